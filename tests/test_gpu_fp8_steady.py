"""FP8 products where every loop of the kernels runs more than once: many tiles
a workgroup, tiles that follow one another with an odd number of K steps and a
short last one, weight scales loaded again; and their precision.

Codes are drawn directly. With codes 0, +-1 and +-2 the 128 products of a block
are whole numbers that add up to 512 at most, which the instruction sums exactly;
what is left is fp32: one rounding of the scales' product, one FMA a block and
three sums of waves, (K / 128 + 6) 2^-24 of the blocks' magnitudes."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import fp8_ckpt_balance_oracle as fo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


VALUES = torch.from_numpy(np.concatenate([np.append(fo.E4M3, np.nan)] * 2))
VALUES[128:] *= -1


class Operands:
    """Codes, scales and segments on the GPU, and the product in 64 bits."""

    def __init__(self, counts, K, N, cap=None, whole=True, seed=0):
        self.n, self.rows = len(counts), int(sum(counts))
        self.cap, self.K, self.N = self.rows if cap is None else cap, K, N
        g = torch.Generator(device="cuda").manual_seed(seed)
        nb, kb = -(-N // 128), -(-K // 128)

        def codes(*shape):
            if whole:  # 0, 1, 2, -1, -2
                pick = torch.tensor([0x00, 0x38, 0x40, 0xB8, 0xC0], dtype=torch.uint8,
                                    device="cuda")
                return pick[torch.randint(0, 5, shape, generator=g, device="cuda")]
            v = torch.randn(*shape, generator=g, device="cuda") * 100
            return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

        def scales(*shape):
            return torch.exp(torch.randn(*shape, generator=g, device="cuda")) * 0.01

        self.xq, self.xs = codes(self.cap, K), scales(kb, self.cap)
        self.wq, self.ws = codes(self.n, N, K), scales(self.n, nb, kb)
        # what lies behind the segments is not looked at
        self.xq[self.rows:], self.xs[:, self.rows:] = 0x7F, float("nan")
        off = np.concatenate([[0], np.cumsum(counts)])
        self.off = torch.tensor(off, dtype=torch.int32, device="cuda")
        lut = VALUES.cuda()
        self.y = torch.zeros(self.rows, N, dtype=torch.float64, device="cuda")
        self.blocks = torch.zeros_like(self.y)   # sum over blocks of |block's part|
        self.mag = torch.zeros_like(self.y)      # sum of |products|
        for e in range(self.n):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            x, w = lut[self.xq[a:b].long()], lut[self.wq[e].long()]
            for j in range(kb):
                s = slice(128 * j, min(128 * j + 128, K))
                sx = self.xs[j, a:b].double()[:, None]
                sw = self.ws[e, :, j].double().repeat_interleave(128)[:N]
                part = (x[:, s] @ w[:, s].t().contiguous()) * sx * sw
                self.y[a:b] += part
                self.blocks[a:b] += part.abs()
                if not whole:
                    self.mag[a:b] += (x[:, s].abs() @ w[:, s].abs().t().contiguous()) * sx * sw

    def down(self, half):
        d = moe.make_desc(T=self.cap, D=self.N, E=self.n, top_k=1, I=self.K, y_fp16=half)
        out = torch.full((self.cap, self.N), -7.0, dtype=torch.float16 if half else torch.float32,
                         device="cuda")
        moe.moe_expert_down_fp8(d, self.n, self.K, self.cap, self.xq, self.xs, self.off, self.wq,
                                self.ws, out)
        assert (out[self.rows:] == -7.0).all()
        return out[:self.rows].double()

    def gate_up(self):
        I = self.N // 2
        d = moe.make_desc(T=self.cap, D=self.K, E=self.n, top_k=1, I=I)
        out = torch.full((self.cap, I), -7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_gate_up_fp8(d, self.n, I, self.cap, self.xq, self.xs, self.off, self.wq,
                                   self.ws, out)
        assert (out[self.rows:] == -7.0).all()
        return out[:self.rows].double()

    def check(self, gated):
        err = self.blocks * (-(-self.K // 128) + 6) * U
        if gated:
            I = self.N // 2
            g, u = self.y[:, :I], self.y[:, I:]
            silu = g / (1 + torch.exp(-g))
            ref = silu * u
            # |SiLU'| <= 1.1, SiLU from exp2 and rcp 2^-19, one bf16 rounding
            bound = (1.1 * err[:, :I] * (u.abs() + err[:, I:]) + silu.abs() * err[:, I:]
                     + (2.0 ** -8 + 2.0 ** -19) * ref.abs() + 1e-30)
            assert ((self.gate_up() - ref).abs() <= bound).all()
            return
        assert ((self.down(False) - self.y).abs() <= err).all()
        half = self.down(True)
        fits = self.y.abs() < 65000
        assert ((half - self.y).abs() <= err + 2.0 ** -11 * self.y.abs() + 2.0 ** -25)[fits].all()


def loads(n, mean, seed):
    """n loads around the mean, two of them none."""
    c = np.random.default_rng(seed).integers(1, 2 * mean, n)
    c[[1, n - 1]] = 0
    return [int(v) for v in c]


# Small tiles beyond one a workgroup (their second rule: at most 32 rows an
# expert, K of 2048 and more, two tiles a CU or more).
@pytest.mark.parametrize("K,N", [(2112, 4096), (4032, 2688)])
@pytest.mark.parametrize("gated", [False, True])
def test_small_tiles_one_after_another(gated, K, N):
    Operands(loads(32, 16, K), K, N, seed=1).check(gated)


# 64 steps of a wave's four cover 32768 columns of K.
@pytest.mark.parametrize("gated", [False, True])
def test_small_tiles_of_more_than_64_steps(gated):
    Operands([5, 17], 33088, 128, seed=2).check(gated)


# Large tiles: more than one a CU, 9 (3, 2, 16) steps each, the last one short.
@pytest.mark.parametrize("K", [1088, 320, 256, 2048, 64])
@pytest.mark.parametrize("gated,N", [(False, 1984), (True, 2176)])
def test_large_tiles_one_after_another(gated, N, K):
    Operands(loads(20, 320, K), K, N, 9000, seed=3).check(gated)


def test_large_tiles_of_more_than_64_steps_one_after_another():
    p = Operands(loads(40, 330, 4), 8384, 1024, 16384, seed=4)   # 66 steps, the last one short
    p.check(False)


@pytest.mark.parametrize("counts,K,N,cap", [(loads(32, 16, 5), 2112, 4096, None),
                                            (loads(20, 320, 6), 1088, 1984, 9000)])
def test_mean_error_of_normal_values(counts, K, N, cap):
    """2^-19 of the sum of the products' magnitudes in the mean, as the header
    says, here twice that at most; no result off by more than its 2^-10."""
    p = Operands(counts, K, N, cap, whole=False, seed=7)
    err = (p.down(False) - p.y).abs() / p.mag
    assert float(err.mean()) <= 2.0 ** -18
    assert float(err.max()) <= 2.0 ** -10


@pytest.mark.parametrize("cap", [None, 9000])   # small tiles, large tiles
def test_gate_far_below_zero_gives_zero(cap):
    """SiLU of a gate of -1e24 is 0, whatever the up value, also where their
    product leaves fp32's range."""
    p = Operands([3, 14], 192, 256, cap, seed=8)
    p.xq[:p.rows], p.wq[:, 128:] = 0x38, 0x38    # all ones: gates < 0 < up values
    p.wq[:, :128] = 0xB8
    p.xs[:, :p.rows] = 1e23
    p.ws[:] = 1.0
    out = p.gate_up()
    assert out.shape == (17, 128) and (out == 0).all()
