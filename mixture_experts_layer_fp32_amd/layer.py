"""Device-buffer owners around the C entry points.

``LayerForward`` allocates the outputs and workspace of ``moe_layer_forward``
once and calls it: the whole layer on one GPU (every expert local). With
``packed=True`` it first packs the expert weights (moe_pack_expert_weights)
into the layout the grouped GEMMs feed to the matrix cores, once.

``LayerForwardMXFP8`` is the same layer with the MXFP8 expert FFN
(include/moe_mxfp8.h): the expert weights are packed once at construction;
a call routes (fp32 router), permutes the bf16 rows, quantizes them, runs the
MXFP8 grouped FFN and combines in fp32 into the bf16 residual.

``LayerForwardFP8`` is the layer with the FP8 expert FFN with block scales
(include/moe_fp8.h): its expert weights, routed and shared, are given as codes
and scales, as fine-grained MoE weights are distributed, or in bf16 and packed
once; a call routes, permutes, quantizes the rows, runs the FP8 FFN and combines.

``LayerTrain`` runs the layer forward through the step entry points, keeping
what the backward needs (routing, offsets, positions, x_perm, y_perm and, with
``save_gu`` (bf16 layers), the fp32 gate and up pre-activations of the routed
and shared experts from ``moe_expert_ffn_train``), and its backward through
``moe_layer_backward`` (include/moe_backward.h): the input gradient and the
router, expert and shared-expert weight gradients. Without ``save_gu`` the
backward recomputes G | U: the same gradients, bit for bit, for
T top_k 2I 4 bytes less memory held between the two passes. With ``norm=True``
it is the pre-norm block out = x + layer(layer_norm(x)): the forward
normalises first (``moe_layer_norm``, include/moe_norm.h) and the residual stays
x; the backward runs the layer's pieces, then ``moe_layer_norm_backward``, which
joins the residual's gradient in. With ``ckpt=True`` (bf16 layers) it keeps 8-bit
checkpoints between the passes (include/moe_ckpt.h): G | U (made in the GEMM's
epilogue), the rows that enter the experts, once a token, and the expert
outputs; the bf16 x_perm and the fp32 y_perm are then scratch, restored in the
backward, which layers that run one after another share (``scratch``): what a
layer keeps is then 0.22 to 0.27 of the plain step's bytes. Without a shared
scratch it holds x_perm and y_perm beside the codes, and only G | U shrinks.
With ``balance`` the forward adds the balance loss
(include/moe_balance.h), and the backward its gradient.

``ExpertMuon`` steps the expert matrices of a ``LayerTrain`` from its gradients
(``moe_muon_update``, include/moe_update.h): gate, up and down matrices of every
expert, and of the shared one, each orthogonalised on its own; it owns the fp32
momentum and the workspace.

``EPRankShareForward`` runs the share of one expert-parallel rank out of
``ep_size`` logical ranks on this GPU, as a sequence of C calls (page "Expert
Parallel (EP)", Communication Pattern; page "Worked Example", Steps 1-5):
  1. moe_route on the rank's own tokens;
  2. moe_permute of the own tokens over all experts ("send" order, with the
     split sizes each rank would receive);
  3. moe_permute over every logical rank's tokens, keeping the pairs whose
     expert is local ("receive" buffer; on a real cluster these rows arrive
     through the all-to-all);
  4. moe_expert_ffn for the local experts;
  5. moe_expert_ffn for the shared expert on the own tokens (if any); with
     ``overlap_shared=True`` (opt-in, off by default) on a second stream
     forked at the start of the step and joined before step 6 (torchtitan
     issue 5554: independent shared experts overlap the routed path and join
     before the combination), else on the step's stream after step 4;
  6. moe_unpermute_combine over every source token: each gets the weighted
     sum of its local slots (the part this rank would send back), and the own
     tokens also get the residual and the shared expert's output.
The other ranks' routing is computed once by ``setup`` (their own routers
would produce it). Torch provides only device memory, streams and events.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import _binding as B


def _layer_desc(desc: B.moe_desc, packed: bool, y_fp16: bool) -> B.moe_desc:
    d = B.moe_desc.from_buffer_copy(desc)
    if packed:
        d.weight_layout = B.MOE_WEIGHTS_PACKED
    d.expert_out_dtype = B.MOE_F16 if y_fp16 else B.MOE_F32
    return d


def _on_own_gpu(method):
    """The method with the GPU of the layer's tensors current. (Of the calls
    that these layers make, some run on the current GPU and some on that of
    their tensors: elsewhere they would not wait for one another.)"""
    @functools.wraps(method)
    def run(self, *args, **kwargs):
        dev = self.out.get_device()
        if dev < 0 or dev == B._current_device():
            return method(self, *args, **kwargs)
        with torch.cuda.device(dev):
            return method(self, *args, **kwargs)
    return run


class LayerForward:
    """packed=True: the expert weights (routed and shared) are packed once here
    (moe_pack_expert_weights) and every call reads the packed copies.
    y_fp16: the layer keeps its expert outputs (y_perm, the shared expert's
    output; workspace-internal) in fp16; default on for bf16 layers."""

    def __init__(self, desc: B.moe_desc, w_router, w_gate_up, w_down, logit_bias=None,
                 shared_gate_up=None, shared_down=None, want_logits=False, device="cuda",
                 packed=False, y_fp16=None):
        if y_fp16 is None:
            y_fp16 = desc.act_dtype == B.MOE_BF16
        desc = _layer_desc(desc, packed, y_fp16)
        if packed:
            w_gate_up, w_down = B.pack_expert_weights(desc, w_gate_up, w_down)
            if shared_gate_up is not None:
                shared_gate_up, shared_down = B.pack_expert_weights(desc, shared_gate_up,
                                                                    shared_down)
        self.d = desc
        T, D, E, k = desc.T, desc.D, desc.E, desc.top_k
        dt = torch.bfloat16 if desc.act_dtype == B.MOE_BF16 else torch.float32
        self.w = dict(w_router=w_router, logit_bias=logit_bias, w_gate_up=w_gate_up,
                      w_down=w_down, shared_gate_up=shared_gate_up, shared_down=shared_down)
        self.out = torch.empty(T, D, dtype=dt, device=device)
        self.logits = torch.empty(T, E, dtype=torch.float32, device=device) if want_logits else None
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=device)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=device)
        self.counts = torch.empty(E, dtype=torch.int32, device=device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.split = torch.empty(desc.ep_size, dtype=torch.int32, device=device)
        self.perm_src = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.pos = torch.empty(T, k, dtype=torch.int32, device=device)
        self.ws = B.workspace(B.moe_workspace_size(desc), device)

    def __call__(self, x, stream=None):
        w = self.w
        B.moe_layer_forward(self.d, x, w["w_router"], w["logit_bias"], w["w_gate_up"],
                            w["w_down"], w["shared_gate_up"], w["shared_down"], self.out,
                            self.logits, self.topk_idx, self.topk_w, self.counts, self.offsets,
                            self.split, self.perm_src, self.pos, self.ws, stream)
        return self.out


class LayerTrain:
    def __init__(self, desc: B.moe_desc, w_router, w_gate_up, w_down, logit_bias=None,
                 shared_gate_up=None, shared_down=None, device="cuda", save_gu=None,
                 norm=False, norm_gamma=None, norm_beta=None, norm_eps=1e-5, ckpt=False,
                 scratch=None, balance=None):
        """norm: a layer norm in front of the layer; norm_gamma, norm_beta [D]
        fp32 or None (ones, zeros), their gradients in dnorm_gamma, dnorm_beta.
        ckpt: 8-bit checkpoints (bf16 layers) in place of save_gu.
        scratch: a dict that LayerTrain(ckpt=True) layers of equal sizes share
        for what no layer needs between its passes (None: the layer's own).
        balance: the coefficient of the balance loss, None for none; the forward
        leaves the loss in balance_loss [1] and balance_counts [E] (int32),
        balance_tokens [1] (int32), balance_prob_sum [E], which ranks of one
        batch add up (all-reduce) before the backward."""
        self.d = desc
        T, D, E, k, I, Is = desc.T, desc.D, desc.E, desc.top_k, desc.I, desc.I_shared
        M = T * k
        # bf: the activation dtype (bf16, or fp32 for fp32 layers)
        f32, i32 = torch.float32, torch.int32
        bf = torch.bfloat16 if desc.act_dtype == B.MOE_BF16 else torch.float32
        self.w = dict(w_router=w_router, logit_bias=logit_bias, w_gate_up=w_gate_up,
                      w_down=w_down, shared_gate_up=shared_gate_up, shared_down=shared_down)
        self.out = torch.empty(T, D, dtype=bf, device=device)
        self.topk_idx = torch.empty(T, k, dtype=i32, device=device)
        self.topk_w = torch.empty(T, k, dtype=f32, device=device)
        self.counts = torch.empty(E, dtype=i32, device=device)
        self.offsets = torch.empty(E + 1, dtype=i32, device=device)
        self.split = torch.empty(desc.ep_size, dtype=i32, device=device)
        self.perm_src = torch.empty(max(M, 1), dtype=i32, device=device)
        self.pos = torch.empty(T, k, dtype=i32, device=device)
        if ckpt and desc.act_dtype != B.MOE_BF16:
            raise ValueError("ckpt: bf16 layers only")
        if ckpt and save_gu:
            raise ValueError("ckpt keeps G | U in 8 bits: not with save_gu")
        if scratch is not None and not ckpt:
            raise ValueError("scratch: only with ckpt=True")
        self.ckpt, self.balance = ckpt, balance
        pool = {} if scratch is None else scratch

        def shared(name, *shape, dtype=f32):
            """A tensor of the scratch (made by the first layer that asks)."""
            t = pool.get(name)
            if t is None:
                t = pool[name] = torch.empty(*shape, dtype=dtype, device=device)
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError(f"scratch: {name} is of a layer of other sizes")
            return same_device(name, t)

        def same_device(name, t):
            if t.device != self.out.device:
                raise ValueError(f"scratch: {name} is on {t.device}, the layer on "
                                 f"{self.out.device}")
            return t

        def shared_ws(name, nbytes):
            t = pool.get(name)
            if t is not None:
                same_device(name, t)
            if t is None or t.numel() < nbytes:
                t = pool[name] = B.workspace(nbytes, device)
            return t

        self.x_perm = shared("x_perm", M, D, dtype=bf)
        self.y_perm = shared("y_perm", M, D)
        self.shared_out = shared("shared_out", T, D) if Is > 0 else None
        if ckpt:
            # What the layer keeps between its passes, in 8 bits.
            i8 = torch.int8
            self.gu_q = torch.empty(M, 2 * I, dtype=i8, device=device)
            self.gu_s = torch.empty(M, 2 * I // 32, dtype=bf, device=device)
            self.x_q = torch.empty(T, D, dtype=i8, device=device)
            self.x_s = torch.empty(T, D // 32, dtype=bf, device=device)
            self.y_q = torch.empty(M, D, dtype=i8, device=device)
            self.y_s = torch.empty(M, D // 32, dtype=bf, device=device)
            if Is > 0:
                self.gu_sh_q = torch.empty(T, 2 * Is, dtype=i8, device=device)
                self.gu_sh_s = torch.empty(T, 2 * Is // 32, dtype=bf, device=device)
            self.x_back = shared("x_back", T, D, dtype=bf)
        # fp32 G | U of the forward (bf16 layers only)
        if save_gu is None:
            save_gu = desc.act_dtype == B.MOE_BF16 and not ckpt
        if save_gu and desc.act_dtype != B.MOE_BF16:
            raise ValueError("save_gu: bf16 layers only")
        self.gu = torch.empty(M, 2 * I, dtype=f32, device=device) if save_gu else None
        self.gu_sh = (torch.empty(T, 2 * Is, dtype=f32, device=device)
                      if save_gu and Is > 0 else None)
        self.ws_route = B.workspace(B.moe_route_workspace_size(desc), device)
        self.ws_perm = B.workspace(B.moe_permute_workspace_size(desc, 0, E), device)
        self.ws_ffn = shared_ws("ws_ffn", B.moe_ffn_workspace_size(desc, I, M))
        self.ws_sh = shared_ws("ws_sh", B.moe_ffn_workspace_size(desc, Is, T)) if Is > 0 else None
        # gradients
        self.dx = torch.empty(T, D, dtype=bf, device=device)
        self.dw_router = torch.empty(E, D, dtype=f32, device=device)
        self.dw_gate_up = torch.empty(E, D, 2 * I, dtype=f32, device=device)
        self.dw_down = torch.empty(E, I, D, dtype=f32, device=device)
        self.dw_shared_gate_up = torch.empty(D, 2 * Is, dtype=f32, device=device) if Is else None
        self.dw_shared_down = torch.empty(Is, D, dtype=f32, device=device) if Is else None
        self.x = None
        self.stepped = False  # a forward has been done
        self.norm = norm
        if not norm and (norm_gamma is not None or norm_beta is not None):
            raise ValueError("norm_gamma, norm_beta: only with norm=True")
        if balance is not None:
            self.logits = torch.empty(T, E, dtype=f32, device=device)
            self.balance_counts = torch.empty(E, dtype=i32, device=device)
            self.balance_tokens = torch.empty(1, dtype=i32, device=device)
            self.balance_prob_sum = torch.empty(E, dtype=f32, device=device)
            self.balance_loss = torch.empty(1, dtype=f32, device=device)
            self.ws_balance = B.workspace(B.moe_balance_loss_workspace_size(T, E), device)
            self.mask = None
        # Without any of the three, moe_layer_backward does it all.
        self.pieces = norm or ckpt or balance is not None
        if not self.pieces:
            self.ws_bwd = B.workspace(B.moe_backward_workspace_size(desc), device)
            return
        ffn = B.moe_ffn_backward_workspace_size(desc, I, M)
        if Is:
            ffn = max(ffn, B.moe_ffn_backward_workspace_size(desc, Is, T))
        need = max(ffn, B.moe_router_backward_workspace_size(desc, M))
        # what the layer's backward leaves between its pieces
        self.dy_perm = shared("dy_perm", M, D, dtype=bf)
        self.dx_perm = shared("dx_perm", M, D)
        self.dx_shared = shared("dx_shared", T, D) if Is or balance is not None else None
        self.dlogit = shared("dlogit", T, k)
        self.dl_perm = shared("dl_perm", max(M, 1))
        if balance is not None:
            self.dlogits = shared("dlogits", T, E)
            need = max(need, B.moe_router_backward_dense_workspace_size(T, E, D))
        if norm:
            self.norm_gamma, self.norm_beta, self.norm_eps = norm_gamma, norm_beta, norm_eps
            self.h = shared("h", T, D, dtype=bf)
            self.mean = torch.empty(T, dtype=f32, device=device)
            self.rstd = torch.empty(T, dtype=f32, device=device)
            self.dh = shared("dh", T, D, dtype=bf)
            self.dnorm_gamma = torch.empty(D, dtype=f32, device=device)
            self.dnorm_beta = torch.empty(D, dtype=f32, device=device)
            need = max(need, B.moe_layer_norm_backward_workspace_size(T, D))
        self.ws_bwd = shared_ws("ws_bwd", need)

    @_on_own_gpu
    def forward(self, x, stream=None, mask=None):
        """mask [T] uint8 or bool: tokens that count in the balance loss (None:
        all). x (but for ckpt=True without a norm) and mask are read again by
        the backward: they stay as they are until then."""
        d, w = self.d, self.w
        E, I, M = d.E, d.I, d.T * d.top_k
        if mask is not None and self.balance is None:
            raise ValueError("mask: only with balance")
        # Refused before anything that the backward of the step before needs is
        # replaced.
        dev = B._device_of(self.out, "out")
        B._device_of(x, "x")
        B._ptr_on(dev, x, "x", self.out.dtype, (d.T, d.D))
        B._mask(dev, mask, d.T)
        res = x
        # The backward's input: kept, or restored from its checkpoint.
        self.x = None if self.ckpt and not self.norm else x
        if self.norm:
            B.moe_layer_norm(x, self.norm_gamma, self.norm_beta, self.norm_eps, self.h, self.mean,
                             self.rstd, stream)
            x = self.h
        logits = self.logits if self.balance is not None else None
        B.moe_route(d, x, w["w_router"], w["logit_bias"], logits, None, self.topk_idx, self.topk_w,
                    ws=self.ws_route, stream=stream)
        if self.balance is not None:
            self.mask = mask
            B.moe_balance_loss(logits, self.topk_idx, self.balance, self.balance_counts,
                               self.balance_tokens, self.balance_prob_sum, self.balance_loss,
                               self.ws_balance, mask=mask, stream=stream)
        B.moe_permute(d, x, self.topk_idx, 0, E, M, self.counts, self.offsets, self.split,
                      self.perm_src, self.pos, self.x_perm, self.ws_perm, stream)
        if self.ckpt:
            B.moe_ckpt_save_rows(x, self.x_q, self.x_s, stream)
            B.moe_expert_ffn_train_ckpt(d, E, I, M, self.x_perm, self.offsets, w["w_gate_up"],
                                        w["w_down"], self.y_perm, self.gu_q, self.gu_s,
                                        self.ws_ffn, stream)
            B.moe_ckpt_save_rows(self.y_perm, self.y_q, self.y_s, stream)
        elif self.gu is not None:
            B.moe_expert_ffn_train(d, E, I, M, self.x_perm, self.offsets, w["w_gate_up"],
                                   w["w_down"], self.y_perm, self.gu, self.ws_ffn, stream)
        else:
            B.moe_expert_ffn(d, E, I, M, self.x_perm, self.offsets, w["w_gate_up"], w["w_down"],
                             self.y_perm, self.ws_ffn, stream)
        if self.shared_out is not None:
            if self.ckpt:
                B.moe_expert_ffn_train_ckpt(d, 1, d.I_shared, d.T, x, None, w["shared_gate_up"],
                                            w["shared_down"], self.shared_out, self.gu_sh_q,
                                            self.gu_sh_s, self.ws_sh, stream)
            elif self.gu_sh is not None:
                B.moe_expert_ffn_train(d, 1, d.I_shared, d.T, x, None, w["shared_gate_up"],
                                       w["shared_down"], self.shared_out, self.gu_sh, self.ws_sh,
                                       stream)
            else:
                B.moe_expert_ffn(d, 1, d.I_shared, d.T, x, None, w["shared_gate_up"],
                                 w["shared_down"], self.shared_out, self.ws_sh, stream)
        B.moe_unpermute_combine(d, self.y_perm, self.pos, self.topk_w, res, self.shared_out, 0,
                                d.T, self.out, stream)
        self.stepped = True
        return self.out

    def _backward_pieces(self, dout, dloss, stream):
        d, w, ws = self.d, self.w, self.ws_bwd
        E, I, M = d.E, d.I, d.T * d.top_k
        if self.ckpt:
            B.moe_ckpt_restore_rows(self.x_q, self.x_s, self.x_back, stream=stream)
            B.moe_ckpt_restore_rows(self.x_q, self.x_s, self.x_perm, self.perm_src[:M], stream)
            B.moe_ckpt_restore_rows(self.y_q, self.y_s, self.y_perm, stream=stream)
            x = self.x_back
        else:
            x = self.h if self.norm else self.x
        B.moe_combine_backward(d, dout, self.y_perm, self.pos, self.topk_w, self.dy_perm, None,
                               self.dlogit, self.dl_perm, stream)
        gate_up, down = w["w_gate_up"], w["w_down"]
        if self.ckpt:
            B.moe_expert_ffn_backward_ckpt(d, E, I, M, self.x_perm, self.offsets, gate_up, down,
                                           self.dy_perm, self.gu_q, self.gu_s, self.dx_perm,
                                           self.dw_gate_up, self.dw_down, ws, stream)
        else:
            B.moe_expert_ffn_backward(d, E, I, M, self.x_perm, self.offsets, gate_up, down,
                                      self.dy_perm, self.dx_perm, self.dw_gate_up, self.dw_down,
                                      ws, stream, gu_saved=self.gu)
        if self.shared_out is not None:
            gate_up, down, dgate_up, ddown = (
                t[None] for t in (w["shared_gate_up"], w["shared_down"], self.dw_shared_gate_up,
                                  self.dw_shared_down))
            if self.ckpt:
                B.moe_expert_ffn_backward_ckpt(d, 1, d.I_shared, d.T, x, None, gate_up, down, dout,
                                               self.gu_sh_q, self.gu_sh_s, self.dx_shared,
                                               dgate_up, ddown, ws, stream)
            else:
                B.moe_expert_ffn_backward(d, 1, d.I_shared, d.T, x, None, gate_up, down, dout,
                                          self.dx_shared, dgate_up, ddown, ws, stream,
                                          gu_saved=self.gu_sh)
        dlogit = self.dlogit
        if self.balance is not None:
            # The router's whole gradient, dense: dx goes the way of the shared
            # expert's.
            B.moe_balance_loss_backward(self.logits, self.topk_idx, self.balance,
                                        self.balance_counts, self.balance_tokens, dloss,
                                        self.dlogits, mask=self.mask, dlogit=dlogit, stream=stream)
            B.moe_router_backward_dense(self.dlogits, x, w["w_router"], self.dx_shared,
                                        self.dw_router, ws,
                                        accumulate=self.shared_out is not None, stream=stream)
            dlogit = None
        else:
            B.moe_router_backward(d, M, self.x_perm, self.offsets, self.dl_perm, self.dw_router,
                                  ws, stream)
        # With a norm the residual's gradient joins behind it, not here.
        B.moe_input_backward(d, self.dx_perm, self.pos, self.topk_idx, dlogit, w["w_router"],
                             self.dx_shared, None if self.norm else dout,
                             self.dh if self.norm else self.dx, stream)
        if self.norm:
            B.moe_layer_norm_backward(self.x, self.dh, self.norm_gamma, self.mean, self.rstd, dout,
                                      self.dx, self.dnorm_gamma, self.dnorm_beta, ws, stream)
        return self.dx

    @_on_own_gpu
    def backward(self, dout, stream=None, dloss=None):
        """dloss [1] fp32: the gradient of balance_loss (None: 1)."""
        if dloss is not None and self.balance is None:
            raise ValueError("dloss: only with balance")
        if not self.stepped:
            # (The positions of the routing are not there yet: they say where
            # gradients are written.)
            raise RuntimeError("backward: no forward before it")
        if self.pieces:
            return self._backward_pieces(dout, dloss, stream)
        w = self.w
        B.moe_layer_backward(self.d, self.x, w["w_router"], w["w_gate_up"], w["w_down"],
                             w["shared_gate_up"], w["shared_down"], self.topk_idx, self.topk_w,
                             self.offsets, self.pos, self.x_perm, self.y_perm, dout, self.dx,
                             self.dw_router, self.dw_gate_up, self.dw_down,
                             self.dw_shared_gate_up, self.dw_shared_down, self.ws_bwd, stream,
                             gu_saved=self.gu, gu_shared_saved=self.gu_sh)
        return self.dx


class ExpertMuon:
    """Muon for the expert matrices of a LayerTrain (and its shared expert's):
    step(lr) updates layer.w in place from layer.dw_*. Each [D, I] gate, [D, I]
    up and [I, D] down matrix is orthogonalised on its own and scaled by
    0.2 sqrt(longer side). The router weight and the norm's parameters are
    the caller's (they are not updated here)."""

    def __init__(self, layer: LayerTrain, mu=0.95, nesterov=True, weight_decay=0.0, steps=5,
                 eps=1e-7):
        self.kw = dict(mu=mu, nesterov=nesterov, weight_decay=weight_decay, steps=steps, eps=eps)
        self.momentum = {}
        self.batches = []
        need = 256
        for w_name, g_name, halves in (("w_gate_up", "dw_gate_up", 2), ("w_down", "dw_down", 1),
                                       ("shared_gate_up", "dw_shared_gate_up", 2),
                                       ("shared_down", "dw_shared_down", 1)):
            w, g = layer.w[w_name], getattr(layer, g_name)
            if g is None:
                continue
            m = self.momentum[w_name] = torch.zeros_like(g)
            for wv, gv, mv in zip(*(t.chunk(halves, dim=-1) for t in (w, g, m))):
                n = wv.shape[0] if wv.dim() == 3 else 1
                rows, cols = wv.shape[-2:]
                need = max(need, B.moe_orthogonalize_workspace_size(n, rows, cols, steps))
                self.batches.append((gv, mv, wv, 0.2 * max(rows, cols) ** 0.5))
        self.ws = B.workspace(need, layer.dx.device)

    def step(self, lr, stream=None):
        for g, m, w, scale in self.batches:
            B.moe_muon_update(g, m, w, self.ws, lr=lr, scale=scale, stream=stream, **self.kw)


class EPRankShareForward:
    def __init__(self, T: int, D: int, E: int, top_k: int, I: int, ep_size: int, ep_rank: int,
                 x_src, w_router, w_gate_up_local, w_down_local, logit_bias=None,
                 shared_gate_up=None, shared_down=None, I_shared: int = 0, dtype="bf16",
                 norm_topk=True, device="cuda", overlap_shared: bool = False,
                 packed: bool = False, y_fp16=None):
        R, r = ep_size, ep_rank
        if E % R:
            raise ValueError("E must be divisible by ep_size")
        self.T, self.D, self.E, self.k, self.I, self.R, self.r = T, D, E, top_k, I, R, r
        self.E_loc = E // R
        self.e_begin, self.e_end = r * self.E_loc, (r + 1) * self.E_loc
        self.Is = I_shared
        if y_fp16 is None:
            y_fp16 = dtype == "bf16"
        kw = dict(D=D, E=E, top_k=top_k, I=I, ep_size=R, ep_rank=r, dtype=dtype,
                  norm_topk=norm_topk, I_shared=I_shared, packed=packed, y_fp16=y_fp16)
        ydt = torch.float16 if y_fp16 else torch.float32
        self.d_own = B.make_desc(T=T, **kw)
        self.d_src = B.make_desc(T=T * R, **kw)
        if packed:
            w_gate_up_local, w_down_local = B.pack_expert_weights(self.d_own, w_gate_up_local,
                                                                  w_down_local)
            if shared_gate_up is not None:
                shared_gate_up, shared_down = B.pack_expert_weights(self.d_own, shared_gate_up,
                                                                    shared_down)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        dev = device
        self.x_src = x_src
        self.x_own = x_src[r * T:(r + 1) * T]
        self.w = dict(w_router=w_router, logit_bias=logit_bias, w_gate_up=w_gate_up_local,
                      w_down=w_down_local, shared_gate_up=shared_gate_up, shared_down=shared_down)
        Ts = T * R
        k = top_k
        # routing of every source token; rows [r*T, (r+1)*T) are this rank's own
        self.idx_src = torch.empty(Ts, k, dtype=torch.int32, device=dev)
        self.w_src = torch.empty(Ts, k, dtype=torch.float32, device=dev)
        self.idx_own = self.idx_src[r * T:(r + 1) * T]
        self.w_own = self.w_src[r * T:(r + 1) * T]
        # send-side permute of the own tokens over all experts
        self.send_counts = torch.empty(E, dtype=torch.int32, device=dev)
        self.send_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.send_split = torch.empty(R, dtype=torch.int32, device=dev)
        self.send_cap = T * k
        self.send_perm_src = torch.empty(max(self.send_cap, 1), dtype=torch.int32, device=dev)
        self.send_pos = torch.empty(T, k, dtype=torch.int32, device=dev)
        self.x_send = torch.empty(self.send_cap, D, dtype=dt, device=dev)
        self.route_ws = B.workspace(B.moe_route_workspace_size(self.d_own), dev)
        self.send_ws = B.workspace(B.moe_permute_workspace_size(self.d_own, 0, E), dev)
        # receive side: every source pair whose expert is local
        n = self.E_loc
        self.recv_cap = Ts * min(k, n)
        self.recv_counts = torch.empty(n, dtype=torch.int32, device=dev)
        self.recv_offsets = torch.empty(n + 1, dtype=torch.int32, device=dev)
        self.recv_split = torch.empty(R, dtype=torch.int32, device=dev)
        self.recv_perm_src = torch.empty(max(self.recv_cap, 1), dtype=torch.int32, device=dev)
        self.recv_pos = torch.empty(Ts, k, dtype=torch.int32, device=dev)
        self.x_recv = torch.empty(self.recv_cap, D, dtype=dt, device=dev)
        self.recv_ws = B.workspace(
            B.moe_permute_workspace_size(self.d_src, self.e_begin, self.e_end), dev)
        self.y_recv = torch.empty(self.recv_cap, D, dtype=ydt, device=dev)
        self.ffn_ws = B.workspace(B.moe_ffn_workspace_size(self.d_src, I, self.recv_cap), dev)
        if I_shared > 0:
            self.shared_out = torch.empty(T, D, dtype=ydt, device=dev)
            self.shared_ws = B.workspace(B.moe_ffn_workspace_size(self.d_own, I_shared, T), dev)
        else:
            self.shared_out = None
        # The shared expert depends only on the own tokens: it runs on a second
        # stream (default priority), forked at the start of the step and joined
        # before the combine (the overlap of the torchtitan shared-expert
        # issue, without the lower stream priority).
        self.aux = None
        if I_shared > 0 and overlap_shared:
            self.aux = torch.cuda.Stream(device=dev)
            self.ev_fork = torch.cuda.Event()
            self.ev_join = torch.cuda.Event()
        self.out_src = torch.empty(Ts, D, dtype=dt, device=dev)

    def setup(self, stream=None):
        """Route every other logical rank's tokens (their own routers' output)."""
        w = self.w
        for q in range(self.R):
            if q == self.r:
                continue
            sl = slice(q * self.T, (q + 1) * self.T)
            B.moe_route(self.d_own, self.x_src[sl], w["w_router"], w["logit_bias"], None, None,
                        self.idx_src[sl], self.w_src[sl], ws=self.route_ws, stream=stream)

    def __call__(self, logits: Optional[torch.Tensor] = None, stream=None):
        w = self.w
        if self.aux is not None:
            main = stream if isinstance(stream, torch.cuda.Stream) else (
                torch.cuda.current_stream(self.x_own.device) if stream is None
                else torch.cuda.ExternalStream(int(stream), device=self.x_own.device))
            self.ev_fork.record(main)
            self.aux.wait_event(self.ev_fork)
            B.moe_expert_ffn(self.d_own, 1, self.Is, self.T, self.x_own, None,
                             w["shared_gate_up"], w["shared_down"], self.shared_out,
                             self.shared_ws, self.aux)
            self.ev_join.record(self.aux)
        B.moe_route(self.d_own, self.x_own, w["w_router"], w["logit_bias"], logits, None,
                    self.idx_own, self.w_own, ws=self.route_ws, stream=stream)
        B.moe_permute(self.d_own, self.x_own, self.idx_own, 0, self.E, self.send_cap,
                      self.send_counts, self.send_offsets, self.send_split, self.send_perm_src,
                      self.send_pos, self.x_send, self.send_ws, stream)
        B.moe_permute(self.d_src, self.x_src, self.idx_src, self.e_begin, self.e_end,
                      self.recv_cap, self.recv_counts, self.recv_offsets, self.recv_split,
                      self.recv_perm_src, self.recv_pos, self.x_recv, self.recv_ws, stream)
        B.moe_expert_ffn(self.d_src, self.E_loc, self.I, self.recv_cap, self.x_recv,
                         self.recv_offsets, w["w_gate_up"], w["w_down"], self.y_recv, self.ffn_ws,
                         stream)
        if self.aux is not None:
            main.wait_event(self.ev_join)
        elif self.shared_out is not None:
            B.moe_expert_ffn(self.d_own, 1, self.Is, self.T, self.x_own, None,
                             w["shared_gate_up"], w["shared_down"], self.shared_out,
                             self.shared_ws, stream)
        B.moe_unpermute_combine(self.d_src, self.y_recv, self.recv_pos, self.w_src, self.x_own,
                                self.shared_out, self.r * self.T, self.T, self.out_src, stream)
        return self.out_src


class LayerForwardMXFP8:
    def __init__(self, desc: B.moe_desc, w_router, w_gate_up, w_down, logit_bias=None,
                 want_logits=False, device="cuda"):
        if desc.act_dtype != B.MOE_BF16 or desc.I_shared != 0:
            raise ValueError("the MXFP8 layer takes a bf16 layer without a shared expert")
        self.d = desc
        T, D, E, k, I = desc.T, desc.D, desc.E, desc.top_k, desc.I
        M = T * k
        u8 = torch.uint8
        self.w_router, self.logit_bias = w_router, logit_bias
        # weights packed once (quantized per output column along K, K contiguous)
        self.guq = torch.empty(E, 2 * I, D, dtype=u8, device=device)
        self.gus = torch.empty(E, 2 * I, D // 32, dtype=u8, device=device)
        self.dq = torch.empty(E, D, I, dtype=u8, device=device)
        self.ds = torch.empty(E, D, I // 32, dtype=u8, device=device)
        B.moe_mxfp8_pack_weights(w_gate_up, self.guq, self.gus)
        B.moe_mxfp8_pack_weights(w_down, self.dq, self.ds)
        self.out = torch.empty(T, D, dtype=torch.bfloat16, device=device)
        self.logits = torch.empty(T, E, dtype=torch.float32, device=device) if want_logits else None
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=device)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=device)
        self.counts = torch.empty(E, dtype=torch.int32, device=device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.split = torch.empty(desc.ep_size, dtype=torch.int32, device=device)
        self.perm_src = torch.empty(max(M, 1), dtype=torch.int32, device=device)
        self.pos = torch.empty(T, k, dtype=torch.int32, device=device)
        self.x_perm = torch.empty(M, D, dtype=torch.bfloat16, device=device)
        self.xq = torch.empty(M, D, dtype=u8, device=device)
        self.xs = torch.empty(M, D // 32, dtype=u8, device=device)
        self.y_perm = torch.empty(M, D, dtype=torch.float32, device=device)
        self.ws_route = B.workspace(B.moe_route_workspace_size(desc), device)
        self.ws_perm = B.workspace(B.moe_permute_workspace_size(desc, 0, E), device)
        self.ws_ffn = B.workspace(B.moe_ffn_mxfp8_workspace_size(desc, I, M), device)

    def __call__(self, x, stream=None):
        d = self.d
        E, I, M = d.E, d.I, d.T * d.top_k
        B.moe_route(d, x, self.w_router, self.logit_bias, self.logits, None, self.topk_idx,
                    self.topk_w, ws=self.ws_route, stream=stream)
        B.moe_permute(d, x, self.topk_idx, 0, E, M, self.counts, self.offsets, self.split,
                      self.perm_src, self.pos, self.x_perm, self.ws_perm, stream)
        B.moe_mxfp8_quantize_rows(self.x_perm, self.xq, self.xs, stream)
        B.moe_expert_ffn_mxfp8(d, E, I, M, self.xq, self.xs, self.offsets, self.guq, self.gus,
                               self.dq, self.ds, self.y_perm, self.ws_ffn, stream)
        B.moe_unpermute_combine(d, self.y_perm, self.pos, self.topk_w, x, None, 0, d.T, self.out,
                                stream)
        return self.out


class LayerForwardFP8:
    """w_gate_up, w_down (and the shared expert's) are bf16 or fp32 tensors,
    stacked as for LayerForward and packed here, or pairs (codes, scales) in the
    layout of include/moe_fp8.h: codes [E, 2I, D] and [E, D, I], scales one for
    each 128 x 128 block. y_fp16: expert outputs in fp16 (default) or fp32."""

    def __init__(self, desc: B.moe_desc, w_router, w_gate_up, w_down, logit_bias=None,
                 shared_gate_up=None, shared_down=None, want_logits=False, device="cuda",
                 y_fp16=True):
        if desc.act_dtype != B.MOE_BF16:
            raise ValueError("the FP8 layer takes a bf16 layer")
        self.d = desc = _layer_desc(desc, False, y_fp16)
        T, D, E, k, I, Is = desc.T, desc.D, desc.E, desc.top_k, desc.I, desc.I_shared
        M = T * k

        def pack(w):
            if isinstance(w, (tuple, list)):
                return tuple(t if t.dim() == 3 else t[None] for t in w)
            return B.pack_expert_weights_fp8(w if w.dim() == 3 else w[None])

        self.w_router, self.logit_bias = w_router, logit_bias
        self.gate_up, self.down = pack(w_gate_up), pack(w_down)
        u8, i32, f32, bf = torch.uint8, torch.int32, torch.float32, torch.bfloat16
        ydt = torch.float16 if y_fp16 else f32
        self.out = torch.empty(T, D, dtype=bf, device=device)
        self.logits = torch.empty(T, E, dtype=f32, device=device) if want_logits else None
        self.topk_idx = torch.empty(T, k, dtype=i32, device=device)
        self.topk_w = torch.empty(T, k, dtype=f32, device=device)
        self.counts = torch.empty(E, dtype=i32, device=device)
        self.offsets = torch.empty(E + 1, dtype=i32, device=device)
        self.split = torch.empty(desc.ep_size, dtype=i32, device=device)
        self.perm_src = torch.empty(max(M, 1), dtype=i32, device=device)
        self.pos = torch.empty(T, k, dtype=i32, device=device)
        self.x_perm = torch.empty(M, D, dtype=bf, device=device)
        self.xq = torch.empty(M, D, dtype=u8, device=device)
        self.xs = torch.empty((D + 127) // 128, M, dtype=f32, device=device)
        self.y_perm = torch.empty(M, D, dtype=ydt, device=device)
        self.ws_route = B.workspace(B.moe_route_workspace_size(desc), device)
        self.ws_perm = B.workspace(B.moe_permute_workspace_size(desc, 0, E), device)
        need = B.moe_ffn_fp8_workspace_size(desc, I, M)
        self.shared_out = None
        if Is > 0:
            self.sh_gate_up, self.sh_down = pack(shared_gate_up), pack(shared_down)
            self.xq_sh = torch.empty(T, D, dtype=u8, device=device)
            self.xs_sh = torch.empty((D + 127) // 128, T, dtype=f32, device=device)
            self.shared_out = torch.empty(T, D, dtype=ydt, device=device)
            need = max(need, B.moe_ffn_fp8_workspace_size(desc, Is, T))
        self.ws_ffn = B.workspace(need, device)

    @_on_own_gpu
    def __call__(self, x, stream=None):
        d = self.d
        E, I, M = d.E, d.I, d.T * d.top_k
        B.moe_route(d, x, self.w_router, self.logit_bias, self.logits, None, self.topk_idx,
                    self.topk_w, ws=self.ws_route, stream=stream)
        B.moe_permute(d, x, self.topk_idx, 0, E, M, self.counts, self.offsets, self.split,
                      self.perm_src, self.pos, self.x_perm, self.ws_perm, stream)
        B.moe_fp8_quantize_rows(self.x_perm, self.xq, self.xs, stream)
        B.moe_expert_ffn_fp8(d, E, I, M, self.xq, self.xs, self.offsets, *self.gate_up, *self.down,
                             self.y_perm, self.ws_ffn, stream)
        if self.shared_out is not None:
            B.moe_fp8_quantize_rows(x, self.xq_sh, self.xs_sh, stream)
            B.moe_expert_ffn_fp8(d, 1, d.I_shared, d.T, self.xq_sh, self.xs_sh, None,
                                 *self.sh_gate_up, *self.sh_down, self.shared_out, self.ws_ffn,
                                 stream)
        B.moe_unpermute_combine(d, self.y_perm, self.pos, self.topk_w, x, self.shared_out, 0, d.T,
                                self.out, stream)
        return self.out
