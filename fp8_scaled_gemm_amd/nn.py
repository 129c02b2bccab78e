"""PyTorch integration of the FP8 scaled linear layer and the GradScaler step,
over the C-ABI library: every FP8 cast, GEMM, unscale, check and scale update
runs in libfp8sg's kernels; this module only allocates buffers, wires
autograd and walks module trees.

  - Float8Linear / _Fp8LinearFn ["FP8训练：量化、自动微分、Torchao", §6: one
    autograd node per linear; the forward takes and returns plain bf16, FP8
    never leaves it; what is saved for the backward pass is the FP8 operands
    and their inverse scales, not the bf16 inputs; §1 for row-wise scaling].
  - convert_to_float8_training [same page, §8: post-order walk over the module
    tree, nn.Linear children replaced in place when module_filter_fn(module,
    fully qualified name) allows, the new module reusing the original weight
    tensor].
  - GradScaler ["第20章 量化与混合精度训练", §20.2.2 and §20.5.33;
    "AMP：Automatic Mixed Precision 技术笔记", §4 and §6]: scale the loss,
    unscale fp16 gradients in place with the non-finite check, skip the
    optimizer step on inf/NaN, update the scale on the device.

Dynamic scaling runs through two registered operators, fp8sg::scaled_linear_fwd
and fp8sg::scaled_linear_bwd (torch.library custom ops with shape-only fake
implementations and an autograd formula), so torch.compile keeps each FP8 linear
as one opaque call in its graph (the same page, §7: the compiler sees the FP8
linear as an opaque call and optimises around it) instead of tracing into the
library calls.  Delayed and row-wise scaling use an autograd.Function in eager
mode; a module keeps its backward scratch (the quantized gradient) across steps.

An fp16 model under loss scaling [PT-CH20 §20.2.2] uses fp16 layers
(Float8Linear with an fp16 weight): fp16 inputs are cast by the fp16-input
kernels, outputs and gradients are fp16, and with a GradScaler attached the
weight gradient leaves the wgrad GEMM unscaled and checked (the scaler's
unscale_ then skips it); the input gradient keeps the loss scale for the layers
below.

  - MXFP4Linear, PackedMXFP4Linear, convert_to_mxfp4_training / _serving: the
    same layer with 4-bit microscaled operands, for training and for serving.
  - SwiGLU, LayerNorm: the gated activation and the norm around those linears,
    which may keep what their backward pass needs in 8 bits.
  - Float8EpilogueLinear, MXFP4EpilogueLinear, PackedMXFP4EpilogueLinear, Dropout: the
    linears with bias, activation, dropout and residual in the product's epilogue,
    and dropout on its own.

Limits of Float8Linear: inputs and weights are bf16 or fp16; no bias (the method's
linear has none; the default filter leaves biased layers alone, biased=True makes
them Float8EpilogueLinear); leading dimensions of the input are flattened into M;
M, N, K must be multiples of 16.
"""
import math
from typing import Callable, Optional

import torch
from torch import nn

from . import (E4M3FN, E5M2, LinearBwdWs, LinearBwdWsRW, LinearSaved, LinearSavedRW, OUT_BF16,
               OUT_F16, SCALE_REC_BYTES, ScaleRec,
               amp_norm_workspace_len, amp_unscale_check, amp_unscale_check_norm,
               amp_update_scale, fp8_amax, fp8_amax_f16, fp8_gemm, fp8_gemm_kmajor,
               fp8_gemm_kmajor_unscale, fp8_linear_copies,
               fp8_quantize_f16, fp8_scaled_linear_bwd, fp8_scaled_linear_bwd_delayed,
               fp8_scaled_linear_bwd_rowwise, fp8_scaled_linear_fwd, fp8_scaled_linear_fwd_delayed,
               fp8_scaled_linear_fwd_rowwise)
from . import (MX_FIT, MX_FLOOR, Act8, Mxfp4, Mxfp4LinearSaved, Mxfp4LinearWs, layer_norm_bwd,
               layer_norm_fwd, layer_norm_workspace_len, mxfp4_linear_apply, mxfp4_linear_bwd,
               mxfp4_linear_fwd, mxfp4_quantize, swiglu_bwd, swiglu_fwd)
from . import (ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, dropout_bwd, dropout_fwd,
               epilogue_workspace_len, fp8_scaled_linear_bwd_epilogue, fp8_scaled_linear_fwd_epilogue,
               mxfp4_linear_apply_epilogue, mxfp4_linear_bwd_epilogue, mxfp4_linear_fwd_epilogue)

SCALINGS = ("dynamic", "delayed", "rowwise")


def _seed_history(hist: torch.Tensor, x: torch.Tensor):
    """Delayed scaling needs a history before its first step: its first entry
    becomes max |x| of the first tensor seen (one amax pass)."""
    rec = ScaleRec(device=x.device)
    fp8_amax(x, rec)
    hist.zero_()
    hist[:1].copy_(rec.buf[0:4].view(torch.float32))  # the record's amax field


# ---------------------------------------------------------------- custom ops
# The dynamic-scaling linear as two operators.  The forward returns y and the
# state the backward needs (codes, transposed codes, the two scale records),
# all fresh outputs; nothing is mutated.  Which transposed copies are made
# follows fp8_linear_copies (the fastest backward on this device); a copy not
# made travels as an empty tensor.

def _present(t):
    return t if t is not None and t.numel() > 0 else None


@torch.library.custom_op("fp8sg::scaled_linear_fwd", mutates_args=())
def _op_fwd(x: torch.Tensor, w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor,
                                                         torch.Tensor, torch.Tensor, torch.Tensor]:
    M, K = x.shape
    N = w.shape[0]
    xt, wt, _ = fp8_linear_copies(M, N, K)
    u8 = dict(dtype=torch.uint8, device=x.device)
    # uninitialised records: the forward writes every field the backward reads
    # (a zero fill would cost one more kernel launch per call)
    saved = LinearSaved(M, N, K, tensors=(
        torch.empty((M, K), **u8), torch.empty((K, M), **u8) if xt else None,
        torch.empty((N, K), **u8), torch.empty((K, N), **u8) if wt else None,
        torch.empty((2, SCALE_REC_BYTES), **u8)))
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    fp8_scaled_linear_fwd(x, w, saved, y, OUT_BF16)
    empty = torch.empty(0, dtype=torch.uint8, device=x.device)
    return (y, saved.x_q, saved.x_qT if xt else empty, saved.w_q, saved.w_qT if wt else empty.clone(),
            saved.recs)


@_op_fwd.register_fake
def _op_fwd_fake(x, w):
    M, K = x.shape
    N = w.shape[0]
    xt, wt, _ = fp8_linear_copies(M, N, K)
    u8 = dict(dtype=torch.uint8, device=x.device)
    return (x.new_empty((M, N), dtype=torch.bfloat16), x.new_empty((M, K), **u8),
            x.new_empty((K, M) if xt else (0,), **u8), x.new_empty((N, K), **u8),
            x.new_empty((K, N) if wt else (0,), **u8), x.new_empty((2, SCALE_REC_BYTES), **u8))


@torch.library.custom_op("fp8sg::scaled_linear_bwd", mutates_args=())
def _op_bwd(gy: torch.Tensor, x_q: torch.Tensor, x_qT: torch.Tensor, w_q: torch.Tensor,
            w_qT: torch.Tensor, recs: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    M, N = gy.shape
    K = x_q.shape[1]
    saved = LinearSaved(M, N, K, tensors=(x_q, _present(x_qT), w_q, _present(w_qT), recs))
    gx = torch.empty((M, K), dtype=torch.bfloat16, device=gy.device)
    gw = torch.empty((N, K), dtype=torch.bfloat16, device=gy.device)
    # the backward writes gy's record before it reads it: no zero fill needed
    rec = ScaleRec(buf=torch.empty(SCALE_REC_BYTES, dtype=torch.uint8, device=gy.device))
    ws = LinearBwdWs(M, N, device=gy.device, transposed=fp8_linear_copies(M, N, K)[2], gy_sc=rec)
    fp8_scaled_linear_bwd(gy, saved, ws, gx, gw, OUT_BF16)
    return gx, gw


@_op_bwd.register_fake
def _op_bwd_fake(gy, x_q, x_qT, w_q, w_qT, recs):
    M, N = gy.shape
    K = x_q.shape[1]
    return (gy.new_empty((M, K), dtype=torch.bfloat16), gy.new_empty((N, K), dtype=torch.bfloat16))


def _op_setup(ctx, inputs, output):
    ctx.save_for_backward(*output[1:])
    # the codes and records are state, not differentiable outputs: without
    # this, autograd passes the backward a zero-filled "gradient" of each (one
    # fill kernel per code tensor, up to 117 MB each in the MLP block)
    ctx.set_materialize_grads(False)


def _op_backward(ctx, gy, *_unused):
    if gy is None:  # y took no part in the loss
        return None, None
    if gy.dtype != torch.bfloat16:
        raise TypeError(f"Float8Linear expects bf16 output gradients, got {gy.dtype}")
    gx, gw = torch.ops.fp8sg.scaled_linear_bwd(gy.contiguous(), *ctx.saved_tensors)
    return gx, gw


_op_fwd.register_autograd(_op_backward, setup_context=_op_setup)


class _Fp8LinearFn(torch.autograd.Function):
    """y = x W^T through the FP8 path with delayed or row-wise scaling; saves
    the FP8 codes (row-major and transposed) and the scale records (delayed) or
    scale vectors (row-wise) for the backward pass."""

    @staticmethod
    def forward(ctx, x2d: torch.Tensor, weight: torch.Tensor, mod: "Float8Linear"):
        M, K = x2d.shape
        N = weight.shape[0]
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x2d.device)
        ctx.mod = mod
        ctx.dims = (M, N, K)
        if mod.scaling == "rowwise":
            saved = LinearSavedRW(M, N, K, device=x2d.device)
            fp8_scaled_linear_fwd_rowwise(x2d, weight, saved, y, OUT_BF16)
            ctx.save_for_backward(*saved.tensors())
            return y
        xt, wt, _ = fp8_linear_copies(M, N, K)
        saved = LinearSaved(M, N, K, device=x2d.device, x_transposed=xt, w_transposed=wt)
        if mod.scaling == "delayed":
            if not mod._seeded_fwd:
                _seed_history(mod.hist_x, x2d)
                _seed_history(mod.hist_w, weight)
                mod._seeded_fwd = True
            fp8_scaled_linear_fwd_delayed(x2d, weight, saved, mod.hist_x, mod.hist_w, y, OUT_BF16)
        else:
            fp8_scaled_linear_fwd(x2d, weight, saved, y, OUT_BF16)
        ctx.save_for_backward(*saved.tensors())
        return y

    @staticmethod
    def backward(ctx, gy: torch.Tensor):
        M, N, K = ctx.dims
        mod = ctx.mod
        if gy.dtype != torch.bfloat16:
            raise TypeError(f"Float8Linear expects bf16 output gradients, got {gy.dtype}")
        gy = gy.contiguous()
        gx = torch.empty((M, K), dtype=torch.bfloat16, device=gy.device)
        gw = torch.empty((N, K), dtype=torch.bfloat16, device=gy.device)
        if mod.scaling == "rowwise":
            saved = LinearSavedRW(M, N, K, tensors=ctx.saved_tensors)
            fp8_scaled_linear_bwd_rowwise(gy, saved, mod._bwd_scratch(M, N, gy.device, True), gx,
                                          gw, OUT_BF16)
            return gx, gw, None
        saved = LinearSaved(M, N, K, tensors=ctx.saved_tensors)
        ws = mod._bwd_scratch(M, N, gy.device, False, fp8_linear_copies(M, N, K)[2])
        if mod.scaling == "delayed":
            if not mod._seeded_bwd:
                _seed_history(mod.hist_gy, gy)
                mod._seeded_bwd = True
            fp8_scaled_linear_bwd_delayed(gy, saved, ws, mod.hist_gy, gx, gw, OUT_BF16)
        else:
            fp8_scaled_linear_bwd(gy, saved, ws, gx, gw, OUT_BF16)
        return gx, gw, None


class _Fp8LinearF16Fn(torch.autograd.Function):
    """y = x W^T for an fp16 model under loss scaling [PT-CH20 §20.2.2; FP8-TRAIN
    §2, §4]: fp16 x and W cast to e4m3, the GEMMs in FP8, fp16 y and
    gradients.  The output gradient carries the loss scale; the input gradient
    keeps it (it flows to the layers below), the weight gradient leaves the
    wgrad GEMM unscaled and checked when a GradScaler is attached (its scale and
    non-finite flag), and the scaler then skips that gradient in unscale_."""

    @staticmethod
    def forward(ctx, x2d: torch.Tensor, weight: torch.Tensor, mod: "Float8Linear"):
        M, K = x2d.shape
        N = weight.shape[0]
        xt, wt, _ = fp8_linear_copies(M, N, K)
        saved = LinearSaved(M, N, K, device=x2d.device, x_transposed=xt, w_transposed=wt)
        fp8_amax_f16(x2d, saved.x_sc)
        fp8_quantize_f16(x2d, E4M3FN, saved.x_sc, saved.x_q, saved.x_qT)
        fp8_amax_f16(weight, saved.w_sc)
        fp8_quantize_f16(weight, E4M3FN, saved.w_sc, saved.w_q, saved.w_qT)
        y = torch.empty((M, N), dtype=torch.float16, device=x2d.device)
        fp8_gemm(saved.x_q, E4M3FN, saved.w_q, E4M3FN, saved.x_sc.inv_ptr(), saved.w_sc.inv_ptr(), y,
                 OUT_F16)
        ctx.mod = mod
        ctx.dims = (M, N, K)
        ctx.save_for_backward(*saved.tensors())
        return y

    @staticmethod
    def backward(ctx, gy: torch.Tensor):
        M, N, K = ctx.dims
        mod = ctx.mod
        if gy.dtype != torch.float16:
            raise TypeError(f"an fp16 Float8Linear expects fp16 output gradients, got {gy.dtype}")
        gy = gy.contiguous()
        saved = LinearSaved(M, N, K, tensors=ctx.saved_tensors)
        ws = mod._bwd_scratch(M, N, gy.device, False, fp8_linear_copies(M, N, K)[2])
        fp8_amax_f16(gy, ws.gy_sc)
        fp8_quantize_f16(gy, E5M2, ws.gy_sc, ws.gy_q, ws.gy_qT)
        # an operand without its transposed copy is read contraction-major
        wk, gk, xk = saved.w_qT is None, ws.gy_qT is None, saved.x_qT is None
        gx = torch.empty((M, K), dtype=torch.float16, device=gy.device)
        fp8_gemm_kmajor(ws.gy_q, E5M2, False, saved.w_q if wk else saved.w_qT, E4M3FN, wk,
                        ws.gy_sc.inv_ptr(), saved.w_sc.inv_ptr(), gx, OUT_F16)
        gw = torch.empty((N, K), dtype=torch.float16, device=gy.device)
        a, b = (ws.gy_q if gk else ws.gy_qT), (saved.x_q if xk else saved.x_qT)
        scaler = mod.grad_scaler
        if scaler is not None:
            fp8_gemm_kmajor_unscale(a, E5M2, gk, b, E4M3FN, xk, ws.gy_sc.inv_ptr(),
                                    saved.x_sc.inv_ptr(), scaler._scale, scaler._found, gw)
            scaler._mark_unscaled(mod.weight)
        else:
            fp8_gemm_kmajor(a, E5M2, gk, b, E4M3FN, xk, ws.gy_sc.inv_ptr(), saved.x_sc.inv_ptr(),
                            gw, OUT_F16)
        return gx, gw, None


class Float8Linear(nn.Module):
    """nn.Linear (no bias) whose forward and backward GEMMs run in FP8 with
    per-tensor scaling, "dynamic" (scale from the current tensor) or
    "delayed" (scale from an amax history of history_len earlier steps), or
    with "rowwise" scaling (one scale per row of every operand along the
    dimension its GEMM does not contract).

    dtype torch.float16 makes an fp16 layer for an fp16 model under loss
    scaling (dynamic scaling): fp16 inputs, weight, output and gradients; with
    attach_grad_scaler(scaler), its weight gradient is unscaled and checked in
    the wgrad GEMM's epilogue."""

    def __init__(self, in_features: int, out_features: int, scaling: str = "dynamic",
                 history_len: int = 16, device=None, dtype=torch.bfloat16):
        super().__init__()
        if scaling not in SCALINGS:
            raise ValueError(f"scaling must be one of {SCALINGS}, not {scaling!r}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"Float8Linear takes bf16 or fp16, not {dtype}")
        if dtype == torch.float16 and scaling != "dynamic":
            raise ValueError("an fp16 Float8Linear uses dynamic scaling")
        self.in_features, self.out_features = in_features, out_features
        self.scaling = scaling
        self.grad_scaler = None
        self.weight = nn.Parameter(torch.empty((out_features, in_features), dtype=dtype,
                                               device=device))
        if scaling == "delayed":
            for name in ("hist_x", "hist_w", "hist_gy"):
                self.register_buffer(name, torch.zeros(history_len, dtype=torch.float32,
                                                       device=device))
        self._seeded_fwd = self._seeded_bwd = False
        self._ws = None

    def _bwd_scratch(self, M, N, device, rowwise, transposed=True):
        """The quantized gradient of the backward pass, kept across steps (its
        contents are written and consumed inside one backward call on the
        current stream, so calls on one stream can share it)."""
        key = (M, N, str(device), rowwise, transposed)
        if self._ws is None or self._ws[0] != key:
            ws = LinearBwdWsRW(M, N, device=device) if rowwise else \
                LinearBwdWs(M, N, device=device, transposed=transposed)
            self._ws = (key, ws)
        return self._ws[1]

    def attach_grad_scaler(self, scaler: "GradScaler") -> "Float8Linear":
        """fp16 layers: unscale and check the weight gradient in the wgrad GEMM
        with this scaler's scale and flag (the scaler's unscale_ then skips it)."""
        if self.weight.dtype != torch.float16:
            raise TypeError("the fused unscale serves fp16 layers (fp16 gradients)")
        self.grad_scaler = scaler
        return self

    @classmethod
    def from_float(cls, lin: nn.Linear, scaling: str = "dynamic",
                   history_len: int = 16) -> "Float8Linear":
        """A Float8Linear sharing lin's weight tensor (no copy); an fp16 weight
        makes an fp16 layer."""
        if lin.bias is not None:
            raise ValueError("Float8Linear has no bias")
        if lin.weight.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"Float8Linear needs a bf16 or fp16 weight, got {lin.weight.dtype}")
        with torch.device("meta"):
            new = cls(lin.in_features, lin.out_features, scaling, history_len,
                      dtype=lin.weight.dtype)
        new.weight = lin.weight
        new._ws = None
        if scaling == "delayed":
            for name in ("hist_x", "hist_w", "hist_gy"):
                setattr(new, name, torch.zeros(history_len, dtype=torch.float32,
                                               device=lin.weight.device))
        return new

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dtype != self.weight.dtype:
            raise TypeError(f"Float8Linear takes inputs of its weight's dtype {self.weight.dtype}")
        lead = x.shape[:-1]
        x2d = x.reshape(-1, self.in_features).contiguous()
        if self.weight.dtype == torch.float16:
            y = _Fp8LinearF16Fn.apply(x2d, self.weight, self)
        elif self.scaling == "dynamic":
            y = torch.ops.fp8sg.scaled_linear_fwd(x2d, self.weight)[0]
        else:
            y = _Fp8LinearFn.apply(x2d, self.weight, self)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, " \
               f"scaling={self.scaling}"


# Layers kept in high precision by name [FP8-TRAIN §8: the output head and the
# MoE router, where FP8 costs more convergence than it saves time]: the last
# component of the fully qualified name.
HIGH_PRECISION_NAMES = ("lm_head", "output", "router")


def default_module_filter(mod: nn.Linear, fqn: str) -> bool:
    """Convert a linear layer when the FP8 path can take it (bf16 weight, no
    bias, in and out features multiples of 16) and its name does not mark it as
    the output head or a MoE router."""
    last = fqn.rsplit(".", 1)[-1]
    return (mod.bias is None and mod.weight.dtype in (torch.bfloat16, torch.float16) and
            mod.in_features % 16 == 0 and mod.out_features % 16 == 0 and
            last not in HIGH_PRECISION_NAMES)


def _has_own_bias(mod) -> bool:
    """A bias in the weight's dtype or fp32, as the products' epilogue takes it."""
    b = getattr(mod, "bias", None)
    return b is not None and b.dtype in (mod.weight.dtype, torch.float32)


def _biased_filter(mod: nn.Linear, fqn: str) -> bool:
    """default_module_filter, layers with a bias included."""
    return ((mod.bias is None or _has_own_bias(mod)) and mod.weight.dtype in (torch.bfloat16, torch.float16) and
            mod.in_features % 16 == 0 and mod.out_features % 16 == 0 and
            fqn.rsplit(".", 1)[-1] not in HIGH_PRECISION_NAMES)


def convert_to_float8_training(model: nn.Module,
                               module_filter_fn: Optional[Callable[[nn.Module, str], bool]] = None,
                               scaling: str = "dynamic", history_len: int = 16,
                               grad_scaler: Optional["GradScaler"] = None, biased: bool = False) -> nn.Module:
    """Replace, in place and post-order, every nn.Linear child that
    module_filter_fn(child, fully_qualified_name) accepts (default:
    default_module_filter) with a Float8Linear sharing its weight.  With
    grad_scaler, the fp16 layers unscale and check their weight gradients in
    the wgrad GEMM's epilogue with that scaler.  With biased (dynamic scaling
    only), layers with a bias are replaced too, by a Float8EpilogueLinear that
    shares both, and the default filter accepts them (grad_scaler is not attached to
    those: its unscale_ takes their gradients)."""
    if biased and scaling != "dynamic":
        raise ValueError("layers with a bias are converted with dynamic scaling only")
    accept = module_filter_fn or (_biased_filter if biased else default_module_filter)
    # every (parent, attribute, module, dotted path) below the root, each
    # module after all of its own descendants; the swaps are made after the
    # walk, so it never iterates over a tree it is changing
    edges = list(_descendants_post_order(model, ()))
    for parent, attr, child, path in edges:
        if type(child) is nn.Linear and accept(child, ".".join(path)):
            if biased and child.bias is not None:
                setattr(parent, attr, Float8EpilogueLinear.from_float(child))
                continue
            new = Float8Linear.from_float(child, scaling, history_len)
            if grad_scaler is not None and new.weight.dtype == torch.float16:
                new.attach_grad_scaler(grad_scaler)
            setattr(parent, attr, new)
    return model


def _descendants_post_order(mod: nn.Module, path: tuple):
    for attr, child in mod.named_children():
        yield from _descendants_post_order(child, path + (attr,))
        yield mod, attr, child, path + (attr,)


class GradScaler:
    """Dynamic loss scaling for fp16 gradients with the scale, growth tracker
    and non-finite flag kept on the device.  scale(loss) multiplies by the
    current scale; unscale_(optimizer) unscales the optimizer's gradients in
    place and checks them (optionally also returning their global 2-norm, for
    clipping); step(optimizer) runs optimizer.step() unless a gradient was
    inf/NaN (this reads the flag: one host synchronisation, as in PyTorch's
    GradScaler); update() applies the halve-on-inf / grow-after-interval rule
    and clears the flag."""

    def __init__(self, init_scale: float = 2.0 ** 16, growth_factor: float = 2.0,
                 backoff_factor: float = 0.5, growth_interval: int = 2000, device="cuda"):
        self._scale = torch.tensor([init_scale], dtype=torch.float32, device=device)
        self._tracker = torch.zeros(1, dtype=torch.int32, device=device)
        self._found = torch.zeros(1, dtype=torch.int32, device=device)
        self.growth_factor, self.backoff_factor = growth_factor, backoff_factor
        self.growth_interval = growth_interval
        self._unscaled = set()
        self._pre_unscaled = set()  # parameters whose gradient a layer unscaled this step

    def scale(self, loss: torch.Tensor) -> torch.Tensor:
        # a 0-dim fp32 factor: torch's promotion keeps the loss's own dtype
        # unless it is lower, as PyTorch's GradScaler does
        return loss * self._scale.view(())

    def _mark_unscaled(self, param):
        """An fp16 Float8Linear wrote param's gradient already unscaled and
        checked (wgrad epilogue): unscale_ leaves it alone this step."""
        self._pre_unscaled.add(id(param))

    def _grads(self, optimizer):
        gs = []
        for group in optimizer.param_groups:
            for p in group["params"]:
                if p.grad is None or id(p) in self._pre_unscaled:
                    continue
                if p.grad.dtype != torch.float16 or not p.grad.is_contiguous():
                    raise TypeError("GradScaler unscales contiguous fp16 gradients only")
                gs.append(p.grad)
        return gs

    def unscale_(self, optimizer, with_norm: bool = False):
        """Unscale and check the optimizer's gradients once per step.  With
        with_norm, returns a device float32[2]: (sum of squares, 2-norm) of the
        unscaled gradients taken together."""
        if id(optimizer) in self._unscaled:
            raise RuntimeError("unscale_() has already been called on this optimizer this step")
        grads = self._grads(optimizer)
        self._unscaled.add(id(optimizer))
        if not with_norm:
            amp_unscale_check(grads, self._scale, self._found)
            return None
        ws = torch.empty(amp_norm_workspace_len([g.numel() for g in grads]), dtype=torch.float32,
                         device=self._scale.device)
        out = torch.empty(2, dtype=torch.float32, device=self._scale.device)
        amp_unscale_check_norm(grads, self._scale, self._found, ws, out)
        return out

    def step(self, optimizer, *args, **kwargs):
        if id(optimizer) not in self._unscaled:
            self.unscale_(optimizer)
        if int(self._found.item()) == 0:
            return optimizer.step(*args, **kwargs)
        return None

    def update(self):
        amp_update_scale(self._scale, self._tracker, self._found, self.growth_factor,
                         self.backoff_factor, self.growth_interval)
        self._unscaled.clear()
        self._pre_unscaled.clear()

    def get_scale(self) -> float:
        return float(self._scale.item())

    def state(self):
        """(scale, growth tracker, non-finite flag), read from the device."""
        return self.get_scale(), int(self._tracker.item()), int(self._found.item())


# ------------------------------------------- MXFP4 linears, gated activation, norm
# Each as a pair of registered operators, forward and backward, with fresh
# outputs (torch.compile keeps them as opaque calls).  Workspaces are taken from
# torch's allocator on the current stream, so calls on several streams share
# nothing.

MX_RULES = {"floor": MX_FLOOR, "fit": MX_FIT}
_MX_DTYPES = (torch.bfloat16, torch.float16, torch.float32)


def _flat(x, cols, who):
    """x, whose last dimension is cols, as a matrix (leading dimensions are rows)."""
    if x.dim() < 1 or x.shape[-1] != cols:
        raise ValueError(f"{who} over {cols} values got {tuple(x.shape)}")
    return x.reshape(math.prod(x.shape[:-1]), cols)


def _u8(like, n):
    return like.new_empty(n, dtype=torch.uint8)


def _mx_bytes(rows, k):
    nk = -(-k // 256)
    return rows * 128 * nk, -(-rows // 32) * 256 * nk


@torch.library.custom_op("fp8sg::mxfp4_linear_fwd", mutates_args=())
def _op_mx_fwd(x: torch.Tensor, w: torch.Tensor, rule: int, save: bool) -> tuple[
        torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    M, K = x.shape
    N = w.shape[0]
    y = x.new_empty((M, N))
    saved = Mxfp4LinearSaved(M, N, K, x.device) if save else None
    mxfp4_linear_fwd(x, w, Mxfp4LinearWs(M, N, K, x.device, backward=False), saved, y, rule)
    return (y,) + (saved.tensors() if save else tuple(_u8(x, 0) for _ in range(4)))


@_op_mx_fwd.register_fake
def _op_mx_fwd_fake(x, w, rule, save):
    M, K = x.shape
    N = w.shape[0]
    sizes = _mx_bytes(K, M) + _mx_bytes(K, N) if save else (0, 0, 0, 0)
    return (x.new_empty((M, N)),) + tuple(_u8(x, n) for n in sizes)


@torch.library.custom_op("fp8sg::mxfp4_linear_bwd", mutates_args=())
def _op_mx_bwd(gy: torch.Tensor, xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, K: int,
               rule: int, need_x: bool, need_w: bool) -> tuple[torch.Tensor, torch.Tensor]:
    M, N = gy.shape
    saved = Mxfp4LinearSaved(M, N, K, gy.device, tensors=(xq, xs, wq, ws))
    gx = gy.new_empty((M, K) if need_x else (0,))
    gw = gy.new_empty((N, K) if need_w else (0,))
    mxfp4_linear_bwd(gy, Mxfp4LinearWs(M, N, K, gy.device, forward=False), saved, gx if need_x else None,
                     gw if need_w else None, rule)
    return gx, gw


@_op_mx_bwd.register_fake
def _op_mx_bwd_fake(gy, xq, xs, wq, ws, K, rule, need_x, need_w):
    M, N = gy.shape
    return gy.new_empty((M, K) if need_x else (0,)), gy.new_empty((N, K) if need_w else (0,))


def _mx_setup(ctx, inputs, output):
    x, _w, rule, save = inputs
    ctx.dims, ctx.rule, ctx.saved = (x.shape[1],), rule, save
    ctx.save_for_backward(*output[1:])
    ctx.set_materialize_grads(False)


def _mx_backward(ctx, gy, *_unused):
    need_x, need_w = ctx.needs_input_grad[:2]
    if gy is None or not (need_x or need_w):
        return None, None, None, None
    if not ctx.saved:
        raise RuntimeError("this MXFP4 linear ran without saving for a backward pass")
    gx, gw = torch.ops.fp8sg.mxfp4_linear_bwd(gy.contiguous(), *ctx.saved_tensors, ctx.dims[0], ctx.rule, need_x, need_w)
    return gx if need_x else None, gw if need_w else None, None, None


_op_mx_fwd.register_autograd(_mx_backward, setup_context=_mx_setup)


def _mx_rule(rule):
    if rule not in MX_RULES:
        raise ValueError(f"rule must be one of {tuple(MX_RULES)}, not {rule!r}")
    return rule


class MXFP4Linear(nn.Module):
    """nn.Linear (no bias) whose forward, input-gradient and weight-gradient
    products run in MXFP4: every operand is quantised in blocks of 32 along the
    dimension its product contracts.  Kept for the backward pass are the 4-bit
    x^T and W^T, not the inputs.  Weights, inputs and gradients share one dtype
    (bf16, fp16 or fp32); any sizes.

    rule: how a block's scale follows from its largest value, "floor" (the MX
    specification's, which saturates the top of some blocks) or "fit" (no
    saturation)."""

    def __init__(self, in_features: int, out_features: int, rule: str = "floor", device=None, dtype=torch.bfloat16):
        super().__init__()
        if dtype not in _MX_DTYPES:
            raise TypeError(f"MXFP4Linear takes bf16, fp16 or fp32, not {dtype}")
        self.in_features, self.out_features, self.rule = in_features, out_features, _mx_rule(rule)
        self.weight = nn.Parameter(torch.empty((out_features, in_features), dtype=dtype, device=device))

    @classmethod
    def from_float(cls, lin: nn.Linear, rule: str = "floor") -> "MXFP4Linear":
        """An MXFP4Linear sharing lin's weight tensor (no copy)."""
        if lin.bias is not None:
            raise ValueError("MXFP4Linear has no bias")
        if lin.weight.dtype not in _MX_DTYPES:
            raise TypeError(f"MXFP4Linear needs a bf16, fp16 or fp32 weight, got {lin.weight.dtype}")
        with torch.device("meta"):
            new = cls(lin.in_features, lin.out_features, rule, dtype=lin.weight.dtype)
        new.weight = lin.weight
        return new

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dtype != self.weight.dtype:
            raise TypeError(f"MXFP4Linear takes inputs of its weight's dtype {self.weight.dtype}")
        x2d = _flat(x, self.in_features, "MXFP4Linear").contiguous()
        save = torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad)
        y = torch.ops.fp8sg.mxfp4_linear_fwd(x2d, self.weight.contiguous(), MX_RULES[self.rule], save)[0]
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, rule={self.rule}"


class PackedMXFP4Linear(nn.Module):
    """A linear for serving: the weight is held as MXFP4 (17/32 byte a value) and
    only inputs are quantised, for a few tokens in the product's own launch.
    No gradients."""

    def __init__(self, in_features: int, out_features: int, rule: str = "floor", device=None):
        super().__init__()
        self.in_features, self.out_features, self.rule = in_features, out_features, _mx_rule(rule)
        nq, ns = _mx_bytes(out_features, in_features)
        self.register_buffer("weight_q", torch.zeros(nq, dtype=torch.uint8, device=device))
        self.register_buffer("weight_s", torch.zeros(ns, dtype=torch.uint8, device=device))

    @classmethod
    def from_float(cls, lin: nn.Module, rule: Optional[str] = None) -> "PackedMXFP4Linear":
        """The packed form of an nn.Linear's or MXFP4Linear's weight.  rule None: the
        one an MXFP4Linear was trained with, "floor" for an nn.Linear."""
        if getattr(lin, "bias", None) is not None:
            raise ValueError("PackedMXFP4Linear has no bias")
        if rule is None:
            rule = lin.rule if isinstance(lin, MXFP4Linear) else "floor"
        w = lin.weight.detach()
        new = cls(w.shape[1], w.shape[0], rule, device=w.device)
        mxfp4_quantize(w.contiguous(), new._packed(), rule=MX_RULES[new.rule])
        return new

    def _packed(self):
        return Mxfp4(self.out_features, self.in_features, tensors=(self.weight_q, self.weight_s))

    @torch.no_grad()
    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2d = _flat(x, self.in_features, "PackedMXFP4Linear").contiguous()
        y = x2d.new_empty((x2d.shape[0], self.out_features))
        mxfp4_linear_apply(x2d, self._packed(), y, Mxfp4(x2d.shape[0], self.in_features, x.device),
                           MX_RULES[self.rule])
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, rule={self.rule}"


def _mx_filter(mod: nn.Module, fqn: str, biased: bool = False) -> bool:
    """As default_module_filter, without its rules on sizes (MXFP4 takes any)."""
    b = getattr(mod, "bias", None)
    return ((b is None or biased and _has_own_bias(mod)) and mod.weight.dtype in _MX_DTYPES and
            fqn.rsplit(".", 1)[-1] not in HIGH_PRECISION_NAMES)


def _mx_accept(module_filter_fn, biased):
    return module_filter_fn or (lambda m, fqn: _mx_filter(m, fqn, biased))


def _replace_linears(model, accept, make):
    for parent, attr, child, path in list(_descendants_post_order(model, ())):
        if type(child) in (nn.Linear, MXFP4Linear, MXFP4EpilogueLinear) and accept(child, ".".join(path)):
            setattr(parent, attr, make(child))
    return model


def convert_to_mxfp4_training(model: nn.Module,
                              module_filter_fn: Optional[Callable[[nn.Module, str], bool]] = None,
                              rule: str = "floor", biased: bool = False) -> nn.Module:
    """convert_to_float8_training's walk with MXFP4Linear: every nn.Linear child
    that module_filter_fn accepts (default: no bias, not an output head or a
    router by name) is replaced in place by one that shares its weight.  With
    biased, layers with a bias too, by an MXFP4EpilogueLinear that shares both."""
    accept = _mx_accept(module_filter_fn, biased)
    return _replace_linears(model, lambda m, fqn: type(m) is nn.Linear and accept(m, fqn),
                            lambda m: MXFP4EpilogueLinear.from_float(m, rule=rule) if biased and m.bias is not None
                            else MXFP4Linear.from_float(m, rule))


def convert_to_mxfp4_serving(model: nn.Module,
                             module_filter_fn: Optional[Callable[[nn.Module, str], bool]] = None,
                             rule: Optional[str] = None, biased: bool = False) -> nn.Module:
    """Replace, in place, every nn.Linear and MXFP4Linear child that the filter
    accepts by a PackedMXFP4Linear holding its quantised weight.  rule None: each
    layer's own, "floor" for an nn.Linear.  With biased, layers with a bias and
    MXFP4EpilogueLinears too, by a PackedMXFP4EpilogueLinear."""
    accept = _mx_accept(module_filter_fn, biased)

    def make(m):
        if type(m) is MXFP4EpilogueLinear or biased and getattr(m, "bias", None) is not None:
            return PackedMXFP4EpilogueLinear.from_float(m, rule=rule)
        return PackedMXFP4Linear.from_float(m, rule)
    return _replace_linears(model, lambda m, fqn: (biased or type(m) is not MXFP4EpilogueLinear) and accept(m, fqn),
                            make)


# ---- gated activation

def _rows_of(t):
    """t with contiguous rows that may be apart, as the kernels read them (a
    column range of a matrix stays as it is)."""
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t
    return t.contiguous()


@torch.library.custom_op("fp8sg::swiglu_fwd", mutates_args=())
def _op_swiglu_fwd(g: torch.Tensor, u: torch.Tensor, save: bool) -> tuple[
        torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    rows, cols = g.shape
    a = g.new_empty((rows, cols))
    c = [Act8(rows, cols, g.device) for _ in range(2)] if save else [None, None]
    swiglu_fwd(g, u, a, *c)
    return (a,) + (c[0].tensors() + c[1].tensors() if save else tuple(_u8(g, 0) for _ in range(4)))


@_op_swiglu_fwd.register_fake
def _op_swiglu_fwd_fake(g, u, save):
    rows, cols = g.shape
    n = -(-cols // 32)
    shapes = ((rows, 32 * n), (rows, n)) * 2 if save else ((0,),) * 4
    return (g.new_empty((rows, cols)),) + tuple(_u8(g, s) for s in shapes)


@torch.library.custom_op("fp8sg::swiglu_bwd", mutates_args=())
def _op_swiglu_bwd(da: torch.Tensor, gq: torch.Tensor, gs: torch.Tensor, uq: torch.Tensor,
                   us: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    rows, cols = da.shape
    dg, du = torch.empty_like(da), torch.empty_like(da)
    swiglu_bwd(da, Act8(rows, cols, tensors=(gq, gs)), Act8(rows, cols, tensors=(uq, us)), dg, du)
    return dg, du


@_op_swiglu_bwd.register_fake
def _op_swiglu_bwd_fake(da, gq, gs, uq, us):
    return torch.empty_like(da), torch.empty_like(da)


@torch.library.custom_op("fp8sg::swiglu_bwd_plain", mutates_args=())
def _op_swiglu_bwd_plain(da: torch.Tensor, g: torch.Tensor, u: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    dg, du = torch.empty_like(da), torch.empty_like(da)
    swiglu_bwd(da, g, u, dg, du)
    return dg, du


@_op_swiglu_bwd_plain.register_fake
def _op_swiglu_bwd_plain_fake(da, g, u):
    return torch.empty_like(da), torch.empty_like(da)


def _swiglu_setup(ctx, inputs, output):
    g, u, save = inputs
    ctx.save_for_backward(*(output[1:] if save else (g, u)))
    ctx.set_materialize_grads(False)


def _swiglu_backward(ctx, da, *_unused):
    if da is None:
        return None, None, None
    op = torch.ops.fp8sg.swiglu_bwd if len(ctx.saved_tensors) == 4 else torch.ops.fp8sg.swiglu_bwd_plain
    return (*op(da.contiguous(), *ctx.saved_tensors), None)


_op_swiglu_fwd.register_autograd(_swiglu_backward, setup_context=_swiglu_setup)


class SwiGLU(nn.Module):
    """silu(gate) * up.  checkpoint: keep both for the backward pass as 8-bit
    blocks (33/32 bytes a value) instead of themselves; the result is the same,
    the gradients are those at the kept values.  gate and up may be the two
    halves of one projection's output."""

    def __init__(self, checkpoint: bool = True):
        super().__init__()
        self.checkpoint = checkpoint

    def forward(self, gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
        if gate.shape != up.shape or gate.dtype != up.dtype:
            raise ValueError(f"gate {tuple(gate.shape)} {gate.dtype} and up {tuple(up.shape)} {up.dtype} differ")
        if gate.dim() < 1:
            raise ValueError("SwiGLU takes at least one dimension")
        g, u = (_rows_of(t if t.dim() == 2 else _flat(t, gate.shape[-1], "SwiGLU")) for t in (gate, up))
        save = self.checkpoint and torch.is_grad_enabled() and (gate.requires_grad or up.requires_grad)
        return torch.ops.fp8sg.swiglu_fwd(g, u, save)[0].reshape(gate.shape)

    def extra_repr(self):
        return f"checkpoint={self.checkpoint}"


# ---- layer norm

@torch.library.custom_op("fp8sg::layer_norm_fwd", mutates_args=())
def _op_ln_fwd(x: torch.Tensor, w: Optional[torch.Tensor], b: Optional[torch.Tensor], eps: float, save: bool) -> tuple[
        torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    rows, cols = x.shape
    y = torch.empty_like(x)
    mean, rstd = (x.new_empty(rows, dtype=torch.float32) for _ in range(2))
    c = Act8(rows, cols, x.device) if save else None
    layer_norm_fwd(x, w, b, eps, y, mean, rstd, c)
    return (y, mean, rstd) + (c.tensors() if save else (_u8(x, 0), _u8(x, 0)))


@_op_ln_fwd.register_fake
def _op_ln_fwd_fake(x, w, b, eps, save):
    rows, cols = x.shape
    n = -(-cols // 32)
    st = x.new_empty(rows, dtype=torch.float32)
    shapes = ((rows, 32 * n), (rows, n)) if save else ((0,), (0,))
    return (torch.empty_like(x), st, torch.empty_like(st)) + tuple(_u8(x, s) for s in shapes)


@torch.library.custom_op("fp8sg::layer_norm_bwd", mutates_args=())
def _op_ln_bwd(dy: torch.Tensor, x: Optional[torch.Tensor], xq: Optional[torch.Tensor], xs: Optional[torch.Tensor],
               w: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, need: int,
               pdtype: torch.dtype) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    rows, cols = dy.shape
    dx = torch.empty_like(dy) if need & 1 else dy.new_empty(0)
    dw, db = (dy.new_empty(cols if need & m else 0, dtype=pdtype) for m in (2, 4))
    ws = dy.new_empty(layer_norm_workspace_len(rows, cols), dtype=torch.float32) if need & 6 else None
    layer_norm_bwd(dy, Act8(rows, cols, tensors=(xq, xs)) if x is None else x, w, mean, rstd,
                   dx if need & 1 else None, dw if need & 2 else None, db if need & 4 else None, ws)
    return dx, dw, db


@_op_ln_bwd.register_fake
def _op_ln_bwd_fake(dy, x, xq, xs, w, mean, rstd, need, pdtype):
    cols = dy.shape[1]
    return (torch.empty_like(dy) if need & 1 else dy.new_empty(0),
            dy.new_empty(cols if need & 2 else 0, dtype=pdtype), dy.new_empty(cols if need & 4 else 0, dtype=pdtype))


def _ln_setup(ctx, inputs, output):
    x, w, b, _eps, save = inputs
    _y, mean, rstd, xq, xs = output
    ctx.kept = save
    ctx.pdtype = w.dtype if w is not None else b.dtype if b is not None else x.dtype
    ctx.save_for_backward(w, mean, rstd, *((xq, xs) if save else (x,)))
    ctx.mark_non_differentiable(mean, rstd, xq, xs)
    ctx.set_materialize_grads(False)


def _ln_backward(ctx, dy, *_unused):
    need = sum(m for m, f in zip((1, 2, 4), ctx.needs_input_grad) if f)
    if dy is None or not need:
        return None, None, None, None, None
    w, mean, rstd, *kept = ctx.saved_tensors
    x, xq, xs = (None, *kept) if ctx.kept else (kept[0], None, None)
    got = torch.ops.fp8sg.layer_norm_bwd(dy.contiguous(), x, xq, xs, w, mean, rstd, need, ctx.pdtype)
    return (*(t if need & m else None for t, m in zip(got, (1, 2, 4))), None, None)


_op_ln_fwd.register_autograd(_ln_backward, setup_context=_ln_setup)


class LayerNorm(nn.Module):
    """Layer norm over the last dimension, with its own forward and backward
    kernels.  Parameters are of the data's dtype or fp32.  checkpoint: keep the
    input for the backward pass as 8-bit blocks instead of itself (mean and rstd
    are kept in fp32 either way)."""

    def __init__(self, normalized_shape: int, eps: float = 1e-5, elementwise_affine: bool = True, bias: bool = True,
                 checkpoint: bool = False, device=None, dtype=torch.float32):
        super().__init__()
        if normalized_shape < 1:
            raise ValueError(f"normalized_shape must be at least 1, not {normalized_shape}")
        self.normalized_shape, self.eps, self.checkpoint = normalized_shape, eps, checkpoint
        kw = dict(device=device, dtype=dtype)
        self.weight = nn.Parameter(torch.ones(normalized_shape, **kw)) if elementwise_affine else None
        self.bias = nn.Parameter(torch.zeros(normalized_shape, **kw)) if elementwise_affine and bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2d = _flat(x, self.normalized_shape, "LayerNorm").contiguous()
        needs = any(t is not None and t.requires_grad for t in (x, self.weight, self.bias))
        save = self.checkpoint and torch.is_grad_enabled() and needs
        return torch.ops.fp8sg.layer_norm_fwd(x2d, self.weight, self.bias, self.eps, save)[0].reshape(x.shape)

    def extra_repr(self):
        return f"{self.normalized_shape}, eps={self.eps}, checkpoint={self.checkpoint}"

# ------------------------------- linears with an epilogue in their product, dropout
# y = residual + dropout(act(x W^T + b)), everything behind the product in its
# epilogue, and dropout on its own.  Dropout's masks come from a counter-based
# generator and are never stored: a pass keeps its two words (16 bytes) instead.  The
# words are drawn from torch's generator of the device, so manual_seed,
# torch.utils.checkpoint and a replayed graph govern them as they govern torch's own
# dropout.

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}
_T = torch.Tensor  # (in the long signatures below)


def dropout_words(device) -> torch.Tensor:
    """Two words for one dropout, from torch's generator of the device."""
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), device=device, dtype=torch.int64)


def _ep_part(like, M, N):
    return like.new_empty(epilogue_workspace_len(M, N), dtype=torch.float32)


def _changes(act, p):
    """Whether the backward step's result is another tensor than its input."""
    return act != ACT_NONE or p > 0


# ------------------------------------------------------------------------- FP8

@torch.library.custom_op("fp8sg::scaled_linear_epilogue_fwd", mutates_args=())
def _op_ep_fwd(x: _T, w: _T, bias: Optional[_T], residual: Optional[_T], rng: Optional[_T], act: int, p: float,
               save: bool) -> tuple[_T, _T, _T, _T, _T, _T, _T]:
    M, K = x.shape
    N = w.shape[0]
    xt, wt, _ = fp8_linear_copies(M, N, K) if save else (False, False, False)
    # uninitialised records: the forward writes every field the backward reads
    saved = LinearSaved(M, N, K, tensors=(
        _u8(x, (M, K)), _u8(x, (K, M)) if xt else None, _u8(x, (N, K)), _u8(x, (K, N)) if wt else None,
        _u8(x, (2, SCALE_REC_BYTES))))
    y = x.new_empty((M, N))
    pre = x.new_empty((M, N)) if save and act != ACT_NONE else None
    fp8_scaled_linear_fwd_epilogue(x, w, saved, y, bias=bias, act=act, residual=residual, pre=pre, p=p, rng=rng)
    kept = saved.tensors() if save else (None,) * 5
    return (y, pre if pre is not None else x.new_empty(0)) + tuple(t if t is not None else _u8(x, 0) for t in kept)


@_op_ep_fwd.register_fake
def _op_ep_fwd_fake(x, w, bias, residual, rng, act, p, save):
    # (which copies are made depends on the sizes: a traced size becomes a constant)
    M, N, K = int(x.shape[0]), int(w.shape[0]), int(x.shape[1])
    xt, wt, _ = fp8_linear_copies(M, N, K) if save else (False, False, False)
    shapes = ((M, K), (K, M) if xt else (0,), (N, K), (K, N) if wt else (0,), (2, SCALE_REC_BYTES)) if save else \
        ((0,),) * 5
    return (x.new_empty((M, N)), x.new_empty((M, N) if save and act != ACT_NONE else (0,))) + \
        tuple(_u8(x, s) for s in shapes)


@torch.library.custom_op("fp8sg::scaled_linear_epilogue_bwd", mutates_args=())
def _op_ep_bwd(gy: _T, pre: _T, rng: Optional[_T], x_q: _T, x_qT: _T, w_q: _T, w_qT: _T, recs: _T, act: int, p: float,
               need_b: bool, bdtype: torch.dtype) -> tuple[_T, _T, _T]:
    M, N = gy.shape
    K = x_q.shape[1]
    saved = LinearSaved(M, N, K, tensors=(x_q, _present(x_qT), w_q, _present(w_qT), recs))
    ws = LinearBwdWs(M, N, device=gy.device, transposed=fp8_linear_copies(M, N, K)[2],
                     gy_sc=ScaleRec(buf=_u8(gy, SCALE_REC_BYTES)))
    gx, gw = gy.new_empty((M, K)), gy.new_empty((N, K))
    gb = gy.new_empty(N if need_b else 0, dtype=bdtype)
    fp8_scaled_linear_bwd_epilogue(gy, saved, ws, gx, gw, gh=torch.empty_like(gy) if _changes(act, p) else None,
                                   gb=gb if need_b else None, pre=_present(pre), act=act, p=p, rng=rng,
                                   part=_ep_part(gy, M, N) if need_b else None)
    return gx, gw, gb


@_op_ep_bwd.register_fake
def _op_ep_bwd_fake(gy, pre, rng, x_q, x_qT, w_q, w_qT, recs, act, p, need_b, bdtype):
    M, N = gy.shape
    K = x_q.shape[1]
    return gy.new_empty((M, K)), gy.new_empty((N, K)), gy.new_empty(N if need_b else 0, dtype=bdtype)


def _ep_setup(ctx, inputs, output):
    x, _w, bias, _res, rng, act, p = inputs[:7]
    ctx.act, ctx.p, ctx.rest = act, p, inputs[7:]
    ctx.saved = inputs[-1]
    ctx.K = x.shape[1]
    ctx.bdtype = bias.dtype if bias is not None else x.dtype
    ctx.save_for_backward(rng, *output[1:])
    ctx.set_materialize_grads(False)


def _ep_gy(ctx, gy):
    """gy for a backward operator; needs the forward to have kept what that reads."""
    if not ctx.saved:
        raise RuntimeError("this linear ran without saving for a backward pass")
    return gy.contiguous()


def _ep_backward(ctx, gy, *_unused):
    need = ctx.needs_input_grad
    if gy is None or not any(need[:4]):
        return (None,) * 8
    gx = gw = gb = None
    if any(need[:3]):
        rng, *kept = ctx.saved_tensors
        gx, gw, gb = torch.ops.fp8sg.scaled_linear_epilogue_bwd(_ep_gy(ctx, gy), kept[0], rng, *kept[1:], ctx.act,
                                                                ctx.p, need[2], ctx.bdtype)
    return (gx if need[0] else None, gw if need[1] else None, gb if need[2] else None, gy if need[3] else None,
            None, None, None, None)


_op_ep_fwd.register_autograd(_ep_backward, setup_context=_ep_setup)


# ------------------------------------------------------------------------- MXFP4

@torch.library.custom_op("fp8sg::mxfp4_linear_epilogue_fwd", mutates_args=())
def _op_mxe_fwd(x: _T, w: _T, bias: Optional[_T], residual: Optional[_T], rng: Optional[_T], act: int, p: float,
                rule: int, save: bool) -> tuple[_T, _T, _T, _T, _T, _T]:
    M, K = x.shape
    N = w.shape[0]
    y = x.new_empty((M, N))
    pre = x.new_empty((M, N)) if save and act != ACT_NONE else None
    saved = Mxfp4LinearSaved(M, N, K, x.device) if save else None
    mxfp4_linear_fwd_epilogue(x, w, Mxfp4LinearWs(M, N, K, x.device, backward=False), saved, y, bias=bias, act=act,
                              residual=residual, pre=pre, p=p, rng=rng, rule=rule)
    return (y, pre if pre is not None else x.new_empty(0)) + \
        (saved.tensors() if save else tuple(_u8(x, 0) for _ in range(4)))


@_op_mxe_fwd.register_fake
def _op_mxe_fwd_fake(x, w, bias, residual, rng, act, p, rule, save):
    M, K = x.shape
    N = w.shape[0]
    sizes = _mx_bytes(K, M) + _mx_bytes(K, N) if save else (0, 0, 0, 0)
    return (x.new_empty((M, N)), x.new_empty((M, N) if save and act != ACT_NONE else (0,))) + \
        tuple(_u8(x, n) for n in sizes)


@torch.library.custom_op("fp8sg::mxfp4_linear_epilogue_bwd", mutates_args=())
def _op_mxe_bwd(gy: _T, pre: _T, rng: Optional[_T], xq: _T, xs: _T, wq: _T, ws: _T, K: int, act: int, p: float,
                rule: int, need: int, bdtype: torch.dtype) -> tuple[_T, _T, _T]:
    M, N = gy.shape
    gx = gy.new_empty((M, K) if need & 1 else (0,))
    gw = gy.new_empty((N, K) if need & 2 else (0,))
    gb = gy.new_empty(N if need & 4 else 0, dtype=bdtype)
    products = need & 3
    mxfp4_linear_bwd_epilogue(gy, Mxfp4LinearWs(M, N, K, gy.device, forward=False),
                              Mxfp4LinearSaved(M, N, K, tensors=(xq, xs, wq, ws)), gx if need & 1 else None,
                              gw if need & 2 else None,
                              gh=torch.empty_like(gy) if products and _changes(act, p) else None,
                              gb=gb if need & 4 else None, pre=pre if act != ACT_NONE else None, act=act, p=p,
                              rng=rng, part=_ep_part(gy, M, N) if need & 4 else None, rule=rule)
    return gx, gw, gb


@_op_mxe_bwd.register_fake
def _op_mxe_bwd_fake(gy, pre, rng, xq, xs, wq, ws, K, act, p, rule, need, bdtype):
    M, N = gy.shape
    return (gy.new_empty((M, K) if need & 1 else (0,)), gy.new_empty((N, K) if need & 2 else (0,)),
            gy.new_empty(N if need & 4 else 0, dtype=bdtype))


def _mxe_backward(ctx, gy, *_unused):
    need = ctx.needs_input_grad
    if gy is None or not any(need[:4]):
        return (None,) * 9
    got = [None] * 3
    if any(need[:3]):
        rng, *kept = ctx.saved_tensors
        bits = sum(m for m, f in zip((1, 2, 4), need) if f)
        got = torch.ops.fp8sg.mxfp4_linear_epilogue_bwd(_ep_gy(ctx, gy), kept[0], rng, *kept[1:], ctx.K, ctx.act, ctx.p,
                                                        ctx.rest[0], bits, ctx.bdtype)
    return (*(t if f else None for t, f in zip(got, need)), gy if need[3] else None, None, None, None, None, None)


_op_mxe_fwd.register_autograd(_mxe_backward, setup_context=_ep_setup)


# ------------------------------------------------------------------------- modules

def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, not {name!r}")
    return name


def _probability(p):
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"dropout must lie in [0, 1], not {p}")
    return float(p)


class _EpilogueLinear(nn.Module):
    """What the layers share: parameters, checks and shapes."""
    _dtypes = _MX_DTYPES

    def __init__(self, in_features, out_features, bias, activation, dropout, device, dtype):
        super().__init__()
        if dtype not in self._dtypes:
            raise TypeError(f"{type(self).__name__} takes {', '.join(str(t) for t in self._dtypes)}, not {dtype}")
        self.in_features, self.out_features = in_features, out_features
        self.activation, self.dropout = _activation(activation), _probability(dropout)
        kw = dict(dtype=dtype, device=device)
        self.weight = nn.Parameter(torch.empty((out_features, in_features), **kw))
        self.bias = nn.Parameter(torch.empty(out_features, **kw)) if bias else None

    @classmethod
    def _share(cls, new, lin):
        new.weight, new.bias = lin.weight, lin.bias
        return new.train(lin.training)  # (a layer in evaluation does not begin to drop)

    @classmethod
    def _check_float(cls, lin):
        w, b = lin.weight, lin.bias
        if w.dtype not in cls._dtypes:
            raise TypeError(f"{cls.__name__} needs a weight of {', '.join(str(t) for t in cls._dtypes)}, got {w.dtype}")
        if b is not None and b.dtype not in (w.dtype, torch.float32):
            raise TypeError(f"{cls.__name__} needs a bias of {w.dtype} or float32, got {b.dtype}")

    def _inputs(self, x, residual):
        """(x, residual) as matrices."""
        if x.dtype != self.weight.dtype:
            raise TypeError(f"{type(self).__name__} takes inputs of its weight's dtype {self.weight.dtype}")
        x2d = _flat(x, self.in_features, type(self).__name__).contiguous()
        return x2d, _residual(residual, x.dtype, x.shape[:-1] + (self.out_features,))

    def _drop(self, x):
        """(p, words) of this pass."""
        p = self.dropout if self.training else 0.0
        return (p, dropout_words(x.device)) if p > 0 else (0.0, None)

    def _saves(self, *tensors):
        return torch.is_grad_enabled() and any(
            t is not None and t.requires_grad for t in (self.weight, self.bias) + tensors)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, " \
               f"activation={self.activation}, dropout={self.dropout}"


def _residual(residual, dtype, shape):
    if residual is None:
        return None
    if residual.dtype != dtype or residual.shape != shape:
        raise ValueError(f"residual {tuple(residual.shape)} {residual.dtype}, expected {tuple(shape)} {dtype}")
    return _rows_of(residual if residual.dim() == 2 else _flat(residual, shape[-1], "residual"))


class Float8EpilogueLinear(_EpilogueLinear):
    """residual + dropout(activation(x W^T + b)) through FP8 products with dynamic
    per-tensor scaling, as Float8Linear's; everything behind the product happens in
    its epilogue, in fp32.  activation: "none", "relu", "silu", "gelu" or "gelu_tanh".
    Kept for the backward pass: the FP8 codes, with an activation also x W^T + b in
    the layer's dtype, with dropout its two words.  bf16 or fp16; the sizes and the
    number of rows are multiples of 16.  Gradients of an fp16 layer carry the loss
    scale; a GradScaler's unscale_ takes them (fp16 ones: with an fp32 bias it raises)."""
    _dtypes = (torch.bfloat16, torch.float16)

    def __init__(self, in_features: int, out_features: int, bias: bool = True, activation: str = "none",
                 dropout: float = 0.0, device=None, dtype=torch.bfloat16):
        super().__init__(in_features, out_features, bias, activation, dropout, device, dtype)

    @classmethod
    def from_float(cls, lin: nn.Linear, activation: str = "none", dropout: float = 0.0) -> "Float8EpilogueLinear":
        """One sharing lin's weight and bias (no copies), in lin's mode."""
        cls._check_float(lin)
        with torch.device("meta"):
            new = cls(lin.in_features, lin.out_features, False, activation, dropout, dtype=lin.weight.dtype)
        return cls._share(new, lin)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        x2d, res = self._inputs(x, residual)
        p, rng = self._drop(x)
        y = torch.ops.fp8sg.scaled_linear_epilogue_fwd(x2d, self.weight.contiguous(), self.bias, res, rng,
                                                       ACTIVATIONS[self.activation], p, self._saves(x))[0]
        return y.reshape(*x.shape[:-1], self.out_features)


class MXFP4EpilogueLinear(_EpilogueLinear):
    """The same layer with MXFP4 operands, as MXFP4Linear's (bf16, fp16 or fp32; any
    sizes; `rule`: see there).  Kept for the backward pass: the 4-bit x^T and W^T, with
    an activation also x W^T + b, with dropout its two words."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, activation: str = "none",
                 dropout: float = 0.0, rule: str = "floor", device=None, dtype=torch.bfloat16):
        super().__init__(in_features, out_features, bias, activation, dropout, device, dtype)
        self.rule = _mx_rule(rule)

    @classmethod
    def from_float(cls, lin: nn.Linear, activation: str = "none", dropout: float = 0.0,
                   rule: str = "floor") -> "MXFP4EpilogueLinear":
        """One sharing lin's weight and bias (no copies), in lin's mode."""
        cls._check_float(lin)
        with torch.device("meta"):
            new = cls(lin.in_features, lin.out_features, False, activation, dropout, rule, dtype=lin.weight.dtype)
        return cls._share(new, lin)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        x2d, res = self._inputs(x, residual)
        p, rng = self._drop(x)
        y = torch.ops.fp8sg.mxfp4_linear_epilogue_fwd(x2d, self.weight.contiguous(), self.bias, res, rng,
                                                      ACTIVATIONS[self.activation], p, MX_RULES[self.rule],
                                                      self._saves(x))[0]
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self):
        return super().extra_repr() + f", rule={self.rule}"


class PackedMXFP4EpilogueLinear(nn.Module):
    """The layer for serving: residual + activation(x W^T + b) with the weight held as
    MXFP4, as PackedMXFP4Linear's.  No dropout, no gradients."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, activation: str = "none",
                 rule: str = "floor", device=None, dtype=torch.bfloat16):
        super().__init__()
        if dtype not in _MX_DTYPES:
            raise TypeError(f"PackedMXFP4EpilogueLinear takes a bias of bf16, fp16 or fp32, not {dtype}")
        self.in_features, self.out_features = in_features, out_features
        self.activation, self.rule = _activation(activation), _mx_rule(rule)
        nq, ns = _mx_bytes(out_features, in_features)
        self.register_buffer("weight_q", torch.zeros(nq, dtype=torch.uint8, device=device))
        self.register_buffer("weight_s", torch.zeros(ns, dtype=torch.uint8, device=device))
        self.register_buffer("bias", torch.zeros(out_features, dtype=dtype, device=device) if bias else None)

    @classmethod
    def from_float(cls, lin: nn.Module, activation: Optional[str] = None,
                   rule: Optional[str] = None) -> "PackedMXFP4EpilogueLinear":
        """The packed form of a linear with or without bias.  activation and rule None:
        those the layer was trained with, "none" and "floor" for an nn.Linear."""
        w, b = lin.weight.detach(), getattr(lin, "bias", None)
        if w.dtype not in _MX_DTYPES:
            raise TypeError(f"PackedMXFP4EpilogueLinear needs a bf16, fp16 or fp32 weight, got {w.dtype}")
        new = cls(w.shape[1], w.shape[0], b is not None,
                  activation if activation is not None else getattr(lin, "activation", "none"),
                  rule if rule is not None else getattr(lin, "rule", "floor"), device=w.device,
                  dtype=b.dtype if b is not None else w.dtype)
        mxfp4_quantize(w.contiguous(), new._packed(), rule=MX_RULES[new.rule])
        if b is not None:
            new.bias.copy_(b.detach())
        return new

    def _packed(self):
        return Mxfp4(self.out_features, self.in_features, tensors=(self.weight_q, self.weight_s))

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        x2d = _flat(x, self.in_features, "PackedMXFP4EpilogueLinear").contiguous()
        shape = x.shape[:-1] + (self.out_features,)
        y = x2d.new_empty((x2d.shape[0], self.out_features))
        mxfp4_linear_apply_epilogue(x2d, self._packed(), y, Mxfp4(x2d.shape[0], self.in_features, x.device),
                                    bias=self.bias, act=ACTIVATIONS[self.activation],
                                    residual=_residual(residual, x.dtype, shape), rule=MX_RULES[self.rule])
        return y.reshape(shape)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, " \
               f"activation={self.activation}, rule={self.rule}"


# ------------------------------------------------------------------------- dropout

@torch.library.custom_op("fp8sg::dropout_fwd", mutates_args=())
def _op_drop(x: _T, residual: Optional[_T], rng: _T, p: float) -> _T:
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dropout_fwd(x, p, rng, y, residual=residual)
    return y


@_op_drop.register_fake
def _op_drop_fake(x, residual, rng, p):
    return x.new_empty(x.shape)


@torch.library.custom_op("fp8sg::dropout_bwd", mutates_args=())
def _op_drop_bwd(gy: _T, rng: _T, p: float) -> _T:
    gx = torch.empty(gy.shape, dtype=gy.dtype, device=gy.device)
    dropout_bwd(gy, p, rng, gx)
    return gx


@_op_drop_bwd.register_fake
def _op_drop_bwd_fake(gy, rng, p):
    return gy.new_empty(gy.shape)


def _drop_setup(ctx, inputs, output):
    ctx.p = inputs[3]
    ctx.save_for_backward(inputs[2])
    ctx.set_materialize_grads(False)


def _drop_backward(ctx, gy):
    need = ctx.needs_input_grad
    if gy is None:
        return None, None, None, None
    gx = torch.ops.fp8sg.dropout_bwd(_rows_of(gy), ctx.saved_tensors[0], ctx.p) if need[0] else None
    return gx, gy if need[1] else None, None, None


_op_drop.register_autograd(_drop_backward, setup_context=_drop_setup)


class Dropout(nn.Module):
    """residual + dropout(x) in one pass, forward and backward, with no stored mask.
    p in steps of 2^-16.  In evaluation x (+ residual)."""

    def __init__(self, p: float = 0.5):
        super().__init__()
        self.p = _probability(p)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if x.dtype not in _MX_DTYPES:
            raise TypeError(f"Dropout takes bf16, fp16 or fp32, not {x.dtype}")
        if x.dim() < 1:
            raise ValueError("Dropout takes at least one dimension")
        res = _residual(residual, x.dtype, x.shape)
        if not self.training or self.p == 0:
            return x if residual is None else x + residual
        x2d = _rows_of(x if x.dim() == 2 else _flat(x, x.shape[-1], "Dropout"))
        return torch.ops.fp8sg.dropout_fwd(x2d, res, dropout_words(x.device), self.p).reshape(x.shape)

    def extra_repr(self):
        return f"p={self.p}"
