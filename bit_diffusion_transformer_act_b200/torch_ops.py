"""PyTorch operator registration and nn.Module layers over libsvdq.

The three device calls of include/svdq.h are registered as ``torch.library`` custom
operators (namespace ``svdq``) with fake implementations, so that the layers can be
traced by ``torch.compile(fullgraph=True)`` / ``torch.export`` without graph breaks; the
real implementations are the ctypes calls of ``ops.py`` (the CUDA kernels, on the current
stream).  Method: "Nunchaku Lite" docs, "Supported quantization types" and the
``NunchakuLiteQuantizationConfig`` section (the layers replace nn.Linear in a model).

Operators (all tensors on one CUDA device):
  svdq::quantize_act_lowrank_down(X bf16 [M,K], smooth_inv bf16 [K], packed_w u8,
      act_global_scale float, rank int) -> (codes u8 [M,K/2], scales u8 [svdq_act_scale_bytes],
      lowrank_act bf16 [M,2 rank])
  svdq::w4a4_nvfp4_linear(codes, scales, lowrank_act, act_global_scale, packed_w,
      w_global_scale float, N int, rank int) -> Y bf16 [M,N]
  svdq::awq_w4a16_linear(X bf16 [M,K], qweight u8 [N,K/2], scales bf16 [N,K/64],
      zeros bf16 [N,K/64], bias bf16 [N] or None) -> Y bf16 [M,N]
  svdq::lora_add_(X bf16 [M,K], Y bf16 [M,N], A bf16 [adapters,rank,K], B bf16 [adapters,N,rank],
      plan u8, plan_sizes int[9]) -> (), adds each request's adapters to Y; refuses tensors that carry gradients
  svdq::lora_add_planned_(the same, plan_sizes int64 [9] on the host): the sizes as data, which a compiled graph
      does not depend on
  svdq::lora_add(as lora_add_planned_) -> Y' bf16 [M,N], Y left as it is
  svdq::qk_norm_rope(q bf16 [M,Hq,D], k bf16 [M,Hk,D], norm_wq, norm_wk bf16 [D] or None, eps float,
      positions int32 or fp32 [P,axes], axes_dims int[], theta float[], pairing str) -> (q', k')
  svdq::rope_axes_tables(positions, axes_dims int[], theta float[], head_dim int, rows int)
      -> (cos, sin fp32 [head_dim/2, rows])

They are for inference: none has a gradient, and a backward pass through any of them raises.
"""

from typing import Callable, List, Optional, Sequence, Tuple

import numpy as np
import torch
from torch import nn

from . import ops


# ---------------------------------------------------------------- operators

@torch.library.custom_op("svdq::quantize_act_lowrank_down", mutates_args=())
def quantize_act_lowrank_down(X: torch.Tensor, smooth_inv: torch.Tensor, packed_w: torch.Tensor,
                              act_global_scale: float, rank: int) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return ops.svdq_quantize_act_lowrank_down(X, smooth_inv, packed_w, act_global_scale, rank)


@quantize_act_lowrank_down.register_fake
def _(X, smooth_inv, packed_w, act_global_scale, rank):
    M, K = X.shape
    # swizzled scales: rows padded to the 128-row atom, one byte per 16 K
    return (X.new_empty((M, K // 2), dtype=torch.uint8),
            X.new_empty((((M + 127) // 128) * 128 * (K // 16),), dtype=torch.uint8),
            X.new_empty((M, 2 * rank), dtype=torch.bfloat16))


@torch.library.custom_op("svdq::w4a4_nvfp4_linear", mutates_args=())
def w4a4_nvfp4_linear(act_codes: torch.Tensor, act_scales: torch.Tensor, lowrank_act: torch.Tensor,
                      act_global_scale: float, packed_w: torch.Tensor, w_global_scale: float, N: int,
                      rank: int) -> torch.Tensor:
    M, half_k = act_codes.shape
    return ops.svdq_w4a4_nvfp4_linear(act_codes, act_scales, lowrank_act, act_global_scale, packed_w,
                                      w_global_scale, M, N, 2 * half_k, rank)


@w4a4_nvfp4_linear.register_fake
def _(act_codes, act_scales, lowrank_act, act_global_scale, packed_w, w_global_scale, N, rank):
    return act_codes.new_empty((act_codes.shape[0], N), dtype=torch.bfloat16)


@torch.library.custom_op("svdq::awq_w4a16_linear", mutates_args=())
def awq_w4a16_linear(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                     bias: Optional[torch.Tensor]) -> torch.Tensor:
    return ops.awq_w4a16_linear(X, qweight, scales, zeros, bias)


@awq_w4a16_linear.register_fake
def _(X, qweight, scales, zeros, bias):
    return X.new_empty((X.shape[0], qweight.shape[0]), dtype=torch.bfloat16)


@torch.library.custom_op("svdq::lora_add_", mutates_args={"Y"})
def lora_add_(X: torch.Tensor, Y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, plan: torch.Tensor,
              plan_sizes: List[int]) -> None:
    ops.svdq_lora_add(X, Y, A, B, ops.LoraPlan.from_parts(plan, plan_sizes), out=Y)


@lora_add_.register_fake
def _(X, Y, A, B, plan, plan_sizes):
    return None


def _carries_gradients(*tensors: torch.Tensor) -> bool:
    return torch.is_grad_enabled() and any(t.requires_grad for t in tensors)


# The launches follow from plan_sizes' values, which inductor's CUDA graphs would keep from the first plan.
_READS_HOST_VALUES = (torch.Tag.cudagraph_unsafe,)


@torch.library.custom_op("svdq::lora_add_planned_", mutates_args={"Y"}, tags=_READS_HOST_VALUES)
def lora_add_planned_(X: torch.Tensor, Y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, plan: torch.Tensor,
                      plan_sizes: torch.Tensor) -> None:
    ops.svdq_lora_add(X, Y, A, B, ops.LoraPlan.from_parts(plan, plan_sizes.tolist()), out=Y)


@lora_add_planned_.register_fake
def _(X, Y, A, B, plan, plan_sizes):
    return None


# An operator that changes its argument can have no gradient formula, and without one Y would keep the gradient of
# what it was before: the adapters' part would be missing from it without an error.
def _refuse_gradients(op):
    def call(X, Y, A, B, plan, plan_sizes):
        if _carries_gradients(X, Y, A, B):
            raise RuntimeError(f"{op} has no gradient: call it under torch.no_grad(), on detached tensors, or use "
                               "svdq::lora_add")
        with torch._C._AutoDispatchBelowAutograd():
            op(X, Y, A, B, plan, plan_sizes)
    return call


_LIB = torch.library.Library("svdq", "FRAGMENT")
_LIB.impl("lora_add_", _refuse_gradients(torch.ops.svdq.lora_add_.default), "Autograd", allow_override=True)
_LIB.impl("lora_add_planned_", _refuse_gradients(torch.ops.svdq.lora_add_planned_.default), "Autograd",
          allow_override=True)


@torch.library.custom_op("svdq::lora_add", mutates_args=(), tags=_READS_HOST_VALUES)
def lora_add(X: torch.Tensor, Y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, plan: torch.Tensor,
             plan_sizes: torch.Tensor) -> torch.Tensor:
    return ops.svdq_lora_add(X, Y, A, B, ops.LoraPlan.from_parts(plan, plan_sizes.tolist()))


@lora_add.register_fake
def _(X, Y, A, B, plan, plan_sizes):
    return Y.new_empty(Y.shape)


@torch.library.custom_op("svdq::no_gradient", mutates_args=())
def no_gradient(grad: torch.Tensor, shape: List[int], name: str) -> torch.Tensor:
    """Stands for a gradient that there is none of.  An operator, so that a compiled forward pass runs and only the
    backward pass raises."""
    raise RuntimeError(f"{name} has no gradient (the adapters are for inference): run it under torch.no_grad()")


@no_gradient.register_fake
def _(grad, shape, name):
    return grad.new_empty(shape)


def _lora_add_context(ctx, inputs, output):
    ctx.shapes = [t.shape for t in inputs[:4]]


def _lora_add_backward(ctx, grad):
    return tuple(no_gradient(grad, list(shape), "svdq::lora_add") if need else None
                 for need, shape in zip(ctx.needs_input_grad, ctx.shapes)) + (None, None)


lora_add.register_autograd(_lora_add_backward, setup_context=_lora_add_context)


@torch.library.custom_op("svdq::qk_norm_rope", mutates_args=())
def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, norm_wq: Optional[torch.Tensor], norm_wk: Optional[torch.Tensor],
                 eps: float, positions: torch.Tensor, axes_dims: List[int], theta: List[float],
                 pairing: str) -> Tuple[torch.Tensor, torch.Tensor]:
    return ops.svdq_qk_norm_rope(q, k, norm_wq, norm_wk, eps, positions, axes_dims, theta, pairing)


@qk_norm_rope.register_fake
def _(q, k, norm_wq, norm_wk, eps, positions, axes_dims, theta, pairing):
    return q.new_empty(q.shape), k.new_empty(k.shape)


@torch.library.custom_op("svdq::rope_axes_tables", mutates_args=())
def rope_axes_tables(positions: torch.Tensor, axes_dims: List[int], theta: List[float], head_dim: int,
                     rows: int) -> Tuple[torch.Tensor, torch.Tensor]:
    return ops.svdq_rope_axes_tables(positions, axes_dims, theta, head_dim, rows)


@rope_axes_tables.register_fake
def _(positions, axes_dims, theta, head_dim, rows):
    shape = (head_dim // 2, rows)
    return positions.new_empty(shape, dtype=torch.float32), positions.new_empty(shape, dtype=torch.float32)


# ---------------------------------------------------------------- layers

def _as_2d(x: torch.Tensor, K: int) -> torch.Tensor:
    if x.shape[-1] != K:
        raise ValueError(f"last dimension {x.shape[-1]} != in_features {K}")
    return x.reshape(-1, K).contiguous()


class SvdqLinear(nn.Module):
    """SVDQuant W4A4 NVFP4 linear layer (rank-32 16-bit low-rank branch), a drop-in for
    nn.Linear on bf16 inputs of any leading shape.

    Built from the exporter's parameters (see ``from_exported``); holds the packed weight
    blob, the bf16 smoothing factors and the two power-of-two per-tensor scales."""

    def __init__(self, in_features: int, out_features: int, rank: int, packed_w: torch.Tensor,
                 smooth_inv: torch.Tensor, act_global_scale: float, w_global_scale: float):
        super().__init__()
        self.in_features, self.out_features, self.rank = in_features, out_features, rank
        self.register_buffer("packed_w", packed_w)
        self.register_buffer("smooth_inv", smooth_inv)
        self.act_global_scale = float(act_global_scale)
        self.w_global_scale = float(w_global_scale)

    @classmethod
    def from_exported(cls, R: np.ndarray, L1_bits: np.ndarray, L2_bits: np.ndarray,
                      bias_bits: Optional[np.ndarray], smooth_inv_bits: np.ndarray, act_global_scale: float,
                      device="cuda") -> "SvdqLinear":
        """R float32 [N, K] (residual), L1 / L2 bf16 bit patterns [K, r] / [r, N], bias [N] or None,
        smooth_inv [K] (bf16 bits), act_global_scale a power of two (calibration)."""
        blob, g_w = ops.svdq_pack_weights(R, L1_bits, L2_bits, bias_bits, smooth_inv_bits)
        N, K = R.shape
        smooth = torch.from_numpy(np.ascontiguousarray(smooth_inv_bits, np.uint16).view(np.int16)) \
            .view(torch.bfloat16)
        return cls(K, N, L1_bits.shape[1], torch.from_numpy(blob).to(device), smooth.to(device),
                   act_global_scale, g_w)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = _as_2d(x, self.in_features)
        codes, scales, lowrank = torch.ops.svdq.quantize_act_lowrank_down(
            x2, self.smooth_inv, self.packed_w, self.act_global_scale, self.rank)
        y = torch.ops.svdq.w4a4_nvfp4_linear(codes, scales, lowrank, self.act_global_scale, self.packed_w,
                                             self.w_global_scale, self.out_features, self.rank)
        return y.reshape(*lead, self.out_features)

    def get_extra_state(self):
        # the per-tensor scales and sizes travel with state_dict() next to the buffers
        return {"in_features": self.in_features, "out_features": self.out_features, "rank": self.rank,
                "act_global_scale": self.act_global_scale, "w_global_scale": self.w_global_scale}

    def set_extra_state(self, state):
        self.in_features, self.out_features = int(state["in_features"]), int(state["out_features"])
        self.rank = int(state["rank"])
        self.act_global_scale = float(state["act_global_scale"])
        self.w_global_scale = float(state["w_global_scale"])

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, rank={self.rank}, nvfp4"


class AwqLinear(nn.Module):
    """AWQ-style W4A16 int4 (group 64) linear layer, a drop-in for nn.Linear on bf16 inputs
    of any leading shape (built for the few rows of the adaptive normalisation; more than 64
    rows after flattening run in 64-row tiles that each re-read the weights)."""

    def __init__(self, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                 bias: Optional[torch.Tensor] = None):
        super().__init__()
        self.out_features, half_k = qweight.shape
        self.in_features = 2 * half_k
        self.register_buffer("qweight", qweight)
        self.register_buffer("scales", scales)
        self.register_buffer("zeros", zeros)
        self.register_buffer("bias", bias)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        y = torch.ops.svdq.awq_w4a16_linear(_as_2d(x, self.in_features), self.qweight, self.scales, self.zeros,
                                            self.bias)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, int4 group 64"


class LoraLinear(nn.Module):
    """A shared projection (an SvdqLinear, an AwqLinear, an nn.Linear) with a pool of low-rank adapters beside
    it, of which each request of a batch uses its own: y = base(x) + sum_j w_j B_j (A_j x).

    A bf16 [adapters, rank, in_features], B bf16 [adapters, out_features, rank], the features multiples of 64, the
    rank of 16 and at most 128 (a plan's slots times the rank too).  Which rows use which adapters is the batch's
    plan (``set_plan``; rows are counted after flattening the leading dimensions); without a plan the layer is its
    base.  A compiled layer takes one plan after another without being compiled again: the plan's sizes are data,
    in a small host tensor (and inductor's CUDA graphs leave the adapters' calls out: the number of blocks launched
    follows from the sizes).  For inference: a backward pass through the adapters raises.  (The adapters are added
    to the base's output in place, into a copy only where gradients are on and something carries them.)"""

    def __init__(self, base: nn.Module, A: torch.Tensor, B: torch.Tensor):
        super().__init__()
        adapters, rank, k = A.shape
        if k != base.in_features or tuple(B.shape) != (adapters, base.out_features, rank):
            raise ValueError(f"A {tuple(A.shape)} and B {tuple(B.shape)} do not fit a projection from "
                             f"{base.in_features} to {base.out_features}")
        if base.in_features % 64 or base.out_features % 64:
            raise ValueError(f"adapters need features in multiples of 64, got {base.in_features} to {base.out_features}")
        if rank == 0 or rank % 16 or rank > ops.LORA_MAX_RANK:
            raise ValueError(f"adapters need a rank in multiples of 16 up to {ops.LORA_MAX_RANK}, got {rank}")
        if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
            raise ValueError(f"adapters must be bfloat16, got {A.dtype} and {B.dtype}")
        self.base = base
        self.in_features, self.out_features = base.in_features, base.out_features
        self.register_buffer("A", A)
        self.register_buffer("B", B)
        self.plan_words: Optional[torch.Tensor] = None
        self.plan_sizes: Optional[torch.Tensor] = None

    @classmethod
    def from_adapters(cls, base: nn.Module, adapters: Sequence[Tuple[torch.Tensor, torch.Tensor]]) -> "LoraLinear":
        """adapters: (A [r, in_features], B [out_features, r]) of any ranks r up to 128, padded here with zeros to
        the largest, rounded up to a multiple of 16."""
        rank = (max(a.shape[0] for a, _ in adapters) + 15) // 16 * 16
        dev = adapters[0][0].device
        A = torch.zeros((len(adapters), rank, base.in_features), dtype=torch.bfloat16, device=dev)
        B = torch.zeros((len(adapters), base.out_features, rank), dtype=torch.bfloat16, device=dev)
        for i, (a, b) in enumerate(adapters):
            if a.shape[0] != b.shape[1]:
                raise ValueError(f"adapter {i}: A has rank {a.shape[0]}, B {b.shape[1]}")
            A[i, : a.shape[0]] = a
            B[i, :, : b.shape[1]] = b
        return cls(base, A, B)

    def check_plan(self, plan: ops.LoraPlan) -> None:
        """Raises where the layer cannot serve the plan."""
        adapters, rank, _ = self.A.shape
        if plan.adapters != adapters:
            raise ValueError(f"the plan is for {plan.adapters} adapters, the layer has {adapters}")
        if plan.slots * rank > ops.LORA_MAX_RANK:
            raise ValueError(f"a plan of {plan.slots} slots needs adapters of rank {ops.LORA_MAX_RANK // plan.slots} at "
                             f"most, the layer's have rank {rank}")

    def set_plan(self, plan: Optional[ops.LoraPlan]) -> None:
        if plan is None:
            self.plan_words = self.plan_sizes = None
            return
        self.check_plan(plan)
        self.plan_words = plan.words
        self.plan_sizes = torch.tensor(plan.sizes(), dtype=torch.int64, device="cpu")
        torch._dynamo.maybe_mark_dynamic(self.plan_words, 0)   # plans differ in length

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y = self.base(x)
        if self.plan_words is None:
            return y
        x2, y2 = _as_2d(x, self.in_features), y.reshape(-1, self.out_features)
        if _carries_gradients(x2, y2, self.A, self.B):
            y2 = torch.ops.svdq.lora_add(x2, y2, self.A, self.B, self.plan_words, self.plan_sizes)
        else:
            torch.ops.svdq.lora_add_planned_(x2, y2, self.A, self.B, self.plan_words, self.plan_sizes)
        return y2.reshape(y.shape)

    def extra_repr(self) -> str:
        return f"adapters={self.A.shape[0]}, rank={self.A.shape[1]}"


def attach_adapters(model: nn.Module, factory: Callable[[str, nn.Module], Optional[nn.Module]]) -> int:
    """Replaces, in place, every SvdqLinear, AwqLinear and nn.Linear of ``model`` for which
    ``factory(qualified_name, layer)`` returns a module (for instance a LoraLinear around it); returns how
    many were replaced."""
    replaced = 0
    for parent_name, parent in list(model.named_modules()):
        if isinstance(parent, LoraLinear):
            continue
        for child_name, child in list(parent.named_children()):
            if isinstance(child, (SvdqLinear, AwqLinear, nn.Linear)):
                new = factory(f"{parent_name}.{child_name}" if parent_name else child_name, child)
                if new is not None:
                    setattr(parent, child_name, new)
                    replaced += 1
    return replaced


def set_lora_plan(model: nn.Module, plan: Optional[ops.LoraPlan]) -> None:
    """Sets the batch's plan (None: no adapters) on every LoraLinear of ``model``; on none where one of them cannot
    serve it."""
    layers = [m for m in model.modules() if isinstance(m, LoraLinear)]
    if plan is not None:
        for m in layers:
            m.check_plan(plan)
    for m in layers:
        m.set_plan(plan)


def swap_linears(model: nn.Module, factory: Callable[[str, nn.Linear], Optional[nn.Module]]) -> int:
    """Replaces, in place, every nn.Linear of ``model`` for which ``factory(qualified_name, linear)``
    returns a module (for instance an SvdqLinear or AwqLinear built from that layer's exported
    parameters); returns how many were replaced."""
    replaced = 0
    for parent_name, parent in list(model.named_modules()):
        for child_name, child in list(parent.named_children()):
            if isinstance(child, nn.Linear):
                name = f"{parent_name}.{child_name}" if parent_name else child_name
                new = factory(name, child)
                if new is not None:
                    setattr(parent, child_name, new)
                    replaced += 1
    return replaced
