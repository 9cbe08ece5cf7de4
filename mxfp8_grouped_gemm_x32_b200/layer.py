"""Device buffers for one grouped MXFP8 MoE expert layer, driven through the
C ABI.  PyTorch only allocates device memory and provides the stream; every
step of the layer runs in the CUDA library (see lib.py).

Steps (names of the C entry points):
  quantize_weights  moe_mlp_quantize_weights: W_gate_up and W_down, along K
                    for the forward and along the other axis for the backward
                    (forward only: moe_mlp_quantize_mxfp8 x2)
  route             moe_router_topk: router logits -> top-k experts + probabilities
  route_losses      moe_router_losses: the same with the load-balance loss, the
                    z-loss and the tokens per expert
  route_backward    moe_router_bwd: gradient of the logits from d(prob) and the
                    losses' gradients
  permute           moe_permute: counting sort by expert, gather + quantise x
  forward           moe_grouped_mlp_fwd: gate_up GEMM + ScaledSwiGLU + requant,
                    down GEMM, top-k combine
  forward_bf16      moe_grouped_mlp_fwd_bf16: the same layer with bf16 operands
                    (routing from permute_index, moe_permute without x)
  backward_bf16     moe_grouped_mlp_bwd_bf16: its backward
  forward_fp8_tensor / backward_fp8_tensor
                    moe_grouped_mlp_fwd/bwd_fp8_tensor: the per-tensor FP8 recipe
  quantize_weights_mxfp4 / load_weights_mxfp4, forward_mxfp4
                    moe_mlp_quantize_mxfp4, moe_grouped_mlp_fwd_mxfp4: the MXFP4
                    (4-bit) serving recipe, routing from permute_index
  backward          moe_grouped_mlp_bwd: dgrad/wgrad of both projections,
                    ScaledSwiGLU backward, d(prob)
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import lib


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def check_tensor(t, name: str, dtype, shape, device) -> None:
    """Raise unless `t` is a contiguous tensor of `dtype` and `shape` on
    `device`.  The library receives raw pointers, so a host tensor or a
    wrong shape must be caught here, before any kernel reads through it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


GUARD_BYTE = 0xA5


class _Alloc:
    """Device buffers of one layer.  With guard > 0 every buffer is followed
    by `guard` bytes of a fixed pattern (a debug aid: check() names every
    buffer whose tail was written, i.e. a write past its end)."""

    def __init__(self, dev, guard: int = 0):
        self.dev, self.guard = dev, (guard + 255) // 256 * 256
        self.tails = []

    def raw(self, nbytes: int, name: str) -> torch.Tensor:
        # 256-byte aligned by the caching allocator; sizes rounded to 16 bytes
        n = max(16, (nbytes + 15) // 16 * 16)
        if not self.guard:
            return torch.empty(n, dtype=torch.uint8, device=self.dev)
        n256 = (n + 255) // 256 * 256
        buf = torch.empty(n256 + self.guard, dtype=torch.uint8, device=self.dev)
        buf[n:].fill_(GUARD_BYTE)
        self.tails.append((name, buf[n:]))
        return buf[:n]

    def typed(self, shape, dtype, name: str) -> torch.Tensor:
        numel = 1
        for d in shape:
            numel *= d
        esz = torch.empty(0, dtype=dtype).element_size()
        return self.raw(numel * esz, name)[: numel * esz].view(dtype).view(*shape)

    def check(self):
        """Names of the buffers whose guard bytes changed."""
        return [name for name, t in self.tails if not bool((t == GUARD_BYTE).all())]


_DTYPES = {torch.float32: lib.MOE_DTYPE_F32, torch.bfloat16: lib.MOE_DTYPE_BF16}


def _logits_dtype(logits) -> int:
    dt = _DTYPES.get(getattr(logits, "dtype", None))
    if dt is None:
        raise TypeError(f"logits: expected float32 or bfloat16, got {getattr(logits, 'dtype', type(logits).__name__)}")
    return dt


def on_device(dev: torch.device):
    """Context in which `dev` is the current device (the library launches on
    the current device; nothing to do when it already is)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _on_layer_device(call):
    """A method that runs with its layer's device current."""
    @functools.wraps(call)
    def wrapped(self, *args, **kwargs):
        with on_device(self.dev):
            return call(self, *args, **kwargs)
    return wrapped


# the raw handle of a device's current stream; the public call builds a Stream
# object first, which takes longer (3 us) than a small kernel's launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class GroupedMLP:
    """One layer: T tokens, hidden H, intermediate I, E experts, top-k.

    mxfp8=False leaves out the buffers of the MXFP8 recipe (quantised weights,
    x and h and its workspaces): a layer that routes and serves in MXFP4, or
    runs one of the recipes on bf16 weights, does not need them.

    Results and workspaces are the layer's buffers, overwritten by the next call
    of the same kind: one stream at a time, and no two captured graphs of one
    layer replayed at the same time.  Layers beside each other are
    independent."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, device="cuda", backward: bool = True,
                 guard: int = 0, mxfp8: bool = True):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.dev = torch.device(device)
        al = self._alloc = _Alloc(self.dev, guard)
        u8 = al.raw
        self.rows_cap = lib.moe_padded_rows(T, k, E)
        rc = self.rows_cap
        sb = lib.moe_mx_scale_bytes
        self.mxfp8 = mxfp8
        if mxfp8:
            # quantised weights (forward: along H for gate_up, along I for down)
            self.w1q = u8(2 * E * I * H, "w1q")
            self.w1sf = u8(sb(2 * E, I, H), "w1sf")
            self.w2q = u8(E * H * I, "w2q")
            self.w2sf = u8(sb(E, H, I), "w2sf")
        # routing
        self.split_sizes = al.typed((E,), torch.int32, "split_sizes")
        self.group_offsets = al.typed((E + 1,), torch.int32, "group_offsets")
        self.row_to_slot = al.typed((rc,), torch.int32, "row_to_slot")
        self.slot_to_row = al.typed((T * k,), torch.int32, "slot_to_row")
        # router outputs: topk_idx and topk_prob are those of the last routing
        # call; route_losses has its own (kept for route_backward)
        self._routed = (al.typed((T, k), torch.int32, "topk_idx"), al.typed((T, k), torch.float32, "topk_prob"))
        self.topk_idx, self.topk_prob = self._routed
        self.prob_perm = al.typed((rc,), torch.float32, "prob_perm")
        if mxfp8:
            self.xq = u8(rc * H, "xq")
            self.xq_sf = u8(sb(1, rc, H), "xq_sf")
            self.hq = u8(rc * I, "hq")
            self.hq_sf = u8(sb(1, rc, I), "hq_sf")
        self.out = al.typed((T, H), torch.bfloat16, "out")
        self.dev = self.out.device      # concrete device (index resolved) for the input checks
        self.ws_perm_bytes = lib.moe_workspace_size(lib.MOE_OP_PERMUTE, T, k, E, H, I)
        self.ws_perm = u8(self.ws_perm_bytes, "ws_perm")
        if mxfp8:
            self.ws_fwd_bytes = lib.moe_workspace_size(lib.MOE_OP_FWD, T, k, E, H, I)
            self.ws_fwd = u8(self.ws_fwd_bytes, "ws_fwd")
        self.backward_enabled = backward
        if backward and mxfp8:
            self.w1tq = u8(E * H * 2 * I, "w1tq")
            self.w1tsf = u8(sb(E, H, 2 * I), "w1tsf")
            self.w2tq = u8(E * I * H, "w2tq")
            self.w2tsf = u8(sb(E, I, H), "w2tsf")
            self.ws_bwd_bytes = lib.moe_workspace_size(lib.MOE_OP_BWD, T, k, E, H, I)
            self.ws_bwd = u8(self.ws_bwd_bytes, "ws_bwd")
        if backward:
            self.saved_a = al.typed((rc, 2 * I), torch.bfloat16, "saved_a")
            self.dX = al.typed((T, H), torch.bfloat16, "dX")
            self.dW1 = al.typed((E, 2 * I, H), torch.bfloat16, "dW1")
            self.dW2 = al.typed((E, H, I), torch.bfloat16, "dW2")
            self.dprob = al.typed((T, k), torch.float32, "dprob")
        else:
            self.saved_a = None
        self.xq_col = self.xq_col_sf = None   # x along tokens: only when permute(..., with_cols=True)
        self._x = None                         # the input of the last permutation (the backward's x)
        self.router_lse = None                 # route_losses' outputs and mask, once it has run
        self._loss_mask = None
        self.dlogits = {}                      # route_backward's, one buffer per type it has met
        self.w1q4 = None                       # MXFP4 weights, once quantised or loaded
        self._permuted = False                 # whether the routing buffers hold a permutation

    def _need_mxfp8(self):
        if not self.mxfp8:
            raise RuntimeError("this layer was built with mxfp8=False")

    def _cols(self, with_cols: bool):
        """Buffers of the optional column form of x (x^T quantised along
        tokens in permuted order); the backward does not need them."""
        if not with_cols:
            return 0, 0
        if self.xq_col is None:
            self.xq_col = self._alloc.raw(self.H * self.rows_cap, "xq_col")
            self.xq_col_sf = self._alloc.raw(lib.moe_mx_scale_bytes(1, self.H, self.rows_cap), "xq_col_sf")
        return _ptr(self.xq_col), _ptr(self.xq_col_sf)

    def permute_index(self, topk_idx: torch.Tensor, topk_prob: torch.Tensor) -> None:
        """Routing outputs of the permutation only (no quantisation of x):
        what the BF16, per-tensor FP8 and MXFP4 forwards need."""
        check_tensor(topk_idx, "topk_idx", torch.int32, (self.T, self.k), self.dev)
        check_tensor(topk_prob, "topk_prob", torch.float32, (self.T, self.k), self.dev)
        with on_device(self.dev):
            lib.moe_permute(0, topk_idx.data_ptr(), topk_prob.data_ptr(), self.T, self.H, self.k, self.E,
                            self.rows_cap, _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                            _ptr(self.slot_to_row), _ptr(self.prob_perm), 0, 0, 0, 0, _ptr(self.ws_perm),
                            self.ws_perm_bytes, self._stream())
        self._permuted = True

    @_on_layer_device
    def forward_bf16(self, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor) -> torch.Tensor:
        """BF16 recipe forward (moe_grouped_mlp_fwd_bf16) on the routing of
        the last permute / permute_index: x bf16 [T, H], w1 bf16 [E, 2I, H],
        w2 bf16 [E, H, I] -> out."""
        E, H, I = self.E, self.H, self.I
        check_tensor(x, "x", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        if getattr(self, "ws_bf16", None) is None:
            self.ws_bf16_bytes = lib.moe_workspace_size(lib.MOE_OP_FWD_BF16, self.T, self.k, E, H, I)
            self.ws_bf16 = self._alloc.raw(self.ws_bf16_bytes, "ws_bf16")
        lib.moe_grouped_mlp_fwd_bf16(w1.data_ptr(), w2.data_ptr(), self.T, H, I, E, self.k, self.rows_cap,
                                     _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                                     _ptr(self.slot_to_row), _ptr(self.prob_perm), x.data_ptr(), _ptr(self.out),
                                     _ptr(self.saved_a), _ptr(self.ws_bf16), self.ws_bf16_bytes, self._stream())
        return self.out

    @_on_layer_device
    def backward_bf16(self, dY: torch.Tensor, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor):
        """BF16 recipe backward (moe_grouped_mlp_bwd_bf16) after forward_bf16
        on the same routing: dY, x bf16 [T, H], w1 bf16 [E, 2I, H], w2 bf16
        [E, H, I] -> (dX, dW1, dW2, dprob)."""
        if not self.backward_enabled:
            raise RuntimeError("this layer was built with backward=False")
        E, H, I = self.E, self.H, self.I
        check_tensor(dY, "dY", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(x, "x", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        if getattr(self, "ws_bwd_bf16", None) is None:
            self.ws_bwd_bf16_bytes = lib.moe_workspace_size(lib.MOE_OP_BWD_BF16, self.T, self.k, E, H, I)
            self.ws_bwd_bf16 = self._alloc.raw(self.ws_bwd_bf16_bytes, "ws_bwd_bf16")
        lib.moe_grouped_mlp_bwd_bf16(w1.data_ptr(), w2.data_ptr(), self.T, H, I, E, self.k, self.rows_cap,
                                     _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                                     _ptr(self.slot_to_row), _ptr(self.prob_perm), dY.data_ptr(),
                                     _ptr(self.saved_a), x.data_ptr(), _ptr(self.dX), _ptr(self.dW1),
                                     _ptr(self.dW2), _ptr(self.dprob), _ptr(self.ws_bwd_bf16),
                                     self.ws_bwd_bf16_bytes, self._stream())
        return self.dX, self.dW1, self.dW2, self.dprob

    @_on_layer_device
    def forward_fp8_tensor(self, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor) -> torch.Tensor:
        """Per-tensor FP8 recipe forward (moe_grouped_mlp_fwd_fp8_tensor) on
        the routing of the last permute / permute_index: x bf16 [T, H], w1
        bf16 [E, 2I, H], w2 bf16 [E, H, I] -> out; the factors land in
        self.fp8_scales (x, h, W_gate_up[E], W_down[E])."""
        E, H, I = self.E, self.H, self.I
        check_tensor(x, "x", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        if getattr(self, "ws_f8t", None) is None:
            self.ws_f8t_bytes = lib.moe_workspace_size(lib.MOE_OP_FWD_FP8_TENSOR, self.T, self.k, E, H, I)
            self.ws_f8t = self._alloc.raw(self.ws_f8t_bytes, "ws_f8t")
            self.fp8_scales = self._alloc.typed((2 + 2 * E,), torch.float32, "fp8_scales")
        lib.moe_grouped_mlp_fwd_fp8_tensor(w1.data_ptr(), w2.data_ptr(), self.T, H, I, E, self.k, self.rows_cap,
                                           _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                                           _ptr(self.slot_to_row), _ptr(self.prob_perm), x.data_ptr(),
                                           _ptr(self.out), _ptr(self.saved_a), _ptr(self.fp8_scales),
                                           _ptr(self.ws_f8t), self.ws_f8t_bytes, self._stream())
        return self.out

    @_on_layer_device
    def backward_fp8_tensor(self, dY: torch.Tensor, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor):
        """Per-tensor FP8 recipe backward (moe_grouped_mlp_bwd_fp8_tensor)
        after forward_fp8_tensor on the same routing, x and weights -> (dX,
        dW1, dW2, dprob); the factors of dY, da and h land in
        self.fp8_bwd_scales."""
        if not self.backward_enabled:
            raise RuntimeError("this layer was built with backward=False")
        if getattr(self, "fp8_scales", None) is None:
            raise RuntimeError("backward_fp8_tensor needs forward_fp8_tensor first")
        E, H, I = self.E, self.H, self.I
        check_tensor(dY, "dY", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(x, "x", torch.bfloat16, (self.T, H), self.dev)
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        if getattr(self, "ws_bwd_f8t", None) is None:
            self.ws_bwd_f8t_bytes = lib.moe_workspace_size(lib.MOE_OP_BWD_FP8_TENSOR, self.T, self.k, E, H, I)
            self.ws_bwd_f8t = self._alloc.raw(self.ws_bwd_f8t_bytes, "ws_bwd_f8t")
            self.fp8_bwd_scales = self._alloc.typed((3,), torch.float32, "fp8_bwd_scales")
        lib.moe_grouped_mlp_bwd_fp8_tensor(w1.data_ptr(), w2.data_ptr(), self.T, H, I, E, self.k, self.rows_cap,
                                           _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                                           _ptr(self.slot_to_row), _ptr(self.prob_perm), dY.data_ptr(),
                                           _ptr(self.saved_a), x.data_ptr(), _ptr(self.fp8_scales), _ptr(self.dX),
                                           _ptr(self.dW1), _ptr(self.dW2), _ptr(self.dprob),
                                           _ptr(self.fp8_bwd_scales), _ptr(self.ws_bwd_f8t), self.ws_bwd_f8t_bytes,
                                           self._stream())
        return self.dX, self.dW1, self.dW2, self.dprob

    def route_losses(self, logits: torch.Tensor, token_mask: torch.Tensor = None):
        """Router for training (moe_router_losses): logits fp32 or bf16
        [T, E], token_mask bool [T] (False: padding) -> (topk_idx int32
        [T, k], topk_prob fp32 [T, k], losses fp32 [2] = load-balance loss and
        z-loss), in this layer's buffers; the tokens per expert land in
        self.expert_counts (int32 [E]), the sums of the experts' softmax
        probabilities in self.prob_sums (fp32 [E]), the number of unmasked
        tokens in self.routed_tokens (int32 [1]).  All of it, ids and
        probabilities too, stays until the next route_losses.  For a loss over a
        data-parallel job's whole batch, add the counts and tokens up over the
        ranks before route_backward."""
        T, E, k = self.T, self.E, self.k
        dt = _logits_dtype(logits)
        check_tensor(logits, "logits", logits.dtype, (T, E), self.dev)
        if token_mask is not None:
            check_tensor(token_mask, "token_mask", torch.bool, (T,), self.dev)
        if self.router_lse is None:
            al = self._alloc
            self._loss_idx = al.typed((T, k), torch.int32, "loss_topk_idx")
            self._loss_prob = al.typed((T, k), torch.float32, "loss_topk_prob")
            self.router_lse = al.typed((T,), torch.float32, "router_lse")
            self.expert_counts = al.typed((E,), torch.int32, "expert_counts")
            self.prob_sums = al.typed((E,), torch.float32, "prob_sums")
            self.routed_tokens = al.typed((1,), torch.int32, "routed_tokens")
            self.router_losses = al.typed((2,), torch.float32, "router_losses")
            self.ws_losses_bytes = lib.moe_workspace_size(lib.MOE_OP_ROUTER_LOSSES, T, k, E, 0, 0)
            self.ws_losses = al.raw(self.ws_losses_bytes, "ws_losses")
        with on_device(self.dev):
            lib.moe_router_losses(logits.data_ptr(), dt, T, E, k, _ptr(token_mask), _ptr(self._loss_idx),
                                  _ptr(self._loss_prob), _ptr(self.router_lse), _ptr(self.expert_counts),
                                  _ptr(self.prob_sums), _ptr(self.routed_tokens), _ptr(self.router_losses),
                                  _ptr(self.ws_losses), self.ws_losses_bytes, self._stream())
        self._loss_mask = token_mask
        self.topk_idx, self.topk_prob = self._loss_idx, self._loss_prob
        return self.topk_idx, self.topk_prob, self.router_losses

    def route_backward(self, logits: torch.Tensor, dprob: torch.Tensor = None, dlosses: torch.Tensor = None,
                       token_mask: torch.Tensor = None) -> torch.Tensor:
        """Gradient of the logits (moe_router_bwd) after route_losses on the
        same logits and mask (other routing calls may have come in between;
        token_mask None: the tensor that route_losses was given): dprob fp32
        [T, k] (as backward() returns it) and dlosses fp32 [2], either None for
        zero -> dlogits [T, E] in the logits' type, in a buffer of this layer
        (one per type)."""
        T, E, k = self.T, self.E, self.k
        dt = _logits_dtype(logits)
        check_tensor(logits, "logits", logits.dtype, (T, E), self.dev)
        if self.router_lse is None:
            raise RuntimeError("route_backward needs route_losses first")
        if dprob is not None:
            check_tensor(dprob, "dprob", torch.float32, (T, k), self.dev)
        if dlosses is not None:
            check_tensor(dlosses, "dlosses", torch.float32, (2,), self.dev)
        if token_mask is not None:
            check_tensor(token_mask, "token_mask", torch.bool, (T,), self.dev)
        else:
            token_mask = self._loss_mask
        if logits.dtype not in self.dlogits:
            self.dlogits[logits.dtype] = self._alloc.typed((T, E), logits.dtype, "dlogits")
        dlogits = self.dlogits[logits.dtype]
        with on_device(self.dev):
            lib.moe_router_bwd(logits.data_ptr(), dt, T, E, k, _ptr(token_mask), _ptr(self._loss_idx),
                               _ptr(self._loss_prob), _ptr(self.router_lse), _ptr(self.expert_counts),
                               _ptr(self.routed_tokens), _ptr(dprob), _ptr(dlosses), _ptr(dlogits), self._stream())
        return dlogits

    def _mxfp4_weights(self):
        if self.w1q4 is None:
            u8, E, H, I = self._alloc.raw, self.E, self.H, self.I
            self.w1sf4 = u8(lib.moe_mxfp4_tiled_scale_bytes(E, I, H, 1), "w1sf4")
            self.w2sf4 = u8(lib.moe_mxfp4_tiled_scale_bytes(E, H, I, 0), "w2sf4")
            # rows of codes start on 128-byte lines
            self.ld1_4, self.ld2_4 = (H // 2 + 127) // 128 * 128, (I // 2 + 127) // 128 * 128
            self.w2q4 = u8(E * H * self.ld2_4, "w2q4")
            self.w1q4 = u8(E * 2 * I * self.ld1_4, "w1q4")

    def quantize_weights_mxfp4(self, w1: torch.Tensor, w2: torch.Tensor) -> None:
        """w1 bf16 [E, 2I, H] (gate rows first), w2 bf16 [E, H, I] -> this
        layer's MXFP4 weights."""
        E, H, I = self.E, self.H, self.I
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        self._mxfp4_weights()
        with on_device(self.dev):
            s, bf = self._stream(), lib.MOE_DTYPE_BF16
            for w, matrices, n, k, q, ld, sf, gate_up in ((w1, 2 * E, I, H, self.w1q4, self.ld1_4, self.w1sf4, 1),
                                                          (w2, E, H, I, self.w2q4, self.ld2_4, self.w2sf4, 0)):
                # the quantiser's blocked scales, in row order, in the GEMMs' order
                blocked = torch.empty(lib.moe_mx_scale_bytes(matrices, n, k), dtype=torch.uint8, device=self.dev)
                plain = torch.empty(matrices * n * (k // 32), dtype=torch.uint8, device=self.dev)
                lib.moe_mlp_quantize_mxfp4(w.data_ptr(), bf, matrices, n, k, _ptr(q), ld, _ptr(blocked), s)
                lib.moe_mx_scales_from_blocked(_ptr(blocked), matrices, n, k, _ptr(plain), k // 32, s)
                lib.moe_mxfp4_tile_scales(_ptr(plain), E, n, k, k // 32, gate_up, _ptr(sf), s)

    def load_weights_mxfp4(self, w1_codes: torch.Tensor, w1_scales: torch.Tensor, w2_codes: torch.Tensor,
                           w2_scales: torch.Tensor) -> None:
        """Weights that are in 4 bits already (a checkpoint): uint8 codes
        [E, 2I, H/2] (gate rows first) and [E, H, I/2], the even element in the
        low half of a byte, and uint8 E8M0 scales in row order [E, 2I, H/32]
        and [E, H, I/32].  Codes are copied, scales laid out for the GEMMs."""
        E, H, I = self.E, self.H, self.I
        check_tensor(w1_codes, "w1_codes", torch.uint8, (E, 2 * I, H // 2), self.dev)
        check_tensor(w1_scales, "w1_scales", torch.uint8, (E, 2 * I, H // 32), self.dev)
        check_tensor(w2_codes, "w2_codes", torch.uint8, (E, H, I // 2), self.dev)
        check_tensor(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32), self.dev)
        self._mxfp4_weights()
        with on_device(self.dev):
            self.w1q4[: E * 2 * I * self.ld1_4].view(E, 2 * I, -1)[..., : H // 2].copy_(w1_codes)
            self.w2q4[: E * H * self.ld2_4].view(E, H, -1)[..., : I // 2].copy_(w2_codes)
            s = self._stream()
            lib.moe_mxfp4_tile_scales(_ptr(w1_scales), E, I, H, H // 32, 1, _ptr(self.w1sf4), s)
            lib.moe_mxfp4_tile_scales(_ptr(w2_scales), E, H, I, I // 32, 0, _ptr(self.w2sf4), s)

    def forward_mxfp4(self, x: torch.Tensor) -> torch.Tensor:
        """MXFP4 recipe forward (moe_grouped_mlp_fwd_mxfp4) on the routing of
        the last permute / permute_index and the weights of the last
        quantize_weights_mxfp4 / load_weights_mxfp4: x bf16 [T, H] -> out."""
        E, H, I = self.E, self.H, self.I
        if self.w1q4 is None:
            raise RuntimeError("forward_mxfp4 needs quantize_weights_mxfp4 or load_weights_mxfp4 first")
        check_tensor(x, "x", torch.bfloat16, (self.T, H), self.dev)
        if not self._permuted:
            raise RuntimeError("forward_mxfp4 needs permute_index, permute or route_permute first")
        if getattr(self, "ws_mxfp4", None) is None:
            self.ws_mxfp4_bytes = lib.moe_workspace_size(lib.MOE_OP_FWD_MXFP4, self.T, self.k, E, H, I)
            self.ws_mxfp4 = self._alloc.raw(self.ws_mxfp4_bytes, "ws_mxfp4")
        with on_device(self.dev):
            lib.moe_grouped_mlp_fwd_mxfp4(_ptr(self.w1q4), self.ld1_4, _ptr(self.w1sf4), _ptr(self.w2q4), self.ld2_4,
                                          _ptr(self.w2sf4), self.T, H, I, E, self.k, self.rows_cap,
                                          _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.slot_to_row),
                                          _ptr(self.prob_perm), x.data_ptr(), _ptr(self.out), _ptr(self.ws_mxfp4),
                                          self.ws_mxfp4_bytes, self._stream())
        return self.out

    def check_guards(self):
        """Names of the buffers written past their end (layers built with
        guard > 0; always empty otherwise)."""
        return self._alloc.check()

    def _stream(self) -> int:
        return _raw_stream(self.dev.index)

    @_on_layer_device
    def quantize_weights(self, w1: torch.Tensor, w2: torch.Tensor) -> None:
        """w1 bf16 [E, 2I, H] (gate rows first), w2 bf16 [E, H, I]."""
        self._need_mxfp8()
        E, H, I, s = self.E, self.H, self.I, self._stream()
        check_tensor(w1, "w_gate_up", torch.bfloat16, (E, 2 * I, H), self.dev)
        check_tensor(w2, "w_down", torch.bfloat16, (E, H, I), self.dev)
        if self.backward_enabled:
            # both directions of both weights from one read of each
            lib.moe_mlp_quantize_weights(w1.data_ptr(), w2.data_ptr(), E, H, I, _ptr(self.w1q), _ptr(self.w1sf),
                                         _ptr(self.w2q), _ptr(self.w2sf), _ptr(self.w1tq), _ptr(self.w1tsf),
                                         _ptr(self.w2tq), _ptr(self.w2tsf), s)
            return
        lib.moe_mlp_quantize_mxfp8(w1.data_ptr(), 2 * E, I, H, lib.MOE_QUANT_ROW, _ptr(self.w1q), _ptr(self.w1sf), s)
        lib.moe_mlp_quantize_mxfp8(w2.data_ptr(), E, H, I, lib.MOE_QUANT_ROW, _ptr(self.w2q), _ptr(self.w2sf), s)

    @_on_layer_device
    def route(self, logits: torch.Tensor):
        """Router logits fp32 or bf16 [T, E] -> (topk_idx int32 [T, k],
        topk_prob float32 [T, k]) in this layer's routing buffers."""
        dt = {torch.float32: lib.MOE_DTYPE_F32, torch.bfloat16: lib.MOE_DTYPE_BF16}.get(logits.dtype)
        if dt is None:
            raise TypeError(f"logits: expected float32 or bfloat16, got {logits.dtype}")
        check_tensor(logits, "logits", logits.dtype, (self.T, self.E), self.dev)
        self.topk_idx, self.topk_prob = self._routed
        lib.moe_router_topk(logits.data_ptr(), dt, self.T, self.E, self.k, _ptr(self.topk_idx),
                            _ptr(self.topk_prob), self._stream())
        return self.topk_idx, self.topk_prob

    @_on_layer_device
    def route_permute(self, logits: torch.Tensor, x: torch.Tensor, with_cols: bool = False):
        """Router and permutation in one call (moe_route_permute): logits fp32
        or bf16 [T, E], x bf16 [T, H]; the routing lands in topk_idx /
        topk_prob, the quantised x in this layer's buffers."""
        self._need_mxfp8()
        dt = {torch.float32: lib.MOE_DTYPE_F32, torch.bfloat16: lib.MOE_DTYPE_BF16}.get(logits.dtype)
        if dt is None:
            raise TypeError(f"logits: expected float32 or bfloat16, got {logits.dtype}")
        check_tensor(logits, "logits", logits.dtype, (self.T, self.E), self.dev)
        check_tensor(x, "x", torch.bfloat16, (self.T, self.H), self.dev)
        xc, xcs = self._cols(with_cols)
        self.topk_idx, self.topk_prob = self._routed
        lib.moe_route_permute(logits.data_ptr(), dt, x.data_ptr(), self.T, self.H, self.k, self.E, self.rows_cap,
                              _ptr(self.topk_idx), _ptr(self.topk_prob), _ptr(self.split_sizes),
                              _ptr(self.group_offsets), _ptr(self.row_to_slot), _ptr(self.slot_to_row),
                              _ptr(self.prob_perm), _ptr(self.xq), _ptr(self.xq_sf), xc, xcs, _ptr(self.ws_perm),
                              self.ws_perm_bytes, self._stream())
        self._x, self._permuted = x, True
        return self.topk_idx, self.topk_prob

    @_on_layer_device
    def permute(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_prob: torch.Tensor,
                with_cols: bool = False) -> None:
        """x bf16 [T, H]; topk_idx int32 [T, k]; topk_prob float32 [T, k].
        with_cols also writes x^T quantised along tokens (xq_col), which the
        backward makes for itself from x."""
        self._need_mxfp8()
        check_tensor(x, "x", torch.bfloat16, (self.T, self.H), self.dev)
        check_tensor(topk_idx, "topk_idx", torch.int32, (self.T, self.k), self.dev)
        check_tensor(topk_prob, "topk_prob", torch.float32, (self.T, self.k), self.dev)
        xc, xcs = self._cols(with_cols)
        lib.moe_permute(x.data_ptr(), topk_idx.data_ptr(), topk_prob.data_ptr(), self.T, self.H, self.k,
                        self.E, self.rows_cap, _ptr(self.split_sizes), _ptr(self.group_offsets),
                        _ptr(self.row_to_slot), _ptr(self.slot_to_row), _ptr(self.prob_perm),
                        _ptr(self.xq), _ptr(self.xq_sf), xc, xcs, _ptr(self.ws_perm), self.ws_perm_bytes,
                        self._stream())
        self._x, self._permuted = x, True

    @_on_layer_device
    def forward(self) -> torch.Tensor:
        self._need_mxfp8()
        lib.moe_grouped_mlp_fwd(_ptr(self.w1q), _ptr(self.w1sf), _ptr(self.w2q), _ptr(self.w2sf), self.T,
                                self.H, self.I, self.E, self.k, self.rows_cap, _ptr(self.split_sizes),
                                _ptr(self.group_offsets), _ptr(self.row_to_slot), _ptr(self.slot_to_row),
                                _ptr(self.prob_perm), _ptr(self.xq), _ptr(self.xq_sf), _ptr(self.out),
                                _ptr(self.saved_a),
                                _ptr(self.hq), _ptr(self.hq_sf), _ptr(self.ws_fwd), self.ws_fwd_bytes,
                                self._stream())
        return self.out

    @_on_layer_device
    def backward(self, dY: torch.Tensor, x: torch.Tensor = None):
        """dY bf16 [T, H]; x defaults to the input of the last permutation."""
        self._need_mxfp8()
        if not self.backward_enabled:
            raise RuntimeError("this layer was built with backward=False")
        x = self._x if x is None else x
        if x is None:
            raise RuntimeError("backward needs x: call permute first or pass x")
        check_tensor(dY, "dY", torch.bfloat16, (self.T, self.H), self.dev)
        check_tensor(x, "x", torch.bfloat16, (self.T, self.H), self.dev)
        lib.moe_grouped_mlp_bwd(_ptr(self.w2tq), _ptr(self.w2tsf), _ptr(self.w1tq), _ptr(self.w1tsf),
                                self.T, self.H, self.I, self.E, self.k, self.rows_cap,
                                _ptr(self.split_sizes), _ptr(self.group_offsets), _ptr(self.row_to_slot),
                                _ptr(self.slot_to_row), _ptr(self.prob_perm), dY.data_ptr(),
                                _ptr(self.saved_a), x.data_ptr(),
                                _ptr(self.dX), _ptr(self.dW1), _ptr(self.dW2), _ptr(self.dprob),
                                _ptr(self.ws_bwd), self.ws_bwd_bytes, self._stream())
        return self.dX, self.dW1, self.dW2, self.dprob

    def step(self, x, topk_idx, topk_prob, w1, w2, dY=None):
        """One pass of the whole layer: weight quantisation, permutation,
        forward and (if dY is given) backward."""
        self.quantize_weights(w1, w2)
        self.permute(x, topk_idx, topk_prob)
        out = self.forward()
        if dY is None:
            return out
        return (out,) + tuple(self.backward(dY, x))

    @_on_layer_device
    def device_status(self) -> int:
        return lib.moe_get_device_status(self._stream())
