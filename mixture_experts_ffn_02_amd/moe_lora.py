"""Thin torch-facing binding of the C calls (argument marshalling only): the layer's own and the
operators around it.

PyTorch provides device memory and streams; every step runs in the HIP
kernels of libmoe_lora.so.  Tensors are passed by data pointer: bf16 tensors may be
``torch.bfloat16`` or 16-bit integer views of the same bits.
"""

from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass, field, fields
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import Adapters, Dims, Grouped, MoELoRAError, Options, check, load  # noqa: F401

ROUTING_RENORMALIZE = _lib.ROUTING_RENORMALIZE
ROUTING_DEEPSEEK_V3 = _lib.ROUTING_DEEPSEEK_V3
# moe_lora_options.packed_weights bits
PACKED_GATE_UP = 1
PACKED_DOWN = 2


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE-LoRA library must be contiguous")
    return t.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        # the current stream's handle, without the Stream object (2.7 us of a call's 8)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream
    return int(s)


def dims(num_tokens: int, hidden: int, inter: int, num_experts: int, top_k: int) -> Dims:
    return Dims(num_tokens, hidden, inter, num_experts, top_k)


@dataclass
class LoRASlots:
    """Resident adapter slots (per-slot compact weights, device tensors).

    shared_outer: the shared-outer layout, where a_gate_up[s] is [r, H] and b_down[s] is
    [H, r], one set used by every expert (b_gate_up and a_down stay per expert).
    """

    token_slot: torch.Tensor  # [T] int32
    rank: Sequence[int]
    scaling: Sequence[float]
    a_gate_up: Sequence[torch.Tensor]  # [E, r, H]  (shared-outer: [r, H])
    b_gate_up: Sequence[torch.Tensor]  # [E, 2I, r]
    a_down: Sequence[torch.Tensor]     # [E, r, I]
    b_down: Sequence[torch.Tensor]     # [E, H, r]  (shared-outer: [H, r])
    shared_outer: bool = False

    def to_c(self) -> Adapters:
        n = len(self.rank)
        if n > _lib.MAX_SLOTS:
            raise ValueError("too many adapter slots")
        a = Adapters()
        a.num_slots = n
        a.token_slot = _ptr(self.token_slot)
        a.shared_outer = 1 if self.shared_outer else 0
        for s in range(n):
            a.rank[s] = int(self.rank[s])
            a.scaling[s] = float(self.scaling[s])
            a.a_gate_up[s] = _ptr(self.a_gate_up[s])
            a.b_gate_up[s] = _ptr(self.b_gate_up[s])
            a.a_down[s] = _ptr(self.a_down[s])
            a.b_down[s] = _ptr(self.b_down[s])
        return a


def moe_lora_route_workspace_size(d: Dims) -> int:
    return int(load().moe_lora_route_workspace_size(ctypes.byref(d)))


def moe_lora_forward_workspace_size(d: Dims, lora: Optional[Adapters]) -> int:
    return int(load().moe_lora_forward_workspace_size(ctypes.byref(d),
                                                       ctypes.byref(lora) if lora else None))


def moe_lora_route(d: Dims, logits, topk_ids, topk_weights, expert_offsets, e2p, p2e, ws,
                   routing: int = ROUTING_RENORMALIZE, grouped: Optional[Grouped] = None,
                   stream=None) -> None:
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    check("moe_lora_route", load().moe_lora_route(
        ctypes.byref(d), int(routing), ctypes.byref(grouped) if grouped is not None else None,
        _ptr(logits), _ptr(topk_ids), _ptr(topk_weights), _ptr(expert_offsets), _ptr(e2p),
        _ptr(p2e), _ptr(ws), ws_bytes, _stream(stream)))


def moe_lora_permute(d: Dims, x, p2e, x_perm, stream=None) -> None:
    check("moe_lora_permute", load().moe_lora_permute(
        ctypes.byref(d), _ptr(x), _ptr(p2e), _ptr(x_perm), _stream(stream)))


def moe_lora_forward(d: Dims, x, x_perm, expert_offsets, p2e, w_gate_up, w_down,
                     lora: Optional[Adapters], y_perm, ws, main=None, side=None,
                     opts: Optional[Options] = None) -> None:
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    check("moe_lora_forward", load().moe_lora_forward(
        ctypes.byref(d), _ptr(x), _ptr(x_perm), _ptr(expert_offsets), _ptr(p2e), _ptr(w_gate_up),
        _ptr(w_down), ctypes.byref(lora) if lora is not None else None, _ptr(y_perm), _ptr(ws),
        ws_bytes, _stream(main), None if side is None else _stream(side),
        ctypes.byref(opts) if opts is not None else None))


def moe_lora_forward_noalloc(d: Dims, x, x_perm, expert_offsets, p2e, w_gate_up, w_down,
                             lora: Optional[Adapters], y_perm, main=None,
                             opts: Optional[Options] = None) -> None:
    check("moe_lora_forward_noalloc", load().moe_lora_forward_noalloc(
        ctypes.byref(d), _ptr(x), _ptr(x_perm), _ptr(expert_offsets), _ptr(p2e), _ptr(w_gate_up),
        _ptr(w_down), ctypes.byref(lora) if lora is not None else None, _ptr(y_perm), _stream(main),
        ctypes.byref(opts) if opts is not None else None))


def moe_lora_forward_fp8(d: Dims, x, x_perm, expert_offsets, p2e, w_gate_up, w_gate_up_scale, w_down,
                         w_down_scale, lora: Optional[Adapters], y_perm, ws, main=None, side=None,
                         opts: Optional[Options] = None) -> None:
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    check("moe_lora_forward_fp8", load().moe_lora_forward_fp8(
        ctypes.byref(d), _ptr(x), _ptr(x_perm), _ptr(expert_offsets), _ptr(p2e), _ptr(w_gate_up),
        _ptr(w_gate_up_scale), _ptr(w_down), _ptr(w_down_scale),
        ctypes.byref(lora) if lora is not None else None, _ptr(y_perm), _ptr(ws), ws_bytes,
        _stream(main), None if side is None else _stream(side),
        ctypes.byref(opts) if opts is not None else None))


def moe_lora_pack_weights(d: Dims, w_gate_up, w_down, w_gate_up_packed, w_down_packed,
                          stream=None) -> None:
    check("moe_lora_pack_weights", load().moe_lora_pack_weights(
        ctypes.byref(d), _ptr(w_gate_up), _ptr(w_down), _ptr(w_gate_up_packed), _ptr(w_down_packed),
        _stream(stream)))


def moe_lora_pack_weights_fp8(d: Dims, w_gate_up, w_down, w_gate_up_packed, w_down_packed,
                              stream=None) -> None:
    check("moe_lora_pack_weights_fp8", load().moe_lora_pack_weights_fp8(
        ctypes.byref(d), _ptr(w_gate_up), _ptr(w_down), _ptr(w_gate_up_packed), _ptr(w_down_packed),
        _stream(stream)))


def moe_lora_finalize(d: Dims, y_perm, topk_weights, e2p, out, stream=None) -> None:
    check("moe_lora_finalize", load().moe_lora_finalize(
        ctypes.byref(d), _ptr(y_perm), _ptr(topk_weights), _ptr(e2p), _ptr(out), _stream(stream)))


# ---- operators around the expert layer.  These check every tensor (device, type, shape,
# contiguity) before the call, and launch on the tensors' device.

def _on(first, *tensors) -> int:
    """Index of the one GPU that all these tensors are on (the first one is not None)."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"a GPU tensor is needed, got one on {first.device}")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors of one call are on {first.device} and {t.device}")
    return dev


def _checked(name: str, t: torch.Tensor, dtype, numel: int) -> int:
    """Data pointer of a contiguous tensor of this type and size."""
    if t.dtype is not dtype and not (dtype is torch.bfloat16 and t.dtype in (torch.int16, torch.uint16)):
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name}: {numel} elements expected, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed")
    return t.data_ptr()


def _workspace(ws: Optional[torch.Tensor]):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor is needed")
    return ws.data_ptr(), ws.nbytes


def _call(fn: str, dev, stream, *args) -> None:
    """The library call with the tensors' device current (its kernels launch there), on the
    given stream or that device's current one."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = getattr(load(), fn)(*args, _stream(stream))
    else:
        status = getattr(load(), fn)(*args, _stream(stream))
    if status != _lib.OK:
        check(fn, status)


@dataclass
class Scoring:
    """How moe_lora_route_scored scores, groups and weights the experts.

    score: "softmax" or "sigmoid"; bias: [E] fp32, added to the scores for the choice only;
    group_score: how many of a group's best experts make its score (1 or 2).
    """

    score: str = "softmax"
    renormalize: bool = True
    n_group: int = 1
    topk_group: int = 1
    group_score: int = 1
    scale: float = 1.0
    bias: Optional[torch.Tensor] = None

    def __eq__(self, other):
        """The same method with the same bias tensor (whose values are not compared)."""
        if not isinstance(other, Scoring):
            return NotImplemented
        return all(getattr(self, f.name) == getattr(other, f.name) for f in fields(self) if f.name != "bias") and \
            self.bias is other.bias

    def to_c(self, logits_dtype: torch.dtype, num_experts: int) -> _lib.ScoringC:
        if self.score not in ("softmax", "sigmoid"):
            raise ValueError(f"score: 'softmax' or 'sigmoid', got {self.score!r}")
        f32 = logits_dtype is torch.float32
        if not f32 and logits_dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise ValueError(f"logits are bf16 or fp32, got {logits_dtype}")
        return _lib.ScoringC(
            _lib.SCORE_SIGMOID if self.score == "sigmoid" else _lib.SCORE_SOFTMAX,
            _lib.DTYPE_F32 if f32 else _lib.DTYPE_BF16, int(bool(self.renormalize)), self.n_group,
            self.topk_group, self.group_score, self.scale,
            None if self.bias is None else _checked("bias", self.bias, torch.float32, num_experts))


def moe_lora_route_scored_workspace_size(d: Dims, scoring: Scoring, logits_dtype=torch.bfloat16) -> int:
    return int(load().moe_lora_route_scored_workspace_size(
        ctypes.byref(d), ctypes.byref(scoring.to_c(logits_dtype, d.num_experts))))


def moe_lora_route_scored(d: Dims, scoring: Scoring, logits, topk_ids, topk_weights, expert_offsets, e2p, p2e,
                          ws, stream=None) -> None:
    T, E, R = d.num_tokens, d.num_experts, d.num_tokens * d.top_k
    sc = scoring.to_c(logits.dtype, E)
    i32 = torch.int32
    _call("moe_lora_route_scored",
          _on(logits, topk_ids, topk_weights, expert_offsets, e2p, p2e, ws, scoring.bias), stream,
          ctypes.byref(d), ctypes.byref(sc), _checked("logits", logits, logits.dtype, T * E),
          _checked("topk_ids", topk_ids, i32, R), _checked("topk_weights", topk_weights, torch.float32, R),
          _checked("expert_offsets", expert_offsets, i32, E + 1), _checked("e2p", e2p, i32, R),
          _checked("p2e", p2e, i32, R), *_workspace(ws))


def moe_lora_route_scored_backward(d: Dims, scoring: Scoring, logits, topk_ids, d_weights, d_logits,
                                   stream=None) -> None:
    T, E, R = d.num_tokens, d.num_experts, d.num_tokens * d.top_k
    sc = scoring.to_c(logits.dtype, E)
    _call("moe_lora_route_scored_backward", _on(logits, topk_ids, d_weights, d_logits), stream,
          ctypes.byref(d), ctypes.byref(sc), _checked("logits", logits, logits.dtype, T * E),
          _checked("topk_ids", topk_ids, torch.int32, R), _checked("d_weights", d_weights, torch.float32, R),
          _checked("d_logits", d_logits, logits.dtype, T * E))


def _rows_cols(name: str, t: torch.Tensor):
    if t.dim() != 2:
        raise ValueError(f"{name}: a matrix is needed, got shape {tuple(t.shape)}")
    return t.shape


def _int32(what: str, *values: int) -> None:
    """Refuses what a 32-bit field of the library's structs would cut off."""
    if max(values) > 0x7FFFFFFF:
        raise ValueError(f"{what}: {max(values)} does not fit 32 bits")


def checkpoint_exps_shape(rows: int, cols: int):
    """Shape of the exponent bytes of a [rows, cols] checkpoint."""
    return rows, (cols + 31) // 32


def moe_lora_checkpoint_pack(x, codes, exps, stream=None) -> None:
    """x [rows, cols] bf16 -> codes [rows, cols] and exps [rows, ceil(cols / 32)], uint8."""
    M, H = _rows_cols("x", x)
    _int32("columns of x", H)
    _call("moe_lora_checkpoint_pack", _on(x, codes, exps), stream, M, H,
          _checked("x", x, torch.bfloat16, M * H), _checked("codes", codes, torch.uint8, M * H),
          _checked("exps", exps, torch.uint8, M * ((H + 31) // 32)))


def moe_lora_checkpoint_unpack(codes, exps, x, stream=None) -> None:
    M, H = _rows_cols("codes", codes)
    _int32("columns of codes", H)
    _call("moe_lora_checkpoint_unpack", _on(codes, exps, x), stream, M, H,
          _checked("codes", codes, torch.uint8, M * H), _checked("exps", exps, torch.uint8, M * ((H + 31) // 32)),
          _checked("x", x, torch.bfloat16, M * H))


def moe_lora_finalize_backward(d: Dims, d_out, topk_weights, e2p, d_y_perm, d_weights, y_perm=None, y_codes=None,
                               y_exps=None, stream=None) -> None:
    """y_perm in bf16, or its checkpoint (y_codes, y_exps)."""
    T, H, R = d.num_tokens, d.hidden, d.num_tokens * d.top_k
    _call("moe_lora_finalize_backward",
          _on(d_out, topk_weights, e2p, d_y_perm, d_weights, y_perm, y_codes, y_exps), stream, ctypes.byref(d),
          _checked("d_out", d_out, torch.bfloat16, T * H),
          None if y_perm is None else _checked("y_perm", y_perm, torch.bfloat16, R * H),
          None if y_codes is None else _checked("y_codes", y_codes, torch.uint8, R * H),
          None if y_exps is None else _checked("y_exps", y_exps, torch.uint8, R * ((H + 31) // 32)),
          _checked("topk_weights", topk_weights, torch.float32, R), _checked("e2p", e2p, torch.int32, R),
          _checked("d_y_perm", d_y_perm, torch.bfloat16, R * H),
          _checked("d_weights", d_weights, torch.float32, R))


@dataclass(frozen=True, eq=False)  # (a pool equals itself: comparing tensors gives no truth value)
class AdapterPool:
    """Resident adapters of a projection (device tensors): a [S, R, in] and b [S, out, R] bf16,
    rank [S] int32 and scaling [S] fp32; token_slot [T] int32 names each token's adapter
    (outside [0, S): none).

    Checked when it is made and then fixed (the tensors' contents may change; with_slots gives
    the same adapters for another batch).  A tensor that was moved to other memory since
    (resized, or given other data) is refused.
    """

    token_slot: torch.Tensor
    rank: torch.Tensor
    scaling: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    _c: _lib.Pool = field(init=False, repr=False, compare=False)
    _shape: tuple = field(init=False, repr=False, compare=False)
    _at: tuple = field(init=False, repr=False, compare=False)
    _device: int = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if self.a.dim() != 3 or self.b.dim() != 3:
            raise ValueError("a is [S, R, in] and b [S, out, R]")
        (S, R, K), N, T = self.a.shape, self.b.shape[1], self.token_slot.numel()
        if self.b.shape != (S, N, R):
            raise ValueError(f"b: [{S}, out, {R}] expected, got shape {tuple(self.b.shape)}")
        bf16 = torch.bfloat16
        _int32("sizes of the pool", S, R)
        object.__setattr__(self, "_c", _lib.Pool(
            S, R, _checked("token_slot", self.token_slot, torch.int32, T),
            _checked("rank", self.rank, torch.int32, S), _checked("scaling", self.scaling, torch.float32, S),
            _checked("a", self.a, bf16, S * R * K), _checked("b", self.b, bf16, S * N * R)))
        object.__setattr__(self, "_shape", (T, K, N))
        object.__setattr__(self, "_at", self._addresses())
        devices = {t.get_device() for t in (self.token_slot, self.rank, self.scaling, self.a, self.b)}
        if len(devices) != 1:
            raise ValueError("the tensors of a pool are on different devices")
        object.__setattr__(self, "_device", devices.pop())

    def _addresses(self):
        return (self.token_slot.data_ptr(), self.rank.data_ptr(), self.scaling.data_ptr(), self.a.data_ptr(),
                self.b.data_ptr())

    def on(self, dev: int) -> int:
        """dev, which has to be the pool's device."""
        if dev != self._device:
            raise ValueError(f"the pool is not on the call's device, cuda:{dev}")
        return dev

    def with_slots(self, token_slot: torch.Tensor) -> "AdapterPool":
        return AdapterPool(token_slot, self.rank, self.scaling, self.a, self.b)

    def to_c(self, T: int, K: int, N: int) -> _lib.Pool:
        if self._shape != (T, K, N):
            raise ValueError(f"the pool is for {self._shape[0]} tokens and a projection of {self._shape[1]} to "
                             f"{self._shape[2]}, the call for {T}, {K} and {N}")
        if self._at != self._addresses():
            raise ValueError("a tensor of the pool was moved to other memory: make a new pool")
        return self._c


def _matrix(name: str, t: torch.Tensor, rows: int, cols: int):
    """Pointer and row pitch of a bf16 matrix [rows, cols] whose rows may lie apart."""
    if t.dtype is not torch.bfloat16 and t.dtype not in (torch.int16, torch.uint16):
        raise ValueError(f"{name}: torch.bfloat16 expected, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: [{rows}, {cols}] expected, got shape {tuple(t.shape)}")
    if rows == 0:
        return t.data_ptr(), cols
    pitch, unit = t.stride()
    if unit != 1 or (rows > 1 and pitch < cols):
        raise ValueError(f"{name}: rows must have unit stride and not overlap")
    return t.data_ptr(), pitch if rows > 1 else cols


def _proj_dims(T: int, K: int, N: int, ldx: int, ldy: int) -> _lib.ProjDims:
    _int32("tokens, features, or elements that rows are apart", T, K, N, ldx, ldy)
    return _lib.ProjDims(T, K, N, ldx, ldy)


def moe_lora_project_workspace_size(T: int, K: int, N: int, pool: AdapterPool) -> int:
    return int(load().moe_lora_project_workspace_size(ctypes.byref(_proj_dims(T, K, N, K, N)),
                                                      ctypes.byref(pool.to_c(T, K, N))))


def moe_lora_project(x, w, pool: AdapterPool, y, ws, v=None, stream=None) -> None:
    """y = x W^T + scaling * (x A^T) B^T with each token's adapter; v [T, R] fp32 keeps x A^T.
    x and y may be column slices of wider matrices."""
    T, K = _rows_cols("x", x)
    N = w.shape[0]
    p = pool.to_c(T, K, N)
    px, ldx = _matrix("x", x, T, K)
    py, ldy = _matrix("y", y, T, N)
    _call("moe_lora_project", pool.on(_on(x, w, y, ws, v)), stream,
          ctypes.byref(_proj_dims(T, K, N, ldx, ldy)), px, _checked("w", w, torch.bfloat16, N * K),
          ctypes.byref(p), py, None if v is None else _checked("v", v, torch.float32, T * p.max_rank),
          *_workspace(ws))


def moe_lora_project_backward_workspace_size(T: int, K: int, N: int, pool: AdapterPool) -> int:
    return int(load().moe_lora_project_backward_workspace_size(ctypes.byref(_proj_dims(T, K, N, K, N)),
                                                               ctypes.byref(pool.to_c(T, K, N))))


def moe_lora_project_backward(dy, w, pool: AdapterPool, v, ws, x=None, x_codes=None, x_exps=None, dx=None, da=None,
                              db=None, stream=None) -> None:
    """Gradients of moe_lora_project: dx [T, in], da [S, R, in], db [S, out, R] (None: not
    wanted).  The input is x in bf16 or its checkpoint (x_codes, x_exps); v the forward's."""
    T, N = _rows_cols("dy", dy)
    K = w.shape[1]
    p = pool.to_c(T, K, N)
    S, R = p.num_slots, p.max_rank
    bf16, u8 = torch.bfloat16, torch.uint8
    px, ldx = (None, K) if x is None else _matrix("x", x, T, K)
    pdy, ldy = _matrix("dy", dy, T, N)
    _call("moe_lora_project_backward",
          pool.on(_on(dy, w, v, ws, x, x_codes, x_exps, dx, da, db)), stream,
          ctypes.byref(_proj_dims(T, K, N, ldx, ldy)), px,
          None if x_codes is None else _checked("x_codes", x_codes, u8, T * K),
          None if x_exps is None else _checked("x_exps", x_exps, u8, T * ((K + 31) // 32)),
          _checked("w", w, bf16, N * K), ctypes.byref(p),
          None if v is None else _checked("v", v, torch.float32, T * R), pdy,
          None if dx is None else _checked("dx", dx, bf16, T * K),
          None if da is None else _checked("da", da, bf16, S * R * K),
          None if db is None else _checked("db", db, bf16, S * N * R),
          *_workspace(ws))


def _device_of(t: torch.Tensor):
    """A context in which t's device is the current one."""
    dev = t.get_device()
    return nullcontext() if dev < 0 or dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


@dataclass
class RouteOut:
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    expert_offsets: torch.Tensor
    e2p: torch.Tensor
    p2e: torch.Tensor


class MoELoRALayer:
    """The routed MoE-LoRA layer on one GPU: route -> permute -> forward -> finalize.

    Buffers (routing outputs, workspaces, intermediates) are allocated once per token
    count and reused, so repeated calls at one shape allocate nothing.  packed_weights
    (PACKED_GATE_UP | PACKED_DOWN bits; True = both) makes the layer keep tile-packed
    copies of those expert weights (written once by moe_lora_pack_weights) and run the
    GEMMs on them; weights_prepacked gives the bits of the weights that are passed in
    already packed.  With w_gate_up_scale / w_down_scale the expert weights are FP8: uint8
    E4M3 codes [E, 2I, H] / [E, H, I] with fp32 scales per 128 x 128 block, run through
    moe_lora_forward_fp8 (packed_weights / weights_prepacked then refer to the FP8
    tile-packed layout of moe_lora_pack_weights_fp8).  routing: one of the ROUTING_ methods,
    or a Scoring (moe_lora_route_scored; logits bf16 or fp32).
    """

    def __init__(self, hidden: int, inter: int, num_experts: int, top_k: int,
                 w_gate_up: torch.Tensor, w_down: torch.Tensor,
                 routing=ROUTING_RENORMALIZE, n_group: int = 1, topk_group: int = 1,
                 routed_scaling_factor: float = 1.0, correction_bias: Optional[torch.Tensor] = None,
                 gather_on_load: bool = True, packed_weights=0, weights_prepacked=0,
                 w_gate_up_scale: Optional[torch.Tensor] = None, w_down_scale: Optional[torch.Tensor] = None,
                 fp8_pow2_scales: bool = False):
        load()
        self.w_scales = None
        if (w_gate_up_scale is None) != (w_down_scale is None):
            raise ValueError("FP8 weights need both block-scale tensors")
        if w_gate_up_scale is not None:
            self.w_scales = (w_gate_up_scale, w_down_scale)
        self.fp8_pow2_scales = bool(fp8_pow2_scales) and self.w_scales is not None
        self.H, self.I, self.E, self.k = hidden, inter, num_experts, top_k
        both = PACKED_GATE_UP | PACKED_DOWN
        to_pack = both if packed_weights is True else int(packed_weights)
        pre = both if weights_prepacked is True else int(weights_prepacked)
        if (to_pack | pre) & ~both:
            raise ValueError("packed_weights / weights_prepacked take PACKED_GATE_UP | PACKED_DOWN bits")
        to_pack &= ~pre
        if to_pack:
            w1p = torch.empty_like(w_gate_up) if to_pack & PACKED_GATE_UP else None
            w2p = torch.empty_like(w_down) if to_pack & PACKED_DOWN else None
            pack = moe_lora_pack_weights_fp8 if self.w_scales is not None else moe_lora_pack_weights
            with _device_of(w_gate_up):
                pack(self.dims(0), w_gate_up if w1p is not None else None, w_down if w2p is not None else None,
                     w1p, w2p)
            w_gate_up = w1p if w1p is not None else w_gate_up
            w_down = w2p if w2p is not None else w_down
        self.packed_weights = to_pack | pre
        self.w_gate_up, self.w_down = w_gate_up, w_down
        if isinstance(routing, Scoring) and (correction_bias is not None or
                                             (n_group, topk_group, routed_scaling_factor) != (1, 1, 1.0)):
            raise ValueError("a Scoring holds its own groups, scale and bias")
        self.routing = routing
        self.correction_bias = correction_bias
        self.grouped = None
        if routing == ROUTING_DEEPSEEK_V3:
            self.grouped = Grouped(n_group, topk_group, routed_scaling_factor,
                                   _ptr(correction_bias) if correction_bias is not None else None)
        self.gather_on_load = gather_on_load
        self._bufs = {}
        self._used = {}  # (tokens, ranks) -> the buffers of the last call with them

    def dims(self, T: int) -> Dims:
        return Dims(T, self.H, self.I, self.E, self.k)

    def _route_form(self):
        """What the routing workspace depends on beside the batch (a Scoring may change between calls)."""
        r = self.routing
        return (r.bias is not None, r.n_group > 1, r.group_score) if isinstance(r, Scoring) else None

    def _route_workspace(self, d: Dims) -> int:
        if isinstance(self.routing, Scoring):
            return moe_lora_route_scored_workspace_size(d, self.routing)
        return moe_lora_route_workspace_size(d)

    def _buffers(self, T: int, lora: Optional[Adapters], device) -> dict:
        key = (T, None if lora is None else tuple(lora.rank[: lora.num_slots]), self._route_form())
        b = self._bufs.get(key)
        if b is None:
            d = self.dims(T)
            R = T * self.k
            i32 = dict(dtype=torch.int32, device=device)
            b = {
                "ids": torch.empty((T, self.k), **i32),
                "w": torch.empty((T, self.k), dtype=torch.float32, device=device),
                "off": torch.empty((self.E + 1,), **i32),
                "e2p": torch.empty((R,), **i32),
                "p2e": torch.empty((R,), **i32),
                # per-workgroup expert histograms of the two-launch routing (written before read)
                "rws": torch.empty((max(1, self._route_workspace(d)),), dtype=torch.uint8, device=device),
                "fws": torch.empty((max(1, moe_lora_forward_workspace_size(d, lora)),),
                                   dtype=torch.uint8, device=device),
                "x_perm": None if self.gather_on_load else torch.empty((R, self.H), dtype=torch.bfloat16,
                                                                       device=device),
                "y": torch.empty((R, self.H), dtype=torch.bfloat16, device=device),
                "out": torch.empty((T, self.H), dtype=torch.bfloat16, device=device),
            }
            self._bufs[key] = b
        self._used[key[:2]] = b
        return b

    def _last(self, T: int, lora: Optional[LoRASlots]) -> dict:
        b = self._used.get((T, None if lora is None else tuple(lora.to_c().rank[: len(lora.rank)])))
        if b is None:
            raise ValueError(f"the layer has not run a batch of {T} tokens with these adapters")
        return b

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, lora: Optional[LoRASlots] = None,
                 side_stream=None, opts: Optional[Options] = None, stream=None) -> torch.Tensor:
        with _device_of(x):  # every launch of the call on x's device, and on its stream where none is given
            return self._run(x, logits, lora, side_stream, opts, stream)

    def _run(self, x, logits, lora, side_stream, opts, stream) -> torch.Tensor:
        T = x.shape[0]
        c_lora = lora.to_c() if lora is not None else None
        b = self._buffers(T, c_lora, x.device)
        d = self.dims(T)
        if isinstance(self.routing, Scoring):
            moe_lora_route_scored(d, self.routing, logits, b["ids"], b["w"], b["off"], b["e2p"], b["p2e"],
                                  b["rws"], stream)
        else:
            moe_lora_route(d, logits, b["ids"], b["w"], b["off"], b["e2p"], b["p2e"], b["rws"],
                           self.routing, self.grouped, stream)
        if not self.gather_on_load:
            moe_lora_permute(d, x, b["p2e"], b["x_perm"], stream)
        if self.packed_weights or self.fp8_pow2_scales:
            o = Options()
            if opts is not None:
                ctypes.memmove(ctypes.byref(o), ctypes.byref(opts), ctypes.sizeof(Options))
            o.packed_weights = self.packed_weights
            o.fp8_pow2_scales = int(self.fp8_pow2_scales)
            opts = o
        if self.w_scales is not None:
            moe_lora_forward_fp8(d, x, b["x_perm"], b["off"], b["p2e"], self.w_gate_up, self.w_scales[0],
                                 self.w_down, self.w_scales[1], c_lora, b["y"], b["fws"], stream,
                                 side_stream, opts)
        else:
            moe_lora_forward(d, x, b["x_perm"], b["off"], b["p2e"], self.w_gate_up, self.w_down,
                             c_lora, b["y"], b["fws"], stream, side_stream, opts)
        moe_lora_finalize(d, b["y"], b["w"], b["e2p"], b["out"], stream)
        return b["out"]

    def last_route(self, T: int, lora: Optional[LoRASlots] = None) -> RouteOut:
        """Routing outputs of the last call with T tokens and these adapters' ranks."""
        b = self._last(T, lora)
        return RouteOut(b["ids"], b["w"], b["off"], b["e2p"], b["p2e"])

    def last_rows(self, T: int, lora: Optional[LoRASlots] = None) -> torch.Tensor:
        """The routed rows [T * k, H] that the last such call summed (moe_lora_finalize_backward
        takes them).  The layer's own buffer: the next call of that size writes it again."""
        return self._last(T, lora)["y"]
