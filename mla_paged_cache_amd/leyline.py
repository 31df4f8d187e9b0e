"""Python binding of libleyline.so (include/leyline.h, include/leyline_step.h,
include/leyline_weight.h, include/leyline_train.h): argument marshalling only.

Every step of the splice / evict path runs in the library's HIP kernels and
C++ host planner; this module turns torch tensors into device pointers and
the current torch stream into a hipStream_t, and turns status codes into
exceptions.  If the library is missing, importing this module fails loudly.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libleyline.so")

LL_OK, LL_EINVAL, LL_ERANGE, LL_ENOMEM, LL_EUNSUPPORTED, LL_EDEVICE, LL_EPOISONED = 0, -1, -2, -3, -4, -5, -6
AMORTIZE, FORGET, PIN, DECAY, SCRATCH = 0, 1, 2, 3, 4
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
SPLICE_PLAN_AUTO, SPLICE_PLAN_HOST = 0, 1
KV_LORA_RANK, ROPE_DIM = 512, 64
ROW = KV_LORA_RANK + ROPE_DIM

# Every symbol include/leyline.h declares.
EXPORTS = (
    "ll_pool_create", "ll_pool_destroy", "ll_seq_alloc", "ll_seq_set_pages", "ll_seq_free",
    "ll_seq_get", "ll_pool_free_pages", "leyline_splice", "kv_evict_compact", "ll_ptable_reindex",
    "ll_rope_delta_table", "ll_last_plan_stats", "ll_pool_set_profiling", "ll_profile_read",
    "ll_last_error", "ll_status_str", "ll_pool_create_gqa",
    "kvs_ctx_create", "kvs_ctx_destroy", "kvs_death_times", "kvs_block_mask", "kvs_dense_mask",
    "ll_rope_rows", "ll_pool_set_splice_planner", "ll_pool_set_page_reuse", "ll_last_plan_bytes", "ll_seq_lengths",
    "leyline_splice_noalloc", "ll_pool_set_dispatch_limit",
)


# Every symbol include/leyline_step.h declares.
STEP_EXPORTS = ("ll_step_create", "ll_step_destroy", "ll_step_begin", "ll_step_append", "ll_step_attend")

# Every symbol include/leyline_weight.h and include/leyline_train.h declare.
WEIGHT_EXPORTS = ("ll_step_attend_capped", "ll_step_weigh", "ll_keep_heaviest")
TRAIN_EXPORTS = ("kvs_attend_workspace", "kvs_attend", "kvs_attend_backward")


class LeylineError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class _PoolDesc(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_seqs", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("kv_lora_rank", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("rope_pairing", ctypes.c_int32),
        ("rope_base", ctypes.c_double),
        ("layer_base", ctypes.POINTER(ctypes.c_void_p)),
        ("page_table", ctypes.c_void_p),
        ("device", ctypes.c_int32),
    ]


class _GqaPoolDesc(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_seqs", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rope_pairing", ctypes.c_int32),
        ("rope_base", ctypes.c_double),
        ("k_layer_base", ctypes.POINTER(ctypes.c_void_p)),
        ("v_layer_base", ctypes.POINTER(ctypes.c_void_p)),
        ("page_table", ctypes.c_void_p),
        ("device", ctypes.c_int32),
    ]


class _Directive(ctypes.Structure):
    _fields_ = [
        ("seq_id", ctypes.c_int32),
        ("mode", ctypes.c_int32),
        ("s_start", ctypes.c_int64),
        ("s_end", ctypes.c_int64),
        ("r_len", ctypes.c_int64),
        ("r_rows", ctypes.c_void_p),
        ("r_layer_stride_bytes", ctypes.c_int64),
        ("r_rows_v", ctypes.c_void_p),
        ("r_layer_stride_bytes_v", ctypes.c_int64),
    ]


class _KvsRolloutLog(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64),
        ("n_events", ctypes.c_int32),
        ("event_time", ctypes.POINTER(ctypes.c_int64)),
        ("mask_len", ctypes.POINTER(ctypes.c_int64)),
        ("mask_offset", ctypes.c_int64),
    ]


class _PlanStats(ctypes.Structure):
    _fields_ = [
        ("alg_bytes", ctypes.c_int64),
        ("rows_moved", ctypes.c_int64),
        ("rows_rotated_inplace", ctypes.c_int64),
        ("fresh_pages", ctypes.c_int64),
        ("freed_pages", ctypes.c_int64),
        ("table_entries", ctypes.c_int64),
        ("planned_on_device", ctypes.c_int64),
    ]


class _StepDesc(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("max_seqs", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
    ]


# ll_append_desc and ll_attend_desc, packed in their C layout
_APPEND_DESC = struct.Struct("@qii Pqq Pqq P Pqq Pqq P f4x")
_ATTEND_DESC = struct.Struct("@qiiq f4x Pqq Pqq Pqq P")
# ll_weigh_desc, kvs_attend_desc and what kvs_attend_backward_desc has behind it
_WEIGH_DESC = struct.Struct("@qiiq ff Pqq Pqq P P q f4x")
_TRAIN_DESC = struct.Struct("@iiq iiiff4x P Pqqq Pqqq Pqqq Pqqq P Pq")
_TRAIN_GRADS = struct.Struct("@Pqqq Pqqq Pqqq Pqqq")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with mla_paged_cache_amd._build.build() "
                          "(the splice path has no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, vp = ctypes.POINTER, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "ll_pool_create": (i32, [P(_PoolDesc), P(vp)]),
        "ll_pool_create_gqa": (i32, [P(_GqaPoolDesc), P(vp)]),
        "ll_pool_destroy": (None, [vp]),
        "ll_seq_alloc": (i32, [vp, i64, P(i32), vp]),
        "ll_seq_set_pages": (i32, [vp, i32, vp, i64, vp]),
        "ll_seq_free": (i32, [vp, i32]),
        "ll_seq_get": (i32, [vp, i32, P(i64), P(i64), P(i32), i32, P(i32)]),
        "ll_pool_free_pages": (i32, [vp, P(i64)]),
        "leyline_splice": (i32, [vp, P(_Directive), i32, vp]),
        "leyline_splice_noalloc": (i32, [vp, P(_Directive), i32, vp]),
        "kv_evict_compact": (i32, [vp, vp, i32, vp, vp, vp]),
        "ll_ptable_reindex": (i32, [vp, i32, vp, i32, vp]),
        "ll_rope_delta_table": (i32, [ctypes.c_double, i32, i64, P(ctypes.c_float), P(ctypes.c_float)]),
        "ll_last_plan_stats": (i32, [vp, P(_PlanStats)]),
        "ll_last_plan_bytes": (i32, [vp, P(i64), P(i64), P(i64)]),
        "ll_seq_lengths": (i32, [vp, vp, i32, vp]),
        "ll_pool_set_profiling": (i32, [vp, i32]),
        "ll_pool_set_splice_planner": (i32, [vp, i32]),
        "ll_pool_set_page_reuse": (i32, [vp, i32]),
        "ll_pool_set_dispatch_limit": (i32, [vp, i64]),
        "ll_profile_read": (i32, [vp, i32, P(i64), P(ctypes.c_double), P(i64), P(ctypes.c_float), i64]),
        "ll_rope_rows": (i32, [vp, i32, i64, i64, vp, vp, i64, vp]),
        "kvs_ctx_create": (i32, [i32, P(vp)]),
        "kvs_ctx_destroy": (None, [vp]),
        "kvs_death_times": (i32, [vp, P(_KvsRolloutLog), i32, i64, vp, vp, vp, vp]),
        "kvs_block_mask": (i32, [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp]),
        "kvs_dense_mask": (i32, [vp, vp, i32, i64, vp, vp]),
        "ll_step_create": (i32, [vp, P(_StepDesc), P(vp)]),
        "ll_step_destroy": (None, [vp]),
        "ll_step_begin": (i32, [vp, vp, vp, i32, i32, vp]),
        "ll_step_append": (i32, [vp, vp, vp]),
        "ll_step_attend": (i32, [vp, vp, vp]),
        "ll_step_attend_capped": (i32, [vp, vp, ctypes.c_float, vp]),
        "ll_step_weigh": (i32, [vp, vp, vp]),
        "ll_keep_heaviest": (i32, [vp, vp, i32, vp, i64, i64, vp, vp, i64, vp, vp, vp]),
        "kvs_attend_workspace": (i32, [vp, i32, P(i64)]),
        "kvs_attend": (i32, [vp, vp, vp]),
        "kvs_attend_backward": (i32, [vp, vp, vp]),
        "ll_last_error": (ctypes.c_char_p, []),
        "ll_status_str": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _status_name(s: int) -> str:
    return _lib.ll_status_str(s).decode()


def _check(status: int) -> None:
    if status != LL_OK:
        raise LeylineError(status, _lib.ll_last_error().decode())


def _i32_array(values):
    """(contiguous int32 array, its address); an int32 ndarray that is
    already contiguous is used as it is."""
    if isinstance(values, np.ndarray) and values.dtype == np.int32 and values.flags.c_contiguous:
        a = values.reshape(-1)
    else:
        a = np.ascontiguousarray(np.asarray(values, dtype=np.int32)).reshape(-1)
    return a, (a.ctypes.data if a.size else None)


def _require(t, name: str, dtype, shape, device) -> None:
    """Raise ValueError unless `t` is a contiguous tensor of `dtype` and
    exactly `shape` on `device` (checked before any kernel sees its pointer)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: need a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ' (not contiguous)'}")


def _stream_handle(stream, device: int) -> int:
    """The hipStream_t of `stream`, or of the current torch stream of
    `device` (the device the pool or context lives on) when stream is None."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(device)
    return torch.cuda.current_stream(device).cuda_stream


def _on(stream, device: int):
    """Context in which new tensors belong to `stream`, where the call that fills
    them runs (None: the current one).  A block of another stream may have work of
    that stream still queued on it, and goes back to that stream when dropped."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def rope_delta_table(delta: int, rope_dim: int = ROPE_DIM, base: float = 10000.0):
    """float32 (cos, sin) of delta * theta_j, as the library computes them."""
    c = np.zeros(rope_dim // 2, np.float32)
    s = np.zeros(rope_dim // 2, np.float32)
    _check(_lib.ll_rope_delta_table(base, rope_dim, int(delta),
                                    c.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                    s.ctypes.data_as(ctypes.POINTER(ctypes.c_float))))
    return c, s


@dataclass
class Directive:
    """D = (s_start, s_end, R, m).  MLA pools: `stub` is a device bf16 tensor
    [L][r_len][576] (or [r_len][576] for a one-layer pool), or None for
    r_len = 0.  GQA / MHA pools: `stub` holds the K rows and `stub_v` the V
    rows, each [L][r_len][H][D]."""
    seq: int
    s_start: int
    s_end: int
    stub: object = None
    mode: int = AMORTIZE
    stub_v: object = None


@dataclass
class PlanStats:
    alg_bytes: int
    rows_moved: int
    rows_rotated_inplace: int
    fresh_pages: int
    freed_pages: int
    table_entries: int
    planned_on_device: int


class Pool:
    """A paged MLA cache over caller-owned torch memory.

    layers: a bf16 CUDA tensor [L][num_pages][page_size][576] or a list of L
    tensors [num_pages][page_size][576]; page_table: int32 CUDA tensor
    [max_seqs][max_pages_per_seq].  Both are kept referenced by the pool."""

    gqa = False

    def __init__(self, layers, page_table, rope_base: float = 10000.0, pairing: int = ROPE_INTERLEAVED):
        import torch
        if isinstance(layers, torch.Tensor):
            layer_list = [layers[i] for i in range(layers.shape[0])]
        else:
            layer_list = list(layers)
        if not layer_list:
            raise ValueError("no layers")
        shape = tuple(layer_list[0].shape)
        for t in layer_list:
            if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError("layers must be contiguous bf16 CUDA tensors of one shape [pages][P][576]")
        if len(shape) != 3 or shape[2] != ROW:
            raise ValueError("layer shape must be [num_pages][page_size][576]")
        if page_table.dtype != torch.int32 or not page_table.is_cuda or page_table.dim() != 2 \
                or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 CUDA tensor [max_seqs][max_pages_per_seq]")
        self._layers = layer_list
        self._keep = layers
        self.page_table = page_table
        self.num_layers = len(layer_list)
        self.num_pages, self.page_size = shape[0], shape[1]
        self.max_seqs, self.max_pages_per_seq = page_table.shape
        self.device = layer_list[0].device
        self._dev = self.device.index or 0
        self._ptrs = (ctypes.c_void_p * self.num_layers)(*[t.data_ptr() for t in layer_list])
        d = _PoolDesc(self.num_layers, self.page_size, self.num_pages, self.max_seqs, self.max_pages_per_seq,
                      KV_LORA_RANK, ROPE_DIM, pairing, rope_base,
                      ctypes.cast(self._ptrs, ctypes.POINTER(ctypes.c_void_p)),
                      page_table.data_ptr(), self.device.index or 0)
        h = ctypes.c_void_p()
        _check(_lib.ll_pool_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h

    # -- lifetime
    def close(self):
        if getattr(self, "_h", None):
            _lib.ll_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- sequences
    def seq_alloc(self, n_tokens: int, stream=None) -> int:
        sid = ctypes.c_int32()
        _check(_lib.ll_seq_alloc(self._h, int(n_tokens), ctypes.byref(sid), _stream_handle(stream, self._dev)))
        return sid.value

    def seq_set_pages(self, seq: int, pages, n_tokens: int, stream=None) -> None:
        arr, ptr = _i32_array(pages)
        _check(_lib.ll_seq_set_pages(self._h, int(seq), ptr, int(n_tokens), _stream_handle(stream, self._dev)))

    def seq_free(self, seq: int) -> None:
        _check(_lib.ll_seq_free(self._h, int(seq)))

    def seq_get(self, seq: int):
        """(length, next_position, page table as np.int32)."""
        n, pos, cnt = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
        _check(_lib.ll_seq_get(self._h, int(seq), ctypes.byref(n), ctypes.byref(pos), None, 0, ctypes.byref(cnt)))
        pages = np.zeros(cnt.value, np.int32)
        _check(_lib.ll_seq_get(self._h, int(seq), None, None,
                               pages.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), cnt.value, None))
        return n.value, pos.value, pages

    def free_pages(self) -> int:
        n = ctypes.c_int64()
        _check(_lib.ll_pool_free_pages(self._h, ctypes.byref(n)))
        return n.value

    # -- the path
    def _stub(self, st):
        """(r_len, pointer, layer stride in bytes) of one stub tensor."""
        import torch
        if st.dtype != torch.bfloat16 or st.device != self.device or st.shape[-1] != ROW:
            raise ValueError(f"stub must be a bf16 tensor [..., r_len, 576] on {self.device}")
        if st.dim() == 2:
            st = st.unsqueeze(0)
        if st.shape[0] != self.num_layers or st.stride(2) != 1 or st.stride(1) != ROW:
            raise ValueError("stub must be [num_layers][r_len][576] with contiguous rows")
        r_len = st.shape[1]
        return r_len, (st.data_ptr() if r_len else None), st.stride(0) * 2

    def splice(self, directives, stream=None, noalloc: bool = False) -> None:
        """Apply the directives (leyline_splice; noalloc=True:
        leyline_splice_noalloc, which allocates no device memory)."""
        n = len(directives)
        arr = (_Directive * max(1, n))()
        for i, d in enumerate(directives):
            r_len, ptr, stride, ptr_v, stride_v = 0, None, 0, None, 0
            if d.stub is not None and d.mode == AMORTIZE:
                r_len, ptr, stride = self._stub(d.stub)
                if self.gqa:
                    if d.stub_v is None:
                        raise ValueError("a GQA / MHA directive needs stub_v with stub")
                    r_v, ptr_v, stride_v = self._stub(d.stub_v)
                    if r_v != r_len:
                        raise ValueError("stub and stub_v hold different row counts")
            elif d.stub_v is not None and d.mode == AMORTIZE:
                raise ValueError("stub_v without stub")
            arr[i] = _Directive(int(d.seq), int(d.mode), int(d.s_start), int(d.s_end), int(r_len), ptr, stride,
                                ptr_v, stride_v)
        fn = _lib.leyline_splice_noalloc if noalloc else _lib.leyline_splice
        _check(fn(self._h, arr, n, _stream_handle(stream, self._dev)))

    def evict(self, seqs, keep, offsets, stream=None) -> None:
        """keep: uint8 CUDA tensor holding every mask; offsets[i]: start of
        sequence seqs[i]'s mask in it (its length is the sequence length)."""
        import torch
        if not isinstance(keep, torch.Tensor) or keep.dtype != torch.uint8 or keep.device != self.device \
                or not keep.is_contiguous():
            raise ValueError(f"keep must be a contiguous uint8 tensor on {self.device}")
        s_arr, s_ptr = _i32_array(seqs)
        o_arr = offsets if isinstance(offsets, np.ndarray) and offsets.dtype == np.int64 and offsets.flags.c_contiguous \
            else np.ascontiguousarray(np.asarray(offsets, dtype=np.int64))
        o_arr = o_arr.reshape(-1)
        if len(o_arr) != len(s_arr):
            raise ValueError(f"{len(s_arr)} sequences but {len(o_arr)} mask offsets")
        if len(s_arr):
            lens = np.empty(len(s_arr), np.int64)
            _check(_lib.ll_seq_lengths(self._h, s_ptr, len(s_arr), lens.ctypes.data))
            # a negative offset is the library's to refuse (LL_EINVAL)
            past = (o_arr >= 0) & (o_arr + lens > keep.numel())
            if past.any():
                i = int(np.argmax(past))
                raise ValueError(f"mask of sequence {int(s_arr[i])}: bytes [{int(o_arr[i])}, {int(o_arr[i] + lens[i])}) "
                                 f"outside keep's {keep.numel()}")
        _check(_lib.kv_evict_compact(self._h, s_ptr, len(s_arr), keep.data_ptr(),
                                     o_arr.ctypes.data if len(o_arr) else None, _stream_handle(stream, self._dev)))

    def _weights(self, w, name: str):
        """Address and rows of a float32 tensor [max_seqs][rows]."""
        import torch
        if not isinstance(w, torch.Tensor) or w.dtype != torch.float32 or w.device != self.device or w.dim() != 2 \
                or w.shape[0] != self.max_seqs or not w.is_contiguous():
            raise ValueError(f"{name}: need a contiguous float32 tensor [{self.max_seqs}][rows] on {self.device}")
        return w.data_ptr(), w.shape[1]

    def keep_heaviest(self, seqs, budgets, weights, sinks: int = 0, recent: int = 0, keep=None, kept_weights=None,
                      stream=None):
        """Keep masks of the heaviest rows (ll_keep_heaviest): of sequence seqs[i]
        min(budgets[i], its rows) rows, the first `sinks` and the last `recent` ones
        before all others, ties to the earlier row.  weights: float32 [max_seqs][rows]
        (see Step.weigh).  kept_weights: the tensor that gets the weights moved as the
        eviction moves the rows (weights itself: in place; None: no one does).  Returns
        (keep, offsets) as evict(seqs, keep, offsets) takes them; keep: a uint8 tensor
        with room for the masks, new when not given."""
        import torch
        s_arr, s_ptr = _i32_array(seqs)
        b_arr = np.ascontiguousarray(np.asarray(budgets, dtype=np.int64)).reshape(-1)
        if len(b_arr) != len(s_arr):
            raise ValueError(f"{len(s_arr)} sequences but {len(b_arr)} budgets")
        w_ptr, w_rows = self._weights(weights, "weights")
        o_ptr = None
        if kept_weights is not None:
            o_ptr, o_rows = self._weights(kept_weights, "kept_weights")
            if o_rows != w_rows:
                raise ValueError("kept_weights and weights must have one shape")
        lens = np.zeros(len(s_arr), np.int64)
        if len(s_arr):
            _check(_lib.ll_seq_lengths(self._h, s_ptr, len(s_arr), lens.ctypes.data))
        total = int(lens.sum())
        offsets = np.cumsum(lens) - lens
        if keep is None:
            with _on(stream, self._dev):
                keep = torch.empty(total, dtype=torch.uint8, device=self.device)
        elif not isinstance(keep, torch.Tensor) or keep.dtype != torch.uint8 or keep.device != self.device \
                or not keep.is_contiguous() or keep.numel() < total:
            raise ValueError(f"keep must be a contiguous uint8 tensor of {total} bytes or more on {self.device}")
        if total:
            _check(_lib.ll_keep_heaviest(self._h, s_ptr, len(s_arr), b_arr.ctypes.data, int(sinks), int(recent), w_ptr,
                                         o_ptr, w_rows, keep.data_ptr(), offsets.ctypes.data,
                                         _stream_handle(stream, self._dev)))
        return keep, offsets

    def rope_rows(self, seq: int, row_begin: int, angles, out=None, stream=None):
        """Turn the RoPE bands of rows [row_begin, row_begin + len(angles)) of
        a sequence by their own angle steps (angles: int64 CUDA tensor).  With
        out=None the pool is rotated in place; with out=True (or a tensor) the
        rows are gathered into [L][n][row] bf16 and returned, the pool left
        as it was."""
        import torch
        if not isinstance(angles, torch.Tensor) or angles.dtype != torch.int64 or angles.device != self.device \
                or angles.dim() != 1 or not angles.is_contiguous():
            raise ValueError(f"angles must be a contiguous 1-D int64 tensor on {self.device}")
        n = angles.numel()
        ptr, stride = None, 0
        if out is not None:
            shape = (self.num_layers, n, self.heads, self.head_dim) if self.gqa else (self.num_layers, n, ROW)
            if out is True:
                with _on(stream, self._dev):
                    out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            if not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16 or out.device != self.device \
                    or tuple(out.shape) != shape or not out[0].is_contiguous() or out.stride(0) < out[0].numel():
                raise ValueError(f"out must be a bf16 tensor {shape} on {self.device} with contiguous layers")
            ptr, stride = out.data_ptr(), out.stride(0) * 2
        _check(_lib.ll_rope_rows(self._h, int(seq), int(row_begin), int(n), angles.data_ptr() if n else None,
                                 ptr, stride, _stream_handle(stream, self._dev)))
        return out

    def step(self, heads: int, max_seqs: int | None = None, max_tokens: int = 8192) -> "Step":
        """A serving step of this pool for `heads` query heads: up to max_seqs
        sequences (None: all the pool can hold) with up to max_tokens new
        tokens together."""
        return Step(self, heads, self.max_seqs if max_seqs is None else max_seqs, max_tokens)

    def ptable_reindex(self, seq: int, keep_pages, stream=None) -> None:
        arr, ptr = _i32_array(keep_pages)
        _check(_lib.ll_ptable_reindex(self._h, int(seq), ptr, len(arr), _stream_handle(stream, self._dev)))

    # -- counters
    def last_stats(self) -> PlanStats:
        s = _PlanStats()
        _check(_lib.ll_last_plan_stats(self._h, ctypes.byref(s)))
        return PlanStats(s.alg_bytes, s.rows_moved, s.rows_rotated_inplace, s.fresh_pages, s.freed_pages,
                         s.table_entries, s.planned_on_device)

    def set_splice_planner(self, planner: int) -> None:
        """SPLICE_PLAN_AUTO (default: small batches are planned on the device
        from kernel arguments) or SPLICE_PLAN_HOST (always staged and
        uploaded)."""
        _check(_lib.ll_pool_set_splice_planner(self._h, int(planner)))

    def set_page_reuse(self, on: bool) -> None:
        """True (default): a new page keeps an old one whose rows stay at their
        offsets.  False: every page of a rewritten sequence is fresh (the
        sequence is compacted into the lowest free pages); not on page size 1."""
        _check(_lib.ll_pool_set_page_reuse(self._h, 1 if on else 0))

    def set_dispatch_limit(self, max_items: int = 0) -> None:
        """Work-items per dispatch of a row-moving kernel (0: the packet's
        2^32 - 1; at least 1024 otherwise).  Larger launches are issued as
        several dispatches; results do not change."""
        _check(_lib.ll_pool_set_dispatch_limit(self._h, int(max_items)))

    def set_profiling(self, enable: bool, every: int = 1) -> None:
        """Time every `every`-th launch of each profiled kernel while enabled."""
        _check(_lib.ll_pool_set_profiling(self._h, max(1, int(every)) if enable else 0))

    def profile_read(self, kernel: int = 0, samples: int = 0):
        """(launches, total_ms, total_bytes) of kernel 0 (row moves), 1 (keep
        scan) or 2 (per-row rotation); with samples = k > 0 a fourth item, the
        milliseconds of the first k timed launches."""
        n, ms, b = ctypes.c_int64(), ctypes.c_double(), ctypes.c_int64()
        each = np.zeros(max(0, int(samples)), np.float32)
        _check(_lib.ll_profile_read(self._h, kernel, ctypes.byref(n), ctypes.byref(ms), ctypes.byref(b),
                                    each.ctypes.data_as(ctypes.POINTER(ctypes.c_float)) if samples else None,
                                    len(each)))
        if samples:
            return n.value, ms.value, b.value, each[:min(n.value, len(each))].astype(float).tolist()
        return n.value, ms.value, b.value


class GqaPool(Pool):
    """A paged GQA / MHA cache over caller-owned torch memory.

    k_layers, v_layers: bf16 CUDA tensors [L][num_pages][page_size][H][D] (or
    lists of L tensors [num_pages][page_size][H][D]); the first rotary_dim
    values of every K head are its RoPE band.  page_table as for Pool."""

    gqa = True

    def __init__(self, k_layers, v_layers, page_table, rotary_dim: int | None = None,
                 rope_base: float = 10000.0, pairing: int = ROPE_INTERLEAVED):
        import torch

        def planes(x):
            return [x[i] for i in range(x.shape[0])] if isinstance(x, torch.Tensor) else list(x)

        k_list, v_list = planes(k_layers), planes(v_layers)
        if not k_list or len(k_list) != len(v_list):
            raise ValueError("k_layers and v_layers must hold the same number (>= 1) of layers")
        shape = tuple(k_list[0].shape)
        if len(shape) != 4:
            raise ValueError("layer shape must be [num_pages][page_size][H][D]")
        for t in k_list + v_list:
            if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError("K and V layers must be contiguous bf16 CUDA tensors of one shape [pages][P][H][D]")
        if page_table.dtype != torch.int32 or not page_table.is_cuda or page_table.dim() != 2 \
                or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 CUDA tensor [max_seqs][max_pages_per_seq]")
        self._layers = k_list + v_list
        self._keep = (k_layers, v_layers)
        self.page_table = page_table
        self.num_layers = len(k_list)
        self.num_pages, self.page_size, self.heads, self.head_dim = shape
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.row = self.heads * self.head_dim
        self.max_seqs, self.max_pages_per_seq = page_table.shape
        self.device = k_list[0].device
        self._dev = self.device.index or 0
        self._kptrs = (ctypes.c_void_p * self.num_layers)(*[t.data_ptr() for t in k_list])
        self._vptrs = (ctypes.c_void_p * self.num_layers)(*[t.data_ptr() for t in v_list])
        d = _GqaPoolDesc(self.num_layers, self.page_size, self.num_pages, self.max_seqs, self.max_pages_per_seq,
                         self.heads, self.head_dim, self.rotary_dim, pairing, rope_base,
                         ctypes.cast(self._kptrs, ctypes.POINTER(ctypes.c_void_p)),
                         ctypes.cast(self._vptrs, ctypes.POINTER(ctypes.c_void_p)),
                         page_table.data_ptr(), self.device.index or 0)
        h = ctypes.c_void_p()
        _check(_lib.ll_pool_create_gqa(ctypes.byref(d), ctypes.byref(h)))
        self._h = h

    def _stub(self, st):
        import torch
        if st.dtype != torch.bfloat16 or st.device != self.device or tuple(st.shape[-2:]) != (self.heads, self.head_dim):
            raise ValueError(f"stub rows must be bf16 tensors [..., r_len, H, D] on {self.device}")
        if st.dim() == 3:
            st = st.unsqueeze(0)
        if st.shape[0] != self.num_layers or st.stride(3) != 1 or st.stride(2) != self.head_dim \
                or st.stride(1) != self.row:
            raise ValueError("stub rows must be [num_layers][r_len][H][D] with contiguous rows")
        r_len = st.shape[1]
        return r_len, (st.data_ptr() if r_len else None), st.stride(0) * 2


@dataclass
class _Logs:
    n: int
    logs: object
    host: list
    keep: object


class KvsMask:
    """KV-streams trainer-side attention mask on one device: death times from
    the engine's eviction logs, then a block mask, a dense bit mask, or the
    attention under them and its gradient (include/leyline_train.h).

    A log is a list of (time, keep) events per rollout, keep being the mask the
    engine passed to its eviction call (uint8 over the rows held then)."""

    def __init__(self, device: int = 0):
        import torch
        h = ctypes.c_void_p()
        _check(_lib.kvs_ctx_create(int(device), ctypes.byref(h)))
        self._h = h
        self.device = device
        self._tdev = torch.device("cuda", device)

    def close(self):
        if getattr(self, "_h", None):
            _lib.kvs_ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_death(self, death):
        import torch
        if not isinstance(death, torch.Tensor) or death.dim() != 2:
            raise ValueError("death must be a 2-D int32 tensor [n][n_pad]")
        _require(death, "death", torch.int32, tuple(death.shape), self._tdev)

    def upload_logs(self, rollouts):
        """Marshal eviction logs once: rollouts is a list of (n_tokens,
        events), events a list of objects with .time and .keep (host uint8
        arrays).  The keep masks go to the device as one buffer."""
        import torch
        n = len(rollouts)
        chunks, logs, host = [], (_KvsRolloutLog * max(1, n))(), []
        off = 0
        for i, (n_tokens, events) in enumerate(rollouts):
            times = np.ascontiguousarray([int(e.time) for e in events], dtype=np.int64)
            lens = np.ascontiguousarray([len(e.keep) for e in events], dtype=np.int64)
            host += [times, lens]
            logs[i] = _KvsRolloutLog(int(n_tokens), len(events),
                                     times.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                     lens.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), off)
            for e in events:
                chunks.append(np.asarray(e.keep, dtype=np.uint8))
                off += len(e.keep)
        keep = torch.from_numpy(np.concatenate(chunks) if chunks else np.zeros(1, np.uint8)).to(
            torch.device("cuda", self.device))
        return _Logs(n, logs, host, keep)

    def death_times(self, rollouts, n_pad: int, stream=None, out=None):
        """Death times of the rollouts (a list as for upload_logs, or its
        result).  Returns (death int32 [n][n_pad], status int32 [n]) CUDA
        tensors."""
        import torch
        dev = self._tdev
        with _on(stream, self.device):
            logs = rollouts if isinstance(rollouts, _Logs) else self.upload_logs(rollouts)
            if out is None:
                out = (torch.empty((logs.n, n_pad), dtype=torch.int32, device=dev),
                       torch.empty(logs.n, dtype=torch.int32, device=dev))
        death, status = out
        _require(death, "death", torch.int32, (logs.n, n_pad), dev)
        _require(status, "status", torch.int32, (logs.n,), dev)
        _check(_lib.kvs_death_times(self._h, logs.logs, logs.n, int(n_pad), logs.keep.data_ptr(), death.data_ptr(),
                                    status.data_ptr(), _stream_handle(stream, self.device)))
        self._last_logs = logs  # the kernel reads the keep buffer after this returns
        return death, status

    def block_mask(self, death, block_q: int, block_k: int, out=None, stream=None):
        """(partial_num [n][nq], partial_idx [n][nq][nk], full_num, full_idx).
        Without `out` the index arrays are new and filled with -1 past each
        count; with `out` (four int32 tensors of those shapes) the entries past
        each count are left as they were."""
        import torch
        self._check_death(death)
        n, n_pad = death.shape
        nq, nk = -(-n_pad // block_q), -(-n_pad // block_k)
        kw = dict(dtype=torch.int32, device=death.device)
        if out is None:
            with _on(stream, self.device):
                pn, fn = torch.zeros((n, nq), **kw), torch.zeros((n, nq), **kw)
                pi, fi = torch.full((n, nq, nk), -1, **kw), torch.full((n, nq, nk), -1, **kw)
        else:
            pn, pi, fn, fi = out
            for x, shape in ((pn, (n, nq)), (pi, (n, nq, nk)), (fn, (n, nq)), (fi, (n, nq, nk))):
                if tuple(x.shape) != shape or x.dtype != torch.int32 or not x.is_contiguous() or x.device != death.device:
                    raise ValueError(f"block_mask out: need contiguous int32 {shape} on {death.device}")
        _check(_lib.kvs_block_mask(self._h, death.data_ptr(), n, n_pad, int(block_q), int(block_k), pn.data_ptr(),
                                   pi.data_ptr(), fn.data_ptr(), fi.data_ptr(), _stream_handle(stream, self.device)))
        return pn, pi, fn, fi

    def dense_mask(self, death, out=None, stream=None):
        """uint32 bits [n][n_pad][n_pad / 32] (as an int32 tensor)."""
        import torch
        self._check_death(death)
        n, n_pad = death.shape
        if out is None:
            with _on(stream, self.device):
                out = torch.empty((n, n_pad, n_pad // 32), dtype=torch.int32, device=death.device)
        _require(out, "out", torch.int32, (n, n_pad, n_pad // 32), self._tdev)
        _check(_lib.kvs_dense_mask(self._h, death.data_ptr(), n, n_pad, out.data_ptr(), _stream_handle(stream, self.device)))
        return out


    # -- the trainer's attention
    def _heads(self, t, name: str, shape):
        """(address, rollout, token and head stride) of a bf16 tensor of `shape`
        [n][n_pad][heads][width] on this device with a dense last axis."""
        import torch
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device != self._tdev \
                or tuple(t.shape) != shape or (t.stride(3) != 1 and t.numel()):
            raise ValueError(f"{name}: need a bf16 tensor {list(shape)} on {self._tdev} with a dense last axis")
        return (t.data_ptr(), *t.stride()[:3])

    def _attend_desc(self, q, k, v, death, scale, cap, out, lse, backward: bool, stream):
        """The packed kvs_attend_desc, with `out` and `lse` (new where None) and the
        workspace that it names."""
        import torch
        self._check_death(death)
        if not all(isinstance(t, torch.Tensor) and t.dim() == 4 for t in (q, k, v)):
            raise ValueError("q, k and v must be 4-D tensors [n][n_pad][heads][width]")
        n, n_pad = death.shape
        heads, kv_heads, dk, dv = q.shape[2], k.shape[2], q.shape[3], v.shape[3]
        q_s = self._heads(q, "q", (n, n_pad, heads, dk))
        k_s = self._heads(k, "k", (n, n_pad, kv_heads, dk))
        v_s = self._heads(v, "v", (n, n_pad, kv_heads, dv))
        with _on(stream, self.device):
            if out is None:
                out = torch.empty((n, n_pad, heads, dv), dtype=torch.bfloat16, device=self._tdev)
            if lse is None:
                lse = torch.empty((n, n_pad, heads), dtype=torch.float32, device=self._tdev)
            o_s = self._heads(out, "out", (n, n_pad, heads, dv))
            _require(lse, "lse", torch.float32, (n, n_pad, heads), self._tdev)

            def pack(work, size):
                try:
                    return _TRAIN_DESC.pack(n, heads, n_pad, kv_heads, dk, dv, scale, cap, death.data_ptr(), *q_s, *k_s,
                                            *v_s, *o_s, lse.data_ptr(), work, size)
                except (struct.error, OverflowError) as e:
                    raise ValueError(f"sizes, scale or cap: {e}") from None

            size = ctypes.c_int64()
            _check(_lib.kvs_attend_workspace(pack(0, 0), 1 if backward else 0, ctypes.byref(size)))
            work = torch.empty(size.value, dtype=torch.uint8, device=self._tdev)
        return pack(work.data_ptr(), size.value), out, lse, work

    def attend(self, q, k, v, death, scale: float | None = None, cap: float = 0.0, out=None, lse=None, stream=None):
        """Attention under death times (kvs_attend): query t of a rollout sees key s iff
        s <= t < death[s].  q [n][n_pad][heads][key width], k [n][n_pad][KV heads][key
        width], v [n][n_pad][KV heads][value width], bf16 views with a dense last axis and
        the other strides multiples of 8 values; death as death_times gives it.  scale
        defaults to the key width ** -0.5; cap > 0: scores are cap * tanh(scale * q . k /
        cap).  Returns (out [n][n_pad][heads][value width], lse float32
        [n][n_pad][heads]).  Nothing of it is differentiable: see attention."""
        if scale is None:
            scale = q.shape[-1] ** -0.5
        desc, out, lse, work = self._attend_desc(q, k, v, death, scale, cap, out, lse, False, stream)
        _check(_lib.kvs_attend(self._h, desc, _stream_handle(stream, self.device)))
        return out, lse

    def attend_backward(self, dout, q, k, v, out, lse, death, scale: float | None = None, cap: float = 0.0, grads=None,
                        stream=None):
        """The gradients (dq, dk, dv) of attend for the gradient dout of its out
        (kvs_attend_backward); out and lse are what attend returned for the same inputs.
        grads: three bf16 tensors shaped as q, k and v to write; new ones when not given."""
        import torch
        if out is None or lse is None:
            raise ValueError("out and lse of the forward pass must be given")
        if scale is None:
            scale = q.shape[-1] ** -0.5
        desc, out, lse, work = self._attend_desc(q, k, v, death, scale, cap, out, lse, True, stream)
        g_s = self._heads(dout, "dout", tuple(out.shape))
        if grads is None:
            with _on(stream, self.device):
                grads = tuple(torch.empty(t.shape, dtype=torch.bfloat16, device=self._tdev) for t in (q, k, v))
        dq, dk, dv = grads
        desc += _TRAIN_GRADS.pack(*g_s, *self._heads(dq, "dq", tuple(q.shape)), *self._heads(dk, "dk", tuple(k.shape)),
                                  *self._heads(dv, "dv", tuple(v.shape)))
        _check(_lib.kvs_attend_backward(self._h, desc, _stream_handle(stream, self.device)))
        return dq, dk, dv

    def attention(self, q, k, v, death, scale: float | None = None, cap: float = 0.0):
        """attend with a gradient: out, differentiable in q, k and v, on the current
        stream.  Not for graph capture, forward or backward: there attend and
        attend_backward are called themselves, so that no autograd state of an eager pass
        takes part."""
        return _attention_function().apply(self, q, k, v, death, scale, cap)


_ATTENTION = None


def _attention_function():
    global _ATTENTION
    if _ATTENTION is not None:
        return _ATTENTION
    import torch

    def eager():
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("attention cannot be captured: call attend and attend_backward")

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, kvs, q, k, v, death, scale, cap):
            eager()
            out, lse = kvs.attend(q, k, v, death, scale, cap)
            ctx.kvs, ctx.scale, ctx.cap = kvs, scale, cap
            ctx.save_for_backward(q, k, v, death, out, lse)
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            eager()
            q, k, v, death, out, lse = ctx.saved_tensors
            # a gradient may come as any view, e.g. one value broadcast
            dout = dout.contiguous()
            if dout.data_ptr() % 16:
                dout = dout.clone()
            return (None, *ctx.kvs.attend_backward(dout, q, k, v, out, lse, death, ctx.scale, ctx.cap), None, None, None)

    _ATTENTION = Attention
    return Attention


class Step:
    """The serving step of a pool (include/leyline_step.h): begin() names the
    sequences and how many tokens each brings, then append() and attend() run
    once per layer.  The tokens of a step are the first sequence's in order, then
    the second's, ...; tensors hold one row per token, or more (the first ones are
    used; under graph capture they hold max_tokens rows).

    Inputs may be views (e.g. of one projection's output): the last axis is dense,
    the other strides are multiples of 8 values and the data is 16-byte aligned.

    A call runs on `stream` (None: the current one), and results that it allocates
    belong to that stream.  Inputs made on another one, and results read on another
    one, are the caller's to order and to keep (torch's record_stream).

    A graph that holds calls of a step needs the step, which owns their workspace:
    keep it open for as long as the graph is replayed."""

    def __init__(self, pool: Pool, heads: int, max_seqs: int, max_tokens: int):
        import torch
        d = _StepDesc(int(heads), int(max_seqs), int(max_tokens))
        h = ctypes.c_void_p()
        _check(_lib.ll_step_create(pool._h, ctypes.byref(d), ctypes.byref(h)))
        self._h = h
        self._pool = pool
        self.gqa, self.heads, self.max_seqs, self.max_tokens = pool.gqa, int(heads), int(max_seqs), int(max_tokens)
        self.device, self._dev = pool.device, pool._dev
        self.tokens = 0
        # widths of a result and of a query's rotated part (append), and the axes
        # behind the tokens of every tensor that append and attend take
        self._dv, self._dr = (pool.head_dim,) * 2 if pool.gqa else (KV_LORA_RANK, ROPE_DIM)
        self._a_tail = (pool.heads, pool.head_dim) if pool.gqa else (KV_LORA_RANK,)
        self._b_tail = (pool.heads, pool.head_dim) if pool.gqa else (ROPE_DIM,)
        self._q_tail, self._r_tail, self._o_tail = (self.heads, ROW), (self.heads, self._dr), (self.heads, self._dv)
        self._l_tail = (self.heads,)
        self._torch, self._bf16, self._f32 = torch, torch.bfloat16, torch.float32
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: _stream_handle(None, d))

    def close(self):
        if getattr(self, "_h", None):
            _lib.ll_step_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def begin(self, seqs, counts, grow: bool = True, stream=None) -> int:
        """counts[i] tokens of sequence seqs[i].  grow=True: new ones, every
        sequence grows by them; grow=False: the last ones it already holds.
        Returns the number of tokens of the step."""
        s_arr, s_ptr = _i32_array(seqs)
        c_arr, c_ptr = _i32_array(counts)
        if len(s_arr) != len(c_arr):
            raise ValueError(f"{len(s_arr)} sequences but {len(c_arr)} token counts")
        _check(_lib.ll_step_begin(self._h, s_ptr, c_ptr, len(s_arr), 1 if grow else 0,
                                  _stream_handle(stream, self._dev)))
        self.tokens = int(c_arr.sum())
        return self.tokens

    def _rows(self, t, name: str, tail, dtype):
        """(tokens, address, token stride, head stride) of a [tokens][*tail] tensor on
        the pool's device (tail: heads and width, or a width alone)."""
        # once per tensor of every call: each attribute is read once
        try:
            if len(tail) == 2:
                n, h, d = t.shape
                ts, hs, one = t.stride()
                ok = h == tail[0] and d == tail[1]
            else:
                n, d = t.shape
                ts, one = t.stride()
                hs, ok = 0, d == tail[0]
            ok = ok and (one == 1 or n == 0) and t.dtype is dtype and t.device == self.device
        except (AttributeError, TypeError, ValueError):   # no tensor, or one of other axes
            ok = False
        if not ok:
            raise ValueError(f"{name}: need a {dtype} tensor [tokens]{list(tail)} on {self.device} with a dense last axis")
        return n, t.data_ptr(), ts, hs

    def _new(self, shape, dtype, stream):
        """A result for a call on `stream`."""
        if stream is None:
            return self._torch.empty(shape, dtype=dtype, device=self.device)
        with _on(stream, self._dev):
            return self._torch.empty(shape, dtype=dtype, device=self.device)

    def _weight(self, w, name: str, n: int):
        """(address, LL_TYPE_*) of a norm's weight."""
        try:
            dt = w.dtype
            ok = (dt is self._bf16 or dt is self._f32) and w.shape == (n,) and w.device == self.device and w.is_contiguous()
        except AttributeError:   # no tensor
            ok = False
        if not ok:
            raise ValueError(f"{name}: need a dense bf16 or float32 tensor [{n}] on {self.device}")
        return w.data_ptr(), 1 if dt is self._f32 else 0

    def append(self, layer: int, a=None, b=None, norm=None, q=None, q_out=None, q_norm=None, eps: float = 1e-6,
               stream=None):
        """Write one layer's new rows and prepare its queries (ll_step_append).

        MLA: a = c_kv [T][512], b = k_pe [T][64], q = the rotated part of the
        queries [T][heads][64]; GQA: a = K, b = V [T][kv_heads][head_dim], q =
        [T][heads][head_dim].  norm / q_norm: RMS-norm weights (bf16 or float32) of
        c_kv or the K heads / the query heads (GQA).  Returns q_out (new when not
        given; q itself turns the queries in place), or None without q."""
        bf16 = self._bf16
        room = 1 << 62
        a_ptr = a_ts = a_hs = b_ptr = b_ts = b_hs = 0
        if a is not None and b is not None:
            room, a_ptr, a_ts, a_hs = self._rows(a, "a", self._a_tail, bf16)
            n, b_ptr, b_ts, b_hs = self._rows(b, "b", self._b_tail, bf16)
            room = min(room, n)
        elif a is not None or b is not None:
            raise ValueError("a and b go together")
        norm_ptr = qn_ptr = f32 = 0
        if norm is not None:
            norm_ptr, f32 = self._weight(norm, "norm", self._dv)
        q_ptr = q_ts = q_hs = o_ptr = o_ts = o_hs = 0
        if q is not None:
            n, q_ptr, q_ts, q_hs = self._rows(q, "q", self._r_tail, bf16)
            room = min(room, n)
            if q_out is None:
                q_out = self._new(q.shape, bf16, stream)
            n, o_ptr, o_ts, o_hs = self._rows(q_out, "q_out", self._r_tail, bf16)
            room = min(room, n)
            if q_norm is not None:
                qn_ptr, kind = self._weight(q_norm, "q_norm", self._dr)
                if norm is not None and kind != f32:
                    raise ValueError("norm and q_norm must have one dtype")
                f32 = kind
        elif q_out is not None or q_norm is not None:
            raise ValueError("q_out and q_norm need q")
        try:
            desc = _APPEND_DESC.pack(room, layer, f32, a_ptr, a_ts, a_hs, b_ptr, b_ts, b_hs, norm_ptr, q_ptr, q_ts, q_hs,
                                     o_ptr, o_ts, o_hs, qn_ptr, eps)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"layer or eps: {e}") from None
        rc = _lib.ll_step_append(self._h, desc, self._raw_stream(self._dev) if stream is None else stream.cuda_stream)
        if rc:
            _check(rc)
        return q_out

    def _queries(self, q, q_pe, scale):
        """(scale, tokens, then address, token and head stride of q and of q_pe) of an
        attention's queries."""
        bf16 = self._bf16
        if scale is None:
            if not self.gqa:
                raise ValueError("scale must be given: the latent width does not say the model's head width")
            scale = self._dv ** -0.5
        p_ptr = p_ts = p_hs = 0
        if self.gqa:
            if q_pe is not None:
                raise ValueError("q_pe is for MLA pools only")
            room, q_ptr, q_ts, q_hs = self._rows(q, "q", self._o_tail, bf16)
        elif q_pe is None:
            room, q_ptr, q_ts, q_hs = self._rows(q, "q", self._q_tail, bf16)
            p_ptr, p_ts, p_hs = q_ptr + 2 * KV_LORA_RANK, q_ts, q_hs
        else:
            room, q_ptr, q_ts, q_hs = self._rows(q, "q", self._o_tail, bf16)
            n, p_ptr, p_ts, p_hs = self._rows(q_pe, "q_pe", self._r_tail, bf16)
            room = min(room, n)
        return scale, room, q_ptr, q_ts, q_hs, p_ptr, p_ts, p_hs

    def attend(self, layer: int, q, q_pe=None, scale: float | None = None, causal: bool = True, window: int = 0,
               out=None, lse=None, stream=None, cap: float = 0.0):
        """Attention of the step's tokens over one layer (ll_step_attend; with a cap:
        ll_step_attend_capped, scores cap * tanh(scale * q . k / cap)).

        MLA: q [T][heads][576] (latent part, then the rotated part), or q
        [T][heads][512] with q_pe [T][heads][64]; the result is [T][heads][512] in
        the latent space, and scale must be given.  GQA: q and the result are
        [T][heads][head_dim], scale defaults to head_dim ** -0.5.  window > 0: a
        token sees the last `window` rows up to its own.  lse=True (or a dense
        float32 tensor [T][heads]) also returns the log sum exp: (out, lse)."""
        bf16 = self._bf16
        scale, room, q_ptr, q_ts, q_hs, p_ptr, p_ts, p_hs = self._queries(q, q_pe, scale)
        if out is None:
            out = self._new((q.shape[0], *self._o_tail), bf16, stream)
        n, o_ptr, o_ts, o_hs = self._rows(out, "out", self._o_tail, bf16)
        room = min(room, n)
        l_ptr = 0
        if lse is True:
            lse = self._new((q.shape[0], self.heads), self._f32, stream)
        if lse is not None and lse is not False:
            n, l_ptr, _, _ = self._rows(lse, "lse", self._l_tail, self._f32)
            if not lse.is_contiguous():
                raise ValueError("lse must be contiguous")
            room = min(room, n)
        else:
            lse = None
        try:
            desc = _ATTEND_DESC.pack(room, layer, 1 if causal else 0, window, scale, q_ptr, q_ts, q_hs, p_ptr, p_ts, p_hs,
                                     o_ptr, o_ts, o_hs, l_ptr)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"layer, window or scale: {e}") from None
        st = self._raw_stream(self._dev) if stream is None else stream.cuda_stream
        if cap:
            try:
                rc = _lib.ll_step_attend_capped(self._h, desc, cap, st)
            except ctypes.ArgumentError as e:
                raise ValueError(f"cap: {e}") from None
        else:
            rc = _lib.ll_step_attend(self._h, desc, st)
        if rc:
            _check(rc)
        return out if lse is None else (out, lse)

    def weigh(self, layer: int, q, lse, weights, q_pe=None, scale: float | None = None, causal: bool = True,
              window: int = 0, cap: float = 0.0, decay: float = 1.0, stream=None):
        """Add the attention that each cached row of the step's sequences gets from the
        step's tokens in one layer, over all heads, to weights (ll_step_weigh): a float32
        tensor [the pool's max_seqs][rows], zeros at first, row s of sequence s.  q, q_pe,
        scale, causal, window and cap as in the attend that gave lse; decay multiplies
        what was there (0: it counts nothing).  Returns weights."""
        scale, room, q_ptr, q_ts, q_hs, p_ptr, p_ts, p_hs = self._queries(q, q_pe, scale)
        n, l_ptr, _, _ = self._rows(lse, "lse", self._l_tail, self._f32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        room = min(room, n)
        w_ptr, w_rows = self._pool._weights(weights, "weights")
        try:
            desc = _WEIGH_DESC.pack(room, layer, 1 if causal else 0, window, scale, cap, q_ptr, q_ts, q_hs, p_ptr, p_ts,
                                    p_hs, l_ptr, w_ptr, w_rows, decay)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"layer, window, scale, cap or decay: {e}") from None
        rc = _lib.ll_step_weigh(self._h, desc, self._raw_stream(self._dev) if stream is None else stream.cuda_stream)
        if rc:
            _check(rc)
        return weights
