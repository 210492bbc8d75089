"""ctypes binding of libdetint (include/detint.h), with the same names.

Argument marshalling only: every step of the forward pass runs in the CUDA
kernels behind the C ABI. PyTorch supplies device memory and streams. If the
library is missing or cannot be loaded, every entry point raises; there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import hashlib
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdetint.so")
_lib = None

ERRORS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "token id outside the vocabulary",
          4: "context capacity exceeded", 5: "unreadable or malformed artifact",
          6: "artifact sha256 mismatch", 7: "CUDA error", 8: "device out of memory",
          9: "bad sequence id", 10: "saturation recorded"}

# every entry point of include/detint.h
SYMBOLS = ["detint_load", "detint_load_kv", "detint_prefill", "detint_decode_step", "detint_gemm_i8",
           "detint_reset_seq", "detint_seq_len", "detint_status", "detint_set_graph",
           "detint_set_option", "detint_argmax_noalloc", "detint_sample", "detint_fork_seq", "detint_reorder_seqs", "detint_gemm_w16", "detint_split_w16",
           "detint_int8_peak_loop", "detint_kv4_append", "detint_kv4_workspace", "detint_kv4_decode",
           "detint_kv4_prefill", "detint_kv4_append_axes", "detint_kv4_weigh", "detint_kv4_weigh_block",
           "detint_kv4_evict", "detint_kv4_copy", "detint_beam_select", "detint_beam_workspace",
           "detint_beam_reorder", "detint_model_info", "detint_free", "detint_strerror", "detint_last_error"]


class DetintError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({detail})" if detail else
                         f"{where}: {ERRORS.get(code, code)}")


def lib():
    """The loaded libdetint; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "deterministic_integer_only_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        vp, i32p = C.c_void_p, C.POINTER(C.c_int32)
        L.detint_load.argtypes = [C.c_char_p, C.c_int, C.c_int, vp, C.POINTER(vp)]
        L.detint_load_kv.argtypes = [C.c_char_p, C.c_int, C.c_int, C.c_int, vp, C.POINTER(vp)]
        L.detint_prefill.argtypes = [vp, C.c_int, i32p, i32p, vp, vp, vp, vp]
        L.detint_decode_step.argtypes = [vp, C.c_int, i32p, vp, vp, vp, vp]
        L.detint_gemm_i8.argtypes = [vp, vp, vp, C.c_int, C.c_int, C.c_int, vp]
        L.detint_reset_seq.argtypes = [vp, C.c_int]
        L.detint_seq_len.argtypes = [vp, C.c_int, i32p]
        L.detint_status.argtypes = [vp, i32p, vp]
        L.detint_set_graph.argtypes = [vp, C.c_int]
        L.detint_set_option.argtypes = [vp, C.c_int, C.c_int]
        L.detint_argmax_noalloc.argtypes = [vp, C.c_int, C.c_int, vp, vp]
        L.detint_fork_seq.argtypes = [vp, C.c_int, C.c_int, C.c_int, vp]
        L.detint_reorder_seqs.argtypes = [vp, C.c_int, i32p, i32p, vp]
        L.detint_gemm_w16.argtypes = [vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp]
        L.detint_split_w16.argtypes = [vp, vp, vp, C.c_longlong, vp]
        L.detint_sample.argtypes = [vp, C.c_int, C.c_int, C.POINTER(SamplingParams), vp, vp]
        L.detint_int8_peak_loop.argtypes = [C.c_int, C.c_int, C.c_int, vp, C.POINTER(C.c_longlong), vp]
        ll = C.c_longlong
        L.detint_kv4_append.argtypes = [vp, vp, vp, ll, vp, vp, C.c_int, vp, vp, vp, vp, vp, vp]
        L.detint_kv4_workspace.argtypes = [vp, C.c_int, C.c_int, C.POINTER(ll)]
        L.detint_kv4_decode.argtypes = [vp, vp, vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, ll, vp, ll, vp]
        L.detint_kv4_prefill.argtypes = [vp, vp, vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, ll, vp]
        L.detint_kv4_append_axes.argtypes = [vp, vp, vp, vp, C.c_int, vp, ll, vp, vp, C.c_int, vp, vp, vp, vp, vp, vp]
        L.detint_kv4_weigh.argtypes = [vp, vp, vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, vp]
        L.detint_kv4_weigh_block.argtypes = [vp, vp, vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, vp]
        L.detint_kv4_evict.argtypes = [vp, vp, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp]
        L.detint_kv4_copy.argtypes = [vp, vp, vp, C.c_int, vp, vp]
        L.detint_beam_select.argtypes = [vp, ll, C.c_int, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp, vp, vp,
                                         ll, vp]
        L.detint_beam_workspace.argtypes = [C.c_int, C.c_int, C.c_int, C.POINTER(ll)]
        L.detint_beam_reorder.argtypes = [vp, vp, C.c_int, vp, vp, C.c_int, C.c_int, vp, vp, vp]
        L.detint_model_info.argtypes = [vp, i32p]
        L.detint_free.argtypes = [vp]
        L.detint_free.restype = None
        L.detint_strerror.restype = C.c_char_p
        L.detint_strerror.argtypes = [C.c_int]
        L.detint_last_error.restype = C.c_char_p
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != 0:
        raise DetintError(rc, where, lib().detint_last_error().decode(errors="replace"))


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def detint_gemm_i8(A, B, C_out, stream=None):
    """C_out[M,N] (int32, cuda) = A[M,K] (int8) @ B[N,K]^T (int8), exact."""
    M, K = A.shape
    N = B.shape[0]
    _check(lib().detint_gemm_i8(_ptr(A), _ptr(B), _ptr(C_out), M, N, K, _stream(stream)),
           "detint_gemm_i8")
    return C_out


def detint_argmax_noalloc(logits, out, stream=None):
    """out[r] = tie-low argmax of logits[r] (int32 cuda tensors), computed
    without any device allocation (partials in a fixed device array)."""
    import torch
    rows, n = logits.shape
    if logits.dtype != torch.int32 or out.dtype != torch.int32 or not logits.is_cuda or not out.is_cuda:
        raise ValueError("detint_argmax_noalloc: int32 cuda tensors expected")
    if not logits.is_contiguous() or not out.is_contiguous() or out.numel() < rows:
        raise ValueError("detint_argmax_noalloc: contiguous logits [rows, n] and out [rows] expected")
    _check(lib().detint_argmax_noalloc(_ptr(logits), rows, n, _ptr(out), _stream(stream)),
           "detint_argmax_noalloc")
    return out


class SamplingParams(C.Structure):
    """detint_sampling_t: seed, counter (SplitMix64 draw index), inv_temp
    (Q16 of 1/T), top_k (0: off), top_p (Q16, 65536: off)."""
    _fields_ = [("seed", C.c_uint64), ("counter", C.c_uint64), ("inv_temp", C.c_int32),
                ("top_k", C.c_int32), ("top_p", C.c_int32), ("reserved", C.c_int32)]


def detint_sample(logits, params, out=None, stream=None):
    """One integer-sampled token per row of an int32 cuda tensor [rows, n];
    params: one dict (or SamplingParams) per row, or one for every row."""
    import torch
    rows, n = logits.shape
    if isinstance(params, (dict, SamplingParams)):
        params = [params] * rows
    arr = (SamplingParams * rows)()
    for r, p in enumerate(params):
        if isinstance(p, SamplingParams):
            arr[r] = p
        else:
            arr[r] = SamplingParams(int(p.get("seed", 0)), int(p.get("counter", 0)),
                                    int(p.get("inv_temp", 65536)), int(p.get("top_k", 0)),
                                    int(p.get("top_p", 65536)), 0)
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    _check(lib().detint_sample(_ptr(logits), rows, n, arr, _ptr(out), _stream(stream)), "detint_sample")
    return out


def detint_split_w16(W, stream=None):
    """(w_hi int8, w_lo uint8) limbs of an int16 cuda tensor, W = 256 hi + lo."""
    import torch
    hi = torch.empty(W.shape, dtype=torch.int8, device=W.device)
    lo = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    _check(lib().detint_split_w16(_ptr(W), _ptr(hi), _ptr(lo), W.numel(), _stream(stream)), "detint_split_w16")
    return hi, lo


def detint_gemm_w16(A, w_hi, w_lo, C=None, stream=None):
    """C = A @ W.T exactly in int64 (int8 A [M, K], W = 256 w_hi + w_lo [N, K])."""
    import torch
    M, K = A.shape
    N = w_hi.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.int64, device=A.device)
    _check(lib().detint_gemm_w16(_ptr(A), _ptr(w_hi), _ptr(w_lo), _ptr(C), M, N, K, _stream(stream)),
           "detint_gemm_w16")
    return C


def detint_int8_peak_loop(kind: int, blocks: int, iters: int, sink, stream=None) -> int:
    """Launch the integer-pipe peak loop (kind 0 mma.sync s8, 1 dp4a); returns
    the integer operations it performs."""
    ops = C.c_longlong(0)
    _check(lib().detint_int8_peak_loop(int(kind), int(blocks), int(iters), _ptr(sink), C.byref(ops),
                                       _stream(stream)), "detint_int8_peak_loop")
    return int(ops.value)


# ------------------------------------------------- the 4-bit paged K/V cache
class _Kv4(C.Structure):
    """detint_kv4_t"""
    _fields_ = [(n, C.c_int32) for n in ("n_q", "n_kv", "head_dim", "n_blocks", "n_seq", "max_blocks")] + \
               [(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "block_table", "params", "status")]


class _Rope(C.Structure):
    """detint_rope_t"""
    _fields_ = [("cos", C.c_void_p), ("sin", C.c_void_p), ("max_pos", C.c_int32), ("rot_dim", C.c_int32),
                ("interleaved", C.c_int32), ("eps", C.c_int32), ("q_gamma", C.c_void_p), ("k_gamma", C.c_void_p)]


def _expect(where, name, t, dtype, numel, device):
    """A contiguous tensor of `dtype` on `device` that holds numel elements."""
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{where}: {name}: a contiguous {dtype} tensor of {numel} elements on {device} expected, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


class KV4Cache:
    """A view of a 4-bit paged K/V cache in caller-owned cuda tensors.

    k, v: uint8 with n_blocks * n_kv * 32 * head_dim elements, k as
    [n_blocks, n_kv, 64, head_dim // 2]; k_scale, v_scale: uint8
    [n_blocks, n_kv, 64]; block_table: int32 [n_seq, max_blocks]; params: int32
    [n_kv, 8 + head_dim]; status: int32 [8] or None. The tensors are kept
    alive with the view, and their memory is used in place."""

    def __init__(self, k, v, k_scale, v_scale, block_table, params, n_q: int, status=None):
        import torch
        n_blocks, n_kv, blk, half = k.shape
        if not k.is_cuda or blk != 64:
            raise ValueError("KV4Cache: k: a cuda tensor [n_blocks, n_kv, 64, head_dim // 2] expected")
        dev, d = k.device, 2 * half
        n_seq, max_blocks = block_table.shape
        pages = n_blocks * n_kv * 64
        for name, t, dt, n in (("k", k, torch.uint8, pages * half), ("v", v, torch.uint8, pages * half),
                               ("k_scale", k_scale, torch.uint8, pages), ("v_scale", v_scale, torch.uint8, pages),
                               ("block_table", block_table, torch.int32, n_seq * max_blocks),
                               ("params", params, torch.int32, n_kv * (8 + d))):
            _expect("KV4Cache", name, t, dt, n, dev)
        if status is not None:
            _expect("KV4Cache", "status", status, torch.int32, 8, dev)
        self.n_q, self.n_kv, self.head_dim, self.device = int(n_q), n_kv, d, dev
        self.n_blocks = n_blocks
        self._index, self._torch = dev.index, torch
        self._keep = (k, v, k_scale, v_scale, block_table, params, status)
        self._c = _Kv4(int(n_q), n_kv, d, n_blocks, n_seq, max_blocks, _ptr(k), _ptr(v), _ptr(k_scale),
                       _ptr(v_scale), _ptr(block_table), _ptr(params), _ptr(status))
        self._ref = C.addressof(self._c)


class RopeNorm:
    """Rotation tables (int16 Q14 cuda tensors [max_pos, rot_dim // 2], or None
    for no rotation), pair layout, and the optional per-head norm (int16 Q12
    gammas, eps = round(eps 2^24)) of detint_kv4_append."""

    def __init__(self, cos, sin, interleaved: bool = False, q_gamma=None, k_gamma=None, eps: int = 0,
                 max_pos: int | None = None):
        import torch
        if (cos is None) != (sin is None) or (cos is None and max_pos is None):
            raise ValueError("RopeNorm: both tables, or none and max_pos")
        rot = 0
        self.device = None
        if cos is not None:
            max_pos, rot = cos.shape[0], 2 * cos.shape[1]
            self.device = cos.device
            _expect("RopeNorm", "cos", cos, torch.int16, max_pos * rot // 2, cos.device)
            _expect("RopeNorm", "sin", sin, torch.int16, max_pos * rot // 2, cos.device)
        for name, t in (("cos", cos), ("q_gamma", q_gamma), ("k_gamma", k_gamma)):
            if t is not None and not t.is_cuda:              # the others have to be where these are
                raise ValueError(f"RopeNorm: {name}: a cuda tensor expected, got one on {t.device}")
        self._gammas = 0 if q_gamma is None else q_gamma.numel()
        for name, t in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
            if t is not None:
                self.device = self.device or t.device
                _expect("RopeNorm", name, t, torch.int16, self._gammas, self.device)
        self._index = None if self.device is None else self.device.index
        if not (abs(max_pos) < 1 << 31 and abs(eps) < 1 << 31):          # (would be cut to 32 bits on the way)
            raise ValueError(f"RopeNorm: max_pos {max_pos} or eps {eps} out of range")
        self._keep = (cos, sin, q_gamma, k_gamma)
        self._c = _Rope(_ptr(cos), _ptr(sin), int(max_pos), rot, int(bool(interleaved)), int(eps), _ptr(q_gamma),
                        _ptr(k_gamma))
        self._ref = C.addressof(self._c)


def _unfit(t, dtype, numel, index) -> bool:
    """Whether t is not a contiguous cuda tensor of that type and device with
    room for numel elements. A decode step makes these calls once per layer:
    the checks stay a few hundred nanoseconds each, and _expect words the
    error once one fails."""
    return t.dtype is not dtype or t.get_device() != index or t.numel() < numel or not t.is_contiguous()


def _row_stride(where, name, t, dtype, rows, width, index) -> int:
    """The stride of rows of at least `width` elements, which may be strided."""
    if t.dtype is dtype and t.get_device() == index:
        if t.numel() == rows * width and t.is_contiguous():
            return width
        if t.dim() == 2 and t.size(0) >= rows and t.size(1) >= width and t.stride(1) == 1:
            return t.stride(0) if t.size(0) > 1 else width
    raise ValueError(f"{where}: {name}: {dtype} rows [{rows}, {width}] on cuda:{index} expected, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}")


def _kv4_current(where, cache):
    if cache._torch._C._cuda_getDevice() != cache._index:
        raise ValueError(f"{where}: the cache is on {cache.device}, which is not the current device")


def _kv4_call(where, cache, q8, mq, kq, tok_seq, tok_pos, stream):
    """The checks the kv4 operators share: tokens and query buffers (None:
    to be made). Returns (tokens, raw stream)."""
    index, torch, n = cache._index, cache._torch, tok_pos.numel()
    i32 = torch.int32
    if torch._C._cuda_getDevice() != index:
        _kv4_current(where, cache)                       # words the error
    rows = n * cache.n_q
    if _unfit(tok_pos, i32, n, index) or _unfit(tok_seq, i32, n, index) or \
            mq is not None and _unfit(mq, i32, rows, index) or kq is not None and _unfit(kq, i32, rows, index) or \
            q8 is not None and _unfit(q8, torch.int8, rows * cache.head_dim, index):
        for name, t, dt, m in (("tok_pos", tok_pos, i32, n), ("tok_seq", tok_seq, i32, n), ("mq", mq, i32, rows),
                               ("kq", kq, i32, rows), ("q8", q8, torch.int8, rows * cache.head_dim)):
            if t is not None:
                _expect(where, name, t, dt, m, cache.device)
    if stream is None:
        return n, torch._C._cuda_getCurrentRawStream(index)
    return n, stream.cuda_stream


def _new(stream, shape, dtype, device):
    """A tensor for a kernel on `stream` (None: the current one)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _kv4_append(w, cache, rope, qkv, tok_seq, tok_pos, axes, q8, mq, kq, k_val, v_val, stream):
    torch, dev, index = cache._torch, cache.device, cache._index
    n, raw = _kv4_call(w, cache, q8, mq, kq, tok_seq, tok_pos, stream)
    nq, d = cache.n_q, cache.head_dim
    stride = _row_stride(w, "qkv", qkv, torch.int32, n, (nq + 2 * cache.n_kv) * d, index)
    if rope._index not in (None, index) or rope._gammas not in (0, d):
        raise ValueError(f"{w}: tables or gammas do not fit the cache")
    q8 = _new(stream, (n, nq, d), torch.int8, dev) if q8 is None else q8
    mq = _new(stream, (n, nq), torch.int32, dev) if mq is None else mq
    kq = _new(stream, (n, nq), torch.int32, dev) if kq is None else kq
    kp = vp = 0
    if k_val is not None:
        if _unfit(k_val, torch.int16, n * cache.n_kv * d, index):
            _expect(w, "k_val", k_val, torch.int16, n * cache.n_kv * d, dev)
        kp = k_val.data_ptr()
    if v_val is not None:
        if _unfit(v_val, torch.int16, n * cache.n_kv * d, index):
            _expect(w, "v_val", v_val, torch.int16, n * cache.n_kv * d, dev)
        vp = v_val.data_ptr()
    if axes is None:
        rc = lib().detint_kv4_append(cache._ref, rope._ref, qkv.data_ptr(), stride, tok_seq.data_ptr(),
                                     tok_pos.data_ptr(), n, q8.data_ptr(), mq.data_ptr(), kq.data_ptr(), kp, vp, raw)
    else:
        rope_pos, axis = axes
        n_axes = rope_pos.size(0) if rope_pos.dim() == 2 else 1
        if _unfit(rope_pos, torch.int32, n_axes * n, index) or rope_pos.numel() != n_axes * n:
            raise ValueError(f"{w}: rope_pos: a contiguous int32 tensor [axes, {n}] on {dev} expected, got "
                             f"{rope_pos.dtype} {tuple(rope_pos.shape)} on {rope_pos.device}")
        ap = 0
        if axis is not None:
            if _unfit(axis, torch.uint8, rope._c.rot_dim // 2, index):
                _expect(w, "axis", axis, torch.uint8, rope._c.rot_dim // 2, dev)
            ap = axis.data_ptr()
        rc = lib().detint_kv4_append_axes(cache._ref, rope._ref, rope_pos.data_ptr(), ap, n_axes, qkv.data_ptr(), stride,
                                          tok_seq.data_ptr(), tok_pos.data_ptr(), n, q8.data_ptr(), mq.data_ptr(),
                                          kq.data_ptr(), kp, vp, raw)
    if rc:
        _check(rc, w)
    return q8, mq, kq


def detint_kv4_append(cache, rope, qkv, tok_seq, tok_pos, q8=None, mq=None, kq=None, k_val=None, v_val=None,
                      stream=None):
    """Norm, rotate and quantise the Q12 projections qkv [n_tok, (n_q + 2 n_kv)
    head_dim] (int32, rows may be strided) and append keys and values to the
    cache; returns (q8, mq, kq). k_val, v_val (int16 [n_tok, n_kv, head_dim])
    receive the cached integers where given."""
    return _kv4_append("detint_kv4_append", cache, rope, qkv, tok_seq, tok_pos, None, q8, mq, kq, k_val, v_val, stream)


def detint_kv4_append_axes(cache, rope, qkv, tok_seq, tok_pos, rope_pos, axis=None, q8=None, mq=None, kq=None,
                           k_val=None, v_val=None, stream=None):
    """detint_kv4_append with rotary positions rope_pos (int32 [n_tok] or [axes,
    n_tok], 1 to 4 axes) beside the places tok_pos in the cache; axis (uint8
    [rot_dim // 2]) names the axis of each rotated pair."""
    return _kv4_append("detint_kv4_append_axes", cache, rope, qkv, tok_seq, tok_pos, (rope_pos, axis), q8, mq, kq, k_val,
                       v_val, stream)


def detint_kv4_workspace(cache, n_tok: int, max_len: int) -> int:
    """Bytes of workspace for every detint_kv4_decode of up to n_tok tokens and
    max_len keys; 0 for most sizes."""
    w, n = "detint_kv4_workspace", C.c_longlong(0)
    if n_tok >> 31 or max_len >> 31:                     # (would be cut to 32 bits on the way)
        raise DetintError(1, w, f"n_tok {n_tok} or max_len {max_len} out of range")
    _kv4_current(w, cache)
    _check(lib().detint_kv4_workspace(cache._ref, int(n_tok), int(max_len), C.byref(n)), w)
    return int(n.value)


def _kv4_out(w, cache, n, max_len, window, out, stream):
    torch, width = cache._torch, cache.n_q * cache.head_dim
    if max_len >> 31 or window >> 31:                    # (would be cut to 32 bits on the way)
        raise DetintError(1, w, f"max_len {max_len} or window {window} out of range")
    if out is None:
        return _new(stream, (n, width), torch.int32, cache.device), width
    return out, _row_stride(w, "out", out, torch.int32, n, width, cache._index)


def detint_kv4_decode(cache, q8, mq, kq, tok_seq, tok_pos, max_len: int, window: int = 0, out=None,
                      workspace=None, stream=None):
    """Attention of single tokens over the cache (detint_kv4_decode): int32 Q12
    rows [n_tok, n_q head_dim]. workspace: a cuda uint8 tensor of the bytes that
    detint_kv4_workspace gives for these or larger sizes (made here when it is
    needed and not given)."""
    w = "detint_kv4_decode"
    n, raw = _kv4_call(w, cache, q8, mq, kq, tok_seq, tok_pos, stream)
    out, stride = _kv4_out(w, cache, n, max_len, window, out, stream)
    ws = size = 0
    if workspace is not None:
        if workspace.get_device() != cache._index or not workspace.is_contiguous():
            raise ValueError(f"{w}: workspace: a contiguous tensor on {cache.device} expected")
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = lib().detint_kv4_decode(cache._ref, q8.data_ptr(), mq.data_ptr(), kq.data_ptr(), tok_seq.data_ptr(),
                                 tok_pos.data_ptr(), n, max_len, window, out.data_ptr(), stride, ws, size, raw)
    if rc and workspace is None:
        size = detint_kv4_workspace(cache, n, max_len)    # refused for want of one?
        if size:
            workspace = _new(stream, size, cache._torch.uint8, cache.device)
            return detint_kv4_decode(cache, q8, mq, kq, tok_seq, tok_pos, max_len, window, out, workspace, stream)
    if rc:
        _check(rc, w)
    return out


def detint_kv4_prefill(cache, q8, mq, kq, tok_seq, tok_pos, max_len: int, window: int = 0, out=None, stream=None):
    """The attention of detint_kv4_decode, bit for bit, for blocks of tokens of
    the same sequence (tokens of a sequence stand together)."""
    w = "detint_kv4_prefill"
    n, raw = _kv4_call(w, cache, q8, mq, kq, tok_seq, tok_pos, stream)
    out, stride = _kv4_out(w, cache, n, max_len, window, out, stream)
    rc = lib().detint_kv4_prefill(cache._ref, q8.data_ptr(), mq.data_ptr(), kq.data_ptr(), tok_seq.data_ptr(),
                                  tok_pos.data_ptr(), n, max_len, window, out.data_ptr(), stride, raw)
    if rc:
        _check(rc, w)
    return out


def _kv4_weight(w, cache, weight):
    need = cache.n_blocks * cache.n_kv * 64
    if _unfit(weight, cache._torch.int64, need, cache._index):
        _expect(w, "weight", weight, cache._torch.int64, need, cache.device)
    return weight.data_ptr()


def _kv4_weigh(w, fn, cache, q8, mq, kq, tok_seq, tok_pos, max_len, weight, window, stream):
    n, raw = _kv4_call(w, cache, q8, mq, kq, tok_seq, tok_pos, stream)
    if max_len >> 31 or window >> 31:                    # (would be cut to 32 bits on the way)
        raise DetintError(1, w, f"max_len {max_len} or window {window} out of range")
    rc = fn(cache._ref, q8.data_ptr(), mq.data_ptr(), kq.data_ptr(), tok_seq.data_ptr(), tok_pos.data_ptr(), n, max_len,
            window, _kv4_weight(w, cache, weight), raw)
    if rc:
        _check(rc, w)
    return weight


def detint_kv4_weigh(cache, q8, mq, kq, tok_seq, tok_pos, max_len: int, weight, window: int = 0, stream=None):
    """Add the attention probabilities (Q24) of single tokens to the weights
    (int64 [n_blocks, n_kv, 64]) of the keys that they see; returns weight."""
    return _kv4_weigh("detint_kv4_weigh", lib().detint_kv4_weigh, cache, q8, mq, kq, tok_seq, tok_pos, max_len, weight,
                      window, stream)


def detint_kv4_weigh_block(cache, q8, mq, kq, tok_seq, tok_pos, max_len: int, weight, window: int = 0, stream=None):
    """The weights of detint_kv4_weigh, bit for bit, for blocks of tokens of the
    same sequence (tokens of a sequence stand together)."""
    return _kv4_weigh("detint_kv4_weigh_block", lib().detint_kv4_weigh_block, cache, q8, mq, kq, tok_seq, tok_pos,
                      max_len, weight, window, stream)


def _fit_all(w, named, index, device):
    """Words the error of the first tensor that does not fit: (name, tensor, type, elements)."""
    for name, t, dtype, numel in named:
        if t is not None and _unfit(t, dtype, numel, index):
            _expect(w, name, t, dtype, numel, device)


def detint_kv4_evict(cache, weight, seq, lens, max_len: int, keep: int, new_table, sinks: int = 0, recent: int = 0,
                     kept=None, stream=None):
    """Move the `keep` tokens of the largest weights (the first `sinks` and last
    `recent` ones always) of every kv head of sequences seq (int32 [n], rows of
    the block table) with lens (int32 [n]) tokens to the pages new_table (int32
    [n, ceil(keep / 64)]); returns their old places, int32 [n, n_kv, keep] with -1
    behind the last."""
    w, n, index, torch = "detint_kv4_evict", seq.numel(), cache._index, cache._torch
    i32 = torch.int32
    if torch._C._cuda_getDevice() != index:
        _kv4_current(w, cache)                           # words the error
    if max_len >> 31 or keep >> 31 or sinks >> 31 or recent >> 31 or keep < 1:
        raise DetintError(1, w, "max_len, keep, sinks or recent out of range")
    if kept is None:
        kept = _new(stream, (n, cache.n_kv, keep), i32, cache.device)
    room, places = n * ((keep + 63) >> 6), n * cache.n_kv * keep
    if _unfit(seq, i32, n, index) or _unfit(lens, i32, n, index) or _unfit(new_table, i32, room, index) or \
            _unfit(kept, i32, places, index):
        _fit_all(w, (("seq", seq, i32, n), ("lens", lens, i32, n), ("new_table", new_table, i32, room),
                     ("kept", kept, i32, places)), index, cache.device)
    rc = lib().detint_kv4_evict(cache._ref, _kv4_weight(w, cache, weight), seq.data_ptr(), lens.data_ptr(), n, max_len, keep,
                                sinks, recent, new_table.data_ptr(), kept.data_ptr(),
                                torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, w)
    return kept


def detint_kv4_copy(cache, src, dst, weight=None, stream=None):
    """Copy whole pages src[i] to dst[i] (int32 lists, a negative entry: none),
    with their weights where given."""
    w, n, index, torch = "detint_kv4_copy", src.numel(), cache._index, cache._torch
    i32 = torch.int32
    if torch._C._cuda_getDevice() != index:
        _kv4_current(w, cache)                           # words the error
    if _unfit(src, i32, n, index) or _unfit(dst, i32, n, index):
        _fit_all(w, (("src", src, i32, n), ("dst", dst, i32, n)), index, cache.device)
    rc = lib().detint_kv4_copy(cache._ref, src.data_ptr(), dst.data_ptr(), n,
                               0 if weight is None else _kv4_weight(w, cache, weight),
                               torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, w)


# ---------------------------------------------------------------- beam search
def _beam_device(w, torch, t):
    """The index of a cuda tensor's device, which has to be the current one."""
    index = t.get_device()
    if index < 0 or torch._C._cuda_getDevice() != index:
        raise ValueError(f"{w}: cuda tensors on the current device expected, got one on {t.device}")
    return index


def detint_beam_workspace(rows: int, n: int, n_out: int) -> int:
    """Bytes of workspace for detint_beam_select of up to `rows` rows (groups
    times beams) of n logits and n_out continuations."""
    w, v = "detint_beam_workspace", C.c_longlong(0)
    if rows >> 31 or n >> 31 or n_out >> 31:             # (would be cut to 32 bits on the way)
        raise DetintError(1, w, f"rows {rows}, n {n} or n_out {n_out} out of range")
    _check(lib().detint_beam_workspace(int(rows), int(n), int(n_out), C.byref(v)), w)
    return int(v.value)


def detint_beam_select(logits, scores, n_out: int, done=None, end_id: int = -1, out=None, workspace=None, stream=None):
    """The n_out best continuations of each group of beams, best first: (parent,
    token, score, done), int32 and for the scores int64 tensors [groups, n_out].
    logits: int32 Q16 [groups * beams, n] (rows may be strided), -2^31 masks a
    token; scores: int64 [groups, beams], Q16 (-2^63: no beam); done: int32
    [groups, beams] or None. out: the four tensors, workspace: a uint8 tensor of
    detint_beam_workspace bytes (made here where they are not given)."""
    import torch
    w, i32, i64 = "detint_beam_select", torch.int32, torch.int64
    index = _beam_device(w, torch, logits)
    if scores.dim() != 2 or logits.dim() != 2 or logits.size(0) != scores.numel():
        raise ValueError(f"{w}: logits [groups * beams, n] and scores [groups, beams] expected, got "
                         f"{tuple(logits.shape)} and {tuple(scores.shape)}")
    groups, beams = scores.shape
    rows, n = logits.shape
    stride = _row_stride(w, "logits", logits, i32, rows, n, index)
    if n_out < 1 or n_out >> 31 or not -(1 << 31) <= end_id < 1 << 31:
        raise DetintError(1, w, f"n_out {n_out} or end_id {end_id} out of range")
    m = groups * n_out
    if out is None:
        shape, dev = (groups, n_out), logits.device
        if stream is None:
            parent, token, score, end = (torch.empty(shape, dtype=i32, device=dev), torch.empty(shape, dtype=i32, device=dev),
                                         torch.empty(shape, dtype=i64, device=dev), torch.empty(shape, dtype=i32, device=dev))
        else:
            parent, token, end = (_new(stream, shape, i32, dev) for _ in range(3))
            score = _new(stream, shape, i64, dev)
    else:
        parent, token, score, end = out
    if workspace is None:
        workspace = _new(stream, detint_beam_workspace(rows, n, n_out), torch.uint8, logits.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"{w}: workspace: a contiguous tensor on {logits.device} expected")
    if _unfit(scores, i64, rows, index) or done is not None and _unfit(done, i32, rows, index) or \
            out is not None and (_unfit(parent, i32, m, index) or _unfit(token, i32, m, index) or
                                 _unfit(score, i64, m, index) or _unfit(end, i32, m, index)):
        _fit_all(w, (("scores", scores, i64, rows), ("done", done, i32, rows), ("parent", parent, i32, m),
                     ("token", token, i32, m), ("score", score, i64, m), ("done", end, i32, m)), index, logits.device)
    rc = lib().detint_beam_select(logits.data_ptr(), stride, n, scores.data_ptr(), 0 if done is None else done.data_ptr(), groups,
                                  beams, end_id, n_out, parent.data_ptr(), token.data_ptr(), score.data_ptr(), end.data_ptr(),
                                  workspace.data_ptr(), workspace.nbytes,
                                  torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, w)
    return parent, token, score, end


def detint_beam_reorder(block_table, parent, lens, out=None, src=None, dst=None, stream=None):
    """Give every beam its parent's pages: block_table int32 [groups * beams,
    max_blocks], parent int32 [groups, beams] (a beam that goes on as it is names
    itself; outside 0..beams - 1 the row holds no beam any more, and the tokens of
    its last page are lost), lens int32 [groups]; out: another table, or None for
    block_table itself. Returns (src, dst), int32 [groups, beams]: the pages that
    detint_kv4_copy has to copy in every layer."""
    import torch
    w, i32 = "detint_beam_reorder", torch.int32
    index = _beam_device(w, torch, block_table)
    if parent.dim() != 2 or block_table.dim() != 2 or block_table.size(0) != parent.numel():
        raise ValueError(f"{w}: parent [groups, beams] and block_table [groups * beams, max_blocks] expected, got "
                         f"{tuple(parent.shape)} and {tuple(block_table.shape)}")
    groups, beams = parent.shape
    rows, size, out = groups * beams, block_table.numel(), block_table if out is None else out
    src = _new(stream, (groups, beams), i32, block_table.device) if src is None else src
    dst = _new(stream, (groups, beams), i32, block_table.device) if dst is None else dst
    if _unfit(block_table, i32, size, index) or _unfit(out, i32, size, index) or _unfit(parent, i32, rows, index) or \
            _unfit(lens, i32, groups, index) or _unfit(src, i32, rows, index) or _unfit(dst, i32, rows, index):
        _fit_all(w, (("block_table", block_table, i32, size), ("out", out, i32, size), ("parent", parent, i32, rows),
                     ("lens", lens, i32, groups), ("src", src, i32, rows), ("dst", dst, i32, rows)), index, block_table.device)
    rc = lib().detint_beam_reorder(block_table.data_ptr(), out.data_ptr(), block_table.size(1), parent.data_ptr(), lens.data_ptr(),
                                   groups, beams, src.data_ptr(), dst.data_ptr(),
                                   torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, w)
    return src, dst


def chain_hash(rows, prev: bytes | None = None) -> bytes:
    """SHA-256 chain over int32 rows (little-endian) from 32 zero bytes
    (DetLLM README, "Demo": the per-step logits chain hash)."""
    h = prev if prev is not None else b"\0" * 32
    for r in rows:
        h = hashlib.sha256(h + np.ascontiguousarray(r, dtype="<i4").tobytes()).digest()
    return h


class Model:
    """A loaded integer model on the current CUDA device (detint_load; kv_bits 4:
    detint_load_kv with the 4-bit K/V cache)."""

    def __init__(self, path: str, max_batch: int, max_ctx: int, stream=None, kv_bits: int = 8):
        import torch
        self.torch = torch
        self.stream = stream if stream is not None else torch.cuda.Stream()
        h = C.c_void_p()
        _check(lib().detint_load_kv(path.encode(), int(max_batch), int(max_ctx), int(kv_bits),
                                    self.stream.cuda_stream, C.byref(h)), "detint_load")
        self._h = h
        self.kv_bits = int(kv_bits)
        info = np.zeros(16, np.int32)
        _check(lib().detint_model_info(self._h, info.ctypes.data_as(C.POINTER(C.c_int32))),
               "detint_model_info")
        (self.n_layers, self.hidden, self.n_q, self.n_kv, self.head_dim, self.ffn, self.vocab,
         self.max_pos, self.qk_norm, self.max_batch, self.max_ctx) = [int(v) for v in info[:11]]

    def close(self):
        if getattr(self, "_h", None):
            lib().detint_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_graph(self, enable: bool):
        _check(lib().detint_set_graph(self._h, int(bool(enable))), "detint_set_graph")

    def set_fused_decode(self, enable: bool):
        _check(lib().detint_set_option(self._h, 1, int(bool(enable))), "detint_set_option")

    def set_staged_decode(self, enable: bool):
        _check(lib().detint_set_option(self._h, 3, int(bool(enable))), "detint_set_option")

    def set_persistent(self, enable: bool):
        _check(lib().detint_set_option(self._h, 4, int(bool(enable))), "detint_set_option")

    def set_wait_test(self, polls: int):
        """While polls > 0, the one-launch decode step's final wait expects a
        tag no CTA writes and gives up after `polls` polls (status slot 6)."""
        _check(lib().detint_set_option(self._h, 5, int(polls)), "detint_set_option")

    def set_tc_prefill(self, enable: bool):
        _check(lib().detint_set_option(self._h, 2, int(bool(enable))), "detint_set_option")

    def reset_seq(self, seq_id: int):
        _check(lib().detint_reset_seq(self._h, int(seq_id)), "detint_reset_seq")

    def fork_seq(self, src: int, dst: int, n_tokens: int):
        """dst starts with src's first n_tokens positions (shared KV blocks)."""
        _check(lib().detint_fork_seq(self._h, int(src), int(dst), int(n_tokens), self.stream.cuda_stream),
               "detint_fork_seq")

    def reorder_seqs(self, seq_ids, parents):
        """seq_ids[i] becomes what seq_ids[parents[i]] was (shared KV blocks)."""
        seq, par = _i32(seq_ids), _i32(parents)
        if seq.size != par.size:
            raise ValueError("reorder_seqs: one parent for each sequence expected")
        _check(lib().detint_reorder_seqs(self._h, seq.size, seq.ctypes.data_as(C.POINTER(C.c_int32)),
                                         par.ctypes.data_as(C.POINTER(C.c_int32)), self.stream.cuda_stream),
               "detint_reorder_seqs")

    def seq_len(self, seq_id: int) -> int:
        v = C.c_int32()
        _check(lib().detint_seq_len(self._h, int(seq_id), C.byref(v)), "detint_seq_len")
        return int(v.value)

    def status(self) -> np.ndarray:
        flags = np.zeros(8, np.int32)
        lib().detint_status(self._h, flags.ctypes.data_as(C.POINTER(C.c_int32)),
                            self.stream.cuda_stream)
        return flags

    def prefill(self, seq_ids, tokens, cu_lens, logits=None, next_tok=None):
        """tokens: int32 cuda tensor (ragged, concatenated); cu_lens: host ints."""
        torch = self.torch
        seq = _i32(seq_ids)
        cu = _i32(cu_lens)
        n = seq.size
        if next_tok is None:
            next_tok = torch.empty(n, dtype=torch.int32, device=tokens.device)
        _check(lib().detint_prefill(self._h, n, seq.ctypes.data_as(C.POINTER(C.c_int32)),
                                    cu.ctypes.data_as(C.POINTER(C.c_int32)), _ptr(tokens),
                                    _ptr(logits), _ptr(next_tok), self.stream.cuda_stream),
               "detint_prefill")
        return next_tok

    def decode_step(self, seq_ids, tok, logits=None, next_tok=None):
        torch = self.torch
        seq = _i32(seq_ids)
        if next_tok is None:
            next_tok = torch.empty(seq.size, dtype=torch.int32, device=tok.device)
        _check(lib().detint_decode_step(self._h, seq.size, seq.ctypes.data_as(C.POINTER(C.c_int32)),
                                        _ptr(tok), _ptr(logits), _ptr(next_tok),
                                        self.stream.cuda_stream), "detint_decode_step")
        return next_tok

    def generate(self, prompts, max_new: int, seq_ids=None, keep_logits: bool = True, sampling=None):
        """Decode a ragged batch of prompts (lists of ids), greedy by default.

        Returns (tokens [B][max_new] int32 numpy, logits rows per step (list of
        [B, V] numpy arrays) or chain-hash digests per row when keep_logits is
        "hash"). Step 0 is the prefill's last-position logits (README, "Usage":
        generate(ids, max_new)). sampling: None (greedy) or a dict of
        detint_sample parameters (seed, inv_temp, top_k, top_p) or one dict per
        row; step s of row b draws with counter = s, so a row's tokens do not
        depend on the rest of the batch.
        """
        torch = self.torch
        B = len(prompts)
        seq_ids = list(range(B)) if seq_ids is None else list(seq_ids)
        dev = torch.device("cuda")
        cu = np.zeros(B + 1, np.int64)
        cu[1:] = np.cumsum([len(p) for p in prompts])
        flat = torch.tensor(np.concatenate([np.asarray(p, np.int32) for p in prompts]),
                            dtype=torch.int32, device=dev)
        logits = torch.empty((B, self.vocab), dtype=torch.int32, device=dev)
        tok = torch.empty(B, dtype=torch.int32, device=dev)
        toks = np.zeros((B, max_new), np.int32)
        rows = []
        hashes = [b"\0" * 32] * B
        if sampling is not None:
            per_row = sampling if isinstance(sampling, (list, tuple)) else [sampling] * B
        with torch.cuda.stream(self.stream):
            self.prefill(seq_ids, flat, cu, logits, tok)
            for step in range(max_new):
                if step:
                    self.decode_step(seq_ids, tok, logits, tok)
                if sampling is not None:
                    detint_sample(logits, [dict(p, counter=step) for p in per_row], out=tok,
                                  stream=self.stream)
                lg = logits.cpu().numpy()
                toks[:, step] = tok.cpu().numpy()
                if keep_logits == "hash":
                    hashes = [chain_hash([lg[b]], hashes[b]) for b in range(B)]
                elif keep_logits:
                    rows.append(lg)
        self.stream.synchronize()
        return toks, (hashes if keep_logits == "hash" else rows)

    def beam_search(self, prompts, beams: int, max_new: int, end_id: int = -1, seq_ids=None):
        """The `beams` best continuations of each prompt by integer beam search.

        Returns (tokens [len(prompts)][beams][max_new] int32 numpy, scores
        [len(prompts)][beams] int64 numpy: log-probabilities in Q16), best first.
        A beam that chose end_id keeps its score and continues with end_id; a
        prompt's search stops early once all of its beams have. The beams of prompt g
        run on the empty sequences seq_ids[g * beams : (g + 1) * beams] (0, 1, ... by
        default) and share their common pages. Scores and tokens, and whether the
        contexts hold them, do not depend on the other prompts of the batch.
        """
        torch = self.torch
        G, dev = len(prompts), torch.device("cuda")
        if G < 1 or not 1 <= beams <= 64 or max_new < 1 or beams > self.vocab:
            raise ValueError("beam_search: at least one prompt and token, 1 to 64 beams expected")
        seq_ids = list(range(G * beams)) if seq_ids is None else list(seq_ids)
        if len(seq_ids) != G * beams:
            raise ValueError(f"beam_search: {G * beams} sequences expected, got {len(seq_ids)}")
        cu = np.zeros(G + 1, np.int64)
        cu[1:] = np.cumsum([len(p) for p in prompts])
        flat = torch.tensor(np.concatenate([np.asarray(p, np.int32) for p in prompts]), dtype=torch.int32, device=dev)
        toks = np.zeros((G, beams, max_new), np.int32)
        with torch.cuda.stream(self.stream):
            logits = torch.empty((G * beams, self.vocab), dtype=torch.int32, device=dev)
            ws = torch.empty(detint_beam_workspace(G * beams, self.vocab, beams), dtype=torch.uint8, device=dev)
            tok = torch.empty(G * beams, dtype=torch.int32, device=dev)
            self.prefill(seq_ids[::beams], flat, cu, logits, tok)
            # the prompts' rows: one beam of each group so far
            parent, token, scores, done = detint_beam_select(logits[:G], torch.zeros((G, 1), dtype=torch.int64, device=dev),
                                                             beams, None, end_id, workspace=ws)
            live, ids, out = np.arange(G), seq_ids, np.zeros((G, beams), np.int64)    # prompts that go on, their sequences
            for step in range(max_new):
                if step:
                    self.decode_step(ids, tok, logits, tok)
                    parent, token, scores, done = detint_beam_select(logits[:len(ids)], scores, beams, done if end_id >= 0 else None,
                                                                     end_id, workspace=ws)
                tok[:len(ids)].copy_(token.view(-1))
                par, new = parent.cpu().numpy(), token.cpu().numpy()
                toks[live] = np.take_along_axis(toks[live], par[:, :, None], 1)
                toks[live, :, step] = new
                over = done.cpu().numpy().all(1) if end_id >= 0 else np.zeros(len(live), bool)
                if step + 1 == max_new:
                    over[:] = True
                if over.any():
                    out[live[over]] = scores.cpu().numpy()[over]
                    toks[live[over], :, step + 1:] = max(end_id, 0)
                    if over.all():
                        break
                    # a finished prompt's beams take no more places of their contexts
                    at = torch.from_numpy(np.flatnonzero(~over)).to(dev)
                    scores, done, live, par = scores[at], done[at], live[~over], par[~over]
                    ids = [seq_ids[g * beams + b] for g in live for b in range(beams)]
                    tok[:len(ids)].copy_(token[at].view(-1))
                self.reorder_seqs(ids, (par + np.arange(len(live))[:, None] * beams).reshape(-1))
        self.stream.synchronize()
        return toks, out
