"""ctypes binding of libspecattn.so: argument marshalling only.

Function names follow the C ABI without the ``sa_`` prefix. Tensors are
torch tensors on the current CUDA device (bf16 data may be passed as
torch.bfloat16 or as int16/uint16 bit patterns); the stream defaults to
torch's current stream. Status codes other than SA_OK raise SpecAttnError.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from .build import LIB

STATUS = {
    0: "SA_OK", 1: "SA_ERR_ARG", 2: "SA_ERR_UNSUPPORTED", 3: "SA_ERR_PAGE_OOB",
    4: "SA_ERR_CUDA", 5: "SA_ERR_TIMEOUT", 6: "SA_ERR_WORKSPACE", 7: "SA_ERR_QLEN",
}


class SpecAttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({status_string(code)})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "num_pages",
        "max_pages_per_seq", "total_q", "max_q_len")]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    """The library this process loads: the in-tree build."""
    return LIB


def load_library() -> ctypes.CDLL:
    """Load the built library; fails loudly when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with speculative_decode_gb300.build.build() "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    I64 = ctypes.c_int64
    DP, RP = ctypes.POINTER(Dims), ctypes.POINTER(_RopeStruct)
    sig = {
        "sa_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "sa_device_sm_count": ([], ctypes.c_int),
        "sa_selftest_bounded_wait": ([ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
        "sa_kv_append": ([DP] + [P] * 8 + [P], ctypes.c_int),
        "sa_plan_create": ([DP, P, P, P, ctypes.POINTER(P)], ctypes.c_int),
        "sa_plan_destroy": ([P], None),
        "sa_plan_analyze": ([DP, P, P, P, I32, P, P, P, P], ctypes.c_int),
        "sa_plan_stats": ([P, P, P, P], ctypes.c_int),
        "sa_paged_attn_workspace_size": ([DP, P], SZ),
        "sa_paged_attn": ([DP, P, P, P, P, P, P, F, P, P, P, SZ, P, P], ctypes.c_int),
        "sa_paged_attn_kernel_count": ([DP, P], ctypes.c_int),
        "sa_paged_attn_noalloc": ([DP, P, P, P, P, P, P, F, P, P, P], ctypes.c_int),
        "sa_spec_verify_workspace_size": ([I32, I32, I32], SZ),
        "sa_spec_verify_greedy": ([P, P, P, I32, I32, I32, P, P, P, P, SZ, P, P], ctypes.c_int),
        "sa_spec_verify_greedy_advance": ([P, P, P, I32, I32, I32, P, P, P, P, P, P, P, SZ, P, P], ctypes.c_int),
        "sa_kv_append_q8": ([DP] + [P] * 11, ctypes.c_int),
        "sa_paged_attn_q8": ([DP, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P], ctypes.c_int),
        "sa_kv_append_q4": ([DP] + [P] * 11, ctypes.c_int),
        "sa_paged_attn_q4": ([DP, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P], ctypes.c_int),
        "sa_defrag_moves": ([DP, P, P, P, P, P, P], ctypes.c_int),
        "sa_defrag_apply": ([DP, P, P, P, I32, P, P], ctypes.c_int),
        "sa_defrag_apply_bytes": ([I32, ctypes.c_int64, P, P, P, I32, P, P], ctypes.c_int),
        "sa_qk_norm_rope": ([RP, I32, I32, I32, I32, P, I64, P, I64, P, P, I64, P, I64, P], ctypes.c_int),
        "sa_kv_append_rope": ([DP, RP, P, I64, P, I64, P, I64] + [P] * 9, ctypes.c_int),
        "sa_kv_append_rope_q8": ([DP, RP, P, I64, P, I64, P, I64] + [P] * 11, ctypes.c_int),
        "sa_kv_append_rope_q4": ([DP, RP, P, I64, P, I64, P, I64] + [P] * 11, ctypes.c_int),
        "sa_beam_select_workspace_size": ([I32, I32, I32, I32], SZ),
        "sa_beam_select": ([P, I64, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, SZ, P], ctypes.c_int),
        "sa_beam_select_bf16": ([P, I64, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, SZ, P], ctypes.c_int),
        "sa_beam_reorder": ([DP, I32] + [P] * 8, ctypes.c_int),
        "sa_beam_reorder_q8": ([DP, I32] + [P] * 10, ctypes.c_int),
        "sa_beam_reorder_q4": ([DP, I32] + [P] * 10, ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().sa_status_string(int(code)).decode()


def sm_count() -> int:
    return int(load_library().sa_device_sm_count())


def selftest_bounded_wait(err_flag, stream=None) -> None:
    """sa_selftest_bounded_wait: one CTA's bounded wait on an mbarrier that
    nothing completes; sets bit 1 << SA_ERR_TIMEOUT of err_flag."""
    _check(load_library().sa_selftest_bounded_wait(_ptr(err_flag), _stream(stream)),
           "sa_selftest_bounded_wait")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _current_stream_getter():
    """The address of torch's current stream: its raw getter, where torch has one,
    makes no Stream object (0.2 us of host time a call instead of 2.9)."""
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


_current_stream = None


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _current_stream_getter()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise SpecAttnError(rc, what)


def dims_for(num_seqs, num_q_heads, num_kv_heads, num_pages, max_pages_per_seq, total_q,
             max_q_len, head_dim=128, page_size=256) -> Dims:
    return Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                max_pages_per_seq, total_q, max_q_len)


def kv_append(dims: Dims, k_new, v_new, k_pages, v_pages, block_table, seq_lens, q_lens,
              err_flag=None, stream=None) -> None:
    rc = load_library().sa_kv_append(ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                                      _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                      _ptr(q_lens), _ptr(err_flag), _stream(stream))
    _check(rc, "sa_kv_append")


class Plan:
    """Shared-run plan (sa_plan_create) built from host copies of the tables."""

    def __init__(self, dims: Dims, block_table_host, seq_lens_host, q_lens_host):
        import numpy as np
        bt = np.ascontiguousarray(block_table_host, dtype=np.int32)
        sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
        ql = np.ascontiguousarray(q_lens_host, dtype=np.int32)
        self._h = ctypes.c_void_p()
        lib = load_library()
        rc = lib.sa_plan_create(ctypes.byref(dims), bt.ctypes.data, sl.ctypes.data, ql.ctypes.data,
                                ctypes.byref(self._h))
        _check(rc, "sa_plan_create")

    @property
    def handle(self) -> int:
        return self._h.value or 0

    def stats(self):
        r, m, p = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(load_library().sa_plan_stats(self._h, ctypes.byref(r), ctypes.byref(m),
                                            ctypes.byref(p)), "sa_plan_stats")
        return {"runs": r.value, "members": m.value, "pages": p.value}

    def close(self) -> None:
        if self._h.value:
            load_library().sa_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_analyze(dims: Dims, block_table_host, seq_lens_host, q_lens_host, sm_count_: int):
    """Host-only dry run of the planner: (skip_pages, run_slots, num_runs, num_tiles)."""
    import numpy as np
    bt = np.ascontiguousarray(block_table_host, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
    ql = np.ascontiguousarray(q_lens_host, dtype=np.int32)
    skip = np.zeros(dims.num_seqs, np.int32)
    slots = np.zeros(dims.num_seqs, np.int32)
    runs, tiles = ctypes.c_int32(), ctypes.c_int32()
    rc = load_library().sa_plan_analyze(ctypes.byref(dims), bt.ctypes.data, sl.ctypes.data,
                                        ql.ctypes.data, int(sm_count_), skip.ctypes.data,
                                        slots.ctypes.data, ctypes.byref(runs), ctypes.byref(tiles))
    _check(rc, "sa_plan_analyze")
    return skip, slots, runs.value, tiles.value


def paged_attn_workspace_size(dims: Dims, plan: Optional[Plan] = None) -> int:
    return int(load_library().sa_paged_attn_workspace_size(ctypes.byref(dims),
                                                           plan.handle if plan else None))


def paged_attn(dims: Dims, q, k_pages, v_pages, block_table, seq_lens, q_lens, scale: float, out,
               workspace, plan: Optional[Plan] = None, err_flag=None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    rc = load_library().sa_paged_attn(ctypes.byref(dims), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                      _ptr(block_table), _ptr(seq_lens), _ptr(q_lens),
                                      float(scale), _ptr(out), plan.handle if plan else None,
                                      _ptr(workspace), nbytes, _ptr(err_flag), _stream(stream))
    _check(rc, "sa_paged_attn")


def paged_attn_noalloc(dims: Dims, q, k_pages, v_pages, block_table, seq_lens, q_lens,
                       scale: float, out, err_flag=None, stream=None) -> None:
    """sa_paged_attn_noalloc: paged attention using the library's fixed 16 MiB
    scratch, for callers that cannot allocate device memory."""
    rc = load_library().sa_paged_attn_noalloc(ctypes.byref(dims), _ptr(q), _ptr(k_pages),
                                              _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                              _ptr(q_lens), float(scale), _ptr(out),
                                              _ptr(err_flag), _stream(stream))
    _check(rc, "sa_paged_attn_noalloc")


def paged_attn_kernel_count(dims: Dims, plan: Optional[Plan] = None) -> int:
    return int(load_library().sa_paged_attn_kernel_count(ctypes.byref(dims),
                                                         plan.handle if plan else None))


def spec_verify_workspace_size(num_seqs: int, k_max: int, vocab: int) -> int:
    return int(load_library().sa_spec_verify_workspace_size(num_seqs, k_max, vocab))


def spec_verify_greedy(logits, candidates, n_cand, accepted, next_tok, workspace, window=None,
                       err_flag=None, stream=None) -> None:
    B, k1, V = logits.shape
    nbytes = workspace.numel() * workspace.element_size()
    rc = load_library().sa_spec_verify_greedy(_ptr(logits), _ptr(candidates), _ptr(n_cand), B,
                                              k1 - 1, V, _ptr(accepted), _ptr(next_tok),
                                              _ptr(window), _ptr(workspace), nbytes,
                                              _ptr(err_flag), _stream(stream))
    _check(rc, "sa_spec_verify_greedy")


def spec_verify_greedy_advance(logits, candidates, n_cand, accepted, next_tok, window, seq_lens, q_lens,
                               n_cand_next, workspace, err_flag=None, stream=None) -> None:
    """spec_verify_greedy plus the next verify call's lengths (window,
    seq_lens and q_lens updated in place, n_cand_next written)."""
    B, k1, V = logits.shape
    nbytes = workspace.numel() * workspace.element_size()
    rc = load_library().sa_spec_verify_greedy_advance(
        _ptr(logits), _ptr(candidates), _ptr(n_cand), B, k1 - 1, V, _ptr(accepted), _ptr(next_tok),
        _ptr(window), _ptr(seq_lens), _ptr(q_lens), _ptr(n_cand_next), _ptr(workspace), nbytes,
        _ptr(err_flag), _stream(stream))
    _check(rc, "sa_spec_verify_greedy_advance")


def defrag_moves(dims: Dims, block_table_host, seq_lens_host):
    """Host compaction plan: (new_table, moves [n, 2] as (from, to), n_live)."""
    import numpy as np
    bt = np.ascontiguousarray(block_table_host, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
    new = np.empty_like(bt)
    moves = np.empty((max(dims.num_pages, 1), 2), np.int32)
    n_moves, n_live = ctypes.c_int32(), ctypes.c_int32()
    rc = load_library().sa_defrag_moves(ctypes.byref(dims), bt.ctypes.data, sl.ctypes.data,
                                        new.ctypes.data, moves.ctypes.data, ctypes.byref(n_moves),
                                        ctypes.byref(n_live))
    _check(rc, "sa_defrag_moves")
    return new, moves[:n_moves.value].copy(), n_live.value


def defrag_apply(dims: Dims, k_pages, v_pages, moves, n_moves: int, err_flag=None, stream=None) -> None:
    """Make the moves (a device int32 [n, 2] tensor) on both page pools."""
    rc = load_library().sa_defrag_apply(ctypes.byref(dims), _ptr(k_pages), _ptr(v_pages), _ptr(moves),
                                        int(n_moves), _ptr(err_flag), _stream(stream))
    _check(rc, "sa_defrag_apply")


def kv_append_q8(dims: Dims, k_new, v_new, k_codes, v_codes, k_scales, v_scales, block_table,
                 seq_lens, q_lens, err_flag=None, stream=None) -> None:
    """kv_append into int8 pages (codes int8 [pages, Hkv, 256, 128], scales fp32 [pages, Hkv, 256])."""
    rc = load_library().sa_kv_append_q8(ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(k_codes),
                                        _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
                                        _ptr(seq_lens), _ptr(q_lens), _ptr(err_flag), _stream(stream))
    _check(rc, "sa_kv_append_q8")


def paged_attn_q8(dims: Dims, q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, q_lens,
                  scale: float, out, workspace, err_flag=None, stream=None) -> None:
    """paged_attn over int8 pages; the workspace is paged_attn_workspace_size(dims)."""
    rc = load_library().sa_paged_attn_q8(ctypes.byref(dims), _ptr(q), _ptr(k_codes), _ptr(v_codes),
                                         _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
                                         _ptr(seq_lens), _ptr(q_lens), float(scale), _ptr(out),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _ptr(err_flag), _stream(stream))
    _check(rc, "sa_paged_attn_q8")


def kv_append_q4(dims: Dims, k_new, v_new, k_codes, v_codes, k_scales, v_scales, block_table,
                 seq_lens, q_lens, err_flag=None, stream=None) -> None:
    """kv_append into int4 pages (nibbles uint8 [pages, Hkv, 256, 64], scales fp32 [pages, Hkv, 256])."""
    rc = load_library().sa_kv_append_q4(ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(k_codes),
                                        _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
                                        _ptr(seq_lens), _ptr(q_lens), _ptr(err_flag), _stream(stream))
    _check(rc, "sa_kv_append_q4")


def paged_attn_q4(dims: Dims, q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, q_lens,
                  scale: float, out, workspace, err_flag=None, stream=None) -> None:
    """paged_attn over int4 pages; the workspace is paged_attn_workspace_size(dims)."""
    rc = load_library().sa_paged_attn_q4(ctypes.byref(dims), _ptr(q), _ptr(k_codes), _ptr(v_codes),
                                         _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
                                         _ptr(seq_lens), _ptr(q_lens), float(scale), _ptr(out),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _ptr(err_flag), _stream(stream))
    _check(rc, "sa_paged_attn_q4")


def defrag_apply_bytes(num_pages: int, page_bytes: int, pool_a, pool_b, moves, n_moves: int,
                       err_flag=None, stream=None) -> None:
    """Make the moves on two pools paged alike (page p = bytes [p * page_bytes, (p + 1) * page_bytes))."""
    rc = load_library().sa_defrag_apply_bytes(int(num_pages), int(page_bytes), _ptr(pool_a), _ptr(pool_b),
                                              _ptr(moves), int(n_moves), _ptr(err_flag), _stream(stream))
    _check(rc, "sa_defrag_apply_bytes")


class _Types:
    """torch dtypes by what the C ABI calls them, and the device that is current
    (torch is imported with the first call that needs it)."""

    def __init__(self):
        import torch
        self.bf16 = (torch.bfloat16, torch.int16, torch.uint16)  # values or bit patterns
        self.f32 = (torch.float32,)
        self.int32 = torch.int32
        self.i32 = (torch.int32,)
        self.i8 = (torch.int8,)
        self.u8 = (torch.uint8,)
        # no device: no tensor is on it, and every call refuses its tensors
        self.here = (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device) if torch.cuda.is_available() \
            else lambda: -2


_types_made = None


def _types() -> _Types:
    global _types_made
    if _types_made is None:
        _types_made = _Types()
    return _types_made


def _refuse(t, name: str, dtypes, here: int, shape=None) -> None:
    if t is None:
        raise ValueError(f"{name} is missing")
    if not t.is_cuda or t.dtype not in dtypes:
        raise ValueError(f"{name}: a CUDA tensor of {dtypes[0]} is wanted, got {t.dtype} on {t.device}")
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, strides {t.stride()}" +
                     (f", wanted {tuple(shape)}" if shape is not None else "") + ", packed")


def _tensor(t, name: str, dtypes, here: int, shape=None) -> int:
    """Address of a packed tensor of one of these dtypes (and of that shape) on the current device."""
    if (t is None or t.dtype not in dtypes or t.get_device() != here or not t.is_contiguous() or
            (shape is not None and t.shape != shape)):
        _refuse(t, name, dtypes, here, shape)
    return t.data_ptr()


def _ints(t, name: str, here: int, count: int) -> int:
    """Address of packed int32 values, `count` of them (the attributes that cost a call least)."""
    if t is None or t.dtype is not _types_made.int32 or t.get_device() != here or t.numel() != count or \
            not t.is_contiguous():
        _refuse(t, name, _types_made.i32, here, (count,))
    return t.data_ptr()


def _heads(t, name: str, tokens: int, heads: int, here: int):
    """(address, token stride) of bf16 rows [tokens, heads, 128] whose heads are packed in their token."""
    bf16 = _types_made.bf16
    if t is None or t.get_device() != here or t.dtype not in bf16 or t.shape != (tokens, heads, 128):
        _refuse(t, name, bf16, here, (tokens, heads, 128))
    step, head, value = t.stride()
    if tokens and (value != 1 or (head != 128 and heads > 1)):
        _refuse(t, name, bf16, here, (tokens, heads, 128))
    return t.data_ptr(), (step if tokens > 1 else heads * 128)


def _here() -> int:
    """The current device: its context takes the launch, so a call's tensors have to be on it."""
    return (_types_made or _types()).here()


class Rope:
    """Norm and rotation of query and key heads (sa_rope): frequencies fp32
    [rotary_dim / 2], weights fp32 [128] or None for no norm. Made once for a
    model's layer; it keeps its tensors."""

    def __init__(self, inv_freq=None, rotary_dim=128, interleaved=False, q_weight=None, k_weight=None, eps=1e-6):
        f32 = _types().f32
        tensors = [(inv_freq, "inv_freq", (rotary_dim // 2,)), (q_weight, "q_weight", (128,)), (k_weight, "k_weight", (128,))]
        if inv_freq is None and rotary_dim:
            raise ValueError("inv_freq is missing")
        for t, name, _ in tensors:
            if t is not None and not t.is_cuda:
                raise ValueError(f"{name}: a CUDA tensor is wanted, got one on {t.device}")
        here = self._device = _here() if any(t is not None for t, _, _ in tensors) else None
        self._struct = _RopeStruct(*[None if t is None else _tensor(t, name, f32, here, shape) for t, name, shape in tensors],
                                   eps, rotary_dim, 1 if interleaved else 0)
        self._kept = (inv_freq, q_weight, k_weight)
        self._ref = ctypes.byref(self._struct)

    def _on(self, here: int):
        """The struct, for a call on this device."""
        if self._device is not None and self._device != here:
            raise ValueError(f"the Rope's tensors are on cuda:{self._device}, the current device is cuda:{here}")
        return self._ref


def qk_norm_rope(rope: Rope, q, k, positions, q_out, k_out, stream=None) -> None:
    """sa_qk_norm_rope: q [tokens, heads, 128] -> q_out and k -> k_out, normalised
    and rotated. q and k may be views with any token stride (a multiple of 8
    values); q with q_out, or k with k_out, may be None."""
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("q with q_out, k with k_out, or both are wanted")
    here = _here()
    n = (k if q is None else q).shape[0]
    hq = hk = qs = qos = ks = kos = 0
    qp = qo = kp = ko = None
    if q is not None:
        hq = q.shape[1]
        qp, qs = _heads(q, "q", n, hq, here)
        qo, qos = _heads(q_out, "q_out", n, hq, here)
    if k is not None:
        hk = k.shape[1]
        kp, ks = _heads(k, "k", n, hk, here)
        ko, kos = _heads(k_out, "k_out", n, hk, here)
    pos = _ints(positions, "positions", here, n)
    rc = load_library().sa_qk_norm_rope(rope._on(here), n, hq, hk, 128, qp, qs, kp, ks, pos, qo, qos, ko, kos,
                                        _stream(stream))
    if rc:
        _check(rc, "sa_qk_norm_rope")


def _pools(dims: Dims, here: int, k_pages, v_pages):
    """Addresses of bf16 page pools."""
    bf16, shape = _types_made.bf16, (dims.num_pages, dims.num_kv_heads, 256, 128)
    return _tensor(k_pages, "k_pages", bf16, here, shape), _tensor(v_pages, "v_pages", bf16, here, shape)


def _code_pools(dims: Dims, here: int, dtypes, row: int, k_codes, v_codes, k_scales, v_scales):
    """Addresses of code pools (rows of `row` bytes) and their scales."""
    f32, rows = _types_made.f32, (dims.num_pages, dims.num_kv_heads, 256)
    codes = (*rows, row)
    return (_tensor(k_codes, "k_codes", dtypes, here, codes), _tensor(v_codes, "v_codes", dtypes, here, codes),
            _tensor(k_scales, "k_scales", f32, here, rows), _tensor(v_scales, "v_scales", f32, here, rows))


def _append_rope(call, what, here, dims, rope, q, k_new, v_new, q_out, pools, block_table, seq_lens, q_lens, positions,
                 err_flag, stream) -> None:
    n, hkv, B = dims.total_q, dims.num_kv_heads, dims.num_seqs
    if q is None and q_out is None:
        qp, qs, qo = None, 0, None
    else:
        hq = dims.num_q_heads
        qp, qs = _heads(q, "q", n, hq, here)
        qo = _tensor(q_out, "q_out", _types_made.bf16, here, (n, hq, 128))
    kp, ks = _heads(k_new, "k_new", n, hkv, here)
    vp, vs = _heads(v_new, "v_new", n, hkv, here)
    rc = call(ctypes.byref(dims), rope._on(here), qp, qs, kp, ks, vp, vs, qo, *pools,
              _tensor(block_table, "block_table", _types_made.i32, here, (B, dims.max_pages_per_seq)),
              _ints(seq_lens, "seq_lens", here, B), _ints(q_lens, "q_lens", here, B),
              None if positions is None else _ints(positions, "positions", here, n),
              None if err_flag is None else _ints(err_flag, "err_flag", here, 1), _stream(stream))
    if rc:
        _check(rc, what)


def kv_append_rope(dims: Dims, rope: Rope, q, k_new, v_new, q_out, k_pages, v_pages, block_table, seq_lens, q_lens,
                   positions=None, err_flag=None, stream=None) -> None:
    """sa_kv_append_rope: kv_append with the keys normalised and rotated on the
    way, and q -> q_out for paged_attn (q and q_out may be None). q, k_new and
    v_new may be views with any token stride (a multiple of 8 values)."""
    here = _here()
    _append_rope(load_library().sa_kv_append_rope, "sa_kv_append_rope", here, dims, rope, q, k_new, v_new, q_out,
                 _pools(dims, here, k_pages, v_pages), block_table, seq_lens, q_lens, positions, err_flag, stream)


def kv_append_rope_q8(dims: Dims, rope: Rope, q, k_new, v_new, q_out, k_codes, v_codes, k_scales, v_scales,
                      block_table, seq_lens, q_lens, positions=None, err_flag=None, stream=None) -> None:
    """kv_append_rope into int8 pages (pools as in kv_append_q8)."""
    here = _here()
    _append_rope(load_library().sa_kv_append_rope_q8, "sa_kv_append_rope_q8", here, dims, rope, q, k_new, v_new, q_out,
                 _code_pools(dims, here, _types_made.i8, 128, k_codes, v_codes, k_scales, v_scales), block_table, seq_lens,
                 q_lens, positions, err_flag, stream)


def kv_append_rope_q4(dims: Dims, rope: Rope, q, k_new, v_new, q_out, k_codes, v_codes, k_scales, v_scales,
                      block_table, seq_lens, q_lens, positions=None, err_flag=None, stream=None) -> None:
    """kv_append_rope into int4 pages (pools as in kv_append_q4)."""
    here = _here()
    _append_rope(load_library().sa_kv_append_rope_q4, "sa_kv_append_rope_q4", here, dims, rope, q, k_new, v_new, q_out,
                 _code_pools(dims, here, _types_made.u8, 64, k_codes, v_codes, k_scales, v_scales), block_table, seq_lens,
                 q_lens, positions, err_flag, stream)


def beam_select_workspace_size(num_groups: int, beam_width: int, vocab: int, num_select: int) -> int:
    return int(load_library().sa_beam_select_workspace_size(num_groups, beam_width, vocab, num_select))


def beam_select(logits, scores, tokens, parents, scores_out, workspace, finished=None, finished_out=None,
                eos_token: int = -1, stream=None) -> None:
    """sa_beam_select (fp32 logits) or sa_beam_select_bf16 (bf16 logits): the best
    continuations of every group. logits [groups, beams, vocab] may be a view
    whose rows are evenly spaced (a padded vocabulary); scores and finished
    [groups, beams]; the outputs [groups, picks]."""
    here, types = _here(), _types_made
    wide = logits.dtype in types.f32
    if logits.dim() != 3 or logits.get_device() != here or not (wide or logits.dtype in types.bf16):
        raise ValueError(f"logits: fp32 or bf16 values [groups, beams, vocab] on cuda:{here} are wanted, got "
                         f"{logits.dtype} {tuple(logits.shape)} on {logits.device}")
    B, W, V = logits.shape
    group, row, value = logits.stride()
    if W == 1:
        row = group
    if (V > 1 and value != 1) or (B > 1 and group != W * row):
        raise ValueError(f"logits: packed values and evenly spaced rows are wanted, strides {logits.stride()}")
    if B * W <= 1:
        row = V
    K = tokens.shape[-1]
    picks, beams, f32 = (B, K), (B, W), types.f32
    sc = _tensor(scores, "scores", f32, here, beams)
    fi = None if finished is None else _ints(finished, "finished", here, B * W)
    to = _tensor(tokens, "tokens", types.i32, here, picks)
    pa = _tensor(parents, "parents", types.i32, here, picks)
    so = _tensor(scores_out, "scores_out", f32, here, picks)
    fo = None if finished_out is None else _ints(finished_out, "finished_out", here, B * K)
    ws = _tensor(workspace, "workspace", types.u8, here)
    lib = load_library()
    rc = (lib.sa_beam_select if wide else lib.sa_beam_select_bf16)(
        logits.data_ptr(), row, sc, fi, B, W, V, K, eos_token, to, pa, so, fo, ws, workspace.numel(), _stream(stream))
    if rc:
        _check(rc, "sa_beam_select" if wide else "sa_beam_select_bf16")


def _beam_reorder(call, what, here, dims, beam_width, parents, block_table, seq_lens, block_table_out, pools, err_flag,
                  stream) -> None:
    i32, B = _types_made.i32, dims.num_seqs
    table = (B, dims.max_pages_per_seq)
    rc = call(ctypes.byref(dims), beam_width, _ints(parents, "parents", here, B),
              _tensor(block_table, "block_table", i32, here, table), _ints(seq_lens, "seq_lens", here, B),
              _tensor(block_table_out, "block_table_out", i32, here, table), *pools,
              None if err_flag is None else _ints(err_flag, "err_flag", here, 1), _stream(stream))
    if rc:
        _check(rc, what)


def beam_reorder(dims: Dims, beam_width: int, parents, block_table, seq_lens, block_table_out, k_pages, v_pages,
                 err_flag=None, stream=None) -> None:
    """sa_beam_reorder: the tables of the chosen continuations, and the copies of
    the tail pages that more than one of them continues."""
    here = _here()
    _beam_reorder(load_library().sa_beam_reorder, "sa_beam_reorder", here, dims, beam_width, parents, block_table, seq_lens,
                  block_table_out, _pools(dims, here, k_pages, v_pages), err_flag, stream)


def beam_reorder_q8(dims: Dims, beam_width: int, parents, block_table, seq_lens, block_table_out, k_codes, v_codes,
                    k_scales, v_scales, err_flag=None, stream=None) -> None:
    """beam_reorder over int8 pages."""
    here = _here()
    _beam_reorder(load_library().sa_beam_reorder_q8, "sa_beam_reorder_q8", here, dims, beam_width, parents, block_table,
                  seq_lens, block_table_out,
                  _code_pools(dims, here, _types_made.i8, 128, k_codes, v_codes, k_scales, v_scales), err_flag, stream)


def beam_reorder_q4(dims: Dims, beam_width: int, parents, block_table, seq_lens, block_table_out, k_codes, v_codes,
                    k_scales, v_scales, err_flag=None, stream=None) -> None:
    """beam_reorder over int4 pages."""
    here = _here()
    _beam_reorder(load_library().sa_beam_reorder_q4, "sa_beam_reorder_q4", here, dims, beam_width, parents, block_table,
                  seq_lens, block_table_out,
                  _code_pools(dims, here, _types_made.u8, 64, k_codes, v_codes, k_scales, v_scales), err_flag, stream)
