"""Thin ctypes binding of the C ABI in include/pkv.h (libpkv.so).

Argument marshalling only: each function turns torch tensors into pkv_tensor
descriptors (pointer, dtype, shape, strides) and calls the library on the
current CUDA stream. Every step of the computation runs in the library's CUDA
kernels; there is no Python or CPU implementation behind these names, and a
missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA = 0, 1, 2, 3
LAYOUTS = {"NHD": 0, "HND": 1}
STYLES = {"neox": 0, "interleaved": 1}
FLAG_SLOT_RANGE = 0x01
FLAG_POSITION_RANGE = 0x02
FLAG_PAGE_RANGE = 0x04
FLAG_SEQ_LEN_RANGE = 0x08
FLAG_DUPLICATE_SLOT = 0x10
FLAG_WAIT_TIMEOUT = 0x20
FLAG_PLAN_RANGE = 0x40
FLAG_DRAFT_RANGE = 0x80
FLAG_POOL_EMPTY = 0x100
FLAG_PAGE_STATE = 0x200
FLAG_ROW_RANGE = 0x400

_DTYPES = {
    torch.bfloat16: 0,
    torch.float8_e4m3fn: 1,
    torch.uint8: 1,
    torch.float32: 2,
    torch.int32: 3,
}
PKV_FP4_E2M1X2 = 4    # uint8 bytes of two E2M1 values (NVFP4 value caches)
_CACHE_DTYPE = {"bf16": 0, "fp8": 1, "nvfp4": PKV_FP4_E2M1X2}

EXPORTED = ("pkv_rope_kv_write", "pkv_paged_gqa_decode", "pkv_lse_merge", "pkv_choose_num_splits",
            "pkv_validate_indices", "pkv_status_string", "pkv_abi_version", "pkv_stream_read",
            "pkv_validate_indices_static", "pkv_rope_kv_write_nvfp4", "pkv_paged_gqa_decode_nvfp4",
            "pkv_mla_cache_write", "pkv_paged_mla_decode", "pkv_choose_num_splits_mla",
            "pkv_selftest_bounded_wait", "pkv_copy", "pkv_plan_splits", "pkv_paged_gqa_decode_planned",
            "pkv_lse_merge_planned", "pkv_plan_splits_mla", "pkv_paged_mla_decode_planned", "pkv_paged_tree_decode",
            "pkv_tree_decode_workspace", "pkv_accept_drafts", "pkv_resize_sequences", "pkv_fork_sequences",
            "pkv_qk_norm_rope_kv_write", "pkv_gather_kv", "pkv_prompt_attention", "pkv_prompt_attention_workspace")


class PkvTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class PkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libpkv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library {LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        T = ctypes.POINTER(PkvTensor)
        P = ctypes.c_void_p
        i32 = ctypes.c_int32
        L.pkv_rope_kv_write.argtypes = [T, T, T, T, T, T, T, T, T, T, i32, i32, P, P]
        L.pkv_paged_gqa_decode.argtypes = [T, T, T, T, T, ctypes.c_float, i32, T, T, T, T, i32, P, P]
        L.pkv_rope_kv_write_nvfp4.argtypes = [T, T, T, T, T, T, T, T, T, T, T, T, i32, i32, P, P]
        L.pkv_paged_gqa_decode_nvfp4.argtypes = [T, T, T, T, T, T, T, ctypes.c_float, i32, T, T, T, T, i32, P, P]
        L.pkv_mla_cache_write.argtypes = [T, T, T, T, T, T, T, T, T, i32, P, P]
        L.pkv_paged_mla_decode.argtypes = [T, T, T, T, T, T, ctypes.c_float, i32, T, T, T, P, P]
        L.pkv_choose_num_splits_mla.argtypes = [i32, i32, ctypes.c_int64, i32, i32]
        L.pkv_lse_merge.argtypes = [T, T, T, T, P]
        L.pkv_choose_num_splits.argtypes = [i32, i32, i32, i32, ctypes.c_int64, i32, i32, i32]
        L.pkv_validate_indices.argtypes = [T, T, T, ctypes.c_int64, T, P, P]
        L.pkv_stream_read.argtypes = [P, ctypes.c_int64, P, i32, P]
        L.pkv_selftest_bounded_wait.argtypes = [ctypes.c_int64, P, P, P]
        L.pkv_copy.argtypes = [P, P, ctypes.c_int64, P]
        L.pkv_validate_indices_static.argtypes = [T, T, T, ctypes.c_int64, P, P]
        L.pkv_plan_splits.argtypes = [P, i32, i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, ctypes.c_int64, P]
        L.pkv_paged_gqa_decode_planned.argtypes = [T, T, T, T, T, T, T, ctypes.c_float, T, T, T, T, T, T, i32, P,
                                                   P]
        L.pkv_lse_merge_planned.argtypes = [T, T, T, T, T, P]
        L.pkv_plan_splits_mla.argtypes = [P, i32, i32, i32, i32, i32, i32, P, P, P, ctypes.c_int64, P]
        L.pkv_paged_mla_decode_planned.argtypes = [T, T, T, T, T, T, ctypes.c_float, T, T, T, T, T, P, P]
        L.pkv_paged_tree_decode.argtypes = [T, T, T, T, T, T, T, ctypes.c_float, T, T, P, ctypes.c_int64, T, T, i32,
                                            P, P]
        L.pkv_tree_decode_workspace.argtypes = [ctypes.c_int64, i32, i32, i32]
        L.pkv_tree_decode_workspace.restype = ctypes.c_int64
        L.pkv_accept_drafts.argtypes = [T, i32, i32, T, T, T, T, T, T, P, P]
        L.pkv_resize_sequences.argtypes = [T, T, T, T, i32, P, P]
        L.pkv_fork_sequences.argtypes = [T, i32, i32, T, T, T, T, T, T, P, P]
        L.pkv_qk_norm_rope_kv_write.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, T, T, T, T, T, T, T, i32, i32, P,
                                                P]
        L.pkv_gather_kv.argtypes = [T, T, T, T, T, T, T, T, T, T, T, i32, P, P]
        L.pkv_prompt_attention.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, P, ctypes.c_int64, P, P]
        L.pkv_prompt_attention_workspace.argtypes = [i32, i32]
        L.pkv_prompt_attention_workspace.restype = ctypes.c_int64
        L.pkv_status_string.argtypes = [i32]
        L.pkv_status_string.restype = ctypes.c_char_p
        for name in ("pkv_rope_kv_write", "pkv_paged_gqa_decode", "pkv_lse_merge", "pkv_validate_indices",
                     "pkv_choose_num_splits", "pkv_abi_version", "pkv_stream_read", "pkv_validate_indices_static",
                     "pkv_rope_kv_write_nvfp4", "pkv_paged_gqa_decode_nvfp4", "pkv_mla_cache_write",
                     "pkv_paged_mla_decode", "pkv_choose_num_splits_mla", "pkv_selftest_bounded_wait", "pkv_copy",
                     "pkv_plan_splits", "pkv_paged_gqa_decode_planned", "pkv_lse_merge_planned",
                     "pkv_plan_splits_mla", "pkv_paged_mla_decode_planned", "pkv_paged_tree_decode",
                     "pkv_accept_drafts", "pkv_resize_sequences", "pkv_fork_sequences",
                     "pkv_qk_norm_rope_kv_write", "pkv_gather_kv", "pkv_prompt_attention"):
            getattr(L, name).restype = ctypes.c_int32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


class Bound:
    """A tensor, or a list of tensors, with its descriptors made once (see
    bind). Keeps the tensors alive."""
    __slots__ = ("tensors", "ptr", "n", "data", "nbytes", "device", "_other")

    def __init__(self, tensors, ptr, n: int):
        self.tensors, self.ptr, self.n = tensors, ptr, n
        first = tensors[0] if tensors else None
        self.data = first.data_ptr() if first is not None else None
        # (as a workspace: None where the elements are not one stretch of memory)
        self.nbytes = 0 if first is None else first.numel() * first.element_size() if first.is_contiguous() else None
        self.device = first.get_device() if first is not None else None
        self._other = None

    def tensor(self) -> torch.Tensor:
        if self.n != 1:
            raise TypeError("a bound list of tensors where one tensor is expected")
        return self.tensors[0]

    def as_dtype(self, dtype: int):
        """The descriptor under another pkv_dtype (the one that _desc's `dtype` gives), made once too."""
        self.tensor()
        if self._other is None or self._other.contents.dtype != dtype:
            d = PkvTensor.from_buffer_copy(self.ptr.contents)
            d.dtype = dtype
            self._other = ctypes.pointer(d)
        return self._other


def _tensor(t):
    return t.tensor() if isinstance(t, Bound) else t


def bind(t):
    """Descriptors of a tensor, or of a list of tensors (the caches of a
    model), made once for buffers that a program passes call after call: every
    call here takes what bind() returns in place of the tensor, and skips the
    descriptor's making. The tensor's memory, shape and strides are those at
    the time of bind()."""
    if t is None or isinstance(t, Bound):
        return t
    if isinstance(t, torch.Tensor):
        return Bound([t], _desc(t), 1)
    ts = list(t)
    if any(x.get_device() != ts[0].get_device() for x in ts):
        raise ValueError("the tensors of one call are on different devices")
    arr = (PkvTensor * len(ts))(*[_desc(x).contents for x in ts])
    return Bound(ts, ctypes.cast(arr, ctypes.POINTER(PkvTensor)) if ts else None, len(ts))


def _on_current_device(*ts) -> None:
    """The kernels run on the current device's stream: a tensor of another
    device would be reached through a peer mapping, or not at all."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is None:
            continue
        d = t.device if isinstance(t, Bound) else t.get_device()
        if d is not None and d != dev and not (isinstance(t, torch.Tensor) and not t.numel()):
            raise ValueError(f"a tensor is on device {d}, the current device is {dev}")


def _desc(t, dtype: Optional[int] = None):
    """Pointer to a descriptor of t (NULL for None); `dtype` overrides the
    pkv_dtype taken from t.dtype (uint8 NVFP4 value caches)."""
    if t is None:
        return None
    if isinstance(t, Bound):
        if dtype is not None:
            return t.as_dtype(dtype)
        if t.n != 1:
            raise TypeError("a bound list of tensors where one tensor is expected")
        return t.ptr
    d = PkvTensor()
    if t.dim() > 4:
        raise ValueError("tensors of more than 4 dims are not part of the ABI")
    if t.dtype not in _DTYPES:
        raise TypeError(f"dtype {t.dtype} is not part of the ABI")
    if t.numel() and not t.is_cuda:
        raise ValueError("the C ABI takes device tensors; copy host data to the GPU first")
    d.ptr = t.data_ptr() if t.numel() else None
    d.dtype = _DTYPES[t.dtype] if dtype is None else dtype
    d.ndim = t.dim()
    for i, (n, s) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = n
        d.stride[i] = s
    return ctypes.pointer(d)


def _descs(dev: int, *ts):
    """_desc of every tensor, each checked to be on device `dev` as
    _on_current_device does: one pass over a call's tensors, for calls short
    enough for the host's share to count."""
    out = []
    for t in ts:
        if type(t) is Bound and t.n == 1 and t.device == dev:
            out.append(t.ptr)
        elif t is None:
            out.append(None)
        else:
            _on_current_device(t)
            out.append(_desc(t))
    return out


def _stream(stream) -> Optional[int]:
    if stream is None:  # (torch.cuda.current_stream() makes a Stream object: 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_of(dev: int, stream) -> Optional[int]:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _flag(dev: int, t):
    """The error flag's address, checked as _descs does."""
    if type(t) is Bound and t.n == 1 and t.device == dev:
        return t.data
    _on_current_device(t)
    return _ptr(t)


def _ptr(t):
    if t is None:
        return None
    return t.data if isinstance(t, Bound) else t.data_ptr()


def _check(fn: str, status: int) -> None:
    if status != PKV_OK:
        raise PkvError(fn, status)


def rope_kv_write(q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, k_scale=None, v_scale=None,
                  layout: str = "HND", rope_style: str = "neox", err_flag=None, stream=None) -> None:
    """Fused RoPE + paged-KV write (pkv_rope_kv_write): q (or None) rotated
    in place, rotated k and v written into the caches at slot_mapping."""
    _check("pkv_rope_kv_write", lib().pkv_rope_kv_write(
        _desc(q), _desc(k), _desc(v), _desc(positions), _desc(cos_sin), _desc(k_cache), _desc(v_cache),
        _desc(slot_mapping), _desc(k_scale), _desc(v_scale), LAYOUTS[layout], STYLES[rope_style],
        _ptr(err_flag), _stream(stream)))


def paged_gqa_decode(q, k_cache, v_cache, block_tables, seq_lens, softmax_scale: float, num_splits: int,
                     out_partial, lse_partial, k_scale=None, v_scale=None, layout: str = "HND", err_flag=None,
                     stream=None) -> None:
    """Paged GQA split-K decode (pkv_paged_gqa_decode) into out_partial
    [B,S,Hq,D] and lse_partial [B,S,Hq]."""
    _check("pkv_paged_gqa_decode", lib().pkv_paged_gqa_decode(
        _desc(q), _desc(k_cache), _desc(v_cache), _desc(block_tables), _desc(seq_lens), float(softmax_scale),
        int(num_splits), _desc(out_partial), _desc(lse_partial), _desc(k_scale), _desc(v_scale), LAYOUTS[layout],
        _ptr(err_flag), _stream(stream)))


def _fp4(t):
    if t is not None and _tensor(t).dtype != torch.uint8:
        raise TypeError("NVFP4 value caches are uint8 tensors of packed E2M1 pairs")
    return _desc(t, PKV_FP4_E2M1X2)


def rope_kv_write_nvfp4(q, k, v, positions, cos_sin, k_cache, v_cache, k_block_scale, v_block_scale,
                        slot_mapping, k_scale, v_scale, layout: str = "HND", rope_style: str = "neox",
                        err_flag=None, stream=None) -> None:
    """pkv_rope_kv_write_nvfp4: as rope_kv_write into NVFP4 caches -- value
    caches uint8 [.., D/2] (packed E2M1 pairs), block-scale caches uint8 or
    float8_e4m3fn [.., D/16], static scales [1] or [Hkv] float32."""
    _check("pkv_rope_kv_write_nvfp4", lib().pkv_rope_kv_write_nvfp4(
        _desc(q), _desc(k), _desc(v), _desc(positions), _desc(cos_sin), _fp4(k_cache), _fp4(v_cache),
        _desc(k_block_scale), _desc(v_block_scale), _desc(slot_mapping), _desc(k_scale), _desc(v_scale),
        LAYOUTS[layout], STYLES[rope_style], _ptr(err_flag), _stream(stream)))


def paged_gqa_decode_nvfp4(q, k_cache, v_cache, k_block_scale, v_block_scale, block_tables, seq_lens,
                           softmax_scale: float, num_splits: int, out_partial, lse_partial, k_scale, v_scale,
                           layout: str = "HND", err_flag=None, stream=None) -> None:
    """pkv_paged_gqa_decode_nvfp4: paged GQA split-K decode over NVFP4
    caches (HND) into out_partial [B,S,Hq,D] and lse_partial [B,S,Hq]."""
    _check("pkv_paged_gqa_decode_nvfp4", lib().pkv_paged_gqa_decode_nvfp4(
        _desc(q), _fp4(k_cache), _fp4(v_cache), _desc(k_block_scale), _desc(v_block_scale), _desc(block_tables),
        _desc(seq_lens), float(softmax_scale), int(num_splits), _desc(out_partial), _desc(lse_partial),
        _desc(k_scale), _desc(v_scale), LAYOUTS[layout], _ptr(err_flag), _stream(stream)))


def mla_cache_write(q_pe, ckv, kpe, positions, cos_sin, ckv_cache, kpe_cache, slot_mapping, ckv_scale,
                    rope_style: str = "interleaved", err_flag=None, stream=None) -> None:
    """pkv_mla_cache_write: ckv [T,512] bf16 -> E4M3 bytes of ckv_cache
    [pages,P,512] (uint8 or float8_e4m3fn), RoPE(kpe [T,64]) -> kpe_cache
    [pages,P,64] bf16, q_pe [T,H,64] (or None) rotated in place."""
    _check("pkv_mla_cache_write", lib().pkv_mla_cache_write(
        _desc(q_pe), _desc(ckv), _desc(kpe), _desc(positions), _desc(cos_sin), _desc(ckv_cache), _desc(kpe_cache),
        _desc(slot_mapping), _desc(ckv_scale), STYLES[rope_style], _ptr(err_flag), _stream(stream)))


def paged_mla_decode(q_lat, q_pe, ckv_cache, kpe_cache, block_tables, seq_lens, softmax_scale: float,
                     num_splits: int, out_partial, lse_partial, ckv_scale, err_flag=None, stream=None) -> None:
    """pkv_paged_mla_decode: q_lat [B,H,512], q_pe [B,H,64] over the latent
    cache into out_partial [B,S,H,512] and lse_partial [B,S,H]."""
    _check("pkv_paged_mla_decode", lib().pkv_paged_mla_decode(
        _desc(q_lat), _desc(q_pe), _desc(ckv_cache), _desc(kpe_cache), _desc(block_tables), _desc(seq_lens),
        float(softmax_scale), int(num_splits), _desc(out_partial), _desc(lse_partial), _desc(ckv_scale),
        _ptr(err_flag), _stream(stream)))


def choose_num_splits_mla(B: int, H: int, total_pages: int, max_pages: int, sm_count: int) -> int:
    """Split count for the MLA decode from the library's heuristic (host only)."""
    return int(lib().pkv_choose_num_splits_mla(B, H, int(total_pages), max_pages, sm_count))


def lse_merge(out_partial, lse_partial, out, lse_out=None, stream=None) -> None:
    """LSE merge of the split partials into out [B,Hq,D] bf16 (pkv_lse_merge)."""
    _check("pkv_lse_merge", lib().pkv_lse_merge(_desc(out_partial), _desc(lse_partial), _desc(out),
                                                 _desc(lse_out), _stream(stream)))


def choose_num_splits(B: int, Hkv: int, Hq: int, D: int, total_pages: int, max_pages: int, cache_dtype: str,
                      sm_count: int) -> int:
    """Split count from the library's heuristic (host only)."""
    return int(lib().pkv_choose_num_splits(B, Hkv, Hq, D, int(total_pages), max_pages,
                                           _CACHE_DTYPE[cache_dtype], sm_count))


def plan_splits(seq_lens, Hkv: int, Hq: int, D: int, max_pages: int, cache_dtype: str, sm_count: int,
                max_splits: int = 4095, target_pages: int = 0):
    """pkv_plan_splits (host only): (splits_per_seq int32 [B], num_records,
    work int32 [W, 2]) for the planned decode and merge."""
    import numpy as np
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = int(sl.size)
    sp = np.zeros(max(B, 1), np.int32)
    nrec = ctypes.c_int32(0)
    nwork = ctypes.c_int64(0)
    f = lib().pkv_plan_splits
    args = (sl.ctypes.data if B else None, B, Hkv, Hq, D, max_pages, _CACHE_DTYPE[cache_dtype], sm_count,
            max_splits, target_pages, sp.ctypes.data)
    _check("pkv_plan_splits", f(*args, ctypes.byref(nrec), None, 0, ctypes.byref(nwork)))
    work = np.zeros((max(int(nwork.value), 1), 2), np.int32)
    _check("pkv_plan_splits", f(*args, ctypes.byref(nrec), work.ctypes.data, int(nwork.value), ctypes.byref(nwork)))
    return sp[:B], int(nrec.value), work[:int(nwork.value)]


def paged_gqa_decode_planned(q, k_cache, v_cache, block_tables, seq_lens, softmax_scale: float, splits_per_seq,
                             work, out_partial, lse_partial, k_scale=None, v_scale=None, layout: str = "HND",
                             err_flag=None, stream=None, k_block_scale=None, v_block_scale=None) -> None:
    """pkv_paged_gqa_decode_planned: the decode under a split plan (device
    splits_per_seq [B] and work [W, 2] int32 from plan_splits); NVFP4 caches
    when the block-scale caches are given."""
    fp4 = k_block_scale is not None
    kc, vc = (_fp4(k_cache), _fp4(v_cache)) if fp4 else (_desc(k_cache), _desc(v_cache))
    _check("pkv_paged_gqa_decode_planned", lib().pkv_paged_gqa_decode_planned(
        _desc(q), kc, vc, _desc(k_block_scale), _desc(v_block_scale), _desc(block_tables), _desc(seq_lens),
        float(softmax_scale), _desc(splits_per_seq), _desc(work), _desc(out_partial), _desc(lse_partial),
        _desc(k_scale), _desc(v_scale), LAYOUTS[layout], _ptr(err_flag), _stream(stream)))


def plan_splits_mla(seq_lens, H: int, max_pages: int, sm_count: int, max_splits: int = 4095, target_pages: int = 0):
    """pkv_plan_splits_mla (host only): (splits_per_seq int32 [B],
    num_records, work int32 [W, 2]) for the planned MLA decode."""
    import numpy as np
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = int(sl.size)
    sp = np.zeros(max(B, 1), np.int32)
    nrec = ctypes.c_int32(0)
    nwork = ctypes.c_int64(0)
    f = lib().pkv_plan_splits_mla
    args = (sl.ctypes.data if B else None, B, H, max_pages, sm_count, max_splits, target_pages, sp.ctypes.data)
    _check("pkv_plan_splits_mla", f(*args, ctypes.byref(nrec), None, 0, ctypes.byref(nwork)))
    work = np.zeros((max(int(nwork.value), 1), 2), np.int32)
    _check("pkv_plan_splits_mla", f(*args, ctypes.byref(nrec), work.ctypes.data, int(nwork.value),
                                    ctypes.byref(nwork)))
    return sp[:B], int(nrec.value), work[:int(nwork.value)]


def paged_mla_decode_planned(q_lat, q_pe, ckv_cache, kpe_cache, block_tables, seq_lens, softmax_scale: float,
                             splits_per_seq, work, out_partial, lse_partial, ckv_scale, err_flag=None,
                             stream=None) -> None:
    """pkv_paged_mla_decode_planned: the MLA decode under a split plan."""
    _check("pkv_paged_mla_decode_planned", lib().pkv_paged_mla_decode_planned(
        _desc(q_lat), _desc(q_pe), _desc(ckv_cache), _desc(kpe_cache), _desc(block_tables), _desc(seq_lens),
        float(softmax_scale), _desc(splits_per_seq), _desc(work), _desc(out_partial), _desc(lse_partial),
        _desc(ckv_scale), _ptr(err_flag), _stream(stream)))


def lse_merge_planned(out_partial, lse_partial, splits_per_seq, out, lse_out=None, stream=None) -> None:
    """pkv_lse_merge_planned: each sequence's own records [0, S_b)."""
    _check("pkv_lse_merge_planned", lib().pkv_lse_merge_planned(
        _desc(out_partial), _desc(lse_partial), _desc(splits_per_seq), _desc(out), _desc(lse_out), _stream(stream)))


def _workspace(t):
    """Address and bytes of a workspace."""
    if t is None:
        return None, 0
    if isinstance(t, Bound):
        t.tensor()
        ptr, nbytes = t.data, t.nbytes
    else:
        ptr, nbytes = t.data_ptr(), t.numel() * t.element_size() if t.is_contiguous() else None
    if nbytes is None:
        raise ValueError("a workspace is a contiguous tensor")
    return ptr, nbytes


def tree_decode_workspace(T: int, Hq: int, D: int, sm_count: int) -> int:
    """Bytes of workspace that paged_tree_decode needs (the same for any T and
    Hq, which are only checked)."""
    return int(lib().pkv_tree_decode_workspace(int(T), Hq, D, sm_count))


def paged_tree_decode(q, k_cache, v_cache, block_tables, seq_lens, q_start, tree_mask, softmax_scale: float, out,
                      lse_out, workspace, k_scale=None, v_scale=None, layout: str = "HND", err_flag=None,
                      stream=None) -> None:
    """Attention of the drafted tokens (rows q_start[b] .. q_start[b+1] of q
    [T,Hq,D] for sequence b) over the paged cache that holds them behind the
    context, under tree_mask [T,W] int32 bits or, with None, as a chain
    (pkv_paged_tree_decode): out [T,Hq,D] bf16, lse_out [T,Hq] float32 or None.
    workspace: a contiguous device tensor of tree_decode_workspace() bytes."""
    _on_current_device(q, k_cache, v_cache, block_tables, seq_lens, q_start, tree_mask, out, lse_out, workspace,
                       k_scale, v_scale, err_flag)
    ws, nbytes = _workspace(workspace)
    _check("pkv_paged_tree_decode", lib().pkv_paged_tree_decode(
        _desc(q), _desc(k_cache), _desc(v_cache), _desc(block_tables), _desc(seq_lens), _desc(q_start),
        _desc(tree_mask), softmax_scale, _desc(out), _desc(lse_out), ws, nbytes, _desc(k_scale), _desc(v_scale),
        LAYOUTS[layout], _ptr(err_flag), _stream(stream)))


def accept_drafts(caches, block_tables, seq_lens, q_start, accepted, num_accepted, seq_lens_out, layout: str = "HND",
                  err_flag=None, stream=None) -> None:
    """Moves the accepted drafted tokens' rows together behind the context, in
    every cache of the list `caches`, and writes the new lengths
    (pkv_accept_drafts)."""
    caches = bind([] if caches is None else caches)
    _on_current_device(caches, block_tables, seq_lens, q_start, accepted, num_accepted, seq_lens_out, err_flag)
    _check("pkv_accept_drafts", lib().pkv_accept_drafts(
        caches.ptr, caches.n, LAYOUTS[layout], _desc(block_tables), _desc(seq_lens), _desc(q_start), _desc(accepted),
        _desc(num_accepted), _desc(seq_lens_out), _ptr(err_flag), _stream(stream)))


def resize_sequences(block_tables, page_counts, new_lens, page_refs, page_size: int = 16, err_flag=None,
                     stream=None) -> None:
    """Returns and takes pages so that every sequence holds those of
    new_lens[b] tokens (< 0: unchanged), the lowest free pages first
    (pkv_resize_sequences)."""
    _on_current_device(block_tables, page_counts, new_lens, page_refs, err_flag)
    _check("pkv_resize_sequences", lib().pkv_resize_sequences(
        _desc(block_tables), _desc(page_counts), _desc(new_lens), _desc(page_refs), page_size, _ptr(err_flag),
        _stream(stream)))


def fork_sequences(caches, block_tables, page_counts, seq_lens, forks, page_refs, copies, layout: str = "HND",
                   err_flag=None, stream=None) -> None:
    """Makes row forks[i][1] continue row forks[i][0]: full pages shared, the
    partial last page copied in every cache of the list `caches`; copies [n,2]
    receives the copied pages (pkv_fork_sequences)."""
    caches = bind([] if caches is None else caches)
    _on_current_device(caches, block_tables, page_counts, seq_lens, forks, page_refs, copies, err_flag)
    _check("pkv_fork_sequences", lib().pkv_fork_sequences(
        caches.ptr, caches.n, LAYOUTS[layout], _desc(block_tables), _desc(page_counts), _desc(seq_lens), _desc(forks),
        _desc(page_refs), _desc(copies), _ptr(err_flag), _stream(stream)))


def qk_norm_rope_kv_write(q, k, v, q_weight, k_weight, eps: float, positions, cos_sin, k_cache, v_cache, slot_mapping,
                          k_scale=None, v_scale=None, k_block_scale=None, v_block_scale=None, k_out=None,
                          layout: str = "HND", rope_style: str = "neox", err_flag=None, stream=None) -> None:
    """rope_kv_write (with block-scale caches: rope_kv_write_nvfp4) with an RMS
    norm of every q and k head, weights q_weight and k_weight [D] float32 or
    bf16, before the rotation; k_out [T,Hkv,D] bf16 (or k itself, or None)
    receives the normed and rotated keys (pkv_qk_norm_rope_kv_write)."""
    dev = torch.cuda.current_device()
    q, k, v, q_weight, k_weight, positions, cos_sin, kc, vc, kbs, vbs, slot_mapping, k_scale, v_scale, k_out = _descs(
        dev, q, k, v, q_weight, k_weight, positions, cos_sin, k_cache, v_cache, k_block_scale, v_block_scale, slot_mapping,
        k_scale, v_scale, k_out)
    if kbs is not None:
        kc, vc = _fp4(k_cache), _fp4(v_cache)
    _check("pkv_qk_norm_rope_kv_write", (_lib or lib()).pkv_qk_norm_rope_kv_write(
        q, k, v, q_weight, k_weight, eps, positions, cos_sin, kc, vc, kbs, vbs, slot_mapping, k_scale, v_scale, k_out,
        LAYOUTS[layout], STYLES[rope_style], _flag(dev, err_flag), _stream_of(dev, stream)))


def gather_kv(k_cache, v_cache, block_tables, start, first, k_out, v_out, k_scale=None, v_scale=None, k_block_scale=None,
              v_block_scale=None, layout: str = "HND", err_flag=None, stream=None) -> None:
    """Cached keys and values as packed bf16 rows (pkv_gather_kv): rows
    start[b] .. start[b+1] of k_out, v_out [T,Hkv,D] receive positions first[b]
    (None: 0) and on of sequence b."""
    dev = torch.cuda.current_device()
    kc, vc, kbs, vbs, block_tables, start, first, k_out, v_out, k_scale, v_scale = _descs(
        dev, k_cache, v_cache, k_block_scale, v_block_scale, block_tables, start, first, k_out, v_out, k_scale, v_scale)
    if kbs is not None:
        kc, vc = _fp4(k_cache), _fp4(v_cache)
    _check("pkv_gather_kv", (_lib or lib()).pkv_gather_kv(
        kc, vc, kbs, vbs, block_tables, start, first, k_out, v_out, k_scale, v_scale, LAYOUTS[layout], _flag(dev, err_flag),
        _stream_of(dev, stream)))


def prompt_attention_workspace(D: int, sm_count: int) -> int:
    """Bytes of workspace that prompt_attention needs, whatever its rows and heads."""
    return int(lib().pkv_prompt_attention_workspace(D, sm_count))


def prompt_attention(q, k, v, q_start, k_start, softmax_scale: float, out, lse_out, workspace, err_flag=None,
                     stream=None) -> None:
    """Causal attention of packed prompts (pkv_prompt_attention): rows
    q_start[b] .. q_start[b+1] of q [T,Hq,D] over rows k_start[b] ..
    k_start[b+1] of k, v [Tk,Hkv,D] (None: q_start), whose last ones are
    theirs: out [T,Hq,D] bf16, lse_out [T,Hq] float32 or None. workspace: a
    contiguous device tensor of prompt_attention_workspace() bytes."""
    dev = torch.cuda.current_device()
    q, k, v, q_start, k_start, out, lse_out = _descs(dev, q, k, v, q_start, k_start, out, lse_out)
    _on_current_device(workspace)
    ws, nbytes = _workspace(workspace)
    _check("pkv_prompt_attention", (_lib or lib()).pkv_prompt_attention(
        q, k, v, q_start, k_start, softmax_scale, out, lse_out, ws, nbytes, _flag(dev, err_flag), _stream_of(dev, stream)))


def validate_indices(block_tables, seq_lens, slot_mapping, num_pages: int, err_flag, slot_bitmap=None,
                     stream=None) -> None:
    """Device check of seq_lens, block tables and slots (pkv_validate_indices)."""
    _check("pkv_validate_indices", lib().pkv_validate_indices(
        _desc(block_tables), _desc(seq_lens), _desc(slot_mapping), int(num_pages), _desc(slot_bitmap),
        _ptr(err_flag), _stream(stream)))


def validate_indices_static(block_tables, seq_lens, slot_mapping, num_pages: int, err_flag, stream=None) -> None:
    """pkv_validate_indices_static: the same check as validate_indices
    (duplicates included) for callers that cannot allocate device memory --
    e.g. an engine whose allocator already holds all free memory for its KV
    pool, or a path that must not call cudaMalloc/cudaFree because they can
    synchronise the device. The bitmap is a fixed 1 MiB device array in the
    library (at most 2**23 cache slots); calls overlapping on the GPU race on
    it, and the first call on a device should come before any stream
    capture."""
    _check("pkv_validate_indices_static", lib().pkv_validate_indices_static(
        _desc(block_tables), _desc(seq_lens), _desc(slot_mapping), int(num_pages), _ptr(err_flag),
        _stream(stream)))


def selftest_bounded_wait(limit_ns: int, err_flag: torch.Tensor, elapsed_ns: torch.Tensor, stream=None) -> None:
    """Self-test of the bounded in-kernel waits (pkv_selftest_bounded_wait):
    err_flag an int32 device word, elapsed_ns two int64 device words."""
    err_flag, elapsed_ns = _tensor(err_flag), _tensor(elapsed_ns)
    if not (err_flag.is_cuda and err_flag.dtype == torch.int32 and elapsed_ns.is_cuda
            and elapsed_ns.dtype == torch.int64 and elapsed_ns.numel() >= 2):
        raise ValueError("int32 device flag and two int64 device words expected")
    _check("pkv_selftest_bounded_wait",
           lib().pkv_selftest_bounded_wait(int(limit_ns), err_flag.data_ptr(), elapsed_ns.data_ptr(), _stream(stream)))


def copy(dst: torch.Tensor, src: torch.Tensor, stream=None) -> None:
    """pkv_copy: dst <- src byte for byte by the SMs; each a contiguous tensor
    in device memory or in pinned host memory (e.g. from pin_memory()), the
    same number of bytes."""
    dst, src = _tensor(dst), _tensor(src)
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy: dst and src must be contiguous")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("copy: dst and src differ in size")
    _check("pkv_copy", lib().pkv_copy(_ptr(dst), _ptr(src), n, _stream(stream)))


def stream_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Streaming-read ceiling (pkv_stream_read): read all of `buf` once in
    one launch of sink.numel() CTAs."""
    buf, sink = _tensor(buf), _tensor(sink)
    if not (buf.is_cuda and sink.is_cuda and sink.dtype == torch.int32):
        raise ValueError("device buffer and int32 device sink expected")
    _check("pkv_stream_read", lib().pkv_stream_read(buf.data_ptr(), buf.numel() * buf.element_size(),
                                                     sink.data_ptr(), sink.numel(), _stream(stream)))
