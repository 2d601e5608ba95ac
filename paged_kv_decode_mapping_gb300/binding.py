"""Thin ctypes binding of libpkv.so: argument marshalling only.

Every function has the name of the C entry point it calls (``include/paged_kv.h``),
takes torch CUDA tensors, checks their dtypes/shapes/contiguity, and passes raw
device pointers, sizes and the current CUDA stream.  All computation happens in
the library's kernels; there is no fallback.  Importing this module raises if
``libpkv.so`` has not been built.
"""

from __future__ import annotations

import array
import ctypes
import struct
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)

PKV_OK = 0
ERRORS = {-1: "PKV_ERR_NULL", -2: "PKV_ERR_SHAPE", -3: "PKV_ERR_UNSUPPORTED",
          -4: "PKV_ERR_WORKSPACE", -5: "PKV_ERR_ALIGN", -6: "PKV_ERR_CUDA", -7: "PKV_ERR_DEVICE",
          -8: "PKV_ERR_NOSPACE"}
DEVERR = {1: "BLOCK_ID", 2: "SLOT", 4: "CONTEXT_LEN", 8: "TIMEOUT", 16: "POSITION"}


class PkvError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = _lib.pkv_last_error().decode(errors="replace")
        super().__init__(f"{where}: {ERRORS.get(code, code)}: {msg}")
        self.code = code


class pkv_cache_desc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class pkv_q8_cache(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("kind", ctypes.c_int32)]


_P = ctypes.c_void_p
_i32, _i64, _f32, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_D = ctypes.POINTER(pkv_cache_desc)
_Q8 = ctypes.POINTER(pkv_q8_cache)

_lib.paged_kv_write.argtypes = [_P, _P, _P, _i64, _P, _P, _D, _P]
_lib.paged_kv_write.restype = ctypes.c_int
_lib.paged_kv_write_rope.argtypes = [_P, _P, _P, _i32, _P, _P, _i64, _P, _i64, _i32, _i32, _P, _P,
                                     _D, _P]
_lib.paged_kv_write_rope.restype = ctypes.c_int
_lib.paged_kv_copy_blocks.argtypes = [_P, _P, _i32, _P, _P, _i64, _D, _P]
_lib.paged_kv_copy_blocks.restype = ctypes.c_int
_lib.paged_kv_compact.argtypes = [_P, _P, _i32, _P, _i64, _P, _i64, _i32, _P, _D, _P]
_lib.paged_kv_compact.restype = ctypes.c_int
_lib.paged_decode_plan.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
_lib.paged_decode_plan.restype = _i32
_lib.paged_decode_path.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
_lib.paged_decode_path.restype = _i32
_lib.pkv_set_decode_consumer.argtypes = [_i32]
_lib.pkv_set_decode_consumer.restype = _i32
_lib.pkv_decode_ctas_per_sm.argtypes = [_i32, _i32]
_lib.pkv_decode_ctas_per_sm.restype = _i32
_lib.paged_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.paged_decode_workspace_size.restype = _sz
_lib.paged_decode_split_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.paged_decode_split_workspace_size.restype = _sz
_lib.paged_decode_attention.argtypes = [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32, _D, _f32,
                                        _P, _sz, _P]
_lib.paged_decode_attention.restype = ctypes.c_int
_lib.pkv_set_shared_prefix.argtypes = [_i32]
_lib.pkv_set_shared_prefix.restype = _i32
_lib.paged_decode_shared_prefix_workspace_size.argtypes = [_i32] * 7
_lib.paged_decode_shared_prefix_workspace_size.restype = _sz
_lib.paged_decode_shared_prefix_attention.argtypes = [_P, _P, _P, _P, _P, _i32, _P, _P, _P, _i32,
                                                      _i32, _i32, _i32, _i32, _D, _f32, _P, _sz, _P]
_lib.paged_decode_shared_prefix_attention.restype = ctypes.c_int
_lib.paged_decode_step.argtypes = [_P, _P, _P, _P, _P, _i64, _P, _P, _P, _i32, _P, _i32, _i32,
                                   _i32, _D, _f32, _P, _sz, _P]
_lib.paged_decode_step.restype = ctypes.c_int
_lib.paged_decode_step_rope.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i64, _i32, _i32, _P, _P, _P,
                                        _i32, _P, _i32, _i32, _i32, _D, _f32, _P, _sz, _P]
_lib.paged_decode_step_rope.restype = ctypes.c_int
_lib.paged_prefill_attention.argtypes = [_P, _P, _P, _P, _P, _i32, _P, _i32, _P, _i32, _i32, _i32,
                                         _D, _f32, _P]
_lib.paged_prefill_attention.restype = ctypes.c_int
_lib.prompt_attention.argtypes = [_P, _P, _P, _P, _i64, _i64, _i64, _i64, _P, _i64, _i32, _i32,
                                  _i32, _i32, _i32, _f32, _P]
_lib.prompt_attention.restype = ctypes.c_int
_lib.paged_kv_write_q8.argtypes = [_P, _P, _i64, _i64, _P, _i64, _i32, _P, _i32, _P, _i32, _Q8, _D, _P]
_lib.paged_kv_write_q8.restype = ctypes.c_int
_lib.paged_kv_write_rope_q8.argtypes = [_P, _P, _i64, _i64, _P, _P, _i64, _i64, _i32, _P, _P, _i64, _i32,
                                        _i32, _P, _i64, _i32, _P, _i32, _P, _i32, _Q8, _D, _P]
_lib.paged_kv_write_rope_q8.restype = ctypes.c_int
_lib.paged_kv_read_q8.argtypes = [_P, _P, _i64, _i64, _P, _i64, _i32, _P, _i32, _P, _i32, _Q8, _D, _P]
_lib.paged_kv_read_q8.restype = ctypes.c_int
_lib.paged_decode_q8_workspace_size.argtypes = [_i32] * 5
_lib.paged_decode_q8_workspace_size.restype = _sz
_lib.paged_decode_attention_q8.argtypes = [_P, _P, _Q8, _P, _i32, _P, _i32, _i32, _i32, _D, _f32, _P, _sz, _P]
_lib.paged_decode_attention_q8.restype = ctypes.c_int
_lib.paged_decode_step_q8.argtypes = [_P, _P, _P, _P, _i64, _i64, _Q8, _P, _i32, _P, _i32, _i32, _i32, _D,
                                      _f32, _P, _sz, _P]
_lib.paged_decode_step_q8.restype = ctypes.c_int
_lib.paged_decode_step_rope_q8.argtypes = [_P, _P, _i64, _P, _P, _P, _i64, _i64, _P, _P, _i64, _i32, _i32,
                                           _Q8, _P, _i32, _P, _i32, _i32, _i32, _D, _f32, _P, _sz, _P]
_lib.paged_decode_step_rope_q8.restype = ctypes.c_int
_lib.paged_prefill_q8_workspace_size.argtypes = [_i32] * 4
_lib.paged_prefill_q8_workspace_size.restype = _sz
_lib.paged_prefill_q8_workspace_size_for.argtypes = [_i64] + [_i32] * 6
_lib.paged_prefill_q8_workspace_size_for.restype = _sz
_lib.paged_prefill_attention_q8.argtypes = [_P, _P, _i64, _Q8, _P, _i32, _P, _i32, _P, _i32, _i32, _i32, _D, _f32,
                                            _P, _sz, _P]
_lib.paged_prefill_attention_q8.restype = ctypes.c_int
_lib.pkv_call_q8.argtypes = [_i32, _P]
_lib.pkv_call_q8.restype = ctypes.c_int
_lib.paged_kv_copy_blocks_q8.argtypes = [_P, _i32, _P, _P, _i64, _D, _P]
_lib.paged_kv_copy_blocks_q8.restype = ctypes.c_int
_lib.paged_kv_compact_q8.argtypes = [_P, _i32, _P, _P, _i64, _P, _i64, _i32, _P, _D, _P]
_lib.paged_kv_compact_q8.restype = ctypes.c_int
_lib.paged_decode_split.argtypes = [_P, _P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32, _D, _f32,
                                    _i32, _P]
_lib.paged_decode_split.restype = ctypes.c_int
_lib.paged_decode_combine.argtypes = [_P, _P, _P, _P, _i32, _i32, _i32, _i32, _i32, _P]
_lib.paged_decode_combine.restype = ctypes.c_int
_lib.paged_decode_attention_noalloc.argtypes = [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32,
                                                _D, _f32, _P]
_lib.paged_decode_attention_noalloc.restype = ctypes.c_int
NOALLOC_SCRATCH_BYTES = 32 << 20  # PKV_NOALLOC_SCRATCH_BYTES in include/paged_kv.h
_lib.pkv_bm_create.argtypes = [_i64, _i32]
_lib.pkv_bm_create.restype = _P
_lib.pkv_bm_destroy.argtypes = [_P]
_lib.pkv_bm_destroy.restype = None
_lib.pkv_bm_num_free_blocks.argtypes = [_P]
_lib.pkv_bm_num_free_blocks.restype = _i64
_lib.pkv_bm_add_sequence.argtypes = [_P, _i64, _i64]
_lib.pkv_bm_add_sequence.restype = ctypes.c_int
_lib.pkv_bm_append_slots.argtypes = [_P, _P, _i32, _P]
_lib.pkv_bm_append_slots.restype = ctypes.c_int
_lib.pkv_bm_free_sequence.argtypes = [_P, _i64]
_lib.pkv_bm_free_sequence.restype = ctypes.c_int
_lib.pkv_bm_fork.argtypes = [_P, _i64, _i64]
_lib.pkv_bm_fork.restype = ctypes.c_int
_lib.pkv_bm_append_slots_cow.argtypes = [_P, _P, _i32, _P, _P, _P, ctypes.POINTER(ctypes.c_int32)]
_lib.pkv_bm_append_slots_cow.restype = ctypes.c_int
_lib.pkv_bm_truncate.argtypes = [_P, _i64, _i64]
_lib.pkv_bm_truncate.restype = ctypes.c_int
_lib.pkv_bm_ref_count.argtypes = [_P, _i32]
_lib.pkv_bm_ref_count.restype = _i32
_lib.pkv_bm_compact.argtypes = [_P, _P, _i64, ctypes.POINTER(ctypes.c_int64), _P]
_lib.pkv_bm_compact.restype = ctypes.c_int
_lib.pkv_bm_preempt_lifo.argtypes = [_P, ctypes.POINTER(ctypes.c_int64)]
_lib.pkv_bm_preempt_lifo.restype = ctypes.c_int
_lib.pkv_bm_block_tables.argtypes = [_P, _P, _i32, _i32, _P, _P]
_lib.pkv_bm_block_tables.restype = ctypes.c_int
_lib.pkv_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
_lib.pkv_device_errors.restype = ctypes.c_int
_lib.pkv_last_error.argtypes = []
_lib.pkv_last_error.restype = ctypes.c_char_p


def lib() -> ctypes.CDLL:
    return _lib


def _check(rc: int, where: str):
    if rc != PKV_OK:
        raise PkvError(rc, where)


def _stream(stream: Optional[torch.cuda.Stream], dev: Optional[int] = None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without the Stream object (0.2 against 2.8 us)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)


def _word(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, ndim: int, host_ok: bool = False):
    """host_ok: a page-locked CPU tensor is accepted too (the kernels address it directly)."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda and not (host_ok and t.is_pinned()):
        raise ValueError(f"{name}: must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def cache_desc(k_cache: torch.Tensor) -> pkv_cache_desc:
    NB, Hkv, BS, D = k_cache.shape
    return pkv_cache_desc(NB, BS, Hkv, D)


def paged_kv_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """k/v [T, Hkv, D] bf16 are copied into k_cache/v_cache [NB, Hkv, BS, D] at their slots
    (k, v and slot_mapping may be pinned host tensors)."""
    _need(k, "k", torch.bfloat16, 3, True)
    _need(v, "v", torch.bfloat16, 3, True)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, True)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    if k.shape != v.shape or k_cache.shape != v_cache.shape:
        raise ValueError("k/v or k_cache/v_cache shapes differ")
    if k.shape[0] != slot_mapping.shape[0] or tuple(k.shape[1:]) != (k_cache.shape[1], k_cache.shape[3]):
        raise ValueError("k [T, Hkv, D] does not match slot_mapping [T] / cache [NB, Hkv, BS, D]")
    d = cache_desc(k_cache)
    _check(_lib.paged_kv_write(_ptr(k), _ptr(v), _ptr(slot_mapping), k.shape[0], _ptr(k_cache),
                               _ptr(v_cache), ctypes.byref(d), _stream(stream)), "paged_kv_write")


def paged_kv_write_rope(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                        positions: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, q: Optional[torch.Tensor] = None,
                        rotary_dim: Optional[int] = None, neox_style: bool = True,
                        stream=None) -> None:
    """RoPE of k (and q, in place) at `positions`, then the slot write of k and v."""
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(positions, "positions", torch.int64, 1)
    _need(cos_sin, "cos_sin", torch.float32, 2)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    if q is not None:
        _need(q, "q", torch.bfloat16, 3)
        if q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
            raise ValueError("q must be [T, Hq, D] with k's T and D")
    r = k.shape[2] if rotary_dim is None else int(rotary_dim)
    if cos_sin.shape[1] != r:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    if not (k.shape[0] == slot_mapping.shape[0] == positions.shape[0]):
        raise ValueError("k, slot_mapping and positions must have the same number of tokens")
    d = cache_desc(k_cache)
    _check(_lib.paged_kv_write_rope(_ptr(k), _ptr(v), _ptr(q), 0 if q is None else q.shape[1],
                                    _ptr(slot_mapping), _ptr(positions), k.shape[0], _ptr(cos_sin),
                                    cos_sin.shape[0], r, 1 if neox_style else 0, _ptr(k_cache),
                                    _ptr(v_cache), ctypes.byref(d), _stream(stream)),
           "paged_kv_write_rope")


def _one_device(where: torch.Tensor, **tensors) -> None:
    """The tensors are on one device, which is the current one (the library launches there)."""
    dev = where.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: on {t.device}, expected {where.device}")
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {where.device}, the current device is "
                         f"{torch.cuda.current_device()}")


def _home(t: torch.Tensor) -> int:
    """The device of t if it is the current one, else -2, which no tensor is on."""
    dev = t.get_device()  # (torch.cuda.current_device() takes 0.13 us more)
    return dev if dev >= 0 and dev == torch._C._cuda_getDevice() else -2


def _fine(dev: int, dtype, *tensors) -> bool:
    """Whether the tensors are contiguous, of `dtype` and on device `dev` (None: not given).  The
    checks that name what is wrong cost 0.5 us a tensor; a call makes them where this fails."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            return False
    return True


def _pointers(values) -> array.array:
    """A host array of device pointers (built faster than a ctypes one)."""
    return array.array("Q", values)


def _layers(k_caches, v_caches, dev: int, where: str):
    """(host arrays of the layers' K and V pointers, layer count, one layer's descriptor, a
    cache tensor) of 4-dim caches (one layer), 5-dim caches [layers, NB, Hkv, BS, D], or
    sequences of 4-dim caches."""
    if isinstance(k_caches, torch.Tensor):
        ndim = k_caches.dim()
        if ndim not in (4, 5):
            raise ValueError(f"{where}: k_caches must be [NB, Hkv, BS, D] or [layers, NB, Hkv, BS, D]")
        if not isinstance(v_caches, torch.Tensor):
            raise TypeError(f"{where}: k_caches and v_caches must be given alike")
        if not _fine(dev, torch.bfloat16, k_caches, v_caches):
            _need(k_caches, "k_caches", torch.bfloat16, ndim)
            _need(v_caches, "v_caches", torch.bfloat16, ndim)
            _one_device(k_caches, v_caches=v_caches)
        if k_caches.shape != v_caches.shape:
            raise ValueError(f"{where}: k_caches and v_caches shapes differ")
        n, NB, Hkv, BS, D = k_caches.shape if ndim == 5 else (1, *k_caches.shape)
        step = 2 * NB * Hkv * BS * D
        k0, v0 = k_caches.data_ptr(), v_caches.data_ptr()
        return (_pointers(range(k0, k0 + n * step, step) if step else [k0] * n),
                _pointers(range(v0, v0 + n * step, step) if step else [v0] * n), n,
                pkv_cache_desc(NB, BS, Hkv, D), k_caches)
    ks, vs = list(k_caches), list(v_caches)
    if len(ks) != len(vs) or not ks:
        raise ValueError(f"{where}: k_caches and v_caches need one cache per layer each")
    if not _fine(dev, torch.bfloat16, *ks, *vs):
        for t in ks + vs:
            _need(t, "a layer's cache", torch.bfloat16, 4)
            _one_device(ks[0], cache=t)
    shape = ks[0].shape
    if len(shape) != 4 or any(t.shape != shape for t in ks + vs):
        raise ValueError(f"{where}: the layers' caches must have one shape [NB, Hkv, BS, D]")
    return (_pointers([t.data_ptr() for t in ks]), _pointers([t.data_ptr() for t in vs]), len(ks),
            cache_desc(ks[0]), ks[0])


def paged_kv_copy_blocks(k_caches, v_caches, block_pairs: torch.Tensor,
                         num_tokens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Pages block_pairs[:, 0] are copied to pages block_pairs[:, 1] ([n, 2] int32) in every
    layer; with num_tokens [n] int32 only the first num_tokens[i] rows of pair i.

    The caches: one layer's [NB, Hkv, BS, D], all layers in one [layers, NB, Hkv, BS, D], or
    a list of the layers' caches.  No destination may be another pair's source or destination.
    """
    dev = _home(block_pairs)
    kp, vp, n, d, first = _layers(k_caches, v_caches, dev, "paged_kv_copy_blocks")
    if not _fine(dev, torch.int32, block_pairs, num_tokens):
        _need(block_pairs, "block_pairs", torch.int32, 2)
        if num_tokens is not None:
            _need(num_tokens, "num_tokens", torch.int32, 1)
        _one_device(first, block_pairs=block_pairs, num_tokens=num_tokens)
    shape = block_pairs.shape
    if len(shape) != 2 or shape[1] != 2:
        raise ValueError("block_pairs must be [n, 2]")
    if num_tokens is not None and num_tokens.shape != shape[:1]:
        raise ValueError("num_tokens must have one entry per pair")
    _check(_lib.paged_kv_copy_blocks(kp.buffer_info()[0], vp.buffer_info()[0], n,
                                     block_pairs.data_ptr(), _ptr(num_tokens), shape[0],
                                     ctypes.byref(d), _stream(stream, dev)), "paged_kv_copy_blocks")


def paged_kv_compact(k_caches, v_caches, block_moves: torch.Tensor,
                     block_tables: Optional[torch.Tensor] = None,
                     block_map: Optional[torch.Tensor] = None, stream=None) -> None:
    """Pages block_moves[:, 0] move to the free pages block_moves[:, 1] ([n, 2] int32) in
    every layer, and block_tables [B, M] int32 is rewritten in place through block_map [NB]
    int32 (BlockManager.compact plans both; caches as in paged_kv_copy_blocks)."""
    dev = _home(block_moves)
    kp, vp, n, d, first = _layers(k_caches, v_caches, dev, "paged_kv_compact")
    if not _fine(dev, torch.int32, block_moves, block_tables, block_map):
        _need(block_moves, "block_moves", torch.int32, 2)
        if block_tables is not None:
            _need(block_tables, "block_tables", torch.int32, 2)
        if block_map is not None:
            _need(block_map, "block_map", torch.int32, 1)
        _one_device(first, block_moves=block_moves, block_tables=block_tables, block_map=block_map)
    shape = block_moves.shape
    if len(shape) != 2 or shape[1] != 2:
        raise ValueError("block_moves must be [n, 2]")
    rows = cols = 0
    if block_tables is not None:
        if block_tables.dim() != 2:
            raise ValueError("block_tables must be [B, M]")
        if block_map is None or block_map.shape != (d.num_blocks,):
            raise ValueError("block_tables need a block_map with one entry per block")
        rows, cols = block_tables.shape
    _check(_lib.paged_kv_compact(kp.buffer_info()[0], vp.buffer_info()[0], n,
                                 block_moves.data_ptr(), shape[0], _ptr(block_tables), rows, cols,
                                 _ptr(block_map), ctypes.byref(d), _stream(stream, dev)),
           "paged_kv_compact")


PATH_PARTITIONS, PATH_CLUSTER, PATH_PERSISTENT = 1, 2, 3
CONSUMER_TENSOR, CONSUMER_FMA = 0, 1


def pkv_set_decode_consumer(consumer: int) -> int:
    """Selects the consumer warps' arithmetic of the partition decode kernel (CONSUMER_*);
    returns the previous one."""
    rc = int(_lib.pkv_set_decode_consumer(consumer))
    if rc < 0:
        _check(rc, "pkv_set_decode_consumer")
    return rc


def pkv_decode_ctas_per_sm(head_dim: int, path: int) -> int:
    """CTAs per SM of the decode kernel of `path` (PATH_*) on the current device."""
    n = int(_lib.pkv_decode_ctas_per_sm(head_dim, path))
    if n < 0:
        _check(n, "pkv_decode_ctas_per_sm")
    return n


def paged_decode_path(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                      max_context_len: int, num_sms: int = 0) -> int:
    """Kernel arrangement paged_decode_attention launches for these sizes (PATH_*; 0 if none)."""
    return int(_lib.paged_decode_path(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                      max_context_len, num_sms))


def paged_decode_plan(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                      max_context_len: int, num_sms: int = 0) -> int:
    """Partition size (tokens) paged_decode_attention cuts each (sequence, kv head) into."""
    return int(_lib.paged_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                      max_context_len, num_sms))


def paged_decode_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                max_context_len: int) -> int:
    return int(_lib.paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                max_context_len))


def paged_decode_split_workspace_size(num_seqs: int, num_q_heads: int, head_dim: int,
                                      max_context_len: int, partition_tokens: int) -> int:
    return int(_lib.paged_decode_split_workspace_size(num_seqs, num_q_heads, head_dim,
                                                      max_context_len, partition_tokens))


def _decode_checks(q, k_cache, v_cache, block_tables, context_lens, host_ok=False):
    _need(q, "q", torch.bfloat16, 3, host_ok)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2, host_ok)
    _need(context_lens, "context_lens", torch.int32, 1, host_ok)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    B = q.shape[0]
    if block_tables.shape[0] != B or context_lens.shape[0] != B or q.shape[2] != k_cache.shape[3]:
        raise ValueError("q [B, Hq, D], block_tables [B, M], context_lens [B], cache [NB, Hkv, BS, D] disagree")


def paged_decode_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, max_context_len: int, scale: float,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """out [B, Hq, D] bf16 = paged GQA decode attention (split + combine when the plan says so).

    ``workspace`` (uint8, CUDA, zero-filled before its first use and before a call with
    another number of sequences or kv heads) may be omitted; then a zeroed buffer of
    ``paged_decode_workspace_size`` bytes is taken from torch's allocator.
    out, q, block_tables and context_lens may be pinned host tensors (read and written
    by the kernels over the host link).
    """
    _decode_checks(q, k_cache, v_cache, block_tables, context_lens, host_ok=True)
    _need(out, "out", torch.bfloat16, 3, True)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    B, Hq, D = q.shape
    need = paged_decode_workspace_size(B, Hq, k_cache.shape[1], D, max_context_len)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=k_cache.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    d = cache_desc(k_cache)
    _check(_lib.paged_decode_attention(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(block_tables), block_tables.shape[1],
                                       _ptr(context_lens), int(max_context_len), B, Hq,
                                       ctypes.byref(d), float(scale), _ptr(workspace), ws_bytes,
                                       _stream(stream)), "paged_decode_attention")


SHARED_AUTO, SHARED_ALWAYS, SHARED_NEVER = 0, 1, 2


def pkv_set_shared_prefix(mode: int) -> int:
    """Whether paged_decode_shared_prefix_attention shares (SHARED_*); returns the previous mode."""
    rc = int(_lib.pkv_set_shared_prefix(mode))
    if rc < 0:
        _check(rc, "pkv_set_shared_prefix")
    return rc


def paged_decode_shared_prefix_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                              head_dim: int, num_groups: int, max_prefix_len: int,
                                              max_suffix_len: int) -> int:
    return int(_lib.paged_decode_shared_prefix_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim, num_groups, max_prefix_len, max_suffix_len))


def paged_decode_shared_prefix_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                                         context_lens: torch.Tensor, group_start: torch.Tensor,
                                         prefix_lens: torch.Tensor, max_prefix_len: int,
                                         max_suffix_len: int, scale: float,
                                         workspace: Optional[torch.Tensor] = None,
                                         stream=None) -> None:
    """paged_decode_attention where the sequences group_start[g] .. group_start[g+1]-1 share
    the pages of their first prefix_lens[g] tokens, which are read once per group.

    max_suffix_len bounds every context_len less the whole pages of its prefix.  ``workspace``
    (uint8, CUDA, ``paged_decode_shared_prefix_workspace_size`` bytes, zero-filled before its
    first use) serves calls of any sizes in turn, but none of paged_decode_attention's; it may
    be omitted as there.
    """
    dev = _home(q)
    if not (_fine(dev, torch.bfloat16, q, out, k_cache, v_cache) and
            _fine(dev, torch.int32, block_tables, context_lens, group_start, prefix_lens)):
        _decode_checks(q, k_cache, v_cache, block_tables, context_lens)
        _need(out, "out", torch.bfloat16, 3)
        _need(group_start, "group_start", torch.int32, 1)
        _need(prefix_lens, "prefix_lens", torch.int32, 1)
        _one_device(q, out=out, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                    context_lens=context_lens, group_start=group_start, prefix_lens=prefix_lens)
    if q.dim() != 3 or k_cache.dim() != 4 or block_tables.dim() != 2 or prefix_lens.dim() != 1:
        raise ValueError("q [B, Hq, D], cache [NB, Hkv, BS, D], block_tables [B, M], prefix_lens [G]")
    B, Hq, D = q.shape
    NB, Hkv, BS, Dk = k_cache.shape
    rows, cols = block_tables.shape
    groups = prefix_lens.shape[0]
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if rows != B or Dk != D or context_lens.shape != (B,):
        raise ValueError("q [B, Hq, D], block_tables [B, M], context_lens [B], cache [NB, Hkv, BS, D] disagree")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if group_start.shape != (groups + 1,):
        raise ValueError("group_start must be [G + 1] for prefix_lens [G]")
    if workspace is None:
        need = paged_decode_shared_prefix_workspace_size(B, Hq, Hkv, D, groups, max_prefix_len,
                                                         max_suffix_len)
        with torch.cuda.stream(stream):  # zeroed, and given back, in that stream's order
            workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the current device")
    d = pkv_cache_desc(NB, BS, Hkv, D)
    _check(_lib.paged_decode_shared_prefix_attention(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), cols, context_lens.data_ptr(), group_start.data_ptr(),
        prefix_lens.data_ptr(), groups, int(max_prefix_len), int(max_suffix_len), B, Hq,
        ctypes.byref(d), float(scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream, dev)), "paged_decode_shared_prefix_attention")


def paged_decode_step(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor,
                      max_context_len: int, scale: float, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """One decode step: the slot write of k/v, then attention over the updated caches.
    out, q, k, v, slot_mapping, block_tables and context_lens may be pinned host tensors:
    the kernels then read and write them over the host link (no copies)."""
    _decode_checks(q, k_cache, v_cache, block_tables, context_lens, host_ok=True)
    _need(out, "out", torch.bfloat16, 3, True)
    _need(k, "k", torch.bfloat16, 3, True)
    _need(v, "v", torch.bfloat16, 3, True)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, True)
    if out.shape != q.shape or k.shape != v.shape or k.shape[0] != slot_mapping.shape[0]:
        raise ValueError("out/q, k/v or slot_mapping shapes disagree")
    B, Hq, D = q.shape
    need = paged_decode_workspace_size(B, Hq, k_cache.shape[1], D, max_context_len)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=k_cache.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    d = cache_desc(k_cache)
    _check(_lib.paged_decode_step(_ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(slot_mapping),
                                  k.shape[0], _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                  block_tables.shape[1], _ptr(context_lens), int(max_context_len),
                                  B, Hq, ctypes.byref(d), float(scale), _ptr(workspace), ws_bytes,
                                  _stream(stream)), "paged_decode_step")


def paged_decode_step_rope(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           slot_mapping: torch.Tensor, positions: torch.Tensor,
                           cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           max_context_len: int, scale: float, rotary_dim: Optional[int] = None,
                           neox_style: bool = True, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """One decode step with RoPE: rotate q (in place) and k at `positions`, write k/v at
    their slots, then attention over the updated caches.  Token b is sequence b's."""
    _decode_checks(q, k_cache, v_cache, block_tables, context_lens)
    _need(out, "out", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(positions, "positions", torch.int64, 1)
    _need(cos_sin, "cos_sin", torch.float32, 2)
    B, Hq, D = q.shape
    if out.shape != q.shape or k.shape != v.shape or k.shape[0] != B or k.shape[2] != D:
        raise ValueError("out/q, k/v shapes disagree (one new token per sequence)")
    if not (slot_mapping.shape[0] == positions.shape[0] == B):
        raise ValueError("slot_mapping and positions need one entry per sequence")
    r = D if rotary_dim is None else int(rotary_dim)
    if cos_sin.shape[1] != r:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    need = paged_decode_workspace_size(B, Hq, k_cache.shape[1], D, max_context_len)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=k_cache.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    d = cache_desc(k_cache)
    _check(_lib.paged_decode_step_rope(_ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(slot_mapping),
                                       _ptr(positions), _ptr(cos_sin), cos_sin.shape[0], r,
                                       1 if neox_style else 0, _ptr(k_cache), _ptr(v_cache),
                                       _ptr(block_tables), block_tables.shape[1],
                                       _ptr(context_lens), int(max_context_len), B, Hq,
                                       ctypes.byref(d), float(scale), _ptr(workspace), ws_bytes,
                                       _stream(stream)), "paged_decode_step_rope")


def paged_prefill_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, max_context_len: int,
                            query_start: torch.Tensor, max_query_len: int, scale: float,
                            stream=None) -> None:
    """Causal attention of each sequence's last n_b cached tokens (packed q [Nq, Hq, D])."""
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(query_start, "query_start", torch.int32, 1)
    B = context_lens.shape[0]
    if out.shape != q.shape or query_start.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("out/q, query_start [B+1] or block_tables [B, M] disagree")
    d = cache_desc(k_cache)
    _check(_lib.paged_prefill_attention(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_tables), block_tables.shape[1],
                                        _ptr(context_lens), int(max_context_len),
                                        _ptr(query_start), int(max_query_len), B, q.shape[1],
                                        ctypes.byref(d), float(scale), _stream(stream)),
           "paged_prefill_attention")


def prompt_attention(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     query_start: torch.Tensor, max_query_len: int, scale: float,
                     stream=None) -> None:
    """Causal attention over whole prompts packed one after another: out, q [T, Hq, D], k, v
    [T, Hkv, D] bf16 (each token's heads contiguous; the tokens may be strided, e.g. slices
    of a fused projection), sequence b at rows query_start[b] .. query_start[b+1]-1."""
    dev, bf = _home(q), torch.bfloat16
    shape, kv = q.shape, k.shape
    so, sq, sk, sv = out.stride(), q.stride(), k.stride(), v.stride()
    if not (q.dtype is bf and k.dtype is bf and v.dtype is bf and out.dtype is bf and
            len(shape) == 3 and len(kv) == 3 and out.shape == shape and v.shape == kv and
            kv[0] == shape[0] and kv[2] == shape[2] and so[2] == sq[2] == sk[2] == sv[2] == 1 and
            (shape[1] == 1 or so[1] == sq[1] == shape[2]) and
            (kv[1] == 1 or sk[1] == sv[1] == shape[2])):
        _prompt_checks(out, q, k, v)
    if not (out.get_device() == dev == k.get_device() == v.get_device() and
            _fine(dev, torch.int32, query_start)):
        _need(query_start, "query_start", torch.int32, 1)
        if not q.is_cuda:
            raise ValueError("q: must be a CUDA tensor")
        _one_device(q, out=out, k=k, v=v, query_start=query_start)
    if query_start.dim() != 1:
        raise ValueError("query_start must be [B + 1]")
    T, Hq, D = shape
    Hkv, seqs = kv[1], query_start.shape[0] - 1
    if seqs < 0:
        raise ValueError("query_start must be [B + 1]")
    if T <= 1:  # one token has no next one: any stride will do
        so = sq = (Hq * D,)
        sk = sv = (Hkv * D,)
    _check(_lib.prompt_attention(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), so[0],
                                 sq[0], sk[0], sv[0], query_start.data_ptr(), T,
                                 int(max_query_len), seqs, Hq, Hkv, D, float(scale),
                                 _stream(stream, dev)), "prompt_attention")


def _prompt_checks(out, q, k, v) -> None:
    """Raises for what is wrong with prompt_attention's rows."""
    T, _, D = q.shape if q.dim() == 3 else (0, 0, 0)
    for t, name in ((out, "out"), (q, "q"), (k, "k"), (v, "v")):
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
        shape = t.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != D:
            raise ValueError(f"{name}: expected [T, heads, D] with q's T and D, got shape {tuple(shape)}")
        step, head, one = t.stride()
        if T > 0 and (one != 1 or (shape[1] > 1 and head != D)):
            raise ValueError(f"{name}: a token's heads must be contiguous")
    if out.shape != q.shape or k.shape != v.shape:
        raise ValueError("out must have q's shape, and v k's")


# ---- the 8-bit cache: codes [NB, Hkv, BS, D] int8 or float8_e4m3fn, scales [NB, Hkv] float32

Q8_E4M3, Q8_INT8 = 0, 1
# pkv_call_q8's words (14 arguments of a call cost ctypes 1.1 us, packed 0.4)
_CALL_WRITE, _CALL_READ, _CALL_WRITE_ROPE, _CALL_DECODE, _CALL_PREFILL, _CALL_STEP, _CALL_STEP_ROPE = range(7)
_call_q8 = _lib.pkv_call_q8
_pack_rows, _pack_rope = struct.Struct("14q7q").pack, struct.Struct("14q7q10q").pack
_pack_decode, _pack_prefill = struct.Struct("14q4qd2q").pack, struct.Struct("14q4qd2q3q").pack
_pack_step, _pack_step_rope = struct.Struct("14q4qd2q4q").pack, struct.Struct("14q4qd2q4q7q").pack
_BF16, _F32, _I32, _I8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.float8_e4m3fn


def _q8_cache(dev: int, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start=None, shape=None):
    """The words of pkv_call_q8 up to num_seqs, of tensors on device `dev`, checked in one expression (a call's
    checks were 9 of its 12 us when each tensor had its own); _q8_wrong names what fails."""
    kt = k_cache.dtype
    if not (kt is v_cache.dtype and (kt is _I8 or kt is _E4M3) and k_scale.dtype is _F32 and
            v_scale.dtype is _F32 and block_tables.dtype is _I32 and context_lens.dtype is _I32 and
            dev == k_cache.get_device() == v_cache.get_device() == k_scale.get_device() ==
            v_scale.get_device() == block_tables.get_device() == context_lens.get_device() and
            k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and
            v_scale.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous() and
            (query_start is None or (query_start.dtype is _I32 and query_start.get_device() == dev and
                                     query_start.is_contiguous()))):
        _q8_wrong(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start)
    if shape is None:
        shape = k_cache.shape
    B, = context_lens.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [NB, Hkv, BS, D], alike")
    NB, Hkv, BS, D = shape
    heads = (NB, Hkv)
    if k_scale.shape != heads or v_scale.shape != heads:
        raise ValueError("k_scale and v_scale must be [NB, Hkv]")
    bt = block_tables.shape
    if len(bt) != 2 or bt[0] != B:
        raise ValueError("block_tables must be [B, M] and context_lens [B]")
    if query_start is not None and query_start.shape != (B + 1,):
        raise ValueError("query_start must be [B + 1] for context_lens [B]")
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            Q8_INT8 if kt is _I8 else Q8_E4M3, NB, BS, Hkv, D, block_tables.data_ptr(), bt[1], context_lens.data_ptr(), B)


def _q8_wrong(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start) -> None:
    """Raises for what is wrong with the 8-bit cache's tensors."""
    if k_cache.dtype not in (_I8, _E4M3):
        raise TypeError(f"k_cache: expected torch.int8 or torch.float8_e4m3fn, got {k_cache.dtype}")
    _need(k_cache, "k_cache", k_cache.dtype, 4)
    _need(v_cache, "v_cache", k_cache.dtype, 4)
    _need(k_scale, "k_scale", _F32, 2)
    _need(v_scale, "v_scale", _F32, 2)
    _need(block_tables, "block_tables", _I32, 2)
    _need(context_lens, "context_lens", _I32, 1)
    if query_start is not None:
        _need(query_start, "query_start", _I32, 1)
    _one_device(k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, block_tables=block_tables,
                context_lens=context_lens, query_start=query_start)
    raise ValueError("the cache and the rows are on different devices")


def _packed(t: torch.Tensor, name: str, tokens: int, D: int, dev: int) -> int:
    """The token stride of rows t [tokens, heads, D] bf16 whose heads are contiguous."""
    shape = t.shape
    if t.dtype is not _BF16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if len(shape) != 3 or shape[0] != tokens or shape[2] != D:
        raise ValueError(f"{name}: expected [{tokens}, heads, {D}], got shape {tuple(shape)}")
    step, head, one = t.stride()
    if tokens > 0 and (one != 1 or (shape[1] > 1 and head != D)):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor")
        raise ValueError(f"{name}: on {t.device}, not where the other tensors and the current device are")
    return step if tokens > 1 else shape[1] * D


def _q8_rows(k, v, cache, names=("k", "v")):
    """(device, tokens, strides) of k and v [T, Hkv, D] for a cache of shape `cache`."""
    shape = k.shape
    if (len(shape) != 3 or len(cache) != 4 or v.shape != shape or shape[1] != cache[1] or
            shape[2] != cache[3]):
        raise ValueError(f"{names[0]} and {names[1]} must be [T, Hkv, D] for a cache [NB, Hkv, BS, D]")
    T, H, D = shape
    dev = _home(k)
    sk, sv = k.stride(), v.stride()
    if (k.dtype is _BF16 and v.dtype is _BF16 and k.get_device() == dev == v.get_device() and T > 1 and
            sk[2] == 1 == sv[2] and sk[1] == D == sv[1]):
        return dev, T, sk[0], sv[0]
    return dev, T, _packed(k, names[0], T, D, dev), _packed(v, names[1], T, D, dev)


def paged_kv_write_q8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, query_start: Optional[torch.Tensor] = None,
                      max_query_len: int = 1, stream=None) -> None:
    """Each sequence's newest tokens, rows query_start[b] .. query_start[b+1]-1 of k and v
    [T, Hkv, D] (the tokens may be strided), quantised into its pages at positions
    context_lens[b] - n .. context_lens[b] - 1.  Without query_start: one token per sequence."""
    shape = k_cache.shape
    dev, T, sk, sv = _q8_rows(k, v, shape)
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start, shape)
    _check(_call_q8(_CALL_WRITE, _pack_rows(
        *cache, _stream(stream, dev), k.data_ptr(), v.data_ptr(), sk, sv, _word(query_start), T, max_query_len)),
        "paged_kv_write_q8")


def paged_kv_write_rope_q8(k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           query_start: Optional[torch.Tensor] = None, max_query_len: int = 1,
                           q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                           positions: Optional[torch.Tensor] = None, rotary_dim: Optional[int] = None,
                           neox_style: bool = True, stream=None) -> None:
    """paged_kv_write_q8 of the rotated k; the rotated q goes to q_out (default: q itself).
    positions [T] int64 default to the tokens' positions in their sequences."""
    shape = k_cache.shape
    dev, T, sk, sv = _q8_rows(k, v, shape)
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start, shape)
    sq = so = heads = 0
    if q is not None:
        q_out = q if q_out is None else q_out
        rows, D = q.shape, shape[3]
        if len(rows) != 3 or q_out.shape != rows:
            raise ValueError("q must be [T, Hq, D], and q_out alike")
        (sq, h, one), (so, h_out, one_out) = q.stride(), q_out.stride()
        if not (q.dtype is _BF16 and q_out.dtype is _BF16 and q.get_device() == dev == q_out.get_device() and
                rows[0] == T > 1 and rows[2] == D and one == 1 == one_out and h == D == h_out):
            sq, so = _packed(q, "q", T, D, dev), _packed(q_out, "q_out", T, D, dev)
        heads = rows[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    r = _rope_table(cos_sin, positions, k.shape[2] if rotary_dim is None else int(rotary_dim), T, dev)
    _check(_call_q8(_CALL_WRITE_ROPE, _pack_rope(
        *cache, _stream(stream, dev), k.data_ptr(), v.data_ptr(), sk, sv, _word(query_start), T, max_query_len,
        _word(q), _word(q_out), sq, so, heads, _word(positions), cos_sin.data_ptr(), cos_sin.shape[0], r,
        1 if neox_style else 0)), "paged_kv_write_rope_q8")


def _rope_table(cos_sin, positions, r: int, tokens: int, dev: int) -> int:
    if not (cos_sin.dtype is _F32 and cos_sin.get_device() == dev and cos_sin.is_contiguous() and
            (positions is None or _fine(dev, torch.int64, positions))):
        _need(cos_sin, "cos_sin", torch.float32, 2)
        if positions is not None:
            _need(positions, "positions", torch.int64, 1)
        raise ValueError("cos_sin and positions: on another device than the rows")
    shape = cos_sin.shape
    if len(shape) != 2 or shape[1] != r:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    if positions is not None and positions.shape != (tokens,):
        raise ValueError("positions must have one entry per token")
    return r


def paged_kv_read_q8(k_out: torch.Tensor, v_out: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                     context_lens: torch.Tensor, query_start: Optional[torch.Tensor] = None,
                     max_query_len: int = 1, stream=None) -> None:
    """Each sequence's newest query_start[b+1] - query_start[b] tokens back as bf16 rows
    query_start[b] .. of k_out and v_out [T, Hkv, D] (the tokens may be strided)."""
    shape = k_cache.shape
    dev, T, sk, sv = _q8_rows(k_out, v_out, shape, ("k_out", "v_out"))
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start, shape)
    _check(_call_q8(_CALL_READ, _pack_rows(
        *cache, _stream(stream, dev), k_out.data_ptr(), v_out.data_ptr(), sk, sv, _word(query_start), T, max_query_len)),
        "paged_kv_read_q8")


def paged_decode_q8_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                   max_context_len: int) -> int:
    return int(_lib.paged_decode_q8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len))


def paged_prefill_q8_workspace_size(num_seqs: int, num_kv_heads: int, head_dim: int, block_size: int,
                                    max_context_len: int) -> int:
    """For any call of these sizes: fp16 rows of num_seqs contexts of max_context_len.  (By tokens: the block
    size makes no difference.)"""
    return int(_lib.paged_prefill_q8_workspace_size(num_seqs, num_kv_heads, head_dim, max_context_len))


def paged_prefill_q8_workspace_size_for(num_queries: int, max_query_len: int, num_seqs: int, num_q_heads: int,
                                        num_kv_heads: int, head_dim: int, max_context_len: int) -> int:
    """For a call of these sizes: a few MB where its few queries need no rows, else rows for all sequences, or 8 GB
    of them at a time.  (Less is taken too, down to one sequence's rows.)"""
    return int(_lib.paged_prefill_q8_workspace_size_for(num_queries, max_query_len, num_seqs, num_q_heads, num_kv_heads,
                                                        head_dim, max_context_len))


def _q8_query(out, q, cache, rows: Optional[int], dev: int) -> None:
    if not (q.dtype is _BF16 and out.dtype is _BF16 and q.get_device() == dev == out.get_device() and
            q.is_contiguous() and out.is_contiguous()):
        _need(q, "q", torch.bfloat16, 3)
        _need(out, "out", torch.bfloat16, 3)
        _one_device(q, out=out)
    shape = q.shape
    if len(shape) != 3 or len(cache) != 4 or shape[2] != cache[3] or (rows is not None and shape[0] != rows):
        raise ValueError("q must be [rows, Hq, D] for a cache [NB, Hkv, BS, D]")
    if out.shape != shape:
        raise ValueError("out must have q's shape")


def _q8_workspace(workspace, need: int, zeroed: bool, like: torch.Tensor, dev: int, stream) -> torch.Tensor:
    if workspace is None:
        with torch.cuda.stream(stream):  # made, and given back, in that stream's order
            make = torch.zeros if zeroed else torch.empty
            return make(max(need, 1), dtype=torch.uint8, device=like.device)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the current device")
    return workspace


def paged_decode_attention_q8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, max_context_len: int, scale: float,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """paged_decode_attention over an 8-bit cache.  ``workspace`` (uint8, CUDA,
    ``paged_decode_q8_workspace_size`` bytes, zero-filled before its first use) serves calls of
    any sizes in turn; it may be omitted as there."""
    dev = _home(q)
    shape = k_cache.shape
    _q8_query(out, q, shape, context_lens.shape[0], dev)
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, None, shape)
    _, Hq, D = q.shape
    workspace = _q8_workspace(workspace, 0 if workspace is not None else paged_decode_q8_workspace_size(
        cache[12], Hq, cache[7], D, int(max_context_len)), True, q, dev, stream)
    _check(_call_q8(_CALL_DECODE, _pack_decode(
        *cache, _stream(stream, dev), out.data_ptr(), q.data_ptr(), max_context_len, Hq, scale, workspace.data_ptr(),
        workspace.nbytes)), "paged_decode_attention_q8")


def paged_decode_step_q8(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                         max_context_len: int, scale: float, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """One decode step over an 8-bit cache: paged_kv_write_q8 of one token per sequence, then
    paged_decode_attention_q8 of q [B, Hq, D] (k, v [B, Hkv, D], tokens may be strided)."""
    shape = k_cache.shape
    dev, T, sk, sv = _q8_rows(k, v, shape)
    _q8_query(out, q, shape, T, dev)
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, None, shape)
    _, Hq, D = q.shape
    if cache[12] != T:
        raise ValueError("q, k and v need one row per sequence")
    workspace = _q8_workspace(workspace, 0 if workspace is not None else paged_decode_q8_workspace_size(
        cache[12], Hq, cache[7], D, int(max_context_len)), True, q, dev, stream)
    _check(_call_q8(_CALL_STEP, _pack_step(
        *cache, _stream(stream, dev), out.data_ptr(), q.data_ptr(), max_context_len, Hq, scale, workspace.data_ptr(),
        workspace.nbytes, k.data_ptr(), v.data_ptr(), sk, sv)), "paged_decode_step_q8")


def paged_decode_step_rope_q8(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, max_context_len: int, scale: float,
                              q_out: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                              rotary_dim: Optional[int] = None, neox_style: bool = True,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """paged_decode_step_q8 with RoPE: q [B, Hq, D] (tokens may be strided) is rotated into the
    contiguous q_out (default: q itself), k on its way into the cache."""
    shape = k_cache.shape
    dev, T, sk, sv = _q8_rows(k, v, shape)
    q_out = q if q_out is None else q_out
    _q8_query(out, q_out, shape, T, dev)
    if q.shape != q_out.shape:
        raise ValueError("q_out must have q's shape")
    sq = _packed(q, "q", T, k.shape[2], dev)
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, None, shape)
    _, Hq, D = q.shape
    if cache[12] != T:
        raise ValueError("q, k and v need one row per sequence")
    r = _rope_table(cos_sin, positions, D if rotary_dim is None else int(rotary_dim), T, dev)
    workspace = _q8_workspace(workspace, 0 if workspace is not None else paged_decode_q8_workspace_size(
        cache[12], Hq, cache[7], D, int(max_context_len)), True, q, dev, stream)
    _check(_call_q8(_CALL_STEP_ROPE, _pack_step_rope(
        *cache, _stream(stream, dev), out.data_ptr(), q.data_ptr(), max_context_len, Hq, scale, workspace.data_ptr(),
        workspace.nbytes, k.data_ptr(), v.data_ptr(), sk, sv, sq, q_out.data_ptr(), _word(positions), cos_sin.data_ptr(),
        cos_sin.shape[0], r, 1 if neox_style else 0)), "paged_decode_step_rope_q8")


def paged_prefill_attention_q8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, max_context_len: int, query_start: torch.Tensor,
                               max_query_len: int, scale: float, workspace: Optional[torch.Tensor] = None,
                               stream=None) -> None:
    """paged_prefill_attention over an 8-bit cache.  ``workspace``: uint8, CUDA,
    ``paged_prefill_q8_workspace_size`` (or ``_size_for``) bytes with any contents; it may be omitted."""
    dev = _home(q)
    shape = k_cache.shape
    _q8_query(out, q, shape, None, dev)
    if query_start is None:
        raise ValueError("query_start must be [B + 1]")
    cache = _q8_cache(dev, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start, shape)
    workspace = _q8_workspace(workspace, 0 if workspace is not None else paged_prefill_q8_workspace_size_for(
        q.shape[0], int(max_query_len), cache[12], q.shape[1], cache[7], cache[8], int(max_context_len)), False, q, dev, stream)
    _check(_call_q8(_CALL_PREFILL, _pack_prefill(
        *cache, _stream(stream, dev), out.data_ptr(), q.data_ptr(), max_context_len, q.shape[1], scale,
        workspace.data_ptr(), workspace.nbytes, q.shape[0], query_start.data_ptr(), max_query_len)),
        "paged_prefill_attention_q8")


def _q8_layers(dev: int, k_caches, v_caches, k_scales, v_scales, where: str):
    """(array of pkv_q8_cache, layers, descriptor, the first k cache) of one layer's tensors, of
    tensors with the layers in front, or of sequences of the layers' tensors."""
    if isinstance(k_caches, torch.Tensor):
        tensors = (k_caches, v_caches, k_scales, v_scales)
        if not all(isinstance(t, torch.Tensor) for t in tensors):
            raise TypeError(f"{where}: the caches and scales must be given alike")
        if k_caches.dim() == 5:
            for t, name, n in zip(tensors, ("k_caches", "v_caches", "k_scales", "v_scales"), (5, 5, 3, 3)):
                if t.dim() != n or t.shape[0] != k_caches.shape[0]:
                    raise ValueError(f"{where}: {name} must have the layers in front, as k_caches has")
            layers = list(zip(*(t.unbind(0) for t in tensors)))
        else:
            layers = [tensors]
    else:
        layers = list(zip(list(k_caches), list(v_caches), list(k_scales), list(v_scales), strict=True))
    if not layers:
        raise ValueError(f"{where}: no layers")
    first = layers[0][0]
    none = torch.empty((0, 0), dtype=torch.int32, device=first.device), torch.empty(0, dtype=torch.int32,
                                                                                   device=first.device)
    out = (pkv_q8_cache * len(layers))()
    for i, tensors in enumerate(layers):
        if tensors[0].shape != first.shape or tensors[0].dtype != first.dtype:
            raise ValueError(f"{where}: the layers' caches must be alike")
        words = _q8_cache(dev, *tensors, *none)
        out[i] = pkv_q8_cache(*words[:5])
    NB, BS, Hkv, D = words[5:9]
    return out, len(layers), pkv_cache_desc(NB, BS, Hkv, D), first


def paged_kv_copy_blocks_q8(k_caches, v_caches, k_scales, v_scales, block_pairs: torch.Tensor,
                            num_tokens: Optional[torch.Tensor] = None, stream=None) -> None:
    """paged_kv_copy_blocks for 8-bit caches: rows and scales.  One layer's tensors [NB, Hkv, BS, D]
    and [NB, Hkv], all layers' with the layers in front, or lists of the layers'."""
    dev = _home(block_pairs)
    caches, n, d, first = _q8_layers(dev, k_caches, v_caches, k_scales, v_scales, "paged_kv_copy_blocks_q8")
    if not _fine(dev, torch.int32, block_pairs, num_tokens):
        _need(block_pairs, "block_pairs", torch.int32, 2)
        if num_tokens is not None:
            _need(num_tokens, "num_tokens", torch.int32, 1)
        _one_device(first, block_pairs=block_pairs, num_tokens=num_tokens)
    shape = block_pairs.shape
    if len(shape) != 2 or shape[1] != 2:
        raise ValueError("block_pairs must be [n, 2]")
    if num_tokens is not None and num_tokens.shape != shape[:1]:
        raise ValueError("num_tokens must have one entry per pair")
    _check(_lib.paged_kv_copy_blocks_q8(ctypes.addressof(caches), n, block_pairs.data_ptr(), _ptr(num_tokens),
                                        shape[0], ctypes.byref(d), _stream(stream, dev)), "paged_kv_copy_blocks_q8")


def paged_kv_compact_q8(k_caches, v_caches, k_scales, v_scales, block_moves: torch.Tensor,
                        block_tables: Optional[torch.Tensor] = None, block_map: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """paged_kv_compact for 8-bit caches (as in paged_kv_copy_blocks_q8)."""
    dev = _home(block_moves)
    caches, n, d, first = _q8_layers(dev, k_caches, v_caches, k_scales, v_scales, "paged_kv_compact_q8")
    if not _fine(dev, torch.int32, block_moves, block_tables, block_map):
        _need(block_moves, "block_moves", torch.int32, 2)
        if block_tables is not None:
            _need(block_tables, "block_tables", torch.int32, 2)
        if block_map is not None:
            _need(block_map, "block_map", torch.int32, 1)
        _one_device(first, block_moves=block_moves, block_tables=block_tables, block_map=block_map)
    shape = block_moves.shape
    if len(shape) != 2 or shape[1] != 2:
        raise ValueError("block_moves must be [n, 2]")
    rows = cols = 0
    if block_tables is not None:
        if block_tables.dim() != 2:
            raise ValueError("block_tables must be [B, M]")
        if block_map is None or block_map.shape != first.shape[:1]:
            raise ValueError("block_tables need a block_map with one entry per block")
        rows, cols = block_tables.shape
    _check(_lib.paged_kv_compact_q8(ctypes.addressof(caches), n, block_moves.data_ptr(), None, shape[0],
                                    _ptr(block_tables), rows, cols, _ptr(block_map), ctypes.byref(d),
                                    _stream(stream, dev)), "paged_kv_compact_q8")


def paged_decode_attention_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, max_context_len: int, scale: float,
                                   stream=None) -> None:
    """paged_decode_attention without a workspace: the library's fixed scratch array is used."""
    _decode_checks(q, k_cache, v_cache, block_tables, context_lens)
    _need(out, "out", torch.bfloat16, 3)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    B, Hq, D = q.shape
    d = cache_desc(k_cache)
    _check(_lib.paged_decode_attention_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                               _ptr(block_tables), block_tables.shape[1],
                                               _ptr(context_lens), int(max_context_len), B, Hq,
                                               ctypes.byref(d), float(scale), _stream(stream)),
           "paged_decode_attention_noalloc")


def paged_decode_split(o_part: torch.Tensor, lse_part: torch.Tensor, q: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, max_context_len: int, scale: float,
                       partition_tokens: int, stream=None) -> None:
    """o_part [B, Hq, n, D] fp32 and lse_part [B, Hq, n] fp32 for n = ceil(max_len / P)."""
    _decode_checks(q, k_cache, v_cache, block_tables, context_lens)
    _need(o_part, "o_part", torch.float32, 4)
    _need(lse_part, "lse_part", torch.float32, 3)
    B, Hq, D = q.shape
    n = -(-int(max_context_len) // int(partition_tokens)) if partition_tokens > 0 else 0
    if tuple(o_part.shape) != (B, Hq, n, D) or tuple(lse_part.shape) != (B, Hq, n):
        raise ValueError(f"o_part must be {(B, Hq, n, D)} and lse_part {(B, Hq, n)}")
    d = cache_desc(k_cache)
    _check(_lib.paged_decode_split(_ptr(o_part), _ptr(lse_part), _ptr(q), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                                   _ptr(context_lens), int(max_context_len), B, Hq,
                                   ctypes.byref(d), float(scale), int(partition_tokens),
                                   _stream(stream)), "paged_decode_split")


def paged_decode_combine(out: torch.Tensor, o_part: torch.Tensor, lse_part: torch.Tensor,
                         context_lens: torch.Tensor, max_context_len: int, partition_tokens: int,
                         stream=None) -> None:
    _need(out, "out", torch.bfloat16, 3)
    _need(o_part, "o_part", torch.float32, 4)
    _need(lse_part, "lse_part", torch.float32, 3)
    _need(context_lens, "context_lens", torch.int32, 1)
    B, Hq, D = out.shape
    _check(_lib.paged_decode_combine(_ptr(out), _ptr(o_part), _ptr(lse_part), _ptr(context_lens),
                                     int(max_context_len), B, Hq, D, int(partition_tokens),
                                     _stream(stream)), "paged_decode_combine")


def pkv_device_errors(clear: bool = True) -> int:
    """Synchronises the device and returns the device error bits (PKV_DEVERR_*)."""
    f = ctypes.c_uint32(0)
    _check(_lib.pkv_device_errors(ctypes.byref(f), 1 if clear else 0), "pkv_device_errors")
    return int(f.value)


def pkv_last_error() -> str:
    return _lib.pkv_last_error().decode(errors="replace")


class BlockManager:
    """The library's host block allocator (pkv_bm_*): block tables and slot mappings."""

    def __init__(self, num_blocks: int, block_size: int):
        self._h = _lib.pkv_bm_create(int(num_blocks), int(block_size))
        if not self._h:
            raise PkvError(-2, "pkv_bm_create")
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            _lib.pkv_bm_destroy(h)

    @property
    def num_free_blocks(self) -> int:
        n = int(_lib.pkv_bm_num_free_blocks(self._h))
        if n < 0:
            raise PkvError(n, "pkv_bm_num_free_blocks")
        return n

    def add_sequence(self, seq_id: int, num_tokens: int) -> None:
        _check(_lib.pkv_bm_add_sequence(self._h, int(seq_id), int(num_tokens)), "pkv_bm_add_sequence")

    def append_slots(self, seq_ids) -> torch.Tensor:
        ids = torch.as_tensor(list(seq_ids), dtype=torch.int64).contiguous()
        out = torch.empty(len(ids), dtype=torch.int64)
        _check(_lib.pkv_bm_append_slots(self._h, ids.data_ptr(), len(ids), out.data_ptr()),
               "pkv_bm_append_slots")
        return out

    def free_sequence(self, seq_id: int) -> None:
        _check(_lib.pkv_bm_free_sequence(self._h, int(seq_id)), "pkv_bm_free_sequence")

    def fork(self, parent_id: int, child_id: int) -> None:
        """Admit child_id sharing every block of parent_id."""
        _check(_lib.pkv_bm_fork(self._h, int(parent_id), int(child_id)), "pkv_bm_fork")

    def append_slots_cow(self, seq_ids):
        """append_slots with copy-on-write: (slots [n] int64, block_pairs [p, 2] int32,
        num_tokens [p] int32); copy the pairs (paged_kv_copy_blocks) before writing the slots."""
        ids = torch.as_tensor(list(seq_ids), dtype=torch.int64).contiguous()
        n = len(ids)
        out = torch.empty(n, dtype=torch.int64)
        pairs, rows = torch.empty(n, 2, dtype=torch.int32), torch.empty(n, dtype=torch.int32)
        got = ctypes.c_int32(0)
        _check(_lib.pkv_bm_append_slots_cow(self._h, ids.data_ptr(), n, out.data_ptr(),
                                            pairs.data_ptr(), rows.data_ptr(), ctypes.byref(got)),
               "pkv_bm_append_slots_cow")
        return out, pairs[:got.value], rows[:got.value]

    def truncate(self, seq_id: int, num_tokens: int) -> None:
        """Shorten a sequence, releasing the blocks past num_tokens."""
        _check(_lib.pkv_bm_truncate(self._h, int(seq_id), int(num_tokens)), "pkv_bm_truncate")

    def ref_count(self, block: int) -> int:
        n = int(_lib.pkv_bm_ref_count(self._h, int(block)))
        if n < 0:
            raise PkvError(n, "pkv_bm_ref_count")
        return n

    def compact(self):
        """Move the blocks in use to the lowest ids: (block_moves [n, 2] int32, block_map
        [num_blocks] int32) for paged_kv_compact; the manager's tables are already moved."""
        moves = torch.empty(self.num_blocks - self.num_free_blocks, 2, dtype=torch.int32)
        block_map = torch.empty(self.num_blocks, dtype=torch.int32)
        got = ctypes.c_int64(0)
        _check(_lib.pkv_bm_compact(self._h, moves.data_ptr(), moves.shape[0], ctypes.byref(got),
                                   block_map.data_ptr()), "pkv_bm_compact")
        return moves[:got.value], block_map

    def preempt_lifo(self) -> int:
        v = ctypes.c_int64(0)
        _check(_lib.pkv_bm_preempt_lifo(self._h, ctypes.byref(v)), "pkv_bm_preempt_lifo")
        return int(v.value)

    def block_tables(self, seq_ids, max_blocks_per_seq: int):
        ids = torch.as_tensor(list(seq_ids), dtype=torch.int64).contiguous()
        tables = torch.empty(len(ids), int(max_blocks_per_seq), dtype=torch.int32)
        lens = torch.empty(len(ids), dtype=torch.int32)
        _check(_lib.pkv_bm_block_tables(self._h, ids.data_ptr(), len(ids), int(max_blocks_per_seq),
                                        tables.data_ptr(), lens.data_ptr()), "pkv_bm_block_tables")
        return tables, lens
