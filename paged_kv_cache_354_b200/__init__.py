"""Python binding of libpa.so: paged KV cache and paged decode attention on B200.

Thin marshalling over the C ABI declared in ``include/pa.h``: every function
here has the C entry point's name and only turns tensors into pointers and
the current CUDA stream into a handle.  All work runs in the library's
kernels; there is no Python or CPU fallback.  Importing this package raises
if ``libpa.so`` is missing (build it with
``python paged_kv_cache_354_b200/_build.py``).

bf16 tensors are ``torch.bfloat16``; shapes follow ``include/pa.h``:
    kv_pool      [num_blocks, 2, num_kv_heads, block_size, head_dim]
    q, out       [batch, num_q_heads, head_dim]
    key, value   [num_tokens, num_kv_heads, head_dim]
    kv_cache     [batch, 2, num_kv_heads, max_len, head_dim]  (contiguous decode)
    block_tables int32 [batch, max_blocks_per_seq]; seq_lens int32 [batch]
    slot_mapping int64 [num_tokens]; block_pairs int32 [num_pairs, 2]
    tree_mask    int32 [num_nodes, words] or [batch, num_nodes, words] (bits)
"""

import ctypes
import os

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpa.so")

PA_OK = 0
PA_ERR_INVALID = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_OOM = -3
PA_ERR_CUDA = -4
PA_ERR_NOT_FOUND = -5
PA_ERR_EXISTS = -6

PA_DEVERR_BLOCK_ID = 0x1
PA_DEVERR_SLOT = 0x2
PA_DEVERR_SEQ_LEN = 0x4
PA_DEVERR_WAIT_TIMEOUT = 0x8
PA_DEVERR_COPY_PAIR = 0x10
PA_DEVERR_NO_BLOCKS = 0x20
PA_DEVERR_PLAN = 0x40
PA_DEVERR_TREE = 0x80
PA_DEVERR_POSITION = 0x100

PA_DECODE_AUTO = 0
PA_DECODE_CUDA_CORE = 1
PA_DECODE_MMA = 2
PA_DECODE_TCGEN05 = 3

PA_SCHEDULE_BALANCED = -1  # partition_tokens value that asks for the balanced schedule

_c = ctypes
_P = _c.c_void_p
_I = _c.c_int
_I64 = _c.c_int64
_SZ = _c.c_size_t

# name -> (restype, argtypes); mirrors include/pa.h
_SIGNATURES = {
    "pa_version": (_I, []),
    "pa_last_error_string": (_c.c_char_p, []),
    "pa_device_error": (_I, [_P, _I]),
    "pa_reshape_and_cache": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "pa_copy_blocks": (_I, [_P, _P, _I, _I, _I, _I, _I, _P]),
    "pa_decode_workspace_size": (_I, [_I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_decode_workspace_size_ex": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "pa_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _c.c_float, _P, _SZ, _P]),
    "pa_decode_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _c.c_float, _P, _SZ,
                          _I, _I, _P]),
    "pa_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _c.c_float, _P]),
    "pa_decode_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _c.c_float, _P,
                              _SZ, _P]),
    "pa_decode_multi_workspace_size": (_I, [_I, _I, _I, _I, _I, _I, _I, _P]),
    "pa_decode_multi": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _c.c_float, _P, _SZ,
                             _P]),
    "pa_decode_contiguous_workspace_size": (_I, [_I, _I, _I, _I, _I, _P]),
    "pa_decode_contiguous": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _c.c_float, _P, _SZ, _I, _P]),
    "pa_plan_append": (_I, [_P] * 7 + [_I] + [_P] * 8 + [_I] * 6 + [_P]),
    "pa_norm_rope_and_cache": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _c.c_float, _P]
                               + [_I] * 3 + [_P, _P] + [_I] * 6 + [_P]),
    "pa_decode_tree_workspace_size": (_I, [_I] * 7 + [_P]),
    "pa_decode_tree": (_I, [_P, _P, _P, _P, _I, _P, _P, _P] + [_I] * 9 + [_c.c_float, _P, _SZ, _P]),
    "pa_tree_accept": (_I, [_P] * 7 + [_I] * 8 + [_P]),
    "pa_selftest_wait_timeout": (_I, [_I64, _P]),
    "pa_alloc_create": (_I, [_I, _I, _P, _P]),
    "pa_alloc_destroy": (_I, [_P]),
    "pa_alloc_add_seq": (_I, [_P, _I64]),
    "pa_alloc_fork": (_I, [_P, _I64, _I64]),
    "pa_alloc_append": (_I, [_P, _I64, _I, _P, _P, _I, _P]),
    "pa_alloc_append_batch": (_I, [_P, _P, _I, _I, _P, _P, _I, _P]),
    "pa_alloc_free_seq": (_I, [_P, _I64]),
    "pa_alloc_num_free": (_I, [_P, _P]),
    "pa_alloc_seq_len": (_I, [_P, _I64, _P]),
    "pa_alloc_refcount": (_I, [_P, _I, _P]),
    "pa_alloc_block_table": (_I, [_P, _I64, _P, _I, _P]),
    "pa_alloc_block_tables": (_I, [_P, _P, _I, _I, _P, _P]),
    "pa_alloc_dump": (_I, [_P, _P, _P, _P]),
    "pa_alloc_stats": (_I, [_P, _P]),
}


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with `python paged_kv_cache_354_b200/_build.py`"
        )
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
LIB_PATH = _LIB_PATH


class PaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib.pa_last_error_string().decode(errors="replace")
        super().__init__(f"{where} returned {status}: {msg}")


class OutOfBlocks(PaError):
    pass


def _check(status, where):
    if status != PA_OK:
        if status == PA_ERR_OOM:
            raise OutOfBlocks(status, where)
        raise PaError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _require(t, dtype, name, pinned_ok=False):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda and not (pinned_ok and t.is_pinned()):
        raise TypeError(f"{name}: expected a CUDA tensor" + (" or a pinned host tensor" if pinned_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


# --------------------------------------------------------------------------
# kernels
# --------------------------------------------------------------------------
def pa_version():
    return lib.pa_version()


def pa_device_error(clear=True):
    """OR of PA_DEVERR_* bits recorded by kernels on the current device."""
    code = ctypes.c_int32(0)
    _check(lib.pa_device_error(ctypes.byref(code), 1 if clear else 0), "pa_device_error")
    return code.value


def pa_reshape_and_cache(key, value, kv_pool, slot_mapping, stream=None):
    import torch

    _require(key, torch.bfloat16, "key")
    _require(value, torch.bfloat16, "value")
    _require(kv_pool, torch.bfloat16, "kv_pool")
    _require(slot_mapping, torch.int64, "slot_mapping")
    nb, two, hkv, bs, d = kv_pool.shape
    t = key.shape[0]
    if key.shape != (t, hkv, d) or value.shape != (t, hkv, d) or slot_mapping.shape != (t,):
        raise ValueError("pa_reshape_and_cache: shape mismatch")
    _check(lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(kv_pool), _ptr(slot_mapping), t, nb,
                                    hkv, bs, d, _stream(stream)), "pa_reshape_and_cache")


def pa_copy_blocks(kv_pool, block_pairs, stream=None):
    import torch

    _require(kv_pool, torch.bfloat16, "kv_pool")
    nb, two, hkv, bs, d = kv_pool.shape
    n = 0 if block_pairs is None else block_pairs.shape[0]
    if n == 0:
        return
    _require(block_pairs, torch.int32, "block_pairs")
    _check(lib.pa_copy_blocks(_ptr(kv_pool), _ptr(block_pairs), n, nb, hkv, bs, d, _stream(stream)),
           "pa_copy_blocks")


def pa_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                             partition_tokens=0, with_schedule=False):
    """(bytes, num_partitions) of the split-K scratch pa_decode needs; with
    ``with_schedule`` also "balanced" or "grid"."""
    nbytes = ctypes.c_size_t(0)
    parts = ctypes.c_int(0)
    balanced = ctypes.c_int(0)
    _check(lib.pa_decode_workspace_size_ex(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                           max_seq_len, partition_tokens, ctypes.byref(nbytes),
                                           ctypes.byref(parts), ctypes.byref(balanced)),
           "pa_decode_workspace_size")
    if with_schedule:
        return nbytes.value, parts.value, ("balanced" if balanced.value else "grid")
    return nbytes.value, parts.value


def pa_decode(out, q, kv_pool, block_tables, seq_lens, max_seq_len, scale, workspace=None,
              variant=PA_DECODE_AUTO, partition_tokens=0, stream=None):
    """Paged decode attention; writes ``out`` (bf16 [B, Hq, D]) in place.
    ``out`` is a CUDA tensor or a pinned host tensor (the kernels then store
    the rows across PCIe as they finish; read it after the stream syncs)."""
    import torch

    _require(out, torch.bfloat16, "out", pinned_ok=True)
    _require(q, torch.bfloat16, "q")
    _require(kv_pool, torch.bfloat16, "kv_pool")
    _require(block_tables, torch.int32, "block_tables")
    _require(seq_lens, torch.int32, "seq_lens")
    nb, two, hkv, bs, d = kv_pool.shape
    b, hq, dq = q.shape
    if out.shape != q.shape or dq != d or block_tables.shape[0] != b or seq_lens.shape != (b,):
        raise ValueError("pa_decode: shape mismatch")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _require(workspace, torch.uint8, "workspace")
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()
    _check(lib.pa_decode_ex(_ptr(out), _ptr(q), _ptr(kv_pool), _ptr(block_tables), _ptr(seq_lens), b, hq,
                            hkv, d, bs, nb, block_tables.shape[1], int(max_seq_len), float(scale), ws_ptr,
                            ws_bytes, int(variant), int(partition_tokens), _stream(stream)), "pa_decode")


def pa_decode_multi_workspace_size(batch, num_query_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                                   max_seq_len):
    nbytes = ctypes.c_size_t(0)
    _check(lib.pa_decode_multi_workspace_size(batch, num_query_tokens, num_q_heads, num_kv_heads, head_dim,
                                              block_size, max_seq_len, ctypes.byref(nbytes)),
           "pa_decode_multi_workspace_size")
    return nbytes.value


def pa_decode_multi(out, q, kv_pool, block_tables, seq_lens, max_seq_len, scale, workspace, stream=None):
    """T causal query tokens per request: q, out bf16 [B, T, Hq, D]."""
    import torch

    _require(out, torch.bfloat16, "out", pinned_ok=True)
    _require(q, torch.bfloat16, "q")
    _require(kv_pool, torch.bfloat16, "kv_pool")
    _require(block_tables, torch.int32, "block_tables")
    _require(seq_lens, torch.int32, "seq_lens")
    _require(workspace, torch.uint8, "workspace")
    nb, two, hkv, bs, d = kv_pool.shape
    b, t, hq, dq = q.shape
    if out.shape != q.shape or dq != d or block_tables.shape[0] != b or seq_lens.shape != (b,):
        raise ValueError("pa_decode_multi: shape mismatch")
    _check(lib.pa_decode_multi(_ptr(out), _ptr(q), _ptr(kv_pool), _ptr(block_tables), _ptr(seq_lens), b, t, hq,
                               hkv, d, bs, nb, block_tables.shape[1], int(max_seq_len), float(scale),
                               _ptr(workspace), workspace.numel(), _stream(stream)), "pa_decode_multi")


def pa_decode_contiguous_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_len):
    nbytes = ctypes.c_size_t(0)
    _check(lib.pa_decode_contiguous_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_len,
                                                   ctypes.byref(nbytes)), "pa_decode_contiguous_workspace_size")
    return nbytes.value


def pa_decode_contiguous(out, q, kv_cache, seq_lens, scale, workspace, variant=PA_DECODE_AUTO, stream=None):
    """Decode over a contiguous per-request cache kv_cache bf16
    [B, 2, Hkv, max_len, D] (no block table); writes ``out`` in place."""
    import torch

    _require(out, torch.bfloat16, "out", pinned_ok=True)
    _require(q, torch.bfloat16, "q")
    _require(kv_cache, torch.bfloat16, "kv_cache")
    _require(seq_lens, torch.int32, "seq_lens")
    _require(workspace, torch.uint8, "workspace")
    b, two, hkv, max_len, d = kv_cache.shape
    bq, hq, dq = q.shape
    if two != 2 or out.shape != q.shape or dq != d or bq != b or seq_lens.shape != (b,):
        raise ValueError("pa_decode_contiguous: shape mismatch")
    _check(lib.pa_decode_contiguous(_ptr(out), _ptr(q), _ptr(kv_cache), _ptr(seq_lens), b, hq, hkv, d, max_len,
                                    float(scale), _ptr(workspace), workspace.numel(), int(variant),
                                    _stream(stream)), "pa_decode_contiguous")


PA_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def pa_decode_noalloc(out, q, kv_pool, block_tables, seq_lens, max_seq_len, scale, stream=None):
    """pa_decode without a workspace argument, for callers that cannot
    allocate device memory: the split-K partials live in a fixed array of
    PA_NOALLOC_SCRATCH_BYTES inside the library (shared by all calls on a
    device; calls that overlap on the GPU race on it)."""
    import torch

    _require(out, torch.bfloat16, "out", pinned_ok=True)
    _require(q, torch.bfloat16, "q")
    _require(kv_pool, torch.bfloat16, "kv_pool")
    _require(block_tables, torch.int32, "block_tables")
    _require(seq_lens, torch.int32, "seq_lens")
    nb, two, hkv, bs, d = kv_pool.shape
    b, hq, dq = q.shape
    if out.shape != q.shape or dq != d or block_tables.shape[0] != b or seq_lens.shape != (b,):
        raise ValueError("pa_decode_noalloc: shape mismatch")
    _check(lib.pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(kv_pool), _ptr(block_tables), _ptr(seq_lens), b,
                                 hq, hkv, d, bs, nb, block_tables.shape[1], int(max_seq_len), float(scale),
                                 _stream(stream)), "pa_decode_noalloc")


def pa_decode_append(out, q, kv_pool, key, value, slot_mapping, block_tables, seq_lens, max_seq_len, scale,
                     workspace=None, stream=None):
    """pa_reshape_and_cache of each request's newest token (key/value
    [B, Hkv, D], slot_mapping [B]) and pa_decode, in one pass."""
    import torch

    _require(out, torch.bfloat16, "out", pinned_ok=True)
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv_pool, torch.bfloat16, "kv_pool"),
                     (key, torch.bfloat16, "key"), (value, torch.bfloat16, "value"),
                     (slot_mapping, torch.int64, "slot_mapping"), (block_tables, torch.int32, "block_tables"),
                     (seq_lens, torch.int32, "seq_lens")):
        _require(t, dt, n)
    nb, two, hkv, bs, d = kv_pool.shape
    b, hq, dq = q.shape
    if (out.shape != q.shape or dq != d or key.shape != (b, hkv, d) or value.shape != (b, hkv, d)
            or slot_mapping.shape != (b,) or block_tables.shape[0] != b or seq_lens.shape != (b,)):
        raise ValueError("pa_decode_append: shape mismatch")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _require(workspace, torch.uint8, "workspace")
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()
    _check(lib.pa_decode_append(_ptr(out), _ptr(q), _ptr(kv_pool), _ptr(key), _ptr(value), _ptr(slot_mapping),
                                _ptr(block_tables), _ptr(seq_lens), b, hq, hkv, d, bs, nb, block_tables.shape[1],
                                int(max_seq_len), float(scale), ws_ptr, ws_bytes, _stream(stream)),
           "pa_decode_append")


# --------------------------------------------------------------------------
# tree speculation
# --------------------------------------------------------------------------
def _fit(dtype, device, tensors):
    """Whether all tensors (None skipped) are contiguous, of ``dtype`` and on
    CUDA device ``device``.  These calls run between two decoding steps, where
    the checks cost as much as the launch: ``_refuse`` says what is wrong."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()):
            return False
    return device >= 0


def _refuse(where, dtype, device, **tensors):
    """Raise for the first tensor that ``_fit`` does not take."""
    for name, t in tensors.items():
        if t is not None:
            _require(t, dtype, name)
            if t.get_device() != device:
                raise ValueError(f"{where}: {name} is on cuda:{t.get_device()}, other tensors on cuda:{device}")


def _raw_stream(torch, device, stream):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _launch(torch, where, device, fn, args):
    """Call fn(*args) with ``device`` current."""
    if device == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != PA_OK:
        _check(status, where)


def _adr(t):
    return None if t is None else t.data_ptr()


def pa_plan_append(block_tables, blocks_held, free_blocks, num_free, seq_lens, new_tokens, slot_mapping, positions,
                   block_size, depths=None, token_starts=None, seq_lens_out=None, blocks_held_out=None,
                   num_free_out=None, appended_out=None, status_out=None, stream=None):
    """Blocks, slots and positions of every request's new tokens, on the GPU.

    ``slot_mapping`` / ``positions`` are [batch, max_new_tokens] (padded) or
    1-d (packed; needs ``token_starts`` [batch + 1]).  The state is updated in
    place unless ``seq_lens_out`` / ``blocks_held_out`` / ``num_free_out`` say
    otherwise.  ``depths``: int32 [batch, max_new_tokens], or
    [max_new_tokens] for one tree shared by all requests."""
    import torch

    where = "pa_plan_append"
    seq_lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    blocks_held_out = blocks_held if blocks_held_out is None else blocks_held_out
    num_free_out = num_free if num_free_out is None else num_free_out
    device = block_tables.get_device()
    if not _fit(torch.int32, device, (block_tables, blocks_held, free_blocks, num_free, seq_lens, new_tokens, positions,
                                      seq_lens_out, blocks_held_out, num_free_out, depths, token_starts, appended_out,
                                      status_out)):
        _refuse(where, torch.int32, device, block_tables=block_tables, blocks_held=blocks_held,
                free_blocks=free_blocks, num_free=num_free, seq_lens=seq_lens, new_tokens=new_tokens,
                positions=positions, seq_lens_out=seq_lens_out, blocks_held_out=blocks_held_out,
                num_free_out=num_free_out, depths=depths, token_starts=token_starts, appended_out=appended_out,
                status_out=status_out)
    if not _fit(torch.int64, device, (slot_mapping,)):
        _refuse(where, torch.int64, device, slot_mapping=slot_mapping)
    b, width = block_tables.shape
    per_request = (b,)
    padded = slot_mapping.dim() == 2
    if (blocks_held.shape != per_request or seq_lens.shape != per_request or new_tokens.shape != per_request
            or seq_lens_out.shape != per_request or blocks_held_out.shape != per_request or num_free.numel() != 1
            or num_free_out.numel() != 1 or free_blocks.dim() != 1 or positions.shape != slot_mapping.shape
            or (padded and slot_mapping.shape[0] != b) or slot_mapping.dim() not in (1, 2)
            or (token_starts is not None and token_starts.shape != (b + 1,))
            or (appended_out is not None and appended_out.shape != per_request)
            or (status_out is not None and status_out.numel() != 1)):
        raise ValueError(f"{where}: shape mismatch")
    most = slot_mapping.shape[1] if padded else 0
    if padded and most == 0:
        raise ValueError(f"{where}: the padded layout needs at least one column")
    stride = 0
    if depths is not None:
        if not padded or depths.shape not in ((most,), (b, most)):
            raise ValueError(f"{where}: shape mismatch")
        stride = most if depths.dim() == 2 else 0
    _launch(torch, where, device, lib.pa_plan_append,
            (block_tables.data_ptr(), blocks_held.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr(),
             seq_lens.data_ptr(), new_tokens.data_ptr(), _adr(depths), stride, slot_mapping.data_ptr(),
             positions.data_ptr(), _adr(token_starts), seq_lens_out.data_ptr(), blocks_held_out.data_ptr(),
             num_free_out.data_ptr(), _adr(appended_out), _adr(status_out), b, most, slot_mapping.numel(),
             free_blocks.shape[0], int(block_size), width, _raw_stream(torch, device, stream)))


def _token_rows(where, device, dtype, name, t, shape):
    """Token stride of a [tokens, heads, head_dim] tensor of ``shape`` whose
    tokens may be strided but whose heads lie together."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    index = t.get_device()
    if index < 0:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if index != device:
        raise ValueError(f"{where}: {name} is on cuda:{index}, other tensors on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{where}: shape mismatch")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if n and h and ((d > 1 and s2 != 1) or (h > 1 and s1 != d)):
        raise ValueError(f"{name}: a token's heads must lie together")
    return s0 if n > 1 else h * d


def pa_norm_rope_and_cache(q_out, q, k, v, kv_pool, slot_mapping, positions, cos_sin, q_weight=None, k_weight=None,
                           eps=1e-6, interleaved=False, k_out=None, stream=None):
    """Norm and rotate queries and keys; queries go to ``q_out`` (may be ``q``),
    keys and values into ``kv_pool`` at ``slot_mapping`` (and / or keys to
    ``k_out``).  q, k, v are [tokens, heads, head_dim], strided by token;
    ``cos_sin`` fp32 [max_position, rotary_dim] (None: no rotation)."""
    import torch

    where = "pa_norm_rope_and_cache"
    bf16 = torch.bfloat16
    device, q_shape, k_shape = q.get_device(), q.shape, k.shape
    n, hq, d = q_shape
    hkv = k_shape[1]
    qs = _token_rows(where, device, bf16, "q", q, q_shape)
    qos = _token_rows(where, device, bf16, "q_out", q_out, q_shape)
    ks = _token_rows(where, device, bf16, "k", k, (n, hkv, d))
    vs = kos = 0
    blocks = block_size = 0
    if kv_pool is None:
        v = slot_mapping = None
    else:
        if not _fit(bf16, device, (kv_pool,)):
            _refuse(where, bf16, device, kv_pool=kv_pool)
        if not _fit(torch.int64, device, (slot_mapping,)):
            _refuse(where, torch.int64, device, slot_mapping=slot_mapping)
        vs = _token_rows(where, device, bf16, "v", v, k_shape)
        blocks, two, pool_heads, block_size, pool_dim = kv_pool.shape
        if slot_mapping.numel() != n or (two, pool_heads, pool_dim) != (2, hkv, d):
            raise ValueError(f"{where}: shape mismatch")
    if k_out is not None:
        kos = _token_rows(where, device, bf16, "k_out", k_out, k_shape)
    most = rotary = 0
    if cos_sin is not None:
        if not _fit(torch.float32, device, (cos_sin,)):
            _refuse(where, torch.float32, device, cos_sin=cos_sin)
        most, rotary = cos_sin.shape
    if positions is not None:
        if not _fit(torch.int32, device, (positions,)):
            _refuse(where, torch.int32, device, positions=positions)
        if positions.numel() != n:
            raise ValueError(f"{where}: shape mismatch")
    if q_weight is not None or k_weight is not None:
        if not _fit(bf16, device, (q_weight, k_weight)):
            _refuse(where, bf16, device, q_weight=q_weight, k_weight=k_weight)
        if (q_weight is not None and q_weight.shape != (d,)) or (k_weight is not None and k_weight.shape != (d,)):
            raise ValueError(f"{where}: shape mismatch")
    _launch(torch, where, device, lib.pa_norm_rope_and_cache,
            (q_out.data_ptr(), qos, _adr(k_out), kos, _adr(kv_pool), q.data_ptr(), qs, k.data_ptr(), ks, _adr(v), vs,
             _adr(q_weight), _adr(k_weight), eps, _adr(cos_sin), most, rotary, 1 if interleaved else 0,
             _adr(positions), _adr(slot_mapping), n, hq, hkv, d, blocks, block_size,
             _raw_stream(torch, device, stream)))


def pa_decode_tree_workspace_size(batch, num_nodes, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len):
    nbytes = ctypes.c_size_t(0)
    _check(lib.pa_decode_tree_workspace_size(batch, num_nodes, num_q_heads, num_kv_heads, head_dim, block_size,
                                             max_seq_len, ctypes.byref(nbytes)), "pa_decode_tree_workspace_size")
    return nbytes.value


def pa_decode_tree(out, q, kv_pool, tree_mask, block_tables, seq_lens, max_seq_len, scale, workspace, tree_lens=None,
                   stream=None):
    """Attention of a tree of drafted tokens per request: q, out bf16
    [B, T, Hq, D]; ``tree_mask`` int32 bits [T, ceil(T/32)] (one tree for all)
    or [B, T, ceil(T/32)]; ``tree_lens`` int32 [B] (None: T each)."""
    import torch

    where = "pa_decode_tree"
    device = q.get_device()
    if not _fit(torch.bfloat16, device, (q, kv_pool, out)):
        _refuse(where, torch.bfloat16, device, q=q, kv_pool=kv_pool)
        _require(out, torch.bfloat16, "out", pinned_ok=True)
        if out.is_cuda:
            _refuse(where, torch.bfloat16, device, out=out)
    if not _fit(torch.int32, device, (tree_mask, block_tables, seq_lens, tree_lens)):
        _refuse(where, torch.int32, device, tree_mask=tree_mask, block_tables=block_tables, seq_lens=seq_lens,
                tree_lens=tree_lens)
    if not _fit(torch.uint8, device, (workspace,)):
        _refuse(where, torch.uint8, device, workspace=workspace)
    nb, two, hkv, bs, d = kv_pool.shape
    b, t, hq, dq = q.shape
    rows = (t, (t + 31) // 32)
    if (out.shape != q.shape or dq != d or two != 2 or block_tables.dim() != 2 or block_tables.shape[0] != b
            or seq_lens.shape != (b,) or (tree_lens is not None and tree_lens.shape != (b,))
            or tree_mask.shape not in (rows, (b,) + rows)):
        raise ValueError(f"{where}: shape mismatch")
    _launch(torch, where, device, lib.pa_decode_tree,
            (out.data_ptr(), q.data_ptr(), kv_pool.data_ptr(), tree_mask.data_ptr(), 1 if tree_mask.dim() == 3 else 0,
             block_tables.data_ptr(), seq_lens.data_ptr(), _adr(tree_lens), b, t, hq, hkv, d, bs, nb,
             block_tables.shape[1], int(max_seq_len), float(scale), workspace.data_ptr(), workspace.numel(),
             _raw_stream(torch, device, stream)))


def pa_tree_accept(kv_pool, path, accept_lens, block_tables, seq_lens, tree_lens, seq_lens_out=None, num_nodes=None,
                   stream=None):
    """Move the rows of each request's accepted path (node indices ``path``
    [B, max_path], the first ``accept_lens[b]`` of them) behind its committed
    prefix; ``seq_lens_out`` (None: not written; may be ``seq_lens``) receives
    the new lengths.  ``tree_lens``: int32 [B] nodes per request, or None and
    ``num_nodes`` for all."""
    import torch

    where = "pa_tree_accept"
    device = kv_pool.get_device()
    if not _fit(torch.bfloat16, device, (kv_pool,)):
        _refuse(where, torch.bfloat16, device, kv_pool=kv_pool)
    if not _fit(torch.int32, device, (path, accept_lens, block_tables, seq_lens, tree_lens, seq_lens_out)):
        _refuse(where, torch.int32, device, path=path, accept_lens=accept_lens, block_tables=block_tables,
                seq_lens=seq_lens, tree_lens=tree_lens, seq_lens_out=seq_lens_out)
    nb, two, hkv, bs, d = kv_pool.shape
    b, most = path.shape
    if (two != 2 or accept_lens.shape != (b,) or seq_lens.shape != (b,) or block_tables.dim() != 2
            or block_tables.shape[0] != b
            or (tree_lens is not None and tree_lens.shape != (b,))
            or (seq_lens_out is not None and seq_lens_out.shape != (b,))):
        raise ValueError(f"{where}: shape mismatch")
    if tree_lens is None and num_nodes is None:
        raise ValueError(f"{where}: tree_lens or num_nodes")
    nodes = 0x7fffffff if num_nodes is None else int(num_nodes)
    _launch(torch, where, device, lib.pa_tree_accept,
            (kv_pool.data_ptr(), path.data_ptr(), accept_lens.data_ptr(), _adr(tree_lens), block_tables.data_ptr(),
             seq_lens.data_ptr(), _adr(seq_lens_out), b, nodes, most, nb, hkv, bs, d, block_tables.shape[1],
             _raw_stream(torch, device, stream)))


def pa_selftest_wait_timeout(limit_ns, stream=None):
    _check(lib.pa_selftest_wait_timeout(int(limit_ns), _stream(stream)), "pa_selftest_wait_timeout")


# --------------------------------------------------------------------------
# host allocator
# --------------------------------------------------------------------------
class PaAlloc:
    """Handle on the C++ block allocator (pa_alloc_* calls).

    Method names match the allocator model used by the tests so one driver
    can run either.
    """

    def __init__(self, num_blocks, block_size, initial_order=None):
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)
        h = ctypes.c_void_p()
        order = None
        if initial_order is not None:
            order = np.ascontiguousarray(np.asarray(initial_order, dtype=np.int32))
            if order.shape != (self.num_blocks,):
                raise ValueError("initial_order must list every block once")
        _check(lib.pa_alloc_create(self.num_blocks, self.block_size,
                                   order.ctypes.data_as(ctypes.c_void_p) if order is not None else None,
                                   ctypes.byref(h)), "pa_alloc_create")
        self._h = h
        self._cow = np.zeros(2 * 1024, dtype=np.int32)

    def close(self):
        if self._h:
            lib.pa_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id):
        _check(lib.pa_alloc_add_seq(self._h, int(seq_id)), "pa_alloc_add_seq")

    def fork(self, parent, child):
        _check(lib.pa_alloc_fork(self._h, int(parent), int(child)), "pa_alloc_fork")

    def free_seq(self, seq_id):
        _check(lib.pa_alloc_free_seq(self._h, int(seq_id)), "pa_alloc_free_seq")

    def append(self, seq_id, num_tokens):
        return self.append_batch([seq_id], num_tokens)

    def append_batch(self, seq_ids, num_tokens, as_numpy=False):
        """(slots, cow_pairs) like the model: slots in (request, token) order."""
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        slots = np.empty(len(ids) * int(num_tokens), dtype=np.int64)
        ncow = ctypes.c_int(0)
        cap = max(1, len(ids))
        if self._cow.size < 2 * cap:
            self._cow = np.zeros(2 * cap, dtype=np.int32)
        _check(lib.pa_alloc_append_batch(self._h, ids.ctypes.data_as(ctypes.c_void_p), len(ids),
                                         int(num_tokens), slots.ctypes.data_as(ctypes.c_void_p),
                                         self._cow.ctypes.data_as(ctypes.c_void_p), cap,
                                         ctypes.byref(ncow)), "pa_alloc_append_batch")
        pairs = self._cow[: 2 * ncow.value].reshape(-1, 2).copy()
        if as_numpy:
            return slots, pairs
        return slots.tolist(), [tuple(int(x) for x in p) for p in pairs]

    def num_free(self):
        n = ctypes.c_int(0)
        _check(lib.pa_alloc_num_free(self._h, ctypes.byref(n)), "pa_alloc_num_free")
        return n.value

    def seq_len(self, seq_id):
        n = ctypes.c_int(0)
        _check(lib.pa_alloc_seq_len(self._h, int(seq_id), ctypes.byref(n)), "pa_alloc_seq_len")
        return n.value

    def refcount(self, block):
        n = ctypes.c_int(0)
        _check(lib.pa_alloc_refcount(self._h, int(block), ctypes.byref(n)), "pa_alloc_refcount")
        return n.value

    def block_table(self, seq_id):
        cap = self.num_blocks
        out = np.empty(cap, dtype=np.int32)
        n = ctypes.c_int(0)
        _check(lib.pa_alloc_block_table(self._h, int(seq_id), out.ctypes.data_as(ctypes.c_void_p), cap,
                                        ctypes.byref(n)), "pa_alloc_block_table")
        return out[: n.value].tolist()

    def block_tables(self, seq_ids, max_blocks_per_seq):
        """Padded int32 [n, max_blocks_per_seq] tables and int32 lengths (numpy)."""
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        tables = np.empty((len(ids), int(max_blocks_per_seq)), dtype=np.int32)
        lens = np.empty(len(ids), dtype=np.int32)
        _check(lib.pa_alloc_block_tables(self._h, ids.ctypes.data_as(ctypes.c_void_p), len(ids),
                                         int(max_blocks_per_seq), tables.ctypes.data_as(ctypes.c_void_p),
                                         lens.ctypes.data_as(ctypes.c_void_p)), "pa_alloc_block_tables")
        return tables, lens

    def dump(self):
        free = np.empty(self.num_blocks, dtype=np.int32)
        refs = np.empty(self.num_blocks, dtype=np.int32)
        n = ctypes.c_int(0)
        _check(lib.pa_alloc_dump(self._h, free.ctypes.data_as(ctypes.c_void_p), ctypes.byref(n),
                                 refs.ctypes.data_as(ctypes.c_void_p)), "pa_alloc_dump")
        return free[: n.value].tolist(), refs.tolist()

    def stats(self):
        """dict: tokens, logical_slots, physical_blocks, live_requests, free_blocks."""
        out = np.zeros(5, dtype=np.int64)
        _check(lib.pa_alloc_stats(self._h, out.ctypes.data_as(ctypes.c_void_p)), "pa_alloc_stats")
        keys = ("tokens", "logical_slots", "physical_blocks", "live_requests", "free_blocks")
        return dict(zip(keys, (int(x) for x in out)))

    def free_list(self):
        return self.dump()[0]

    def refcounts(self):
        return self.dump()[1]
