"""Python binding of the C ABI in ``include/pkv.h`` (ctypes).

Argument marshalling only: every function here turns torch tensors into the
pointers, sizes and strides the C entry point takes and raises on a non-OK
status.  All arithmetic runs in the CUDA kernels of ``libpkv.so``; if the
library has not been built this module raises instead of falling back to
anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA = range(5)
PKV_BF16, PKV_F16, PKV_F32 = range(3)
MASKS = {"none": 0, "causal": 1, "block_causal": 2}
PKV_FLAG_CHECKED = 0x1
PKV_FLAG_SIMT_ONLY = 0x2
PKV_FLAG_TEST_WAIT_TIMEOUT = 0x4
PKV_FLAG_TILE_GRID = 0x8
PKV_FLAG_STREAM_K = 0x10
PKV_ERRBIT_SLOT, PKV_ERRBIT_SRC, PKV_ERRBIT_PAGE, PKV_ERRBIT_LEN, PKV_ERRBIT_TIMEOUT = (
    0x1, 0x2, 0x4, 0x8, 0x10)

# every symbol include/pkv.h declares
EXPORTED = ("pkv_status_string", "pkv_last_error", "kv_scatter_slots",
            "paged_attention_workspace_size", "paged_attention", "merge_attn_states",
            "rotate_rows", "paged_attention_no_alloc", "rope_write_kv_paged", "copy_kv_slots",
            "causal_layout", "plan_shared_prefix", "shared_prefix_attention",
            "shared_prefix_attention_workspace_size", "pkv_plan_attention", "kv_append_fp8",
            "paged_attention_fp8_workspace_size", "paged_attention_fp8",
            "paged_attention_window_workspace_size", "paged_attention_window", "assign_step_pages",
            "kv_append_latent", "paged_attention_latent_workspace_size", "paged_attention_latent",
            "ragged_attention_latent")
NO_ALLOC_SCRATCH_BYTES = 32 << 20

_vp, _i64, _i32, _u32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_uint, ctypes.c_float, ctypes.c_size_t)
_SIGNATURES = {
    "pkv_status_string": (ctypes.c_char_p, [_i32]),
    "pkv_last_error": (ctypes.c_char_p, []),
    "kv_scatter_slots": (_i32, [_vp, _vp, _i64, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _vp,
                                _vp, _vp, _i64, _i32, _i64, _i32, _u32, _vp, _vp]),
    "paged_attention_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _u32]),
    "pkv_plan_attention": (_i32, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _u32, _i32, _vp, _vp, _vp,
                                  _vp]),
    "paged_attention": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _i64, _vp, _vp,
                               _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp,
                               _i32, _vp, _vp, _sz, _i32, _u32, _vp, _vp]),
    "paged_attention_no_alloc": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _i64,
                                        _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                        _i32, _f32, _vp, _i32, _vp, _i32, _u32, _vp, _vp]),
    "merge_attn_states": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp,
                                 _vp]),
    "rotate_rows": (_i32, [_vp, _i64, _i64, _i64, _i32, _i64, _vp]),
    "rope_write_kv_paged": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _i32, _i32,
                                   _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _i64, _u32, _vp,
                                   _vp]),
    "copy_kv_slots": (_i32, [_vp, _vp, _i32, _i64, _i64, _i32, _i64, _i32, _i32, _i32, _vp, _vp,
                             _i64, _u32, _vp, _vp]),
    "causal_layout": (_i32, [_vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _i32, _i32, _vp, _i64,
                             _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
    "plan_shared_prefix": (_i32, [_vp, _i64, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp]),
    "shared_prefix_attention_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "shared_prefix_attention": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _i64, _vp, _vp,
                                       _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                       _i32, _f32, _vp, _i32, _vp, _vp, _sz, _i32, _u32, _vp, _vp]),
    "kv_append_fp8": (_i32, [_vp, _vp, _i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                             _i32, _vp, _vp, _i64, _i32, _i64, _vp, _vp, _i64, _u32, _vp, _vp]),
    "paged_attention_fp8_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _u32]),
    "paged_attention_fp8": (_i32, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _i64, _vp, _i64,
                                   _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _f32, _vp, _i32, _vp, _vp, _sz, _u32, _vp, _vp]),
    "paged_attention_window_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _u32]),
    "paged_attention_window": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _i64, _vp, _vp, _vp,
                                      _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp,
                                      _vp, _sz, _u32, _vp, _vp]),
    "assign_step_pages": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp]),
    "kv_append_latent": (_i32, [_vp, _i64, _i64, _vp, _f32, _vp, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _i64,
                                _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _i32, _u32, _vp, _vp]),
    "paged_attention_latent_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _u32]),
    "paged_attention_latent": (_i32, [_vp, _i64, _i64, _vp, _i64, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _i32,
                                      _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp, _vp, _sz, _u32,
                                      _vp, _vp]),
    "ragged_attention_latent": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _vp,
                                       _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp,
                                       _u32, _vp, _vp]),
}

_lib = None


class PkvError(RuntimeError):
    def __init__(self, func, status, message):
        self.status = status
        super().__init__(f"{func}: {status_string(status)}: {message}")


def lib(path: str | None = None) -> ctypes.CDLL:
    """The loaded library with its C signatures declared."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libpkv.so is not built ({p}); call __graft_entry__.build() or "
                           "paged_kv_cache_189_gb300.build.build() first")
    L = ctypes.CDLL(p)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = L
    return L


def status_string(status: int) -> str:
    return lib().pkv_status_string(status).decode()


def last_error() -> str:
    return lib().pkv_last_error().decode()


def _check(func, status):
    if status != PKV_OK:
        raise PkvError(func, status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(stream)


_DTYPES = {torch.bfloat16: PKV_BF16, torch.float16: PKV_F16, torch.float32: PKV_F32}


def _dtype(t):
    return _DTYPES[t.dtype]


def _pool_geometry(pool):
    """[num_pages, page_size, Hkv, D] with dense slots; page stride may be larger."""
    assert pool.dim() == 4, "pool must be [num_pages, page_size, num_kv_heads, head_dim]"
    n, P, H, D = pool.shape
    if pool.stride(3) != 1 or pool.stride(2) != D or pool.stride(1) != H * D:
        raise ValueError("pool slots must be dense [num_kv_heads, head_dim] rows")
    return n, P, H, D, pool.stride(0)


# ----------------------------------------------------------------------------
def kv_scatter_slots(k_src, v_src, slots, k_pool, v_pool, slots2=None, src_idx=None,
                     checked=False, err=None, stream=None):
    """Write rows of ``k_src``/``v_src`` ``[T, Hkv, D]`` (any token/head stride,
    unit dim stride) into pool slots ``slots`` (and ``slots2``) in place."""
    assert k_src.stride() == v_src.stride() and k_src.shape == v_src.shape
    assert k_src.stride(2) == 1
    n, P, H, D, page_stride = _pool_geometry(k_pool)
    assert v_pool.shape == k_pool.shape and v_pool.stride() == k_pool.stride()
    T = slots.numel()
    st = lib().kv_scatter_slots(
        _ptr(k_src), _ptr(v_src), T, k_src.shape[0], H, D, k_src.stride(0), k_src.stride(1),
        _ptr(slots), _ptr(slots2), _ptr(src_idx), _ptr(k_pool), _ptr(v_pool), n, P, page_stride,
        _dtype(k_pool), PKV_FLAG_CHECKED if checked else 0, _ptr(err), _stream(stream))
    _check("kv_scatter_slots", st)


def paged_attention_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim,
                                   max_kv_len, num_splits=0, flags=0) -> int:
    return int(lib().paged_attention_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads,
                                                    head_dim, max_kv_len, num_splits, flags))


PKV_KERNEL_NONE, PKV_KERNEL_DECODE, PKV_KERNEL_TILE, PKV_KERNEL_SIMT, PKV_KERNEL_TILE_STREAM_K = range(5)


def plan_attention(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim, max_kv_len,
                   num_splits=0, flags=0, num_sms=0) -> dict:
    """The launch plan of ``paged_attention`` for these host bounds on a GPU
    with ``num_sms`` SMs (0: the current device's): kernel, splits, keys per
    split and workspace bytes."""
    k, s, sk, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    st = lib().pkv_plan_attention(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim, max_kv_len,
                                  num_splits, flags, num_sms, ctypes.byref(k), ctypes.byref(s),
                                  ctypes.byref(sk), ctypes.byref(ws))
    _check("pkv_plan_attention", st)
    return {"kernel": k.value, "splits": s.value, "split_keys": sk.value, "workspace_bytes": ws.value}


def paged_attention(q, k_pool, v_pool, block_table, kv_lens, q_indptr, out, *, q_real=None,
                    lse=None, batch=None, max_q_rows, max_kv_len, mask="causal",
                    causal_block=0, scale=0.0, workspace=None, num_splits=0, flags=0, err=None,
                    stream=None):
    """Paged attention of packed query rows ``q [rows, Hq, D]`` (bf16) into
    ``out [rows, Hq, D]`` (bf16 or f32) and ``lse [rows, Hq]`` (f32)."""
    n, P, H, D, page_stride = _pool_geometry(k_pool)
    assert v_pool.shape == k_pool.shape and v_pool.stride() == k_pool.stride()
    assert q.stride(2) == 1 and out.is_contiguous()
    if batch is None:
        batch = kv_lens.numel()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().paged_attention(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k_pool), _ptr(v_pool), n, P, page_stride,
        _ptr(block_table), block_table.stride(0), _ptr(kv_lens), _ptr(q_indptr), _ptr(q_real),
        batch, max_q_rows, max_kv_len, q.shape[1], H, D, MASKS[mask], causal_block,
        float(scale), _ptr(out), _dtype(out), _ptr(lse), _ptr(workspace), ws_bytes, num_splits,
        flags, _ptr(err), _stream(stream))
    _check("paged_attention", st)


def paged_attention_no_alloc(q, k_pool, v_pool, block_table, kv_lens, q_indptr, out, *,
                             q_real=None, lse=None, batch=None, max_q_rows, max_kv_len,
                             mask="causal", causal_block=0, scale=0.0, num_splits=0, flags=0,
                             err=None, stream=None):
    """``paged_attention`` without a workspace argument, for callers that
    cannot allocate: the scratch is the library's fixed device array of
    ``NO_ALLOC_SCRATCH_BYTES`` (see include/pkv.h).  Calls on one device share
    it, so they must not overlap on the GPU."""
    n, P, H, D, page_stride = _pool_geometry(k_pool)
    assert v_pool.shape == k_pool.shape and v_pool.stride() == k_pool.stride()
    assert q.stride(2) == 1 and out.is_contiguous()
    if batch is None:
        batch = kv_lens.numel()
    st = lib().paged_attention_no_alloc(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k_pool), _ptr(v_pool), n, P, page_stride,
        _ptr(block_table), block_table.stride(0), _ptr(kv_lens), _ptr(q_indptr), _ptr(q_real),
        batch, max_q_rows, max_kv_len, q.shape[1], H, D, MASKS[mask], causal_block,
        float(scale), _ptr(out), _dtype(out), _ptr(lse), num_splits, flags, _ptr(err),
        _stream(stream))
    _check("paged_attention_no_alloc", st)


def merge_attn_states(o_a, lse_a, o_b, lse_b, o_out, lse_out=None, stream=None):
    """Exact LSE merge of two states ``[rows, heads, D]`` into ``o_out``."""
    rows, heads, D = o_a.shape
    assert o_b.shape == o_a.shape and o_out.shape == o_a.shape and o_a.dtype == o_b.dtype
    st = lib().merge_attn_states(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _dtype(o_a),
                                 rows, heads, D, _ptr(o_out), _dtype(o_out), _ptr(lse_out),
                                 _stream(stream))
    _check("merge_attn_states", st)


def rotate_rows(x, shift, rows=None, cols=None, row_stride=None, elem_size=None, stream=None):
    """Rotate every row of ``x`` left by ``shift`` elements in place.  By
    default ``x`` is viewed as ``[rows, cols]`` of its own element type."""
    if rows is None:
        if x.dim() == 1:
            rows, cols, row_stride = 1, x.shape[0], x.shape[0]
        else:
            assert x.dim() == 2 and x.stride(1) == 1
            rows, cols, row_stride = x.shape[0], x.shape[1], x.stride(0)
        elem_size = x.element_size()
    st = lib().rotate_rows(_ptr(x), rows, cols, row_stride, elem_size, shift, _stream(stream))
    _check("rotate_rows", st)


def rope_write_kv_paged(q, k_src, v_src, positions, cos_sin, slots, k_pool, v_pool,
                        checked=False, err=None, stream=None):
    """Rotate ``q [T, Hq, D]`` in place and write the rotated ``k_src`` and the
    ``v_src`` rows ``[T, Hkv, D]`` into pool slots ``slots`` (NeoX pairs,
    angles from the table ``cos_sin [max_position, D]``)."""
    assert q.stride(2) == 1 and k_src.stride(2) == 1 and k_src.stride() == v_src.stride()
    n, P, H, D, page_stride = _pool_geometry(k_pool)
    assert v_pool.shape == k_pool.shape and v_pool.stride() == k_pool.stride()
    assert cos_sin.dtype == torch.float32 and cos_sin.is_contiguous() and cos_sin.shape[1] == D
    st = lib().rope_write_kv_paged(
        _ptr(q), q.stride(0), q.stride(1), q.shape[1], _ptr(k_src), _ptr(v_src), k_src.stride(0),
        k_src.stride(1), q.shape[0], H, D, _ptr(positions), _ptr(cos_sin), cos_sin.shape[0],
        _ptr(slots), _ptr(k_pool), _ptr(v_pool), n, P, page_stride,
        PKV_FLAG_CHECKED if checked else 0, _ptr(err), _stream(stream))
    _check("rope_write_kv_paged", st)


def copy_kv_slots(k_pools, v_pools, src_slots, dst_slots, checked=False, err=None, stream=None):
    """Copy slot rows ``src -> dst`` in every layer of ``k_pools``/``v_pools``
    ``[layers, pages, P, Hkv, D]`` (a 4-D pool is one layer); negative entries
    are skipped."""
    if k_pools.dim() == 4:
        k_pools, v_pools = k_pools.unsqueeze(0), v_pools.unsqueeze(0)
    layers = k_pools.shape[0]
    n, P, H, D, page_stride = _pool_geometry(k_pools[0])
    assert v_pools.shape == k_pools.shape and v_pools.stride() == k_pools.stride()
    st = lib().copy_kv_slots(_ptr(k_pools), _ptr(v_pools), layers, k_pools.stride(0), n, P,
                             page_stride, H, D, _dtype(k_pools), _ptr(src_slots), _ptr(dst_slots),
                             src_slots.numel(), PKV_FLAG_CHECKED if checked else 0, _ptr(err),
                             _stream(stream))
    _check("copy_kv_slots", st)


LAYOUT_COMMITTED_PER_BLOCK = 93
LAYOUT_CURRENT_PER_BLOCK = 62


def causal_layout_buffers(num_staged, block_size, row_stride, device="cuda"):
    """Output tensors of :func:`causal_layout` for a forward of ``num_staged``
    tokens in blocks of ``block_size`` (allocated here, by the caller's side)."""
    import torch
    nb = (num_staged + block_size - 1) // block_size
    i32 = dict(dtype=torch.int32, device=device)
    i64 = dict(dtype=torch.int64, device=device)
    return dict(rows=torch.full((nb, row_stride), -1, **i32), kv_lens=torch.zeros(nb, **i32),
                q_indptr=torch.zeros(nb + 1, **i32), staged_slots=torch.full((num_staged,), -1, **i64),
                staged_slots2=torch.full((num_staged,), -1, **i64),
                committed_src=torch.full((nb * LAYOUT_COMMITTED_PER_BLOCK,), -1, **i64),
                committed_dst=torch.full((nb * LAYOUT_COMMITTED_PER_BLOCK,), -1, **i64),
                current_src_idx=torch.full((nb * LAYOUT_CURRENT_PER_BLOCK,), -1, **i64),
                current_dst=torch.full((nb * LAYOUT_CURRENT_PER_BLOCK,), -1, **i64))


def causal_layout(table, committed, pin_tokens, window_tokens, num_staged, block_size,
                  private_pages, out, err=None, stream=None):
    """Per-block rows over exact windows (see ``include/pkv.h``).  ``table``:
    int32 logical page table; ``committed``: int64 device scalar (history
    tokens); ``private_pages``: int32 ``[blocks, stride]``; ``out``: the dict of
    :func:`causal_layout_buffers`, rewritten in place."""
    assert private_pages.dim() == 2 and private_pages.is_contiguous()
    rows = out["rows"]
    st = lib().causal_layout(_ptr(table), table.numel(), _ptr(committed), pin_tokens, window_tokens,
                             num_staged, block_size, _ptr(private_pages), private_pages.shape[1], 32,
                             _ptr(rows), rows.shape[1], _ptr(out["kv_lens"]), _ptr(out["q_indptr"]),
                             _ptr(out["staged_slots"]), _ptr(out["staged_slots2"]),
                             _ptr(out["committed_src"]), _ptr(out["committed_dst"]),
                             out["committed_src"].numel(), _ptr(out["current_src_idx"]),
                             _ptr(out["current_dst"]), out["current_src_idx"].numel(), _ptr(err),
                             _stream(stream))
    _check("causal_layout", st)


def plan_buffers(batch, group_row_stride, device="cuda"):
    """Output tensors of :func:`plan_shared_prefix` for a batch of ``batch`` rows."""
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    return dict(group_rows=torch.full((batch, group_row_stride), -1, **i32),
                run_lens=torch.zeros(batch, **i32), group_indptr=torch.zeros(batch + 1, **i32),
                perm=torch.zeros(batch, **i32), group_of=torch.zeros(batch, **i32),
                tail_start=torch.zeros(batch, **i32), tail_lens=torch.zeros(batch, **i32),
                num_groups=torch.zeros(1, **i32))


def plan_shared_prefix(block_table, kv_lens, q_indptr, out, max_pages=None, err=None, stream=None):
    """Shared-prefix grouping of the batch's rows (see ``include/pkv.h``);
    ``out``: the dict of :func:`plan_buffers`, rewritten in place."""
    B = kv_lens.numel()
    mp = block_table.shape[1] if max_pages is None else max_pages
    gr = out["group_rows"]
    st = lib().plan_shared_prefix(_ptr(block_table), block_table.stride(0), _ptr(kv_lens), _ptr(q_indptr), B,
                                  mp, _ptr(gr), gr.shape[1], _ptr(out["run_lens"]), _ptr(out["group_indptr"]),
                                  _ptr(out["perm"]), _ptr(out["group_of"]), _ptr(out["tail_start"]),
                                  _ptr(out["tail_lens"]), _ptr(out["num_groups"]), _ptr(err),
                                  _stream(stream))
    _check("plan_shared_prefix", st)


def shared_prefix_attention_workspace_size(batch, max_q_len, max_group_tokens, max_group_keys,
                                           num_q_heads, num_kv_heads, head_dim, num_splits=0) -> int:
    return int(lib().shared_prefix_attention_workspace_size(batch, max_q_len, max_group_tokens,
                                                            max_group_keys, num_q_heads, num_kv_heads,
                                                            head_dim, num_splits))


def shared_prefix_attention(q, k_pool, v_pool, plan, q_indptr, out, *, max_q_len, max_group_tokens,
                            max_group_keys, lse=None, scale=0.0, workspace=None, num_splits=0, flags=0,
                            err=None, stream=None):
    """One-launch attention of a planned batch (``plan``: the dict of
    :func:`plan_buffers` after :func:`plan_shared_prefix`); outputs at the
    tokens' own positions in ``out [tokens, Hq, D]`` / ``lse [tokens, Hq]``."""
    n, P, H, D, page_stride = _pool_geometry(k_pool)
    assert v_pool.shape == k_pool.shape and v_pool.stride() == k_pool.stride()
    assert q.stride(2) == 1 and out.is_contiguous()
    B = q_indptr.numel() - 1
    gr = plan["group_rows"]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().shared_prefix_attention(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k_pool), _ptr(v_pool), n, P, page_stride, _ptr(gr),
        gr.stride(0), _ptr(plan["run_lens"]), _ptr(plan["group_indptr"]), _ptr(plan["perm"]),
        _ptr(plan["tail_start"]), _ptr(plan["tail_lens"]), _ptr(plan["num_groups"]), _ptr(q_indptr), B,
        max_q_len, max_group_tokens, max_group_keys, q.shape[1], H, D, scale, _ptr(out), _dtype(out),
        _ptr(lse), _ptr(workspace), ws_bytes, num_splits, flags, _ptr(err), _stream(stream))
    _check("shared_prefix_attention", st)


# ----------------------------------------------------------------------------
# The entry points below check their tensors here: a wrong type, shape, stride
# or device raises ValueError before a pointer is handed out.  The checks are
# written flat, since a small call's cost is its host time.
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_FP8_TYPES = (torch.float8_e4m3fn, torch.uint8)


def _pools(k_pool, v_pool):
    """Shape and page stride of two like pools with dense slots."""
    shape, st = k_pool.shape, k_pool.stride()
    if len(shape) != 4:
        raise ValueError("pools must be [num_pages, page_size, num_kv_heads, head_dim]")
    n, P, H, D = shape
    if st[3] != 1 or st[2] != D or st[1] != H * D:
        raise ValueError("pool slots must be dense [num_kv_heads, head_dim] rows")
    if v_pool.shape != shape or v_pool.stride() != st or v_pool.dtype != k_pool.dtype:
        raise ValueError("K and V pools must have the same shape, strides and type")
    return n, P, H, D, st[0]


def _scales(k_scale, v_scale, n, H):
    """Page stride of the f32 scales ``[num_pages, Hkv]`` (unit head stride)."""
    st = k_scale.stride()
    if (k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or k_scale.shape != (n, H) or
            v_scale.shape != (n, H) or v_scale.stride() != st or (H > 1 and st[1] != 1)):
        raise ValueError("scales must be float32 [num_pages, num_kv_heads] with unit head stride, K's and V's alike")
    if n <= 1:  # one page: whatever its stride says, nothing is taken by it
        return H
    if st[0] < H:
        raise ValueError("scales of different pages must not overlap (an expanded tensor needs a copy)")
    return st[0]


def _tables(block_table, kv_lens, q_indptr, q_real, batch, keys):
    """The batch size and the table's row stride, for up to ``keys`` keys a row."""
    count = kv_lens.numel()
    if batch is None:
        batch = count
    if (kv_lens.dtype is not _I32 or q_indptr.dtype is not _I32 or count < batch or q_indptr.numel() <= batch or
            not kv_lens.is_contiguous() or not q_indptr.is_contiguous()):
        raise ValueError("kv_lens [batch] and q_indptr [batch + 1] must be dense int32")
    if q_real is not None and (q_real.dtype is not _I32 or q_real.numel() < batch or not q_real.is_contiguous()):
        raise ValueError("q_real must be dense int32 [batch]")
    st, shape = block_table.stride(), block_table.shape
    if (block_table.dtype is not _I32 or len(shape) != 2 or shape[0] < batch or (st[1] != 1 and shape[1] > 1) or
            shape[1] * 32 < keys):
        raise ValueError("block_table must be int32 [batch, pages] with unit last stride and room for max_kv_len keys")
    return batch, shape[1] if shape[0] == 1 else st[0]


def _states(q, out, lse, D):
    """Token and head stride of packed query rows, after the outputs are checked."""
    shape, st = q.shape, q.stride()
    if q.dtype is not _BF16 or len(shape) != 3 or shape[2] != D or st[2] != 1:
        raise ValueError("q must be bf16 [rows, num_q_heads, head_dim] with unit last stride")
    if out.shape != shape or not out.is_contiguous() or out.dtype not in _DTYPES:
        raise ValueError("out must be dense bf16 or float32 with the shape of q")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse must be dense float32 [rows, num_q_heads]")
    return st


def _mask(name):
    if name not in MASKS:
        raise ValueError(f"mask {name!r} (one of {', '.join(MASKS)})")
    return MASKS[name]


def _scratch(workspace, err):
    """The tensors whose bytes are written without regard to their type."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("the workspace must be dense")
    if err is not None and (err.dtype is not _I32 or not err.numel()):
        raise ValueError("err must be an int32")


def _on_device(tensors):
    """All on the current CUDA device: the launch goes there."""
    devs = {t.get_device() for t in tensors if t is not None}
    dev = devs.pop()
    if devs or dev < 0:
        raise ValueError("tensors must be on one CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _launch_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _address(t):
    return None if t is None else t.data_ptr()


def _bytes(workspace):
    return 0 if workspace is None else workspace.nbytes


def kv_append_fp8(k_src, v_src, block_table, kv_lens, q_indptr, k_pool, v_pool, k_scale, v_scale, *,
                  q_real=None, batch=None, max_q_rows, max_kv_len, checked=False, err=None, stream=None):
    """Quantise this step's rows ``k_src``/``v_src [rows, Hkv, D]`` (bf16, f16
    or f32, any token/head stride of whole 16 bytes) into e4m3 pools and their
    per-page, per-head scales, in place (see ``include/pkv.h``)."""
    n, P, H, D, page_stride = _pools(k_pool, v_pool)
    if k_pool.dtype not in _FP8_TYPES:
        raise ValueError("8-bit pools must be float8_e4m3fn (or its bytes as uint8)")
    scale_stride = _scales(k_scale, v_scale, n, H)
    shape, st = k_src.shape, k_src.stride()
    if v_src.shape != shape or v_src.stride() != st or v_src.dtype != k_src.dtype:
        raise ValueError("k_src and v_src must have the same shape, strides and dtype")
    if len(shape) != 3 or shape[1] != H or shape[2] != D or st[2] != 1:
        raise ValueError("sources must be [rows, num_kv_heads, head_dim] with unit last stride")
    if k_src.dtype not in (_BF16, torch.float16, _F32):
        raise ValueError("sources must be bf16, f16 or f32")
    batch, table_stride = _tables(block_table, kv_lens, q_indptr, q_real, batch, max_kv_len)
    _scratch(None, err)
    dev = _on_device((k_src, v_src, block_table, kv_lens, q_indptr, q_real, k_pool, v_pool, k_scale, v_scale, err))
    status = lib().kv_append_fp8(
        k_src.data_ptr(), v_src.data_ptr(), _dtype(k_src), st[0], st[1], block_table.data_ptr(), table_stride,
        kv_lens.data_ptr(), q_indptr.data_ptr(), _address(q_real), batch, max_q_rows, max_kv_len, H, D,
        k_pool.data_ptr(), v_pool.data_ptr(), n, P, page_stride, k_scale.data_ptr(), v_scale.data_ptr(),
        scale_stride, PKV_FLAG_CHECKED if checked else 0, _address(err), _launch_stream(stream, dev))
    if status:
        _check("kv_append_fp8", status)


def paged_attention_fp8_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim, max_kv_len,
                                       window=0, num_sinks=0, flags=0) -> int:
    return int(lib().paged_attention_fp8_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim,
                                                        max_kv_len, window, num_sinks, flags))


def paged_attention_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, kv_lens, q_indptr, out, *,
                        q_real=None, lse=None, batch=None, max_q_rows, max_kv_len, mask="causal",
                        causal_block=0, window=0, num_sinks=0, scale=0.0, workspace=None, flags=0, err=None,
                        stream=None):
    """``paged_attention`` over e4m3 pools with a scale per page and head (as
    :func:`kv_append_fp8` writes them); ``window`` > 0 limits causal rows to
    their last ``window`` keys and the first ``num_sinks``."""
    n, P, H, D, page_stride = _pools(k_pool, v_pool)
    if k_pool.dtype not in _FP8_TYPES:
        raise ValueError("8-bit pools must be float8_e4m3fn (or its bytes as uint8)")
    scale_stride = _scales(k_scale, v_scale, n, H)
    st = _states(q, out, lse, D)
    batch, table_stride = _tables(block_table, kv_lens, q_indptr, q_real, batch, max_kv_len)
    _scratch(workspace, err)
    mask = _mask(mask)
    dev = _on_device((q, k_pool, v_pool, k_scale, v_scale, block_table, kv_lens, q_indptr, q_real, out, lse,
                      workspace, err))
    status = lib().paged_attention_fp8(
        q.data_ptr(), st[0], st[1], k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        scale_stride, n, P, page_stride, block_table.data_ptr(), table_stride, kv_lens.data_ptr(),
        q_indptr.data_ptr(), _address(q_real), batch, max_q_rows, max_kv_len, q.shape[1], H, D, mask,
        causal_block, window, num_sinks, scale, out.data_ptr(), _dtype(out), _address(lse), _address(workspace),
        _bytes(workspace), flags, _address(err), _launch_stream(stream, dev))
    if status:
        _check("paged_attention_fp8", status)


def paged_attention_window_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads, head_dim, max_kv_len,
                                          window, num_sinks=0, flags=0) -> int:
    return int(lib().paged_attention_window_workspace_size(batch, max_q_rows, num_q_heads, num_kv_heads,
                                                           head_dim, max_kv_len, window, num_sinks, flags))


def paged_attention_window(q, k_pool, v_pool, block_table, kv_lens, q_indptr, out, *, window, num_sinks=0,
                           q_real=None, lse=None, batch=None, max_q_rows, max_kv_len, scale=0.0,
                           workspace=None, flags=0, err=None, stream=None):
    """Causal ``paged_attention`` of bf16 pools in which a row sees its last
    ``window`` keys (its own among them) and the first ``num_sinks``; pages
    that no row sees are not read."""
    n, P, H, D, page_stride = _pools(k_pool, v_pool)
    if k_pool.dtype is not _BF16:
        raise ValueError("pools must be bf16")
    st = _states(q, out, lse, D)
    batch, table_stride = _tables(block_table, kv_lens, q_indptr, q_real, batch, max_kv_len)
    _scratch(workspace, err)
    dev = _on_device((q, k_pool, v_pool, block_table, kv_lens, q_indptr, q_real, out, lse, workspace, err))
    status = lib().paged_attention_window(
        q.data_ptr(), st[0], st[1], k_pool.data_ptr(), v_pool.data_ptr(), n, P, page_stride,
        block_table.data_ptr(), table_stride, kv_lens.data_ptr(), q_indptr.data_ptr(), _address(q_real), batch,
        max_q_rows, max_kv_len, q.shape[1], H, D, window, num_sinks, scale, out.data_ptr(), _dtype(out),
        _address(lse), _address(workspace), _bytes(workspace), flags, _address(err),
        _launch_stream(stream, dev))
    if status:
        _check("paged_attention_window", status)


# ----------------------------------------------------------------------------
LATENT_DIM, LATENT_ROPE = 512, 64
NOPE_DIM, EXPANDED_V = 128, 128
_I64 = torch.int64


def _vector(t, name, dtype, count):
    if t.dtype is not dtype or t.numel() < count or not t.is_contiguous():
        raise ValueError(f"{name} must be dense {dtype} with room for {count}")


def _heads(t, name, rows, heads, width):
    """Token and head stride of a bf16 [rows, heads, width] tensor with unit last
    stride (rows or heads None: any); axes of one element take the dense stride,
    as theirs may say anything.  Also its rows and heads."""
    shape, st = t.shape, t.stride()
    if t.dtype is not _BF16 or len(shape) != 3 or st[2] != 1:
        raise ValueError(f"{name} must be bf16 [rows, heads, {width}] with unit last stride")
    n, h, w = shape
    if w != width or (rows is not None and n != rows) or (heads is not None and h != heads):
        raise ValueError(f"{name} must have the shape [{rows or 'rows'}, {heads or 'heads'}, {width}]")
    head = st[1] if h > 1 else width
    return st[0] if n > 1 else head * h, head, n, h


def _latent_pool(pool):
    """Pages, page size and page stride of a latent pool."""
    shape, st = pool.shape, pool.stride()
    if pool.dtype is not _BF16 or len(shape) != 3 or st[2] != 1:
        raise ValueError("the pool must be bf16 [num_pages, page_size, 512 + 64] with unit last stride")
    n, P, row = shape
    if row != LATENT_DIM + LATENT_ROPE or (P > 1 and st[1] != row):
        raise ValueError("the pool must hold dense slots of 512 + 64")
    return n, P, st[0] if n > 1 else P * row


def assign_step_pages(new_lens, kv_lens, num_free, free_pages, block_table, *, kv_lens_out, num_free_out, q_indptr,
                      slots, positions, err=None, stream=None):
    """Block tables, query ranges and slot map of a step, built on the device:
    ``new_lens [batch]`` tokens are asked for by sequences of ``kv_lens`` keys
    (below zero: finished), pages come from and go back to the stack
    ``free_pages[:num_free]`` (see ``include/pkv.h``).  ``kv_lens_out`` and
    ``num_free_out`` may be the inputs themselves.  Requests are granted in
    order: one that does not fit holds back those behind it, so one that never
    can (more tokens than ``slots`` has, more pages than the table's width) must
    be withdrawn or asked for in pieces.  An empty batch leaves an empty step:
    no slot, no query row."""
    batch, tokens, shape = new_lens.numel(), slots.numel(), block_table.shape
    _vector(new_lens, "new_lens", _I32, batch)
    _vector(kv_lens, "kv_lens", _I32, batch)
    _vector(num_free, "num_free", _I32, 1)
    _vector(free_pages, "free_pages", _I32, 0)
    _vector(kv_lens_out, "kv_lens_out", _I32, batch)
    _vector(num_free_out, "num_free_out", _I32, 1)
    _vector(q_indptr, "q_indptr", _I32, batch + 1)
    _vector(slots, "slots", _I64, tokens)
    _vector(positions, "positions", _I64, tokens)
    if block_table.dtype is not _I32 or len(shape) != 2 or shape[0] < batch or not block_table.is_contiguous():
        raise ValueError("block_table must be dense int32 [batch, pages]: its width bounds a sequence's pages")
    _scratch(None, err)
    dev = _on_device((new_lens, kv_lens, num_free, free_pages, block_table, kv_lens_out, num_free_out, q_indptr, slots,
                      positions, err))
    if not batch:
        _empty_step(num_free, free_pages, num_free_out, q_indptr, slots, positions, err, stream, dev)
        return
    status = lib().assign_step_pages(
        new_lens.data_ptr(), kv_lens.data_ptr(), num_free.data_ptr(), free_pages.data_ptr(), free_pages.numel(),
        block_table.data_ptr(), shape[1], batch, tokens, 32, kv_lens_out.data_ptr(), num_free_out.data_ptr(),
        q_indptr.data_ptr(), slots.data_ptr(), positions.data_ptr(), _address(err), _launch_stream(stream, dev))
    if status:
        _check("assign_step_pages", status)


def _empty_step(num_free, free_pages, num_free_out, q_indptr, slots, positions, err, stream, dev):
    """The outputs of a step without sequences, which the library leaves
    unwritten: an earlier step's slots must not be taken for this one's."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        # (an external stream of address 0 would be a new one, not the default one)
        stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        slots.fill_(-1)
        positions.zero_()
        q_indptr[(0,) * q_indptr.dim()].zero_()
        free = num_free[(0,) * num_free.dim()]
        height = free.clamp(0, free_pages.numel())
        if err is not None:
            err[(0,) * err.dim()].bitwise_or_((height != free).int() * PKV_ERRBIT_PAGE)
        num_free_out[(0,) * num_free_out.dim()].copy_(height)


def kv_append_latent(src, positions, cos_sin, slots, pool, *, norm_weight=None, eps=1e-6, q_pe=None, q_out=None,
                     interleaved=False, checked=False, err=None, stream=None):
    """Normalise ``src[:, :512]`` by its root mean square (with
    ``norm_weight``), rotate ``src[:, 512:]`` and write the rows into pool slots
    ``slots``; rotate ``q_pe [T, H, 64]`` into ``q_out`` (see ``include/pkv.h``)."""
    n, P, page_stride = _latent_pool(pool)
    st = src.stride()
    T, row = src.shape
    if src.dtype is not _BF16 or row != LATENT_DIM + LATENT_ROPE or st[1] != 1:
        raise ValueError("src must be bf16 [tokens, 512 + 64] with unit last stride")
    _vector(positions, "positions", _I64, T)
    _vector(slots, "slots", _I64, T)
    table = cos_sin.shape
    if cos_sin.dtype is not _F32 or len(table) != 2 or table[1] != LATENT_ROPE or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be dense float32 [max_position, 64]")
    if norm_weight is not None:
        _vector(norm_weight, "norm_weight", _BF16, LATENT_DIM)
    qt = qh = ot = oh = heads = 0
    if q_pe is not None and q_out is not None:
        qt, qh, _, heads = _heads(q_pe, "q_pe", T, None, LATENT_ROPE)
        ot, oh, _, _ = _heads(q_out, "q_out", T, heads, LATENT_ROPE)
    elif q_pe is not None or q_out is not None:
        raise ValueError("q_pe and q_out come together")
    _scratch(None, err)
    dev = _on_device((src, positions, cos_sin, slots, pool, norm_weight, q_pe, q_out, err))
    status = lib().kv_append_latent(
        src.data_ptr(), st[0] if T > 1 else row, T, _address(norm_weight), eps, positions.data_ptr(),
        cos_sin.data_ptr(), table[0], interleaved, slots.data_ptr(), pool.data_ptr(), n, P, page_stride,
        LATENT_DIM, LATENT_ROPE, _address(q_pe), qt, qh, _address(q_out), ot, oh, heads,
        PKV_FLAG_CHECKED if checked else 0, _address(err), _launch_stream(stream, dev))
    if status:
        _check("kv_append_latent", status)


def paged_attention_latent_workspace_size(batch, max_q_rows, num_heads, max_kv_len, flags=0) -> int:
    return int(lib().paged_attention_latent_workspace_size(batch, max_q_rows, num_heads, max_kv_len, LATENT_DIM,
                                                           LATENT_ROPE, flags))


def _outputs(out, lse, rows, heads, width):
    if out.shape != (rows, heads, width) or not out.is_contiguous() or out.dtype not in _DTYPES:
        raise ValueError(f"out must be dense bf16 or float32 [rows, num_heads, {width}]")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (rows, heads) or not lse.is_contiguous()):
        raise ValueError("lse must be dense float32 [rows, num_heads]")


def paged_attention_latent(q, pool, block_table, kv_lens, q_indptr, out, *, q_real=None, lse=None, batch=None,
                           max_q_rows, max_kv_len, mask="causal", scale, workspace=None, flags=0, err=None,
                           stream=None):
    """Attention of absorbed queries ``q [rows, H, 512 + 64]`` over the latent
    rows of ``pool``, into ``out [rows, H, 512]`` (bf16 or f32) and ``lse``."""
    n, P, page_stride = _latent_pool(pool)
    qt, qh, rows, heads = _heads(q, "q", None, None, LATENT_DIM + LATENT_ROPE)
    _outputs(out, lse, rows, heads, LATENT_DIM)
    batch, table_stride = _tables(block_table, kv_lens, q_indptr, q_real, batch, max_kv_len)
    _scratch(workspace, err)
    mask = _mask(mask)
    dev = _on_device((q, pool, block_table, kv_lens, q_indptr, q_real, out, lse, workspace, err))
    status = lib().paged_attention_latent(
        q.data_ptr(), qt, qh, pool.data_ptr(), n, P, page_stride, block_table.data_ptr(), table_stride,
        kv_lens.data_ptr(), q_indptr.data_ptr(), _address(q_real), batch, max_q_rows if rows else 0, max_kv_len, heads,
        LATENT_DIM, LATENT_ROPE, mask, scale, out.data_ptr(), _dtype(out), _address(lse), _address(workspace),
        _bytes(workspace), flags, _address(err), _launch_stream(stream, dev))
    if status:
        _check("paged_attention_latent", status)


def ragged_attention_latent(q, k, k_pe, v, q_indptr, kv_indptr, out, *, lse=None, batch=None, max_q_rows, max_kv_len,
                            mask="causal", scale, flags=0, err=None, stream=None):
    """Attention of ``q [rows, H, 128 + 64]`` over ragged expanded keys ``k
    [keys, H, 128]`` with the shared ``k_pe [keys, 64]`` and values ``v [keys, H,
    128]``, into ``out [rows, H, 128]`` (bf16 or f32) and ``lse``."""
    qt, qh, rows, heads = _heads(q, "q", None, None, NOPE_DIM + LATENT_ROPE)
    _outputs(out, lse, rows, heads, EXPANDED_V)
    kt, kh, keys, _ = _heads(k, "k", None, heads, NOPE_DIM)
    vt, vh, _, _ = _heads(v, "v", keys, heads, EXPANDED_V)
    if k_pe.dtype is not _BF16 or k_pe.shape != (keys, LATENT_ROPE) or k_pe.stride(1) != 1:
        raise ValueError("k_pe must be bf16 [keys, 64] with unit last stride")
    if batch is None:
        batch = q_indptr.numel() - 1
    _vector(q_indptr, "q_indptr", _I32, batch + 1)
    _vector(kv_indptr, "kv_indptr", _I32, batch + 1)
    _scratch(None, err)
    mask = _mask(mask)
    dev = _on_device((q, k, k_pe, v, q_indptr, kv_indptr, out, lse, err))
    status = lib().ragged_attention_latent(
        q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, k_pe.data_ptr(), k_pe.stride(0) if keys > 1 else LATENT_ROPE,
        v.data_ptr(), vt, vh, keys, q_indptr.data_ptr(), kv_indptr.data_ptr(), batch, max_q_rows if rows else 0, max_kv_len,
        heads, NOPE_DIM, LATENT_ROPE, EXPANDED_V, mask, scale, out.data_ptr(), _dtype(out), _address(lse), flags, _address(err),
        _launch_stream(stream, dev))
    if status:
        _check("ragged_attention_latent", status)
