"""Full attention over a paged cache: rotary positions, appending new tokens, attention of
them over the cache, and the bookkeeping of its pages.  Argument marshalling only, as in the
package's __init__; the functions are reached through the package.
"""
from __future__ import annotations

import ctypes

import torch

from . import (GDN_FLAG_ROPE_BACKWARD, GDN_FLAG_ROPE_INTERLEAVED, GDN_FLAG_SIMT, GDN_FLAG_TEST_NO_WAIT,
               GDN_MAX_POOLS, GDN_ROPE_SCALING, GdnCacheShape, GdnPagePools, GdnPageTables, Workspace, _check,
               _dtype_code, _need_cuda, _ptr, _stream, _ws_cache, load)


def _handle(t, stream):
    """The stream of a call on t's device, as an integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return _stream(t, stream).value or 0


def gdn_rope_inv_freq(rotary_dim, base=10000.0, scaling="none", factor=1.0, orig_len=0, alpha=1.0, beta=32.0):
    """Frequencies of the rotary pairs, fp64 on the CPU [rotary_dim / 2]: base^(-2i / rotary_dim), with
    scaling "linear" (over factor), "base" (a larger base) or "parts" (by parts, over orig_len positions)."""
    out = torch.empty(max(0, rotary_dim // 2), dtype=torch.float64)
    _check(load().gdn_rope_inv_freq(rotary_dim, base, GDN_ROPE_SCALING[scaling], factor, orig_len, alpha, beta,
                                    _ptr(out)), "gdn_rope_inv_freq")
    return out


def gdn_rope_freqs(inv_freq, device="cuda"):
    """The device table that gdn_rope and gdn_kv_append read (made once): int64 words holding each
    frequency of inv_freq (fp64, CPU) in turns as a 64-bit fraction."""
    inv = inv_freq.detach().to("cpu", torch.float64).contiguous()
    assert inv.dim() == 1
    out = torch.empty(inv.numel(), dtype=torch.int64)
    _check(load().gdn_rope_freqs(_ptr(inv), inv.numel(), _ptr(out)), "gdn_rope_freqs")
    return out.to(device)


def _heads(name, t, D=None):
    """Token stride of t [n_tok, H, D] whose heads and features are contiguous within a token."""
    n, h, d = t.shape
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError(f"{name}: heads and features must be contiguous within a token")
    if D is not None and d != D:
        raise ValueError(f"{name}: head width {d}, expected {D}")
    return s[0] if n > 1 else h * d


def _rotary(freqs, D):
    if freqs is None:
        return 0
    if freqs.dtype != torch.int64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise TypeError("freqs must be a table of gdn_rope_freqs")
    if 2 * freqs.numel() > D:
        raise ValueError("freqs holds more pairs than a head")
    return 2 * freqs.numel()


def gdn_rope(q, k, positions, freqs, interleaved=False, scale=1.0, backward=False, q_out=None, k_out=None,
             stream=None):
    """Rotary positions of q [n_tok, Hq, D] and k [n_tok, Hk, D] (either may be None) over the first
    2 * len(freqs) elements of each head, times scale there; positions int64 [n_tok].  backward=True
    takes gradients of the outputs to those of the inputs.  q_out / k_out may be q / k.
    Returns (q_out, k_out)."""
    x = q if q is not None else k
    _need_cuda(q, k, positions, freqs, q_out, k_out)
    n_tok, _, D = x.shape
    if positions.dtype != torch.int64 or positions.numel() != n_tok or not positions.is_contiguous():
        raise TypeError("positions must be contiguous int64 [n_tok]")
    rd = _rotary(freqs, D)
    dtype = x.dtype

    def side(name, t, out):
        """(input, output, heads, input stride, output stride, output tensor)"""
        if t is None:
            return None, None, 0, 0, 0, None
        if t.shape[0] != n_tok or t.dtype != dtype:
            raise ValueError("q and k must have the same tokens and dtype")
        stride = _heads(name, t, D)
        if out is None:
            out = torch.empty(t.shape, dtype=dtype, device=t.device)
            out_stride = 0
        else:
            if out.shape != t.shape or out.dtype != dtype:
                raise ValueError(f"{name}_out must have {name}'s shape and dtype")
            out_stride = _heads(name + "_out", out, D)
        return t.data_ptr(), out.data_ptr(), t.shape[1], stride, out_stride, out

    qp, qop, hq, qs, qos, q_out = side("q", q, q_out)
    kp, kop, hk, ks, kos, k_out = side("k", k, k_out)
    flags = (GDN_FLAG_ROPE_INTERLEAVED if interleaved else 0) | (GDN_FLAG_ROPE_BACKWARD if backward else 0)
    st = load().gdn_rope(qp, kp, positions.data_ptr(), None if freqs is None else freqs.data_ptr(), _dtype_code(dtype),
                         n_tok, hq, hk, D, rd, qs, ks, qos, kos, scale, flags, qop, kop, _handle(x, stream))
    if st:
        _check(st, "gdn_rope")
    return q_out, k_out


_cache_shapes = {}


def cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, k=None, v=None) -> GdnCacheShape:
    """Shape of a paged call: q [n_tok, Hq, D] (or None), caches [n_pages, page_size, Hkv, D] (any order of
    pages, slots and heads in memory; D contiguous), page_table int32 [n_seqs, max_pages], seq_lens
    int32 [n_seqs], cu_seqlens int32 [n_seqs + 1] or None, new k, v [n_tok, Hkv, D]."""
    x = q if q is not None else k
    key = (None if q is None else (q.shape, q.stride()), k_cache.shape, k_cache.stride(), v_cache.shape,
           v_cache.stride(), page_table.shape, page_table.stride(), seq_lens.shape,
           None if cu_seqlens is None else cu_seqlens.shape, x.dtype, k_cache.dtype, v_cache.dtype,
           None if k is None else (k.shape, k.stride(), k.dtype), None if v is None else (v.shape, v.stride(), v.dtype),
           page_table.dtype, seq_lens.dtype, None if cu_seqlens is None else cu_seqlens.dtype)
    sh = _cache_shapes.get(key)
    if sh is not None:
        return sh
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must be [n_pages, page_size, Hkv, D] with the same strides")
    n_pages, page_size, Hkv, D = k_cache.shape
    if D > 1 and k_cache.stride(3) != 1:
        raise ValueError("the caches' last dimension must be contiguous")
    if any(t is not None and t.dtype != x.dtype for t in (k_cache, v_cache, k, v)):
        raise TypeError("q, k, v and the caches must have one dtype")
    for name, t in (("page_table", page_table), ("seq_lens", seq_lens), ("cu_seqlens", cu_seqlens)):
        if t is not None and t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    n_seqs, max_pages = page_table.shape
    if max_pages > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be contiguous")
    if seq_lens.shape != (n_seqs,) or (n_seqs > 1 and seq_lens.stride(0) != 1):
        raise ValueError("seq_lens must be contiguous [n_seqs]")
    n_tok = x.shape[0]
    if cu_seqlens is None and n_tok != n_seqs:
        raise ValueError("without cu_seqlens every sequence has one new token")
    if cu_seqlens is not None and (cu_seqlens.shape != (n_seqs + 1,) or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be contiguous [n_seqs + 1]")
    for name, t in (("k", k), ("v", v)):
        if t is not None and t.shape != (n_tok, Hkv, D):
            raise ValueError(f"{name} must be [n_tok, Hkv, D]")
    Hq = Hkv if q is None else q.shape[1]
    if Hq % Hkv:
        raise ValueError("Hq must be a multiple of Hkv")
    st = k_cache.stride()
    sh = GdnCacheShape(n_seqs, n_tok, Hq, Hkv, D, _dtype_code(x.dtype), page_size, n_pages, max_pages,
                       page_table.stride(0) if n_seqs > 1 else max_pages, st[0], st[1], st[2],
                       0 if q is None else _heads("q", q, D), 0 if k is None else _heads("k", k, D),
                       0 if v is None else _heads("v", v, D))
    if len(_cache_shapes) >= 4096:
        _cache_shapes.clear()
    _cache_shapes[key] = sh
    return sh


def _own_workspace(kind, nbytes, t, stream):
    """A workspace of this kind for calls on this device and stream, which run one after another."""
    handle = _handle(t, stream)
    key = (kind, t.get_device(), handle)
    ws = _ws_cache.get(key)
    if ws is None or ws.nbytes < nbytes:
        ws = _ws_cache[key] = Workspace(nbytes, t.device)
    return ws, handle


def gdn_kv_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, q=None, freqs=None,
                  positions=None, interleaved=False, scale=1.0, q_out=None, workspace=None, stream=None):
    """The new tokens' k, v [n_tok, Hkv, D] into the cache at the end of their sequences (seq_lens counts
    them already), k rotated on the way with freqs, and q [n_tok, Hq, D] rotated into q_out (a new
    tensor, or q itself).  positions int64 [n_tok] replaces the places in the sequences as rotary
    positions.  Returns q_out (None without q)."""
    _need_cuda(q, k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens, freqs, positions, q_out)
    sh = cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, k, v)
    rd = _rotary(freqs, sh.D)
    if positions is not None and (positions.dtype != torch.int64 or positions.shape != (sh.n_tok,)
                                  or not positions.is_contiguous()):
        raise TypeError("positions must be contiguous int64 [n_tok]")
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape or q_out.dtype != q.dtype or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous with q's shape and dtype")
    ws, handle = ((workspace, _handle(k, stream)) if workspace is not None
                  else _own_workspace("cache", 256, k, stream))
    flags = GDN_FLAG_ROPE_INTERLEAVED if interleaved else 0
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _check(load().gdn_kv_append(p(q), k.data_ptr(), v.data_ptr(), p(positions), p(freqs), rd, scale, flags,
                                page_table.data_ptr(), seq_lens.data_ptr(), p(cu_seqlens), ctypes.byref(sh),
                                None if q is None else p(q_out), k_cache.data_ptr(), v_cache.data_ptr(), ws.ptr(),
                                ws.nbytes, handle), "gdn_kv_append")
    return q_out if q is not None else None


def gdn_paged_attn_workspace_bytes(shape: GdnCacheShape, max_new: int) -> int:
    return int(load().gdn_paged_attn_workspace_bytes(ctypes.byref(shape), int(max_new)))


_attn_bytes = {}


def gdn_paged_attn(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, max_new=None, scale=None, window=0,
                   want_lse=False, o=None, lse=None, simt=False, workspace=None, stream=None, _test_no_wait=False):
    """Attention of the new tokens q [n_tok, Hq, D] over the paged cache, which holds their k and v already:
    the token at position p of its sequence sees the last `window` positions up to p (0: all).
    max_new: a bound on the new tokens of one sequence (default: all of them).  Returns
    (o [n_tok, Hq, D], lse [n_tok, Hq] fp32 or None)."""
    _need_cuda(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, o, lse)
    sh = cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens)
    if max_new is None:
        max_new = sh.n_tok if cu_seqlens is not None else 1
    if scale is None:
        scale = sh.D ** -0.5
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous():
        raise ValueError("o must be contiguous with q's shape and dtype")
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    elif lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [n_tok, Hq]")
    if workspace is None:
        nbytes = gdn_paged_attn_workspace_bytes(sh, max_new)
        ws, handle = _own_workspace("attn", nbytes, q, stream)
    else:
        ws, handle = workspace, _handle(q, stream)
    flags = (GDN_FLAG_SIMT if simt else 0) | (GDN_FLAG_TEST_NO_WAIT if _test_no_wait else 0)
    _check(load().gdn_paged_attn(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                 seq_lens.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(),
                                 ctypes.byref(sh), max_new, scale, window, flags, o.data_ptr(),
                                 None if lse is None else lse.data_ptr(), ws.ptr(), ws.nbytes, handle),
           "gdn_paged_attn")
    return o, lse


def gdn_pages_workspace_bytes(n_pages: int, n_rows: int) -> int:
    return int(load().gdn_pages_workspace_bytes(int(n_pages), int(n_rows)))


def _page_tables(page_table, seq_lens, refs, page_size):
    _need_cuda(page_table, seq_lens, refs)
    for name, t, dims in (("page_table", page_table, 2), ("seq_lens", seq_lens, 1), ("refs", refs, 1)):
        if t.dtype != torch.int32 or t.dim() != dims or (t.numel() > 1 and t.stride(-1) != 1 and t.shape[-1] > 1):
            raise TypeError(f"{name} must be int32 with contiguous rows")
    n_rows, max_pages = page_table.shape
    if seq_lens.shape[0] != n_rows:
        raise ValueError("seq_lens must have one entry a row of page_table")
    return GdnPageTables(page_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), n_rows, max_pages,
                         page_table.stride(0) if n_rows > 1 else max_pages, refs.shape[0], page_size)


def _page_list(name, t, n=None):
    _need_cuda(t)
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise TypeError(f"{name} must be a contiguous int32 list" + ("" if n is None else f" of {n}"))
    return t.shape[0]


def _page_pools(pools, n_pages):
    """The pools as the library takes them; each page must be one contiguous block of its pool."""
    pools = tuple(pools)
    if len(pools) > GDN_MAX_POOLS:
        raise ValueError(f"at most {GDN_MAX_POOLS} pools")
    page_bytes = stride = 0
    for t in pools:
        _need_cuda(t)
        if t.dim() < 2 or t.shape[0] != n_pages:
            raise ValueError("a pool must be [n_pages, ...]")
        span = 1 + sum((n - 1) * s for n, s in zip(t.shape[1:], t.stride()[1:]))
        n = t.numel() // n_pages if n_pages else 0
        if n_pages and span != n:
            raise ValueError("a pool's pages must each be contiguous")
        b, s = n * t.element_size(), (t.stride(0) if n_pages > 1 else n) * t.element_size()
        if page_bytes and (b, s) != (page_bytes, stride):
            raise ValueError("the pools' pages must have one size and stride")
        page_bytes, stride = b, s
    arr = (ctypes.c_void_p * max(1, len(pools)))(*[t.data_ptr() for t in pools])
    return GdnPagePools(arr, len(pools), page_bytes, stride)


def _pages_workspace(tables, t, workspace, stream):
    if workspace is not None:
        return workspace, _handle(t, stream)
    return _own_workspace("pages", gdn_pages_workspace_bytes(tables.n_pages, tables.n_rows), t, stream)


def gdn_pages_grow(page_table, seq_lens, refs, seqs, new_lens, page_size, workspace=None, stream=None):
    """Sequences `seqs` grow to `new_lens` tokens (device int32 lists): missing pages come from the free
    ones in rising order.  Nothing changes (GDN_ERR_PAGES in the workspace's status) if they do not suffice."""
    t = _page_tables(page_table, seq_lens, refs, page_size)
    n = _page_list("seqs", seqs)
    _page_list("new_lens", new_lens, n)
    ws, handle = _pages_workspace(t, page_table, workspace, stream)
    _check(load().gdn_pages_grow(ctypes.byref(t), seqs.data_ptr(), new_lens.data_ptr(), n, ws.ptr(), ws.nbytes,
                                 handle), "gdn_pages_grow")


def gdn_pages_free(page_table, seq_lens, refs, seqs, page_size, workspace=None, stream=None):
    """Sequences `seqs` give their pages back and become empty."""
    t = _page_tables(page_table, seq_lens, refs, page_size)
    n = _page_list("seqs", seqs)
    ws, handle = _pages_workspace(t, page_table, workspace, stream)
    _check(load().gdn_pages_free(ctypes.byref(t), seqs.data_ptr(), n, ws.ptr(), ws.nbytes, handle),
           "gdn_pages_free")


def gdn_pages_fork(page_table, seq_lens, refs, parents, children, pools, page_size, workspace=None, stream=None):
    """The empty rows `children` become copies of the rows `parents`: full pages shared, a part-filled last
    page copied in every pool ([n_pages, ...] tensors: the k and v caches of every layer)."""
    t = _page_tables(page_table, seq_lens, refs, page_size)
    n = _page_list("parents", parents)
    _page_list("children", children, n)
    p = _page_pools(pools, refs.shape[0])
    ws, handle = _pages_workspace(t, page_table, workspace, stream)
    _check(load().gdn_pages_fork(ctypes.byref(t), parents.data_ptr(), children.data_ptr(), n, ctypes.byref(p),
                                 ws.ptr(), ws.nbytes, handle), "gdn_pages_fork")


def gdn_pages_compact(page_table, seq_lens, refs, pools, page_size, workspace=None, stream=None):
    """The live pages come together at the start of the pools; tables and refs follow."""
    t = _page_tables(page_table, seq_lens, refs, page_size)
    p = _page_pools(pools, refs.shape[0])
    ws, handle = _pages_workspace(t, page_table, workspace, stream)
    _check(load().gdn_pages_compact(ctypes.byref(t), ctypes.byref(p), ws.ptr(), ws.nbytes, handle),
           "gdn_pages_compact")


def gdn_pages_copy(pools, src, dst, workspace=None, stream=None):
    """Page src[i] over page dst[i] in every pool (device int32 lists; no page in both, none twice in dst)."""
    pools = tuple(pools)
    n = _page_list("src", src)
    _page_list("dst", dst, n)
    n_pages = pools[0].shape[0] if pools else 0
    p = _page_pools(pools, n_pages)
    ws, handle = ((workspace, _handle(src, stream)) if workspace is not None
                  else _own_workspace("pages", 256, src, stream))
    _check(load().gdn_pages_copy(src.data_ptr(), dst.data_ptr(), n, n_pages, ctypes.byref(p), ws.ptr(), ws.nbytes,
                                 handle), "gdn_pages_copy")
