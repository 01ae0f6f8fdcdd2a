"""Full attention over a paged cache: rotary positions, appending new tokens, attention of
them over the cache, and the bookkeeping of its pages.  Argument marshalling only, as in the
package's __init__; the functions are reached through the package.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import struct

import torch

from . import build as _build
from . import (GDN_FLAG_ROPE_BACKWARD, GDN_FLAG_ROPE_INTERLEAVED, GDN_FLAG_SIMT, GDN_FLAG_TEST_NO_WAIT,
               GDN_MAX_POOLS, GDN_ROPE_SCALING, GdnCacheShape, GdnPagePools, GdnPageTables, _check, _dtype_code,
               _need_cuda, _ptr, _stream, load)


def _load_marshal():
    """lays, like and pack of the C++ module, and itself; the three in Python where there is none for this torch."""
    if os.path.exists(_build.MARSHAL):
        try:
            spec = importlib.util.spec_from_file_location("gdn_marshal", _build.MARSHAL)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            if module.torch_version == torch.__version__.split("+")[0]:
                return module.lays, module.like, module.pack, module
        except (ImportError, AttributeError):  # another torch's, or an older build's
            pass

    def lays(*tensors):
        return tuple(None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors)

    def like(t, dims, f32):
        return torch.empty(t.shape[:dims], dtype=torch.float32 if f32 else t.dtype, device=t.device)

    def pack(tail, *pointers):
        at = [p.data_ptr() if isinstance(p, torch.Tensor) else ctypes.cast(p, ctypes.c_void_p).value or 0
              for p in pointers]
        return struct.pack(f"{len(at)}P", *at) + tail

    return lays, like, pack, None


_lays, _like, _pack, _marshal = _load_marshal()

# What a call's layouts come to (sizes, strides, flags, the workspace's size), worked out and
# checked once for each combination of shapes, strides, dtypes and devices; addresses are never
# part of it.
_plans = {}


def _plan(key, make):
    plan = _plans.get(key)
    if plan is None:
        plan = make()
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = plan
    return plan


_entries = {}
_TAKE_SCRATCH = ("gdn_paged_attn", "gdn_pages_grow", "gdn_pages_fork", "gdn_pages_compact")


def _entry(name):
    """The library's function of this name, taking tensors, bytes, addresses or None for pointers.  Those that take
    scratch get it from the allocator where their workspace is None: memory of the current stream for this call alone,
    for calls of several threads enqueue their kernels between each other's, and a captured graph goes on using what it
    was captured with."""
    f = _entries.get(name)
    if f is None:
        fn = getattr(load(), name)
        if _marshal is not None:
            f = functools.partial(getattr(_marshal, name), ctypes.cast(fn, ctypes.c_void_p).value)
        else:
            def f(*args):
                if args[-3] is None and name in _TAKE_SCRATCH:
                    scratch = torch.empty(max(256, args[-2]), dtype=torch.uint8, device="cuda")
                    args = (*args[:-3], scratch, scratch.numel(), args[-1])
                return fn(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args])
        _entries[name] = f
    return f


def _handle(t, stream):
    """The stream of a call on t's device, as an integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return _stream(t, stream).value or 0


def _empty(t, dims, f32, stream):
    """An output of a call on `stream`: memory of that stream, so that its earlier users are done."""
    if stream is None:
        return _like(t, dims, f32)
    with torch.cuda.stream(_as_stream(t, stream)):
        return _like(t, dims, f32)


def _as_stream(like, stream):
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=like.device)


_words = {}


def _status_words(index):
    """Address of the library's 256 bytes on a device: the status word of its calls without a workspace."""
    at = _words.get(index)
    if at is None:
        out = ctypes.c_void_p()
        with torch.cuda.device(index):
            _check(load().gdn_status_words(ctypes.byref(out)), "gdn_status_words")
        at = _words[index] = out.value
    return at


def _device_words(device, stream):
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    if stream is None:
        stream = torch.cuda.current_stream(index)
    return ctypes.c_void_p(_status_words(index)), ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def gdn_paged_status(device="cuda", stream=None) -> int:
    """The status of a device's gdn_kv_append, gdn_paged_attn and gdn_pages_* calls without a workspace (those with
    one leave theirs in it): GDN_OK, or the first error that one of them found on the GPU since the last
    gdn_paged_status_reset: GDN_ERR_PAGES (a grow or fork was refused), GDN_ERR_BOUNDS, GDN_ERR_TIMEOUT.
    Synchronises `stream` (default: the current one)."""
    words, stream = _device_words(device, stream)
    out = ctypes.c_int32(0)
    _check(load().gdn_workspace_status(words, ctypes.byref(out), stream), "gdn_workspace_status")
    return out.value


def gdn_paged_status_reset(device="cuda", stream=None):
    """gdn_paged_status is GDN_OK again once `stream` comes to here."""
    words, stream = _device_words(device, stream)
    _check(load().gdn_workspace_reset(words, 256, stream), "gdn_workspace_reset")


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
    return _row_stride(name, n, s[0], h * d)


def _row_stride(name, n, stride, row):
    """Stride of n rows of `row` elements as the library takes it, where 0 would mean dense: a broadcast
    tensor (stride 0) or one whose rows overlap is refused."""
    if n > 1 and stride < row:
        raise ValueError(f"{name}: rows overlap (a broadcast tensor?): use .contiguous()")
    return stride if n > 1 else row


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
    Returns (q_out, k_out), with gradients where q or k has them (then without q_out and k_out)."""
    x = q if q is not None else k
    if ((q is not None and q.requires_grad) or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out take no gradients: leave them out, or call under torch.no_grad()")
        if stream is None:
            return _Rope.apply(q, k, positions, freqs, interleaved, scale, backward)
        with torch.cuda.stream(_as_stream(x, stream)):  # the gradients then come on that stream too
            return _Rope.apply(q, k, positions, freqs, interleaved, scale, backward)

    def make():
        _need_cuda(q, k, positions, freqs, q_out, k_out)
        n_tok, _, D = x.shape
        if positions.dtype != torch.int64 or positions.numel() != n_tok or not positions.is_contiguous():
            raise TypeError("positions must be contiguous int64 [n_tok]")
        sides = []
        for name, t, out in (("q", q, q_out), ("k", k, k_out)):
            if t is None:
                sides.append((0, 0, 0))
                continue
            if t.shape[0] != n_tok or t.dtype != x.dtype:
                raise ValueError("q and k must have the same tokens and dtype")
            if out is not None and (out.shape != t.shape or out.dtype != t.dtype):
                raise ValueError(f"{name}_out must have {name}'s shape and dtype")
            sides.append((t.shape[1], _heads(name, t, D), 0 if out is None else _heads(name + "_out", out, D)))
        (hq, qs, qos), (hk, ks, kos) = sides
        return _dtype_code(x.dtype), n_tok, hq, hk, D, _rotary(freqs, D), qs, ks, qos, kos

    plan = _plan(("rope", _lays(q, k, positions, freqs, q_out, k_out)), make)
    if q_out is None and q is not None:
        q_out = _empty(q, 3, False, stream)
    if k_out is None and k is not None:
        k_out = _empty(k, 3, False, stream)
    flags = (GDN_FLAG_ROPE_INTERLEAVED if interleaved else 0) | (GDN_FLAG_ROPE_BACKWARD if backward else 0)
    st = _entry("gdn_rope")(q, k, positions, freqs, *plan, scale, flags, q_out, k_out, _handle(x, stream))
    if st:
        _check(st, "gdn_rope")
    return q_out, k_out


class _Rope(torch.autograd.Function):
    """gdn_rope with its gradient: the transposed rotation of the outputs' gradients."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, interleaved, scale, backward):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions, freqs)
        ctx.how = interleaved, scale, not backward
        return gdn_rope(q, k, positions, freqs, interleaved, scale, backward)

    @staticmethod
    def backward(ctx, dq, dk):
        dq, dk = (t.contiguous() if t is not None and need else None for t, need in zip((dq, dk), ctx.needs_input_grad))
        if dq is not None or dk is not None:
            dq, dk = gdn_rope(dq, dk, *ctx.saved_tensors, *ctx.how)
        return dq, dk, None, None, None, None, None


def cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, k=None, v=None) -> GdnCacheShape:
    """Shape of a paged call: q [n_tok, Hq, D] (or None), caches [n_pages, page_size, Hkv, D] (any order of
    pages, slots and heads in memory; D contiguous), page_table int32 [n_seqs, max_pages], seq_lens
    int32 [n_seqs], cu_seqlens int32 [n_seqs + 1] or None, new k, v [n_tok, Hkv, D]."""
    x = q if q is not None else k
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must be [n_pages, page_size, Hkv, D] with the same strides")
    n_pages, page_size, Hkv, D = k_cache.shape
    if D > 1 and k_cache.stride(3) != 1:
        raise ValueError("the caches' last dimension must be contiguous")
    if any(n > 1 and s < D for n, s in zip(k_cache.shape[:3], k_cache.stride()[:3])):
        raise ValueError("the caches' pages, slots and heads must not overlap")
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
    return GdnCacheShape(n_seqs, n_tok, Hq, Hkv, D, _dtype_code(x.dtype), page_size, n_pages, max_pages,
                         _row_stride("page_table", n_seqs, page_table.stride(0), max_pages), st[0], st[1], st[2],
                         0 if q is None else _heads("q", q, D), 0 if k is None else _heads("k", k, D),
                         0 if v is None else _heads("v", v, D))


def _call(name, t, nbytes, workspace, stream, *args):
    """A library call with a workspace or with scratch of its own: its arguments up to that."""
    buf = None
    if workspace is not None:
        buf, nbytes = workspace.buf, workspace.nbytes
    if stream is None:
        st = _entry(name)(*args, buf, nbytes, _handle(t, None))
    else:
        with torch.cuda.stream(_as_stream(t, stream)):
            st = _entry(name)(*args, buf, nbytes, _handle(t, stream))
    if st:
        _check(st, name)


def gdn_kv_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, q=None, freqs=None,
                  positions=None, interleaved=False, scale=1.0, q_out=None, workspace=None, stream=None):
    """The new tokens' k, v [n_tok, Hkv, D] into the cache at the end of their sequences (seq_lens counts
    them already), k rotated on the way with freqs, and q [n_tok, Hq, D] rotated into q_out (a new
    tensor, or q itself).  positions int64 [n_tok] replaces the places in the sequences as rotary
    positions.  Returns q_out (None without q), without gradients."""

    def make():
        _need_cuda(q, k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens, freqs, positions, q_out)
        sh = cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, k, v)
        if positions is not None and (positions.dtype != torch.int64 or positions.shape != (sh.n_tok,)
                                      or not positions.is_contiguous()):
            raise TypeError("positions must be contiguous int64 [n_tok]")
        if q_out is not None and (q is None or q_out.shape != q.shape or q_out.dtype != q.dtype
                                  or not q_out.is_contiguous()):
            raise ValueError("q_out must be contiguous with q's shape and dtype")
        return sh, ctypes.addressof(sh), _rotary(freqs, sh.D)

    _, shape, rd = _plan(("append", _lays(q, k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens, freqs, positions,
                                          q_out)), make)
    if q is not None and q_out is None:
        q_out = _empty(q, 3, False, stream)
    buf, nbytes = (workspace.buf, workspace.nbytes) if workspace is not None else (_status_words(k.get_device()), 256)
    st = _entry("gdn_kv_append")(q, k, v, positions, freqs, rd, scale, GDN_FLAG_ROPE_INTERLEAVED if interleaved else 0,
                                 page_table, seq_lens, cu_seqlens, shape, q_out, k_cache, v_cache, buf, nbytes,
                                 _handle(k, stream))
    if st:
        _check(st, "gdn_kv_append")
    return q_out


def gdn_paged_attn_workspace_bytes(shape: GdnCacheShape, max_new: int) -> int:
    return int(load().gdn_paged_attn_workspace_bytes(ctypes.byref(shape), int(max_new)))


def gdn_paged_attn(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, max_new=None, scale=None, window=0,
                   want_lse=False, o=None, lse=None, simt=False, workspace=None, stream=None, _test_no_wait=False):
    """Attention of the new tokens q [n_tok, Hq, D] over the paged cache, which holds their k and v already:
    the token at position p of its sequence sees the last `window` positions up to p (0: all).
    max_new: a bound on the new tokens of one sequence (default: all of them).  Returns
    (o [n_tok, Hq, D], lse [n_tok, Hq] fp32 or None), without gradients."""

    def make():
        _need_cuda(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, o, lse)
        sh = cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens)
        if o is not None and (o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous()):
            raise ValueError("o must be contiguous with q's shape and dtype")
        if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()):
            raise ValueError("lse must be contiguous fp32 [n_tok, Hq]")
        new = max_new if max_new is not None else sh.n_tok if cu_seqlens is not None else 1
        if workspace is None:
            sh.status = _status_words(q.get_device())
        return sh, ctypes.addressof(sh), new, gdn_paged_attn_workspace_bytes(sh, new), sh.D ** -0.5

    _, shape, new, nbytes, unit = _plan(
        ("attn", max_new, workspace is None,
         _lays(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, o, lse)), make)
    if o is None:
        o = _empty(q, 3, False, stream)
    if lse is None and want_lse:
        lse = _empty(q, 2, True, stream)
    flags = (GDN_FLAG_SIMT if simt else 0) | (GDN_FLAG_TEST_NO_WAIT if _test_no_wait else 0)
    _call("gdn_paged_attn", q, nbytes, workspace, stream, q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, shape,
          new, unit if scale is None else scale, window, flags, o, lse)
    return o, lse


def gdn_pages_workspace_bytes(n_pages: int, n_rows: int) -> int:
    return int(load().gdn_pages_workspace_bytes(int(n_pages), int(n_rows)))


def _page_list(name, t, n=None):
    _need_cuda(t)
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise TypeError(f"{name} must be a contiguous int32 list" + ("" if n is None else f" of {n}"))
    return t.shape[0]


def _page_tables(page_table, seq_lens, refs, page_size, workspace, names=(), *lists):
    """The tables as the library takes them, the length of the lists of rows, and a workspace's size."""
    def make():
        _need_cuda(page_table, seq_lens, refs)
        for name, t, dims in (("page_table", page_table, 2), ("seq_lens", seq_lens, 1), ("refs", refs, 1)):
            if t.dtype != torch.int32 or t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise TypeError(f"{name} must be int32 with contiguous rows")
        n_rows, max_pages = page_table.shape
        if seq_lens.shape[0] != n_rows:
            raise ValueError("seq_lens must have one entry a row of page_table")
        n_pages, n = refs.shape[0], None
        for name, t in zip(names, lists):
            n = _page_list(name, t, n)
        t = GdnPageTables(None, None, None, n_rows, max_pages,
                          _row_stride("page_table", n_rows, page_table.stride(0), max_pages), n_pages, page_size,
                          None if workspace is not None else _status_words(page_table.get_device()))
        return bytes(t)[3 * ctypes.sizeof(ctypes.c_void_p):], n, gdn_pages_workspace_bytes(n_pages, n_rows)

    tail, n, nbytes = _plan(
        ("tables", page_size, names, workspace is None, _lays(page_table, seq_lens, refs, *lists)), make)
    return _pack(tail, page_table, seq_lens, refs), n, nbytes


def _page_pools(pools, n_pages):
    """The pools as the library takes them, and what that points to; a page must be one contiguous block of its pool."""
    pools = tuple(pools)
    if len(pools) > GDN_MAX_POOLS:
        raise ValueError(f"at most {GDN_MAX_POOLS} pools")

    def make():
        _need_cuda(*pools)
        page_bytes = stride = 0
        for t in pools:
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
        return bytes(GdnPagePools(None, len(pools), page_bytes, stride))[ctypes.sizeof(ctypes.c_void_p):]

    tail = _plan(("pools", n_pages, _lays(*pools)), make)
    at = _pack(b"", *pools)
    return _pack(tail, at), at


def gdn_pages_grow(page_table, seq_lens, refs, seqs, new_lens, page_size, workspace=None, stream=None):
    """Sequences `seqs` grow to `new_lens` tokens (device int32 lists): missing pages come from the free
    ones in rising order.  Nothing changes, the lengths included, if they do not suffice: GDN_ERR_PAGES in
    the status of the workspace, or of gdn_paged_status without one."""
    t, n, nbytes = _page_tables(page_table, seq_lens, refs, page_size, workspace, ("seqs", "new_lens"), seqs, new_lens)
    _call("gdn_pages_grow", page_table, nbytes, workspace, stream, t, seqs, new_lens, n)


def gdn_pages_free(page_table, seq_lens, refs, seqs, page_size, workspace=None, stream=None):
    """Sequences `seqs` give their pages back and become empty."""
    t, n, nbytes = _page_tables(page_table, seq_lens, refs, page_size, workspace, ("seqs",), seqs)
    _call("gdn_pages_free", page_table, nbytes, workspace, stream, t, seqs, n)


def gdn_pages_fork(page_table, seq_lens, refs, parents, children, pools, page_size, workspace=None, stream=None):
    """The empty rows `children` become copies of the rows `parents`: full pages shared, a part-filled last
    page copied in every pool ([n_pages, ...] tensors: the k and v caches of every layer).  Nothing changes
    if the lists cannot be carried out or the free pages do not suffice: GDN_ERR_PAGES, as for gdn_pages_grow."""
    t, n, nbytes = _page_tables(page_table, seq_lens, refs, page_size, workspace, ("parents", "children"), parents,
                                children)
    p, _keep = _page_pools(pools, refs.shape[0])
    _call("gdn_pages_fork", page_table, nbytes, workspace, stream, t, parents, children, n, p)


def gdn_pages_compact(page_table, seq_lens, refs, pools, page_size, workspace=None, stream=None):
    """The live pages come together at the start of the pools; tables and refs follow."""
    t, _, nbytes = _page_tables(page_table, seq_lens, refs, page_size, workspace)
    p, _keep = _page_pools(pools, refs.shape[0])
    _call("gdn_pages_compact", page_table, nbytes, workspace, stream, t, p)


def gdn_pages_copy(pools, src, dst, workspace=None, stream=None):
    """Page src[i] over page dst[i] in every pool (device int32 lists; no page in both, none twice in dst)."""
    pools = tuple(pools)
    n = _page_list("src", src)
    _page_list("dst", dst, n)
    n_pages = pools[0].shape[0] if pools else 0
    p, _keep = _page_pools(pools, n_pages)
    buf, nbytes = (workspace.buf, workspace.nbytes) if workspace is not None else (_status_words(src.get_device()), 256)
    st = _entry("gdn_pages_copy")(src, dst, n, n_pages, p, buf, nbytes, _handle(src, stream))
    if st:
        _check(st, "gdn_pages_copy")
