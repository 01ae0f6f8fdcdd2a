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
               GDN_MAX_POOLS, GDN_ROPE_SCALING, GdnCacheShape, GdnPageHeads, GdnPagePools, GdnPageTables, _check,
               _dtype_code, _need_cuda, _ptr, _stream, load)


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
_TAKE_SCRATCH = ("gdn_paged_attn", "gdn_paged_attn_shared", "gdn_paged_mass", "gdn_pages_grow", "gdn_pages_fork",
                 "gdn_pages_compact", "gdn_pages_evict")


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
    """The status of a device's gdn_kv_append, gdn_paged_attn, gdn_paged_attn_shared, gdn_paged_mass and gdn_pages_* calls
    without a workspace (those with one leave theirs in it): GDN_OK, or the first error that one of them found on the GPU
    since the last gdn_paged_status_reset: GDN_ERR_PAGES (a grow, fork or eviction was refused), GDN_ERR_BOUNDS,
    GDN_ERR_TIMEOUT.
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


def _groups(group_offsets, prefix_lens):
    _need_cuda(group_offsets, prefix_lens)
    for name, t in (("group_offsets", group_offsets), ("prefix_lens", prefix_lens)):
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
            raise TypeError(f"{name} must be contiguous int32")
    if group_offsets.shape[0] != prefix_lens.shape[0] + 1:
        raise ValueError("group_offsets must have one entry more than prefix_lens")
    return prefix_lens.shape[0]


def gdn_paged_attn_shared_workspace_bytes(shape: GdnCacheShape, n_groups: int, max_group_new: int) -> int:
    return int(load().gdn_paged_attn_shared_workspace_bytes(ctypes.byref(shape), int(n_groups), int(max_group_new)))


def gdn_paged_attn_shared(q, k_cache, v_cache, page_table, seq_lens, group_offsets, prefix_lens, cu_seqlens=None,
                          max_group_new=None, scale=None, want_lse=False, o=None, lse=None, simt=False, workspace=None,
                          stream=None, _test_no_wait=False):
    """gdn_paged_attn where groups of sequences share a prefix: sequences group_offsets[g] .. group_offsets[g + 1] - 1 hold
    the same tokens in their first prefix_lens[g] positions (device int32 [n_groups + 1], from 0 to n_seqs, and
    [n_groups]), which are read once for the group, from its first sequence's pages.  max_group_new: a bound on
    the new tokens of one group (default: all of them).  Returns (o, lse or None) as gdn_paged_attn, without gradients.
    For few sequences, short prefixes and long chunks gdn_paged_attn is the faster one; include/gdn.h has the figures."""

    def make():
        _need_cuda(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens, o, lse)
        n_groups = _groups(group_offsets, prefix_lens)
        sh = cache_shape(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens)
        if o is not None and (o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous()):
            raise ValueError("o must be contiguous with q's shape and dtype")
        if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()):
            raise ValueError("lse must be contiguous fp32 [n_tok, Hq]")
        new = sh.n_tok if max_group_new is None else max_group_new
        if workspace is None:
            sh.status = _status_words(q.get_device())
        return sh, ctypes.addressof(sh), n_groups, new, gdn_paged_attn_shared_workspace_bytes(sh, n_groups, new), sh.D ** -0.5

    _, shape, n_groups, new, nbytes, unit = _plan(
        ("shared", max_group_new, workspace is None,
         _lays(q, k_cache, v_cache, page_table, seq_lens, group_offsets, prefix_lens, cu_seqlens, o, lse)), make)
    if o is None:
        o = _empty(q, 3, False, stream)
    if lse is None and want_lse:
        lse = _empty(q, 2, True, stream)
    flags = (GDN_FLAG_SIMT if simt else 0) | (GDN_FLAG_TEST_NO_WAIT if _test_no_wait else 0)
    _call("gdn_paged_attn_shared", q, nbytes, workspace, stream, q, k_cache, v_cache, page_table, seq_lens, cu_seqlens,
          group_offsets, prefix_lens, n_groups, shape, new, unit if scale is None else scale, flags, o, lse)
    return o, lse


def gdn_paged_mass_workspace_bytes(shape: GdnCacheShape) -> int:
    return int(load().gdn_paged_mass_workspace_bytes(ctypes.byref(shape)))


def gdn_paged_mass(q, k_cache, page_table, seq_lens, lse, mass, cu_seqlens=None, max_new=None, scale=None, window=0,
                   accumulate=True, simt=False, workspace=None, stream=None, _test_no_wait=False):
    """The softmax weight that each cached position gets from the new tokens q [n_tok, Hq, D] whose attention left lse
    [n_tok, Hq] (fp32), summed over them and the heads of a kv head's group: added to mass [n_seqs, Hkv, length] (fp32,
    contiguous rows), or with accumulate=False written over it, up to each sequence's length.  Other arguments as for
    gdn_paged_attn.  Returns mass, without gradients."""

    def make():
        _need_cuda(q, k_cache, page_table, seq_lens, cu_seqlens, lse, mass)
        sh = cache_shape(q, k_cache, k_cache, page_table, seq_lens, cu_seqlens)
        if lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError("lse must be contiguous fp32 [n_tok, Hq]")
        if mass.dtype != torch.float32 or mass.dim() != 3 or (mass.shape[2] > 1 and mass.stride(2) != 1):
            raise TypeError("mass must be fp32 [n_seqs, Hkv, length] with contiguous rows")
        if mass.shape[:2] != (sh.n_seqs, sh.Hkv):
            raise ValueError("mass must have a row a sequence and kv head")
        length = mass.shape[2]
        st = [length if n == 1 else s for n, s in zip(mass.shape, mass.stride()[:2])]
        if any(s < length for s in st):
            raise ValueError("mass's rows overlap (a broadcast tensor?): use .contiguous()")
        new = max_new if max_new is not None else sh.n_tok if cu_seqlens is not None else 1
        if workspace is None:
            sh.status = _status_words(q.get_device())
        return sh, ctypes.addressof(sh), new, (*st, length), gdn_paged_mass_workspace_bytes(sh), sh.D ** -0.5

    _, shape, new, rows, nbytes, unit = _plan(
        ("mass", max_new, workspace is None,
         _lays(q, k_cache, page_table, seq_lens, lse, mass, cu_seqlens)), make)
    flags = (GDN_FLAG_SIMT if simt else 0) | (GDN_FLAG_TEST_NO_WAIT if _test_no_wait else 0)
    _call("gdn_paged_mass", q, nbytes, workspace, stream, q, k_cache, page_table, seq_lens, cu_seqlens, lse, shape, new,
          unit if scale is None else scale, window, 1 if accumulate else 0, flags, mass, *rows)
    return mass


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


def gdn_pages_evict_workspace_bytes(n_pages: int, n_rows: int, max_pages: int, n: int, max_keep: int, n_layers: int,
                                    heads: int) -> int:
    t = GdnPageTables(n_rows=int(n_rows), max_pages=int(max_pages), n_pages=int(n_pages))
    return int(load().gdn_pages_evict_workspace_bytes(ctypes.byref(t), int(n), int(max_keep), int(n_layers), int(heads)))


def gdn_pages_evict(page_table, seq_lens, refs, seqs, keep, mass, pools, page_size, max_keep, recent=0, want_kept=False,
                    workspace=None, stream=None):
    """Sequences `seqs` are cut to `keep` tokens (device int32 lists, at most max_keep) where they have more: in each layer
    and for each kv head the last `recent` positions stay and those of the others with the largest mass (fp32
    [n_layers, n_rows, heads, length]; ties to the lowest position), moved in their order to fresh pages.
    pools: each layer's [n_pages, page_size, heads, D] caches in turn (k0, v0, k1, v1, ...).  Masses move along, the tables
    follow.  Returns the positions that stayed, int32 [n_layers, n, heads, max_keep] filled up with -1, or None without
    want_kept.  Nothing changes, and nothing is returned that means anything, if a list cannot be carried out (pages held more
    often than refs says among the reasons) or the free pages do not suffice, ceil(keep / page_size) for each sequence that is
    cut, before its old ones are given back: GDN_ERR_PAGES, as for gdn_pages_grow."""
    pools = tuple(pools)
    t, n, _ = _page_tables(page_table, seq_lens, refs, page_size, workspace, ("seqs", "keep"), seqs, keep)
    p, _keep = _page_pools(pools, refs.shape[0])

    def make():
        _need_cuda(mass)
        if mass.dtype != torch.float32 or mass.dim() != 4 or (mass.shape[3] > 1 and mass.stride(3) != 1):
            raise TypeError("mass must be fp32 [n_layers, n_rows, heads, length] with contiguous rows")
        n_layers, n_rows, heads, length = mass.shape
        if n_rows != page_table.shape[0]:
            raise ValueError("mass must have one row a row of page_table")
        if n_layers == 0 or len(pools) % n_layers:
            raise ValueError("the pools must be as many for each of mass's layers")
        st = [max(s, length) if k == 1 else s for s, k in zip(mass.stride()[:3], mass.shape[:3])]
        if any(s < length for s in st):
            raise ValueError("mass's rows overlap (a broadcast tensor?): use .contiguous()")
        row_bytes = slot = head = 1
        if pools:
            x = pools[0]
            if any(c.dim() != 4 or c.shape[1:3] != (page_size, heads) or c.shape[3] != x.shape[3] or c.dtype != x.dtype
                   or (c.shape[3] > 1 and c.stride(3) != 1) or c.stride()[1:3] != x.stride()[1:3] for c in pools):
                raise ValueError("the pools must be [n_pages, page_size, heads, D] with the same strides")
            row_bytes = x.shape[3] * x.element_size()
            slot, head = (s * x.element_size() for s in x.stride()[1:3])
            slot, head = slot if page_size > 1 else row_bytes, head if heads > 1 else row_bytes
        tail = bytes(GdnPageHeads(None, n_layers, heads, length, *st, row_bytes, slot, head))
        nbytes = gdn_pages_evict_workspace_bytes(refs.shape[0], n_rows, page_table.shape[1], n, max_keep, n_layers, heads)
        return tail[ctypes.sizeof(ctypes.c_void_p):], (n_layers, n, heads, max_keep), nbytes

    tail, shape, nbytes = _plan(("evict", page_size, max_keep, _lays(page_table, refs, seqs, mass), _lays(*pools)), make)
    kept = None
    if want_kept:
        if stream is None:
            kept = torch.empty(shape, dtype=torch.int32, device=mass.device)
        else:
            with torch.cuda.stream(_as_stream(mass, stream)):
                kept = torch.empty(shape, dtype=torch.int32, device=mass.device)
    _call("gdn_pages_evict", page_table, nbytes, workspace, stream, t, seqs, keep, n, max_keep, recent,
          _pack(tail, mass), p, kept)
    return kept
