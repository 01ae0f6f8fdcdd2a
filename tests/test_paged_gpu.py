"""GPU parity of the full-attention operators (rotary positions, append, attention over a paged cache, pages)
against plain 64-bit implementations.

Tolerances count roundings.  A stored bf16 is off by at most 2^-8 of its value, fp32 by 2^-24.
Attention: with A = softmax @ |v| an output may be off by
    u_out |o| + (u_P + 4 ds + n 2^-23) A,     ds = (D + 8) 2^-24 c max_j sum_d |q_d k_jd| + 2^-20,
u_P = 2^-8 where the weights are rounded to bf16 for the tensor cores, else 0; ds is the error of a
score (a sum of D products, and the exponent's argument and base-2 exponential), n the keys summed.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def crg():
    import chunked_recurrence_gb300 as m
    m.load()
    return m


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(TYPES[dtype])


# ------------------------------------------------------------------- rotary

def rope_ref(x, pos, inv, rd, inter, scale, sign):
    y = x.copy()
    a = pos[:, None, None].astype(np.float64) * inv
    c, s = scale * np.cos(a), scale * sign * np.sin(a)
    i1, i2 = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, rd // 2), slice(rd // 2, rd))
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    size = np.zeros_like(x)
    size[..., i1] = size[..., i2] = scale * (np.abs(x1) + np.abs(x2))
    return y, size


def assert_rope(got, x, pos, inv, rd, inter, scale=1.0, sign=1.0):
    """Angle to 2^-25 turns and sincospi to two ulps: 2^-21 of |x1| + |x2|, and the stored rounding."""
    ref, size = rope_ref(f64(x), pos, inv, rd, inter, scale, sign)
    off = np.abs(f64(got) - ref)
    assert np.all(off <= HALF[got.dtype] * np.abs(ref) + 2.0 ** -21 * size), off.max()
    assert torch.equal(got[..., rd:], x[..., rd:])


ROPE = [  # dtype, n_tok, Hq, Hk, D, rotary_dim, interleaved
    ("bf16", 1, 4, 1, 128, 128, False), ("bf16", 1300, 3, 1, 128, 128, True), ("bf16", 37, 5, 0, 256, 64, False),
    ("bf16", 37, 2, 3, 256, 64, True), ("f32", 33, 0, 3, 64, 64, False), ("f32", 33, 2, 2, 64, 32, True),
    ("bf16", 19, 2, 1, 80, 40, False), ("f32", 19, 2, 1, 10, 6, True), ("f32", 5, 1, 1, 7, 2, False),
    ("bf16", 1217, 1, 1, 64, 0, False), ("bf16", 9, 33, 2, 96, 96, False),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(crg, case, backward):
    dtype, n, hq, hk, d, rd, inter = case
    g = gen(n + d + rd)
    q, k = (randn(g, (n, h, d), dtype) if h else None for h in (hq, hk))
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV)
    pos[0] = 0
    inv = crg.gdn_rope_inv_freq(rd, scaling="parts", factor=4.0, orig_len=4096) if rd else torch.zeros(0).double()
    qo, ko = crg.gdn_rope(q, k, pos, crg.gdn_rope_freqs(inv, DEV), inter, 1.25, backward)
    torch.cuda.synchronize()
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            assert y is None
        else:
            assert_rope(y, x, pos.cpu().numpy(), inv.numpy(), rd, inter, 1.25, -1.0 if backward else 1.0)


def test_rope_far_and_negative_positions(crg):
    """The angle is exact at any 64-bit position: turns by exact integer arithmetic in Python."""
    inv = crg.gdn_rope_inv_freq(64)
    table = crg.gdn_rope_freqs(inv, DEV)
    pos = torch.tensor([2 ** 31, -7, 2 ** 40 + 3, -(2 ** 62), 2 ** 63 - 1], device=DEV)
    q = torch.ones((5, 1, 64), device=DEV)
    out, _ = crg.gdn_rope(q, None, pos, table)
    for t, p in enumerate(pos.tolist()):
        for i, w in enumerate(table.tolist()):
            a = 2 * math.pi * (((p * w) % 2 ** 64) / 2 ** 64)
            assert abs(out[t, 0, i].item() - (math.cos(a) - math.sin(a))) <= 2.0 ** -20
            assert abs(out[t, 0, 32 + i].item() - (math.cos(a) + math.sin(a))) <= 2.0 ** -20


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(crg, inter):
    """The backward against differences: the step is linear, so (f(x + e u) - f(x - e u)) / 2e = f(u), and
    <dy, f(u)> = <backward(dy), u>."""
    g = gen(5)
    n, h, d, rd = 29, 3, 64, 48
    x, u, dy = (torch.randn((n, h, d), generator=g, device=DEV) for _ in range(3))
    pos = torch.arange(n, device=DEV) * 1000
    table = crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(rd), DEV)
    f = lambda t: f64(crg.gdn_rope(t, None, pos, table, inter, 1.1)[0])  # noqa: E731
    diff = (f(x + 0.5 * u) - f(x - 0.5 * u))
    dx = f64(crg.gdn_rope(dy, None, pos, table, inter, 1.1, backward=True)[0])
    lhs, rhs = (f64(dy) * diff).sum((1, 2)), (dx * f64(u)).sum((1, 2))
    size = np.abs(f64(dy)).sum((1, 2)) * 8  # |x|, |u| < 8
    assert np.all(np.abs(lhs - rhs) <= 2.0 ** -20 * size)


def test_rope_views_and_in_place(crg):
    """q and k as views of one projection's rows, rotated in place; the rest of the row is untouched."""
    g = gen(6)
    n, hq, hk, d = 41, 4, 2, 64
    x = randn(g, (n, (hq + 2 * hk) * d + 24), "bf16")
    before = x.clone()
    view = lambda t, h0, h: t.as_strided((n, h, d), (t.stride(0), d, 1), h0 * d)  # noqa: E731
    q, k = view(x, 0, hq), view(x, hq, hk)
    inv = crg.gdn_rope_inv_freq(d)
    pos = torch.arange(n, device=DEV)
    crg.gdn_rope(q, k, pos, crg.gdn_rope_freqs(inv, DEV), q_out=q, k_out=k)
    assert_rope(q, view(before, 0, hq), pos.cpu().numpy(), inv.numpy(), d, False)
    assert_rope(k, view(before, hq, hk), pos.cpu().numpy(), inv.numpy(), d, False)
    assert torch.equal(x[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_rope_unaligned_and_empty(crg):
    g = gen(7)
    buf = torch.zeros(20 * 3 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    q = buf[1:].view(20, 3, 64)
    q.copy_(randn(g, (20, 3, 64), "bf16"))
    inv, pos = crg.gdn_rope_inv_freq(64), torch.arange(20, device=DEV)
    out, _ = crg.gdn_rope(q, None, pos, crg.gdn_rope_freqs(inv, DEV))
    assert_rope(out, q, pos.cpu().numpy(), inv.numpy(), 64, False)
    out, _ = crg.gdn_rope(q[:0], None, pos[:0], crg.gdn_rope_freqs(inv, DEV))
    assert out.shape == (0, 3, 64)


# -------------------------------------------------------------------- cache

class Cache:
    """A cache with its sequences' pages anywhere in it, NaN wherever no sequence's token lies."""

    def __init__(self, seed, dtype, lens, hkv, d, page, order="token", gap=0, spare=3):
        g = gen(seed)
        self.page, self.lens_list = page, list(lens)
        need = [-(-m // page) for m in lens]
        n_pages = sum(need) + spare
        width = max(need + [1]) + 1
        perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            table[s, :n] = torch.tensor([perm.pop() for _ in range(n)], dtype=torch.int32)
        self.table = table.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        both = []
        for _ in range(2):
            if order == "head":  # [page][head][slot]
                t = randn(g, (n_pages, hkv, page + gap, d), dtype)[:, :, :page].permute(0, 2, 1, 3)
            else:                # [page][slot][head], pages `gap` slots apart
                t = randn(g, (n_pages, page + gap, hkv, d), dtype)[:, :page]
            both.append(t)
        self.k, self.v = both
        free = torch.ones((n_pages, page), dtype=torch.bool, device=DEV)
        for s, m in enumerate(lens):
            for i in range(need[s]):
                free[int(table[s, i]), : min(page, m - i * page)] = False
        self.k[free] = math.nan
        self.v[free] = math.nan

    def rows(self, s, t):
        """Sequence s's tokens of cache t, in order, in 64 bits [len, hkv, d]."""
        m = self.lens_list[s]
        pages = self.table[s, : -(-m // self.page)].long()
        return f64(t[pages].reshape(-1, *t.shape[2:])[:m]) if m else np.zeros((0, *t.shape[2:]))


def attn_ref(q, cache, new, window, scale):
    """(o, lse, A, ds) of every token and head, from the definition."""
    q64 = f64(q)
    n_tok, hq, d = q64.shape
    hkv = cache.k.shape[2]
    o, a = np.zeros_like(q64), np.zeros_like(q64)
    lse, ds = np.full((n_tok, hq), -np.inf), np.zeros((n_tok, hq))
    t = 0
    for s, n in enumerate(new):
        k, v = cache.rows(s, cache.k), cache.rows(s, cache.v)
        m = cache.lens_list[s]
        p = np.arange(m - n, m)
        j = np.arange(m)
        seen = (j[None] <= p[:, None]) & ((j[None] > p[:, None] - window) if window else True)
        for h in range(hq if n and m else 0):
            x = scale * (q64[t: t + n, h] @ k[:, h * hkv // hq].T)
            size = scale * (np.abs(q64[t: t + n, h]) @ np.abs(k[:, h * hkv // hq]).T)
            x = np.where(seen, x, -np.inf)
            top = np.max(x, 1, keepdims=True, initial=-1e300)
            e = np.exp(x - top)
            z = e.sum(1, keepdims=True)
            with np.errstate(divide="ignore", invalid="ignore"):
                w = np.where(z > 0, e / z, 0.0)
                lse[t: t + n, h] = np.where(z > 0, np.log(z) + top, -np.inf)[:, 0]
            o[t: t + n, h] = w @ v[:, h * hkv // hq]
            a[t: t + n, h] = w @ np.abs(v[:, h * hkv // hq])
            ds[t: t + n, h] = np.max(np.where(seen, size, 0.0), 1, initial=0.0) * (d + 8) * 2.0 ** -24 + 2.0 ** -20
        t += n
    return o, lse, a, ds


def assert_attn(o, lse, q, cache, new, window=0, scale=None, tensor=True):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    ro, rl, a, ds = attn_ref(q, cache, new, window, scale)
    n = max(cache.lens_list + [1])
    u_p = 2.0 ** -8 if tensor else 0.0
    off = np.abs(f64(o) - ro)
    tol = HALF[o.dtype] * np.abs(ro) + (u_p + 4 * ds[..., None] + n * 2.0 ** -23) * a
    assert np.all(np.isfinite(f64(o)))
    assert np.all(off <= tol), (off - tol).max()
    if lse is not None:
        g = f64(lse)
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(g), none)
        lt = 2 * ds + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(none, 0, rl))
        assert np.all(np.abs(g - rl)[~none] <= lt[~none])


def cu_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)


def run_attn(crg, seed, dtype, new, lens, hq, hkv, d, page, window=0, order="token", gap=0, simt=False, max_new=None,
             one=False, scale=None, tensor=None):
    cache = Cache(seed, dtype, lens, hkv, d, page, order, gap)
    q = randn(gen(seed + 1), (sum(new), hq, d), dtype)
    ws = crg.Workspace(1 << 28, DEV)
    o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, None if one else cu_of(new),
                                max_new=max_new, window=window, want_lse=True, simt=simt, workspace=ws, scale=scale)
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert_attn(o, lse, q, cache, new, window, scale, tensor=dtype == "bf16" and not simt if tensor is None else tensor)
    return cache, q, o, lse


SIMT = [  # dtype, new, lens, hq, hkv, d, page, window
    ("f32", [1, 1, 1], [1, 17, 300], 4, 2, 64, 16, 0),
    ("f32", [5, 0, 37], [5, 0, 90], 6, 2, 64, 16, 0),
    ("f32", [33], [200], 3, 1, 128, 1, 50),
    ("bf16", [9, 3], [40, 3], 4, 4, 96, 5, 0),
    ("bf16", [7], [33], 8, 1, 256, 16, 1),
    ("f32", [4, 2], [2, 1], 2, 1, 7, 3, 0),       # more new tokens than cached ones: rows that see nothing
    ("f32", [3], [700], 2, 1, 250, 48, 0),
]


@pytest.mark.parametrize("case", SIMT, ids=str)
def test_attn_simt(crg, case):
    run_attn(crg, 11, *case, simt=True)


F32 = [  # dtype, new, lens, hq, hkv, d, page, window: what the tcgen05 kernel does not take
    ("f32", [1, 4], [900, 65], 8, 2, 128, 16, 0),
    ("f32", [1, 1, 1], [1, 17, 3000], 4, 2, 64, 16, 0),
    ("f32", [5, 0, 37], [5, 0, 90], 6, 2, 64, 16, 0),
    ("f32", [130, 1], [200, 1], 3, 1, 128, 1, 50),
    ("f32", [90], [400], 4, 2, 256, 48, 0),
    ("f32", [1, 1], [400, 70], 5, 1, 256, 48, 33),
    ("f32", [20, 2], [7, 1], 4, 2, 96, 3, 0),      # rows that see nothing
    ("f32", [33], [70], 2, 1, 7, 5, 0),
    ("bf16", [9, 3], [40, 3], 4, 4, 96, 5, 0),
    ("bf16", [70], [133], 8, 1, 200, 12, 1),
    ("bf16", [1, 1], [1000, 64], 3, 1, 40, 16, 0),
    ("bf16", [3], [77], 130, 1, 64, 16, 0),        # more heads a group than a tile has rows
]


@pytest.mark.parametrize("case", F32, ids=str)
def test_attn_f32(crg, case):
    run_attn(crg, 12, *case, tensor=False)


TC = [  # new, lens, hq, hkv, d, page, window
    ([1], [1], 1, 1, 128, 16, 0),
    ([1, 1, 1], [1, 127, 129], 4, 2, 128, 16, 0),
    ([1, 1, 1, 1], [0, 128, 1000, 3], 8, 1, 128, 64, 0),   # a sequence without a token
    ([1, 1], [513, 77], 3, 3, 64, 8, 0),
    ([1, 1, 1], [300, 257, 64], 14, 2, 256, 32, 0),        # groups of seven
    ([13, 1, 0, 40], [13, 500, 9, 333], 4, 2, 128, 48, 0),
    ([20, 3], [7, 3], 8, 2, 128, 16, 0),                   # rows that see nothing
    ([130], [130], 1, 1, 64, 128, 0),
    ([257, 5, 1], [400, 5, 1000], 2, 1, 64, 16, 0),
    ([300], [300], 3, 1, 128, 64, 0),
    ([65, 1, 129], [700, 513, 129], 8, 2, 128, 24, 0),
    ([200, 1], [200, 900], 4, 2, 256, 64, 0),
    ([70], [1500], 5, 1, 256, 16, 0),
    ([2, 1], [5000, 4001], 8, 1, 128, 256, 0),             # one kv head split over many blocks
    ([1], [20000], 8, 1, 64, 64, 0),
    # windows
    ([1, 1, 1], [1000, 100, 129], 4, 2, 128, 16, 100),
    ([150, 9], [800, 9], 4, 2, 128, 16, 1),
    ([300, 33], [1000, 400], 2, 1, 64, 32, 129),
    ([90, 1], [900, 700], 4, 1, 256, 16, 260),
]


@pytest.mark.parametrize("case", TC, ids=str)
def test_attn_tensor_cores(crg, case):
    run_attn(crg, 13, "bf16", *case)


@pytest.mark.parametrize("order,gap", [("token", 3), ("head", 0), ("head", 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_cache_layouts(crg, d, order, gap):
    run_attn(crg, 14, "bf16", [40, 1], [150, 400], 4, 2, d, 16, order=order, gap=gap)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_new", [1, 200])
def test_attn_max_new_is_a_hint(crg, d, max_new):
    """One or two row tiles a block: both right for chunks shorter and longer than the hint."""
    run_attn(crg, 15, "bf16", [1, 90, 17], [300, 200, 17], 8, 2, d, 16, max_new=max_new)


def test_attn_one_token_each(crg):
    run_attn(crg, 16, "bf16", [1] * 37, [1 + 61 * i % 900 for i in range(37)], 8, 2, 128, 16, one=True)


def test_attn_many_sequences(crg):
    """More sequences than a block has threads."""
    new = [i % 3 for i in range(400)]
    run_attn(crg, 17, "bf16", new, [n + (7 * i) % 40 for i, n in enumerate(new)], 2, 1, 64, 8)


def test_attn_scores_far_apart(crg):
    """Scores over hundreds of e-folds, rising along the sequence, so that the running maximum moves often."""
    for scale in (3.0, 0.01):
        run_attn(crg, 18, "bf16", [150, 1], [700, 700], 4, 2, 128, 16, scale=scale)
    cache = Cache(19, "bf16", [1200], 1, 128, 16)
    q = torch.ones((260, 1, 128), dtype=torch.bfloat16, device=DEV)
    for i in range(75):
        cache.k[int(cache.table[0, i])] *= 0.02
        cache.k[int(cache.table[0, i])] += 0.002 * i
    o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([260]), want_lse=True, scale=3.0)
    assert_attn(o, lse, q, cache, [260], scale=3.0)


def test_attn_strided_q_and_given_outputs(crg):
    cache = Cache(20, "bf16", [100, 60], 2, 128, 16)
    x = randn(gen(21), (24, 8 * 128 + 64), "bf16")
    q = x.as_strided((24, 8, 128), (x.stride(0), 128, 1), 64)
    o = torch.empty((24, 8, 128), dtype=torch.bfloat16, device=DEV)
    r, _ = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([20, 4]), o=o)
    assert r.data_ptr() == o.data_ptr()
    assert_attn(o, None, q, cache, [20, 4])


def test_attn_unaligned(crg):
    cache = Cache(22, "bf16", [90], 2, 64, 16)
    buf = torch.zeros(3 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    q = buf[1:].view(3, 4, 64)
    q.copy_(randn(gen(23), (3, 4, 64), "bf16"))
    o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([3]), want_lse=True)
    assert_attn(o, lse, q, cache, [3], tensor=False)


def test_attn_window_never_reads_released_pages(crg):
    """Pages wholly before every query's window may be given back (-1 in the table)."""
    cache = Cache(24, "bf16", [1000, 600], 2, 128, 16)
    q = randn(gen(25), (31, 4, 128), "bf16")
    ws = crg.Workspace(1 << 28, DEV)
    table = cache.table.clone()
    for s, (n, m) in enumerate(((30, 1000), (1, 600))):
        table[s, : max(0, m - n - 200 + 1) // 16] = -1
    o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, table, cache.lens, cu_of([30, 1]), window=200, want_lse=True,
                                workspace=ws)
    assert ws.status() == 0
    assert_attn(o, lse, q, cache, [30, 1], 200)


@pytest.mark.parametrize("simt", [False, True])
def test_attn_bad_pages_and_lengths_are_reported(crg, simt):
    """A page outside the cache or a length past the table: GDN_ERR_BOUNDS, nothing read there, and the other
    sequences as they should be."""
    cache = Cache(26, "bf16", [100, 60, 80], 2, 128, 16)
    q = randn(gen(27), (9, 4, 128), "bf16")
    for what in ("page", "negative", "length"):
        ws = crg.Workspace(1 << 28, DEV)
        table, lens = cache.table.clone(), cache.lens.clone()
        if what == "length":
            lens[1] = 100000
        else:
            table[1, 2] = 10 ** 9 if what == "page" else -5
        o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, table, lens, cu_of([4, 2, 3]), want_lse=True, workspace=ws,
                                    simt=simt)
        assert ws.status() == crg.GDN_ERR_BOUNDS, what
        ro, rl, a, ds = attn_ref(q, cache, [4, 2, 3], 0, 128 ** -0.5)
        for rows in (slice(0, 4), slice(6, 9)):
            off = np.abs(f64(o)[rows] - ro[rows])
            assert np.all(off <= 2.0 ** -8 * np.abs(ro[rows]) + (2.0 ** -8 + 4 * ds[rows][..., None] + 2.0 ** -16) * a[rows])


def test_attn_offsets_past_32_bits(crg):
    """Pages more than 2^31 elements apart."""
    stride = (1 << 31) + 128
    buf = torch.empty(2 * stride + 16 * 128 + 64, dtype=torch.bfloat16, device=DEV)
    view = lambda o: buf.as_strided((3, 8, 1, 128), (stride, 128, 128, 1), o)  # noqa: E731
    k, v = view(0), view(8 * 128)
    cache = Cache(28, "bf16", [20], 1, 128, 8, spare=0)
    k.copy_(cache.k)
    v.copy_(cache.v)
    q = randn(gen(29), (3, 4, 128), "bf16")
    for simt in (False, True):
        o, lse = crg.gdn_paged_attn(q, k, v, cache.table, cache.lens, cu_of([3]), want_lse=True, simt=simt)
        assert_attn(o, lse, q, cache, [3], tensor=not simt)


def test_attn_empty_calls(crg):
    cache = Cache(30, "bf16", [10], 1, 64, 16)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    o, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([0]), want_lse=True)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    o, _ = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table[:0], cache.lens[:0], None)
    assert o.shape == (0, 2, 64)


def test_attn_stream_and_graph(crg):
    """On another stream, and captured: a replay follows the lengths, tables and contents of the moment."""
    cache = Cache(31, "bf16", [300, 200], 2, 128, 16)
    q = randn(gen(32), (2, 8, 128), "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, _ = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens)
    side.synchronize()
    assert_attn(o, None, q, cache, [1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, o=o)
    cache.lens -= 37
    cache.lens_list = [263, 163]
    cache.table = cache.table.flip(0)[[1, 0]].contiguous()
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert_attn(o, None, q, cache, [1, 1])


def test_attn_wait_that_runs_out_is_reported(crg):
    """The test mode gives up at the first wait: the status says so and the context stays usable."""
    cache = Cache(33, "bf16", [300, 200], 2, 128, 16)
    q = randn(gen(34), (2, 8, 128), "bf16")
    ws = crg.Workspace(1 << 28, DEV)
    crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, workspace=ws, _test_no_wait=True)
    assert ws.status() == crg.GDN_ERR_TIMEOUT
    ws.reset()
    o, _ = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, workspace=ws)
    assert ws.status() == 0
    assert_attn(o, None, q, cache, [1, 1])


# ------------------------------------------------------------------- append

APPEND = [  # dtype, new, lens (with them), hq, hkv, d, rd, page, interleaved, order
    ("bf16", [1, 1, 1], [1, 16, 33], 4, 2, 128, 128, 16, False, "token"),
    ("bf16", [5, 0, 40], [5, 7, 90], 4, 2, 256, 64, 48, True, "token"),
    ("f32", [3, 9], [3, 30], 2, 1, 64, 32, 5, False, "head"),
    ("bf16", [1300], [1400], 3, 3, 64, 64, 64, False, "head"),
    ("bf16", [20], [7], 2, 1, 128, 0, 16, False, "token"),   # thirteen tokens before the start are dropped
    ("f32", [6], [11], 1, 1, 10, 6, 4, True, "token"),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(crg, case):
    dtype, new, lens, hq, hkv, d, rd, page, inter, order = case
    cache = Cache(40, dtype, lens, hkv, d, page, order)
    g = gen(41)
    n = sum(new)
    q, k, v = randn(g, (n, hq, d), dtype), randn(g, (n, hkv, d), dtype), randn(g, (n, hkv, d), dtype)
    inv = crg.gdn_rope_inv_freq(rd) if rd else None
    freqs = crg.gdn_rope_freqs(inv, DEV) if rd else None
    k0, v0 = cache.k.clone(), cache.v.clone()
    ws = crg.Workspace(256, DEV)
    qo = crg.gdn_kv_append(k, v, cache.k, cache.v, cache.table, cache.lens, cu_of(new), q=q, freqs=freqs,
                           interleaved=inter, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    pos = np.concatenate([np.arange(m - a, m) for a, m in zip(new, lens)]).astype(np.int64)
    inv64 = inv.numpy() if rd else np.zeros(0)
    assert_rope(qo, q, pos, inv64, rd, inter)
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device=DEV)
    t = 0
    for s, (a, m) in enumerate(zip(new, lens)):
        for i in range(a):
            p = m - a + i
            if p >= 0:
                pg, sl = int(cache.table[s, p // page]), p % page
                touched[pg, sl] = True
                assert torch.equal(cache.v[pg, sl], v[t])
                assert_rope(cache.k[pg, sl][None], k[t][None], np.array([p]), inv64, rd, inter)
            t += 1
    same = lambda a, b: torch.equal(a[~touched].nan_to_num(7.0), b[~touched].nan_to_num(7.0))  # noqa: E731
    assert same(cache.k, k0) and same(cache.v, v0)


def test_append_given_positions_in_place_and_without_q(crg):
    cache = Cache(42, "bf16", [30, 50], 2, 64, 16)
    g = gen(43)
    q, k, v = (randn(g, (7, h, 64), "bf16") for h in (4, 2, 2))
    inv = crg.gdn_rope_inv_freq(64)
    freqs = crg.gdn_rope_freqs(inv, DEV)
    pos = torch.randint(0, 10 ** 6, (7,), generator=g, device=DEV)
    q0 = q.clone()
    r = crg.gdn_kv_append(k, v, cache.k, cache.v, cache.table, cache.lens, cu_of([3, 4]), q=q, freqs=freqs,
                          positions=pos, q_out=q)
    assert r.data_ptr() == q.data_ptr()
    assert_rope(q, q0, pos.cpu().numpy(), inv.numpy(), 64, False)
    assert_rope(cache.k[int(cache.table[1, 3]), 1][None], k[6:], pos[6:].cpu().numpy(), inv.numpy(), 64, False)
    assert crg.gdn_kv_append(k, v, cache.k, cache.v, cache.table, cache.lens, cu_of([3, 4])) is None
    assert torch.equal(cache.k[int(cache.table[1, 3]), 1], k[6])


def test_append_bad_pages_are_reported(crg):
    cache = Cache(44, "bf16", [30, 50], 2, 64, 16)
    k0 = cache.k.clone()
    k = randn(gen(45), (2, 2, 64), "bf16")
    ws = crg.Workspace(256, DEV)
    table = cache.table.clone()
    table[1, 3] = 1 << 30
    crg.gdn_kv_append(k, k, cache.k, cache.v, table, cache.lens, workspace=ws)
    assert ws.status() == crg.GDN_ERR_BOUNDS
    pg, sl = int(table[0, 1]), 13
    assert torch.equal(cache.k[pg, sl], k[0])
    k0[pg, sl] = k[0]
    assert torch.equal(cache.k.nan_to_num(7.0), k0.nan_to_num(7.0))


# -------------------------------------------------------------------- pages

class Pages:
    """The bookkeeping in plain Python, beside the device's."""

    def __init__(self, n_rows, max_pages, n_pages, page, pools):
        self.table = [[-1] * max_pages for _ in range(n_rows)]
        self.lens, self.refs, self.page = [0] * n_rows, [0] * n_pages, page
        self.pools = [p.cpu().clone() for p in pools]

    def need(self, n):
        return -(-n // self.page)

    def free_pages(self, n):
        got = [i for i, r in enumerate(self.refs) if r == 0][:n]
        return got if len(got) == n else None

    def grow(self, seqs, lens):
        pages = self.free_pages(sum(self.need(m) - self.need(self.lens[s]) for s, m in zip(seqs, lens)))
        if pages is None:
            return False
        for s, m in zip(seqs, lens):
            for i in range(self.need(self.lens[s]), self.need(m)):
                self.table[s][i] = pages.pop(0)
                self.refs[self.table[s][i]] = 1
            self.lens[s] = m
        return True

    def free(self, seqs):
        for s in seqs:
            for i in range(self.need(self.lens[s])):
                self.refs[self.table[s][i]] -= 1
                self.table[s][i] = -1
            self.lens[s] = 0

    def fork(self, parents, children):
        pages = self.free_pages(sum(self.lens[p] % self.page > 0 for p in parents))
        if pages is None:
            return False
        for p, c in zip(parents, children):
            full = self.lens[p] // self.page
            for i in range(full):
                self.table[c][i] = self.table[p][i]
                self.refs[self.table[p][i]] += 1
            if self.lens[p] % self.page:
                new = self.table[c][full] = pages.pop(0)
                self.refs[new] = 1
                for t in self.pools:
                    t[new] = t[self.table[p][full]]
            self.lens[c] = self.lens[p]
        return True

    def compact(self):
        L = sum(r > 0 for r in self.refs)
        src = [i for i, r in enumerate(self.refs) if r > 0 and i >= L]
        dst = [i for i, r in enumerate(self.refs) if r == 0 and i < L]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
            for t in self.pools:
                t[d] = t[s]
        self.table = [[to.get(x, x) for x in row] for row in self.table]


@pytest.mark.parametrize("n_pages,page,width,dtype", [(40, 16, 7, torch.uint8), (150, 4, 24, torch.bfloat16),
                                                      (5000, 16, 640, torch.float32)])
def test_pages_follow_the_model(crg, n_pages, page, width, dtype):
    """Random grow, fork, free, compact against the plain model: tables, lengths, refs and contents equal."""
    rng = np.random.default_rng(n_pages)
    rows, most = 24, 30
    pools = [(torch.rand((n_pages, width), device=DEV) * 100).to(dtype) for _ in range(3)]
    model = Pages(rows, most, n_pages, page, pools)
    table = torch.full((rows, most + 3), -1, dtype=torch.int32, device=DEV)[:, :most]
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    ws = crg.Workspace(crg.gdn_pages_workspace_bytes(n_pages, rows), DEV)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    refused = 0
    for step in range(60):
        kind = ["grow", "fork", "free", "compact", "grow", "fork"][step % 6]
        done = True
        if kind == "grow":
            seqs = rng.permutation(rows)[: rng.integers(1, 8)].tolist()
            want = [min(most * page, model.lens[s] + int(rng.integers(0, 5 * page))) for s in seqs]
            done = model.grow(seqs, want)
            crg.gdn_pages_grow(table, lens, refs, dev(seqs), dev(want), page, workspace=ws)
        elif kind == "free":
            seqs = rng.permutation(rows)[:6].tolist()
            model.free(seqs)
            crg.gdn_pages_free(table, lens, refs, dev(seqs + seqs[:2]), page, workspace=ws)  # twice counts once
        elif kind == "fork":
            children = [s for s in range(rows) if model.lens[s] == 0][: int(rng.integers(1, 6))]
            parents = [s for s in range(rows) if model.lens[s] > 0]
            if not children or not parents:
                continue
            parents = rng.choice(parents, len(children)).tolist()
            done = model.fork(parents, children)
            crg.gdn_pages_fork(table, lens, refs, dev(parents), dev(children), pools, page, workspace=ws)
        else:
            model.compact()
            crg.gdn_pages_compact(table, lens, refs, pools, page, workspace=ws)
        assert ws.status() == (0 if done else crg.GDN_ERR_PAGES), (step, kind)
        if not done:
            refused += 1
            ws.reset()
        assert refs.tolist() == model.refs, (step, kind)
        assert lens.tolist() == model.lens, (step, kind)
        for s in range(rows):
            n = model.need(model.lens[s])
            assert table[s, :n].tolist() == model.table[s][:n], (step, kind, s)
        held = torch.tensor([r > 0 for r in model.refs])
        for a, b in zip(pools, model.pools):
            assert torch.equal(a.cpu()[held], b[held]), (step, kind)
    assert refused > 0 or n_pages > 40


def test_pages_refuse_bad_lists_and_change_nothing(crg):
    page, n_pages = 16, 12
    table = torch.full((5, 4), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(5, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    pool = torch.rand((n_pages, 64), device=DEV)
    ws = crg.Workspace(crg.gdn_pages_workspace_bytes(n_pages, 5), DEV)
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    crg.gdn_pages_grow(table, lens, refs, dev(0, 1), dev(40, 16), page, workspace=ws)
    assert ws.status() == 0
    before = [t.clone() for t in (table, lens, refs, pool)]
    grow = lambda s, n: crg.gdn_pages_grow(table, lens, refs, dev(*s), dev(*n), page, workspace=ws)  # noqa: E731
    fork = lambda p, c: crg.gdn_pages_fork(table, lens, refs, dev(*p), dev(*c), [pool], page, workspace=ws)  # noqa: E731
    for f, a, b in ((grow, (0, 9), (50, 20)), (grow, (0, -1), (50, 20)), (grow, (0, 0), (50, 60)), (grow, (2, 0), (8, 39)),
                    (grow, (2, 0), (8, 65)), (grow, (2, 3, 4), (64, 64, 64)), (fork, (0, 0), (2, 2)), (fork, (0,), (1,)),
                    (fork, (0, 2), (2, 3)), (fork, (2,), (2,)), (fork, (7,), (2,)), (fork, (0,), (7,)), (fork, (0,), (-3,))):
        f(a, b)
        assert ws.status() == crg.GDN_ERR_PAGES, (a, b)
        ws.reset()
        for x, y in zip(before, (table, lens, refs, pool)):
            assert torch.equal(x, y), (a, b)
    crg.gdn_pages_free(table, lens, refs, dev(9, -2), page, workspace=ws)
    assert ws.status() == crg.GDN_ERR_PAGES
    assert torch.equal(before[2], refs)


def test_pages_released_entries_and_bad_pages(crg):
    """-1 inside a row (a page given back under a window) is skipped; a page outside the cache is reported."""
    page, n_pages = 16, 8
    table = torch.tensor([[-1, 3, 5, -1], [-1, -1, -1, -1], [2, 99, -1, -1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([45, 0, 32], dtype=torch.int32, device=DEV)
    refs = torch.tensor([0, 0, 1, 1, 0, 1, 0, 0], dtype=torch.int32, device=DEV)
    pool = torch.arange(8, device=DEV, dtype=torch.float32)[:, None].repeat(1, 5)
    ws = crg.Workspace(crg.gdn_pages_workspace_bytes(n_pages, 3), DEV)
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    crg.gdn_pages_fork(table, lens, refs, dev(0), dev(1), [pool], page, workspace=ws)
    assert ws.status() == 0
    assert table[1].tolist() == [-1, 3, 0, -1] and refs.tolist() == [1, 0, 1, 2, 0, 1, 0, 0]
    assert pool[0].tolist() == [5.0] * 5
    crg.gdn_pages_compact(table, lens, refs, [pool], page, workspace=ws)
    assert ws.status() == crg.GDN_ERR_BOUNDS
    ws.reset()
    assert table.tolist() == [[-1, 3, 1, -1], [-1, 3, 0, -1], [2, 99, -1, -1]]
    assert refs.tolist() == [1, 1, 1, 2, 0, 0, 0, 0] and pool[:4, 0].tolist() == [5.0, 5.0, 2.0, 3.0]
    crg.gdn_pages_free(table, lens, refs, dev(2, 0), page, workspace=ws)
    assert ws.status() == crg.GDN_ERR_BOUNDS
    assert refs.tolist() == [1, 0, 0, 1, 0, 0, 0, 0] and lens.tolist() == [0, 45, 0]


@pytest.mark.parametrize("shape,dtype", [((9, 3, 5), torch.uint8), ((9, 6), torch.float32), ((9, 32, 128), torch.bfloat16)])
def test_pages_copy(crg, shape, dtype):
    """Pages of one, four and sixteen byte multiples, in strided pools; pairs outside the cache are skipped."""
    big = [(torch.rand((shape[0], 2) + shape[1:], device=DEV) * 100).to(dtype) for _ in range(2)]
    pools = [b[:, 1] for b in big]
    want = [b.clone() for b in big]
    for w in want:
        w[[4, 0, 7], 1] = w[[1, 2, 1], 1]
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = crg.Workspace(256, DEV)
    crg.gdn_pages_copy(pools, dev(1, 2, 1), dev(4, 0, 7), workspace=ws)
    assert ws.status() == 0 and all(torch.equal(a, b) for a, b in zip(big, want))
    crg.gdn_pages_copy(pools, dev(9, -1, 3), dev(5, 5, 9), workspace=ws)
    assert ws.status() == crg.GDN_ERR_BOUNDS and all(torch.equal(a, b) for a, b in zip(big, want))
