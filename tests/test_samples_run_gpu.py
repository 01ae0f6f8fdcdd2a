"""Samples of one prompt as they are served, every step against a plain 64-bit model: the prompt appended and attended to,
the weight of its positions, eviction by it, forks, tokens of the samples at their own rotary positions over the cut
prompt, weights gathered further, one sample evicted while others share its pages.

The model keeps each row's keys and values per kv head as the cache has them (the keys as gdn_kv_append rotated them, read back
where they were appended), so attention and weights are compared by test_paged_gpu's and test_paged_mass_gpu's tolerances
and everything that moves has to be equal."""
import numpy as np
import pytest
import torch

from tests.test_paged_gpu import DEV, HALF, f64, gen, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("bf16", 64, 32), ("f32", 64, 16), ("bf16", 256, 16)])
def test_prompt_to_samples(dtype, d, page):
    import chunked_recurrence_gb300 as crg
    hq, hkv, n_prompt, keep, recent, samples, steps = 8, 2, 203, 70, 16, 4, 5
    group, scale, rows = hq // hkv, d ** -0.5, 6
    g = gen(d + page)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    n_pages = 60
    caches = [randn(g, (n_pages, page, hkv, d), dtype) for _ in range(2)]
    table = torch.full((rows, -(-300 // page)), -1, dtype=torch.int32, device=DEV)
    lens, refs = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    mass = torch.zeros((1, rows, hkv, 300), device=DEV)
    freqs = crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(d), DEV)
    crg.gdn_paged_status_reset()
    tables = (table, lens, refs)
    K, V = {}, {}  # row -> [hkv, len, d] in 64 bits
    u_p = 2.0 ** -8 if dtype == "bf16" and d in (64, 128, 256) else 0.0

    def held(row):
        pages = table[row, : -(-int(lens[row]) // page)].long()
        return [f64(c[pages].flatten(0, 1)[: int(lens[row])].transpose(0, 1)) for c in caches]

    def attend(q, row, first):
        """(o, lse, A, ds, weights [hq, n, len]) of new tokens at cached positions first ... of a row."""
        q64, k, v = f64(q), K[row], V[row]
        o, a, lse = np.zeros_like(q64), np.zeros_like(q64), np.zeros(q64.shape[:2])
        ds, w = np.zeros(q64.shape[:2]), np.zeros((hq, q64.shape[0], k.shape[1]))
        for h in range(hq):
            x = scale * q64[:, h] @ k[h // group].T
            size = scale * np.abs(q64[:, h]) @ np.abs(k[h // group]).T
            seen = np.arange(k.shape[1])[None] <= first + np.arange(len(q64))[:, None]
            x = np.where(seen, x, -np.inf)
            top = x.max(1, keepdims=True)
            e = np.exp(x - top)
            z = e.sum(1, keepdims=True)
            w[h] = e / z
            lse[:, h] = (np.log(z) + top)[:, 0]
            o[:, h], a[:, h] = w[h] @ v[h // group], w[h] @ np.abs(v[h // group])
            ds[:, h] = np.where(seen, size, 0).max(1) * (d + 8) * 2.0 ** -24 + 2.0 ** -20
        return o, lse, a, ds, w

    def check(o, lse, refs_):
        ro, rl, a, ds = (np.concatenate(x) for x in zip(*[r[:4] for r in refs_]))
        n = 300 * 2.0 ** -23
        assert np.all(np.abs(f64(o) - ro) <= HALF[o.dtype] * np.abs(ro) + (u_p + 4 * ds[..., None] + n) * a)
        assert np.all(np.abs(f64(lse) - rl) <= 2 * ds + n + 2.0 ** -22 * np.abs(rl))

    # the prompt, in row 2
    crg.gdn_pages_grow(*tables, i32(2), i32(n_prompt), page)
    q, k, v = (randn(g, (n_prompt, h, d), dtype) for h in (hq, hkv, hkv))
    cu = i32(0, n_prompt)
    q = crg.gdn_kv_append(k, v, *caches, table[2:3], lens[2:3], cu, q=q, freqs=freqs)
    K[2], V[2] = held(2)
    o, lse = crg.gdn_paged_attn(q, *caches, table[2:3], lens[2:3], cu, want_lse=True)
    ref = attend(q, 2, 0)
    check(o, lse, [ref])
    crg.gdn_paged_mass(q, caches[0], table[2:3], lens[2:3], lse, mass[0, 2:3], cu, accumulate=False)
    want = np.zeros((rows, hkv, 300))
    want[2, :, :n_prompt] = ref[4].reshape(hkv, group, n_prompt, n_prompt).sum((1, 2))
    # a weight is off by the lse's error and its own: (4 ds + n 2^-23) of it, some 1e-4 in all for scores of this size
    near = lambda: np.all(np.abs(f64(mass[0]) - want) <= 2.0 ** -12 * want + 1e-30)  # noqa: E731
    assert near()

    def evict(row, m, r):
        before = int(lens[row])
        masses = mass[0, row].cpu().numpy().copy()
        kept = crg.gdn_pages_evict(*tables, i32(row), i32(m), mass, caches, page, max_keep=m, recent=r, want_kept=True)
        kept = kept[0, 0].cpu().numpy()
        for h in range(hkv):
            stay = sorted(np.argsort(-masses[h, : before - r], kind="stable")[: m - r]) + list(range(before - r, before))
            assert kept[h].tolist() == stay
        K[row], V[row] = (np.stack([x[row][h, kept[h]] for h in range(hkv)]) for x in (K, V))
        want[row, :, :m] = np.stack([want[row, h, kept[h]] for h in range(hkv)])
        want[row, :, m:] = 0
        assert all(np.array_equal(a, b) for a, b in zip(held(row), (K[row], V[row])))

    evict(2, keep, recent)
    assert lens[2].item() == keep and (refs > 0).sum().item() == -(-keep // page) and near()
    # samples of it: rows 2, 0, 4, 5 (as the call lists them)
    order = [2, 0, 4, 5]
    crg.gdn_pages_fork(*tables, i32(2, 2, 2), i32(0, 4, 5), caches, page)
    mass[0, order[1:]] = mass[0, 2].clone()
    for r in order[1:]:
        K[r], V[r], want[r] = K[2].copy(), V[2].copy(), want[2].copy()
    groups, prefix = i32(0, samples), i32(keep)
    where = torch.tensor(order, device=DEV)
    for step in range(steps):
        crg.gdn_pages_grow(*tables, i32(*order), lens[where] + 1, page)
        q, k, v = (randn(g, (samples, h, d), dtype) for h in (hq, hkv, hkv))
        at = torch.full((samples,), n_prompt + step, device=DEV)
        t, n = table[where], lens[where]
        q = crg.gdn_kv_append(k, v, *caches, t, n, q=q, freqs=freqs, positions=at)
        for r in order:
            K[r], V[r] = held(r)
        o, lse = crg.gdn_paged_attn_shared(q, *caches, t, n, groups, prefix, want_lse=True)
        ref = [attend(q[i: i + 1], r, keep + step) for i, r in enumerate(order)]
        check(o, lse, ref)
        mass[0, where] = crg.gdn_paged_mass(q, caches[0], t, n, lse, mass[0, where])
        for r, x in zip(order, ref):
            want[r, :, : keep + step + 1] += x[4].reshape(hkv, group, -1).sum(1)
        assert near()
    # one of them is cut again while the others go on with its pages
    others = {r: held(r) for r in (2, 0, 5)}
    evict(4, 33, 8)
    assert all(np.array_equal(a, b) for r, x in others.items() for a, b in zip(held(r), x))
    assert near()
    crg.gdn_pages_free(*tables, i32(*order), page)
    assert refs.sum().item() == 0 and crg.gdn_paged_status() == crg.GDN_OK
