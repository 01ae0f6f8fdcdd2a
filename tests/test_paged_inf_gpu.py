"""Infinities and NaN in q, k and v of attention on the paths that multiply in fp32: they reach the rows that see them, as
the definition says, and no others.

Reference: 64-bit sums over a row's own positions.  Tolerance of the finite values as in test_paged_gpu (no weights
rounded): u_out |o| + (4 ds + n 2^-23) A.
"""
import math

import numpy as np
import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

INF, NAN = math.inf, math.nan
CASES = [  # dtype, new, length, query heads, kv heads, D, page, window
    (torch.float32, 1, 900, 4, 2, 128, 16, 0),     # few rows, positions in parts
    (torch.float32, 3, 70, 4, 2, 64, 16, 0),
    (torch.float32, 90, 200, 4, 1, 96, 5, 0),      # many rows
    (torch.float32, 90, 200, 2, 1, 256, 16, 40),
    (torch.float32, 40, 60, 2, 1, 7, 3, 0),
    (torch.bfloat16, 70, 133, 4, 2, 96, 12, 0),
    (torch.bfloat16, 2, 133, 4, 2, 200, 12, 30),
]
# what is put where: tensor, token (from the end of the sequence, or of the new ones for q), column, value
ODD = {
    "k +inf": [("k", 2, 0, INF)], "k -inf": [("k", 2, 0, -INF), ("k", 30, 1, -INF)], "k nan": [("k", 2, 1, NAN)],
    "v +inf": [("v", 2, 0, INF), ("v", 40, 3, INF)], "v both": [("v", 2, 0, INF), ("v", 20, 0, -INF)],
    "v nan": [("v", 2, 5, NAN), ("v", 35, 2, NAN)], "q inf": [("q", 1, 0, INF)], "q nan": [("q", 1, 0, NAN)],
    "largest": [("k", 2, 0, 3.3e38), ("v", 2, 1, 3.3e38)], "first": [("v", -1, 0, INF), ("k", -1, 1, NAN)],
}


def _reference(q, k, v, window):
    """o, lse, A, ds of [new, heads], row by row over what each sees."""
    new, hq, d = q.shape
    m, hkv = k.shape[:2]
    o, a = np.zeros((new, hq, d)), np.zeros((new, hq, d))
    lse, ds = np.full((new, hq), -np.inf), np.zeros((new, hq))
    with np.errstate(all="ignore"):
        for i in range(new):
            p = m - new + i
            rows = slice(max(0, p - window + 1) if window else 0, p + 1)
            for h in range(hq):
                kk, vv = k[rows, h * hkv // hq], v[rows, h * hkv // hq]
                s = (q[i, h] * kk).sum(1) * d ** -0.5
                size = (np.abs(q[i, h]) * np.abs(kk)).sum(1) * d ** -0.5
                top = s.max()
                if top == -np.inf:
                    continue
                e = np.exp(s - top)
                e[s == -np.inf] = 0
                z = e.sum()
                w = e / z
                o[i, h], lse[i, h] = (w[:, None] * vv).sum(0), np.log(z) + top
                a[i, h] = (w[:, None] * np.abs(vv)).sum(0)
                ds[i, h] = np.max(size[np.isfinite(size)], initial=0.0) * (d + 8) * 2.0 ** -24 + 2.0 ** -20
    return o, lse, a, ds


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("what", ODD)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_they_reach_who_sees_them(case, what, simt):
    dtype, new, length, hq, hkv, d, page, window = case
    g = torch.Generator().manual_seed(length + d)
    q = torch.randn(new, hq, d, generator=g)
    k, v = (torch.randn(length, hkv, d, generator=g) for _ in range(2))
    q[..., 0] = q[..., 0].abs() + 0.5  # an infinite k has the same sign of score for every row,
    if new > 1:
        q[::2, :, 0] *= -1             # or for every second one
    q[..., 1] = q[..., 1].abs() + 0.5
    for name, token, col, value in ODD[what]:
        x = {"q": q, "k": k, "v": v}[name]
        x[max(0, x.shape[0] - 1 - token) if token >= 0 else 0, 0, col] = value
    q, k, v = (x.to(dtype) for x in (q, k, v))
    n = -(-length // page)
    order = torch.randperm(n, generator=g)
    caches = []
    for x in (k, v):
        c = torch.full((n * page, hkv, d), NAN, dtype=dtype)
        c[:length] = x
        caches.append(c.view(n, page, hkv, d)[order.argsort()].cuda())
    ws = crg.Workspace(1 << 27, "cuda")
    o, lse = crg.gdn_paged_attn(q.cuda(), *caches, order.to(torch.int32)[None].cuda(),
                                torch.tensor([length], dtype=torch.int32, device="cuda"),
                                torch.tensor([0, new], dtype=torch.int32, device="cuda"), window=window, want_lse=True,
                                simt=simt, workspace=ws)
    assert ws.status() == 0
    got, got_lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    ro, rl, a, ds = _reference(*(x.double().numpy() for x in (q, k, v)), window)
    if what == "largest":  # past fp32 where it is an infinity there: compared where it is not
        keep = np.isfinite(got) & (np.abs(ro) < 1e37) & np.isfinite(rl)[..., None]
        assert not np.isnan(got[np.abs(rl) < 1e30]).any()
    else:
        for x, y in ((got, ro), (got_lse, rl)):
            assert np.array_equal(np.isnan(x), np.isnan(y))
            assert np.array_equal(np.isposinf(x), np.isposinf(y)) and np.array_equal(np.isneginf(x), np.isneginf(y))
        keep = np.isfinite(ro)
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    with np.errstate(invalid="ignore"):
        off = np.abs(got - ro)
        tol = u * np.abs(ro) + (4 * ds[..., None] + length * 2.0 ** -23) * a
    assert np.all(off[keep] <= tol[keep])
    ok = np.isfinite(rl) & (np.abs(rl) < 1e30)
    assert np.all(np.abs(got_lse - rl)[ok] <= (2 * ds + length * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl))[ok])
