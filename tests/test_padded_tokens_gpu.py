"""Tokens behind the last sequence (a batch padded to a captured graph's size): their rows of o and lse stay as they were,
on every path of gdn_paged_attn and gdn_paged_attn_shared, and gdn_paged_mass counts none of them."""
import pytest
import torch

from tests.test_paged_gpu import DEV, assert_attn, cu_of, gen, randn
from tests.test_paged_groups_gpu import Shared, crg  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

CASES = [  # dtype, new, lens, hq, hkv, d, simt
    ("bf16", [1, 1, 1], [200, 217, 300], 4, 2, 128, False),     # a join of few rows
    ("bf16", [200, 90, 400], [400, 390, 700], 32, 8, 128, False),  # of many
    ("bf16", [3, 1, 2], [2000, 3000, 900], 8, 1, 256, False),
    ("f32", [1, 1, 1], [900, 617, 2000], 4, 2, 64, False),      # parts and their join
    ("f32", [40, 3, 1], [240, 617, 200], 4, 2, 64, False),
    ("bf16", [1, 2, 1], [900, 617, 2000], 4, 2, 96, False),
    ("bf16", [1, 1, 5], [900, 617, 2000], 4, 2, 128, True),
]


@pytest.mark.parametrize("spare", [1, 50])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rows_behind_the_last_sequence(crg, case, spare):  # noqa: F811
    dtype, new, lens, hq, hkv, d, simt = case
    cache = Shared(160, dtype, [0, 2, 3], [150, 0], lens, hkv, d, 16)
    n = sum(new)
    q = randn(gen(161), (n + spare, hq, d), dtype)
    cu = cu_of(new)
    args = (q, cache.k, cache.v, cache.table, cache.lens)
    for call in (lambda **kw: crg.gdn_paged_attn(*args, cu, **kw),
                 lambda **kw: crg.gdn_paged_attn_shared(*args, cache.groups, cache.prefix, cu, **kw)):
        # what the scratch held before is not zeros
        big = torch.full((1 << 26,), 3.0, device=DEV)
        del big
        o, lse = torch.full_like(q, 7.0), torch.full((n + spare, hq), 7.0, device=DEV)
        call(o=o, lse=lse, simt=simt)
        assert_attn(o[:n], lse[:n], q[:n], cache, new, tensor=dtype == "bf16" and d != 96 and not simt)
        assert (o[n:] == 7).all() and (lse[n:] == 7).all()
    mass = torch.zeros((3, hkv, max(lens)), device=DEV)
    lse[n:] = -1000.0  # a weight of these would show
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu, max_new=max(new), simt=simt)
    total = mass.double().sum(-1)
    want = torch.tensor(new, device=DEV, dtype=torch.float64)[:, None] * (hq // hkv)
    assert ((total / want - 1).abs() < 2.0 ** -8).all()
