"""gdn_pages_evict at the ends of its selection's forms (4096, 16384 and 32768 weights in registers, more read again),
against test_pages_evict_gpu's model; equal results each time."""
import math

import pytest
import torch

from tests.test_pages_evict_gpu import DEV, crg, i32, make, run  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("n", [4096, 4097, 16384, 16385, 32768, 32769])  # weights before the recent ones
def test_forms_of_the_selection(crg, n):  # noqa: F811
    page, recent = 64, 5
    for part in (7, 2):
        state = make(n + part, [n + recent], 1, 4, 8, page, torch.float32, spare=-(-n // page) + 1)
        mass = state[3]
        g = torch.Generator(device=DEV)
        g.manual_seed(n)
        mass[0, 0, 1] = torch.randint(0, 5, (n + recent,), generator=g, device=DEV).float()
        mass[0, 0, 2] = 1 + torch.rand(n + recent, generator=g, device=DEV) / 16  # their numbers begin alike
        odd = torch.tensor([0.0, -0.0, -1.0, math.inf, -math.inf, math.nan, 1e-40], device=DEV)
        mass[0, 0, 3] = odd.repeat(-(-(n + recent) // 7))[: n + recent]
        assert run(crg, state, page, [0], [recent + n - n // part], recent) is not None


def test_the_same_each_time(crg):  # noqa: F811
    """Many lists at once, whose candidates are listed in any order."""
    page = 16
    lens = [700 + 211 * i for i in range(24)]
    table, lens_, refs, mass, pools = make(20, lens, 3, 4, 8, page, torch.float32, spare=24 * 32)
    seqs, keep = i32(list(range(24))), i32([500] * 24)
    first = None
    for _ in range(30):
        state = [t.clone() for t in (table, lens_, refs)]
        m = mass.clone()
        kept = crg.gdn_pages_evict(*state, seqs, keep, m, [p.clone() for p in pools], page, 500, 20, want_kept=True)
        got = [kept, m, *state]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    for i, n in enumerate(lens):
        top = torch.sort(mass[:, i, :, : n - 20], dim=-1, descending=True, stable=True).indices[..., :480]
        assert torch.equal(torch.sort(top, dim=-1).values.int(), first[0][:, i, :, :480])
