"""GPU parity of gdn_paged_mass for few query rows where a warp has several tiles, against test_paged_mass_gpu's 64-bit
implementation and by its tolerances."""
import pytest
import torch

from tests.test_paged_mass_gpu import crg, run  # noqa: F401
from tests.test_paged_mass_held_host import FURTHER

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def tiles_a_warp(lens, new, hkv, d, window):
    """Of 64 positions and a kv head, over the warps of the kernel's 152 blocks (at least)."""
    tiles = sum(-(-n // 64) - (max(0, n - k - window + 1) // 64 if window else 0) for n, k in zip(lens, new)) * hkv
    return tiles / (152 * (6 if d == 256 else 12))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d,hq,hkv,new,window", [
    (64, 32, 8, 4, 1000), (128, 32, 8, 8, 1024), (128, 8, 8, 32, 1500), (256, 16, 8, 4, 700), (64, 32, 8, 2, 900),
    (128, 32, 8, 4, 0), (64, 16, 8, 1, 800),
])
def test_windows_over_many_tiles(crg, d, hq, hkv, new, window, accumulate):  # noqa: F811
    """Drafted tokens in a sliding-window layer.  Of the first tile in sight the last tokens may see nothing, of the next
    tiles they do: the first position in sight lies up to 30 before a tile's end."""
    lens = [window + new - 1 + 64 * (s % 11) + 34 + s % 30 for s in range(40)] if window else [900 + 62 * s for s in range(32)]
    assert tiles_a_warp(lens, [new] * len(lens), hkv, d, window) > 2
    run(crg, 150, "bf16", [new] * len(lens), lens, hq, hkv, d, 16, window, accumulate, max_new=new)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", FURTHER, ids=str)
def test_more_rows_than_the_call_said(crg, case, accumulate):  # noqa: F811
    """max_new picks the kernel; a warp takes each tile again for the rows past it while the next tile's keys are on their way.
    The same bits each time."""
    d, group, new, said, window = case
    lens = [900 + 62 * s for s in range(32)]
    cache, q, lse, mass = run(crg, 151, "bf16", [new] * 32, lens, 8 * group, 8, d, 16, window, accumulate, max_new=said)
    cu = torch.arange(0, 32 * new + 1, new, dtype=torch.int32, device=q.device)
    first = torch.zeros_like(mass)
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, first, cu, max_new=said, window=window)
    for _ in range(20):
        again = torch.zeros_like(mass)
        crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, again, cu, max_new=said, window=window)
        assert torch.equal(first, again)
