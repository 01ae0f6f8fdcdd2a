"""Tensors whose rows lie on top of each other (broadcast ones) are refused before the library sees their stride of 0,
which it reads as dense: the kernels would address rows that are not there."""
import pytest
import torch

import chunked_recurrence_gb300 as crg
from chunked_recurrence_gb300 import paged


def _args(**kw):
    cache = torch.zeros(8, 16, 2, 64)
    return {**dict(q=torch.zeros(5, 4, 64), k_cache=cache, v_cache=cache, page_table=torch.zeros(5, 4, dtype=torch.int32),
                   seq_lens=torch.ones(5, dtype=torch.int32), k=torch.zeros(5, 2, 64), v=torch.zeros(5, 2, 64)), **kw}


OVERLAPPING = [
    dict(q=torch.zeros(1, 4, 64).expand(5, 4, 64)), dict(k=torch.zeros(1, 2, 64).expand(5, 2, 64)),
    dict(v=torch.zeros(1, 2, 64).expand(5, 2, 64)), dict(page_table=torch.zeros(1, 4, dtype=torch.int32).expand(5, 4)),
    dict(seq_lens=torch.ones(1, dtype=torch.int32).expand(5)),
    dict(q=torch.zeros(1000).as_strided((5, 4, 64), (128, 64, 1))),  # half over each other
]


@pytest.mark.parametrize("kw", OVERLAPPING, ids=lambda kw: "-".join(kw))
def test_paged_shapes(kw):
    assert crg.cache_shape(**_args()).q_stride == 256
    with pytest.raises(ValueError):
        crg.cache_shape(**_args(**kw))


@pytest.mark.parametrize("shape", [(64,), (2, 64), (16, 2, 64), (8, 1, 1, 64), (8, 16, 1, 64), (8, 1, 2, 64), (1, 16, 2, 64)])
def test_paged_caches(shape):
    cache = torch.zeros(shape).expand(8, 16, 2, 64)
    with pytest.raises(ValueError, match="overlap"):
        crg.cache_shape(**_args(k_cache=cache, v_cache=cache))


def test_single_rows_have_any_stride():
    """One row has nothing to lie upon: its stride is not looked at."""
    one = crg.cache_shape(torch.zeros(4, 64).as_strided((1, 4, 64), (0, 64, 1)), *[torch.zeros(1, 16, 2, 64)] * 2,
                          torch.zeros(4, dtype=torch.int32).as_strided((1, 4), (0, 1)), torch.ones(1, dtype=torch.int32))
    assert (one.q_stride, one.table_stride) == (256, 4)


@pytest.fixture
def no_launch(monkeypatch):
    """The binding on CPU tensors, up to the library call."""
    calls = []

    def entry(name):
        return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(paged, "_entry", entry)
    monkeypatch.setattr(paged, "_need_cuda", lambda *t: None)
    monkeypatch.setattr(paged, "_handle", lambda t, stream: 0)
    monkeypatch.setattr(paged, "_plans", {})
    return calls


def test_rope(no_launch):
    x, pos = torch.zeros(5, 4, 64), torch.arange(5)
    freqs = crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(64), "cpu")
    wide = torch.zeros(1, 4, 64).expand(5, 4, 64)
    crg.gdn_rope(x, x, pos, freqs)
    assert no_launch == ["gdn_rope"]
    for kw in (dict(q=wide), dict(k=wide), dict(q_out=wide), dict(k_out=wide)):
        with pytest.raises(ValueError, match="overlap"):
            crg.gdn_rope(**{**dict(q=x, k=x, positions=pos, freqs=freqs), **kw})
    assert no_launch == ["gdn_rope"]


@pytest.mark.parametrize("name", ["grow", "free", "fork", "compact"])
def test_page_tables(no_launch, name):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    lists = {"grow": (i32(2), i32(2)), "free": (i32(2),), "fork": (i32(2), i32(2), [i32(8, 4)]), "compact": ([i32(8, 4)],)}
    with pytest.raises(ValueError, match="overlap"):
        getattr(crg, "gdn_pages_" + name)(i32(1, 4).expand(5, 4), i32(5), i32(8), *lists[name], 16)
    assert no_launch == []


@pytest.mark.parametrize("which", [0, 1, 2])
def test_recurrent_shapes(which):
    qkv = [torch.zeros(6, 2, 64), torch.zeros(6, 2, 64), torch.zeros(6, 4, 32)]
    assert crg.make_shape(*qkv).q_stride == 128
    qkv[which] = qkv[which][:1].expand(6, -1, -1)
    with pytest.raises(ValueError, match="overlap"):
        crg.make_shape(*qkv)
    one = [t[:1] for t in qkv]  # a single token has nothing to lie upon
    one[which] = one[which].as_strided(one[which].shape, (0, one[which].shape[2], 1))
    crg.make_shape(*one)
