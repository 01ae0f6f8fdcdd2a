"""Work and inputs of the full-attention operators: rotary positions, appending to a paged
cache, attention over it, and the cache's pages.

`own` chooses the side: False runs the plain form of an operator in elementary torch
operations, True the package's entry points.
"""
import math
import random

import torch

own = False

BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the rotary step of one layer's q and k over a training batch's tokens
        dict(name="rope_train", op="rope", n_tok=8192, hq=32, hk=8, d=128, rd=128, interleaved=False,
             backward=False, factor=1.0, far=8192, dtype="bf16"),
        # its gradient for a quarter of a wide head, at the far positions of an extended context
        dict(name="rope_grad_far", op="rope", n_tok=5003, hq=16, hk=4, d=256, rd=64, interleaved=True,
             backward=True, factor=8.0, far=1000000, dtype="bf16"),
        # a short prompt in 32 bits
        dict(name="rope_f32_short", op="rope", n_tok=77, hq=6, hk=2, d=64, rd=64, interleaved=False,
             backward=False, factor=1.0, far=4096, dtype="f32"),
        # a decode step's new tokens of a batch of sequences
        dict(name="append_decode", op="append", n_seqs=64, max_new=1, max_len=1000, hq=32, hkv=8, d=128, rd=128,
             interleaved=False, page=16, dtype="bf16"),
        # ragged prompt chunks of several sequences, part of a wide head rotated
        dict(name="append_chunk", op="append", n_seqs=9, max_new=1700, max_len=4000, hq=16, hkv=4, d=256, rd=64,
             interleaved=False, page=64, dtype="bf16"),
        # a few users' next tokens over short contexts: latency
        dict(name="attn_decode_small", op="attn", n_seqs=3, max_new=1, min_len=1, max_len=900, hq=16, hkv=4, d=128,
             page=16, window=0, dtype="bf16"),
        # a full batch's next tokens over long ragged contexts: the cache is read once
        dict(name="attn_decode_batch", op="attn", n_seqs=64, max_new=1, min_len=500, max_len=16000, hq=32, hkv=8, d=128,
             page=64, window=0, dtype="bf16"),
        # prompt chunks and single tokens in one step, wide heads, few kv heads, an odd number of tokens
        dict(name="attn_chunk_mixed", op="attn", n_seqs=16, max_new=509, min_len=1, max_len=6000, hq=16, hkv=2, d=256,
             page=32, window=0, dtype="bf16"),
        # the second half of a long prompt over its first
        dict(name="attn_prefill", op="attn", n_seqs=1, max_new=8192, min_len=16384, max_len=16384, hq=32, hkv=8, d=128,
             page=64, window=0, dtype="bf16"),
        # a sliding window in 32 bits, a small model's debugging run
        dict(name="attn_window_f32", op="attn", n_seqs=5, max_new=37, min_len=1, max_len=700, hq=6, hkv=2, d=64,
             page=16, window=200, dtype="f32"),
        # a beam step: the losing beams are freed and forked again from the winners
        dict(name="pages_beam", op="beam", n_seqs=48, forks=24, max_len=3000, hkv=8, d=128, page=64, dtype="bf16"),
        # a cache whose pages are half free, brought together
        dict(name="pages_compact", op="compact", n_seqs=61, max_len=8000, hkv=8, d=128, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "beam", "compact"])
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        rd = rng.choice([x for x in (32, 64, 128, 256) if x <= d])
        return dict(op=op, n_tok=_log(rng, 1, 8192), hq=hkv * group, hk=hkv, d=d, rd=rd,
                    interleaved=rng.random() < 0.5, backward=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 8.0]),
                    far=_log(rng, 1000, 1000000), dtype=dtype)
    if op == "append":
        max_len = _log(rng, 16, 4000)
        return dict(op=op, n_seqs=_log(rng, 1, 48), max_new=min(max_len, _log(rng, 1, 1000)), max_len=max_len,
                    hq=hkv * group, hkv=hkv, d=d, rd=rng.choice([x for x in (32, 64, 128, 256) if x <= d]),
                    interleaved=rng.random() < 0.5, page=page, dtype=dtype)
    if op == "attn":
        dtype = rng.choice(["bf16"] * 5 + ["f32"])
        far = 1000 if dtype == "f32" else 12000
        kind = rng.choice(["tokens", "chunks", "chunks"])
        max_len = _log(rng, 16, far)
        if kind == "tokens":
            n_seqs, max_new = _log(rng, 1, 64), 1
        else:
            max_new = min(max_len, _log(rng, 2, 200 if dtype == "f32" else 3000))
            n_seqs = _log(rng, 1, max(1, min(24, int(3e9 / (max_new * max_len * hkv * group)))))
        return dict(op=op, n_seqs=n_seqs, max_new=max_new, min_len=1, max_len=max_len, hq=hkv * group, hkv=hkv, d=d,
                    page=page, window=rng.choice([0, 0, 0, _log(rng, 10, 4000)]), dtype=dtype)
    n_seqs = _log(rng, 2, 60)
    case = dict(op=op, n_seqs=n_seqs, max_len=_log(rng, 100, 4000), hkv=hkv, d=d, page=page, dtype=dtype)
    if op == "beam":
        case["forks"] = max(1, int(n_seqs * rng.uniform(0.2, 0.6)))
    return case


# The lengths belong to the case (work() counts them); the values and pages to the seed.
def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    r = random.Random("%s %s %s" % (case["n_seqs"], case["max_len"], case.get("max_new", 1)))
    n, top, most = case["n_seqs"], case["max_len"], case.get("max_new", 1)
    new, lens = [], []
    for s in range(n):
        k = most if s == 0 else 1 if r.random() < 0.4 else r.randint(1, most)
        m = top if s == n - 1 else r.randint(min(case.get("min_len", 1), top), top)
        new.append(min(k, top))
        lens.append(max(m, new[-1]))
    return new, lens


def _cdiv(a, b):
    return -(-a // b)


def _visible(case):
    """Pairs of a query and a key that it sees, over all sequences; keys that some query sees."""
    pairs = keys = 0
    w = case["window"] or (1 << 60)
    for k, m in zip(*_lengths(case)):
        first = m - k
        pairs += sum(min(p + 1, w) for p in range(first, m))
        keys += m - max(0, first - w + 1)
    return pairs, keys


def _beam_lists(case):
    """(sequences freed and used again as children, their parents)."""
    r = random.Random("%s %s" % (case["n_seqs"], case["forks"]))
    order = list(range(case["n_seqs"]))
    r.shuffle(order)
    n = min(case["forks"], case["n_seqs"] - 1)
    return order[:n], [r.choice(order[n:]) for _ in range(n)]


def _n_pages(case):
    _, lens = _lengths(case)
    used = sum(_cdiv(m, case["page"]) for m in lens)
    return 2 * used + 2 if case["op"] == "compact" else used + used // 8 + case["n_seqs"] + 2


def work(case):
    b = BYTES[case["dtype"]]
    op = case["op"]
    if op == "rope":
        rows = case["n_tok"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * rows * case["d"] * b + 8 * case["n_tok"], "flops": 3 * rows * case["rd"]}
    if op == "append":
        n_tok = sum(_lengths(case)[0])
        rows = n_tok * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 2 * rows * case["d"] * b, "flops": 3 * n_tok * (case["hq"] + case["hkv"]) * case["rd"]}
    if op == "attn":
        pairs, keys = _visible(case)
        n_tok = sum(_lengths(case)[0])
        return {"bytes": (2 * keys * case["hkv"] + 2 * n_tok * case["hq"]) * case["d"] * b,
                "flops": 4 * pairs * case["hq"] * case["d"]}
    page_bytes = 2 * case["page"] * case["hkv"] * case["d"] * b
    lens, page = _lengths(case)[1], case["page"]
    table = 4 * case["n_seqs"] * _cdiv(case["max_len"], page) + 4 * _n_pages(case)
    if op == "beam":
        _, parents = _beam_lists(case)
        moved = sum(1 for p in parents if lens[p] % page)
        return {"bytes": 2 * moved * page_bytes + 2 * table, "flops": 0}
    live, n = sum(_cdiv(m, page) for m in lens), _n_pages(case)
    return {"bytes": 2 * (live * (n - live) / n) * page_bytes + 2 * table, "flops": 0}  # expected for random pages


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _inv_freq(rd, factor):
    """Frequencies of the rotary pairs in 64 bits; with a factor, scaled by parts: pairs that turn fewer than
    once over the 4096 original positions are slowed by the factor, those over 32 times are left, a ramp between."""
    inv = BASE ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    if factor == 1.0:
        return inv, 1.0
    keep = ((4096 * inv / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return (1 - keep) * inv / factor + keep * inv, 0.1 * math.log(factor) + 1.0


def _freqs(inv):
    """The table of frequencies that a user of the package makes once."""
    import chunked_recurrence_gb300 as crg
    return crg.gdn_rope_freqs(inv, device="cuda")


def _cache(case, g, lens, junk):
    """A cache whose sequences' pages lie anywhere in it; what no sequence holds is junk."""
    page, dtype = case["page"], DTYPES[case["dtype"]]
    n_pages, width = _n_pages(case), _cdiv(max(lens), page)
    shape = (n_pages, page, case["hkv"], case["d"])
    k, v = _randn(g, shape, dtype), _randn(g, shape, dtype)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    need = torch.tensor([_cdiv(m, page) for m in lens], device="cuda")
    col = torch.arange(width, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    used = col < need[:, None]
    table = torch.where(used, order[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
    if junk:  # slots past a sequence's end and pages of no sequence
        slot = (torch.arange(page, device="cuda") + page * col[:, None]).expand(len(lens), width, page)
        past = slot >= torch.tensor(lens, device="cuda")[:, None, None]
        bad = torch.ones((n_pages, page), dtype=torch.bool, device="cuda")
        bad[table[used].long()] = past[used]
        k[bad] = math.nan
        v[bad] = math.nan
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[used].long()] = 1
    return k, v, table, refs


def _cu(new):
    return torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    g, dtype, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    st = dict(case=case)
    if op == "rope":
        n, d = case["n_tok"], case["d"]
        st["q"] = _randn(g, (n, case["hq"], d), dtype)
        st["k"] = _randn(g, (n, case["hk"], d), dtype)
        start = torch.randint(0, max(1, case["far"] - n) + 1, (1,), generator=g, device="cuda")
        st["positions"] = torch.arange(n, device="cuda") + start
        st["inv"], st["scale"] = _inv_freq(case["rd"], case["factor"])
        st["inv_cuda"] = st["inv"].cuda()
        st["freqs"] = _freqs(st["inv"]) if own else None
        return st
    new, lens = _lengths(case)
    st["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    st["k_cache"], st["v_cache"], st["table"], refs = _cache(case, g, lens, junk=op == "attn")
    if op in ("append", "attn"):
        st["cu"] = None if case["max_new"] == 1 else _cu(new)
        st["q"] = _randn(g, (sum(new), case["hq"], case["d"]), dtype)
        if op == "append":
            st["k"] = _randn(g, (sum(new), case["hkv"], case["d"]), dtype)
            st["v"] = _randn(g, (sum(new), case["hkv"], case["d"]), dtype)
            st["inv"], _ = _inv_freq(case["rd"], 1.0)
            st["inv_cuda"] = st["inv"].cuda()
            st["freqs"] = _freqs(st["inv"]) if own else None
        return st
    # the tables of the cache in one buffer, so that a pass can begin again from the same ones
    parts = [st["table"], st["lens"], refs]
    st["begin"] = torch.cat([p.reshape(-1) for p in parts])
    st["now"] = st["begin"].clone()
    a, b = parts[0].numel(), parts[0].numel() + parts[1].numel()
    st["table"], st["lens"], st["refs"] = st["now"][:a].view_as(parts[0]), st["now"][a:b], st["now"][b:]
    if op == "beam":
        children, parents = _beam_lists(case)
        st["children"] = torch.tensor(children, device="cuda", dtype=torch.int32)
        st["parents"] = torch.tensor(parents, device="cuda", dtype=torch.int32)
    return st


# ------------------------------------------------------------- plain forms

def _tokens(st, n_tok, n_seqs):
    """Of each new token: its sequence, its place among the sequence's new ones, its position."""
    dev = st["lens"].device
    cu = torch.arange(n_seqs + 1, device=dev) if st["cu"] is None else st["cu"].long()
    t = torch.arange(n_tok, device=dev)
    s = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[s]
    return cu, s, i, st["lens"].long()[s] - (cu[s + 1] - cu[s]) + i


def _rotate(x, positions, inv, rd, interleaved, scale, sign):
    angle = positions.double()[:, None] * inv
    c, s = (scale * angle.cos()).float()[:, None], (sign * scale * angle.sin()).float()[:, None]
    xf = x.float()
    r = xf[..., :rd]
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rd // 2], r[..., rd // 2:])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, xf[..., rd:]), -1).to(x.dtype)


def _plain_rope(st):
    case = st["case"]
    args = (st["positions"], st["inv_cuda"], case["rd"], case["interleaved"], st["scale"], -1.0 if case["backward"] else 1.0)
    return _rotate(st["q"], *args), _rotate(st["k"], *args)


def _plain_append(st):
    case = st["case"]
    _, s, _, p = _tokens(st, st["q"].shape[0], case["n_seqs"])
    page, slot = st["table"].long()[s, p // case["page"]], p % case["page"]
    st["k_cache"][page, slot] = _rotate(st["k"], p, st["inv_cuda"], case["rd"], case["interleaved"], 1.0, 1.0)
    st["v_cache"][page, slot] = st["v"]
    return _rotate(st["q"], p, st["inv_cuda"], case["rd"], case["interleaved"], 1.0, 1.0), st["k_cache"], st["v_cache"]


def _plain_attn(st):
    case = st["case"]
    q, page, hkv, d, n = st["q"], case["page"], case["hkv"], case["d"], case["n_seqs"]
    cu, s, i, p = _tokens(st, q.shape[0], n)
    at = st["table"].long().clamp(min=0)
    there = torch.arange(at.shape[1] * page, device=q.device)
    held = there < st["lens"][:, None]  # [n, L]
    k = st["k_cache"][at].flatten(1, 2).float().permute(0, 2, 3, 1)  # [n, hkv, d, L]
    v = torch.where(held[:, :, None, None], st["v_cache"][at].flatten(1, 2), 0).float().permute(0, 2, 1, 3)
    rows = torch.zeros((n, case["max_new"], hkv, case["hq"] // hkv, d), device=q.device)
    rows[s, i] = q.float().view(-1, hkv, case["hq"] // hkv, d)
    rows = rows.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, hkv, group * new, d]
    scores = torch.matmul(rows, k).mul_(d ** -0.5).view(n, hkv, -1, case["max_new"], there.numel())
    mine = torch.full((n, case["max_new"]), -1, device=q.device)
    mine[s, i] = p
    seen = (there <= mine[:, :, None]) & (there > mine[:, :, None] - (case["window"] or 1 << 40)) & held[:, None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-1e30)
    scores.sub_(top).exp_()
    total = scores.sum(-1)
    o = torch.matmul(scores.flatten(2, 3), v).view(n, hkv, -1, case["max_new"], d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0)
    lse = total.log() + top.squeeze(-1)
    return (o.permute(0, 3, 1, 2, 4)[s, i].reshape(q.shape).to(q.dtype),
            lse.permute(0, 3, 1, 2)[s, i].reshape(q.shape[:2]))


def _plain_beam(st):
    case, page = st["case"], st["case"]["page"]
    st["now"].copy_(st["begin"])
    table, lens, refs, c, p = st["table"], st["lens"], st["refs"], st["children"].long(), st["parents"].long()
    col = torch.arange(table.shape[1], device=table.device)
    # free the children's pages
    gone = col < (lens[c, None] + page - 1) // page
    refs.index_put_((table[c].long().clamp(min=0),), -gone.int(), accumulate=True)
    table[c] = -1
    # share the parents' full pages, copy the part-filled ones to the lowest free pages
    full, part = lens[p] // page, lens[p] % page > 0
    row = table[p]
    shared = col < full[:, None]
    refs.index_put_((row.long().clamp(min=0),), shared.int(), accumulate=True)
    rank = torch.where(refs == 0, torch.arange(refs.numel(), device=refs.device), refs.numel()).sort().values
    fresh = rank[(part.cumsum(0) - 1).clamp(min=0)].to(torch.int32)
    last = (col == full[:, None]) & part[:, None]
    table[c] = torch.where(last, fresh[:, None], torch.where(shared, row, -1))
    lens[c] = lens[p]
    src = row.gather(1, full.long().clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()[part]
    dst = fresh.long()[part]
    refs[dst] = 1
    st["k_cache"][dst] = st["k_cache"][src]
    st["v_cache"][dst] = st["v_cache"][src]
    return table, lens, refs, st["k_cache"], st["v_cache"]


def _plain_compact(st):
    st["now"].copy_(st["begin"])
    table, refs = st["table"], st["refs"]
    n = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    below = n < live.sum()
    src = (live & ~below).nonzero()[:, 0]  # in rising order, as many as
    dst = (~live & below).nonzero()[:, 0]
    to = n.clone()
    to[src] = dst
    st["k_cache"][dst] = st["k_cache"][src]
    st["v_cache"][dst] = st["v_cache"][src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), table))
    return table, st["lens"], refs, st["k_cache"], st["v_cache"]


# --------------------------------------------------------- package's calls

def _own(st):
    import chunked_recurrence_gb300 as crg
    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        return crg.gdn_rope(st["q"], st["k"], st["positions"], st["freqs"], interleaved=case["interleaved"],
                            scale=st["scale"], backward=case["backward"])
    if op == "append":
        q = crg.gdn_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"],
                              q=st["q"], freqs=st["freqs"], interleaved=case["interleaved"])
        return q, st["k_cache"], st["v_cache"]
    if op == "attn":
        return crg.gdn_paged_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"],
                                  max_new=case["max_new"], window=case["window"], want_lse=True)
    st["now"].copy_(st["begin"])
    tables = (st["table"], st["lens"], st["refs"])
    pools = (st["k_cache"], st["v_cache"])
    if op == "beam":
        crg.gdn_pages_free(*tables, st["children"], case["page"])
        crg.gdn_pages_fork(*tables, st["parents"], st["children"], pools, case["page"])
    else:
        crg.gdn_pages_compact(*tables, pools, case["page"])
    return (*tables, *pools)


PLAIN = {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "beam": _plain_beam,
         "compact": _plain_compact}


def run(st):
    return _own(st) if own else PLAIN[st["case"]["op"]](st)


# ---------------------------------------------------------- the definition

def exact(case, seed):
    """Outputs from the definition in 64 bits, token by token or head by head."""
    op = case["op"]
    if op in ("beam", "compact"):
        return None  # pages and whole numbers: moved, not computed
    st = prepare(case, seed)

    def turn(x, positions):
        """Pairs as complex numbers, each turned by its angle."""
        x, rd = x.double(), case["rd"]
        sign = -1.0 if case.get("backward") else 1.0
        w = st.get("scale", 1.0) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                               sign * torch.outer(positions.double(), st["inv"].cuda()))
        y = x.clone()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous()) * w[:, None]
            y[..., :rd] = torch.view_as_real(z).reshape(*x.shape[:-1], rd)
        else:
            z = torch.complex(x[..., : rd // 2].contiguous(), x[..., rd // 2: rd].contiguous()) * w[:, None]
            y[..., : rd // 2], y[..., rd // 2: rd] = z.real, z.imag
        return y

    if op == "rope":
        return turn(st["q"], st["positions"]), turn(st["k"], st["positions"])
    new, lens = _lengths(case)
    page, table = case["page"], st["table"].tolist()
    if op == "append":
        pos = torch.cat([torch.arange(m - k, m) for k, m in zip(new, lens)]).cuda()
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        k = turn(st["k"], pos)
        t = 0
        for s, (a, m) in enumerate(zip(new, lens)):
            rows = torch.tensor([table[s][p // page] * page + p % page for p in range(m - a, m)], device="cuda")
            kc.flatten(0, 1)[rows] = k[t: t + a]
            vc.flatten(0, 1)[rows] = st["v"][t: t + a].double()
            t += a
        return turn(st["q"], pos), kc, vc
    o = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    t, group, w = 0, case["hq"] // case["hkv"], case["window"] or (1 << 40)
    for s, (a, m) in enumerate(zip(new, lens)):
        pages = table[s][: _cdiv(m, page)]
        ks, vs = (st[c][pages].flatten(0, 1)[:m].double() for c in ("k_cache", "v_cache"))
        p = torch.arange(m - a, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")
        hide = (j > p) | (j <= p - w)
        for h in range(case["hq"]):
            x = (st["q"][t: t + a, h].double() @ ks[:, h // group].T) / math.sqrt(case["d"])
            x = x.masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[t: t + a, h] = z
            o[t: t + a, h] = torch.exp(x - z[:, None]) @ vs[:, h // group]
        t += a
    return o, lse
