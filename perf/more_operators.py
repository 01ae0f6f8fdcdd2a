"""Work and inputs of the operators for many samples of long prompts over a paged cache: attention of
sequences that share a prefix, the attention weight that each cached position gathers, and eviction by it.

`own` chooses the side: False runs the plain form of an operator in elementary torch operations, True the
package's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a few samples' next tokens over a short common prompt: latency
        dict(name="shared_small", op="shared", groups=1, members=4, prefix=600, own=40, max_new=1, hq=16, hkv=4, d=128,
             page=16, dtype="bf16"),
        # many samples of one long prompt, their next tokens
        dict(name="shared_samples", op="shared", groups=1, members=64, prefix=16000, own=500, max_new=1, hq=32, hkv=8,
             d=128, page=64, dtype="bf16"),
        # several prompts with samples each, wide heads, up to 7 drafted tokens to verify
        dict(name="shared_drafts", op="shared", groups=7, members=12, prefix=6000, own=900, max_new=7, hq=16, hkv=2,
             d=256, page=32, dtype="bf16"),
        # questions of ragged lengths after one long document
        dict(name="shared_chunks", op="shared", groups=1, members=15, prefix=9001, own=300, max_new=300, hq=32, hkv=8,
             d=128, page=64, dtype="bf16"),
        # a small model's debugging run in 32 bits, three prompts
        dict(name="shared_f32", op="shared", groups=3, members=5, prefix=700, own=60, max_new=3, hq=6, hkv=2, d=64,
             page=16, dtype="f32"),
        # a decode step of a full batch over long ragged contexts: the keys are read once
        dict(name="mass_decode", op="mass", n_seqs=64, max_new=1, min_len=500, max_len=16000, window=0, add=True, hq=32,
             hkv=8, d=128, page=64, dtype="bf16"),
        # all tokens of a long prompt, after its attention
        dict(name="mass_prompt", op="mass", n_seqs=1, max_new=8192, min_len=8192, max_len=8192, window=0, add=False,
             hq=32, hkv=8, d=128, page=64, dtype="bf16"),
        # the last tokens of ragged prompts as the ones that judge, wide heads
        dict(name="mass_last", op="mass", n_seqs=9, max_new=33, min_len=100, max_len=12000, window=0, add=False, hq=16,
             hkv=2, d=256, page=32, dtype="bf16"),
        # a sliding window in 32 bits, a few short chunks
        dict(name="mass_f32", op="mass", n_seqs=5, max_new=37, min_len=1, max_len=700, window=200, add=True, hq=6, hkv=2,
             d=64, page=16, dtype="f32"),
        # a page's worth of tokens out of a few short contexts: latency
        dict(name="evict_small", op="evict", layers=1, n_seqs=3, min_len=400, max_len=500, keep=384, recent=32, forks=0,
             hkv=4, d=128, page=16, dtype="bf16"),
        # a long prompt cut to an eighth in every layer before decoding
        dict(name="evict_prompt", op="evict", layers=6, n_seqs=1, min_len=16000, max_len=16000, keep=2001, recent=64,
             forks=0, hkv=8, d=128, page=64, dtype="bf16"),
        # ragged sequences of a batch, some of them sharing their first pages, some shorter than what is kept
        dict(name="evict_batch", op="evict", layers=2, n_seqs=24, min_len=700, max_len=6000, keep=1900, recent=256,
             forks=9, hkv=2, d=256, page=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "mass", "mass", "mass", "evict", "evict"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16"] * 4 + ["f32"])
    f32 = dtype == "f32"
    if op == "shared":
        groups = _log(rng, 1, 12)
        prefix = _log(rng, 10, 1500 if f32 else 12000)
        members = _log(rng, 1, max(1, (24 if f32 else 64) // groups))
        max_new = rng.choice([1, 1, _log(rng, 2, 12), _log(rng, 12, 40 if f32 else 300)])
        while groups * members * max_new * prefix * hkv * group * d > (5e9 if f32 else 8e10) and max_new > 1:
            max_new //= 2
        return dict(op=op, groups=groups, members=members, prefix=prefix, own=max_new + _log(rng, 1, 600), max_new=max_new,
                    hq=hkv * group, hkv=hkv, d=d, page=page, dtype=dtype)
    if op == "mass":
        max_len = _log(rng, 16, 1000 if f32 else 10000)
        kind = rng.choice(["tokens", "last", "chunks"])
        if kind == "tokens":
            n_seqs, max_new = _log(rng, 1, 48), 1
        else:
            max_new = min(max_len, _log(rng, 2, 64 if kind == "last" else 200 if f32 else 4000))
            while max_new * max_len * hkv * group * d > (1e10 if f32 else 1.3e11):
                max_new //= 2
            n_seqs = _log(rng, 1, max(1, min(16, int((1e10 if f32 else 1.3e11) / (max_new * max_len * hkv * group * d)))))
        return dict(op=op, n_seqs=n_seqs, max_new=max_new, min_len=1, max_len=max_len,
                    window=rng.choice([0, 0, 0, _log(rng, 10, 4000)]), add=rng.random() < 0.5, hq=hkv * group, hkv=hkv, d=d,
                    page=page, dtype=dtype)
    max_len = _log(rng, 60, 8000)
    n_seqs = _log(rng, 1, 24)
    keep = max(1, int(max_len * rng.uniform(0.1, 0.9)))
    layers = rng.randint(1, 3)
    n_seqs = max(1, min(n_seqs, int(3e8 / (layers * max_len * hkv * d * BYTES[dtype]))))
    return dict(op=op, layers=layers, n_seqs=n_seqs, min_len=max_len // 8, max_len=max_len, keep=keep,
                recent=min(keep, _log(rng, 1, 300)), forks=rng.choice([0, n_seqs // 3]), hkv=hkv, d=d, page=page,
                dtype=dtype)


# The lengths belong to the case (work() counts them); the values and pages to the seed.
def _shared_lengths(case):
    """Of each group its members and prefix; of each sequence its new and its own tokens (the new ones among them)."""
    r = random.Random("%s %s %s" % (case["groups"], case["prefix"], case["own"]))
    members = [case["members"] if g == 0 else r.randint(1, case["members"]) for g in range(case["groups"])]
    prefix = [case["prefix"] if g == 0 else r.randint(0, case["prefix"]) for g in range(case["groups"])]
    new, mine = [], []
    for s in range(sum(members)):
        new.append(case["max_new"] if s == 0 else r.randint(1, case["max_new"]))
        mine.append(max(new[-1], case["own"] if s == 0 else r.randint(1, case["own"])))
    return members, prefix, new, mine


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    n, top, most = case["n_seqs"], case["max_len"], case.get("max_new", 1)
    r = random.Random("%s %s %s" % (n, top, most))
    new, lens = [], []
    for s in range(n):
        new.append(min(top, most if s == 0 else r.randint(1, most)))
        lens.append(max(new[-1], top if s == n - 1 else r.randint(min(case["min_len"], top), top)))
    return new, lens


def _cdiv(a, b):
    return -(-a // b)


def _visible(new, lens, window):
    """Pairs of a query and a key that it sees, over all sequences; keys that some query sees."""
    pairs = keys = 0
    w = window or (1 << 60)
    for k, m in zip(new, lens):
        first = m - k
        pairs += sum(min(p + 1, w) for p in range(first, m))
        keys += m - max(0, first - w + 1)
    return pairs, keys


def _evict_layout(case):
    """Of each sequence: its length, what it keeps, and the sequence whose first pages it shares (or -1)."""
    lens = _lengths(case)[1]
    n = case["n_seqs"]
    forks = min(case["forks"], n - 1)
    parent = [-1] * (n - forks) + [(i * 7) % (n - forks) for i in range(forks)]
    return lens, [min(m, case["keep"]) for m in lens], parent


def work(case):
    b = BYTES[case["dtype"]]
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "shared":
        members, prefix, new, mine = _shared_lengths(case)
        of = [g for g, m in enumerate(members) for _ in range(m)]
        lens = [prefix[g] + m for g, m in zip(of, mine)]
        pairs, _ = _visible(new, lens, 0)
        return {"bytes": (2 * (sum(prefix) + sum(mine)) * hkv + 2 * sum(new) * case["hq"]) * d * b,
                "flops": 4 * pairs * case["hq"] * d}
    if op == "mass":
        new, lens = _lengths(case)
        pairs, keys = _visible(new, lens, case["window"])
        masses = keys if case["add"] else 0
        return {"bytes": (keys * hkv + sum(new) * case["hq"]) * d * b + 4 * sum(new) * case["hq"]
                + 4 * hkv * (sum(lens) + masses), "flops": 2 * pairs * case["hq"] * d}
    lens, keep, _ = _evict_layout(case)
    moved = sum(k for k, m in zip(keep, lens) if k < m)
    weighed = sum(m for k, m in zip(keep, lens) if k < m)
    return {"bytes": case["layers"] * hkv * (2 * 2 * moved * d * b + 4 * (2 * weighed + moved)), "flops": 0}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _i32(a):
    return torch.tensor(a, device="cuda", dtype=torch.int32)


def _tables(g, lens, shared, page, spare):
    """A table of pages that lie anywhere in the cache: sequence s has the first shared[s][1] tokens in common with
    sequence shared[s][0], as full pages.  Returns the table, the refs and the number of pages."""
    width = max(1, max(_cdiv(m, page) for m in lens))
    at, rows, used = 0, [], []
    for m, (other, common) in zip(lens, shared):
        head = rows[other][: common // page] if other >= 0 else []
        n = _cdiv(m, page) - len(head)
        rows.append(head + list(range(at, at + n)))
        used += rows[-1]
        at += n
    n_pages = at + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = _i32([r + [-1] * (width - len(r)) for r in rows])
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], -1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs.index_put_((order[torch.tensor(used, device="cuda").long()].long(),), torch.ones((), dtype=torch.int32, device="cuda"),
                    accumulate=True)
    return table, refs, n_pages


def _junk(caches, table, lens, page):
    """NaN in the slots past a sequence's end and in pages of no sequence."""
    col = torch.arange(table.shape[1], device="cuda")
    slot = (torch.arange(page, device="cuda") + page * col[:, None]).expand(len(lens), -1, page)
    held = slot < torch.tensor(lens, device="cuda")[:, None, None]
    good = torch.zeros((caches[0].shape[0], page), dtype=torch.bool, device="cuda")
    used = table >= 0
    good.index_put_((table[used].long(),), held[used].bool())  # sequences that share a page fill it
    for c in caches:
        c[~good] = math.nan


def _cu(new):
    return torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    g, dtype, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    page, hkv, d = case["page"], case["hkv"], case["d"]
    st = dict(case=case)
    if op == "shared":
        members, prefix, new, mine = _shared_lengths(case)
        first = [sum(members[:i]) for i in range(len(members) + 1)]
        of = [i for i, m in enumerate(members) for _ in range(m)]
        lens = [prefix[i] + m for i, m in zip(of, mine)]
        shared = [(first[i] if s > first[i] else -1, prefix[i]) for s, i in enumerate(of)]
        st["table"], _, n_pages = _tables(g, lens, shared, page, 3)
        caches = [_randn(g, (n_pages, page, hkv, d), dtype) for _ in range(2)]
        for s, i in enumerate(of):  # the part-filled last page of a prefix is each sequence's own copy
            if s > first[i] and prefix[i] % page:
                a, b = st["table"][first[i], prefix[i] // page].long(), st["table"][s, prefix[i] // page].long()
                for c in caches:
                    c[b, : prefix[i] % page] = c[a, : prefix[i] % page]
        _junk(caches, st["table"], lens, page)
        st["k_cache"], st["v_cache"] = caches
        st["lens"], st["groups"], st["prefix"] = _i32(lens), _i32(first), _i32(prefix)
        st["cu"] = None if case["max_new"] == 1 else _cu(new)
        st["q"] = _randn(g, (sum(new), case["hq"], d), dtype)
        st["most"] = max(sum(new[a:b]) for a, b in zip(first, first[1:]))
        return st
    if op == "mass":
        new, lens = _lengths(case)
        st["table"], _, n_pages = _tables(g, lens, [(-1, 0)] * len(lens), page, 3)
        st["k_cache"] = _randn(g, (n_pages, page, hkv, d), dtype)
        _junk([st["k_cache"]], st["table"], lens, page)
        st["lens"], st["cu"] = _i32(lens), None if case["max_new"] == 1 else _cu(new)
        st["q"] = _randn(g, (sum(new), case["hq"], d), dtype)
        st["begin"] = torch.rand((len(lens), hkv, max(lens)), generator=g, device="cuda")
        st["mass"] = st["begin"].clone()
        st["lse"] = torch.empty((sum(new), case["hq"]), device="cuda")
        for h, rows, tok, heads, x in _scores(st, torch.float32):  # what the attention before left
            st["lse"][tok[:, None], heads] = torch.logsumexp(x, -1).T
        return st
    lens, keep, parent = _evict_layout(case)
    shared = [(p, min(lens[p], m) // 2 if p >= 0 else 0) for p, m in zip(parent, lens)]
    fresh = sum(_cdiv(k, page) for k, m in zip(keep, lens) if k < m)
    table, refs, n_pages = _tables(g, lens, shared, page, fresh + 2)
    st["pools"] = [_randn(g, (n_pages, page, hkv, d), dtype) for _ in range(2 * case["layers"])]
    # weights as softmax sums gather them: a few positions have most, many are tiny, later ones have seen fewer queries
    mass = torch.randn((case["layers"], len(lens), hkv, max(lens)), generator=g, device="cuda").mul_(2).exp_()
    mass[torch.rand(mass.shape, generator=g, device="cuda") < 0.05] = 0.0
    # the tables and weights in one buffer, so that a pass can begin again from the same ones
    parts = [table, _i32(lens), refs]
    st["begin"] = torch.cat([p.reshape(-1) for p in parts] + [mass.view(torch.int32).reshape(-1)])
    st["now"] = st["begin"].clone()
    a, b, c = table.numel(), table.numel() + len(lens), table.numel() + len(lens) + n_pages
    st["table"], st["lens"], st["refs"] = st["now"][:a].view_as(table), st["now"][a:b], st["now"][b:c]
    st["mass"] = st["now"][c:].view(torch.float32).view(mass.shape)
    st["seqs"], st["keep"] = torch.arange(len(lens), device="cuda", dtype=torch.int32), _i32(keep)
    return st


# ------------------------------------------------------------- plain forms

def _tokens(st, n_tok, n_seqs):
    """Of each new token: its sequence, its place among the sequence's new ones, its position."""
    cu = torch.arange(n_seqs + 1, device="cuda") if st["cu"] is None else st["cu"].long()
    t = torch.arange(n_tok, device="cuda")
    s = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[s]
    return cu, s, i, st["lens"].long()[s] - (cu[s + 1] - cu[s]) + i


def _gather(cache, table, page, held):
    """Rows of the sequences' positions [n, hkv, L, d] in 32 bits; those not held are zeros."""
    x = cache[table.long().clamp(min=0)].flatten(1, 2)[:, : held.shape[1]]
    return torch.where(held[:, :, None, None], x, 0).float().permute(0, 2, 1, 3)


def _plain_shared(st):
    """A group's rows against its prefix in one product, each sequence's against its own positions in a padded one, and
    one softmax over both."""
    case = st["case"]
    members, prefix, new, mine = _shared_lengths(case)
    q, page, hkv, d, n_seqs = st["q"], case["page"], case["hkv"], case["d"], sum(members)
    group = case["hq"] // hkv
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    cu, s, i, p = _tokens(st, q.shape[0], n_seqs)
    at = s0 = 0
    for m, P in zip(members, prefix):
        n = sum(new[s0: s0 + m])
        tok = torch.arange(at, at + n, device=q.device)
        sl, il, pl = s[tok] - s0, i[tok], p[tok]
        most, far = max(new[s0: s0 + m]), max(mine[s0: s0 + m])
        rows = q[tok].float().view(n, hkv, group, d)
        # the prefix: [hkv, n * group, P]
        table = st["table"][s0: s0 + m]
        there = torch.arange(P, device=q.device)
        kp, vp = (_gather(st[c], table[:1], page, (there >= 0)[None])[0] for c in ("k_cache", "v_cache"))
        x1 = torch.matmul(rows.permute(1, 0, 2, 3).reshape(hkv, n * group, d), kp.transpose(1, 2)).mul_(d ** -0.5)
        x1 = x1.view(hkv, n, group, P).masked_fill_(there > pl[:, None, None], -math.inf)
        # their own positions, a row a new token of a sequence: [m, hkv, most * group, far]
        skip = P // page
        there = torch.arange(P - skip * page, P - skip * page + far, device=q.device)
        own_len = st["lens"][s0: s0 + m].long() - skip * page
        held = torch.arange(there[-1] + 1, device=q.device) < own_len[:, None]
        width = min(table.shape[1], skip + _cdiv(int(held.shape[1]), page))
        held = held[:, : (width - skip) * page]
        ko, vo = (_gather(st[c], table[:, skip: width], page, held)[:, :, P - skip * page:] for c in ("k_cache", "v_cache"))
        far = ko.shape[2]
        pad = torch.zeros((m, most, hkv, group, d), device=q.device)
        pad[sl, il] = rows
        x2 = torch.matmul(pad.permute(0, 2, 1, 3, 4).reshape(m, hkv, most * group, d), ko.transpose(2, 3)).mul_(d ** -0.5)
        x2 = x2.view(m, hkv, most, group, far).permute(0, 2, 1, 3, 4)[sl, il].permute(1, 0, 2, 3)  # [hkv, n, group, far]
        x2 = x2.masked_fill(P + torch.arange(far, device=q.device) > pl[:, None, None], -math.inf)
        top = x2.amax(-1, keepdim=True)
        if P:
            top = torch.maximum(top, x1.amax(-1, keepdim=True))
        top = top.clamp(min=-1e30)
        w1, w2 = (x1 - top).exp(), (x2 - top).exp()
        total = w1.sum(-1) + w2.sum(-1)
        num = torch.matmul(w1.view(hkv, n * group, P), vp).view(hkv, n, group, d)
        pad2 = torch.zeros((m, most, hkv, group, far), device=q.device)
        pad2[sl, il] = w2.permute(1, 0, 2, 3)
        y = torch.matmul(pad2.permute(0, 2, 1, 3, 4).reshape(m, hkv, most * group, far), vo)
        num = num + y.view(m, hkv, most, group, d).permute(0, 2, 1, 3, 4)[sl, il].permute(1, 0, 2, 3)
        o[tok] = (num / total[..., None]).permute(1, 0, 2, 3).reshape(n, case["hq"], d).to(q.dtype)
        lse[tok] = (total.log() + top.squeeze(-1)).permute(1, 0, 2).reshape(n, case["hq"])
        at, s0 = at + n, s0 + m
    return o, lse


def _scores(st, dtype):
    """The scaled and masked scores of the cases of op mass, sequence by sequence and kv head by kv head: the head, the
    sequence, its tokens, the query heads and [group, new, len]."""
    case = st["case"]
    new, lens = _lengths(case)
    page, d, group, w = case["page"], case["d"], case["hq"] // case["hkv"], case["window"] or (1 << 40)
    t = 0
    for s, (a, m) in enumerate(zip(new, lens)):
        k = st["k_cache"][st["table"][s, : _cdiv(m, page)].long()].flatten(0, 1)[:m].to(dtype)
        tok = torch.arange(t, t + a, device="cuda")
        p, j = torch.arange(m - a, m, device="cuda")[:, None], torch.arange(m, device="cuda")
        hide = (j > p) | (j <= p - w)
        for h in range(case["hkv"]):
            heads = torch.arange(h * group, (h + 1) * group, device="cuda")
            x = torch.matmul(st["q"][t: t + a, h * group: (h + 1) * group].to(dtype).transpose(0, 1), k[:, h].T)
            yield h, s, tok, heads, (x * d ** -0.5).masked_fill_(hide, -math.inf)
        t += a


def _plain_mass(st):
    case = st["case"]
    if case["add"]:
        st["mass"].copy_(st["begin"])
    if case["max_new"] > 1:
        for h, s, tok, heads, x in _scores(st, torch.float32):
            w = x.sub_(st["lse"][tok[:, None], heads].T[..., None]).exp_().sum((0, 1))
            row = st["mass"][s, h, : w.numel()]
            row.copy_(row + w if case["add"] else w)
        return st["mass"]
    # single tokens: one padded product for all sequences
    n, hkv, group, far = case["n_seqs"], case["hkv"], case["hq"] // case["hkv"], st["mass"].shape[2]
    there = torch.arange(far, device="cuda")
    held = there < st["lens"][:, None]
    k = _gather(st["k_cache"], st["table"], case["page"], held)
    x = torch.matmul(st["q"].float().view(n, hkv, group, -1), k.transpose(2, 3)).mul_(case["d"] ** -0.5)
    seen = held & (there >= st["lens"][:, None] - (case["window"] or 1 << 30))
    x.sub_(st["lse"].view(n, hkv, group, 1)).masked_fill_(~seen[:, None, None], -math.inf)
    w = x.exp_().sum(2)
    st["mass"].copy_(st["mass"] + w if case["add"] else torch.where(held[:, None], w, st["mass"]))
    return st["mass"]


def _plain_evict(st):
    case, page = st["case"], st["case"]["page"]
    st["now"].copy_(st["begin"])
    table, lens, refs, mass = st["table"], st["lens"], st["refs"], st["mass"]
    L, hkv = mass.shape[3], case["hkv"]
    there = torch.arange(L, device=mass.device)
    cut = st["keep"] < lens
    # a sequence's last `recent` positions first, then the largest weights, ties to the lowest position
    recent = torch.minimum(st["keep"], torch.full_like(lens, case["recent"]))
    late = (there >= (lens - recent)[:, None]) & (there < lens[:, None])
    rank = torch.where(late[None, :, None], math.inf, mass)
    rank = torch.where((there < lens[:, None])[None, :, None], rank, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., : case["keep"]]
    mine = torch.arange(order.shape[-1], device=mass.device) < st["keep"][:, None]  # [n, keep]
    kept = torch.where(mine[None, :, None], order, L).sort(-1).values
    # fresh pages, the lowest free ones
    need = torch.where(cut, (st["keep"] + page - 1) // page, 0)
    free = (refs == 0).nonzero()[:, 0].to(torch.int32)
    col = torch.arange(table.shape[1], device=table.device)
    at = (need.cumsum(0) - need)[:, None] + col
    fresh = torch.where(col < need[:, None], free[at.clamp(max=free.numel() - 1)], -1)
    # the rows move: [n, hkv, keep] of every layer
    move = mine & cut[:, None]
    s, i = move.nonzero(as_tuple=True)
    dst, slot = fresh[s, i // page].long(), i % page
    heads = torch.arange(hkv, device=table.device)
    for layer in range(case["layers"]):
        j = kept[layer][s, :, i]  # [moved, hkv]
        src = table[s[:, None], j // page].long()
        for pool in st["pools"][2 * layer: 2 * layer + 2]:
            pool[dst, slot] = pool[src, j % page, heads]
    w = torch.where(mine[None, :, None], mass.gather(-1, kept.clamp(max=L - 1)), 0.0)
    past = there < lens[:, None]
    out = torch.zeros_like(mass)
    out[..., : w.shape[-1]] = w
    mass.copy_(torch.where((past & cut[:, None])[None, :, None], out, mass))
    # the tables follow
    old = table[cut].long()
    refs.index_put_((old.clamp(min=0),), -(old >= 0).int(), accumulate=True)
    refs[fresh[fresh >= 0].long()] = 1
    table.copy_(torch.where(cut[:, None], fresh, table))
    lens.copy_(st["keep"])
    return table, lens, refs, mass, torch.where(kept < L, kept, -1).to(torch.int32), *st["pools"]


# --------------------------------------------------------- package's calls

def _own(st):
    import chunked_recurrence_gb300 as crg
    case, op = st["case"], st["case"]["op"]
    if op == "shared":
        return crg.gdn_paged_attn_shared(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["groups"],
                                         st["prefix"], st["cu"], max_group_new=st["most"], want_lse=True)
    if op == "mass":
        if case["add"]:
            st["mass"].copy_(st["begin"])
        return crg.gdn_paged_mass(st["q"], st["k_cache"], st["table"], st["lens"], st["lse"], st["mass"], st["cu"],
                                  max_new=case["max_new"], window=case["window"], accumulate=case["add"])
    st["now"].copy_(st["begin"])
    kept = crg.gdn_pages_evict(st["table"], st["lens"], st["refs"], st["seqs"], st["keep"], st["mass"], st["pools"],
                               case["page"], max_keep=case["keep"], recent=case["recent"], want_kept=True)
    return st["table"], st["lens"], st["refs"], st["mass"], kept, *st["pools"]


PLAIN = {"shared": _plain_shared, "mass": _plain_mass, "evict": _plain_evict}


def run(st):
    return _own(st) if own else PLAIN[st["case"]["op"]](st)


# ---------------------------------------------------------- the definition

def exact(case, seed):
    """Outputs from the definition in 64 bits, sequence by sequence and head by head."""
    op = case["op"]
    if op == "evict":
        return None  # whole numbers, and rows that move: nothing is computed
    st = prepare(case, seed)
    page, scale = case["page"], 1.0 / math.sqrt(case["d"])
    group = case["hq"] // case["hkv"]
    if op == "shared":
        members, prefix, new, mine = _shared_lengths(case)
        lens = [prefix[g] + m for g, m in zip([g for g, m in enumerate(members) for _ in range(m)], mine)]
    else:
        new, lens = _lengths(case)
    pages = st["table"].tolist()
    w = case.get("window") or (1 << 40)
    o = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if op == "mass" else None
    t = 0
    for s, (a, m) in enumerate(zip(new, lens)):
        held = pages[s][: _cdiv(m, page)]
        ks = st["k_cache"][held].flatten(0, 1)[:m].double()
        vs = st["v_cache"][held].flatten(0, 1)[:m].double() if op == "shared" else None
        i = torch.arange(a, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")
        sees = (j <= m - a + i) & (j > m - a + i - w)
        if op == "mass" and not case["add"]:
            mass[s, :, :m] = 0
        for h in range(case["hq"]):
            x = torch.einsum("id,jd->ij", st["q"][t: t + a, h].double() * scale, ks[:, h // group])
            if op == "mass":
                e = torch.exp(x - st["lse"][t: t + a, h].double()[:, None])
                mass[s, h // group, :m] += torch.where(sees, e, 0.0).sum(0)
                continue
            top = torch.where(sees, x, -math.inf).amax(1, keepdim=True)
            e = torch.where(sees, torch.exp(x - top), 0.0)
            z = e.sum(1, keepdim=True)
            lse[t: t + a, h] = (top + z.log())[:, 0]
            o[t: t + a, h] = (e @ vs[:, h // group]) / z
        t += a
    return mass if op == "mass" else (o, lse)
