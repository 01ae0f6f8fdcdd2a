"""A small hybrid model served end to end: Gated DeltaNet layers with a full-attention layer after every
third, prompts in, then tokens one at a time for several beams, losing beams dropped and forked again from
the winners, the cache's pages brought together now and then.

    python examples/hybrid_beam.py [--tokens 24] [--beams 4] [--dtype bf16] [--keep 0]

Weights are random.  Projections are plain torch products; the layers between them are this package's:
    recurrent layer:  gdn_layer_fwd for a prompt, gdn_decode_step for a token, its state a row of a tensor
    attention layer:  gdn_kv_append (rotary positions on q and k on the way), gdn_paged_attn; for beams whose prompt is
                      long enough gdn_paged_attn_shared, which reads it once for all of them
    sequences:        gdn_pages_grow / fork / free / compact for the pages, gdn_pages_copy for the recurrent state
    a long prompt:    with --keep, gdn_paged_mass counts the attention weight of its positions and gdn_pages_evict
                      leaves that many of them in the cache before the beams begin
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_recurrence_gb300 as crg  # noqa: E402


@dataclass
class Config:
    vocab: int = 500
    width: int = 256
    layers: str = "rrra"       # r: recurrent, a: attention
    Hqk: int = 2               # recurrent layers: q/k heads, v heads, widths
    Hv: int = 4
    K: int = 64
    V: int = 64
    conv: int = 4
    heads: int = 8             # attention layers: query heads, kv heads, width, its rotary part
    kv_heads: int = 2
    D: int = 128
    rotary: int = 32
    page: int = 16
    pages: int = 96
    rows: int = 8              # sequences that may live at once
    max_len: int = 256
    keep: int = 0              # of a prompt, positions left in the cache (0: all); a quarter of them its last
    pays: int = 1 << 28        # bytes of a layer's k and v of the prompt, counted once a beam, from which it is read once for
                               # all (16 beams over 4000 positions, 4096 bytes each, 39 -> 32 us; 4 over 37 11 -> 20)
    dtype: torch.dtype = torch.bfloat16


class Hybrid:
    """The weights, and the state of up to `rows` sequences."""

    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        self.cfg, c = cfg, cfg
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g, device=device) / math.sqrt(s[0])).to(c.dtype)  # noqa: E731
        self.channels = 2 * c.Hqk * c.K + c.Hv * c.V
        self.embed, self.head = w(c.vocab, c.width) * math.sqrt(c.vocab), w(c.width, c.vocab)
        self.layers = []
        for kind in c.layers:
            if kind == "r":
                self.layers.append(dict(
                    x=w(c.width, self.channels), ab=w(c.width, 2 * c.Hv), z=w(c.width, c.Hv * c.V),
                    conv=(torch.randn((self.channels, c.conv), generator=g, device=device) / 2).to(c.dtype),
                    A_log=torch.rand(c.Hv, generator=g, device=device).mul_(2.0),
                    dt=torch.rand(c.Hv, generator=g, device=device) - 0.5, out=w(c.Hv * c.V, c.width),
                    state=torch.zeros((c.rows, c.Hv, c.V, c.K), device=device),
                    last=torch.zeros((c.rows, c.conv - 1, self.channels), dtype=c.dtype, device=device)))
            else:
                cache = lambda: torch.zeros((c.pages, c.page, c.kv_heads, c.D), dtype=c.dtype, device=device)  # noqa: E731
                self.layers.append(dict(q=w(c.width, c.heads * c.D), k=w(c.width, c.kv_heads * c.D),
                                        v=w(c.width, c.kv_heads * c.D), out=w(c.heads * c.D, c.width), k_cache=cache(),
                                        v_cache=cache()))
        self.pools = [x[n] for x in self.layers for n in ("k_cache", "v_cache") if n in x]
        self.freqs = crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(c.rotary), device)
        self.table = torch.full((c.rows, -(-c.max_len // c.page)), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(c.rows, dtype=torch.int32, device=device)
        self.refs = torch.zeros(c.pages, dtype=torch.int32, device=device)
        self.at = torch.zeros(c.rows, dtype=torch.int64, device=device)  # rotary position of a row's next token
        n_attn = c.layers.count("a")
        self.mass = torch.zeros((n_attn, c.rows, c.kv_heads, c.max_len), device=device) if c.keep else None
        self.pages_ws = crg.Workspace(crg.gdn_pages_workspace_bytes(c.pages, c.rows), device)

    # ------------------------------------------------------------- sequences

    def _list(self, x):
        return torch.as_tensor(x, dtype=torch.int32, device=self.table.device)

    def _pages(self, f, *args):
        f(self.table, self.lens, self.refs, *args, self.cfg.page, workspace=self.pages_ws)

    def grow(self, rows, by):
        rows = self._list(rows)
        self._pages(crg.gdn_pages_grow, rows, self.lens[rows.long()] + self._list(by))

    def fork(self, parents, children):
        """Rows `children` (empty) become copies of rows `parents`."""
        parents, children = self._list(parents), self._list(children)
        self._pages(crg.gdn_pages_fork, parents, children, self.pools)
        for name in ("state", "last"):
            crg.gdn_pages_copy([x[name] for x in self.layers if name in x], parents, children)
        self.at[children.long()] = self.at[parents.long()]

    def free(self, rows):
        self._pages(crg.gdn_pages_free, self._list(rows))
        self.at[self._list(rows).long()] = 0

    def evict(self, rows):
        """Rows cut to `keep` positions: in each layer, for each kv head, those that their tokens looked at most."""
        c = self.cfg
        keep = [c.keep] * len(rows)
        crg.gdn_pages_evict(self.table, self.lens, self.refs, self._list(rows), self._list(keep), self.mass, self.pools,
                            c.page, max_keep=c.keep, recent=c.keep // 4)

    def compact(self):
        self._pages(crg.gdn_pages_compact, self.pools)

    def check(self):
        """Synchronises; whether every page operation could be carried out, and every other call found its pages."""
        return self.pages_ws.status() == crg.GDN_OK == crg.gdn_paged_status(self.table.device)

    # ---------------------------------------------------------------- layers

    def _norm(self, h):
        x = h.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(h.dtype)

    def _recurrent(self, p, x, rows, cu, lengths):
        c = self.cfg
        ab = x @ p["ab"]
        a, b = ab[:, : c.Hv].contiguous(), ab[:, c.Hv:].contiguous()
        xs, z = x @ p["x"], (x @ p["z"]).view(-1, c.Hv, c.V)
        if cu is not None:  # prompts: from empty states
            o, h = crg.gdn_layer_fwd(xs, p["conv"], a, b, p["A_log"], p["dt"], c.Hqk, c.Hv, c.K, c.V, cu_seqlens=cu,
                                     z=z)
            p["state"][rows] = h
            ends = cu[1:].long()
            back = torch.arange(c.conv - 1, 0, -1, device=x.device)
            at = ends[:, None] - back
            there = at >= cu[:-1].long()[:, None]
            p["last"][rows] = torch.where(there[..., None], xs[at.clamp(min=0)], 0)
        else:
            state, last = p["state"][rows].contiguous(), p["last"][rows].contiguous()
            o, after = crg.gdn_decode_step(xs, last, p["conv"], a, b, p["A_log"], p["dt"], state, c.Hqk, c.Hv, c.K, c.V)
            p["state"][rows], p["last"][rows] = state, after
            o = crg.gdn_gated_rmsnorm(o, z)
        return o.view(-1, c.Hv * c.V) @ p["out"]

    def _attention(self, p, x, rows, cu, longest, positions, mass, groups):
        c, n = self.cfg, x.shape[0]
        q, k, v = ((x @ p[w]).view(n, -1, c.D) for w in "qkv")
        table, lens = self.table[rows], self.lens[rows]
        q = crg.gdn_kv_append(k, v, p["k_cache"], p["v_cache"], table, lens, cu, q=q, freqs=self.freqs, q_out=q,
                              positions=positions)
        if groups is not None:
            o, lse = crg.gdn_paged_attn_shared(q, p["k_cache"], p["v_cache"], table, lens, *groups, cu)
        else:
            o, lse = crg.gdn_paged_attn(q, p["k_cache"], p["v_cache"], table, lens, cu, max_new=longest,
                                        want_lse=mass is not None)
        if mass is not None and cu is not None:
            mass[rows] = crg.gdn_paged_mass(q, p["k_cache"], table, lens, lse, mass[rows], cu, max_new=longest,
                                            accumulate=False)
        return o.view(n, -1) @ p["out"]

    def forward(self, tokens, rows, lengths=None, shared=0):
        """New tokens of the sequences in `rows`: whole prompts (lengths, rows empty before), or one token each, of rows
        that have their first `shared` positions in common.  Returns the logits of all of them."""
        rows_t = torch.as_tensor(rows, device=tokens.device)
        new = lengths if lengths is not None else [1] * len(rows)
        self.grow(rows, new)
        positions = torch.cat([torch.arange(n, device=tokens.device) for n in new]) + \
            self.at[rows_t].repeat_interleave(self._list(new), output_size=sum(new))
        self.at[rows_t] += self._list(new)
        groups = (self._list([0, len(rows)]), self._list([shared])) if shared else None
        masses = iter(self.mass if self.mass is not None else [None] * len(self.layers))
        cu = None if lengths is None else self._list([0] + list(lengths)).cumsum(0).to(torch.int32)
        h = self.embed[tokens]
        for kind, p in zip(self.cfg.layers, self.layers):
            x = self._norm(h)
            if kind == "r":
                h = h + self._recurrent(p, x, rows_t, cu, lengths)
            else:
                h = h + self._attention(p, x, rows_t, cu, max(new), positions, next(masses), groups)
        return (self._norm(h) @ self.head).float()


def beams(model: Hybrid, prompt, n_beams, n_tokens):
    """Beam search from one prompt: [n_beams] token lists and their scores, best first."""
    rows = list(range(n_beams))
    logits = model.forward(prompt, [0], [prompt.numel()])[-1:]
    score = logits.log_softmax(-1)
    best = score[0].topk(n_beams)
    c, shared = model.cfg, prompt.numel()
    if c.keep:
        model.evict([0])
        shared = min(shared, c.keep)
    if n_beams * shared * 2 * c.kv_heads * c.D * c.dtype.itemsize < c.pays:
        shared = 0
    model.fork([0] * (n_beams - 1), rows[1:])
    texts, scores = [[t] for t in best.indices.tolist()], best.values
    for step in range(n_tokens - 1):
        logp = model.forward(torch.tensor([t[-1] for t in texts], device=prompt.device), rows,
                             shared=shared).log_softmax(-1)
        best = (scores[:, None] + logp).flatten().topk(n_beams)
        parents, tokens = (best.indices // logp.shape[1]).tolist(), (best.indices % logp.shape[1]).tolist()
        # a row goes on as its own first child; rows without one are dropped and forked again
        kept, again = {}, []
        for i, p in enumerate(parents):
            if p in kept:
                again.append(i)
            else:
                kept[p] = i
        spare = [r for r in range(n_beams) if r not in kept]
        if again:
            model.free([rows[r] for r in spare])
            model.fork([rows[parents[i]] for i in again], [rows[r] for r in spare])
        order = [None] * n_beams
        for p, i in kept.items():
            order[i] = rows[p]
        for i, r in zip(again, spare):
            order[i] = rows[r]
        texts = [texts[p] + [t] for p, t in zip(parents, tokens)]
        rows, scores = order, best.values
        if step % 8 == 7:
            model.compact()
    model.free(rows)
    if not model.check():
        raise RuntimeError("the cache has no page left")
    return texts, scores


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--keep", type=int, default=0)
    args = ap.parse_args()
    model = Hybrid(Config(dtype=torch.bfloat16 if args.dtype == "bf16" else torch.float32, keep=args.keep))
    prompt = torch.arange(37, device="cuda") * 11 % model.cfg.vocab
    texts, scores = beams(model, prompt, args.beams, args.tokens)
    for text, score in zip(texts, scores.tolist()):
        print(f"{score:9.3f}  {text}")


if __name__ == "__main__":
    main()
