"""A small hybrid model served end to end: Gated DeltaNet layers with a full-attention layer after every
third, prompts in, then tokens one at a time for several beams, losing beams dropped and forked again from
the winners, the cache's pages brought together now and then.

    python examples/hybrid_beam.py [--tokens 24] [--beams 4] [--dtype bf16]

Weights are random.  Projections are plain torch products; the layers between them are this package's:
    recurrent layer:  gdn_layer_fwd for a prompt, gdn_decode_step for a token, its state a row of a tensor
    attention layer:  gdn_kv_append (rotary positions on q and k on the way), gdn_paged_attn
    sequences:        gdn_pages_grow / fork / free / compact for the pages, gdn_pages_copy for the recurrent state
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

    def free(self, rows):
        self._pages(crg.gdn_pages_free, self._list(rows))

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

    def _attention(self, p, x, rows, cu, longest):
        c, n = self.cfg, x.shape[0]
        q, k, v = ((x @ p[w]).view(n, -1, c.D) for w in "qkv")
        table, lens = self.table[rows], self.lens[rows]
        q = crg.gdn_kv_append(k, v, p["k_cache"], p["v_cache"], table, lens, cu, q=q, freqs=self.freqs, q_out=q)
        o, _ = crg.gdn_paged_attn(q, p["k_cache"], p["v_cache"], table, lens, cu, max_new=longest)
        return o.view(n, -1) @ p["out"]

    def forward(self, tokens, rows, lengths=None):
        """New tokens of the sequences in `rows`: whole prompts (lengths, rows empty before), or one token each.
        Returns the logits of all of them."""
        rows_t = torch.as_tensor(rows, device=tokens.device)
        self.grow(rows, lengths if lengths is not None else [1] * len(rows))
        cu = None if lengths is None else self._list([0] + list(lengths)).cumsum(0).to(torch.int32)
        h = self.embed[tokens]
        for kind, p in zip(self.cfg.layers, self.layers):
            x = self._norm(h)
            if kind == "r":
                h = h + self._recurrent(p, x, rows_t, cu, lengths)
            else:
                h = h + self._attention(p, x, rows_t, cu, max(lengths) if lengths else 1)
        return (self._norm(h) @ self.head).float()


def beams(model: Hybrid, prompt, n_beams, n_tokens):
    """Beam search from one prompt: [n_beams] token lists and their scores, best first."""
    rows = list(range(n_beams))
    logits = model.forward(prompt, [0], [prompt.numel()])[-1:]
    score = logits.log_softmax(-1)
    best = score[0].topk(n_beams)
    model.fork([0] * (n_beams - 1), rows[1:])
    texts, scores = [[t] for t in best.indices.tolist()], best.values
    for step in range(n_tokens - 1):
        logp = model.forward(torch.tensor([t[-1] for t in texts], device=prompt.device), rows).log_softmax(-1)
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
    args = ap.parse_args()
    model = Hybrid(Config(dtype=torch.bfloat16 if args.dtype == "bf16" else torch.float32))
    prompt = torch.arange(37, device="cuda") * 11 % model.cfg.vocab
    texts, scores = beams(model, prompt, args.beams, args.tokens)
    for text, score in zip(texts, scores.tolist()):
        print(f"{score:9.3f}  {text}")


if __name__ == "__main__":
    main()
