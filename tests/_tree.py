"""Drafted trees: small seeded cases and their plain references in 64 bits (CPU), with error bounds.

Bounds are derived, not fitted.  A dot product of bf16 values has exact fp32 products; its W-term fp32 sum is off
by at most W * 2^-23 * sum|a b| in any order and with truncating adders.  A rounding to bf16 is off by at most
2^-8 of the value."""
from __future__ import annotations

from dataclasses import dataclass

import torch

PAGE = 128


@dataclass
class Tree:
    """Host description of a batch of trees over a paged cache."""
    off: list
    parents: list
    ctx: list
    depth: list
    anc: list          # python ints, bit m: node m on the row's path
    block_table: torch.Tensor
    n_pages: int

    @property
    def n_rows(self):
        return len(self.parents)

    @property
    def max_blocks(self):
        return self.block_table.shape[1]

    def rows(self, b):
        return range(self.off[b], self.off[b + 1])

    def q_pos(self):
        return [self.ctx[b] + self.depth[r] for b in range(len(self.ctx)) for r in self.rows(b)]

    def q_req(self):
        return [b for b in range(len(self.ctx)) for _ in self.rows(b)]

    def dev(self, device, pad=0):
        """node_off, parents, ctx, block_table, anc on the device, with `pad` padding rows."""
        i32 = dict(dtype=torch.int32, device=device)
        par = self.parents + [123456] * pad
        return (torch.tensor(self.off, **i32), torch.tensor(par, **i32), torch.tensor(self.ctx, **i32),
                self.block_table.to(device), torch.tensor(signed(self.anc) + [0] * pad, dtype=torch.int64, device=device))


def signed(words):
    words = [w & (1 << 64) - 1 for w in words]
    return [w - (1 << 64) if w >> 63 else w for w in words]


def make_tree(ctx, counts, seed, shape="random", extra_blocks=0, spare=2):
    """Trees of counts[b] nodes after ctx[b] cached tokens; pages in random order."""
    g = torch.Generator().manual_seed(seed)
    off, parents, depth, anc = [0], [], [], []
    for n in counts:
        r0 = off[-1]
        for i in range(n):
            if i == 0:
                p = -1
            elif shape == "chain":
                p = i - 1
            elif shape == "star":
                p = 0
            else:
                p = int(torch.randint(max(0, i - 4), i, (1,), generator=g))
            parents.append(p)
            depth.append(0 if p < 0 else depth[r0 + p] + 1)
            anc.append((1 << i) | (0 if p < 0 else anc[r0 + p]))
        off.append(r0 + n)
    need = []
    for b, c in enumerate(ctx):
        deep = max([depth[r] for r in range(off[b], off[b + 1])], default=-1) + 1
        need.append((c + deep + PAGE - 1) // PAGE)
    mb = max(max(need), 1) + extra_blocks
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    bt = torch.full((len(ctx), mb), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[at:at + k]
        at += k
    return Tree(off, parents, list(ctx), depth, anc, bt, pool)


def bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def cached(pool, t: Tree, b):
    """Request b's cached rows in order, 64 bits: [ctx][G][width]."""
    c = t.ctx[b]
    pages = t.block_table[b, :(c + PAGE - 1) // PAGE].long()
    return pool[pages].reshape(-1, *pool.shape[2:])[:c].double()


def random_sel(t: Tree, G, topk, seed, drop_own=0.1, empty=0.1):
    """Any choice of candidate blocks: mostly with the own block, some rows with nothing at all."""
    g = torch.Generator().manual_seed(seed)
    sel = torch.full((t.n_rows, G, topk), -1, dtype=torch.int32)
    pos = t.q_pos()
    for r in range(t.n_rows):
        for x in range(G):
            if float(torch.rand((), generator=g)) < empty:
                continue
            own = pos[r] // PAGE
            perm = torch.randperm(own, generator=g)[:topk - 1].tolist() if own else []
            ids = perm + ([] if float(torch.rand((), generator=g)) < drop_own else [own])
            sel[r, x, :len(ids)] = torch.tensor(sorted(ids), dtype=torch.int32)
    return sel


def ref_scores(t: Tree, q_idx, kidx, kidx_new):
    """(scores, bound) fp64 [rows][G][max_blocks]."""
    R, G, Di = q_idx.shape
    s = torch.full((R, G, t.max_blocks), -torch.inf, dtype=torch.float64)
    tol = torch.zeros_like(s)
    for b in range(len(t.ctx)):
        keys = cached(kidx, t, b)
        for r in t.rows(b):
            pos = list(range(t.ctx[b]))
            kk = [keys]
            for m in range(t.off[b + 1] - t.off[b]):
                if t.anc[r] >> m & 1:
                    kk.append(kidx_new[t.off[b] + m].double()[None])
                    pos.append(t.ctx[b] + t.depth[t.off[b] + m])
            kk = torch.cat(kk)
            blk = torch.tensor(pos) // PAGE
            q = q_idx[r].double()
            dots = torch.einsum("gd,tgd->gt", q, kk)
            mag = torch.einsum("gd,tgd->gt", q.abs(), kk.abs()) * Di * 2.0 ** -23
            s[r].scatter_reduce_(1, blk.expand(G, -1), dots, "amax")
            tol[r].scatter_reduce_(1, blk.expand(G, -1), mag, "amax")
    return s, tol


def ref_attend(t: Tree, q, k_cache, v_cache, k_new, v_new, sel, sm_scale):
    """(out, lse, out bound, lse bound) fp64."""
    R, Hq, D = q.shape
    G = k_new.shape[1]
    hpg = Hq // G
    out = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), -torch.inf, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(t.ctx)):
        kc, vc = cached(k_cache, t, b), cached(v_cache, t, b)
        for r in t.rows(b):
            path = [m for m in range(t.off[b + 1] - t.off[b]) if t.anc[r] >> m & 1]
            rows = [t.off[b] + m for m in path]
            pos = torch.tensor(list(range(t.ctx[b])) + [t.ctx[b] + t.depth[x] for x in rows])
            for g in range(G):
                pick = {int(j) for j in sel[r, g] if j >= 0}
                see = torch.tensor([int(p) // PAGE in pick for p in pos], dtype=torch.bool)
                if not bool(see.any()):
                    continue
                kk = torch.cat([kc[:, g], k_new[rows, g].double()])[see]
                vv = torch.cat([vc[:, g], v_new[rows, g].double()])[see]
                qq = q[r, g * hpg:(g + 1) * hpg].double()
                s = qq @ kk.T * sm_scale
                # logits: the dot's sum, the scale's rounding and the exponent's fp32 argument
                ds = ((qq.abs() @ kk.abs().T) * sm_scale * (D + 4) * 2.0 ** -23).amax(-1) + 2.0 ** -20
                p = torch.softmax(s, -1)
                o = p @ vv
                mass = p @ vv.abs()
                h = slice(g * hpg, (g + 1) * hpg)
                out[r, h], lse[r, h] = o, torch.logsumexp(s, -1)
                b_lse[r, h] = 2 * ds + lse[r, h].abs() * 2.0 ** -21
                # probabilities rounded to bf16, exponent errors, fp32 sums, the result rounded to bf16
                b_out[r, h] = mass * (2.0 ** -8 + 2 * ds[:, None] + len(pos) * 2.0 ** -23) * 1.01 + \
                    o.abs() * 2.0 ** -8 + 1e-30
    return out, lse, b_out, b_lse


def assert_within(got, want, bound, what):
    got = got.detach().cpu().double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    d = (got[~inf] - want[~inf]).abs() - bound[~inf]
    assert not bool(torch.isnan(d).any()), f"{what}: NaN"
    assert d.numel() == 0 or float(d.max()) <= 0, f"{what}: {int((d > 0).sum())} outside the bound by {float(d.max()):.3e}"


def ref_verify(t: Tree, p, q, tokens, u_accept, u_next):
    """(path, n_accepted, next_token): the chain of rejections written out with normalised residuals."""
    path, n_acc, nxt = [], [], []
    for b in range(len(t.ctx)):
        r0, n = t.off[b], t.off[b + 1] - t.off[b]
        if n == 0:
            n_acc.append(0)
            nxt.append(-1)
            continue
        at, taken = 0, []
        while True:
            taken.append(at)
            dist = p[r0 + at].double().clamp(min=0)
            step = None
            for x in range(at + 1, n):
                if t.parents[r0 + x] != at:
                    continue
                tok = int(tokens[r0 + x])
                draft = 1.0 if q is None else float(q[r0 + at, tok])
                if float(u_accept[r0 + x]) * draft < float(dist[tok]):
                    step = x
                    break
                if q is None:
                    rest = dist.clone()
                    rest[tok] = 0.0
                else:
                    rest = (dist - q[r0 + at].double()).clamp(min=0)
                # the first residual's p is taken to sum to one, as probabilities do
                mass = 1.0 - float(dist[tok]) if q is None else float(rest.sum())
                dist = rest / mass if mass > 0 else rest * 0
            if step is None:
                break
            at = step
        if not float(dist.sum()) > 0:
            dist = p[r0 + at].double()
        cum = dist.cumsum(0)
        nxt.append(int((cum <= cum[-1] * float(u_next[b])).sum()))
        path += taken + [-1] * (n - len(taken))
        n_acc.append(len(taken))
    i32 = dict(dtype=torch.int32)
    return torch.tensor(path, **i32), torch.tensor(n_acc, **i32), torch.tensor(nxt, **i32)


def verify_inputs(t: Tree, vocab, seed, drafts, sharp=2.5, noise=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((t.n_rows, vocab), generator=g) * sharp
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + noise * torch.randn((t.n_rows, vocab), generator=g), -1)
    tokens, seen = torch.zeros(t.n_rows, dtype=torch.int32), {}
    for b in range(len(t.ctx)):
        for r in t.rows(b):
            if t.parents[r] < 0:
                continue
            up = t.off[b] + t.parents[r]
            if drafts:
                tokens[r] = int(torch.multinomial(q[up], 1, generator=g))
            else:
                k = seen.get(up, 0)
                seen[up] = k + 1
                tokens[r] = int(q[up].argsort(descending=True)[k % vocab])
    return p, q if drafts else None, tokens, torch.rand(t.n_rows, generator=g), torch.rand(len(t.ctx), generator=g)
