"""Drafted trees on the GPU at the edges of their arithmetic: references that rise within an item, infinite keys and
values, flat tails and empty residuals, layouts that are refused.  References in 64 bits; bounds as in tests/_tree.py."""
import pytest
import torch

from tests import _tree as T

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def msa():
    import block_sparse_attention_06_gb300 as m
    return m


def _inputs(t, Hq, G, D, seed):
    return [T.bf16(s, seed + i) for i, s in enumerate(((t.n_rows, Hq, D), (t.n_pages, 128, G, D), (t.n_pages, 128, G, D),
                                                       (t.n_rows, G, D), (t.n_rows, G, D)))]


def _attend(msa, t, dims, x, sel):
    off, _, ctx, bt, anc = t.dev(DEV)
    err = msa.new_err_word(DEV)
    out, lse = msa.msa_sparse_attn_tree(*[v.to(DEV) for v in x], bt, ctx, off, anc, sel.to(DEV), dims, err_word=err)
    msa.msa_check(err)
    return out, lse


def _check(t, out, lse, x, sel, D):
    ro, rl, bo, bl = T.ref_attend(t, *x, sel, D ** -0.5)
    T.assert_within(lse, rl, bl, "lse")
    T.assert_within(out, ro, bo, "out")


# ------------------------------------------------------------------ attention: a reference that rises within an item

@pytest.mark.parametrize("nodes", [9, 64])                      # one 128-row half, and two or more
@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (16, 2, 64), (8, 2, 128), (4, 1, 64)])
@pytest.mark.parametrize("ctx,block", [(128, 0), (100, 0), (384, 1), (230, 1)])
def test_reference_rises_in_later_columns(msa, ctx, block, Hq, G, D, nodes):
    """Tokens 40 and 100 of a block pass one row's other logits by far more than 2^40, after that row's and its
    neighbours' weights of the first tokens are already stored: a whole block and a partial one, the first item
    and a later one."""
    t = T.make_tree([ctx], [nodes], 91, "chain")
    x = _inputs(t, Hq, G, D, 92)
    q, kc = x[0], x[1]
    q[..., 0] = 0.0
    page = int(t.block_table[0, block])
    kc[page, 40, :, 0], kc[page, min(100, ctx - 1 - 128 * block), :, 0] = 64.0, 96.0
    for node in range(0, nodes, 5):                             # one row of a node, so few of a warp's 32
        q[node, 3, 0] = 8.0                                     # 64 * 8 / sqrt(128) = 45 = 65 in units of log 2
    sel = torch.arange(4, dtype=torch.int32).expand(nodes, G, 4).contiguous()
    sel[sel >= t.max_blocks] = -1
    out, lse = _attend(msa, t, msa.Dims(Hq, G, D, 64, 4, t.max_blocks), x, sel)
    _check(t, out, lse, x, sel, D)


@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (8, 2, 64)])
def test_reference_rises_among_drafted_tokens(msa, Hq, G, D):
    t = T.make_tree([300], [60], 93, "chain")
    x = _inputs(t, Hq, G, D, 94)
    q, kn = x[0], x[3]
    q[..., 0] = 0.0
    kn[45, :, 0] = 64.0
    q[::5, 3, 0] = 8.0
    sel = torch.tensor([0, 1, 2, -1], dtype=torch.int32).expand(60, G, 4).contiguous()
    out, lse = _attend(msa, t, msa.Dims(Hq, G, D, 64, 4, t.max_blocks), x, sel)
    _check(t, out, lse, x, sel, D)


# ------------------------------------------------------------------ attention: infinite keys

def _check_finite(t, out, lse, x, sel, D):
    """As _check, over the tokens whose logit is finite: a weight of exp(-inf) is no weight, and no part of a bound."""
    q, kc, vc, kn, vn = x
    G = kn.shape[1]
    hpg = q.shape[1] // G
    for b in range(len(t.ctx)):
        kb, vb = T.cached(kc, t, b), T.cached(vc, t, b)
        for r in t.rows(b):
            rows = [t.off[b] + m for m in range(t.off[b + 1] - t.off[b]) if t.anc[r] >> m & 1]
            blk = torch.tensor(list(range(t.ctx[b])) + [t.ctx[b] + t.depth[y] for y in rows]) // 128
            for g in range(G):
                see = torch.isin(blk, sel[r, g][sel[r, g] >= 0])
                k, v = torch.cat([kb[:, g], kn[rows, g].double()])[see], torch.cat([vb[:, g], vn[rows, g].double()])[see]
                h = slice(g * hpg, (g + 1) * hpg)
                qq = q[r, h].double()
                fin = torch.isfinite(qq @ k.T).all(0)
                assert torch.equal(fin, torch.isfinite(qq @ k.T).any(0))   # the same tokens for all heads
                k, v = k[fin], v[fin]
                s = qq @ k.T * D ** -0.5
                ds = ((qq.abs() @ k.abs().T) * D ** -0.5 * (D + 4) * 2.0 ** -23).amax(-1) + 2.0 ** -20
                p = torch.softmax(s, -1)
                o, want = p @ v, torch.logsumexp(s, -1)
                bound = (p @ v.abs()) * (2.0 ** -8 + 2 * ds[:, None] + len(see) * 2.0 ** -23) * 1.01 + \
                    o.abs() * 2.0 ** -8 + 1e-30
                T.assert_within(lse[r, h], want, 2 * ds + want.abs() * 2.0 ** -21, f"lse of row {r}")
                T.assert_within(out[r, h], o, bound, f"out of row {r}")


@pytest.mark.parametrize("nodes", [5, 64])
@pytest.mark.parametrize("Hq,G,D", [(8, 1, 128), (8, 1, 64), (4, 1, 128), (4, 1, 64)])
@pytest.mark.parametrize("blocks,tokens", [((0,), 32), ((0, 1), 32), ((0, 1, 2), 32), ((0, 2), 96), ((0, 1), 128),
                                           ((1,), 33)])
def test_infinite_keys_at_the_start_of_blocks(msa, blocks, tokens, Hq, G, D, nodes):
    """The first tokens of whole blocks have logits of -inf (a cache masked by infinite keys): they weigh nothing, and
    the tokens behind them count like any others."""
    t = T.make_tree([400], [nodes], 95, "chain")
    x = _inputs(t, Hq, G, D, 96)
    q, kc, vc = x[:3]
    q[..., 0] = q[..., 0].abs() + 0.5
    for j in range(3):
        page = int(t.block_table[0, j])
        vc[page] += 2 - 2 * j                                   # blocks told apart by their values
        if j in blocks:
            kc[page, :tokens, :, 0] = -float("inf")
    sel = torch.full((nodes, G, 4), -1, dtype=torch.int32)
    for r in range(nodes):                                      # one to three blocks, the first of them always there
        n = 1 + r % 3
        sel[r, :, :n] = torch.arange(n, dtype=torch.int32)
        if tokens == 128:
            sel[r, :, n] = 3
    out, lse = _attend(msa, t, msa.Dims(Hq, G, D, 64, 4, t.max_blocks), x, sel)
    _check_finite(t, out, lse, x, sel, D)


def test_rows_whose_logits_are_all_infinite(msa):
    """Nothing but logits of -inf: 0 and -inf, like a row that sees no token, and the neighbours are unharmed."""
    t = T.make_tree([256], [6], 98, "star")
    x = _inputs(t, 8, 1, 128, 99)
    x[0][..., 0] = x[0][..., 0].abs() + 0.5
    x[1][int(t.block_table[0, 0]), :, :, 0] = -float("inf")
    sel = torch.tensor([0, 1], dtype=torch.int32).repeat(6, 1, 1)
    sel[::2, :, 1] = -1
    out, lse = _attend(msa, t, msa.Dims(8, 1, 128, 64, 2, t.max_blocks), x, sel)
    assert bool((out[::2] == 0).all()) and bool((lse[::2] == -float("inf")).all())
    x = [v[1::2].contiguous() if i in (0, 3, 4) else v for i, v in enumerate(x)]
    alone = T.make_tree([256], [3], 98, "star")
    alone.block_table, alone.n_pages = t.block_table, t.n_pages
    _check_finite(alone, out[1::2], lse[1::2], x, torch.full((3, 1, 2), 1, dtype=torch.int32), 128)


# ------------------------------------------------------------------ verification: sums of flat tails, rows of any mass

def _flat_tail(V, head, x1, x2):
    """A likely token and a flat tail: x1 in its first half, x2 in the second.  Returns the row, and the tail's entries
    as whole numbers of 2^-60 with their sum (fp32 numbers from 2^-36 on are whole numbers of 2^-60)."""
    x = torch.full((V,), x1, dtype=torch.float32)
    x[V // 2:] = x2
    x[head] = 0.0
    units = (x.double() * 2.0 ** 60).long()
    row = x.clone()
    row[head] = 1.0 - float(x.double().sum())
    return row, units, int(units.sum())


def _border(cum, total, u):
    """The smallest t with cum[t] > u * total, exactly (u an fp32 number: a whole number of 2^-24 over [0, 1))."""
    n = int(float(u) * 2 ** 48)
    assert n == float(u) * 2 ** 48
    want = n * total
    lo, hi = 0, len(cum) - 1
    while lo < hi:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if (int(cum[mid]) << 48) > want else (mid + 1, hi)
    return lo


@pytest.mark.parametrize("B", [3, 200])                         # clusters of CTAs, and more requests than SMs
@pytest.mark.parametrize("V", [131072, 130999])
@pytest.mark.parametrize("drafts", [True, False])
def test_sums_of_a_flat_tail(msa, V, B, drafts):
    """A likely token was drafted and rejected: the flat tail behind it is all that is left, and the next token's
    border is placed a small part of a token's share away from a token's end."""
    head = 777
    row, units, total = _flat_tail(V, head, 2.0 ** -23, 1.1920e-7)
    cum = units.cumsum(0)
    g = torch.Generator().manual_seed(101)
    # borders half a hundredth of a share and more away from a token's end, on both sides
    ends = torch.randint(V // 8, V // 2 - 2, (B,), generator=g)
    share = cum[ends].double() / total
    u = (share + torch.where(torch.arange(B) % 2 == 0, 1.0, -1.0) * 2.0 ** -17 / 40).float()
    want = [_border(cum, total, x) for x in u]
    tok = torch.tensor([0, head], dtype=torch.int32).repeat(B)
    ua = torch.tensor([0.0, 1 - 2.0 ** -24]).repeat(B)
    off = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device=DEV)
    par = torch.tensor([-1, 0], dtype=torch.int32, device=DEV).repeat(B)
    P = row.to(DEV).expand(2 * B, V).contiguous()
    Q = None
    if drafts:
        Q = torch.zeros(V)
        Q[head] = 1.0
        Q = Q.to(DEV).expand(2 * B, V).contiguous()
    err = msa.new_err_word(DEV)
    path, acc, nxt = msa.msa_verify_tree(P, Q, tok.to(DEV), off, par, ua.to(DEV), u.to(DEV), err_word=err)
    msa.msa_check(err)
    assert acc.tolist() == [1] * B
    assert nxt.tolist() == want


@pytest.mark.parametrize("B", [4, 200])
def test_mass_of_a_flat_tail(msa, B):
    """The second child is held to the mass of that tail: accepted just below the border, rejected just above it."""
    V, head, tok = 131072, 5, 100000
    row, units, total = _flat_tail(V, head, 2.0 ** -23, 1.1920e-7)
    mass = total * 2.0 ** -60                                   # of the residual once the head is rejected, but for q
    q = torch.zeros(V)
    q[head] = 1.0
    q[tok] = float(row[tok]) / (1 + mass / 2)                   # r(tok) is about half of mass * q(tok)
    qt = int(float(q[tok].double() * 2.0 ** 60))
    left, rest = int(units[tok]) - qt, total - qt               # whole numbers of 2^-60: r(tok) and M
    border = left * 2 ** 60 / (qt * rest)
    assert 0.4 < border < 0.6
    u0 = torch.tensor([border], dtype=torch.float64).float()
    step = 2.0 ** -24                                           # fp32 numbers in [0.5, 1); half of it below
    u = torch.stack([u0 + k * step for k in (-3, -2, 2, 3)]).flatten().repeat(B // 4)
    want = [2 if int(float(x) * 2 ** 48) * qt * rest < left << 108 else 1 for x in u]
    assert sorted(set(want)) == [1, 2]
    off = torch.arange(0, 3 * B + 1, 3, dtype=torch.int32, device=DEV)
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device=DEV).repeat(B)
    toks = torch.tensor([0, head, tok], dtype=torch.int32, device=DEV).repeat(B)
    ua = torch.stack([torch.zeros(B), torch.full((B,), 1 - 2.0 ** -24), u], 1).flatten().to(DEV)
    P, Q = row.to(DEV).expand(3 * B, V).contiguous(), q.to(DEV).expand(3 * B, V).contiguous()
    err = msa.new_err_word(DEV)
    path, acc, _ = msa.msa_verify_tree(P, Q, toks, off, par, ua, torch.full((B,), 0.5, device=DEV), err_word=err)
    msa.msa_check(err)
    assert acc.tolist() == want
    assert path.view(B, 3)[:, 1].tolist() == [2 if w == 2 else -1 for w in want]


@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** -20])
def test_next_token_of_rows_of_any_mass(msa, scale):
    """Weights that do not sum to one: the next token goes by their share all the same."""
    V, B = 5003, 64
    g = torch.Generator().manual_seed(102)
    w = torch.randint(1, 2 ** 20, (V,), generator=g)
    row = (w.double() * 2.0 ** -20 * scale).float()             # exact
    cum = w.cumsum(0)
    u = torch.rand(B, generator=g)
    # a border between two tokens, from either side
    ends = torch.randint(V // 8, V, (B,), generator=g)
    near = cum[ends].double() / int(cum[-1])
    u[::2] = (near + torch.where(torch.arange(B) % 4 == 0, 1.0, -1.0) * 2.0 ** -23).clamp(max=1 - 2.0 ** -24).float()[::2]
    want = [_border(cum, int(cum[-1]), x) for x in u]
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    par = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    zero = torch.zeros(B, device=DEV)
    err = msa.new_err_word(DEV)
    _, acc, nxt = msa.msa_verify_tree(row.to(DEV).expand(B, V).contiguous(), None, par * 0, off, par, zero, u.to(DEV),
                                      err_word=err)
    msa.msa_check(err)
    assert acc.tolist() == [1] * B and nxt.tolist() == want


# ------------------------------------------------------------------ attention: values that are not finite, next to no weight

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("nodes,ctx", [(3, 256), (3, 512), (3, 1024), (3, 2048), (40, 2048)])
def test_seen_nonfinite_values_of_no_weight(msa, bad, nodes, ctx):
    """A value that is not finite reaches the rows that see it, however little its token weighs, whether or not the
    token's block and the heavy one fall to the same range of work."""
    t = T.make_tree([ctx], [nodes], 103, "star")
    x = _inputs(t, 8, 1, 128, 104)
    q, kc, vc = x[:3]
    q[..., 0] = 8.0
    kc[..., 0] = 0.0
    x[3][..., 0] = 0.0
    kc[int(t.block_table[0, ctx // 128 - 1]), 60, :, 0] = 160.0   # 113 above the others: e^-113 is 0 in 32 bits
    vc[int(t.block_table[0, 0]), 3, 0, 7] = bad
    sel = torch.arange(16, dtype=torch.int32).repeat(nodes, 1, 1)
    sel[sel >= ctx // 128] = -1
    sel[1, :, 0] = -1                                             # node 1 does not see it
    out, lse = _attend(msa, t, msa.Dims(8, 1, 128, 64, 16, t.max_blocks), x, sel)
    hit = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(hit)
    want[:, :, 7] = True
    want[1] = False
    assert torch.equal(hit, want) and bool(torch.isfinite(lse).all())


# ------------------------------------------------------------------ layouts that are refused

@pytest.mark.parametrize("off,good", [
    ([1, 5, 9], (5, 9)),            # does not begin at 0
    ([7, 5, 9], (5, 9)),
    ([0, 12, 9], ()),               # past the rows, then down
    ([0, 5, 10], (0, 5)),           # past the rows
    ([0, 5, 3], (0, 5)),            # down
    ([-3, 5, 9], (5, 9)),           # below 0
    ([0, -2, 4], ()),
    ([2, 2, 2], ()),                # no node at all, but rows before the first request
    ([20, 30, 40], ()),
    ([-3, -3, -3], ()),
    ([0, 5, 12, 9], (0, 5)),        # past the rows, then down, behind a good one
])
def test_every_row_of_a_bad_layout_is_written(msa, off, good):
    """Rows that a bad node_off leaves to no good request are padding, whatever the buffers held: the calls that follow
    read them."""
    ctx = [10, 20, 30][:len(off) - 1]
    old = [torch.full((9,), 77, dtype=d, device=DEV) for d in (torch.int32, torch.int32, torch.int64)]
    par = torch.arange(9, dtype=torch.int32) - 1 - (good[0] if good else 0)
    if good:
        par[good[0]] = -1
    err = msa.new_err_word(DEV)
    q_req, q_pos, anc = msa.msa_tree_rows(torch.tensor(off, dtype=torch.int32, device=DEV), par.to(DEV),
                                          torch.tensor(ctx, dtype=torch.int32, device=DEV),
                                          msa.Dims(16, 2, 128, 64, 4, 3), *old, err_word=err)
    with pytest.raises(msa.MsaError, match="BOUNDS"):
        msa.msa_check(err)
    b = off.index(good[0]) if good else 0
    for r in range(9):
        mine = bool(good) and good[0] <= r < good[1]
        k = r - good[0] if mine else 0
        assert int(q_req[r]) == (b if mine else -1), r
        assert int(q_pos[r]) == (ctx[b] + k if mine else 0), r
        assert int(anc[r]) == ((2 << k) - 1 if mine else 0), r


def test_a_refused_request_among_many(msa):
    """One request with too many nodes in the middle of 40,000 rows, and padding behind the last."""
    counts = [40] * 1000
    counts[819] = 70                                             # rows 32,760 to 32,829
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    R = off[-1] + 100
    node = torch.cat([torch.arange(n) for n in counts] + [torch.zeros(100, dtype=torch.long)])
    req = torch.cat([torch.full((n,), b) for b, n in enumerate(counts)] + [torch.full((100,), -1)])
    req[off[819]:off[820]] = -1
    old = [torch.full((R,), 77, dtype=d, device=DEV) for d in (torch.int32, torch.int32, torch.int64)]
    err = msa.new_err_word(DEV)
    q_req, q_pos, anc = msa.msa_tree_rows(torch.tensor(off, dtype=torch.int32, device=DEV), (node - 1).int().to(DEV),
                                          torch.arange(1000, dtype=torch.int32, device=DEV),
                                          msa.Dims(16, 2, 128, 64, 4, 9), *old, err_word=err)
    with pytest.raises(msa.MsaError, match="UNSUPPORTED"):
        msa.msa_check(err)
    live = req >= 0
    assert torch.equal(q_req.cpu().long(), req)
    assert torch.equal(q_pos.cpu().long(), torch.where(live, req + node, 0))
    assert torch.equal(anc.cpu(), torch.where(live, (2 << node.clamp(max=61)) - 1, 0))


# ------------------------------------------------------------------ a step against a sequential decode, to the rounding

def test_tree_step_and_decode_within_the_rounding(msa):
    """The attention of every accepted node, from the tree and from decoding its path token by token, lies within the
    roundings of the 64-bit result over the selection that both made; a reference without one drafted token on the
    path, or with another value for it, does not."""
    t = T.make_tree([700, 250, 0, 126], [9, 20, 4, 12], 105, extra_blocks=1)
    Hq, G, D, Di, topk = 16, 2, 128, 64, 4
    dims = msa.Dims(Hq, G, D, Di, topk, t.max_blocks)
    q, kc, vc, kn, vn = _inputs(t, Hq, G, D, 106)
    qi, ic, ixn = T.bf16((t.n_rows, G, Di), 111), T.bf16((t.n_pages, 128, G, Di), 112), T.bf16((t.n_rows, G, Di), 113)
    off, par, ctx, bt, _ = t.dev(DEV)
    step = msa.TreeStep(dims, t.n_rows, 4, DEV)
    step.layout(off, par, ctx)
    dev = [v.to(DEV) for v in (kn, vn, ixn, kc, vc, ic)]
    out, lse = step.attend(q.to(DEV), qi.to(DEV), *dev, bt)
    msa.msa_check(step.err)
    sel = step.sel.cpu()
    x = [q, kc, vc, kn, vn]
    _check(t, out, lse, x, sel, D)
    # the deepest path of each tree, appended and decoded token by token
    ro, rl, bo, bl = T.ref_attend(t, *x, sel, D ** -0.5)
    dec = msa.DecodeStep(dims, 1, 1, t.n_pages, DEV)
    nodes = []
    for b in range(4):
        best = max(t.rows(b), key=lambda r: t.depth[r])
        rows = [r for r in t.rows(b) if t.anc[best] >> (r - t.off[b]) & 1]
        nodes += rows[-1:] if len(rows) > 2 else []
        for k, r in enumerate(rows):
            page, at = int(t.block_table[b, (t.ctx[b] + k) // 128]), (t.ctx[b] + k) % 128
            for c, n in zip(dev[3:], dev[:3]):
                c[page, at] = n[r]
            n = torch.tensor([t.ctx[b] + k + 1], dtype=torch.int32, device=DEV)
            o, s = dec(q[r:r + 1].to(DEV), qi[r:r + 1].to(DEV), *dev[3:], bt[b:b + 1].contiguous(), n)
            msa.msa_check(dec.err)
            assert torch.equal(dec.sel[0].cpu(), sel[r])
            T.assert_within(o[0], ro[r], bo[r], "decoded out")
            T.assert_within(s[0], rl[r], bl[r], "decoded lse")
    # mistakes planted in the reference
    assert len(nodes) >= 3
    for what in ("dropped", "value"):
        for r in nodes:
            b = t.q_req()[r]
            up = t.off[b] + t.parents[r]
            bad = T.Tree(t.off, t.parents, t.ctx, t.depth, list(t.anc), t.block_table, t.n_pages)
            vn2 = vn.clone()
            if what == "dropped":
                bad.anc[r] &= ~(1 << t.parents[r])
            else:
                vn2[up] += 1
            o2, l2, _, _ = T.ref_attend(bad, q, kc, vc, kn, vn2, sel, D ** -0.5)
            miss = (out[r].cpu().double() - o2[r]).abs() > bo[r]
            assert bool(miss.any()), (what, r)


# ------------------------------------------------------------------ attention: the order of a tile's nodes

def _inherited(n, G, full, seed, changed):
    """15 blocks a node: seven that all nodes have, and eight of its parent's, `changed` of them new."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda k: int(torch.randint(k, (1,), generator=g))
    sel = []
    for _ in range(G):
        ids = torch.randperm(full, generator=g).tolist()
        core, rest, own = ids[:7], ids[7:], []
        for i in range(n):
            s = list(own[i - 1]) if i else rest[:8]
            for _ in range(changed if i else 0):
                s[rnd(8)] = [j for j in rest if j not in s][rnd(len(rest) - 8)]
            own.append(s)
        sel.append([sorted(core + s) for s in own])
    return torch.tensor(sel, dtype=torch.int32).permute(1, 0, 2)


def _windows(n, G, full, seed):
    """The same, but of eight blocks one after another in a pool of 96: nodes twelve apart have the same."""
    g = torch.Generator().manual_seed(seed)
    sel = []
    for _ in range(G):
        ids = torch.randperm(full, generator=g).tolist()
        sel.append([sorted(ids[:7] + [ids[7 + (8 * i + k) % 80] for k in range(8)]) for i in range(n)])
    return torch.tensor(sel, dtype=torch.int32).permute(1, 0, 2)


@pytest.mark.parametrize("pattern", ["inherited", "inherited_2", "windows"])
def test_nodes_keep_their_order_where_it_reads_less(msa, pattern):
    """A tile reads the blocks that any of its 32 nodes selected.  Where a child keeps most of its parent's blocks the
    tree's own order makes the smaller tiles, where like nodes lie far apart another one does; the plan's tiles are
    never larger than those of the tree's own order."""
    n, G, Hq, D = 64, 2, 16, 128
    t = T.make_tree([12000, 11990], [n, n], 107, "chain")
    full = 93
    both = [_windows(n, G, full, 108 + b) if pattern == "windows" else
            _inherited(n, G, full, 108 + b, 2 if pattern == "inherited_2" else 1) for b in range(2)]
    sel = torch.full((2 * n, G, 16), -1, dtype=torch.int32)
    sel[:, :, :15] = torch.cat(both)
    sel[:, :, 15] = (torch.tensor(t.q_pos()) // 128)[:, None]
    x = _inputs(t, Hq, G, D, 109)
    dims = msa.Dims(Hq, G, D, 64, 16, t.max_blocks)
    ws = torch.empty(msa.msa_workspace_bytes(msa.MSA_OP_TREE, 2 * n, 2, dims), dtype=torch.uint8, device=DEV)
    off, _, ctx, bt, anc = t.dev(DEV)
    err = msa.new_err_word(DEV)
    out, lse = msa.msa_sparse_attn_tree(*[v.to(DEV) for v in x], bt, ctx, off, anc, sel.to(DEV), dims, workspace=ws,
                                        err_word=err)
    msa.msa_check(err)
    _check(t, out, lse, x, sel, D)
    # the plan's records: a tile's items in the first word, 2^30 for the item of the drafted tokens
    tiles = 2 * 2 * G
    items = ws[:16 * tiles].view(torch.int32).view(tiles, 4)[:, 0].cpu()
    assert bool((items >> 30 == 1).all())
    blocks = (items & (1 << 30) - 1) - 1
    own = sum(len({int(j) for j in sel[r0:r0 + 32, g].flatten() if 0 <= int(j) * 128 < t.ctx[r0 // n]})
              for r0 in range(0, 2 * n, 32) for g in range(G))
    assert int(blocks.sum()) < own if pattern == "windows" else int(blocks.sum()) <= own


@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("counts", [[17, 31], [33, 16], [40, 63], [48, 1]])
def test_wide_trees_in_their_own_order(msa, counts, Hq, G, D):
    """Selections that follow the tree, at sizes that leave a tile's second half or a second tile partly filled; the
    rows behind each tree belong to the next one, or are padding full of NaN."""
    t = T.make_tree([2900, 2950], counts, 110, "chain")
    full = 22
    sel = torch.cat([_inherited(n, G, full, 111 + b, 1) for b, n in enumerate(counts)])
    own = (torch.tensor(t.q_pos()) // 128)[:, None, None].expand(-1, G, 1).int()
    sel = torch.cat([sel, own], -1).contiguous()
    x = _inputs(t, Hq, G, D, 112)
    pad = 9
    wide = [torch.cat([v, torch.full((pad, *v.shape[1:]), float("nan"), dtype=v.dtype)]) if i in (0, 3, 4) else v
            for i, v in enumerate(x)]
    off, _, ctx, bt, anc = t.dev(DEV, pad)
    err = msa.new_err_word(DEV)
    out, lse = msa.msa_sparse_attn_tree(*[v.to(DEV) for v in wide], bt, ctx, off, anc,
                                        torch.cat([sel, torch.full((pad, G, 16), -1, dtype=torch.int32)]).to(DEV),
                                        msa.Dims(Hq, G, D, 64, 16, t.max_blocks), err_word=err)
    msa.msa_check(err)
    _check(t, out[:t.n_rows], lse[:t.n_rows], x, sel, D)
