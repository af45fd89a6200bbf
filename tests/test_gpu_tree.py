"""Drafted trees on the GPU: layout, scoring, attention, verification and commit against plain references in 64
bits, at the sizes and masks where they can go wrong, and one speculative step against a sequential decode."""
import pytest
import torch

from tests import _tree as T

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def msa():
    import block_sparse_attention_06_gb300 as m
    return m


def _dims(msa, t, Hq=16, G=2, D=128, Di=64, topk=4):
    return msa.Dims(Hq, G, D, Di, topk, t.max_blocks)


# ------------------------------------------------------------------ layout

@pytest.mark.parametrize("ctx,counts,shape,pad", [
    ([0], [1], "chain", 0),
    ([5, 0, 700], [64, 1, 17], "random", 0),
    ([127, 128, 129], [64, 64, 64], "chain", 5),
    ([10, 20, 30, 40], [3, 0, 0, 9], "star", 70),
    ([2 ** 20], [33], "random", 1),
])
def test_tree_rows(msa, ctx, counts, shape, pad):
    t = T.make_tree(ctx, counts, 3, shape)
    off, par, ctxd, _, _ = t.dev(DEV, pad)
    err = msa.new_err_word(DEV)
    q_req, q_pos, anc = msa.msa_tree_rows(off, par, ctxd, _dims(msa, t), err_word=err)
    msa.msa_check(err)
    assert q_req.tolist() == t.q_req() + [-1] * pad
    assert q_pos.tolist() == t.q_pos() + [0] * pad
    assert anc.tolist() == T.signed(t.anc) + [0] * pad


@pytest.mark.parametrize("what", ["parent_ahead", "parent_self", "second_root", "no_root", "off_down", "off_past",
                                  "off_start", "ctx_negative", "past_end", "too_many"])
def test_tree_rows_flags_bad_layouts(msa, what):
    counts = [5, 65 if what == "too_many" else 4]
    t = T.make_tree([10, 20], counts, 4, "chain")
    off, par, ctx, _, _ = t.dev(DEV)
    dims = _dims(msa, t)
    if what == "parent_ahead":
        par[5 + 2] = 3
    elif what == "parent_self":
        par[5 + 2] = 2
    elif what == "second_root":
        par[5 + 2] = -1
    elif what == "no_root":
        par[5] = 0
    elif what == "off_down":
        off[1] = 12
    elif what == "off_past":
        off[2] = 10
    elif what == "off_start":
        off[0] = 1
    elif what == "ctx_negative":
        ctx[1] = -1
    elif what == "past_end":
        ctx[1] = t.max_blocks * 128 - 3
    err = msa.new_err_word(DEV)
    q_req, q_pos, anc = msa.msa_tree_rows(off, par, ctx, dims, err_word=err)
    with pytest.raises(msa.MsaError, match="UNSUPPORTED" if what == "too_many" else "BOUNDS"):
        msa.msa_check(err)
    if what not in ("off_down", "off_past", "off_start"):   # the good request is unharmed, the bad one padding
        assert q_req.tolist()[:5] == [0] * 5 and anc.tolist()[:5] == t.anc[:5]
        assert q_req.tolist()[5:] == [-1] * counts[1] and anc.tolist()[5:] == [0] * counts[1]


# ------------------------------------------------------------------ scores

SHAPES = [
    ([0], [1], "chain"),                               # nothing cached
    ([1], [1], "chain"),
    ([0, 3], [64, 40], "chain"),                       # nothing cached, the widest trees
    ([127, 128, 129], [16, 17, 15], "random"),         # around a block's edge
    ([100, 250, 640], [64, 33, 8], "chain"),           # paths that cross into the next block
    ([1000, 0, 2049, 300], [5, 0, 64, 1], "random"),   # a request without nodes, one n-tile to four
    ([383], [7], "star"),
]


@pytest.mark.parametrize("G,Di", [(8, 64), (2, 32), (16, 64), (1, 64)])
@pytest.mark.parametrize("ctx,counts,shape", SHAPES)
def test_tree_scores(msa, ctx, counts, shape, G, Di):
    t = T.make_tree(ctx, counts, 11, shape, extra_blocks=2)
    pad = 3
    q, kn = T.bf16((t.n_rows + pad, G, Di), 1), T.bf16((t.n_rows + pad, G, Di), 2)
    kidx = T.bf16((t.n_pages, 128, G, Di), 3)
    # nothing behind a context's end, no padding row is seen
    for b, c in enumerate(ctx):
        if c % 128:
            kidx[int(t.block_table[b, c // 128]), c % 128:] = float("inf")
    kn[t.n_rows:] = float("inf")
    off, _, ctxd, bt, anc = t.dev(DEV, pad)
    dims = _dims(msa, t, 8 * G, G, 128, Di)
    err = msa.new_err_word(DEV)
    scores = torch.full((t.n_rows + pad, G, t.max_blocks), 77.0, device=DEV)
    msa.msa_tree_index_score(q.to(DEV), kidx.to(DEV), kn.to(DEV), bt, ctxd, off, anc, dims, scores, err_word=err)
    msa.msa_check(err)
    want, tol = T.ref_scores(t, q[:t.n_rows], kidx, kn[:t.n_rows])
    T.assert_within(scores[:t.n_rows], want, tol, "scores")
    assert bool((scores[t.n_rows:] == 77.0).all()), "padding rows were written"


@pytest.mark.parametrize("G,Di", [(1, 64), (2, 32), (4, 64), (16, 64)])
def test_tree_scores_many_requests(msa, G, Di):
    """Requests of one block or none, several to a range of work, so that a CTA changes its queries often."""
    B = 700
    t = T.make_tree([(37 * b) % 150 for b in range(B)], [(7 * b) % 5 for b in range(B)], 12)
    q, kn = T.bf16((t.n_rows, G, Di), 1), T.bf16((t.n_rows, G, Di), 2)
    kidx = T.bf16((t.n_pages, 128, G, Di), 3)
    off, _, ctxd, bt, anc = t.dev(DEV)
    err = msa.new_err_word(DEV)
    want, tol = T.ref_scores(t, q, kidx, kn)
    q, kn, kidx = q.to(DEV), kn.to(DEV), kidx.to(DEV)
    for _ in range(3):
        scores = msa.msa_tree_index_score(q, kidx, kn, bt, ctxd, off, anc, _dims(msa, t, 8 * G, G, 128, Di),
                                          err_word=err)
        msa.msa_check(err)
        T.assert_within(scores, want, tol, "scores")


def test_tree_scores_flag_bad_page(msa):
    t = T.make_tree([300], [4], 5)
    off, _, ctxd, bt, anc = t.dev(DEV)
    dims = _dims(msa, t)
    q, kn = T.bf16((4, 2, 64), 1).to(DEV), T.bf16((4, 2, 64), 2).to(DEV)
    kidx = T.bf16((t.n_pages, 128, 2, 64), 3).to(DEV)
    for bad in (-1, t.n_pages):
        bt2 = bt.clone()
        bt2[0, 1] = bad
        err = msa.new_err_word(DEV)
        msa.msa_tree_index_score(q, kidx, kn, bt2, ctxd, off, anc, dims, err_word=err)
        with pytest.raises(msa.MsaError, match="BOUNDS"):
            msa.msa_check(err)


# ------------------------------------------------------------------ attention

def _attn_inputs(t, Hq, G, D, seed, pad=0):
    R = t.n_rows + pad
    return (T.bf16((R, Hq, D), seed), T.bf16((t.n_pages, 128, G, D), seed + 1), T.bf16((t.n_pages, 128, G, D), seed + 2),
            T.bf16((R, G, D), seed + 3), T.bf16((R, G, D), seed + 4))


def _attend(msa, t, dims, q, kc, vc, kn, vn, sel, pad=0, out=None, lse=None, ws=None):
    off, _, ctxd, bt, anc = t.dev(DEV, pad)
    if pad:
        sel = torch.cat([sel, torch.full((pad, *sel.shape[1:]), 1 << 30, dtype=torch.int32)])
    err = msa.new_err_word(DEV)
    out, lse = msa.msa_sparse_attn_tree(q.to(DEV), kc.to(DEV), vc.to(DEV), kn.to(DEV), vn.to(DEV), bt, ctxd, off, anc,
                                        sel.to(DEV), dims, out, lse, ws, err_word=err)
    msa.msa_check(err)
    return out, lse


def _check_attend(t, out, lse, q, kc, vc, kn, vn, sel, D, scale=None):
    n = t.n_rows
    ro, rl, bo, bl = T.ref_attend(t, q[:n], kc, vc, kn[:n], vn[:n], sel[:n], scale or D ** -0.5)
    T.assert_within(lse[:n], rl, bl, "lse")
    T.assert_within(out[:n], ro, bo, "out")


@pytest.mark.parametrize("Hq,G,D,topk", [(16, 2, 128, 4), (8, 2, 64, 3), (16, 2, 64, 1), (4, 1, 128, 32)])
@pytest.mark.parametrize("ctx,counts,shape", SHAPES)
def test_tree_attention(msa, ctx, counts, shape, Hq, G, D, topk):
    t = T.make_tree(ctx, counts, 21, shape, extra_blocks=1)
    x = _attn_inputs(t, Hq, G, D, 31, pad=2)
    sel = T.random_sel(t, G, topk, 41)
    out = torch.full((t.n_rows + 2, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((t.n_rows + 2, Hq), 7.0, device=DEV)
    _attend(msa, t, _dims(msa, t, Hq, G, D, 64, topk), *x, sel, pad=2, out=out, lse=lse)
    _check_attend(t, out, lse, *x, sel, D)
    assert bool((out[t.n_rows:] == 7).all()) and bool((lse[t.n_rows:] == 7).all()), "padding rows were written"


@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (8, 2, 64)])
def test_tree_attention_long_context(msa, Hq, G, D):
    """Rows that agree on most blocks and rows that share none; the union runs over several ranges of work."""
    t = T.make_tree([20000, 9000, 131], [40, 64, 2], 22)
    x = _attn_inputs(t, Hq, G, D, 32)
    sel = T.random_sel(t, G, 16, 42, drop_own=0.0, empty=0.02)
    sel[:t.off[1]:2] = sel[0]      # every other row of the first tree: one selection
    out, lse = _attend(msa, t, _dims(msa, t, Hq, G, D, 64, 16), *x, sel)
    _check_attend(t, out, lse, *x, sel, D)


def test_tree_attention_many_requests(msa):
    """More tiles than SMs, of every size from nothing on."""
    counts = [(7 * b) % 20 for b in range(90)]
    t = T.make_tree([(37 * b) % 600 for b in range(90)], counts, 23)
    x = _attn_inputs(t, 16, 2, 64, 33)
    sel = T.random_sel(t, 2, 4, 43)
    out, lse = _attend(msa, t, _dims(msa, t, 16, 2, 64, 64, 4), *x, sel)
    _check_attend(t, out, lse, *x, sel, 64)


def test_tree_attention_large_logits(msa):
    """Logits far apart within a row, growing along the context: the running maximum rises block after block."""
    t = T.make_tree([1500], [20], 24, "random")
    q, kc, vc, kn, vn = _attn_inputs(t, 16, 2, 128, 34)
    pos = torch.zeros(t.n_pages, dtype=torch.float32)
    for j in range(12):
        pos[int(t.block_table[0, j])] = j
    kc = (kc.float() * (1 + pos)[:, None, None, None]).to(torch.bfloat16)
    sel = T.random_sel(t, 2, 12, 44, drop_own=0.0, empty=0.0)
    dims = _dims(msa, t, 16, 2, 128, 64, 12)
    out, lse = _attend(msa, t, dims, q, kc, vc, kn, vn, sel)
    _check_attend(t, out, lse, q, kc, vc, kn, vn, sel, 128)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (8, 2, 64)])
def test_tree_attention_unseen_values(msa, bad, Hq, G, D):
    """Page tails, padding rows, other branches, and blocks that only other rows selected hold NaN or infinities:
    the rows that do not see them come out as if they held zeros."""
    t = T.make_tree([300, 700], [10, 12], 25, "star")
    pad = 60
    q, kc, vc, kn, vn = _attn_inputs(t, Hq, G, D, 35, pad)
    sel = T.random_sel(t, G, 4, 45, drop_own=0.0, empty=0.0)
    # block 1 of request 1: selected by row 3 of it alone; the leaf 5 of request 0: seen by itself alone
    lone, leaf = t.off[1] + 3, t.off[0] + 5
    for r in t.rows(1):
        for g in range(G):
            own = int(t.q_pos()[r]) // 128
            sel[r, g] = torch.tensor(sorted({0, 2, 3, own})[:4] if r != lone else [1, 2, own, -1][:4], dtype=torch.int32)
    clean = [x.clone() for x in (kc, vc, kn, vn)]
    page = int(t.block_table[1, 1])
    vc[page, 5, :, 3] = bad
    kc[page, 77] = bad
    kn[leaf], vn[leaf] = bad, bad
    for b, c in enumerate(t.ctx):
        tail = int(t.block_table[b, c // 128])
        kc[tail, c % 128:], vc[tail, c % 128:] = bad, bad
    q[t.n_rows:], kn[t.n_rows:], vn[t.n_rows:] = bad, bad, bad
    dims = _dims(msa, t, Hq, G, D, 64, 4)
    out, lse = _attend(msa, t, dims, q, kc, vc, kn, vn, sel, pad=pad)
    keep = [r for r in range(t.n_rows) if r not in (lone, leaf)]
    ro, rl, bo, bl = T.ref_attend(t, q[:t.n_rows], *[c for c in clean[:2]], clean[2][:t.n_rows], clean[3][:t.n_rows], sel,
                                  D ** -0.5)
    T.assert_within(lse[keep], rl[keep], bl[keep], "lse")
    T.assert_within(out[keep], ro[keep], bo[keep], "out")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_attention_seen_nonfinite_values(msa, bad):
    """A NaN or infinity in a value that a row does see reaches that row's column, and only it."""
    t = T.make_tree([300], [6], 26, "star")
    q, kc, vc, kn, vn = _attn_inputs(t, 16, 2, 128, 36)
    sel = torch.tensor([0, 1, 2, -1], dtype=torch.int32).expand(6, 2, 4).contiguous()
    sel[2] = torch.tensor([0, 2, -1, -1], dtype=torch.int32)
    vc[int(t.block_table[0, 1]), 9, 0, 17] = bad
    vn[4, 1, 100] = bad
    out, _ = _attend(msa, t, _dims(msa, t), q, kc, vc, kn, vn, sel)
    want = torch.zeros((6, 16, 128), dtype=torch.bool)
    want[[0, 1, 3, 4, 5], :8, 17] = True
    want[4, 8:, 100] = True
    got = out.cpu()
    hit = torch.isnan(got) | torch.isinf(got)
    assert torch.equal(hit, want)


def test_tree_attention_flags(msa):
    t = T.make_tree([300], [4], 27)
    x = [v.to(DEV) for v in _attn_inputs(t, 16, 2, 128, 37)]
    off, _, ctxd, bt, anc = t.dev(DEV)
    dims = _dims(msa, t)
    sel = torch.tensor([0, 1, 2, -1], dtype=torch.int32, device=DEV).expand(4, 2, 4).contiguous()
    for what in ("page", "page_high", "block", "ctx"):
        bt2, sel2, ctx2 = bt.clone(), sel.clone(), ctxd.clone()
        if what == "page":
            bt2[0, 1] = -1
        elif what == "page_high":
            bt2[0, 1] = t.n_pages
        elif what == "block":
            sel2[3, 1, 2] = t.max_blocks
        else:
            ctx2[0] = -1
        err = msa.new_err_word(DEV)
        msa.msa_sparse_attn_tree(*x, bt2, ctx2, off, anc, sel2, dims, err_word=err)
        with pytest.raises(msa.MsaError, match="BOUNDS"):
            msa.msa_check(err)
    # an unread table entry (a block past the cached tokens) is not an error
    bt2 = bt.clone()
    t2 = T.make_tree([256], [4], 27)
    x2 = [v.to(DEV) for v in _attn_inputs(t2, 16, 2, 128, 37)]
    off, _, ctxd, bt, anc = t2.dev(DEV)
    bt[0, 2] = -1
    err = msa.new_err_word(DEV)
    msa.msa_sparse_attn_tree(*x2, bt, ctxd, off, anc, sel, _dims(msa, t2), err_word=err)
    msa.msa_check(err)


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 32000, 131071])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("shape", ["random", "chain", "star"])
def test_verify(msa, vocab, drafts, shape):
    counts = [1, 8, 0, 17, 3] if vocab > 50000 else [1, 8, 0, 64, 3, 30, 2]
    t = T.make_tree([0] * len(counts), counts, 51, shape)
    for seed in range(4):
        # drafts close to the target, and drafts far from it (many rejections)
        x = T.verify_inputs(t, vocab, 61 + seed, drafts, sharp=2.5, noise=(0.3, 3.0)[seed % 2])
        off, par, _, _, _ = t.dev(DEV)
        p, q, tok, ua, un = x
        err = msa.new_err_word(DEV)
        got = msa.msa_verify_tree(p.to(DEV), None if q is None else q.to(DEV), tok.to(DEV), off, par, ua.to(DEV),
                                  un.to(DEV), err_word=err)
        msa.msa_check(err)
        want = T.ref_verify(t, *x)
        for g, w, name in zip(got, want, ("path", "n_accepted", "next_token")):
            assert torch.equal(g.cpu(), w), (name, g.tolist(), w.tolist())


def test_verify_follows_the_target(msa):
    """The emitted first token has the target's distribution: 20,000 trees of three sampled children each."""
    vocab, n = 11, 20000
    g = torch.Generator().manual_seed(5)
    p, q = (torch.softmax(torch.randn(vocab, generator=g), -1) for _ in range(2))
    kids = torch.multinomial(q, 3 * n, replacement=True, generator=g).view(n, 3).int()
    tokens = torch.cat([torch.zeros((n, 1), dtype=torch.int32), kids], 1).reshape(-1).to(DEV)
    off = torch.arange(0, 4 * n + 1, 4, dtype=torch.int32, device=DEV)
    par = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device=DEV).repeat(n)
    P, Q = p.to(DEV).repeat(4 * n, 1), q.to(DEV).repeat(4 * n, 1)
    ua, un = torch.rand(4 * n, generator=g).to(DEV), torch.rand(n, generator=g).to(DEV)
    err = msa.new_err_word(DEV)
    path, acc, nxt = msa.msa_verify_tree(P, Q, tokens, off, par, ua, un, err_word=err)
    msa.msa_check(err)
    path, acc = path.view(n, 4).long(), acc.long()
    first = torch.where(acc > 1, tokens.view(n, 4).gather(1, path[:, 1:2].clamp(min=0))[:, 0], nxt)
    freq = torch.bincount(first.long().cpu(), minlength=vocab).double() / n
    # six standard deviations of a frequency over n independent draws
    assert bool(((freq - p.double()).abs() <= 6 * (p.double() * (1 - p.double()) / n).sqrt()).all())


def test_verify_edges(msa):
    """u at both ends of [0, 1), a target without the drafted token, equal distributions, one-hot targets."""
    t = T.make_tree([0] * 6, [3] * 6, 52, "star")
    V = 257
    p, q, tok, ua, un = T.verify_inputs(t, V, 71, True)
    top = 1 - 2.0 ** -24
    ua[:], un[:] = top, top
    un[0] = 0.0
    p[t.off[1]] = q[t.off[1]]                                     # accepted whatever u
    p[t.off[2], tok[t.off[2] + 1:t.off[2] + 3].long()] = 0.0      # rejected whatever u
    ua[t.off[2]:t.off[3]] = 0.0
    p[t.off[3]] = 0.0
    p[t.off[3], 200] = 1.0
    p[t.off[4]], un[4] = p[t.off[4]] * 0, 0.5
    p[t.off[4], 0] = 1.0
    q[t.off[4]] = p[t.off[4]]                                     # residual empty after a rejection: p again
    tok[t.off[4] + 1:t.off[4] + 3] = 5
    x = (p, q, tok, ua, un)
    off, par, _, _, _ = t.dev(DEV)
    err = msa.new_err_word(DEV)
    got = msa.msa_verify_tree(*[v.to(DEV) for v in (p, q, tok)], off, par, ua.to(DEV), un.to(DEV), err_word=err)
    msa.msa_check(err)
    want = T.ref_verify(t, *x)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w), (g.tolist(), w.tolist())
    assert int(got[2][4]) == 0 and int(got[2][3]) == 200 and int(got[1][1]) == 2


def test_verify_flags(msa):
    t = T.make_tree([0, 0], [3, 3], 53, "chain")
    p, q, tok, ua, un = [v.to(DEV) for v in T.verify_inputs(t, 100, 72, True)]
    off, par, _, _, _ = t.dev(DEV)
    for what in ("token", "token_low", "parent", "mass", "infinite"):
        p2, tok2, par2 = p.clone(), tok.clone(), par.clone()
        if what == "token":
            tok2[4] = 100
        elif what == "token_low":
            tok2[4] = -1
        elif what == "parent":
            par2[4] = 2
        elif what == "mass":
            p2[3:] = 0
        else:
            p2[3:, 7] = float("inf")
            tok2[4:] = 8
        err = msa.new_err_word(DEV)
        path, acc, nxt = msa.msa_verify_tree(p2, q, tok2, off, par2, ua, un, err_word=err)
        with pytest.raises(msa.MsaError, match="NaN" if what in ("mass", "infinite") else "out of range"):
            msa.msa_check(err)
        assert int(acc[1]) >= 1 and (int(nxt[1]) == -1) == (what in ("mass", "infinite"))


def test_verify_leaves_padding(msa):
    t = T.make_tree([0, 0], [3, 2], 54)
    p, q, tok, ua, un = T.verify_inputs(t, 100, 73, True)
    pad = 4
    nan = torch.full((pad, 100), float("nan"))
    off, par, _, _, _ = t.dev(DEV, pad)
    path = torch.full((5 + pad,), 99, dtype=torch.int32, device=DEV)
    err = msa.new_err_word(DEV)
    got = msa.msa_verify_tree(torch.cat([p, nan]).to(DEV), torch.cat([q, nan]).to(DEV),
                              torch.cat([tok, torch.full((pad,), -7, dtype=torch.int32)]).to(DEV), off, par,
                              torch.cat([ua, torch.zeros(pad)]).to(DEV), un.to(DEV), path=path, err_word=err)
    msa.msa_check(err)
    want = T.ref_verify(t, p, q, tok, ua, un)
    assert got[0].tolist() == want[0].tolist() + [99] * pad
    assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[2].cpu(), want[2])


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("layers,G,D,Di", [(1, 8, 128, 64), (3, 2, 64, 32), (5, 1, 128, 32), (2, 16, 64, 64)])
def test_commit(msa, layers, G, D, Di):
    t = T.make_tree([0, 100, 127, 300, 128], [64, 40, 3, 0, 9], 55, "random")
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    R, pad = t.n_rows, 2
    new = [rnd(layers, R + pad, G, w) for w in (D, D, Di)]
    caches = [rnd(layers, t.n_pages, 128, G, w) for w in (D, D, Di)]
    path, acc = torch.full((R + pad,), -1, dtype=torch.int32), []
    for b in range(5):
        rows = list(t.rows(b))
        if not rows:
            acc.append(0)
            continue
        best = max(rows, key=lambda r: t.depth[r])
        nodes = [m for m in range(len(rows)) if t.anc[best] >> m & 1]
        nodes = nodes[:-1] if b == 4 and len(nodes) > 1 else nodes
        path[rows[0]:rows[0] + len(nodes)] = torch.tensor(nodes, dtype=torch.int32)
        acc.append(len(nodes))
    off, _, ctxd, bt, _ = t.dev(DEV, pad)
    dev_new, dev_c = [x.to(DEV) for x in new], [x.to(DEV) for x in caches]
    err = msa.new_err_word(DEV)
    dims = msa.Dims(8 * G, G, D, Di, 1, t.max_blocks)
    if layers == 1:   # one layer: the leading dimension may be left out
        args = [x[0] for x in dev_new] + [x[0] for x in dev_c]
    else:
        args = dev_new + dev_c
    lens = msa.msa_commit_tree(*args, bt, ctxd, off, path.to(DEV), torch.tensor(acc, dtype=torch.int32, device=DEV),
                               dims, err_word=err)
    msa.msa_check(err)
    for b in range(5):
        for k in range(acc[b]):
            pos = t.ctx[b] + k
            page = int(t.block_table[b, pos // 128])
            for c, x in zip(caches, new):
                c[:, page, pos % 128] = x[:, t.off[b] + int(path[t.off[b] + k])]
    for c, d in zip(caches, dev_c):
        assert torch.equal(c, d.cpu())
    assert lens.tolist() == [c + a for c, a in zip(t.ctx, acc)]


def test_commit_flags(msa):
    t = T.make_tree([126], [4], 56, "chain")
    dims = msa.Dims(8, 1, 64, 32, 1, t.max_blocks)
    new = [T.bf16((4, 1, w), w).to(DEV) for w in (64, 64, 32)]
    off, _, ctxd, bt, _ = t.dev(DEV)
    path = torch.arange(4, dtype=torch.int32, device=DEV)
    acc = torch.tensor([4], dtype=torch.int32, device=DEV)
    for what in ("page", "path", "acc", "end"):
        caches = [torch.zeros((t.n_pages, 128, 1, w), dtype=torch.bfloat16, device=DEV) for w in (64, 64, 32)]
        bt2, path2, acc2, ctx2 = bt.clone(), path.clone(), acc.clone(), ctxd.clone()
        if what == "page":
            bt2[0, 1] = t.n_pages
        elif what == "path":
            path2[2] = 4
        elif what == "acc":
            acc2[0] = 5
        else:
            ctx2[0] = t.max_blocks * 128 - 2
        err = msa.new_err_word(DEV)
        msa.msa_commit_tree(*new, *caches, bt2, ctx2, off, path2, acc2, dims, err_word=err)
        with pytest.raises(msa.MsaError, match="BOUNDS"):
            msa.msa_check(err)
        written = {"page": 2, "path": 3, "acc": 0, "end": 2}[what]
        assert int((caches[0] != 0).any(-1).sum()) == written


# ------------------------------------------------------------------ a whole step

def _model_step(msa, seed, ctx, counts, pad, Hq=16, G=2, D=128, Di=64, topk=4, layers=2):
    t = T.make_tree(ctx, counts, seed, extra_blocks=1)
    R = t.n_rows + pad
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)
    caches = [rnd(layers, t.n_pages, 128, G, w) for w in (D, D, Di)]
    rows = [rnd(layers, R, G, w) for w in (D, D, Di)]
    q, q_idx = rnd(layers, R, Hq, D), rnd(layers, R, G, Di)
    return t, msa.Dims(Hq, G, D, Di, topk, t.max_blocks), caches, rows, q, q_idx


def test_tree_step_equals_sequential_decode(msa):
    """A speculative step -- layout, scoring, top-k and attention per layer, verification, commit -- against
    appending the accepted path token by token and decoding each token on its own."""
    pad = 3
    t, dims, caches, rows, q, q_idx = _model_step(msa, 81, [700, 250, 0, 126], [9, 20, 4, 12], pad)
    off, par, ctxd, bt, _ = t.dev(DEV, pad)
    B, L = 4, 2
    step = msa.TreeStep(dims, t.n_rows + pad, B, DEV)
    step.layout(off, par, ctxd)
    outs, lses, sels = [], [], []
    for l in range(L):
        out, lse = step.attend(q[l], q_idx[l], rows[0][l], rows[1][l], rows[2][l], *[c[l] for c in caches], bt)
        outs.append(out.clone())
        lses.append(lse.clone())
        sels.append(step.sel.clone())
    # a target that accepts the deepest leaf's path up to its last node
    V = 50
    p = torch.full((t.n_rows + pad, V), 1.0 / V, device=DEV)
    tokens = torch.zeros(t.n_rows + pad, dtype=torch.int32, device=DEV)
    want_path = []
    for b in range(B):
        best = max(t.rows(b), key=lambda r: t.depth[r])
        nodes = [m for m in range(t.off[b + 1] - t.off[b]) if t.anc[best] >> m & 1]
        want_path.append(nodes)
        for r in t.rows(b):
            tokens[r] = 1 + (r - t.off[b]) % 40
        for a, c in zip(nodes, nodes[1:]):
            p[t.off[b] + a] = 0
            p[t.off[b] + a, 1 + c % 40] = 1.0
    u = torch.full((t.n_rows + pad,), 0.5, device=DEV)
    path, acc, nxt = step.verify(p, None, tokens, u, torch.full((B,), 0.25, device=DEV))
    lens = step.commit(*rows, *caches, bt)
    msa.msa_check(step.err)
    for b in range(B):
        assert path.tolist()[t.off[b]:t.off[b] + int(acc[b])] == want_path[b]
        assert int(lens[b]) == t.ctx[b] + len(want_path[b]) and 0 <= int(nxt[b]) < V
    # every accepted token again, alone, over the cache that now holds its path
    dec = msa.DecodeStep(dims, 1, 1, t.n_pages, DEV)
    for b in range(B):
        for k, node in enumerate(want_path[b]):
            r = t.off[b] + node
            n = torch.tensor([t.ctx[b] + k + 1], dtype=torch.int32, device=DEV)
            for l in range(L):
                o, s = dec(q[l, r:r + 1], q_idx[l, r:r + 1], *[c[l] for c in caches], bt[b:b + 1].contiguous(), n)
                msa.msa_check(dec.err)
                assert torch.equal(dec.sel[0], sels[l][r]), (b, node, l)
                # both round P and the result to bf16
                tol = 2 * 2.0 ** -8 * (o.float().abs() + 1.0)
                assert bool(((o.float() - outs[l][r].float()).abs() <= tol).all())
                assert torch.allclose(s[0], lses[l][r], rtol=1e-5, atol=1e-4)


def test_tree_step_captured_and_replayed(msa):
    """One captured step replayed for trees of other shapes and sizes, and on a side stream, gives what eager calls give."""
    first = _model_step(msa, 82, [700, 250], [9, 20], 45, layers=1)
    t, dims, caches, rows, q, q_idx = first
    R = t.n_rows + 45
    off, par, ctxd, bt, _ = t.dev(DEV, 45)
    step = msa.TreeStep(dims, R, 2, DEV)
    V = 300
    g = torch.Generator().manual_seed(4)
    p = torch.softmax(torch.randn((R, V), generator=g), -1).to(DEV)
    d = torch.softmax(torch.randn((R, V), generator=g), -1).to(DEV)
    tok = torch.randint(0, V, (R,), generator=g).int().to(DEV)
    ua, un = torch.rand(R, generator=g).to(DEV), torch.rand(2, generator=g).to(DEV)

    def run(s, c):
        s.layout(off, par, ctxd)
        s.attend(q[0], q_idx[0], rows[0][0], rows[1][0], rows[2][0], *[x[0] for x in c], bt)
        s.verify(p, d, tok, ua, un)
        s.commit(*rows, *c, bt)

    caps = [c.clone() for c in caches]
    run(step, caps)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(step, caps)
    side = torch.cuda.Stream()
    for seed, ctx, counts in ((83, [640, 255], [1, 64]), (84, [0, 300], [0, 37]), (82, [700, 250], [9, 20])):
        t2 = T.make_tree(ctx, counts, seed)
        o2, p2, c2, _, _ = t2.dev(DEV, R - t2.n_rows)
        off.copy_(o2)
        par.copy_(p2)
        ctxd.copy_(c2)
        want = msa.TreeStep(dims, R, 2, DEV)
        wc, gc = [c.clone() for c in caches], [c.clone() for c in caches]
        run(want, wc)
        msa.msa_check(want.err)
        for a, b in zip(caps, gc):
            a.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        msa.msa_check(step.err)
        n = t2.n_rows
        assert torch.equal(step.out[:n], want.out[:n]) and torch.equal(step.lse[:n], want.lse[:n])
        assert torch.equal(step.path[:n], want.path[:n]) and torch.equal(step.next_token, want.next_token)
        assert torch.equal(step.new_lens, want.new_lens)
        for a, b in zip(caps, wc):
            assert torch.equal(a, b)


def test_tree_attention_repeats_bit_for_bit(msa):
    t = T.make_tree([20000, 300], [30, 64], 28)
    x = _attn_inputs(t, 16, 2, 128, 38)
    sel = T.random_sel(t, 2, 16, 46, drop_own=0.0)
    dims = _dims(msa, t, 16, 2, 128, 64, 16)
    first = _attend(msa, t, dims, *x, sel)
    for _ in range(3):
        again = _attend(msa, t, dims, *x, sel)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_steps_at_once(msa):
    """Two steps on two streams with their own workspaces."""
    runs = []
    for seed in (85, 86):
        t = T.make_tree([9000 + seed, 300], [30, 64], seed)
        x = [v.to(DEV) for v in _attn_inputs(t, 16, 2, 128, seed)]
        sel = T.random_sel(t, 2, 16, seed, drop_own=0.0).to(DEV)
        off, _, ctxd, bt, anc = t.dev(DEV)
        dims = _dims(msa, t, 16, 2, 128, 64, 16)
        err = msa.new_err_word(DEV)
        ws = torch.empty(msa.msa_workspace_bytes(msa.MSA_OP_TREE, t.n_rows, 2, dims), dtype=torch.uint8, device=DEV)
        runs.append((x, bt, ctxd, off, anc, sel, dims, err, ws))

    def go(r):
        x, bt, ctxd, off, anc, sel, dims, err, ws = r
        return msa.msa_sparse_attn_tree(*x, bt, ctxd, off, anc, sel, dims, workspace=ws, err_word=err)

    want = [go(r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        got = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(go(r))
        torch.cuda.synchronize()
        for (a, b), (c, d), r in zip(got, want, runs):
            assert torch.equal(a, c) and torch.equal(b, d)
            msa.msa_check(r[7])


# ------------------------------------------------------------------ calls at the edges of what is documented

def test_verify_counts_bad_draft_entries_as_zero(msa):
    """Draft entries that are negative or not a number, anywhere in a row and at the drafted tokens."""
    t = T.make_tree([0] * 8, [5] * 8, 55, "star")
    V = 1003
    p, q, tok, ua, un = T.verify_inputs(t, V, 74, True)
    q[::2, 3::7] = float("nan")
    q[1::2, 2::5] = -0.25
    q[:, 11] = -float("inf")
    for b in range(8):
        q[t.off[b], tok[t.off[b] + 1].long()] = float("nan") if b % 2 else -1.0
    off, par, _, _, _ = t.dev(DEV)
    err = msa.new_err_word(DEV)
    got = msa.msa_verify_tree(p.to(DEV), q.to(DEV), tok.to(DEV), off, par, ua.to(DEV), un.to(DEV), err_word=err)
    msa.msa_check(err)
    want = T.ref_verify(t, p, torch.nan_to_num(q, nan=0.0, neginf=0.0).clamp(min=0), tok, ua, un)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w), (g.tolist(), w.tolist())


@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (8, 2, 64), (128, 16, 128)])
def test_tree_attention_refused_page_of_wide_trees(msa, Hq, G, D):
    """A bad page is reported and the rows that did not select its block are as without it, also where the page
    leaves a tile's item without any node."""
    t = T.make_tree([900, 1700], [60, 23], 28)
    x = _attn_inputs(t, Hq, G, D, 38)
    sel = T.random_sel(t, G, 5, 45, drop_own=0.2, empty=0.05)
    off, _, ctxd, bt, anc = t.dev(DEV)
    bt[0, 3], bt[1, 0] = -5, t.n_pages
    err = msa.new_err_word(DEV)
    out, lse = msa.msa_sparse_attn_tree(*[v.to(DEV) for v in x], bt, ctxd, off, anc, sel.to(DEV),
                                        _dims(msa, t, Hq, G, D, 64, 5), err_word=err)
    with pytest.raises(msa.MsaError, match="BOUNDS"):
        msa.msa_check(err)
    ro, rl, bo, bl = T.ref_attend(t, *x, sel, D ** -0.5)
    bad = torch.where(torch.arange(t.n_rows) < t.off[1], 3, 0)[:, None, None]
    keep = (~(sel == bad).any(-1)).repeat_interleave(Hq // G, 1)          # [n_rows][Hq]
    assert 0.2 < float(keep.float().mean()) < 0.98
    T.assert_within(lse[keep.to(DEV)], rl[keep], bl[keep], "lse")
    T.assert_within(out[keep.to(DEV)], ro[keep], bo[keep], "out")


def test_tree_attention_block_named_twice(msa):
    """The selection is a set."""
    t = T.make_tree([700], [20], 29)
    x = _attn_inputs(t, 16, 2, 128, 39)
    sel = T.random_sel(t, 2, 3, 46)
    dims = _dims(msa, t, topk=6)
    once = torch.cat([sel, torch.full_like(sel, -1)], -1)
    a = _attend(msa, t, dims, *x, once)
    b = _attend(msa, t, dims, *x, torch.cat([sel, sel.flip(-1)], -1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hq,G,D,Di", [(128, 16, 128, 64), (4, 1, 64, 32)])
def test_largest_tree_at_the_longest_context(msa, Hq, G, D, Di):
    """64 nodes with 32 blocks each that end at the last position of the largest table of the attention; the pages
    repeat, so the cache is small."""
    MB, n_pages = 16384, 96
    ctx = MB * 128 - 64
    t = T.make_tree([ctx % 8192 + 64], [64], 30, "chain")     # for its parents alone
    g = torch.Generator().manual_seed(40)
    bt = torch.randint(n_pages, (1, MB), generator=g, dtype=torch.int32)
    off, par = torch.tensor([0, 64], dtype=torch.int32, device=DEV), torch.tensor(t.parents, dtype=torch.int32, device=DEV)
    ctxd = torch.tensor([ctx], dtype=torch.int32, device=DEV)
    dims = msa.Dims(Hq, G, D, Di, 32, MB)
    step = msa.TreeStep(dims, 64, 1, DEV)
    step.layout(off, par, ctxd)
    assert int(step.q_pos[-1]) == MB * 128 - 1
    q, qi = T.bf16((64, Hq, D), 47), T.bf16((64, G, Di), 48)
    kc, vc, ic = T.bf16((n_pages, 128, G, D), 49), T.bf16((n_pages, 128, G, D), 50), T.bf16((n_pages, 128, G, Di), 51)
    kn, vn, ixn = T.bf16((64, G, D), 52), T.bf16((64, G, D), 53), T.bf16((64, G, Di), 54)
    dev = [v.to(DEV) for v in (q, qi, kn, vn, ixn, kc, vc, ic, bt)]
    out, lse = step.attend(*dev)
    msa.msa_check(step.err)
    # scores of the repeated pages: one product per page
    dots = torch.einsum("rgd,ptgd->rgpt", qi.double(), ic.double())
    per_page = dots.amax(-1)
    want = per_page[..., bt[0].long()]
    tail = ctx % 128                                          # cached tokens of the last block
    drafted = torch.einsum("rgd,mgd->rgm", qi.double(), ixn.double())
    drafted.masked_fill_(~torch.ones(64, 64).tril().bool()[:, None], -torch.inf)
    want[..., -1] = torch.maximum(dots[:, :, bt[0, -1].long(), :tail].amax(-1), drafted.amax(-1))
    # |dot - its fp32 sum| <= Di ulps of the sum of the products' sizes
    size = torch.einsum("rgd,ptgd->rgpt", qi.double().abs(), ic.double().abs()).amax() + \
        torch.einsum("rgd,mgd->rgm", qi.double().abs(), ixn.double().abs()).amax()
    assert bool(((step.scores.cpu().double() - want).abs() <= Di * 2.0 ** -23 * float(size)).all())
    sel = step.sel.cpu()
    assert bool((sel[..., 0] >= 0).all()) and int(sel.max()) == MB - 1
    # the attention of three rows, by the selection that was made
    for r in (0, 31, 63):
        for h in range(0, Hq, Hq // G):
            grp = h // (Hq // G)
            ks, vs = [], []
            for j in sel[r, grp].tolist():
                if j < 0:
                    continue
                lim = tail if j == MB - 1 else 128
                ks.append(kc[bt[0, j], :lim, grp])
                vs.append(vc[bt[0, j], :lim, grp])
                if j == MB - 1:
                    ks.append(kn[:r + 1, grp])
                    vs.append(vn[:r + 1, grp])
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            s = (k @ q[r, h].double()) * D ** -0.5
            w = torch.softmax(s, 0)
            # P and the output rounded to bf16 (half a step each), and the logits' fp32 sums
            slack = D * 2.0 ** -23 * float((k.abs() @ q[r, h].double().abs()).max()) * D ** -0.5 + 1e-5
            bound = (2.0 ** -8 + 2 * slack) * (w @ v.abs()) * (1 + 2.0 ** -8) + 2.0 ** -8 * (w @ v).abs()
            assert bool(((out[r, h].cpu().double() - w @ v).abs() <= bound).all()), (r, h)
            assert abs(float(lse[r, h]) - float(s.logsumexp(0))) <= slack + 2.0 ** -22 * abs(float(s.logsumexp(0)))


def test_step_with_padding_and_old_scores(msa):
    """Scores that an earlier use of the buffers left, NaN among them, do not reach a padded step."""
    t = T.make_tree([500, 90], [9, 4], 31)
    pad = 7
    off, par, ctxd, bt, _ = t.dev(DEV, pad)
    dims = _dims(msa, t)
    x = _attn_inputs(t, 16, 2, 128, 41, pad)
    qi, ic, ixn = T.bf16((t.n_rows + pad, 2, 64), 42), T.bf16((t.n_pages, 128, 2, 64), 43), T.bf16((t.n_rows + pad, 2, 64), 44)
    got = []
    for fill in (0.0, float("nan")):
        step = msa.TreeStep(dims, t.n_rows + pad, 2, DEV)
        step.scores.fill_(fill)
        step.layout(off, par, ctxd)
        q, kc, vc, kn, vn = [v.to(DEV) for v in x]
        out, lse = step.attend(q, qi.to(DEV), kn, vn, ixn.to(DEV), kc, vc, ic.to(DEV), bt)
        msa.msa_check(step.err)
        got.append((out.clone(), lse.clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool((got[0][0][t.n_rows:] == 0).all())
