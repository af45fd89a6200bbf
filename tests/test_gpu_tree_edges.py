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
