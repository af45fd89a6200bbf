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
