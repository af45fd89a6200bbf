"""Drafted trees without a GPU: what the calls refuse on the host, and the references' own consistency."""
import ctypes

import pytest
import torch

from tests import _tree as T
from tests.test_abi_cpu import FAKE, good_dims, lib  # noqa: F401  (fixture)

ODD = ctypes.c_void_p(0x1008)
BIG = ctypes.c_size_t(1 << 40)


def _rows(lib, d, n_rows=8, n_req=2, first=FAKE):
    return lib.msa_tree_rows(first, FAKE, FAKE, n_rows, n_req, ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, None)


def _score(lib, d, n_rows=8, n_req=2, n_pages=10, q=FAKE, scores=FAKE):
    return lib.msa_tree_index_score(q, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, n_rows, n_req, n_pages, ctypes.byref(d),
                                    scores, FAKE, None)


def _attn(lib, d, n_rows=8, n_req=2, n_pages=10, q=FAKE, out=FAKE, ws=FAKE, ws_bytes=BIG):
    return lib.msa_sparse_attn_tree(q, *([FAKE] * 9), n_rows, n_req, n_pages, ctypes.byref(d), out, FAKE, ws, ws_bytes,
                                    FAKE, None)


def _verify(lib, n_rows=8, n_req=2, vocab=100, p=FAKE, path=FAKE):
    return lib.msa_verify_tree(p, None, vocab, FAKE, FAKE, FAKE, FAKE, FAKE, n_rows, n_req, path, FAKE, FAKE, FAKE, None)


def _commit(lib, d, layers=1, n_rows=8, n_req=2, n_pages=10, k=FAKE, lens=ctypes.c_void_p(0x2000)):
    return lib.msa_commit_tree(k, FAKE, FAKE, layers, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, n_rows, n_req,
                               n_pages, ctypes.byref(d), lens, FAKE, None)


@pytest.mark.parametrize("call", [_rows, _score, _attn, _commit])
@pytest.mark.parametrize("kw,status", [(dict(page_size=64), 2), (dict(topk=0), 1), (dict(max_blocks=0), 1),
                                       (dict(Hq=63), 1)])
def test_bad_dims(lib, call, kw, status):  # noqa: F811
    assert call(lib, good_dims(**kw)) == status


def test_unsupported_shapes(lib):  # noqa: F811
    assert _attn(lib, good_dims(Hq=16, G=8)) == 2 and _attn(lib, good_dims(D=96)) == 2
    assert _attn(lib, good_dims(max_blocks=16385)) == 2
    assert _score(lib, good_dims(Di=48)) == 2 and _score(lib, good_dims(G=3, Hq=24)) == 2
    assert _score(lib, good_dims(max_blocks=65536)) == 2
    assert _commit(lib, good_dims(Di=48)) == 2 and _commit(lib, good_dims(D=96)) == 2
    d = good_dims()
    for call in (_rows, _score, _attn, _commit):
        assert call(lib, d, n_req=65536) == 2
    assert _verify(lib, n_req=65536) == 2


def test_refuses_sizes_past_32_bits(lib):  # noqa: F811
    """Index arithmetic that would leave 32 bits is refused before anything is launched."""
    assert _verify(lib, vocab=(1 << 30) + 1) == 2
    assert _score(lib, good_dims(Hq=128, G=16, max_blocks=65535), n_rows=4000, n_req=4000) == 2
    assert _attn(lib, good_dims(Hq=128, G=16, topk=32, max_blocks=16384), n_rows=65535, n_req=65535) == 2


def test_bad_sizes_and_pointers(lib):  # noqa: F811
    d = good_dims()
    for call in (_rows, _score, _attn, _commit):
        assert call(lib, d, n_rows=-1) == 1 and call(lib, d, n_req=0) == 1
    for call in (_score, _attn, _commit):
        assert call(lib, d, n_pages=0) == 1
    assert _verify(lib, n_rows=-1) == 1 and _verify(lib, n_req=0) == 1 and _verify(lib, vocab=0) == 1
    assert _commit(lib, d, layers=0) == 1
    assert _rows(lib, d, first=None) == 1 and _score(lib, d, q=None) == 1 and _attn(lib, d, q=None) == 1
    assert _verify(lib, p=None) == 1 and _verify(lib, path=None) == 1 and _commit(lib, d, k=None) == 1
    assert _score(lib, d, q=ODD) == 1 and _attn(lib, d, q=ODD) == 1 and _attn(lib, d, out=ODD) == 1
    assert _attn(lib, d, ws=ODD) == 1 and _commit(lib, d, k=ODD) == 1
    assert _commit(lib, d, lens=FAKE) == 1   # the lengths would overwrite ctx_lens
    lib.msa_last_error.restype = ctypes.c_char_p
    assert b"new_lens" in lib.msa_last_error()


def test_commit_refuses_lengths_that_overlap(lib):  # noqa: F811
    """A CTA of one layer would write a length that another has still to read."""
    d = good_dims()
    for shift in (-4, 4):
        assert _commit(lib, d, n_req=2, lens=ctypes.c_void_p(FAKE.value + shift)) == 1


def test_nothing_to_do(lib):  # noqa: F811
    d = good_dims()
    assert _rows(lib, d, n_rows=0) == 0 and _score(lib, d, n_rows=0) == 0 and _attn(lib, d, n_rows=0) == 0


def test_workspace(lib):  # noqa: F811
    lib.msa_workspace_bytes.restype = ctypes.c_size_t
    d = good_dims()
    need = lib.msa_workspace_bytes(5, 64, 8, ctypes.byref(d))
    assert need > 0 and lib.msa_workspace_bytes(5, 64, 0, ctypes.byref(d)) == 0
    assert _attn(lib, d, n_rows=64, n_req=8, ws=None) == 6 or need == 0
    assert _attn(lib, d, n_rows=64, n_req=8, ws_bytes=ctypes.c_size_t(need - 1)) == 6


def test_binding_refuses_before_the_call():
    """Types, shapes and devices are refused in Python (CPU tensors never reach the library)."""
    import block_sparse_attention_06_gb300 as m
    dims = m.Dims(16, 2, 128, 64, 4, 3)
    off, par = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([-1, 0], dtype=torch.int32)
    ctx = torch.tensor([5], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.msa_tree_rows(off, par, ctx, dims)
    with pytest.raises(TypeError, match="torch.Tensor"):
        m.msa_verify_tree(None, None, par, [0, 2], par, None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.msa_commit_tree(*[torch.zeros(1, 2, 2, 128, dtype=torch.bfloat16)] * 6, par, ctx, off, par, ctx, dims)


def test_reference_scores_are_those_of_the_committed_path():
    """A node's reference scores are the oracle's block scores once its path is in the cache."""
    import oracle
    t = T.make_tree([250, 120], [12, 9], 3)
    q, kn, kidx = T.bf16((t.n_rows, 2, 32), 1), T.bf16((t.n_rows, 2, 32), 2), T.bf16((t.n_pages, 128, 2, 32), 3)
    got, _ = T.ref_scores(t, q, kidx, kn)
    for b in range(2):
        for r in t.rows(b):
            cache = kidx.clone()
            path = [m for m in range(t.off[b + 1] - t.off[b]) if t.anc[r] >> m & 1]
            for k, m in enumerate(path):
                pos = t.ctx[b] + k
                cache[int(t.block_table[b, pos // 128]), pos % 128] = kn[t.off[b] + m]
            want = oracle.block_scores(q[r:r + 1], cache, t.block_table[b:b + 1], torch.zeros(1, dtype=torch.int32),
                                       torch.tensor([t.q_pos()[r]], dtype=torch.int32), t.max_blocks)
            assert torch.allclose(got[r], want[0].double(), rtol=1e-12, atol=1e-12)


def test_reference_attention_is_that_of_the_committed_path():
    import oracle
    t = T.make_tree([250], [12], 4)
    q, kn, vn = T.bf16((12, 8, 64), 1), T.bf16((12, 2, 64), 2), T.bf16((12, 2, 64), 3)
    kc, vc = T.bf16((t.n_pages, 128, 2, 64), 4), T.bf16((t.n_pages, 128, 2, 64), 5)
    sel = T.random_sel(t, 2, 3, 6, drop_own=0.0, empty=0.0)
    out, lse, _, _ = T.ref_attend(t, q, kc, vc, kn, vn, sel, 0.125)
    for r in t.rows(0):
        k2, v2 = kc.clone(), vc.clone()
        for k, m in enumerate(m for m in range(12) if t.anc[r] >> m & 1):
            pos = t.ctx[0] + k
            k2[int(t.block_table[0, pos // 128]), pos % 128] = kn[m]
            v2[int(t.block_table[0, pos // 128]), pos % 128] = vn[m]
        o, s = oracle.attention(q[r:r + 1], k2, v2, t.block_table, torch.zeros(1, dtype=torch.int32),
                                torch.tensor([t.q_pos()[r]], dtype=torch.int32), sel[r:r + 1], 0.125)
        assert torch.allclose(out[r], o[0].double(), atol=1e-9) and torch.allclose(lse[r], s[0].double(), atol=1e-9)


def test_reference_verification_keeps_the_targets_distribution():
    """Exact, over a grid of both uniform numbers and all pairs of sampled children, at a small vocabulary."""
    p = torch.tensor([[0.5, 0.25, 0.25, 0.0]] * 3)
    q = torch.tensor([[0.25, 0.25, 0.0, 0.5]] * 3)
    t = T.make_tree([0], [3], 1, "star")
    N = 16
    mass = torch.zeros(4, dtype=torch.float64)
    for x in range(4):
        for y in range(4):
            w = float(q[0, x] * q[0, y])
            if not w:
                continue
            for i in range(N):
                for j in range(N):
                    ua = torch.tensor([0.0, (i + 0.5) / N, (j + 0.5) / N])
                    for u in range(N):
                        _, acc, nxt = T.ref_verify(t, p, q, torch.tensor([0, x, y]), ua, torch.tensor([(u + 0.5) / N]))
                        tok = int(nxt[0])
                        if int(acc[0]) > 1:
                            path = T.ref_verify(t, p, q, torch.tensor([0, x, y]), ua, torch.tensor([(u + 0.5) / N]))[0]
                            tok = (x, y)[int(path[1]) - 1]
                        mass[tok] += w / N ** 3
    # the grid's own error: at most one cell per comparison
    assert bool(((mass - p[0].double()).abs() <= 3 / N).all()) and float(mass[3]) == 0.0


def test_attention_refuses_more_requests_and_groups_than_its_records_number(lib):  # noqa: F811
    """A (request, group)'s place in the workspace is kept in 30 bits, 64 nodes each."""
    big = dict(n_rows=1, n_req=65535, n_pages=1)
    assert _attn(lib, good_dims(Hq=4 * 257, G=257, topk=1), **big) == 2
    lib.msa_workspace_bytes.restype = ctypes.c_size_t
    small = good_dims(Hq=4 * 256, G=256, topk=1)
    assert _attn(lib, small, **big, ws_bytes=ctypes.c_size_t(0)) == 6   # 2^24 - 256 of them: only the workspace is short
