"""8-bit caches on the GPU, where it can go wrong: rows of V without a nonzero code, rows that cannot be answered among
rows that can, q and unseen tokens of any bits, lengths and windows at the ends of their ranges, the last bit of cosines
and sines, and long streams (more items than CTAs, many refills of a ring).  References and bounds: tests/_q8.py."""
import math

import pytest
import torch

from tests import _q8 as Q
from tests.test_gpu_q8 import E4M3, E8M0, cuda, i32, make_cache, msa, u8  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ rows of zeros in V

ZERO_ROWS = list(range(5)) + [37] + list(range(64, 97)) + [255]      # parts of a unit of 32 tokens, a whole one, the last token


def _zero_rows(D, G, exp, logit, negative=False):
    """256 tokens in two pages, V of 2^exp but for rows of zeros whose logits lie `logit` above the others'."""
    bt, pool = Q.tables([256], 1)
    k = Q.normal((pool, G, 128, D), 2, 0.3).double()
    v = Q.normal((pool, G, 128, D), 3).double() * 2.0 ** exp
    for t in ZERO_ROWS:
        page = int(bt[0, t // 128])
        v[page, :, t % 128] = 0.0
        k[page, :, t % 128, 0] = logit
    kc, vc = Q.to_cache(k), Q.to_cache(v)
    assert all(int(u8(vc[1])[int(bt[0, t // 128]), 0, t % 128]) == 127 for t in ZERO_ROWS)
    if negative:
        u8(vc[0])[vc[0].float() == 0] = 0x80                                     # -0 is a zero too
    q = Q.normal((4, 8 * G, D), 4, 0.3)
    q[..., 0] = 1.0
    return bt, kc, vc, q


@pytest.mark.parametrize("D,G", [(64, 2), (128, 1)])
@pytest.mark.parametrize("exp,logit,negative", [(-7, 0.0, False), (-24, 0.0, True), (-40, 0.0, False), (-60, 30.0, False),
                                                (-60, -30.0, True), (-90, 14.0, False), (-30, 400.0, False)])
@pytest.mark.parametrize("call", ["paged", "decode", "chunk"])
def test_rows_of_zeros_in_v_take_no_bits_of_the_others(msa, call, D, G, exp, logit, negative):  # noqa: F811
    bt, kc, vc, q = _zero_rows(D, G, exp, logit, negative)
    cache = msa.CacheQ8(*cuda(*kc, *vc))
    k, v = Q.stored(*kc), Q.stored(*vc)
    # with logits 400 apart what is left of the others is flushed: the bound says so; 1 / 16 keeps the rest in range
    sc = 1.0 if logit == 400.0 else 1.0 / 16 if abs(logit) < 20 else 0.5
    dims = msa.Dims(8 * G, G, D, 64, 2, bt.shape[1], sc)
    pos = i32([255, 254, 130, 60])
    if call == "paged":
        table = bt.repeat(4 * G, 1)
        lens = (pos + 1).repeat_interleave(G).to(torch.int32)
        out, lse = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
        o, s, bo, bs = Q.ref_paged(q, k, v, table, lens, sc)
    else:
        req = i32([0] * 4)
        out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 200, 3, dims, int(call == "chunk"))
        o, s, bo, bs = Q.ref_window(q, k, v, bt, req, pos, 200, 3, sc)
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")
    if logit == 0.0:
        assert bool((o.abs() > 4 * bo).any())                                    # the bound leaves something to tell


@pytest.mark.parametrize("phase", [0, 1])
def test_rows_of_zeros_alone_and_beside_nan(msa, phase):  # noqa: F811
    dims = msa.Dims(8, 1, 128, 64, 1, 2)
    cache, (k, v, _) = make_cache(msa, dims, 2, 3)
    u8(cache.v).zero_()
    u8(cache.v_scale).fill_(127)
    q = Q.normal((2, 8, 128), 1)
    args = i32([[0, 1]]).cuda(), i32([0, 0]).cuda(), i32([40, 200]).cuda(), 256, 0, dims, phase
    out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *args)
    want = Q.ref_window(q, k, v * 0, i32([[0, 1]]), [0, 0], [40, 200], 256, 0, 1 / math.sqrt(128))
    assert bool((out == 0).all())
    Q.assert_within(lse, want[1], want[3], "lse")
    u8(cache.v_scale)[0, 0, 100] = 255                                           # a row of NaN whose codes are zeros
    out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *args)
    assert bool((out[0] == 0).all()) and bool(torch.isnan(out[1]).all())


# ------------------------------------------------------------------------------------------------ rows that cannot be answered

@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("Hq,G,D", [(16, 2, 128), (4, 1, 128), (8, 2, 64), (8, 1, 64)])
def test_window_bad_rows_among_good_ones(msa, phase, Hq, G, D):  # noqa: F811
    """Bad requests and positions in the same tiles as good rows, over pages that every good row sees whole: 0 and
    -inf, as alone; the others as without them."""
    bt, pool = Q.tables([900], 1)
    dims = msa.Dims(Hq, G, D, 64, 1, bt.shape[1])
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    R = 150
    req, pos = i32([0] * R), torch.arange(700, 700 + R, dtype=torch.int32)
    low = -2 ** 31
    for r, a, p in ((3, 1, 710), (9, -2, 710), (17, low, 5), (31, 0, -1), (40, 0, low), (63, 0, bt.shape[1] * 128),
                    (64, 0, 2 ** 31 - 1), (70, 2 ** 31 - 1, 0), (100, 7, -9), (149, 1, 849)):
        req[r], pos[r] = a, p
    bad = (req != 0) | (pos < 0) | (pos >= bt.shape[1] * 128)
    pad = torch.zeros(R, dtype=torch.bool)
    pad[[20, 21, 148]] = True
    req[pad], pos[pad] = -1, low
    q = Q.normal((R, Hq, D), 5)
    q[31], q[21] = math.nan, math.inf
    out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R, Hq), 7.0, device="cuda")
    err = msa.new_err_word("cuda")
    for window, sinks in ((650, 0), (100, 300), (1 << 30, 0)):
        out.fill_(7.0), lse.fill_(7.0), err.zero_()
        msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), window, sinks, dims, phase, out, lse, err_word=err)
        assert int(err) == 1
        assert bool((out[bad.cuda()] == 0).all()) and bool((lse[bad.cuda()] == -math.inf).all())
        assert bool((out[pad.cuda()] == 7.0).all()) and bool((lse[pad.cuda()] == 7.0).all())
        rows = torch.nonzero(~bad & ~pad)[::5, 0]
        o, s, bo, bs = Q.ref_window(q[rows], k, v, bt, req[rows], pos[rows], window, sinks, 1 / math.sqrt(D))
        Q.assert_within(out.cpu()[rows], o, bo, "out")
        Q.assert_within(lse.cpu()[rows], s, bs, "lse")


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("D,G", [(128, 2), (64, 1)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_window_of_q_that_is_not_finite(msa, phase, D, G, bad, sign):  # noqa: F811
    """A component that no key has 0 in, so that all logits of its row may be -inf: NaN in out and lse, and the
    other rows and heads as without it."""
    bt, pool = Q.tables([500], 1)
    dims = msa.Dims(8 * G, G, D, 64, 1, bt.shape[1])
    k = Q.normal((pool, G, 128, D), 2).double()
    k[..., 9] = sign
    cache = msa.CacheQ8(*cuda(*Q.to_cache(k), *Q.pages(pool, G, D, 3)))
    q = Q.normal((40, 8 * G, D), 5).cuda()
    args = bt.cuda(), i32([0] * 40).cuda(), torch.arange(400, 440, dtype=torch.int32).cuda(), 300, 5, dims, phase
    want = msa.msa_window_attn_q8(q, cache, *args)
    good = torch.ones((40, 8 * G), dtype=torch.bool)
    for r, h in ((0, 5), (17, 0), (39, 8 * G - 1)):
        q[r, h, 9] = bad
        good[r, h] = False
    out, lse = msa.msa_window_attn_q8(q, cache, *args)
    assert bool(torch.isnan(out.cpu()[~good]).all()) and bool(torch.isnan(lse.cpu()[~good]).all())
    assert torch.equal(out.cpu()[good], want[0].cpu()[good]) and torch.equal(lse.cpu()[good], want[1].cpu()[good])


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("scale", [0, 247, 250, 254])
@pytest.mark.parametrize("code", [0x7e, 0xfe, 0x7f, 0x01])
def test_window_unseen_tokens_of_any_scale(msa, phase, scale, code):  # noqa: F811
    """What lies in pages beside a row's tokens (memory as it came) under scales whose values pass every number."""
    bt, pool = Q.tables([600], 1)
    for D, G in ((128, 2), (64, 1)):
        dims = msa.Dims(8 * G, G, D, 64, 1, bt.shape[1])
        cache, _ = make_cache(msa, dims, pool, 3)
        pos = [500 + 3 * i for i in range(20)]
        q = Q.normal((20, 8 * G, D), 5).cuda()
        args = (bt.cuda(), i32([0] * 20).cuda(), i32(pos).cuda(), 100, 5, dims, phase)
        want = msa.msa_window_attn_q8(q, cache, *args)
        assert bool(torch.isfinite(want[0].float()).all())
        for t in list(range(5, 401)) + list(range(558, 600)):
            page = int(bt[0, t // 128])
            u8(cache.k)[page, :, t % 128] = u8(cache.v)[page, :, t % 128] = code
            u8(cache.k_scale)[page, :, t % 128] = u8(cache.v_scale)[page, :, t % 128] = scale
        got = msa.msa_window_attn_q8(q, cache, *args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------------------ ends of the ranges

def test_read_of_lengths_below_zero(msa):  # noqa: F811
    dims = msa.Dims(8, 2, 64, 32, 2, 3)
    cache, (k, _, _) = make_cache(msa, dims, 4, 3)
    out = [torch.full((6, 128, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    tables = i32([[0, 1, 2], [3, 0, 1]]).cuda(), i32([[0, 1, 2], [3, 4, 5]]).cuda()
    err = msa.new_err_word("cuda")
    for low in (-2 ** 31, -2 ** 31 + 200, -1, 0):
        msa.msa_cache_read_q8(cache, *tables, i32([low, 130]).cuda(), dims, *out, err_word=err)
        msa.msa_check(err)
        assert bool((out[0][:3] == 7.0).all()) and bool((out[1][:3] == 7.0).all()), low
    assert torch.equal(out[0][3].cpu().double(), k[3].transpose(0, 1)) and bool((out[0][4, 2:] == 7.0).all())


@pytest.mark.parametrize("phase", [0, 1])
def test_windows_past_32_bits(msa, phase):  # noqa: F811
    """A window or a number of first tokens past the longest context says no more than that one, however large."""
    bt, pool = Q.tables([300], 1)
    dims = msa.Dims(8, 1, 64, 64, 1, bt.shape[1])
    cache, _ = make_cache(msa, dims, pool, 3)
    q = Q.normal((2, 8, 64), 5).cuda()
    args = q, cache, bt.cuda(), i32([0, 0]).cuda(), i32([299, 100]).cuda()
    dense = msa.msa_window_attn_q8(*args, 300, 0, dims, phase)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31, 0), (2 ** 32 + 1, 0), (2 ** 63, 0), (300, 2 ** 32), (300, 2 ** 40 + 3)):
        got = msa.msa_window_attn_q8(*args, window, sinks, dims, phase)
        assert torch.equal(got[0], dense[0]) and torch.equal(got[1], dense[1]), (window, sinks)
    for window, sinks in ((0, 0), (-2 ** 32 + 5, 0), (5, -1), (5, -2 ** 32)):
        with pytest.raises(msa.MsaError, match="window"):
            msa.msa_window_attn_q8(*args, window, sinks, dims, phase)


# ------------------------------------------------------------------------------------------------ the angle

@pytest.mark.parametrize("pos", [1, 1000003])
def test_cosines_and_sines_are_rounded_once(msa, pos):  # noqa: F811
    """Pairs (1, b) turned by nearly arc cot b: the first component is cos - b sin, in fp32 next to 0, and shows both
    to their last bit.  Each is a neighbour of the 64-bit value, and the farther one only where the two are as near
    as 2^-28 of it."""
    rounds, n = 128, 64
    dims = msa.Dims(4, 1, 128, 64, 1, pos // 128 + 1)
    table = torch.zeros((1, dims.max_blocks), dtype=torch.int32, device="cuda")
    caches = [torch.empty((1, 128, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(pos)
    b = 1.0 + torch.randint(0, 24, (rounds, n), generator=g).double() / 128      # bf16 numbers; angles of 0.11 to 0.13 turns
    f = (torch.atan(1 / b) + (2 * torch.rand((rounds, n), generator=g).double() - 1) * 2.0 ** -18) / pos
    x = torch.zeros((rounds, 1, 4, 128), dtype=torch.bfloat16)
    x[:, 0, :, :64], x[:, 0, :, 64:] = 1.0, b[:, None].to(torch.bfloat16)
    x, fd = x.cuda(), f.cuda()
    zero, at = i32([0]).cuda(), i32([pos]).cuda()
    got = torch.stack([msa.msa_rope_append(x[i], kv, kv, None, None, *caches, None, table, zero, at, msa.Rope(128, fd[i]),
                                           dims)[0][0, 0] for i in range(rounds)]).cpu()
    w = f * pos

    def near(y):                         # the fp32 numbers that y may have been rounded to
        y32 = y.float()
        z32 = torch.nextafter(y32, torch.where(y > y32.double(), 1.0, -1.0).float())
        half = (z32.double() - y32.double()).abs() / 2
        return (y32.double(), torch.where((z32.double() - y).abs() <= half + 2.0 ** -28 * y.abs(), z32.double(), y32.double()))
    c, s = near(torch.cos(w)), near(torch.sin(w))
    ok = torch.zeros(rounds, n, dtype=torch.bool)
    for cc in c:
        for ss in s:
            ok |= (cc - b * ss).float().to(torch.bfloat16) == got[:, :64]
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} pairs"


# ------------------------------------------------------------------------------------------------ long streams

@pytest.mark.parametrize("Hq,G,D,n", [(64, 8, 128, 1500), (16, 4, 128, 5200), (32, 4, 64, 2600), (16, 4, 64, 5200)])
def test_window_more_items_than_ctas(msa, Hq, G, D, n):  # noqa: F811
    """Several items per CTA: rows of three requests, padding and bad rows, items of padding and of bad rows alone."""
    lens = [n // 2 + 700, n // 3 + 90, n // 6]
    bt, pool = Q.tables(lens, 1)
    dims = msa.Dims(Hq, G, D, 64, 1, bt.shape[1])
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    rows = [(b, p) for b, m in zip(range(3), (n // 2, n // 3, n // 6)) for p in range(lens[b] - m, lens[b])]
    rows += [(-1, 0)] * (n - len(rows))
    req, pos = i32([b for b, _ in rows]), i32([p for _, p in rows])
    req[256:512] = -1                                                            # whole items of padding
    req[640:900:2] = -1
    req[900:1156] = 3                                                            # and of rows without a request
    q = Q.normal((n, Hq, D), 5)
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    err = msa.new_err_word("cuda")
    args = q.cuda(), cache, *cuda(bt, req, pos), 150, 9, dims, 1
    msa.msa_window_attn_q8(*args, out, lse, err_word=err)
    assert int(err) == 1
    again = msa.msa_window_attn_q8(*args)
    live = (req >= 0).cuda()
    assert torch.equal(out[live], again[0][live]) and torch.equal(lse[live], again[1][live])
    assert bool((out[~live] == 7.0).all()) and bool((out[(req == 3).cuda()] == 0).all())
    at = torch.nonzero((req >= 0) & (req < 3))[:, 0]
    at = at[torch.randperm(at.numel(), generator=torch.Generator().manual_seed(1))[:300]]
    o, s, bo, bs = Q.ref_window(q[at], k, v, bt, req[at], pos[at], 150, 9, 1 / math.sqrt(D))
    Q.assert_within(out.cpu()[at], o, bo, "out")
    Q.assert_within(lse.cpu()[at], s, bs, "lse")
    # every row against the rows taken one by one: each of the two rounds P and the output, by 2^-8 of the largest value
    # that a row can see, and 2^-10 of it is more than all else in the bound
    one = msa.msa_window_attn_q8(*args[:-1], 0)
    d = (out.float() - one[0].float()).abs()[live]
    assert float(d.max()) <= float(v.abs().max()) * 2 * (2 * 2.0 ** -8 + 2.0 ** -10)


def test_window_second_cta_of_a_pair_with_four_heads(msa):  # noqa: F811
    bt, pool = Q.tables([600], 1)
    dims = msa.Dims(8, 2, 128, 64, 1, bt.shape[1])
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    for n in (65, 128, 200):             # a pair takes 128 rows, 64 a CTA
        req, pos = i32([0] * n), torch.arange(600 - n, 600, dtype=torch.int32)
        q = Q.normal((n, 8, 128), 5)
        out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 140, 2, dims, 1)
        o, s, bo, bs = Q.ref_window(q, k, v, bt, req, pos, 140, 2, 1 / math.sqrt(128))
        Q.assert_within(out, o, bo, "out")
        Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("Di,G,rows", [(64, 8, 8), (32, 16, 5), (64, 4, 40)])
def test_score_long_streams(msa, Di, G, rows):  # noqa: F811
    """Many units per warp: stages filled again and again, runs of more than 32 blocks of one (row, group).  Pages are
    shared, so the reference needs each once."""
    pool, MB = 12, 800
    dims = msa.Dims(4 * G, G, 64, Di, 2, MB)
    cache, (_, _, x) = make_cache(msa, dims, pool, 3)
    g = torch.Generator().manual_seed(4)
    bt = torch.randint(0, pool, (rows, MB), generator=g).to(torch.int32)
    pos = torch.randint(MB * 128 - 9000, MB * 128, (rows,), generator=g).to(torch.int32)
    pos[0], pos[1], pos[2] = MB * 128 - 1, 5, 127
    req = torch.arange(rows, dtype=torch.int32)
    q = Q.normal((rows, G, Di), 9)
    err = msa.new_err_word("cuda")
    got = msa.msa_index_score_q8(q.cuda(), cache, *cuda(bt, req, pos), dims, err_word=err)
    msa.msa_check(err)
    assert torch.equal(got, msa.msa_index_score_q8(q.cuda(), cache, *cuda(bt, req, pos), dims))
    s = torch.einsum("rgd,pgtd->rgpt", Q.f64(q), x)
    mag = torch.einsum("rgd,pgtd->rgpt", Q.f64(q).abs(), x.abs()).amax(-1) * 1.2 * (Di + 8) * 2.0 ** -23
    tol = mag + Q.f64(q).abs().amax(-1)[..., None] * x.abs().sum(-1).amax(-1).T[None] * 2.0 ** -39   # as in ref_scores
    want, bound = torch.full((rows, G, MB), -math.inf).double(), torch.zeros((rows, G, MB)).double()
    for r in range(rows):
        last = int(pos[r]) // 128
        pages = bt[r, :last + 1].long()
        want[r, :, :last + 1] = s[r].amax(-1)[:, pages]
        want[r, :, last] = s[r, :, int(pages[-1]), :int(pos[r]) % 128 + 1].amax(-1)
        bound[r, :, :last + 1] = tol[r][:, pages]
    Q.assert_within(got, want, bound, "scores")


@pytest.mark.parametrize("rows,MB,D", [(80, 160, 64), (80, 150, 128), (1, 1100, 64), (9, 300, 128)])
def test_window_of_many_units_per_warp(msa, rows, MB, D):  # noqa: F811
    """More than 32 units per warp: pages are looked up again.  Pages are shared."""
    pool = 8
    dims = msa.Dims(8, 1, D, 64, 1, MB)
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    g = torch.Generator().manual_seed(4)
    bt = torch.randint(0, pool, (rows, MB), generator=g).to(torch.int32)
    req = torch.arange(rows, dtype=torch.int32)
    pos = torch.randint(MB * 128 - 4000, MB * 128, (rows,), generator=g).to(torch.int32)
    pos[0] = MB * 128 - 1
    q = Q.normal((rows, 8, D), 9)
    for window, sinks in ((1 << 30, 0), (MB * 128 - 9000, 700)):
        out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), window, sinks, dims, 0)
        for r in range(0, rows, 11):
            p = int(pos[r])
            t = torch.arange(p + 1)
            t = t[(t > p - window) | (t < sinks)]
            page, slot = bt[r].long()[t // 128], t % 128
            want = Q.ref_attend(Q.f64(q[r]), k[page, 0, slot], v[page, 0, slot], 1 / math.sqrt(D))
            Q.assert_within(out[r], want[0], want[2], "out")
            Q.assert_within(lse[r], want[1], want[3], "lse")


# ------------------------------------------------------------------------------------------------ caches

def test_a_cache_whose_tensors_changed_is_refused(msa):  # noqa: F811
    dims = msa.Dims(8, 1, 64, 32, 1, 2)
    cache, _ = make_cache(msa, dims, 4, 3)
    q, z = Q.normal((1, 8, 64), 5).cuda(), i32([0]).cuda()
    table = i32([[3, 3]]).cuda()
    calls = [lambda: msa.msa_window_attn_q8(q, cache, table, z, z, 5, 0, dims, 0),
             lambda: msa.msa_index_score_q8(q[:, :1, :32].contiguous(), cache, table, z, z, dims)]
    for call, name in zip(calls, ("v", "kidx")):
        call()
        x = getattr(cache, name)
        x.data = x[:2].clone()
        with pytest.raises(ValueError, match="shape"):
            call()


# ------------------------------------------------------------------------------------------------ shapes

@pytest.mark.parametrize("Hq,G,D", [(12, 3, 64), (40, 5, 128), (24, 3, 128), (80, 20, 64)])
def test_groups_that_are_no_power_of_two(msa, Hq, G, D):  # noqa: F811
    """Calls without the index take any number of groups: append, read back, decode and window attention."""
    n = 200
    bt, pool = Q.tables([n], 1)
    dims = msa.Dims(Hq, G, D, 64, 2, bt.shape[1])
    cache = msa.CacheQ8.zeros(dims, pool, "cuda", index=False)
    rows = [Q.normal((n, h, D), 7 + i) for i, h in enumerate((Hq, G, G))]
    req, pos = i32([0] * n), torch.arange(n, dtype=torch.int32)
    f = 10000.0 ** (-2 * torch.arange(16).double() / 32)
    err = msa.new_err_word("cuda")
    q, _ = msa.msa_rope_append_q8(*cuda(*rows), None, None, cache, *cuda(bt, req, pos), msa.Rope(32, f.cuda()), dims,
                                  err_word=err)
    y, t = Q.rotated(rows[0], 32, f, pos.long(), False, 1.0)
    Q.assert_within(q, y, t + (y.abs() + t) * 2.0 ** -8, "q")
    page, slot = bt.long()[0, pos.long() // 128], pos.long() % 128
    for x, s, row, rot in ((cache.k, cache.k_scale, rows[1], 32), (cache.v, cache.v_scale, rows[2], 0)):
        y, t = Q.rotated(row, rot, f, pos.long(), False, 1.0)
        Q.check_rows8(u8(x).cpu()[page, :, slot].view(E4M3), u8(s).cpu()[page, :, slot].view(E8M0), y, t, "cache")
    k, v = (Q.stored(x.cpu(), s.cpu()) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    out = [torch.zeros((pool, 128, G, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_cache_read_q8(cache, bt.cuda(), bt.cuda(), i32([n]).cuda(), dims, *out, err_word=err)
    for x, val in zip(out, (k, v)):
        assert torch.equal(x.cpu().double().transpose(1, 2), val * (x.cpu() != 0).any(-1)[..., None].transpose(1, 2).double())
        assert torch.equal(x.cpu()[page, slot].double(), val[page, :, slot])
    q = q.cpu()
    at = torch.arange(0, n, 23)
    o, s, bo, bs = Q.ref_window(q[at], k, v, bt, req[at], pos[at], 90, 5, 1 / math.sqrt(D))
    for phase in (0, 1):
        got, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 90, 5, dims, phase, err_word=err)
        Q.assert_within(got.cpu()[at], o, bo, "out")
        Q.assert_within(lse.cpu()[at], s, bs, "lse")
    table, lens = bt.repeat(3 * G, 1), i32([200, 77, 1]).repeat_interleave(G).to(torch.int32)
    got, lse = msa.msa_sparse_attn_decode_q8(q[:3].cuda(), cache, *cuda(table, lens), dims, err_word=err)
    o, s, bo, bs = Q.ref_paged(q[:3], k, v, table, lens, 1 / math.sqrt(D))
    Q.assert_within(got, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")
    msa.msa_check(err)


def test_append_of_index_vectors_in_place(msa):  # noqa: F811
    dims = msa.Dims(8, 2, 64, 32, 2, 3)
    got = []
    for inplace in (False, True):
        cache = msa.CacheQ8.zeros(dims, 3, "cuda")
        rows = [Q.normal((300, h, w), 20 + i).cuda() for i, (h, w) in enumerate(((8, 64), (2, 64), (2, 64), (2, 32), (2, 32)))]
        q, qi = msa.msa_rope_append_q8(*rows, cache, i32([[2, 0, 1]]).cuda(), i32([0] * 300).cuda(),
                                       torch.arange(300, dtype=torch.int32).cuda(), msa.Rope.of_base(48, 32), dims,
                                       *((rows[0], rows[3]) if inplace else ()))
        got.append([q, qi] + [u8(getattr(cache, f)) for f in ("k", "v", "kidx", "k_scale", "v_scale", "kidx_scale")])
    for x, y in zip(*got):
        assert torch.equal(x, y)
