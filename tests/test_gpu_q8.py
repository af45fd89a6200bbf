"""8-bit caches on the GPU: rotation and append, read back, scan, decode and window attention against 64-bit references
(tests/_q8.py, with derived bounds), and a run of them together as a serving loop makes it."""
import math

import pytest
import torch

from tests import _q8 as Q

pytestmark = pytest.mark.gpu

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_attention_06_gb300 as m
    return m


def cuda(*xs):
    return [x.cuda() for x in xs]


def u8(x):
    return x.view(torch.uint8)


def make_cache(msa, dims, pool, seed):
    """(CacheQ8 on the GPU, its stored k, v, kidx in 64 bits)."""
    parts, values = [], []
    for i, w in enumerate((dims.D, dims.D, dims.Di)):
        code, scale = Q.pages(pool, dims.G, w, seed + i)
        parts += cuda(code, scale)
        values.append(Q.stored(code, scale))
    return msa.CacheQ8(*parts), values


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------------------------------------ append

APPENDS = [
    # Hq, G, D, Di, rot, rot_idx, interleaved, ctx, rows each, pad, fused, index
    (16, 2, 128, 64, 128, 64, False, [0], 1, 0, False, True),
    (64, 8, 128, 64, 64, 64, False, [127, 5, 300], 2, 3, True, True),
    (16, 4, 64, 32, 48, 16, True, [1, 126], 131, 1, True, True),
    (8, 1, 64, 32, 0, 0, False, [63], 5, 0, False, True),
    (4, 1, 64, 64, 64, 32, True, [2097000], 9, 2, True, True),
    (32, 8, 128, 32, 16, 32, False, [1000003], 3, 0, False, True),
    (32, 4, 128, 64, 112, 48, True, [60, 500], 700, 5, True, True),
    (16, 2, 128, 64, 64, 32, False, [60, 500], 300, 3, True, True),
    (16, 2, 64, 64, 32, 0, False, [100], 40, 2, True, False),
]


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("Hq,G,D,Di,rot,rot_idx,inter,ctx,n,pad,fused,index", APPENDS)
def test_append(msa, q8, Hq, G, D, Di, rot, rot_idx, inter, ctx, n, pad, fused, index):
    gain = 1.25 if rot == 48 else 1.0
    bt, pool = Q.tables([c + n for c in ctx], 1, first=ctx)
    dims = msa.Dims(Hq, G, D, Di, 4, bt.shape[1])
    R = len(ctx) * n + pad
    order = torch.randperm(R, generator=torch.Generator().manual_seed(5))       # rows in any order
    req = i32([b for b in range(len(ctx)) for _ in range(n)] + [-1] * pad)[order]
    pos = i32([c + i for c in ctx for i in range(n)] + [-7] * pad)[order]
    widths = [Hq * D, G * D, G * D, G * Di, G * Di]
    # one projection's output with a few columns more, or five tensors
    wide = Q.normal((R, sum(widths) + 8), 2, 3.0).cuda()
    parts = [x.unflatten(1, (h, -1)) for x, h in zip(wide[:, :sum(widths)].split(widths, 1), (Hq, G, G, G, G))]
    if not fused:
        parts = [x.contiguous() for x in parts]
    host = [x.cpu() for x in parts]
    f, fi = (10000.0 ** (-2 * torch.arange(r // 2).double() / max(r, 1)) for r in (rot, rot_idx))
    rope = msa.Rope(rot, f.cuda(), rot_idx, fi.cuda(), inter, gain)
    if not index:
        parts[3] = parts[4] = None
    q_out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qi_out = torch.full((R, G, Di), 7.0, dtype=torch.bfloat16, device="cuda") if index else None
    err = msa.new_err_word("cuda")
    t = cuda(bt, req, pos)
    if q8:
        cache, _ = make_cache(msa, dims, pool, 11)
        if not index:
            cache = msa.CacheQ8(cache.k, cache.k_scale, cache.v, cache.v_scale)
        parts8 = (cache.k, cache.k_scale, cache.v, cache.v_scale, cache.kidx, cache.kidx_scale)
        before = [None if x is None else u8(x).clone() for x in parts8]
        out = msa.msa_rope_append_q8(*parts, cache, *t, rope, dims, q_out, qi_out, err_word=err)
        after = [None if x is None else u8(x) for x in parts8]
    else:
        caches = [Q.normal((pool, 128, G, w), 20 + w).cuda() for w in (D, D, Di)]
        before = [x.clone() for x in caches]
        out = msa.msa_rope_append(*parts, *caches[:2], caches[2] if index else None, *t, rope, dims, q_out, qi_out,
                                  err_word=err)
        after = caches
    msa.msa_check(err)
    assert out[0] is q_out and out[1] is qi_out
    live = req >= 0
    p = pos.long()
    yq, tq = Q.rotated(host[0], rot, f, p, inter, gain)
    yk, tk = Q.rotated(host[1], rot, f, p, inter, gain)
    yi, ti = Q.rotated(host[3], rot_idx, fi, p, inter, gain)
    yj, tj = Q.rotated(host[4], rot_idx, fi, p, inter, gain)
    Q.assert_within(q_out.cpu()[live], yq[live], (tq + (yq.abs() + tq) * 2.0 ** -8)[live], "q")
    assert bool((q_out.cpu()[~live] == 7.0).all())
    if index:
        Q.assert_within(qi_out.cpu()[live], yi[live], (ti + (yi.abs() + ti) * 2.0 ** -8)[live], "q_idx")
        assert bool((qi_out.cpu()[~live] == 7.0).all())
    page = bt.long()[req[live].long(), p[live] // 128]
    slot = p[live] % 128
    new = [(yk, tk), (Q.f64(host[2]), torch.zeros_like(Q.f64(host[2]))), (yj, tj)]
    for i, (y, tol) in enumerate(new[:3 if index else 2]):
        if q8:
            code, scale = after[2 * i].cpu(), after[2 * i + 1].cpu()
            Q.check_rows8(code[page, :, slot].view(E4M3), scale[page, :, slot].view(E8M0), y[live], tol[live], f"cache {i}")
            for x, old in ((code, before[2 * i].cpu()), (scale, before[2 * i + 1].cpu())):   # nothing else is written
                old[page, :, slot] = x[page, :, slot]
                assert torch.equal(x, old), f"cache {i}"
        else:
            x, old = after[i].cpu(), before[i].cpu()
            Q.assert_within(x[page, slot], y[live], (tol + (y.abs() + tol) * 2.0 ** -8)[live], f"cache {i}")
            if i == 1:
                assert torch.equal(x[page, slot], host[2][live])                 # v as it is
            old[page, slot] = x[page, slot]
            assert torch.equal(x, old), f"cache {i}"
    # what is not rotated is q as it is, and v's codes are the reference's
    assert torch.equal(q_out.cpu()[live][..., rot:], host[0][live][..., rot:])
    if q8:
        want, e = Q.quantise(Q.f64(host[2][live]))
        assert torch.equal(Q.f64(after[2].cpu()[page, :, slot].view(E4M3)), want)
        assert torch.equal(after[3].cpu()[page, :, slot].long() - 127, e)


def _append_small(msa, k=None, v=None, req=(0, 1, 1), pos=(3, 0, 129), table=((0, -1), (1, 2)), n_pages=3, inplace=False):
    """Three rows of two requests, D 64, one group; -> (q, cache, cache before, error word, dims)."""
    dims = msa.Dims(4, 1, 64, 32, 2, 2)
    n = len(req)
    q = Q.normal((n, 4, 64), 1).cuda()
    k = Q.normal((n, 1, 64), 2).cuda() if k is None else k.cuda()
    v = Q.normal((n, 1, 64), 3).cuda() if v is None else v.cuda()
    qi, ki = Q.normal((n, 1, 32), 4).cuda(), Q.normal((n, 1, 32), 5).cuda()
    cache = msa.CacheQ8.zeros(dims, n_pages, "cuda")
    err = msa.new_err_word("cuda")
    rope = msa.Rope.of_base(64, 32, device="cuda")
    out, out_i = msa.msa_rope_append_q8(q, k, v, qi, ki, cache, i32(table).cuda(), i32(req).cuda(), i32(pos).cuda(), rope,
                                        dims, q if inplace else None, err_word=err)
    return out, cache, err, dims


def test_append_in_place(msa):
    a, c1, _, _ = _append_small(msa)
    b, c2, _, _ = _append_small(msa, inplace=True)
    assert torch.equal(a, b) and torch.equal(u8(c1.k), u8(c2.k))


@pytest.mark.parametrize("req,pos,table", [((0, 1, 2), (3, 0, 129), ((0, -1), (1, 2))),      # no such request
                                           ((0, 1, -2), (3, 0, 129), ((0, -1), (1, 2))),
                                           ((0, 1, 1), (3, 0, 256), ((0, -1), (1, 2))),      # past the table
                                           ((0, 1, 1), (3, 0, -1), ((0, -1), (1, 2))),
                                           ((0, 1, 0), (3, 0, 129), ((0, -1), (1, 2))),      # no page
                                           ((0, 1, 1), (3, 0, 129), ((0, -1), (1, 3)))])     # no such page
def test_append_flags_bad_rows_and_writes_nothing_of_them(msa, req, pos, table):
    _, cache, err, _ = _append_small(msa, req=req, pos=pos, table=table)
    assert int(err) == 1
    with pytest.raises(msa.MsaError):
        msa.msa_check(err)
    assert int((cache.k.float().abs().amax(-1) > 0).sum()) == 2                 # the two good rows


def test_append_extreme_rows(msa):
    """Zeros, subnormal and huge magnitudes; a row whose largest number is just past a power of two times 448."""
    v = torch.zeros((9, 1, 64), dtype=torch.bfloat16)
    v[1, 0, 5] = 2.0 ** -133                                                     # the smallest bf16
    v[2, 0, 0], v[2, 0, 1] = 3.3e38, -1.0
    v[3, 0, 0] = 448.0
    v[4, 0, 0] = 450.0
    v[5, 0, :] = torch.linspace(-1, 1, 64).to(torch.bfloat16)
    v[6, 0, 3], v[6, 0, 4] = 2.0 ** -92, 2.0 ** -110                             # near the lowest scale
    v[7, 0, 0], v[7, 0, 1] = 1.0, 2.0 ** -18                                     # under half of the lowest step
    v[8, 0, 0], v[8, 0, 1] = 1.0, 2.0 ** -17.0
    _, cache, err, _ = _append_small(msa, k=v.clone(), v=v, req=[0] * 9, pos=list(range(9)))
    msa.msa_check(err)
    code, scale = cache.v[0, 0, :9].cpu(), cache.v_scale[0, 0, :9].cpu()
    want, e = Q.quantise(Q.f64(v[:, 0]))
    assert torch.equal(u8(scale).long() - 127, e) and torch.equal(Q.f64(code), want)
    assert bool(torch.isfinite(cache.k.float()).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_stores_rows_that_are_not_finite_as_nan(msa, bad):
    v = Q.normal((3, 1, 64), 3)
    v[1, 0, 17] = bad
    _, cache, err, _ = _append_small(msa, v=v)
    assert int(err) == 8
    vals = cache.v.float() * cache.v_scale.float()[..., None]
    assert bool(torch.isnan(vals[1, 0, 0]).all()) and int(torch.isnan(vals).sum()) == 64
    assert int(u8(cache.v_scale)[1, 0, 0]) == 255


def test_append_without_the_index(msa):
    dims = msa.Dims(8, 2, 64, 32, 2, 1)
    cache = msa.CacheQ8.zeros(dims, 1, "cuda", index=False)
    q, k, v = (Q.normal((2, h, 64), h).cuda() for h in (8, 2, 2))
    out, none = msa.msa_rope_append_q8(q, k, v, None, None, cache, i32([[0]]).cuda(), i32([0, 0]).cuda(),
                                       i32([0, 1]).cuda(), msa.Rope(0), dims)
    assert none is None and torch.equal(out, q)
    with pytest.raises(TypeError):
        msa.msa_rope_append_q8(q, k, v, Q.normal((2, 2, 32), 1).cuda(), None, cache, i32([[0]]).cuda(), i32([0, 0]).cuda(),
                               i32([0, 1]).cuda(), msa.Rope(0), dims)


def test_append_refuses_shapes(msa):
    dims = msa.Dims(8, 2, 64, 32, 2, 1)
    cache = msa.CacheQ8.zeros(dims, 1, "cuda", index=False)
    q, k, v = (Q.normal((2, h, 64), h).cuda() for h in (8, 2, 2))
    bt, req, pos = i32([[0]]).cuda(), i32([0, 0]).cuda(), i32([0, 1]).cuda()
    call = lambda q=q, k=k, v=v, c=cache, rope=msa.Rope(0), r=req: msa.msa_rope_append_q8(  # noqa: E731
        q, k, v, None, None, c, bt, r, pos, rope, dims)
    with pytest.raises(ValueError):
        call(k=k[:1])
    with pytest.raises(TypeError):
        call(v=v.float())
    with pytest.raises(ValueError, match="dense"):
        call(q=Q.normal((2, 64, 8), 1).cuda().transpose(1, 2))
    with pytest.raises(TypeError):
        call(rope=None)
    with pytest.raises(msa.MsaError, match="strides"):                          # rows that overlap
        call(q=torch.zeros(1024, dtype=torch.bfloat16, device="cuda").as_strided((2, 8, 64), (256, 64, 1)))
    with pytest.raises(ValueError):
        call(r=req[:1])
    with pytest.raises(TypeError):
        call(c=msa.CacheQ8(u8(cache.k), cache.k_scale, cache.v, cache.v_scale))


# ------------------------------------------------------------------------------------------------ read back

@pytest.mark.parametrize("G,D,Di,lens", [(2, 128, 64, [1]), (8, 64, 32, [129, 300, 0, 127]), (1, 128, 32, [5000]),
                                         (16, 64, 64, [128, 256])])
def test_read(msa, G, D, Di, lens):
    bt, pool = Q.tables([max(n, 1) for n in lens], 1, extra_blocks=2)
    dims = msa.Dims(4 * G, G, D, Di, 2, bt.shape[1])
    cache, values = make_cache(msa, dims, pool, 3)
    to = torch.full_like(bt, -1)
    n_out = int((bt >= 0).sum()) + 1
    to[bt >= 0] = torch.randperm(n_out - 1, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    if lens == [5000]:
        to[0, ::3] = -1                                                          # blocks that are not wanted
    out = [torch.full((n_out, 128, G, w), 7.0, dtype=torch.bfloat16, device="cuda") for w in (D, D, Di)]
    err = msa.new_err_word("cuda")
    got = msa.msa_cache_read_q8(cache, bt.cuda(), to.cuda(), i32(lens).cuda(), dims, *out, err_word=err)
    msa.msa_check(err)
    for x, val, name in zip(got, values, ("k", "v", "kidx")):
        want = torch.full((n_out, 128, G, val.shape[-1]), 7.0).double()
        for b, n in enumerate(lens):
            for j in range((n + 127) // 128):
                if to[b, j] >= 0:
                    m = min(128, n - j * 128)
                    want[int(to[b, j]), :m] = val[int(bt[b, j])].transpose(0, 1)[:m]
        assert torch.equal(x.cpu().double(), want), name


def test_read_without_the_index_and_bad_pages(msa):
    dims = msa.Dims(8, 2, 64, 32, 2, 3)
    cache, _ = make_cache(msa, dims, 4, 3)
    out = [torch.full((2, 128, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens = i32([300]).cuda()
    err = msa.new_err_word("cuda")
    cache = msa.CacheQ8(cache.k, cache.k_scale, cache.v, cache.v_scale)
    for bt, to, flag, written in (([[0, 1, 9]], [[0, 1, -1]], 0, 2), ([[0, 4, 9]], [[0, 1, -1]], 1, 1),
                                  ([[0, 1, -1]], [[0, 2, -1]], 1, 1), ([[-1, 1, 1]], [[0, 1, -1]], 1, 1)):
        for x in out:
            x.fill_(7.0)
        assert msa.msa_cache_read_q8(cache, i32(bt).cuda(), i32(to).cuda(), lens, dims, *out, err_word=err)[2] is None
        assert int(err) == flag, (bt, to)
        err.zero_()
        assert sum(bool((out[0][p] != 7.0).any()) for p in range(2)) == written


def test_read_of_nan_rows(msa):
    dims = msa.Dims(8, 2, 64, 32, 2, 1)
    cache, _ = make_cache(msa, dims, 1, 3)
    u8(cache.v_scale)[0, 1, 5] = 255
    u8(cache.k)[0, 0, 3, 7] = 0x7f
    out = [torch.zeros((1, 128, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    zero = i32([[0]]).cuda()
    k, v, _ = msa.msa_cache_read_q8(cache, zero, zero, i32([128]).cuda(), dims, *out)
    assert bool(torch.isnan(v[0, 5, 1]).all()) and int(torch.isnan(v).sum()) == 64
    assert bool(torch.isnan(k[0, 3, 0, 7])) and int(torch.isnan(k).sum()) == 1


# ------------------------------------------------------------------------------------------------ scan

@pytest.mark.parametrize("G,Di,lens,more", [(8, 64, [1], 0), (4, 32, [128, 129, 1000], 3), (1, 64, [517], 0),
                                            (16, 32, [40, 300], 1), (2, 64, [2600, 31], 0)])
def test_score(msa, G, Di, lens, more):
    bt, pool = Q.tables(lens, 1, extra_blocks=more)
    dims = msa.Dims(4 * G, G, 64, Di, 2, bt.shape[1])
    cache, values = make_cache(msa, dims, pool, 3)
    rows = [(b, p) for b, n in enumerate(lens) for p in sorted({0, n // 2, n - 1})]
    req, pos = i32([b for b, _ in rows]), i32([p for _, p in rows])
    q = Q.normal((len(rows), G, Di), 9, 2.0)
    q[:, :, 0] = 300.0                                                           # one component far above the others
    q[:, :, 1] = 2.0 ** -14
    err = msa.new_err_word("cuda")
    got = msa.msa_index_score_q8(q.cuda(), cache, *cuda(bt, req, pos), dims, err_word=err)
    msa.msa_check(err)
    want, tol = Q.ref_scores(q, cache.kidx.cpu(), cache.kidx_scale.cpu(), bt, req, pos)
    Q.assert_within(got, want, tol, "scores")


def test_score_many_rows(msa):
    """More rows than a warp has lanes, bad ones among them: every range of units starts in its own row."""
    lens = [1 + 37 * (i % 19) for i in range(300)]
    bt, pool = Q.tables([max(lens)], 1)
    dims = msa.Dims(8, 2, 64, 64, 2, bt.shape[1] + 1)
    bt = torch.cat([bt, i32([[-1]])], 1)
    cache, _ = make_cache(msa, dims, pool, 3)
    q = Q.normal((300, 2, 64), 9)
    pos = i32([n - 1 for n in lens])
    req = i32([0] * 300)
    err = msa.new_err_word("cuda")
    got = msa.msa_index_score_q8(q.cuda(), cache, *cuda(bt, req, pos), dims, err_word=err)
    msa.msa_check(err)
    want, tol = Q.ref_scores(q, cache.kidx.cpu(), cache.kidx_scale.cpu(), bt, req, pos)
    Q.assert_within(got, want, tol, "scores")
    req[7], pos[200] = 1, -1
    got = msa.msa_index_score_q8(q.cuda(), cache, *cuda(bt, req, pos), dims, err_word=err)
    assert int(err) == 1
    want[7], want[200] = -math.inf, -math.inf
    Q.assert_within(got, want, tol, "scores")


def test_score_small_components_count(msa):
    """Components 2^-16 and 2^-30 of the largest, alone with a key: the third piece holds them."""
    dims = msa.Dims(4, 1, 64, 32, 1, 1)
    for small, rel in ((2.0 ** -16 * 1.0078125, 0.0), (2.0 ** -30 * 1.5, 2.0 ** -9)):
        q = torch.zeros((1, 1, 32), dtype=torch.bfloat16)
        q[0, 0, 3], q[0, 0, 7] = 1.0, small
        key = torch.zeros((1, 1, 128, 32)).double()
        key[..., 7] = 1.0
        cache = msa.CacheQ8(None, None, None, None, *cuda(*Q.to_cache(key)))
        z = i32([0]).cuda()
        got = msa.msa_index_score_q8(q.cuda(), cache, z[None], z, z, dims)
        assert abs(float(got) - float(q[0, 0, 7])) <= rel * small


def test_score_nan_and_what_is_not_seen(msa):
    dims = msa.Dims(8, 2, 64, 64, 2, 2)
    cache, _ = make_cache(msa, dims, 2, 3)
    bt, req, pos = i32([[1, 0]]).cuda(), i32([0]).cuda(), i32([130]).cuda()
    q = Q.normal((1, 2, 64), 9).cuda()
    want = msa.msa_index_score_q8(q, cache, bt, req, pos, dims)
    u8(cache.kidx)[0, :, 3:] = 0x7f                                              # past the row's position: not seen
    u8(cache.kidx_scale)[0, :, 3:] = 255
    assert torch.equal(msa.msa_index_score_q8(q, cache, bt, req, pos, dims), want)
    u8(cache.kidx_scale)[1, 1, 100] = 255                                        # block 0, group 1
    got = msa.msa_index_score_q8(q, cache, bt, req, pos, dims)
    assert bool(torch.isnan(got[0, 1, 0])) and int(torch.isnan(got).sum()) == 1
    u8(cache.kidx_scale)[1, 1, 100] = 127
    q[0, 0, 5] = math.inf
    got = msa.msa_index_score_q8(q, cache, bt, req, pos, dims)
    assert bool(torch.isnan(got[0, 0]).all()) and torch.equal(got[0, 1, 1], want[0, 1, 1])


def test_score_flags(msa):
    dims = msa.Dims(8, 2, 64, 64, 2, 2)
    cache, _ = make_cache(msa, dims, 2, 3)
    q = Q.normal((1, 2, 64), 9).cuda()
    err = msa.new_err_word("cuda")
    for bt, req, pos, flag in (([[0, 1]], 0, 200, 0), ([[0, 2]], 0, 200, 1), ([[0, -1]], 0, 200, 1), ([[0, -1]], 0, 127, 0),
                               ([[0, 1]], 1, 0, 1), ([[0, 1]], -1, 0, 1), ([[0, 1]], 0, -1, 1), ([[0, 1]], 0, 256, 1)):
        msa.msa_index_score_q8(q, cache, i32(bt).cuda(), i32([req]).cuda(), i32([pos]).cuda(), dims, err_word=err)
        assert int(err) == flag, (bt, req, pos)
        err.zero_()


# ------------------------------------------------------------------------------------------------ decode attention

def _paged(msa, Hq, G, D, topk, row_len, seed=1, spread=0.4):
    B = len(row_len)
    dims = msa.Dims(Hq, G, D, 64, topk, 4)
    g = torch.Generator().manual_seed(seed)
    pool = 2 * topk + 3
    table = torch.stack([torch.randperm(pool, generator=g)[:topk] for _ in range(B * G)]).to(torch.int32)
    lens = i32([n for n in row_len for _ in range(G)])
    for r in range(B * G):
        used = (int(lens[r]) + 127) // 128
        table[r, used:] = -1
    parts = [Q.pages(pool, G, D, seed + 7 + i, spread) for i in range(2)]
    cache = msa.CacheQ8(*cuda(*parts[0], *parts[1]))
    return dims, table, lens, cache, [Q.stored(*p) for p in parts], Q.normal((B, Hq, D), seed + 3)


@pytest.mark.parametrize("Hq,G,D,topk,row_len", [
    (16, 2, 128, 4, [0, 1, 31, 32, 33, 127, 128, 129, 500, 512]),
    (16, 4, 64, 3, [384, 1, 200]),
    (8, 2, 128, 32, [4096, 3000]),
    (8, 1, 64, 1, [77]),
    (64, 8, 128, 16, [2048, 1999]),
    (4, 1, 128, 2, list(range(1, 257, 5))),
    (128, 16, 64, 2, [256] * 40),
])
def test_attend(msa, Hq, G, D, topk, row_len):
    dims, table, lens, cache, (k, v), q = _paged(msa, Hq, G, D, topk, row_len)
    err = msa.new_err_word("cuda")
    out, lse = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims, err_word=err)
    msa.msa_check(err)
    o, s, bo, bs = Q.ref_paged(q, k, v, table, lens, 1 / math.sqrt(D))
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("spread", [3.0, 8.0])
def test_attend_rows_of_unlike_scale(msa, spread):
    """Scales that differ by many binades from token to token, and peaked weights."""
    dims, table, lens, cache, (k, v), q = _paged(msa, 16, 2, 128, 4, [500, 130], 2, spread)
    sc = 2.0 ** -8 if spread == 8.0 else 0.05
    dims = msa.Dims(16, 2, 128, 64, 4, 4, sc)
    out, lse = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
    o, s, bo, bs = Q.ref_paged(q, k, v, table, lens, sc)
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40])
def test_attend_huge_logits(msa, scale):
    """Logits whose steps in fp32 are whole numbers or more: the output stays a mean of values that the row sees (here
    mostly one token's), whatever the scales of V."""
    dims, table, lens, cache, (k, v), q = _paged(msa, 16, 2, 128, 4, [500, 130], 2, 3.0)
    dims = msa.Dims(16, 2, 128, 64, 4, 4, scale)
    out, lse = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
    o, s, bo, bs = Q.ref_paged(q, k, v, table, lens, scale)
    Q.assert_within(out, o, bo, "out")
    assert bool(torch.isfinite(lse).all())
    for r in range(4):
        idx = [(int(p), t) for j, p in enumerate(table[r]) for t in range(min(128, int(lens[r]) - j * 128))]
        seen = v[[p for p, _ in idx], r % 2, [t for _, t in idx]]
        got = out[r // 2, r % 2 * 8:r % 2 * 8 + 8].double().cpu()
        top, low = seen.amax(0) * (1 + seen.amax(0).sign() * 2.0 ** -7), seen.amin(0) * (1 - seen.amin(0).sign() * 2.0 ** -7)
        assert bool((got <= top).all()) and bool((got >= low).all())


def test_attend_all_codes(msa):
    """Every finite code, subnormal ones among them, reaches the output: one token seen at a time."""
    dims = msa.Dims(8, 1, 128, 64, 1, 1)
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8)
    k = torch.zeros((2, 1, 128, 128), dtype=torch.uint8)
    v = k.clone()
    v[0, 0, 0], v[1, 0, 0, :126] = codes[:128], codes[128:]
    sc = torch.full((2, 1, 128), 127, dtype=torch.uint8)
    cache = msa.CacheQ8(k.view(E4M3).cuda(), sc.view(E8M0).cuda(), v.view(E4M3).cuda(), sc.view(E8M0).cuda())
    q = Q.normal((2, 8, 128), 1).cuda()
    out, lse = msa.msa_sparse_attn_decode_q8(q, cache, i32([[0], [1]]).cuda(), i32([1, 1]).cuda(), dims)
    want = v.view(E4M3).float()[:, 0, 0]
    assert torch.equal(out.float().cpu(), want[:, None].expand(2, 8, 128))
    assert float(lse.abs().max()) == 0.0


def test_attend_what_is_not_seen_does_not_reach_a_row(msa):
    dims, table, lens, cache, (k, v), q = _paged(msa, 16, 2, 128, 4, [1, 45, 130, 400])
    args = (q.cuda(), cache, *cuda(table, lens), dims)
    want = msa.msa_sparse_attn_decode_q8(*args)
    clean = [u8(x).clone() for x in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    seen = torch.zeros(cache.k.shape[:3], dtype=torch.bool)                      # by any row
    for r in range(table.shape[0]):
        for s in range(4):
            n = min(128, int(lens[r]) - 128 * s)
            if n > 0:
                seen[int(table[r, s]), r % 2, :n] = True
    hide = ~seen.cuda()
    u8(cache.k)[hide], u8(cache.v)[hide] = 0x7f, 0xff
    u8(cache.k_scale)[hide], u8(cache.v_scale)[hide] = 255, 255
    got = msa.msa_sparse_attn_decode_q8(*args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for x, c in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), clean):
        u8(x).copy_(c)
    # a NaN that one row sees makes that row NaN: request 3, group 1
    page = int(table[7, 1])
    others = [r for r in range(8) if r != 7 and r % 2 == 1 and page in table[r, :(int(lens[r]) + 127) // 128].tolist()]
    for x in (cache.v_scale, cache.k_scale):
        old = int(u8(x)[page, 1, 0])
        u8(x)[page, 1, 0] = 255
        got = msa.msa_sparse_attn_decode_q8(*args)
        u8(x)[page, 1, 0] = old
        assert bool(torch.isnan(got[0][3, 8:]).all())
        good = torch.ones((4, 2), dtype=torch.bool)
        good[3, 1] = False
        for r in others:
            good[r // 2, 1] = False
        good = good.repeat_interleave(8, 1).cuda()
        assert torch.equal(got[0][good], want[0][good])


def test_attend_flags_and_empty_slots(msa):
    dims, table, lens, cache, (k, v), q = _paged(msa, 16, 2, 128, 4, [500, 300])
    err = msa.new_err_word("cuda")
    table[1, 1] = -1                                                             # skipped, as in msa_sparse_attn_decode
    out, lse = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims, err_word=err)
    msa.msa_check(err)
    o, s, bo, bs = Q.ref_paged(q, k, v, table, lens, 1 / math.sqrt(128))
    Q.assert_within(out, o, bo, "out")
    table[2, 0] = cache.k.shape[0]
    msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims, err_word=err)
    assert int(err) == 1


def test_attend_of_q_that_is_not_finite(msa):
    dims, table, lens, cache, _, q = _paged(msa, 16, 2, 128, 2, [200])
    want = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
    q[0, 5, 9] = math.inf
    got = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
    assert bool(torch.isnan(got[0][0, 5]).all()) and bool(torch.isnan(got[1][0, 5]))
    keep = [h for h in range(16) if h != 5]
    assert torch.equal(got[0][0, keep], want[0][0, keep])


def test_attend_as_the_bf16_call_on_pages_read_back(msa):
    dims, table, lens, cache, _, q = _paged(msa, 64, 8, 128, 16, [2048, 1000, 5])
    n = cache.k.shape[0]
    ids = torch.arange(n, dtype=torch.int32).cuda()[None]
    d2 = msa.Dims(64, 8, 128, 64, 16, n)
    pages = [torch.empty((n, 128, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_cache_read_q8(cache, ids, ids, i32([n * 128]).cuda(), d2, *pages)
    a, la = msa.msa_sparse_attn_decode_q8(q.cuda(), cache, *cuda(table, lens), dims)
    b, lb = msa.msa_sparse_attn_decode(q.cuda(), *pages, *cuda(table, lens), dims)
    # both round P and the output to bf16
    assert float((a.float() - b.float()).abs().max()) < 4 * 2.0 ** -8 * float(b.float().abs().max())
    assert float((la - lb).abs().max()) < 1e-4


# ------------------------------------------------------------------------------------------------ window

WINDOWS = [
    # Hq, G, D, ctx, rows each, window, sinks, pad
    (16, 2, 128, [0], 1, 1, 0, 0),
    (16, 2, 128, [300, 5], 3, 64, 4, 2),
    (16, 4, 64, [1000], 2, 129, 130, 0),
    (8, 1, 64, [511, 128], 1, 1 << 30, 0, 1),
    (8, 2, 128, [700], 2, 33, 40, 0),
    (64, 8, 128, [2000, 31, 64], 1, 512, 1, 0),
    (8, 2, 64, [250], 1, 200, 300, 0),
    (16, 2, 128, [96], 70, 32, 31, 5),
    (4, 1, 64, [0, 3], 40, 7, 2, 1),
    (8, 1, 64, [9000], 2, 1 << 30, 0, 0),
    (8, 1, 128, [8300, 20], 1, 8200, 50, 0),
]


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("Hq,G,D,ctx,n,window,sinks,pad", WINDOWS)
def test_window(msa, phase, Hq, G, D, ctx, n, window, sinks, pad):
    bt, pool = Q.tables([c + n for c in ctx], 1, extra_blocks=1)
    dims = msa.Dims(Hq, G, D, 64, 1, bt.shape[1])
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    R = len(ctx) * n + pad
    req = i32([b for b in range(len(ctx)) for _ in range(n)] + [-1] * pad)
    pos = i32([c + i for c in ctx for i in range(n)] + [-1] * pad)
    q = Q.normal((R, Hq, D), 5)
    # blocks that no row sees may have no page
    for b, c in enumerate(ctx):
        for j in range(bt.shape[1]):
            if (j + 1) * 128 <= c - window + 1 and j * 128 >= sinks:
                bt[b, j] = -1
    out = torch.zeros((R, Hq, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((R, Hq), device="cuda")
    err = msa.new_err_word("cuda")
    msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), window, sinks, dims, phase, out, lse, err_word=err)
    msa.msa_check(err)
    o, s, bo, bs = Q.ref_window(q, k, v, bt, req, pos, window, sinks, 1 / math.sqrt(D))
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("exp", [-100, -7, 0, 9, 60])
def test_window_all_codes(msa, phase, exp):
    """Every finite code in V, subnormal ones among them, under small and large scales: rows that see one token."""
    dims = msa.Dims(8, 1, 128, 64, 1, 2)
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8)
    k = torch.zeros((2, 1, 128, 128), dtype=torch.uint8)
    v = k.clone()
    v[0, 0, 0], v[1, 0, 0, :126] = codes[:128], codes[128:]
    sc = torch.full((2, 1, 128), 127 + exp, dtype=torch.uint8)
    cache = msa.CacheQ8(k.view(E4M3).cuda(), sc.view(E8M0).cuda(), v.view(E4M3).cuda(), sc.view(E8M0).cuda())
    q = Q.normal((2, 8, 128), 1).cuda()
    out, lse = msa.msa_window_attn_q8(q, cache, i32([[0, 1]]).cuda(), i32([0, 0]).cuda(), i32([0, 128]).cuda(), 1, 0, dims,
                                      phase)
    want = v.view(E4M3).float()[:, 0, 0] * 2.0 ** exp
    assert torch.equal(out.float().cpu(), want[:, None].expand(2, 8, 128))
    assert float(lse.abs().max()) == 0.0


@pytest.mark.parametrize("phase", [0, 1])
def test_window_all_key_codes(msa, phase):
    """Every finite code in K: the log-sum of a row that sees one token is its logit."""
    dims = msa.Dims(8, 1, 128, 64, 1, 2, 1.0)
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8)
    k = torch.zeros((2, 1, 128, 128), dtype=torch.uint8)
    flat = k[:, 0].reshape(-1, 128)
    flat[torch.arange(254), torch.arange(254) % 128] = codes
    one = torch.full((2, 1, 128), 127, dtype=torch.uint8)
    cache = msa.CacheQ8(k.view(E4M3).cuda(), one.view(E8M0).cuda(), torch.zeros_like(k).view(E4M3).cuda(),
                        one.view(E8M0).cuda())
    q = torch.zeros((254, 8, 128), dtype=torch.bfloat16)
    q[torch.arange(254), :, torch.arange(254) % 128] = 1.0
    out, lse = msa.msa_window_attn_q8(q.cuda(), cache, i32([[0, 1]]).cuda(), i32([0] * 254).cuda(),
                                      torch.arange(254, dtype=torch.int32).cuda(), 1, 0, dims, phase)
    want = codes.view(E4M3).float()[:, None].expand(254, 8)
    assert float((lse.cpu() - want).abs().max() / 448) < 2.0 ** -22 and bool((out == 0).all())
    assert float(((lse.cpu() - want).abs() / want.abs().clamp(min=2.0 ** -9)).max()) < 2.0 ** -20


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 1)])
@pytest.mark.parametrize("shape", ["rising", "falling", "teeth"])
@pytest.mark.parametrize("size", [-60, 0, 70])
def test_window_logits_far_apart(msa, phase, D, G, shape, size):
    """Logits that pass one another by far within a page and from page to page, upwards in every other head and
    downwards in the rest, over small and large values."""
    n = 700
    bt, pool = Q.tables([n], 1)
    t = torch.arange(n)
    a = {"rising": t / 4, "falling": (n - t) / 4, "teeth": (t % 96) * 1.0}[shape].double()
    k = torch.zeros((pool, G, 128, D)).double()
    k[bt[0].long()[t // 128], :, t % 128] = a[:, None, None].expand(n, G, D)
    v = Q.normal((pool, G, 128, D), 2).double() * 2.0 ** size
    kc, vc = Q.to_cache(k), Q.to_cache(v)
    cache = msa.CacheQ8(*cuda(*kc, *vc))
    R = 150
    q = (Q.normal((R, 8 * G, D), 3, 0.05).float() + (1.0 - 2.0 * (torch.arange(8 * G) % 2))[:, None]).to(torch.bfloat16)
    req, pos = i32([0] * R), torch.arange(n - R, n, dtype=torch.int32)
    dims = msa.Dims(8 * G, G, D, 64, 1, bt.shape[1], 1.0 / D)
    out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 400, 5, dims, phase)
    o, s, bo, bs = Q.ref_window(q, Q.stored(*kc), Q.stored(*vc), bt, req, pos, 400, 5, 1.0 / D)
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40])
def test_window_huge_logits_of_chunks(msa, scale):
    """As of decode rows: with logits whose steps in fp32 are whole numbers or more, the output stays a mean of values
    that the row sees."""
    n, dims = 300, msa.Dims(16, 2, 128, 64, 1, 3, scale)
    bt, pool = Q.tables([n], 1)
    cache, (k, v, _) = make_cache(msa, dims, pool, 2)
    q = Q.normal((n, 16, 128), 3)
    req, pos = i32([0] * n), torch.arange(n, dtype=torch.int32)
    out, lse = msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 100, 0, dims, msa.MSA_PHASE_PREFILL)
    assert bool(torch.isfinite(lse).all())
    for r in range(0, n, 7):
        t = torch.arange(max(0, r - 99), r + 1)
        for g in range(2):
            seen = v[bt[0].long()[t // 128], g, t % 128]
            got = out[r, 8 * g:8 * g + 8].double().cpu()
            top, low = seen.amax(0), seen.amin(0)
            top, low = top * (1 + top.sign() * 2.0 ** -7), low * (1 - low.sign() * 2.0 ** -7)
            assert bool((got <= top).all()) and bool((got >= low).all())


@pytest.mark.parametrize("phase", [0, 1])
def test_window_rows_in_any_order(msa, phase):
    """Rows of several requests, shuffled, with padding among them; one row twice."""
    bt, pool = Q.tables([400, 260, 150], 1)
    dims = msa.Dims(16, 2, 128, 64, 1, bt.shape[1])
    cache, (k, v, _) = make_cache(msa, dims, pool, 3)
    rows = [(0, 399), (2, 0), (1, 259), (-1, 0), (0, 3), (2, 149), (0, 200), (0, 399), (1, 100), (2, 77), (-1, 5)] + \
        [(b, p) for b, p in zip([0, 1, 2] * 10, range(100, 130))]
    req, pos = i32([b for b, _ in rows]), i32([p for _, p in rows])
    q = Q.normal((len(rows), 16, 128), 5)
    out = torch.zeros((len(rows), 16, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((len(rows), 16), device="cuda")
    msa.msa_window_attn_q8(q.cuda(), cache, *cuda(bt, req, pos), 90, 3, dims, phase, out, lse)
    o, s, bo, bs = Q.ref_window(q, k, v, bt, req, pos, 90, 3, 1 / math.sqrt(128))
    Q.assert_within(out, o, bo, "out")
    Q.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("phase", [0, 1])
def test_window_what_is_not_seen_does_not_reach_a_row(msa, phase):
    """NaN before the window, between sinks and window, behind the row and in another row's token."""
    bt, pool = Q.tables([600], 1)
    dims = msa.Dims(16, 2, 128, 64, 1, bt.shape[1])
    cache, _ = make_cache(msa, dims, pool, 3)
    pos = [500 + 3 * i for i in range(20)]
    q = Q.normal((20, 16, 128), 5).cuda()
    args = (i32([0] * 20).cuda(), i32(pos).cuda(), 100, 5, dims, phase)
    want = msa.msa_window_attn_q8(q, cache, bt.cuda(), *args)
    assert bool(torch.isfinite(want[0].float()).all())
    for t in list(range(5, 401)) + list(range(558, 600)):
        page = int(bt[0, t // 128])
        u8(cache.k)[page, :, t % 128], u8(cache.v)[page, :, t % 128] = 0xff, 0x7f
        u8(cache.k_scale)[page, :, t % 128] = u8(cache.v_scale)[page, :, t % 128] = 255
    got = msa.msa_window_attn_q8(q, cache, bt.cuda(), *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    page = int(bt[0, 557 // 128])                                                # the last row's own token
    for x in (cache.v_scale, cache.k_scale):
        old = int(u8(x)[page, 0, 557 % 128])
        u8(x)[page, 0, 557 % 128] = 255
        got = msa.msa_window_attn_q8(q, cache, bt.cuda(), *args)
        u8(x)[page, 0, 557 % 128] = old
        assert bool(torch.isnan(got[0][19, :8]).all())
        assert torch.equal(got[0][:19], want[0][:19]) and torch.equal(got[0][19, 8:], want[0][19, 8:])
    page = int(bt[0, 450 // 128])                                                # seen by the rows up to 549
    u8(cache.v_scale)[page, 1, 450 % 128] = 255
    got = msa.msa_window_attn_q8(q, cache, bt.cuda(), *args)
    for i, p in enumerate(pos):
        if p < 550:
            assert bool(torch.isnan(got[0][i, 8:]).all()) and torch.equal(got[0][i, :8], want[0][i, :8])
        else:
            assert torch.equal(got[0][i], want[0][i])


@pytest.mark.parametrize("phase", [0, 1])
def test_window_flags(msa, phase):
    bt, pool = Q.tables([300], 1)
    dims = msa.Dims(16, 2, 128, 64, 1, bt.shape[1])
    cache, _ = make_cache(msa, dims, pool, 3)
    q = Q.normal((1, 16, 128), 5).cuda()
    err = msa.new_err_word("cuda")
    gone, past = bt.clone(), bt.clone()
    gone[0, 1], past[0, 1] = -1, pool
    for table, req, p, window, sinks, flag in ((bt, 0, 299, 300, 0, 0), (gone, 0, 299, 300, 0, 1), (past, 0, 299, 300, 0, 1),
                                               (gone, 0, 299, 44, 128, 0), (gone, 0, 299, 44, 129, 1), (bt, 1, 0, 5, 0, 1),
                                               (bt, -2, 0, 5, 0, 1), (bt, 0, -1, 5, 0, 1), (bt, 0, 384, 5, 0, 1)):
        msa.msa_window_attn_q8(q, cache, table.cuda(), i32([req]).cuda(), i32([p]).cuda(), window, sinks, dims, phase,
                               err_word=err)
        assert int(err) == flag, (req, p, window, sinks)
        err.zero_()


# ------------------------------------------------------------------------------------------------ together

def _loop_case(msa, lens, Hq=32, G=4, D=128, Di=64, topk=4, steps=3):
    bt, pool = Q.tables([n + steps for n in lens], 1)
    dims = msa.Dims(Hq, G, D, Di, topk, bt.shape[1])
    return dims, bt, pool


def test_step_is_the_separate_calls(msa):
    dims, bt, pool = _loop_case(msa, [700, 129, 2000, 1])
    cache, _ = make_cache(msa, dims, pool, 3)
    B, lens = 4, i32([701, 130, 2001, 2]).cuda()
    q, qi = Q.normal((B, 32, 128), 1).cuda(), Q.normal((B, 4, 64), 2).cuda()
    out, lse, sel, pt, row_len, scores = msa.msa_decode_step_q8(q, qi, cache, bt.cuda(), lens, dims)
    req = torch.arange(B, dtype=torch.int32).cuda()
    s2 = msa.msa_index_score_q8(qi, cache, bt.cuda(), req, lens - 1, dims)
    sel2 = msa.msa_topk_blocks(s2, lens - 1, dims)
    pt2, rl2 = msa.msa_build_page_table(sel2, bt.cuda(), lens, pool, dims)
    o2, l2 = msa.msa_sparse_attn_decode_q8(q, cache, pt2, rl2, dims)
    for x, y in ((scores, s2), (sel, sel2), (pt, pt2), (row_len, rl2), (out, o2), (lse, l2)):
        assert torch.equal(x, y)
    host = torch.empty((B, 32, 128), dtype=torch.bfloat16).pin_memory(), torch.empty((B, 32)).pin_memory()
    msa.msa_decode_step_q8(q, qi, cache, bt.cuda(), lens, dims, out=host[0], lse=host[1])
    torch.cuda.synchronize()
    assert torch.equal(host[0], out.cpu()) and torch.equal(host[1], lse.cpu())


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(msa, captured):
    """A prompt appended in two chunks and attended through pages read back, then tokens decoded one by one: every
    result against 64 bits computed from what the caches hold and from the unrotated inputs."""
    steps, lens = 3, [300, 129]
    dims, bt, pool = _loop_case(msa, lens, steps=steps)
    B, G, D, Di, Hq = 2, 4, 128, 64, 32
    cache = msa.CacheQ8.zeros(dims, pool, "cuda")
    rope = msa.Rope.of_base(64, 32, scaling="yarn", factor=8.0, original_len=128, device="cuda")
    f, gain = msa.rope_inv_freq(64, scaling="yarn", factor=8.0, original_len=128)
    err = msa.new_err_word("cuda")
    bt_d = bt.cuda()
    # the prompt, in chunks that end anywhere
    total = sum(lens)
    req = i32([b for b, n in enumerate(lens) for _ in range(n)])
    pos = i32([i for n in lens for i in range(n)])
    x = [Q.normal((total, h, w), 30 + i) for i, (h, w) in enumerate(((Hq, D), (G, D), (G, D), (G, Di), (G, Di)))]
    rot = torch.empty((total, Hq, D), dtype=torch.bfloat16).cuda()
    for a, z in ((0, 201), (201, total)):
        part = [t[a:z].cuda() for t in x]
        qo, qio = msa.msa_rope_append_q8(*part, cache, bt_d, req[a:z].cuda(), pos[a:z].cuda(), rope, dims, err_word=err)
        rot[a:z] = qo
    msa.msa_check(err)
    yk, tk = Q.rotated(x[1], 64, f, pos.long(), False, gain)
    page, slot = bt.long()[req.long(), pos.long() // 128], pos.long() % 128
    Q.check_rows8(u8(cache.k).cpu()[page, :, slot].view(E4M3), u8(cache.k_scale).cpu()[page, :, slot].view(E8M0), yk, tk,
                  "k")
    # prefill of the last rows over pages read back
    out_pages = [torch.zeros((pool, 128, G, w), dtype=torch.bfloat16, device="cuda") for w in (D, D, Di)]
    msa.msa_cache_read_q8(cache, bt_d, bt_d, i32(lens).cuda(), dims, *out_pages, err_word=err)
    tail = torch.arange(total - 40, total)
    pre = msa.PrefillStep(dims, 40, B, "cuda")
    o, lse = pre(rot[tail], qio[-40:], *out_pages, bt_d, req[tail].cuda(), pos[tail].cuda())
    msa.msa_check(pre.err)
    vals = [Q.stored(c.cpu(), s.cpu()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    sel = pre.sel.cpu()
    for i, r in enumerate(tail.tolist()[::13]):
        i *= 13
        for g in range(G):
            blocks = [int(j) for j in sel[i, g] if j >= 0]
            t = torch.tensor([t for j in blocks for t in range(j * 128, min(j * 128 + 128, int(pos[r]) + 1))])
            pg, sl = bt[int(req[r])].long()[t // 128], t % 128
            want, _, tol, _ = Q.ref_attend(Q.f64(rot[r, g * 8:(g + 1) * 8].cpu()), vals[0][pg, g, sl], vals[1][pg, g, sl],
                                           1 / math.sqrt(D))
            # partials are rounded to bf16 once more
            Q.assert_within(o[i, g * 8:(g + 1) * 8], want, tol + 2.0 ** -8 * vals[1][pg, g, sl].abs().amax(0), "prefill")
    # decode, in a window layer of the same caches too
    step = msa.DecodeStepQ8(dims, B, "cuda", rope)
    bufs = [torch.zeros((B, h, w), dtype=torch.bfloat16, device="cuda") for h, w in ((Hq, D), (G, D), (G, D), (G, Di), (G, Di))]
    p, n = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def fill(k):
        for i, b in enumerate(bufs):
            b.copy_(Q.normal(tuple(b.shape), 100 * k + i))
        p.copy_(i32([m + k for m in lens]))
        n.copy_(p + 1)

    fill(0)
    if captured:
        step.capture(*bufs, cache, bt_d, p, n)
    for k in range(steps):
        fill(k)
        out, lse = step.replay() if captured else step.step(*bufs, cache, bt_d, p, n)
        w_out, w_lse = msa.msa_window_attn_q8(step.q, cache, bt_d, step.q_req, p, 140, 4, dims, msa.MSA_PHASE_DECODE,
                                              err_word=err)
        msa.msa_check(step.err)
        msa.msa_check(err)
        yq, tq = Q.rotated(bufs[0].cpu(), 64, f, p.cpu().long(), False, gain)
        Q.assert_within(step.q, yq, tq + (yq.abs() + tq) * 2.0 ** -8, "q")
        s, ts = Q.ref_scores(step.q_idx.cpu(), cache.kidx.cpu(), cache.kidx_scale.cpu(), bt, range(B), p.tolist())
        Q.assert_within(step.scores, s, ts, "scores")
        vals = [Q.stored(c.cpu(), s.cpu()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        o, l, bo, bl = Q.ref_paged(step.q.cpu(), *vals, step.page_table.cpu(), step.row_len.cpu(), 1 / math.sqrt(D))
        Q.assert_within(out, o, bo, "out")
        Q.assert_within(lse, l, bl, "lse")
        o, l, bo, bl = Q.ref_window(step.q.cpu(), *vals, bt, range(B), p.tolist(), 140, 4, 1 / math.sqrt(D))
        Q.assert_within(w_out, o, bo, "window out")
        Q.assert_within(w_lse, l, bl, "window lse")


def test_on_another_stream(msa):
    dims, bt, pool = _loop_case(msa, [500, 60])
    cache, _ = make_cache(msa, dims, pool, 3)
    q, qi, lens = Q.normal((2, 32, 128), 1).cuda(), Q.normal((2, 4, 64), 2).cuda(), i32([501, 61]).cuda()
    bt = bt.cuda()
    want = msa.msa_decode_step_q8(q, qi, cache, bt, lens, dims)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a, b = torch.zeros_like(q), torch.zeros_like(qi)
    big = torch.empty(1 << 28, device="cuda")
    with torch.cuda.stream(side):
        big.normal_()                                                            # the copies wait behind it
        a.copy_(q)
        b.copy_(qi)
        got = msa.msa_decode_step_q8(a, b, cache, bt, lens, dims)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_results_do_not_depend_on_timing(msa):
    dims, table, lens, cache, _, q = _paged(msa, 64, 8, 128, 16, [2048, 1999, 700])
    args = (q.cuda(), cache, *cuda(table, lens), dims)
    first = msa.msa_sparse_attn_decode_q8(*args)
    for _ in range(20):
        got = msa.msa_sparse_attn_decode_q8(*args)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_pages_past_32_bits(msa):
    """Pages whose codes, and whose bf16 rows, lie past 2^32 bytes: every call as on the same pages in front."""
    dims = msa.Dims(64, 8, 128, 64, 4, 4)
    bt, pool = Q.tables([500], 1)
    small, _ = make_cache(msa, dims, pool, 3)
    far, n_out = 33000, 17000
    assert (far - pool) * 8 * 128 * 128 > 1 << 32 and (n_out - pool) * 128 * 8 * 128 * 2 > 1 << 32
    fields = ("k", "k_scale", "v", "v_scale", "kidx", "kidx_scale")

    def moved(x):
        big = torch.empty((far, *x.shape[1:]), dtype=torch.uint8, device="cuda")
        big[far - pool:] = u8(x)
        return big.view(x.dtype)
    large = msa.CacheQ8(*(moved(getattr(small, f)) for f in fields))
    tables = bt.cuda(), torch.where(bt >= 0, bt + (far - pool), bt).cuda()
    rows = [Q.normal((3, 64 if i == 0 else 8, 64 if i > 2 else 128), 40 + i).cuda() for i in range(5)]
    req, pos, lens = i32([0] * 3).cuda(), i32([497, 498, 499]).cuda(), i32([500]).cuda()
    rope = msa.Rope.of_base(64, 32)
    got = []
    for cache, table in zip((small, large), tables):
        res = list(msa.msa_rope_append_q8(*rows, cache, table, req, pos, rope, dims))
        q, qi = res
        page = table[0, 3].item()
        res += [u8(getattr(cache, f)[page].contiguous()) for f in fields]
        res.append(msa.msa_index_score_q8(qi, cache, table, req, pos, dims))
        res += msa.msa_decode_step_q8(q[2:].contiguous(), qi[2:].contiguous(), cache, table, lens, dims)[:2]
        for phase in (0, 1):
            res += msa.msa_window_attn_q8(q, cache, table, req, pos, 300, 5, dims, phase)
        base = 0 if cache is small else n_out - pool
        n = pool if cache is small else n_out
        out = [torch.empty((n, 128, 8, w), dtype=torch.bfloat16, device="cuda") for w in (128, 128, 64)]
        to = torch.where(bt >= 0, bt + base, bt).cuda()
        for x in out:
            x[base:] = 0
        msa.msa_cache_read_q8(cache, table, to, lens, dims, *out)
        msa.msa_rope_append(*rows, *out, to, req, pos - 200, rope, dims)
        res += [x[base:].clone() for x in out]
        got.append(res)
    for i, (x, y) in enumerate(zip(*got)):
        assert torch.equal(x, y), i


def test_calls_of_no_rows(msa):
    dims = msa.Dims(16, 2, 128, 64, 2, 4)
    cache = msa.CacheQ8.zeros(dims, 3, "cuda")
    bt = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    none = torch.zeros((0,), dtype=torch.int32, device="cuda")
    rows = [torch.zeros((0, h, w), dtype=torch.bfloat16, device="cuda")
            for h, w in ((16, 128), (2, 128), (2, 128), (2, 64), (2, 64))]
    msa.msa_rope_append_q8(*rows, cache, bt, none, none, msa.Rope(0), dims)
    assert msa.msa_index_score_q8(rows[3], cache, bt, none, none, dims).numel() == 0
    for phase in (0, 1):
        out, lse = msa.msa_window_attn_q8(rows[0], cache, bt, none, none, 5, 1, dims, phase)
        assert out.numel() == 0 and lse.numel() == 0
    out, lse = msa.msa_sparse_attn_decode_q8(rows[0], cache, bt.new_zeros((0, 2)), none, dims)
    assert out.numel() == 0 and lse.numel() == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("D,G", [(128, 2), (64, 1)])
def test_window_captured_and_two_at_once(msa, phase, D, G):
    """Two graphs over the same caches, replayed side by side on what their tensors then hold."""
    dims = msa.Dims(8 * G, G, D, 64, 1, 8)
    bt, pool = Q.tables([1000], 1)
    bt = torch.cat([bt, bt.flip(1)])[:, :8].contiguous()
    cache, _ = make_cache(msa, dims, pool, 3)
    sets = []
    for k in range(2):
        q = torch.zeros((200, 8 * G, D), dtype=torch.bfloat16, device="cuda")
        table, req = bt.clone().cuda(), torch.zeros(200, dtype=torch.int32, device="cuda")
        pos = torch.zeros(200, dtype=torch.int32, device="cuda")
        args = (q, cache, table, req, pos, 333, 7, dims, phase)
        out, lse = msa.msa_window_attn_q8(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            msa.msa_window_attn_q8(*args, out, lse)
        sets.append((graph, args, out, lse, torch.cuda.Stream()))
    for k, (_, args, _, _, _) in enumerate(sets):
        args[0].copy_(Q.normal((200, 8 * G, D), 50 + k))
        args[3].copy_(i32([k] * 190 + [-1] * 10))
        args[4].copy_(torch.arange(700 + 50 * k, 900 + 50 * k, dtype=torch.int32))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, _, _, _, stream in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, args, out, lse, _ in sets:
        want = msa.msa_window_attn_q8(*args)
        assert torch.equal(out[:190], want[0][:190]) and torch.equal(lse[:190], want[1][:190])


def test_two_captured_steps_at_once(msa):
    """Two steps of their own buffers and caches, replayed side by side."""
    dims = msa.Dims(16, 2, 128, 64, 2, 4)
    bt, pool = Q.tables([300, 400], 1)
    steps = []
    for k in range(2):
        cache, _ = make_cache(msa, dims, pool, 3 + 10 * k)
        step = msa.DecodeStepQ8(dims, 2, "cuda", msa.Rope.of_base(64, 32))
        rows = [Q.normal((2, 16 if i == 0 else 2, 64 if i > 2 else 128), 60 + 10 * k + i).cuda() for i in range(5)]
        args = (*rows, cache, bt.cuda(), i32([299, 399]).cuda(), i32([300, 400]).cuda())
        step.capture(*args)
        steps.append((step, args, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for step, _, stream in steps:
            with torch.cuda.stream(stream):
                step.replay()
    torch.cuda.synchronize()
    for step, args, _ in steps:
        got = step.out.clone(), step.lse.clone()
        want = step.step(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
