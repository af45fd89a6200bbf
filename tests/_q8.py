"""8-bit caches: small seeded cases and their plain references in 64 bits (CPU), with error bounds.

Bounds are derived, not fitted.  e4m3 has four significant bits: a code is off by at most 2^-4 of a normal value, and by
half of the lowest step, 2^-10 in units of the scale, below 2^-6.  A rounding to bf16 is off by at most 2^-8 of the
value.  The MMAs' products (of f16 or bf16 factors) are exact; an fp32 sum of W terms is off by at most W * 2^-23 of the
sum of their magnitudes, in any order and with truncating adders."""
from __future__ import annotations

import torch

PAGE = 128
LOWEST = -100


def f64(x):
    """bf16, e4m3 or e8m0 as 64 bits."""
    return x.float().double()


def exponent(amax):
    """Exponent of a row's scale: smallest e >= LOWEST with amax <= 448 * 2^e; 0 for a row of zeros."""
    out = torch.zeros(amax.shape, dtype=torch.int64)
    e = LOWEST
    todo = amax > 0
    while bool(todo.any()):
        fits = todo & (amax <= 448.0 * 2.0 ** e)
        out[fits] = e
        todo &= ~fits
        e += 1
    return out


def step_of(y):
    """Distance of neighbouring e4m3 numbers at |y| (in units of the scale)."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)


def quantise(x):
    """(codes as values, exponents) of rows in 64 bits: nearest, ties to even."""
    e = exponent(x.abs().amax(-1))
    y = x * torch.exp2(-e.double())[..., None]
    step = step_of(y)
    return torch.round(y / step) * step, e


def to_cache(x):
    """Rows [pages][G][128][width] in 64 bits -> (e4m3 codes, e8m0 scales) tensors."""
    code, e = quantise(x)
    return code.float().to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def stored(code, scale):
    return f64(code) * f64(scale)[..., None]


def tables(lens, seed, extra_blocks=0, spare=2, first=None):
    """Block table of pages in random order for tokens [first, len) of each request (-1 elsewhere), pool size."""
    g = torch.Generator().manual_seed(seed)
    first = [0] * len(lens) if first is None else first
    last = [(n + PAGE - 1) // PAGE for n in lens]
    pool = sum(b - a // PAGE for a, b in zip(first, last)) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    bt = torch.full((len(lens), max(max(last), 1) + extra_blocks), -1, dtype=torch.int32)
    at = 0
    for b, (a, z) in enumerate(zip(first, last)):
        bt[b, a // PAGE:z] = perm[at:at + z - a // PAGE]
        at += z - a // PAGE
    return bt, pool


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def pages(pool, G, width, seed, spread=0.4):
    """Quantised rows of unlike size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((pool, G, PAGE, width), generator=g).double()
    return to_cache(x * torch.exp(spread * torch.randn((pool, G, PAGE, 1), generator=g).double()))


def rotated(x, rot, inv_freq, pos, interleaved, gain):
    """(rows rotated in 64 bits, bound of an fp32 rotation) of x [R][heads][width]."""
    x = f64(x)
    y, tol = x.clone(), torch.zeros_like(x)
    if rot:
        w = pos.double()[:, None, None] * inv_freq
        i = torch.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = gain * torch.cos(w), gain * torch.sin(w)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        # the cosine and the sine, the gain, two products and a sum, each below 2^-23 of |a| + |b|, and 2^-22 besides (the
        # cosine and the sine are known far better than that: test_gpu_q8_edges.py holds them to their last bit)
        tol[..., a] = tol[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(gain) * (2.0 ** -22 + 6 * 2.0 ** -23)
    return y, tol


def check_rows8(code, scale, want, tol, what):
    """Stored rows against rows in 64 bits that the writer knew within tol: a scale of some row that near, and codes
    within half a step."""
    amax, slack = want.abs().amax(-1), tol.amax(-1)
    e = torch.log2(f64(scale)).round().long()
    lo, hi = exponent((amax - slack).clamp(min=0)), exponent(amax + slack)
    ok = (e == lo) | (e == hi)
    assert bool(ok.all()), f"{what}: scale {e[~ok][:4].tolist()}, expected {lo[~ok][:4].tolist()}"
    unit = torch.exp2(e.double())[..., None]
    y = want / unit
    # half a step at the value, or at its neighbour above where tol reaches the next binade
    half = step_of(y.abs() + tol / unit) / 2
    off = (f64(code) - y).abs() - (half + tol / unit)
    assert float(off.max()) <= 0, f"{what}: code off by {float(off.max()):.3e} more than its rounding"


def ref_scores(q_idx, kidx, kscale, bt, req, pos):
    """(scores, bound) in 64 bits [rows][G][max_blocks]."""
    R, G, Di = q_idx.shape
    s = torch.full((R, G, bt.shape[1]), -torch.inf, dtype=torch.float64)
    tol = torch.zeros_like(s)
    k = stored(kidx, kscale)
    for r in range(R):
        q = f64(q_idx[r])
        for j in range(int(pos[r]) // PAGE + 1):
            n = min(PAGE, int(pos[r]) + 1 - j * PAGE)
            x = k[int(bt[req[r], j]), :, :n]
            s[r, :, j] = torch.einsum("gd,gtd->gt", q, x).amax(-1)
            # q in f16, the largest component in [2^14, 2^15): half of the lowest step, 2^-25, is under 2^-39 of it;
            # fp32 sums
            mag = torch.einsum("gd,gtd->gt", q.abs(), x.abs()) * 1.2 * (Di + 8) * 2.0 ** -23
            lost = q.abs().amax(-1)[:, None] * x.abs().sum(-1) * 2.0 ** -39
            tol[r, :, j] = (mag + lost).amax(-1)
    return s, tol


def ref_attend(q, k, v, sm_scale):
    """(out, lse, bounds) of heads q [h][D] over the tokens k, v [t][D] (64 bits) that they see."""
    D, n = q.shape[1], k.shape[0]
    if n == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), -torch.inf, dtype=torch.float64), z, torch.zeros(q.shape[0]).double()
    s = q @ k.T * sm_scale
    # the dot product's sum, its factors' roundings, q in f16, and the exponent's argument in log2 units
    ds = ((q.abs() @ k.abs().T) * sm_scale * (D + 16) * 1.2 * 2.0 ** -23).amax(-1) + s.abs().amax(-1) * 2.0 ** -22
    ds += q.abs().amax(-1) * k.abs().sum(-1).max() * sm_scale * 2.0 ** -39 + 2.0 ** -20
    p = torch.softmax(s, -1)
    o, lse = p @ v, torch.logsumexp(s, -1)
    mass = p @ v.abs()
    tol = mass * (2.0 ** -8 + 2 * ds[:, None] + n * 2.0 ** -23) * 1.01 + o.abs() * 2.0 ** -8
    # weights below 2^-126 of the largest are flushed
    tol = tol + v.abs().amax(0) * n * 2.0 ** -125
    return o, lse, tol, 2 * ds + lse.abs() * 2.0 ** -21


def ref_paged(q, k, v, table, row_len, sm_scale):
    """Decode attention over page tables: q [B][Hq][D], stored pages k, v [pages][G][128][D]; table [B*G][topk]."""
    B, Hq, D = q.shape
    G = k.shape[1]
    hpg = Hq // G
    res = [torch.zeros((B, Hq, D)).double(), torch.zeros((B, Hq)).double(), torch.zeros((B, Hq, D)).double(),
           torch.zeros((B, Hq)).double()]
    for r in range(B * G):
        b, g = r // G, r % G
        idx = [(int(p), t) for s, p in enumerate(table[r]) for t in range(min(PAGE, int(row_len[r]) - s * PAGE)) if p >= 0]
        page, slot = torch.tensor([i for i, _ in idx]).long(), torch.tensor([t for _, t in idx]).long()
        h = slice(g * hpg, (g + 1) * hpg)
        for x, y in zip(res, ref_attend(f64(q[b, h]), k[page, g, slot], v[page, g, slot], sm_scale)):
            x[b, h] = y
    return res


def ref_window(q, k, v, bt, req, pos, window, n_sink, sm_scale):
    """Rows with req -1 keep zeros; the bounds of the others."""
    R, Hq, D = q.shape
    G = k.shape[1]
    hpg = Hq // G
    res = [torch.zeros((R, Hq, D)).double(), torch.zeros((R, Hq)).double(), torch.zeros((R, Hq, D)).double(),
           torch.zeros((R, Hq)).double()]
    for r in range(R):
        if int(req[r]) < 0:
            continue
        p = int(pos[r])
        t = torch.tensor(sorted(set(range(min(n_sink, p + 1))) | set(range(max(0, p - window + 1), p + 1))))
        page, slot = bt[int(req[r])].long()[t // PAGE], t % PAGE
        for g in range(G):
            h = slice(g * hpg, (g + 1) * hpg)
            for x, y in zip(res, ref_attend(f64(q[r, h]), k[page, g, slot], v[page, g, slot], sm_scale)):
                x[r, h] = y
    return res


def assert_within(got, want, bound, what):
    got = got.detach().cpu().double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    d = (got[~inf] - want[~inf]).abs() - bound[~inf]
    assert not bool(torch.isnan(d).any()), f"{what}: NaN"
    assert d.numel() == 0 or float(d.max()) <= 0, f"{what}: {int((d > 0).sum())} outside the bound by {float(d.max()):.3e}"
