"""An 8-bit paged cache: the operators that write it, read it back and attend over it, as measured cases.

A serving step rotates the projected queries, keys and index vectors to their positions and appends the new tokens'
K, V and index keys to the paged caches.  In 8 bits a cached row (one token, one group) is stored as e4m3 codes and
one power-of-two scale, so a page takes half the bytes and every stored value is also a bf16 value.  Five operators
are measured here, each by a plain form in elementary torch operations and by the framework's own calls (`own`):

  append   msa_rope_append (bf16 caches), msa_rope_append_q8: rotary positions and the write into the caches
  read     msa_cache_read_q8: blocks of the 8-bit caches as bf16 pages, as a prefill chunk takes them
  score    msa_index_score_q8: block scores of decode rows over 8-bit index keys
  attend   msa_sparse_attn_decode_q8: decode attention over the pages of the selected blocks
  window   msa_window_attn_q8: attention to the last `window` tokens and the first `sinks`, decode rows and chunks

Pages hold 128 tokens; 8-bit pages are laid out [group][token][width], bf16 pages [token][group][width]."""
import math

import torch

own = False

PAGE = 128
TOP = 448.0          # the largest e4m3 value
LOWEST = -100        # exponent of the smallest scale


# ------------------------------------------------------------------------------------------------ cases

def _append(name, B, ctx, rows, q8, Hq=64, G=8, D=128, Di=64, rot=64, rot_idx=64, interleaved=False, scaling="none",
            pad=0):
    return {"name": name, "op": "append", "B": B, "ctx": ctx, "rows": rows, "q8": q8, "Hq": Hq, "G": G, "D": D,
            "Di": Di, "rot": rot, "rot_idx": rot_idx, "interleaved": interleaved, "scaling": scaling, "pad": pad}


def _read(name, B, ctx, G=8, D=128, Di=64, ragged=False):
    return {"name": name, "op": "read", "B": B, "ctx": ctx, "G": G, "D": D, "Di": Di, "ragged": ragged}


def _score(name, B, ctx, G=8, Di=64, ragged=False):
    return {"name": name, "op": "score", "B": B, "ctx": ctx, "G": G, "Di": Di, "ragged": ragged}


def _attend(name, B, ctx, Hq=64, G=8, D=128, topk=16, ragged=False):
    return {"name": name, "op": "attend", "B": B, "ctx": ctx, "Hq": Hq, "G": G, "D": D, "topk": topk, "ragged": ragged}


def _window(name, B, ctx, rows, window, sinks, Hq=64, G=8, D=128, prefill=False, pad=0, ragged=False):
    return {"name": name, "op": "window", "B": B, "ctx": ctx, "rows": rows, "window": window, "sinks": sinks, "Hq": Hq,
            "G": G, "D": D, "prefill": prefill, "pad": pad, "ragged": ragged}


def listed():
    return [
        # a decode batch: one new token for each of eight requests of 60,000 tokens, half of the head rotated
        _append("append_decode", 8, 60000, 1, True),
        # a prefill chunk into bf16 caches, whole heads in interleaved pairs, positions scaled for long contexts
        _append("append_chunk_bf16", 1, 60000, 8192, False, rot=128, interleaved=True, scaling="yarn"),
        # the same chunk into 8-bit caches, half of the head rotated
        _append("append_chunk", 1, 60000, 8192, True, scaling="yarn"),
        # the last turn of a short conversation, before a small prefill chunk
        _read("read_chat", 3, 1501, G=4, D=64, Di=32, ragged=True),
        # the prefix and chunk of a long prefill
        _read("read_prefix", 1, 68192),
        # one short conversation: the latency of the scan
        _score("score_chat", 1, 1500),
        # the agentic shape: eight requests of 60,000 tokens
        _score("score_agentic", 8, 60000),
        # unequal lengths, four heads per group, half the head width, odd sizes
        _attend("attend_ragged", 6, 20011, Hq=16, G=4, D=64, topk=11, ragged=True),
        # the agentic shape
        _attend("attend_agentic", 8, 60000),
        # one token of a short conversation in a window layer
        _window("window_chat", 1, 1500, 1, 1024, 4),
        # a decode batch in a window layer
        _window("window_decode", 32, 30000, 1, 4096, 4, ragged=True),
        # the long prefill's chunk in a window layer
        _window("window_chunk", 1, 60000, 8192, 4096, 4, prefill=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "append", "read", "score", "attend", "window", "window"])
    G, D, Di = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([32, 64])
    Hq = G * rng.choice([4, 8])
    ctx = _log_int(rng, 1, 60000)
    ragged = rng.random() < 0.5
    if op == "append":
        B = _log_int(rng, 1, 32)
        rows = 1 if rng.random() < 0.4 else _log_int(rng, 1, 8192 // B)
        c = _append("", B, ctx, rows, rng.random() < 0.7, Hq, G, D, Di, 16 * rng.randint(0, D // 16),
                    16 * rng.randint(0, Di // 16), rng.random() < 0.5,
                    rng.choice(["none", "linear", "ntk", "yarn"]), rng.randint(0, 5))
    elif op == "read":
        c = _read("", _log_int(rng, 1, max(1, min(16, 68192 // ctx))), ctx, G, D, Di, ragged)
    elif op == "score":
        c = _score("", _log_int(rng, 1, max(1, min(64, 480000 // ctx))), ctx, G, Di, ragged)
    elif op == "attend":
        c = _attend("", _log_int(rng, 1, max(1, min(64, 480000 // ctx))), ctx, Hq, G, D, rng.randint(1, 16), ragged)
    else:
        prefill = rng.random() < 0.5
        window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 130])
        if prefill:
            B = rng.randint(1, 3)
            rows = _log_int(rng, 1, 4096 // B)
        else:
            B, rows = _log_int(rng, 1, max(1, min(32, 960000 // ctx))), rng.randint(1, 2)
        c = _window("", B, ctx, rows, window, sinks, Hq, G, D, prefill, rng.randint(0, 5), ragged)
    del c["name"]
    return c


def _lens(case):
    """Tokens of each request before the call's own rows (append, window) or in all (the others)."""
    B, ctx = case["B"], case["ctx"]
    if not case.get("ragged"):
        return [ctx] * B
    return [max(1, ctx * (b + 1) // B - 37 * b) for b in range(B)]


# ------------------------------------------------------------------------------------------------ inputs

def _freqs(rot, scaling, base=10000.0, factor=16.0, original=4096):
    """Radians per position of each pair, and what cosines and sines are multiplied by (64 bits, host)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":       # a larger base: the lowest frequency is stretched by the factor, the highest kept
        base = base * factor ** (rot / max(rot - 2, 1))
    f = base ** (-2.0 * i / max(rot, 1))
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":      # pairs with many turns over the original length are kept, with few are stretched
        turn = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _tables(ends, gc, starts=None, spare=3):
    """Block table of pages in random order for the tokens [start, end) of each request, and the size of the pool;
    the pool's last page belongs to no block."""
    first = [0] * len(ends) if starts is None else [s // PAGE for s in starts]
    last = [(e + PAGE - 1) // PAGE for e in ends]
    pool = sum(b - a for a, b in zip(first, last)) + spare
    perm = torch.randperm(pool - 1, generator=gc).to(torch.int32)
    bt = torch.full((len(ends), max(last)), -1, dtype=torch.int32)
    at = 0
    for b, (x, y) in enumerate(zip(first, last)):
        bt[b, x:y] = perm[at:at + y - x]
        at += y - x
    return bt, pool


def _channels(shape, gd):
    """bf16 rows as projections give them: normal, with channels of different size."""
    x = torch.randn(shape, generator=gd, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(shape[-1], generator=gd, device="cuda"))).to(torch.bfloat16)


def _codes(pages, G, width, gd):
    """Pages of e4m3 codes and scales as quantised normal rows of unlike size have them."""
    code = torch.empty((pages, G, PAGE, width), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, G, PAGE), dtype=torch.uint8, device="cuda")
    for i in range(0, pages, 256):
        n = min(256, pages - i)
        x = torch.randn((n, G, PAGE, width), generator=gd, device="cuda")
        x *= torch.exp(0.4 * torch.randn((n, G, PAGE, 1), generator=gd, device="cuda"))
        c, e = _quantised(x)
        code[i:i + n], scale[i:i + n] = c, (e + 127).to(torch.uint8)
    return code, scale.view(torch.float8_e8m0fnu)


def _exponent(amax):
    """The power of two of a row's scale: the smallest with amax / 2^e <= 448 (0 for a row of zeros)."""
    m, e = torch.frexp(amax)                                   # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=LOWEST)
    return torch.where(amax > 0, e, 0)


def _quantised(x):
    """Codes of rows (the last axis) and the exponents of their scales."""
    e = _exponent(x.abs().amax(-1))
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), e


def prepare(case, seed):
    gc = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    op, G = case["op"], case["G"]
    lens = _lens(case)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": dict(case), "err": torch.zeros(1, **i32)}
    if op in ("append", "window"):
        n, pad = case["rows"], case["pad"]
        s["q_req"] = torch.tensor([b for b in range(case["B"]) for _ in range(n)] + [-1] * pad, **i32)
        s["q_pos"] = torch.tensor([x + i for x in lens for i in range(n)] + [0] * pad, **i32)
        bt, pool = _tables([x + n for x in lens], gc, lens if op == "append" else None)
        R = s["q_req"].numel()
    else:
        bt, pool = _tables(lens, gc)
        s["lens"] = torch.tensor(lens, **i32)
    s["bt"], s["pool"] = bt.cuda(), pool
    if op == "append":
        Hq, D, Di = case["Hq"], case["D"], case["Di"]
        widths = [Hq * D, G * D, G * D, G * Di, G * Di]         # one projection holds all five, row by row
        x = torch.cat([_channels((R, w), gd) for w in widths], 1)
        for name, part, h in zip(("q", "k", "v", "q_idx", "k_idx"), x.split(widths, 1), (Hq, G, G, G, G)):
            s[name] = part.unflatten(1, (h, -1))
        s["q_out"] = torch.zeros((R, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["q_idx_out"] = torch.zeros((R, G, Di), dtype=torch.bfloat16, device="cuda")
        (f, a), (g, _) = _freqs(case["rot"], case["scaling"]), _freqs(case["rot_idx"], case["scaling"])
        s["freq"], s["freq_idx"], s["gain"] = f.cuda(), g.cuda(), a
        if case["q8"]:
            for name, w in (("k", D), ("v", D), ("kidx", Di)):
                s[name + "8"], s[name + "_scale"] = _codes(pool, G, w, gd)
        else:
            for name, w in (("k", D), ("v", D), ("kidx", Di)):
                s[name + "_cache"] = _channels((pool, PAGE, G, w), gd)
    elif op == "read":
        D, Di = case["D"], case["Di"]
        for name, w in (("k", D), ("v", D), ("kidx", Di)):
            s[name + "8"], s[name + "_scale"] = _codes(pool, G, w, gd)
            s[name + "_out"] = torch.zeros((pool, PAGE, G, w), dtype=torch.bfloat16, device="cuda")
        s["bt_out"] = torch.where(bt >= 0, (bt + 1) % (pool - 1), -1).to(torch.int32).cuda()
    elif op == "score":
        s["kidx8"], s["kidx_scale"] = _codes(pool, G, case["Di"], gd)
        s["q_idx"] = _channels((case["B"], G, case["Di"]), gd)
        s["q_req"], s["q_pos"] = torch.arange(case["B"], **i32), s["lens"] - 1
    elif op == "attend":
        s["k8"], s["k_scale"] = _codes(pool, G, case["D"], gd)
        s["v8"], s["v_scale"] = _codes(pool, G, case["D"], gd)
        s["q"] = _channels((case["B"], case["Hq"], case["D"]), gd)
        table, row_len = [], []
        for b, n in enumerate(lens):                            # the own block, last, and topk - 1 others
            blocks = (n + PAGE - 1) // PAGE
            k = min(case["topk"], blocks)
            pick = torch.rand((G, max(blocks - 1, 1)), generator=gc).argsort(1)[:, :k - 1].sort(1).values
            row = torch.full((G, case["topk"]), -1, dtype=torch.long)
            row[:, :k - 1], row[:, k - 1] = pick, blocks - 1
            table.append(torch.where(row >= 0, bt[b].long()[row.clamp(min=0)], -1))
            row_len += [(k - 1) * PAGE + n - (blocks - 1) * PAGE] * G
        s["pt"] = torch.cat(table).to(torch.int32).cuda()
        s["row_len"] = torch.tensor(row_len, **i32)
    else:
        s["k8"], s["k_scale"] = _codes(pool, G, case["D"], gd)
        s["v8"], s["v_scale"] = _codes(pool, G, case["D"], gd)
        s["q"] = _channels((R, case["Hq"], case["D"]), gd)
        s["out"] = torch.zeros((R, case["Hq"], case["D"]), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((R, case["Hq"]), dtype=torch.float32, device="cuda")
        s["ctx"] = torch.tensor(lens, **i32)
    return s


# ------------------------------------------------------------------------------------------------ the calls

def _own(s):
    import block_sparse_attention_06_gb300 as msa
    c, err = s["case"], s["err"]
    if "dims" not in s:      # the handles that a serving loop keeps: sizes, the caches, the rotation's frequencies
        G, D, Di = c["G"], c.get("D", 64), c.get("Di", 32)
        s["dims"] = msa.Dims(c.get("Hq", 8 * G), G, D, Di, c.get("topk", 1), s["bt"].shape[1])
        s["cache"] = msa.CacheQ8(*(s.get(n) for n in ("k8", "k_scale", "v8", "v_scale", "kidx8", "kidx_scale")))
        if c["op"] == "append":
            s["rope"] = msa.Rope(c["rot"], s["freq"], c["rot_idx"], s["freq_idx"], interleaved=c["interleaved"],
                                 gain=s["gain"])
    d = s["dims"]
    if c["op"] == "append":
        new = (s["q"], s["k"], s["v"], s["q_idx"], s["k_idx"])
        where = (s["bt"], s["q_req"], s["q_pos"], s["rope"], d, s["q_out"], s["q_idx_out"])
        if c["q8"]:
            q, q_idx = msa.msa_rope_append_q8(*new, s["cache"], *where, err_word=err)
        else:
            q, q_idx = msa.msa_rope_append(*new, s["k_cache"], s["v_cache"], s["kidx_cache"], *where, err_word=err)
        return _appended(s, q, q_idx)
    if c["op"] == "read":
        k, v, kidx = msa.msa_cache_read_q8(s["cache"], s["bt"], s["bt_out"], s["lens"], d, s["k_out"], s["v_out"],
                                           s["kidx_out"], err_word=err)
        return {"k": k, "v": v, "kidx": kidx}
    if c["op"] == "score":
        return {"scores": msa.msa_index_score_q8(s["q_idx"], s["cache"], s["bt"], s["q_req"], s["q_pos"], d,
                                                 err_word=err)}
    if c["op"] == "attend":
        out, lse = msa.msa_sparse_attn_decode_q8(s["q"], s["cache"], s["pt"], s["row_len"], d, err_word=err)
        return {"out": out, "lse": lse}
    phase = msa.MSA_PHASE_PREFILL if c["prefill"] else msa.MSA_PHASE_DECODE
    out, lse = msa.msa_window_attn_q8(s["q"], s["cache"], s["bt"], s["q_req"], s["q_pos"], c["window"], c["sinks"], d,
                                      phase, s["out"], s["lse"], err_word=err)
    return {"out": out, "lse": lse}


def _appended(s, q, q_idx):
    names = [n for n in ("k8", "k_scale", "v8", "v_scale", "kidx8", "kidx_scale", "k_cache", "v_cache", "kidx_cache")
             if n in s]
    return {"q": q, "q_idx": q_idx, **{n: s[n] for n in names}}


# ------------------------------------------------------------------------------------------------ plain forms

def _rotated(x, rot, cos, sin, interleaved):
    """x [R, heads, width] in 32 bits with its first `rot` components rotated in pairs; cos, sin [R, rot / 2]."""
    if rot == 0:
        return x
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    live, pos = s["q_req"] >= 0, s["q_pos"].long()
    wave = [pos.double()[:, None] * f for f in (s["freq"], s["freq_idx"])]       # in 64 bits: far positions
    (cos, sin), (cos_i, sin_i) = [((torch.cos(w) * s["gain"]).float(), (torch.sin(w) * s["gain"]).float()) for w in wave]
    q, k = (_rotated(s[n].float(), c["rot"], cos, sin, c["interleaved"]) for n in ("q", "k"))
    qi, ki = (_rotated(s[n].float(), c["rot_idx"], cos_i, sin_i, c["interleaved"]) for n in ("q_idx", "k_idx"))
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(torch.bfloat16), s["q_out"]))
    s["q_idx_out"].copy_(torch.where(live[:, None, None], qi.to(torch.bfloat16), s["q_idx_out"]))
    # rows of no request rewrite what the page of no block holds
    page = torch.where(live, s["bt"].long()[s["q_req"].long().clamp(min=0), pos // PAGE], s["pool"] - 1)
    slot = torch.where(live, pos % PAGE, 0)
    keep = live[:, None, None]
    for name, x in (("k", k), ("v", s["v"].float()), ("kidx", ki)):
        if c["q8"]:
            code, e = _quantised(x)
            codes, scales = s[name + "8"].view(torch.uint8), s[name + "_scale"].view(torch.uint8)
            new, scale = code.view(torch.uint8), (e + 127).to(torch.uint8)
            codes[page, :, slot] = torch.where(keep, new, codes[page, :, slot])
            scales[page, :, slot] = torch.where(keep[..., 0], scale, scales[page, :, slot])
        else:
            cache = s[name + "_cache"]
            cache[page, slot] = torch.where(keep, x.to(torch.bfloat16), cache[page, slot])
    return _appended(s, s["q_out"], s["q_idx_out"])


def _plain_read(s):
    bt, to = s["bt"].long().flatten(), s["bt_out"].long().flatten()
    B, MB = s["bt"].shape
    token = torch.arange(MB * PAGE, device="cuda").reshape(1, MB, PAGE)
    live = ((token < s["lens"].long()[:, None, None]) & (s["bt_out"] >= 0)[..., None]).reshape(B * MB, PAGE, 1, 1)
    to = torch.where((to >= 0) & (bt >= 0), to, s["pool"] - 1)     # the page of no block is rewritten as it is
    out = {}
    for name in ("k", "v", "kidx"):
        at = bt.clamp(min=0)
        x = s[name + "8"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        x *= s[name + "_scale"].view(torch.uint8)[at].view(torch.float8_e8m0fnu).float()[..., None]
        x = x.transpose(1, 2).to(torch.bfloat16)
        pages = s[name + "_out"]
        pages[to] = torch.where(live, x, pages[to])
        out[name] = pages
    return out


def _values(s, name, pages, groups=slice(None)):
    """Stored rows in 32 bits: pages [...] (and groups) of the pool -> [..., token, width]."""
    code = s[name + "8"].view(torch.uint8)[pages, groups].view(torch.float8_e4m3fn).float()
    return code * s[name + "_scale"].view(torch.uint8)[pages, groups].view(torch.float8_e8m0fnu).float()[..., None]


def _plain_score(s):
    B, MB = s["bt"].shape
    keys = _values(s, "kidx", s["bt"].long().clamp(min=0))                             # [B, MB, G, PAGE, Di]
    dots = torch.einsum("bgd,bjgtd->bgjt", s["q_idx"].float(), keys)
    token = torch.arange(MB * PAGE, device="cuda").reshape(1, 1, MB, PAGE)
    seen = token <= s["q_pos"][:, None, None, None]
    return {"scores": torch.where(seen, dots, -torch.inf).amax(-1)}


def _softmax(logits):
    """Weights that are not normalised yet, their sum and the log-sum; rows that see nothing get 0 and -inf."""
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total > 0, total, 1.0), (top + torch.log(total))[..., 0]


def _plain_attend(s):
    c = s["case"]
    B, G, D, K = c["B"], c["G"], c["D"], c["topk"]
    pages = s["pt"].long().reshape(B, G, K).clamp(min=0)
    group = torch.arange(G, device="cuda")[None, :, None]
    k = _values(s, "k", pages, group).reshape(B, G, K * PAGE, D)
    v = _values(s, "v", pages, group).reshape(B, G, K * PAGE, D)
    q = s["q"].float().reshape(B, G, -1, D)
    logits = torch.einsum("bghd,bgtd->bght", q, k) * (1.0 / D ** 0.5)
    seen = torch.arange(K * PAGE, device="cuda") < s["row_len"].reshape(B, G, 1, 1)
    e, total, lse = _softmax(torch.where(seen, logits, -torch.inf))
    out = torch.einsum("bght,bgtd->bghd", e, v) / total
    return {"out": out.reshape(B, c["Hq"], D).to(torch.bfloat16), "lse": lse.reshape(B, c["Hq"])}


def _plain_window(s):
    """Decode rows gather the tokens they see; a chunk takes all tokens that any of its rows sees, and masks."""
    c = s["case"]
    G, D, W, S = c["G"], c["D"], c["window"], c["sinks"]
    pos, req = s["q_pos"].long(), s["q_req"].long()
    R = pos.numel()
    q = s["q"].float().reshape(R, G, -1, D) * (1.0 / D ** 0.5)
    if c["prefill"]:
        n = c["B"] * (S + W - 1 + c["rows"])
        one = n // c["B"]                                       # tokens taken of each request
        tr = torch.arange(n, device="cuda") // one
        i = torch.arange(n, device="cuda") % one
        first = (s["ctx"].long() - (W - 1))[tr]                 # of the window of the first row
        token = torch.where(i < S, i, first + i - S)
        fresh = (i < S) | (token >= S)                          # no token twice
        at = s["bt"].long()[tr, (token // PAGE).clamp(0, s["bt"].shape[1] - 1)].clamp(min=0)
        k, v = (_row(s, name, at, token % PAGE) for name in ("k", "v"))               # [n, G, D]
        seen = (tr == req[:, None]) & fresh & (token >= 0) & (token <= pos[:, None])
        seen &= (token > pos[:, None] - W) | (token < S)
        logits = torch.einsum("rghd,tgd->rght", q, k)
        e, total, lse = _softmax(torch.where(seen[:, None, None], logits, -torch.inf))
        out = torch.einsum("rght,tgd->rghd", e, v) / total
    else:
        i = torch.arange(S + min(W, s["bt"].shape[1] * PAGE), device="cuda")
        token = torch.where(i < S, i, pos[:, None] - (i - S))
        fresh = (i < S) | (token >= S)
        seen = fresh & (token >= 0) & (token <= pos[:, None])
        at = s["bt"].long()[req.clamp(min=0)[:, None], (token // PAGE).clamp(0, s["bt"].shape[1] - 1)].clamp(min=0)
        k, v = (_row(s, name, at, token % PAGE) for name in ("k", "v"))               # [R, n, G, D]
        logits = torch.einsum("rghd,rtgd->rght", q, k)
        e, total, lse = _softmax(torch.where(seen[:, None, None], logits, -torch.inf))
        out = torch.einsum("rght,rtgd->rghd", e, v) / total
    live = req >= 0
    s["out"].copy_(torch.where(live[:, None, None], out.reshape(R, c["Hq"], D).to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(live[:, None], lse.reshape(R, c["Hq"]), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _row(s, name, page, slot):
    """Stored rows of single tokens in 32 bits: [..., G, width]."""
    code = s[name + "8"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return code * s[name + "_scale"].view(torch.uint8)[page, :, slot].view(torch.float8_e8m0fnu).float()[..., None]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "score": _plain_score, "attend": _plain_attend,
            "window": _plain_window}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass costs

def work(case):
    op, G, lens = case["op"], case["G"], _lens(case)
    if op == "append":
        Hq, D, Di, n = case["Hq"], case["D"], case["Di"], case["B"] * case["rows"]
        read = (Hq + 2 * G) * D * 2 + 2 * G * Di * 2
        stored = G * (2 * D + Di + 3) if case["q8"] else G * (2 * D + Di) * 2
        return {"bytes": n * (read + Hq * D * 2 + G * Di * 2 + stored + 8),
                "flops": n * 3 * ((Hq + G) * case["rot"] + 2 * G * case["rot_idx"])}
    if op == "read":
        D, Di = case["D"], case["Di"]
        return {"bytes": sum(lens) * G * ((2 * D + Di) * 3 + 3), "flops": 0}
    if op == "score":
        blocks = max((n + PAGE - 1) // PAGE for n in lens)
        Di = case["Di"]
        return {"bytes": sum(lens) * G * (Di + 1) + case["B"] * G * (Di * 2 + blocks * 4),
                "flops": 2 * sum(lens) * G * Di}
    Hq, D = case["Hq"], case["D"]
    if op == "attend":
        seen = sum(min(n, (min(case["topk"], (n + PAGE - 1) // PAGE) - 1) * PAGE + (n - 1) % PAGE + 1) for n in lens)
        return {"bytes": seen * G * 2 * (D + 1) + case["B"] * (Hq * (D * 4 + 4) + G * (case["topk"] + 1) * 4),
                "flops": 4 * seen * Hq * D}
    W, S, n = case["window"], case["sinks"], case["rows"]
    pairs = touched = 0
    for x in lens:
        full = [min(x + i + 1, W) + min(S, max(0, x + i + 1 - W)) for i in (0, n - 1)]
        pairs += n * (full[0] + full[1]) // 2
        touched += min(x + n, W + n - 1 + min(S, max(0, x + 1 - W)))
    return {"bytes": touched * G * 2 * (D + 1) + case["B"] * n * Hq * (D * 4 + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "score": _exact_score, "attend": _exact_attend,
            "window": _exact_window}[case["op"]](s)


def _stored(s, name):
    """All pages in 64 bits: [pages][G][token][width]."""
    return s[name + "8"].double() * s[name + "_scale"].double()[..., None]


def _exact_append(s):
    c = s["case"]
    req, pos = s["q_req"].tolist(), s["q_pos"].tolist()
    live = [r for r in range(len(req)) if req[r] >= 0]
    page = torch.tensor([int(s["bt"][req[r], pos[r] // PAGE]) for r in live[:1]] if not live else
                        s["bt"].cpu()[[req[r] for r in live], [pos[r] // PAGE for r in live]].tolist())
    slot = torch.tensor([pos[r] % PAGE for r in live])

    def turned(x, rot, freq):
        """Pairs as complex numbers, turned by their angle."""
        x = x.double().clone()
        if rot:
            half = rot // 2
            first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
            second = first + (1 if c["interleaved"] else half)
            angle = s["q_pos"].double()[:, None, None] * freq[None, None]
            z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(angle, s["gain"]), angle)
            x[..., first], x[..., second] = z.real, z.imag
        return x

    out = {}
    for name, rot, f in (("q", c["rot"], s["freq"]), ("q_idx", c["rot_idx"], s["freq_idx"])):
        out[name] = s[name + "_out"].double()
        out[name][live] = turned(s[name], rot, f)[live]
    for name, x in (("k", turned(s["k"], c["rot"], s["freq"])), ("v", s["v"].double()),
                    ("kidx", turned(s["k_idx"], c["rot_idx"], s["freq_idx"]))):
        x = x[live]
        if not c["q8"]:
            out[name + "_cache"] = s[name + "_cache"].double()
            out[name + "_cache"][page, slot] = x
            continue
        top = x.abs().amax(-1)
        scale = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(min=LOWEST))
        scale = torch.where(scale * TOP < top, scale * 2, scale)
        scale = torch.where((scale / 2 * TOP >= top) & (scale > 2.0 ** LOWEST), scale / 2, scale)
        scale = torch.where(top > 0, scale, 1.0)
        y = x / scale[..., None]
        # e4m3: three bits behind the leading one, the lowest step 2^-9, ties to even
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        out[name + "8"] = s[name + "8"].double()
        out[name + "8"][page, :, slot] = torch.round(y / step) * step
        out[name + "_scale"] = s[name + "_scale"].double()
        out[name + "_scale"][page, :, slot] = scale
    return out


def _exact_read(s):
    out = {n: s[n + "_out"].double() for n in ("k", "v", "kidx")}
    for name in out:
        x = _stored(s, name)
        for b, n in enumerate(s["lens"].tolist()):
            for j in range((n + PAGE - 1) // PAGE):
                m = min(PAGE, n - j * PAGE)
                out[name][int(s["bt_out"][b, j]), :m] = x[int(s["bt"][b, j])].transpose(0, 1)[:m]
    return out


def _exact_score(s):
    lens, MB = s["lens"].tolist(), s["bt"].shape[1]
    scores = torch.full((len(lens), s["case"]["G"], MB), -torch.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        blocks = (n + PAGE - 1) // PAGE
        at = s["bt"][b, :blocks].long()
        x = s["kidx8"][at].double() * s["kidx_scale"][at].double()[..., None]
        dots = (x * s["q_idx"][b].double()[None, :, None]).sum(-1)                     # [blocks, G, PAGE]
        if n % PAGE:
            dots[-1, :, n % PAGE:] = -torch.inf
        scores[b, :, :blocks] = dots.amax(-1).T
    return {"scores": scores}


def _one_row(q, k, v, D):
    """Attention of the heads q [h, D] over tokens k, v [t, D]; nothing seen gives 0 and -inf."""
    if not k.shape[0]:
        return torch.zeros_like(q), torch.full((q.shape[0],), -torch.inf, dtype=torch.float64, device=q.device)
    a = q @ k.T / D ** 0.5
    return torch.softmax(a, -1) @ v, torch.logsumexp(a, -1)


def _exact_attend(s):
    c = s["case"]
    G, D, hpg = c["G"], c["D"], c["Hq"] // c["G"]
    out = torch.zeros((c["B"], c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], c["Hq"]), dtype=torch.float64, device="cuda")
    pt, lens = s["pt"].tolist(), s["row_len"].tolist()
    for r in range(len(pt)):
        b, g = r // G, r % G
        at = [p for p in pt[r] if p >= 0]
        k, v = ((s[n + "8"][at, g].double() * s[n + "_scale"][at, g].double()[..., None]).flatten(0, 1)[:lens[r]]
                for n in ("k", "v"))
        h = slice(g * hpg, (g + 1) * hpg)
        out[b, h], lse[b, h] = _one_row(s["q"][b, h].double(), k, v, D)
    return {"out": out, "lse": lse}


def _exact_window(s):
    c = s["case"]
    G, D, W, S, hpg, n = c["G"], c["D"], c["window"], c["sinks"], c["Hq"] // c["G"], c["rows"]
    out, lse = s["out"].double(), s["lse"].double()
    step = max(1, (1 << 26) // ((W + S + n) * hpg))              # rows at once
    for b, x in enumerate(s["ctx"].tolist()):
        bt = s["bt"][b].long()
        first = max(0, x - W + 1)
        where = torch.tensor(sorted(set(range(min(S, x + n))) | set(range(first, x + n))), device="cuda")
        at, slot = bt[where // PAGE], where % PAGE
        for g in range(G):
            k, v = (s[m + "8"][at, g, slot].double() * s[m + "_scale"][at, g, slot].double()[:, None] for m in ("k", "v"))
            for i in range(0, n, step):
                m = min(step, n - i)
                p = x + i + torch.arange(m, device="cuda")
                see = (where <= p[:, None]) & ((where > p[:, None] - W) | (where < S))
                rows, h = slice(b * n + i, b * n + i + m), slice(g * hpg, (g + 1) * hpg)
                a = s["q"][rows, h].double() @ k.T / D ** 0.5
                a = a.masked_fill(~see[:, None], -torch.inf)
                lse[rows, h] = torch.logsumexp(a, -1)
                out[rows, h] = torch.softmax(a, -1) @ v
    return {"out": out, "lse": lse}
