"""Drafted-tree decoding: the operators of one speculative decode step, as measured cases.

A step drafts a small tree of tokens after each request's cached context, runs the target model over the whole
tree at once, keeps the longest path that the target accepts, and appends that path to the caches.  Four
operators of that step are measured here, each by a plain form in elementary torch operations and by the
framework's own calls (`own`):

  score    msa_tree_rows + msa_tree_index_score: the tree's layout and the block scores of every node
  attend   msa_sparse_attn_tree: sparse attention of every node over its selected blocks and its ancestors
  verify   msa_verify_tree: the accepted path and the next token, from given uniform random numbers
  commit   msa_commit_tree: the accepted path's K, V and k-index written into the paged caches of all layers

A request's nodes are numbered so that a parent precedes its children; node 0, the root, is the last token that
was sampled.  Node i of a request with `ctx` cached tokens stands at position ctx + depth(i)."""
import torch

own = False

PAGE = 128
MAX_NODES = 64


# ------------------------------------------------------------------------------------------------ cases

def _score(name, B, ctx, nodes, G=8, Di=64, chain=False, ragged=False):
    return {"name": name, "op": "score", "B": B, "ctx": ctx, "nodes": nodes, "G": G, "Di": Di, "chain": chain,
            "ragged": ragged}


def _attend(name, B, ctx, nodes, Hq=64, G=8, D=128, topk=16, spread=4, chain=False, ragged=False):
    return {"name": name, "op": "attend", "B": B, "ctx": ctx, "nodes": nodes, "Hq": Hq, "G": G, "D": D, "topk": topk,
            "spread": spread, "chain": chain, "ragged": ragged}


def _verify(name, B, vocab, nodes, drafts, chain=False, ragged=False):
    return {"name": name, "op": "verify", "B": B, "vocab": vocab, "nodes": nodes, "drafts": drafts, "chain": chain,
            "ragged": ragged}


def _commit(name, B, layers, nodes, G=8, D=128, Di=64, chain=False, ragged=False):
    return {"name": name, "op": "commit", "B": B, "layers": layers, "nodes": nodes, "G": G, "D": D, "Di": Di,
            "chain": chain, "ragged": ragged}


def listed():
    return [
        # one short conversation with a chain of drafts: the latency of the whole scan
        _score("score_chat", 1, 1500, 5, chain=True),
        # requests of unequal lengths and trees, four groups, the narrow index
        _score("score_ragged", 6, 30011, 23, G=4, Di=32, ragged=True),
        # the agentic shape: eight requests of 60,000 tokens, a tree of 16 each
        _score("score_agentic", 8, 60000, 16),
        # the same contexts with the widest trees
        _score("score_wide", 8, 60000, 64),
        # a short conversation: latency of the attention, boundary block and drafts only a few pages long
        _attend("attend_chat", 1, 1500, 5, chain=True),
        # half the head width, four heads per group, unequal lengths, odd sizes
        _attend("attend_ragged", 6, 20011, 23, Hq=16, G=4, D=64, topk=11, ragged=True),
        # the agentic shape
        _attend("attend_agentic", 8, 60000, 16),
        # the widest trees, whose nodes agree on fewer blocks
        _attend("attend_wide", 8, 60000, 64, spread=12),
        # one request, drafts taken from a lookup (no draft distribution), a small vocabulary
        _verify("verify_chain", 1, 32000, 5, False, chain=True),
        # a batch with sampled trees over a large vocabulary
        _verify("verify_batch", 32, 131072, 16, True),
        # one layer's commit for one request
        _commit("commit_one", 1, 1, 8, chain=True),
        # all layers of a deep model for a batch
        _commit("commit_batch", 32, 32, 16, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["score", "attend", "attend", "verify", "commit"])
    shape = {"chain": rng.random() < 0.3, "ragged": rng.random() < 0.5}
    if op in ("score", "attend"):
        ctx = _log_int(rng, 1, 60000)
        B = _log_int(rng, 1, max(1, min(64, 480000 // ctx)))
        nodes = _log_int(rng, 1, max(1, min(64, 512 // B)))
        if op == "score":
            c = _score("", B, ctx, nodes, G=rng.choice([1, 2, 4, 8]), Di=rng.choice([32, 64]), **shape)
        else:
            G = rng.choice([1, 2, 4, 8])
            c = _attend("", B, ctx, nodes, Hq=G * rng.choice([4, 8]), G=G, D=rng.choice([64, 128]),
                        topk=rng.randint(1, 16), spread=rng.randint(1, 12), **shape)
    elif op == "verify":
        vocab = _log_int(rng, 1000, 131072)
        B = _log_int(rng, 1, 32)
        c = _verify("", B, vocab, _log_int(rng, 1, min(64, 512 // B)), rng.random() < 0.6, **shape)
    else:
        B = _log_int(rng, 1, 32)
        c = _commit("", B, _log_int(rng, 1, 32), _log_int(rng, 1, min(64, 512 // B)), G=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 128]), Di=rng.choice([32, 64]), **shape)
    del c["name"]
    return c


def _per_request(case):
    """(cached tokens, nodes) of each request."""
    B, n = case["B"], case["nodes"]
    if not case["ragged"]:
        return [case.get("ctx", 0)] * B, [n] * B
    ctx = [max(1, case.get("ctx", 0) * (b + 1) // B - 37 * b) for b in range(B)]
    return ctx, [max(1, n - 5 * b % n) for b in range(B)]


def _accepted(case):
    """Accepted nodes of each request (commit): between one and its path's length, eight at most."""
    return [min(n, 1 + (3 * b + 4) % 8) for b, n in enumerate(_per_request(case)[1])]


# ------------------------------------------------------------------------------------------------ inputs

def _tree(case, gc):
    """node_off, parents (numbers within the request) of random trees: a node hangs under one of the four before it."""
    counts = _per_request(case)[1]
    parents = []
    for n in counts:
        i = torch.arange(n)
        back = torch.ones(n, dtype=torch.long) if case["chain"] else torch.randint(1, 5, (n,), generator=gc)
        p = torch.clamp(i - back, min=0)
        p[0] = -1
        parents.append(p)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    return off, torch.cat(parents).to(torch.int32)


def _depths(off, parents):
    """Depth of every node and the rows of its path (host)."""
    off, parents = off.tolist(), parents.tolist()
    depth, anc = [0] * len(parents), [0] * len(parents)
    for b in range(len(off) - 1):
        for i in range(off[b + 1] - off[b]):
            r, p = off[b] + i, parents[off[b] + i]
            depth[r] = depth[off[b] + p] + 1 if p >= 0 else 0
            anc[r] = (anc[off[b] + p] if p >= 0 else 0) | (1 << i)
    return depth, anc


def _tables(ctx, extra, gc, spare=3):
    """Block table of pages in random order for ctx + extra tokens a request, and the size of the pool."""
    blocks = [(c + e + PAGE - 1) // PAGE for c, e in zip(ctx, extra)]
    pool = sum(blocks) + spare
    perm = torch.randperm(pool, generator=gc).to(torch.int32)
    bt = torch.full((len(ctx), max(blocks)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, pool


def _normal(shape, gd):
    return torch.randn(shape, generator=gd, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _pool(pages, width, gd):
    out = torch.empty((pages, PAGE, *width), dtype=torch.bfloat16, device="cuda")
    for i in range(0, pages, 256):
        out[i:i + 256] = _normal((min(256, pages - i), PAGE, *width), gd)
    return out


def _union(case, ctx, n):
    """(shared blocks, blocks a node adds, pool they come from) of a request: the nodes of a tree agree on half of
    their blocks, and take the rest from a pool `spread` times what one node adds."""
    full, k = ctx // PAGE, case["topk"] - 1
    core = min(full, k // 2)
    add = min(full - core, k - core)
    return core, add, min(full - core, add * case["spread"])


def _selection(case, ctx, off, depth, gc):
    """sel int32 [rows][G][topk]: ascending block ids with the node's own block, -1 behind."""
    G, topk = case["G"], case["topk"]
    counts = _per_request(case)[1]
    big = 1 << 30
    sel = []
    for b, n in enumerate(counts):
        core, add, pool = _union(case, ctx[b], n)
        full = ctx[b] // PAGE
        ids = torch.rand((G, max(full, 1)), generator=gc).argsort(1)
        i = torch.arange(n)
        s = torch.full((n, G, topk), big, dtype=torch.long)
        s[:, :, :core] = ids[None, :, :core]
        if add:
            take = core + (i[:, None] * add + torch.arange(add)) % pool
            s[:, :, core:core + add] = ids[:, take].permute(1, 0, 2)
        own_block = (ctx[b] + torch.tensor(depth[int(off[b]):int(off[b + 1])])) // PAGE
        # the block that the cached context ends in, where a node already stands past it
        past = (own_block > full) & (i % 2 == 1) & (topk > core + add + 1)
        if topk > core + add + 1:
            s[past, :, core + add + 1] = full
        s[:, :, core + add if core + add < topk else topk - 1] = own_block[:, None]
        s = s.sort(-1).values
        sel.append(torch.where(s == big, -1, s))
    return torch.cat(sel).to(torch.int32)


def prepare(case, seed):
    gc = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    ctx, counts = _per_request(case)
    off, parents = _tree(case, gc)
    depth, anc = _depths(off, parents)
    rows = len(depth)
    s = {"case": dict(case), "off": off.cuda(), "parents": parents.cuda(),
         "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    op = case["op"]
    if op in ("score", "attend", "commit"):
        if op == "commit":   # contexts that end anywhere in a page; only the pages around their end are held
            ctx = [1 + (29 * b + 100) % PAGE for b in range(case["B"])]
        bt, pool = _tables(ctx, counts, gc)
        s["bt"], s["ctx"] = bt.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    if op == "score":
        G, Di = case["G"], case["Di"]
        s["q_idx"], s["kidx_new"] = _normal((rows, G, Di), gd), _normal((rows, G, Di), gd)
        s["kidx"] = _pool(pool, (G, Di), gd)
    elif op == "attend":
        G, D = case["G"], case["D"]
        s["q"] = _normal((rows, case["Hq"], D), gd)
        s["k_new"], s["v_new"] = _normal((rows, G, D), gd), _normal((rows, G, D), gd)
        s["k"], s["v"] = _pool(pool, (G, D), gd), _pool(pool, (G, D), gd)
        s["sel"] = _selection(case, ctx, off, depth, gc).cuda()
        s["anc"] = torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64, device="cuda")
    elif op == "verify":
        V = case["vocab"]
        logits = torch.randn((rows, V), generator=gd, device="cuda") * 2.5
        s["p"] = torch.softmax(logits, -1)
        q = torch.softmax(logits + torch.randn((rows, V), generator=gd, device="cuda") * 0.7, -1)
        above = torch.clamp(parents, min=0).cuda() + torch.repeat_interleave(s["off"][:-1], torch.tensor(counts).cuda())
        rank = _ranks(off, parents)
        s["children"] = min(max(rank) + 1, case["nodes"] - 1)   # of any node, at most
        if case["drafts"]:   # children drawn from the draft model's distribution at their parent
            s["q"] = q
            tokens = torch.multinomial(q[above.long()], 1, generator=gd)[:, 0]
        else:                # children looked up: the likeliest continuations in order
            s["q"] = None
            top = q.topk(max(rank) + 1, -1).indices
            tokens = top[above.long(), torch.tensor(rank, device="cuda")]
        s["tokens"] = tokens.to(torch.int32)
        s["u_accept"] = torch.rand(rows, generator=gd, device="cuda")
        s["u_next"] = torch.rand(case["B"], generator=gd, device="cuda")
    else:
        L, G, D, Di = case["layers"], case["G"], case["D"], case["Di"]
        for name, w in (("k", D), ("v", D), ("kidx", Di)):
            s[name] = torch.randn((L, pool, PAGE, G, w), generator=gd, device="cuda", dtype=torch.bfloat16)
            s[name + "_new"] = torch.randn((L, rows, G, w), generator=gd, device="cuda", dtype=torch.bfloat16)
        path, n_acc = torch.full((rows,), -1, dtype=torch.int32), []
        for b, want in enumerate(_accepted(case)):
            r0, r1 = int(off[b]), int(off[b + 1])
            best = max(range(r0, r1), key=lambda r: (min(depth[r] + 1, want), -r))
            nodes = [i for i in range(r1 - r0) if anc[best] >> i & 1][:want]
            path[r0:r0 + len(nodes)] = torch.tensor(nodes, dtype=torch.int32)
            n_acc.append(len(nodes))
        s["path"], s["n_acc"] = path.cuda(), torch.tensor(n_acc, dtype=torch.int32, device="cuda")
    return s


def _ranks(off, parents):
    """Each node's number among the children of its parent (host)."""
    off, parents = off.tolist(), parents.tolist()
    rank, seen = [], {}
    for b in range(len(off) - 1):
        for r in range(off[b], off[b + 1]):
            key = (b, parents[r])
            rank.append(seen.get(key, 0))
            seen[key] = rank[-1] + 1
    return rank


# ------------------------------------------------------------------------------------------------ the calls

def _own(s):
    import block_sparse_attention_06_gb300 as msa
    c = s["case"]
    if "dims" not in s:   # the handle and the workspace that a decode loop keeps
        G, D, Di = c.get("G", 1), c.get("D", 64), c.get("Di", 32)
        mb = s["bt"].shape[1] if "bt" in s else 1
        s["dims"] = msa.Dims(c.get("Hq", 8 * G), G, D, Di, c.get("topk", 1), mb)
        if c["op"] == "attend":
            need = msa.msa_workspace_bytes(msa.MSA_OP_TREE, s["q"].shape[0], c["B"], s["dims"])
            s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    d, err = s["dims"], s["err"]
    if c["op"] == "score":
        q_req, q_pos, anc = msa.msa_tree_rows(s["off"], s["parents"], s["ctx"], d, err_word=err)
        scores = msa.msa_tree_index_score(s["q_idx"], s["kidx"], s["kidx_new"], s["bt"], s["ctx"], s["off"], anc, d,
                                          err_word=err)
        return {"q_req": q_req, "q_pos": q_pos, "anc": anc, "scores": scores}
    if c["op"] == "attend":
        out, lse = msa.msa_sparse_attn_tree(s["q"], s["k"], s["v"], s["k_new"], s["v_new"], s["bt"], s["ctx"], s["off"],
                                            s["anc"], s["sel"], d, workspace=s["ws"], err_word=err)
        return {"out": out, "lse": lse}
    if c["op"] == "verify":
        path, n_acc, token = msa.msa_verify_tree(s["p"], s["q"], s["tokens"], s["off"], s["parents"], s["u_accept"],
                                                 s["u_next"], err_word=err)
        return {"path": path, "n_acc": n_acc, "token": token}
    lens = msa.msa_commit_tree(s["k_new"], s["v_new"], s["kidx_new"], s["k"], s["v"], s["kidx"], s["bt"], s["ctx"],
                               s["off"], s["path"], s["n_acc"], d, err_word=err)
    return {"k": s["k"], "v": s["v"], "kidx": s["kidx"], "lens": lens}


# ------------------------------------------------------------------------------------------------ plain forms

def _layout(s):
    """Per row: its request, its number there; per request: reach [B, N, N] (node i's path holds m) and depth [B, N]."""
    off, parents, N = s["off"].long(), s["parents"].long(), s["case"]["nodes"]
    B, R = off.numel() - 1, parents.numel()
    row = torch.arange(R, device="cuda")
    req = torch.searchsorted(off, row, right=True) - 1
    num = row - off[req]
    step = torch.zeros((B, N, N), dtype=torch.float64, device="cuda")
    step[req, num, torch.clamp(parents, min=0)] = (parents >= 0).double()
    eye = torch.eye(N, dtype=torch.float64, device="cuda")
    reach = torch.linalg.matrix_power(step + eye, max(N - 1, 1)) > 0
    live = torch.arange(N, device="cuda")[None] < (off[1:] - off[:-1])[:, None]
    reach = reach & live[:, :, None] & live[:, None, :]
    return req, num, reach, reach.sum(-1) - 1


def _padded(x, req, num, B, N):
    out = torch.zeros((B, N, *x.shape[1:]), dtype=torch.float32, device="cuda")
    out[req, num] = x.float()
    return out


def _plain_score(s):
    c = s["case"]
    B, N, MB = c["B"], c["nodes"], s["bt"].shape[1]
    req, num, reach, depth = _layout(s)
    ctx = s["ctx"].long()
    pos = ctx[:, None] + depth
    bits = torch.ones(N, dtype=torch.int64, device="cuda") << torch.arange(N, device="cuda")
    anc = (reach.long() * bits).sum(-1)
    q, kn = _padded(s["q_idx"], req, num, B, N), _padded(s["kidx_new"], req, num, B, N)
    keys = s["kidx"][torch.clamp(s["bt"], min=0).long()].float().reshape(B, MB * PAGE, c["G"], -1)
    dots = torch.einsum("bngd,btgd->bngt", q, keys)
    cached = torch.arange(MB * PAGE, device="cuda")[None] < ctx[:, None]
    dots = torch.where(cached[:, None, None, :], dots, -torch.inf)
    scores = dots.reshape(B, N, c["G"], MB, PAGE).amax(-1)
    drafted = torch.einsum("bngd,bmgd->bngm", q, kn)
    drafted = torch.where(reach[:, :, None, :], drafted, -torch.inf)
    at = (pos // PAGE).clamp(max=MB - 1)[:, None, None, :].expand(drafted.shape)
    scores = scores.scatter_reduce(-1, at, drafted, "amax")
    return {"q_req": req.int(), "q_pos": pos[req, num].int(), "anc": anc[req, num], "scores": scores[req, num]}


def _plain_attend(s):
    c = s["case"]
    B, N, G, D, K = c["B"], c["nodes"], c["G"], c["D"], c["topk"]
    req, num, reach, depth = _layout(s)
    R, ctx, sel = req.numel(), s["ctx"].long(), s["sel"].long()
    pages = torch.clamp(s["bt"].long()[req[:, None, None], torch.clamp(sel, min=0)], min=0)
    group = torch.arange(G, device="cuda")[None, :, None]
    k = s["k"].transpose(1, 2)[pages, group].float().reshape(R, G, K * PAGE, D)
    v = s["v"].transpose(1, 2)[pages, group].float().reshape(R, G, K * PAGE, D)
    token = (sel[..., None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(R, G, K * PAGE)
    seen = (token >= 0) & (token < ctx[req][:, None, None])
    kn = _padded(s["k_new"], req, num, B, N)[req].transpose(1, 2)
    vn = _padded(s["v_new"], req, num, B, N)[req].transpose(1, 2)
    block = ((ctx[:, None] + depth) // PAGE)[req]                                     # of each drafted token
    chosen = (sel[..., None] == block[:, None, None, :]).any(2)                       # [R, G, N]
    seen = torch.cat([seen, chosen & reach[req, num][:, None, :]], -1)
    k, v = torch.cat([k, kn], 2), torch.cat([v, vn], 2)
    q = s["q"].float().reshape(R, G, -1, D)
    logits = torch.einsum("rghd,rgtd->rght", q, k) * (1.0 / D ** 0.5)
    logits = torch.where(seen[:, :, None, :], logits, -torch.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("rght,rgtd->rghd", e, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.reshape(R, c["Hq"], D).to(torch.bfloat16), "lse": lse.reshape(R, c["Hq"])}


def _plain_verify(s):
    """For every node at once: which of its children, in order, is the first accepted, and what distribution is
    left when none is.  Then the path from each root.  In 64 bits: the sums are long and the comparisons sharp."""
    c = s["case"]
    B, N, V = c["B"], c["nodes"], c["vocab"]
    req, num, reach, depth = _layout(s)
    off, R = s["off"].long(), req.numel()
    p, tok, u = s["p"].double(), s["tokens"].long(), s["u_accept"].double()
    q = None if s["q"] is None else s["q"].double()
    up = torch.where(s["parents"] >= 0, s["parents"].long() + off[req], R)            # row R: above the roots
    child = torch.full((R + 1, N), -1, dtype=torch.long, device="cuda")              # children in order
    same = (up[:, None] == up[None, :]) & (torch.arange(R, device="cuda")[None] < torch.arange(R, device="cuda")[:, None])
    child[up, torch.where(up < R, same.sum(1), 0)] = torch.arange(R, device="cuda")
    child = child[:R]
    at = torch.arange(R, device="cuda")
    left = p.clone()                                                                  # what the next child is held to
    mass, scale = torch.ones(R, dtype=torch.float64, device="cuda"), torch.zeros(R, dtype=torch.float64, device="cuda")
    took = torch.full((R,), -1, dtype=torch.long, device="cuda")
    for k in range(s["children"]):
        x = child[:, k]
        open_ = (x >= 0) & (took < 0)
        t = tok[torch.clamp(x, min=0)]
        r, ux = left[at, t], u[torch.clamp(x, min=0)]
        yes = open_ & (ux * (1.0 if q is None else q[at, t]) * mass < r)
        took = torch.where(yes, x, took)
        no = open_ & ~yes
        if q is None:
            mass = torch.where(no, mass - r, mass)
            left[at, t] = torch.where(no, 0.0, r)
        else:
            scale = torch.where(no, scale + mass, scale)
            left = torch.where(no[:, None], torch.clamp(p - scale[:, None] * q, min=0), left)
            mass = torch.where(no, left.sum(-1), mass)
    here = off[:-1].clone()
    path = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    n_acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    on, last = torch.ones(B, dtype=torch.bool, device="cuda"), here.clone()
    for d in range(N):
        slot = torch.where(on, off[:-1] + d, R)
        path = torch.cat([path, path[:1]]).scatter(0, slot, (here - off[:-1]).int())[:R]
        n_acc += on
        last = torch.where(on, here, last)
        nxt = took[here]
        on = on & (nxt >= 0)
        here = torch.where(on, nxt, here)
    left = left[last]
    left = torch.where((left.sum(-1) > 0)[:, None], left, p[last])
    run_ = left.cumsum(-1)
    over = run_ > s["u_next"].double()[:, None] * run_[:, -1:]
    token = torch.where(over.any(-1), over.int().argmax(-1), V - 1)
    return {"path": path, "n_acc": n_acc, "token": token.int()}


def _plain_commit(s):
    off, ctx, path = s["off"].long(), s["ctx"].long(), s["path"].long()
    row = torch.arange(path.numel(), device="cuda")
    req = torch.searchsorted(off, row, right=True) - 1
    k = row - off[req]
    taken = k < s["n_acc"].long()[req]
    src, req, pos = (off[req] + path)[taken], req[taken], (ctx[req] + k)[taken]
    page, at = s["bt"].long()[req, pos // PAGE], pos % PAGE
    for name in ("k", "v", "kidx"):
        s[name][:, page, at] = s[name + "_new"][:, src]
    return {"k": s["k"], "v": s["v"], "kidx": s["kidx"], "lens": (s["ctx"] + s["n_acc"])}


def run(state):
    if own:
        return _own(state)
    return {"score": _plain_score, "attend": _plain_attend, "verify": _plain_verify,
            "commit": _plain_commit}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass costs

def work(case):
    ctx, counts = _per_request(case)
    rows, op = sum(counts), case["op"]
    if op == "score":
        G, Di = case["G"], case["Di"]
        blocks = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, counts)]
        scores = sum(n for n in counts) * G * max(blocks) * 4
        return {"bytes": sum(ctx) * G * Di * 2 + 2 * rows * G * Di * 2 + scores + rows * 20,
                "flops": 2 * Di * G * sum(n * (c + n) for c, n in zip(ctx, counts))}
    if op == "attend":
        Hq, G, D = case["Hq"], case["G"], case["D"]
        kv, flops = 0, 0
        for c, n in zip(ctx, counts):
            core, add, pool = _union(case, c, n)
            kv += (min(c // PAGE, core + min(pool, add * n)) * PAGE + c % PAGE + n) * G * D * 4
            flops += 4 * D * Hq * n * min(c, (core + add) * PAGE + c % PAGE)
        return {"bytes": kv + 2 * rows * Hq * D * 2 + rows * (Hq * 4 + G * case["topk"] * 4 + 8), "flops": flops}
    if op == "verify":
        per = case["vocab"] * 4 * (2 if case["drafts"] else 1)   # the row that the next token is drawn from
        return {"bytes": case["B"] * per + rows * 24, "flops": case["B"] * case["vocab"] * 3}
    moved = sum(_accepted(case)) * case["layers"] * case["G"] * (2 * case["D"] + case["Di"]) * 2
    return {"bytes": 2 * moved + rows * 4, "flops": 0}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"score": _exact_score, "attend": _exact_attend, "verify": _exact_verify,
            "commit": _exact_commit}[case["op"]](s)


def _cached(pool, s, b, ctx):
    """The cached rows of request b in order, in 64 bits: [ctx][G][width]."""
    pages = s["bt"][b, :(ctx + PAGE - 1) // PAGE].long()
    return pool[pages].flatten(0, 1)[:ctx].double()


def _exact_score(s):
    c, off, ctx = s["case"], s["off"].tolist(), s["ctx"].tolist()
    depth, anc = _depths(s["off"], s["parents"])
    R, MB = len(depth), s["bt"].shape[1]
    scores = torch.full((R, c["G"], MB), -torch.inf, dtype=torch.float64, device="cuda")
    req, pos = [], []
    for b in range(len(ctx)):
        keys = _cached(s["kidx"], s, b, ctx[b])
        n = off[b + 1] - off[b]
        req += [b] * n
        pos += [ctx[b] + d for d in depth[off[b]:off[b + 1]]]
        q = s["q_idx"][off[b]:off[b + 1]].double()
        for g in range(c["G"]):
            dots = q[:, g] @ keys[:, g].T
            full = ctx[b] // PAGE
            if full:
                scores[off[b]:off[b + 1], g, :full] = dots[:, :full * PAGE].reshape(n, full, PAGE).amax(-1)
            if ctx[b] % PAGE:
                scores[off[b]:off[b + 1], g, full] = dots[:, full * PAGE:].amax(-1)
        for i in range(n):
            for m in range(i + 1):
                if anc[off[b] + i] >> m & 1:
                    d = (s["q_idx"][off[b] + i].double() * s["kidx_new"][off[b] + m].double()).sum(-1)
                    j = (ctx[b] + depth[off[b] + m]) // PAGE
                    scores[off[b] + i, :, j] = torch.maximum(scores[off[b] + i, :, j], d)
    anc = [a - (1 << 64) if a >> 63 else a for a in anc]
    return {"q_req": torch.tensor(req, dtype=torch.int32), "q_pos": torch.tensor(pos, dtype=torch.int32),
            "anc": torch.tensor(anc, dtype=torch.int64), "scores": scores}


def _exact_attend(s):
    c, off, ctx = s["case"], s["off"].tolist(), s["ctx"].tolist()
    depth, anc = _depths(s["off"], s["parents"])
    hpg, D, MB = c["Hq"] // c["G"], c["D"], s["bt"].shape[1]
    outs, lses = [], []
    for b in range(len(ctx)):
        r0, n = off[b], off[b + 1] - off[b]
        keys, vals = _cached(s["k"], s, b, ctx[b]), _cached(s["v"], s, b, ctx[b])
        pos = torch.tensor(list(range(ctx[b])) + [ctx[b] + d for d in depth[r0:r0 + n]], device="cuda")
        path = torch.tensor([[bool(anc[r0 + i] >> m & 1) for m in range(n)] for i in range(n)], device="cuda")
        path = torch.cat([torch.ones((n, ctx[b]), dtype=torch.bool, device="cuda"), path], 1)
        out = torch.empty((n, c["Hq"], D), dtype=torch.float64, device="cuda")
        lse = torch.empty((n, c["Hq"]), dtype=torch.float64, device="cuda")
        for g in range(c["G"]):
            has = torch.zeros((n, MB + 1), dtype=torch.bool, device="cuda")
            pick = s["sel"][r0:r0 + n, g].long()
            has.scatter_(1, torch.where(pick < 0, MB, pick), True)
            see = has[:, pos // PAGE] & path
            need = see.any(0)                                          # no row sees the others
            kk = torch.cat([keys[:, g], s["k_new"][r0:r0 + n, g].double()])[need]
            vv = torch.cat([vals[:, g], s["v_new"][r0:r0 + n, g].double()])[need]
            see = see[:, need]
            for h in range(g * hpg, (g + 1) * hpg):
                a = s["q"][r0:r0 + n, h].double() @ kk.T / D ** 0.5
                a = a.masked_fill(~see, -torch.inf)
                lse[:, h] = torch.logsumexp(a, -1)
                out[:, h] = torch.nan_to_num(torch.softmax(a, -1)) @ vv
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_verify(s):
    off, parents = s["off"].tolist(), s["parents"].tolist()
    tok, u = s["tokens"].tolist(), s["u_accept"].tolist()
    path, n_acc, nxt = [], [], []
    for b in range(len(off) - 1):
        r0, n = off[b], off[b + 1] - off[b]
        at, taken = 0, []
        while True:
            taken.append(at)
            p = s["p"][r0 + at].double()
            q = None if s["q"] is None else s["q"][r0 + at].double()
            left, whole, step = p.clone(), 1.0, None
            for x in range(at + 1, n):
                if parents[r0 + x] != at:
                    continue
                t = tok[r0 + x]
                draft = 1.0 if q is None else float(q[t])
                if u[r0 + x] * draft * whole < float(left[t]):
                    step = x
                    break
                if q is None:
                    whole -= float(left[t])
                    left[t] = 0.0
                else:                       # unnormalised: left is whole times the distribution that is left
                    left = torch.clamp(left - whole * q, min=0)
                    whole = float(left.sum())
            if step is None:
                break
            at = step
        if not float(left.sum()) > 0:
            left = p
        total = left.cumsum(0)
        token = int(torch.searchsorted(total, total[-1:] * float(s["u_next"][b]), right=True)[0])
        path += taken + [-1] * (n - len(taken))
        n_acc.append(len(taken))
        nxt.append(min(token, p.numel() - 1))
    return {"path": torch.tensor(path, dtype=torch.int32), "n_acc": torch.tensor(n_acc, dtype=torch.int32),
            "token": torch.tensor(nxt, dtype=torch.int32)}


def _exact_commit(s):
    off, ctx, path, acc = s["off"].tolist(), s["ctx"].tolist(), s["path"].tolist(), s["n_acc"].tolist()
    out = {name: s[name].clone() for name in ("k", "v", "kidx")}
    for b in range(len(ctx)):
        for k in range(acc[b]):
            pos = ctx[b] + k
            page = int(s["bt"][b, pos // PAGE])
            for name in out:
                out[name][:, page, pos % PAGE] = s[name + "_new"][:, off[b] + path[off[b] + k]]
    return {**{k: v.double() for k, v in out.items()}, "lens": torch.tensor([c + a for c, a in zip(ctx, acc)],
                                                                           dtype=torch.int32)}
