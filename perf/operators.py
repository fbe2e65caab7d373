"""The operators of a drafted decode step, as they are measured.

One step of speculative decoding passes, for every sequence, its last token and the tokens drafted
after it (a chain, or a tree) through the model at once. Beside the expert layer and the lm_head
that takes four operators over one paged key/value cache:

* rope:   rotary positions of the new queries and keys, the keys and values written into the cache
* attend: attention of the drafted tree's rows over the cached tokens and their own ancestors
* verify: drafted tokens tested against the target's probabilities, from given random numbers
* keep:   the accepted path's keys and values moved to where the next step expects them

`own` False: each in its plain form (elementary torch operations). True: this repository's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence, one new token: the smallest call, where latency counts
        _rope("rope one row", seqs=1, rows=1, length=777, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
              layout="half", rotary=128, scaling="none", far=0),
        # eight sequences with trees of up to 13 rows, fp16, interleaved pairs over half of each head
        _rope("rope trees partial", seqs=8, rows=13, length=1500, heads=40, kv_heads=8, dim=128, page=16,
              dtype="f16", layout="interleaved", rotary=64, scaling="linear", far=100000),
        # a prompt of the largest prefill pass, frequencies scaled by parts for a long context
        _rope("rope prompt", seqs=1, rows=4096, length=0, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
              layout="half", rotary=128, scaling="parts", far=0),
        # one sequence, one token, a short cache: plain decode at its smallest
        _attend("attend one row", seqs=1, rows=1, length=777, heads=32, kv_heads=8, dim=128, page=64,
                dtype="bf16", tree=False),
        # ordinary serving: ragged lengths, trees of up to 16 rows
        _attend("attend trees", seqs=8, rows=16, length=8200, heads=32, kv_heads=8, dim=128, page=64,
                dtype="bf16", tree=True),
        # the widest trees, fp16, small heads
        _attend("attend wide trees", seqs=4, rows=64, length=4100, heads=32, kv_heads=4, dim=64, page=16,
                dtype="f16", tree=True),
        # long caches, a chain of drafts: the largest call
        _attend("attend long", seqs=16, rows=5, length=32700, heads=40, kv_heads=8, dim=128, page=128,
                dtype="bf16", tree=False),
        # one sequence, a chain of four drafts over the lm_head's vocabulary
        _verify("verify one chain", seqs=1, rows=5, vocab=131072, logits="f32", sampled=True, branch=1),
        # trees whose drafts were chosen without chance, bf16 logits, some sequences greedy
        _verify("verify trees", seqs=8, rows=16, vocab=131072, logits="bf16", sampled=False, branch=3),
        # a full batch, drafts drawn from given probabilities, an odd vocabulary
        _verify("verify batch", seqs=64, rows=6, vocab=100003, logits="f32", sampled=True, branch=1),
        # the path of one tree
        _keep("keep one", seqs=1, rows=16, length=777, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # a full batch's paths
        _keep("keep batch", seqs=64, rows=24, length=1000, kv_heads=8, dim=128, page=16, dtype="f16"),
    ]


def _rope(name=None, **c):
    return _named(name, dict(op="rope", **c))


def _attend(name=None, **c):
    return _named(name, dict(op="attend", **c))


def _verify(name=None, **c):
    return _named(name, dict(op="verify", **c))


def _keep(name=None, **c):
    return _named(name, dict(op="keep", **c))


def _named(name, c):
    return c if name is None else dict(c, name=name)


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


#: (query heads, key/value heads, head width)
HEADS = [(8, 2, 64), (32, 8, 128), (40, 8, 128), (32, 4, 64), (16, 16, 96), (64, 4, 128), (24, 8, 80), (16, 2, 256),
         (28, 4, 128), (71, 1, 64)]


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "verify", "keep"])
    heads, kv_heads, dim = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    if op == "rope":
        seqs = _log(rng, 1, 64)
        rotary = rng.choice([dim, dim // 2, dim // 4])
        return _rope(seqs=seqs, rows=_log(rng, 1, max(1, 4096 // seqs * 32 * 128 // (heads * dim))), length=_log(rng, 1, 2000),
                     heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype,
                     layout=rng.choice(["half", "interleaved"]), rotary=rotary,
                     scaling=rng.choice(["none", "linear", "base", "parts"]), far=rng.choice([0, 30000, 900000]))
    if op == "attend":
        seqs = _log(rng, 1, 64)
        most = min(16 * 32700 * 8 * 128 // (2 * kv_heads), 16 * 32700 * 5 * 40 * 128 // heads) // (seqs * dim)
        length = _log(rng, 1, min(131072, most))
        return _attend(seqs=seqs, rows=_log(rng, 1, min(64, max(1, most // length))), length=length,
                       heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, tree=rng.random() < 0.6)
    if op == "verify":
        vocab = rng.choice([32000, 50257, 131072, 151936, _log(rng, 1000, 200000)])
        seqs = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, min(40, 64 * 6 * 100003 // (vocab * seqs))))
        return _verify(seqs=seqs, rows=rows, vocab=vocab, logits=rng.choice(["f32", "bf16"]), sampled=rng.random() < 0.6,
                       branch=rng.choice([1, 1, 2, 4]))
    return _keep(seqs=_log(rng, 1, 64), rows=_log(rng, 2, 64), length=_log(rng, 1, 1000), kv_heads=kv_heads, dim=dim,
                 page=page, dtype=dtype)


# ------------------------------------------------------------------ shapes of a case (the same for every seed)

def _plan(case):
    """Per sequence: cached tokens, rows of this pass, parents of the rows, kept path; from the case alone."""
    B, most = case["seqs"], case["rows"]
    r = random.Random(7 * B + 11 * most + 13 * case.get("length", 0) + 17 * case.get("vocab", 0))
    lens, rows, parents, paths = [], [], [], []
    for b in range(B):
        full = case.get("length", 0)
        lens.append(full if b == 0 or full < 8 else r.randint(full // 4, full))
        n = most if b == 0 or most < 4 else r.randint(most // 2, most)
        if b == B - 1 and B >= 8:          # one sequence of a full batch starts here: nothing is cached yet
            lens[b] = 0
        rows.append(n)
        width = case.get("branch", 3 if case.get("tree") or case["op"] in ("keep", "rope") else 1)
        par = [-1]
        for i in range(1, n):
            par.append(i - 1 if width == 1 else r.randint(max(0, (i - 1) // width), i - 1))
        parents.append(par)
        path, i = [0], 0
        while True:                        # a walk down the tree
            kids = [c for c in range(1, n) if par[c] == i]
            if not kids or r.random() < 0.05:
                break
            i = r.choice(kids)
            path.append(i)
        paths.append(path)
    return lens, rows, parents, paths


def _depths(par):
    d = []
    for i, p in enumerate(par):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _masks(par, tree):
    m = []
    for i, p in enumerate(par):
        m.append((1 << i) | (m[p] if p >= 0 else 0) if tree else (1 << (i + 1)) - 1)
    return m


def work(case):
    lens, rows, parents, paths = _plan(case)
    R = sum(rows)
    if case["op"] == "verify":
        e = 4 if case["logits"] == "f32" else 2
        V = case["vocab"]
        # every row's logits once; the draft probabilities of the row where a sequence stops
        return {"bytes": R * V * e + (case["seqs"] * V * 4 if case["sampled"] else 0), "flops": 6 * R * V}
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "keep":
        moved = sum(i != p for path in paths for i, p in enumerate(path))
        return {"bytes": moved * 2 * 2 * Hk * D * 2 + 8 * R, "flops": 0}
    H = case["heads"]
    if case["op"] == "rope":
        return {"bytes": R * D * 2 * (2 * H + 4 * Hk), "flops": R * (H + Hk) * case["rotary"] * 3}
    tokens = sum(t + n for t, n in zip(lens, rows))
    seen = 0
    for t, n, par in zip(lens, rows, parents):
        seen += n * t + sum(bin(m).count("1") for m in _masks(par, case["tree"]))
    return {"bytes": tokens * Hk * D * 2 * 2 + R * H * D * 2 * 2, "flops": 4 * seen * H * D}


# ------------------------------------------------------------------ inputs

def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


def _starts(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return s


def frequencies(rotary, scaling, base=10000.0, factor=8.0, trained=8192):
    """Radians per position of each pair, and the factor on cosine and sine, scaled for a context
    `factor` times the trained one: by stretching positions, by a larger base, or by parts (pairs
    that turn often in the trained length keep their speed, slow ones are stretched)."""
    j = torch.arange(rotary // 2, dtype=torch.float64)
    if scaling == "base" and rotary > 2:
        base = base * factor ** (rotary / (rotary - 2))
    f = base ** (-2.0 * j / rotary)
    if scaling == "linear":
        f = f / factor
    if scaling != "parts":
        return f, 1.0
    turns = trained * f / (2 * math.pi)
    ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)      # 0: at most one turn, 1: 32 turns and more
    return f / factor * (1 - ramp) + f * ramp, 0.1 * math.log(factor) + 1.0


def _cache(case, lens, rows, g):
    """A paged cache of every sequence's tokens: pages in random order, all slots filled."""
    P, Hk, D = case["page"], case["kv_heads"], case["dim"]
    need = [-(-(t + n) // P) for t, n in zip(lens, rows)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, P, Hk, D)
    dt = DTYPES[case["dtype"]]
    k = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    return k, v, table


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, rows, parents, paths = _plan(case)
    starts = _starts(rows)
    R, B, N = starts[-1], len(rows), max(rows)
    s = {"case": case, "lens": lens, "rows": rows, "most_len": max(lens), "N": N, "R": R, "row_start": _ints(starts)}
    # for the plain forms: the row of (sequence, i), and of each row its sequence and i
    grid = torch.tensor([[starts[b] + min(i, max(rows[b] - 1, 0)) for i in range(N)] for b in range(B)])
    s["grid"] = grid.cuda()
    s["valid"] = torch.tensor([[i < rows[b] for i in range(N)] for b in range(B)]).cuda()
    s["row_seq"] = torch.tensor([b for b in range(B) for _ in range(rows[b])]).cuda()
    s["row_at"] = torch.tensor([i for b in range(B) for i in range(rows[b])]).cuda()
    if case["op"] == "verify":
        return _prepare_verify(case, g, s, parents, starts)
    dt = DTYPES[case["dtype"]]
    s["k"], s["v"], s["table"] = _cache(case, lens, rows, g)
    s["len"] = _ints(lens)
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "keep":
        s["n_keep"] = _ints([len(p) for p in paths])
        s["path"] = _ints([(p + [-1] * n)[:n][i] for p, n in zip(paths, rows) for i in range(n)])
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    H = case["heads"]
    if case["op"] == "rope":
        # one projection's output holds the queries, keys and values of a row side by side
        qkv = torch.empty((R, (H + 2 * Hk) * D), dtype=dt, device="cuda").normal_(generator=g)
        s["q"], s["kn"], s["vn"] = qkv[:, :H * D], qkv[:, H * D:(H + Hk) * D], qkv[:, (H + Hk) * D:]
        f, m = frequencies(case["rotary"], case["scaling"])
        s["freqs"], s["magnitude"] = f.cuda(), m
        flat = case["rows"] > 64           # a prompt: one token after another; else a drafted tree
        s["pos"] = _ints([case["far"] + t + (i if flat else d) for t, par in zip(lens, parents)
                          for i, d in enumerate(_depths(par))])
        s["q_out"] = torch.zeros((R, H * D), dtype=dt, device="cuda")
        return s
    s["q"] = torch.empty((R, H * D), dtype=dt, device="cuda").normal_(generator=g)
    s["mask"] = _ints([_signed(m) for par in parents for m in _masks(par, case["tree"])], torch.int64)
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.zeros((R, H * D), dtype=dt, device="cuda")
    return s


def _prepare_verify(case, g, s, parents, starts):
    R, V, B = s["R"], case["vocab"], case["seqs"]
    z = torch.empty((R, V), device="cuda").normal_(0, 2.5, generator=g)
    s["logits"] = z.to(DTYPES[case["logits"]])
    T = [0.0 if not case["sampled"] and b % 4 == 3 else 0.7 + 0.1 * (b % 4) for b in range(B)]
    s["temperature"] = _ints(T, torch.float32)
    q = torch.softmax((z + torch.empty_like(z).normal_(0, 0.5, generator=g)) / 0.9, dim=1)
    del z
    # the drafted tokens: drawn from the draft's probabilities at their parent, or its most likely ones
    par = _ints([starts[b] + max(p, 0) for b, ps in enumerate(parents) for p in ps], torch.int64)
    if case["sampled"]:
        s["tokens"] = torch.multinomial(q[par], 1, generator=g)[:, 0].to(torch.int32) if R * V < 1 << 28 else torch.cat(
            [torch.multinomial(q[c], 1, generator=g)[:, 0].to(torch.int32) for c in par.split(64)])
        s["draft"] = q
    else:
        nth = [sum(p == ps[i] for p in ps[:i]) for ps in parents for i in range(len(ps))]
        top = torch.topk(q, max(nth) + 1, dim=1).indices
        s["tokens"] = top[par, _ints(nth, torch.int64)].to(torch.int32)
        s["draft"] = None
    s["parent"] = _ints([p for ps in parents for p in ps])
    s["u_test"] = torch.rand(R, device="cuda", generator=g)
    s["u_pick"] = torch.rand(R, device="cuda", generator=g)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_rope, "attend": _plain_attend, "verify": _plain_verify, "keep": _plain_keep}[s["case"]["op"]](s)


def _run_own(s):
    op = s["case"]["op"]
    h = s.get("handle")
    if h is None:                          # what a program sets up once: the cache's descriptor, the workspaces
        h = s["handle"] = _handle(s)
    if op == "rope":
        h[0].append(h[1], s["q"], s["kn"], s["vn"], s["row_start"], positions=s["pos"], out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "attend":
        h[0].attend(s["q"], s["row_start"], mask=s["mask"], scale=s["scale"], out=s["out"])
        return {"out": s["out"]}
    if op == "keep":
        h[0].keep(s["row_start"], s["n_keep"], s["path"], new_len=s["new_len"])
        return {"k": s["k"], "v": s["v"], "len": s["new_len"]}
    n_keep, path, tokens, logprobs = h[0].verify(
        s["logits"], s["tokens"], s["row_start"], s["u_test"], s["u_pick"], parent=s["parent"],
        draft_probs=s["draft"], temperature=s["temperature"])
    return {"n_keep": n_keep, "path": path, "tokens": tokens, "logprobs": logprobs}


def _handle(s):
    from latent_mixture_experts_bf16_amd import drafted
    c = s["case"]
    if c["op"] == "verify":
        return (drafted.Verifier(c["vocab"], max_rows=s["R"], max_seqs=c["seqs"]),)
    cache = drafted.PagedCache(s["k"], s["v"], s["table"], s["len"])
    if c["op"] == "rope":
        return cache, drafted.Rope(s["freqs"], layout=c["layout"], magnitude=s["magnitude"])
    return (cache,)


# ------------------------------------------------------------------ the plain forms

def _slots(s, b, token):
    """Index into the cache's (page, slot) pairs of tokens `token` of sequences `b`."""
    P = s["case"]["page"]
    return s["table"][b, token // P].long() * P + token % P


def _turn(x, cos, sin, layout, rd):
    x = x.float()
    r = x[..., :rd]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rd // 2], r[..., rd // 2:])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([ya, yb], dim=-1).flatten(-2) if layout == "interleaved" else torch.cat([ya, yb], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    H, Hk, D, rd, R = c["heads"], c["kv_heads"], c["dim"], c["rotary"], s["R"]
    angle = s["pos"].double()[:, None, None] * s["freqs"]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    q = _turn(s["q"].reshape(R, H, D), cos, sin, c["layout"], rd).to(s["q"].dtype)
    k = _turn(s["kn"].reshape(R, Hk, D), cos, sin, c["layout"], rd).to(s["k"].dtype)
    at = _slots(s, s["row_seq"], s["len"].long()[s["row_seq"]] + s["row_at"])
    s["k"].view(-1, Hk, D)[at] = k
    s["v"].view(-1, Hk, D)[at] = s["vn"].reshape(R, Hk, D)
    return {"q": q.reshape(R, H * D), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    H, Hk, D, R, N, B = c["heads"], c["kv_heads"], c["dim"], s["R"], s["N"], c["seqs"]
    G, L = H // Hk, s["most_len"] + N
    ln = s["len"].long()
    last = (ln + s["valid"].sum(1) - 1).clamp(min=0)
    t = torch.arange(L, device="cuda")
    at = _slots(s, torch.arange(B, device="cuda")[:, None], torch.minimum(t, last[:, None]))
    q = s["q"][s["grid"]].float().reshape(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * G, D)
    k = s["k"].view(-1, Hk, D)[at].float().permute(0, 2, 3, 1).contiguous()
    sc = torch.matmul(q, k) * s["scale"]
    del k
    j = (t[None] - ln[:, None])[:, None]                       # [B,1,L]: the row's number among the drafted ones
    bits = (s["mask"][s["grid"]][:, :, None] >> j.clamp(0, 63)) & 1
    see = (j < 0) | ((j < 64) & (bits == 1))                   # [B,N,L]
    see = see[:, None, :, None, :].expand(B, Hk, N, G, L).reshape(B, Hk, N * G, L)
    sc = torch.where(see, sc, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    del sc, see
    p = p / p.sum(-1, keepdim=True)
    v = s["v"].view(-1, Hk, D)[at].float().permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(p, v).reshape(B, Hk, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * D)
    s["out"][:] = o[s["row_seq"], s["row_at"]].to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_verify(s):
    # in 64 bits: whole tokens come out, and a draw may lie next to the border of two
    N, R, B = s["N"], s["R"], s["case"]["seqs"]
    grid, valid, q = s["grid"], s["valid"], s["draft"]
    T = s["temperature"].double()
    z = s["logits"].double()
    top = z.amax(1, keepdim=True)
    best = torch.argmax((z == top).to(torch.int8), dim=1)      # the lowest index among equals
    Tr = T[s["row_seq"]][:, None]
    p = torch.exp((z - top) / torch.where(Tr > 0, Tr, torch.ones_like(Tr)))
    p = p / p.sum(1, keepdim=True)
    ids = torch.arange(z.shape[1], device="cuda")
    p = torch.where(Tr > 0, p, (ids == best[:, None]).double())
    parent = torch.where(valid, s["parent"][grid], -2)
    token = s["tokens"].long()[grid]
    ut, up = s["u_test"].double(), s["u_pick"].double()
    if q is None:
        cum = p.cumsum(1)
        pick = (cum <= up[:, None] * cum[:, -1:]).sum(1)
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    S, rest = torch.zeros(B, dtype=torch.float64, device="cuda"), torch.ones(B, dtype=torch.float64, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    said = torch.full((B, N), -1, dtype=torch.long, device="cuda")
    logp = torch.zeros((B, N), dtype=torch.float64, device="cuda")
    kept = torch.ones(B, dtype=torch.long, device="cuda")
    seq = torch.arange(B, device="cuda")
    at = lambda: grid[seq, cur]  # noqa: E731
    for r in range(1, N):
        child = parent[:, r] == cur
        x = token[:, r]
        row = at()
        px = p[row, x]
        if q is None:
            yes = child & (pick[row] == x)
        else:
            qx = q[row, x].double()
            yes = child & (ut[grid[:, r]] * qx * rest < (px - S * qx).clamp(min=0))
            no = child & ~yes
            S = torch.where(no, S + rest, S)
            rest = torch.where(no, (p[row] - S[:, None] * q[row]).clamp(min=0).sum(1), rest)
            S, rest = torch.where(yes, 0.0, S), torch.where(yes, 1.0, rest)
        here = yes[:, None] & (torch.arange(N, device="cuda") == (kept - 1)[:, None])
        said, logp = torch.where(here, x[:, None], said), torch.where(here, px.log()[:, None], logp)
        path = torch.where(yes[:, None] & (torch.arange(N, device="cuda") == kept[:, None]), r, path)
        kept, cur = kept + yes, torch.where(yes, r, cur)
    row = at()
    if q is None:
        t = pick[row]
    else:
        w = (p[row] - S[:, None] * q[row]).clamp(min=0)
        w = torch.where(w.sum(1, keepdim=True) > 0, w, p[row])
        cum = w.cumsum(1)
        t = (cum <= up[row][:, None] * cum[:, -1:]).sum(1)
    here = torch.arange(N, device="cuda") == (kept - 1)[:, None]
    said, logp = torch.where(here, t[:, None], said), torch.where(here, p[row, t].log()[:, None], logp)
    b, i = s["row_seq"], s["row_at"]
    return {"n_keep": kept.int(), "path": path[b, i].int(), "tokens": said[b, i].int(), "logprobs": logp[b, i].float()}


def _plain_keep(s):
    b, i = s["row_seq"], s["row_at"]
    Hk, D = s["case"]["kv_heads"], s["case"]["dim"]
    ln = s["len"].long()[b]
    live = i < s["n_keep"].long()[b]
    src = _slots(s, b, ln + torch.where(live, s["path"].long(), i))   # rows that are not kept stay
    dst = _slots(s, b, ln + i)
    k, v = s["k"].view(-1, Hk, D), s["v"].view(-1, Hk, D)
    nk, nv = k[src], v[src]
    k[dst] = nk
    v[dst] = nv
    torch.add(s["len"], s["n_keep"], out=s["new_len"])
    return {"k": s["k"], "v": s["v"], "len": s["new_len"]}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, rows, parents, paths = _plan(case)
    starts = _starts(rows)
    return {"rope": _exact_rope, "attend": _exact_attend, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](
        case, s, lens, rows, parents, paths, starts)


def _places(s, case, b, tokens):
    table = s["table"][b].tolist()
    return [(table[t // case["page"]], t % case["page"]) for t in tokens]


def _exact_rope(case, s, lens, rows, parents, paths, starts):
    H, Hk, D, rd = case["heads"], case["kv_heads"], case["dim"], case["rotary"]
    R = s["R"]
    turn = torch.polar(torch.full((R, 1, rd // 2), float(s["magnitude"]), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None, None] * s["freqs"])

    def spin(x, heads):
        x = x.double().reshape(R, heads, D).clone()
        r = x[..., :rd]
        pair = torch.view_as_complex(r.reshape(R, heads, rd // 2, 2).contiguous() if case["layout"] == "interleaved"
                                     else r.reshape(R, heads, 2, rd // 2).transpose(-1, -2).contiguous())
        y = torch.view_as_real(pair * turn)
        x[..., :rd] = (y if case["layout"] == "interleaved" else y.transpose(-1, -2)).reshape(R, heads, rd)
        return x

    k, v = s["k"].double(), s["v"].double()
    kn, vn = spin(s["kn"], Hk), s["vn"].double().reshape(R, Hk, D)
    for b, (t, n) in enumerate(zip(lens, rows)):
        if n:
            at = torch.tensor(_places(s, case, b, range(t, t + n)), device="cuda")
            k[at[:, 0], at[:, 1]] = kn[starts[b]:starts[b] + n]
            v[at[:, 0], at[:, 1]] = vn[starts[b]:starts[b] + n]
    return {"q": spin(s["q"], H).reshape(R, H * D), "k": k, "v": v}


def _exact_attend(case, s, lens, rows, parents, paths, starts):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    out = torch.zeros((s["R"], H, D), dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(lens, rows)):
        at = torch.tensor(_places(s, case, b, range(t + n)), device="cuda")
        see = torch.ones((n, t + n), dtype=torch.bool)
        for i, m in enumerate(_masks(parents[b], case["tree"])):
            see[i, t:] = torch.tensor([bool(m >> j & 1) for j in range(n)])
        see = see.cuda()
        for h in range(Hk):
            k, v = s["k"][at[:, 0], at[:, 1], h].double(), s["v"][at[:, 0], at[:, 1], h].double()
            for g in range(G):
                q = s["q"][starts[b]:starts[b] + n].double().reshape(n, H, D)[:, h * G + g]
                w = torch.softmax((q @ k.T * s["scale"]).masked_fill(~see, -math.inf), dim=1)
                out[starts[b]:starts[b] + n, h * G + g] = w @ v
    return {"out": out.reshape(s["R"], H * D)}


def _exact_verify(case, s, lens, rows, parents, paths, starts):
    n_keep, path, tokens, logp = [], [], [], []
    T, tok = s["temperature"].tolist(), s["tokens"].tolist()
    ut, up = s["u_test"].tolist(), s["u_pick"].tolist()

    def inverse(w, u):
        cum = torch.cumsum(w, 0)
        return int(torch.searchsorted(cum, cum[-1:] * u, right=True).item())

    for b, n in enumerate(rows):
        o = starts[b]

        def target(i):
            z = s["logits"][o + i].double()
            if T[b] == 0:
                w = torch.zeros_like(z)
                w[int(torch.nonzero(z == z.max())[0].item())] = 1.0
                return w
            return torch.softmax(z / T[b], 0)

        cur, walk, said, lp = 0, [0], [], []
        while True:
            p = target(cur)
            kids = [c for c in range(cur + 1, n) if parents[b][c] == cur]
            went = None
            if s["draft"] is None:
                t = inverse(p, up[o + cur])
                went = next((c for c in kids if tok[o + c] == t), None)
            else:
                q = s["draft"][o + cur].double()
                w, total, S = p, 1.0, 0.0
                for c in kids:
                    x = tok[o + c]
                    if ut[o + c] * float(q[x]) * total < float(w[x]):
                        went = c
                        break
                    S += total
                    w = (p - S * q).clamp(min=0)
                    total = float(w.sum())
                if went is None:
                    t = inverse(w if total > 0 else p, up[o + cur])
            x = tok[o + went] if went is not None else t
            said.append(x)
            lp.append(float(p[x].log()))
            if went is None:
                break
            walk.append(went)
            cur = went
        n_keep.append(len(walk))
        path += walk + [-1] * (n - len(walk))
        tokens += said + [-1] * (n - len(said))
        logp += lp + [0.0] * (n - len(lp))
    return {"n_keep": _ints(n_keep), "path": _ints(path), "tokens": _ints(tokens), "logprobs": _ints(logp, torch.float64)}


def _exact_keep(case, s, lens, rows, parents, paths, starts):
    k, v = s["k"].double(), s["v"].double()
    for b, (t, p) in enumerate(zip(lens, paths)):
        for i, node in enumerate(p):       # in order: a path's node never comes before its place
            (src, dst) = _places(s, case, b, [t + node, t + i])
            k[dst], v[dst] = k[src].clone(), v[src].clone()
    return {"k": k, "v": v, "len": _ints([t + len(p) for t, p in zip(lens, paths)])}
