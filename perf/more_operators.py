"""The operators of a served batch's decode step, as they are measured.

Beside the expert layer, the lm_head and the drafted step's operators, a batch of requests takes:

* norm:   queries and keys normed for each head, rotated and appended to the paged cache, in one pass
* write:  the same into a cache held in 8 or 4 bits (blocks of 32 values under a power of two), and read back
* attend: attention that reads such a cache
* shared: attention of a batch whose requests begin with the same long prompt, whose part is computed once
* sample: a token for each row from given random numbers, with temperature, top-k, top-p and min-p

`own` False: each in its plain form (elementary torch operations). True: this repository's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
#: of a code: bits, largest value, exponent of the smallest normal value, bits of the fraction
FORMATS = {"mx8": (8, 448.0, -6, 3), "mx4": (4, 6.0, 0, 1)}
BLOCK = 32
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence, one new token: the smallest call, where latency counts
        _case("norm", "norm one row", seqs=1, rows=1, length=777, heads=32, kv_heads=8, dim=128, page=64,
              dtype="bf16", format="none", layout="half", rotary=128, norm="shared"),
        # a prompt with an odd number of rows, half of each head rotated in neighbouring pairs, a weight for every head
        _case("norm", "norm prompt", seqs=1, rows=2001, length=0, heads=40, kv_heads=8, dim=128, page=16,
              dtype="f16", format="none", layout="interleaved", rotary=64, norm="each"),
        # one new token into an 8-bit cache
        _case("write", "write one row", seqs=1, rows=1, length=777, heads=32, kv_heads=8, dim=128, page=64,
              dtype="bf16", format="mx8", layout="half", rotary=128, norm="shared"),
        # the largest prefill pass's rows into a 4-bit cache
        _case("write", "write prompts", seqs=3, rows=1365, length=100, heads=32, kv_heads=8, dim=128, page=64,
              dtype="bf16", format="mx4", layout="half", rotary=128, norm="none"),
        # plain decode at its smallest over an 8-bit cache
        _case("attend", "attend one row", seqs=1, rows=1, length=777, heads=32, kv_heads=8, dim=128, page=64,
              dtype="bf16", format="mx8", tree=False),
        # drafted trees over ragged lengths in 4 bits
        _case("attend", "attend trees", seqs=8, rows=16, length=8200, heads=32, kv_heads=8, dim=128, page=64,
              dtype="bf16", format="mx4", tree=True),
        # long caches in 8 bits, single tokens: where the bytes of the cache are the step's time
        _case("attend", "attend long", seqs=16, rows=1, length=32700, heads=40, kv_heads=8, dim=128, page=128,
              dtype="f16", format="mx8", tree=False),
        # four requests after one prompt, its end inside a page
        _case("shared", "shared few", seqs=4, rows=1, length=300, shared=1999, groups=1, heads=32, kv_heads=4, dim=64,
              page=16, dtype="f16", format="none", tree=False),
        # a full batch after one long prompt: the largest call
        _case("shared", "shared batch", seqs=64, rows=1, length=700, shared=16000, groups=1, heads=32, kv_heads=8, dim=128,
              page=64, dtype="bf16", format="none", tree=False),
        # one row over the lm_head's vocabulary
        _case("sample", "sample one row", rows=1, vocab=131072, logits="f32", top_k=50, top_p=0.95, min_p=0.0),
        # a batch, bf16 logits: many equal ones; every cut, and greedy rows among them
        _case("sample", "sample batch", rows=64, vocab=131072, logits="bf16", top_k=1000, top_p=0.9, min_p=0.02),
        # many rows, an odd vocabulary, no cut but top-p
        _case("sample", "sample many", rows=256, vocab=100003, logits="f32", top_k=0, top_p=0.92, min_p=0.0),
    ]


def _case(op, name=None, **c):
    return dict(op=op, **c) if name is None else dict(op=op, name=name, **c)


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))


#: (query heads, key/value heads, head width)
HEADS = [(8, 2, 64), (32, 8, 128), (40, 8, 128), (32, 4, 64), (16, 16, 96), (64, 4, 128), (16, 2, 256), (28, 4, 128),
         (71, 1, 64), (10, 2, 192)]


def draw(rng):
    op = rng.choice(["norm", "write", "attend", "attend", "shared", "sample", "sample"])
    if op == "sample":
        vocab = rng.choice([32000, 50257, 131072, 151936, _log(rng, 1000, 200000)])
        return _case(op, rows=_log(rng, 1, min(256, 256 * 100003 // vocab)), vocab=vocab, logits=rng.choice(["f32", "bf16", "f16"]),
                     top_k=rng.choice([0, 0, 1, _log(rng, 2, 2000)]), top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                     min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.3), 3)]))
    heads, kv_heads, dim = rng.choice(HEADS)
    common = dict(heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128, 256]),
                  dtype=rng.choice(["bf16", "f16"]))
    if op in ("norm", "write"):
        seqs = _log(rng, 1, 64)
        return _case(op, seqs=seqs, rows=_log(rng, 1, max(1, 4095 // seqs * 32 * 128 // (heads * dim))), length=_log(rng, 1, 2000),
                     format="none" if op == "norm" else rng.choice(["mx8", "mx4"]), layout=rng.choice(["half", "interleaved"]),
                     rotary=rng.choice([dim, dim // 2, dim // 4]),
                     norm=rng.choice(["shared", "each"] if op == "norm" else ["none", "shared", "each"]), **common)
    if op == "attend":
        seqs = _log(rng, 1, 64)
        most = 16 * 32700 * 8 * 128 // (kv_heads * seqs * dim)
        length = _log(rng, 1, min(131072, most))
        return _case(op, seqs=seqs, rows=_log(rng, 1, min(64, max(1, 16 * 32700 * 40 * 128 * 2 // (heads * dim * seqs * length)))),
                     length=length, format=rng.choice(["mx8", "mx4"]), tree=rng.random() < 0.5, **common)
    seqs = _log(rng, 2, 64)
    most = 64 * 16700 * 32 * 128 // (heads * dim * seqs)
    groups = rng.choice([1, 1, min(3, seqs)])
    shared = _log(rng, 64, min(50000 // groups, most))
    return _case(op, seqs=seqs, rows=_log(rng, 1, min(16, max(1, most // (2 * shared)))), length=_log(rng, 1, 1000), shared=shared,
                 groups=groups, format=rng.choice(["none", "none", "mx8", "mx4"]),
                 tree=rng.random() < 0.4, **common)


# ------------------------------------------------------------------ shapes of a case (the same for every seed)

def _plan(case):
    """Per sequence: cached tokens, rows of this pass, parents of the rows; the groups' starts. From the case alone."""
    B, most, S = case["seqs"], case["rows"], case.get("shared", 0)
    r = random.Random(7 * B + 11 * most + 13 * case["length"] + 17 * S)
    lens, rows, parents = [], [], []
    for b in range(B):
        full = case["length"]
        lens.append(S + (full if b == 0 or full < 8 else r.randint(full // 4, full)))
        n = most if b == 0 or most < 4 else r.randint(most // 2, most)
        if b == B - 1 and B >= 8 and case["op"] != "attend":      # one of a full batch has only the prompt that all share, or nothing
            lens[b] = S
        rows.append(n)
        par = [-1]
        for i in range(1, n):
            par.append(r.randint(max(0, (i - 1) // 3), i - 1) if case.get("tree") else i - 1)
        parents.append(par)
    G = case.get("groups", 1)
    return lens, rows, parents, [b * B // G for b in range(G + 1)]


def _masks(par, tree):
    m = []
    for i, p in enumerate(par):
        m.append((1 << i) | (m[p] if p >= 0 else 0) if tree else (1 << (i + 1)) - 1)
    return m


def _row_bytes(case):
    """Of one head's key, or value, of a token in the cache."""
    D, f = case["dim"], case["format"]
    return 2 * D if f == "none" else D * FORMATS[f][0] // 8 + D // BLOCK


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["logits"] == "f32" else 2) + case["rows"] * 28, "flops": 4 * n}
    lens, rows, parents, groups = _plan(case)
    R, H, Hk, D = sum(rows), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("norm", "write"):
        # the rows read, the queries and the cache's part written; read back, the latter again and 16 bits a value
        n = R * D * 2 * (2 * H + 2 * Hk) + R * Hk * 2 * _row_bytes(case)
        if case["op"] == "write":
            n += R * Hk * 2 * (_row_bytes(case) + 2 * D)
        return {"bytes": n, "flops": R * (H + Hk) * (case["rotary"] * 3 + (0 if case["norm"] == "none" else 4 * D))}
    S, G = case.get("shared", 0), case.get("groups", 1)
    tokens = G * S + sum(t - S + n for t, n in zip(lens, rows))
    seen = 0
    for t, n, par in zip(lens, rows, parents):
        seen += n * t + sum(bin(m).count("1") for m in _masks(par, case["tree"]))
    return {"bytes": tokens * Hk * 2 * _row_bytes(case) + R * H * D * 2 * 2, "flops": 4 * seen * H * D}


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


def _tables(case, lens, rows, groups, g):
    """Pages of every sequence, in random order; those that the shared prompt fills are the same within a group."""
    P, S = case["page"], case.get("shared", 0)
    need = [-(-(t + n) // P) for t, n in zip(lens, rows)]
    common = S // P
    leaders = {b: groups[i] for i in range(len(groups) - 1) for b in range(groups[i], groups[i + 1])}
    pages = sum(n - (common if leaders[b] != b else 0) for b, n in enumerate(need)) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        first = 0
        if leaders[b] != b:
            first = common
            table[b, :first] = table[leaders[b], :first]
        table[b, first:n] = order[at:at + n - first]
        at += n - first
    return pages, table, [(leaders[b], b) for b in range(len(lens)) if leaders[b] != b and S % P]


def _fill(case, pages, g):
    """Keys or values of every slot as the cache holds them: [pages][page][heads][dim], or codes and scales of such, a head's
    tokens of a page side by side."""
    P, Hk, D, f = case["page"], case["kv_heads"], case["dim"], case["format"]
    dt = DTYPES[case["dtype"]]
    if f == "none":
        return torch.empty((pages, P, Hk, D), dtype=dt, device="cuda").normal_(generator=g), None
    bits = FORMATS[f][0]
    codes = torch.empty((pages, Hk, P, D * bits // 8), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, Hk, P, D // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (P * Hk * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        codes[i:i + n], scales[i:i + n] = quantise(torch.empty((n, Hk, P, D), device="cuda").normal_(generator=g), f, case["dtype"])
    return codes.permute(0, 2, 1, 3), scales.permute(0, 2, 1, 3)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, seed, g)
    lens, rows, parents, groups = _plan(case)
    starts = _starts(rows)
    R, B, N = starts[-1], len(rows), max(rows)
    s = {"case": case, "most_len": max(lens), "N": N, "R": R, "row_start": _ints(starts), "len": _ints(lens)}
    # for the plain forms: the row of (sequence, i), and of each row its sequence and i
    s["grid"] = torch.tensor([[starts[b] + min(i, rows[b] - 1) for i in range(N)] for b in range(B)]).cuda()
    s["valid"] = torch.tensor([[i < rows[b] for i in range(N)] for b in range(B)]).cuda()
    s["row_seq"] = torch.tensor([b for b in range(B) for _ in range(rows[b])]).cuda()
    s["row_at"] = torch.tensor([i for b in range(B) for i in range(rows[b])]).cuda()
    dt = DTYPES[case["dtype"]]
    pages, s["table"], halves = _tables(case, lens, rows, groups, g)
    s["k"], s["ks"] = _fill(case, pages, g)
    s["v"], s["vs"] = _fill(case, pages, g)
    for a, b in halves:                    # the page that the prompt ends in: every sequence has its own copy
        at, n = case["shared"] // case["page"], case["shared"] % case["page"]
        for t in (s["k"], s["ks"], s["v"], s["vs"]):
            if t is not None:
                t[int(s["table"][b, at]), :n] = t[int(s["table"][a, at]), :n]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("norm", "write"):
        # one projection's output holds the queries, keys and values of a row side by side; some channels are large
        qkv = torch.empty((R, (H + 2 * Hk) * D), dtype=dt, device="cuda").normal_(generator=g)
        qkv *= (1 + 4 * (torch.rand((H + 2 * Hk) * D, device="cuda", generator=g) < 0.02)).to(dt)
        s["q"], s["kn"], s["vn"] = qkv[:, :H * D], qkv[:, H * D:(H + Hk) * D], qkv[:, (H + Hk) * D:]
        j = torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda")
        s["freqs"] = 10000.0 ** (-2.0 * j / case["rotary"])
        s["pos"] = _ints([t + i for t, n in zip(lens, rows) for i in range(n)])
        s["qw"] = s["kw"] = None
        if case["norm"] != "none":
            each = case["norm"] == "each"
            s["qw"], s["kw"] = ((1 + 0.2 * torch.empty((h, D) if each else (D,), device="cuda").normal_(generator=g)).to(dt)
                                for h in (H, Hk))
        s["q_out"] = torch.zeros((R, H * D), dtype=dt, device="cuda")
        return s
    s["q"] = torch.empty((R, H * D), dtype=dt, device="cuda").normal_(0, 2, generator=g)      # some tokens stand out
    s["mask"] = _ints([_signed(m) for par in parents for m in _masks(par, case["tree"])], torch.int64)
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.zeros((R, H * D), dtype=dt, device="cuda")
    if case["op"] == "shared":
        s["group_start"] = _ints(groups)
        s["shared"] = _ints([case["shared"]] * case["groups"])
    return s


def _prepare_sample(case, seed, g):
    R, V = case["rows"], case["vocab"]
    r = random.Random(seed)
    z = torch.empty((R, V), device="cuda").normal_(0, 2.5, generator=g)
    s = {"case": case, "logits": z.to(DTYPES[case["logits"]]), "u": torch.rand(R, device="cuda", generator=g)}
    # requests differ: temperatures, and where a cut is asked for, some without it
    s["temperature"] = _ints([0.0 if R > 3 and i % 9 == 4 else round(r.uniform(0.5, 1.3), 3) for i in range(R)], torch.float32)
    s["top_k"] = _ints([case["top_k"] if R < 4 or i % 5 else 0 for i in range(R)]) if case["top_k"] else None
    s["top_p"] = _ints([case["top_p"] if R < 4 or i % 7 else 1.0 for i in range(R)], torch.float32) if case["top_p"] < 1 else None
    s["min_p"] = _ints([case["min_p"] if R < 4 or i % 4 else 0.0 for i in range(R)], torch.float32) if case["min_p"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_write, "write": _plain_write, "attend": _plain_attend, "shared": _plain_attend,
            "sample": _plain_sample}[s["case"]["op"]](s)


def _run_own(s):
    op = s["case"]["op"]
    h = s.get("handle")
    if h is None:                          # what a program sets up once: the cache's descriptor, weights, workspaces
        h = s["handle"] = _handle(s)
    if op == "sample":
        tokens, logprobs = h.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                    min_p=s["min_p"])
        return {"tokens": tokens, "logprobs": logprobs}
    if op in ("norm", "write"):
        cache, rope, norm = h
        cache.append(rope, s["q"], s["kn"], s["vn"], s["row_start"], positions=s["pos"], out=s["q_out"], norm=norm)
        if op == "norm":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        k, v = cache.read(s["row_start"], s["R"])
        return {"q": s["q_out"], "k": k, "v": v}
    cache, shared = h
    cache.attend(s["q"], s["row_start"], mask=s["mask"], scale=s["scale"], out=s["out"], shared=shared)
    return {"out": s["out"]}


def _handle(s):
    from latent_mixture_experts_bf16_amd import drafted, serving
    c = s["case"]
    if c["op"] == "sample":
        return serving.Sampler(c["vocab"], max_rows=c["rows"])
    if c["format"] == "none":
        cache = drafted.PagedCache(s["k"], s["v"], s["table"], s["len"])
    else:
        cache = serving.MxCache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"], format=c["format"],
                                dtype=DTYPES[c["dtype"]])
    if c["op"] in ("norm", "write"):
        return (cache, drafted.Rope(s["freqs"], layout=c["layout"]),
                None if s["qw"] is None else serving.HeadNorm(s["qw"], s["kw"], eps=EPS))
    return cache, serving.SharedPrefix(s["group_start"], s["shared"]) if c["op"] == "shared" else None


# ------------------------------------------------------------------ the plain forms

def _two(e):
    """2^e of whole numbers from -126 to 127, fp32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def quantise(x, format, dtype):
    """Codes and scale bytes of x [..., dim] (fp32): blocks of 32 under the smallest power of two (2^-126 at least) that leaves no
    value above the code's largest; a byte e stands for 2^(e - 127). In f16 what the cache stands for stays finite there."""
    bits, top, _, _ = FORMATS[format]
    y = x.unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True))
    tm, te = math.frexp(top)
    e = torch.where(m > tm, e - te + 1, e - te).clamp(min=-126)
    e = torch.where(m == 0, -126, e)
    if dtype == "f16":
        e = e.clamp(max=16 - te)
    y = (y * _two(-e)).clamp(-top, top)
    if bits == 8:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:
        a = y.abs()
        n = sum((a >= t if even else a > t).to(torch.uint8)     # a tie goes to the code that is even
                for t, even in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)))
        n = (n + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2).unflatten(-1, (-1, 2))
        codes = n[..., 0] + 16 * n[..., 1]
    return codes, (e.squeeze(-1) + 127).to(torch.uint8)


def stands_for(codes, scales, format):
    """The values of codes and scale bytes, fp32."""
    if FORMATS[format][0] == 8:
        x = codes.contiguous().view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        x = table[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, BLOCK)) * _two(scales.int().unsqueeze(-1) - 127)).flatten(-2)


def _slots(s, b, token):
    """Page and slot of tokens `token` of sequences `b`."""
    P = s["case"]["page"]
    return s["table"][b, token // P].long(), token % P


def _held(s, name, page, slot):
    """Keys or values of those slots, fp32 [..., heads, dim]."""
    x = s[name][page, slot]
    return x.float() if s["case"]["format"] == "none" else stands_for(x, s[name + "s"][page, slot], s["case"]["format"])


def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _turn(x, cos, sin, layout, rd):
    r = x[..., :rd]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rd // 2], r[..., rd // 2:])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([ya, yb], dim=-1).flatten(-2) if layout == "interleaved" else torch.cat([ya, yb], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_write(s):
    c = s["case"]
    H, Hk, D, rd, R, f = c["heads"], c["kv_heads"], c["dim"], c["rotary"], s["R"], c["format"]
    angle = s["pos"].double()[:, None, None] * s["freqs"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _turn(_normed(s["q"].float().reshape(R, H, D), s["qw"]), cos, sin, c["layout"], rd)
    k = _turn(_normed(s["kn"].float().reshape(R, Hk, D), s["kw"]), cos, sin, c["layout"], rd)
    v = s["vn"].float().reshape(R, Hk, D)
    s["q_out"][:] = q.reshape(R, H * D).to(s["q"].dtype)
    page, slot = _slots(s, s["row_seq"], s["len"].long()[s["row_seq"]] + s["row_at"])
    for name, x in (("k", k), ("v", v)):
        if f == "none":
            s[name][page, slot] = x.to(s[name].dtype)
        else:
            s[name][page, slot], s[name + "s"][page, slot] = quantise(x, f, c["dtype"])
    if c["op"] == "norm":
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    k, v = (_held(s, name, page, slot).reshape(R, Hk * D).to(s["q"].dtype) for name in ("k", "v"))
    return {"q": s["q_out"], "k": k, "v": v}


def _plain_attend(s):
    c = s["case"]
    H, Hk, D, R, N, B = c["heads"], c["kv_heads"], c["dim"], s["R"], s["N"], c["seqs"]
    G, L = H // Hk, s["most_len"] + N
    ln = s["len"].long()
    last = (ln + s["valid"].sum(1) - 1).clamp(min=0)
    t = torch.arange(L, device="cuda")
    page, slot = _slots(s, torch.arange(B, device="cuda")[:, None], torch.minimum(t, last[:, None]))
    q = s["q"][s["grid"]].float().reshape(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * G, D)
    k = _held(s, "k", page, slot).permute(0, 2, 3, 1).contiguous()
    sc = torch.matmul(q, k) * s["scale"]
    del k
    j = (t[None] - ln[:, None])[:, None]                       # [B,1,L]: the row's number among the step's
    bits = (s["mask"][s["grid"]][:, :, None] >> j.clamp(0, 63)) & 1
    see = (j < 0) | ((j < 64) & (bits == 1))                   # [B,N,L]
    see = see[:, None, :, None, :].expand(B, Hk, N, G, L).reshape(B, Hk, N * G, L)
    sc = torch.where(see, sc, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    del sc, see
    p = p / p.sum(-1, keepdim=True)
    v = _held(s, "v", page, slot).permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(p, v).reshape(B, Hk, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * D)
    s["out"][:] = o[s["row_seq"], s["row_at"]].to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_sample(s):
    # in 64 bits: whole tokens come out, and a draw may lie next to the border of two
    z, T, u = s["logits"].double(), s["temperature"].double(), s["u"].double()
    V = z.shape[1]
    greedy = T <= 0
    z, order = torch.sort(z, dim=1, descending=True, stable=True)      # equal ones: the lowest index first
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, T)[:, None])
    mass = w.cumsum(1)
    at = torch.arange(V, device=z.device)
    k = torch.full_like(at[:1], V).expand(len(u))
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"].long(), V).clamp(max=V)
    k = torch.where(greedy, 1, k)
    n = k
    if s["top_p"] is not None:
        p = s["top_p"].double()
        short = (mass < p[:, None] * mass.gather(1, k[:, None] - 1)).sum(1) + 1
        n = torch.where(p < 1, torch.minimum(n, short), n)
    if s["min_p"] is not None:
        n = torch.minimum(n, (w >= s["min_p"].double().clamp(max=1)[:, None]).sum(1))
    kept = mass.gather(1, n[:, None] - 1)
    i = torch.minimum((mass <= u[:, None] * kept).sum(1), n - 1)[:, None]
    logp = (w.gather(1, i) / mass[:, -1:]).log()[:, 0]
    return {"tokens": order.gather(1, i)[:, 0].int(), "logprobs": torch.where(greedy, 0.0, logp).float()}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    lens, rows, parents, groups = _plan(case)
    return (_exact_write if case["op"] in ("norm", "write") else _exact_attend)(case, s, lens, rows, parents, _starts(rows))


def _places(s, case, b, tokens):
    table = s["table"][b].tolist()
    return torch.tensor([(table[t // case["page"]], t % case["page"]) for t in tokens], device="cuda").T


def _nearest(x, case):
    """x [..., dim] in 64 bits as the cache's format holds it."""
    if case["format"] == "none":
        return x
    _, top, low, frac = FORMATS[case["format"]]
    y = x.reshape(*x.shape[:-1], -1, BLOCK)
    big = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(big.clamp(min=1e-300) / top)).clamp(-126, 7 if top > 6 else 13) if case["dtype"] == "f16" else \
        torch.ceil(torch.log2(big.clamp(min=1e-300) / top)).clamp(min=-126)
    unit = torch.exp2(e)
    y = (y / unit).clamp(-top, top)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1e-300))).clamp(min=low) - frac)
    return (torch.round(y / step) * step * unit).reshape(x.shape)


def _exact_write(case, s, lens, rows, parents, starts):
    H, Hk, D, rd, R = case["heads"], case["kv_heads"], case["dim"], case["rotary"], s["R"]
    turn = torch.polar(torch.ones((R, 1, rd // 2), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None, None] * s["freqs"])

    def spin(x, heads, w):
        x = x.double().reshape(R, heads, D).clone()
        if w is not None:
            x = w.double() * x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        r = x[..., :rd]
        pair = torch.view_as_complex(r.reshape(R, heads, rd // 2, 2).contiguous() if case["layout"] == "interleaved"
                                     else r.reshape(R, heads, 2, rd // 2).transpose(-1, -2).contiguous())
        y = torch.view_as_real(pair * turn)
        return torch.cat([(y if case["layout"] == "interleaved" else y.transpose(-1, -2)).reshape(R, heads, rd), x[..., rd:]], -1)

    q = spin(s["q"], H, s["qw"]).reshape(R, H * D)
    kn, vn = _nearest(spin(s["kn"], Hk, s["kw"]), case), _nearest(s["vn"].double().reshape(R, Hk, D), case)
    if case["op"] == "write":
        return {"q": q, "k": kn.reshape(R, Hk * D), "v": vn.reshape(R, Hk * D)}
    k, v = s["k"].double(), s["v"].double()
    for b, (t, n) in enumerate(zip(lens, rows)):
        page, slot = _places(s, case, b, range(t, t + n))
        k[page, slot] = kn[starts[b]:starts[b] + n]
        v[page, slot] = vn[starts[b]:starts[b] + n]
    return {"q": q, "k": k, "v": v}


def _meant(s, case, name, page, slot, h):
    """Keys or values of one head at those slots, in 64 bits, from the formats' bits."""
    x = s[name][page, slot, h]
    if case["format"] == "none":
        return x.double()
    bits, _, low, frac = FORMATS[case["format"]]
    c = x.long()
    if bits == 4:
        c = torch.stack([c % 16, c // 16], dim=-1).reshape(c.shape[0], -1)
    sign, mag = c >> (bits - 1), c & ((1 << (bits - 1)) - 1)
    e, m = mag >> frac, (mag & ((1 << frac) - 1)).double() / (1 << frac)
    val = torch.where(e == 0, m * 2.0 ** low, (1 + m) * torch.exp2((e - 1 + low).double())) * (1 - 2 * sign)
    unit = torch.exp2(s[name + "s"][page, slot, h].double() - 127)
    return val * unit.repeat_interleave(BLOCK, dim=-1)


def _exact_attend(case, s, lens, rows, parents, starts):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    out = torch.zeros((s["R"], H, D), dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(lens, rows)):
        page, slot = _places(s, case, b, range(t + n))
        see = torch.ones((n, t + n), dtype=torch.bool)
        for i, m in enumerate(_masks(parents[b], case["tree"])):
            see[i, t:] = torch.tensor([bool(m >> j & 1) for j in range(n)])
        see = see.cuda()
        for h in range(Hk):
            k, v = _meant(s, case, "k", page, slot, h), _meant(s, case, "v", page, slot, h)
            for g in range(G):
                q = s["q"][starts[b]:starts[b] + n].double().reshape(n, H, D)[:, h * G + g]
                w = torch.softmax((q @ k.T * s["scale"]).masked_fill(~see, -math.inf), dim=1)
                out[starts[b]:starts[b] + n, h * G + g] = w @ v
    return {"out": out.reshape(s["R"], H * D)}


def _exact_sample(case, s):
    tokens, logp = [], []
    Z, U, T = s["logits"].double().cpu().numpy(), s["u"].tolist(), s["temperature"].tolist()
    cut = {name: [None] * len(U) if s[name] is None else s[name].tolist() for name in ("top_k", "top_p", "min_p")}
    for i, z in enumerate(Z):
        if T[i] <= 0:
            tokens.append(int(z.argmax()))
            logp.append(0.0)
            continue
        p = np.exp((z - z.max()) / T[i])
        p /= p.sum()
        order = np.lexsort((np.arange(len(z)), -z))
        if cut["top_k"][i]:
            order = order[:cut["top_k"][i]]
        left = np.ones(len(order), dtype=bool)
        if cut["top_p"][i] is not None and cut["top_p"][i] < 1:
            before = np.concatenate([[0.0], np.cumsum(p[order])])
            left &= before[:-1] < cut["top_p"][i] * before[-1]
        if cut["min_p"][i]:
            left &= p[order] / p.max() >= cut["min_p"][i]
        order = order[left]
        run = np.cumsum(p[order])
        x = order[min(int(np.searchsorted(run, U[i] * run[-1], side="right")), len(order) - 1)]
        tokens.append(int(x))
        logp.append(float(np.log(p[x])))
    return {"tokens": _ints(tokens), "logprobs": _ints(logp, torch.float64)}
