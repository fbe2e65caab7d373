"""The served batch's operators on the GPU against their definitions in 64 bits.

Tolerances, derived from the arithmetic that include/moe_serving.h states (eps is the type's
torch.finfo(t).eps; rounding to it is off by eps / 2 of the value, or half the smallest subnormal):

append   a head's sum of squares rounds at most 13 times (8 fused steps, 5 joins), its root halves that; the mean, eps, root and
         quotient round 4 times, the products with them 3 times; cosine and sine are within 4 units in the last place after the
         angle's rest is turned in, and round twice with the magnitude; the rotation's product and fused sum round twice: fewer than
         24 roundings of 2^-24, of the pair's length after the norm. One rounding to the type. Codes: half a step of the
         code (2^-4 or 2^-2 of a value, half the least step of the block below its smallest normal code); the block's power is the least
         that holds its largest value, with the 24 roundings at the border.
read     bit for bit; what codes stand for is exact in both types for the scales used here.
attend   as in test_gpu_drafted.py, on the values that the codes stand for; a shared prompt's sums are joined once more.
sample   whole tokens equal; log p to fp32.
"""
import numpy as np
import pytest
import torch

from latent_mixture_experts_bf16_amd import binding as B
from latent_mixture_experts_bf16_amd import drafted as D
from latent_mixture_experts_bf16_amd import serving as S
from test_gpu_drafted import TINY, TYPES, Paged, _attend_check, _gen, _i32, _starts, _trees

pytestmark = pytest.mark.gpu

FOURS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
EIGHTS = torch.tensor([(-1) ** (c >> 7) * (float("nan") if c & 127 == 127 else (c & 7) * 2.0 ** -9 if not c & 120 else
                                           (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) for c in range(256)], dtype=torch.float64)
LARGEST = {"mx8": 448.0, "mx4": 6.0}
HALF_STEP = {"mx8": (2.0 ** -4, 2.0 ** -10), "mx4": (2.0 ** -2, 0.25)}      # of a value; of the block's power


def _means(codes, scales, format):
    """What codes and scale bytes stand for, in 64 bits (host tensors)."""
    if format == "mx8":
        x = EIGHTS[codes.long()]
    else:
        x = FOURS[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    unit = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return x * unit.repeat_interleave(32, -1)


class Mx(Paged):
    """A cache of codes over random bytes: k and v are what they stand for, in the rows' type."""

    def __init__(self, lens, rows, heads, dim, page, dtype, seed, format="mx8", heads_first=True):
        super().__init__(lens, rows, heads, dim, page, dtype, seed)
        g = _gen(seed + 100)
        self.format, pages = format, self.k.shape[0]
        wide = dim if format == "mx8" else dim // 2

        def raw(width, lo, hi):
            shape = (pages, heads, page, width) if heads_first else (pages, page, heads, width)
            t = torch.randint(lo, hi, shape, generator=g).to(torch.uint8)
            return t.cuda().transpose(1, 2) if heads_first else t.cuda()

        self.codes = [raw(wide, 0, 256) for _ in range(2)]
        if format == "mx8":
            for t in self.codes:       # values of about 1 under the scales below, no NaN
                t.copy_(torch.where((t & 127) > 119, t & 0x80, t))
        lo = 117 if format == "mx8" else 124
        self.scales = [raw(dim // 32, lo, lo + 4) for _ in range(2)]
        self.cache = S.MxCache(*self.codes, *self.scales, self.table, self.len, format=format, dtype=dtype)
        self.look()

    def look(self):
        self.k, self.v = (_means(c.cpu(), s.cpu(), self.format).to(self.k.dtype).cuda() for c, s in zip(self.codes, self.scales))


def _cache(kind, *a, **k):
    return Paged(*a, **k) if kind == "none" else Mx(*a, format=kind, **k)


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("format", ["mx8", "mx4"])
def test_every_code_is_read_as_what_it_stands_for(dtype, format):
    """All 256 bytes under every scale whose values the type holds exactly, and under the NaN scale."""
    dt, dim, page = TYPES[dtype], 256, 16
    wide = dim if format == "mx8" else 128
    low, high = (20, 240) if dtype == "bf16" else (112, 134) if format == "mx8" else (104, 140)
    scales = list(range(low, high + 1)) + [255]
    pages = -(-len(scales) // page)
    P = Mx([0], [pages * page], 1, dim, page, dt, seed=1, format=format)
    table = P.table_host[0]
    for i in range(pages * page):
        at = (int(table[i // page]), i % page, 0)
        for c, s in zip(P.codes, P.scales):
            c[at] = torch.arange(wide, dtype=torch.uint8) + (128 if format == "mx4" and i % 2 else 0)
            s[at] = scales[min(i, len(scales) - 1)]
    P.look()
    k, v = P.cache.read(_i32([0, pages * page]), pages * page)
    P.cache.status()
    for got, want in ((k, P.k), (v, P.v)):
        want = torch.stack([want[int(table[i // page]), i % page, 0] for i in range(pages * page)])
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    if format == "mx4":
        assert torch.isnan(k[-1]).all()


CASES = [
    # heads, kv_heads, dim, rotary, lens, rows, page, far, pad, norm
    (4, 2, 64, 64, [5], [1], 16, 0, 0, "shared"),
    (8, 2, 128, 64, [0, 15, 33], [3, 1, 17], 16, 100000, 8, "each"),
    (3, 1, 96, 24, [31, 0, 7], [2, 0, 9], 32, 900000, 4, "none"),       # an empty sequence
    (5, 5, 192, 192, [100, 1], [40, 5], 48, 30000, 2, "shared"),        # pages of 48
    (2, 2, 256, 128, [63], [66], 64, 0, 0, "each"),
    (2, 1, 32, 6, [3, 3], [2, 2], 16, 12345, 1, "shared"),              # three pairs, rows aligned to 2 bytes
    (40, 8, 128, 20, [9] * 70, [1] * 70, 16, 0, 0, "each"),             # ten pairs of a head, many sequences
]


def _rows_of(P, heads, kv_heads, dim, rotary, lens, rows, far, pad, norm, layout, seed=3):
    """Inputs of an append, the rope, the norm, and in 64 bits what rows become, with the 24 roundings' bound."""
    dt, R, g = P.k.dtype, sum(rows), _gen(seed)
    width = (heads + 2 * kv_heads) * dim + pad
    qkv = torch.randn((R, width), generator=g).to(dt).cuda()
    q, k, v = (qkv[:, a * dim:b * dim] for a, b in ((0, heads), (heads, heads + kv_heads), (heads + kv_heads, heads + 2 * kv_heads)))
    freqs, mag = D.rope_frequencies(rotary, scaling="parts", factor=8.0)
    w = hn = None
    if norm != "none":
        w = [(0.3 * torch.randn((n, dim) if norm == "each" else (dim,), generator=g)).to(dt).cuda() for n in (heads, kv_heads)]
        hn = S.HeadNorm(*w, eps=1e-5, offset=1.0)
    seq = [b for b, n in enumerate(rows) for _ in range(n)]
    at = [i for n in rows for i in range(n)]
    pos = None if not far else [far + lens[b] + i // 2 for b, i in zip(seq, at)]
    t = torch.tensor(pos if pos else [lens[b] + i for b, i in zip(seq, at)], dtype=torch.float64)
    angle = t[:, None, None] * freqs
    h = rotary // 2
    ia = torch.arange(0, rotary, 2) if layout == "interleaved" else torch.arange(h)
    ib = ia + 1 if layout == "interleaved" else ia + h

    def turn(x, n, w):
        x = x.double().cpu().reshape(R, n, dim)
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + float(np.float32(1e-5))).sqrt() * (1 + w.double().cpu())
        y, size = x.clone(), x.abs()
        a, b = x[..., ia], x[..., ib]
        m = float(np.float32(mag))
        y[..., ia], y[..., ib] = m * (a * angle.cos() - b * angle.sin()), m * (a * angle.sin() + b * angle.cos())
        size[..., ia] = size[..., ib] = m * (a * a + b * b).sqrt()
        return y, 24 * 2.0 ** -24 * size

    want = dict(q=turn(q, heads, w and w[0]), k=turn(k, kv_heads, w and w[1]),
                v=(v.double().cpu().reshape(R, kv_heads, dim), torch.zeros(R, kv_heads, dim, dtype=torch.float64)))
    return qkv, q, k, v, D.Rope(freqs, mag, layout), hn, None if pos is None else _i32(pos), seq, at, want


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary,lens,rows,page,far,pad,norm", [c for c in CASES if c[-1] != "none"] + [
    (3, 1, 80, 20, [31, 0, 7], [2, 0, 9], 32, 900000, 4, "each"), (2, 1, 112, 112, [1], [5], 16, 0, 0, "shared")])
def test_normed_append(dtype, layout, heads, kv_heads, dim, rotary, lens, rows, page, far, pad, norm):
    dt = TYPES[dtype]
    pad += layout == "interleaved" and pad % 2
    P = Paged(lens, rows, kv_heads, dim, page, dt, seed=dim + rotary)
    qkv, q, k, v, rope, hn, pos, seq, at, want = _rows_of(P, heads, kv_heads, dim, rotary, lens, rows, far, pad, norm, layout)
    starts, before, k0, v0 = _i32(_starts(rows)), qkv.clone(), P.k.clone(), P.v.clone()
    out = P.cache.append(rope, q, k, v, starts, positions=pos, norm=hn)
    P.cache.status()
    assert torch.equal(qkv, before) and torch.equal(P.len, _i32(lens))

    def near(got, y, tol):
        return ((got.double().cpu().reshape(y.shape) - y).abs() <= tol + torch.finfo(dt).eps / 2 * (y.abs() + tol) + TINY[dt]).all()

    assert near(out, *want["q"])
    for r, (b, i) in enumerate(zip(seq, at)):
        place = P.place(b, lens[b] + i)
        assert near(P.k[place], want["k"][0][r], want["k"][1][r]), r
        assert torch.equal(P.v[place], v[r].reshape(kv_heads, dim)), r
        k0[place], v0[place] = P.k[place], P.v[place]
    assert torch.equal(P.k, k0) and torch.equal(P.v, v0)      # nothing else was written
    assert P.cache.append(rope, q, k, v, starts, positions=pos, norm=hn, out=q) is q
    assert torch.equal(q, out) and torch.equal(P.k, k0) and torch.equal(qkv[:, heads * dim:], before[:, heads * dim:])


@pytest.mark.parametrize("format", ["mx8", "mx4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary,lens,rows,page,far,pad,norm", CASES)
def test_append_of_codes(format, dtype, layout, heads, kv_heads, dim, rotary, lens, rows, page, far, pad, norm):
    dt = TYPES[dtype]
    pad += layout == "interleaved" and pad % 2
    P = Mx(lens, rows, kv_heads, dim, page, dt, seed=dim + rotary, format=format, heads_first=page != 48)
    qkv, q, k, v, rope, hn, pos, seq, at, want = _rows_of(P, heads, kv_heads, dim, rotary, lens, rows, far, pad, norm, layout)
    starts, before = _i32(_starts(rows)), qkv.clone()
    held = [t.clone() for t in P.codes + P.scales]
    out = P.cache.append(rope, q, k, v, starts, positions=pos, norm=hn)
    P.cache.status()
    assert torch.equal(qkv, before) and torch.equal(P.len, _i32(lens))
    y, tol = want["q"]
    assert ((out.double().cpu().reshape(y.shape) - y).abs() <= tol + torch.finfo(dt).eps / 2 * (y.abs() + tol) + TINY[dt]).all()
    most, (half, least) = LARGEST[format], HALF_STEP[format]
    kr, vr = P.cache.read(starts, sum(rows))
    for j, (name, back) in enumerate((("k", kr), ("v", vr))):
        y, tol = want[name]
        for r, (b, i) in enumerate(zip(seq, at)):
            place = P.place(b, lens[b] + i)
            codes, scales = P.codes[j][place].cpu(), P.scales[j][place].cpu()
            got, unit = _means(codes, scales, format), torch.exp2(scales.double() - 127)
            top = y[r].reshape(kv_heads, -1, 32).abs().amax(-1)
            off = tol[r].reshape(kv_heads, -1, 32).amax(-1)
            assert (top - off <= most * unit).all() and (top + off > most * unit / 2).all(), (name, r)
            unit = unit.repeat_interleave(32, -1)
            far_ = (got - y[r]).abs() - tol[r] - torch.maximum(half * (y[r].abs() + tol[r]), least * unit)
            assert (far_ <= 0).all(), (name, r, float(far_.max()))
            assert torch.equal(back[r].cpu().double().reshape(kv_heads, dim), got), (name, r)
            held[j][place], held[2 + j][place] = P.codes[j][place], P.scales[j][place]
    for a, b in zip(P.codes + P.scales, held):
        assert torch.equal(a, b)      # nothing else was written
    assert P.cache.append(rope, q, k, v, starts, positions=pos, norm=hn, out=q) is q
    assert torch.equal(q, out)
    for a, b in zip(P.codes + P.scales, held):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("format", ["mx8", "mx4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,rows,width", [
    (4, 1, 64, 16, [0], [1], None),                     # the first token of all
    (8, 2, 128, 64, [777], [1], None),
    (2, 2, 96, 16, [15, 16, 17, 31, 32, 33], [1] * 6, None),
    (10, 2, 128, 32, [300, 0, 129], [5, 3, 7], None),   # chains; one sequence with nothing cached
    (8, 2, 128, 64, [200, 1000, 64], [16, 13, 1], 3),
    (8, 1, 64, 16, [500, 40], [64, 33], 3),             # the widest trees: 512 rows of one key head
    (6, 2, 96, 48, [95, 47, 48], [2, 17, 0], 2),        # pages of 48, a sequence without rows
    (2, 2, 256, 128, [129, 5], [9, 3], 2),
    (4, 4, 192, 16, [70], [4], 2),
    (4, 2, 32, 32, [70, 71], [4, 21], 2),
    (71, 1, 64, 256, [1025], [3], None),                # 71 query heads on one key head
    (4, 2, 64, 16, [40], [150], None),                  # a prompt's rows behind a cache
    (4, 4, 128, 64, [4000, 100], [2, 1], None),         # split along the tokens
])
def test_attend_over_codes(format, dtype, heads, kv_heads, dim, page, lens, rows, width):
    P = Mx(lens, rows, kv_heads, dim, page, TYPES[dtype], seed=dim + page, format=format, heads_first=page != 48)
    _attend_check(P, heads, None if width is None else _trees(rows, width, 5), pad=8 * (dim == 128))


class Shares:
    """A cache whose `attend` computes the groups' common tokens once, for _attend_check."""

    def __init__(self, P, groups, lengths):
        self.P, self.shared = P, S.SharedPrefix(_i32(groups), _i32(lengths))
        self.real, P.cache = P.cache, self

    def attend(self, *a, **k):
        return self.real.attend(*a, shared=self.shared, **k)

    def status(self):
        self.real.status()


def _share(P, groups, lengths):
    """The first lengths[g] tokens of group g's sequences the same: the pages they fill, and copies of the rest."""
    for g, n in enumerate(lengths):
        a = groups[g]
        for b in range(a + 1, groups[g + 1]):
            full = n // P.page
            P.table_host[b, :full] = P.table_host[a, :full]
            for t in range(full * P.page, n):
                for x in ([P.k, P.v] if not isinstance(P, Mx) else P.codes + P.scales):
                    x[P.place(b, t)] = x[P.place(a, t)]
    P.table.copy_(P.table_host[:, :P.table.shape[1]])
    if isinstance(P, Mx):
        P.look()
    return Shares(P, groups, lengths)


@pytest.mark.parametrize("format", ["none", "mx8", "mx4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,rows,width,groups,lengths", [
    (4, 1, 64, 16, [70], [1], None, [0, 1], [64]),                              # one sequence, one tile
    (8, 2, 128, 64, [640, 645, 640, 900], [1] * 4, None, [0, 4], [640]),        # the prompt ends where a page does
    (8, 2, 128, 64, [333, 400, 333], [1, 3, 2], None, [0, 3], [333]),           # and inside a page and a tile
    (4, 4, 96, 16, [63, 63], [1, 2], None, [0, 2], [63]),                       # too short to be shared
    (2, 2, 192, 32, [500, 130, 131, 7], [2, 1, 1, 1], 2, [0, 1, 3, 4], [200, 130, 0]),
    (4, 2, 64, 16, [300, 300, 290, 280, 280], [5, 0, 9, 1, 2], 2, [0, 3, 3, 5], [290, 5, 280]),   # an empty group
    (6, 1, 256, 128, [256, 257], [17, 30], 3, [0, 2], [256]),                   # tiles of 128 queries
    (71, 1, 64, 48, [1000, 1001, 1100], [1, 1, 2], None, [0, 3], [999]),
    (4, 2, 32, 16, [3000] * 12, [1] * 12, None, [0, 12], [2990]),               # split along the prompt
    (16, 8, 64, 16, [70 + b % 61 for b in range(700)], [1 + (b % 9 == 4) for b in range(700)], None,    # many items a workgroup,
     [0, 3, 400, 400, 640, 700], [64, 70, 0, 68, 0]),                                                   # a row's query a wave
])
def test_attend_after_a_shared_prompt(format, dtype, heads, kv_heads, dim, page, lens, rows, width, groups, lengths):
    P = _cache(format, lens, rows, kv_heads, dim, page, TYPES[dtype], seed=dim + page)
    plain = P.cache
    _share(P, groups, lengths)
    masks = None if width is None else _trees(rows, width, 5)
    got = _attend_check(P, heads, masks, pad=8 * (dim == 128))
    # near what the same call without sharing gives
    q = torch.randn((sum(rows), heads * dim + 8 * (dim == 128)), generator=_gen(11)).to(TYPES[dtype]).cuda()[:, :heads * dim]
    m = None if masks is None else torch.tensor(masks, dtype=torch.int64, device="cuda")
    want = plain.attend(q, _i32(_starts(rows)), mask=m)
    assert (got.float() - want.float()).norm() <= 2 * torch.finfo(TYPES[dtype]).eps * want.float().norm()


# ------------------------------------------------------------------ sampling

def _sample_ref(z, u, T, top_k, top_p, min_p):
    """Tokens, log p and the number of tokens left, in 64 bits, row by row (host arrays; NaN counts as -infinity)."""
    tokens, logp, left = [], [], []
    for i in range(len(z)):
        x = np.where(np.isnan(z[i]), -np.inf, z[i].astype(np.float64))
        order = np.lexsort((np.arange(len(x)), -x))
        order = order[x[order] > -np.inf]
        t = T[i] if T is not None else 1.0
        if not t > 0:
            tokens.append(int(order[0]))
            logp.append(0.0)
            left.append(1)
            continue
        top = x[order[0]]
        w = np.exp((x[order] - top) / t) if np.isfinite(top) else (x[order] == top).astype(np.float64)
        run, n = np.cumsum(w), len(order)
        k = top_k[i] if top_k is not None and top_k[i] > 0 else n
        n = k = min(n, k)
        if top_p is not None and top_p[i] < 1:
            n = min(n, int((run < top_p[i] * run[k - 1]).sum()) + 1)
        if min_p is not None and min_p[i] > 0:
            n = min(n, int((w >= min(min_p[i], 1.0)).sum()))
        j = min(int((run <= np.float64(u[i]) * run[n - 1]).sum()), n - 1)
        tokens.append(int(order[j]))
        logp.append(float(np.log(w[j] / run[-1])))
        left.append(n)
    return tokens, logp, left


def _sample_check(z, u, T=None, top_k=None, top_p=None, min_p=None, pad=0):
    dev = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    f32 = lambda v: None if v is None else [float(np.float32(x)) for x in v]  # noqa: E731
    rows, V = z.shape
    wide = torch.zeros((rows, V + pad), dtype=z.dtype, device="cuda")
    wide[:, :V] = z.cuda()
    s = S.Sampler(V, max_rows=rows)
    args = dict(temperature=dev(T, torch.float32), top_k=dev(top_k, torch.int32), top_p=dev(top_p, torch.float32),
                min_p=dev(min_p, torch.float32))
    tokens, logp = s.sample(wide[:, :V], dev(u, torch.float32), **args)
    s.status()
    want, lp, left = _sample_ref(z.float().numpy(), f32(u), f32(T), top_k, f32(top_p), f32(min_p))
    assert tokens.tolist() == want, [(i, a, b, left[i]) for i, (a, b) in enumerate(zip(tokens.tolist(), want)) if a != b][:5]
    assert np.allclose(logp.cpu().numpy(), lp, rtol=2.0 ** -22, atol=2.0 ** -22)
    again, lp2 = s.sample(wide[:, :V], dev(u, torch.float32), **args)
    assert torch.equal(again, tokens) and torch.equal(lp2, logp)
    return tokens, left


@pytest.mark.parametrize("logits", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,rows,pad", [(1, 2, 0), (2, 3, 1), (63, 5, 0), (1000, 9, 24), (4096, 4, 0), (4097, 4, 3), (32000, 6, 0),
                                        (100003, 5, 1), (131072, 8, 0), (1 << 20, 3, 0)])
def test_sample(logits, V, rows, pad):
    r = np.random.default_rng(V)
    z = (torch.randn((rows, V), generator=_gen(V)) * 2.5).to({"f32": torch.float32, **TYPES}[logits])
    u = r.random(rows).astype(np.float32)
    T = [[0.7, 1.0, 1.3, 0.0, 0.2][i % 5] for i in range(rows)]
    k = [[0, 1, 50, 700, V][(i + 1) % 5] for i in range(rows)]
    p = [[0.9, 1.0, 0.5, 0.999, 0.0][(i + 2) % 5] for i in range(rows)]
    m = [[0.0, 0.05, 0.3, 1.0][i % 4] for i in range(rows)]
    _sample_check(z, u, pad=pad)
    _sample_check(z, u, T=T, pad=pad)
    _sample_check(z, u, T=T, top_k=k)
    _sample_check(z, u, T=T, top_p=p)
    _sample_check(z, u, T=T, min_p=m)
    _sample_check(z, u, T=T, top_k=k, top_p=p, min_p=m)
