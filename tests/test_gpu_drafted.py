"""The drafted step's operators on the GPU against their definitions in 64 bits.

Tolerances, derived from the arithmetic that include/moe_drafted.h states (eps is the type's
torch.finfo(t).eps; rounding to it is off by eps / 2 of the value, or half the smallest subnormal):

append   the angle's fraction of a turn is rounded once to 32 bits (2 pi 2^-25 of angle), cosine and
         sine and the two products and their sum round a few times more: at most 6e-7 of
         magnitude * (|a| + |b|), then one rounding to the type. Values are copied bit for bit.
attend   with A = sum p |v| over what a row sees: probabilities round to the type (eps / 2 of A); scores
         are fp32 dot products of D terms (D 2^-24 of scale * sum |q k| at most, as a relative
         change of p, in numerator and sum); 2^-24 per token of the sums; f16 probabilities may be
         subnormal (2^-25 per token, against the largest |v|); one rounding of the result.
verify   whole tokens and paths equal; log p to fp32.
keep     bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from latent_mixture_experts_bf16_amd import binding as B
from latent_mixture_experts_bf16_amd import drafted as D

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half the smallest subnormal


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _starts(rows):
    return [0] + list(np.cumsum(rows))


def _tree(n, width, seed):
    r = np.random.default_rng(seed)
    return [-1] + [i - 1 if width == 1 else int(r.integers(max(0, (i - 1) // width), i)) for i in range(1, n)]


class Paged:
    """A cache with pages in random order, two pages that no sequence holds, and its host copies."""

    def __init__(self, lens, rows, heads, dim, page, dtype, seed, heads_first=False):
        g = _gen(seed)
        self.lens, self.rows, self.page, self.heads, self.dim = lens, rows, page, heads, dim
        need = [max(1, -(-(t + n) // page)) for t, n in zip(lens, rows)]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        # table rows lie in a wider table, entries past a sequence's pages name none
        table = torch.full((len(lens), max(need) + 3), -7, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([order.pop() for _ in range(n)])
        self.table_host = table
        shape = (pages, heads, page, dim) if heads_first else (pages, page, heads, dim)
        kv = [torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2)]
        self.k, self.v = [t.transpose(1, 2) if heads_first else t for t in kv]
        self.table = table.cuda()[:, :max(need) + 1]
        self.len = _i32(lens)
        self.cache = D.PagedCache(self.k, self.v, self.table, self.len)

    def place(self, b, t):
        return int(self.table_host[b, t // self.page]), t % self.page


# ------------------------------------------------------------------ rotary append

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary,lens,rows,page,far,pad", [
    (4, 2, 64, 64, [5], [1], 16, 0, 0),
    (8, 2, 128, 64, [0, 15, 33], [3, 1, 17], 16, 100000, 8),
    (3, 1, 80, 20, [31, 0, 7], [2, 0, 9], 32, 900000, 4),       # a quarter of an odd width; an empty sequence
    (5, 5, 96, 24, [100, 1], [40, 5], 48, 30000, 2),            # pages of 48
    (2, 2, 256, 256, [63], [66], 64, 0, 0),
    (2, 1, 32, 6, [3, 3], [2, 2], 16, 12345, 1),                # three pairs, rows aligned to 2 bytes
])
def test_append(dtype, layout, heads, kv_heads, dim, rotary, lens, rows, page, far, pad):
    dt = TYPES[dtype]
    if layout == "interleaved" and pad % 2:
        pad += 1
    P = Paged(lens, rows, kv_heads, dim, page, dt, seed=dim + rotary)
    R, starts = sum(rows), _starts(rows)
    g = _gen(3)
    width = (heads + 2 * kv_heads) * dim + pad
    qkv = torch.randn((R, width), generator=g).to(dt).cuda()
    q, k, v = qkv[:, :heads * dim], qkv[:, heads * dim:(heads + kv_heads) * dim], qkv[:, (heads + kv_heads) * dim:
                                                                                        (heads + 2 * kv_heads) * dim]
    freqs, mag = D.rope_frequencies(rotary, scaling="parts", factor=8.0)
    rope = D.Rope(freqs, mag, layout)
    seq = [b for b, n in enumerate(rows) for _ in range(n)]
    at = [i for n in rows for i in range(n)]
    pos = None if not far else [far + lens[b] + i // 2 for b, i in zip(seq, at)]
    before = qkv.clone()
    k0, v0 = P.k.clone(), P.v.clone()
    out = P.cache.append(rope, q, k, v, _i32(starts), positions=None if pos is None else _i32(pos))
    P.cache.status()
    assert torch.equal(qkv, before) and torch.equal(P.len, _i32(lens))

    t = torch.tensor(pos if pos else [lens[b] + i for b, i in zip(seq, at)], dtype=torch.float64)
    angle = t[:, None, None] * freqs
    h = rotary // 2
    ia = torch.arange(0, rotary, 2) if layout == "interleaved" else torch.arange(h)
    ib = ia + 1 if layout == "interleaved" else ia + h

    def turn(x, n):
        x = x.double().cpu().reshape(R, n, dim)
        y, near = x.clone(), torch.zeros_like(x)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = mag * (a * angle.cos() - b * angle.sin()), mag * (a * angle.sin() + b * angle.cos())
        d = 6e-7 * mag * (a.abs() + b.abs())
        near[..., ia] = near[..., ib] = d
        return y, near + (torch.finfo(dt).eps / 2 * (y.abs() + near) + TINY[dt]) * (near > 0)

    y, tol = turn(q, heads)
    assert ((out.double().cpu().reshape(R, heads, dim) - y).abs() <= tol).all()
    y, tol = turn(k, kv_heads)
    for r, (b, i) in enumerate(zip(seq, at)):
        page_, slot = P.place(b, lens[b] + i)
        assert ((P.k[page_, slot].double().cpu() - y[r]).abs() <= tol[r]).all(), r
        assert torch.equal(P.v[page_, slot], v[r].reshape(kv_heads, dim)), r
        k0[page_, slot], v0[page_, slot] = P.k[page_, slot], P.v[page_, slot]
    assert torch.equal(P.k, k0) and torch.equal(P.v, v0)      # nothing else was written
    # in place, beside the keys and values of the same rows: the same bits
    assert P.cache.append(rope, q, k, v, _i32(starts), positions=None if pos is None else _i32(pos), out=q) is q
    assert torch.equal(q, out) and torch.equal(P.k, k0) and torch.equal(qkv[:, heads * dim:], before[:, heads * dim:])


# ------------------------------------------------------------------ tree attention

def _see(lens, rows, masks):
    """Per sequence [n][len + n] of what each row sees; masks None: rows up to its own."""
    out, at = [], 0
    for t, n in zip(lens, rows):
        s = torch.zeros((n, t + n), dtype=torch.bool)
        s[:, :t] = True
        for i in range(n):
            for j in range(n):
                s[i, t + j] = j <= i if masks is None else j < 64 and bool(masks[at + i] >> j & 1)
        out.append(s)
        at += n
    return out


def _attend_ref(P, q, see, heads, scale):
    """The definition in 64 bits and the tolerance, [rows][heads][dim]; a row that sees nothing: 0."""
    dt, dim, hk = q.dtype, P.dim, P.heads
    eps, outs, tols, at = torch.finfo(dt).eps, [], [], 0
    K, V = P.k.double().cpu(), P.v.double().cpu()
    q = q.double().cpu().reshape(-1, heads, dim)
    for b, s in enumerate(see):
        n, T = s.shape
        if n == 0:
            continue
        where = [P.place(b, t) for t in range(T)]
        pg, sl = [w[0] for w in where], [w[1] for w in where]
        for i in range(n):
            ok = s[i].nonzero()[:, 0]
            o, tol = torch.zeros(heads, dim, dtype=torch.float64), torch.zeros(heads, dim, dtype=torch.float64)
            if len(ok):
                k = K[pg, sl][ok].repeat_interleave(heads // hk, 1)
                v = V[pg, sl][ok].repeat_interleave(heads // hk, 1)
                x = torch.einsum("hd,thd->ht", q[at + i], k) * scale
                p = torch.softmax(x, 1)
                o = torch.einsum("ht,thd->hd", p, v)
                A = torch.einsum("ht,thd->hd", p, v.abs())
                ds = (torch.einsum("hd,thd->ht", q[at + i].abs(), k.abs()).amax(1) * abs(scale) * (dim + 4) * 2.0 ** -24)
                tol = A * (eps / 2 + 2 * ds[:, None] + (len(ok) + 64) * 2.0 ** -24) + eps / 2 * o.abs() + TINY[dt]
                if dt == torch.float16:
                    tol = tol + len(ok) * 2.0 ** -25 * v.abs().amax(0)
            outs.append(o)
            tols.append(tol * (1 + eps))
        at += n
    return torch.stack(outs), torch.stack(tols)


def _attend_check(P, heads, masks, seed=11, scale=None, pad=0, q=None):
    dt = P.k.dtype
    R = sum(P.rows)
    if q is None:
        q = torch.randn((R, heads * P.dim + pad), generator=_gen(seed)).to(dt).cuda()[:, :heads * P.dim]
    out = torch.full((R, heads * P.dim + pad), 7.0, dtype=dt, device="cuda")
    m = None if masks is None else torch.tensor(masks, dtype=torch.int64, device="cuda")
    got = P.cache.attend(q, _i32(_starts(P.rows)), mask=m, scale=scale, out=out[:, :heads * P.dim])
    P.cache.status()
    assert (out[:, heads * P.dim:] == 7).all()
    y, tol = _attend_ref(P, q, _see(P.lens, P.rows, masks), heads, P.dim ** -0.5 if scale is None else scale)
    far = (got.double().cpu().reshape(y.shape) - y).abs() - tol
    assert (far <= 0).all(), float(far.max())
    again = P.cache.attend(q, _i32(_starts(P.rows)), mask=m, scale=scale)
    assert torch.equal(again, got)
    return got


def _trees(rows, width, seed):
    return [m for b, n in enumerate(rows) for m in D.tree_masks(_tree(n, width, seed + b))[:n]] if max(rows) else []


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,rows,width", [
    (4, 1, 64, 16, [0], [1], None),                     # the first token of all
    (4, 2, 64, 16, [1], [1], None),
    (8, 2, 128, 64, [777], [1], None),
    (2, 2, 96, 16, [15, 16, 17, 31, 32, 33], [1] * 6, None),
    (10, 2, 128, 32, [300, 0, 129], [5, 3, 7], None),   # chains; one sequence with nothing cached
    (8, 2, 128, 64, [200, 1000, 64], [16, 13, 1], 3),
    (8, 1, 64, 16, [500, 40], [64, 33], 3),             # the widest trees: 512 rows of one key head
    (6, 2, 80, 48, [95, 47, 48], [2, 17, 0], 2),        # pages of 48, a sequence without rows
    (2, 2, 256, 128, [129, 5], [9, 3], 2),
    (4, 4, 192, 16, [70], [4], 2),
    (4, 2, 112, 32, [70], [4], 2),
    (4, 2, 32, 32, [70, 71], [4, 21], 2),
    (71, 1, 64, 256, [1025], [3], None),                # 71 query heads on one key head
    (4, 2, 64, 16, [40], [150], None),                  # a prompt's rows behind a cache
    (4, 4, 128, 64, [4000, 100], [2, 1], None),         # split along the tokens
])
def test_attend(dtype, heads, kv_heads, dim, page, lens, rows, width):
    P = Paged(lens, rows, kv_heads, dim, page, TYPES[dtype], seed=dim + page)
    masks = None if width is None else _trees(rows, width, 5)
    _attend_check(P, heads, masks, pad=8 * (dim == 128))


def test_attend_heads_first_cache():
    P = Paged([75, 16], [3, 2], 4, 128, 32, torch.bfloat16, seed=1, heads_first=True)
    _attend_check(P, 8, None)


def test_attend_many_sequences():
    r = np.random.default_rng(2)
    lens = [int(v) for v in r.integers(0, 90, 130)]
    rows = [int(v) for v in r.integers(0, 4, 130)]
    P = Paged(lens, rows, 1, 64, 16, torch.float16, seed=4)
    _attend_check(P, 2, None)


def test_attend_odd_masks():
    """Rows that see nothing, only later rows, not themselves; bits past the sequence's rows."""
    P = Paged([0, 20, 0], [4, 5, 2], 2, 64, 16, torch.bfloat16, seed=5)
    masks = [0, 0b1100, 0b0001, -1, 0, 0b10000, -1, 1 << 62, 0b00110, 0, 0b11]
    got = _attend_check(P, 4, masks)
    assert (got[0] == 0).all() and (got[9] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_does_not_use_what_is_not_seen(dtype):
    """Infinities and NaN where nothing looks: unused pages, slots behind the last row, drafted rows
    outside a row's mask. Rows that do see them are NaN or infinite and spoil no other."""
    dt = TYPES[dtype]
    lens, rows = [37, 0], [20, 9]
    masks = _trees(rows, 2, 9)
    P = Paged(lens, rows, 2, 64, 16, dt, seed=6)
    q = torch.randn((29, 4 * 64), generator=_gen(1)).to(dt).cuda()
    want = _attend_check(P, 4, masks, q=q).clone()
    used = {P.place(b, t) for b in range(2) for t in range(lens[b] + rows[b])}
    for page in range(P.k.shape[0]):
        for slot in range(16):
            if (page, slot) not in used:
                P.k[page, slot] = float("nan")
                P.v[page, slot] = float("inf")
    got = P.cache.attend(q, _i32(_starts(rows)), mask=torch.tensor(masks, device="cuda"))
    assert torch.equal(got, want)
    for b, j, bad in ((0, 3, float("nan")), (1, 2, float("inf")), (0, 11, -float("inf"))):
        page, slot = P.place(b, lens[b] + j)
        keep = P.v[page, slot].clone(), P.k[page, slot].clone()
        P.v[page, slot] = bad
        P.k[page, slot] = float("nan") if j == 11 else keep[1]
        got = P.cache.attend(q, _i32(_starts(rows)), mask=torch.tensor(masks, device="cuda"))
        at = _starts(rows)[b]
        for r in range(29):
            sees = at <= r < at + rows[b] and masks[r] >> j & 1
            if sees:
                assert not torch.isfinite(got[r]).any(), (b, j, r)
            else:
                assert torch.equal(got[r], want[r]), (b, j, r)
        P.v[page, slot], P.k[page, slot] = keep
    # a row of queries that is NaN spoils no other row
    q[5] = float("nan")
    got = P.cache.attend(q, _i32(_starts(rows)), mask=torch.tensor(masks, device="cuda"))
    assert torch.isnan(got[5]).all()
    assert torch.equal(torch.cat([got[:5], got[6:]]), torch.cat([want[:5], want[6:]]))


def test_attend_far_scores():
    """Scores that grow along the cache by hundreds, and a scale that is not the default: the running
    maximum moves at nearly every tile, and what it leaves behind underflows to nothing."""
    P = Paged([700], [2], 1, 64, 16, torch.bfloat16, seed=8)
    q = torch.ones((2, 128), dtype=torch.bfloat16, device="cuda")
    q[:, 64:] = -1
    for t in range(702):
        page, slot = P.place(0, t)
        P.k[page, slot] = float(t % 128) / 8 if t < 350 else t / 16.0
    _attend_check(P, 2, None, q=q, scale=0.25)


def test_attend_on_another_stream_and_in_a_graph():
    P = Paged([400, 90], [4, 4], 2, 128, 64, torch.bfloat16, seed=12)
    q = torch.randn((8, 8 * 128), generator=_gen(1)).to(torch.bfloat16).cuda()
    starts, out = _i32([0, 4, 8]), torch.zeros((8, 8 * 128), dtype=torch.bfloat16, device="cuda")
    want = P.cache.attend(q, starts).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.cache.attend(q, starts, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.cache.attend(q, starts, out=out)
    for step in range(4):
        q.copy_(torch.randn((8, 8 * 128), generator=_gen(20 + step)).to(torch.bfloat16))
        P.len.copy_(_i32([400 - 7 * step, 90 - step]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, P.cache.attend(q, starts)), step


def test_bad_pages_and_lengths_are_reported_not_read():
    """Host-made bad values: each is caught by the kernels' own bounds, sets its bit and reads nothing."""
    P = Paged([40, 20], [2, 2], 1, 64, 16, torch.bfloat16, seed=3)
    q = torch.randn((4, 64), generator=_gen(1)).to(torch.bfloat16).cuda()
    starts = _i32([0, 2, 4])
    want = P.cache.attend(q, starts).clone()
    rope = D.Rope(D.rope_frequencies(64)[0])

    def met(text, f):
        f()
        with pytest.raises(B.MoeError, match=text) as e:
            P.cache.status()
        assert e.value.name == "MOE_ERR_DEVICE_CHECK"
        P.cache.status()      # cleared

    kept = P.table.clone()
    for bad in (-1, P.k.shape[0], 1 << 30):
        P.table[0, 1] = bad
        met("page", lambda: P.cache.attend(q, starts))
        P.table.copy_(kept)
        P.table[1, 1] = bad       # where sequence 1's new rows would go
        k0 = P.k.clone()
        met("page", lambda: P.cache.append(rope, q, q, q, starts))
        P.table.copy_(kept)
        same = torch.ones(P.k.shape[:2], dtype=torch.bool)
        for t in (40, 41):
            same[P.place(0, t)] = False
        assert torch.equal(P.k[same], k0[same])
        P.k.copy_(k0)
    for bad in (-3, 1 << 30, 2 ** 31 - 1):
        P.len.copy_(_i32([bad, 20]))
        met("length", lambda: P.cache.attend(q, starts))
        met("page|length", lambda: P.cache.append(rope, q, q, q, starts))
        P.len.copy_(_i32([40, 20]))
    for bad in ([0, 3, 2], [0, 2, 5], [-1, 2, 4], [0, 2, 3]):
        met("row_start", lambda: P.cache.attend(q, _i32(bad)))
    P2 = Paged([40, 20], [2, 2], 1, 64, 16, torch.bfloat16, seed=3)
    assert torch.equal(P2.cache.attend(q, starts), want)
    P2.cache.status()


# ------------------------------------------------------------------ path keeping

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv_heads,dim,page,lens,rows,in_place", [
    (2, 64, 16, [0], [1], True), (8, 128, 64, [777, 62, 0], [16, 5, 30], False), (3, 80, 16, [15, 16, 31], [40, 64, 0], True),
    (1, 256, 48, [100] * 5, [7, 20, 33, 64, 2], False)])
def test_keep(dtype, kv_heads, dim, page, lens, rows, in_place):
    P = Paged(lens, rows, kv_heads, dim, page, TYPES[dtype], seed=dim)
    r = np.random.default_rng(dim)
    n_keep, path = [], []
    for n in rows:
        kept = [0] + sorted(r.choice(np.arange(1, n), int(r.integers(0, n)), replace=False).tolist()) if n else []
        n_keep.append(len(kept))
        path += kept + [-1] * (n - len(kept))
    k0, v0 = P.k.clone(), P.v.clone()
    wk, wv = P.k.clone(), P.v.clone()
    for b, t in enumerate(lens):
        for i in range(n_keep[b]):
            s, d = P.place(b, t + path[_starts(rows)[b] + i]), P.place(b, t + i)
            wk[d], wv[d] = k0[s], v0[s]
    new = None if in_place else torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    path_dev = _i32(path) if path else torch.zeros(1, dtype=torch.int32, device="cuda")
    got = P.cache.keep(_i32(_starts(rows)), _i32(n_keep), path_dev, new_len=new)
    P.cache.status()
    assert got.tolist() == [t + n for t, n in zip(lens, n_keep)]
    assert (P.len if in_place else new) is got and (in_place or P.len.tolist() == lens)
    assert torch.equal(P.k, wk) and torch.equal(P.v, wv)


def test_keep_refuses_bad_paths():
    P = Paged([20, 20], [4, 4], 1, 64, 16, torch.bfloat16, seed=3)
    k0 = P.k.clone()
    starts, new = _i32([0, 4, 8]), _i32([0, 0])
    for n, path in (([4, 1], [0, 2, 2, 3, 0, -1, -1, -1]), ([2, 1], [1, 0, 0, 0, 0, 0, 0, 0]),
                    ([2, 1], [0, 4, 0, 0, 0, 0, 0, 0]), ([5, 1], [0, 1, 2, 3, 0, 0, 0, 0]),
                    ([1, 1], [-1, 0, 0, 0, 0, 0, 0, 0]), ([-1, 1], [0] * 8)):
        P.cache.keep(starts, _i32(n), _i32(path), new_len=new)
        with pytest.raises(B.MoeError, match="path"):
            P.cache.status()
        assert torch.equal(P.k, k0) and new.tolist() == [20, 21], (n, path)


# ------------------------------------------------------------------ verification

def _verify_ref(z, tokens, rows, parents, ut, up, q, T):
    """The definition in float64, walking one sequence after another."""
    z = z.double().cpu().numpy()
    z = np.where(np.isnan(z), -np.inf, z)
    q = None if q is None else q.double().cpu().numpy()
    ut, up = [np.asarray(x, dtype=np.float64) for x in (ut, up)]
    n_keep, path, said, logp, at = [], [], [], [], 0

    def target(r, t):
        top = z[r].max()
        if not t > 0:
            p = np.zeros(z.shape[1])
            p[int(np.argmax(z[r]))] = 1
            return p
        with np.errstate(invalid="ignore"):
            p = np.exp(np.where(z[r] == top, 0.0, (z[r] - top) / t))
        return p / p.sum()

    def draw(w, u):
        c = np.cumsum(w)
        return int(np.searchsorted(c, c[-1] * u, side="right"))

    for b, n in enumerate(rows):
        cur, walk, out, lp = 0, [0], [], []
        while n:
            p = target(at + cur, T[b])
            kids = [c for c in range(cur + 1, n) if parents[b][c] == cur and 0 <= tokens[at + c] < z.shape[1]]
            went = None
            if q is None:
                t = draw(p, up[at + cur])
                went = next((c for c in kids if tokens[at + c] == t), None)
            else:
                w, rest, S = p, 1.0, 0.0
                for c in kids:
                    x = tokens[at + c]
                    if ut[at + c] * q[at + cur][x] * rest < w[x]:
                        went, t = c, x
                        break
                    S += rest
                    w = np.maximum(p - S * q[at + cur], 0)
                    rest = w.sum()
                if went is None:
                    t = draw(w if rest > 0 else p, up[at + cur])
            out.append(t)
            with np.errstate(divide="ignore"):
                lp.append(np.log(p[t]))
            if went is None:
                break
            walk.append(went)
            cur = went
        if not n:
            walk = []
        n_keep.append(len(walk))
        path += walk + [-1] * (n - len(walk))
        said += out + [-1] * (n - len(out))
        logp += lp + [0.0] * (n - len(lp))
        at += n
    return n_keep, path, said, logp


def _verify_check(z, tokens, rows, parents, ut, up, q, T, chain=False, verifier=None):
    R, V = z.shape
    v = verifier or D.Verifier(V, max_rows=R, max_seqs=len(rows))
    f = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    par = None if chain else _i32([p for ps in parents for p in ps])
    got = v.verify(z, _i32(tokens), _i32(_starts(rows)), None if ut is None else f(ut), f(up), parent=par,
                   draft_probs=q, temperature=None if T is None else f(T))
    v.status()
    Th = [1.0] * len(rows) if T is None else np.asarray(T, np.float32).astype(np.float64).tolist()
    want = _verify_ref(z, tokens, rows, parents, None if ut is None else np.asarray(ut, np.float32),
                       np.asarray(up, np.float32), q, Th)
    for g, w, name in zip(got, want, ("n_keep", "path", "tokens")):
        assert g.tolist() == list(w), name
    lp, wl = got[3].double().cpu().numpy(), np.asarray(want[3])
    with np.errstate(invalid="ignore"):
        assert (np.where(lp == wl, 0, np.abs(lp - wl)) <= 2.0 ** -24 * np.abs(wl) + 1e-12).all()
    again = v.verify(z, _i32(tokens), _i32(_starts(rows)), None if ut is None else f(ut), f(up), parent=par,
                     draft_probs=q, temperature=None if T is None else f(T))
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


@pytest.mark.parametrize("logits", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,rows,width,sampled,pad", [
    (1, [1, 2], 1, True, 0), (7, [3, 1, 5], 2, True, 1), (7, [3, 1, 5], 2, False, 0), (1000, [6, 6, 0, 4], 1, True, 3),
    (2047, [9, 8], 3, True, 0), (2048, [9, 8], 3, False, 5), (2049, [16], 4, True, 0), (4099, [40, 3], 4, True, 2),
    (50257, [5, 6], 1, True, 0), (131072, [7], 2, False, 0), (200003, [4, 3], 2, True, 1)])
def test_verify(logits, V, rows, width, sampled, pad):
    r = np.random.default_rng(V + len(rows))
    dt = {"f32": torch.float32, **TYPES}[logits]
    R = sum(rows)
    base = torch.randn((R, V + pad), generator=_gen(V)) * 2.5
    z = base.to(dt).cuda()[:, :V]
    noisy = torch.randn((R, V), generator=_gen(V + 1)) * 0.5 + base[:, :V]
    q = torch.softmax(noisy / 0.9, 1).cuda()
    parents = [_tree(n, width, 3 + b) if n else [] for b, n in enumerate(rows)]
    tokens, at = [], 0
    for b, n in enumerate(rows):
        for i in range(n):
            pr = q[at + max(parents[b][i], 0)].double().cpu().numpy()
            nth = sum(p == parents[b][i] for p in parents[b][:i])
            tokens.append(int(r.choice(V, p=pr / pr.sum())) if sampled else int(np.argsort(-pr, kind="stable")[nth % V]))
        at += n
    T = [0.0 if b % 4 == 1 else 0.7 + 0.1 * b for b in range(len(rows))]
    for trial in range(3):
        ut, up = r.random(R).astype(np.float32), r.random(R).astype(np.float32)
        if trial == 2:
            T = None
        _verify_check(z, tokens, rows, parents, ut if sampled else None, up, q if sampled else None, T,
                      chain=width == 1)


def test_verify_rejections_in_a_row():
    """Drafts the target hardly wants: sibling after sibling is refused, down to an empty residual."""
    V, n = 5000, 12
    g = _gen(5)
    z = (torch.randn((2 * n, V), generator=g) * 2).cuda()
    q = torch.softmax(torch.randn((2 * n, V), generator=g) * 2, 1).cuda()
    rows, parents = [n, n], [[-1] + [0] * (n - 1), [-1, 0, 0, 0, 1, 1, 1, 2, 2, 3, 3, 3]]
    r = np.random.default_rng(0)
    tokens = [int(r.choice(V, p=(lambda p: p / p.sum())(q[n * b + max(p, 0)].double().cpu().numpy())))
              for b in range(2) for p in parents[b]]
    for t in range(3):
        _verify_check(z, tokens, rows, parents, r.random(2 * n), r.random(2 * n), q, [1.0, 0.8])
    # the draft's probabilities are the target's but for their rounding
    q = torch.softmax(z.double(), 1).float()
    last = float(np.nextafter(np.float32(1), np.float32(0)))
    _verify_check(z, tokens, rows, parents, [last] * (2 * n), r.random(2 * n), q, None)
    # a greedy target whose token the draft was sure of, and drafted tokens that are others: the residual
    # is empty, and the token comes from the target
    q = torch.nn.functional.one_hot(z.argmax(1), V).float()
    wrong = [int(t + 1) % V for t in z.argmax(1).tolist()]
    got = _verify_check(z, wrong, rows, parents, r.random(2 * n), r.random(2 * n), q, [0.0, 0.0])
    assert got[0].tolist() == [1, 1]


def test_verify_picks_at_the_ends():
    """u of 0 and just under 1, weights of 0 at both ends, equal largest logits, infinities."""
    V = 4100
    inf = float("inf")
    z = torch.full((6, V), -inf)
    z[0, 3], z[0, 4000] = 1.0, 1.0          # u = 0: the first with weight
    z[1, 3], z[1, 4000] = 1.0, 1.0          # u just under 1: the last with weight
    z[2, 100], z[2, 50], z[2, 60] = 2.0, 2.0, 2.0    # greedy: the lowest of equals
    z[3, 7], z[3, 9] = inf, inf             # all weight on the infinite ones
    z[4] = torch.linspace(-1, 1, V)
    z[4, 5] = float("nan")                  # weighs nothing
    z[5, V - 1] = -3.4e38
    z = z.cuda()
    last = float(np.nextafter(np.float32(1), np.float32(0)))
    got = _verify_check(z, [0] * 6, [1] * 6, [[-1]] * 6, None, [0.0, last, 0.5, 0.75, 0.0, last], None,
                        [1.0, 0.5, 0.0, 1.0, 1.0, 2.0], chain=True)
    assert got[2].tolist() == [3, 4000, 50, 9, 0, V - 1]


def test_verify_reports_bad_tokens_and_logits():
    V = 300
    z = torch.randn((4, V), generator=_gen(1)).cuda()
    q = torch.softmax(z, 1)
    v = D.Verifier(V, max_rows=4, max_seqs=1)
    one = torch.full((4,), 0.5, device="cuda")
    for bad in (-1, V, 1 << 30):
        got = v.verify(z, _i32([0, bad, bad, bad]), _i32([0, 4]), one, one, parent=_i32([-1, 0, 0, 0]), draft_probs=q)
        with pytest.raises(B.MoeError, match="token"):
            v.status()
        # such a draft changes nothing: the token is drawn from the target itself
        want = v.verify(z[:1], _i32([0]), _i32([0, 1]), one[:1], one[:1], draft_probs=q[:1])
        assert got[0].tolist() == [1] and got[2][0] == want[2][0]
        v.status()
    z[0] = -float("inf")
    got = v.verify(z, _i32([0, 1, 2, 3]), _i32([0, 4]), None, one)
    with pytest.raises(B.MoeError, match="logits"):
        v.status()
    assert got[0].tolist()[0] >= 1 and 0 <= int(got[2][0]) < V
    for bad in ([1, 4], [0, 5], [-1, 4]):
        v.verify(z[1:].contiguous(), _i32([0, 1, 2]), _i32(bad), None, one[:3])
        with pytest.raises(B.MoeError, match="row_start"):
            v.status()


def test_verify_follows_the_target():
    """20000 sequences of two drafted siblings each over a small vocabulary: the first token's counts
    follow the target's probabilities whatever the drafts (chi-squared, 31 degrees of freedom; its
    0.99999 quantile is 81.6, with a fixed seed)."""
    V, B_ = 32, 20000
    g = _gen(77)
    z = torch.randn((1, V), generator=g).repeat(3 * B_, 1).cuda()
    q1 = torch.softmax(torch.randn((1, V), generator=g), 1)
    q = q1.repeat(3 * B_, 1).cuda()
    tokens = torch.multinomial(q1[0], 3 * B_, replacement=True, generator=g).int().cuda()
    ut, up = torch.rand(3 * B_, generator=g).cuda(), torch.rand(3 * B_, generator=g).cuda()
    v = D.Verifier(V, max_rows=3 * B_, max_seqs=B_)
    starts = torch.arange(0, 3 * B_ + 1, 3, dtype=torch.int32, device="cuda")
    parent = _i32([-1, 0, 0] * B_)
    n_keep, _, said, _ = v.verify(z, tokens, starts, ut, up, parent=parent, draft_probs=q)
    v.status()
    p = torch.softmax(z[0].double(), 0).cpu().numpy()
    seen = np.bincount(said[::3].cpu().numpy(), minlength=V)
    assert (((seen - B_ * p) ** 2) / (B_ * p)).sum() < 81.6
    assert 0.3 < float((n_keep == 2).float().mean()) < 0.999


def test_the_operators_in_a_graph():
    """append, attend, verify and keep captured together and replayed on changing inputs equal eager calls."""
    def state(seed):
        P = Paged([90, 33], [5, 4], 2, 64, 16, torch.bfloat16, seed=13)
        g = _gen(seed)
        return P, torch.randn((9, 8 * 64), generator=g).to(torch.bfloat16).cuda(), torch.randn((9, 512), generator=g).cuda()

    starts, tokens = _i32([0, 5, 9]), _i32([3, 1, 4, 1, 5, 9, 2, 6, 5])
    u = torch.full((9,), 0.4, device="cuda")
    rope = D.Rope(D.rope_frequencies(64)[0])
    v = D.Verifier(512, 9, 2)

    def step(P, x, z, q_out, o, new_len):
        P.cache.append(rope, x[:, :256], x[:, 256:384], x[:, 384:], starts, out=q_out)
        P.cache.attend(q_out, starts, out=o)
        n, path, said, lp = v.verify(z, tokens, starts, None, u)
        P.cache.keep(starts, n, path, new_len=new_len)
        return n, path, said, lp

    def buffers():
        return (torch.zeros((9, 256), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((9, 256), dtype=torch.bfloat16, device="cuda"), _i32([0, 0]))

    P, x, z = state(0)
    b1 = buffers()
    k0, v0 = P.k.clone(), P.v.clone()
    step(P, x, z, *b1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(P, x, z, *b1)
    for s in range(4):
        P2, x2, z2 = state(30 + s)
        x.copy_(x2), z.copy_(z2), P.k.copy_(k0), P.v.copy_(v0)
        graph.replay()
        b2 = buffers()
        want = step(P2, x2, z2, *b2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), s
        assert all(torch.equal(a, b) for a, b in zip(b1, b2)), s
        assert torch.equal(P.k, P2.k) and torch.equal(P.v, P2.v)
    P.cache.status(), v.status()


@pytest.mark.parametrize("rows", [[20, 5], [700, 5]])
def test_keep_with_a_bad_page_moves_nothing(rows):
    """A page that the cache does not have, at a source or a place of the path, early or late in it: the whole path stays
    where it was and the length too; the other sequence's path is kept."""
    lens = [20, 33]
    path = [0] + list(range(2, rows[0])) + [-1] + [0, 2, 4, -1, -1]
    keep = [rows[0] - 1, 3]
    P = Paged(lens, rows, 2, 64, 16, torch.bfloat16, seed=3)
    starts, n_keep, path_dev, new = _i32(_starts(rows)), _i32(keep), _i32(path), _i32([0, 0])
    k0, v0, table = P.k.clone(), P.v.clone(), P.table.clone()
    wk, wv = k0.clone(), v0.clone()
    for i, s in enumerate((0, 2, 4)):
        wk[P.place(1, 33 + i)], wv[P.place(1, 33 + i)] = k0[P.place(1, 33 + s)], v0[P.place(1, 33 + s)]
    last = (lens[0] + rows[0] - 1) // 16      # the page of the last source
    for entry in (lens[0] // 16, last):       # that of the first place, too
        for bad in (-1, P.k.shape[0], 1 << 30):
            P.table[0, entry] = bad
            P.cache.keep(starts, n_keep, path_dev, new_len=new)
            P.table.copy_(table)
            with pytest.raises(B.MoeError, match="page") as e:
                P.cache.status()
            assert "path" not in str(e.value)
            assert torch.equal(P.k, wk) and torch.equal(P.v, wv) and new.tolist() == [20, 36], (entry, bad)
            P.k.copy_(k0), P.v.copy_(v0)


def test_keep_long_paths():
    """Paths of more rows than a workgroup has threads, bit for bit."""
    lens, rows = [5, 100], [900, 513]
    P = Paged(lens, rows, 1, 64, 48, torch.float16, seed=4)
    r = np.random.default_rng(3)
    kept = [[0] + sorted(r.choice(np.arange(1, n), n * 2 // 3, replace=False).tolist()) for n in rows]
    wk, wv = P.k.clone(), P.v.clone()
    for b, t in enumerate(lens):
        for i, s in enumerate(kept[b]):
            wk[P.place(b, t + i)], wv[P.place(b, t + i)] = P.k[P.place(b, t + s)], P.v[P.place(b, t + s)]
    path = [x for k, n in zip(kept, rows) for x in k + [-1] * (n - len(k))]
    got = P.cache.keep(_i32(_starts(rows)), _i32([len(k) for k in kept]), _i32(path))
    P.cache.status()
    assert got.tolist() == [t + len(k) for t, k in zip(lens, kept)]
    assert torch.equal(P.k, wk) and torch.equal(P.v, wv)


def test_append_with_a_bad_length_writes_nothing():
    """Rows of a sequence whose length is negative or past the table: token len + i of a later row may be a cached one.
    Its keys and values stay as they were, the other sequence's are appended, the queries are rotated all the same."""
    P = Paged([40, 20], [5, 2], 1, 64, 16, torch.bfloat16, seed=3)
    rope, starts = D.Rope(D.rope_frequencies(64)[0]), _i32([0, 5, 7])
    q = torch.randn((7, 64), generator=_gen(1)).to(torch.bfloat16).cuda()
    pos = _i32([40, 41, 42, 43, 44, 20, 21])
    k0, v0 = P.k.clone(), P.v.clone()
    want = P.cache.append(rope, q, q, q, starts, positions=pos)
    P.cache.status()
    wk, wv = k0.clone(), v0.clone()
    for t in (20, 21):
        wk[P.place(1, t)], wv[P.place(1, t)] = P.k[P.place(1, t)], P.v[P.place(1, t)]
    for bad in (-1, -3, -2 ** 31, P.table.shape[1] * 16 + 1, 2 ** 31 - 1):
        P.k.copy_(k0), P.v.copy_(v0), P.len.copy_(_i32([bad, 20]))
        got = P.cache.append(rope, q, q, q, starts, positions=pos)
        with pytest.raises(B.MoeError, match="length"):
            P.cache.status()
        assert torch.equal(got, want) and torch.equal(P.k, wk) and torch.equal(P.v, wv), bad


@pytest.mark.parametrize("bad", [[1, 4, 7], [0, 4, 6], [0, 4, 8], [2, 2, 7], [0, 0, 0]])
def test_starts_that_do_not_cover_the_rows_are_reported(bad):
    """row_start that does not begin at 0 or does not end at the number of rows, by every operator of the step."""
    P = Paged([40, 20], [4, 3], 1, 64, 16, torch.bfloat16, seed=3)
    q = torch.randn((7, 64), generator=_gen(1)).to(torch.bfloat16).cuda()
    rope, starts = D.Rope(D.rope_frequencies(64)[0]), _i32(bad)
    z, u, tokens = torch.randn((7, 300), generator=_gen(2)).cuda(), torch.full((7,), 0.5, device="cuda"), _i32([1] * 7)
    v = D.Verifier(300, max_rows=7, max_seqs=2)
    none = _i32([0, 0])
    for status, call in ((P.cache.status, lambda: P.cache.append(rope, q, q, q, starts)),
                         (P.cache.status, lambda: P.cache.attend(q, starts)),
                         (P.cache.status, lambda: P.cache.keep(starts, none, tokens, new_len=_i32([0, 0]))),
                         (v.status, lambda: v.verify(z, tokens, starts, None, u)),
                         (v.status, lambda: v.verify(z, tokens, starts, u, u, draft_probs=torch.softmax(z, 1)))):
        call()
        with pytest.raises(B.MoeError, match="row_start"):
            status()
        status()


def test_keep_of_layers_that_share_lengths():
    """Three layers' caches over one table and one length tensor, and one with a length of its own: each moves its own
    rows from where they were, and every length advances once."""
    lens, rows = [40, 0, 15], [6, 4, 9]
    layers = [Paged(lens, rows, 2, 64, 16, torch.bfloat16, seed=3) for _ in range(4)]
    shared, own = layers[0], layers[3]
    for j, P in enumerate(layers[1:3]):
        P.k.copy_(torch.randn(P.k.shape, generator=_gen(50 + j)))
        P.cache = D.PagedCache(P.k, P.v, shared.table, shared.len)
    path = [[0, 2, 5], [0, 1], [0, 3, 4, 8]]
    flat = [x for p, n in zip(path, rows) for x in p + [-1] * (n - len(p))]
    want = []
    for P in layers:
        k, v = P.k.clone(), P.v.clone()
        for b, p in enumerate(path):
            for i, s in enumerate(p):
                k[P.place(b, lens[b] + i)] = P.k[P.place(b, lens[b] + s)]
                v[P.place(b, lens[b] + i)] = P.v[P.place(b, lens[b] + s)]
        want.append((k, v))
    D.keep_paths([P.cache for P in layers], _i32(_starts(rows)), _i32([len(p) for p in path]), _i32(flat))
    for P, (k, v) in zip(layers, want):
        P.cache.status()
        assert torch.equal(P.k, k) and torch.equal(P.v, v)
    assert shared.len.tolist() == own.len.tolist() == [43, 2, 19]


def test_one_row_of_an_odd_stride():
    """A single row cut out of rows that are not aligned to each other: aligned itself, so it is taken."""
    P = Paged([37], [1], 2, 64, 16, torch.bfloat16, seed=6)
    x = torch.randn((2, 1001), generator=_gen(1)).to(torch.bfloat16).cuda()
    q, starts = x[:1, :256], _i32([0, 1])
    rope = D.Rope(D.rope_frequencies(64)[0], layout="interleaved")
    want = P.cache.append(rope, q.contiguous(), x[:1, 256:384].contiguous(), x[:1, 384:512].contiguous(), starts)
    k = P.k.clone()
    assert torch.equal(P.cache.append(rope, q, x[:1, 256:384], x[:1, 384:512], starts), want) and torch.equal(P.k, k)
    assert torch.equal(P.cache.attend(q, starts), P.cache.attend(q.contiguous(), starts))
    P.cache.status()
