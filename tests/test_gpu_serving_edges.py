"""The served batch's operators where they can go wrong: values that are not finite, bad pages, lengths, groups and starts, other
streams and graphs, and for sampling every way that logits can lie. Tolerances as derived in test_gpu_serving.py."""
import numpy as np
import pytest
import torch

from latent_mixture_experts_bf16_amd import binding as B
from latent_mixture_experts_bf16_amd import drafted as D
from latent_mixture_experts_bf16_amd import serving as S
from test_gpu_drafted import TINY, TYPES, Paged, _attend_check, _attend_ref, _gen, _i32, _see, _starts, _trees
from test_gpu_serving import Mx, _cache, _means, _sample_check, _sample_ref, _share

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("format", ["mx8", "mx4"])
def test_codes_at_the_ends_of_the_range(dtype, format):
    """Blocks of zeros, of numbers that are exactly a code, just past the largest one, tiny, the type's largest, infinite and NaN;
    a rotation by nothing, so that values reach the codes as they are."""
    dt, most = TYPES[dtype], {"mx8": 448.0, "mx4": 6.0}[format]
    big = torch.finfo(dt).max
    blocks = torch.zeros(12, 32)
    blocks[1] = torch.linspace(-6, 6, 32)
    blocks[2, :4] = torch.tensor([most, -most, most / 2, 1.0])
    blocks[3, :2] = torch.tensor([most * (1 + 2.0 ** -7), 1.0])        # twice the power
    blocks[4] = 2.0 ** -20
    blocks[5, 7] = -torch.finfo(dt).tiny
    blocks[6, 0], blocks[6, 1] = big, -big
    blocks[7, 3] = float("inf")
    blocks[8, 9] = float("nan")
    blocks[9, 31] = -float("inf")
    blocks[10] = -0.0
    blocks[11, 0], blocks[11, 1:] = 1.0, 2.0 ** -8                     # far below the block's largest
    x = blocks.to(dt).reshape(6, 64).cuda()
    P = Mx([0], [6], 1, 64, 16, dt, seed=1, format=format)
    starts, q = _i32([0, 6]), torch.zeros((6, 64), dtype=dt, device="cuda")
    rope = D.Rope(torch.zeros(32))
    P.cache.append(rope, q, x, x, starts)
    P.cache.status()
    k, v = P.cache.read(starts, 6)
    # (a rotation takes what is not finite to the other of the pair, in the keys' other block)
    assert torch.equal(k[[0, 1, 2, 5]], v[[0, 1, 2, 5]]) and torch.isnan(k[[3, 4]]).all()
    got, src = v.cpu().double().reshape(12, 32), blocks.to(dt).double()
    for i in (7, 8, 9):
        assert torch.isnan(got[i]).all()
    assert torch.isfinite(got[[j for j in range(12) if j not in (7, 8, 9)]]).all()
    half, least = {"mx8": (2.0 ** -4, 2.0 ** -10), "mx4": (2.0 ** -2, 0.25)}[format]
    scales = torch.stack([P.scales[1][P.place(0, t)] for t in range(6)]).cpu().reshape(12)
    for i in range(12):
        if i in (7, 8, 9):
            assert scales[i] == 255
            continue
        unit, top = 2.0 ** (float(scales[i]) - 127), float(src[i].abs().max())
        if i == 6:      # the power stops where the largest code is finite in the type
            assert float(scales[i]) == {"mx8": 126, "mx4": 132}[format] + {"f16": 8, "bf16": 120}[dtype]
            assert float(got[i].abs().max()) == most * unit
            continue
        assert top <= most * unit and (scales[i] == 1 or top > most * unit / 2), i
        assert ((got[i] - src[i]).abs() <= torch.maximum(half * src[i].abs(), torch.tensor(least * unit, dtype=torch.float64))).all(), i
    assert (got[0] == 0).all() and (got[2, :4] == src[2, :4]).all()


@pytest.mark.parametrize("format", ["mx8", "mx4"])
def test_blocks_that_are_nan_reach_only_the_rows_that_see_them(format):
    dt = torch.bfloat16
    lens, rows = [37, 0], [20, 9]
    masks = _trees(rows, 2, 9)
    P = Mx(lens, rows, 2, 64, 16, dt, seed=6, format=format)
    q = torch.randn((29, 4 * 64), generator=_gen(1)).to(dt).cuda()
    want = _attend_check(P, 4, masks, q=q).clone()
    used = {P.place(b, t) for b in range(2) for t in range(lens[b] + rows[b])}
    for page in range(P.k.shape[0]):
        for slot in range(16):
            if (page, slot) not in used:
                for s in P.scales:
                    s[page, slot] = 255
    m = torch.tensor(masks, device="cuda")
    assert torch.equal(P.cache.attend(q, _i32(_starts(rows)), mask=m), want)
    for b, j in ((0, 3), (1, 2), (0, 11)):
        place = P.place(b, lens[b] + j)
        keep = [s[place].clone() for s in P.scales]
        P.scales[1][place] = 255
        if j == 11:
            P.scales[0][place] = 255
        got = P.cache.attend(q, _i32(_starts(rows)), mask=m)
        at = _starts(rows)[b]
        for r in range(29):
            if at <= r < at + rows[b] and masks[r] >> j & 1:
                assert torch.isnan(got[r]).all(), (b, j, r)
            else:
                assert torch.equal(got[r], want[r]), (b, j, r)
        for s, k in zip(P.scales, keep):
            s[place] = k


@pytest.mark.parametrize("format", ["mx8", "mx4"])
@pytest.mark.parametrize("kv_heads,dim,page,heads_first", [(2, 64, 16, True), (3, 96, 48, False), (1, 256, 32, True)])
def test_keep_moves_codes_and_scales(format, kv_heads, dim, page, heads_first):
    lens, rows = [5, 0, 100], [30, 4, 13]
    P = Mx(lens, rows, kv_heads, dim, page, torch.bfloat16, seed=4, format=format, heads_first=heads_first)
    kept = [[0, 2, 3, 9, 29], [0], [0, 1, 12]]
    want = [t.clone() for t in P.codes + P.scales]
    for b, path in enumerate(kept):
        for i, s in enumerate(path):
            for w, t in zip(want, P.codes + P.scales):
                w[P.place(b, lens[b] + i)] = t[P.place(b, lens[b] + s)]
    flat = [x for p, n in zip(kept, rows) for x in p + [-1] * (n - len(p))]
    D.keep_paths([P.cache], _i32(_starts(rows)), _i32([len(p) for p in kept]), _i32(flat))
    P.cache.status()
    assert P.len.tolist() == [t + len(p) for t, p in zip(lens, kept)]
    for w, t in zip(want, P.codes + P.scales):
        assert torch.equal(w, t)


def test_read_any_tokens_and_none():
    """Tokens before the length, the same ones twice (two sequences over one table), past the table and on a bad page: the last two
    leave their rows and are reported."""
    P = Mx([70, 40], [3, 1], 2, 64, 16, torch.float16, seed=5)
    starts = _i32([0, 9, 11])
    k, v = P.cache.read(starts, 11, start=_i32([33, 2]))
    P.cache.status()
    for r, (b, t) in enumerate([(0, 33 + i) for i in range(9)] + [(1, 2), (1, 3)]):
        assert torch.equal(k[r].reshape(2, 64), P.k[P.place(b, t)]) and torch.equal(v[r].reshape(2, 64), P.v[P.place(b, t)])
    cap = P.table.shape[1] * 16
    wide = [torch.full((11, 136), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    out = tuple(t[:, :128] for t in wide)
    assert P.cache.read(starts, 11, start=_i32([cap - 2, 2]), out=out) is out
    with pytest.raises(B.MoeError, match="page"):
        P.cache.status()
    assert (wide[0][:9] == 5).all() and (wide[0][:, 128:] == 5).all()      # the pages past a sequence's own are no pages
    assert torch.equal(out[0][9:], k[9:]) and torch.equal(out[1][9:], v[9:])
    P.cache.read(starts, 11, start=_i32([-1, 2]), out=out)
    with pytest.raises(B.MoeError, match="length"):
        P.cache.status()
    assert (wide[0][:9] == 5).all()


@pytest.mark.parametrize("kind", ["none", "mx8", "mx4"])
def test_append_with_a_bad_length_or_page_writes_nothing(kind):
    P = _cache(kind, [40, 20], [5, 2], 1, 64, 16, torch.bfloat16, seed=3)
    held = [P.k, P.v] if kind == "none" else P.codes + P.scales
    rope, starts = D.Rope(D.rope_frequencies(64)[0]), _i32([0, 5, 7])
    norm = S.HeadNorm(torch.ones(64, device="cuda"), torch.ones(1, 64, device="cuda"))
    q = torch.randn((7, 64), generator=_gen(1)).to(torch.bfloat16).cuda()
    pos = _i32([40, 41, 42, 43, 44, 20, 21])
    before = [t.clone() for t in held]
    want = P.cache.append(rope, q, q, q, starts, positions=pos, norm=norm)
    P.cache.status()
    after = [b.clone() for b in before]
    for t in (20, 21):
        for a, h in zip(after, held):
            a[P.place(1, t)] = h[P.place(1, t)]
    table = P.table.clone()
    for what, bad in [("length", v) for v in (-1, -2 ** 31, P.table.shape[1] * 16 + 1, 2 ** 31 - 1)] + [
            ("page", v) for v in (-1, P.k.shape[0], 1 << 30)]:
        for h, b in zip(held, before):
            h.copy_(b)
        if what == "length":
            P.len.copy_(_i32([bad, 20]))
        else:
            P.len.copy_(_i32([40, 20]))
            P.table[0, 40 // 16] = bad
        got = P.cache.append(rope, q, q, q, starts, positions=pos, norm=norm)
        P.table.copy_(table)
        with pytest.raises(B.MoeError, match=what):
            P.cache.status()
        assert torch.equal(got, want), bad
        for h, a in zip(held, after):
            assert torch.equal(h, a), (what, bad)


@pytest.mark.parametrize("bad", [[1, 4, 7], [0, 4, 6], [0, 4, 8], [2, 2, 7], [0, 0, 0]])
def test_starts_that_do_not_cover_the_rows_are_reported(bad):
    q = torch.randn((7, 64), generator=_gen(1)).to(torch.bfloat16).cuda()
    rope, starts = D.Rope(D.rope_frequencies(64)[0]), _i32(bad)
    norm = S.HeadNorm(torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    shared = S.SharedPrefix(_i32([0, 2]), _i32([20]))
    for kind in ("none", "mx8"):
        P = _cache(kind, [40, 20], [4, 3], 1, 64, 16, torch.bfloat16, seed=3)
        calls = [lambda: P.cache.append(rope, q, q, q, starts, norm=norm), lambda: P.cache.attend(q, starts, shared=shared)]
        if kind == "mx8":
            calls += [lambda: P.cache.read(starts, 7), lambda: P.cache.attend(q, starts),
                      lambda: P.cache.keep(starts, _i32([0, 0]), _i32([0] * 7), new_len=_i32([0, 0]))]
        for call in calls:
            call()
            with pytest.raises(B.MoeError, match="row_start"):
                P.cache.status()
            P.cache.status()


def test_norms_of_zero_one_and_large_heads():
    """A head of zeros stays zero (also with eps 0), one of equal values becomes ones, weights in three types and of heads apart,
    and a row of NaN spoils no other."""
    P = Paged([3], [4], 1, 128, 16, torch.bfloat16, seed=2)
    rope, starts = D.Rope(torch.zeros(64)), _i32([0, 4])
    q = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    q[1, :128], q[1, 128:] = 3.0, -2.0 ** 40
    q[2] = 2.0 ** -60
    q[3] = float("nan")
    k = q[:, :128].contiguous()
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        w = torch.tensor([[1.0], [2.0]], device="cuda").expand(2, 128).to(dt).contiguous()
        out = P.cache.append(rope, q, k, k, starts, norm=S.HeadNorm(w, w[0], eps=0.0))
        P.cache.status()
        assert (out[0] == 0).all() and torch.isnan(out[3]).all()
        assert (out[1, :128] == 1).all() and (out[1, 128:] == -2).all()
        assert (out[2, :128] == 1).all() and (out[2, 128:] == 2).all()
        kept = torch.stack([P.k[P.place(0, 3 + i)][0] for i in range(4)])
        assert torch.equal(kept[:3], out[:3, :128]) and torch.isnan(kept[3]).all()
    # rows and weights of odd strides, eps that outweighs the values
    wide = torch.randn((3, 131), generator=_gen(4)).cuda()[:, :128]
    x = torch.randn((4, 3 * 128 + 5), generator=_gen(5)).to(torch.bfloat16).cuda()[:, 3:3 + 384]
    out = P.cache.append(rope, x[:, :256], x[:, 256:], x[:, 256:], starts, norm=S.HeadNorm(wide[:2], wide[2:], eps=1e4, offset=1.0))
    y = x[:, :256].double().reshape(4, 2, 128)
    y = y / (y.square().mean(-1, keepdim=True) + 1e4).sqrt() * (1 + wide[:2].double())
    assert ((out.double().reshape(4, 2, 128) - y).abs() <= (2.0 ** -8 + 24 * 2.0 ** -24) * y.abs()).all()


@pytest.mark.parametrize("dim", [32, 96, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_values_whose_squares_leave_fp32(dim, eps):
    """bf16 holds values whose squares fp32 does not: the norm is that of the formula for them too."""
    powers = [0, 59, 60, 64, 100, 124, -49, -51, -60, -100, -130]
    n, g = len(powers), _gen(5)
    P = Paged([0], [n], 2, dim, 16, torch.bfloat16, seed=3)
    x = torch.randn((n, 6, dim), generator=g).clamp(-7, 7) * 2.0 ** torch.tensor(powers, dtype=torch.float64)[:, None, None]
    x = x.to(torch.bfloat16).reshape(n, 6 * dim).cuda()
    q, k, v = x[:, :2 * dim], x[:, 2 * dim:4 * dim], x[:, 4 * dim:]
    w = torch.randn(dim, generator=g)
    out = P.cache.append(D.Rope(torch.zeros(dim // 2)), q, k, v, _i32([0, n]), norm=S.HeadNorm(w.cuda(), w.cuda(), eps=eps))
    P.cache.status()

    def near(got, t):
        t = t.double().cpu().reshape(n, 2, dim)
        y = t / (t.square().mean(-1, keepdim=True) + float(np.float32(eps))).sqrt() * w.double()
        tol = 24 * 2.0 ** -24 * y.abs()
        return ((got.double().cpu().reshape(n, 2, dim) - y).abs() <= tol + 2.0 ** -8 * (y.abs() + tol) + TINY[torch.bfloat16]).all()

    assert near(out, q)
    assert near(torch.stack([P.k[P.place(0, t)] for t in range(n)]), k)
    assert torch.equal(torch.stack([P.v[P.place(0, t)] for t in range(n)]).reshape(n, 2 * dim), v)


# ------------------------------------------------------------------ a shared prompt

def test_shared_prompts_that_are_wrong_are_reported():
    lens, rows = [300, 310, 290, 305], [2, 1, 1, 3]
    P = Paged(lens, rows, 2, 64, 16, torch.bfloat16, seed=7)
    plain = P.cache
    _share(P, [0, 3, 4], [280, 100])
    q = torch.randn((7, 256), generator=_gen(1)).to(torch.bfloat16).cuda()
    starts = _i32(_starts(rows))
    want = P.cache.attend(q, starts).clone()
    for groups, lengths, says in [([0, 3, 4], [291, 100], "length"), ([0, 3, 4], [-5, 100], "length"),
                                  ([0, 3, 4], [2 ** 31 - 1, 100], "length"), ([0, 3, 3], [280, 100], "group_start"),
                                  ([1, 3, 4], [280, 100], "group_start"), ([0, 5, 4], [280, 100], "group_start"),
                                  ([0, -1, 4], [280, 100], "group_start"), ([3, 0, 4], [280, 100], "group_start")]:
        plain.attend(q, starts, shared=S.SharedPrefix(_i32(groups), _i32(lengths)))
        with pytest.raises(B.MoeError, match=says):
            plain.status()
    table = P.table.clone()
    P.table[0, 2] = 1 << 20
    P.cache.attend(q, starts)
    with pytest.raises(B.MoeError, match="page"):
        plain.status()
    P.table.copy_(table)
    assert torch.equal(P.cache.attend(q, starts), want)
    plain.status()


def test_shared_prompt_hides_nothing_and_uses_no_one_elses_tokens():
    """The followers' own pages of the prompt are not read (they may hold anything), and a value that is not finite in the shared
    part reaches every row of its group alone."""
    lens, rows = [200, 210, 150], [1, 2, 1]
    P = Paged(lens, rows, 1, 64, 16, torch.bfloat16, seed=9)
    _share(P, [0, 2, 3], [192, 64])
    q = torch.randn((4, 128), generator=_gen(1)).to(torch.bfloat16).cuda()
    starts = _i32(_starts(rows))
    want = _attend_check(P, 2, None, q=q).clone()
    P.table[1, :12] = P.k.shape[0] - 1           # names pages, but none that matters
    assert torch.equal(P.cache.attend(q, starts), want)
    P.v[P.place(0, 70)] = float("inf")
    got = P.cache.attend(q, starts)
    assert not torch.isfinite(got[:3]).any() and torch.equal(got[3], want[3])


@pytest.mark.parametrize("kind", ["none", "mx8", "mx4"])
def test_shared_and_codes_in_graphs_and_on_other_streams(kind):
    """Two graphs of the same calls, replayed in turn with changed inputs, against eager calls; and a side stream."""
    lens, rows = [400, 390, 395], [4, 1, 2]
    P = _cache(kind, lens, rows, 2, 128, 64, torch.bfloat16, seed=12)
    _share(P, [0, 3], [390])
    rope, norm = D.Rope(D.rope_frequencies(128)[0]), S.HeadNorm(torch.ones(128, device="cuda"), torch.ones(128, device="cuda"))
    starts = _i32(_starts(rows))
    x = torch.randn((7, 12 * 128), generator=_gen(1)).to(torch.bfloat16).cuda()
    shared, cache = P.cache.shared, P.cache.real
    held = [P.k, P.v] if kind == "none" else P.codes + P.scales
    outs = [torch.zeros((7, 1024), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    u = torch.rand(7, device="cuda")
    picks = [None, None]
    sampler = S.Sampler(1024, max_rows=7)

    def step(i):
        q = cache.append(rope, x[:, :1024], x[:, 1024:1280], x[:, 1280:], starts, norm=norm)
        cache.attend(q, starts, shared=shared, out=outs[i])
        picks[i] = sampler.sample(outs[i], u)

    step(0)
    want = outs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1)
    side.synchronize()
    assert torch.equal(outs[1], want) and torch.equal(picks[0][0], picks[1][0])
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(i)
    graph_picks = list(picks)
    for n in range(6):
        x.copy_(torch.randn(x.shape, generator=_gen(20 + n)).to(torch.bfloat16))
        u.copy_(torch.rand(7, generator=_gen(40 + n)))
        P.len.copy_(_i32([400 - n, 390, 395 - n]))
        for o in outs:
            o.zero_()
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        got, tokens, state = outs[n % 2].clone(), graph_picks[n % 2][0].clone(), [t.clone() for t in held]
        step(n % 2)
        assert torch.equal(got, outs[n % 2]) and torch.equal(tokens, picks[n % 2][0]), n
        for a, b in zip(state, held):
            assert torch.equal(a, b), n
    cache.status()
    sampler.status()


@pytest.mark.parametrize("kind", ["none", "mx8", "mx4"])
def test_attend_from_a_workspace_that_holds_anything(kind):
    """NaN in all the memory that the next allocations get changes nothing."""
    P = _cache(kind, [700, 690], [3, 2], 2, 64, 16, torch.bfloat16, seed=3)
    _share(P, [0, 2], [640])
    q = torch.randn((5, 512), generator=_gen(2)).to(torch.bfloat16).cuda()
    starts = _i32([0, 3, 5])
    want = P.cache.attend(q, starts).clone()
    logits = torch.randn((9, 70001), generator=_gen(3)).cuda()
    u, s = torch.rand(9, device="cuda"), S.Sampler(70001, max_rows=9)
    tokens = s.sample(logits, u)[0].clone()
    for _ in range(2):
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(12)]
        del junk
        assert torch.equal(P.cache.attend(q, starts), want)
        assert torch.equal(s.sample(logits, u)[0], tokens)


def test_a_step_of_a_served_batch():
    """The operators as they are used: requests after one prompt decode some tokens over an 8-bit cache; every step's attention
    against 64 bits on what the cache holds, every token against the definition."""
    lens, heads, kv, dim, V = [150, 150, 160], 8, 2, 64, 512
    P = Mx(lens, [6] * 3, kv, dim, 16, torch.bfloat16, seed=21)
    _share(P, [0, 3], [150])
    g = _gen(5)
    embed, qkv, head = ((torch.randn(s, generator=g) * f).to(torch.bfloat16).cuda()
                        for s, f in (((V, 256), 1.0), ((256, (heads + 2 * kv) * dim), 0.06), ((heads * dim, V), 0.3)))
    norm = S.HeadNorm(*(1 + 0.1 * torch.randn((n, dim), generator=g).cuda() for n in (heads, kv)))
    rope, sampler = D.Rope(*D.rope_frequencies(dim)), S.Sampler(V, max_rows=3)
    starts, tokens = _i32([0, 1, 2, 3]), torch.tensor([3, 77, 401], device="cuda")
    T, k, p = torch.tensor([0.8, 0.0, 1.1], device="cuda"), _i32([50, 0, 0]), torch.tensor([0.9, 1.0, 0.95], device="cuda")
    for step in range(5):
        x = embed[tokens.long()] @ qkv
        a, b = heads * dim, (heads + kv) * dim
        q = P.cache.real.append(rope, x[:, :a], x[:, a:b], x[:, b:], starts, norm=norm)
        o = P.cache.attend(q, starts)
        logits = (o @ head).float()
        u = torch.rand(3, generator=g)
        tokens, logp = sampler.sample(logits, u.cuda(), temperature=T, top_k=k, top_p=p)
        P.look()
        P.rows = [1] * 3
        y, tol = _attend_ref(P, q, _see(lens, P.rows, None), heads, dim ** -0.5)
        assert ((o.double().cpu().reshape(y.shape) - y).abs() <= tol).all(), step
        want, lp, _ = _sample_ref(logits.cpu().numpy(), u.tolist(), T.tolist(), k.tolist(), p.tolist(), None)
        assert tokens.tolist() == want and np.allclose(logp.cpu().numpy(), lp, rtol=2.0 ** -22, atol=2.0 ** -22), step
        P.len += 1
        lens = [t + 1 for t in lens]
        P.lens = lens
    P.cache.status()
    sampler.status()


# ------------------------------------------------------------------ sampling

CUTS = dict(top_k=[0, 1, 3, 40, 0, 7, 100000, 0], top_p=[1.0, 0.5, 0.9, 1.0, 0.3, 0.99, 1e-6, 0.0],
            min_p=[0.0, 0.2, 0.0, 0.01, 1.0, 0.5, 0.0, 2.0])


@pytest.mark.parametrize("logits", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["equal", "two values", "flat", "steep", "one high", "masked", "lowest", "negative zero", "rising",
                                  "infinite", "nan"])
def test_sample_logits_of_every_kind(logits, kind):
    V, R = 20011, 8
    z = torch.randn((R, V), generator=_gen(3))
    if kind == "equal":
        z = torch.full((R, V), 0.75)
    elif kind == "two values":
        z = (z > 1).float()
    elif kind == "flat":
        z = z * 0.01
    elif kind == "steep":
        z = z * 300
    elif kind == "one high":
        z[:, 12345] = 60.0
    elif kind == "masked":
        z[:, 5:19000] = -float("inf")
    elif kind == "lowest":
        z[:, 5:19000] = torch.finfo({"f32": torch.float32, **TYPES}[logits]).min
    elif kind == "negative zero":
        z = torch.where(z > 0, 0.0, -0.0)
        z[:, 77] = -1.0
    elif kind == "rising":
        z = torch.linspace(-20, 20, V).expand(R, V).clone()
    elif kind == "infinite":
        z[:, [7, 100, 15000]] = float("inf")
    elif kind == "nan":
        z[:, ::3] = float("nan")
    z = z.to({"f32": torch.float32, **TYPES}[logits])
    r = np.random.default_rng(7)
    T = [1.0, 0.7, 1.3, 0.05, 3.0, 1e-4, 0.0, 50.0]
    for u in (r.random(R).astype(np.float32), np.zeros(R, np.float32), np.full(R, np.float32(1 - 2.0 ** -24))):
        _sample_check(z, u)
        _sample_check(z, u, T=T)
        _sample_check(z, u, T=T, **CUTS)
        _sample_check(z, u, top_k=[5000] * R, top_p=[0.999] * R)


def test_sample_large_vocabularies_and_cells():
    """More logits in one cell than a list holds, in f32 (all different) and f16."""
    for dt in (torch.float32, torch.float16):
        z = (torch.rand((3, 200000), generator=_gen(1)) * 0.1).to(dt)
        u = np.array([0.001, 0.5, 0.9999], np.float32)
        _sample_check(z, u)
        _sample_check(z, u, top_k=[70000, 150000, 3], top_p=[0.9, 0.5, 1.0], min_p=[0.0, 0.93, 0.5])


def test_sample_odd_arguments():
    """Temperatures, cuts and random numbers that are NaN, infinite or out of range count as the header says."""
    V = 3001
    z = torch.randn((6, V), generator=_gen(2))
    nan, inf = float("nan"), float("inf")
    s, dev = S.Sampler(V, max_rows=6), lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    zc, u = z.cuda(), [0.1, 0.9, 0.5, 0.2, 0.7, 0.99]
    plain = s.sample(zc, dev(u))[0]
    assert torch.equal(s.sample(zc, dev(u), top_p=dev([nan, 2.0, inf, 1.0, nan, 1.5]), min_p=dev([nan, -1.0, 0.0, -inf, nan, 0.0]),
                                top_k=_i32([0, -5, -2 ** 31, V, V + 1, 2 ** 31 - 1]))[0], plain)
    best = z.argmax(1).tolist()
    assert s.sample(zc, dev(u), temperature=dev([0.0, -1.0, nan, -inf, 0.0, -0.0]))[0].tolist() == best
    assert s.sample(zc, dev(u), top_p=dev([0.0, -3.0, -inf, 1e-30, 0.0, 0.0]))[0].tolist() == best
    assert s.sample(zc, dev(u), min_p=dev([1.0, 7.0, inf, 1.0, 2.0, 1.0]))[0].tolist() == best
    low, high = s.sample(zc, dev([0.0] * 6))[0], s.sample(zc, dev([1 - 2.0 ** -24] * 6))[0]
    assert torch.equal(s.sample(zc, dev([nan, -1.0, -inf, 0.0, -0.0, nan]))[0], low)
    assert torch.equal(s.sample(zc, dev([1.0, 5.0, inf, 1.5, 1.0, 1.0]))[0], high)
    # an infinite temperature: all alike
    got = s.sample(zc, dev([0.5] * 6), temperature=dev([inf, 3e38, inf, inf, 1e30, inf]))
    want = [int(np.lexsort((np.arange(V), -z[i].double().numpy()))[V // 2]) for i in range(6)]
    assert got[0].tolist() == want and np.allclose(got[1].cpu(), -np.log(V), rtol=1e-6)
    s.status()


def test_sample_rows_without_logits_are_reported():
    z = torch.randn((4, 5000), generator=_gen(2))
    z[1], z[2] = -float("inf"), float("nan")
    s, u = S.Sampler(5000, max_rows=4), torch.full((4,), 0.5, device="cuda")
    tokens, logp = s.sample(z.cuda(), u)
    with pytest.raises(B.MoeError, match="logits without"):
        s.status()
    s.status()
    assert tokens[[1, 2]].tolist() == [0, 0] and logp[[1, 2]].tolist() == [0.0, 0.0]
    want, _, _ = _sample_ref(z[[0, 3]].numpy(), [0.5, 0.5], None, None, None, None)
    assert tokens[[0, 3]].tolist() == want


def test_sample_follows_the_weights():
    """Evenly spaced random numbers give each token its share to within one of the 20000 draws."""
    V, n = 50, 20000
    z = torch.randn(V, generator=_gen(9)) * 1.5
    u = (torch.arange(n, dtype=torch.float64) / n).float().cuda()
    tokens = S.Sampler(V, max_rows=n).sample(z.expand(n, V).contiguous().cuda(), u, top_p=torch.full((n,), 0.9, device="cuda"))[0]
    p = torch.softmax(z.double(), 0)
    order = torch.argsort(p, descending=True)
    kept = order[:int((p[order].cumsum(0) < float(np.float32(0.9))).sum()) + 1]
    share = torch.zeros(V, dtype=torch.float64)
    share[kept] = p[kept] / p[kept].sum()
    # a share's two ends may each fall on the other side of a number of 24 bits, and the next of the spaced ones
    assert (torch.bincount(tokens.cpu().long(), minlength=V).double() - n * share).abs().max() <= 2


def test_sample_many_rows():
    z = torch.randn((40000, 9), generator=_gen(4))
    u = torch.rand(40000, generator=_gen(5))
    tokens, _ = S.Sampler(9, max_rows=40000).sample(z.cuda(), u.cuda())
    zd, order = torch.sort(z.double(), dim=1, descending=True, stable=True)
    run = torch.softmax(zd, 1).cumsum(1)
    want = order.gather(1, (run <= u.double()[:, None] * run[:, -1:]).sum(1, keepdim=True).clamp(max=8))[:, 0]
    assert torch.equal(tokens.cpu().long(), want)
