"""More shapes of the drafted step's attention and verification: every query tile, caches cut into many parts,
many short sequences, scales of either sign. Tolerances as derived in test_gpu_drafted.py."""
import ctypes
import math

import numpy as np
import pytest
import torch

from latent_mixture_experts_bf16_amd import binding as B
from latent_mixture_experts_bf16_amd import drafted as D
from test_gpu_drafted import (Paged, TYPES, _attend_check, _gen, _i32, _starts, _tree, _trees, _verify_check)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 80, 96, 112, 128, 192, 256])
@pytest.mark.parametrize("group,rows", [(1, 3), (3, 9), (6, 10), (4, 40)])     # query tiles of 16, 32, 64, 128 (two of them)
def test_every_query_tile(dtype, dim, group, rows):
    P = Paged([70, 9], [rows, rows], 2, dim, 16, TYPES[dtype], seed=dim + rows)
    _attend_check(P, 2 * group, _trees([rows, rows], 2, 3))


@pytest.mark.parametrize("group,rows", [(1, 3), (3, 9), (6, 10), (4, 40)])
@pytest.mark.parametrize("dim", [80, 128])
def test_values_that_are_not_finite_in_every_query_tile(dim, group, rows):
    dt, n = torch.bfloat16, 2 * rows
    masks = _trees([rows, rows], 2, 5)
    P = Paged([37, 66], [rows, rows], 2, dim, 16, dt, seed=7)
    q = torch.randn((n, 2 * group * dim), generator=_gen(1)).to(dt).cuda()
    starts, m = _i32([0, rows, n]), torch.tensor(masks, device="cuda")
    want = P.cache.attend(q, starts, mask=m).clone()
    for b, j in ((0, rows - 1), (1, 1)):
        at = P.place(b, P.lens[b] + j)
        keep = P.v[at].clone()
        P.v[at][:, 5] = float("inf")
        got = P.cache.attend(q, starts, mask=m).view(n, -1, dim)
        P.v[at] = keep
        for r in range(n):
            sees = r // rows == b and masks[r] >> j & 1
            ok = torch.ones(dim, dtype=torch.bool, device="cuda")
            if sees:      # that dim and no other
                ok[5] = False
                assert (got[r][:, 5] == float("inf")).all()
            assert torch.equal(got[r][:, ok], want[r].view(-1, dim)[:, ok]), (b, j, r)
    P.cache.status()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-12, 3.0])
def test_scales(scale):
    P = Paged([150, 3], [5, 2], 2, 64, 32, torch.float16, seed=3)
    _attend_check(P, 4, None, scale=scale)


@pytest.mark.parametrize("page", [16, 48, 256])
def test_one_row_over_a_long_cache(page):
    """One item cut into hundreds of parts."""
    P = Paged([9001], [1], 1, 64, page, torch.bfloat16, seed=4)
    _attend_check(P, 5, None)


def test_a_long_sequence_among_short_ones():
    r = np.random.default_rng(8)
    lens = [int(v) for v in r.integers(0, 4, 300)]
    lens[7], lens[299] = 3000, 0
    rows = [int(v) for v in r.integers(0, 3, 300)]
    rows[7], rows[299] = 5, 1
    P = Paged(lens, rows, 1, 64, 16, torch.bfloat16, seed=4)
    _attend_check(P, 3, None)


def test_a_prompt_of_several_query_tiles():
    P = Paged([0, 100], [300, 130], 2, 64, 64, torch.float16, seed=4)
    _attend_check(P, 4, None)


def test_a_fresh_workspace_holds_anything():
    """The parts' records are written before they are read: whatever the memory held."""
    P = Paged([2000, 0, 31], [3, 1, 2], 2, 128, 64, torch.bfloat16, seed=9)
    q = torch.randn((6, 4 * 128), generator=_gen(1)).to(torch.bfloat16).cuda()
    starts, out = _i32([0, 3, 4, 6]), torch.zeros((6, 4 * 128), dtype=torch.bfloat16, device="cuda")
    lib, got = B.lib(), []
    need = lib.moe_tree_attend_workspace(P.cache._ref, 6, 4)
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        B._check(lib.moe_tree_attend(P.cache._ref, 6, q.data_ptr(), 512, 4, starts.data_ptr(), None, 128 ** -0.5,
                                     out.data_ptr(), 512, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert (ws[need:] == fill).all()
        got.append(out.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_verify_infinite_temperature_and_logits():
    """T of infinity: every finite logit weighs the same; logits of -infinity still nothing."""
    V = 2500
    z = torch.randn((3, V), generator=_gen(2)) * 4
    z[0, ::2] = -math.inf
    z[2, 9] = math.inf
    u = [0.25, 0.7501, 0.5]
    v = D.Verifier(V, 3, 3)
    got = v.verify(z.cuda(), _i32([0, 0, 0]), _i32([0, 1, 2, 3]), None, torch.tensor(u, device="cuda"),
                   temperature=torch.full((3,), math.inf, device="cuda"))
    v.status()
    assert got[2].tolist() == [2 * (V // 2 // 4) + 1, V * 3 // 4, 9]
    want = torch.tensor([-math.log(V / 2), -math.log(V), 0.0])
    assert (got[3].cpu() - want).abs().max() <= 2.0 ** -24 * 8 + 1e-12


@pytest.mark.parametrize("logits", ["f32", "bf16"])
def test_verify_refusals_along_a_path(logits):
    """Wide trees over several chunks whose drafts are refused one after another and at one row after another:
    more sums of what is left than there are launches for them."""
    V, n, B_ = 3001, 40, 5
    g = _gen(31)
    z = (torch.randn((B_ * n, V), generator=g) * 2)
    q = torch.softmax(z * 0.5 + torch.randn((B_ * n, V), generator=g), 1).cuda()
    z = z.to({"f32": torch.float32, **TYPES}[logits]).cuda()
    rows, parents = [n] * B_, [_tree(n, 8, 4 + b) for b in range(B_)]
    r = np.random.default_rng(5)
    tokens = []
    for b in range(B_):
        for i in range(n):
            pr = q[b * n + max(parents[b][i], 0)].double().cpu().numpy()
            tokens.append(int(r.choice(V, p=pr / pr.sum())))
    for _ in range(3):
        _verify_check(z, tokens, rows, parents, r.random(B_ * n).astype(np.float32), r.random(B_ * n).astype(np.float32), q,
                      [1.0, 0.7, 0.0, 1.5, 1.0])


@pytest.mark.parametrize("n", [64, 65, 130, 200])
def test_verify_long_chains(n):
    """More rows than a wave has lanes, most drafts accepted."""
    V = 300
    z = torch.randn((n + 3, V), generator=_gen(n)) * 6
    z[:, 0] = -math.inf
    tokens = [0] + [int(t) for t in z.argmax(1)[:-1]]
    rows = [n, 3]
    r = np.random.default_rng(n)
    up = (r.random(n + 3) * 0.3).astype(np.float32)
    q = torch.softmax(z, 1).cuda()
    par = [[-1] + list(range(n - 1)), [-1, 0, 1]]
    z = z.cuda()
    _verify_check(z, tokens, rows, par, None, up, None, [0.0, 1.0], chain=True)
    _verify_check(z, tokens, rows, par, [0.999] * (n + 3), up, q, [1.0, 1.0])


def test_verify_a_fresh_workspace_holds_anything():
    V, n = 5000, 9
    g = _gen(6)
    z, q = (torch.randn((n, V), generator=g) * 2).cuda(), torch.softmax(torch.randn((n, V), generator=g), 1).cuda()
    tokens = torch.multinomial(q, 1)[:, 0].int()
    starts, par = _i32([0, 6, 9]), _i32([-1, 0, 0, 1, 1, 1, -1, 0, 0])
    u = torch.rand(n, generator=g).cuda()
    lib, got = B.lib(), []
    need = lib.moe_draft_verify_workspace(n, 2, V)
    desc = B.make_tensor(z.data_ptr(), B.MOE_DT_F32, (n, V), (V, 1))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        out = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (2, n, n)] + [torch.zeros(n, device="cuda")]
        B._check(lib.moe_draft_verify(ctypes.byref(desc), tokens.data_ptr(), starts.data_ptr(), 2, par.data_ptr(), u.data_ptr(),
                                      u.data_ptr(), q.data_ptr(), V, None, *[o.data_ptr() for o in out], flags.data_ptr(),
                                      ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert int(flags) == 0 and (ws[need:] == fill).all()
        got.append(out)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(*got))


def test_rope_rows_of_many_sequences():
    """Each row finds its sequence among thousands, empty ones between."""
    r = np.random.default_rng(1)
    rows = [int(v) for v in r.integers(0, 2, 5000)]
    rows[0], rows[-1] = 1, 1
    lens = [int(v) for v in r.integers(0, 16, 5000)]
    P = Paged(lens, rows, 1, 32, 16, torch.bfloat16, seed=2)
    R = sum(rows)
    x = torch.randn((R, 32), generator=_gen(1)).to(torch.bfloat16).cuda()
    rope = D.Rope([0.0] * 16)
    out = P.cache.append(rope, x, x, x, _i32(_starts(rows)))
    P.cache.status()
    assert torch.equal(out, x)
    pages = [P.place(b, lens[b]) for b in range(5000) if rows[b]]
    pg, sl = torch.tensor([p for p, _ in pages]), torch.tensor([s for _, s in pages])
    assert torch.equal(P.k[pg, sl].view(R, 32), x) and torch.equal(P.v[pg, sl].view(R, 32), x)


@pytest.mark.parametrize("seqs,V", [(64, 131072), (300, 16385)])
def test_verify_refusals_of_a_full_batch(seqs, V):
    """Sampled trees whose siblings are refused one after another, over more chunks than the card's workgroups hold at
    once (seqs * V / 4096 of 1024): a workgroup that starts late finds others' arrivals counted, in every launch. The
    drafts are drawn apart from the target, so most sequences refuse two siblings or more at one row."""
    parent = [-1, 0, 0, 0, 0, 1]
    n, R = len(parent), len(parent) * seqs
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    z = torch.empty((R, V), device="cuda").normal_(0, 3, generator=g)
    q = torch.softmax(torch.empty((R, V), device="cuda").normal_(0, 3, generator=g), 1)
    at = torch.tensor([b * n + max(p, 0) for b in range(seqs) for p in parent], device="cuda")
    tokens = torch.multinomial(q[at], 1, generator=g)[:, 0].tolist()
    r = np.random.default_rng(seqs)
    T = (0.7 + 0.1 * (np.arange(seqs) % 5)).tolist()
    for _ in range(2):
        ut, up = r.random(R).astype(np.float32), r.random(R).astype(np.float32)
        got = _verify_check(z, tokens, [n] * seqs, [parent] * seqs, ut, up, q, T)
        assert (got[0] == 1).sum() > seqs // 2      # all four siblings refused
