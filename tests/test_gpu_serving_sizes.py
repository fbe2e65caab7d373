"""Calls of the served batch's operators at sizes where a launch's own limits come near. Tolerances as in test_gpu_drafted.py."""
import pytest
import torch

from latent_mixture_experts_bf16_amd import drafted as D
from latent_mixture_experts_bf16_amd import serving as S
from test_gpu_drafted import _i32

pytestmark = pytest.mark.gpu


def test_shared_prompt_of_more_queries_than_one_grid_dimension_holds():
    """2^26 + 2^16 queries, a wave each, are more than 2^32 threads: 1025 rows of 65536 heads on one, after a prompt of 64 tokens. All
    results against the same attention without groups, some of them, the last ones too, against 64 bits."""
    seqs, rows, heads, dim, page, T = 65, 1025, 65536, 32, 16, 64
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB of memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n = [16] * 64 + [1]
    k, v = (torch.rand((4 + seqs, page, 1, dim), generator=g, device="cuda").mul_(2).sub_(1).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[0, 1, 2, 3, 4 + b] for b in range(seqs)], dtype=torch.int32, device="cuda")
    cache = D.PagedCache(k, v, table, _i32([T] * seqs))
    first = [16 * b for b in range(seqs)] + [rows]
    q = torch.empty((rows, heads * dim), dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 64):
        q[r:r + 64] = torch.rand((min(64, rows - r), heads * dim), generator=g, device="cuda").mul_(2).sub_(1)
    out = torch.full_like(q, float("nan"))
    cache.attend(q, _i32(first), out=out, shared=S.SharedPrefix(_i32([0, seqs]), _i32([T])))
    cache.status()

    # |q|, |k|, |v| <= 1: scores' error ds, then as A <= 1 and |o| <= 1
    eps, ds = torch.finfo(torch.bfloat16).eps, dim * dim ** -0.5 * (dim + 4) * 2.0 ** -24
    most = (eps + 2 * ds + (T + 16 + 64) * 2.0 ** -24) * (1 + eps)
    plain = cache.attend(q, _i32(first))
    for r in range(0, rows, 64):
        assert ((out[r:r + 64].float() - plain[r:r + 64].float()).abs().amax() <= 2 * most).item(), r      # false of a NaN
    del plain

    K, V = (t.reshape(4 + seqs, page, dim).double().cpu() for t in (k, v))
    scale = dim ** -0.5
    for r in (0, 1, 15, 16, 511, 1023, 1024):
        b = r // 16
        seen = T + r - 16 * b + 1
        kk, vv = (torch.cat([t[:4].reshape(-1, dim), t[4 + b]])[:seen] for t in (K, V))
        for h in (0, 1, 127, 128, 32767, 65535):
            x = q[r, h * dim:(h + 1) * dim].double().cpu()
            p = torch.softmax(kk @ x * scale, 0)
            o, A = p @ vv, p @ vv.abs()
            d = float((kk.abs() @ x.abs()).amax()) * scale * (dim + 4) * 2.0 ** -24
            tol = (A * (eps / 2 + 2 * d + (seen + 64) * 2.0 ** -24) + eps / 2 * o.abs()) * (1 + eps)
            got = out[r, h * dim:(h + 1) * dim].double().cpu()
            assert ((got - o).abs() <= tol).all(), (r, h)
