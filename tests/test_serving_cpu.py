"""The served batch's C ABI and its Python classes without a GPU: the library exports what include/moe_serving.h declares,
and every bad argument is refused by name before a device is touched."""
import ctypes
import math
import os
import re

import pytest
import torch

from latent_mixture_experts_bf16_amd import binding as B
from latent_mixture_experts_bf16_amd import drafted as D
from latent_mixture_experts_bf16_amd import serving as S
from test_drafted_cpu import FAKE, F16, F32, BF, I32, T, _cache, _refused, _says

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U8 = B.MOE_DT_U8
FAR = 0x400000


def test_library_exports_every_declared_function():
    with open(os.path.join(ROOT, "include", "moe_serving.h")) as f:
        declared = sorted(set(re.findall(r"^\w[\w ]*\b(moe_\w+)\(", f.read(), re.M)))
    assert declared == sorted(B.SERVING)
    for name in declared:
        assert hasattr(B.lib(), name), name


def _mx(**over):
    c = B.moe_mx_cache()
    shape = over.pop("shape", [4, 16, 2, 64])
    scales = over.pop("scales", shape[:3] + [max(1, shape[3] // 32)])
    for name, s in (("k", shape), ("v", shape), ("k_scale", scales), ("v_scale", scales)):
        setattr(c, name, over.pop(name, T(FAKE, U8, s)))
    c.table = over.pop("table", T(FAKE, I32, [3, 5]))
    c.len = over.pop("len", T(FAKE, I32, [3]))
    c.flags = over.pop("flags", FAKE)
    c.format = over.pop("format", B.MOE_MX8)
    c.dtype = over.pop("dtype", BF)
    assert not over
    return c


@pytest.mark.parametrize("over,status,text", [
    (dict(format=0), "MOE_ERR_INVALID_ARG", "format 0"),
    (dict(format=3), "MOE_ERR_INVALID_ARG", "format 3"),
    (dict(dtype=F32), "MOE_ERR_DTYPE", "cache: dtype f32"),
    (dict(k=T(0, U8, [4, 16, 2, 64])), "MOE_ERR_MISSING_TENSOR", "cache k"),
    (dict(v=T(FAKE, BF, [4, 16, 2, 64])), "MOE_ERR_DTYPE", "cache v: dtype bf16"),
    (dict(k_scale=T(FAKE, F32, [4, 16, 2, 2])), "MOE_ERR_DTYPE", "cache k_scale"),
    (dict(v_scale=T(FAKE, U8, [4, 16, 4])), "MOE_ERR_LAYOUT", "cache v_scale: rank 3"),
    (dict(shape=[4, 8, 2, 64]), "MOE_ERR_SHAPE", "page of 8"),
    (dict(shape=[4, 16, 2, 80]), "MOE_ERR_SHAPE", "head width 80"),
    (dict(shape=[4, 16, 2, 160]), "MOE_ERR_SHAPE", "head width 160"),
    (dict(shape=[4, 16, 2, 256], format=B.MOE_MX4), "MOE_ERR_SHAPE", "head width 512"),
    (dict(shape=[4, 16, 2, 64], format=B.MOE_MX4), "MOE_ERR_SHAPE", "k_scale: dim 3 is 2, expected 4"),
    (dict(scales=[4, 16, 2, 3]), "MOE_ERR_SHAPE", "k_scale: dim 3 is 3"),
    (dict(v_scale=T(FAKE, U8, [4, 16, 1, 2])), "MOE_ERR_SHAPE", "v_scale: dim 2 is 1"),
    (dict(v=T(FAKE, U8, [5, 16, 2, 64])), "MOE_ERR_SHAPE", "cache v: dim 0"),
    (dict(k=T(FAKE + 8, U8, [4, 16, 2, 64])), "MOE_ERR_LAYOUT", "16-byte"),
    (dict(k=T(FAKE, U8, [4, 16, 2, 64], [2112, 132, 64, 1])), "MOE_ERR_LAYOUT", "stride[1]"),
    (dict(k=T(FAKE, U8, [4, 16, 2, 64], [2048, 128, 32, 1])), "MOE_ERR_LAYOUT", "overlap"),
    (dict(k=T(FAKE, U8, [4, 16, 2, 64], [2048, 64, 64, 1])), "MOE_ERR_LAYOUT", "overlap"),
    (dict(v_scale=T(FAKE, U8, [4, 16, 2, 2], [32, 2, 16, 1])), "MOE_ERR_LAYOUT", "overlap"),
    (dict(k_scale=T(FAKE, U8, [4, 16, 2, 2], [64, 4, 2, 4])), "MOE_ERR_LAYOUT", "last dim"),
    (dict(table=T(FAKE, I32, [3, 5], [1, 3])), "MOE_ERR_LAYOUT", "cache table"),
    (dict(len=T(FAKE, I32, [2])), "MOE_ERR_SHAPE", "cache len"),
    (dict(flags=0), "MOE_ERR_INVALID_ARG", "flags"),
])
def test_mx_cache_refusals(over, status, text):
    c = _mx(**over)
    _says(B.lib().moe_mx_cache_check(ctypes.byref(c)), status, text)
    assert B.lib().moe_mx_attend_workspace(ctypes.byref(c), 0, 1, 4) < 0


def test_mx_caches_that_are_taken():
    for shape, f in (([4, 16, 2, 64], 1), ([1, 48, 1, 96], 1), ([7, 256, 8, 128], 2), ([2, 16, 3, 16], 2)):
        dim = shape[3] * f
        assert B.lib().moe_mx_cache_check(ctypes.byref(_mx(shape=shape, scales=shape[:3] + [dim // 32], format=f))) == 0
    apart = T(FAKE, U8, [4, 16, 2, 64], [2048, 64, 1024, 1])
    scales = T(FAKE + 1, U8, [4, 16, 2, 2], [64, 2, 32, 1])
    assert B.lib().moe_mx_cache_check(ctypes.byref(_mx(k=apart, v=apart, k_scale=scales, v_scale=scales))) == 0


def _append(mx, norm=None, rope=None, rows=2, q=FAKE, qs=256, heads=4, k=FAKE + 0x10000, ks=128, v=FAKE + 0x20000, vs=128,
            starts=FAKE, pos=None, out=FAKE + 0x30000, os_=256):
    c = _mx() if mx else _cache()
    f = B.lib().moe_mx_append if mx else B.lib().moe_norm_rope_append
    rope = rope or B.moe_rope(FAKE, 32, B.MOE_ROPE_HALF, 1.0)
    return f(ctypes.byref(c), norm and ctypes.byref(norm), ctypes.byref(rope), rows, q, qs, heads, k, ks, v, vs, starts, pos, out,
             os_, None)


def _norm(q=FAKE, k=FAKE, qs=64, ks=64, dtype=BF, eps=1e-6, offset=0.0):
    return B.moe_head_norm(q, k, qs, ks, dtype, eps, offset)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("over,status,text", [
    (dict(rows=0), "MOE_ERR_ROWS", "rows 0"),
    (dict(heads=3, qs=192, os_=192), "MOE_ERR_SHAPE", "3 heads"),
    (dict(norm=_norm(q=None)), "MOE_ERR_INVALID_ARG", "norm q_weight"),
    (dict(norm=_norm(k=FAKE + 1)), "MOE_ERR_LAYOUT", "norm k_weight"),
    (dict(norm=_norm(q=FAKE + 2, dtype=F32)), "MOE_ERR_LAYOUT", "norm q_weight"),
    (dict(norm=_norm(dtype=I32)), "MOE_ERR_DTYPE", "norm: dtype i32"),
    (dict(norm=_norm(qs=63)), "MOE_ERR_LAYOUT", "norm: row stride 63"),
    (dict(norm=_norm(ks=-64)), "MOE_ERR_LAYOUT", "norm: row stride -64"),
    (dict(norm=_norm(eps=-1e-6)), "MOE_ERR_INVALID_ARG", "norm: eps"),
    (dict(norm=_norm(eps=math.nan)), "MOE_ERR_INVALID_ARG", "norm: eps"),
    (dict(norm=_norm(offset=math.inf)), "MOE_ERR_INVALID_ARG", "offset"),
    (dict(rope=B.moe_rope(FAKE, 33, 1, 1.0)), "MOE_ERR_SHAPE", "33 pairs"),
    (dict(qs=255), "MOE_ERR_LAYOUT", "q: row stride"),
    (dict(pos=FAKE + 2), "MOE_ERR_LAYOUT", "positions"),
    (dict(out=FAKE + 2), "MOE_ERR_ALIAS", "q_out partially"),
    (dict(out=FAKE + 0x10000), "MOE_ERR_ALIAS", "q_out overlaps k"),
    (dict(rope=B.moe_rope(FAKE, 32, 2, 1.0), q=FAKE + 2), "MOE_ERR_LAYOUT", "interleaved"),
])
def test_append_refusals(mx, over, status, text):
    _says(_append(mx, **over), status, text)


@pytest.mark.parametrize("over,status,text", [
    (dict(rows=0), "MOE_ERR_ROWS", "rows 0"),
    (dict(starts=None), "MOE_ERR_INVALID_ARG", "row_start"),
    (dict(start=FAKE + 2), "MOE_ERR_LAYOUT", "start"),
    (dict(k=FAKE + 8), "MOE_ERR_LAYOUT", "k_out: pointer"),
    (dict(vs=120), "MOE_ERR_LAYOUT", "v_out: row stride"),
    (dict(ks=132), "MOE_ERR_LAYOUT", "k_out: pointer and row stride"),
    (dict(v=FAKE), "MOE_ERR_ALIAS", "k_out overlaps v_out"),
])
def test_read_refusals(over, status, text):
    def call(rows=2, starts=FAKE, start=None, k=FAKE, ks=128, v=FAKE + FAR, vs=128):
        return B.lib().moe_mx_read(ctypes.byref(_mx()), rows, starts, start, k, ks, v, vs, None)
    _says(call(**over), status, text)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("over,status,text", [
    (dict(rows=0), "MOE_ERR_ROWS", "rows"),
    (dict(q=FAKE + 8), "MOE_ERR_LAYOUT", "q: pointer"),
    (dict(mask=FAKE + 4), "MOE_ERR_LAYOUT", "mask"),
    (dict(scale=math.nan), "MOE_ERR_INVALID_ARG", "scale"),
    (dict(out=FAKE), "MOE_ERR_ALIAS", "out overlaps q"),
    (dict(shared=B.moe_shared_prefix(None, FAKE, 1)), "MOE_ERR_INVALID_ARG", "shared group_start"),
    (dict(shared=B.moe_shared_prefix(FAKE, FAKE + 2, 1)), "MOE_ERR_LAYOUT", "shared len"),
    (dict(shared=B.moe_shared_prefix(FAKE, FAKE, 0)), "MOE_ERR_SHAPE", "0 groups"),
    (dict(shared=B.moe_shared_prefix(FAKE, FAKE, 4)), "MOE_ERR_SHAPE", "4 groups"),
    (dict(ws=None), "MOE_ERR_INVALID_ARG", "workspace: NULL"),
    (dict(ws=FAKE + 8), "MOE_ERR_LAYOUT", "workspace"),
    (dict(short=1), "MOE_ERR_SHAPE", "needed"),
])
def test_attend_refusals(mx, over, status, text):
    c = _mx() if mx else _cache()
    f, size = ((B.lib().moe_mx_attend, B.lib().moe_mx_attend_workspace) if mx else
               (B.lib().moe_shared_attend, B.lib().moe_shared_attend_workspace))

    def call(shared=B.moe_shared_prefix(FAKE, FAKE, 2), rows=2, q=FAKE, mask=None, scale=0.1, out=FAKE + FAR, ws=FAKE, short=0):
        need = max(size(ctypes.byref(c), 2, max(rows, 1), 4), 0)
        return f(ctypes.byref(c), ctypes.byref(shared), rows, q, 256, 4, FAKE, mask, scale, out, 256, ws, need - short, None)
    _says(call(**over), status, text)


def test_workspaces():
    lib = B.lib()
    for c, size in ((_cache(), lib.moe_shared_attend_workspace), (_mx(), lib.moe_mx_attend_workspace)):
        assert 0 < size(ctypes.byref(c), 0, 7, 4) < size(ctypes.byref(c), 1, 7, 4) <= size(ctypes.byref(c), 1, 70, 4)
        assert size(ctypes.byref(c), 4, 7, 4) < 0 and size(ctypes.byref(c), -1, 7, 4) < 0 and size(ctypes.byref(c), 1, 0, 4) < 0
    assert lib.moe_shared_attend_workspace(ctypes.byref(_cache()), 0, 7, 4) == lib.moe_tree_attend_workspace(ctypes.byref(_cache()), 7, 4)
    _says(lib.moe_shared_attend(ctypes.byref(_cache()), None, 2, FAKE, 256, 4, FAKE, None, 0.1, FAKE + FAR, 256, FAKE, 1 << 30, None),
          "MOE_ERR_INVALID_ARG", "shared: NULL")
    assert 0 < lib.moe_sample_workspace(1, 1) < lib.moe_sample_workspace(2, 5000)
    for rows, vocab in ((0, 5), (1, 0), (1, (1 << 20) + 1), ((1 << 20) + 1, 5)):
        assert lib.moe_sample_workspace(rows, vocab) < 0


def test_keep_refusals():
    c = _mx()
    call = lambda *a: B.lib().moe_mx_keep(ctypes.byref(c), *a, None)  # noqa: E731
    _says(call(FAKE, 0, FAKE, FAKE, FAKE), "MOE_ERR_ROWS", "rows")
    _says(call(FAKE, 4, FAKE + 1, FAKE, FAKE), "MOE_ERR_LAYOUT", "n_keep")
    _says(call(FAKE, 4, FAKE, None, FAKE), "MOE_ERR_INVALID_ARG", "path")


@pytest.mark.parametrize("over,status,text", [
    (dict(z=T(0, F32, [4, 1000])), "MOE_ERR_MISSING_TENSOR", "logits"),
    (dict(z=T(FAKE, I32, [4, 1000])), "MOE_ERR_DTYPE", "logits"),
    (dict(z=T(FAKE, F32, [4000])), "MOE_ERR_LAYOUT", "rank 1"),
    (dict(z=T(FAKE, F32, [4, (1 << 20) + 1])), "MOE_ERR_SHAPE", "vocabulary"),
    (dict(z=T(FAKE, F32, [0, 1000])), "MOE_ERR_ROWS", "rows 0"),
    (dict(z=T(FAKE, F32, [4, 1000], [999, 1])), "MOE_ERR_LAYOUT", "strides"),
    (dict(z=T(FAKE + 2, F32, [4, 1000])), "MOE_ERR_LAYOUT", "logits"),
    (dict(u=None), "MOE_ERR_INVALID_ARG", "u: NULL"),
    (dict(t=FAKE + 2), "MOE_ERR_LAYOUT", "temperature"),
    (dict(k=FAKE + 2), "MOE_ERR_LAYOUT", "top_k"),
    (dict(p=FAKE + 2), "MOE_ERR_LAYOUT", "top_p"),
    (dict(m=FAKE + 2), "MOE_ERR_LAYOUT", "min_p"),
    (dict(tokens=None), "MOE_ERR_INVALID_ARG", "tokens"),
    (dict(lp=None), "MOE_ERR_INVALID_ARG", "logprobs"),
    (dict(flags=None), "MOE_ERR_INVALID_ARG", "flags"),
    (dict(ws=None), "MOE_ERR_INVALID_ARG", "workspace"),
    (dict(ws=FAKE + 4), "MOE_ERR_LAYOUT", "workspace"),
    (dict(wsb=100), "MOE_ERR_SHAPE", "needed"),
])
def test_sample_refusals(over, status, text):
    def call(z=None, u=FAKE, t=None, k=None, p=None, m=None, tokens=FAKE, lp=FAKE, flags=FAKE, ws=FAKE, wsb=1 << 30):
        z = z or T(FAKE, F32, [4, 1000])
        return B.lib().moe_sample(ctypes.byref(z), u, t, k, p, m, tokens, lp, flags, ws, wsb, None)
    _says(call(**over), status, text)


# ------------------------------------------------------------------ the Python classes, on host tensors

def _table():
    return torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)


def test_python_caches_of_codes():
    for f, dim in (("mx8", 64), ("mx4", 128), ("mx4", 32), ("mx8", 256)):
        c = S.mx_cache(4, 16, 2, dim, *_table(), format=f, dtype=torch.float16)
        assert c.k.shape == (4, 16, 2, dim if f == "mx8" else dim // 2) and c.v_scale.shape == (4, 16, 2, dim // 32)
        assert c.k[1, :, 1].is_contiguous() and c.k_scale[1, :, 1].is_contiguous()      # a head's tokens of a page
        assert (c.dim, c.kv_heads, c.seqs, c.dtype, c.format) == (dim, 2, 3, torch.float16, f)
    _refused("MOE_ERR_INVALID_ARG", "format", S.mx_cache, 4, 16, 2, 64, *_table(), format="int8")
    _refused("MOE_ERR_SHAPE", "head width 80", S.mx_cache, 4, 16, 2, 80, *_table())
    _refused("MOE_ERR_SHAPE", "head width 160", S.mx_cache, 4, 16, 2, 160, *_table())
    _refused("MOE_ERR_DTYPE", "cache: dtype", S.mx_cache, 4, 16, 2, 64, *_table(), dtype=torch.float32)
    c = S.mx_cache(4, 16, 2, 64, *_table())
    _refused("MOE_ERR_SHAPE", "k_scale", S.MxCache, c.k, c.v, c.k_scale[..., :1], c.v_scale, c.table, c.length)
    _refused("MOE_ERR_DTYPE", "cache v", S.MxCache, c.k, c.v.to(torch.int32), c.k_scale, c.v_scale, c.table, c.length)
    q, kv = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    starts, rope = torch.tensor([0, 1, 2, 4], dtype=torch.int32), D.Rope([1.0] * 32, device="cpu")
    _refused("MOE_ERR_DEVICE", "GPU", c.append, rope, q, kv, kv, starts)
    _refused("MOE_ERR_DEVICE", "GPU", c.attend, q, starts)
    _refused("MOE_ERR_DEVICE", "GPU", c.read, starts, 4)
    _refused("MOE_ERR_DEVICE", "GPU", c.keep, starts, torch.ones(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    _refused("MOE_ERR_DTYPE", "q:", c.attend, q.half(), starts)
    _refused("MOE_ERR_SHAPE", "start:", c.read, starts, 4, start=torch.zeros(2, dtype=torch.int32))
    _refused("MOE_ERR_SHAPE", "out v", c.read, starts, 4, out=(kv, kv[:3]))


def test_python_norms():
    c = D.PagedCache(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), *_table())
    q, kv = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    starts, rope = torch.tensor([0, 1, 2, 4], dtype=torch.int32), D.Rope([1.0] * 32, device="cpu")
    one = torch.ones(64)
    _refused("MOE_ERR_DTYPE", "k_weight", S.HeadNorm, one, one.half())
    _refused("MOE_ERR_DTYPE", "q_weight", S.HeadNorm, one.double(), one.double())
    _refused("MOE_ERR_LAYOUT", "q_weight", S.HeadNorm, one[None, None], one)
    _refused("MOE_ERR_LAYOUT", "k_weight", S.HeadNorm, one, torch.ones(64, 2).T)
    _refused("MOE_ERR_INVALID_ARG", "eps", S.HeadNorm, one, one, eps=-1.0)
    _refused("MOE_ERR_INVALID_ARG", "offset", S.HeadNorm, one, one, offset=math.nan)
    for bad, text in ((S.HeadNorm(one[:32], one), "q_weight"), (S.HeadNorm(one, torch.ones(4, 64)), "k_weight"),
                      (S.HeadNorm(torch.ones(3, 64), one), "q_weight")):
        _refused("MOE_ERR_SHAPE", text, c.append, rope, q, kv, kv, starts, norm=bad)
    _refused("MOE_ERR_DEVICE", "GPU", c.append, rope, q, kv, kv, starts, norm=S.HeadNorm(torch.ones(4, 64), torch.ones(2, 64)))


def test_python_shared_prefixes():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    _refused("MOE_ERR_DTYPE", "group_start", S.SharedPrefix, torch.tensor([0, 3]), i32(5))
    _refused("MOE_ERR_DTYPE", "length", S.SharedPrefix, i32(0, 3), torch.tensor([5]))
    _refused("MOE_ERR_SHAPE", "starts of 2 groups", S.SharedPrefix, i32(0, 3), i32(5, 5))
    _refused("MOE_ERR_SHAPE", "starts of 0 groups", S.SharedPrefix, i32(0), i32())
    _refused("MOE_ERR_LAYOUT", "group_start", S.SharedPrefix, i32(0, 1, 3, 9)[::2], i32(5))
    c = D.PagedCache(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), *_table())
    q, starts = torch.zeros(4, 256, dtype=torch.bfloat16), i32(0, 1, 2, 4)
    _refused("MOE_ERR_SHAPE", "4 groups, 3 sequences", c.attend, q, starts, shared=S.SharedPrefix(i32(0, 1, 2, 3, 3), i32(1, 1, 1, 1)))
    _refused("MOE_ERR_DEVICE", "GPU", c.attend, q, starts, shared=S.SharedPrefix(i32(0, 3), i32(5)))


def test_python_sampler():
    s = S.Sampler(1000, max_rows=4, device="cpu")
    z, u = torch.zeros(4, 1000), torch.zeros(4)
    _refused("MOE_ERR_DEVICE", "GPU", s.sample, z, u)
    _refused("MOE_ERR_LAYOUT", "rank 1", s.sample, z[0], u)
    _refused("MOE_ERR_ROWS", "5 rows", s.sample, torch.zeros(5, 1000), u)
    _refused("MOE_ERR_ROWS", "0 rows", s.sample, z[:0], u[:0])
    _refused("MOE_ERR_DTYPE", "logits", s.sample, z.double(), u)
    _refused("MOE_ERR_SHAPE", "logits", s.sample, z[:, :999], u)
    _refused("MOE_ERR_LAYOUT", "columns", s.sample, torch.zeros(1000, 4).T, u)
    _refused("MOE_ERR_DTYPE", "u:", s.sample, z, u.double())
    _refused("MOE_ERR_SHAPE", "u:", s.sample, z, u[:3])
    _refused("MOE_ERR_DTYPE", "top_k", s.sample, z, u, top_k=torch.ones(4, dtype=torch.int64))
    _refused("MOE_ERR_SHAPE", "top_p", s.sample, z, u, top_p=torch.ones(1))
    _refused("MOE_ERR_LAYOUT", "min_p", s.sample, z, u, min_p=torch.ones(8)[::2])
    _refused("MOE_ERR_DTYPE", "temperature", s.sample, z, u, temperature=torch.ones(4, dtype=torch.float16))
    _refused("MOE_ERR_SHAPE", "vocabulary", S.Sampler, 0, 4, device="cpu")
    _refused("MOE_ERR_ROWS", "rows", S.Sampler, 1000, 0, device="cpu")
