"""Sampling where a border of a cut, or the draw, falls exactly between two equal logits.

n logits hold the row's largest value, all others weigh nothing: each of the n weighs exactly 1, so top-p of top_p leaves the
first ceil(top_p n) of them, and the draw of u over m is the one with number floor(u m). Both are whole-number arithmetic (a float times
a whole number below 2^21 has at most 45 digits), with no tolerance. log p is -log(n), to fp32.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from latent_mixture_experts_bf16_amd import serving as S
from test_gpu_drafted import TYPES

pytestmark = pytest.mark.gpu

LOGITS = {"f32": torch.float32, **TYPES}
VALUES = [0.0, 0.75, 1.0, 2.0, 2.5, 3.875, 5.0, 7.5, 10.0, 12.0, 20.0, -0.375, -6.5, 0.0625]
TEMPERATURES = [None, 0.7, 1.3, 0.05, 3.0, 50.0, 1e-4, 1e8]
PARTS = [0.25, 0.5, 0.75]


def _want(at, u, top_p, top_k):
    n = min(len(at), top_k) if top_k > 0 else len(at)
    if top_p < 1:
        n = min(n, max(1, math.ceil(Fraction(float(np.float32(top_p))) * n)))
    return at[math.floor(Fraction(float(np.float32(u))) * n)]


def _check(V, at, rest, values, temperature, cuts, dtype):
    """A row for each (value, u, top_p, top_k); `rest` in all other places."""
    rows = [(z, *c) for z in values for c in cuts]
    z = torch.full((len(rows), V), rest, dtype=torch.float64, device="cuda").to(LOGITS[dtype])
    z[:, torch.tensor(at, device="cuda")] = torch.tensor([r[0] for r in rows], device="cuda").to(LOGITS[dtype])[:, None]
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    s = S.Sampler(V, max_rows=len(rows))
    T = None if temperature is None else torch.full((len(rows),), temperature, **f32)
    tokens, logp = s.sample(z, torch.tensor([r[1] for r in rows], **f32), temperature=T,
                            top_p=torch.tensor([r[2] for r in rows], **f32), top_k=torch.tensor([r[3] for r in rows], **i32))
    s.status()
    want = [_want(at, *r[1:]) for r in rows]
    bad = [(r, a, b) for r, a, b in zip(rows, tokens.tolist(), want) if a != b]
    assert not bad, (len(bad), len(rows), bad[:5])
    assert np.allclose(logp.cpu().numpy(), -math.log(len(at)), rtol=2.0 ** -22, atol=2.0 ** -22)


@pytest.mark.parametrize("dtype", list(LOGITS))
@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("n", [2, 4, 6, 64])
def test_borders_between_few_equal_logits(n, temperature, dtype):
    """In one chunk of the vocabulary and spread over several, beside -infinity; with and without top-k."""
    cuts = [(u, p, k) for u in [0.0] + PARTS for p in PARTS + [1.0] for k in (0, 2, n)]
    for V, at in ((5000, list(range(7, 7 + n))), (20011, [13 + i * (19900 // n) for i in range(n)])):
        _check(V, at, -float("inf"), VALUES, temperature, cuts, dtype)


@pytest.mark.parametrize("dtype", list(LOGITS))
@pytest.mark.parametrize("rest", [-1e4, "lowest", 0.0])
def test_borders_beside_logits_that_weigh_nothing(rest, dtype):
    """The rest at finite numbers: a mask's, or far below (60 octaves and more at a temperature of 1 / 10), or kept out by top-k
    alone."""
    cuts = [(u, p, 0) for u in PARTS for p in PARTS + [1.0]]
    rest = torch.finfo(LOGITS[dtype]).min if rest == "lowest" else rest
    _check(9001, [0, 1, 4095, 4096, 8999, 9000], rest, [5.0, 7.5, 12.0, 20.0], 0.1, cuts, dtype)


@pytest.mark.parametrize("dtype", list(LOGITS))
@pytest.mark.parametrize("n", [16384, 131072])
def test_borders_between_many_equal_logits(n, dtype):
    """Whole rows of equal logits, and every eighth of a row."""
    cuts = [(u, p, k) for u in PARTS + [1 / 128, 127 / 128] for p in (0.5, 1.0) for k in (0, 4096)]
    at = list(range(0, 131072, 131072 // n))
    for T in (None, 0.7):
        _check(131072, at, -float("inf"), [0.75, 5.0, 7.5], T, cuts, dtype)


@pytest.mark.parametrize("dtype", list(LOGITS))
def test_borders_between_equal_logits_of_a_top_k(dtype):
    """The largest ones are equal, and others little below them are cut by top-k alone."""
    V, at = 6000, [5, 900, 4500, 5999]
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    cuts = [(u, p) for u in PARTS for p in PARTS + [1.0]]
    for value in VALUES:
        z = torch.full((len(cuts), V), value - 0.25, device="cuda").to(LOGITS[dtype])
        z[:, at] = torch.tensor(value, device="cuda").to(LOGITS[dtype])
        s = S.Sampler(V, max_rows=len(cuts))
        tokens, _ = s.sample(z, torch.tensor([c[0] for c in cuts], **f32), top_p=torch.tensor([c[1] for c in cuts], **f32),
                             top_k=torch.full((len(cuts),), 4, **i32))
        assert tokens.tolist() == [_want(at, u, p, 4) for u, p in cuts], value
