"""The drafted decode example against plain decoding of the same model: the cache after many accepted paths
holds what one row a step would have written, and every token is the one plain decoding would say.

Both sides round activations to bf16 about eight times between the embedding and the logits (2^-8 of the
value each, at most half of it, of random sign), and differ only in the order of fp32 sums before those
roundings: the logits agree to 8 * 2^-8 of their root mean square. A token that plain decoding would not
say must therefore come within twice that of its largest logit; keys after one projection, a rotation and
their rounding agree to a step of bf16.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("drafted_decode", os.path.join(ROOT, "examples", "drafted_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_drafted_decoding_equals_plain_decoding():
    ex = _example()
    torch.manual_seed(1)
    model = ex.Model(vocab=256, seed=3)
    prompts = [[5, 17, 200], [9], [31, 44, 7, 12, 90]]
    texts, steps = ex.decode(model, prompts, 40)
    assert all(len(t) - len(p) >= 40 for t, p in zip(texts, prompts)) and steps <= 40
    for t, p in zip(texts, prompts):
        cache = ex.new_cache(1, len(t) + 1)
        for i in range(len(t) - 1):
            z = model.step(cache, ex.i32([t[i]]), ex.i32([0, 1]), None, None)[0].double()
            cache.length.add_(1)
            if i >= len(p) - 1:
                assert float(z.max() - z[t[i + 1]]) <= 2 * 8 * 2.0 ** -8 * float(z.square().mean().sqrt()), i
        cache.status()


def test_a_sequence_ahead_of_the_others_stays_in_its_cache():
    """Sequences whose drafts are accepted more often have their tokens first; they wait for the others then."""
    ex = _example()
    torch.manual_seed(1)
    prompts = [[5, 17, 200], [9], [31, 44, 7, 12, 90]]
    texts, _ = ex.decode(ex.Model(vocab=256, seed=3), prompts, 120)
    # the last step's path has at most three accepted drafts
    assert all(120 <= len(t) - len(p) <= 123 for t, p in zip(texts, prompts))


def test_accepted_and_moved_rows_leave_what_plain_decoding_sees(monkeypatch):
    """The same over 120 tokens, in which drafts are accepted and rows that are not in their place are moved there."""
    ex = _example()
    torch.manual_seed(1)
    model, kept = ex.Model(vocab=256, seed=3), []
    keep = ex.drafted.PagedCache.keep

    def noting(self, row_start, n_keep, path, new_len=None):
        kept.append((row_start.tolist(), n_keep.tolist(), path.tolist()))
        return keep(self, row_start, n_keep, path, new_len=new_len)

    monkeypatch.setattr(ex.drafted.PagedCache, "keep", noting)
    prompts = [[5, 17, 200], [9], [31, 44, 7, 12, 90]]
    texts, steps = ex.decode(model, prompts, 120)
    # every step gives one token at least; more come from accepted drafts alone
    accepted = sum(k - 1 for _, n, _ in kept for k in n if k)
    assert accepted >= 12 and steps < 120 and steps == len(kept)
    assert sum(path[at + i] != i for start, n, path in kept for at, k in zip(start, n) for i in range(k)) > 0
    for t, p in zip(texts, prompts):
        cache = ex.new_cache(1, len(t) + 1)
        for i in range(len(t) - 1):
            z = model.step(cache, ex.i32([t[i]]), ex.i32([0, 1]), None, None)[0].double()
            cache.length.add_(1)
            if i >= len(p) - 1:
                assert float(z.max() - z[t[i + 1]]) <= 2 * 8 * 2.0 ** -8 * float(z.square().mean().sqrt()), i
        cache.status()
