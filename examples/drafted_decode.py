"""Drafted decoding over a paged cache: the operators of a drafted step beside the expert layer and the lm_head.

A small random model (embedding, one attention block, one latent mixture-of-experts layer, lm_head)
decodes several sequences at once. Each step drafts a tree of guesses after every sequence's last
token (from what followed the same token before), passes it through the model in one go, tests the
guesses against the target's probabilities and keeps the accepted path. Greedy, so the tokens are
those of plain decoding, in fewer steps:

    python examples/drafted_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from latent_mixture_experts_bf16_amd import binding as B  # noqa: E402
from latent_mixture_experts_bf16_amd import drafted, synth  # noqa: E402
from latent_mixture_experts_bf16_amd import layer as LY  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE, MOST_ROWS = 8, 2, 64, 16, 256


class Model:
    """One attention block and one expert layer over a vocabulary of `vocab` tokens, random weights."""

    def __init__(self, vocab=512, seed=0, rotary=DIM):
        dims, arrays = next(synth.workload_layers(0, rows=1))
        self.layer = LY.DeviceLayer(dims, arrays, max_rows=MOST_ROWS)
        self.vocab, self.hidden = vocab, dims.hidden
        g = torch.Generator()
        g.manual_seed(seed)
        draw = lambda *s, std: (torch.randn(s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
        self.embed = draw(vocab, self.hidden, std=1.0)
        self.qkv = draw(self.hidden, (HEADS + 2 * KV_HEADS) * DIM, std=self.hidden ** -0.5)
        self.out = draw(HEADS * DIM, self.hidden, std=(HEADS * DIM) ** -0.5)
        self.head = draw(vocab, self.hidden, std=self.hidden ** -0.5)
        self.head_desc = B.make_tensor(self.head.data_ptr(), B.MOE_DT_BF16, [vocab, self.hidden])
        self.rope = drafted.Rope(*drafted.rope_frequencies(rotary))

    def step(self, cache, tokens, row_start, positions, mask):
        """Logits [rows][vocab] (fp32) of one pass; the rows' keys and values lie in the cache after it."""
        x = self.embed[tokens.long()]
        qkv = x @ self.qkv
        at = HEADS * DIM
        q = cache.append(self.rope, qkv[:, :at], qkv[:, at:at + KV_HEADS * DIM], qkv[:, at + KV_HEADS * DIM:], row_start,
                         positions=positions)
        x = x + cache.attend(q, row_start, mask=mask) @ self.out
        y = torch.empty_like(x)
        # the layer and the lm_head run on the null stream, which waits for torch's default stream's work and is it
        self.layer.forward(x, y)
        logits = torch.empty((x.shape[0], self.vocab), device="cuda")
        B.moe_lm_head_gemv(self.head_desc, x.shape[0], y.data_ptr(), logits.data_ptr(), B.MOE_DT_F32)
        return logits


def new_cache(seqs, length):
    pages = -(-length // PAGE)
    k = torch.zeros((seqs * pages, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(seqs * pages).view(seqs, pages).to(torch.int32).cuda()
    return drafted.PagedCache(k, torch.zeros_like(k), table, torch.zeros(seqs, dtype=torch.int32, device="cuda"))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def draft_tree(text, followers, wide=2, deep=3):
    """Tokens and parents of a tree after the text's last token: `wide` guesses, the first drawn out to `deep`."""
    tokens, parents = [text[-1]], [-1]
    at = 0
    for d in range(deep):
        guesses = followers.get(tokens[at], [])[:wide]
        for g in guesses:
            tokens.append(g)
            parents.append(at)
        if not guesses:
            break
        at = len(tokens) - len(guesses)
    return tokens, parents


def decode(model, prompts, n_new):
    """Greedy continuation of each prompt by n_new tokens (a few more where the last step's drafts were accepted);
    returns the texts and the number of steps."""
    seqs = len(prompts)
    texts = [list(p) for p in prompts]
    cache = new_cache(seqs, max(map(len, texts)) + n_new + 16)
    verifier = drafted.Verifier(model.vocab, max_rows=MOST_ROWS, max_seqs=seqs)
    # the prompts but for their last tokens
    starts = [0]
    for t in texts:
        starts.append(starts[-1] + len(t) - 1)
    model.step(cache, i32([x for t in texts for x in t[:-1]]), i32(starts), None, None)
    cache.length.copy_(i32([len(t) - 1 for t in texts]))
    followers = [{} for _ in texts]
    steps = 0
    while min(len(t) - len(p) for t, p in zip(texts, prompts)) < n_new:
        tokens, parents, masks, positions, starts = [], [], [], [], [0]
        for t, p, f in zip(texts, prompts, followers):
            # a sequence that has its tokens passes no more rows while the others go on
            tok, par = draft_tree(t, f) if len(t) - len(p) < n_new else ([], [])
            tokens += tok
            parents += par
            masks += drafted.tree_masks(par)
            positions += [len(t) - 1 + d for d in drafted.tree_depths(par)]
            starts.append(len(tokens))
        rows, row_start, drafts = len(tokens), i32(starts), i32(tokens)
        logits = model.step(cache, drafts, row_start, i32(positions), torch.tensor(masks, dtype=torch.int64, device="cuda"))
        half = torch.full((rows,), 0.5, device="cuda")
        n_keep, path, said, _ = verifier.verify(logits, drafts, row_start, None, half, parent=i32(parents),
                                                temperature=torch.zeros(seqs, device="cuda"))
        cache.keep(row_start, n_keep, path)
        n_keep, said = n_keep.tolist(), said.tolist()
        for b, t in enumerate(texts):
            for x in said[starts[b]:starts[b] + n_keep[b]]:
                seen = followers[b].setdefault(t[-1], [])
                if x in seen:
                    seen.remove(x)
                seen.insert(0, x)
                t.append(x)
        steps += 1
    cache.status()
    verifier.status()
    model.layer.status()
    return texts, steps


if __name__ == "__main__":
    torch.manual_seed(0)
    m = Model()
    done, n = decode(m, [[5, 17, 200], [9], [301, 44, 7, 12, 90]], 96)
    for t in done:
        print(" ".join(map(str, t[:24])), "...")
    print(f"{sum(map(len, done)) - 9} tokens of {len(done)} sequences in {n} steps")
