"""Speculative decoding of a small random model with LoRA adapters over a paged cache.

    python examples/speculative_decode.py [--steps 12] [--temperature 0.7]

Every request has an adapter of its own on qkv.  The prompts are prefilled, the first one is
forked into a second sample that shares its pages, and each step then drafts a tree of tokens per
request, runs the model over all trees at once, verifies the drafts against the model's
distribution, and keeps the accepted tokens' keys and values.  The draft model is the same model
without its layers.  Nothing is copied to the host until the end.

With temperature 0 every emitted token is checked against the model computed densely in float32.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_gemm_amd as sgg  # noqa: E402

LAYERS, HIDDEN, HEADS, KV_HEADS, HEAD_DIM, VOCAB, MAX_LEN = 2, 256, 4, 2, 64, 1000, 512
ADAPTERS, RANK, PAGE = 4, 16, 16
OFFSETS = [0, HEADS * HEAD_DIM, (HEADS + KV_HEADS) * HEAD_DIM, (HEADS + 2 * KV_HEADS) * HEAD_DIM]
# children of each node of a level; nodes are numbered level by level
WIDTHS = (3, 2, 1)


def norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Model:
    """Random weights; ``forward`` on the cache and adapters, ``dense`` in float32 without them."""

    def __init__(self, device, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16).to(device)

        n = HIDDEN ** -0.5
        self.embed = draw(VOCAB, HIDDEN, scale=1.0)
        self.place = draw(MAX_LEN, HIDDEN, scale=0.3)
        self.qkv = draw(LAYERS, HIDDEN, OFFSETS[-1], scale=n)
        self.out = draw(LAYERS, HEADS * HEAD_DIM, HIDDEN, scale=0.3 * n)
        self.up = draw(LAYERS, HIDDEN, 2 * HIDDEN, scale=n)
        self.down = draw(LAYERS, 2 * HIDDEN, HIDDEN, scale=0.3 * n)
        self.head = draw(HIDDEN, VOCAB, scale=3 * n)
        self.lora_a = draw(LAYERS, ADAPTERS, 3 * RANK, HIDDEN, scale=n)
        self.lora_b = draw(LAYERS, ADAPTERS, OFFSETS[-1], RANK, scale=0.3)

    def draft(self, tokens, positions, temperature):
        """The draft model's probabilities after each token: the embedding straight to the head."""
        x = norm(self.embed[tokens] + self.place[positions])
        return torch.softmax((x @ self.head).float() / (temperature or 1.0), -1)

    def forward(self, lora, cache, tokens, positions, q_indptr, rows, max_q, max_kv, mask=None):
        x = self.embed[tokens] + self.place[positions]
        n = tokens.numel()
        for i in range(LAYERS):
            h = norm(x)
            qkv = lora.run_qkv_lora(h, self.lora_a[i], self.lora_b[i], OFFSETS, OFFSETS[1],
                                    h @ self.qkv[i])
            q, k, v = (y.view(n, -1, HEAD_DIM) for y in
                       (qkv[:, a:b] for a, b in zip(OFFSETS, OFFSETS[1:])))
            cache.write(i, k, v, q_indptr, rows)
            o = cache.attention(i, q, q_indptr, max_q, max_kv, tree_mask=mask, rows=rows)
            x = x + o.reshape(n, -1) @ self.out[i]
            x = x + torch.nn.functional.silu(norm(x) @ self.up[i]) @ self.down[i]
        return (norm(x) @ self.head).float()

    def dense(self, tokens, adapter, scaling):
        """Logits after every token of one sequence, float32."""
        n = len(tokens)
        x = (self.embed[tokens] + self.place[:n]).float()
        later = torch.ones(n, n, device=x.device).triu(1).bool()
        for i in range(LAYERS):
            h = norm(x)
            a, b = self.lora_a[i, adapter].float(), self.lora_b[i, adapter].float()
            parts = []
            for s, (lo, hi) in enumerate(zip(OFFSETS, OFFSETS[1:])):
                low = h @ a[s * RANK:(s + 1) * RANK].T
                y = h @ self.qkv[i, :, lo:hi].float() + scaling * (low @ b[lo:hi].T)
                parts.append(y.view(n, -1, HEAD_DIM).transpose(0, 1))
            q, k, v = parts
            k, v = (y.repeat_interleave(HEADS // KV_HEADS, 0).contiguous() for y in (k, v))
            w = (q @ k.transpose(1, 2).contiguous()) * HEAD_DIM ** -0.5
            o = torch.softmax(w.masked_fill(later, float("-inf")), -1) @ v
            x = x + o.transpose(0, 1).reshape(n, -1) @ self.out[i].float()
            x = x + torch.nn.functional.silu(norm(x) @ self.up[i].float()) @ self.down[i].float()
        return norm(x) @ self.head.float()


def tree_parents():
    """Parents of the tree's nodes, and the first node of each level."""
    parents, levels, first = [-1], [0], 0
    for width in WIDTHS:
        last = len(parents)
        levels.append(last)
        parents += [node for node in range(first, last) for _ in range(width)]
        first = last
    return parents, levels


def decode(steps=12, temperature=0.0, seed=0, device="cuda"):
    """Returns (model, sequences, prompt lengths, adapters, scalings): prompt and emitted tokens
    of every request, and the tokens emitted per step and request."""
    gen = torch.Generator(device).manual_seed(seed)
    model = Model(device, seed)
    prompts = [torch.randint(VOCAB, (n,), generator=gen, device=device) for n in (37, 5, 64, 18)]
    adapters = [0, 1, 2, 3, 0]                   # the fifth request is forked from the first
    ranks, scalings = [RANK] * ADAPTERS, [0.5, 1.0, 2.0, 1.0]
    parents, levels = tree_parents()
    T, depth, bs = len(parents), len(WIDTHS), len(adapters)
    longest = max(len(p) for p in prompts) + steps * (depth + 1) + T
    pages = -(-longest // PAGE)
    cache = sgg.PagedKVCache(LAYERS, bs * pages, PAGE, KV_HEADS, HEAD_DIM, bs, pages,
                             device=device)
    lora = sgg.ChunkedSgmvLoRA(ADAPTERS, 128, device)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    # prefill: all tokens but the last, which is the first tree's root
    held = [len(p) - 1 for p in prompts]
    first = i32(list(range(len(prompts))))
    missing = [cache.reserve(first, i32(held))]
    lora.prepare_lora_batch(held, adapters[:-1], ranks, scalings)
    model.forward(lora, cache, torch.cat([p[:-1] for p in prompts]),
                  torch.cat([torch.arange(n, device=device) for n in held]),
                  i32([0] + torch.tensor(held).cumsum(0).tolist()), first, max(held), max(held))
    cache.commit(first, i32(held))
    missing.append(cache.fork(i32([0]), i32([bs - 1])))

    rows = i32(list(range(bs)))
    q_indptr = i32([T * r for r in range(bs + 1)])
    tree = i32(parents * bs)
    root = torch.stack([p[-1] for p in prompts] + [prompts[0][-1]])
    lora.prepare_lora_batch([T] * bs, adapters, ranks, scalings)
    emitted, counts = [], []
    for _ in range(steps):
        missing.append(cache.reserve(rows, cache.kv_lens + T))
        mask, positions = sgg.spec_tree_mask(tree, q_indptr, cache.kv_lens, 1, rows)
        at = positions.long().view(bs, T)
        # the drafts, level by level
        tokens = torch.zeros((bs, T), dtype=torch.int64, device=device)
        tokens[:, 0] = root
        probs = torch.zeros((bs, T, VOCAB), device=device)
        for level, width in enumerate(WIDTHS):
            a, b = levels[level], levels[level + 1]
            probs[:, a:b] = p = model.draft(tokens[:, a:b], at[:, a:b], temperature)
            flat = p.reshape(-1, VOCAB)
            pick = torch.multinomial(flat, width, replacement=True, generator=gen) \
                if temperature else flat.topk(width).indices
            tokens[:, b:b + (b - a) * width] = pick.view(bs, -1)
        logits = model.forward(lora, cache, tokens.view(-1), at.view(-1), q_indptr, rows, T,
                               longest, mask)
        target = torch.softmax(logits / temperature, -1) if temperature else \
            torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()
        coins = torch.rand(bs * T + bs, generator=gen, device=device)
        path, accepted, root32 = sgg.spec_verify(
            tokens.view(-1).int(), tree, q_indptr, target, coins[:bs * T], coins[bs * T:],
            depth + 1, draft_probs=probs.view(-1, VOCAB) if temperature else None)
        cache.commit(rows, cache.compact(path, accepted, rows))
        root = root32.long()
        # the accepted drafts (the root was emitted before), then the model's own next token
        got = tokens.gather(1, path.clamp(min=0).long())
        got = torch.cat([got[:, 1:], got.new_zeros(bs, 1)], 1)
        emitted.append(got.scatter(1, accepted.long().view(-1, 1) - 1, root.view(-1, 1)))
        counts.append(accepted)
    assert not torch.stack(missing).any(), "the cache has no page left"
    counts = torch.stack(counts, 1).tolist()
    tokens = torch.stack(emitted, 1).tolist()
    sequences = [(prompts + prompts[:1])[r].tolist() +
                 [t for step, n in zip(tokens[r], counts[r]) for t in step[:n]]
                 for r in range(bs)]
    starts = [len(p) for p in prompts + prompts[:1]]
    return model, sequences, starts, [(a, scalings[a]) for a in adapters], counts


def behind(model, sequence, start, adapter, scaling):
    """How far, in standard deviations of the logits, the emitted tokens' logits lie behind the
    largest ones in float32 (0: the same choice)."""
    tokens = torch.tensor(sequence, device=model.embed.device)
    logits = model.dense(tokens[:-1], adapter, scaling)[start - 1:]
    mine = logits.gather(1, tokens[start:].view(-1, 1))[:, 0]
    return ((logits.amax(-1) - mine) / logits.std(-1)).max().item()


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=12)
    parser.add_argument("--temperature", type=float, default=0.0)
    args = parser.parse_args()
    model, sequences, starts, adapters, counts = decode(args.steps, args.temperature)
    for r, (seq, start, n) in enumerate(zip(sequences, starts, counts)):
        line = f"request {r}: {len(seq) - start} tokens in {len(n)} steps"
        if not args.temperature:
            line += f", at most {behind(model, seq, start, *adapters[r]):.3f} behind the largest"
        print(line + f": {' '.join(map(str, seq[start:start + 12]))} ..")


if __name__ == "__main__":
    main()
