"""Generation from a one-layer decoder with a 4-bit key-value cache.

Prompts of different lengths enter a paged cache in one call (cache_extend:
heads normed and rotated, rows rounded to 4 bits with a scale every 32
elements); from then on each step extends every sequence by a token, attends
over the cache (cache_attend), and draws the next token from the logits
(sample).  Where a cache has reached its budget it is cut back to the slots
that have drawn the most attention (cache_evict).  A step can be captured into
a graph once and replayed.  Weights are random: what is shown is how the calls
fit together, not text.

    python examples/generate.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_selection_two_amd as ltk  # noqa: E402

PAGE, SINKS, RECENT = 16, 4, 16


class Decoder:
    """Embedding, one attention layer, and a head."""

    def __init__(self, vocab, heads, group, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            x = torch.randn(rows, cols, generator=g, device="cuda")
            return (x / cols ** 0.5).to(torch.bfloat16)

        self.heads, self.q_heads, self.dim = heads, heads * group, dim
        wide = self.q_heads * dim
        self.embedding = weight(vocab, wide) * wide ** 0.5
        self.project = weight((self.q_heads + 2 * heads) * dim, wide)
        self.back = weight(wide, wide)
        self.head = weight(vocab, wide) * 3
        self.q_norm = torch.ones(dim, device="cuda")
        self.k_norm = torch.ones(dim, device="cuda")
        self.freqs = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda",
                                               dtype=torch.float32) / dim)

    def projected(self, tokens):
        """Rows of the tokens [N] and their heads: q, k, v [N, ., dim], all
        slices of one array."""
        x = self.embedding[tokens]
        y = (x @ self.project.t()).view(len(tokens), -1, self.dim)
        return (x, *y.split([self.q_heads, self.heads, self.heads], 1))

    def logits(self, x, out):
        return (x + out.flatten(1) @ self.back.t()) @ self.head.t()


class Cache:
    """Paged 4-bit rows, their scales, and a weight and position a slot."""

    def __init__(self, batch, heads, dim, slots):
        width = -(-slots // PAGE)
        size = (batch * width, heads, PAGE)

        def rows():
            return torch.zeros(*size, dim // 2, dtype=torch.uint8,
                               device="cuda").view(torch.float4_e2m1fn_x2)

        def blocks():
            return torch.zeros(*size, dim // 32,
                               dtype=torch.uint8,
                               device="cuda").view(torch.float8_e8m0fnu)

        self.k, self.v = rows(), rows()
        self.k_blocks, self.v_blocks = blocks(), blocks()
        self.table = torch.arange(batch * width, dtype=torch.int32,
                                  device="cuda").view(batch, width)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.seen = torch.zeros_like(self.lens)  # tokens so far
        self.weights = torch.zeros(batch, heads, width * PAGE, device="cuda")
        self.positions = torch.zeros_like(self.weights, dtype=torch.int32)

    def extend(self, model, q, k, v, starts):
        """The heads of new tokens enter; the queries are turned in place."""
        lens, _ = ltk.cache_extend(
            k, v, self.k, self.v, self.table, self.lens, starts,
            seen=self.seen, q=q, freqs=model.freqs, q_norm=model.q_norm,
            k_norm=model.k_norm, weights=self.weights,
            positions=self.positions, k_blocks=self.k_blocks,
            v_blocks=self.v_blocks, out=q)
        self.lens.copy_(lens)
        self.seen += starts[1:] - starts[:-1]
        return q

    def attend(self, q):
        return ltk.cache_attend(q, self.k, self.v, self.table, self.lens,
                                weights=self.weights, k_blocks=self.k_blocks,
                                v_blocks=self.v_blocks)[0]

    def evict(self, keep):
        weights, positions, lens = ltk.cache_evict(
            self.k, self.v, self.table, self.lens, self.seen, self.weights,
            self.positions, keep, sinks=SINKS, recent=RECENT,
            k_blocks=self.k_blocks, v_blocks=self.v_blocks)
        self.weights[..., :keep] = weights
        self.positions[..., :keep] = positions
        self.lens.copy_(lens)


def generate(model, prompts, steps, budget, graph=False, seed=1, top_k=50,
             top_p=0.95, temperature=0.8):
    """Tokens [steps, B] after the prompts (lists of tokens), log
    probabilities, and the cache; a sequence's cache is cut to half of
    `budget` slots when it is full.  With `graph` the current stream is one
    that can be captured (not the default one), and has waited for whatever
    made the model."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch = len(prompts)
    longest = max(map(len, prompts))
    cache = Cache(batch, model.heads, model.dim, max(longest, budget))
    starts = torch.tensor([0, *map(len, prompts)], dtype=torch.int32,
                          device="cuda").cumsum(0, dtype=torch.int32)
    flat = torch.tensor(sum(prompts, []), device="cuda")
    x, q, k, v = model.projected(flat)
    cache.extend(model, q, k, v, starts)
    last = (starts[1:] - 1).long()
    x, q = x[last], q[last]
    u = torch.rand(steps + 1, batch, generator=g, device="cuda")
    how = dict(temperature=temperature, top_k=top_k, top_p=top_p)
    out = cache.attend(q)
    cache.evict(budget // 2)
    token, logprob = ltk.sample(model.logits(x, out), u[0], **how)
    tokens, logprobs = [token.clone()], [logprob.clone()]
    one_each = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    now = u[1].clone() if steps else None

    def step():
        x, q, k, v = model.projected(token)
        q = cache.extend(model, q, k, v, one_each)
        ltk.sample(model.logits(x, cache.attend(q)), now, **how,
                   out=(token, logprob))

    run, used = step, budget // 2  # no sequence holds more slots
    for i in range(steps):
        if used == budget:
            cache.evict(budget // 2)
            used = budget // 2
        now.copy_(u[i + 1])
        run()
        used += 1
        tokens.append(token.clone())
        logprobs.append(logprob.clone())
        if graph and i == 0:  # the first step has made its workspaces
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded, stream=torch.cuda.current_stream()):
                step()
            run = recorded.replay
    return torch.stack(tokens), torch.stack(logprobs), cache


def main():
    model = Decoder(vocab=32000, heads=8, group=4, dim=128)
    r = torch.Generator().manual_seed(2)
    prompts = [torch.randint(32000, (n,), generator=r).tolist()
               for n in (700, 3, 251, 1024)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())  # which makes the weights
    with torch.cuda.stream(side):
        tokens, logprobs, cache = generate(model, prompts, 200, budget=512,
                                           graph=True)
    side.synchronize()
    print("200 steps of %d sequences; lengths seen %s, held %s; mean log "
          "probability %.2f" % (len(prompts), cache.seen.tolist(),
                                cache.lens.tolist(), float(logprobs.mean())))


if __name__ == "__main__":
    main()
