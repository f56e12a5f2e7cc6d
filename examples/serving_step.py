"""Speculative serving with one decoder layer: latent attention over a paged
cache, the routed expert layer, tree drafts, verification and kept rows, put
together as a serving loop uses them.

    python examples/serving_step.py

The model is random and tiny (width 256, 8 heads of 192 + 64 / 256, 16 experts,
512 tokens); its dense projections are ordinary torch products.  A prompt goes
through the expanded attention, each following step drafts a tree of seven
nodes with a bigram-like drafter, runs them as one batch through the absorbed
attention and the experts, and verifies them."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from int4_routed_expert_layer_amd import binding, configs, inputs  # noqa: E402
from int4_routed_expert_layer_amd.serve import LATENT, ROPE, ROW, Serve  # noqa: E402

SPEC = configs.Spec("example_h256_i128_e16_k4", 256, 128, 16, 4, 64, "bf16", True, "gauss", seed=77)
HEADS, NOPE, V, VOCAB, PAGE, EPS = 8, 192, 256, 512, 16, 1e-6
TEMPERATURE = 32.0   # an untrained model with tied embeddings mostly repeats its last token
# The draft tree: the two likeliest continuations of the last token, then of each of those.
PARENTS = [-1, 0, 0, 1, 1, 2, 2]


def rms(x, eps=EPS):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)).bfloat16()


class Model:
    def __init__(self, seed=0, max_tokens=256, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g, device=device) / fan ** 0.5).bfloat16()

        d = SPEC.hidden
        self.device = device
        self.embed = weight(VOCAB, d, fan=1)
        self.w_q = weight(d, HEADS * (NOPE + ROPE), fan=d)
        self.w_kv = weight(d, ROW, fan=d)
        self.kv_norm = (1 + 0.1 * torch.randn(LATENT, generator=g, device=device)).bfloat16()
        up = weight(HEADS, NOPE + V, LATENT, fan=LATENT)          # the up-projection of latents, by head
        self.w_up = up.reshape(-1, LATENT)
        self.w_uk = up[:, :NOPE].contiguous()                      # absorbed into the queries
        self.w_uv = up[:, NOPE:].transpose(1, 2).contiguous()      # absorbed into the output
        self.w_o = weight(HEADS * V, d, fan=HEADS * V)
        angle = torch.arange(4096, device=device)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, device=device) / ROPE)
        self.cos, self.sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        self.scale = (NOPE + ROPE) ** -0.5
        self.serve = Serve(HEADS, max_tokens, 4, PAGE, NOPE, V)
        self.moe = binding.MoELayer.from_spec(SPEC, max_tokens=max_tokens)
        self.moe.set_router(inputs.router_weight(SPEC), inputs.router_bias(SPEC))
        for e, blob in inputs.expert_blobs(SPEC, 0, range(SPEC.n_experts), threads=4).items():
            self.moe.place(e, blob)
        self.moe.place(binding.SHARED, inputs.expert_blobs(SPEC, 0, [-1], threads=1)[-1])

    def close(self):
        self.serve.close()
        self.moe.close()

    def layer(self, tokens, positions, slots, cache, attend):
        """Logits of a batch of tokens, whose rows are written to the cache first."""
        x = self.embed[tokens.long()]
        h = rms(x)
        q = (h @ self.w_q).view(-1, HEADS, NOPE + ROPE)
        q_pe = self.serve.append(h @ self.w_kv, self.kv_norm, EPS, self.cos, self.sin, positions, slots, cache, q_pe=q[..., NOPE:])
        o = attend(q[..., :NOPE], q_pe)
        x = x + o.reshape(len(tokens), -1) @ self.w_o
        y, _, _, _ = self.moe.layer(rms(x))
        return rms(x.float() + y).float() @ self.embed.float().t()

    def expanded(self, slots, cache, starts):
        """Attention of whole prompts: keys and values expanded from the rows just written."""
        def attend(q_nope, q_pe):
            rows = cache.view(-1, ROW)[slots]
            kv = (rows[:, :LATENT] @ self.w_up.t()).view(-1, HEADS, NOPE + V)
            return self.serve.prompt(torch.cat([q_nope, q_pe], -1), kv, rows[:, LATENT:], starts, starts, self.scale)
        return attend

    def absorbed(self, cache, table, tree_mask=None):
        """Attention over the cache: the up-projection moves into queries and outputs."""
        def attend(q_nope, q_pe):
            q_lat = torch.bmm(q_nope.transpose(0, 1).float().contiguous(), self.w_uk.float()).bfloat16().transpose(0, 1)
            o = self.serve.decode(q_lat, q_pe, cache, table, self.scale, tree_mask=tree_mask)
            return torch.bmm(o.transpose(0, 1).float().contiguous(), self.w_uv.float()).bfloat16().transpose(0, 1)
        return attend


def ancestor_bits(parents):
    bits = []
    for j, p in enumerate(parents):
        bits.append((1 << j) | (bits[p] if p >= 0 else 0))
    return bits


def ints(values, device, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=device)


def generate(model, prompt, steps, seed=0):
    """Returns the generated tokens, the nodes accepted per step, and the
    sequence's cache rows (in order)."""
    dev, n = model.device, len(PARENTS)
    g = torch.Generator(device=dev).manual_seed(seed)
    longest = len(prompt) + steps * n + n
    pages = -(-longest // PAGE)
    cache = torch.zeros(pages, PAGE, ROW, dtype=torch.bfloat16, device=dev)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()   # pages lie anywhere
    table = ints([order], dev)

    def slots(first, count):
        return ints([order[p // PAGE] * PAGE + p % PAGE for p in range(first, first + count)], dev, torch.int64)

    # The prompt, by expanded attention; all but its last token's row stay
    # (the last is the root of the first draft).
    at = slots(0, len(prompt))
    model.layer(ints(prompt, dev), torch.arange(len(prompt), device=dev, dtype=torch.int32), at, cache,
                model.expanded(at, cache, ints([0, len(prompt)], dev)))
    tokens, length, accepted = list(prompt), len(prompt) - 1, []
    mask = ints([[b] for b in ancestor_bits(PARENTS)], dev, torch.int64)
    parents, starts = ints(PARENTS, dev), ints([0, n], dev)
    depth = [0, 1, 1, 2, 2, 2, 2]
    for _ in range(steps):
        # Draft: the tokens nearest to the last one's embedding.
        def nearest(token):
            return torch.topk(model.embed[token].float() @ model.embed.float().t(), 2).indices.tolist()
        first = nearest(tokens[-1])
        draft = [tokens[-1], *first, *nearest(first[0]), *nearest(first[1])]
        kv_len = ints([length + n], dev)
        model.serve.plan(starts, kv_len, n_tok=n)
        logits = model.layer(ints(draft, dev), ints([length + d for d in depth], dev), slots(length, n), cache, model.absorbed(cache, table, mask))
        probs = torch.softmax(logits / TEMPERATURE, 1)
        race = torch.empty(1, VOCAB, device=dev).exponential_(generator=g).reciprocal_()
        path, count, nxt = model.serve.verify(probs, ints(draft, dev), starts, torch.rand(n, generator=g, device=dev), race, parents=parents, max_path=n)
        model.serve.keep(cache, table, starts, kv_len, path)
        kept = int(count[0])
        tokens += nxt[0, :kept].tolist()
        length += kept
        accepted.append(kept - 1)
    assert model.serve.device_errors() == 0 and model.moe.device_errors() == 0
    rows = cache.view(-1, ROW)[slots(0, length)]
    return tokens, accepted, rows


def main():
    model = Model()
    tokens, accepted, _ = generate(model, list(range(3, 40)), 12)
    print("tokens:", tokens[37:])
    print("drafted tokens accepted per step:", accepted)
    model.close()


if __name__ == "__main__":
    main()
