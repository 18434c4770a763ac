"""A small transformer that decodes with drafted tokens, on the operators of the package.

Every step takes the last token and a tree of drafted ones through two layers of

    moe_linear_int4 (q, k, v) -> moe_rope_append -> moe_tree_attention -> moe_linear_int4 (output)
    -> fused_moe_gated (the FFN: 8 experts, INT4) -> ... -> moe_linear_int4 (vocabulary) -> moe_verify_draft

and then moves the keys and values of the kept tokens to their places in the paged cache.  The weights are random, so
the drafts come from a stand-in for a draft model: it knows the continuation and is wrong now and then.

    python examples/speculative_decode.py [--tokens 48] [--hit 0.7]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from mixture_experts_ffn_moe_gb300 import build, gbmoe, synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, LAYERS, PAGE = 512, 8, 2, 64, 1000, 2, 16
EXPERTS, TOPK, INTER = 8, 2, 256


class Model:
    """Random INT4 weights, a paged cache for one sequence, and the step that runs nodes of a tree."""

    def __init__(self, seed=0, pages=32, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def int4(rows, cols, std):
            w, s = synth.quantize_int4_group(torch.randn(rows, cols, generator=g) * std)
            return w.to(device).contiguous(), s.to(device).contiguous()

        self.embed = torch.randn(VOCAB, HIDDEN, generator=g).to(device, torch.bfloat16)
        self.head = int4(VOCAB, HIDDEN, 0.2)
        self.layers = []
        for _ in range(LAYERS):
            w13 = [int4(2 * INTER, HIDDEN, 0.06) for _ in range(EXPERTS)]
            w2 = [int4(HIDDEN, INTER, 0.1) for _ in range(EXPERTS)]
            self.layers.append({
                "qkv": int4((HEADS + 2 * KV_HEADS) * DIM, HIDDEN, 0.06), "out": int4(HIDDEN, HEADS * DIM, 0.06),
                "router": (torch.randn(HIDDEN, EXPERTS, generator=g) * 0.05).to(device),
                "w13": [torch.stack(p).contiguous() for p in zip(*w13)],
                "w2": [torch.stack(p).contiguous() for p in zip(*w2)],
                "k": torch.zeros(pages, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device=device),
                "v": torch.zeros(pages, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device=device)})
        # the sequence's pages, in any order
        self.table = torch.randperm(pages, generator=g).to(torch.int32).to(device).view(1, pages)
        self.inv_freq, self.rope_scale = gbmoe.rope_frequencies(DIM, 10000.0, "yarn", 4.0, 128, device=device)
        self.gate = gbmoe.gate_config()
        self.device = device

    def slots(self, places):
        """Cache slots of the sequence's places."""
        return (self.table[0, places // PAGE] * PAGE + places % PAGE).to(torch.int32)

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def step(self, tokens, depth, mask, length):
        """Logits of the nodes `tokens` (depth below the committed end, ancestor masks) after `length` slots."""
        n = len(tokens)
        x = self.embed[tokens]
        positions = (length + depth).to(torch.int32)
        slots = self.slots(length + torch.arange(n, device=self.device))
        lens = torch.tensor([length], dtype=torch.int32, device=self.device)
        offsets = torch.tensor([0, n], dtype=torch.int32, device=self.device)
        for p in self.layers:
            qkv = gbmoe.moe_linear_int4(self.norm(x), *p["qkv"]).view(n, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            q = gbmoe.moe_rope_append(q, k, v, positions, self.inv_freq, slots, p["k"], p["v"], scale=self.rope_scale)
            a = gbmoe.moe_tree_attention(q, p["k"], p["v"], self.table, lens, offsets, mask)
            x = x + gbmoe.moe_linear_int4(a.view(n, HEADS * DIM), *p["out"])
            h = self.norm(x)
            y, _, _ = gbmoe.fused_moe_gated(gbmoe.MOE_WEIGHT_INT4, h, h.float() @ p["router"], self.gate, TOPK, *p["w13"],
                                            *p["w2"])
            x = x + y
        return gbmoe.moe_linear_int4(self.norm(x), *self.head).float()

    def keep(self, length, path):
        """Moves the kept drafted tokens' keys and values (node indices) to the places after `length`."""
        if path:
            src = self.slots(length + torch.tensor(path, device=self.device)).long()
            dst = self.slots(length + 1 + torch.arange(len(path), device=self.device)).long()
            for p in self.layers:
                for c in (p["k"], p["v"]):
                    flat = c.view(-1, KV_HEADS, DIM)
                    flat[dst] = flat[src].clone()


def probabilities(logits, temperature):
    if temperature == 0.0:  # all on the best token
        return torch.zeros_like(logits).scatter_(1, logits.argmax(-1, keepdim=True), 1.0)
    return torch.softmax(logits / temperature, -1)


def draft_tree(known, at, hit, rng):
    """Candidates after token `at`: (tokens, parents), parents counted among the drafted; -1 is the last token."""
    tokens, parents, tip = [], [], -1
    for level in range(4):
        right = known[at + 1 + level] if at + 1 + level < len(known) else 0
        pair = [right if torch.rand((), generator=rng) < hit else int(torch.randint(VOCAB, (), generator=rng)),
                int(torch.randint(VOCAB, (), generator=rng))]
        first = len(tokens)
        tokens += pair
        parents += [tip, tip]
        tip = first
    return tokens, parents


def generate(model, start, count, known=None, hit=0.7, temperature=0.0, seed=0):
    """`count` tokens after `start`; with `known`, drafts from it.  Returns (tokens, steps)."""
    rng, dev = torch.Generator().manual_seed(seed), model.device
    out, length, steps = [start], 0, 0  # `length` slots are committed; the last token is not among them yet
    i32 = torch.int32
    while len(out) <= count:
        tokens, parents = draft_tree(known, len(out) - 1, hit, rng) if known else ([], [])
        nodes = [out[-1]] + tokens
        depth, masks = [0], [1]
        for j, p in enumerate(parents):  # node j + 1 of the step hangs below node p + 1
            depth.append(depth[p + 1] + 1)
            masks.append(masks[p + 1] | (1 << (j + 1)))
        logits = model.step(torch.tensor(nodes, device=dev), torch.tensor(depth, device=dev),
                            torch.tensor(masks, device=dev), length)
        kept, path, accepted = gbmoe.moe_verify_draft(
            probabilities(logits, temperature), torch.tensor(tokens, dtype=i32, device=dev),
            torch.tensor([0, len(tokens)], dtype=i32, device=dev), torch.rand(len(nodes), generator=rng).to(dev),
            torch.rand(1, generator=rng).to(dev), len(tokens), torch.tensor(parents, dtype=i32, device=dev))
        n = int(accepted)
        if n < 0:
            raise RuntimeError("the step's drafted tokens were refused")
        model.keep(length, [1 + j for j in path[0, :n].tolist()])
        out += kept[0, :n + 1].tolist()
        length += 1 + n
        steps += 1
    return out[:count + 1], steps


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--hit", type=float, default=0.7, help="how often the stand-in draft knows the next token")
    args = ap.parse_args()
    build.build()
    plain, steps = generate(Model(), 7, args.tokens)
    print(f"one token a step: {steps} steps")
    drafted, steps = generate(Model(), 7, args.tokens, known=plain, hit=args.hit)
    same = sum(a == b for a, b in zip(plain, drafted))
    print(f"with drafted trees: {steps} steps, {same} of {len(plain)} tokens alike")


if __name__ == "__main__":
    main()
