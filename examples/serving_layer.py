"""One attention layer as it serves a language model, on the library's operators.

    x --Gemm--> q, k, v --norm and rotation (in place)--> q, k --+--> 8-bit paged cache
                                                                 +--> attention --Gemm--> out

`prompt` takes the packed whole prompts of several sequences, `token` one new
token of each sequence over the cache.  (A later piece of a prompt needs the keys
and values of the tokens before it, at 16 bits and in front of its own, with
cumulative lengths of the keys of its own; this layer keeps them in the cache alone.)
Weights and inputs are random.

    python examples/serving_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import layout_general_tensor_gb300 as lgt


class AttentionLayer:
    def __init__(self, hidden, q_heads, k_heads, head_dim, pages, page_size=64, sequences=64, seed=0):
        self.hidden, self.hq, self.hk, self.d, self.page_size = hidden, q_heads, k_heads, head_dim, page_size
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):  # stored [out][in], as a product reads it K-contiguously
            return (torch.randn(rows, cols, generator=g, device="cuda") / cols ** 0.5).bfloat16()

        self.w_qkv = weight((q_heads + 2 * k_heads) * head_dim, hidden)
        self.w_out = weight(hidden, q_heads * head_dim)
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.rope = lgt.QKNormRope(q_heads, k_heads, head_dim, base=500000.0)
        self.attend = lgt.PromptAttention(q_heads, k_heads, head_dim)
        self.cache = lgt.KVCache.empty(pages, page_size, k_heads, head_dim)
        self.attend_cache = lgt.CacheAttention(q_heads, k_heads, head_dim, page_size, batch=sequences)
        self.products = {}

    def _product(self, x, w):
        """x [rows][in] times w [out][in], by a plan kept for the shape."""
        m, (n, k) = x.shape[0], w.shape
        if (m, n, k) not in self.products:
            self.products[m, n, k] = lgt.Gemm(lgt.make_desc(m, n, k, lgt.GEMM_K_CONTIG, lgt.GEMM_K_CONTIG, lgt.GEMM_BF16,
                                                            split_k=0))
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        self.products[m, n, k].run(x, w, out)
        return out

    def _heads(self, x, positions, slots):
        """Queries, keys and values of x, the first two normed and turned in place; keys and values to the cache."""
        qkv = self._product(x, self.w_qkv)
        q, k, v = (y.unflatten(1, (-1, self.d)) for y in
                   qkv.split([self.hq * self.d, self.hk * self.d, self.hk * self.d], dim=1))
        self.rope.run(q, k, positions, q, k, self.q_norm, self.k_norm)
        self.cache.write(k, v, slots)
        return q, k, v

    def prompt(self, x, positions, slots, cu):
        """x [tokens][hidden] of packed whole prompts, each from its first token on, whose cumulative lengths are cu."""
        q, k, v = self._heads(x, positions, slots)
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        self.attend.run(q, k, v, cu, cu, out)
        return self._product(out.flatten(1), self.w_out)

    def token(self, x, positions, slots, table, lengths):
        """x [sequences][hidden], one new token of each; lengths with the new token."""
        q, _, _ = self._heads(x, positions, slots)
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        self.attend_cache.run(q, self.cache, table, lengths, out)
        return self._product(out.flatten(1), self.w_out)


def serve(prompts=(300, 17, 1000, 1), new_tokens=3, hidden=1024, q_heads=8, k_heads=2, head_dim=128, page_size=64, seed=0):
    """Prompts of these lengths, then new tokens for all of them; returns the
    layer's outputs: the prompts' [tokens][hidden], then each step's [sequences][hidden]."""
    n = len(prompts)
    per_seq = -(-(max(prompts) + new_tokens) // page_size)
    layer = AttentionLayer(hidden, q_heads, k_heads, head_dim, n * per_seq, page_size, n, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    table = torch.randperm(n * per_seq, generator=g, device="cuda").int().view(n, per_seq)  # pages as an allocator deals them

    def slots_of(sequence, position):
        return (table[sequence, position // page_size] * page_size + position % page_size).int()

    sequence = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(prompts, device="cuda"))
    position = torch.cat([torch.arange(p, device="cuda") for p in prompts])
    cu = torch.tensor([0, *torch.tensor(prompts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(prompts), hidden, generator=g, device="cuda").bfloat16()
    outputs = [layer.prompt(x, position.int(), slots_of(sequence, position), cu)]
    everyone, lengths = torch.arange(n, device="cuda"), torch.tensor(prompts, device="cuda")
    for _ in range(new_tokens):
        x = torch.randn(n, hidden, generator=g, device="cuda").bfloat16()
        outputs.append(layer.token(x, lengths.int(), slots_of(everyone, lengths), table, (lengths + 1).int()))
        lengths = lengths + 1
    torch.cuda.synchronize()
    return outputs


if __name__ == "__main__":
    for i, y in enumerate(serve()):
        print("prompts" if i == 0 else f"token {i}", tuple(y.shape), f"rms {float(y.float().square().mean().sqrt()):.4f}")
