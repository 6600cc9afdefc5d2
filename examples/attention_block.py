"""The attention half of a transformer block on an MI355X, as a program runs it.

    python examples/attention_block.py [--tokens 4608] [--hidden 5120] [--heads 40] [--kv-heads 8]

Prompt: packed sequences of odd lengths go through the W4A4 ConvRot projections
(one quantised activation feeds q, k and v), the head norms with rotary
positions, causal attention and the output projection. Their keys and values
fill a cache, and one new token of every sequence attends to it. Training: the
gradients of the block's attention part with respect to q, k, v and the norm
weights. Synthetic weights and activations.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_w4a4_quantized_amd as ck  # noqa: E402


class Block:
    def __init__(self, hidden: int, heads: int, kv_heads: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.d = heads, kv_heads, hidden // heads
        sizes = {"q": heads * self.d, "k": kv_heads * self.d, "v": kv_heads * self.d, "o": hidden}
        self.weights = {n: ck.quantize_weight_convrot(0.02 * torch.randn(m, hidden, generator=g, device="cuda"))
                        for n, m in sizes.items()}
        self.q_norm = 1 + 0.1 * torch.randn(self.d, generator=g, device="cuda")
        self.k_norm = 1 + 0.1 * torch.randn(self.d, generator=g, device="cuda")
        self.freqs = (10000.0 ** -(torch.arange(self.d // 2, dtype=torch.float64) / (self.d // 2))).float().cuda()

    def project(self, x):
        """q, k and v of activation rows, as heads: one quantised activation for the three."""
        xq, sx = ck.rotate_quantize_act(x)
        return [ck.linear_w4a4(xq, sx, *self.weights[n]).unflatten(1, (-1, self.d)) for n in "qkv"]

    def norm(self, q, k, positions, **out):
        return ck.qk_norm_rope(q, k, self.q_norm, self.k_norm, positions, self.freqs, interleaved=False, **out)

    def output(self, heads):
        return ck.w4a4_linear(heads.flatten(1), *self.weights["o"])

    def prompt(self, x, cu, positions):
        """Packed prompts: the block's output, and its (normed, turned) keys and values for a cache."""
        q, k, v = self.project(x)
        q, k = self.norm(q, k, positions)
        out, _ = ck.attention(q, k, v, cu, cu, causal=True)
        return self.output(out), k, v

    def token(self, x, k_cache, v_cache, lengths):
        """One new token per sequence: its key and value go to the cache's next slot."""
        q, k, v = self.project(x)
        q, k = self.norm(q, k, lengths)
        rows = torch.arange(x.shape[0], device=x.device)
        k_cache[rows, lengths.long()], v_cache[rows, lengths.long()] = k, v
        out, _ = ck.attention_decode(q, k_cache, v_cache, lengths + 1)
        return self.output(out)

    def gradients(self, x, cu, positions, dout):
        """Gradients of the attention part (from the heads that the projections gave to the heads it returns): they end there,
        as the quantised projections have none."""
        q, k, v = self.project(x)
        qn, kn = self.norm(q, k, positions)
        out, lse = ck.attention(qn, kn, v, cu, cu, causal=True)
        dqn, dkn, dv = ck.attention_backward(dout, qn, kn, v, out, lse, cu, cu, causal=True)
        dq, dk, dq_norm, dk_norm = ck.qk_norm_rope_backward(dqn, dkn, q, k, self.q_norm, self.k_norm, positions,
                                                            self.freqs, interleaved=False, dq=dqn, dk=dkn)
        return {"q": dq, "k": dk, "v": dv, "q_norm": dq_norm, "k_norm": dk_norm}


def run(tokens: int = 4608, hidden: int = 5120, heads: int = 40, kv_heads: int = 8) -> dict:
    block = Block(hidden, heads, kv_heads)
    lens = [n for n in (tokens // 2 + 1, tokens // 5, 1) if n]
    lens.append(tokens - sum(lens))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    positions = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    y, k, v = block.prompt(x, cu, positions)

    slots = max(lens) + 16
    caches = [torch.zeros(len(lens), slots, kv_heads, block.d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i, n in enumerate(lens):
        a = int(cu[i])
        caches[0][i, :n], caches[1][i, :n] = k[a:a + n], v[a:a + n]
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = torch.randn(len(lens), hidden, generator=g, device="cuda").bfloat16()
    z = block.token(new, *caches, lengths)

    dout = torch.randn(tokens, heads, block.d, generator=g, device="cuda").bfloat16()
    grads = block.gradients(x, cu, positions, dout)
    return {"block": block, "lens": lens, "cu": cu, "x": x, "new": new, "prompt": y, "token": z, "grads": grads}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4608)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--heads", type=int, default=40)
    ap.add_argument("--kv-heads", type=int, default=8)
    a = ap.parse_args()
    r = run(a.tokens, a.hidden, a.heads, a.kv_heads)
    torch.cuda.synchronize()
    print("sequences of", r["lens"])
    for name, t in [("prompt", r["prompt"]), ("token", r["token"])] + [("d" + n, t) for n, t in r["grads"].items()]:
        print(f"{name:8} {tuple(t.shape)} rms {t.float().square().mean().sqrt().item():.4g}")
