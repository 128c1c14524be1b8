"""One W4A4 transformer block on packed prompts, every operator from this package.

    x  -> layer norm -> quantize -> W4A4 linear (QKV, bias)
       -> attention over the packed prompts
       -> quantize -> W4A4 linear (output projection, bias, residual)
       -> layer norm -> quantize -> W4A4 linear (bias, GELU)
       -> quantize -> W4A4 linear (bias, residual)

    python examples/transformer_block.py [--width 1152 --heads 16 --kv-heads 16
        --lengths 1024,333,17,0,2048 --hidden 4608 --tune]

Activations are quantized by the KroQuant transform, weights by its inverse
transpose, once.  Every operator's output is compared with elementary torch
operations in fp32 on the inputs it had, and the whole block with the same block
on the unquantized operands (the difference is what four bits cost).  ``--tune``
then takes a step of the first norm's weight and bias along the gradient that
kq_layer_norm_backward gives.  Weights and inputs are random.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

from w4a4_mxfp4_activation_gb300 import kq, synth

BLOCKED = kq.KQ_SF_BLOCKED_128x4


class Linear:
    """A W4A4 layer: the weight W T^-T quantized once, the activations' transform
    records kept beside it."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor, seed: int):
        self.n, self.k = weight.shape
        self.weight, self.bias = weight, bias
        factors = kq.kq_lu_to_factors(synth.lu_params(self.k // 32, seed), 1)
        inverse = torch.from_numpy(kq.kq_invert_transpose_factors(factors)).cuda()
        self.records = kq.kq_expand_blocks(torch.from_numpy(factors).cuda(), kq.KQ_K_BF16X3)
        self.q, self.sf, _ = kq.kq_quantize_mxfp4(weight, self.k, factors=inverse, layout=BLOCKED)

    def __call__(self, x, act="none", residual=None):
        m = x.shape[0]
        qa, sfa, _ = kq.kq_quantize_mxfp4(x, self.k, K_expanded=self.records, layout=BLOCKED)
        return kq.kq_w4a4_linear(qa, sfa, self.q, self.sf, m, self.n, self.k, bias=self.bias,
                                 act=act, residual=residual)

    def reference(self, x):
        """x W^T + bias in fp32 on the quantized operands."""
        qa, sfa, _ = kq.kq_quantize_mxfp4(x, self.k, K_expanded=self.records, layout=BLOCKED)
        a = kq.kq_dequantize(qa, sfa, x.shape[0], self.k, layout=BLOCKED)
        w = kq.kq_dequantize(self.q, self.sf, self.n, self.k, layout=BLOCKED)
        return a @ w.t() + self.bias

    def unquantized(self, x):
        return x.float() @ self.weight.float().t() + self.bias


class Block:
    def __init__(self, width: int, heads: int, kv_heads: int, hidden: int, seed: int = 0):
        self.width, self.heads, self.kv_heads = width, heads, kv_heads
        self.dim = width // heads
        g = torch.Generator(device="cuda").manual_seed(seed)

        def linear(n, k, s):
            w = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
            return Linear(w.bfloat16(), 0.1 * torch.randn(n, generator=g, device="cuda"), s)

        self.qkv = linear((heads + 2 * kv_heads) * self.dim, width, seed + 1)
        self.proj = linear(width, width, seed + 2)
        self.up = linear(hidden, width, seed + 3)
        self.down = linear(width, hidden, seed + 4)
        self.norm1 = [1 + 0.1 * torch.randn(width, generator=g, device="cuda"),
                      0.1 * torch.randn(width, generator=g, device="cuda")]
        self.norm2 = [1 + 0.1 * torch.randn(width, generator=g, device="cuda"),
                      0.1 * torch.randn(width, generator=g, device="cuda")]

    def split(self, qkv):
        """q, k, v [tokens, heads, dim] as views of the packed projection."""
        t = qkv.view(qkv.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        h, hk = self.heads, self.kv_heads
        return t[:, :h], t[:, h:h + hk], t[:, h + hk:]

    def forward(self, x, cu, longest: int, causal: bool = True, seen=None):
        """The block's output.  ``seen``: a dict that receives every operator's
        output."""
        seen = {} if seen is None else seen
        seen["norm1"] = y = kq.kq_layer_norm(x, *self.norm1)
        seen["qkv"] = y = self.qkv(y)
        q, k, v = self.split(y)
        seen["attention"] = a = kq.kq_attention(q, k, v, cu, cu, longest, longest, causal=causal)
        seen["proj"] = x = self.proj(a.reshape(x.shape), residual=x)
        seen["norm2"] = y = kq.kq_layer_norm(x, *self.norm2)
        seen["up"] = y = self.up(y, act="gelu_tanh")
        seen["down"] = x = self.down(y, residual=x)
        return x

    def norm(self, x, parameters):
        return torch.nn.functional.layer_norm(x.float(), (self.width,), *parameters, eps=1e-6)

    def attend(self, qkv, lengths, causal: bool):
        """Softmax attention, one prompt after the other, in fp32."""
        q, k, v = self.split(qkv.float())
        out, at, grp = [], 0, self.heads // self.kv_heads
        for n in lengths:
            of = lambda t: t[at:at + n].transpose(0, 1)
            kk, vv = of(k).repeat_interleave(grp, 0), of(v).repeat_interleave(grp, 0)
            s = of(q) @ kk.transpose(1, 2) / math.sqrt(self.dim)
            if causal:
                s = s + torch.full((n, n), -math.inf, device=s.device).triu(1)
            out.append((torch.softmax(s, -1) @ vv).transpose(0, 1))
            at += n
        return torch.cat(out)

    def check(self, x, lengths, causal: bool, seen):
        """Relative distance (2-norm) of every operator's output from torch's on the
        inputs that the operator had."""
        gelu = lambda t: torch.nn.functional.gelu(t, approximate="tanh")
        flat = seen["attention"].reshape(x.shape)
        want = {
            "norm1": self.norm(x, self.norm1),
            "qkv": self.qkv.reference(seen["norm1"]),
            "attention": self.attend(seen["qkv"], lengths, causal),
            "proj": x.float() + self.proj.reference(flat),
            "norm2": self.norm(seen["proj"], self.norm2),
            "up": gelu(self.up.reference(seen["norm2"])),
            "down": seen["proj"].float() + self.down.reference(seen["up"])}
        return {name: relative(seen[name], t) for name, t in want.items()}

    def unquantized(self, x, lengths, causal: bool):
        """The block in fp32 on the unquantized operands."""
        a = self.attend(self.qkv.unquantized(self.norm(x, self.norm1)), lengths, causal)
        x = x.float() + self.proj.unquantized(a.reshape(x.shape))
        up = torch.nn.functional.gelu(self.up.unquantized(self.norm(x, self.norm2)), approximate="tanh")
        return x + self.down.unquantized(up)

    def tune_norm(self, x, target):
        """One step of norm1's weight and bias down the gradient of the mean square
        distance from ``target``; the losses before and after.  The step is half the
        inverse of the loss's largest curvature, which decreases it."""
        def loss(y):
            return float((y.float() - target.float()).square().mean())

        y, mean, rstd = kq.kq_layer_norm(x, *self.norm1, stats=True)
        dy = (y.float() - target.float()).bfloat16()
        _, dw, db = kq.kq_layer_norm_backward(dy, x, self.norm1[0], mean, rstd)
        before, m = loss(y), x.shape[0]
        rate = 0.5 / (1 + kq.kq_layer_norm(x).float().square().mean(0).max())
        self.norm1 = [self.norm1[0] - rate * dw[0] / m, self.norm1[1] - rate * db[0] / m]
        return before, loss(kq.kq_layer_norm(x, *self.norm1))


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--width", type=int, default=1152)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4608)
    ap.add_argument("--lengths", default="1024,333,17,0,2048")
    ap.add_argument("--full", action="store_true", help="every token sees its whole prompt")
    ap.add_argument("--tune", action="store_true")
    a = ap.parse_args(argv)
    if a.width % 32 or a.hidden % 32 or a.width % a.heads or a.heads % a.kv_heads:
        ap.error("widths are multiples of 32, heads divide the width, kv-heads the heads")
    lengths = [int(n) for n in a.lengths.split(",")]
    m = sum(lengths)
    block = Block(a.width, a.heads, a.kv_heads, a.hidden)
    bits = synth.activations(m, a.width, synth.SEED_A, "gauss_outlier8")
    x = (torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16) / 8).contiguous()
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    seen = {}
    out = block.forward(x, cu, max(lengths), not a.full, seen)
    off = block.check(x, lengths, not a.full, seen)
    exact = block.unquantized(x, lengths, not a.full)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        block.forward(x, cu, max(lengths), not a.full)
    end.record()
    end.synchronize()
    cost = relative(out - x, exact - x.float())          # of what the block adds to x
    print(f"block {m} x {a.width}, {a.heads}/{a.kv_heads} heads, hidden {a.hidden}: "
          f"{start.elapsed_time(end) / 10:.3f} ms; four bits cost {cost:.3f} of its output")
    print("off from torch on the same inputs: " + ", ".join(f"{k} {v:.4f}" for k, v in off.items()))
    result = {"off": off, "cost": cost}
    if a.tune:
        target = torch.nn.functional.layer_norm(x.float(), (a.width,))
        before, after = block.tune_norm(x, target)
        print(f"norm tuned by one step: loss {before:.5f} -> {after:.5f}")
        result.update(before=before, after=after)
    return result


if __name__ == "__main__":
    main()
