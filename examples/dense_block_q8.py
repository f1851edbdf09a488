"""A decoder's dense feed-forward block with 8-bit activations.

    h  = x + r                                    the residual stream
    a  = e4m3 rows of rmsnorm(h) * w              b200q_rmsnorm_q8
    m  = silu(Wg a) * (Wu a)                      b200q_glu_q8
    m8 = e4m3 rows of m                           b200q_quantize_q8
    y  = Wd m8 + h                                b200q_matmul_q8

Random int4 weights; the result is compared with the same block on f32
activations, and the chain is timed for one token and for a prompt:

    python examples/dense_block_q8.py [--hidden 6144] [--inner 12288] [--tokens 1 16 512]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_weight_quant_gb300 as q  # noqa: E402


class Weights:
    """An int4 matrix on the GPU and its f32 values for the comparison."""

    def __init__(self, O, I, seed):
        rng = np.random.default_rng(seed)
        codes = rng.integers(0, 256, (O, (I + 1) // 2), dtype=np.uint8)
        scale = (rng.uniform(0.5, 1.5, O) / (4.6 * np.sqrt(I))).astype(np.float32)
        self.t = q.tensor_upload(q.I4, O, I, codes, scale)
        c = torch.from_numpy(codes).cuda()
        v = torch.stack((c & 15, c >> 4), 2).reshape(O, -1)[:, :I].float() - 8
        self.f32 = v * torch.from_numpy(scale).cuda()[:, None]


class DenseBlock:
    def __init__(self, hidden, inner, max_tokens):
        self.hidden, self.inner = hidden, inner
        self.gate, self.up, self.down = (Weights(*s, k) for k, s in
                                         enumerate([(inner, hidden), (inner, hidden), (hidden, inner)]))
        self.w = 0.5 + torch.rand(hidden, device="cuda")
        self.a, self.m8 = q.Q8Rows(max_tokens, hidden), q.Q8Rows(max_tokens, inner)
        self.m = torch.empty(max_tokens, inner, dtype=torch.bfloat16, device="cuda")

    def forward(self, x, r, h, y, S):
        q.rmsnorm_q8(x, self.w, self.a, S, self.hidden, 1e-6, r=r, h=h)
        q.glu_q8(self.gate.t, self.up.t, self.a, self.m, S, act=q.ACT_SILU)
        q.quantize_q8(self.m, self.m8, S, self.inner)
        q.matmul_q8(self.down.t, self.m8, y, S, res=h)

    def reference(self, x, r):
        h = x.float() + r.float()
        a = h * self.w / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
        m = torch.nn.functional.silu(a @ self.gate.f32.t()) * (a @ self.up.f32.t())
        return h, m @ self.down.f32.t()


def run(hidden, inner, tokens, time_it=True):
    """Relative error of the block's own contribution (y - h) per token count."""
    block = DenseBlock(hidden, inner, max(tokens))
    torch.manual_seed(0)
    errors = []
    for S in tokens:
        x, r = (torch.randn(S, hidden, device="cuda").bfloat16() for _ in range(2))
        h, y = torch.empty_like(x), torch.empty_like(x)
        block.forward(x, r, h, y, S)
        h32, want = block.reference(x, r)
        got = y.float() - h.float()
        errors.append(float((got - want).norm() / want.norm()))
        line = "%5d tokens: error %.3f of the f32 block" % (S, errors[-1])
        if time_it:
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            for _ in range(3):
                block.forward(x, r, h, y, S)
            a.record()
            for _ in range(20):
                block.forward(x, r, h, y, S)
            b.record()
            torch.cuda.synchronize()
            line += ", %.1f us" % (a.elapsed_time(b) * 50)
        print(line)
    assert q.device_status() == q.OK
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--hidden", type=int, default=6144)
    p.add_argument("--inner", type=int, default=12288)
    p.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 512])
    a = p.parse_args()
    run(a.hidden, a.inner, a.tokens)
