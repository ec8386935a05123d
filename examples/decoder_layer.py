"""One decoder layer as it is served: attention over the paged 8-bit cache, then the sparse expert layer.

    python examples/decoder_layer.py [--prompt 512] [--steps 32] [--batch 4]

A batch of prompts goes through the layer at once, then the sequences are decoded token by token; the last decoded state is
compared with that of the whole sequences sent as prompts.  Random weights; the projections are torch matrix products.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_fwd_gb300 as moe  # noqa: E402


class DecoderLayer:
    """hidden [T, H] -> hidden [T, H]: norm, attention, norm, experts, with the residual stream beside them."""

    def __init__(self, H=1024, Hq=16, Hkv=2, E=16, k=4, I=256, n_pages=256, page=64, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, device="cuda", generator=g) * s[-1] ** -0.5).to(torch.bfloat16)
        one = lambda n: torch.ones(n, device="cuda", dtype=torch.bfloat16)
        D = 128
        self.H, self.E, self.k, self.I = H, E, k, I
        self.w_qkv, self.w_o = w((Hq + 2 * Hkv) * D, H), w(H, Hq * D)
        self.norm1, self.norm2 = one(H), one(H)
        self.w_gate, self.w13, self.w2 = w(E, H), moe.moe_prepack_w13(w(E, 2 * I, H)), w(E, H, I)
        self.attention = moe.AttentionLayer(n_pages, Hq, Hkv, D, page, max_pos, q_norm_weight=one(D), k_norm_weight=one(D))
        self.experts = {}

    def forward(self, hidden, q_start, kv_len, page_table, max_q):
        T = hidden.shape[0]
        _, x, _ = moe.moe_add_rms_norm_cast(hidden, None, self.norm1, 1e-6)
        a = self.attention.forward(x @ self.w_qkv.T, q_start, kv_len, page_table, max_q) @ self.w_o.T
        x32, x, residual = moe.moe_add_rms_norm_cast(a, hidden, self.norm2, 1e-6)
        if T not in self.experts:
            self.experts[T] = moe.MoELayer(T, self.H, self.E, self.k, self.I)
        y = self.experts[T].forward(x, moe.moe_router_logits(x32, self.w_gate), self.w13, self.w2)
        return residual + y


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(prompt=512, steps=32, batch=4, page=64, k=4, say=print):
    """Returns the largest difference between decoding step by step and sending everything at once, over the largest value."""
    total = prompt + steps
    per = -(-total // page)
    layer = DecoderLayer(k=k, n_pages=2 * batch * per, page=page, max_pos=total)
    torch.manual_seed(1)
    tokens = torch.randn(batch, total, layer.H, device="cuda").to(torch.bfloat16)
    table = torch.randperm(2 * batch * per)[:batch * per].view(batch, per).to(torch.int32).cuda()

    def send(n, length):
        """The tokens length - n .. length - 1 of every sequence."""
        x = tokens[:, length - n:length].reshape(batch * n, layer.H).contiguous()
        return layer.forward(x, i32([b * n for b in range(batch + 1)]), i32([length] * batch), table, n)

    send(prompt, prompt)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for step in range(steps):
        last = send(1, prompt + step + 1)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / max(1, steps) * 1e3
    whole = send(total, total).view(batch, total, layer.H)[:, -1]
    assert layer.attention.status() == moe.MOE_OK
    off = float((last.float() - whole.float()).abs().max() / whole.float().abs().max())
    say(f"{batch} sequences of {prompt} + {steps} tokens: {ms:.3f} ms a decode step, last states differ by {off:.2e}")
    return off


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("--prompt", 512), ("--steps", 32), ("--batch", 4)):
        p.add_argument(name, type=int, default=value)
    run(**vars(p.parse_args()))
