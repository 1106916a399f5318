"""The expert half of a transformer block with int8 weights, for prefill and for
decoding: output projection of the attention, block boundary norm, router,
experts, and the boundary to the next block.

    python examples/int8_block.py [--tokens T] [--hidden H] [--experts E] [--topk K] [--ffn N]

builds random weights, runs the block and prints its time per call, for T
tokens and for one.  The functions below are what a model would call:
`quantise_weights` once when the weights are loaded, `Int8Block.__call__` in
every step.  Steps of a few tokens take the few-token layer, whose results are
those of the whole layer bit for bit, from the same packed weights.  Nothing is kept
per length, so that a call of any length can be captured in a graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_route_count_prefix_gb300 import binding as B  # noqa: E402

FEW_ROUTES = 512         # what moe_layer_few_tokens takes
FEW_PER_EXPERT = 16      # above so many routes an expert, on average, the whole layer is faster


def quantise_weights(w):
    """[E, N, Kd] -> int8 of the same shape and one fp32 scale per output channel."""
    scale = w.abs().amax(2).clamp(min=1e-30) / 127.0
    return torch.round(w / scale[:, :, None]).to(torch.int8), scale


class Int8Block:
    """hidden H, E experts of width N (SwiGLU halves it), top-K routing by a
    softmax over the router's logits."""

    def __init__(self, o_proj, o_scale, post_weight, weight, next_weight, gate, router, w1, scale1, w2,
                 scale2, topk):
        """o_proj int8 [1, H, A]; post_weight, weight, next_weight bf16 [H]: the norms
        behind the attention, before the experts, before the next block; gate bf16
        [1, H]: what scales the attention's branch per channel."""
        self.o_scale, self.scale1, self.scale2, self.topk = o_scale, scale1, scale2, topk
        self.post_weight, self.weight, self.next_weight, self.gate = post_weight, weight, next_weight, gate
        self.router = router
        self.E, self.N, self.H = w1.shape
        self.o_owner, self.o_packed = B.pack_int8(o_proj)
        shape = B.make_shape(1, 1, self.H, self.E, topk, self.N, ffn_path="auto")
        (self.w1_owner, self.w1), (self.w2_owner, self.w2) = B.pack_weights(shape, w1, w2)

    def __call__(self, attention, residual, mask=None, stages=None):
        """attention bf16 [T, A], residual bf16 [T, H]; mask uint8 [T] (0: padding).
        Returns the new residual stream and the next block's input, bf16 [T, H].
        `stages`, a dict, collects the intermediate tensors."""
        T = attention.shape[0]
        one_group = torch.linspace(0, T, 2, dtype=torch.int32, device=attention.device)      # [0, T], on the GPU
        o, _ = B.grouped_gemm_int8(one_group, attention, self.o_packed, self.o_scale)
        n = B.block_norm(o, residual, self.weight, post_weight=self.post_weight, gate=self.gate,
                         gate_act="sigmoid", with_q=False)
        logits = n["y"].float() @ self.router.t()
        r = B.gate(logits, self.topk, mask=mask)
        shape = B.make_shape(T, 1, self.H, self.E, self.topk, self.N, mask_kind=2, ffn_path="auto")
        few = T * self.topk <= min(FEW_ROUTES, FEW_PER_EXPERT * self.E)
        layer = B.layer_few_tokens if few else B.layer
        y, _ = layer(shape, n["y"], r["expert_ids"], r["expert_scales"], self.w1, self.scale1, self.w2,
                     self.scale2, mask=r["route_mask"])
        out = B.block_norm(y, n["residual_out"], self.next_weight, with_q=False)
        if stages is not None:
            stages.update(o=o, norm=n, logits=logits, routes=r, layer=y)
        return out["residual_out"], out["y"]


def random_block(H, A, E, K, N, seed=0, device="cuda", stages=None):
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device=device)

    o_proj, o_scale = quantise_weights(randn(1, H, A) * A ** -0.5)
    w1 = torch.empty(E, N, H, dtype=torch.int8, device=device)
    w2 = torch.empty(E, H, N // 2, dtype=torch.int8, device=device)
    s1, s2 = torch.empty(E, N, device=device), torch.empty(E, H, device=device)
    for e in range(E):      # one expert at a time: the fp32 weights of all would not be small
        q, s = quantise_weights(randn(1, N, H) * H ** -0.5)
        w1[e], s1[e] = q[0], s[0]
        q, s = quantise_weights(randn(1, H, N // 2) * (N // 2) ** -0.5)
        w2[e], s2[e] = q[0], s[0]
    if stages is not None:
        stages.update(o_proj=o_proj, w1=w1, w2=w2)
    norms = [(1 + 0.1 * randn(H)).bfloat16() for _ in range(3)]
    return Int8Block(o_proj, o_scale, *norms, randn(1, H).bfloat16(), randn(E, H) * H ** -0.5, w1, s1, w2,
                     s2, K)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--ffn", type=int, default=4096)
    a = ap.parse_args()
    block = random_block(a.hidden, a.hidden, a.experts, a.topk, a.ffn)
    for T in (a.tokens, 1):
        x = torch.randn(T, a.hidden, device="cuda").bfloat16()
        residual = torch.randn(T, a.hidden, device="cuda").bfloat16()
        for _ in range(5):
            block(x, residual)
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            out, _ = block(x, residual)
        stop.record()
        torch.cuda.synchronize()
        print(f"{T} tokens, hidden {a.hidden}, {a.experts} experts, top-{a.topk}, FFN {a.ffn}: "
              f"{start.elapsed_time(stop) / 20 * 1e3:.1f} us per call, "
              f"output rms {out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
