"""One MoE block of a transformer with experts in block-scaled 8-bit floating
point: residual addition and norm, router, dispatch, expert FFN, combine.

    python examples/fp8_moe_block.py [--tokens T] [--hidden H] [--experts E] [--topk K] [--ffn N]

builds random weights, runs the block and prints its time per call.  The
functions below are what a model would call: `quantise_weights` once when the
weights are loaded, `Fp8MoeBlock.__call__` in every step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_route_count_prefix_gb300 import binding as B  # noqa: E402

BLOCK = 128


def quantise_weights(w):
    """[E, N, Kd] -> e4m3 codes of the same shape and one fp32 scale per 128 x 128 block."""
    E, N, Kd = w.shape
    nb, kb = -(-N // BLOCK), -(-Kd // BLOCK)
    p = torch.zeros(E, nb * BLOCK, kb * BLOCK, device=w.device)
    p[:, :N, :Kd] = w
    p = p.view(E, nb, BLOCK, kb, BLOCK)
    scale = p.abs().amax((2, 4)).clamp(min=2.0 ** -100) / 448.0
    q = (p / scale[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(E, nb * BLOCK, kb * BLOCK)[:, :N, :Kd].contiguous(), scale


class Fp8MoeBlock:
    """hidden H, E experts of width N (SwiGLU halves it), top-K routing by
    sigmoid scores with a balance bias over `groups` groups of experts."""

    def __init__(self, norm_weight, router, bias, w1, w1_scales, w2, w2_scales, topk, groups=1,
                 topk_groups=1, scale=1.0):
        self.norm_weight, self.router, self.bias = norm_weight, router, bias
        self.w1, self.w1_scales, self.w2, self.w2_scales = w1, w1_scales, w2, w2_scales
        self.topk, self.groups, self.topk_groups, self.scale = topk, groups, topk_groups, scale

    def __call__(self, x, residual, mask=None, stages=None):
        """x, residual bf16 [T, H]; mask uint8 [T] (0: padding).  Returns the new
        residual stream, bf16 [T, H].  `stages`, a dict, collects the intermediate tensors."""
        T, H = x.shape
        E, N, _ = self.w1.shape
        n = B.add_rms_norm(x, self.norm_weight, residual=residual)
        logits = n["y"].float() @ self.router.t()
        r = B.gate(logits, self.topk, bias=self.bias, mask=mask, score="sigmoid",
                   groups=self.groups, topk_groups=self.topk_groups, group_score="top2",
                   scale=self.scale)
        # bookkeeping only: the FFN takes its rows straight from the tokens
        d = B.dispatch(None, r["expert_ids"], E, 1, mask=r["route_mask"], with_rows=False)
        shape = B.make_shape(T, 1, H, E, self.topk, N)
        # its workspace, like the outputs, comes from the allocator for this call
        # alone: calls on other streams, or of other lengths, share nothing with it
        y, _ = B.grouped_ffn_fp8(shape, n["q"], n["scales"], d["expert_offsets"], self.w1,
                                 self.w1_scales, self.w2, self.w2_scales, assist=d["assist"])
        # the residual joins the experts' weighted sum in the combine
        out = B.combine(y, d["route_row"], r["expert_scales"], E, 1, mask=r["route_mask"],
                        shared=n["residual_out"])
        if stages is not None:
            stages.update(norm=n, logits=logits, routes=r, dispatch=d, y=y)
        return out


def random_block(H, E, K, N, groups=1, topk_groups=1, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device=device)

    w1 = torch.empty(E, N, H, dtype=torch.float8_e4m3fn, device=device)
    w2 = torch.empty(E, H, N // 2, dtype=torch.float8_e4m3fn, device=device)
    s1 = torch.empty(E, N // BLOCK, -(-H // BLOCK), device=device)
    s2 = torch.empty(E, -(-H // BLOCK), N // 2 // BLOCK, device=device)
    for e in range(E):      # one expert at a time: the fp32 weights of all would not be small
        q, s = quantise_weights(randn(1, N, H) * H ** -0.5)
        w1[e], s1[e] = q[0], s[0]
        q, s = quantise_weights(randn(1, H, N // 2) * (N // 2) ** -0.5)
        w2[e], s2[e] = q[0], s[0]
    return Fp8MoeBlock((1 + 0.1 * randn(H)).bfloat16(), randn(E, H) * H ** -0.5, 0.05 * randn(E),
                       w1, s1, w2, s2, K, groups, topk_groups, 2.5)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--ffn", type=int, default=4096)
    a = ap.parse_args()
    groups = 8 if a.experts % 8 == 0 and a.topk <= a.experts // 2 else 1
    block = random_block(a.hidden, a.experts, a.topk, a.ffn, groups, max(1, groups // 2))
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    residual = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    for _ in range(5):
        block(x, residual)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        out = block(x, residual)
    stop.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts, top-{a.topk}, FFN {a.ffn}: "
          f"{start.elapsed_time(stop) / 20 * 1e3:.1f} us per call, "
          f"output rms {out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
