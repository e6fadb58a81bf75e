"""One routed FP8 layer over a prompt: residual + RMSNorm + quantisation, router, routed experts and shared expert.

    python examples/prompt_layer.py [--tokens T]

Random weights of the DeepSeek-V3 layer shape with fewer experts (1.8 GB). The same weights then serve a decode batch
through the one-launch layer call; the two are compared on the prompt's last tokens.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp4_moe_expert_gb300 as fme  # noqa: E402

H, I, E, TOP_K = 7168, 2048, 40, 8
LIMIT, SCALE, EPS = 7.0, 2.5, 1e-5


def fp8_weights(experts, rows, cols):
    """E4M3 bytes [experts, rows, cols] and FP32 scales per 128 x 128 block."""
    w = torch.empty(experts, rows, cols, dtype=torch.uint8, device="cuda")
    for e in range(experts):
        w[e] = torch.randn(rows, cols, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    return w, torch.exp2(torch.rand(experts, rows // 128, cols // 128, device="cuda") * 3 - 10)


def shared_expert(xq, sx, w13, s13, w2, s2):
    """The shared expert of a prompt: the grouped products with one group that holds every token."""
    all_tokens = torch.tensor([0, xq.shape[0]], dtype=torch.int32, device="cuda")
    hq, sh = fme.moe_grouped_swiglu_fp8(xq, sx, w13, s13, all_tokens, limit=LIMIT, gate_first=True)
    return fme.moe_grouped_gemm_fp8(hq, sh, w2, s2, all_tokens)


def prompt_layer(x, residual, gamma, router, bias, routed, shared):
    """(layer output [T, H], new residual [T, H], normed [T, H], router logits) of a prompt x [T, H]."""
    xq, sx, residual, normed = fme.add_rmsnorm_fp8(x, gamma, residual, EPS, want_normed=True)
    logits = normed @ router
    y, _, _ = fme.moe_prompt_fp8(xq, sx, logits, bias, *routed, TOP_K, LIMIT, SCALE, False,
                                 shared_out=shared_expert(xq, sx, *shared))
    return y, residual, normed, logits


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2000)
    T = ap.parse_args().tokens
    torch.manual_seed(0)
    x = torch.randn(T, H, device="cuda").bfloat16()
    residual = (3 * torch.randn(T, H, device="cuda")).bfloat16()
    gamma = (1 + 0.1 * torch.randn(H, device="cuda")).bfloat16()
    router = (torch.randn(H, E, device="cuda") / H ** 0.5).bfloat16()
    bias = 0.05 * torch.randn(E, device="cuda")
    routed = (*fp8_weights(E, 2 * I, H), *fp8_weights(E, H, I))
    shared = (*fp8_weights(1, 2 * I, H), *fp8_weights(1, H, I))
    args = (x, residual, gamma, router, bias, routed, shared)

    y, _, normed, logits = prompt_layer(*args)
    # The last tokens again as a decode batch on the same weights. It quantises the BF16 norm, the prompt the FP32 one:
    # some codes differ, and the outputs by about as much as one FP8 rounding changes them.
    M = min(8, T)
    out, _, weights, shared_out = fme.moe_layer_fp8(
        normed[-M:].contiguous(), logits[-M:].contiguous(), bias, *routed, TOP_K, LIMIT, SCALE, False,
        *(w[0] for w in shared), LIMIT, False)
    ref = fme.moe_finalize(out, weights, shared_out).float()
    err = ((y[-M:].float() - ref).norm() / ref.norm()).item()

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(10):
        prompt_layer(*args)
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 100
    print(f"{T} tokens: {us:.0f} us a layer, {T / us:.2f} tokens/us; last {M} tokens against the decode layer: "
          f"relative difference {err:.2e}")
    return err


if __name__ == "__main__":
    main()
