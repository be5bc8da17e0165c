"""Time the kernels of the gated projection, the 8-bit checkpoints and the
post-training losses on one GPU, with the products or the bytes they cannot do
without over the time taken.

    python examples/time_block.py [--op gated|int8|policy|preference] [--rows N] [--cols C] [--hidden F] [--reps R]

Inputs rotate through two sets, so that no set is found in the caches.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_deterministic_exact_amd as det  # noqa: E402

DEFAULTS = {"gated": (8192, 4096), "int8": (16384, 8192), "policy": (1024, 8192), "preference": (2048, 4096)}
BF16 = torch.bfloat16


def timed(name: str, call, sets, reps: int, flops: float = 0.0, nbytes: float = 0.0) -> None:
    for s in sets:
        call(*s)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for i in range(reps):
        call(*sets[i % len(sets)])
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) / reps * 1e3
    print(f"{name:34s} {us:10.1f} us " + (f"{flops / us / 1e6:8.0f} TFLOP/s" if flops else f"{nbytes / us / 1e3:8.0f} GB/s"),
          flush=True)


def gated(N: int, C: int, F: int, reps: int) -> None:
    randn = lambda *s: torch.randn(*s, device="cuda")
    sets = [((randn(N, C)).to(BF16), (randn(F, C) / C ** 0.5).to(BF16), (randn(F, C) / C ** 0.5).to(BF16)) for _ in range(2)]
    label, flops = f"gated {N}x{C}x{F}", 4.0 * N * C * F
    timed(label + " forward", lambda *s: det.gated_linear(*s), sets, reps, flops)
    for ck in (None, "int8"):
        name = f"{label} {ck or 'fp16'}"
        timed(name + " forward", lambda *s: det.gated_linear_forward(*s, checkpoint=ck), sets, reps, flops)
        grads = [((randn(N, F) / N ** 0.5).to(BF16), det.pack_int8(s[0]) if ck else s[0], *s[1:],
                  det.gated_linear_forward(*s, checkpoint=ck)[1]) for s in sets]
        timed(name + " gradients", det.gated_linear_backward, grads, reps, 2 * flops)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--op", choices=sorted(DEFAULTS), default=None)
    ap.add_argument("--rows", type=int, default=None)
    ap.add_argument("--cols", type=int, default=None)
    ap.add_argument("--hidden", type=int, default=11008)
    ap.add_argument("--reps", type=int, default=12)
    a = ap.parse_args(argv)
    for op in [a.op] if a.op else sorted(DEFAULTS):
        N, C = a.rows or DEFAULTS[op][0], a.cols or DEFAULTS[op][1]
        n = N * C
        if op == "gated":
            gated(N, C, a.hidden, a.reps)
            continue
        if op == "int8":
            sets = [(torch.randn(N, C, device="cuda").to(BF16),) for _ in range(2)]
            timed(f"int8 {N}x{C} bf16 pack", det.pack_int8, sets, a.reps, nbytes=n * (3 + 1 / 32))
            packed = [(det.pack_int8(*s), BF16) for s in sets]
            timed(f"int8 {N}x{C} bf16 unpack", det.unpack_int8, packed, a.reps, nbytes=n * (3 + 1 / 32))
            continue
        lp = [-torch.rand(N, C, device="cuda") for _ in range(8)]
        mask = torch.arange(C, device="cuda") < torch.randint(C // 4, C + 1, (N, 1), device="cuda")
        one = torch.ones((), device="cuda")
        if op == "policy":
            sets = [(lp[k], lp[k + 1], lp[k + 2], lp[k + 3]) for k in (0, 4)]
            opts = dict(kl_weight=0.05)
            timed(f"policy {N}x{C}", lambda l, o, v, r: det.policy_loss_forward(l, o, v, mask, ref_logprob=r, **opts), sets, a.reps,
                  nbytes=17 * n)
            count = det.policy_loss_forward(lp[0], lp[1], lp[2], mask)[1]
            timed(f"policy {N}x{C} gradient",
                  lambda l, o, v, r: det.policy_loss_backward(one, l, o, v, mask, count, ref_logprob=r, **opts), sets, a.reps,
                  nbytes=21 * n)
            continue
        sets = [(lp[k], lp[k + 1], lp[k + 2], lp[k + 3]) for k in (0, 4)]
        timed(f"preference 2x{N}x{C}", lambda *s: det.preference_loss(*s, chosen_mask=mask, rejected_mask=mask), sets, a.reps,
              nbytes=18 * n)
        slope = det.preference_loss_forward(*sets[0], chosen_mask=mask, rejected_mask=mask)[1]
        timed(f"preference 2x{N}x{C} gradient",
              lambda *s: det.preference_loss_backward(one.expand(N), slope, (N, C), (N, C), chosen_mask=mask, rejected_mask=mask),
              sets, a.reps, nbytes=10 * n)


if __name__ == "__main__":
    main()
