"""Time the head operators' kernels on one GPU: forward and gradient of layer
norm, token log probabilities and distillation at given sizes, with the bytes
they cannot do without over the time taken.

    python examples/time_head.py [--op norm|score|top|distill] [--rows N] [--cols C] [--dtype f32|bf16] [--reps R]

Inputs rotate through three sets, so that no set is found in the caches.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_deterministic_exact_amd as det  # noqa: E402

DEFAULTS = {"norm": (16384, 8192), "score": (4096, 131072), "top": (1024, 131072), "distill": (4096, 131072)}


def timed(name: str, call, sets, nbytes: int, reps: int) -> None:
    for s in sets:
        call(*s)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for i in range(reps):
        call(*sets[i % len(sets)])
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) / reps * 1e3
    print(f"{name:28s} {us:10.1f} us  {nbytes / us / 1e3:8.0f} GB/s", flush=True)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--op", choices=sorted(DEFAULTS), default=None)
    ap.add_argument("--rows", type=int, default=None)
    ap.add_argument("--cols", type=int, default=None)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="bf16")
    ap.add_argument("--reps", type=int, default=21)
    a = ap.parse_args(argv)
    dt = torch.float32 if a.dtype == "f32" else torch.bfloat16
    for op in [a.op] if a.op else sorted(DEFAULTS):
        N, C = a.rows or DEFAULTS[op][0], a.cols or DEFAULTS[op][1]
        n = N * C * (4 if a.dtype == "f32" else 2)
        label = f"{op} {N}x{C} {a.dtype}"
        xs = [torch.randn(N, C, device="cuda").to(dt) for _ in range(3)]
        if op == "norm":
            w, b = torch.ones(C, device="cuda", dtype=dt), torch.zeros(C, device="cuda", dtype=dt)
            stats = [(x, x.flip(0), *det.layer_norm_forward(x, w, b)[1:]) for x in xs]
            timed(label + " forward", lambda x: det.layer_norm(x, w, b), [(x,) for x in xs], 2 * n, a.reps)
            timed(label + " gradient", lambda x, dy, m, r: det.layer_norm_backward(dy, x, w, m, r), stats, 3 * n,
                  a.reps)
            continue
        t = torch.randint(0, C, (N,), device="cuda")
        if op in ("score", "top"):
            top = 20 if op == "top" else 0
            timed(label + " forward", lambda x: det.token_logprobs(x, t, top=top), [(x,) for x in xs], n, a.reps)
            if op == "top":
                continue
            stats = [(x, det.token_logprobs_forward(x, t)[1]) for x in xs]
            g = torch.rand(N, device="cuda")
            timed(label + " gradient", lambda x, s: det.token_logprobs_backward(x, t, s, g_logprob=g, g_entropy=g),
                  stats, 2 * n, a.reps)
            continue
        K = 64
        teacher, index = torch.randn(N, K, device="cuda"), torch.randint(0, C, (N, K), device="cuda")
        timed(label + " forward", lambda x: det.distill_forward(x, teacher, index), [(x,) for x in xs], n, a.reps)
        stats = [(x, *det.distill_forward(x, teacher, index)[1:]) for x in xs]
        g = torch.rand(N, device="cuda")
        timed(label + " gradient", lambda x, s, q: det.distill_backward(x, index, s, q, g), stats, 2 * n, a.reps)


if __name__ == "__main__":
    main()
