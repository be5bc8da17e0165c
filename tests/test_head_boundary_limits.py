"""The limits that Python repeats are the header's (CPU)."""
import os
import re

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from bitwise_deterministic_exact_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _header(name: str) -> int:
    with open(os.path.join(ROOT, "include", "detgemm.h")) as f:
        value = re.search(rf"^#define {name} (.+?)(?:/\*.*)?$", f.read(), re.M).group(1)
    return eval(value.replace("(int64_t)", ""))


def test_python_limits_are_the_headers():
    assert _lib.NORM_C_MAX == _header("DET_NORM_C_MAX")
    assert _lib.NORM_SHARD_ROWS == det.NORM_SHARD_ROWS == _header("DET_NORM_SHARD_ROWS")


def test_both_layers_refuse_from_the_header_s_limits_on():
    top, entries = _header("DET_HEAD_TOP_MAX"), _header("DET_HEAD_ENTRIES_MAX")
    lib = _lib.load()
    assert lib.det_head_workspace_bytes(1, 1 << 20, top) > 0 and lib.det_head_workspace_bytes(1, 1 << 20, top + 1) == 0
    z = torch.empty(1, 9999, device="meta")

    def teacher(k):
        return torch.empty(1, k, device="meta"), torch.empty(1, k, dtype=torch.int64, device="meta")
    for call, match in ((lambda: det.token_logprobs(z, top=top), "GPU"), (lambda: det.token_logprobs(z, top=top + 1), "top"),
                        (lambda: det.distill_loss(z, *teacher(entries)), "GPU"),
                        (lambda: det.distill_loss(z, *teacher(entries + 1)), str(entries))):
        with pytest.raises(ValueError, match=match):
            call()
