"""The 8-bit path's fixed tables against the largest calls that it accepts (CPU only)."""
import os
import re

import numpy as np
import pytest

import sparse_activation_quantization_b200 as sq

CSRC = os.path.join(os.path.dirname(sq.__file__), "csrc")


def constants(name):
    """the integer constants of a source file that are written as `constexpr int a = ..., b = ...;`"""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = {}
    for line in re.findall(r"constexpr int ([^;]*);", text):
        for part in line.split(","):
            key, _, expr = part.partition("=")
            try:
                found.setdefault(key.strip(), eval(expr.replace("/", "//"), {"__builtins__": {}}, found))
            except (NameError, SyntaxError, TypeError):
                pass  # depends on a template's parameter
    return found


def skewed_choices(T=64, topk=16, E=512):
    """[T, topk] experts, distinct in a row, that make as many groups of 8 as `T` tokens can: 64 experts of nine tokens
    each and 448 of one"""
    assert (T, topk, E) == (64, 16, 512)
    t = np.arange(T)[:, None]
    return np.concatenate([(t + np.arange(9)) % 64, 64 + 7 * t + np.arange(7)], axis=1)


def groups_of(counts, size):
    return int(sum(-(-int(c) // size) for c in counts))


def most_groups(T, topk, E, size):
    """over every routing of T tokens: n experts of one token each are n groups, and each further `size` tokens of an
    expert (of T at most) one more"""
    n = min(E, T * topk)
    return min(n + (T * topk - n) // size, E * -(-T // size))


def test_skewed_routing_is_the_worst():
    ids = skewed_choices()
    assert all(len(set(row)) == 16 for row in ids.tolist()) and ids.min() == 0 and ids.max() == 511
    counts = np.bincount(ids.reshape(-1), minlength=512)
    assert groups_of(counts, 8) == most_groups(64, 16, 512, 8) == 576


@pytest.mark.parametrize("E", [1, 2, 16, 64, 100, 255, 256, 300, 511, 512])
def test_moe_group_table_holds_every_routing(E):
    c = constants("fp8_moe.cu")
    assert (c["kMoeMaxTokens"], c["kMoeMaxTopk"], c["kMoeMaxExperts"]) == (
        sq.SHARQ_FP8_MOE_MAX_T, sq.SHARQ_FP8_MOE_MAX_TOPK, sq.SHARQ_FP8_MOE_MAX_E)
    for T in range(1, 65):
        for topk in range(1, min(16, E) + 1):
            small = T <= c["kSmallGroup"] or T * topk <= 4 * E  # launch_moe
            size = c["kSmallGroup"] if small else c["kGroup"]
            assert most_groups(T, topk, E, size) <= c["kMaxGroups"]


@pytest.mark.parametrize("device", ["cpu", "cpu:0", "meta"])
def test_buffers_are_cuda_buffers(device):
    """a kernel would be given the address of host memory"""
    from sparse_activation_quantization_b200 import build
    build.build()
    for make in (lambda: sq.Fp8Act(4, 256, device=device), lambda: sq.Fp8Workspace(256, device=device),
                 lambda: sq.Fp8Workspace.for_linear(4, 256, 256, device=device)):
        with pytest.raises(ValueError, match="CUDA device"):
            make()
