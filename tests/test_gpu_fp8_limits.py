"""The 8-bit path at the ends of what its calls accept (GPU), against oracle/fp8.py with the bounds of
tests/test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

import sparse_activation_quantization_b200 as sq
from oracle import fp8 as O
from tests import gpu_helpers as H
from tests.test_fp8_limits_host import groups_of, skewed_choices
from tests.test_gpu_fp8 import (F8, check_linear, check_moe, check_quant, check_untouched, f64, linear_reference,
                                make_act, moe_inputs, norm_delta, operands)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.ensure_built()


def fp8_moe(x, lg, w13, s13, w2, s2, topk, **kw):
    """fp8_moe with a workspace of its own, whose error word is read"""
    a, b = sq.Fp8Weight.from_parts(w13.cuda(), s13.cuda()), sq.Fp8Weight.from_parts(w2.cuda(), s2.cuda())
    ws = sq.Fp8Workspace.for_moe(x.shape[0], topk, a, b)
    out = sq.fp8_moe(x.cuda(), lg.cuda(), a, b, topk, ws=ws, return_routing=True, **kw)
    assert ws.check() == 0
    return out


@pytest.mark.parametrize("topk", [13, 16])
@pytest.mark.parametrize("Hd,I", [(128, 32), (272, 80)])
def test_moe_routing_with_the_most_groups(topk, Hd, I):
    """64 tokens over all of 512 experts, 64 of them chosen by nine tokens (topk = 16): groups of 8, 576 of them"""
    x, lg, *w = moe_inputs(64, 512, Hd, I, 21)
    ids = torch.from_numpy(skewed_choices())
    lg = (lg * 0.25).clamp(-4, 4)
    lg.scatter_(1, ids, lg.gather(1, ids) + 10)
    assert topk < 16 or groups_of(np.bincount(lg.topk(topk).indices.reshape(-1), minlength=512), 8) == 576
    out = fp8_moe(x, lg, *w, topk)
    check_moe(out, x, lg, *w, topk)
    again = fp8_moe(x, lg, *w, topk)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,K,x_exp,gamma_exp", [
    (3, 64, 56, 74), (3, 64, -45, -110),         # a warp per row
    (3, 2064, 54, 76), (3, 2064, -48, -105),     # a vector per thread
    (160, 1040, 54, 76), (160, 1040, -47, -106),  # four vectors per thread
    (2, 33008, 50, 80), (2, 33008, -50, -105),   # rows that are read twice
])
def test_prep_norm_before_gamma(T, K, x_exp, gamma_exp, residual):
    """x * (1 / rms) * gamma from left to right: x * gamma leaves float32, x / rms and the result do not"""
    g = np.random.default_rng(T + K)
    x = torch.from_numpy(((g.random((T, K)) + 1) * g.choice([-1.0, 1.0], (T, K)) * 2.0 ** x_exp).astype(np.float32))
    gamma = torch.from_numpy(((g.random(K) + 0.5) * 2.0 ** gamma_exp).astype(np.float32))
    x, gamma = x.bfloat16(), gamma.bfloat16()
    act, codes, scales = make_act(T, K)
    if residual:
        act.prep_residual(x.cuda(), torch.zeros_like(x).cuda(), None, gamma.cuda(), 0.0)
    else:
        act.prep(x.cuda(), gamma.cuda(), 0.0)
    check_quant(act, O.rms_norm(x.float().numpy(), gamma.float().numpy(), 0.0), norm_delta(K))
    check_untouched(act, codes, scales)


def test_scale_columns_further_apart_than_32_bits_say():
    """the struct holds the distance of two columns as an int: beyond that the scales are copied"""
    far = 2 ** 32 + 4
    x, xs, w, ws = operands(4, 256, 40, 7)
    big = torch.empty(2 * far, device="cuda")
    scales = big.as_strided((4, 2), (1, far))
    scales.copy_(xs)
    big[4:8] = -1.0  # where a distance cut to 32 bits would look
    act = sq.Fp8Act.from_parts(x.cuda(), scales)
    assert act.scales.data_ptr() != big.data_ptr() and torch.equal(act.scales.cpu(), xs)
    y = sq.fp8_linear(act, sq.Fp8Weight.from_parts(w.cuda(), ws.cuda()))
    ref, bound = linear_reference(x, xs, w, ws)
    check_linear(y, ref, bound, torch.bfloat16)
    del big, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,E", [(1, 1), (12, 4), (64, 1)])  # one token; groups of 8; groups of 32
def test_moe_h_of_one_block_from_large_to_small(T, E):
    """y = h through a unit w2: h is off by 2^-12 of itself or 2^-25 of its block's largest, and bf16 (8 significant bits,
    so a spacing of 2^-7 from 1 to 2) by half a spacing, 2^-8 of itself"""
    n = 128
    x = torch.zeros(T, n, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    w13 = torch.zeros(E, 2 * n, n)
    w13[:, :n, 0] = torch.exp2(torch.arange(n) % 13 - 9.0)             # gates from 2^-9 to 8
    w13[:, n:, 0] = torch.exp2(torch.arange(n) // 8 - 8.0) * 1.125     # up from 2^-8 to 2^7
    one13, one2 = torch.ones(E, 2, 1), torch.ones(E, 1, 1)
    w2 = torch.eye(n).repeat(E, 1, 1)
    lg = torch.full((T, E), -100.0)
    lg[:, 0] = 100.0
    y, ids, p = fp8_moe(x, lg, w13.to(F8), one13, w2.to(F8), one2, 1)
    assert (ids == 0).all() and (p == 1).all()
    v = f64(w13.to(F8)[0, :, 0])  # what the codes hold: 1.125 * 2^-8 lies between two of E4M3's smallest numbers
    h = O.silu(v[:n]) * v[n:]
    assert h.max() / h.min() > 2.0 ** 25
    own = np.maximum(2.0 ** -12 * np.abs(h), 2.0 ** -25 * np.abs(h).max()) + 2.0 ** -18 * np.abs(h)  # and silu, float32 sums
    err = np.abs(f64(y) - h)
    assert (err <= own + 2.0 ** -8 * (np.abs(h) + own)).all()
    assert (err > 2.0 ** -11 * np.abs(h) + 2.0 ** -8 * np.abs(h)).any()  # so 2^-12 of itself alone does not hold
