"""Host side of the 8-bit path (CPU only): size queries, views, refusals before
any device work, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_activation_quantization_b200 as sq
from oracle import fp8 as O


@pytest.fixture(scope="module")
def L():
    from sparse_activation_quantization_b200 import build
    build.build()
    return sq.lib()


BASE = 1 << 20  # a fake, aligned address: no call below reaches the device


def act(T=4, K=256, lds=4, codes=BASE, scales=BASE + (1 << 16)):
    return sq.SharqFp8Act(codes, scales, T, K, lds)


def weight(K=256, D=256, E=1, codes=BASE, scales=BASE + (1 << 18)):
    return sq.SharqFp8Weight(codes, scales, K, D, E)


def test_sizes(L):
    assert sq.sharq_fp8_weight_bytes(256, 256, 1) == 65536 + 256
    assert sq.sharq_fp8_weight_bytes(2000, 1111, 3) >= 3 * (2000 * 1111 + 4 * 16 * 9)
    assert sq.sharq_fp8_act_bytes(5, 272) >= 5 * 272 + 3 * 8 * 4
    assert sq.sharq_fp8_act_bytes(0, 16) > 0
    for K, D, E in [(0, 16, 1), (8, 16, 1), (24, 16, 1), (16, 0, 1), (16, 16, 0), (1 << 18, 16, 1), (16, 1 << 19, 1)]:
        assert sq.sharq_fp8_weight_bytes(K, D, E) == 0
    assert sq.sharq_fp8_act_bytes(-1, 16) == 0 and sq.sharq_fp8_act_bytes(1, 20) == 0
    assert sq.sharq_fp8_linear_workspace_bytes(1, 256, 1) >= 4
    assert sq.sharq_fp8_linear_workspace_bytes(1, 250, 1) == 0
    assert sq.sharq_fp8_moe_workspace_bytes(64, 8, 2048, 768, 128) >= 64 * 8 * 768 * 4
    for bad in [(65, 8, 256, 256, 16), (1, 17, 256, 256, 64), (1, 5, 256, 256, 4), (1, 0, 256, 256, 4),
                (1, 1, 250, 256, 4), (1, 1, 256, 8, 4), (1, 1, 256, 256, 513), (-1, 1, 256, 256, 4)]:
        assert sq.sharq_fp8_moe_workspace_bytes(*bad) == 0


def test_views(L):
    a = sq.sharq_fp8_act_view(BASE, 5, 272)
    assert (a.T, a.K, a.lds) == (5, 272, 8) and a.codes == BASE and a.scales % 16 == 0
    assert a.codes + 5 * 272 <= a.scales and a.scales + 3 * 8 * 4 <= BASE + sq.sharq_fp8_act_bytes(5, 272)
    w = sq.sharq_fp8_weight_view(BASE, 272, 300, 2)
    assert (w.K, w.D, w.E) == (272, 300, 2)
    assert w.codes + 2 * 272 * 300 <= w.scales
    assert w.scales + 2 * 3 * 3 * 4 <= BASE + sq.sharq_fp8_weight_bytes(272, 300, 2)
    for call in (lambda: sq.sharq_fp8_act_view(BASE + 8, 5, 272), lambda: sq.sharq_fp8_weight_view(BASE + 16, 272, 3)):
        with pytest.raises(sq.SharqError) as e:
            call()
        assert e.value.status == -1
    with pytest.raises(sq.SharqError) as e:
        sq.sharq_fp8_act_view(BASE, 5, 270)
    assert e.value.status == -2


X, Y, G = BASE + (1 << 22), BASE + (1 << 24), BASE + (1 << 26)


@pytest.mark.parametrize("args,status", [
    ((X, 256, None, 1e-5, None), -1),                        # no act
    ((X, 256, None, 1e-5, act(K=250)), -2),
    ((X, 256, None, 1e-5, act(T=-1)), -2),
    ((X, 256, None, 1e-5, act(lds=3)), -1),                  # lds < T
    ((X, 256, None, 1e-5, act(lds=6)), -1),                  # lds % 4
    ((X, 256, None, 1e-5, act(codes=None)), -1),
    ((X, 256, None, 1e-5, act(codes=BASE + 8)), -1),
    ((X, 256, None, 1e-5, act(scales=BASE + 4)), -1),
    ((None, 256, None, 1e-5, act()), -1),
    ((X + 8, 256, None, 1e-5, act()), -1),                   # misaligned input
    ((X, 252, None, 1e-5, act()), -1),                       # stride < K
    ((X, 260, None, 1e-5, act()), -1),                       # stride % 8
    ((X, 256, G + 2, 1e-5, act()), -1),
    ((X, 256, G, -1.0, act()), -1),
    ((X, 256, G, float("nan"), act()), -1),
])
def test_prep_refusals(L, args, status):
    x, ldx, g, eps, a = args
    assert L.sharq_fp8_prep(x, ldx, g, eps, ctypes.byref(a) if a is not None else None, None) == status


@pytest.mark.parametrize("out,ldo", [
    (X, 256),              # the sublayer's output itself
    (X + 512 * 2, 256),    # its rows from the second on
    (Y + 16, 256),         # the stream, shifted
    (Y, 512),              # the stream's first row in another stride
    (Y + 8, 256),
])
def test_residual_overlaps_are_refused(L, out, ldo):
    a = act()
    assert L.sharq_fp8_prep_residual(X, 256, Y, 256, out, ldo, None, 1e-5, ctypes.byref(a), None) == -1


def test_silu_refusals(L):
    a = act()
    assert L.sharq_fp8_prep_silu_mul(X, 256, None, 256, ctypes.byref(a), None) == -1
    assert L.sharq_fp8_prep_silu_mul(X, 256, Y, 128, ctypes.byref(a), None) == -1


def test_linear_refusals(L):
    def call(a=None, w=None, y=Y, ldy=256, dt=0, ws=G, n=256):
        return L.sharq_fp8_linear(ctypes.byref(a or act()), ctypes.byref(w or weight()), y, ldy, dt, ws, n, None)
    assert call(w=weight(K=512)) == -2
    assert call(w=weight(E=2)) == -1
    assert call(w=weight(D=0)) == -2
    assert call(w=weight(codes=BASE + 4)) == -1
    assert call(w=weight(scales=None)) == -1
    assert call(y=None) == -1
    assert call(y=Y + 1) == -1
    assert call(y=Y + 2, dt=1) == -1
    assert call(ldy=255) == -1
    assert call(dt=7) == -1
    assert call(ws=None) == -6 and call(n=16) == -6 and call(ws=G + 4) == -6
    assert L.sharq_fp8_linear(None, ctypes.byref(weight()), Y, 256, 0, G, 256, None) == -1
    assert L.sharq_fp8_pack_weight(None, ctypes.byref(weight()), None) == -1
    assert L.sharq_fp8_pack_weight(X, None, None) == -1


def test_moe_refusals(L):
    w13, w2 = weight(K=256, D=512, E=8), weight(K=256, D=256, E=8)
    n = sq.sharq_fp8_moe_workspace_bytes(4, 2, 256, 256, 8)

    def call(x=X, ldx=256, lg=Y, ldl=8, T=4, k=2, a=w13, b=w2, y=Y, ldy=256, ids=None, p=None, ws=G, ws_n=n):
        return L.sharq_fp8_moe(x, ldx, lg, ldl, T, k, 1, ctypes.byref(a), ctypes.byref(b), y, ldy, ids, p, ws, ws_n,
                               None)
    assert call(T=65) == -2 and call(T=-1) == -2
    assert call(k=0) == -2 and call(k=9) == -2 and call(k=17) == -2
    assert call(b=weight(K=128, D=256, E=8)) == -2     # I of w2 is not half of w13's rows
    assert call(b=weight(K=256, D=128, E=8)) == -2
    assert call(b=weight(K=256, D=256, E=4)) == -2
    assert call(x=None) == -1 and call(x=X + 4) == -1 and call(ldx=250) == -1
    assert call(lg=None) == -1 and call(ldl=7) == -1
    assert call(y=None) == -1 and call(ldy=255) == -1
    assert call(ids=Y + 2) == -1 and call(p=Y + 1) == -1
    assert call(ws=None) == -6 and call(ws_n=n - 1) == -6


def test_conveniences_check_before_the_library():
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    for bad in (lambda: sq.Fp8Weight(t), lambda: sq.Fp8Weight.from_parts(t, t), lambda: sq.Fp8Act.from_parts(t, t)):
        with pytest.raises(TypeError):
            bad()


# ------------------------------------------------------------- oracle pins ---


def test_oracle_e4m3_rounds_as_the_format():
    """every E4M3 value is a fixed point, midpoints go to the even mantissa"""
    vals = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_round(vals), vals) and vals[-1] == 448
    mid = (vals[:-1] + vals[1:]) / 2
    want = np.where(np.arange(126) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(O.e4m3_round(mid), want)
    assert O.e4m3_round(1e9) == 448 and O.e4m3_round(-460.0) == -448
    x = np.random.default_rng(0).standard_normal(20000) * np.exp(np.random.default_rng(1).uniform(-9, 5, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_round(x), got)


def test_oracle_quant_scales():
    v = np.zeros((2, 272), np.float32)
    v[0, 3], v[0, 200], v[1, 271] = -7.0, 448.0, 1e-38
    q, s = O.quant(v)
    assert s[0, 0] == np.float32(7.0) / np.float32(448) and s[0, 1] == 1.0 and s[0, 2] == 1.0
    assert s[1, 2] == np.float32(2.0 ** -126) and q[0, 3] == -448 and q[0, 200] == 448


def test_oracle_routing_ties_and_empty():
    lg = np.array([[1.0, 3.0, 3.0, 3.0], [-np.inf, -np.inf, -np.inf, -np.inf], [0.0, -np.inf, np.nan, -1.0]])
    ids, p = O.route(lg, 2)
    assert ids[0].tolist() == [1, 2] and np.allclose(p[0], 0.5)
    assert ids[1].tolist() == [0, 1] and not p[1].any()
    assert ids[2].tolist() == [0, 3] and abs(p[2].sum() - 1) < 1e-15
    ids, p = O.route(lg, 4, renormalize=False)
    assert ids[2].tolist() == [0, 3, 1, 2] and p[2, 2] == 0 and p[2, 3] == 0
