"""The 8-bit path at the ends of what its calls accept (GPU), against oracle/fp8.py with the bounds of
tests/test_gpu_fp8.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_activation_quantization_b200 as sq
import synthetic
from oracle import fp8 as O
from tests import gpu_helpers as H
from tests.gpu_helpers import bf16_dev as bf
from tests.test_fp8_limits_host import groups_of, skewed_choices
from tests.test_gpu_fp8 import (F8, Layer, check_linear, check_moe, check_quant, check_untouched, f64, linear_reference,
                                make_act, moe_inputs, norm_delta, operands)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


@pytest.mark.parametrize("T,E,topk", [(1, 2, 1), (2, 3, 2), (9, 8, 1), (40, 3, 2)])
def test_moe_of_more_row_tiles_than_share_sums(T, E, topk):
    """65 tiles of 128 rows in down: no tile is shared by several clusters"""
    args = moe_inputs(T, E, 8208, 32, 31)
    check_moe(fp8_moe(*args, topk), *args, topk)


@pytest.mark.parametrize("T,E,topk", [(1, 16, 4), (8, 16, 4), (9, 16, 4), (17, 16, 2), (64, 256, 8), (64, 16, 4)])
def test_moe_error_word_stays_clear(T, E, topk):
    args = moe_inputs(T, E, 640, 144, 32)
    check_moe(fp8_moe(*args, topk), *args, topk)


def test_layer_error_words_stay_clear():
    layer = Layer(48, seed=33)
    layer.run()
    layer.check()
    assert layer.wm.check() == 0


def test_library_functions_by_their_names():
    """the sharq_fp8_* functions on plain addresses write the bits that the torch conveniences return"""
    T, K, D, stream = 12, 272, 136, torch.cuda.current_stream().cuda_stream
    W, X, R = (bf(synthetic.weights(41, K, D)), bf(synthetic.activations(42, T, K)), bf(synthetic.activations(43, T, K)))
    G = bf(synthetic.gamma(44, K))

    def buffer(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    wb, ab = buffer(sq.sharq_fp8_weight_bytes(K, D)), buffer(sq.sharq_fp8_act_bytes(T, K))
    w, a = sq.sharq_fp8_weight_view(wb.data_ptr(), K, D), sq.sharq_fp8_act_view(ab.data_ptr(), T, K)
    sq.sharq_fp8_pack_weight(W.data_ptr(), w, stream)
    weight, act = sq.Fp8Weight(W), sq.Fp8Act(T, K)
    assert torch.equal(wb[:K * D], weight.codes.view(torch.uint8).reshape(-1))
    off = w.scales - w.codes
    assert torch.equal(wb[off:off + weight.scales.numel() * 4].view(torch.float32), weight.scales.reshape(-1))

    def same():
        b = O.blocks(K)
        sc = ab[a.scales - a.codes:][:4 * b * a.lds].view(torch.float32).view(b, a.lds)[:, :T].t()
        return torch.equal(ab[:T * K], act.codes.view(torch.uint8).reshape(-1)) and torch.equal(sc, act.scales)

    sq.sharq_fp8_prep(X.data_ptr(), K, G.data_ptr(), 1e-5, a, stream)
    act.prep(X, G)
    assert same()
    gu = torch.cat([X, R], 1)
    sq.sharq_fp8_prep_silu_mul(gu.data_ptr(), 2 * K, gu.data_ptr() + 2 * K, 2 * K, a, stream)
    act.prep_silu_mul(gu[:, :K], gu[:, K:])
    assert same()
    out = torch.empty_like(R)
    sq.sharq_fp8_prep_residual(X.data_ptr(), K, R.data_ptr(), K, out.data_ptr(), K, G.data_ptr(), 1e-5, a, stream)
    act.prep_residual(X, R, R, G)
    assert same() and torch.equal(out, R)
    ws, y = buffer(sq.sharq_fp8_linear_workspace_bytes(T, K, D)), torch.empty(T, D, device="cuda")
    sq.sharq_fp8_linear(a, w, y.data_ptr(), D, sq.SHARQ_OUT_F32, ws.data_ptr(), ws.numel(), stream)
    assert torch.equal(y, sq.fp8_linear(act, weight, out_dtype=torch.float32))
    x, lg, *parts = (t.cuda() for t in moe_inputs(T, 6, 256, 64, 45))
    w13, w2 = sq.Fp8Weight.from_parts(*parts[:2]), sq.Fp8Weight.from_parts(*parts[2:])
    wm, y = buffer(sq.sharq_fp8_moe_workspace_bytes(T, 2, 256, 64, 6)), torch.empty_like(x)
    ids, p = torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda")
    sq.sharq_fp8_moe(x.data_ptr(), 256, lg.data_ptr(), 6, T, 2, 1, w13.view, w2.view, y.data_ptr(), 256, ids.data_ptr(),
                     p.data_ptr(), wm.data_ptr(), wm.numel(), stream)
    for got, want in zip((y, ids, p), sq.fp8_moe(x, lg, w13, w2, 2, return_routing=True)):
        assert torch.equal(got, want)
    assert sq.sharq_check_status(ws.data_ptr(), stream) == 0 and sq.sharq_check_status(wm.data_ptr(), stream) == 0
    with pytest.raises(sq.SharqError):
        sq.sharq_fp8_linear(a, w, y.data_ptr(), D, sq.SHARQ_OUT_F32, ws.data_ptr(), 16, stream)


def test_captured_layers_replayed_at_once():
    """two graphs with a workspace each, replayed side by side on two streams"""
    layers, graphs, want = [Layer(16, seed=51), Layer(64, seed=52)], [], []
    for la in layers:
        la.run()
        torch.cuda.synchronize()
        want.append(la.outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            la.run()
        graphs.append(g)
    for la in layers:
        for t in (la.h, la.gu, la.down, la.y):
            t.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for la, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(la.outputs(), w))
        assert la.ws.check() == 0 and la.wm.check() == 0


def test_beside_the_fp4_path_on_another_stream():
    """both paths' kernels hold TMEM and clusters on the same SMs"""
    T, K, D = 600, 1024, 2048
    fp4 = sq.PackedWeight(bf(synthetic.weights(61, K, D)))
    x, gamma = bf(synthetic.activations(62, T, K)), bf(synthetic.gamma(63, K))
    rows = {n: (sq.PreparedAct(n, K), sq.Workspace(n, K, D)) for n in (8, T)}

    def four(stream=None):
        return [sq.linear(a.prep(x[:n], gamma, 1e-5, stream=stream), fp4, ws=ws, stream=stream)
                for n, (a, ws) in rows.items()]

    layers = [Layer(n, seed=64 + n) for n in (8, 64)]
    want4 = four()
    for la in layers:
        la.run()
    torch.cuda.synchronize()
    want8 = [la.outputs() for la in layers]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            got4 = four(a)
        for la in layers:
            la.run(stream=b)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got4, want4))
    for la, w in zip(layers, want8):
        assert all(torch.equal(g, v) for g, v in zip(la.outputs(), w)) and la.wm.check() == 0
    assert all(ws.check() == 0 for _, ws in rows.values())


FIRST = """
import torch
import sparse_activation_quantization_b200 as sq
from tests.test_gpu_fp8 import Layer
layer, g = Layer(%d, seed=71), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    layer.run()
layer.y.fill_(float("nan"))
g.replay()
layer.check()
assert layer.wm.check() == 0
print("captured first")
"""


@pytest.mark.parametrize("T", [3, 40])
def test_first_call_of_a_process_may_be_captured(T):
    """what a kernel's first launch looks up (attributes, resident clusters) is allowed while a stream is captured"""
    r = subprocess.run([sys.executable, "-c", FIRST % T], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------- the largest of each size ---


@pytest.mark.parametrize("T,K,D", [(1, 131072, 40), (40, 131072, 130), (70, 131072, 24), (300, 131072, 140),  # sums of 1024 blocks
                                   (1, 16, 262144), (65, 16, 262144),
                                   (300001, 16, 9), (70000, 144, 16)])
def test_linear_of_the_largest_sizes(T, K, D):
    x, xs, w, ws = operands(T, K, D, 3)
    act = sq.Fp8Act.from_parts(x.cuda(), xs.cuda())
    wt = sq.Fp8Weight.from_parts(w.cuda(), ws.cuda())
    work = sq.Fp8Workspace.for_linear(T, K, D)
    y = sq.fp8_linear(act, wt, out_dtype=torch.float32, ws=work)
    ref, bound = linear_reference(x, xs, w, ws)
    check_linear(y, ref, bound, torch.float32)
    assert work.check() == 0


@pytest.mark.parametrize("T,K", [(2, 131072), (70001, 16), (70001, 272)])
def test_prep_of_the_largest_sizes(T, K):
    x, r, gamma = synthetic.activations(91, T, K), synthetic.activations(92, T, K), synthetic.gamma(93, K)
    act, codes, scales = make_act(T, K)
    X, R, G = bf(x), bf(r), bf(gamma)
    act.prep(X)
    q, s = O.quant(x)
    assert np.array_equal(act.scales.cpu().numpy(), s) and np.array_equal(f64(act.codes.float()), q)
    act.prep(X, G)
    check_quant(act, O.rms_norm(x, gamma, np.float32(1e-5)), norm_delta(K))
    act.prep_silu_mul(X, R)
    check_quant(act, O.silu(x) * r, (2 + 1.2 * 88 + 8) * 2.0 ** -23)
    act.prep_residual(X, R, R, G)
    h = (torch.from_numpy(x) + torch.from_numpy(r)).bfloat16()
    assert torch.equal(R.cpu(), h)
    check_quant(act, O.rms_norm(h.float().numpy(), gamma, np.float32(1e-5)), norm_delta(K))
    check_untouched(act, codes, scales)


@pytest.mark.parametrize("E,K,D", [(1, 131072, 17), (1, 16, 262144), (4096, 16, 3), (3, 144, 70000)])
def test_pack_of_the_largest_sizes(E, K, D):
    W = synthetic.weights(94, E * K, D).reshape(E, K, D)
    w = sq.Fp8Weight(bf(W))
    codes, scales = f64(w.codes.float()), w.scales.cpu().numpy()
    for e in range(0, E, max(1, E // 8)):
        q, s = O.pack(W[e])
        assert np.array_equal(scales[e], s) and np.array_equal(codes[e], q)


@pytest.mark.parametrize("T,E,topk,Hd,I", [(1, 1, 1, 131072, 16), (9, 3, 1, 131072, 16), (33, 2, 2, 131072, 16),
                                           (1, 2, 1, 16, 131072), (9, 4, 1, 16, 131072), (34, 2, 1, 16, 131072)])
def test_moe_of_the_largest_sizes(T, E, topk, Hd, I):
    args = moe_inputs(T, E, Hd, I, 95)
    if I == 131072:  # sums of 131072 products: keeps |W2| within what check_moe takes
        args = (*args[:5], args[5] * 2.0 ** -4)
    check_moe(fp8_moe(*args, topk), *args, topk)


def test_rows_further_apart_than_32_bits_say():
    """strides of more than 2^31 elements: input, output and in-place stream"""
    far, T, K, D = 2 ** 31 + 8, 3, 272, 24
    big = torch.empty(2 * far + K, dtype=torch.bfloat16, device="cuda")
    x, r = synthetic.activations(96, T, K), synthetic.activations(97, T, K)
    X = big.as_strided((T, K), (far, 1))
    X.copy_(bf(x))
    act, near = sq.Fp8Act(T, K), sq.Fp8Act(T, K)
    act.prep(X)
    near.prep(bf(x))
    assert torch.equal(act.codes.view(torch.uint8), near.codes.view(torch.uint8)) and torch.equal(act.scales, near.scales)
    G = bf(synthetic.gamma(98, K))
    act.prep_residual(bf(r), X, X, G)  # the stream is updated where it lies
    R = bf(x)
    near.prep_residual(bf(r), R, R, G)
    assert torch.equal(X, R) and torch.equal(act.codes.view(torch.uint8), near.codes.view(torch.uint8))
    w = sq.Fp8Weight(bf(synthetic.weights(99, K, D)))
    out = big.as_strided((T, D), (far, 1))
    sq.fp8_linear(near, w, out=out)
    assert torch.equal(out, sq.fp8_linear(near, w))
    x, lg, *p = (t.cuda() for t in moe_inputs(3, 4, K, 48, 101))
    a, b = sq.Fp8Weight.from_parts(*p[:2]), sq.Fp8Weight.from_parts(*p[2:])
    want = sq.fp8_moe(x, lg, a, b, 2)
    X.copy_(x)
    assert torch.equal(sq.fp8_moe(X, lg, a, b, 2, out=X), want)
    del big, X
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E,topk", [(129, 1), (300, 16), (512, 3)])
def test_moe_without_renormalizing_over_many_experts(E, topk):
    args = moe_inputs(7, E, 128, 32, 102, spread=3.0)
    check_moe(fp8_moe(*args, topk, renormalize=False), *args, topk, renormalize=False)


def test_two_threads_call_at_once():
    """the host side's tables (attributes, resident clusters) are filled by whoever comes first"""
    code = """
import threading, torch
from tests.test_gpu_fp8 import Layer
layers = [Layer(5, seed=111), Layer(40, seed=112)]
streams = [torch.cuda.Stream() for _ in layers]
torch.cuda.synchronize()
def work(la, s):
    torch.cuda.set_device(0)
    for _ in range(30):
        la.run(stream=s)
ts = [threading.Thread(target=work, args=a) for a in zip(layers, streams)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
for la in layers:
    la.check()
    assert la.wm.check() == 0
print("both right")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "both right" in r.stdout, r.stderr[-2000:]
