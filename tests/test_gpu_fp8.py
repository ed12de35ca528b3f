"""The 8-bit (E4M3, block-scaled) path on the GPU against oracle/fp8.py.

Tolerances.  A quantized value: half an E4M3 step (2^-4 relative, 2^-10 of the
scale below the smallest normal) plus the float32 error of the value itself.
A product of two E4M3 values has at most 8 significant bits, so it is exact in
float32; a sum of n of them is off by at most n 2^-23 of the sum of magnitudes
(also where an adder truncates), and so are sums of scaled blocks.  One final
rounding: 2^-8 (bf16).
"""
import numpy as np
import pytest
import torch

import sparse_activation_quantization_b200 as sq
import synthetic
from oracle import fp8 as O
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.ensure_built()


def values(codes):
    return codes.float().double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def strided(x, pad):
    """bf16 CUDA tensor whose rows lie x.shape[1] + pad apart, and its whole buffer (NaN between)"""
    T, K = x.shape
    buf = torch.full((T, K + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :K] = H.bf16_dev(x)
    return buf[:, :K], buf


def make_act(T, K, lds_pad=0):
    """Fp8Act over a buffer full of 0xAB with `lds_pad` more scale columns than rows"""
    lds = -(-T // 4) * 4 + lds_pad
    codes = torch.full((T * K + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((O.blocks(K), lds), -7.0, device="cuda")
    act = sq.Fp8Act.from_parts(codes[:T * K].view(F8).view(T, K), scales[:, :T].t())
    assert act.codes.data_ptr() == codes.data_ptr() and act.scales.data_ptr() == scales.data_ptr()
    return act, codes, scales


def check_untouched(act, codes, scales):
    assert (codes[act.T * act.K:] == 0xAB).all()
    assert (scales[:, act.T:] == -7.0).all()


def check_quant(act, v, delta):
    """codes and scales of `v` (float64), which float32 holds to `delta` relative"""
    T, K = v.shape
    s = f64(act.scales)
    pad = np.zeros((T, O.blocks(K) * 128))
    pad[:, :K] = np.abs(v)
    want = O.block_scale(np.zeros(1))  # dtype only
    amax = pad.reshape(T, -1, 128).max(-1)
    want = np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 1.0)
    assert (np.abs(s - want) <= (delta + 2.0 ** -23) * want).all()
    se = O.expand(s, K, 1)
    err = np.abs(values(act.codes) * se - v)
    # v * f32(1/s) rounds twice in float32 before the code does
    assert (err <= np.abs(v) * (2.0 ** -4 + delta + 2.0 ** -22) + se * 2.0 ** -10 * (1 + 2.0 ** -20)).all()


SHAPES = [(1, 16), (1, 128), (3, 272), (5, 1040), (33, 3584), (7, 8208), (130, 512), (4, 18944), (2, 33008)]


@pytest.mark.parametrize("T,K", SHAPES)
def test_prep_plain_is_bit_exact(T, K):
    x = synthetic.activations(10 + T, T, K)
    x[0, :min(K, 128)] = 0.0  # a block of zeros
    act, codes, scales = make_act(T, K, lds_pad=4)
    X, _ = strided(x, 8)
    act.prep(X)
    q, s = O.quant(x)
    assert np.array_equal(act.scales.cpu().numpy(), s)
    assert np.array_equal(values(act.codes), q)
    check_untouched(act, codes, scales)


def norm_delta(K):
    """relative float32 error of x * 1/rms * gamma: half of the sum's (one thread's chain of squares, ten levels of
    joining, all positive) and eight roundings"""
    return (max(32, K // 1024 + 8) + 20) * 2.0 ** -24


@pytest.mark.parametrize("T,K", SHAPES)
def test_prep_norm(T, K):
    x, gamma = synthetic.activations(20 + T, T, K), synthetic.gamma(21, K)
    act, codes, scales = make_act(T, K)
    X, _ = strided(x, 16)
    act.prep(X, H.bf16_dev(gamma), EPS)
    check_quant(act, O.rms_norm(x, gamma, np.float32(EPS)), norm_delta(K))
    check_untouched(act, codes, scales)


@pytest.mark.parametrize("out", ["new", "inplace", "none"])
@pytest.mark.parametrize("T,K,norm", [(t, k, n) for t, k in SHAPES for n in (True, False)])
def test_prep_residual(T, K, norm, out):
    x = synthetic.activations(30 + T, T, K)
    r = (synthetic.activations(31 + T, T, K) * np.float32(4)).astype(np.float32)
    r[-1] = -x[-1]  # a row that cancels
    h = (torch.from_numpy(x) + torch.from_numpy(r)).bfloat16().float().numpy()
    gamma = synthetic.gamma(32, K) if norm else None
    act, codes, scales = make_act(T, K)
    X, xb = strided(x, 8)
    R, rb = strided(r, 24)
    keep = xb.clone()
    dst, db = {"new": strided(np.zeros_like(x), 40), "inplace": (R, rb), "none": (None, None)}[out]
    act.prep_residual(X, R, dst, H.bf16_dev(gamma) if norm else None, EPS)
    if norm:
        check_quant(act, O.rms_norm(h, gamma, np.float32(EPS)), norm_delta(K))
    else:
        q, s = O.quant(h)
        assert np.array_equal(act.scales.cpu().numpy(), s) and np.array_equal(values(act.codes), q)
    if dst is not None:
        assert np.array_equal(dst.float().cpu().numpy(), h)
        assert db[:, K:].isnan().all()  # between the rows
    if out != "inplace":
        assert np.array_equal(R.float().cpu().numpy(), r)
    assert torch.equal(xb.view(torch.int16), keep.view(torch.int16))
    check_untouched(act, codes, scales)


@pytest.mark.parametrize("T,K", SHAPES)
def test_prep_silu_mul_of_halves(T, K):
    g = synthetic.activations(40 + T, T, K) * np.float32(0.5)
    u = synthetic.activations(41 + T, T, K, base="student_t")
    g[0, :8] = [0.0, -0.0, 80.0, -80.0, 1e4, -1e4, 3e38, -3e38]
    u[0, 6] = 1.0  # 3e38 * 1 stays finite
    u[0, 7] = 1.0
    gu = H.bf16_dev(np.concatenate([g, u], axis=1))
    g, u = f64(gu[:, :K]), f64(gu[:, K:])
    act, codes, scales = make_act(T, K)
    act.prep_silu_mul(gu[:, :K], gu[:, K:])
    # exp of a float32 x by the fast instruction: 2 + 1.2 |x| units of 2^-23 and |x| <= 88 where e^x matters; the
    # quotient 2 more, sum, products and the scale's roundings 6
    check_quant(act, O.silu(g) * u, (2 + 1.2 * 88 + 8) * 2.0 ** -23)
    check_untouched(act, codes, scales)


@pytest.mark.parametrize("mag", [2.0 ** -120, 2.0 ** -60, 2.0 ** 70, 2.0 ** 120])
@pytest.mark.parametrize("K", [512, 4096, 40000])
def test_prep_norm_of_rows_whose_squares_leave_float32(mag, K):
    x = (synthetic.activations(50, 3, K) * np.float32(mag)).astype(np.float32)
    x = torch.from_numpy(x).bfloat16().float().numpy()
    assert np.isfinite(x).all()
    gamma = synthetic.gamma(51, K)
    act, _, _ = make_act(3, K)
    act.prep(H.bf16_dev(x), H.bf16_dev(gamma), 0.0)
    check_quant(act, O.rms_norm(x, gamma, 0.0), norm_delta(K))


@pytest.mark.parametrize("K", [256, 2064])
def test_prep_keeps_non_finite_values_to_their_block_or_row(K):
    x = synthetic.activations(60, 4, K)
    x[1, 3], x[2, 130] = np.nan, np.inf
    act, _, _ = make_act(4, K)
    act.prep(H.bf16_dev(x))
    clean = np.where(np.isfinite(x), x, 0).astype(np.float32)
    q, s = O.quant(clean)
    got, gs = values(act.codes), act.scales.cpu().numpy()
    assert np.isnan(got[1, 3])
    got[1, 3] = q[1, 3]
    deq = got * O.expand(gs.astype(np.float64), K, 1)
    blk = slice(128, min(256, K))
    with np.errstate(invalid="ignore"):
        assert np.isnan(deq[2, blk]).all() or np.isnan(got[2, 130]) and np.isinf(gs[2, 1])
    keep = np.ones_like(x, bool)
    keep[2, blk] = False
    assert np.array_equal(got[keep], q[keep])
    act.prep(H.bf16_dev(x), H.bf16_dev(synthetic.gamma(61, K)), EPS)
    row = values(act.codes)
    assert np.isfinite(row[[0, 3]]).all()
    check = sq.Fp8Act(4, K)
    check.prep(H.bf16_dev(clean), H.bf16_dev(synthetic.gamma(61, K)), EPS)
    assert np.array_equal(row[[0, 3]], values(check.codes)[[0, 3]])


# Rows enough that each thread holds four vectors of one: up to 8192 columns, up to 20480, and beyond
MANY = [(200, 1040), (161, 3584), (300, 4112), (150, 8192), (149, 8208), (5, 20480), (3, 24000)]


@pytest.mark.parametrize("T,K", MANY)
def test_prep_of_many_rows(T, K):
    x = synthetic.activations(80 + K, T, K)
    r = synthetic.activations(81 + K, T, K)
    x[0, :K // 2] = 0.0
    gamma = synthetic.gamma(82, K)
    X, _ = strided(x, 8)
    R, _ = strided(r, 16)
    act, codes, scales = make_act(T, K, lds_pad=4)
    act.prep(X)
    q, s = O.quant(x)
    assert np.array_equal(act.scales.cpu().numpy(), s) and np.array_equal(values(act.codes), q)
    act.prep(X, H.bf16_dev(gamma), EPS)
    check_quant(act, O.rms_norm(x, gamma, np.float32(EPS)), norm_delta(K))
    h = (torch.from_numpy(x) + torch.from_numpy(r)).bfloat16().float().numpy()
    act.prep_residual(X, R, R, H.bf16_dev(gamma), EPS)
    check_quant(act, O.rms_norm(h, gamma, np.float32(EPS)), norm_delta(K))
    assert np.array_equal(R.float().cpu().numpy(), h)
    act.prep_silu_mul(X, R)
    check_quant(act, O.silu(x) * h, (2 + 1.2 * 88 + 8) * 2.0 ** -23)
    check_untouched(act, codes, scales)


@pytest.mark.parametrize("K", [512, 1040, 4096, 9000 // 16 * 16])
def test_prep_norm_of_blocks_far_below_their_row(K):
    """a row of small root mean square with a block so small that its scale is the smallest normal number: the factor
    gamma / rms / scale leaves float32 although the codes are ordinary"""
    x = np.full((3, K), 2.0 ** -20, np.float32)
    x[:, :128] = 2.0 ** -133 * np.arange(1, 129)  # bf16 values, some subnormal
    x[1, :128] = 0.0
    x = torch.from_numpy(x).bfloat16().float().numpy()
    gamma = np.ones(K, np.float32)
    act, _, _ = make_act(3, K)
    act.prep(H.bf16_dev(x), H.bf16_dev(gamma), 0.0)
    v = O.rms_norm(x, gamma, 0.0)
    s = f64(act.scales)
    assert s[1, 0] == 1.0 and (s > 0).all()
    # below 2^-126 a float32 product is off by up to half its spacing 2^-149, which is 2^-24 of the smallest scale
    err = np.abs(values(act.codes) * O.expand(s, K, 1) - v)
    se = O.expand(s, K, 1)
    assert (err <= np.abs(v) * (2.0 ** -4 + norm_delta(K) + 2.0 ** -22) + se * (2.0 ** -10 * (1 + 2.0 ** -20) + 2.0 ** -23)).all()


def test_prep_without_rows():
    act = sq.Fp8Act(0, 256)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    act.prep(e, H.bf16_dev(synthetic.gamma(1, 256))).prep_residual(e, e, e).prep_silu_mul(e, e)
    w = sq.Fp8Weight(H.bf16_dev(synthetic.weights(1, 256, 40)))
    assert sq.fp8_linear(act, w).shape == (0, 40)
    torch.cuda.synchronize()


@pytest.mark.parametrize("E,K,D", [(1, 16, 1), (1, 128, 128), (1, 272, 129), (3, 2000, 1100), (2, 144, 264), (1, 4096, 512), (2, 300 // 16 * 16, 130),
                                   (1, 160, 77)])
def test_pack_is_bit_exact(E, K, D):
    W = synthetic.weights(70 + E, E * K, D).reshape(E, K, D).copy()
    W[0, :128, :128] = 0.0
    w = sq.Fp8Weight(H.bf16_dev(W) if E > 1 else H.bf16_dev(W[0]))
    codes, scales = values(w.codes).reshape(E, D, K), w.scales.cpu().numpy().reshape(E, O.blocks(D), O.blocks(K))
    for e in range(E):
        q, s = O.pack(W[e])
        assert np.array_equal(scales[e], s) and np.array_equal(codes[e], q)


def test_pack_of_a_misaligned_or_strided_weight():
    W = synthetic.weights(75, 256, 130)
    flat = torch.zeros(256 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:] = H.bf16_dev(W[:, :128]).reshape(-1)
    for t, ref in ((flat[1:].view(256, 128), W[:, :128]), (H.bf16_dev(W)[:, 1:129], W[:, 1:129])):
        w = sq.Fp8Weight(t)
        q, s = O.pack(ref)
        assert np.array_equal(values(w.codes), q) and np.array_equal(w.scales.cpu().numpy(), s)


# ------------------------------------------------------------------ linear ---


def operands(T, K, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, K, generator=g) * 60).clamp(-448, 448).to(F8)
    w = (torch.randn(D, K, generator=g) * 90).clamp(-448, 448).to(F8)
    xs = torch.exp2(torch.rand(T, O.blocks(K), generator=g) * 6 - 9)
    ws = torch.exp2(torch.rand(O.blocks(D), O.blocks(K), generator=g) * 4 - 12)
    return x, xs, w, ws


def linear_reference(x, xs, w, ws):
    K = x.shape[1]
    xd = torch.from_numpy(O.dequant_act(values(x), f64(xs)))
    wd = torch.from_numpy(O.dequant_weight(values(w), f64(ws)))
    y = (xd @ wd.T).numpy()
    mag = (xd.abs() @ wd.abs().T).numpy()
    return y, (128 + O.blocks(K) + 8) * 2.0 ** -23 * mag


def check_linear(y, ref, bound, dtype):
    got = f64(y)
    assert (np.abs(got - ref) <= bound + (np.abs(ref) + bound) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)).all()
    if dtype == torch.float32:
        # the sums' errors are not all one way: far below the bound over the whole product
        assert H.rel_fro(got, ref) <= 2e-6


LINEAR = [(1, 16, 1), (1, 3584, 512), (2, 144, 15), (7, 1024, 17), (8, 4112, 129), (9, 272, 264), (16, 18944, 96),
          (17, 128, 128), (17, 16, 1), (32, 1040, 640), (33, 4112, 250), (65, 400, 130), (3, 272, 38100), (64, 3584, 640), (127, 1040, 129), (128, 128, 127),
          (129, 272, 1111), (200, 4096, 257), (333, 2064, 300), (700, 144, 2000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,D", LINEAR)
def test_linear(T, K, D, dtype):
    x, xs, w, ws = operands(T, K, D, T + K + D)
    act = sq.Fp8Act.from_parts(x.cuda(), xs.cuda())
    wt = sq.Fp8Weight.from_parts(w.cuda(), ws.cuda())
    work = sq.Fp8Workspace.for_linear(T, K, D)
    y = sq.fp8_linear(act, wt, out_dtype=dtype, ws=work)
    ref, bound = linear_reference(x, xs, w, ws)
    check_linear(y, ref, bound, dtype)
    assert work.check() == 0
    assert torch.equal(y, sq.fp8_linear(act, wt, out_dtype=dtype, ws=work))  # the same bits again


# enough 256 x 256 tiles for the pair kernel: whole tiles, and both axes (and the second CTA's half) ragged
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,D", [(2048, 512, 2560), (2100, 400, 2500), (2180, 144, 2705), (260, 272, 19000),
                                   (19000, 272, 260), (2049, 1040, 2560), (4000, 640, 5000)])
def test_linear_pair(T, K, D, dtype):
    x, xs, w, ws = operands(T, K, D, T + K + D)
    act = sq.Fp8Act.from_parts(x.cuda(), xs.cuda())
    wt = sq.Fp8Weight.from_parts(w.cuda(), ws.cuda())
    work = sq.Fp8Workspace.for_linear(T, K, D)
    y = sq.fp8_linear(act, wt, out_dtype=dtype, ws=work)
    ref, bound = linear_reference(x, xs, w, ws)
    check_linear(y, ref, bound, dtype)
    assert work.check() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D,off,width", [(5, 40, 3, 47), (5, 48, 8, 64), (40, 200, 1, 202), (40, 200, 8, 216),
                                           (2100, 2500, 4, 2511), (2100, 2504, 8, 2520)])
def test_linear_into_columns_of_a_wider_tensor(T, D, off, width, dtype):
    x, xs, w, ws = operands(T, 272, D, T)
    wide = torch.full((T + 1, width), 77.0, dtype=dtype, device="cuda")
    out = wide[:T, off:off + D]
    sq.fp8_linear(sq.Fp8Act.from_parts(x.cuda(), xs.cuda()), sq.Fp8Weight.from_parts(w.cuda(), ws.cuda()), out=out)
    ref, bound = linear_reference(x, xs, w, ws)
    check_linear(out, ref, bound, dtype)
    wide[:T, off:off + D] = 77.0
    assert (wide == 77.0).all()  # nothing else was written


@pytest.mark.parametrize("T,D", [(9, 150), (150, 300), (2100, 2500)])
def test_linear_keeps_nan_to_its_row_and_column(T, D):
    x, xs, w, ws = operands(T, 272, D, 3)
    x.view(torch.uint8)[T - 2, 270] = 0x7F
    w.view(torch.uint8)[D - 3, 5] = 0xFF
    y = sq.fp8_linear(sq.Fp8Act.from_parts(x.cuda(), xs.cuda()), sq.Fp8Weight.from_parts(w.cuda(), ws.cuda()),
                      out_dtype=torch.float32).cpu()
    nan = torch.zeros(T, D, dtype=torch.bool)
    nan[T - 2], nan[:, D - 3] = True, True
    assert torch.equal(y.isnan(), nan)


def test_linear_refuses_what_does_not_fit():
    x, xs, w, ws = (t.cuda() for t in operands(4, 256, 64, 0))
    act, wt = sq.Fp8Act.from_parts(x, xs), sq.Fp8Weight.from_parts(w, ws)
    with pytest.raises(ValueError):
        sq.fp8_linear(act, wt, out=torch.empty(4, 65, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        sq.fp8_linear(act, wt, out=torch.empty(64, 4, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(TypeError):
        sq.fp8_linear(act, wt, out_dtype=torch.float16)
    with pytest.raises(sq.SharqError):
        sq.fp8_linear(sq.Fp8Act(4, 272), wt)
    with pytest.raises(ValueError):
        act.prep(torch.empty(5, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        act.prep(torch.empty(4, 256, device="cuda"))
    with pytest.raises(ValueError):
        sq.Fp8Act.from_parts(x, xs[:, :1])
    with pytest.raises(ValueError):
        sq.Fp8Weight.from_parts(w, ws.t())


# --------------------------------------------------------------------- moe ---


def moe_inputs(T, E, Hd, I, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.from_numpy(synthetic.activations(seed, T, Hd)) if T else torch.zeros(0, Hd)
    x = (x / x.square().mean(-1, keepdim=True).sqrt()).bfloat16()
    lg = (torch.randn(T, E, generator=g) * spread).bfloat16().float()
    w13 = (torch.randn(E, 2 * I, Hd, generator=g) * 90).clamp(-448, 448).to(F8)
    w2 = (torch.randn(E, Hd, I, generator=g) * 90).clamp(-448, 448).to(F8)
    s13 = torch.exp2(torch.rand(E, O.blocks(2 * I), O.blocks(Hd), generator=g) * 2 - 13)
    s2 = torch.exp2(torch.rand(E, O.blocks(Hd), O.blocks(I), generator=g) * 2 - 13)
    return x, lg, w13, s13, w2, s2


def run_moe(x, lg, w13, s13, w2, s2, topk, **kw):
    a, b = sq.Fp8Weight.from_parts(w13.cuda(), s13.cuda()), sq.Fp8Weight.from_parts(w2.cuda(), s2.cuda())
    return sq.fp8_moe(x.cuda(), lg.cuda(), a, b, topk, return_routing=True, **kw)


def check_moe(out, x, lg, w13, s13, w2, s2, topk, renormalize=True):
    y, ids, p = out
    ref, rid, rp, bound = O.moe(f64(x), f64(lg), O.dequant_weight(values(w13), f64(s13)),
                                O.dequant_weight(values(w2), f64(s2)), topk, renormalize)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # exp to 2 units, a sum of up to 512 positive terms in a tree, a quotient
    assert (np.abs(f64(p) - rp) <= 2.0 ** -23 * 40 * rp + 1e-37).all()
    # results near zero: the spacing of bf16 below 2^-126 is 2^-133, so its rounding is off by up to 2^-134 however
    # small the value, and h (spacing 2^-149 in float32) adds at most 2^-149 sum |w2| < 2^-134
    assert (np.abs(O.dequant_weight(values(w2), f64(s2))).sum(-1) < 2.0 ** 15).all()
    bound = bound + 2.0 ** -23 * 40 * np.abs(ref) + 2.0 ** -133
    assert (np.abs(f64(y) - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8).all()


MOE = [(1, 1, 1, 16, 16), (1, 4, 2, 128, 64), (1, 128, 8, 256, 96), (2, 8, 2, 272, 144), (7, 16, 4, 2064, 48),
       (16, 8, 2, 256, 768), (33, 60, 6, 144, 272), (64, 8, 8, 256, 128), (64, 512, 16, 128, 32), (64, 128, 8, 512, 96), (1, 1, 1, 2064, 64), (2, 300, 3, 1040, 16),
       (8, 9, 9, 128, 80), (9, 40, 4, 640, 128), (24, 3, 2, 272, 128), (40, 4, 2, 1040, 272)]


@pytest.mark.parametrize("T,E,topk,Hd,I", MOE)
def test_moe(T, E, topk, Hd, I):
    args = moe_inputs(T, E, Hd, I, T + E)
    check_moe(run_moe(*args, topk), *args, topk)


@pytest.mark.parametrize("topk", [1, 3, 6])
def test_moe_without_renormalizing(topk):
    args = moe_inputs(9, 12, 256, 128, 5)
    check_moe(run_moe(*args, topk, renormalize=False), *args, topk, renormalize=False)


def test_moe_ties_masked_and_empty_rows():
    x, lg, *w = moe_inputs(8, 40, 256, 128, 6)
    lg[0] = 0.5                                   # all equal: the lowest indices
    lg[1, ::2] = lg[1].max()
    lg[2, 3:] = float("-inf")                     # fewer experts than choices
    lg[3] = float("-inf")                         # none
    lg[4] = torch.finfo(torch.float32).min        # masked by the lowest value, all alike
    lg[5, 7] = float("nan")
    lg[6, 9], lg[6, 30] = float("inf"), float("inf")
    lg[7, :20] = -0.0
    lg[7, 20:] = 0.0                              # equal to -0
    for renorm in (True, False):
        out = run_moe(x, lg, *w, 5, renormalize=renorm)
        check_moe(out, x, lg, *w, 5, renormalize=renorm)
        assert (out[0][3] == 0).all()


def test_moe_all_tokens_on_the_same_experts():
    x, lg, *w = moe_inputs(64, 16, 272, 144, 7)
    lg[:, 4:6] += 50
    check_moe(run_moe(x, lg, *w, 2), x, lg, *w, 2)


@pytest.mark.parametrize("T", [4, 20, 60])
def test_moe_padded_rows_may_hold_anything(T):
    """tokens whose logits are all -inf take no part: y = 0 whatever their x, and nobody else's result changes"""
    x, lg, *w = moe_inputs(T, 12, 272, 144, 11)
    pad = torch.arange(T) % 3 == 2
    lg[pad] = float("-inf")
    x = x.clone()
    x[pad] = float("nan")
    y, ids, p = run_moe(x, lg, *w, 3)
    assert (y[pad] == 0).all() and (p[pad] == 0).all()
    keep = ~pad
    check_moe((y[keep], ids[keep], p[keep]), x[keep], lg[keep], *w, 3)
    assert np.array_equal(ids[pad].cpu().numpy(), O.route(f64(lg[pad]), 3)[0])


@pytest.mark.parametrize("T", [5, 20, 64])
def test_moe_nan_and_inf_stay_with_their_token(T):
    x, lg, *w = moe_inputs(T, 10, 272, 144, 12)
    x = x.clone()
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    y, _, _ = run_moe(x, lg, *w, 2)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[1] = bad[2] = True
    assert y[1].isnan().all()
    assert not y[2].isfinite().any()
    ref, _, _ = run_moe(torch.where(bad[:, None], torch.zeros_like(x), x), lg, *w, 2)
    assert torch.equal(y[~bad], ref[~bad])


def test_moe_one_workspace_for_calls_of_every_size():
    """the arrival counts that calls leave behind are zero again, whatever the sizes"""
    args = {T: moe_inputs(T, 16, 640, 128, T) for T in (1, 8, 9, 30, 64)}
    a = {T: (sq.Fp8Weight.from_parts(v[2].cuda(), v[3].cuda()), sq.Fp8Weight.from_parts(v[4].cuda(), v[5].cuda()))
         for T, v in args.items()}
    ws = sq.Fp8Workspace.for_moe(64, 4, *a[64])
    for T in (64, 1, 30, 8, 9, 64, 30, 1):
        x, lg = args[T][:2]
        out = sq.fp8_moe(x.cuda(), lg.cuda(), *a[T], 4, ws=ws, return_routing=True)
        check_moe(out, *args[T], 4)
        again = sq.fp8_moe(x.cuda(), lg.cuda(), *a[T], 4, ws=ws)
        assert torch.equal(out[0], again)  # the same bits again
    assert ws.check() == 0


def test_weights_beyond_two_gigabytes():
    """offsets that pass 32 bits: the last experts of a large layer, the last columns of a large linear"""
    E, Hd, I = 140, 4096, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    bytes_ = torch.randint(0, 256, (2 * I * Hd + 1,), generator=g, device="cuda", dtype=torch.uint8)
    bytes_ = torch.where(bytes_ & 0x7F >= 0x70, bytes_ & 0x8F, bytes_)  # no NaN, nothing above 15
    one13, one2 = bytes_[:-1].view(2 * I, Hd), bytes_[1:1 + Hd * I].view(Hd, I)
    w13, w2 = (torch.zeros(E, *t.shape, dtype=torch.uint8, device="cuda") for t in (one13, one2))
    for e in (0, 130, 139):
        w13[e], w2[e] = one13.roll(e, 0), one2.roll(e, 0)
    s13 = torch.full((E, 2 * I // 128, Hd // 128), 2.0 ** -9, device="cuda")
    s2 = torch.full((E, Hd // 128, I // 128), 2.0 ** -9, device="cuda")
    x = torch.randn(2, Hd, generator=g, device="cuda").bfloat16()
    lg = torch.full((2, E), -9.0, device="cuda")
    lg[0, 139], lg[0, 0], lg[1, 130], lg[1, 139] = 3.0, 2.0, 1.0, 0.5
    y, ids, p = sq.fp8_moe(x, lg, sq.Fp8Weight.from_parts(w13.view(F8), s13), sq.Fp8Weight.from_parts(w2.view(F8), s2),
                           2, return_routing=True)
    assert ids.tolist() == [[139, 0], [130, 139]]
    for t in range(2):
        ref, size = 0.0, 0.0
        for j in range(2):
            a13, a2 = (w[int(ids[t, j])].view(F8).double() * 2.0 ** -9 for w in (w13, w2))
            gu = a13 @ x[t].double()
            h = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            ref = ref + float(p[t, j]) * (a2 @ h)
            size = size + float(p[t, j]) * (a2.abs() @ h.abs())
        # h off by 2^-12 of itself as three terms and less by its own sums; sums of I terms; bf16
        assert ((y[t].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * I * 2.0 ** -23) * size).all()
    del w13, w2
    K, D = 16384, 140000
    code = torch.empty(D, K, dtype=torch.uint8, device="cuda")
    for d in range(0, D, 2 * I):
        n = min(2 * I, D - d)
        code[d:d + n] = bytes_[:n * Hd].view(n, Hd).repeat(1, K // Hd).roll(d // 7, 0)
    scale = torch.full((O.blocks(D), K // 128), 2.0 ** -9, device="cuda")
    act = sq.Fp8Act(3, K).prep(torch.randn(3, K, generator=g, device="cuda").bfloat16())
    y = sq.fp8_linear(act, sq.Fp8Weight.from_parts(code.view(F8), scale), out_dtype=torch.float32)
    xd = act.codes.double() * act.scales.double().repeat_interleave(128, 1)
    for d in (0, 131000, D - 300):
        wd = code[d:d + 300].view(F8).double() * 2.0 ** -9
        ref, size = xd @ wd.T, xd.abs() @ wd.abs().T
        assert ((y[:, d:d + 300].double() - ref).abs() <= (128 + K // 128 + 8) * 2.0 ** -23 * size + 2.0 ** -24 * ref.abs()).all()


@pytest.mark.parametrize("mag", [2.0 ** -110, 2.0 ** -40, 2.0 ** 40])
def test_moe_activations_far_from_one(mag):
    """E4M3 terms hold any bf16 activation: its 128-block is scaled by a power of two"""
    x, lg, w13, s13, w2, s2 = moe_inputs(5, 4, 256, 128, 8)
    x = (x.float() * mag).bfloat16()
    x[3, :128] = 0
    x[4, 128:] *= 2.0 ** -20
    s13 = s13 / mag if mag > 1 else s13
    args = (x, lg, w13, s13, w2, s2)
    check_moe(run_moe(*args, 2), *args, 2)


def test_moe_strides_and_in_place():
    x, lg, w13, s13, w2, s2 = moe_inputs(6, 10, 256, 64, 9)
    xb = torch.full((7, 300 // 4 * 4 + 4), 5.0, dtype=torch.bfloat16, device="cuda")
    xb[:6, :256] = x.cuda()
    lb = torch.full((6, 13), 1e9, device="cuda")
    lb[:, :10] = lg.cuda()
    a, b = sq.Fp8Weight.from_parts(w13.cuda(), s13.cuda()), sq.Fp8Weight.from_parts(w2.cuda(), s2.cuda())
    xin = xb[:6, :256]
    out = sq.fp8_moe(xin, lb[:, :10], a, b, 3, out=xin, return_routing=True)
    check_moe(out, x, lg, w13, s13, w2, s2, 3)
    assert (xb[6] == 5.0).all() and (xb[:, 256:] == 5.0).all()


@pytest.mark.parametrize("T,E", [(20, 40), (20, 3), (64, 4)])
def test_moe_strides_and_in_place_above_eight_tokens(T, E):
    x, lg, w13, s13, w2, s2 = moe_inputs(T, E, 272, 144, 13)
    xb = torch.full((T + 1, 288), 5.0, dtype=torch.bfloat16, device="cuda")
    xb[:T, :272] = x.cuda()
    lb = torch.full((T, E + 3), 1e9, device="cuda")
    lb[:, :E] = lg.cuda()
    a, b = sq.Fp8Weight.from_parts(w13.cuda(), s13.cuda()), sq.Fp8Weight.from_parts(w2.cuda(), s2.cuda())
    xin = xb[:T, :272]
    out = sq.fp8_moe(xin, lb[:, :E], a, b, 2, out=xin, return_routing=True)
    check_moe(out, x, lg, w13, s13, w2, s2, 2)
    assert (xb[T] == 5.0).all() and (xb[:, 272:] == 5.0).all()


def test_moe_refusals():
    x, lg, w13, s13, w2, s2 = (t.cuda() for t in moe_inputs(4, 8, 256, 64, 1))
    a, b = sq.Fp8Weight.from_parts(w13, s13), sq.Fp8Weight.from_parts(w2, s2)
    with pytest.raises(sq.SharqError):
        sq.fp8_moe(x, lg, a, b, 9)
    with pytest.raises(sq.SharqError):
        sq.fp8_moe(x.repeat(17, 1), lg.repeat(17, 1), a, b, 2)
    with pytest.raises(ValueError):
        sq.fp8_moe(x[:, :128], lg, a, b, 2)
    with pytest.raises(ValueError):
        sq.fp8_moe(x, lg[:, :4], a, b, 2)
    with pytest.raises(TypeError):
        sq.fp8_moe(x, lg.bfloat16(), a, b, 2)
    with pytest.raises(sq.SharqError):
        sq.fp8_moe(x, lg, a, a, 2)
    y = sq.fp8_moe(x[:0], lg[:0], a, b, 2)
    assert y.shape == (0, 256)


# ---------------------------------------------------------------- together ---


class Layer:
    """The 8-bit half of a decoder layer: residual + norm -> gate+up -> SwiGLU -> down, and a mixture of experts."""

    def __init__(self, T, Hd=512, I=640, E=8, topk=2, seed=0):
        self.T, self.Hd, self.I, self.topk = T, Hd, I, topk
        self.wgu = sq.Fp8Weight(H.bf16_dev(synthetic.weights(seed, Hd, 2 * I)))
        self.wd = sq.Fp8Weight(H.bf16_dev(synthetic.weights(seed + 1, I, Hd)))
        ex = synthetic.weights(seed + 2, E * Hd, 256).reshape(E, Hd, 256)
        self.w13 = sq.Fp8Weight(H.bf16_dev(ex))
        self.w2 = sq.Fp8Weight(H.bf16_dev(synthetic.weights(seed + 3, E * 128, Hd).reshape(E, 128, Hd)))
        self.gamma = H.bf16_dev(synthetic.gamma(seed + 4, Hd))
        self.x = H.bf16_dev(synthetic.activations(seed + 5, T, Hd))
        self.res = H.bf16_dev(synthetic.activations(seed + 6, T, Hd))
        self.logits = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)).cuda()
        self.h = torch.empty_like(self.res)
        self.a1, self.a2 = sq.Fp8Act(T, Hd), sq.Fp8Act(T, I)
        self.gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.down = torch.empty(T, Hd, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty_like(self.down)
        self.ws = sq.Fp8Workspace.for_linear(T, Hd, 2 * I)
        self.wm = sq.Fp8Workspace.for_moe(T, topk, self.w13, self.w2)

    def run(self, stream=None):
        self.a1.prep_residual(self.x, self.res, self.h, self.gamma, EPS, stream=stream)
        sq.fp8_linear(self.a1, self.wgu, out=self.gu, ws=self.ws, stream=stream)
        self.a2.prep_silu_mul(self.gu[:, :self.I], self.gu[:, self.I:], stream=stream)
        sq.fp8_linear(self.a2, self.wd, out=self.down, ws=self.ws, stream=stream)
        sq.fp8_moe(self.h, self.logits, self.w13, self.w2, self.topk, out=self.y, ws=self.wm, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.h, self.gu, self.down, self.y)]

    def check(self):
        h = (self.x.float() + self.res.float()).bfloat16()
        assert torch.equal(self.h, h)
        check_quant(self.a1, O.rms_norm(f64(h), f64(self.gamma), np.float32(EPS)), norm_delta(self.Hd))
        for a, w, y in ((self.a1, self.wgu, self.gu), (self.a2, self.wd, self.down)):
            ref, bound = linear_reference(a.codes.cpu(), a.scales.cpu(), w.codes.cpu(), w.scales.cpu())
            check_linear(y, ref, bound, torch.bfloat16)
        check_quant(self.a2, O.silu(f64(self.gu[:, :self.I])) * f64(self.gu[:, self.I:]), (2 + 1.2 * 88 + 8) * 2.0 ** -23)
        ref, _, _, bound = O.moe(f64(h), f64(self.logits), O.dequant_weight(values(self.w13.codes), f64(self.w13.scales)),
                                 O.dequant_weight(values(self.w2.codes), f64(self.w2.scales)), self.topk)
        bound = bound + 2.0 ** -23 * 40 * np.abs(ref)
        assert (np.abs(f64(self.y) - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8).all()
        assert self.ws.check() == 0


@pytest.mark.parametrize("T", [1, 12, 50, 64])
def test_layer_runs_as_one_chain(T):
    layer = Layer(T)
    layer.run()
    layer.check()


def test_layer_captured_and_replayed_with_new_inputs():
    layer = Layer(20)
    side = torch.cuda.Stream()
    layer.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        layer.run()
    for seed in (100, 200):
        layer.x.copy_(H.bf16_dev(synthetic.activations(seed, 20, 512)))
        layer.logits.copy_(torch.randn(20, 8, generator=torch.Generator().manual_seed(seed)))
        for t in (layer.h, layer.gu, layer.down, layer.y):
            t.fill_(float("nan"))
        g.replay()
        layer.check()


def test_two_layers_at_once_on_two_streams():
    layers = [Layer(16, seed=s) for s in (300, 400)]
    want = []
    for la in layers:
        la.run()
        torch.cuda.synchronize()
        want.append(la.outputs())
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for la, s in zip(layers, streams):
            la.run(stream=s)
    torch.cuda.synchronize()
    for la, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(la.outputs(), w))


def test_allocations_of_a_call_belong_to_its_stream():
    """weights and workspaces made by a call on another stream are not handed out again while it runs"""
    s = torch.cuda.Stream()
    W = H.bf16_dev(synthetic.weights(1, 2048, 2048)).t()  # not contiguous: copied inside
    x = H.bf16_dev(synthetic.activations(2, 24, 2048))
    torch.cuda.synchronize()
    ref_w = sq.Fp8Weight(W)
    ref_a = sq.Fp8Act(24, 2048).prep(x)
    want = sq.fp8_linear(ref_a, ref_w)
    torch.cuda.synchronize()
    for _ in range(5):
        w = sq.Fp8Weight(W, stream=s)
        y = sq.fp8_linear(ref_a, w, stream=s)
        torch.full((2048 * 2048,), 9.0, dtype=torch.bfloat16, device="cuda")  # this stream's allocations meanwhile
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    with torch.cuda.stream(s):
        with pytest.raises(TypeError):
            sq.Fp8Weight(W.cpu())
