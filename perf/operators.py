"""The 8-bit (E4M3) block-scaled operators: what is measured of them, and on which cases.

Four operators that are used together in a decoder layer whose linears run in 8 bits:

  prep    RMS norm of the residual stream (or the SwiGLU product, or a plain activation) to E4M3 with one float32
          scale per row and 128 columns
  pack    a bf16 weight [E, K, D] to E4M3 [E, D, K] with one float32 scale per 128 x 128 block
  linear  Y = X W of such operands, float32 sums, bf16 or float32 output
  moe     a whole mixture-of-experts layer for a few tokens: top-k of the router's logits, gate and up projections,
          SwiGLU, down projection, weighted sum; E4M3 weights, bf16 activations

`run` computes them in their plain form (elementary torch operations in float32) or, where `own` is true, by the calls
a user makes.  `exact` restates each definition in float64.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9  # spacing of E4M3 below 2^-6
EPS = 1e-5
F8 = torch.float8_e4m3fn

# ------------------------------------------------------------------ cases ---


def listed():
    return [
        # decode step of the 3584-wide decoder layer: one row enters the qkv or gate+up projection
        {"name": "prep_decode", "op": "prep", "kind": "residual", "T": 1, "K": 3584},
        # prefill of the same layer: the largest norm of the layer stack
        {"name": "prep_prefill", "op": "prep", "kind": "residual", "T": 8192, "K": 3584},
        # a batch of odd length whose rows end inside a block of 128
        {"name": "prep_ragged", "op": "prep", "kind": "norm", "T": 777, "K": 4112},
        # input of the down projection: SwiGLU of the two halves of one gate+up output
        {"name": "prep_swiglu", "op": "prep", "kind": "silu", "T": 1024, "K": 18944},
        # loading a model: a square projection
        {"name": "pack_square", "op": "pack", "E": 1, "K": 4096, "D": 4096},
        # loading a model: eight experts, with both axes ending inside a block
        {"name": "pack_experts", "op": "pack", "E": 8, "K": 2000, "D": 1100},
        # decode, one request: the qkv projection
        {"name": "linear_decode", "op": "linear", "T": 1, "K": 3584, "D": 4608, "out": "bf16"},
        # decode, a small batch: the down projection, long sums
        {"name": "linear_batch", "op": "linear", "T": 16, "K": 18944, "D": 3584, "out": "bf16"},
        # a short prompt with odd sizes and a float32 output (logits, or a check against another path)
        {"name": "linear_ragged", "op": "linear", "T": 333, "K": 4112, "D": 1111, "out": "f32"},
        # prefill: the gate+up projection, the largest product of the layer stack
        {"name": "linear_prefill", "op": "linear", "T": 8192, "K": 3584, "D": 37888, "out": "bf16"},
        # one request through the 128-expert layer: eight experts are read
        {"name": "moe_decode", "op": "moe", "T": 1, "E": 128, "topk": 8, "H": 2048, "I": 768},
        # a decode batch through the same layer: nearly every expert is read, four tokens each
        {"name": "moe_batch", "op": "moe", "T": 64, "E": 128, "topk": 8, "H": 2048, "I": 768},
    ]


def _log(rng, lo, hi, step=1):
    """a multiple of `step` in [lo, hi], spread over the logarithm"""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["prep", "prep", "pack", "linear", "linear", "linear", "moe", "moe"])
    if op == "prep":
        T, K = _log(rng, 1, 8192), _log(rng, 128, 18944, 16)
        T = max(1, min(T, 8192 * 3584 // K))
        return {"op": op, "kind": rng.choice(["residual", "norm", "plain", "silu"]), "T": T, "K": K}
    if op == "pack":
        K, D = _log(rng, 128, 8192, 16), _log(rng, 64, 8192)
        return {"op": op, "E": rng.choice([1, 1, rng.randint(2, 8)]) if K * D <= 1 << 24 else 1, "K": K, "D": D}
    if op == "linear":
        T, K, D = _log(rng, 1, 8192), _log(rng, 256, 18944, 16), _log(rng, 64, 37888)
        while T * K * D > 8192 * 3584 * 37888 or K * D > 3584 * 37888:
            D //= 2
        return {"op": op, "T": T, "K": K, "D": D, "out": rng.choice(["bf16", "bf16", "f32"])}
    E, H, I = _log(rng, 8, 128), _log(rng, 256, 4096, 16), _log(rng, 64, 2048, 16)
    while E * H * I > 128 * 2048 * 768:
        E = max(8, E // 2)
        if E == 8:
            break
    return {"op": op, "T": _log(rng, 1, 64), "E": E, "topk": rng.randint(1, min(8, E)), "H": H, "I": I}


# ----------------------------------------------------------------- inputs ---


def _activations(g, T, K):
    """N(0, 1) with 0.5 % of the channels 20 to 60 times larger and 0.1 % of the entries spikes of 8 to 16"""
    dev = "cuda"
    x = torch.randn(T, K, generator=g, device=dev)
    n = max(1, round(0.005 * K))
    ch = torch.randperm(K, generator=g, device=dev)[:n]
    x[:, ch] *= torch.rand(n, generator=g, device=dev) * 40 + 20
    hit = torch.rand(T, K, generator=g, device=dev) < 0.001
    spike = (torch.rand(T, K, generator=g, device=dev) * 8 + 8) * torch.randn(T, K, generator=g, device=dev).sign()
    return torch.where(hit, spike, x).bfloat16()


def _blocks(n):
    return -(-n // BLOCK)


def _weight_codes(g, E, D, K):
    """E4M3 codes [E, D, K] and scales [E, D/128, K/128] of N(0, 0.02) weights"""
    pd, pk = _blocks(D) * BLOCK, _blocks(K) * BLOCK
    codes = torch.empty(E, D, K, dtype=F8, device="cuda")
    scales = torch.empty(E, _blocks(D), _blocks(K), device="cuda")
    for e in range(E):
        w = torch.zeros(pd, pk, device="cuda")
        w[:D, :K] = torch.randn(D, K, generator=g, device="cuda") * 0.02
        t = w.view(pd // BLOCK, BLOCK, pk // BLOCK, BLOCK)
        s = t.abs().amax(dim=(1, 3)) / E4M3_MAX
        codes[e] = (t / s[:, None, :, None]).view(pd, pk)[:D, :K].to(F8)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "prep":
        T, K = c["T"], c["K"]
        s = {"x": _activations(g, T, K)}
        if c["kind"] == "residual":
            s["res"] = (_activations(g, T, K).float() * 4).bfloat16()
        if c["kind"] in ("residual", "norm"):
            s["gamma"] = (torch.rand(K, generator=g, device="cuda") + 0.5).bfloat16()
        if c["kind"] == "silu":  # one gate+up output, its halves side by side
            s["x"] = torch.cat([(s["x"].float() * 0.5).bfloat16(), _activations(g, T, K)], dim=1)
        return {**c, **s}
    if c["op"] == "pack":
        W = (torch.randn(c["E"], c["K"], c["D"], generator=g, device="cuda") * 0.02).bfloat16()
        return {**c, "W": W}
    if c["op"] == "linear":
        T, K, D = c["T"], c["K"], c["D"]
        codes, scales = _plain_quant(_activations(g, T, K).float())
        ld = -(-T // 4) * 4  # scales lie column by column, each column padded to 16 bytes
        xs = torch.zeros(_blocks(K), ld, device="cuda")
        xs[:, :T] = scales.t()
        wq, ws = _weight_codes(g, 1, D, K)
        return {**c, "x": codes, "xs": xs[:, :T].t(), "w": wq[0], "ws": ws[0]}
    T, E, H, I = c["T"], c["E"], c["H"], c["I"]
    x = _activations(g, T, H)
    x = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS)).bfloat16()
    # router outputs as a bf16 projection leaves them: equal logits occur
    logits = (torch.randn(T, E, generator=g, device="cuda") * 1.5).bfloat16().float()
    w13, s13 = _weight_codes(g, E, 2 * I, H)
    w2, s2 = _weight_codes(g, E, H, I)
    return {**c, "x": x, "logits": logits, "w13": w13, "s13": s13, "w2": w2, "s2": s2}


# ------------------------------------------------------------ plain forms ---


def _plain_quant(v):
    """float32 [T, K] -> E4M3 [T, K] and scales [T, K/128]"""
    T, K = v.shape
    kb = _blocks(K)
    t = torch.nn.functional.pad(v, (0, kb * BLOCK - K)).view(T, kb, BLOCK)
    amax = t.abs().amax(-1)
    s = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), torch.ones_like(amax))
    q = (t * (1.0 / s)[..., None]).to(F8).view(T, kb * BLOCK)[:, :K]
    return q.contiguous(), s


def _plain_prep(s):
    x, out = s["x"].float(), {}
    if s["kind"] == "silu":
        gate, up = x[:, :s["K"]], x[:, s["K"]:]
        v = gate / (1 + torch.exp(-gate)) * up
    else:
        if s["kind"] == "residual":
            out["h"] = (x + s["res"].float()).bfloat16()
            x = out["h"].float()
        v = x
        if "gamma" in s:
            v = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    out["codes"], out["scales"] = _plain_quant(v)
    return out


def _plain_pack(s):
    E, K, D = s["W"].shape
    kb, db = _blocks(K), _blocks(D)
    w = torch.nn.functional.pad(s["W"].float().transpose(1, 2), (0, kb * BLOCK - K, 0, db * BLOCK - D))
    t = w.reshape(E, db, BLOCK, kb, BLOCK)
    amax = t.abs().amax(dim=(2, 4))
    sc = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), torch.ones_like(amax))
    q = (t * (1.0 / sc)[:, :, None, :, None]).to(F8).view(E, db * BLOCK, kb * BLOCK)
    return {"codes": q[:, :D, :K].contiguous(), "scales": sc}


def _spread(s, n, dim):
    """one value per 128 -> one per element, n of them"""
    return s.repeat_interleave(BLOCK, dim=dim).narrow(dim, 0, n)


def _plain_linear(s):
    x = s["x"].float() * _spread(s["xs"], s["K"], 1)
    w = s["w"].float() * _spread(_spread(s["ws"], s["D"], 0), s["K"], 1)
    y = x @ w.t()
    return y if s["out"] == "f32" else y.bfloat16()


def _plain_moe(s):
    T, k, H, I = s["T"], s["topk"], s["H"], s["I"]
    order = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    ids = order.indices[:, :k]
    w = torch.exp(order.values[:, :k] - order.values[:, :1])
    w = w / w.sum(-1, keepdim=True)
    pick = ids.reshape(-1)
    w13 = s["w13"].view(torch.uint8)[pick].view(F8).float()
    w13 = w13 * _spread(_spread(s["s13"][pick], 2 * I, 1), H, 2)
    gu = torch.bmm(w13, s["x"].float().repeat_interleave(k, dim=0).unsqueeze(-1)).squeeze(-1)
    del w13
    h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
    w2 = s["w2"].view(torch.uint8)[pick].view(F8).float()
    w2 = w2 * _spread(_spread(s["s2"][pick], H, 1), I, 2)
    y = torch.bmm(w2, h.unsqueeze(-1)).view(T, k, H)
    return {"y": (y * w[..., None]).sum(1).bfloat16(), "ids": ids.int(), "weights": w}


# -------------------------------------------------------- framework calls ---


def _held(s, name, make):
    """a weight, buffer or workspace that the caller's program keeps beside its data"""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    import sparse_activation_quantization_b200 as sq
    if s["op"] == "prep":
        act = _held(s, "_act", lambda: sq.Fp8Act(s["T"], s["K"], device=s["x"].device))
        if s["kind"] == "silu":
            act.prep_silu_mul(s["x"][:, :s["K"]], s["x"][:, s["K"]:])
        elif s["kind"] == "residual":
            h = _held(s, "_h", lambda: torch.empty_like(s["x"]))
            act.prep_residual(s["x"], s["res"], h, s["gamma"], EPS)
            return {"h": h, "codes": act.codes, "scales": act.scales}
        else:
            act.prep(s["x"], s.get("gamma"), EPS)
        return {"codes": act.codes, "scales": act.scales}
    if s["op"] == "pack":
        w = sq.Fp8Weight(s["W"])
        return {"codes": w.codes, "scales": w.scales}
    if s["op"] == "linear":
        act = _held(s, "_act", lambda: sq.Fp8Act.from_parts(s["x"], s["xs"]))
        w = _held(s, "_w", lambda: sq.Fp8Weight.from_parts(s["w"], s["ws"]))
        ws = _held(s, "_ws", lambda: sq.Fp8Workspace.for_linear(s["T"], s["K"], s["D"], device=s["x"].device))
        return sq.fp8_linear(act, w, out_dtype=torch.float32 if s["out"] == "f32" else torch.bfloat16, ws=ws)
    w13 = _held(s, "_w13", lambda: sq.Fp8Weight.from_parts(s["w13"], s["s13"]))
    w2 = _held(s, "_w2", lambda: sq.Fp8Weight.from_parts(s["w2"], s["s2"]))
    ws = _held(s, "_ws", lambda: sq.Fp8Workspace.for_moe(s["T"], s["topk"], w13, w2, device=s["x"].device))
    y, ids, weights = sq.fp8_moe(s["x"], s["logits"], w13, w2, s["topk"], ws=ws, return_routing=True)
    return {"y": y, "ids": ids, "weights": weights}


_PLAIN = {"prep": _plain_prep, "pack": _plain_pack, "linear": _plain_linear, "moe": _plain_moe}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------- the floor ---


def work(case):
    """bytes: each input read once, each output written once; flops: of the products (norms and quantizers: per value)"""
    c = case
    if c["op"] == "prep":
        n = c["T"] * c["K"]
        reads = {"residual": 4, "silu": 4}.get(c["kind"], 2)  # bf16 inputs per value
        writes = 1 + (2 if c["kind"] == "residual" else 0)    # code, new stream
        return {"bytes": n * (reads + writes) + 4 * c["T"] * _blocks(c["K"]) + 2 * c["K"], "flops": 8 * n}
    if c["op"] == "pack":
        n = c["E"] * c["K"] * c["D"]
        return {"bytes": 3 * n + 4 * c["E"] * _blocks(c["K"]) * _blocks(c["D"]), "flops": 3 * n}
    if c["op"] == "linear":
        T, K, D = c["T"], c["K"], c["D"]
        return {"bytes": T * K + K * D + T * D * (4 if c["out"] == "f32" else 2) +
                4 * (T * _blocks(K) + _blocks(K) * _blocks(D)), "flops": 2 * T * K * D}
    T, E, k, H, I = c["T"], c["E"], c["topk"], c["H"], c["I"]
    active = E * (1 - (1 - k / E) ** T)  # distinct experts that uniform routing reads, on average
    return {"bytes": int(active * 3 * H * I + 4 * T * H + 4 * T * E + 8 * T * k), "flops": 6 * T * k * H * I}


# ------------------------------------------------------- exact, in 64 bits ---


def _round_e4m3(v):
    """float64 -> the nearest E4M3 value, ties to the even mantissa"""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(v) * torch.round(a / step.clamp_min(E4M3_TINY)).mul(step.clamp_min(E4M3_TINY)).clamp_max(E4M3_MAX)


def _block_scale(t, dims):
    amax = t.abs().amax(dim=dims, keepdim=True)
    return torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), torch.ones_like(amax))


def _pad_to(v, *sizes):
    out = v.new_zeros(*v.shape[:-len(sizes)], *sizes)
    out[tuple([...] + [slice(0, n) for n in v.shape[-len(sizes):]])] = v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "prep":
        T, K, kb = s["T"], s["K"], _blocks(s["K"])
        x, out = s["x"].double(), {}
        if s["kind"] == "silu":
            v = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        elif s["kind"] == "plain":
            v = x
        else:
            if s["kind"] == "residual":
                x = (x + s["res"].double()).bfloat16().double()
                out["h"] = x
            v = x / torch.sqrt((x * x).sum(-1, keepdim=True) / K + EPS) * s["gamma"].double()
        t = _pad_to(v, kb * BLOCK).view(T, kb, BLOCK)
        sc = _block_scale(t, -1)
        out["codes"] = _round_e4m3(t / sc).view(T, -1)[:, :K]
        out["scales"] = sc[..., 0]
        return out
    if s["op"] == "pack":
        E, K, D = s["W"].shape
        db, kb = _blocks(D), _blocks(K)
        t = _pad_to(s["W"].double().mT, db * BLOCK, kb * BLOCK).view(E, db, BLOCK, kb, BLOCK)
        sc = _block_scale(t, (2, 4))
        q = _round_e4m3(t / sc).view(E, db * BLOCK, kb * BLOCK)[:, :D, :K]
        return {"codes": q, "scales": sc[:, :, 0, :, 0]}
    if s["op"] == "linear":
        T, K, D = s["T"], s["K"], s["D"]
        row = torch.arange(K, device="cuda") // BLOCK
        col = torch.arange(D, device="cuda") // BLOCK
        x = s["x"].double() * s["xs"].double()[:, row]
        w = s["w"].double() * s["ws"].double()[col][:, row]
        return torch.mm(x, w.mT)
    T, E, k, H, I = s["T"], s["E"], s["topk"], s["H"], s["I"]
    lg = s["logits"].double()
    # the k largest, the lower index first among equals: order by (-logit, index)
    rank = (lg[:, None, :] > lg[:, :, None]).sum(-1) + \
        ((lg[:, None, :] == lg[:, :, None]) & (torch.arange(E, device="cuda")[None, None, :] <
                                               torch.arange(E, device="cuda")[None, :, None])).sum(-1)
    ids = torch.argsort(rank, dim=-1)[:, :k]
    p = torch.softmax(torch.gather(lg, 1, ids), dim=-1)
    rh, ri = torch.arange(H, device="cuda") // BLOCK, torch.arange(I, device="cuda") // BLOCK
    r2 = torch.arange(2 * I, device="cuda") // BLOCK
    x, y = s["x"].double(), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = x[t] @ (s["w13"][e].double() * s["s13"][e].double()[r2][:, rh]).mT
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y[t] += p[t, j, None] * (h @ (s["w2"][e].double() * s["s2"][e].double()[rh][:, ri]).mT)
    return {"y": y, "ids": ids.int(), "weights": p}
