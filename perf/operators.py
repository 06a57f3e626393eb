"""The layer's operators around the routed experts, as cases to be timed and compared: the residual
RMS norm (forward, with bf16 and MXFP8 outputs, and backward), the dense gated feed-forward block
(the shared expert; forward and backward) and the AdamW step over many tensors.

With ``own`` false ``run`` computes a case with elementary torch operations in fp32; with ``own``
true it makes the library's calls. ``exact`` computes the same outputs in fp64, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
EPS_NORM = 1e-6
LR, BETA1, BETA2, EPS_ADAM, STEP = 1e-3, 0.9, 0.95, 1e-8, 100
SEED, STREAM = 7, 40


def _lib():
    import precision_moe_numerics_amd as P
    return P


# ---- cases ------------------------------------------------------------------------------------


def _norm(name, rows, cols, res, y, mx, save):
    """res: the residual stream's type ("" without one); y / mx: bf16 / MXFP8 output; save: the
    reciprocal norms are kept for a backward pass."""
    return {"name": name, "op": "norm_fwd", "rows": rows, "cols": cols, "res": res, "y": y, "mx": mx, "save": save}


def _norm_bwd(name, rows, cols, z, dy, dres):
    return {"name": name, "op": "norm_bwd", "rows": rows, "cols": cols, "z": z, "dy": dy, "dres": dres}


def _ffn(name, op, tokens, hidden, ffn, add=False, save=False):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "ffn": ffn, "add": add, "save": save}


def _adamw(name, bits, tensors, total, grad):
    return {"name": name, "op": "adamw", "bits": bits, "tensors": tensors, "total": total, "grad": grad}


def listed():
    return [
        # one decoded token before an MXFP8 layer: latency of one launch
        _norm("norm_token", 1, 7168, "bf16", True, True, False),
        # the tokens of the 32-expert layer in training: both outputs, the statistics saved
        _norm("norm_tokens", 16384, 4096, "bf16", True, True, True),
        # a ragged prefill batch with an fp32 residual stream, straight to 8 bits
        _norm("norm_ragged_f32", 1003, 7168, "f32", False, True, False),
        # the backward of the training case: the gradient along the residual joins in
        _norm_bwd("norm_bwd_tokens", 16384, 4096, "bf16", "bf16", True),
        # a short microbatch with fp32 gradients and stream
        _norm_bwd("norm_bwd_ragged_f32", 777, 7168, "f32", "f32", True),
        # the shared expert of the 48-expert layer for one decoded token: the weights' bytes
        _ffn("ffn_token", "ffn_fwd", 1, 7168, 2048, add=True),
        # a serving batch of decoded tokens, odd
        _ffn("ffn_batch_45", "ffn_fwd", 45, 7168, 2048, add=True),
        # the same block in training on 8192 tokens
        _ffn("ffn_train", "ffn_fwd", 8192, 7168, 2048, add=True, save=True),
        # a small microbatch's backward with odd tokens
        _ffn("ffn_bwd_501", "ffn_bwd", 501, 4096, 1024),
        # the training case's backward
        _ffn("ffn_bwd_train", "ffn_bwd", 8192, 7168, 2048),
        # norm weights, biases and router weights of many layers: many small tensors
        _adamw("adamw32_many", 32, 280, 2_400_000, "f32"),
        # the expert matrices of a rank, states in 8 bits, bf16 gradients
        _adamw("adamw8_large", 8, 24, 150_000_000, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ffn_fwd", "ffn_bwd", "adamw"])
    if op == "norm_fwd":
        outs = rng.choice([(True, False), (False, True), (True, True)])
        c = _norm("", _log(rng, 1, 16384), 32 * _log(rng, 2, 256), rng.choice(["", "bf16", "f32"]), *outs,
                  rng.random() < 0.5)
    elif op == "norm_bwd":
        c = _norm_bwd("", _log(rng, 1, 16384), 8 * _log(rng, 8, 1024), rng.choice(["bf16", "f32"]),
                      rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    elif op == "ffn_fwd":
        save = rng.random() < 0.4
        c = _ffn("", op, _log(rng, 1, 8192), 8 * _log(rng, 32, 896), 8 * _log(rng, 16, 256), rng.random() < 0.5, save)
    elif op == "ffn_bwd":
        c = _ffn("", op, _log(rng, 1, 8192), 8 * _log(rng, 32, 896), 8 * _log(rng, 16, 256))
    else:
        total = _log(rng, 1000, 100_000_000)
        c = _adamw("", rng.choice([32, 8]), min(rng.randint(1, 300), max(1, total // 200)), total,
                   rng.choice(["f32", "bf16"]))
    del c["name"]
    return c


# ---- inputs -----------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "": 0}


def _lengths(case):
    """The lengths of an AdamW case's tensors: spread over their logarithm, odd ones among them, in
    a flat buffer where each begins at a multiple of 32 values."""
    n = case["tensors"]
    w = [math.exp(2.0 * math.sin(1.7 * i + 0.3)) for i in range(n)]
    s = sum(w)
    lens = [max(1, int(case["total"] * x / s)) for x in w]
    spans = [-(-k // 32) * 32 for k in lens]
    return lens, spans


def _norm_state(case, seed, g):
    rows, cols = case["rows"], case["cols"]
    s = {"case": case, "gamma": 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)}
    # a stream whose rows differ in size, with a few channels far above the rest, as residual
    # streams have
    ch = torch.ones(cols, device=DEV)
    ch[:: max(cols // 8, 1)] = 12.0
    row = torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    stream = torch.randn((rows, cols), generator=g, device=DEV) * row * ch
    return s, stream


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norm_fwd":
        s, stream = _norm_state(case, seed, g)
        if case["res"]:
            s["residual"] = stream.to(DT[case["res"]])
            s["x"] = _normal(g, (case["rows"], case["cols"]), 0.3)
        else:
            s["residual"], s["x"] = None, stream.to(torch.bfloat16)
        return s
    if op == "norm_bwd":
        s, stream = _norm_state(case, seed, g)
        shape = (case["rows"], case["cols"])
        s["z"] = stream.to(DT[case["z"]])
        s["rstd"] = torch.rsqrt(s["z"].float().square().mean(1) + EPS_NORM)
        s["dy"] = _normal(g, shape, 1e-3, DT[case["dy"]])
        s["dres"] = _normal(g, shape, 1e-3, DT[case["z"]]) if case["dres"] else None
        return s
    if op in ("ffn_fwd", "ffn_bwd"):
        M, H, F = case["tokens"], case["hidden"], case["ffn"]
        s = {"case": case, "x": _normal(g, (M, H), 1.0), "w13": _normal(g, (2 * F, H), 1.2 / math.sqrt(H)),
             "w2": _normal(g, (H, F), 1.0 / math.sqrt(F))}
        if op == "ffn_fwd":
            s["add"] = _normal(g, (M, H), 0.5) if case["add"] else None
        else:
            s["dy"] = _normal(g, (M, H), 1e-3)
            s["h13"] = _normal(g, (M, 2 * F), 1.2)
        return s
    # AdamW in the middle of a run: moments of past gradients of very different sizes per tensor
    lens, spans = _lengths(case)
    n = sum(spans)
    T = len(lens)
    s = {"case": case}
    spans_t = torch.tensor(spans, device=DEV)
    s["lens"], s["spans"], s["spans_list"] = torch.tensor(lens, device=DEV), spans_t, spans
    begin = torch.cumsum(spans_t, 0) - spans_t
    s["begin"] = begin
    s["decay"] = torch.tensor([0.1 if i % 3 else 0.0 for i in range(T)], device=DEV)
    tid = torch.repeat_interleave(torch.arange(T, device=DEV), spans_t, output_size=n)
    valid = torch.arange(n, device=DEV) - begin[tid] < s["lens"][tid]
    size = torch.exp(torch.randn(T, generator=g, device=DEV))[tid].mul_(1e-3).mul_(valid)
    s["p"] = torch.randn(n, generator=g, device=DEV).mul_(0.02).mul_(valid)
    s["copy"] = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    s["g"] = torch.randn(n, generator=g, device=DEV).mul_(size).to(DT[case["grad"]])
    m = torch.randn(n, generator=g, device=DEV).mul_(size).mul_(0.25)
    v = torch.randn(n, generator=g, device=DEV).mul_(0.4).exp_().mul_(size).square_()
    del size, tid, valid
    if case["bits"] == 8:
        s["m"], s["me"] = _mxfp8_plain(m.view(-1, 32))
        s["v"], s["ve"] = _mxfp8_plain(v.sqrt_().view(-1, 32))
        for k in ("m", "v"):
            s[k] = s[k].view(torch.uint8).view(-1)
    else:
        s["m"], s["v"] = m, v
    s["lens_list"] = lens
    if own:
        s["plan"] = _plan(s)   # the list of tensors, kept by a program from step to step
    return s


def _plan(s):
    P = _lib()
    tensors, at = [], 0
    for i, (n, span) in enumerate(zip(s["lens_list"], s["spans_list"])):
        f = slice(at, at + n)
        b = slice(at // 32, (at + span) // 32)
        e8 = dict(m_e8m0=s["me"][b], v_e8m0=s["ve"][b]) if s["case"]["bits"] == 8 else {}
        tensors.append(P.AdamWTensor(param=s["p"][f], grad=s["g"][f], m=s["m"][f], v=s["v"][f], copy=s["copy"][f],
                                     weight_decay=0.1 if i % 3 else 0.0, **e8))
        at += span
    return P.AdamWPlan(tensors)


# ---- plain forms ------------------------------------------------------------------------------


def _mxfp8_exponent(amax):
    """Smallest e in [-127, 127] with amax <= 448 * 2^e."""
    _, ex = torch.frexp(amax)
    e = ex - 9
    e = e + (amax > torch.ldexp(torch.full_like(amax, 448.0), e))
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _mxfp8_plain(y):
    """y fp32 [..., 32]: E4M3 codes (rounded to nearest even) and E8M0 bytes."""
    e = _mxfp8_exponent(y.abs().amax(-1))
    codes = torch.ldexp(y, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _norm_fwd_plain(s):
    c = s["case"]
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    rstd = torch.rsqrt(z.square().mean(1, keepdim=True) + EPS_NORM)
    y = z * rstd * s["gamma"]
    out = {}
    if s["residual"] is not None:
        out["z"] = z.to(s["residual"].dtype)
    if c["save"]:
        out["rstd"] = rstd.squeeze(1)
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    if c["mx"]:
        codes, e = _mxfp8_plain(y.view(c["rows"], -1, 32))
        out["codes"], out["scales"] = codes.view(c["rows"], -1), e.view(torch.float8_e8m0fnu)
    return out


def _norm_bwd_plain(s):
    z, dy, rstd = s["z"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    xh = z * rstd
    gy = dy * s["gamma"]
    dz = rstd * (gy - xh * (gy * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dz = dz + s["dres"].float()
    return {"dz": dz.to(s["z"].dtype), "dgamma": (dy * xh).sum(0)}


def _ffn_fwd_plain(s):
    F = s["case"]["ffn"]
    h = s["x"].float() @ s["w13"].float().t()
    h1, h3 = h[:, :F], h[:, F:]
    y = (h1 * torch.sigmoid(h1) * h3) @ s["w2"].float().t()
    if s["add"] is not None:
        y = y + s["add"].float()
    out = {"y": y.to(torch.bfloat16)}
    if s["case"]["save"]:
        out["h13"] = h.to(torch.bfloat16)
    return out


def _ffn_bwd_plain(s):
    F = s["case"]["ffn"]
    x, w13, w2, dy, h = (s[k].float() for k in ("x", "w13", "w2", "dy", "h13"))
    h1, h3 = h[:, :F], h[:, F:]
    sg = torch.sigmoid(h1)
    act = h1 * sg
    da = dy @ w2
    dh = torch.cat([da * h3 * (sg + act * (1 - sg)), da * act], 1)
    grads = {"dx": dh @ w13, "dw13": dh.t() @ x, "dw2": dy.t() @ (act * h3)}
    return {k: v.to(torch.bfloat16) for k, v in grads.items()}


def _mulhilo(a, k):
    """High and low 32 bits of a * k for a, k < 2^32 held in int64."""
    lo, hi = (a & 0xFFFF) * k, (a >> 16) * k
    t = hi + (lo >> 16)
    return (t >> 16) & 0xFFFFFFFF, ((t & 0xFFFF) << 16) | (lo & 0xFFFF)


def _rand16(blk, stream, seed):
    """The 16-bit random values of elements 8 blk .. 8 blk + 7 under (seed, stream), [n, 8]:
    Philox4x32-10 on the counter (blk, stream, 0)."""
    c0, c1, c2, c3 = blk & 0xFFFFFFFF, blk >> 32, stream, torch.zeros_like(blk)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([w & 0xFFFF, w >> 16], 2).view(-1, 8)


def _mxfp8_sr_plain(y, r16, positive):
    """y fp32 [n, 32] to E4M3 codes and E8M0 bytes, rounded up where r16 < floor(f 2^16), f the
    position between the two neighbours. positive: a value above zero never becomes zero."""
    e = _mxfp8_exponent(y.abs().amax(-1))
    a = torch.ldexp(y.abs(), -e.unsqueeze(-1))
    ex = (torch.frexp(a)[1] - 1).clamp_min(-6) - 3
    q = torch.ldexp(a, -ex)
    lo = torch.floor(q)
    up = r16.view(a.shape) < torch.floor((q - lo) * 65536.0)
    q = lo + up
    if positive:
        q = torch.where((a > 0) & (q == 0), torch.ones_like(q), q)
    return torch.copysign(torch.ldexp(q, ex), y).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _adamw_plain(s):
    c = s["case"]
    n, g = s["p"].numel(), s["g"].float()
    decay = torch.repeat_interleave(s["decay"], s["spans"], output_size=n)
    if c["bits"] == 8:
        unpack = lambda q, e: torch.ldexp(s[q].view(torch.float8_e4m3fn).float().view(-1, 32),  # noqa: E731
                                          s[e].int().unsqueeze(1) - 127).view(-1)
        m, v = unpack("m", "me"), unpack("v", "ve").square()
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    mh, vh = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    s["p"].copy_(s["p"] - LR * (mh / (vh.sqrt() + EPS_ADAM) + decay * s["p"]))
    s["copy"].copy_(s["p"])
    if c["bits"] == 8:
        spans8 = s["spans"] // 8
        tid = torch.repeat_interleave(torch.arange(c["tensors"], device=DEV), spans8, output_size=n // 8)
        blk = torch.arange(n // 8, device=DEV) - (s["begin"] // 8)[tid]
        for q, e, value, k in (("m", "me", m, 0), ("v", "ve", v.sqrt(), 1)):
            r16 = _rand16(blk, STREAM + 2 * tid + k, SEED + STEP)
            codes, scales = _mxfp8_sr_plain(value.view(-1, 32), r16, k == 1)
            s[q].copy_(codes.view(torch.uint8).view(-1))
            s[e].copy_(scales)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    out = {"p": s["p"], "copy": s["copy"]}
    if s["case"]["bits"] == 8:
        out.update(m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn),
                   m_scales=s["me"].view(torch.float8_e8m0fnu), v_scales=s["ve"].view(torch.float8_e8m0fnu))
    else:
        out.update(m=s["m"], v=s["v"])
    return out


# ---- the library's calls ----------------------------------------------------------------------


def _run_own(s):
    P = _lib()
    c = s["case"]
    if c["op"] == "norm_fwd":
        r = P.rmsnorm_residual_fwd(s["x"], s["gamma"], EPS_NORM, residual=s["residual"], want_y=c["y"],
                                   want_mxfp8=c["mx"], want_rstd=c["save"])
        out = {}
        if s["residual"] is not None:
            out["z"] = r.z
        if c["save"]:
            out["rstd"] = r.rstd
        if c["y"]:
            out["y"] = r.y
        if c["mx"]:
            out["codes"], out["scales"] = r.codes.view(torch.float8_e4m3fn), r.e8m0.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "norm_bwd":
        dz, dgamma = P.rmsnorm_residual_bwd(s["dy"], s["z"], s["gamma"], s["rstd"], dres=s["dres"])
        return {"dz": dz, "dgamma": dgamma}
    if c["op"] == "ffn_fwd":
        y, h13 = P.swiglu_ffn_fwd(s["x"], s["w13"], s["w2"], add=s["add"], save_h13=c["save"])
        return {"y": y, "h13": h13} if c["save"] else {"y": y}
    if c["op"] == "ffn_bwd":
        dx, dw13, dw2 = P.swiglu_ffn_bwd(s["dy"], s["x"], s["w13"], s["w2"], s["h13"], dw_dtype=torch.bfloat16)
        return {"dx": dx, "dw13": dw13, "dw2": dw2}
    P.adamw_step(s["plan"], lr=LR, step=STEP, beta1=BETA1, beta2=BETA2, eps=EPS_ADAM, seed=SEED, rng_stream=STREAM)
    return _adamw_out(s)


def run(state):
    if own:
        return _run_own(state)
    return {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "ffn_fwd": _ffn_fwd_plain,
            "ffn_bwd": _ffn_bwd_plain, "adamw": _adamw_plain}[state["case"]["op"]](state)


# ---- least work -------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "norm_fwd":
        n, r = case["rows"] * case["cols"], SIZE[case["res"]]
        b = n * (2 + 2 * r + 2 * case["y"] + 33 / 32 * case["mx"]) + 4 * case["cols"] + 4 * case["rows"] * case["save"]
        return {"bytes": b, "flops": 6 * n}
    if op == "norm_bwd":
        n, z = case["rows"] * case["cols"], SIZE[case["z"]]
        return {"bytes": n * (SIZE[case["dy"]] + z * (3 if case["dres"] else 2)) + 8 * case["cols"] + 4 * case["rows"],
                "flops": 12 * n}
    if op == "ffn_fwd":
        M, H, F = case["tokens"], case["hidden"], case["ffn"]
        return {"bytes": 2 * (M * H * (3 if case["add"] else 2) + 3 * H * F + (2 * M * F if case["save"] else 0)),
                "flops": 6 * M * H * F}
    if op == "ffn_bwd":
        M, H, F = case["tokens"], case["hidden"], case["ffn"]
        return {"bytes": 2 * (3 * M * H + 2 * M * F + 6 * H * F), "flops": 12 * M * H * F}
    n = sum(_lengths(case)[0])
    state = 16 if case["bits"] == 32 else 4 * 33 / 32
    return {"bytes": n * (8 + SIZE[case["grad"]] + 2 + state), "flops": 16 * n}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _exact_blocks(y):
    """E4M3 values and scales of y fp64 [rows, blocks, 32] by the definition: the smallest power of
    two that holds the block within 448, then the nearest value of the grid, ties to even."""
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448.0).clamp(-127, 127))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((e > -127) & (amax <= 448.0 * torch.exp2(e - 1)), e - 1, e)
    scale = torch.exp2(e)
    t = y / scale
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(t / step) * step, scale.squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = lambda k: s[k].double()  # noqa: E731
    if op == "norm_fwd":
        z = D("x") if s["residual"] is None else D("x") + D("residual")
        r = 1.0 / torch.sqrt((z * z).sum(1) / case["cols"] + EPS_NORM)
        y = z * r[:, None] * D("gamma")
        out = {"z": z if s["residual"] is not None else None, "rstd": r if case["save"] else None,
               "y": y if case["y"] else None}
        if case["mx"]:
            codes, scales = _exact_blocks(y.view(case["rows"], -1, 32))
            out["codes"], out["scales"] = codes.reshape(case["rows"], -1), scales
        return {k: v for k, v in out.items() if v is not None}
    if op == "norm_bwd":
        z, dy, r = D("z"), D("dy"), D("rstd")[:, None]
        t = dy * D("gamma")
        dot = (t * z).sum(1, keepdim=True) / case["cols"]
        dz = r * t - r ** 3 * dot * z
        if s["dres"] is not None:
            dz = dz + D("dres")
        return {"dz": dz, "dgamma": (dy * z * r).sum(0)}
    if op == "ffn_fwd":
        F = case["ffn"]
        x = D("x")
        h1, h3 = x @ D("w13")[:F].t(), x @ D("w13")[F:].t()
        y = (h1 / (1 + torch.exp(-h1)) * h3) @ D("w2").t()
        if s["add"] is not None:
            y = y + D("add")
        return {"y": y, "h13": torch.cat([h1, h3], 1)} if case["save"] else {"y": y}
    if op == "ffn_bwd":
        F = case["ffn"]
        h1, h3 = D("h13").split(F, 1)
        sg = 1 / (1 + torch.exp(-h1))
        da = D("dy") @ D("w2")
        d1, d3 = da * h3 * sg * (1 + h1 * (1 - sg)), da * h1 * sg
        return {"dx": d1 @ D("w13")[:F] + d3 @ D("w13")[F:],
                "dw13": torch.cat([d1.t() @ D("x"), d3.t() @ D("x")], 0), "dw2": D("dy").t() @ (h1 * sg * h3)}
    g = D("g")
    if case["bits"] == 8:
        value = lambda q, e: (s[q].view(torch.float8_e4m3fn).double().view(-1, 32)  # noqa: E731
                              * torch.exp2(s[e].double() - 127)[:, None]).view(-1)
        m0, v0 = value("m", "me"), value("v", "ve") ** 2
    else:
        m0, v0 = D("m"), D("v")
    m = m0 + (1 - BETA1) * (g - m0)
    v = v0 + (1 - BETA2) * (g * g - v0)
    decay = torch.cat([s["decay"][i].expand(k) for i, k in enumerate(s["spans_list"])]).double()
    step = m / (1 - BETA1 ** STEP) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS_ADAM)
    p = D("p") * (1 - LR * decay) - LR * step
    # states in 8 bits are rounded at random: their values are held by the plain form alone
    return {"p": p, "copy": p} if case["bits"] == 8 else {"p": p, "copy": p, "m": m, "v": v}
