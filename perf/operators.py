"""Measured cases of the FP8 block-scaled matmul and the mixture-of-experts layer.

Each operator has its plain form here (elementary torch operations, 32 bits, one rounding at
the end) beside the call a user makes of the library (`own`), and `exact` gives the same
result from the definitions in 64 bits.

Operators:
  quant    e4m3 codes with an f32 scale per 1 x 128 block of an activation, or per 128 x 128
           block of a weight. Returned as the values the codes stand for, and the scales.
  gemm     y = x . W^T, W in e4m3 with 128 x 128 scales, x quantised in the call per 1 x 128.
  backward dx = dy . W for the same weights (input gradient of a frozen layer), dy quantised
           in the call per 1 x 128 along N.
  moe      router (softmax top-k), experts' gate and up products, silu(g) * u, down product
           and weighted sum for a few tokens; Q4_0 weights, Q8_0 activations.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest scale, so that its reciprocal is finite
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
LARGEST_MNK = 4096 * 14336 * 4096     # multiply-adds of the largest listed product
LARGEST_EXPERTS = 8 * 4096 * 14336    # experts x hidden x intermediate of the largest listed layer


# ------------------------------------------------------------------ cases
def listed():
    return [
        # an activation of a prefill chunk, quantised once for several projections
        {"name": "quant_act_2048x4096", "op": "quant", "block": "row", "M": 2048, "K": 4096, "x": "bf16"},
        # a weight matrix quantised when a checkpoint is loaded, ragged in both directions
        {"name": "quant_weight_14300x4000", "op": "quant", "block": "tile", "M": 14300, "K": 4000, "x": "f32"},
        # one token through a square projection: the weights' bytes and the call itself
        {"name": "gemm_decode_1x4096x4096", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "x": "bf16", "y": "bf16",
         "bias": False},
        # a small decode batch through an MLP projection
        {"name": "gemm_batch_16x14336x4096", "op": "gemm", "M": 16, "N": 14336, "K": 4096, "x": "bf16", "y": "bf16",
         "bias": False},
        # a short prompt, no size a multiple of a tile, f32 in and out
        {"name": "gemm_ragged_201x1531x1936", "op": "gemm", "M": 201, "N": 1531, "K": 1936, "x": "f32", "y": "f32",
         "bias": True},
        # a long prompt through an MLP projection: the matrix units' rate
        {"name": "gemm_prefill_4096x14336x4096", "op": "gemm", "M": 4096, "N": 14336, "K": 4096, "x": "bf16",
         "y": "bf16", "bias": False},
        # input gradient of a training step on a frozen square projection
        {"name": "backward_1024x4096x4096", "op": "backward", "M": 1024, "N": 4096, "K": 4096, "x": "bf16",
         "y": "bf16"},
        # input gradient for a few tokens, ragged
        {"name": "backward_ragged_9x1000x2064", "op": "backward", "M": 9, "N": 1000, "K": 2064, "x": "f32",
         "y": "f32"},
        # one token, many small experts
        {"name": "moe_1tok_64x2048x1024_top8", "op": "moe", "T": 1, "E": 64, "H": 2048, "I": 1024, "k": 8,
         "renorm": True},
        # a small decode batch, few large experts
        {"name": "moe_4tok_8x4096x14336_top2", "op": "moe", "T": 4, "E": 8, "H": 4096, "I": 14336, "k": 2,
         "renorm": True},
        # a larger decode batch: every expert used, several tokens each
        {"name": "moe_64tok_64x2048x1024_top8", "op": "moe", "T": 64, "E": 64, "H": 2048, "I": 1024, "k": 8,
         "renorm": False},
        # odd numbers of tokens, experts and blocks
        {"name": "moe_13tok_11x1504x736_top3", "op": "moe", "T": 13, "E": 11, "H": 1504, "I": 736, "k": 3,
         "renorm": False},
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], spread over its logarithm, a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "backward", "backward", "moe", "moe", "moe", "quant"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "quant":
        block = rng.choice(["row", "tile"])
        M = _log(rng, 1, 14336)
        return {"op": op, "block": block, "M": M, "K": _log(rng, 128, 14336, 16), "x": x}
    if op == "moe":
        while True:
            E = _log(rng, 4, 64)
            H, inter = _log(rng, 256, 4096, 32), _log(rng, 128, 14336, 32)
            if E * H * inter <= LARGEST_EXPERTS:
                break
        return {"op": op, "T": _log(rng, 1, 64), "E": E, "H": H, "I": inter, "k": _log(rng, 1, min(8, E)),
                "renorm": rng.random() < 0.5}
    while True:
        M, N, K = _log(rng, 1, 4096), _log(rng, 64, 14336), _log(rng, 128, 14336, 16)
        if M * N * K <= LARGEST_MNK:
            break
    case = {"op": op, "M": M, "N": N, "K": K, "x": x, "y": rng.choice(["bf16", "bf16", "f32"])}
    if op == "gemm":
        case["bias"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _over(v, by):
    """v / by, correctly rounded (dividing a tensor by a number multiplies by its reciprocal)."""
    return v / torch.full_like(v, by)


def _pack_tiles(w):
    """e4m3 codes and 128 x 128 scales of a weight matrix (what a checkpoint holds)."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    amax = torch.nn.functional.pad(w.abs(), (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128).amax((1, 3))
    s = _over(amax, E4M3_MAX).clamp_min(TINY)
    inv = (1.0 / s).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return (w * inv).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _pack_q4_0(w):
    """Q4_0 codes (rows, K/2) and fp16 scale bits (rows, K/32) of a matrix."""
    rows, K = w.shape
    b = w.view(rows, K // 32, 32)
    mx = b.gather(2, b.abs().argmax(2, keepdim=True))
    d = mx / -8.0
    inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
    q = (b * inv + 8.5).clamp_(0, 15.99).to(torch.uint8)
    codes = (q[..., :16] | (q[..., 16:] << 4)).reshape(rows, K // 2).contiguous()
    return codes, d.squeeze(2).to(torch.float16).view(torch.int16).contiguous()


def _experts(gen, E, rows, cols):
    """Stacked Q4_0 experts, one drawn at a time to keep the f32 weights small."""
    parts = [_pack_q4_0(torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)) for _ in range(E)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _activation(gen, M, K, dtype):
    """Activations as a norm layer leaves them: rows of different size, a few large channels."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=gen, device="cuda"))
    x *= torch.exp(0.5 * torch.randn(1, K, generator=gen, device="cuda"))
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "quant":
        M, K = case["M"], case["K"]
        if case["block"] == "row":
            st["x"] = _activation(gen, M, K, case["x"])
        else:
            st["x"] = (torch.randn(M, K, generator=gen, device="cuda") * 0.02).to(DTYPES[case["x"]])
    elif case["op"] == "moe":
        T, E, H, inter = case["T"], case["E"], case["H"], case["I"]
        st["x"] = _activation(gen, T, H, "bf16")
        st["router"] = (torch.randn(E, H, generator=gen, device="cuda") / math.sqrt(H)).to(torch.bfloat16)
        st["gu_qs"], st["gu_d"] = _experts(gen, E, 2 * inter, H)
        st["dn_qs"], st["dn_d"] = _experts(gen, E, H, inter)
        if own:
            import block_quantized_w4a8_b200 as w4a8
            st["ws"] = w4a8.moe_workspace(T, E, H, inter, case["k"], "cuda")
    else:
        M, N, K = case["M"], case["N"], case["K"]
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
        w *= torch.exp(0.5 * torch.randn(N, 1, generator=gen, device="cuda"))
        st["wq"], st["wsc"] = _pack_tiles(w)
        st["x"] = _activation(gen, M, K if case["op"] == "gemm" else N, case["x"])
        st["bias"] = torch.randn(N, generator=gen, device="cuda") if case.get("bias") else None
        if own:
            import block_quantized_w4a8_b200 as w4a8
            st["ws"] = w4a8.fp8_workspace(M, N, K, "cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _quant_rows(x):
    """e4m3 codes (as f32) and scales of 1 x 128 blocks along the last axis."""
    M, K = x.shape
    kb = -(-K // 128)
    b = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(M, kb, 128)
    s = _over(b.abs().amax(2), E4M3_MAX).clamp_min(TINY)
    q = (b * (1.0 / s).unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    return q.view(M, kb * 128)[:, :K], s


def _spread(s, rows, cols):
    """128 x 128 block scales spread over the matrix."""
    return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _dequant_q4_0(codes, d, K):
    lo, hi = (codes & 15).view(*codes.shape[:-1], K // 32, 16), (codes >> 4).view(*codes.shape[:-1], K // 32, 16)
    q = torch.cat([lo, hi], -1).float() - 8.0
    return (q * d.view(torch.float16).float().unsqueeze(-1)).view(*codes.shape[:-1], K)


def _q8_0(x):
    """x quantised to Q8_0 along the last axis, as the values the codes stand for."""
    b = x.view(*x.shape[:-1], x.shape[-1] // 32, 32)
    d = _over(b.abs().amax(-1, keepdim=True), 127.0)
    inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
    v = (b * inv).double()
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)
    return (q.clamp(-127, 127).float() * d).view(x.shape)


def _route(x, router, k, renorm):
    """Chosen experts (largest logit first, the lower index on ties) and their weights."""
    logits = x.double() @ router.double().T
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(top - top[:, :1])
    p = e[:, :k] / (e[:, :k] if renorm else e).sum(1, keepdim=True)
    return ids[:, :k].to(torch.int32).contiguous(), p.float()


def _plain_moe(st):
    c = st["case"]
    x = st["x"]
    ids, p = _route(x, st["router"], c["k"], c["renorm"])
    gu = torch.matmul(_q8_0(x.float()), _dequant_q4_0(st["gu_qs"], st["gu_d"], c["H"]).transpose(1, 2))  # E, T, 2I
    g, u = gu[..., : c["I"]], gu[..., c["I"]:]
    h = _q8_0((g / (1.0 + torch.exp(-g)) * u).contiguous())
    y = torch.matmul(h, _dequant_q4_0(st["dn_qs"], st["dn_d"], c["I"]).transpose(1, 2))  # E, T, H
    share = torch.zeros(c["T"], c["E"], device=x.device).scatter_add_(1, ids.long(), p)
    return (y * share.T.unsqueeze(2)).sum(0).to(torch.bfloat16), ids, p


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import block_quantized_w4a8_b200 as w4a8
        if op == "quant":
            q, s = w4a8.quant_act_fp8(state["x"]) if c["block"] == "row" else w4a8.pack_fp8(state["x"])
            return q, s
        if op == "moe":
            return w4a8.moe_layer_q4_0(state["x"], state["router"], state["gu_qs"], state["gu_d"], state["dn_qs"],
                                       state["dn_d"], c["k"], renorm=c["renorm"], out_dtype=torch.bfloat16,
                                       ws=state["ws"])
        if op == "gemm":
            return w4a8.gemm_fp8(state["x"], state["wq"], state["wsc"], bias=state["bias"],
                                 out_dtype=DTYPES[c["y"]], ws=state["ws"])
        return w4a8.gemm_fp8_backward(state["x"], state["wq"], state["wsc"], out_dtype=DTYPES[c["y"]],
                                      ws=state["ws"])
    if op == "moe":
        return _plain_moe(state)
    if op == "quant":
        if c["block"] == "row":
            q, s = _quant_rows(state["x"])
            return q.to(torch.float8_e4m3fn), s
        return _pack_tiles(state["x"].float())
    N, K = state["wq"].shape
    w = state["wq"].float() * _spread(state["wsc"], N, K)
    q, s = _quant_rows(state["x"])
    v = q * s.repeat_interleave(128, 1)[:, : q.shape[1]]
    y = v @ w.T if op == "gemm" else v @ w
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(DTYPES[c["y"]])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "quant":
        M, K = case["M"], case["K"]
        scales = (M if case["block"] == "row" else -(-M // 128)) * -(-K // 128)
        return {"bytes": M * K * (BYTES[case["x"]] + 1) + 4 * scales, "flops": 2 * M * K}
    if case["op"] == "moe":
        T, E, H, inter, k = case["T"], case["E"], case["H"], case["I"], case["k"]
        used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token chose, for an even router
        weights = used * 3 * H * inter * (0.5 + 2 / 32)
        return {"bytes": weights + 2 * E * H + 4 * T * H + 8 * T * k,
                "flops": 6 * T * k * H * inter + 2 * T * E * H}
    M, N, K = case["M"], case["N"], case["K"]
    scales = 4 * -(-N // 128) * -(-K // 128)
    a, b = (K, N) if case["op"] == "gemm" else (N, K)
    return {"bytes": N * K + scales + M * a * BYTES[case["x"]] + M * b * BYTES[case["y"]]
            + (4 * N if case.get("bias") else 0), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3(v):
    """v (f64, |v| <= 448) rounded to the nearest e4m3 value, ties to even, by arithmetic:
    a spacing of 2^(e-3) in each binade e >= -6, 2^-9 below."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return torch.round(v / step) * step


def _codes(x, amax):
    """Scales (f32, as the definition rounds them) and code values of x against amax; the
    quotient is the f32 product with the f32 reciprocal, computed here in 64 bits and
    rounded to 32 at the definition's two places."""
    s = torch.clamp_min((amax.double() / E4M3_MAX).float(), TINY)
    inv = (1.0 / s.double()).float()
    v = (x.double() * inv.double()).float().double().clamp(-E4M3_MAX, E4M3_MAX)
    return _e4m3(v), s


def _exact_rows(x):
    M, K = x.shape
    cols = torch.arange(K, device=x.device) // 128
    nb = int(cols[-1]) + 1
    amax = torch.stack([x[:, 128 * b: 128 * b + 128].float().abs().amax(1) for b in range(nb)], 1)
    s_all = amax[:, cols]
    q, s = _codes(x.float(), s_all)
    return q, s, _codes(amax, amax)[1]


def _exact_tiles(x):
    N, K = x.shape
    rb, cb = torch.arange(N, device=x.device) // 128, torch.arange(K, device=x.device) // 128
    amax = torch.stack([torch.stack([x[128 * i: 128 * i + 128, 128 * j: 128 * j + 128].float().abs().max()
                                     for j in range(-(-K // 128))]) for i in range(-(-N // 128))])
    return _codes(x.float(), amax[rb][:, cb])[0], _codes(amax, amax)[1]


def _exact_q8_0(x):
    """Q8_0 values along the last axis: d = f32(amax/127), codes rounded half away from zero."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = (b.abs().amax(-1, keepdim=True) / 127.0).float().double()
    inv = torch.where(d > 0, (1.0 / d).float().double(), torch.zeros_like(d))
    v = (b * inv).float().double()
    q = torch.where(v < 0, -torch.floor(0.5 - v), torch.floor(v + 0.5)).clamp(-127, 127)
    return (q * d).reshape(x.shape)


def _exact_q4_0(codes, d):
    blocks = codes.reshape(codes.shape[0], -1, 16)
    scale = d.view(torch.float16).double().unsqueeze(-1)
    out = torch.empty(*blocks.shape[:2], 32, dtype=torch.float64, device=codes.device)
    out[..., :16] = ((blocks % 16).double() - 8) * scale
    out[..., 16:] = (torch.div(blocks, 16, rounding_mode="floor").double() - 8) * scale
    return out.reshape(codes.shape[0], -1)


def _exact_moe(st):
    c = st["case"]
    x = st["x"].double()
    logits = (x.unsqueeze(1) * st["router"].double().unsqueeze(0)).sum(2)
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    order = [sorted(range(c["E"]), key=lambda e, row=row: (-row[e], e))[: c["k"]] for row in logits.tolist()]
    ids = torch.tensor(order, dtype=torch.int32, device="cuda")
    chosen = logits.gather(1, ids.long())
    total = chosen if c["renorm"] else logits
    p = torch.exp(chosen - torch.logsumexp(total, 1, keepdim=True))
    xq = _exact_q8_0(x)
    for e in sorted({e for row in order for e in row}):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        gu = xq[t] @ _exact_q4_0(st["gu_qs"][e], st["gu_d"][e]).T
        g, u = gu[:, : c["I"]], gu[:, c["I"]:]
        h = _exact_q8_0(g * torch.sigmoid(g) * u)
        y.index_add_(0, t, p[t, slot].unsqueeze(1) * (h @ _exact_q4_0(st["dn_qs"][e], st["dn_d"][e]).T))
    return y, ids, p


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "moe":
        return _exact_moe(st)
    if op == "quant":
        if case["block"] == "tile":
            return _exact_tiles(st["x"])
        q, _, s = _exact_rows(st["x"])
        return q, s
    N, K = st["wq"].shape
    rb, cb = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    w = st["wq"].double() * st["wsc"].double()[rb][:, cb]
    q, s, _ = _exact_rows(st["x"])
    v = q * s.double()
    y = v @ (w.T if op == "gemm" else w)
    return y + st["bias"].double() if st["bias"] is not None else y
