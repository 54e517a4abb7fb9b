"""The mixture-of-experts layer on the GPU against its definition in 64 bits. Two kinds of
inputs: random ones, held to the bound that follows a relative error of 1e-5 * sum |terms|
per dot through h and its int8 rounding, and ones whose gate and up products are exact in f32
(integer activations, power-of-two weight scales), where next to nothing may differ."""
import numpy as np
import pytest
import torch

import block_quantized_w4a8_b200 as w4a8
from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
TOL = 1e-5


def pack(w):
    """Stacked experts (E, rows, K) -> packed codes, scales and dequantised f64 values."""
    E, rows, K = w.shape
    qs, d = w4a8.pack_q4_0(w.reshape(E * rows, K).cuda())
    v = ref.dequant_q4_0(qs.cpu().numpy(), d.cpu().numpy()).reshape(E, rows, K)
    return qs.view(E, rows, K // 2), d.view(E, rows, K // 32), v


def make(T, E, H, I, k, seed, dtype=torch.float32, exact=False):
    g = torch.Generator().manual_seed(seed)
    if exact:
        x = torch.randint(-6, 7, (T, H), generator=g).float()
        x[:, ::64], x[:, 32::64] = 127.0, -127.0  # every block's scale is 1
        gu = torch.randint(-7, 8, (E, 2 * I, H), generator=g).float() * 2.0 ** -9
        gu[:, :, ::32] = -8 * 2.0 ** -9  # every block's scale is 2^-9
        gu[:, :, 1::32] = 8 * 2.0 ** -9  # clipped to 7: keeps g and u of moderate size
    else:
        x = torch.randn(T, H, generator=g)
        gu = torch.randn(E, 2 * I, H, generator=g) / H ** 0.5
    dn = torch.randn(E, H, I, generator=g) / I ** 0.5
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    weights = torch.rand(T, k, generator=g) + 0.1
    return x.to(dtype), pack(gu), pack(dn), ids, weights


def check(y, yref, bound, what=""):
    got = y.float().cpu().numpy().astype(np.float64)
    if y.dtype == torch.bfloat16:  # half a step of the result
        bound = bound * (1 + 2.0 ** -8) + np.abs(yref) * 2.0 ** -8 + 2.0 ** -134
    err = np.abs(got - yref)
    assert got.shape == yref.shape
    assert np.all(err <= bound), f"{what}: {np.sum(err > bound)} of {err.size} outside, worst {np.max(err / bound)}"


def run(x, gu, dn, ids, weights, out=torch.float32, ws=None):
    return w4a8.moe_q4_0(x.cuda(), ids.cuda(), weights.cuda(), gu[0], gu[1], dn[0], dn[1], out_dtype=out, ws=ws)


def verify(x, gu, dn, ids, weights, out, rel, what=""):
    y = run(x, gu, dn, ids, weights, out)
    yref, bound = ref.experts(x.float().numpy(), ids.numpy(), weights.numpy().astype(np.float64), gu[2], dn[2], rel)
    check(y, yref, bound, what)
    assert w4a8.w4a8_last_device_error() == 0
    return y, yref, bound


# (T, E, H, I, top_k): one token, one block, odd counts, row tails of 32 rows, several row
# tiles, more tokens per expert than one tile of 8, all 64 tokens on one expert
SHAPES = [(1, 1, 32, 32, 1), (1, 8, 512, 96, 2), (2, 3, 96, 32, 2), (3, 5, 160, 224, 3), (5, 4, 256, 256, 1),
          (13, 11, 736, 352, 3), (16, 2, 512, 512, 2), (40, 3, 288, 128, 2), (64, 1, 256, 64, 1), (64, 16, 512, 256, 8),
          (1, 64, 2048, 1024, 8), (9, 2, 4096, 288, 1), (64, 9, 512, 1024, 5), (33, 4, 96, 2048, 4), (64, 256, 128, 64, 16),
          (20, 8, 160, 4160, 6)]


@pytest.mark.parametrize("T,E,H,I,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts(T, E, H, I, k, dtype):
    verify(*make(T, E, H, I, k, T + H, dtype), dtype, TOL)


@pytest.mark.parametrize("T,E,H,I,k", [s for s in SHAPES if s[2] <= 1024])
def test_experts_with_exact_gate_and_up(T, E, H, I, k):
    """|g| < 2^24 * 2^-9 with every partial sum a multiple of 2^-9: g and u have no error, so
    only the steps after them are bounded. H <= 1024: sums below 1024 * 127 * 8 < 2^24."""
    x, gu, dn, ids, weights = make(T, E, H, I, k, T + H + 1, exact=True)
    y = run(x, gu, dn, ids, weights)
    yref, bound = ref.experts(x.numpy(), ids.numpy(), weights.numpy().astype(np.float64), gu[2], dn[2], 0.0)
    A = np.zeros_like(yref)
    xv = ref.values(*ref.q8_0(x.numpy()))
    for t in range(T):  # the down product's own f32 sums
        for s in range(k):
            gus = gu[2][ids[t, s]] @ xv[t]
            h = gus[:I] / (1 + np.exp(-gus[:I])) * gus[I:]
            A[t] += abs(float(weights[t, s])) * (np.abs(dn[2][ids[t, s]]) @ (np.abs(h) * 1.01 + np.abs(h).max() / 127))
    check(y, yref, bound + TOL * A)


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("H,I", [(256, 256), (256, 288), (288, 256), (288, 288)])
def test_scale_rows_with_and_without_a_tensor_map(T, H, I):
    """Scale rows of 16-byte units come by TMA, others by plain loads; each product for itself."""
    verify(*make(T, 4, H, I, 2, H + 2 * I + T), torch.float32, TOL)


@pytest.mark.parametrize("T,E,H,I,k", [(33, 2, 4096, 64, 1), (64, 3, 2432, 288, 2), (1, 2, 4768, 96, 2), (40, 2, 2048, 512, 1),
                                       (5, 2, 1216, 96, 1), (2, 2, 2368, 320, 2)])
def test_every_cluster_size_of_down(T, E, H, I, k):
    """CTAs per 32 rows of H on 148 SMs: 1 (the first three), 2, 4, 4; smaller layers take 8."""
    verify(*make(T, E, H, I, k, T + H + I), torch.float32, TOL)


def test_empty_slots_repeated_experts_and_empty_tokens():
    T, E, H, I, k = 6, 5, 256, 96, 3
    x, gu, dn, ids, weights = make(T, E, H, I, k, 3)
    ids[0] = torch.tensor([-1, 2, -7])      # two empty slots
    ids[1] = -1                             # an empty token
    ids[2] = torch.tensor([4, 4, 4])        # one expert three times
    ids[3] = torch.tensor([5, 1000, 0])     # out of range: empty
    ids[4] = torch.tensor([1, 3, 1])        # twice, not next to each other
    y, yref, _ = verify(x, gu, dn, ids, weights, torch.float32, TOL)
    assert torch.equal(y[1], torch.zeros_like(y[1]))
    ids[:] = -1
    assert torch.equal(run(x, gu, dn, ids, weights), torch.zeros(T, H, device="cuda"))


@pytest.mark.parametrize("T,E,k", [(20, 5, 3), (64, 16, 16), (64, 40, 8)])
def test_random_slots(T, E, k):
    """Slots drawn with repeats and empty ones among them (more than 32 slots)."""
    H, I = 96, 64
    x, gu, dn, _, _ = make(T, E, H, I, 1, 4)
    g = torch.Generator().manual_seed(T + k)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).int()
    weights = torch.rand(T, k, generator=g)
    verify(x, gu, dn, ids, weights, torch.float32, TOL)


@pytest.mark.parametrize("T", [1, 2, 12])
def test_nan_in_h_reaches_its_token_and_no_other(T):
    """An infinite input block gives NaN gates (inf - inf); the tokens beside it do not change."""
    E, H, I, k = 2, 128, 96, 2
    x, gu, dn, ids, weights = make(T, E, H, I, k, 6)
    y = run(x, gu, dn, ids, weights)
    x[0, 40] = float("inf")
    z = run(x, gu, dn, ids, weights)
    assert not torch.isfinite(z[0]).any()
    assert torch.equal(z[1:], y[1:])


@pytest.mark.parametrize("T", [1, 2, 12, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k0", [0, 45, 287])
def test_nan_in_x_reaches_its_token_and_no_other(T, dtype, k0):
    """With the caller's ids and weights: the row is NaN whichever element of whichever block is, the
    others keep every bit, and a token without an expert stays zero."""
    E, H, I, k = 2, 288, 96, 2
    x, gu, dn, ids, weights = make(T, E, H, I, k, 7, dtype)
    y = run(x, gu, dn, ids, weights)
    for t in {0, T - 1}:
        bad = x.clone()
        bad[t, k0] = float("nan")
        z = run(bad, gu, dn, ids, weights)
        rest = [i for i in range(T) if i != t]
        assert torch.isnan(z[t]).all() and torch.equal(z[rest], y[rest])
        none = ids.clone()
        none[t] = -1
        assert torch.equal(run(bad, gu, dn, none, weights)[t], torch.zeros(H, device="cuda"))


def test_a_token_does_not_depend_on_the_others():
    """Each token alone gives what it gives in the batch (up to the order of its sums); other
    values in the neighbours' rows, NaN among them, do not change a bit."""
    T, E, H, I, k = 20, 6, 256, 160, 2
    x, gu, dn, ids, weights = make(T, E, H, I, k, 8)
    y, yref, bound = verify(x, gu, dn, ids, weights, torch.float32, TOL)
    for t in (0, 7, 19):
        check(run(x[t:t + 1], gu, dn, ids[t:t + 1], weights[t:t + 1]), yref[t:t + 1], bound[t:t + 1])
    assert torch.equal(run(x, gu, dn, ids, weights), y)
    x[3] = float("nan")
    weights[5] = float("inf")
    z = run(x, gu, dn, ids, weights)
    keep = [t for t in range(T) if t not in (3, 5)]
    assert torch.equal(z[keep], y[keep]) and not torch.isfinite(z[5]).any()


def test_large_and_zero_gates():
    """silu at both ends: exp overflows to infinity (h = -0 * u) or underflows (h = g * u)."""
    T, E, H, I, k = 2, 1, 64, 32, 1
    x, gu, dn, ids, weights = make(T, E, H, I, k, 5)
    x = x * 1e4
    verify(x, gu, dn, ids, weights, torch.float32, TOL)
    x[1] = 0
    y, _, _ = verify(x, gu, dn, ids, weights, torch.float32, TOL)
    assert torch.all(y[1] == 0)


def dot_error(width):
    """What a dot may be off by, relative to the sum of its terms' magnitudes."""
    return max(TOL, (150 + width / 4096) * 2.0 ** -24)


def equal_terms(T, E, H, I, k, dg, du, dd, x, used):
    """(y / expected - 1) of the used tokens, where all weight codes are 7, all scales of a kind equal and
    every token's elements equal: all block terms of a dot are one number, so the roundings of a long
    sum add up instead of averaging out. Expected: from the definition in 64 bits."""
    f16 = lambda rows, K, v: torch.full((E, rows, K // 32), v, dtype=torch.float16, device="cuda")
    code = lambda rows, K: torch.full((E, rows, K // 2), 0xFF, dtype=torch.uint8, device="cuda")
    gd = f16(2 * I, H, dg)
    gd[:, I:] = du
    dg, du, dd = (float(torch.tensor(v, dtype=torch.float16)) for v in (dg, du, dd))
    ids = torch.full((T, k), -1, dtype=torch.int32)
    ids[:used] = torch.arange(k, dtype=torch.int32)
    xs = np.resize(np.asarray(x, dtype=np.float32), used)
    full = torch.zeros(T, H)
    full[:used] = torch.from_numpy(xs)[:, None]
    y = w4a8.moe_q4_0(full.cuda(), ids.cuda(), torch.ones(T, k, device="cuda"), code(2 * I, H), gd.view(torch.int16),
                      code(H, I), f16(H, I, dd).view(torch.int16))
    assert w4a8.w4a8_last_device_error() == 0 and torch.all(y[used:] == 0)
    xv = (xs / np.float32(127)).astype(np.float64) * 127  # amax / 127, every code 127
    g, u = 7 * dg * xv * H, 7 * du * xv * H
    want = k * 7 * dd * I * (g / (1 + np.exp(-g)) * u)
    return np.abs(y[:used].cpu().numpy().astype(np.float64) / want[:, None] - 1).max()


@pytest.mark.parametrize("T,E,H,I,k", [(1, 1, 1 << 18, 32, 1), (7, 1, 1 << 18, 32, 1), (64, 16, 1 << 17, 320, 16)])
@pytest.mark.parametrize("dg", [0.0011, 0.0007, 0.00053, 0.0019])
def test_long_sums_in_gate_and_up(T, E, H, I, k, dg):
    """g = u, so h errs by twice a dot's error (g / silu(g) * silu'(g) - 1 < 1e-7 for g >= 20). Besides: 32
    steps of 2^-24 for exp, division, products, the scale of h and down's sum of I / 32 <= 10 terms, and
    the weighted sum's 3 per slot."""
    worst = max(equal_terms(T, E, H, I, k, dg, dg, 0.0005, (20 + 1.7 * np.arange(7) + off) / (7 * dg * H), T)
                for off in (0.0, 0.61, 1.13))
    assert worst <= 2 * dot_error(H) + (32 + 3 * k) * 2.0 ** -24


@pytest.mark.parametrize("T,E,H,I,k,used", [(40, 1, 2432, 1 << 17, 1, 40), (33, 8, 2432, 1 << 16, 8, 1)])
def test_long_sums_in_down(T, E, H, I, k, used):
    """x = 127 * 2^-a and scales of g and u of one and of four bits: their sums are exact (multiples of
    one unit, below 2^24 of it: 889 * 15 * 76). So only the down product's sum errs beside the 32 steps above
    and the order in which a token's slots are added, I / 4096 + 2 steps per slot. A grid of one
    CTA per tile (H / 32 * ceil(T / 32) > 148), whose warps take the longest runs of boxes."""
    worst = 0.0
    for dd in (0.0011, 0.0007, 0.00053, 0.0019, 0.00131, 0.00087):
        for du in (1.25, 1.875):
            worst = max(worst, equal_terms(T, E, H, I, k, 2.0 ** -10, du * 2.0 ** -10, dd, 127 * 2.0 ** -np.array([6, 7]), used))
    assert worst <= dot_error(I) + (32 + k * (I / 4096 + 2)) * 2.0 ** -24


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("T,E,H,k", [(1, 1, 32, 1), (3, 8, 96, 2), (5, 11, 1504, 3), (64, 64, 2048, 8), (2, 256, 512, 16),
                                     (300, 7, 256, 7)])
@pytest.mark.parametrize("xd,wd", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                   (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, H, k, xd, wd, renorm):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(xd)
    wr = (torch.randn(E, H, generator=g) / H ** 0.5).to(wd)
    ids, p = w4a8.moe_route(x.cuda(), wr.cuda(), k, renorm)
    rid, rp, logits = ref.route(x.float().numpy(), wr.float().numpy(), k, renorm)
    # a logit errs by at most (H/8 + 8) * 2^-24 * sum |terms|; two that close may change places
    err = (H / 8 + 8) * 2.0 ** -24 * (np.abs(x.float().numpy()) @ np.abs(wr.float().numpy()).T).max(1)
    got = ids.cpu().numpy()
    chosen = np.take_along_axis(logits, got, 1)
    want = np.take_along_axis(logits, rid, 1)
    assert np.all(np.abs(chosen - want) <= 2 * err[:, None])
    assert all(len(set(r)) == k for r in got.tolist())
    same = np.all(got == rid, axis=1)
    assert same.mean() > 0.9
    # exp of a difference of logits and a sum of at most 256 of them
    assert np.all(np.abs(p.cpu().numpy() - rp)[same] <= rp[same] * (4 * err[same, None] + 300 * 2.0 ** -24))


def test_route_ties_and_special_logits():
    H, E = 64, 40
    wr = torch.zeros(E, H)
    x = torch.zeros(3, H)
    x[:, 0] = 1.0
    ids, p = w4a8.moe_route(x.cuda(), wr.cuda(), 4)  # all equal: the lowest indices
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 3 and torch.equal(p.cpu(), torch.full((3, 4), 0.25))
    wr[37, 0], wr[33, 0], wr[5, 0] = 2.0, 2.0, 1.0
    ids, _ = w4a8.moe_route(x.cuda(), wr.cuda(), 4)
    assert ids.cpu().tolist() == [[33, 37, 5, 0]] * 3
    wr[37, 0] = float("nan")
    wr[0, 0] = float("-inf")
    ids, p = w4a8.moe_route(x.cuda(), wr.cuda(), 16)
    assert ids[0].tolist()[:3] == [33, 5, 1] and 37 not in ids[0].tolist() and 0 not in ids[0].tolist()
    assert torch.isfinite(p).all()
    x[1] = float("nan")
    ids, p = w4a8.moe_route(x.cuda(), wr.cuda(), 4)
    assert ids[1].tolist() == [0, 1, 2, 3] and torch.isnan(p[1]).all() and torch.isfinite(p[0]).all()


# ------------------------------------------------------------------ the layer in one call
@pytest.mark.parametrize("T,E,H,I,k,renorm", [(1, 64, 512, 128, 8, True), (7, 9, 288, 96, 3, False),
                                              (64, 8, 256, 160, 2, True)])
def test_layer_is_route_and_experts(T, E, H, I, k, renorm):
    x, gu, dn, _, _ = make(T, E, H, I, k, 21, torch.bfloat16)
    wr = torch.randn(E, H, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ex = (gu[0], gu[1], dn[0], dn[1])
    y, ids, p = w4a8.moe_layer_q4_0(x.cuda(), wr, *ex, k, renorm=renorm, out_dtype=torch.bfloat16)
    i2, p2 = w4a8.moe_route(x.cuda(), wr, k, renorm)
    assert torch.equal(ids, i2) and torch.equal(p, p2)
    assert torch.equal(y, w4a8.moe_q4_0(x.cuda(), ids, p, *ex, out_dtype=torch.bfloat16))
    yref, bound = ref.experts(x.float().numpy(), ids.cpu().numpy(), p.cpu().numpy().astype(np.float64), gu[2], dn[2], TOL)
    check(y, yref, bound)


@pytest.mark.parametrize("T", [1, 33])
def test_a_decoder_blocks_matmuls(T):
    """An FP8 projection with its bias, then the routed layer on its output, and the
    projection's input gradient: the pieces as one program runs them, on one stream."""
    from tests import fp8_reference as f8
    H, E, I, k = 256, 8, 96, 2
    x, gu, dn, _, _ = make(T, E, H, I, k, 31)
    g = torch.Generator().manual_seed(2)
    wp, bias = torch.randn(H, H, generator=g) / 16, torch.randn(H, generator=g)
    q, s = w4a8.pack_fp8(wp.cuda())
    wr = torch.randn(E, H, generator=g).cuda()
    h = w4a8.gemm_fp8(x.cuda(), q, s, bias=bias.cuda())
    y, ids, p = w4a8.moe_layer_q4_0(h, wr, gu[0], gu[1], dn[0], dn[1], k)
    dx = w4a8.gemm_fp8_backward(y, q, s)
    wq, ws = f8.decode(q.view(torch.uint8).cpu().numpy()), s.cpu().numpy()
    href, Th = f8.gemm(x.numpy(), wq, ws, bias.numpy().astype(np.float64))
    assert np.all(np.abs(h.cpu().numpy() - href) <= TOL * Th)
    yref, bound = ref.experts(h.cpu().numpy(), ids.cpu().numpy(), p.cpu().numpy().astype(np.float64), gu[2], dn[2], TOL)
    check(y, yref, bound)
    dref, Td = f8.backward(y.cpu().numpy(), wq, ws)
    assert np.all(np.abs(dx.cpu().numpy() - dref) <= TOL * Td)


# ------------------------------------------------------------------ memory, streams, graphs
@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 512, 96, 2), (13, 11, 736, 352, 3), (64, 4, 256, 160, 2)])
def test_nothing_outside_the_outputs_is_written(T, E, H, I, k):
    x, gu, dn, ids, weights = make(T, E, H, I, k, 41)
    x, ids, weights = x.cuda(), ids.cuda(), weights.cuda()
    need = w4a8.w4a8_moe_workspace_bytes(T, E, H, I, k)
    outs = []
    for fill in (0x5A, 0xA5):
        buf = torch.full((1024 + T * H * 4,), fill, dtype=torch.uint8, device="cuda")
        ws = torch.full((1024 + need,), fill, dtype=torch.uint8, device="cuda")
        y = buf[512: 512 + T * H * 4].view(torch.float32).view(T, H)
        w4a8.w4a8_moe_q4_0(x, ids, weights, gu[0], gu[1], dn[0], dn[1], y, ws[512: 512 + need])
        torch.cuda.synchronize()
        for b, inner in ((buf, T * H * 4), (ws, need)):
            assert torch.all(b[:512] == fill) and torch.all(b[512 + inner:] == fill)
        outs.append(y.clone())
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T", [1, 24])
def test_side_streams_and_captured_graphs(T):
    E, H, I, k = 6, 512, 160, 2
    x, gu, dn, _, _ = make(T, E, H, I, k, 51)
    x, ex = x.cuda(), (gu[0], gu[1], dn[0], dn[1])
    wr = torch.randn(E, H, generator=torch.Generator().manual_seed(3)).cuda()
    y0, i0, p0 = w4a8.moe_layer_q4_0(x, wr, *ex, k)
    torch.cuda.synchronize()
    side, ws = [torch.cuda.Stream() for _ in range(2)], [w4a8.moe_workspace(T, E, H, I, k) for _ in range(2)]
    outs = []
    for i, st in enumerate(side):
        with torch.cuda.stream(st):
            outs += [w4a8.moe_layer_q4_0(x, wr, *ex, k, ws=ws[i]) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, y0) and torch.equal(i, i0) and torch.equal(p, p0) for y, i, p in outs)
    y, ids, p = torch.empty_like(y0), torch.empty_like(i0), torch.empty_like(p0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4a8.w4a8_moe_layer_q4_0(x, wr, *ex, k, ids, p, y, ws[0])
    for _ in range(3):
        y.zero_(), ids.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(ids, i0)
    x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(9)))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, w4a8.moe_layer_q4_0(x, wr, *ex, k)[0])
