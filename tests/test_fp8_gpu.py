"""The FP8 matmul on the GPU against its definition in 64 bits: codes and scales exact,
outputs within 1e-5 * sum |terms| (the accumulation in f32) plus, for a bf16 output, half a
step of the result (2^-8 relative, 2^-134 at the smallest)."""
import numpy as np
import pytest
import torch

import block_quantized_w4a8_b200 as w4a8
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu
TOL = 1e-5


def rand(shape, seed, dtype=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[0], 1, generator=g))
    return x.to(dtype)


def check(y, yref, T, what=""):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = TOL * T
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(yref) * 2.0 ** -8 + 2.0 ** -134
    err = np.abs(got - yref)
    assert got.shape == yref.shape
    assert np.all(err <= tol), f"{what}: {np.sum(err > tol)} of {err.size} outside, worst {np.max(err / np.maximum(T, 1e-300))}"


def weights(N, K, seed):
    w = rand((N, K), seed, spread=0.5)
    q, s = w4a8.pack_fp8(w.cuda())
    return q, s, ref.decode(q.view(torch.uint8).cpu().numpy()), s.cpu().numpy()


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 400), (130, 1936), (257, 4096)])
def test_codes_and_scales_are_exact(M, K, dtype):
    x = rand((M, K), M + K, dtype)
    q, s = w4a8.quant_act_fp8(x.cuda())
    rq, rs = ref.quant_rows(x.float().numpy())
    assert np.array_equal(q.float().cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    q, s = w4a8.pack_fp8(x.cuda())
    rq, rs = ref.pack(x.float().numpy())
    assert np.array_equal(q.float().cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_special_values_in_the_codes():
    x = torch.zeros(4, 256)
    x[0, 3] = float("nan")
    x[0, 4] = 2.0
    x[1, 130] = float("inf")
    x[1, 131] = 5.0
    x[2, 0] = 1e-44
    x[3, :] = torch.linspace(-3e38, 3e38, 256)
    for fn, r in ((w4a8.quant_act_fp8, ref.quant_rows), (w4a8.pack_fp8, ref.pack)):
        q, s = fn(x.cuda())
        rq, rs = r(x.numpy())
        assert np.array_equal(q.float().cpu().numpy(), rq, equal_nan=True)
        assert np.array_equal(s.cpu().numpy(), rs)


# ------------------------------------------------------------------ forward and gradient
SHAPES = [(1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 129, 144), (3, 200, 272), (8, 64, 4096), (16, 1000, 1040),
          (17, 257, 512), (33, 130, 400), (64, 640, 1936), (65, 384, 256), (127, 127, 112), (128, 1536, 384),
          (129, 256, 2048), (201, 1531, 1936), (256, 2048, 512), (300, 777, 4096), (1025, 520, 640),
          # whole grids of 256 x 256 tiles (CTA pairs) in both directions, ragged and even
          (1025, 2100, 2064), (2500, 1024, 1040), (2048, 1280, 1280), (513, 3333, 4000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm(M, N, K, dtype):
    q, s, wq, ws = weights(N, K, N + K)
    x = rand((M, K), M, dtype)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1)) if N % 2 else None
    y = w4a8.gemm_fp8(x.cuda(), q, s, bias=None if bias is None else bias.cuda(), out_dtype=dtype)
    yref, T = ref.gemm(x.float().numpy(), wq, ws, None if bias is None else bias.numpy().astype(np.float64))
    check(y, yref, T, f"{M}x{N}x{K}")
    assert w4a8.w4a8_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(M, N, K, dtype):
    q, s, wq, ws = weights(N, K, N + K + 1)
    dy = rand((M, N), M + 1, dtype)
    dx = w4a8.gemm_fp8_backward(dy.cuda(), q, s, out_dtype=dtype)
    dref, T = ref.backward(dy.float().numpy(), wq, ws)
    check(dx, dref, T, f"{M}x{N}x{K}")
    assert w4a8.w4a8_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(70, 18969, 144), (100, 19008, 272), (65, 19012, 128), (300, 9000, 400)])
@pytest.mark.parametrize("bias_dtype", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_outputs_with_a_bias(M, N, K, bias_dtype, dtype):
    """Wide outputs of few rows: rows of 16-byte units or not, ends inside a tile, each bias."""
    q, s, wq, ws = weights(N, K, N + K)
    x = rand((M, K), M, dtype)
    bias = None
    if bias_dtype is not None:
        bias = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(bias_dtype)
    y = w4a8.gemm_fp8(x.cuda(), q, s, bias=None if bias is None else bias.cuda(), out_dtype=dtype)
    yref, T = ref.gemm(x.float().numpy(), wq, ws, None if bias is None else bias.float().numpy().astype(np.float64))
    check(y, yref, T, f"{M}x{N}x{K}")
    assert w4a8.w4a8_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(1, 19001, 1024), (1, 32000, 2048), (3, 19072, 1040), (16, 19072, 1040), (20, 19001, 784),
                                   (40, 19072, 1040), (64, 20000, 400)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_outputs_of_few_tokens(M, N, K, dtype):
    """More than 148 column tiles for at most 64 tokens: one CTA walks all blocks of its tile and stores
    without a join, with a bias, in whole 16-byte rows or not; quantised inside or before."""
    q, s, wq, ws = weights(N, K, N + K)
    x = rand((M, K), M, dtype)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1))
    for b in (None, bias):
        y = w4a8.gemm_fp8(x.cuda(), q, s, bias=None if b is None else b.cuda(), out_dtype=dtype)
        yref, T = ref.gemm(x.float().numpy(), wq, ws, None if b is None else b.numpy().astype(np.float64))
        check(y, yref, T, f"{M}x{N}x{K}")
    assert w4a8.w4a8_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(1, 1000, 19008), (16, 1040, 19008), (33, 777, 20000)])
def test_wide_gradients_of_few_tokens(M, N, K):
    q, s, wq, ws = weights(N, K, N + K + 1)
    dy = rand((M, N), M + 1)
    dx = w4a8.gemm_fp8_backward(dy.cuda(), q, s)
    dref, T = ref.backward(dy.numpy(), wq, ws)
    check(dx, dref, T, f"{M}x{N}x{K}")
    assert w4a8.w4a8_last_device_error() == 0


def test_backward_agrees_with_differences_of_the_forward():
    """With x and dy on the e4m3 grid (scale 1 in every block, so neither call rounds its
    input), <dy, y(x + e) - y(x - e)> = <dx, 2e> up to the f32 sums of both calls."""
    M, N, K = 4, 256, 256
    q, s, _, _ = weights(N, K, 5)
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-7, 8, (M, K), generator=g).float() * 32
    dy = torch.randint(-7, 8, (M, N), generator=g).float() * 32
    x[:, ::128], dy[:, ::128] = 448.0, 448.0
    e = torch.zeros(M, K)
    e[:, 1::2] = 32.0  # steps of the grid: |x + e| <= 256, x + e is a code
    x = x.cuda()
    yp, ym = w4a8.gemm_fp8(x + e.cuda(), q, s).double(), w4a8.gemm_fp8(x - e.cuda(), q, s).double()
    dx = w4a8.gemm_fp8_backward(dy.cuda(), q, s).double().cpu()
    lhs = float((dy.double() * (yp - ym).cpu()).sum())
    rhs = float((dx * 2 * e.double()).sum())
    W = np.abs(ref.dequant(ref.decode(q.view(torch.uint8).cpu().numpy()), s.cpu().numpy()))
    size = np.abs(dy.numpy()) @ W  # sum |terms| of dx
    bound = 2 * TOL * float(np.sum(size * (2 * e.numpy() + 2 * (x.abs().cpu().numpy() + e.numpy()))))
    assert abs(lhs - rhs) <= bound
    assert bound < 0.05 * abs(rhs) + 0.05 * float(np.sum(size * 2 * e.numpy()))  # the bound says something


@pytest.mark.parametrize("M", [1, 40, 300, 5000])
def test_nan_and_infinity_reach_the_outputs_that_use_them_and_no_other(M):
    N, K = 300, 512
    q, s, _, _ = weights(N, K, 9)
    x = rand((M, K), 3)
    clean = w4a8.gemm_fp8(x.cuda(), q, s)
    x[0, 5] = float("nan")
    if M > 1:
        x[M - 1, 200] = float("inf")
    y = w4a8.gemm_fp8(x.cuda(), q, s)
    assert torch.isnan(y[0]).all()
    if M > 1:
        assert not torch.isfinite(y[M - 1]).any()
    if M > 2:
        assert torch.equal(y[1:M - 1], clean[1:M - 1])


@pytest.mark.parametrize("M", [1, 20, 200])
def test_zero_rows_give_zero(M):
    N, K = 130, 272
    q, s, _, _ = weights(N, K, 11)
    x = rand((M, K), 4)
    x[M // 2] = 0
    y = w4a8.gemm_fp8(x.cuda(), q, s, out_dtype=torch.bfloat16)
    assert torch.equal(y[M // 2], torch.zeros_like(y[M // 2]))


@pytest.mark.parametrize("M,N,K", [(1, 130, 16384), (20, 130, 16384), (300, 130, 16384), (2600, 1030, 16384)])
def test_long_sums_of_one_sign(M, N, K):
    """All terms positive, so |y| = sum |terms|: the worst case for a long chain of f32 sums, held
    to 1e-5 at the longest axis the header promises it for (128 blocks)."""
    g = torch.Generator().manual_seed(K)
    q, s = w4a8.pack_fp8(torch.rand(N, K, generator=g).cuda())
    x = torch.rand(M, K, generator=g).cuda()
    y = w4a8.gemm_fp8(x, q, s).double()
    qx, sx = w4a8.quant_act_fp8(x)
    w = q.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    want = (qx.double() * sx.double().repeat_interleave(128, 1)) @ w.T
    assert float(((y - want).abs() / want).max()) <= TOL
    if M > 16:  # the gradient contracts M x N: the same weights turned round
        q2, s2 = w4a8.pack_fp8(torch.rand(K, 144, generator=g).cuda())
        dx = w4a8.gemm_fp8_backward(x, q2, s2).double()
        w2 = q2.double() * s2.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :144]
        want = (qx.double() * sx.double().repeat_interleave(128, 1)) @ w2
        assert float(((dx - want).abs() / want).max()) <= TOL


@pytest.mark.parametrize("M,N,K", [(1, 130, 512), (20, 257, 2048), (300, 384, 400), (2600, 1030, 272)])
@pytest.mark.parametrize("size", [1e-31, 1e-34, 1e-36, 1e-38])
def test_scales_whose_product_is_subnormal(M, N, K, size):
    """Rows so small that a block's two scales multiply to less than 2^-126: the product is off by up
    to 2^-150, times the codes' products, and so is each block's f32 sum."""
    w = rand((N, K), 7, spread=0.5) * 0.01
    q, s = w4a8.pack_fp8(w.cuda())
    wq, ws = ref.decode(q.view(torch.uint8).cpu().numpy()), s.cpu().numpy()
    x, dy = rand((M, K), M) * size, rand((M, N), M + 1) * size
    for inp, call, plain, side in ((x, w4a8.gemm_fp8, ref.gemm, np.abs(wq).T), (dy, w4a8.gemm_fp8_backward, ref.backward, np.abs(wq))):
        y = call(inp.cuda(), q, s).cpu().numpy().astype(np.float64)
        yref, T = plain(inp.numpy(), wq, ws)
        codes = np.abs(ref.quant_rows(inp.numpy())[0]) @ side
        blocks = -(-inp.shape[1] // 128)
        assert np.all(np.abs(y - yref) <= TOL * T + 2.0 ** -150 * (codes + blocks + 1))


# ------------------------------------------------------------------ memory, streams, graphs
@pytest.mark.parametrize("M,N,K", [(1, 1000, 1040), (16, 129, 144), (70, 333, 400), (201, 1531, 1936),
                                   (1100, 2090, 2064)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing_outside_the_outputs_is_written(M, N, K, dtype):
    """Outputs and workspace sit between guard words, and every byte of the output is written."""
    q, s, _, _ = weights(N, K, 13)
    x, dy = rand((M, K), 1, dtype).cuda(), rand((M, N), 2, dtype).cuda()
    need = w4a8.w4a8_fp8_workspace_bytes(M, N, K)
    size = torch.empty(0, dtype=dtype).element_size()
    for n, call in ((M * N, lambda o, w: w4a8.w4a8_gemm_fp8(x, q, s, o.view(M, N), w)),
                    (M * K, lambda o, w: w4a8.w4a8_gemm_fp8_backward(dy, q, s, o.view(M, K), w))):
        outs = []
        for fill in (0x5A, 0xA5):
            buf = torch.full((512 + n * size + 512,), fill, dtype=torch.uint8, device="cuda")
            ws = torch.full((512 + need + 512,), fill, dtype=torch.uint8, device="cuda")
            call(buf[512: 512 + n * size].view(dtype), ws[512: 512 + need])
            torch.cuda.synchronize()
            for b, inner in ((buf, n * size), (ws, need)):
                assert torch.all(b[:512] == fill) and torch.all(b[512 + inner:] == fill)
            outs.append(buf[512: 512 + n * size].clone())
        assert torch.equal(outs[0], outs[1])  # also: the result does not depend on the workspace's contents


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (48, 512, 1024), (300, 512, 1024), (2560, 1024, 1024)])
def test_side_streams_and_captured_graphs(M, N, K):
    q, s, _, _ = weights(N, K, 17)
    x, dy = rand((M, K), 1).cuda(), rand((M, N), 2).cuda()
    y0, d0 = w4a8.gemm_fp8(x, q, s), w4a8.gemm_fp8_backward(dy, q, s)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    ws = [w4a8.fp8_workspace(M, N, K) for _ in side]
    out = []
    for i, st in enumerate(side):  # two calls at once, each with a workspace of its own
        with torch.cuda.stream(st):
            out.append((w4a8.gemm_fp8(x, q, s, ws=ws[i]), w4a8.gemm_fp8_backward(dy, q, s, ws=ws[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, y0) and torch.equal(b, d0) for a, b in out)
    y, dx = torch.empty_like(y0), torch.empty_like(d0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4a8.w4a8_gemm_fp8(x, q, s, y, ws[0])
        w4a8.w4a8_gemm_fp8_backward(dy, q, s, dx, ws[0])
    for _ in range(3):
        y.zero_(), dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(dx, d0)
    x.copy_(rand((M, K), 7))  # the graph reads the new contents
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, w4a8.gemm_fp8(x, q, s))


def test_beside_the_other_tensor_core_kernels():
    """Few-token tiles and CTA pairs in FP8 next to the int8 and fp16 kernels on four streams, all of which
    share the SMs' tensor memory: each gives what it gives alone."""
    N, K = 1024, 2048
    q, s, _, _ = weights(N, K, 27)
    qs, d = w4a8.pack_q4_0(rand((N, K), 28).cuda())
    jobs = [lambda x=rand((M, K), M).cuda(): w4a8.gemm_fp8(x, q, s) for M in (1, 64, 200, 2500)]
    jobs += [lambda x=rand((M, K), M + 1).cuda(): w4a8.gemm(x, qs, d) for M in (16, 64, 300)]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(40):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(((i + 2 * j) % len(jobs), jobs[(i + 2 * j) % len(jobs)]()))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k, y in got)
    assert w4a8.w4a8_last_device_error() == 0


def test_helpers_on_a_stream_argument_keep_their_memory():
    """Outputs and workspace of a call on another stream are not handed out again while it waits
    there: the current stream allocates and fills memory of the same sizes meanwhile."""
    M, N, K = 40, 384, 512
    q, s, _, _ = weights(N, K, 17)
    x, dy = rand((M, K), 18).cuda(), rand((M, N), 19).cuda()
    E, H, I, k = 4, 512, 96, 2
    gu, dn, wr = rand((E * 2 * I, H), 20).cuda(), rand((E * H, I), 21).cuda(), rand((E, H), 22).cuda()
    gq, gd = (t.view(E, 2 * I, -1) for t in w4a8.pack_q4_0(gu))
    dq, dd = (t.view(E, H, -1) for t in w4a8.pack_q4_0(dn))
    ids, p = w4a8.moe_route(x, wr, k)

    def calls(stream):
        yield from w4a8.quant_act_fp8(x, stream=stream)
        yield from w4a8.pack_fp8(x, stream=stream)
        yield w4a8.gemm_fp8(x, q, s, stream=stream)
        yield w4a8.gemm_fp8_backward(dy, q, s, stream=stream)
        yield from w4a8.moe_route(x, wr, k, stream=stream)
        yield w4a8.moe_q4_0(x, ids, p, gq, gd, dq, dd, stream=stream)
        yield from w4a8.moe_layer_q4_0(x, wr, gq, gd, dq, dd, k, stream=stream)

    want = list(calls(None))
    sizes = {t.nbytes for t in want} | {w4a8.w4a8_fp8_workspace_bytes(M, N, K),
                                        w4a8.w4a8_moe_workspace_bytes(M, E, H, I, k)}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got, junk = [], []
    for t in calls(side):
        got.append(t)
        junk += [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("K", [128, 16384])
def test_a_quantised_row_is_a_weight_of_one_row(K):
    """The codes and scales of one activation row are those of a 1 x K weight, and a call that
    reads them as its weight directly afterwards sees them complete."""
    x, rows = rand((1, K), 23).cuda(), rand((8, K), 24).cuda()
    want = [w4a8.gemm_fp8(x, *w4a8.pack_fp8(r[None])) for r in rows]
    q, s = torch.zeros(1, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(1, K // 128, device="cuda")
    y, ws = [torch.empty(1, 1, device="cuda") for _ in range(8)], w4a8.fp8_workspace(1, 1, K)
    torch.cuda.synchronize()
    for i in range(8):
        w4a8.w4a8_quant_act_fp8(rows[i][None], q, s)
        w4a8.w4a8_gemm_fp8(x, q, s, y[i], ws)
    torch.cuda.synchronize()
    assert all(torch.equal(y[i], want[i]) for i in range(8))
