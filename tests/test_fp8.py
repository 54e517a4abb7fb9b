"""Host side of the FP8 matmul (no GPU): the reference the GPU tests use, refusals with the
documented status codes, workspace sizes, and the binding's checks."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_w4a8_b200 as w4a8
from tests import fp8_reference as ref
from tests.test_binding import fake  # noqa: F401  (the stand-in library)

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from block_quantized_w4a8_b200 import build
    build.build()
    return w4a8.load_library()


# ------------------------------------------------------------------ the reference
def test_reference_rounding_is_the_e4m3_grid():
    """Every f32 midpoint and neighbour between adjacent e4m3 values goes where torch's own
    conversion sends it, and decode inverts the codes."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.decode(codes.numpy()), vals, equal_nan=True)
    grid = np.sort(vals[np.isfinite(vals)])
    mid = (grid[1:] + grid[:-1]) / 2
    pts = np.concatenate([grid, mid, np.nextafter(mid, np.float32(1e9)), np.nextafter(mid, np.float32(-1e9))])
    pts = pts.astype(np.float32)
    assert np.array_equal(ref.e4m3_value(pts), torch.from_numpy(pts).to(torch.float8_e4m3fn).float().numpy())


def test_reference_scales_of_empty_and_tiny_blocks():
    x = np.zeros((2, 256), dtype=np.float32)
    x[1, 130] = 1e-44  # below the floor of the scale: finite reciprocal, code 0
    q, s = ref.quant_rows(x)
    assert np.all(q == 0) and np.all(s == np.float32(2.0 ** -126))
    x[0, 0] = 448.0
    q, s = ref.quant_rows(x)
    assert s[0, 0] == 1.0 and q[0, 0] == 448.0


def test_reference_backward_is_the_derivative():
    """dx is the gradient of sum(dy * (v W^T)) with respect to v when dy is on the e4m3 grid:
    central differences of the (linear) forward agree to rounding of the differences."""
    rng = np.random.default_rng(0)
    wq, ws = ref.pack(rng.standard_normal((40, 32)).astype(np.float32))
    W = ref.dequant(wq, ws)
    dy = rng.integers(-7, 8, (3, 40)).astype(np.float32) * 32.0  # multiples of 32 below 256 are e4m3 values
    dy[:, 0] = 448.0  # amax 448: scale 1
    assert np.array_equal(ref.quant_rows(dy)[0], dy)
    v = rng.standard_normal((3, 32))
    dx, _ = ref.backward(dy, wq, ws)
    for m, k in [(0, 0), (1, 17), (2, 31)]:
        e = np.zeros_like(v)
        e[m, k] = 0.5
        diff = np.sum(dy * ((v + e) @ W.T)) - np.sum(dy * ((v - e) @ W.T))
        assert abs(diff - dx[m, k]) <= 1e-12 * np.sum(np.abs(dy) @ np.abs(W))


# ------------------------------------------------------------------ the C ABI's refusals
def _gemm(lib, M=8, N=8, K=128, x=FAKE, dt=0, q=FAKE, s=FAKE, epi=None, y=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.w4a8_gemm_fp8(M, N, K, P(x), dt, P(q), P(s), epi, P(y), P(ws), wsb, P(0))


def _back(lib, M=8, N=8, K=128, dy=FAKE, dt=0, q=FAKE, s=FAKE, odt=0, dx=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.w4a8_gemm_fp8_backward(M, N, K, P(dy), dt, P(q), P(s), odt, P(dx), P(ws), wsb, P(0))


@pytest.mark.parametrize("call,first", [(_gemm, "x"), (_back, "dy")])
def test_gemm_argument_errors(lib, call, first):
    assert call(lib, M=0) == 1 and call(lib, N=-1) == 1 and call(lib, K=0) == 1
    assert call(lib, K=24) == 1 and call(lib, M=(1 << 20) + 1) == 1
    assert call(lib, q=0) == 1 and call(lib, s=0) == 1 and call(lib, **{first: 0}) == 1
    assert call(lib, dt=5) == 2
    assert call(lib, q=FAKE + 8) == 6 and call(lib, **{first: FAKE + 4}) == 6 and call(lib, ws=FAKE + 8) == 6
    assert call(lib, ws=0) == 3 and call(lib, wsb=16) == 3


def test_gemm_output_errors(lib):
    assert _gemm(lib, y=0) == 1 and _gemm(lib, y=FAKE + 2) == 6
    assert _back(lib, dx=0) == 1 and _back(lib, dx=FAKE + 2) == 6 and _back(lib, odt=3) == 2
    e = w4a8.Epilogue(None, 0, 9)
    assert _gemm(lib, epi=ctypes.byref(e)) == 2
    e = w4a8.Epilogue(FAKE + 1, 0, 0)
    assert _gemm(lib, epi=ctypes.byref(e)) == 6


def test_quant_argument_errors(lib):
    for f in (lib.w4a8_quant_act_fp8, lib.w4a8_pack_fp8):
        assert f(P(FAKE), 0, 0, 128, P(FAKE), P(FAKE), P(0)) == 1
        assert f(P(FAKE), 0, 4, 40, P(FAKE), P(FAKE), P(0)) == 1
        assert f(P(FAKE), 0, 4, 128, P(FAKE), P(0), P(0)) == 1
        assert f(P(FAKE), 2, 4, 128, P(FAKE), P(FAKE), P(0)) == 2
        assert f(P(FAKE + 2), 0, 4, 128, P(FAKE), P(FAKE), P(0)) == 6


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 4096, 4096), (201, 1531, 1936), (4096, 14336, 4096)])
def test_workspace_holds_the_quantised_operand(lib, M, N, K):
    """Codes of either operand plus one f32 scale per row and 128 columns, at least."""
    n = w4a8.w4a8_fp8_workspace_bytes(M, N, K)
    for R in (N, K):
        assert n >= M * R + 4 * M * -(-R // 128)
    assert n % 16 == 0


@pytest.mark.parametrize("shape", [(0, 8, 128), (8, 0, 128), (8, 8, 8), (8, 8, 130), (8, 8, 1 << 21)])
def test_workspace_rejects(lib, shape):
    assert w4a8.w4a8_fp8_workspace_bytes(*shape) == 0
    with pytest.raises(w4a8.W4A8Error):
        w4a8.fp8_workspace(*shape, device="cpu")


# ------------------------------------------------------------------ the binding
def _tensors():
    M, N, K = 3, 200, 272
    e4 = torch.float8_e4m3fn
    w = dict(q=torch.zeros(N, K, dtype=torch.uint8).view(e4), s=torch.zeros(2, 3))
    ws = torch.zeros(4096, dtype=torch.uint8)
    return [
        ("w4a8_quant_act_fp8", w4a8.w4a8_quant_act_fp8,
         dict(x=torch.zeros(M, K), q=torch.zeros(M, K, dtype=torch.uint8), s=torch.zeros(M, 3)), {"x"}),
        ("w4a8_pack_fp8", w4a8.w4a8_pack_fp8, dict(w=torch.zeros(N, K), **w), {"w"}),
        ("w4a8_gemm_fp8", w4a8.w4a8_gemm_fp8,
         dict(x=torch.zeros(M, K), **w, y=torch.zeros(M, N, dtype=torch.bfloat16), ws=ws, bias=torch.zeros(N)),
         {"x", "ws"}),
        ("w4a8_gemm_fp8_backward", w4a8.w4a8_gemm_fp8_backward,
         dict(dy=torch.zeros(M, N), **w, dx=torch.zeros(M, K), ws=ws), {"dy", "ws"}),
    ]


@pytest.mark.parametrize("case", _tensors(), ids=lambda c: c[0])
def test_binding_passes_exact_sizes_and_refuses_short_tensors(fake, case):  # noqa: F811
    name, fn, tensors, free = case
    fn(**tensors)
    assert [c[0] for c in fake.calls] == [name]
    ptrs = {a.value for a in fake.calls[0][1] if isinstance(a, ctypes.c_void_p)}
    assert {v.data_ptr() for k, v in tensors.items() if k != "bias"} <= ptrs
    fake.calls.clear()
    for key, v in tensors.items():
        if key in free:
            continue
        cut = v.view(torch.uint8)[:, :-1].contiguous().view(v.dtype) if v.element_size() == 1 else v.flatten()[:-1]
        if v.dim() == 2:
            cut = v[:-1].contiguous()  # one row short
            if (key, name) == ("q", "w4a8_gemm_fp8"):
                continue  # q's rows set N
        with pytest.raises(ValueError, match=rf"libw4a8: {key} holds"):
            fn(**{**tensors, key: cut})
    assert fake.calls == []


def test_binding_refuses_other_element_types(fake):  # noqa: F811
    _, fn, tensors, _ = _tensors()[2]
    for key, bad in [("q", tensors["q"].float()), ("s", tensors["s"].double())]:
        with pytest.raises(ValueError, match=f"libw4a8: {key} is"):
            fn(**{**tensors, key: bad})
    with pytest.raises(ValueError, match="contiguous"):
        fn(**{**tensors, "x": torch.zeros(272, 3).T})
    assert fake.calls == []


@pytest.mark.parametrize("which", [2, 3])
def test_binding_refuses_codes_of_another_width(fake, which):  # noqa: F811
    name, fn, tensors, _ = _tensors()[which]
    q = tensors["q"]
    tensors["q"] = torch.zeros(q.shape[0], q.shape[1] + 16, dtype=q.dtype)
    with pytest.raises(ValueError, match="rows of"):
        fn(**tensors)
    assert not fake.calls


@pytest.mark.parametrize("which,key,shape", [
    (0, "q", (272, 3)), (0, "s", (1, 9)), (1, "q", (272, 200)), (1, "s", (3, 2)), (2, "s", (3, 2)), (2, "s", (3, 3)),
    (2, "y", (200, 3)), (2, "q", (200, 1, 272)), (3, "q", (201, 272)), (3, "q", (456, 272)), (3, "s", (3, 2))])
def test_binding_refuses_tensors_laid_out_otherwise(fake, which, key, shape):  # noqa: F811
    """The bytes are there, but in other rows; a gradient's weight of more rows than dy has columns is
    another layer's."""
    _, fn, tensors, _ = _tensors()[which]
    tensors[key] = torch.zeros(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn) if key == "q" else torch.zeros(*shape)
    with pytest.raises(ValueError, match=f"libw4a8: {key} "):
        fn(**tensors)
    assert not fake.calls


def test_binding_takes_larger_and_flat_outputs_and_flat_scales(fake):  # noqa: F811
    _, fn, tensors, _ = _tensors()[2]
    fn(**{**tensors, "y": torch.zeros(64, 200), "s": torch.zeros(6)})
    fn(**{**tensors, "y": torch.zeros(600)})
    _, fn, tensors, _ = _tensors()[0]
    fn(**{**tensors, "q": torch.zeros(9, 272, dtype=torch.uint8), "s": torch.zeros(9, 3)})
    assert len(fake.calls) == 3
