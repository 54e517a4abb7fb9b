"""Host side of the mixture-of-experts layer (no GPU): the reference the GPU tests use,
refusals with the documented status codes, workspace sizes, and the binding's checks."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_w4a8_b200 as w4a8
import oracle
from tests import moe_reference as ref
from tests.test_binding import fake  # noqa: F401  (the stand-in library)

FAKE = 0x10000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from block_quantized_w4a8_b200 import build
    build.build()
    return w4a8.load_library()


# ------------------------------------------------------------------ the reference
def test_reference_codes_are_the_oracles():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((5, 96)).astype(np.float32)
    qs, d = oracle.pack_q4_0(w)
    assert np.array_equal(ref.dequant_q4_0(qs, d), oracle.dequant_q4_0(qs, d))
    q, dx, _ = oracle.quant_act_q8_0(w)
    codes, scales = ref.q8_0(w)
    assert np.array_equal(codes.reshape(5, 96), q) and np.array_equal(scales, dx)


def test_reference_route_breaks_ties_by_the_lower_index():
    x = np.ones((1, 32))
    wr = np.zeros((6, 32))
    wr[2], wr[4], wr[5] = 1, 1, 2
    ids, p, _ = ref.route(x, wr, 4, True)
    assert ids.tolist() == [[5, 2, 4, 0]] and abs(p.sum() - 1) < 1e-15


def test_reference_layer_is_the_plain_formula_up_to_its_bound():
    """Against h kept in 64 bits: the difference is at most half a code step per element."""
    rng = np.random.default_rng(4)
    T, E, H, I = 3, 4, 64, 96
    x = rng.standard_normal((T, H)).astype(np.float32)
    gu, dn = rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    ids = np.array([[0, 3], [1, -1], [9, -5]])
    w = rng.random((T, 2))
    y, bound = ref.experts(x, ids, w, gu, dn, 0.0)
    xv = ref.values(*ref.q8_0(x))
    assert np.all(y[2] == 0)
    for t in range(2):
        want, slack = np.zeros(H), np.zeros(H)
        for s in range(2):
            if ids[t, s] < 0:
                continue
            a = gu[ids[t, s]] @ xv[t]
            h = a[:I] / (1 + np.exp(-a[:I])) * a[I:]
            step = np.repeat(np.abs(h).reshape(-1, 32).max(1) / 127, 32)
            want += w[t, s] * dn[ids[t, s]] @ h
            slack += w[t, s] * np.abs(dn[ids[t, s]]) @ (step / 2)
        assert np.all(np.abs(y[t] - want) <= slack * (1 + 1e-6) + bound[t])
    assert np.all(bound < 1e-3 * np.abs(y).max() + 1e-9)  # with exact dots almost nothing may flip


# ------------------------------------------------------------------ copies in flight
RING_SIM = """
#include <cstdio>
#include <set>
#include "ring_count.cuh"
using w4a8::moe::RingCount;
// A warp's loop over n boxes, as the expert kernels run it: two requests ahead, then wait,
// read, count, request. The wait for box `lost` runs out (lost = n: none does).
int main() {
    for (int n = 0; n < 12; ++n)
        for (int lost = 0; lost <= n; ++lost) {
            RingCount r;
            r.reset();
            std::set<int> flight;
            auto fetch = [&] {
                if (r.issued == n || r.dead) return;
                for (int f : flight)
                    if (RingCount::stage(f) == RingCount::stage(r.issued)) return (void)std::printf("overrun\\n");
                flight.insert(r.issued++);
            };
            fetch();
            fetch();
            for (int box = 0; box < n; ++box) {
                if (box == lost) r.dead = true;
                if (!r.dead) flight.erase(r.used);
                ++r.used;
                fetch();
            }
            for (int i = r.first_pending(); i < r.issued; ++i) flight.erase(i);  // the drain
            if (!flight.empty()) std::printf("n %d lost %d: %zu in flight at the end\\n", n, lost, flight.size());
        }
}
"""


def test_no_copy_is_left_in_flight_after_a_wait_that_ran_out(tmp_path):
    """A block that ends while a copy into its shared memory is in flight may overwrite its
    successor's: whatever the box whose wait runs out, the drain covers what was requested."""
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(RING_SIM)
    csrc = os.path.join(os.path.dirname(w4a8.__file__), "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-x", "c++", "-I", csrc, str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True) == ""


# ------------------------------------------------------------------ the C ABI's refusals
def _route(lib, T=4, E=8, H=64, k=2, x=FAKE, dt=0, wr=FAKE, wdt=0, ids=FAKE, w=FAKE):
    return lib.w4a8_moe_route(T, E, H, k, 1, P(x), dt, P(wr), wdt, P(ids), P(w), P(0))


def _moe(lib, T=4, E=8, H=64, I=96, k=2, x=FAKE, dt=0, ids=FAKE, w=FAKE, gq=FAKE, gd=FAKE, dq=FAKE, dd=FAKE, odt=0,
         y=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.w4a8_moe_q4_0(T, E, H, I, k, P(x), dt, P(ids), P(w), P(gq), P(gd), P(dq), P(dd), odt, P(y), P(ws), wsb,
                             P(0))


def _layer(lib, T=4, E=8, H=64, I=96, k=2, x=FAKE, dt=0, wr=FAKE, wdt=0, ids=FAKE, w=FAKE, gq=FAKE, gd=FAKE, dq=FAKE,
           dd=FAKE, odt=0, y=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.w4a8_moe_layer_q4_0(T, E, H, I, k, 1, P(x), dt, P(wr), wdt, P(gq), P(gd), P(dq), P(dd), P(ids), P(w),
                                   odt, P(y), P(ws), wsb, P(0))


@pytest.mark.parametrize("call", [_route, _moe, _layer])
def test_argument_errors(lib, call):
    assert call(lib, T=0) == 1 and call(lib, E=0) == 1 and call(lib, k=0) == 1 and call(lib, H=-32) == 1
    assert call(lib, H=48) == 1 and call(lib, H=1 << 21) == 1
    assert call(lib, x=0) == 1 and call(lib, ids=0) == 1 and call(lib, w=0) == 1
    assert call(lib, dt=7) == 2 and call(lib, E=257) == 2 and call(lib, k=9) == 2 and call(lib, E=64, k=17) == 2
    assert call(lib, x=FAKE + 4) == 6 and call(lib, ids=FAKE + 4) == 6 and call(lib, w=FAKE + 8) == 6


@pytest.mark.parametrize("call", [_moe, _layer])
def test_expert_argument_errors(lib, call):
    assert call(lib, I=40) == 1 and call(lib, I=0) == 1
    assert call(lib, T=65) == 2 and call(lib, odt=5) == 2 and call(lib, I=(1 << 19) + 32) == 2
    for name in ("gq", "gd", "dq", "dd", "y"):
        assert call(lib, **{name: 0}) == 1 and call(lib, **{name: FAKE + 4}) == 6
    assert call(lib, ws=0) == 3 and call(lib, wsb=64) == 3 and call(lib, ws=FAKE + 4) == 6


def test_router_argument_errors(lib):
    for call in (_route, _layer):
        assert call(lib, wr=0) == 1 and call(lib, wr=FAKE + 4) == 6 and call(lib, wdt=9) == 2


@pytest.mark.parametrize("shape", [(0, 8, 64, 64, 2), (65, 8, 64, 64, 2), (1, 257, 64, 64, 2), (1, 8, 64, 64, 9),
                                   (1, 64, 64, 64, 17), (1, 8, 40, 64, 2), (1, 8, 64, 40, 2), (1, 8, 64, 64, 0)])
def test_workspace_rejects(lib, shape):
    assert w4a8.w4a8_moe_workspace_bytes(*shape) == 0
    with pytest.raises(w4a8.W4A8Error):
        w4a8.moe_workspace(*shape, device="cpu")


@pytest.mark.parametrize("T,E,H,I,k", [(1, 1, 32, 32, 1), (64, 64, 2048, 1024, 8), (4, 8, 4096, 14336, 2)])
def test_workspace_holds_the_activations(lib, T, E, H, I, k):
    """At least the Q8_0 form (codes and f32 scales) of x and of every slot's h."""
    assert w4a8.w4a8_moe_workspace_bytes(T, E, H, I, k) >= T * H * 9 // 8 + T * k * I * 9 // 8


# ------------------------------------------------------------------ the binding
def _tensors():
    T, E, H, I, k = 3, 4, 64, 96, 2
    u8, i16 = torch.uint8, torch.int16
    ex = dict(gu_qs=torch.zeros(E, 2 * I, H // 2, dtype=u8), gu_d=torch.zeros(E, 2 * I, H // 32, dtype=i16),
              dn_qs=torch.zeros(E, H, I // 2, dtype=u8), dn_d=torch.zeros(E, H, I // 32, dtype=i16))
    r = dict(ids=torch.zeros(T, k, dtype=torch.int32), weights=torch.zeros(T, k))
    x, wr, ws = torch.zeros(T, H), torch.zeros(E, H), torch.zeros(4096, dtype=u8)
    y = torch.zeros(T, H, dtype=torch.bfloat16)
    return [
        ("w4a8_moe_route", w4a8.w4a8_moe_route, dict(x=x, wr=wr, **r), {"top_k": k}, {"x", "wr"}),
        ("w4a8_moe_q4_0", w4a8.w4a8_moe_q4_0, dict(x=x, **r, **ex, y=y, ws=ws), {}, {"x", "ids", "gu_qs", "ws"}),
        ("w4a8_moe_layer_q4_0", w4a8.w4a8_moe_layer_q4_0, dict(x=x, wr=wr, **ex, **r, y=y, ws=ws), {"top_k": k},
         {"x", "gu_qs", "ws"}),
    ]


@pytest.mark.parametrize("case", _tensors(), ids=lambda c: c[0])
def test_binding_passes_exact_sizes_and_refuses_short_tensors(fake, case):  # noqa: F811
    name, fn, tensors, other, free = case
    fn(**tensors, **other)
    assert [c[0] for c in fake.calls] == [name]
    ptrs = {a.value for a in fake.calls[0][1] if isinstance(a, ctypes.c_void_p)}
    assert {v.data_ptr() for v in tensors.values()} <= ptrs
    fake.calls.clear()
    for key, v in tensors.items():
        if key not in free:
            with pytest.raises(ValueError, match=rf"libw4a8: {key} holds"):
                fn(**{**tensors, key: v[:-1].contiguous()}, **other)
    for key, bad in (("ids", tensors["ids"].long()), ("weights", tensors["weights"].double())):
        with pytest.raises(ValueError, match=f"libw4a8: {key} is"):
            fn(**{**tensors, key: bad}, **other)
    with pytest.raises(ValueError, match="contiguous"):
        fn(**{**tensors, "x": torch.zeros(64, 3).T}, **other)
    assert fake.calls == []


@pytest.mark.parametrize("change", [dict(gu_qs=(4, 193, 32)), dict(gu_qs=(4, 192, 48)), dict(dn_qs=(4, 65, 48)),
                                    dict(wr=(5, 64)), dict(wr=(4, 96))])
def test_binding_refuses_tensors_that_do_not_fit_together(fake, change):  # noqa: F811
    """Large enough, but of other rows, widths or experts than the call reads them with."""
    name, fn, tensors, other, _ = _tensors()[2]
    for key, shape in change.items():
        tensors[key] = torch.zeros(*shape, dtype=tensors[key].dtype)
    with pytest.raises(ValueError):
        fn(**tensors, **other)
    assert not fake.calls


@pytest.mark.parametrize("which,key,bad", [
    (0, "ids", torch.zeros(2, 3, dtype=torch.int32)), (0, "weights", torch.zeros(2, 3)),
    (1, "weights", torch.zeros(2, 3)), (1, "gu_qs", torch.zeros(4, 192, 32, dtype=torch.int32)),
    (1, "gu_d", torch.zeros(4, 2, 192, dtype=torch.int16)), (1, "gu_d", torch.zeros(4, 192, 2)),
    (1, "gu_d", torch.zeros(8, 192, 2, dtype=torch.int16)), (1, "dn_d", torch.zeros(4, 3, 64, dtype=torch.int16)),
    (1, "dn_d", torch.zeros(4, 64, 3)), (1, "dn_qs", torch.zeros(4, 64, 48, dtype=torch.int16)),
    (1, "y", torch.zeros(64, 3)), (2, "ids", torch.zeros(2, 3, dtype=torch.int32)), (2, "y", torch.zeros(64, 3))],
    ids=lambda v: str(tuple(v.shape)) if isinstance(v, torch.Tensor) else str(v))
def test_binding_refuses_tensors_laid_out_otherwise(fake, which, key, bad):  # noqa: F811
    """The bytes are there, but in other rows, as turned round, or of another element type."""
    _, fn, tensors, other, _ = _tensors()[which]
    with pytest.raises(ValueError, match=f"libw4a8: {key} "):
        fn(**{**tensors, key: bad}, **other)
    assert not fake.calls


def test_binding_takes_larger_and_flat_outputs(fake):  # noqa: F811
    _, fn, tensors, other, _ = _tensors()[2]
    fn(**{**tensors, "y": torch.zeros(9, 64), "ids": torch.zeros(9, 2, dtype=torch.int32), "weights": torch.zeros(6)}, **other)
    assert len(fake.calls) == 1
