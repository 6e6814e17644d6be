"""The few-token operators without a GPU: the float64 oracle's functions against hand-worked and
brute-force values, and every refusal of the C entry points and of the Python binding, which come
before any CUDA call."""
import numpy as np
import pytest
import torch

import blockwise_adaptive_transforms_b200 as W
from blockwise_adaptive_transforms_b200 import _build
from oracle import wush_oracle as O

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A = 0x10000          # a fake, never dereferenced, 16-byte aligned address
A4, A1 = A + 4, A + 1
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return W.load_library()


# ---------------------------------------------------------------- oracle pins

def test_gemv_by_hand():
    # one MXFP4 row: codes 1.0 and -6.0 in the first two places, scale 2^1; x = (3, 5, 0, ...)
    codes = np.zeros((1, 16), np.uint8)
    codes[0, 0] = 0x2 | (0xF << 4)
    x = np.zeros((1, 32))
    x[0, :2] = 3, 5
    assert O.gemv(x, None, codes, np.array([[128]]), None, 32, "mxfp4").tolist() == [[2 * (3 - 30)]]
    swap = np.eye(32)[[1, 0] + list(range(2, 32))]
    assert O.gemv(x, swap, codes, np.array([[128]]), None, 32, "mxfp4").tolist() == [[2 * (5 - 18)]]
    assert O.gemv(x, swap[None], codes, np.array([[128]]), None, 32, "mxfp4").tolist() == [[2 * (5 - 18)]]


def test_route_by_hand():
    x = np.array([[1.0, 0.0]])
    router = np.array([[0.0, 9.0], [np.log(2.0), 9.0], [0.0, -9.0], [np.log(5.0), 0.0]])
    ids, w = O.moe_route(x, router, 3, renormalise=False)
    assert ids.tolist() == [[3, 1, 0]]                      # the tie 0 / 2 goes to 0
    np.testing.assert_allclose(w, [[5 / 9, 2 / 9, 1 / 9]], rtol=1e-14)
    np.testing.assert_allclose(O.moe_route(x, router, 3)[1], [[5 / 8, 2 / 8, 1 / 8]], rtol=1e-14)


def test_experts_by_hand():
    # INT4, G = 16, width and hidden 16, expert 1: gate_0 = 2 x_0, up_0 = 3 x_1, out_5 = 4 h_0
    z = lambda r: (np.zeros((2, r, 8), np.uint8), np.ones((2, r, 1), np.float32), None)
    w_in, w_out = z(32), z(16)
    w_in[0][1, 0, 0] = 2
    w_in[0][1, 16, 0] = 3 << 4
    w_out[0][1, 5, 0] = 4
    x = np.zeros((1, 16))
    x[0, :2] = 0.5, 7
    g, u = 1.0, 21.0
    y = O.moe_experts(x, np.array([[-1, 1, 2]]), np.array([[np.nan, 0.25, np.nan]]), None, w_in, None, w_out, 16,
                      "int4")
    want = np.zeros(16)
    want[5] = 0.25 * 4 * g / (1 + np.exp(-g)) * u
    np.testing.assert_allclose(y[0], want, rtol=1e-14)


# ---------------------------------------------------------------- refusals of the C entry points

def gemv(lib, x=A, T=A, shared=0, codes=A, scales=A, ts=A, n=1, rows=64, d=64, G=32, fmt=0, y=A, f32=0, ws=A, wn=BIG):
    return lib.wush_gemv(x, T, shared, codes, scales, ts, n, rows, d, G, fmt, y, f32, ws, wn, None)


def test_gemv_refusals(lib):
    for name in ("x", "codes", "scales", "y", "ws"):
        assert gemv(lib, **{name: None}) == INVALID, name
    assert gemv(lib, fmt=1, G=16, ts=None) == INVALID
    for name in ("x", "T", "codes", "y", "ws"):
        assert gemv(lib, **{name: A4}) == MISALIGNED, name
    assert gemv(lib, fmt=2, scales=A1) == MISALIGNED
    assert gemv(lib, fmt=1, G=16, ts=A1) == MISALIGNED
    for bad in (dict(n=-1), dict(rows=0), dict(rows=-5), dict(rows=2 ** 31), dict(d=0), dict(d=48),
                dict(d=2 ** 20 + 32), dict(wn=W.wush_gemv_workspace_bytes(1, 64) - 1)):
        assert gemv(lib, **bad) == INVALID, bad
    for bad in (dict(n=65), dict(G=16), dict(G=64), dict(fmt=1), dict(fmt=3), dict(fmt=-1), dict(fmt=2, G=8)):
        assert gemv(lib, **bad) == UNSUPPORTED, bad
    assert gemv(lib, n=0, x=None, T=None, codes=None, scales=None, y=None, ws=None) == OK


def route(lib, x=A, r=A, f32=0, n=1, d=64, E=8, k=2, ids=A, w=A):
    return lib.wush_moe_route(x, r, f32, n, d, E, k, 1, ids, w, None)


def test_route_refusals(lib):
    for name in ("x", "r", "ids", "w"):
        assert route(lib, **{name: None}) == INVALID, name
    for bad in (dict(x=A4), dict(r=A4), dict(ids=A1), dict(w=A1)):
        assert route(lib, **bad) == MISALIGNED, bad
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(d=0), dict(d=63), dict(d=2 ** 20 + 8), dict(E=0), dict(k=0),
                dict(k=9), dict(k=-1)):
        assert route(lib, **bad) == INVALID, bad
    for bad in (dict(E=1025), dict(E=64, k=33)):
        assert route(lib, **bad) == UNSUPPORTED, bad
    assert route(lib, n=0, x=None, r=None, ids=None, w=None) == OK


def experts(lib, layer=False, x=A, ids=A, w=A, r=A, Ti=A, ic=A, isc=A, its=A, To=A, oc=A, osc=A, ots=A, n=1, d=64, f=64,
            E=8, k=2, G=32, fmt=0, y=A, ws=A, wn=BIG):
    tail = (Ti, 0, ic, isc, its, To, 0, oc, osc, ots, n, d, f, E, k, G, fmt, y, ws, wn, None)
    return lib.wush_moe_layer(x, r, 0, 1, ids, w, *tail) if layer else lib.wush_moe_experts(x, ids, w, *tail)


@pytest.mark.parametrize("layer", [False, True])
def test_experts_refusals(lib, layer):
    call = lambda **a: experts(lib, layer, **a)
    for name in ("x", "ids", "w", "ic", "isc", "oc", "osc", "y", "ws") + (("r",) if layer else ()):
        assert call(**{name: None}) == INVALID, name
    for name in ("its", "ots"):
        assert call(fmt=1, G=16, **{name: None}) == INVALID
        assert call(fmt=1, G=16, **{name: A1}) == MISALIGNED
    for name in ("x", "Ti", "ic", "To", "oc", "y", "ws") + (("r",) if layer else ()):
        assert call(**{name: A4}) == MISALIGNED, name
    for bad in (dict(ids=A1), dict(w=A1), dict(fmt=2, isc=A1), dict(fmt=2, osc=A1)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(n=-1), dict(d=0), dict(d=48), dict(f=0), dict(f=48), dict(E=0), dict(k=0), dict(d=2 ** 20 + 32),
                dict(f=2 ** 20 + 32), dict(wn=W.wush_moe_workspace_bytes(1, 64, 64, 2) - 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n=65), dict(E=1025), dict(E=64, k=33), dict(G=16), dict(fmt=1), dict(fmt=7)):
        assert call(**bad) == UNSUPPORTED, bad
    if layer:
        assert call(k=9) == INVALID                          # more slots than experts
    assert call(n=0, x=None, ids=None, w=None, r=None, ic=None, y=None, ws=None) == OK


def test_workspace_sizes(lib):
    assert W.wush_gemv_workspace_bytes(0, 32) >= 0
    assert W.wush_gemv_workspace_bytes(64, 4096) >= 64 * 4096 * 4
    for bad in ((-1, 64), (65, 64), (1, 0), (1, 2 ** 20 + 1)):
        assert W.wush_gemv_workspace_bytes(*bad) == -1
    assert W.wush_moe_workspace_bytes(1, 64, 64, 2) > 0
    for bad in ((-1, 64, 64, 1), (65, 64, 64, 1), (1, 0, 64, 1), (1, 64, 0, 1), (1, 64, 64, 0), (1, 64, 64, 33)):
        assert W.wush_moe_workspace_bytes(*bad) == -1


def test_packed_calls(lib):
    """The packed form takes the same arguments, in the same order."""
    import struct
    pack = lambda *a: struct.pack(f"{len(a)}q", *a)
    good = [A, A, 0, A, A, 0, 1, 64, 64, 32, 0, A, 0, A, BIG, 0]
    for place, value, want in ((0, 0, INVALID), (0, A4, MISALIGNED), (3, 0, INVALID), (6, 65, UNSUPPORTED),
                               (7, 0, INVALID), (8, 48, INVALID), (9, 16, UNSUPPORTED), (10, 3, UNSUPPORTED),
                               (11, A4, MISALIGNED), (13, 0, INVALID), (14, 1, INVALID), (6, 0, OK),
                               (9, 32 + 2 ** 32, INVALID)):
        words = list(good)
        words[place] = value
        assert lib.wush_call_packed(0, pack(*words)) == want, (place, value)
    assert lib.wush_call_packed(1, pack(A, A, 0, 1, 64, 8, 9, 1, A, A, 0)) == INVALID
    assert lib.wush_call_packed(1, pack(A, A, 0, 0, 64, 8, 2, 1, A, A, 0)) == OK
    experts = [A, A, A, A, 0, A, A, 0, A, 0, A, A, 0, 1, 64, 64, 8, 2, 32, 0, A, A, BIG, 0]
    assert lib.wush_call_packed(2, pack(*experts[:13], 65, *experts[14:])) == UNSUPPORTED
    assert lib.wush_call_packed(2, pack(*experts[:20], A4, *experts[21:])) == MISALIGNED
    layer = [A, A, 0, 1, A, A, A, 0, A, A, 0, A, 0, A, A, 0, 1, 64, 64, 8, 2, 32, 0, A, A, BIG, 0]
    assert lib.wush_call_packed(3, pack(*layer[:20], 9, *layer[21:])) == INVALID
    assert lib.wush_call_packed(3, pack(*layer[:16], 0, *layer[17:])) == OK
    assert lib.wush_call_packed(4, pack(*layer)) == UNSUPPORTED
    assert lib.wush_call_packed(0, None) == INVALID


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        W.wush_gemv(x, None, c, s, None, 32, "mxfp4")
    with pytest.raises(TypeError):
        W.wush_moe_route(x, x, 1)
    with pytest.raises(TypeError):
        W.wush_moe_experts(x, None, None, None, (c, s, None), None, (c, s, None), 32, "mxfp4")
    with pytest.raises(TypeError):
        W.wush_moe_layer(x, x, 1, None, (c, s, None), None, (c, s, None), 32, "mxfp4")


@pytest.mark.parametrize("layer", [False, True])
def test_sizes_beyond_the_counters_are_refused_before_any_launch(lib, layer):
    """Rows of a stack and steps of a product are checked with the other sizes, before the pointers (a null one here)
    and so before the router or the transform is launched; what fits a device is not refused for its steps."""
    top = 2 ** 20
    call = lambda **a: experts(lib, layer, x=None, **a)
    for bad in (dict(E=1024, f=top), dict(E=1024, k=1, d=top, f=top), dict(n=64, E=512, k=32, d=top, f=top),
                dict(n=64, E=64, k=32, d=top // 2, f=top)):
        assert call(**bad) == UNSUPPORTED, bad
    for good in (dict(n=64, E=32, k=32, d=2 ** 16, f=2 ** 16), dict(n=64, E=1023, k=32, f=top),
                 dict(n=64, E=1023, k=32, d=top), dict(n=1, E=1, k=1, d=top, f=2 ** 18)):
        assert call(**good) == INVALID, good                 # the pointer
    if not layer:                                            # 4 x 3 x 2^34 weights of 4 bits: 103 GB
        assert call(n=64, E=4, k=32, d=2 ** 17, f=2 ** 17) == INVALID
    for bad in (dict(rows=2 ** 30 - 1, d=top), dict(rows=2 ** 30 - 1, d=2 ** 15, n=64)):
        assert gemv(lib, x=None, **bad) == UNSUPPORTED, bad
    for good in (dict(rows=2 ** 30 - 1, d=512, n=64, f32=1), dict(rows=2 ** 18, d=top, n=64, f32=1)):
        assert gemv(lib, x=None, **good) == INVALID, good


def test_layer_checks_everything_before_the_router(lib):
    """With every pointer in place (the addresses are never read), a size that only the experts refuse."""
    assert experts(lib, True, E=1024, k=2, f=2 ** 20) == UNSUPPORTED
    assert experts(lib, False, E=1024, k=2, f=2 ** 20) == UNSUPPORTED


def test_the_overlap_of_launches_has_one_switch():
    """Wherever a launch asks to overlap with the one before it, the switch WUSH_USE_PDL decides."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(W.__file__), "csrc")
    found = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu")) + glob.glob(os.path.join(csrc, "*.cuh"))):
        text = open(path).read()
        for m in re.finditer(r"programmaticStreamSerializationAllowed", text):
            begin = max(0, text.rfind("\n}\n", 0, m.start()))     # the function around it
            body = text[begin:text.index("\n}\n", m.end())]
            assert "WUSH_USE_PDL" in body, (path, text.count("\n", 0, m.start()) + 1)
            found += 1
    assert found >= 5


def test_binding_does_without_torchs_inner_names(monkeypatch):
    """A torch without the inner calls that the binding prefers: the public ones take their place."""
    import types
    seen = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=100 + dev))
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, device=None, stream=None: seen.append((n, stream)) or 64)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda p: seen.append(p))
    handle, take, give_back = W._torch_calls(types.SimpleNamespace())
    assert handle(3) == 103 and take(512, 7) == 64
    give_back(64)
    assert seen == [(512, 7), 64]
    inner = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda dev: dev)
    assert W._torch_calls(inner)[0] is inner._cuda_getCurrentRawStream
