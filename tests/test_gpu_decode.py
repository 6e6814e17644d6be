"""The few-token operators on 4-bit weights against the float64 oracle (needs a B200).

Tolerances, from the arithmetic.  With S = |W| |T| |x| (sums of absolute values) and r the exact result:
  - the transform sums G products in fp32: G 2^-24 S;
  - for bf16 results the transformed activations may be held in fp16 under a power-of-two scale per
    group: half a step, 2^-11 S, plus the subnormal floor, under 2^-38 max|y| sum|w|; for fp32 results in
    two such terms: 2^-22 S;
  - the sums: tensor-core partial sums of up to 32 terms may truncate (2^-23 each), then at most
    K / 32 + 64 fp32 additions: (64 + K / 32) 2^-23 S;
  - the result is rounded once: 2^-8 |r| (bf16) or 2^-24 |r| (fp32)."""
import numpy as np
import pytest
import torch

import blockwise_adaptive_transforms_b200 as W
from oracle import wush_oracle as O

pytestmark = pytest.mark.gpu

FORMATS = [("mxfp4", 32), ("nvfp4", 16), ("int4", 16), ("int4", 32)]


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.float().numpy().astype(np.float64)


def ok():
    torch.cuda.synchronize()
    st, bits = W.wush_device_status()
    assert st == 0 and bits == 0, f"device error word {bits:#x}"


def make_matrix(rng, lead, K, G, fmt, wide=False):
    """Random codes (every nibble) and scales; ``wide``: scales over most of the format's range."""
    codes = rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)
    shape, ts = (*lead, K // G), None
    if fmt == "mxfp4":
        scales = rng.integers(20 if wide else 117, 210 if wide else 128, shape, dtype=np.uint8)
    elif fmt == "nvfp4":
        scales = rng.integers(0 if wide else 40, 0x7F, shape, dtype=np.uint8)
        ts = rng.uniform(0.001, 0.01, lead[:-1] if len(lead) > 1 else (1,)).astype(np.float32)
    else:
        scales = (np.exp(rng.normal(0, 20 if wide else 1, shape)) * 0.01).astype(np.float32)
    if fmt == "int4":     # the quantiser never writes -8
        for half in (0, 4):
            codes = np.where((codes >> half) & 15 == 8, codes & ~np.uint8(15 << half), codes)
    return codes, scales, ts


def make_T(rng, kind, K, G):
    if kind == "none":
        return None
    if kind == "shared":
        return rng.normal(0, G ** -0.5, (G, G)).astype(np.float32)
    return (np.eye(G) + 0.2 * rng.normal(0, 1, (K // G, G, G))).astype(np.float32)


def make_x(rng, n, K):
    x = rng.normal(0, 1, (n, K)) * np.exp(rng.normal(0, 1, K))
    x[:, rng.integers(0, K, max(1, K // 100))] *= 40
    return bf16(x)


def values(m, e, G, fmt):
    return O.dequant(O.unpack_nibbles(m[0][e]), m[1][e], fmt, G, None if m[2] is None else m[2][e])


def product_bound(x, T, w, G, f32):
    """(exact result, error before the last rounding) for values w [rows][K]."""
    K = x.shape[1]
    y = O.activations(x, T, G)
    S = O.activations(np.abs(x), None if T is None else np.abs(T), G)
    aw = np.abs(w)
    coef = (2.0 ** -22 if f32 else 2.0 ** -11) + (G + 64 + K / 32) * 2.0 ** -23
    floor = 2.0 ** -38 * np.abs(y).max(1, initial=0.0)[:, None] * aw.sum(1)
    return y @ w.T, coef * (S @ aw.T) + floor


def check_gemv(x, T, m, G, fmt, f32, got, x_exact=None):
    x = f64(x)
    w = O.dequant(O.unpack_nibbles(m[0]), m[1], fmt, G, None if m[2] is None else m[2][0])
    r, e = product_bound(x, T, w, G, f32)
    got = got.float().cpu().numpy().astype(np.float64)
    step = 2.0 ** -24 if f32 else 2.0 ** -8
    bad = np.abs(got - r) > e + step * (np.abs(r) + e) + 1e-37
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} {r[bad][0]}"


def run_gemv(x, T, m, G, fmt, f32, **kw):
    return W.wush_gemv(x.cuda(), dev(T), dev(m[0]), dev(m[1]), dev(m[2]), G, fmt,
                       out_dtype=torch.float32 if f32 else torch.bfloat16, **kw)


SIZES = [(1, 1, 1), (1, 37, 3), (2, 64, 4), (3, 129, 33), (4, 200, 8), (5, 40, 130), (7, 33, 65), (8, 257, 17),
         (9, 100, 7), (16, 65, 40), (17, 16, 5), (33, 70, 9), (64, 31, 6)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,rows,blocks", SIZES)
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv(fmt, G, n, rows, blocks, f32):
    rng = np.random.default_rng(n * 1000 + rows + blocks)
    K = G * blocks
    kind = ("block", "shared", "none")[(n + rows + blocks) % 3]
    x, T, m = make_x(rng, n, K), make_T(rng, kind, K, G), make_matrix(rng, (rows,), K, G, fmt)
    y = run_gemv(x, T, m, G, fmt, f32)
    ok()
    check_gemv(x, T, m, G, fmt, f32, y)


@pytest.mark.parametrize("kind", ["block", "shared", "none"])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_transforms(fmt, G, kind):
    rng = np.random.default_rng(7)
    x, T, m = make_x(rng, 3, 14 * G), make_T(rng, kind, 14 * G, G), make_matrix(rng, (50,), 14 * G, G, fmt)
    y = run_gemv(x, T, m, G, fmt, True)
    ok()
    check_gemv(x, T, m, G, fmt, True, y)


@pytest.mark.parametrize("n", [1, 6, 16])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_wide_scales(fmt, G, n):
    """Group scales over most of the format's range, and activations that differ by 2^60 between groups."""
    rng = np.random.default_rng(n)
    K = 40 * G
    x = rng.normal(0, 1, (n, K)) * np.repeat(np.exp2(rng.integers(-30, 30, (n, 40))), G, axis=1)
    x, m = bf16(x), make_matrix(rng, (45,), K, G, fmt, wide=True)
    for f32 in (False, True):
        y = run_gemv(x, None, m, G, fmt, f32)
        ok()
        check_gemv(x, None, m, G, fmt, f32, y)


@pytest.mark.parametrize("n", [1, 2, 5, 12])
def test_gemv_every_code_and_scale(n):
    """Row b holds byte b in one group and zero codes elsewhere: its result is that byte's two values."""
    for fmt, G in FORMATS:
        K = 8 * G
        codes = np.zeros((256, K // 2), np.uint8)
        for b in range(256):
            codes[b, (b * 7) % (K // 2)] = b
        rng = np.random.default_rng(3)
        _, scales, ts = make_matrix(rng, (256,), K, G, fmt)
        if fmt == "mxfp4":
            scales[:, :] = 127
        x = bf16(rng.integers(1, 9, (n, K)))
        if fmt == "int4":
            codes = np.where((codes & 15 == 8) | (codes >> 4 == 8), 0, codes).astype(np.uint8)
        y = run_gemv(x, None, (codes, scales, ts), G, fmt, True)
        ok()
        check_gemv(x, None, (codes, scales, ts), G, fmt, True, y)


@pytest.mark.parametrize("blocks", [8, 9, 64])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 12])
def test_gemv_nan_scales(n, blocks):
    """A scale byte that is a NaN (255 in E8M0, 0x7F in E4M3) makes its row NaN, and no other."""
    for fmt, G, byte in (("mxfp4", 32, 255), ("nvfp4", 16, 0x7F)):
        rng = np.random.default_rng(n + blocks)
        rows, C = 150, blocks
        m = make_matrix(rng, (rows,), C * G, G, fmt)
        hit = rng.choice(rows, 20, replace=False)
        m[1][hit, rng.integers(0, C, 20)] = byte
        m[1][hit[0], C - 1] = byte
        x = make_x(rng, n, C * G)
        for f32 in (False, True):
            got = run_gemv(x, None, m, G, fmt, f32).float().cpu().numpy()
            ok()
            want = np.zeros((n, rows), bool)
            want[:, hit] = True
            assert np.array_equal(np.isnan(got), want) and np.isfinite(got[~want]).all()


def test_gemv_scale_extremes():
    """E8M0 0 is 2^-127 (subnormal in fp32); E4M3's subnormals and its largest value."""
    codes = np.full((4, 16), 0x22, np.uint8)                       # all ones
    scales = np.array([[0], [1], [126], [253]], np.uint8)
    x = torch.zeros(1, 32, dtype=torch.bfloat16)
    x[0, 5] = 1.0
    y = run_gemv(x, None, (codes, scales, None), 32, "mxfp4", True)
    ok()
    assert y[0].tolist() == [2.0 ** -127, 2.0 ** -126, 0.5, 2.0 ** 126]
    scales = np.array([[1], [7], [8], [0x7E]], np.uint8)
    y = run_gemv(x[:, :16], None, (codes[:, :8], scales, np.array([1.0], np.float32)), 16, "nvfp4", True)
    ok()
    assert y[0].tolist() == [2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 448.0]


@pytest.mark.parametrize("n", [1, 3, 8, 16])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_small_and_zero_activations(fmt, G, n):
    """Zero groups, zero tokens, subnormal bf16 and bf16's largest finite values."""
    rng = np.random.default_rng(5)
    K = 12 * G
    x = make_x(rng, n, K)
    x[:, :3 * G] = 0
    x[:, 3 * G:4 * G] *= 1e-38
    x[:, 4 * G:5 * G] = 0
    x[0, 5 * G:] = 0
    m = make_matrix(rng, (40,), K, G, fmt)
    y = run_gemv(x, None, m, G, fmt, True)
    ok()
    check_gemv(x, None, m, G, fmt, True, y)
    assert torch.equal(run_gemv(torch.zeros_like(x), None, m, G, fmt, False).float(), torch.zeros(n, 40).cuda())
    top = torch.zeros(n, K, dtype=torch.bfloat16)
    top[:, 7] = torch.finfo(torch.bfloat16).max / 256
    y = run_gemv(top, None, m, G, fmt, True)
    ok()
    check_gemv(top, None, m, G, fmt, True, y)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_bad_values_stay_with_their_token(fmt, G, bad):
    rng = np.random.default_rng(8)
    K = 9 * G
    x, T, m = make_x(rng, 5, K), make_T(rng, "block", K, G), make_matrix(rng, (70,), K, G, fmt)
    clean = run_gemv(x, T, m, G, fmt, False)
    x[2, 2 * G + 3] = bad
    y = run_gemv(x, T, m, G, fmt, False)
    ok()
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], clean[keep])
    w = O.dequant(O.unpack_nibbles(m[0]), m[1], fmt, G, None if m[2] is None else m[2][0])
    touched = torch.from_numpy((w[:, 2 * G:3 * G] != 0).any(1)).cuda()
    assert not torch.isfinite(y[2][touched]).any()


@pytest.mark.parametrize("n", [1, 4, 8, 16])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_long_rows_and_exact_repeats(fmt, G, n):
    rng = np.random.default_rng(n)
    K = 14336 if G == 32 else 14320
    x, T, m = make_x(rng, n, K), make_T(rng, "block", K, G), make_matrix(rng, (75,), K, G, fmt)
    ys = [run_gemv(x, T, m, G, fmt, False) for _ in range(3)]
    ok()
    check_gemv(x, T, m, G, fmt, False, ys[0])
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_gemv_large_matrix_against_float64_on_device():
    """More rows than one wave of CTAs; 64-bit products on the device."""
    rng = np.random.default_rng(2)
    rows, K, G, n = 40001, 2080, 32, 6
    x, T, m = make_x(rng, n, K), make_T(rng, "block", K, G), make_matrix(rng, (rows,), K, G, "mxfp4")
    y = run_gemv(x, T, m, G, "mxfp4", False)
    ok()
    w = W.wush_dequant(dev(m[0]), dev(m[1]), None, G, "mxfp4").double()
    xt = torch.from_numpy(O.activations(f64(x), T, G)).cuda()
    ax = torch.from_numpy(O.activations(np.abs(f64(x)), np.abs(T), G)).cuda()
    r, S = xt @ w.T, ax @ w.abs().T
    e = (2.0 ** -11 + (G + 64 + K / 32) * 2.0 ** -23) * S + 2.0 ** -37 * S.max()
    assert bool(((y.double() - r).abs() <= e + 2.0 ** -8 * (r.abs() + e)).all())


@pytest.mark.parametrize("n", [1, 2, 3, 8, 13])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_writes_inside_its_buffers(fmt, G, n):
    rng = np.random.default_rng(1)
    rows, K = 45, 11 * G
    x, T, m = make_x(rng, n, K), make_T(rng, "block", K, G), make_matrix(rng, (rows,), K, G, fmt)
    for dt in (torch.bfloat16, torch.float32):
        big = torch.full((n + 8, rows), 7.0, dtype=dt, device="cuda")
        need = W.wush_gemv_workspace_bytes(n, K)
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")   # any bytes may be left in it
        y = W.wush_gemv(x.cuda(), dev(T), dev(m[0]), dev(m[1]), dev(m[2]), G, fmt, out_dtype=dt, out=big[:n],
                        workspace=ws[:need])
        ok()
        check_gemv(x, T, m, G, fmt, dt is torch.float32, y)
        assert bool((big[n:] == 7).all()) and bool((ws[need:] == 0xA5).all())


def test_gemv_empty_batch():
    m = make_matrix(np.random.default_rng(0), (8,), 64, 32, "mxfp4")
    y = run_gemv(torch.zeros(0, 64, dtype=torch.bfloat16), None, m, 32, "mxfp4", False)
    assert y.shape == (0, 8)


# ---------------------------------------------------------------- router

@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,d,E,k", [(1, 8, 1, 1), (1, 64, 8, 2), (3, 136, 33, 5), (2, 4096, 64, 8), (130, 256, 7, 7),
                                     (5, 520, 256, 8), (9, 1032, 100, 1), (1, 8200, 1024, 32), (65, 24, 1000, 6)])
def test_route(n, d, E, k, f32):
    rng = np.random.default_rng(n + d + E)
    x = bf16(rng.normal(0, 1, (n, d)))
    r = torch.from_numpy((rng.normal(0, 2, (E, d)) * d ** -0.5).astype(np.float32))
    r = r if f32 else r.to(torch.bfloat16)
    for renorm in (True, False):
        ids, w = W.wush_moe_route(x.cuda(), r.cuda(), k, renormalise=renorm)
        ok()
        want_ids, want_w = O.moe_route(f64(x), f64(r), k, renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        # fp32 results of 64-bit arithmetic: half a step, and the float64 sums' own rounding
        assert np.all(np.abs(w.cpu().numpy() - want_w) <= (2.0 ** -24 + 1e-10) * want_w + 1e-44)


def test_route_ties_go_to_the_lower_index():
    x = torch.ones(2, 64, dtype=torch.bfloat16)
    r = torch.zeros(50, 64, dtype=torch.bfloat16)
    r[[3, 7, 31, 32, 49]] = 1.0
    ids, w = W.wush_moe_route(x.cuda(), r.cuda(), 7)
    ok()
    assert ids.tolist() == [[3, 7, 31, 32, 49, 0, 1]] * 2
    rng = np.random.default_rng(0)                       # equal rows with rounding in their sums
    row = bf16(rng.normal(0, 1, (1, 520)))
    ids, _ = W.wush_moe_route(bf16(rng.normal(0, 1, (3, 520))).cuda(), row.repeat(300, 1).cuda(), 9)
    ok()
    assert ids.tolist() == [list(range(9))] * 3


def test_route_close_logits():
    """Logits that differ by 1 part in 10^9: a 32-bit sum could not order them."""
    d = 2048
    x = torch.ones(1, d, dtype=torch.bfloat16)
    r = torch.full((4, d), 1.0, dtype=torch.float32)
    for e, tiny in enumerate((1e-6, 4e-6, 0.0, 2e-6)):
        r[e, 100] = tiny
    ids, _ = W.wush_moe_route(x.cuda(), r.cuda(), 4)
    ok()
    assert ids.tolist() == [[1, 3, 0, 2]]


def test_route_with_bad_values():
    rng = np.random.default_rng(0)
    x = bf16(rng.normal(0, 1, (3, 64)))
    r = bf16(rng.normal(0, 1, (40, 64)))
    clean_ids, clean_w = W.wush_moe_route(x.cuda(), r.cuda(), 4)
    x[1, 5] = float("nan")
    ids, w = W.wush_moe_route(x.cuda(), r.cuda(), 4)
    ok()
    assert torch.equal(ids[[0, 2]], clean_ids[[0, 2]]) and torch.equal(w[[0, 2]], clean_w[[0, 2]])
    assert ids[1].tolist() == [0, 1, 2, 3] and bool(torch.isnan(w[1]).all())
    r[11, 3] = float("nan")                               # one expert's logit: it ranks last
    x[1, 5] = 0.0
    ids, w = W.wush_moe_route(x.cuda(), r[:33].contiguous().cuda(), 32)
    ok()
    assert bool((ids != 11).all()) and bool(torch.isnan(w).all())
    assert all(len(set(row)) == 32 for row in ids.tolist())


def test_route_large_logits():
    x = torch.full((1, 64), 100.0, dtype=torch.bfloat16)
    r = torch.zeros(5, 64)
    r[2], r[4] = 1000.0, 999.0
    ids, w = W.wush_moe_route(x.cuda(), r.cuda(), 2)
    ok()
    assert ids.tolist() == [[2, 4]] and w.tolist() == [[1.0, 0.0]]
    assert W.wush_moe_route(torch.zeros(0, 64, dtype=torch.bfloat16).cuda(), r.cuda(), 2)[0].shape == (0, 2)


# ---------------------------------------------------------------- experts

def moe_reference(x, ids, weights, T_in, w_in, T_out, w_out, G, fmt):
    """(exact y, its error bound before the last rounding)."""
    E, hidden = w_in[0].shape[0], w_in[0].shape[1] // 2
    y, err = np.zeros((x.shape[0], w_out[0].shape[1])), np.zeros((x.shape[0], w_out[0].shape[1]))
    cache = {}
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            if e not in cache:
                cache[e] = values(w_in, e, G, fmt), values(w_out, e, G, fmt)
            wi, wo = cache[e]
            gu, ge = product_bound(x[t:t + 1], T_in, wi, G, False)
            g, u, eg, eu = gu[0, :hidden], gu[0, hidden:], ge[0, :hidden], ge[0, hidden:]
            s = g / (1.0 + np.exp(-g))
            h = s * u
            # |silu'| < 1.1; eight roundings in exp, division and product
            eh = 1.1 * eg * np.abs(u) + (np.abs(s) + 1.1 * eg) * eu + 8 * 2.0 ** -24 * np.abs(h)
            r, e2 = product_bound(h[None], T_out, wo, G, False)
            through = O.activations(eh[None], None if T_out is None else np.abs(T_out), G) @ np.abs(wo).T
            a = abs(float(weights[t, j]))
            y[t] += float(weights[t, j]) * r[0]
            err[t] += a * (1.01 * e2[0] + 1.01 * through[0]) + 40 * 2.0 ** -24 * a * np.abs(r[0])
    return y, err


def make_layer(rng, E, d, f, G, fmt, kind="block"):
    w_in = make_matrix(rng, (E, 2 * f), d, G, fmt)
    w_out = make_matrix(rng, (E, d), f, G, fmt)
    # scale the input side so that gates are of order one
    if fmt == "nvfp4":
        w_in = w_in[0], w_in[1], (w_in[2] * 0.1 * d ** -0.5).astype(np.float32)
    elif fmt == "int4":
        w_in = w_in[0], (w_in[1] * 10 * d ** -0.5).astype(np.float32), None
    else:
        w_in = w_in[0], (w_in[1] - 2).astype(np.uint8), None
    return make_T(rng, kind, d, G), w_in, make_T(rng, kind, f, G), w_out


def on_device(m):
    return tuple(dev(a) for a in m)


def run_experts(x, ids, weights, layer, G, fmt, **kw):
    T_in, w_in, T_out, w_out = layer
    return W.wush_moe_experts(x.cuda(), dev(ids), dev(weights), dev(T_in), on_device(w_in), dev(T_out),
                              on_device(w_out), G, fmt, **kw)


def check_experts(x, ids, weights, layer, G, fmt, got):
    r, e = moe_reference(f64(x), ids, weights, *layer, G, fmt)
    got = got.float().cpu().numpy().astype(np.float64)
    bad = np.abs(got - r) > e + 2.0 ** -8 * (np.abs(r) + e) + 1e-37
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} {r[bad][0]}"


def some_routing(rng, n, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    w = rng.uniform(0.05, 1, (n, k)).astype(np.float32)
    return ids, w


@pytest.mark.parametrize("n,E,k,db,fb", [(1, 1, 1, 1, 1), (1, 4, 2, 3, 5), (2, 8, 8, 9, 2), (3, 5, 3, 16, 33),
                                         (5, 64, 4, 7, 12), (8, 3, 2, 40, 9), (17, 6, 5, 8, 4), (33, 4, 1, 5, 6),
                                         (64, 16, 6, 4, 3)])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts(fmt, G, n, E, k, db, fb):
    rng = np.random.default_rng(n + E + db)
    kind = ("block", "shared", "none")[(n + db + fb) % 3]
    x = bf16(rng.normal(0, 1, (n, db * G)))
    layer = make_layer(rng, E, db * G, fb * G, G, fmt, kind)
    ids, w = some_routing(rng, n, E, k)
    y = run_experts(x, ids, w, layer, G, fmt)
    ok()
    check_experts(x, ids, w, layer, G, fmt, y)


@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_dropped_slots(fmt, G):
    """Ids outside the experts (their weights NaN), a token with none left, an expert nobody chose."""
    rng = np.random.default_rng(4)
    x = bf16(rng.normal(0, 1, (6, 5 * G)))
    layer = make_layer(rng, 7, 5 * G, 3 * G, G, fmt)
    ids, w = some_routing(rng, 6, 6, 3)
    ids[0, 1], ids[2, 0], ids[2, 2], ids[4, 1] = -1, 7, -2 ** 31, 2 ** 31 - 1
    ids[3] = -1
    w[(ids < 0) | (ids >= 7)] = np.nan
    y = run_experts(x, ids, w, layer, G, fmt)
    ok()
    check_experts(x, ids, w, layer, G, fmt, y)
    assert bool((y[3] == 0).all())
    ids[:] = -1
    y = run_experts(x, ids, w, layer, G, fmt)
    ok()
    assert bool((y == 0).all())


@pytest.mark.parametrize("n", [1, 4, 9, 64])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_all_on_one_and_the_same_twice(fmt, G, n):
    rng = np.random.default_rng(n)
    x = bf16(rng.normal(0, 1, (n, 6 * G)))
    layer = make_layer(rng, 5, 6 * G, 4 * G, G, fmt)
    ids = np.full((n, 3), 3, np.int32)
    ids[:, 1] = 1
    w = rng.uniform(-1, 1, (n, 3)).astype(np.float32)
    y = run_experts(x, ids, w, layer, G, fmt)
    again = run_experts(x, ids, w, layer, G, fmt)
    ok()
    check_experts(x, ids, w, layer, G, fmt, y)
    assert torch.equal(y, again)


def test_experts_many_slots():
    """As many slots as a call takes, over many experts, one of them taken by every token."""
    rng = np.random.default_rng(6)
    n, E, k = 64, 1024, 32
    x = bf16(rng.normal(0, 1, (n, 64)))
    layer = make_layer(rng, E, 64, 32, 32, "mxfp4")
    ids, w = some_routing(rng, n, E, k)
    ids[:, 5] = 17
    y = run_experts(x, ids, w, layer, 32, "mxfp4")
    ok()
    check_experts(x, ids, w, layer, 32, "mxfp4", y)


@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_write_inside_their_buffers(fmt, G):
    rng = np.random.default_rng(4)
    n, d, f, k = 3, 5 * G, 3 * G, 2
    x = bf16(rng.normal(0, 1, (n, d)))
    layer = make_layer(rng, 4, d, f, G, fmt)
    ids, w = some_routing(rng, n, 4, k)
    need = W.wush_moe_workspace_bytes(n, d, f, k)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    big = torch.full((n + 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
    y = run_experts(x, ids, w, layer, G, fmt, out=big[:n], workspace=ws[:need])
    y2 = run_experts(x, ids, w, layer, G, fmt, workspace=ws[:need])        # as the first call left it
    ok()
    check_experts(x, ids, w, layer, G, fmt, y)
    assert torch.equal(y, y2)
    assert bool((big[n:] == 7).all()) and bool((ws[need:] == 0xFF).all())


def test_experts_bad_values_stay_with_their_token():
    rng = np.random.default_rng(4)
    x = bf16(rng.normal(0, 1, (5, 160)))
    layer = make_layer(rng, 3, 160, 96, 32, "mxfp4")
    ids, w = some_routing(rng, 5, 3, 2)
    clean = run_experts(x, ids, w, layer, 32, "mxfp4")
    x[1, 3] = float("nan")
    y = run_experts(x, ids, w, layer, 32, "mxfp4")
    ok()
    assert torch.equal(y[[0, 2, 3, 4]], clean[[0, 2, 3, 4]]) and bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_layer_is_the_router_and_the_experts(fmt, G, f32):
    rng = np.random.default_rng(9)
    n, E, k, d, f = 5, 12, 3, 6 * G, 5 * G
    x = bf16(rng.normal(0, 1, (n, d)))
    r = torch.from_numpy((rng.normal(0, 2, (E, d)) * d ** -0.5).astype(np.float32))
    r = (r if f32 else r.to(torch.bfloat16)).cuda()
    layer = make_layer(rng, E, d, f, G, fmt)
    T_in, w_in, T_out, w_out = dev(layer[0]), on_device(layer[1]), dev(layer[2]), on_device(layer[3])
    for renorm in (True, False):
        y, ids, w = W.wush_moe_layer(x.cuda(), r, k, T_in, w_in, T_out, w_out, G, fmt, renormalise=renorm)
        ids2, w2 = W.wush_moe_route(x.cuda(), r, k, renormalise=renorm)
        y2 = W.wush_moe_experts(x.cuda(), ids2, w2, T_in, w_in, T_out, w_out, G, fmt)
        ok()
        assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(y, y2)
        check_experts(x, ids.cpu().numpy(), w.cpu().numpy(), layer, G, fmt, y)


def test_empty_batches():
    rng = np.random.default_rng(9)
    layer = make_layer(rng, 4, 64, 64, 32, "mxfp4")
    x = torch.zeros(0, 64, dtype=torch.bfloat16)
    y = run_experts(x, np.zeros((0, 2), np.int32), np.zeros((0, 2), np.float32), layer, 32, "mxfp4")
    assert y.shape == (0, 64)
    r = torch.zeros(4, 64, dtype=torch.bfloat16).cuda()
    y, ids, w = W.wush_moe_layer(x.cuda(), r, 2, dev(layer[0]), on_device(layer[1]), dev(layer[2]), on_device(layer[3]),
                                 32, "mxfp4")
    assert y.shape == (0, 64) and ids.shape == (0, 2) and w.shape == (0, 2)


# ---------------------------------------------------------------- a decoding step

class Step:
    """x -> x + attention projection -> x + experts -> logits, on weights that the library quantised."""

    def __init__(self, fmt, G, d=256, f=192, E=6, vocab=517, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.fmt, self.G, self.k = fmt, G, 2
        cal = rnd(512, d).to(torch.bfloat16).cuda()
        calf = rnd(512, f).to(torch.bfloat16).cuda()
        quant = lambda w, T: W.wush_quant_weight(w, T, G, fmt)
        attn = (rnd(d, d) * d ** -0.5).cuda()
        self.T_attn, Tw = W.wush_build_transforms(attn, cal, G)
        self.attn = quant(attn, Tw)
        w_in = (rnd(E, 2 * f, d) * d ** -0.5).cuda()
        w_out = (rnd(E, d, f) * f ** -0.5).cuda()
        self.T_in, Tw_in = W.wush_build_transforms(w_in.reshape(-1, d), cal, G)
        self.T_out, Tw_out = W.wush_build_transforms(w_out.reshape(-1, f), calf, G)
        stack = lambda ms: (torch.stack([m[0] for m in ms]), torch.stack([m[1] for m in ms]),
                            torch.cat([m[2] for m in ms]) if fmt == "nvfp4" else None)
        self.w_in = stack([quant(w_in[e].contiguous(), Tw_in) for e in range(E)])
        self.w_out = stack([quant(w_out[e].contiguous(), Tw_out) for e in range(E)])
        self.router = (rnd(E, d) * 2 * d ** -0.5).to(torch.bfloat16).cuda()
        head = (rnd(vocab, d) * d ** -0.5).cuda()
        self.T_head, Tw = W.wush_build_transforms(head, cal, G)
        self.head = quant(head, Tw)
        self.float = attn.double(), w_in.double(), w_out.double(), head.double()

    def __call__(self, x, stream=None):
        kw = dict(stream=stream)
        a = x + W.wush_gemv(x, self.T_attn, *self.attn, self.G, self.fmt, **kw)
        y, ids, w = W.wush_moe_layer(a, self.router, self.k, self.T_in, self.w_in, self.T_out, self.w_out, self.G,
                                     self.fmt, **kw)
        b = a + y
        return a, y, ids, w, b, W.wush_gemv(b, self.T_head, *self.head, self.G, self.fmt, out_dtype=torch.float32, **kw)


def host(m):
    return tuple(None if t is None else t.cpu().numpy() for t in m)


@pytest.mark.parametrize("n", [1, 4, 11])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_decoding_step(fmt, G, n):
    s = Step(fmt, G)
    x = torch.randn(n, 256, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    a, y, ids, w, b, logits = s(x.cuda())
    ok()
    # each operator on what it was given
    proj = W.wush_gemv(x.cuda(), s.T_attn, *s.attn, G, fmt)
    check_gemv(x, s.T_attn.cpu().numpy(), host(s.attn), G, fmt, False, proj)
    want_ids, _ = O.moe_route(f64(a.cpu()), f64(s.router.cpu()), s.k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    layer = s.T_in.cpu().numpy(), host(s.w_in), s.T_out.cpu().numpy(), host(s.w_out)
    check_experts(a.cpu(), ids.cpu().numpy(), w.cpu().numpy(), layer, G, fmt, y)
    check_gemv(b.cpu(), s.T_head.cpu().numpy(), host(s.head), G, fmt, True, logits)
    # and the unquantised layer they stand for: 4 bits leave about a tenth (T_act and T_w cancel)
    full = b.double() @ s.float[3].T
    assert float((logits.double() - full).norm() / full.norm()) < 0.25


def test_decoding_step_in_a_graph_on_a_side_stream():
    s = Step("mxfp4", 32)
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    eager = [t.clone() for t in s(x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    static = torch.zeros_like(x)
    with torch.cuda.stream(side):
        s(static)
        g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = s(static)
        with torch.cuda.graph(g2, stream=side):
            out2 = s(static)
        for v in (x, torch.zeros_like(x), x):
            static.copy_(v)
            g.replay()
            g2.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(eager, out, out2):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_calls_on_two_streams_at_once():
    s, s2 = Step("nvfp4", 16, seed=1), Step("int4", 32, seed=2)
    gen = torch.Generator().manual_seed(5)
    xs = [torch.randn(2, 256, generator=gen).to(torch.bfloat16).cuda() for _ in range(6)]
    want = [[t.clone() for t in f(x)] for x in xs for f in (s, s2)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for x in xs:
        for f, st in zip((s, s2), streams):
            with torch.cuda.stream(st):
                got.append(f(x))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def device_values(m, G, fmt):
    """[E][rows][K] fp64 values of stacked device matrices."""
    return torch.stack([W.wush_dequant(m[0][e], m[1][e], None if m[2] is None else m[2][e:e + 1], G, fmt).double()
                        for e in range(m[0].shape[0])])


@pytest.mark.parametrize("n,k", [(1, 4), (3, 4), (8, 2), (20, 5), (64, 6)])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_at_layer_sizes(fmt, G, n, k):
    """Several units per CTA, tiles shared by CTAs and several passes per expert, against 64-bit products
    on the device.  Bound: the two products' 2^-11 each on sums of absolute values, through the activation
    (|silu'| < 1.1), and the sums' (64 + K / 32) 2^-23, well inside 2^-10 of those sums."""
    rng = np.random.default_rng(n)
    E, d, f = 12, 1072 if G == 16 else 1056, 1040 if G == 16 else 1120
    x = bf16(rng.normal(0, 1, (n, d)))
    layer = make_layer(rng, E, d, f, G, fmt, "none")
    ids, w = some_routing(rng, n, E, k)
    ids[:, 0] = np.where(np.arange(n) % 3 == 0, 5, ids[:, 0])
    w_in, w_out = on_device(layer[1]), on_device(layer[3])
    y = run_experts(x, ids, w, layer, G, fmt)
    again = run_experts(x, ids, w, layer, G, fmt)
    ok()
    assert torch.equal(y, again)
    a, b, xd = device_values(w_in, G, fmt), device_values(w_out, G, fmt), x.double().cuda()
    r, bound = torch.zeros(n, d, dtype=torch.float64).cuda(), torch.zeros(n, d, dtype=torch.float64).cuda()
    for t in range(n):
        for j in range(k):
            e, wt = int(ids[t, j]), float(w[t, j])
            gu, sa = a[e] @ xd[t], a[e].abs() @ xd[t].abs()
            g, u, sg, su = gu[:f], gu[f:], sa[:f], sa[f:]
            s = g * torch.sigmoid(g)
            dh = 2.0 ** -10 * (1.1 * sg * u.abs() + (s.abs() + 2.0 ** -10 * sg) * su) + 2.0 ** -20 * (s * u).abs()
            r[t] += wt * (b[e] @ (s * u))
            bound[t] += abs(wt) * (b[e].abs() @ (dh + 2.0 ** -10 * (s * u).abs()))
    bad = (y.double() - r).abs() > bound + 2.0 ** -8 * (r.abs() + bound)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,rows,K", [(1, 9001, 1056), (2, 4096, 4096), (4, 3001, 2080), (7, 8197, 1184), (16, 6000, 2048),
                                      (40, 2500, 1120)])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_at_layer_sizes(fmt, G, n, rows, K, f32):
    """Clusters, shares that begin and end inside tiles, whole tiles: 64-bit products on the device."""
    rng = np.random.default_rng(rows)
    K += 16 if G == 16 and rows % 2 else 0
    x, m = make_x(rng, n, K), make_matrix(rng, (rows,), K, G, fmt)
    y = run_gemv(x, None, m, G, fmt, f32)
    again = run_gemv(x, None, m, G, fmt, f32)
    ok()
    assert torch.equal(y, again)
    v = W.wush_dequant(dev(m[0]), dev(m[1]), dev(m[2]), G, fmt).double()
    xd = x.double().cuda()
    r, S = xd @ v.T, xd.abs() @ v.abs().T
    e = ((2.0 ** -22 if f32 else 2.0 ** -11) + (G + 64 + K / 32) * 2.0 ** -23) * S + 2.0 ** -38 * xd.abs().max() * v.abs().sum(1)
    bad = (y.double() - r).abs() > e + (2.0 ** -24 if f32 else 2.0 ** -8) * (r.abs() + e)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off"


def test_decode_bench_runs():
    """The per-layer benchmark's few-token rows, on small layers."""
    from blockwise_adaptive_transforms_b200 import layer_bench
    r = layer_bench.decode_shape(3, 256, 256)
    assert set(r["us"]) == {"bf16", "mxfp4", "nvfp4", "int4"} and min(r["us"].values()) > 0
    r = layer_bench.decode_experts(2, 128, 64, 4, 2)
    assert set(r["us"]) == {"mxfp4", "nvfp4", "int4"} and min(r["us"].values()) > 0


def test_stream_argument():
    """``stream=`` launches there: a call queued behind slow work sees what that work writes."""
    rng = np.random.default_rng(1)
    m = make_matrix(rng, (64,), 128, 32, "mxfp4")
    x = make_x(rng, 2, 128).cuda()
    want = run_gemv(x.cpu(), None, m, 32, "mxfp4", False)
    codes, scales = dev(m[0]), dev(m[1])
    side = torch.cuda.Stream()
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        late.copy_(x)
    y = W.wush_gemv(late, None, codes, scales, None, 32, "mxfp4", stream=side)
    y2 = W.wush_gemv(late, None, codes, scales, None, 32, "mxfp4", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want)


def test_binding_refusals():
    rng = np.random.default_rng(1)
    m = make_matrix(rng, (64,), 128, 32, "mxfp4")
    c, s = dev(m[0]), dev(m[1])
    x = make_x(rng, 2, 128).cuda()
    call = lambda x=x, T=None, c=c, s=s, ts=None, G=32, fmt="mxfp4", **kw: W.wush_gemv(x, T, c, s, ts, G, fmt, **kw)
    for bad, err in [(dict(x=x.float()), TypeError), (dict(x=x[0]), ValueError), (dict(x=x[:, :96]), ValueError),
                     (dict(x=x.t()), ValueError), (dict(c=c[:, :32]), ValueError), (dict(c=c.view(torch.int8)), TypeError),
                     (dict(s=s[:63]), ValueError), (dict(s=s.float()), TypeError), (dict(fmt="nvfp4", G=16), ValueError),
                     (dict(T=torch.zeros(3, 32, 32).cuda()), ValueError), (dict(T=torch.zeros(4, 32, 32)), TypeError),
                     (dict(out=torch.zeros(2, 63, dtype=torch.bfloat16).cuda()), ValueError),
                     (dict(out=torch.zeros(2, 64).cuda()), TypeError), (dict(out_dtype=torch.float16), TypeError),
                     (dict(workspace=torch.zeros(16, dtype=torch.uint8).cuda()), W.WushError),
                     (dict(x=torch.zeros(65, 128, dtype=torch.bfloat16).cuda()), W.WushError),
                     (dict(G=48), ValueError), (dict(G=0), ValueError)]:
        with pytest.raises(err):
            call(**bad)
    r = torch.zeros(8, 128, dtype=torch.bfloat16).cuda()
    for bad, err in [((x, r.half(), 2), TypeError), ((x, r[:, :64], 2), ValueError), ((x, r, 9), W.WushError),
                     ((x, r, 0), W.WushError), ((x.float(), r, 2), TypeError)]:
        with pytest.raises(err):
            W.wush_moe_route(*bad)
    layer = make_layer(rng, 4, 128, 64, 32, "mxfp4")
    T_in, w_in, T_out, w_out = dev(layer[0]), on_device(layer[1]), dev(layer[2]), on_device(layer[3])
    ids, w = torch.zeros(2, 2, dtype=torch.int32).cuda(), torch.ones(2, 2).cuda()
    ok_args = dict(x=x, ids=ids, weights=w, T_in=T_in, w_in=w_in, T_out=T_out, w_out=w_out, G=32, fmt="mxfp4")
    for bad, err in [(dict(ids=ids.long()), TypeError), (dict(weights=w[:, :1]), ValueError),
                     (dict(w_in=(w_in[0][:, :64], w_in[1], None)), ValueError), (dict(T_out=T_in), ValueError),
                     (dict(w_out=(w_out[0][:3], w_out[1], None)), ValueError), (dict(fmt="nvfp4", G=16), ValueError)]:
        with pytest.raises(err):
            W.wush_moe_experts(**{**ok_args, **bad})
    with pytest.raises(ValueError):
        W.wush_moe_layer(x, torch.zeros(5, 128, dtype=torch.bfloat16).cuda(), 2, T_in, w_in, T_out, w_out, 32, "mxfp4")
    ok()


def test_short_wait_limit():
    """With waits limited to 1 ns the results are right (a first look at a barrier may itself last until the copy
    lands) or the device error word says that a wait gave up; calls after that, on the same workspace, are right."""
    rng = np.random.default_rng(3)
    m = make_matrix(rng, (3000,), 4096, 32, "mxfp4")
    layer = make_layer(rng, 6, 1024, 512, 32, "mxfp4")
    ids, w = some_routing(rng, 10, 6, 2)
    cases = [(make_x(rng, n, 4096), f32) for n, f32 in ((1, False), (3, True), (9, False))]
    xe = bf16(rng.normal(0, 1, (10, 1024)))
    want = [run_gemv(x, None, m, 32, "mxfp4", f32) for x, f32 in cases] + [run_experts(xe, ids, w, layer, 32, "mxfp4")]
    ok()
    space = torch.empty(max(W.wush_gemv_workspace_bytes(9, 4096), W.wush_moe_workspace_bytes(10, 1024, 512, 2)),
                        dtype=torch.uint8, device="cuda")
    try:
        W.wush_set_wait_limit_ns(1)
        hasty = [run_gemv(x, None, m, 32, "mxfp4", f32, workspace=space) for x, f32 in cases]
        hasty.append(run_experts(xe, ids, w, layer, 32, "mxfp4", workspace=space))
        torch.cuda.synchronize()
    finally:
        W.wush_set_wait_limit_ns(0)
    _, bits = W.wush_device_status()
    assert bits in (0, 256)
    if bits == 0:
        for a, b in zip(hasty, want):
            assert torch.equal(a, b)
    got = [run_gemv(x, None, m, 32, "mxfp4", f32, workspace=space) for x, f32 in cases]
    got.append(run_experts(xe, ids, w, layer, 32, "mxfp4", workspace=space))
    ok()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_experts_behind_four_gigabytes():
    """The last expert of a stack whose codes and rows' offsets pass 32 bits gives what it gives in a short stack."""
    E, d, f = 66, 8192, 8192
    gen = torch.Generator(device="cuda").manual_seed(1)

    def stack(rows, K):
        return (torch.randint(0, 256, (E, rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen),
                torch.randint(110, 118, (E, rows, K // 32), dtype=torch.uint8, device="cuda", generator=gen), None)
    w_in, w_out = stack(2 * f, d), stack(d, f)
    assert w_in[0].numel() > 2 ** 32
    few = [tuple(None if t is None else t[E - 8:].clone() for t in s) for s in (w_in, w_out)]
    for n in (1, 4, 12):
        x = torch.randn(n, d, device="cuda", generator=gen).to(torch.bfloat16)
        ids = torch.full((n, 1), E - 1, dtype=torch.int32, device="cuda")
        weights = torch.rand(n, 1, device="cuda", generator=gen)
        y = W.wush_moe_experts(x, ids, weights, None, w_in, None, w_out, 32, "mxfp4")
        short = W.wush_moe_experts(x, torch.full_like(ids, 7), weights, None, few[0], None, few[1], 32, "mxfp4")
        ok()
        assert bool(y.isfinite().all()) and bool((y != 0).any())
        assert torch.equal(y, short)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_bad_scales_stay_with_their_expert(fmt, G, n):
    """Scales of one expert that are not finite reach the tokens that chose it, in the rows they belong to, and
    nothing else: every other result keeps its bits."""
    rng = np.random.default_rng(n)
    for db, fb in ((9, 5), (33, 40)):
        E, k, d, f = 5, 2, db * G, fb * G
        x = bf16(rng.normal(0, 1, (n, d)))
        layer = make_layer(rng, E, d, f, G, fmt)
        ids = np.array([[2, 4] if t % 3 != 1 else [1, 3] for t in range(n)], np.int32)
        w = rng.uniform(0.1, 1, (n, k)).astype(np.float32)
        clean = run_experts(x, ids, w, layer, G, fmt)
        chose = torch.from_numpy((ids == 2).any(1)).cuda()
        T_in, w_in, T_out, w_out = layer
        bad = (255,) if fmt == "mxfp4" else (0x7F,) if fmt == "nvfp4" else (np.nan, np.inf)
        for value in bad:
            scales = w_out[1].copy()
            hit = rng.choice(d, 7, replace=False)
            scales[2, hit, rng.integers(0, fb, 7)] = value
            scales[0, :, :] = value                        # nobody chose this one
            y = run_experts(x, ids, w, (T_in, w_in, T_out, (w_out[0], scales, w_out[2])), G, fmt)
            ok()
            touched = torch.zeros(n, d, dtype=torch.bool, device="cuda")
            touched[:, torch.from_numpy(hit).cuda()] = True
            touched &= chose[:, None]
            assert not bool(torch.isfinite(y[touched]).any())
            assert torch.equal(y[~touched], clean[~touched])
            scales = w_in[1].copy()
            scales[2, rng.integers(0, 2 * f), rng.integers(0, db)] = value
            y = run_experts(x, ids, w, (T_in, (w_in[0], scales, w_in[2]), T_out, w_out), G, fmt)
            ok()
            assert torch.equal(y[~chose], clean[~chose])
            assert not bool(torch.isfinite(y[chose]).all())
        if fmt == "nvfp4":
            for which in (w_in, w_out):
                ts = which[2].copy()
                ts[2] = np.nan
                m = which[0], which[1], ts
                y = run_experts(x, ids, w, (T_in, m if which is w_in else w_in, T_out, m if which is w_out else w_out),
                                G, fmt)
                ok()
                assert torch.equal(y[~chose], clean[~chose]) and bool(torch.isnan(y[chose]).all())


def test_calls_right_after_an_expired_wait():
    """Calls whose waits are limited to 1 ns leave nothing behind them: the products that follow at once, on the same
    SMs and shared memory, and those on another stream beside them, are right.  Shares of one or two units (a
    cluster's), of many, tiles shared by CTAs, and the layer."""
    rng = np.random.default_rng(8)
    cases = []
    for fmt, G, n, rows, K in (("mxfp4", 32, 1, 4096, 4096), ("mxfp4", 32, 1, 3000, 4096), ("nvfp4", 16, 3, 700, 1040),
                               ("int4", 32, 8, 8197, 2048), ("int4", 16, 12, 3001, 1008), ("mxfp4", 32, 16, 20000, 1024)):
        m = make_matrix(rng, (rows,), K, G, fmt)
        cases.append((make_x(rng, n, K).cuda(), None, dev(m[0]), dev(m[1]), dev(m[2]), G, fmt))
    layer = make_layer(rng, 6, 1024, 512, 32, "mxfp4")
    parts = dev(layer[0]), on_device(layer[1]), dev(layer[2]), on_device(layer[3])
    routed = []
    for n in (2, 10):
        ids, w = some_routing(rng, n, 6, 2)
        routed.append((bf16(rng.normal(0, 1, (n, 1024))).cuda(), dev(ids), dev(w), *parts, 32, "mxfp4"))
    calls = [lambda c=c: W.wush_gemv(*c) for c in cases] + [lambda c=c: W.wush_moe_experts(*c) for c in routed]
    want = [c() for c in calls]
    ok()
    side = torch.cuda.Stream()
    got = []
    try:
        for i, hasty in enumerate(calls * 2):
            W.wush_set_wait_limit_ns(1)
            for _ in range(3):
                hasty()
            W.wush_set_wait_limit_ns(0)
            a, b = i % len(calls), (i * 3 + 1) % len(calls)
            got.append((a, calls[a]()))
            with torch.cuda.stream(side):
                got.append((b, calls[b]()))
        torch.cuda.synchronize()
    finally:
        W.wush_set_wait_limit_ns(0)
    assert W.wush_device_status()[1] in (0, 256)
    for i, y in got:
        assert torch.equal(y, want[i])


def test_bounded_wait_gives_up_and_reports():
    st, bits = W.wush_selftest_decode_wait_timeout(2_000_000)     # 2 ms
    assert st == 5 and bits == 256
    ok()
    rng = np.random.default_rng(1)                                # the context is still usable afterwards
    x, m = make_x(rng, 2, 256), make_matrix(rng, (64,), 256, 32, "mxfp4")
    y = run_gemv(x, None, m, 32, "mxfp4", False)
    ok()
    check_gemv(x, None, m, 32, "mxfp4", False, y)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d", [8, 264, 1032, 8192])
@pytest.mark.parametrize("n,E,k", [(15, 64, 8), (16, 5, 3), (16, 256, 8), (17, 100, 9), (24, 1000, 6), (29, 256, 1), (30, 64, 8),
                                   (31, 1000, 32), (31, 5, 5), (32, 100, 2), (129, 256, 8), (129, 64, 4)])
def test_route_batches(n, E, k, d, f32):
    """Batches around the changes of form (one, two and eight tokens per cluster), rows of one and many pieces, odd
    ends: against 64-bit sums, and each token against a call of its own.

    The weights are fp32 roundings of 64-bit values whose own error is far below: half a step from the exact ones,
    and a step, 2^-23, from those of another order of summation."""
    rng = np.random.default_rng(n + d + E)
    x = bf16(rng.normal(0, 1, (n, d)))
    r = torch.from_numpy((rng.normal(0, 2, (E, d)) * d ** -0.5).astype(np.float32))
    r = (r if f32 else r.to(torch.bfloat16)).cuda()
    xg = x.cuda()
    for renorm in (True, False):
        ids, w = W.wush_moe_route(xg, r, k, renormalise=renorm)
        ok()
        want_ids, want_w = O.moe_route(f64(x), f64(r.cpu()), k, renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.all(np.abs(w.cpu().numpy() - want_w) <= (2.0 ** -24 + 1e-10) * want_w + 1e-44)
        for t in {0, 1, 7, 8, n // 2, n - 2, n - 1}:
            one, ow = W.wush_moe_route(xg[t:t + 1].contiguous(), r, k, renormalise=renorm)
            assert torch.equal(one[0], ids[t])
            assert bool(((ow[0] - w[t]).abs() <= 2.0 ** -23 * ow[0] + 1e-44).all())


@pytest.mark.parametrize("n", [15, 16, 17, 30, 31, 65])
def test_route_batches_ties_and_bad_values(n):
    rng = np.random.default_rng(n)
    E, d, k = 100, 1032, 9
    x = bf16(rng.normal(0, 1, (n, d)))
    row = bf16(rng.normal(0, 1, (1, d)))
    ids, w = W.wush_moe_route(x.cuda(), row.repeat(E, 1).cuda(), k)
    ok()
    assert ids.tolist() == [list(range(k))] * n                 # equal rows, with rounding in their sums
    assert bool((w == torch.tensor(1 / k, device="cuda")).all())
    r = bf16(rng.normal(0, 1, (E, d)))
    r[40] = r[7]
    clean_ids, clean_w = W.wush_moe_route(x.cuda(), r.cuda(), k)
    both = ((clean_ids == 7).any(1) & (clean_ids == 40).any(1)).nonzero()[:, 0].tolist()
    for t in both:                                              # a tie inside the chosen ones
        row_ids = clean_ids[t].tolist()
        assert row_ids.index(40) == row_ids.index(7) + 1
    assert not bool(((clean_ids == 40).any(1) & ~(clean_ids == 7).any(1)).any())
    hit = [1, n // 2, n - 1]
    keep = [t for t in range(n) if t not in hit]
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[hit, 700] = bad
        ids, w = W.wush_moe_route(y.cuda(), r.cuda(), k)
        ok()
        assert torch.equal(ids[keep], clean_ids[keep]) and torch.equal(w[keep], clean_w[keep])
        assert bool(torch.isnan(w[hit]).all()) and all(len(set(q)) == k for q in ids[hit].tolist())
    r[11, 900] = float("nan")                                   # one expert's logit, of every token: it ranks last
    ids, w = W.wush_moe_route(x.cuda(), r.cuda(), k)
    ok()
    assert bool((ids != 11).all()) and bool(torch.isnan(w).all())


def test_calls_by_torchs_public_names(monkeypatch):
    """The binding on a torch that has none of the inner calls it prefers."""
    import types
    s = Step("mxfp4", 32)
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = [t.clone() for t in s(x)]
    for name, call in zip(("_current_handle", "_take", "_give_back"), W._torch_calls(types.SimpleNamespace())):
        monkeypatch.setattr(W, name, call)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s(x)
    with torch.cuda.stream(side):
        beside = s(x)
    ok()
    for a, b, c in zip(want, got, beside):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_precision_beside_a_large_channel(fmt, G):
    """Token e holds 1 in one channel and 1.2345678 2^-e, a value of 24 bits, in another of the same 128; the row sees
    the small one alone.  Held in fp16 under a scale that puts 1 at 2^14: half a step is 2^-11 of the value,
    or 2^-25 2^-14 = 2^-39; of the remainder 2^-22, or 2^-36 2^-14 = 2^-50; then the result's rounding, and for fp32
    results the sum of the two terms, half a step each."""
    K, n = 128, 56
    T = np.eye(G, dtype=np.float32)
    T[5, 5] = np.float32(1.2345678)
    x = torch.zeros(n, K, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[:, 64 + 5] = torch.exp2(-torch.arange(n).float()).to(torch.bfloat16)
    codes = np.zeros((3, K // 2), np.uint8)
    codes[1, 32 + 2] = (1 if fmt == "int4" else 2) << 4                     # channel 69
    one = {"mxfp4": 127, "nvfp4": 0x38, "int4": 1.0}[fmt]
    scales = np.full((3, K // G), one, np.float32 if fmt == "int4" else np.uint8)
    m = codes, scales, np.ones(1, np.float32) if fmt == "nvfp4" else None
    r = float(T[5, 5]) * np.exp2(-np.arange(n, dtype=np.float64))
    for f32, bits, floor, step in ((False, 11, 39, 2.0 ** -8), (True, 22, 50, 2.0 ** -23)):
        y = run_gemv(x, T, m, G, fmt, f32)
        ok()
        got = y.float().cpu().numpy().astype(np.float64)
        assert not got[:, [0, 2]].any()
        held = np.maximum(2.0 ** -bits * r, 2.0 ** -floor)
        assert np.all(np.abs(got[:, 1] - r) <= held + step * (r + held)), (fmt, f32)


def shifted(a, by):
    """On the device, ``by`` bytes behind an address that is a multiple of 256."""
    a = np.ascontiguousarray(a)
    room = torch.zeros(a.nbytes + by, dtype=torch.uint8, device="cuda")
    room[by:] = torch.from_numpy(a.reshape(-1).view(np.uint8)).cuda()
    t = room[by:]
    return (t if a.dtype == np.uint8 else t.view(torch.float32)).reshape(a.shape)


@pytest.mark.parametrize("blocks", [7, 8, 16, 33])
@pytest.mark.parametrize("fmt,G,by", [("mxfp4", 32, 1), ("mxfp4", 32, 2), ("mxfp4", 32, 3), ("mxfp4", 32, 4), ("nvfp4", 16, 1),
                                      ("nvfp4", 16, 3), ("nvfp4", 16, 4), ("nvfp4", 16, 8), ("int4", 16, 4), ("int4", 16, 8),
                                      ("int4", 32, 4), ("int4", 32, 8)])
def test_scales_at_any_address(fmt, G, by, blocks):
    """Scales that begin where their alignment lets them: the same bits as from an aligned copy."""
    rng = np.random.default_rng(blocks)
    K = G * blocks
    m = make_matrix(rng, (130,), K, G, fmt)
    c, ts = dev(m[0]), dev(m[2])
    for n in (1, 3, 7, 13):
        x = make_x(rng, n, K).cuda()
        a = W.wush_gemv(x, None, c, dev(m[1]), ts, G, fmt)
        b = W.wush_gemv(x, None, c, shifted(m[1], by), ts, G, fmt)
        ok()
        check_gemv(x.cpu(), None, m, G, fmt, False, b)
        assert torch.equal(a, b)
    layer = make_layer(rng, 3, K, 5 * G, G, fmt, "none")
    w_in, w_out = on_device(layer[1]), on_device(layer[3])
    s_in = w_in[0], shifted(layer[1][1], by), w_in[2]
    s_out = w_out[0], shifted(layer[3][1], by), w_out[2]
    for n in (1, 4, 6, 10):
        ids, w = some_routing(rng, n, 3, 2)
        x = bf16(rng.normal(0, 1, (n, K))).cuda()
        a = W.wush_moe_experts(x, dev(ids), dev(w), None, w_in, None, w_out, G, fmt)
        b = W.wush_moe_experts(x, dev(ids), dev(w), None, s_in, None, s_out, G, fmt)
        ok()
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 4, 8, 64])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_gemv_longest_rows(fmt, G, n):
    """2^20 channels, the most there are, with the bound of the other sizes on 64-bit products."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    K, rows = 2 ** 20, 5
    x = torch.randn(n, K, device="cuda", generator=gen).to(torch.bfloat16)
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    ts = torch.tensor([0.004], device="cuda") if fmt == "nvfp4" else None
    if fmt == "int4":
        codes &= 0x77
        scales = torch.rand(rows, K // G, device="cuda", generator=gen) * 0.01
    else:
        scales = torch.randint(*((110, 120) if fmt == "mxfp4" else (40, 0x7F)), (rows, K // G), dtype=torch.uint8, device="cuda",
                               generator=gen)
    v = W.wush_dequant(codes, scales, ts, G, fmt).double()
    r, S = x.double() @ v.T, x.double().abs() @ v.abs().T
    for f32 in (False, True):
        y = W.wush_gemv(x, None, codes, scales, ts, G, fmt, out_dtype=torch.float32 if f32 else torch.bfloat16)
        again = W.wush_gemv(x, None, codes, scales, ts, G, fmt, out_dtype=torch.float32 if f32 else torch.bfloat16)
        ok()
        # x itself fits fp16 under its scale down to 2^-28 of the largest of 128: the sums alone are rounded
        e = (G + 64 + K / 32) * 2.0 ** -23 * S
        assert bool(((y.double() - r).abs() <= e + (2.0 ** -24 if f32 else 2.0 ** -8) * (r.abs() + e)).all())
        assert torch.equal(y, again)


@pytest.mark.parametrize("d,f", [(2 ** 20, 32), (32, 2 ** 20)])
@pytest.mark.parametrize("n,k", [(1, 2), (6, 2), (64, 32)])
def test_experts_longest_rows(n, k, d, f):
    """A layer 2^20 wide, or with 2^20 hidden values; with 64 tokens of 32 slots the hidden columns, or the slots' products,
    pass 4 GB.  A few tokens against 64-bit products; bounds as for layers of ordinary sizes."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    E = 32
    make = lambda rows, K: (torch.randint(0, 256, (E, rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen),
                            torch.randint(112, 116, (E, rows, K // 32), dtype=torch.uint8, device="cuda", generator=gen), None)
    w_in, w_out = make(2 * f, d), make(d, f)
    if f > d:
        w_in[1].add_(10)                                    # gates of order one
    x = torch.randn(n, d, device="cuda", generator=gen).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:k] for _ in range(n)]).to(torch.int32)
    w = torch.rand(n, k, device="cuda", generator=gen)
    y = W.wush_moe_experts(x, ids, w, None, w_in, None, w_out, 32, "mxfp4")
    ok()
    for t in {0, n // 2, n - 1}:
        r, bound = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
        xt = x[t].double()
        for e, wt in zip(ids[t].tolist(), w[t].tolist()):
            a, b = (W.wush_dequant(m[0][e], m[1][e], None, 32, "mxfp4").double() for m in (w_in, w_out))
            gu, sa = a @ xt, a.abs() @ xt.abs()
            g, u, sg, su = gu[:f], gu[f:], sa[:f], sa[f:]
            h = g * torch.sigmoid(g) * u
            # fp16 columns 2^-11, sums (G + 64 + K / 32) 2^-23: of the gate and up rows, then of the hidden values
            c1, c2 = (2.0 ** -11 + (96 + q / 32) * 2.0 ** -23 for q in (d, f))
            dh = c1 * (1.1 * sg * u.abs() + ((g * torch.sigmoid(g)).abs() + 1.1 * c1 * sg) * su) + 2.0 ** -20 * h.abs()
            r += wt * (b @ h)
            bound += wt * (b.abs() @ (dh + c2 * h.abs()))
        bad = (y[t].double() - r).abs() > bound + 2.0 ** -8 * (r.abs() + bound)
        assert not bool(bad.any()), f"token {t}: {int(bad.sum())} off"


@pytest.mark.parametrize("n", [3, 8, 9, 64])
@pytest.mark.parametrize("fmt,G", FORMATS)
def test_experts_more_slots_than_experts_and_bad_weights(fmt, G, n):
    """Slots that repeat experts, and a routing weight that is not finite: it stays with its token."""
    rng = np.random.default_rng(n)
    E, k, d, f = 2, 7, 5 * G, 3 * G
    x = bf16(rng.normal(0, 1, (n, d)))
    layer = make_layer(rng, E, d, f, G, fmt)
    ids = rng.integers(-1, E + 1, (n, k)).astype(np.int32)
    ids[1, 2] = 1
    w = rng.uniform(0.05, 1, (n, k)).astype(np.float32)
    y = run_experts(x, ids, w, layer, G, fmt)
    ok()
    check_experts(x, ids, w, layer, G, fmt, y)
    for bad in (np.nan, np.inf):
        w2 = w.copy()
        w2[1, 2] = bad
        z = run_experts(x, ids, w2, layer, G, fmt)
        ok()
        keep = [t for t in range(n) if t != 1]
        assert torch.equal(z[keep], y[keep]) and not bool(torch.isfinite(z[1]).any())
