"""GPU tests of the SwiGLU that keeps its input in 8 bits, and of its backward pass."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])


def _input(rows, F, dt, seed=1, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, 2 * F, generator=g) * spread).to(dt), torch.randn(rows, F, generator=g).to(dt)


def _kept(codes, scales, F):
    """Decoded halves (float64) of the kept copy."""
    c, s = codes.cpu().numpy().astype(np.int64), scales.cpu().numpy().astype(np.int64)
    return [torch.from_numpy(P.e4m3_values(c[:, i * F:(i + 1) * F], s[:, i], F)) for i in (0, 1)]


# The kernels divide by 1 + e^-a with __fdividef, which is defined to give 0 for a divisor in (2^126, 2^128): there the sigmoid,
# itself below 2^-126, is off by at most its own value.  So every result gets that times the factors beside the sigmoid.
S0 = 2.0 ** -126


def _check_forward(h13, out, F, dt):
    x = h13.double().numpy()
    for i in (0, 1):
        code, byte = P.e4m3(x[:, i * F:(i + 1) * F])
        P.assert_same(out["codes"][:, i * F:(i + 1) * F], torch.from_numpy(code).to(torch.uint8), f"codes {i}")
        P.assert_same(out["scales"][:, i], torch.from_numpy(byte).to(torch.uint8), f"scales {i}")
    a, b = h13.double()[:, :F], h13.double()[:, F:]
    ref = a * P.sigmoid(a) * b
    e = (P.sigmoid_err(a) + 2 * 2.0 ** -24) * ref.abs() + S0 * ((a * b).abs() + 1)
    P.assert_within(out["h"], ref, e + P.u(dt) * (ref.abs() + e) + P.tiny(dt), "h")


def _check_backward(dh, out, got, F, dt):
    a, b = _kept(out["codes"], out["scales"], F)
    d, s, r = dh.double(), P.sigmoid(a), P.sigmoid_err(a)
    h = a * s * b
    e = (r + 2 * 2.0 ** -24) * h.abs() + S0 * ((a * b).abs() + 1)
    P.assert_within(got["h"], h, e + P.u(dt) * (h.abs() + e) + P.tiny(dt), "h again")
    db = d * a * s
    e = (r + 2 * 2.0 ** -24) * db.abs() + S0 * ((d * a).abs() + 1)
    P.assert_within(got["dh13"][:, F:], db, e + P.u(dt) * (db.abs() + e) + P.tiny(dt), "db")
    br = 1 + a * (1 - s)
    da = d * b * s * br
    # bracket: 1 - s is off by s r + 2^-24, the product and the sum by half a step each
    eb = a.abs() * (s * r + 2.0 ** -24) + 2.0 ** -24 * (a.abs() * (1 - s) + br.abs())
    e = (d * b).abs() * s * eb + (r + 3 * 2.0 ** -24) * da.abs() + S0 * ((d * b).abs() * (1 + a.abs()) + 1)
    P.assert_within(got["dh13"][:, :F], da, e + P.u(dt) * (da.abs() + e) + P.tiny(dt), "da")


@DTYPES
@pytest.mark.parametrize("rows,F", [(1, 8), (3, 24), (2, 32), (37, 40), (5, 264), (129, 1416), (64, 512), (700, 96)])
def test_forward_and_backward(rows, F, dt):
    h13, dh = _input(rows, F, dt)
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    assert out["scales"].shape == (rows, 2, (F + 31) // 32)
    _check_forward(h13, out, F, dt)
    got = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"])
    _check_backward(dh, out, got, F, dt)
    alone = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"], want_h=False)
    assert alone["h"] is None and torch.equal(alone["dh13"], got["dh13"])


def test_copy_is_the_row_cast():
    """With whole blocks the copy is mxfp8_quantize's ROW codes and scales, and mxfp8_dequantize reads it."""
    h13, _ = _input(70, 256, BF, seed=2)
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    ref = mxk.mxfp8_quantize(h13.to(DEV), mxk.ROW)
    assert torch.equal(out["codes"], ref["row_codes"]) and torch.equal(out["scales"].reshape(70, -1), ref["row_scales"])


@DTYPES
def test_every_scale_of_the_type(dt):
    """Rows over the type's whole exponent range, subnormals and zeros included."""
    F = 64
    g = torch.Generator().manual_seed(3)
    lo, hi = (-132, 127) if dt == BF else (-24, 15)
    e = torch.linspace(lo, hi, hi - lo + 1, dtype=torch.float64)
    x = (torch.rand(e.numel(), 2 * F, generator=g, dtype=torch.float64) * 2 - 1) * torch.pow(2.0, e).unsqueeze(1)
    h13 = x.to(dt)
    h13[5] = 0
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    for i in (0, 1):
        code, byte = P.e4m3(h13.double().numpy()[:, i * F:(i + 1) * F])
        P.assert_same(out["codes"][:, i * F:(i + 1) * F], torch.from_numpy(code).to(torch.uint8), "codes")
        P.assert_same(out["scales"][:, i], torch.from_numpy(byte).to(torch.uint8), "scales")


@DTYPES
def test_nan_and_infinity_stay_in_their_block(dt):
    h13, dh = _input(4, 72, dt, seed=4)
    h13[1, 3], h13[2, 72 + 40] = float("nan"), float("-inf")
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    got = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"])
    bad = torch.zeros(4, 72, dtype=torch.bool)
    bad[1, :32], bad[2, 32:64] = True, True
    for t in (got["h"], got["dh13"][:, :72]):
        assert torch.equal(torch.isnan(t).cpu(), bad)
    assert out["scales"].cpu()[1, 0].tolist()[0] == 255 and out["scales"].cpu()[2, 1].tolist()[1] == 255
    clean, dcl = _input(4, 72, dt, seed=4)
    ref = mxk.mxfp8_swiglu_ckpt(clean.to(DEV))
    assert torch.equal(out["h"][0], ref["h"][0]) and torch.equal(out["codes"][3], ref["codes"][3])


@DTYPES
def test_far_gates(dt):
    """Gates far on both sides: the exponential over- and underflows, nothing else does."""
    F = 32
    a = torch.cat([torch.linspace(-300, 300, F * 4), torch.linspace(-20, 20, F * 4)]).reshape(8, F)
    h13 = torch.cat([a, torch.ones(8, F)], dim=1).to(dt)
    dh = torch.ones(8, F, dtype=dt)
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    _check_forward(h13, out, F, dt)
    _check_backward(dh, out, mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"]), F, dt)


def test_gradient_against_differences():
    """dh13 against central differences of sum(dh * h) at the kept values, in 64 bits."""
    F, dt = 40, FP
    h13, dh = _input(6, F, dt, seed=5)
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    got = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"])["dh13"].cpu().double()
    a, b = _kept(out["codes"], out["scales"], F)
    f = lambda x, y: x * P.sigmoid(x) * y  # noqa: E731
    eps = 1e-5
    da = dh.double() * (f(a + eps, b) - f(a - eps, b)) / (2 * eps)
    db = dh.double() * (f(a, b + eps) - f(a, b - eps)) / (2 * eps)
    # the difference's own error: third derivative eps^2 / 6 < 1e-10, 64-bit cancellation 1e-16 / eps, times |dh b| <= 100
    for x, y in ((got[:, :F], da), (got[:, F:], db)):
        P.assert_within(x, y, P.u(dt) * y.abs() * 1.01 + 1e-5 + P.tiny(dt), "difference")


@DTYPES
def test_rows_past_the_device_count_are_left(dt):
    rows, F = 50, 104
    h13, dh = _input(rows, F, dt, seed=6)
    full = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    for n in (0, 1, 33, 50, 90):
        cnt = torch.tensor([n], dtype=torch.int32, device=DEV)
        poisoned = h13.clone()
        poisoned[n:] = float("nan")
        bufs = dict(h=torch.full((rows, F), 5.0, dtype=dt, device=DEV), codes=torch.full((rows, 2 * F), 9, dtype=torch.uint8, device=DEV),
                    scales=torch.full((rows, 2, 4), 9, dtype=torch.uint8, device=DEV))
        o = mxk.mxfp8_swiglu_ckpt(poisoned.to(DEV), rows_dev=cnt, **bufs)
        for k in bufs:
            assert torch.equal(o[k][:n], full[k][:n]) and (o[k][n:] == (5 if k == "h" else 9)).all(), k
        dh13, h = torch.full((rows, 2 * F), 5.0, dtype=dt, device=DEV), torch.full((rows, F), 5.0, dtype=dt, device=DEV)
        g = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), full["codes"], full["scales"], rows_dev=cnt, dh13=dh13, h=h)
        ref = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), full["codes"], full["scales"])
        for k in ("dh13", "h"):
            assert torch.equal(g[k][:n], ref[k][:n]) and (g[k][n:] == 5).all(), k


def test_no_rows():
    o = mxk.mxfp8_swiglu_ckpt(torch.empty(0, 64, dtype=BF, device=DEV))
    assert o["h"].shape == (0, 32)
    g = mxk.mxfp8_swiglu_ckpt_bwd(torch.empty(0, 32, dtype=BF, device=DEV), o["codes"], o["scales"])
    assert g["dh13"].shape == (0, 64)


def test_large_gradients_of_far_gates():
    """dh up beyond fp32 where the gate's factor is zero or small: the gradients are what the formula gives, not NaN."""
    F = 32
    gates = torch.tensor([-3e38, -1e30, -200.0, -90.0, -60.0, -30.0, 0.0, 3.0])
    h13 = torch.cat([gates.unsqueeze(1).expand(8, F), torch.full((8, F), 2.0 ** 80)], dim=1).to(BF)
    dh = torch.full((8, F), 2.0 ** 60, dtype=BF)
    out = mxk.mxfp8_swiglu_ckpt(h13.to(DEV))
    got = mxk.mxfp8_swiglu_ckpt_bwd(dh.to(DEV), out["codes"], out["scales"])
    a, b = _kept(out["codes"], out["scales"], F)
    d, s = dh.double(), P.sigmoid(a)
    t = s * (1 + a * (1 - s))
    da, db = (d * t * b).to(BF).double(), (d * a * s).to(BF).double()
    # the sigmoid's own error and its flush below 2^-126 (S0), as above; beyond bf16's range: the same infinity
    r = P.sigmoid_err(a) + 2.0 ** -20
    for x, y, m, what in ((got["dh13"][:, :F], da, d * b, "da"), (got["dh13"][:, F:], db, d * a, "db")):
        x = x.cpu().double()
        assert not torch.isnan(x).any(), what
        big = ~torch.isfinite(y)
        assert torch.equal(x[big], y[big]), what
        # (the bracket's own relative error is up to |a| times the sigmoid's)
        e = torch.nan_to_num((2 * r * (1 + a.abs()) + 2 * P.u(BF)) * y.abs(), posinf=0.0) + S0 * (m.abs().clamp(max=2.0 ** 200) * (1 + a.abs().clamp(max=200.0)) + 1)
        P.assert_within(x[~big], y[~big], e[~big], what)
