"""GPU tests of the 4-bit weight cast, the routed matrix-vector product and the decode layer."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])


def _np(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------------------------------------ cast
@DTYPES
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (257, 352), (2, 5, 64), (3, 128, 256)])
def test_cast_and_back(shape, dt):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(*shape, generator=g).to(dt)
    q = mxk.mxfp4_quantize(w.to(DEV))
    assert q["codes"].shape == (*shape[:-1], shape[-1] // 2) and q["scales"].shape == (*shape[:-1], shape[-1] // 32)
    code, byte = P.fp4(_np(w).reshape(-1, shape[-1]))
    got = P.fp4_unpack(q["codes"].cpu().numpy().reshape(-1, shape[-1] // 2))
    assert np.array_equal(got, code) and np.array_equal(q["scales"].cpu().numpy().reshape(byte.shape), byte)
    back = mxk.mxfp4_dequantize(q["codes"], q["scales"], dtype=dt)
    assert back.shape == shape
    P.assert_same(back.reshape(-1, shape[-1]), torch.from_numpy(P.fp4_values(code, byte)).to(dt), "values")


@DTYPES
def test_cast_over_the_types_range_and_ties(dt):
    lo, hi = (-133, 127) if dt == BF else (-24, 15)
    rows = []
    for e in range(lo, hi + 1):
        # half-way values, their neighbours and the largest ones
        v = np.array([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 4.0, 0.24, 0.26, 1.24, 1.26] * 2) * 2.0 ** (e - 2)
        rows.append(np.where(np.arange(32) >= 16, -v, v))
    w = torch.tensor(np.stack(rows)).to(dt)
    w[~torch.isfinite(w)] = 0
    q = mxk.mxfp4_quantize(w.to(DEV))
    code, byte = P.fp4(_np(w))
    assert np.array_equal(q["scales"].cpu().numpy(), byte)
    assert np.array_equal(P.fp4_unpack(q["codes"].cpu().numpy()), code)
    P.assert_same(mxk.mxfp4_dequantize(q["codes"], q["scales"], dtype=dt), torch.from_numpy(P.fp4_values(code, byte)).to(dt), "values")


@DTYPES
def test_cast_of_nan_and_infinity(dt):
    w = torch.ones(4, 64, dtype=dt)
    w[0, 5], w[1, 40], w[2, 0] = float("nan"), float("inf"), float("-inf")
    q = mxk.mxfp4_quantize(w.to(DEV))
    assert q["scales"].cpu().tolist() == [[255, 125], [125, 255], [255, 125], [125, 125]]
    back = mxk.mxfp4_dequantize(q["codes"], q["scales"], dtype=dt).cpu()
    bad = torch.zeros(4, 64, dtype=torch.bool)
    bad[0, :32], bad[1, 32:], bad[2, :32] = True, True, True
    assert torch.equal(torch.isnan(back), bad) and (back[~bad] == 1).all()


def test_decode_of_every_code_and_byte():
    codes = torch.arange(256, dtype=torch.uint8).reshape(16, 16).repeat(256, 1)          # every byte under every scale byte
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).reshape(-1, 1)
    v = P.fp4_values(P.fp4_unpack(codes.numpy()), scales.numpy().astype(np.int64))
    for dt in (BF, FP):
        P.assert_same(mxk.mxfp4_dequantize(codes.to(DEV), scales.to(DEV), dtype=dt), torch.from_numpy(v).to(torch.float32).to(dt)
                      if dt == FP else torch.from_numpy(v).to(dt), "values")


@DTYPES
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,R,K", [(1, 16, 128), (3, 48, 384), (2, 256, 256)])
def test_tile_layouts(E, R, K, gated, dt):
    g = torch.Generator().manual_seed(2)
    w = torch.randn(E, R, K, generator=g).to(DEV, dt)
    plain, tile = mxk.mxfp4_quantize(w), mxk.mxfp4_quantize(w, mxk.TILE_GATED if gated else mxk.TILE)
    iw, isc = P.fp4_tile_index(R, K, gated)
    assert len(np.unique(iw)) == iw.size and len(np.unique(isc)) == isc.size
    for e in range(E):
        words = tile["codes"][e].cpu().numpy().reshape(-1).view(np.uint32)
        assert np.array_equal(words[iw], plain["codes"][e].cpu().numpy().view(np.uint32))
        assert np.array_equal(tile["scales"][e].cpu().numpy().reshape(-1)[isc], plain["scales"][e].cpu().numpy())


# ------------------------------------------------------------------------------------------------ matvec
def _weights(r, E, N, K, lo=120, hi=126):
    """Random codes and scale bytes: packed PLAIN, and float64 values."""
    codes = r.integers(0, 16, size=(E, N, K))
    byte = r.integers(lo, hi + 1, size=(E, N, K // 32))
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    return packed, byte.astype(np.uint8), torch.from_numpy(P.fp4_values(codes, byte))


def _tiled(packed, byte, gated):
    E, R, h = packed.shape
    iw, isc = P.fp4_tile_index(R, 2 * h, gated)
    c, s = np.empty((E, R * h // 4), np.uint32), np.empty((E, byte[0].size), np.uint8)
    for e in range(E):
        c[e][iw] = np.ascontiguousarray(packed[e]).view(np.uint32)
        s[e][isc] = byte[e]
    return torch.from_numpy(c.view(np.uint8).reshape(packed.shape)).to(DEV), torch.from_numpy(s.reshape(byte.shape)).to(DEV)


@DTYPES
@pytest.mark.parametrize("S,E,N,K", [(1, 1, 16, 128), (3, 4, 48, 256), (8, 2, 32, 384), (9, 1, 16, 128), (30, 3, 64, 2176),
                                     (17, 5, 16, 4096), (5, 2, 80, 16384), (70, 1024, 16, 128)])
def test_matvec_of_whole_numbers_is_exact(S, E, N, K, dt):
    """Whole activations and scales of one power: every product and sum is exact in fp32."""
    r = np.random.default_rng(3)
    packed, byte, w = _weights(r, E, N, K, lo=127, hi=128)
    ids = r.integers(0, E, size=S).astype(np.int32)
    x = torch.from_numpy(r.integers(-3, 4, size=(S, K)).astype(np.float64))
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x.to(DEV, dt), torch.from_numpy(ids).to(DEV), c, s)
    ref = torch.stack([w[ids[i]] @ x[i] for i in range(S)])
    P.assert_same(y, ref.to(dt), "y")
    assert mxk.device_error() == 0


@DTYPES
@pytest.mark.parametrize("spread", [0, 30])
def test_matvec_within_the_bound(spread, dt):
    """Normal activations over many powers of two.  Off by one rounding, fp32's sums, and what f16 cuts off below 2^-37 of a
    row's largest value."""
    r = np.random.default_rng(4)
    S, E, N, K = 11, 3, 32, 1024
    packed, byte, w = _weights(r, E, N, K)
    ids = r.integers(0, E, size=S).astype(np.int32)
    sc = np.ldexp(1.0, r.integers(-spread // (2 if dt == FP else 1), 1, size=(S, K))) if spread else 1.0
    x = torch.from_numpy(r.standard_normal((S, K)) * sc).to(dt)
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x.to(DEV), torch.from_numpy(ids).to(DEV), c, s)
    xd = x.double()
    ref = torch.stack([w[ids[i]] @ xd[i] for i in range(S)])
    mag = torch.stack([w[ids[i]].abs() @ xd[i].abs() for i in range(S)])
    cut = torch.stack([w[ids[i]].abs().sum(1) * xd[i].abs().max() * 2.0 ** -37 for i in range(S)])
    e = K * 2.0 ** -23 * mag + cut
    P.assert_within(y, ref, e + P.u(dt) * (ref.abs() + e) + P.tiny(dt), "y")


def test_matvec_scale_bytes_at_their_ends():
    """Byte 0 is 2^-127 and byte 255 NaN; a NaN block reaches its own row only."""
    r = np.random.default_rng(5)
    packed, byte, _ = _weights(r, 1, 16, 128, lo=127, hi=127)
    byte[0, 3, 1], byte[0, 5] = 255, 0
    x = torch.ones(1, 128, dtype=BF, device=DEV)
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x, torch.zeros(1, dtype=torch.int32, device=DEV), c, s).cpu()[0]
    assert torch.isnan(y).tolist() == [i == 3 for i in range(16)]
    ref = P.fp4_values(P.fp4_unpack(packed[0, 5]), np.zeros(4, np.int64)).sum()
    assert abs(float(y[5]) - ref) <= abs(ref) * 2.0 ** -8 + 2.0 ** -133


@DTYPES
def test_matvec_nan_and_infinite_activations_stay_in_their_row(dt):
    r = np.random.default_rng(6)
    packed, byte, _ = _weights(r, 2, 16, 256, lo=127, hi=127)
    packed[packed == 0] = 0x11
    w = torch.from_numpy(P.fp4_values(P.fp4_unpack(packed), byte.astype(np.int64)))
    ids = torch.tensor([0, 1, 0], dtype=torch.int32)
    x = torch.from_numpy(r.integers(-3, 4, size=(3, 256)).astype(np.float64)).to(dt)
    bad = x.clone()
    bad[0, 7], bad[1, 100] = float("nan"), float("inf")
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(bad.to(DEV), ids.to(DEV), c, s).cpu()
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[1]).any()
    P.assert_same(y[2:], (w[0] @ x[2].double()).to(dt).unsqueeze(0), "clean row")


def test_matvec_bad_ids_are_reported_and_left():
    r = np.random.default_rng(7)
    packed, byte, w = _weights(r, 2, 16, 128, lo=127, hi=127)
    c, s = _tiled(packed, byte, False)
    x = torch.ones(4, 128, dtype=BF, device=DEV)
    out = torch.full((4, 16), 3.0, dtype=BF, device=DEV)
    mxk.mxfp4_expert_matvec(x, torch.tensor([1, -1, 2, 0], dtype=torch.int32, device=DEV), c, s, out=out)
    assert mxk.device_error() == 9
    y = out.cpu()
    assert (y[1:3] == 3).all()
    for i, e in ((0, 1), (3, 0)):
        P.assert_same(y[i], w[e].sum(1).to(BF), "row")
    mxk.mxfp4_expert_matvec(x[:0], torch.empty(0, dtype=torch.int32, device=DEV), c, s)
    assert mxk.device_error() == 0


# ------------------------------------------------------------------------------------------------ decode layer
def _layer(r, T, k, E, D, F, dt, distinct=True):
    p13, b13, w13 = _weights(r, E, 2 * F, D, lo=118, hi=121)
    p2, b2, w2 = _weights(r, E, D, F, lo=118, hi=121)
    ids = np.stack([r.permutation(E)[:k] if distinct else r.integers(0, E, size=k) for _ in range(T)]).astype(np.int32)
    x = torch.from_numpy(r.standard_normal((T, D))).to(dt)
    wt = torch.from_numpy(r.random((T, k))).float()
    t13, t2 = _tiled(p13, b13, True), _tiled(p2, b2, False)
    qw = dict(w13_codes=t13[0], w13_scales=t13[1], w2_codes=t2[0], w2_scales=t2[1])
    return qw, w13, w2, torch.from_numpy(ids), x, wt


def _layer_ref(w13, w2, ids, x, wt, dt):
    """(result, bound): f16's half step on h (fp16 layers: of its second piece), fp32's sums in both products and the combine,
    one rounding."""
    T, k = ids.shape
    F = w2.shape[2]
    out, err = torch.zeros(T, x.shape[1], dtype=torch.float64), torch.zeros(T, x.shape[1], dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            z = w13[e] @ x[t].double()
            zm = (w13[e].abs() @ x[t].double().abs()) * x.shape[1] * 2.0 ** -23 + (w13[e].abs().sum(1)) * x[t].double().abs().max() * 2.0 ** -37
            a, b, ea, eb = z[:F], z[F:], zm[:F], zm[F:]
            s = P.sigmoid(a)
            h = a * s * b
            # |d silu / da| <= 1.1; the sigmoid's own error; products
            eh = 1.1 * ea * (b.abs() + eb) + (a * s).abs() * eb + (P.sigmoid_err(a) + 2.0 ** -22) * h.abs()
            eh = eh + 2.0 ** (-11 if dt == BF else -22) * (h.abs() + eh) + h.abs().max() * 2.0 ** -37
            y = w2[e] @ h
            m = w2[e].abs() @ (h.abs() + eh)
            out[t] += wt[t, j].double() * y
            err[t] += wt[t, j].double().abs() * (w2[e].abs() @ eh + (F + k + 2) * 2.0 ** -23 * m)
    return out, err + P.u(dt) * (out.abs() + err) + P.tiny(dt)


@DTYPES
@pytest.mark.parametrize("T,k,E,D,F", [(1, 1, 1, 128, 128), (1, 6, 8, 256, 128), (5, 3, 4, 384, 256), (13, 2, 2, 128, 384), (40, 8, 64, 128, 128)])
def test_decode_layer(T, k, E, D, F, dt):
    qw, w13, w2, ids, x, wt = _layer(np.random.default_rng(8), T, k, E, D, F, dt)
    out = mxk.moe_layer_decode_fp4(x.to(DEV), ids.to(DEV), wt.to(DEV), qw)
    ref, bound = _layer_ref(w13, w2, ids, x, wt, dt)
    P.assert_within(out, ref, bound, "out")
    assert mxk.device_error() == 0


def test_decode_layer_with_repeated_and_bad_ids():
    qw, w13, w2, ids, x, wt = _layer(np.random.default_rng(9), 6, 3, 4, 128, 128, BF, distinct=False)
    ids[0] = 2                                                     # one expert three times
    ref, bound = _layer_ref(w13, w2, ids, x, wt, BF)
    P.assert_within(mxk.moe_layer_decode_fp4(x.to(DEV), ids.to(DEV), wt.to(DEV), qw), ref, bound, "repeated")
    bad = ids.clone()
    bad[1, 1], bad[2] = 4, -7
    zeroed = wt.clone()
    zeroed[1, 1], zeroed[2] = 0, 0
    safe = bad.clone()
    safe[1, 1], safe[2] = 0, 0
    ref, bound = _layer_ref(w13, w2, safe, x, zeroed, BF)
    out = mxk.moe_layer_decode_fp4(x.to(DEV), bad.to(DEV), wt.to(DEV), qw)
    assert mxk.device_error() == 9
    P.assert_within(out, ref, bound, "bad ids add nothing")
    assert (out[2] == 0).all()


def test_decode_layer_captured_with_its_own_workspaces():
    """Two graphs with a workspace each, replayed on two streams at once, on new inputs."""
    T, k, E, D, F = 3, 2, 4, 256, 128
    jobs = []
    for seed in (10, 11):
        qw, w13, w2, ids, x, wt = _layer(np.random.default_rng(seed), T, k, E, D, F, BF)
        n = mxk.lib().mxfp4_decode_workspace_size(T, k, D, F)
        j = dict(qw=qw, w13=w13, w2=w2, ids=ids.to(DEV), x=x.to(DEV), wt=wt.to(DEV), out=torch.zeros(T, D, dtype=BF, device=DEV),
                 ws=torch.empty(n, dtype=torch.uint8, device=DEV), s=torch.cuda.Stream())
        run = lambda j=j: mxk.moe_layer_decode_fp4(j["x"], j["ids"], j["wt"], j["qw"], out=j["out"], workspace=j["ws"])  # noqa: E731
        run()
        torch.cuda.synchronize()
        j["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(j["graph"]):
            run()
        j["x"].copy_(j["x"].roll(1, 0)), j["ids"].copy_(j["ids"].flip(0))
        jobs.append(j)
    torch.cuda.synchronize()
    for _ in range(4):
        for j in jobs:
            with torch.cuda.stream(j["s"]):
                j["graph"].replay()
    torch.cuda.synchronize()
    for j in jobs:
        ref, bound = _layer_ref(j["w13"], j["w2"], j["ids"].cpu(), j["x"].cpu(), j["wt"].cpu(), BF)
        P.assert_within(j["out"], ref, bound, "replayed")


def test_decode_layer_from_16_bit_weights_next_to_the_cast():
    """mxfp4_quantize_experts feeds the layer: the same as the matvecs on the weights that the cast gives back."""
    g = torch.Generator().manual_seed(12)
    E, D, F, T, k = 3, 256, 128, 4, 2
    w13 = (torch.randn(E, 2 * F, D, generator=g) * D ** -0.5).to(BF).to(DEV)
    w2 = (torch.randn(E, D, F, generator=g) * F ** -0.5).to(BF).to(DEV)
    qw = mxk.mxfp4_quantize_experts(w13, w2)
    v13, v2 = ((lambda q: mxk.mxfp4_dequantize(q["codes"], q["scales"]))(mxk.mxfp4_quantize(w)).cpu().double() for w in (w13, w2))
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    x, wt = torch.randn(T, D, generator=g).to(BF), torch.rand(T, k, generator=g)
    ref, bound = _layer_ref(v13, v2, ids, x, wt, BF)
    P.assert_within(mxk.moe_layer_decode_fp4(x.to(DEV), ids.to(DEV), wt.to(DEV), qw), ref, bound, "out")


def test_decode_layer_without_tokens():
    qw = _layer(np.random.default_rng(13), 1, 1, 2, 128, 128, BF)[0]
    out = mxk.moe_layer_decode_fp4(torch.empty(0, 128, dtype=BF, device=DEV), torch.empty(0, 1, dtype=torch.int32, device=DEV),
                                   torch.empty(0, 1, device=DEV), qw)
    assert out.shape == (0, 128)


@pytest.mark.parametrize("S,E,N,K", [(300, 2, 128, 128), (320, 64, 128, 256), (2048, 3, 32, 128)])
def test_matvec_with_many_groups_of_an_expert(S, E, N, K):
    """An expert's slots fill many groups whose tiles are spread over blocks: all blocks must group them alike."""
    r = np.random.default_rng(14)
    packed, byte, w = _weights(r, E, N, K, lo=127, hi=128)
    ids = r.integers(0, E, size=S).astype(np.int32)
    x = torch.from_numpy(r.integers(-3, 4, size=(S, K)).astype(np.float64))
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x.to(DEV, BF), torch.from_numpy(ids).to(DEV), c, s)
    P.assert_same(y, torch.stack([w[ids[i]] @ x[i] for i in range(S)]).to(BF), "y")


# ------------------------------------------------------------------------------------------------ refusals of the bindings
def test_bindings_refuse_wrong_tensors():
    g = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    u8 = lambda *s: g(*s, dt=torch.uint8)  # noqa: E731
    i32 = lambda *s: g(*s, dt=torch.int32)  # noqa: E731
    qw = dict(w13_codes=u8(2, 256, 64), w13_scales=u8(2, 256, 4), w2_codes=u8(2, 128, 64), w2_scales=u8(2, 128, 4))
    x, ids, wt = g(3, 128), i32(3, 2), torch.zeros(3, 2, device=DEV)
    cases = [
        (ValueError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 24), off)),                       # K differs
        (ValueError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(3, 8, 16), off)),                       # E differs
        (TypeError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 16, dt=FP), off)),                 # types differ
        (TypeError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 16), off.long())),
        (TypeError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 16), None)),
        (ValueError, lambda: mxk.mxmoe_ragged_gemm(g(4, 32)[:, ::2], g(2, 8, 16), off)),               # not contiguous
        (ValueError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 16), off, out=g(4, 16))),
        (ValueError, lambda: mxk.mxmoe_ragged_gemm(g(4, 16), g(2, 8, 16), off.cpu())),
        (mxk.MXMOEError, lambda: mxk.mxmoe_ragged_gemm(g(4, 12), g(2, 8, 12), off)),
        (mxk.MXMOEError, lambda: mxk.mxmoe_ragged_gemm(g(65)[1:].view(4, 16), g(2, 8, 16), off)),      # not 16-byte aligned
        (ValueError, lambda: mxk.mxmoe_ragged_gemm_wgrad(g(4, 16), g(5, 8), off)),
        (ValueError, lambda: mxk.mxfp8_swiglu_ckpt(g(4, 15))),
        (mxk.MXMOEError, lambda: mxk.mxfp8_swiglu_ckpt(g(4, 24))),
        (TypeError, lambda: mxk.mxfp8_swiglu_ckpt_bwd(g(4, 16), None, None)),
        (ValueError, lambda: mxk.mxfp8_swiglu_ckpt_bwd(g(4, 16), u8(4, 32), u8(4, 2))),
        (mxk.MXMOEError, lambda: mxk.mxfp4_quantize(g(4, 48))),
        (mxk.MXMOEError, lambda: mxk.mxfp4_quantize(g(24, 128), mxk.TILE)),
        (ValueError, lambda: mxk.mxfp4_dequantize(u8(4, 32), u8(4, 3))),
        (ValueError, lambda: mxk.mxfp4_expert_matvec(x, i32(4), u8(2, 16, 64), u8(2, 16, 4))),
        (ValueError, lambda: mxk.mxfp4_expert_matvec(x, i32(3), u8(2, 16, 32), u8(2, 16, 4))),
        (ValueError, lambda: mxk.moe_layer_decode_fp4(x, i32(2, 2), wt, qw)),
        (ValueError, lambda: mxk.moe_layer_decode_fp4(x, ids, wt[:, :1].contiguous(), qw)),
        (mxk.MXMOEError, lambda: mxk.moe_layer_decode_fp4(x, ids, wt, qw, workspace=u8(16))),
        (ValueError, lambda: mxk.mxfp4_quantize_experts(g(2, 256, 128), g(2, 128, 256))),
    ]
    for i, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            pytest.fail(f"case {i} was accepted")
    assert mxk.device_error() == 0
