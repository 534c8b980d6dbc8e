"""The operators beside the MXFP8 path refuse bad arguments on the host (no GPU needed), and their plain forms agree with facts."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P16

P = ctypes.c_void_p
FAKE = 0x10000          # aligned dummy device address: never dereferenced on the paths below
MIS = 0x10008           # misaligned


@pytest.fixture(scope="module")
def L():
    return mxk.lib()


def _err(L):
    return L.mxmoe_last_error_message().decode()


def test_ragged_refusals(L):
    ok = dict(a=FAKE, M=10, w=FAKE, E=2, N=16, K=24, off=FAKE, tr=0, dt=0, out=FAKE, ws=None, n=0)

    def call(**kw):
        v = {**ok, **kw}
        return L.mxmoe_ragged_gemm(v["a"], v["M"], v["w"], v["E"], v["N"], v["K"], v["off"], v["tr"], v["dt"], v["out"], v["ws"], v["n"], None)

    for kw, status, word in ((dict(N=12), 2, "N=12"), (dict(K=0), 2, "K=0"), (dict(M=-1), 2, "M=-1"), (dict(M=(1 << 31) - 1023), 2, "M="),
                             (dict(E=0), 2, "E=0"), (dict(E=1025), 2, "E=1025"), (dict(off=None), 1, "expert_offsets"),
                             (dict(a=None), 1, "a is NULL"), (dict(w=MIS), 3, "w is not"), (dict(out=MIS), 3, "out is not"),
                             (dict(dt=2), 9, "dtype=2"), (dict(tr=3), 9, "transpose_w=3"), (dict(N=1 << 30), 2, "2^30")):
        assert call(**kw) == status and word in _err(L), kw
    assert call(M=0) == 0                                          # nothing to do, nothing touched


def test_ragged_workspace_arithmetic(L):
    f = L.mxmoe_ragged_workspace_size
    assert f(49152, 2816, 2048, 64, 0) == 0 and f(49152, 2816, 2048, 64, 2) == 0        # tiles enough
    assert f(10, 16, 24, 2, 0) == 0 and f(64, 16, 24, 1, 2) == 0                          # a short contraction
    assert f(128, 2048, 7168, 1, 0) == 256 + 9 * 128 * 2048 * 4                           # 8 tiles: 74 / 8 units each
    assert f(128, 2048, 7168, 1, 1) == 0                                                  # 32 blocks: not worth a launch
    assert f(128, 4096, 7168, 1, 1) == 256 + 2 * 128 * 7168 * 4                           # 28 tiles, 64 blocks
    assert f(31134, 24, 704, 1, 2) == 256 + 24 * 24 * 704 * 4                             # 3 tiles, 487 blocks
    s = L.mxmoe_ragged_gemm(FAKE, 128, FAKE, 1, 2048, 7168, FAKE, 0, 0, FAKE, FAKE, 1000, None)
    assert s == 8 and "workspace of 1000 bytes" in _err(L)
    s = L.mxmoe_ragged_gemm(FAKE, 128, FAKE, 1, 2048, 7168, FAKE, 0, 0, FAKE, MIS, 1 << 30, None)
    assert s == 3 and "workspace is not" in _err(L)
    s = L.mxmoe_ragged_gemm_wgrad(FAKE, 24, FAKE, 704, 31134, FAKE, 1, 0, FAKE, FAKE, 1000, None)
    assert s == 8
    assert f(0, 16, 24, 1, 0) == 0 and f(10, 16, 24, 0, 0) == 0 and f(10, 16, 24, 1, 3) == 0


def test_ragged_workspace_of_refused_sizes_is_zero(L):
    f = L.mxmoe_ragged_workspace_size
    assert f(4096, 24, 72, 1024, 2) >= 0
    for M, N, K, E, which in ((4096, 24, 72, 1025, 2), ((1 << 31) + 1, 24, 72, 1, 2), (4096, 1 << 30, 72, 1, 2), (4096, 24, 1 << 30, 1, 2),
                              (4096, (1 << 30) - 8, (1 << 30) - 8, (1 << 31) - 1, 2), (4096, 24, 72, 1, 3), (4096, 24, 72, 0, 2), (-1, 24, 72, 1, 2)):
        assert f(M, N, K, E, which) == 0, (M, N, K, E, which)


def test_ragged_wgrad_refusals(L):
    ok = dict(g=FAKE, N=16, a=FAKE, K=24, M=10, off=FAKE, E=2, dt=1, out=FAKE)

    def call(**kw):
        v = {**ok, **kw}
        return L.mxmoe_ragged_gemm_wgrad(v["g"], v["N"], v["a"], v["K"], v["M"], v["off"], v["E"], v["dt"], v["out"], None, 0, None)

    for kw, status, word in ((dict(N=4), 2, "N=4"), (dict(K=28), 2, "K=28"), (dict(E=-3), 2, "E=-3"), (dict(off=None), 1, "expert_offsets"),
                             (dict(g=None), 1, "g is NULL"), (dict(a=MIS), 3, "a is not"), (dict(out=None), 1, "dw is NULL"), (dict(dt=-1), 9, "dtype=-1")):
        assert call(**kw) == status and word in _err(L), kw


def test_ckpt_refusals(L):
    f = lambda h13=FAKE, rows=4, F=16, dt=0, h=FAKE, c=FAKE, s=FAKE: L.mxfp8_swiglu_ckpt(h13, rows, F, None, dt, h, c, s, None)  # noqa: E731
    b = lambda dh=FAKE, c=FAKE, s=FAKE, rows=4, F=16, dt=0, g=FAKE, h=None: L.mxfp8_swiglu_ckpt_bwd(dh, c, s, rows, F, None, dt, g, h, None)  # noqa: E731
    for st, status, word in ((lambda: f(F=12), 2, "F=12"), (lambda: f(rows=-1), 2, "rows=-1"), (lambda: f(dt=5), 9, "dtype"), (lambda: f(h13=None), 1, "h13"),
                             (lambda: f(h=MIS), 3, "h is not"), (lambda: f(c=MIS), 3, "codes"), (lambda: f(s=None), 1, "scales"), (lambda: f(F=1 << 28), 2, "too large"),
                             (lambda: f(rows=1 << 62), 2, "too large"), (lambda: b(F=4), 2, "F=4"), (lambda: b(dh=MIS), 3, "dh"), (lambda: b(g=None), 1, "dh13"),
                             (lambda: b(h=MIS), 3, "h is not"), (lambda: b(s=None), 1, "scales")):
        assert st() == status and word in _err(L), word
    assert f(rows=0) == 0 and b(rows=0) == 0


def test_fp4_refusals(L):
    q = lambda x=FAKE, b=1, r=16, c=128, dt=0, lay=0, k=FAKE, s=FAKE: L.mxfp4_quantize(x, b, r, c, dt, lay, k, s, None)  # noqa: E731
    d = lambda k=FAKE, s=FAKE, r=4, c=64, dt=0, o=FAKE: L.mxfp4_dequantize(k, s, r, c, dt, o, None)  # noqa: E731
    m = lambda x=FAKE, S=2, K=128, i=FAKE, k=FAKE, s=FAKE, E=2, N=16, dt=0, y=FAKE: L.mxfp4_expert_matvec(x, S, K, i, k, s, E, N, dt, y, None)  # noqa: E731
    for st, status, word in ((lambda: q(c=48), 2, "cols=48"), (lambda: q(lay=1, c=96), 2, "cols=96"), (lambda: q(lay=2, r=24), 2, "rows=24"), (lambda: q(lay=3), 9, "layout=3"),
                             (lambda: q(b=0), 2, "batch=0"), (lambda: q(dt=7), 9, "dtype"), (lambda: q(x=None), 1, "x is NULL"), (lambda: q(k=MIS), 3, "codes"),
                             (lambda: q(r=1 << 58), 2, "too large"), (lambda: d(c=16), 2, "cols=16"), (lambda: d(o=MIS), 3, "out"), (lambda: d(r=0), 2, "rows=0"),
                             (lambda: m(K=64), 2, "K=64"), (lambda: m(N=8), 2, "N=8"), (lambda: m(S=2049), 2, "2049 slots"), (lambda: m(S=-1), 2, "slots"),
                             (lambda: m(E=1025), 2, "E=1025"), (lambda: m(i=None), 1, "expert_ids"), (lambda: m(x=MIS), 3, "x is not"), (lambda: m(K=1 << 20), 2, "shared memory")):
        assert st() == status and word in _err(L), word
    assert m(S=0) == 0


def test_decode_refusals(L):
    qw = mxk._Q4Weights(FAKE, FAKE, FAKE, FAKE)
    T, k, D, F, E = 4, 2, 256, 128, 4
    need = L.mxfp4_decode_workspace_size(T, k, D, F)
    assert need >= T * k * (D + F) * 4
    assert L.mxfp4_decode_workspace_size(0, k, D, F) == 0 and L.mxfp4_decode_workspace_size(1 << 40, 1 << 30, D, F) == 0

    def call(x=FAKE, T=T, D=D, ids=FAKE, w=FAKE, k=k, q=ctypes.byref(qw), E=E, F=F, dt=0, o=FAKE, ws=FAKE, n=need):
        return L.moe_layer_decode_fp4(x, T, D, ids, w, k, q, E, F, dt, o, ws, n, None)

    bad = mxk._Q4Weights(FAKE, FAKE, MIS, FAKE)
    for kw, status, word in ((dict(D=192), 2, "D=192"), (dict(F=64), 2, "F=64"), (dict(k=5), 2, "top_k=5"), (dict(T=2000), 2, "slots"), (dict(T=-1), 2, "T=-1"),
                             (dict(dt=2), 9, "dtype"), (dict(x=None), 1, "x_tokens"), (dict(o=MIS), 3, "out_tokens"), (dict(ids=None), 1, "topk_ids"),
                             (dict(q=None), 1, "qweights"), (dict(q=ctypes.byref(bad)), 3, "w2_codes"), (dict(ws=None), 8, "workspace"), (dict(n=need - 1), 8, "workspace")):
        assert call(**kw) == status and word in _err(L), kw
    assert call(T=0) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: mxk.mxmoe_ragged_gemm(x, x, x), lambda: mxk.mxfp8_swiglu_ckpt(x), lambda: mxk.mxfp4_quantize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        mxk.mxfp4_quantize(x.float())
    with pytest.raises(TypeError, match="a must be a torch.Tensor"):
        mxk.mxmoe_ragged_gemm([1.0], x, x)
    with pytest.raises(TypeError, match="dtype"):
        mxk.mxfp4_dequantize(x, x, dtype=torch.float32)


def test_plain_forms_against_known_values():
    # OCP MX: 6 is E2M1's largest value, ties go to the even code, the scale is the largest power of two below the maximum / 4
    x = np.zeros((1, 32))
    x[0, :8] = [6, 5, 2.5, 0.25, 0.75, -3.5, 7, 0.2]
    code, byte = P16.fp4(x)
    assert byte[0, 0] == 127 and code[0, :8].tolist() == [7, 6, 4, 0, 2, 14, 7, 0]
    assert P16.fp4_values(code, byte)[0, :8].tolist() == [6, 4, 2, 0, 1, -4, 6, 0]
    c, b = P16.e4m3(np.array([[448.0, 464.0, -1.0, 2.0 ** -9]]))
    assert b[0, 0] == 127 and c[0].tolist() == [0x7E, 0x7E, 0xB8, 0x01]
    iw, isc = P16.fp4_tile_index(32, 256, False)
    assert sorted(iw.reshape(-1).tolist()) == list(range(32 * 32)) and sorted(isc.reshape(-1).tolist()) == list(range(32 * 8))


def test_decode_sizes_that_shared_memory_holds(L):
    """h goes in as two f16 pieces: fp16 layers are refused where a row of them does not fit, bf16 layers take one piece there."""
    qw = mxk._Q4Weights(FAKE, FAKE, FAKE, FAKE)
    f = lambda F, dt: L.moe_layer_decode_fp4(FAKE, 1, 128, FAKE, FAKE, 1, ctypes.byref(qw), 1, F, dt, FAKE, None, 0, None)  # noqa: E731
    assert f(36224, 0) == f(36224, 1) == 8 and "workspace" in _err(L)          # fits; the workspace is missing
    assert f(36352, 1) == 2 and "shared memory" in _err(L)
    assert f(36352, 0) == 8 and f(72448, 0) == 8
    assert f(72576, 0) == 2 and "shared memory" in _err(L)


def test_matvec_sizes_that_shared_memory_holds(L):
    """The header's limits on K: at the largest S and E, and at one."""
    f = lambda K, S, E: L.mxfp4_expert_matvec(None, S, K, FAKE, FAKE, FAKE, E, 16, 0, FAKE, None)  # noqa: E731
    for K, S, E in ((54016, 2048, 1024), (72448, 1, 1)):
        assert f(K, S, E) == 1 and "x is NULL" in _err(L)          # fits; refused for its pointer
        assert f(K + 128, S, E) == 2 and "shared memory" in _err(L)
