"""The operators beside the MXFP8 path together: a training step of a routed-experts layer on unpadded segments with an 8-bit
checkpoint, then the same weights in 4 bits for single tokens.  Each link is checked on its own inputs."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _near(got, ref, mag, depth, what):
    s = depth * 2.0 ** -23 * mag
    P.assert_within(got, ref, P.u(BF) * (ref.abs() + s) + s + P.tiny(BF), what)


def test_training_step_and_decode():
    g = torch.Generator().manual_seed(1)
    T, k, E, D, F = 203, 2, 5, 256, 384
    w13 = (torch.randn(E, 2 * F, D, generator=g) * D ** -0.5).to(BF)
    w2 = (torch.randn(E, D, F, generator=g) * F ** -0.5).to(BF)
    x = torch.randn(T, D, generator=g).to(BF)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int()      # the last expert gets no token
    wt = torch.softmax(torch.randn(T, k, generator=g), dim=1)
    W13, W2, X = w13.to(DEV), w2.to(DEV), x.to(DEV)
    r = mxk.mxmoe_route(ids.to(DEV), E, 1, m_cap=T * k)
    off = r["offsets"]
    rows = X[(r["row_slot"] // k).long()]
    o = off.cpu()
    # forward
    h13 = mxk.mxmoe_ragged_gemm(rows, W13, off)
    _near(h13, *P.ragged(rows.cpu(), w13, o, False), D, "h13")
    f = mxk.mxfp8_swiglu_ckpt(h13, rows_dev=off[E:])
    y = mxk.mxmoe_ragged_gemm(f["h"], W2, off)
    _near(y, *P.ragged(f["h"].cpu(), w2, o, False), F, "y")
    out = mxk.mxmoe_unpermute_combine(y, r["slot_row"], k, weights=wt.to(DEV))
    # backward of sum(out * dout)
    dout = torch.randn(T, D, generator=g).to(BF).to(DEV)
    slot = r["row_slot"].long()
    dy = (dout[slot // k].float() * wt.to(DEV).reshape(-1)[slot].unsqueeze(1)).to(BF)
    dh = mxk.mxmoe_ragged_gemm(dy, W2, off, transpose_w=True)
    b = mxk.mxfp8_swiglu_ckpt_bwd(dh, f["codes"], f["scales"], rows_dev=off[E:])
    dw2 = mxk.mxmoe_ragged_gemm_wgrad(dy, b["h"], off)
    dx = mxk.mxmoe_ragged_gemm(b["dh13"], W13, off, transpose_w=True)
    dw13 = mxk.mxmoe_ragged_gemm_wgrad(b["dh13"], rows, off)
    depth = int((o[1:] - o[:-1]).max())
    _near(dh, *P.ragged(dy.cpu(), w2, o, True), D, "dh")
    _near(dw2, *P.wgrad(dy.cpu(), b["h"].cpu(), o), depth, "dw2")
    _near(dx, *P.ragged(b["dh13"].cpu(), w13, o, True), 2 * F, "dx")
    _near(dw13, *P.wgrad(b["dh13"].cpu(), rows.cpu(), o), depth, "dw13")
    assert (dw2[E - 1] == 0).all() and (dw13[E - 1] == 0).all()
    dxt = mxk.mxmoe_unpermute_combine(dx, r["slot_row"], k)
    assert out.shape == dxt.shape == (T, D) and torch.isfinite(out.float()).all() and torch.isfinite(dxt.float()).all()
    # a few of the tokens through the 4-bit copy: what the ragged products give on the values that it stands for
    qw = mxk.mxfp4_quantize_experts(W13, W2)
    v13, v2 = ((lambda q: mxk.mxfp4_dequantize(q["codes"], q["scales"]))(mxk.mxfp4_quantize(w)) for w in (W13, W2))
    n = 3
    d = mxk.moe_layer_decode_fp4(X[:n].contiguous(), ids[:n].to(DEV), wt[:n].to(DEV), qw).cpu().double()
    for t in range(n):
        ref = torch.zeros(D, dtype=torch.float64)
        mag = torch.zeros(D, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            z = v13[e].cpu().double() @ x[t].double()
            h = z[:F] * P.sigmoid(z[:F]) * z[F:]
            ref += wt[t, j].double() * (v2[e].cpu().double() @ h)
            # h: f16's half step, and fp32's sums of D products through both factors (a generous 2 D 2^-23 of the magnitudes)
            zm = v13[e].cpu().double().abs() @ x[t].double().abs()
            eh = 2.0 ** -11 * h.abs() + 2 * D * 2.0 ** -23 * (zm[:F] * z[F:].abs() + z[:F].abs() * zm[F:] + zm[:F] * zm[F:] * D * 2.0 ** -23) + 2.0 ** -30
            mag += wt[t, j].double() * (v2[e].cpu().double().abs() @ (eh + F * 2.0 ** -23 * h.abs()))
        P.assert_within(d[t], ref, mag * 1.1 + P.u(BF) * (ref.abs() + mag) + P.tiny(BF), f"decode of token {t}")
    assert mxk.device_error() == 0


def test_step_captured_while_an_eager_step_lives():
    """The chain captured into a graph beside buffers of an eager run, replayed on new rows: the same as an eager run."""
    g = torch.Generator(device=DEV).manual_seed(2)
    E, D, F, R = 3, 128, 64, 90
    off = P.offsets_of([40, 0, 50]).to(DEV)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g).to(BF)  # noqa: E731
    w13, w2, x, dy = rn(E, 2 * F, D), rn(E, D, F), rn(R, D), rn(R, D)

    def step():
        h13 = mxk.mxmoe_ragged_gemm(x, w13, off)
        f = mxk.mxfp8_swiglu_ckpt(h13)
        y = mxk.mxmoe_ragged_gemm(f["h"], w2, off)
        dh = mxk.mxmoe_ragged_gemm(dy, w2, off, transpose_w=True)
        b = mxk.mxfp8_swiglu_ckpt_bwd(dh, f["codes"], f["scales"])
        return (y, mxk.mxmoe_ragged_gemm(b["dh13"], w13, off, transpose_w=True), mxk.mxmoe_ragged_gemm_wgrad(dy, b["h"], off),
                mxk.mxmoe_ragged_gemm_wgrad(b["dh13"], x, off))

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    x.copy_(rn(R, D))
    off.copy_(torch.tensor([0, 13, 60, 90], dtype=torch.int32))
    graph.replay()
    fresh = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fresh, captured))
    assert np.isfinite(fresh[0].float().cpu().numpy()).all()
