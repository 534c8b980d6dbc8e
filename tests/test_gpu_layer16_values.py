"""The 16-bit layer's result and its token gradient, against the sums over a token's rows in 64 bits."""
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_output_and_token_gradient():
    g = torch.Generator().manual_seed(61)
    T, k, E, D, F = 203, 3, 5, 264, 136
    w13 = (torch.randn(E, 2 * F, D, generator=g) * D ** -0.5).to(BF).to(DEV)
    w2 = (torch.randn(E, D, F, generator=g) * F ** -0.5).to(BF).to(DEV)
    x, dout = torch.randn(T, D, generator=g).to(BF).to(DEV), torch.randn(T, D, generator=g).to(BF).to(DEV)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int()
    wt = torch.softmax(torch.randn(T, k, generator=g), dim=1)
    r = mxk.mxmoe_route(ids.to(DEV), E, 1, m_cap=T * k)
    off, slot = r["offsets"], r["row_slot"].long()
    rows = x[slot // k]
    f = mxk.mxfp8_swiglu_ckpt(mxk.mxmoe_ragged_gemm(rows, w13, off))
    y = mxk.mxmoe_ragged_gemm(f["h"], w2, off)
    out = mxk.mxmoe_unpermute_combine(y, r["slot_row"], k, weights=wt.to(DEV))
    dy = (dout[slot // k].float() * wt.to(DEV).reshape(-1)[slot].unsqueeze(1)).to(BF)
    dh = mxk.mxmoe_ragged_gemm(dy, w2, off, transpose_w=True)
    dx_rows = mxk.mxmoe_ragged_gemm(mxk.mxfp8_swiglu_ckpt_bwd(dh, f["codes"], f["scales"])["dh13"], w13, off, transpose_w=True)
    dx = mxk.mxmoe_unpermute_combine(dx_rows, r["slot_row"], k)
    # the route: a token's j-th slot lies in its expert's segment
    o, sr = off.cpu(), r["slot_row"].cpu().long().reshape(T, k)
    for t in range(T):
        for j in range(k):
            assert o[ids[t, j]] <= sr[t, j] < o[ids[t, j] + 1]
    assert sr.reshape(-1).unique().numel() == T * k
    # k products summed in fp32 (half a step each, k - 1 sums), rounded once
    for got, v, c, what in ((out, y, wt, "out"), (dx, dx_rows, torch.ones(T, k), "token gradient")):
        p = c.double().unsqueeze(2) * v.cpu().double()[sr]
        ref, e = p.sum(1), (k + 1) * 2.0 ** -24 * p.abs().sum(1)
        P.assert_within(got, ref, e + P.u(BF) * (ref.abs() + e) + P.tiny(BF), what)
    # the whole chain in 64 bits from the layer's inputs, each 16-bit intermediate off by a rounding: the result agrees to the
    # size of those (h13, h, y: u each through the products, at most 4 u of the magnitudes that reach it)
    z = torch.einsum("tjnd,td->tjn", w13.cpu().double()[ids.long()], x.cpu().double())
    zm = torch.einsum("tjnd,td->tjn", w13.cpu().double().abs()[ids.long()], x.cpu().double().abs())
    a, b = z[..., :F], z[..., F:]
    h = a * P.sigmoid(a) * b
    u = P.u(BF)
    dz = u * z.abs() + D * 2.0 ** -23 * zm                          # h13: one rounding and fp32's sums
    dh_ = 1.1 * dz[..., :F] * (b.abs() + dz[..., F:]) + (a * P.sigmoid(a)).abs() * dz[..., F:]
    dh_ = dh_ + (u + 2.0 ** -16) * (h.abs() + dh_)
    W2 = w2.cpu().double()[ids.long()]
    yv, ym = torch.einsum("tjdf,tjf->tjd", W2, h), torch.einsum("tjdf,tjf->tjd", W2.abs(), h.abs() + dh_)
    ey = torch.einsum("tjdf,tjf->tjd", W2.abs(), dh_) + F * 2.0 ** -23 * ym
    ey = ey + u * (yv.abs() + ey)
    c = wt.double().unsqueeze(2)
    ref, e = (c * yv).sum(1), (c * (ey + (k + 1) * 2.0 ** -24 * (yv.abs() + ey))).sum(1)
    P.assert_within(out, ref, e + u * (ref.abs() + e) + P.tiny(BF), "layer")
    assert mxk.device_error() == 0
