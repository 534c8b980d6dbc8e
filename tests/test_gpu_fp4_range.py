"""GPU tests of the 4-bit products at the ends of the exponent ranges: rows of any size under block scales of any size."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P
from test_gpu_fp4 import _layer_ref, _tiled, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def _whole(r, S, K, power):
    """Whole numbers -3..3 times 2^power (a number or one per row)."""
    return torch.from_numpy(np.ldexp(r.integers(-3, 4, size=(S, K)).astype(np.float64), power))


@pytest.mark.parametrize("K", [128, 1152])
@pytest.mark.parametrize("dt,power,lo", [(BF, -133, 253), (BF, -130, 250), (BF, -127, 127), (BF, -112, 253), (BF, -100, 237), (BF, -10, 0),
                                         (BF, 0, 236), (BF, 2, 234), (BF, 110, 0), (BF, 125, 0), (FP, -24, 127), (FP, -24, 145), (FP, 13, 90)])
def test_small_and_large_rows_are_exact(dt, power, lo, K):
    """Every product and sum is a whole multiple of one power of two, so fp32 holds it, and the result, exactly: subnormal rows,
    scales near 2^127 and 2^-127, sums that 2^12 would lift over the range.  |sum| <= 3 * 12 * 1152 < 2^16 units."""
    r = np.random.default_rng(31)
    S, E, N = 11, 3, 48
    packed, byte, w = _weights(r, E, N, K, lo=lo, hi=lo + 1)
    ids = r.integers(0, E, size=S).astype(np.int32)
    x = _whole(r, S, K, power)
    assert torch.equal(x.to(dt).double(), x)
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x.to(DEV, dt), torch.from_numpy(ids).to(DEV), c, s)
    ref = torch.stack([w[ids[i]] @ x[i] for i in range(S)]).to(dt)
    assert torch.isfinite(ref).all() and (ref != 0).any()
    P.assert_same(y, ref, "y")


def test_rows_of_all_sizes_in_one_group():
    """Eight rows of one expert, from subnormal to the largest: each keeps its own power of two."""
    r = np.random.default_rng(32)
    K, N = 256, 32
    packed, byte, w = _weights(r, 1, N, K, lo=127, hi=128)
    power = np.array([-133, -126, -113, -60, 0, 40, 90, 112])[:, None]
    x = _whole(r, 8, K, power)
    x[2] = 0
    c, s = _tiled(packed, byte, False)
    y = mxk.mxfp4_expert_matvec(x.to(DEV, BF), torch.zeros(8, dtype=torch.int32, device=DEV), c, s)
    P.assert_same(y, (x @ w[0].t()).to(BF), "y")


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_decode_with_a_small_and_a_large_product(dt):
    """The up half makes h small, the second weights make up for it: the layer's result is of ordinary size."""
    r = np.random.default_rng(33)
    T, k, E, D, F = 3, 2, 4, 256, 128
    p13, b13, _ = _weights(r, E, 2 * F, D, lo=118, hi=121)
    b13[:, F:] -= 114                                              # up: 2^-114 of the gate's size
    p2, b2, w2 = _weights(r, E, D, F, lo=230, hi=233)
    w13 = torch.from_numpy(P.fp4_values(P.fp4_unpack(p13), b13.astype(np.int64)))
    ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    x, wt = torch.from_numpy(r.standard_normal((T, D))).to(dt), torch.from_numpy(r.random((T, k))).float()
    (c13, s13), (c2, s2) = _tiled(p13, b13, True), _tiled(p2, b2, False)
    out = mxk.moe_layer_decode_fp4(x.to(DEV), ids.to(DEV), wt.to(DEV), dict(w13_codes=c13, w13_scales=s13, w2_codes=c2, w2_scales=s2))
    ref, bound = _layer_ref(w13, w2, ids, x, wt, dt)
    assert torch.isfinite(ref).all() and 2.0 ** -20 < float(ref.abs().median()) < 2.0 ** 14
    P.assert_within(out, ref, bound, "out")
