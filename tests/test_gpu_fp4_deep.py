"""GPU tests of the 4-bit products where every team of warps takes several tiles of a group and blocks cross from group to group."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P
from test_gpu_fp4 import _layer, _layer_ref, _tiled, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
SMS = 148


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("S,E,N,K", [(30, 3, 4112, 2048), (40, 2, 8208, 1152), (100, 2, 6416, 640), (100, 2, 6416, 128)])
def test_matvec_of_many_tiles_is_exact(S, E, N, K, dt):
    """Whole numbers; teams of four, two and one warps, shares of cells that differ between them."""
    r = np.random.default_rng(51)
    packed, byte, w = _weights(r, E, N, K, lo=127, hi=128)
    ids = r.integers(0, E, size=S).astype(np.int32)
    groups = sum(-(-int((ids == e).sum()) // 8) for e in range(E))
    teams = 4 if K >= 2048 else 8 if K >= 1024 else 16
    assert groups * (N // 16) > 2 * teams * SMS                    # every team of every block takes two tiles or more
    x = torch.from_numpy(r.integers(-3, 4, size=(S, K)).astype(np.float64))
    c, s = _tiled(packed, byte, False)
    xd, idd = x.to(DEV, dt), torch.from_numpy(ids).to(DEV)
    ref = torch.stack([w[ids[i]] @ x[i] for i in range(S)]).to(dt)
    for _ in range(3):
        P.assert_same(mxk.mxfp4_expert_matvec(xd, idd, c, s, out=torch.full((S, N), 7.0, dtype=dt, device=DEV)), ref, "y")
    assert mxk.device_error() == 0


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,D,F", [(5, 2, 3, 2048, 2048), (12, 2, 2, 1152, 2176), (1, 2, 2, 4096, 1408)])
def test_decode_layer_with_teams(T, k, E, D, F, dt):
    qw, w13, w2, ids, x, wt = _layer(np.random.default_rng(52), T, k, E, D, F, dt)
    ref, bound = _layer_ref(w13, w2, ids, x, wt, dt)
    args = (x.to(DEV), ids.to(DEV), wt.to(DEV), qw)
    out = mxk.moe_layer_decode_fp4(*args)
    P.assert_within(out, ref, bound, "out")
    assert torch.equal(out, mxk.moe_layer_decode_fp4(*args)) and mxk.device_error() == 0
