"""GPU tests of the ragged products where every pair of SMs works through many tiles.

Whole numbers, so results equal the once-rounded exact ones bit for bit; the reference is a float64 product per expert.
Sizes give each of the 74 pairs more than 16 tiles of several K blocks: stages, accumulators, staging buffers and the
announced places are all reused, and the parities of their barriers flip several times.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
PAIRS = 74


def _ints(g, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).double()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lens(seed, E, mean):
    """Odd lengths around the mean (never a multiple of 16), a few experts without rows."""
    r = np.random.default_rng(seed)
    n = r.integers(mean // 2, mean + mean // 2 + 1, size=E) | 1
    n[r.integers(0, E, size=3)] = 0
    return n.tolist()


def _same(got, ref, what):
    bad = got != ref
    assert not bad.any(), f"{what}: {int(bad.sum())} values differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("E,mean,N,K", [(48, 60, 1304, 1296), (48, 60, 1304, 1288), (40, 450, 1304, 1296), (24, 150, 2056, 1800)])
def test_weight_gradients_next_to_nan(E, mean, N, K, dt):
    """Every other expert's rows are NaN: the rows behind each clean segment's end, up to the next multiple of 16, must have
    been cleared in both SMs of a pair before the products read them."""
    g, lens = _gen(1), _lens(1, E, mean)
    off = P.offsets_of(lens)
    M = sum(lens)
    assert E * -(-N // 256) * -(-K // 256) > 16 * PAIRS
    a, gr = _ints(g, M, K), _ints(g, M, N)
    pa, pg = a.clone(), gr.clone()
    for e in range(1, E, 2):
        pa[off[e]:off[e + 1]], pg[off[e]:off[e + 1]] = float("nan"), float("nan")
    pa, pg, o = pa.to(dt), pg.to(dt), off.to(DEV)
    out = torch.full((E, N, K), 7.0, dtype=dt, device=DEV)
    for _ in range(3):
        out.fill_(7.0)
        mxk.mxmoe_ragged_gemm_wgrad(pg, pa, o, out=out)
        for e in range(E):
            s = slice(int(off[e]), int(off[e + 1]))
            if e % 2 and lens[e]:
                assert torch.isnan(out[e]).all(), e
            else:
                _same(out[e], (gr[s].t() @ a[s]).to(dt), f"expert {e} of {lens[e]} rows")
    assert mxk.device_error() == 0


def test_a_contraction_of_seconds():
    """An unsplit tile of 15.6 million K blocks (one expert's 10^9 rows, 38 experts, so no split) takes over three seconds: the
    waits that last as long as the tile hold, and rows beyond 2^32 bytes are found.  Few rows are not zero, so sums are exact."""
    M, E, N, K = 1_000_000_000, 38, 8, 8
    assert mxk.ragged_workspace_bytes(M, N, K, E, 2) == 0
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB of device memory")
    g = _gen(2)
    rows = torch.tensor([0, 1, 63, 64, 4_000_003, 2 ** 28 - 1, 2 ** 28, 2 ** 29 + 77, M - 14, M - 12, M - 11], device=DEV)
    lens = [5] + [0] * 19 + [M - 5 - 11] + [0] * 16 + [11]          # the last expert's rows lie behind the long one's tail
    off = P.offsets_of(lens)
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    d = torch.zeros(M, N, dtype=BF, device=DEV)
    vx, vd = _ints(g, rows.numel(), K), _ints(g, rows.numel(), N)
    x[rows], d[rows] = vx.to(BF), vd.to(BF)
    dw = mxk.mxmoe_ragged_gemm_wgrad(d, x, off.to(DEV))
    for e in range(E):
        s = (rows >= int(off[e])) & (rows < int(off[e + 1]))
        _same(dw[e], (vd[s].t() @ vx[s]).to(BF), f"expert {e}")
    del x, d
    torch.cuda.empty_cache()
    assert mxk.device_error() == 0


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
@pytest.mark.parametrize("E,mean,rows,deep", [(24, 700, 4360, 328), (48, 60, 6664, 136), (24, 1100, 4104, 1288)])
def test_products_of_many_tiles(E, mean, rows, deep, trans, dt):
    """Blocks of eight row tiles (the last one short) over several token tiles, ragged in every dimension."""
    g, lens = _gen(3), _lens(3, E, mean)
    off = P.offsets_of(lens)
    R, M = sum(lens), sum(lens) + 5
    tiles = sum(-(-n // 256) for n in lens) * -(-rows // 256)
    assert tiles > 16 * PAIRS and rows > 8 * 256
    N, K = (deep, rows) if trans else (rows, deep)
    a, w = _ints(g, M, deep), _ints(g, E, N, K).to(dt)
    a[R:] = float("nan")
    out = torch.full((M, rows), 7.0, dtype=dt, device=DEV)
    x, o = a.to(dt), off.to(DEV)
    for _ in range(2):
        out.fill_(7.0)
        mxk.mxmoe_ragged_gemm(x, w, o, transpose_w=trans, out=out)
        for e in range(E):
            s = slice(int(off[e]), int(off[e + 1]))
            we = w[e].double()
            _same(out[s], (a[s] @ (we if trans else we.t())).to(dt), f"expert {e} of {lens[e]} rows")
        assert (out[R:] == 7).all()
    assert mxk.device_error() == 0
