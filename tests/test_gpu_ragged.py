"""GPU tests of the ragged 16-bit products (mxmoe_ragged_gemm and its weight gradient).

Small whole numbers: every product and sum is exact in fp32, so the results must equal the once-rounded exact ones bit for
bit.  Normal values: a result is off by one rounding plus fp32's sums, at most K additions of 2^-23 of the magnitudes' sum
(2^-23, not 2^-24: the tensor cores may cut instead of rounding).
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16

# segment lengths, N, K: empty experts in every place, one row, tile edges (256 tokens, 128 rows, 64 deep, 16 of the MMA), odd
SHAPES = [
    ([1], 8, 8),
    ([0, 3, 0], 16, 24),
    ([5, 0, 17, 1], 136, 72),
    ([256, 0, 257, 255], 128, 64),
    ([15, 16, 17, 63, 64, 65, 0], 264, 200),
    ([300, 2, 0, 511, 33], 520, 328),
    ([0, 0, 700], 384, 1032),
]


def _ints(g, *shape, top=2):
    return torch.from_numpy(g.integers(-top, top + 1, size=shape).astype(np.float32))


def _round(x, dt):
    return x.to(dt)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
@pytest.mark.parametrize("lens,N,K", SHAPES)
def test_whole_numbers_are_exact(lens, N, K, trans, dt):
    g = np.random.default_rng(1)
    off = P.offsets_of(lens)
    R, E, tail = sum(lens), len(lens), 3
    a = _ints(g, R + tail, N if trans else K)
    w = _ints(g, E, N, K)
    out = torch.full((R + tail, K if trans else N), 7.0, dtype=dt, device=DEV)
    got = mxk.mxmoe_ragged_gemm(a.to(DEV, dt), w.to(DEV, dt), off.to(DEV), transpose_w=trans, out=out)
    assert got is out
    ref, _ = P.ragged(a, w, off, trans)
    ref[R:] = 7.0                                                   # rows behind the last segment stay as they were
    P.assert_same(got, _round(ref, dt), "out")
    assert mxk.device_error() == 0


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,N,K", SHAPES)
def test_weight_gradient_of_whole_numbers_is_exact(lens, N, K, dt):
    g = np.random.default_rng(2)
    off = P.offsets_of(lens)
    R, E = sum(lens), len(lens)
    gr, a = _ints(g, R + 2, N), _ints(g, R + 2, K)
    out = torch.full((E, N, K), float("nan"), dtype=dt, device=DEV)
    got = mxk.mxmoe_ragged_gemm_wgrad(gr.to(DEV, dt), a.to(DEV, dt), off.to(DEV), out=out)
    ref, _ = P.wgrad(gr, a, off)
    P.assert_same(got, _round(ref, dt), "dw")
    assert mxk.device_error() == 0


@pytest.mark.parametrize("lens", [[3, 0, 40], [500, 410], [0, 2000]], ids=["short", "long", "one"])
@pytest.mark.parametrize("N,K", [(136, 272), (264, 288), (24, 16), (520, 600), (8, 344), (40, 200)])
def test_weight_gradient_edges_of_store_boxes(lens, N, K):
    """Boxes of 32 and of 64 columns (few or many rows an expert, row pitch), odd numbers of 32-column pieces,
    bytes behind the matrix untouched."""
    g = np.random.default_rng(21)
    off = P.offsets_of(lens)
    R, E = sum(lens), len(lens)
    gr, a = _ints(g, R, N), _ints(g, R, K)
    flat = torch.full((E * N * K + 64,), 5.0, dtype=BF, device=DEV)
    out = flat[: E * N * K].view(E, N, K)
    mxk.mxmoe_ragged_gemm_wgrad(gr.to(DEV, BF), a.to(DEV, BF), off.to(DEV), out=out)
    P.assert_same(out, _round(P.wgrad(gr, a, off)[0], BF), "dw")
    assert (flat[E * N * K :] == 5.0).all() and mxk.device_error() == 0


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_normal_values_within_the_bound(dt):
    g = torch.Generator().manual_seed(3)
    lens, N, K = [130, 0, 77, 401], 328, 1096
    off = P.offsets_of(lens)
    R, E = sum(lens), len(lens)
    w = (torch.randn(E, N, K, generator=g) * K ** -0.5).to(dt)
    a, gr = torch.randn(R, K, generator=g).to(dt), torch.randn(R, N, generator=g).to(dt)
    dev = lambda *t: [v.to(DEV) for v in t]  # noqa: E731
    for trans, x, depth in ((False, a, K), (True, gr, N)):
        ref, mag = P.ragged(x, w, off, trans)
        got = mxk.mxmoe_ragged_gemm(*dev(x, w, off), transpose_w=trans)
        s = depth * 2.0 ** -23 * mag
        P.assert_within(got, ref, P.u(dt) * (ref.abs() + s) + s + P.tiny(dt), f"trans={trans}")
    ref, mag = P.wgrad(gr, a, off)
    s = max(lens) * 2.0 ** -23 * mag
    P.assert_within(mxk.mxmoe_ragged_gemm_wgrad(*dev(gr, a, off)), ref, P.u(dt) * (ref.abs() + s) + s + P.tiny(dt), "dw")


def test_gradients_are_the_differences():
    """The product is linear: for whole numbers sum(g * (f(a + v) - f(a))) is exactly sum(da * v), and the same for w."""
    r = np.random.default_rng(4)
    lens, N, K = [9, 0, 70], 24, 40
    off = P.offsets_of(lens).to(DEV)
    R, E = sum(lens), len(lens)
    a, v, g = (_ints(r, R, n, top=1).to(DEV, BF) for n in (K, K, N))
    w, x = (_ints(r, E, N, K, top=1).to(DEV, BF) for _ in range(2))
    f = lambda a_, w_: mxk.mxmoe_ragged_gemm(a_, w_, off).double()  # noqa: E731
    dot = lambda s, t: float((s.double() * t.double()).sum())  # noqa: E731
    da = mxk.mxmoe_ragged_gemm(g, w, off, transpose_w=True)
    dw = mxk.mxmoe_ragged_gemm_wgrad(g, a, off)
    assert dot(g, f(a + v, w) - f(a, w)) == dot(da, v)
    assert dot(g, f(a, w + x) - f(a, w)) == dot(dw, x)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_neighbours_and_tail_rows_do_not_leak(dt):
    """NaN in the rows of other experts and behind the last segment reaches no other expert's results."""
    r = np.random.default_rng(5)
    lens, N, K = [19, 41, 3], 72, 136
    off = P.offsets_of(lens)
    R = sum(lens)
    a, g, w = _ints(r, R + 9, K), _ints(r, R + 9, N), _ints(r, 3, N, K)
    mid = slice(19, 60)
    pa, pg = torch.full_like(a, float("nan")), torch.full_like(g, float("nan"))
    pa[mid], pg[mid] = a[mid], g[mid]
    dw = mxk.mxmoe_ragged_gemm_wgrad(pg.to(DEV, dt), pa.to(DEV, dt), off.to(DEV))
    P.assert_same(dw[1], _round(P.wgrad(g, a, off)[0][1], dt), "dw of the clean expert")
    y = mxk.mxmoe_ragged_gemm(pa.to(DEV, dt), w.to(DEV, dt), off.to(DEV))
    P.assert_same(y[mid], _round(P.ragged(a, w, off, False)[0][mid], dt), "rows of the clean expert")
    assert torch.isnan(y[:19]).all() and torch.isnan(y[60:63]).all()


def test_infinite_weights_of_another_expert_do_not_leak():
    r = np.random.default_rng(6)
    lens, N, K = [20, 20], 200, 72
    off = P.offsets_of(lens)
    a, w = _ints(r, 40, K), _ints(r, 2, N, K)
    pw = w.clone()
    pw[1] = float("inf")
    for trans, x in ((False, a), (True, _ints(r, 40, N))):
        y = mxk.mxmoe_ragged_gemm(x.to(DEV, BF), pw.to(DEV, BF), off.to(DEV), transpose_w=trans)
        P.assert_same(y[:20], _round(P.ragged(x, w, off, trans)[0][:20], BF), "rows of the clean expert")


def test_many_experts_and_no_rows():
    r = np.random.default_rng(7)
    lens = r.integers(0, 3, size=1024).tolist()
    off = P.offsets_of(lens)
    a, w, g = _ints(r, sum(lens), 16), _ints(r, 1024, 8, 16), _ints(r, sum(lens), 8)
    P.assert_same(mxk.mxmoe_ragged_gemm(a.to(DEV, BF), w.to(DEV, BF), off.to(DEV)), _round(P.ragged(a, w, off, False)[0], BF), "out")
    P.assert_same(mxk.mxmoe_ragged_gemm_wgrad(g.to(DEV, BF), a.to(DEV, BF), off.to(DEV)), _round(P.wgrad(g, a, off)[0], BF), "dw")
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    wd = torch.ones(3, 8, 16, dtype=BF, device=DEV)
    y = mxk.mxmoe_ragged_gemm(torch.ones(5, 16, dtype=BF, device=DEV), wd, none, out=torch.full((5, 8), 2.0, dtype=BF, device=DEV))
    assert (y == 2).all()
    dw = mxk.mxmoe_ragged_gemm_wgrad(torch.ones(5, 8, dtype=BF, device=DEV), torch.ones(5, 16, dtype=BF, device=DEV), none)
    assert dw.shape == (3, 8, 16) and (dw == 0).all()
    e = torch.empty
    assert mxk.mxmoe_ragged_gemm(e(0, 16, dtype=BF, device=DEV), wd, none).shape == (0, 8)
    dw = mxk.mxmoe_ragged_gemm_wgrad(e(0, 8, dtype=BF, device=DEV), e(0, 16, dtype=BF, device=DEV), none)
    assert (dw == 0).all()
    assert mxk.device_error() == 0


@pytest.mark.parametrize("table", [[1, 5, 9], [0, 6, 5], [0, 4, 11], [0, -1, 3]])
def test_bad_tables_write_nothing_and_are_reported(table):
    off = torch.tensor(table, dtype=torch.int32, device=DEV)
    a = torch.ones(10, 16, dtype=BF, device=DEV)
    w = torch.ones(2, 8, 16, dtype=BF, device=DEV)
    out = torch.full((10, 8), 3.0, dtype=BF, device=DEV)
    mxk.mxmoe_ragged_gemm(a, w, off, out=out)
    assert mxk.device_error() == 4 and (out == 3).all()
    dw = torch.full((2, 8, 16), 3.0, dtype=BF, device=DEV)
    mxk.mxmoe_ragged_gemm_wgrad(out, a, off, out=dw)
    assert mxk.device_error() == 4 and (dw == 3).all()


def test_captured_on_a_stream_and_replayed_on_new_data():
    r = np.random.default_rng(8)
    lens, N, K = [40, 7, 0, 130], 136, 264
    R, E = sum(lens), len(lens)
    a, w, g = (t.to(DEV, BF) for t in (_ints(r, R, K), _ints(r, E, N, K), _ints(r, R, N)))
    off = P.offsets_of(lens).to(DEV)
    y, dx, dw = (torch.empty(s, dtype=BF, device=DEV) for s in ((R, N), (R, K), (E, N, K)))

    def step():
        mxk.mxmoe_ragged_gemm(a, w, off, out=y)
        mxk.mxmoe_ragged_gemm(g, w, off, transpose_w=True, out=dx)
        mxk.mxmoe_ragged_gemm_wgrad(g, a, off, out=dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens2 = [0, 100, 60, 17]
    a.copy_(_ints(r, R, K)), w.copy_(_ints(r, E, N, K)), g.copy_(_ints(r, R, N)), off.copy_(P.offsets_of(lens2))
    graph.replay()
    torch.cuda.synchronize()
    c = [t.cpu() for t in (a, w, g, off)]
    P.assert_same(y, _round(P.ragged(c[0], c[1], c[3], False)[0], BF), "y")
    P.assert_same(dx, _round(P.ragged(c[2], c[1], c[3], True)[0], BF), "dx")
    P.assert_same(dw, _round(P.wgrad(c[2], c[0], c[3])[0], BF), "dw")


def test_two_streams_at_once():
    r = np.random.default_rng(9)
    off = P.offsets_of([300, 100]).to(DEV)
    jobs = []
    for i in range(2):
        a, w = _ints(r, 400, 520).to(DEV, BF), _ints(r, 2, 264, 520).to(DEV, BF)
        jobs.append((torch.cuda.Stream(), a, w, torch.zeros(400, 264, dtype=BF, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, a, w, y in jobs:
            with torch.cuda.stream(s):
                mxk.mxmoe_ragged_gemm(a, w, off, out=y)
    torch.cuda.synchronize()
    for s, a, w, y in jobs:
        P.assert_same(y, _round(P.ragged(a.cpu(), w.cpu(), off.cpu(), False)[0], BF), "y")


def test_repeats_are_bitwise_equal():
    g = torch.Generator(device=DEV).manual_seed(10)
    off = P.offsets_of([900, 0, 333]).to(DEV)
    a, w, d = (torch.randn(*s, device=DEV, generator=g).to(BF) for s in ((1233, 520), (3, 392, 520), (1233, 392)))
    first = (mxk.mxmoe_ragged_gemm(a, w, off), mxk.mxmoe_ragged_gemm_wgrad(d, a, off))
    for _ in range(3):
        again = (mxk.mxmoe_ragged_gemm(a, w, off), mxk.mxmoe_ragged_gemm_wgrad(d, a, off))
        assert all(torch.equal(x, y) for x, y in zip(first, again))


# ------------------------------------------------------------------------------------------------ split contractions
SPLIT = [  # segment lengths, N, K, which of (forward, input gradient, weight gradient) are split
    ([70, 0, 13], 40, 4104, (0,)),
    ([5], 4104, 264, (1,)),
    ([0, 3001, 0, 130, 77], 24, 72, (2,)),
    ([3100, 1], 136, 264, (2,)),
    ([300], 264, 3080, (0,)),
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,N,K,which", SPLIT)
def test_split_whole_numbers_are_exact(lens, N, K, which, dt):
    """Few tiles with a long contraction: units share a tile and a second launch joins their sums."""
    g = np.random.default_rng(11)
    off = P.offsets_of(lens)
    R, E, tail = sum(lens), len(lens), 3
    M = R + tail
    a, gr, w = _ints(g, M, K, top=1), _ints(g, M, N, top=1), _ints(g, E, N, K, top=1)
    d = [t.to(DEV, dt) for t in (a, gr, w)]
    for k in (0, 1, 2):
        assert (mxk.ragged_workspace_bytes(M, N, K, E, k) > 0) or k not in which, k
    for tr, x in ((False, 0), (True, 1)):
        out = torch.full((M, K if tr else N), 7.0, dtype=dt, device=DEV)
        mxk.mxmoe_ragged_gemm(d[x], d[2], off.to(DEV), transpose_w=tr, out=out)
        ref, _ = P.ragged(gr if tr else a, w, off, tr)
        ref[R:] = 7.0
        P.assert_same(out, _round(ref, dt), f"out, transpose_w={tr}")
    dw = mxk.mxmoe_ragged_gemm_wgrad(d[1], d[0], off.to(DEV), out=torch.full((E, N, K), float("nan"), dtype=dt, device=DEV))
    P.assert_same(dw, _round(P.wgrad(gr, a, off)[0], dt), "dw")
    assert mxk.device_error() == 0


def test_split_bad_table_writes_nothing():
    off = torch.tensor([0, 9000], dtype=torch.int32, device=DEV)
    a, g = torch.ones(4000, 72, dtype=BF, device=DEV), torch.ones(4000, 24, dtype=BF, device=DEV)
    assert mxk.ragged_workspace_bytes(4000, 24, 72, 1, 2) > 0
    dw = torch.full((1, 24, 72), 3.0, dtype=BF, device=DEV)
    mxk.mxmoe_ragged_gemm_wgrad(g, a, off, out=dw)
    assert mxk.device_error() == 4 and (dw == 3).all()


def test_split_captured_with_a_workspace_each():
    """Two graphs with their own workspaces on two streams at once; the split and the unsplit product on whole numbers agree."""
    r = np.random.default_rng(12)
    jobs = []
    for _ in range(2):
        a, g = _ints(r, 5000, 72, top=1).to(DEV, BF), _ints(r, 5000, 24, top=1).to(DEV, BF)
        off = P.offsets_of([4000, 1000]).to(DEV)
        ws = torch.empty(mxk.ragged_workspace_bytes(5000, 24, 72, 2, 2), dtype=torch.uint8, device=DEV)
        out = torch.empty(2, 24, 72, dtype=BF, device=DEV)
        run = lambda a=a, g=g, off=off, ws=ws, out=out: mxk.mxmoe_ragged_gemm_wgrad(g, a, off, out=out, workspace=ws)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        off.copy_(P.offsets_of([1, 4500]))
        a.copy_(_ints(r, 5000, 72, top=1))
        jobs.append((graph, torch.cuda.Stream(), a, g, off, out))
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, s, *_ in jobs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, a, g, off, out in jobs:
        P.assert_same(out, _round(P.wgrad(g.cpu(), a.cpu(), off.cpu())[0], BF), "dw")


def test_split_normal_values_within_the_bound():
    g = torch.Generator().manual_seed(13)
    lens, N, K = [4000, 0, 500], 40, 136
    off = P.offsets_of(lens)
    a, gr = torch.randn(4500, K, generator=g).to(BF), torch.randn(4500, N, generator=g).to(BF)
    ref, mag = P.wgrad(gr, a, off)
    s = max(lens) * 2.0 ** -23 * mag
    P.assert_within(mxk.mxmoe_ragged_gemm_wgrad(gr.to(DEV), a.to(DEV), off.to(DEV)), ref, P.u(BF) * (ref.abs() + s) + s + P.tiny(BF), "dw")
