"""Plain 64-bit forms and error bounds for the tests of the operators beside the MXFP8 path (CPU, float64).

u(t) is a rounding's largest relative error: half a step, finfo(t).eps / 2.
"""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def u(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the smallest subnormal: the absolute part of a rounding."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def offsets_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def ragged(a, w, off, trans):
    """(sum, sum of magnitudes) of the grouped product; rows of no segment are zero."""
    a, w = a.double(), w.double()
    out = torch.zeros(a.shape[0], w.shape[2] if trans else w.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(w.shape[0]):
        r = slice(int(off[e]), int(off[e + 1]))
        m = w[e] if trans else w[e].t()
        out[r] = a[r] @ m
        mag[r] = a[r].abs() @ m.abs()
    return out, mag


def wgrad(g, a, off):
    g, a = g.double(), a.double()
    E = off.numel() - 1
    seg = [slice(int(off[e]), int(off[e + 1])) for e in range(E)]
    return (torch.stack([g[r].t() @ a[r] for r in seg]), torch.stack([g[r].abs().t() @ a[r].abs() for r in seg]))


def assert_within(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs() - bound
    bad = ~(off <= 0)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst by {float(off[bad].max()):.3e} at {bad.nonzero()[0].tolist()}"


def assert_same(got, ref, what):
    got = got.detach().cpu()
    assert got.dtype == ref.dtype and got.shape == ref.shape, (what, got.dtype, ref.dtype, got.shape, ref.shape)
    bad = (got != ref) & ~((got != got) & (ref != ref)) if got.is_floating_point() else got != ref
    assert not bad.any(), f"{what}: {int(bad.sum())} values differ, first at {bad.nonzero()[0].tolist()}"


def floor_log2(m):
    """floor(log2 m) of positive float64 values, exactly."""
    return np.frexp(m)[1] - 1


def block_bytes(x, top):
    """Scale bytes of blocks [.., 32] (float64): the OCP rule, 0 for zero blocks, 255 for NaN or infinity."""
    m = np.abs(x)
    bad = ~np.isfinite(x).all(-1)
    m = np.where(np.isfinite(m), m, 0).max(-1)
    b = np.where(m > 0, np.clip(floor_log2(np.where(m > 0, m, 1)) - top + 127, 0, 254), 0)
    return np.where(bad, 255, b).astype(np.int64)


def nearest(v, grid):
    """Index of the nearest grid value by magnitude, ties to the even index, saturating."""
    m = np.abs(v)
    hi = np.clip(np.searchsorted(grid, m), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = m - grid[lo], grid[hi] - m
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def fp4(x):
    """(codes one per value, bytes) of [rows, cols]."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, 32)
    byte = block_bytes(b, 2)
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.where(byte[..., None] == 255, np.where(np.signbit(b), -6.0, 6.0), b * np.ldexp(1.0, 127 - byte)[..., None])
    code = nearest(v, E2M1) | (np.signbit(v).astype(np.int64) << 3)
    return code.reshape(x.shape), byte


def fp4_values(codes, byte):
    """float64 values of one-per-value codes [.., cols] with bytes [.., cols / 32]."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return v * np.repeat(s, 32, axis=-1)


def fp4_unpack(packed):
    p = np.asarray(packed).astype(np.int64)
    return np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], -1)


def fp4_tile_index(R, K, gated):
    """Index arrays [R, K / 8] (of four-byte words) and [R, K / 32] (of scale bytes) of one expert's tile layout."""
    r = np.arange(R)[:, None]
    if gated:
        F = R // 2
        half, f = r // F, r % F
        t, row = f // 8, 8 * half + f % 8
    else:
        t, row = r // 16, r % 16
    c8, kb = np.arange(K // 8)[None], np.arange(K // 32)[None]
    words = ((t * (K // 128) + c8 // 16) * 1024 + (row // 8) * 512 + (row % 8) * 64 + (c8 % 4) * 16 + ((c8 // 4) % 4) * 4) // 4
    return words, (t * (K // 128) + kb // 4) * 64 + row * 4 + kb % 4


E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [2.0 ** e * (1 + m / 8) for e in range(-6, 9) for m in range(8)][:-1])


def e4m3(x):
    """(codes, bytes) of [rows, cols], blocks of 32, the last one short."""
    rows, cols = x.shape
    pad = -cols % 32
    b = np.pad(np.asarray(x, dtype=np.float64), ((0, 0), (0, pad))).reshape(rows, -1, 32)
    byte = block_bytes(b, 8)
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.where(byte[..., None] == 255, 0.0, b * np.ldexp(1.0, 127 - byte)[..., None])
    code = np.where(byte[..., None] == 255, 0x7F, nearest(v, E4M3)) | (np.signbit(b).astype(np.int64) << 7)
    return code.reshape(rows, -1)[:, :cols], byte


def e4m3_values(code, byte, cols):
    v = np.where((code & 0x7F) == 0x7F, np.nan, np.append(E4M3, 0.0)[code & 0x7F]) * np.where(code & 0x80, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return v * np.repeat(s, 32, axis=-1)[:, :cols]


def sigmoid(a):
    return 1 / (1 + torch.exp(-a))


def sigmoid_err(a):
    """Relative error of the kernels' sigmoid: __expf is off by at most 2 + 1.173 |a| units, the addition by one half,
    __fdividef by 2 (units of 2^-23), and no more than the exponential's share reaches the sum."""
    return (6 + 1.2 * a.abs()) * 2.0 ** -23
