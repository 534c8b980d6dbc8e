"""GPU tests of what the decode layer keeps of h between its two products."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_routed_b200 as mxk
import plain16 as P
from test_gpu_fp4 import _layer, _layer_ref, _tiled

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 20])
def test_differences_of_neighbouring_h_survive(T, dt):
    """Pairs of h near 2^17 that differ by 32, and second weights that subtract them: the layer's result is that difference.
    Eleven bits of h would leave steps of 64 to 128.  Slots of one expert from one to a full group of eight and beyond.

    x = 1, gates 32, ups 6 * 2^9 + r and one more (whole numbers, exact in fp32), so h = 32 s up with s = 1 - e^-32: each is off
    by at most (6 + 1.2 * 32) 2^-23 + 2^-22 for the sigmoid and the products and 2^-22 for the pieces, and the result by twice that."""
    r = np.random.default_rng(41)
    E, D, F = 2, 128, 128
    code13, byte13 = np.zeros((E, 2 * F, D), np.int64), np.full((E, 2 * F, D // 32), 127, np.int64)
    code13[:, :F, 0], byte13[:, :F, 0] = 6, 127 + 3                # gate: 4 * 2^3
    code13[:, F:, 0], byte13[:, F:, 0] = 7, 127 + 9                # up: 6 * 2^9 + r, r + 1
    rest = r.integers(0, 12, size=(E, F // 2))
    for e in range(E):
        for i in range(F // 2):
            for odd in (0, 1):
                n = rest[e, i] + odd                               # a whole number up to 12 as two codes
                lo, hi = min(n, 6), n - min(n, 6)
                for col, v in ((32, lo), (64, hi)):
                    a, b = (v, 0) if v != 5 else (4, 1)
                    code13[e, F + 2 * i + odd, col] = np.flatnonzero(P.E2M1 == a)[0]
                    code13[e, F + 2 * i + odd, col + 1] = np.flatnonzero(P.E2M1 == b)[0]
    code2, byte2 = np.zeros((E, D, F), np.int64), np.full((E, D, F // 32), 127, np.int64)
    for n in range(F // 2):
        code2[:, n, 2 * n], code2[:, n, 2 * n + 1] = 2, 2 | 8      # + 1, - 1
    pack = lambda c: (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)  # noqa: E731
    w13, w2 = (torch.from_numpy(P.fp4_values(c, b)) for c, b in ((code13, byte13), (code2, byte2)))
    (c13, s13), (c2, s2) = _tiled(pack(code13), byte13.astype(np.uint8), True), _tiled(pack(code2), byte2.astype(np.uint8), False)
    ids = torch.ones(T, 1, dtype=torch.int32)
    ids[T - 1] = 0                                                 # T - 1 slots of one expert, one of the other
    out = mxk.moe_layer_decode_fp4(torch.ones(T, D, dtype=dt, device=DEV), ids.to(DEV), torch.ones(T, 1, device=DEV),
                                   dict(w13_codes=c13, w13_scales=s13, w2_codes=c2, w2_scales=s2))
    z = w13.sum(2)
    h = z[:, :F] * P.sigmoid(z[:, :F]) * z[:, F:]
    ref = torch.einsum("enf,ef->en", w2, h)[ids[:, 0].long()]
    assert (ref[:, : F // 2].abs() > 31).all() and (ref[:, F // 2:] == 0).all() and (h > 2.0 ** 16).all() and (h < 2.0 ** 17).all()
    e = 2 * 2.0 ** 17 * ((6 + 1.2 * 32) * 2.0 ** -23 + 2 * 2.0 ** -22) + 64 * 2.0 ** -23
    P.assert_within(out, ref, torch.full_like(ref, e) + P.u(dt) * (ref.abs() + e), "out")
    assert mxk.device_error() == 0


def test_bf16_layer_beyond_two_pieces_of_shared_memory():
    """One row of h as two f16 pieces does not fit shared memory: one piece for bf16 layers (fp16 layers are refused)."""
    qw, w13, w2, ids, x, wt = _layer(np.random.default_rng(42), 2, 1, 1, 128, 36352, BF)
    out = mxk.moe_layer_decode_fp4(x.to(DEV), ids.to(DEV), wt.to(DEV), qw)
    ref, bound = _layer_ref(w13, w2, ids, x, wt, BF)
    P.assert_within(out, ref, bound, "out")
    with pytest.raises(mxk.MXMOEError, match="shared memory"):
        mxk.moe_layer_decode_fp4(x.to(DEV, FP), ids.to(DEV), wt.to(DEV), qw)
    assert mxk.device_error() == 0
