"""Refusals of the serving operators at the borders of their ranges (no GPU needed): every call
here is refused before anything is launched."""
import ctypes

import pytest

import long_context_sparse_head_b200 as fs

PTR = 0x10000                                  # a stand-in for a device pointer, never followed


# ---------------------------------------------------------------- rotary positions
def rope(strides, B=2, H=4, N=8, d=64, Hk=0):
    """fs_rope of contiguous inputs into outputs of these strides (b, h, n)."""
    c = fs.FsRopeParams(B, N, H, Hk, d)
    for x, v, w in zip("bhn", (H * N * d, N * d, d), (Hk * N * d, N * d, d)):
        setattr(c, "q_" + x, v)
        setattr(c, "k_" + x, w)
    for name in ("qo_", "ko_"):
        for x, v in zip("bhn", strides):
            setattr(c, name + x, v)
    Q, Qo, K, Ko = (PTR, PTR + (1 << 20)) * 2
    return fs.load().fs_rope(ctypes.byref(c), fs.Rotary(64).ref(), Q, Qo, K, Ko, None, 0, 0, None)


@pytest.mark.parametrize("strides", [
    (2048, 512, 32),                           # a token's row reaches into the next
    (2048, 8, 64),                             # a head's into the next
    (64, 512, 64),                             # both sequences are the same
    (2048, 64, 64),                            # heads and tokens are the same
    (2048, 64, 192),                           # four heads span 256
    (1984, 512, 64), (-1984, 512, 64), (2048, 512, -32), (2048, -448, 64),
    (2048, 512, 0), (0, 512, 64), (1 << 62, 512, 64), (-(1 << 63), 512, 64),
])
def test_rope_refuses_outputs_folded_together(strides):
    assert rope(strides) == 1
    assert rope(strides, Hk=4, H=0) == 1       # the second tensor's output alike
