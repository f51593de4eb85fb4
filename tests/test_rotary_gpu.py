"""fs_rope and fs_rope_backward on the GPU against the rotation in float64."""
import numpy as np
import pytest
import torch

import long_context_sparse_head_b200 as fs
from tests._paged import DTYPES, rotate, rotate_bound, thetas

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def make(shape, dtype, seed, tokens_first=False):
    g = torch.Generator().manual_seed(seed)
    B, H, N, d = shape
    x = torch.randn((B, N, H, d) if tokens_first else shape, generator=g).to(DTYPES[dtype]).cuda()
    return x.transpose(1, 2) if tokens_first else x


def check(x, y, pos, rot, theta, layout, dtype, sign=1.0, mscale=1.0):
    """pos [B,N] (numpy)."""
    a = f64(x)
    want = rotate(a, pos[:, None, :], theta, layout, mscale, sign)
    r = 2 * len(theta)
    err = np.abs(f64(y) - want)
    assert (err <= rotate_bound(a, want, r, layout, dtype, mscale)).all(), err.max()
    assert np.array_equal(f64(y)[..., r:], a[..., r:])       # what is not rotated is copied


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d,r", [(64, 64), (128, 32), (256, 256), (96, 24), (20, 6), (2, 2), (67, 10)])
@pytest.mark.parametrize("tokens_first", [False, True])
def test_rope_and_gradient(dtype, layout, d, r, tokens_first):
    """Vector and element-wise forms (r or d that no 16-byte vector divides), both memory orders."""
    B, H, Hk, N = 3, 5, 2, 37
    q, k = make((B, H, N, d), dtype, 1, tokens_first), make((B, Hk, N, d), dtype, 2, tokens_first)
    pos = np.random.default_rng(3).integers(0, 1 << 20, (B, N))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    rot, theta = fs.Rotary(r, layout), thetas(r)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    fs.rope(rot, q, qo, k, ko, positions=p)
    check(q, qo, pos, rot, theta, layout, dtype)
    check(k, ko, pos, rot, theta, layout, dtype)
    fs.rope_backward(rot, q, qo, k, ko, positions=p)
    check(q, qo, pos, rot, theta, layout, dtype, sign=-1.0)
    check(k, ko, pos, rot, theta, layout, dtype, sign=-1.0)


@pytest.mark.parametrize("scaling,kw", [
    ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("by_parts", dict(factor=16.0, orig_len=4096, slow=1.0, fast=32.0, mscale=1.28)),
    ("by_parts", dict(factor=8.0, orig_len=8192, slow=1.0, fast=4.0)),
])
def test_scaled_positions(scaling, kw):
    N, d = 4100, 64
    kw = dict(kw)
    mscale = kw.pop("mscale", 1.0)
    x = make((1, 2, N, d), "f32", 5)
    y = torch.empty_like(x)
    rot = fs.Rotary(d, "half", base=500000.0, scaling=scaling, mscale=mscale, **kw)
    fs.rope(rot, x, y, pos0=123456)
    check(x, y, 123456 + np.arange(N)[None], rot, thetas(d, 500000.0, scaling, **kw), "half", "f32", mscale=mscale)


def test_far_and_negative_positions():
    pos = np.array([[0, 1, -1, 262143, (1 << 31) - 1, -(1 << 31), 12345678]])
    x = make((1, 3, 7, 64), "f32", 7)
    y = torch.empty_like(x)
    fs.rope(fs.Rotary(64), x, y, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    # the angle in float64 is itself off by 2^-53 of its size: nothing at these positions
    check(x, y, pos, None, thetas(64), "interleaved", "f32")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("r", [64, 32])
def test_in_place_and_there_and_back(layout, r):
    x = make((2, 4, 129, 64), "f32", 9, True)
    keep = x.clone()
    rot = fs.Rotary(r, layout)
    fs.rope(rot, x, x)
    check(keep, x, np.broadcast_to(np.arange(129), (2, 129)), rot, thetas(r), layout, "f32")
    fs.rope_backward(rot, x, x)
    a = f64(keep)
    # two rotations: twice the bound, the second one's terms as large as the first one's results
    assert (np.abs(f64(x) - a) <= 2 * rotate_bound(a, a, r, layout, "f32") + np.abs(a).max() * 2.0 ** -21).all()


def test_gradient_by_differences():
    """The operator is linear: <dy, rope(x + h) - rope(x)> = <rope_backward(dy), h>."""
    x, h, dy = (make((2, 3, 65, 128), "f32", s) for s in (11, 12, 13))
    rot = fs.Rotary(64, "half", scaling="by_parts", factor=4.0, orig_len=64, mscale=1.1)
    out, dx = [torch.empty_like(x) for _ in range(2)], torch.empty_like(x)
    fs.rope(rot, x + h, out[0])
    fs.rope(rot, x, out[1])
    fs.rope_backward(rot, dy, dx)
    left, right = (dy.double() * (out[0].double() - out[1].double())).sum(), (dx.double() * h.double()).sum()
    # each of the 49920 elements is off by at most 4 x 2^-21 of the pair's size
    size = (dy.abs().double() * (x.abs() + h.abs()).double()).sum() * 2.0 ** -18
    assert abs(float(left - right)) <= float(size)


def test_broadcast_and_shared_inputs():
    """Inputs of stride 0 (a key shared by the heads) and positions shared by the rows."""
    k = make((2, 1, 33, 64), "bf16", 15).expand(2, 6, 33, 64)
    out = torch.empty((2, 6, 33, 64), dtype=k.dtype, device="cuda")
    pos = np.random.default_rng(1).integers(0, 9999, 33)
    fs.rope(fs.Rotary(64), k, out, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    check(k, out, np.broadcast_to(pos, (2, 33)), None, thetas(64), "interleaved", "bf16")


def test_rows_off_the_16_byte_grid():
    """Rows of 65 elements, a base off by one element: the element-wise form."""
    base = torch.randn(1 + 2 * 3 * 9 * 65, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    x = base[1:].view(2, 3, 9, 65)[..., :64]
    out = torch.full((2, 3, 9, 70), 7.0, dtype=x.dtype, device="cuda")
    y = out[..., 3:67]
    fs.rope(fs.Rotary(64, "half"), x, y)
    check(x, y, np.broadcast_to(np.arange(9), (2, 9)), None, thetas(64), "half", "bf16")
    assert (out[..., :3] == 7).all() and (out[..., 67:] == 7).all()


def test_offsets_past_32_bits():
    far = (1 << 32) + 64
    store = torch.empty(far + 64 * 5, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((2, 1, 5, 64), (far, 64, 64, 1))
    v = make((2, 1, 5, 64), "bf16", 21)
    x.copy_(v)
    fs.rope(fs.Rotary(64), x, x)
    check(v, x, np.broadcast_to(np.arange(5), (2, 5)), None, thetas(64), "interleaved", "bf16")


def test_nothing_to_do_and_many_heads():
    rot = fs.Rotary(64)
    for shape in ((0, 3, 4, 64), (2, 0, 4, 64), (2, 3, 0, 64)):
        e = torch.empty(shape, device="cuda")
        fs.rope(rot, e, torch.empty_like(e))
    x = make((1, 300, 3, 64), "f16", 22)
    y = torch.empty_like(x)
    fs.rope(rot, x, y, pos0=7)
    check(x, y, 7 + np.arange(3)[None], None, thetas(64), "interleaved", "f16")


def test_on_another_stream_and_captured():
    x = make((1, 4, 64, 64), "bf16", 23)
    y = torch.zeros_like(x)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    rot = fs.Rotary(64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fs.rope(rot, x, y, positions=pos)
    torch.cuda.current_stream().wait_stream(s)
    pos += 1000                                              # a replay reads the positions of its time
    g.replay()
    check(x, y, 1000 + np.arange(64)[None], None, thetas(64), "interleaved", "bf16")
    # on a stream that is not the current one
    fs.rope(rot, x, y, pos0=5, stream=s)
    s.synchronize()
    check(x, y, 5 + np.arange(64)[None], None, thetas(64), "interleaved", "bf16")
