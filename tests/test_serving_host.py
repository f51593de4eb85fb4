"""Refusals of the serving operators at the borders of their ranges (no GPU needed): every call
here is refused before anything is launched."""
import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("mscale", [3.5e38, -1e300])
def test_rotary_refuses_a_factor_that_float_does_not_hold(mscale):
    with pytest.raises(fs.FsError) as e:
        fs.Rotary(64, mscale=mscale)
    assert e.value.code == 1


# ---------------------------------------------------------------- what the binding passes on
class Seen(Exception):
    pass


@pytest.fixture
def passed(monkeypatch):
    """The binding's calls stop where they would enter the library, with the arguments, and take CPU
    tensors for a device's: what is refused is refused by the check under test."""
    def call(fn, where, dev, stream, *args):
        raise Seen(args)

    monkeypatch.setattr(fs, "_call", call)
    monkeypatch.setattr(fs, "_one_device", lambda where, *tensors: 0)


def cache():
    p = fs.PagedParams(B=2, H=4, Hkv=2, d=64, page_size=16, num_pages=8, max_pages=4)
    K, V, refs, table, lens = fs.alloc_pages(p, "cpu")
    return p, K, V, refs, table, lens, fs.alloc_paged_workspace(p, "cpu")


def test_windows_of_any_size(passed):
    """A window past what the library counts in is the whole sequence, not its remainder by 2^32."""
    p, K, V, _, table, lens, ws = cache()
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for window, want in ((0, 0), (511, 511), (-1, -1), (-7, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                         (2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 32 + 5, -1)):
        with pytest.raises(Seen) as e:
            fs.paged_attend(p, q, K, V, table, lens, torch.zeros_like(q), ws, window=window)
        assert e.value.args[0][7] == want


def test_sizes_past_32_bits_are_refused(passed):
    big = (1 << 32) + 2
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    p, K, V, refs, table, lens, ws = cache()
    rows = torch.zeros((1, 2, 64), dtype=torch.bfloat16).expand(big, 2, 64)
    many = torch.empty(big, dtype=torch.int32, device="meta")
    calls = [
        lambda: fs.rope(fs.Rotary(64), x.expand(1, 1, big, 64), x.expand(1, 1, big, 64)),
        lambda: fs.rope(fs.Rotary(64), x.expand(1, big, 1, 64), x.expand(1, big, 1, 64)),
        lambda: fs.rope(fs.Rotary(64), x, x, x.expand(1, big, 1, 64), x.expand(1, big, 1, 64)),
        lambda: fs.rope_backward(fs.Rotary(64), x.expand(big, 1, 1, 64), x.expand(big, 1, 1, 64)),
        lambda: fs.paged_append(p, rows, rows, K, V, table, lens, ws, cu=torch.zeros(3, dtype=torch.int32)),
        lambda: fs.pages_copy(p, K, V, many, many, ws),
        lambda: fs.pages_fork(p, K, V, refs, table, lens, many, many, ws),
        lambda: fs.pages_free(p, refs, table, lens, many, ws),
        lambda: fs.PagedParams(B=big, H=2, Hkv=2, d=64, page_size=16, num_pages=8, max_pages=4),
        lambda: fs.PagedParams(B=1, H=2, Hkv=2, d=64, page_size=big, num_pages=8, max_pages=4),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.code == 2, i
