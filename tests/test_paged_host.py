"""Refusals of the serving operators, before anything touches a device (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import long_context_sparse_head_b200 as fs

PTR = 0x10000                                  # a stand-in for a device pointer, never followed


def paged(**kw):
    base = dict(B=2, H=4, Hkv=2, d=64, page_size=16, num_pages=8, max_pages=4)
    base.update(kw)
    return fs.PagedParams(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(H=5), 1), (dict(page_size=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages=0), 1), (dict(d=96), 2), (dict(d=0), 1), (dict(num_pages=2000001), 2),
    (dict(max_pages=1 << 26), 2), (dict(dtype="f64"), 1), (dict(layout="other"), 1),
    (dict(strides=(2048, 1024, 32)), 1),       # tokens overlap
    (dict(strides=(1024, 1024, 64)), 1),       # pages overlap
    (dict(strides=(2048, 1024, 72)), 1),       # the last token reaches into the next head
    (dict(strides=(4096, 2048, 68)), 2),       # rows off the 16-byte boundaries
    (dict(strides=(-2048, 1024, 64)), 1),
    (dict(strides=(0, 0, 0)), 1),
])
def test_paged_params_refused(kw, code):
    with pytest.raises(fs.FsError) as e:
        paged(**kw)
    assert e.value.code == code


def test_paged_params_accepted():
    for kw in (dict(), dict(layout="tokens_first"), dict(page_size=1, Hkv=1, H=3, strides=(64, 0, 0)), dict(d=256, dtype="f32"),
               dict(strides=(1 << 33, 1024, 64)), dict(strides=(4096, 1024, 64)), dict(num_pages=1, strides=(0, 1024, 64))):
        assert fs.paged_workspace_size(paged(**kw)) > 0
    # flag and counters lie in the same place whatever the batch; the size covers the larger one
    assert fs.paged_workspace_size(paged(num_pages=100000)) >= fs.paged_workspace_size(paged())


def attend(p, **kw):
    a = dict(Q=PTR, qs=256, K=PTR, V=PTR, table=PTR, lens=PTR, window=-1, scale=0.125, O=PTR, os=256, lse=None, ws=PTR,
             n=1 << 30)
    a.update(kw)
    return fs.load().fs_paged_attend(p.ref(), a["Q"], a["qs"], a["K"], a["V"], a["table"], a["lens"], a["window"],
                                     a["scale"], a["O"], a["os"], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(O=None), 1),
    (dict(ws=None), 3), (dict(n=100), 3), (dict(ws=PTR + 4), 1), (dict(Q=PTR + 2), 1), (dict(K=PTR + 8), 1),
    (dict(qs=260), 2), (dict(os=252), 2), (dict(os=128), 1), (dict(os=0), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
])
def test_attend_refused(kw, code):
    assert attend(paged(), **kw) == code


def test_attend_of_too_much_refused():
    assert attend(paged(B=1 << 20, max_pages=1 << 25)) == 2


def append(p, **kw):
    a = dict(rot=None, T=2, Q=None, qs=0, Qo=None, qos=0, k=PTR, ks=128, v=PTR, vs=128, cu=None, K=PTR, V=PTR, table=PTR,
             lens=PTR, ws=PTR, n=1 << 30)
    a.update(kw)
    rot = a["rot"].ref() if a["rot"] is not None else None
    return fs.load().fs_paged_append(p.ref(), rot, a["T"], a["Q"], a["qs"], a["Qo"], a["qos"], a["k"], a["ks"], a["v"],
                                     a["vs"], a["cu"], a["K"], a["V"], a["table"], a["lens"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=3), 1), (dict(T=-1, cu=PTR), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(K=None), 1), (dict(lens=None), 1),
    (dict(Q=PTR, Qo=PTR, qs=256, qos=256), 1),                               # nothing to do to Q without a rotation
    (dict(Q=PTR, qs=256, rot=fs.Rotary(64)), 1),
    (dict(Q=PTR, Qo=PTR, qs=256, qos=512, rot=fs.Rotary(64)), 1),            # in place with other strides
    (dict(Q=PTR, Qo=PTR + 65536, qs=256, qos=64, rot=fs.Rotary(64)), 1),     # rows of Qo overlap
    (dict(rot=fs.Rotary(128)), 1),                                           # more than a row has
    (dict(ks=132), 2), (dict(vs=132), 2), (dict(k=PTR + 8), 1), (dict(ws=None), 3), (dict(n=64), 3),
])
def test_append_refused(kw, code):
    assert append(paged(), **kw) == code


def test_append_of_nothing():
    assert append(paged(), T=0, cu=PTR, k=None, v=None) == 0


def test_page_calls_refused():
    L, p, n = fs.load(), paged(), 1 << 30
    assert L.fs_pages_copy(p.ref(), PTR, PTR, PTR, PTR, -1, PTR, n, None) == 1
    assert L.fs_pages_copy(p.ref(), PTR, PTR, PTR, PTR, 0, PTR, n, None) == 0
    assert L.fs_pages_copy(p.ref(), None, PTR, PTR, PTR, 1, PTR, n, None) == 1
    assert L.fs_pages_copy(p.ref(), PTR, PTR + 2, PTR, PTR, 1, PTR, n, None) == 1
    assert L.fs_pages_copy(p.ref(), PTR, PTR, PTR, PTR, 1, PTR, 16, None) == 3
    assert L.fs_pages_fork(p.ref(), PTR, PTR, PTR, PTR, PTR, PTR, PTR, 3, PTR, n, None) == 1     # more than sequences
    assert L.fs_pages_fork(p.ref(), PTR, PTR, PTR, PTR, PTR, PTR, PTR, 0, PTR, n, None) == 0
    assert L.fs_pages_fork(p.ref(), PTR, PTR, None, PTR, PTR, PTR, PTR, 1, PTR, n, None) == 1
    assert L.fs_pages_free(p.ref(), PTR, PTR, PTR, PTR, -1, PTR, n, None) == 1
    assert L.fs_pages_free(p.ref(), PTR, PTR, PTR, None, 1, PTR, n, None) == 1
    assert L.fs_pages_free(p.ref(), PTR, PTR, PTR, PTR, 0, PTR, n, None) == 0
    assert L.fs_pages_reserve(p.ref(), None, PTR, PTR, PTR, PTR, n, None) == 1
    assert L.fs_pages_reserve(p.ref(), PTR, PTR + 4, PTR, PTR, PTR, n, None) == 1
    assert L.fs_pages_compact(p.ref(), PTR, PTR, PTR, PTR, None, PTR, None, PTR, n, None) == 1
    assert L.fs_pages_compact(p.ref(), PTR, PTR, PTR, PTR, PTR, PTR, None, None, n, None) == 3
    assert L.fs_paged_workspace_size(p.ref(), None) == 1
    assert L.fs_paged_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == 1


@pytest.mark.parametrize("args,kw,code", [
    ((0,), {}, 1), ((3,), {}, 1), ((-2,), {}, 1), ((258,), {}, 2), ((64, "spiral"), {}, 1), ((64,), dict(base=0.5), 1),
    ((64,), dict(base=math.inf), 1), ((64,), dict(scaling="other"), 1), ((64,), dict(scaling="linear", factor=0.5), 1),
    ((64,), dict(scaling="linear", factor=math.nan), 1), ((2,), dict(scaling="ntk", factor=2.0), 1),
    ((64,), dict(scaling="by_parts", factor=2.0), 1),
    ((64,), dict(scaling="by_parts", factor=2.0, orig_len=4096, slow=4.0, fast=4.0), 1),
    ((64,), dict(mscale=math.nan), 1),
])
def test_rotary_refused(args, kw, code):
    with pytest.raises(fs.FsError) as e:
        fs.Rotary(*args, **kw)
    assert e.value.code == code


def rope(rot, **kw):
    c = fs.FsRopeParams(2, 8, 4, 2, 64)
    for name in ("q", "qo", "k", "ko"):
        heads = 4 if name[0] == "q" else 2
        for x, v in zip("bhn", kw.pop(name + "_strides", (heads * 8 * 64, 8 * 64, 64))):
            setattr(c, name + "_" + x, v)
    c.dtype = kw.pop("dtype", 0)
    a = dict(Q=PTR, Qo=PTR + 65536, K=PTR, Ko=PTR + 65536)
    for n in ("B", "N", "H", "Hk", "d"):
        if n in kw:
            setattr(c, n, kw.pop(n))
    a.update(kw)
    return fs.load().fs_rope(ctypes.byref(c), rot.ref(), a["Q"], a["Qo"], a["K"], a["Ko"], None, 0, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(H=-1), 1), (dict(d=0), 1), (dict(d=32), 1), (dict(d=257), 2), (dict(dtype=3), 1),
    (dict(Q=None), 1), (dict(Ko=None), 1), (dict(qo_strides=(2048, 0, 64)), 1), (dict(ko_strides=(0, 512, 64)), 1),
    (dict(Qo=PTR, qo_strides=(2048, 64, 256)), 1), (dict(Q=PTR + 1), 1), (dict(dtype=1, Q=PTR + 2), 1),
    (dict(B=1 << 16, N=1 << 16), 2), (dict(H=65536), 2),
])
def test_rope_refused(kw, code):
    assert rope(fs.Rotary(64), **kw) == code


def test_rope_of_nothing():
    assert rope(fs.Rotary(64), B=0) == 0 and rope(fs.Rotary(64), N=0) == 0 and rope(fs.Rotary(64), H=0, Hk=0) == 0


def test_frequencies():
    """A pair's fraction of a turn per position, to 2^-65 of a turn."""
    for kw in (dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
               dict(scaling="by_parts", factor=8.0, orig_len=8192, slow=1.0, fast=4.0)):
        from tests._paged import thetas
        rot = fs.Rotary(64, **kw)
        for m, t in enumerate(thetas(64, **{"base": 10000.0, **kw})):
            # float64 holds theta to 2^-53 of itself (a few steps in its computing)
            assert abs(rot.c.turns[m] / 2.0 ** 64 - t / (2 * math.pi)) <= 2.0 ** -49 * t + 2.0 ** -65


def test_binding_checks_its_tensors():
    p = paged()
    K, V, refs, table, lens = fs.alloc_pages(p, "cpu")
    ws = fs.alloc_paged_workspace(p, "cpu")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    calls = [
        lambda: fs.paged_attend(p, q, K, V, table, lens, q, ws),                         # not on a GPU
        lambda: fs.paged_attend(p, q.float(), K, V, table, lens, q, ws),
        lambda: fs.paged_attend(p, q[:1], K, V, table, lens, q, ws),
        lambda: fs.paged_attend(p, q.transpose(0, 1), K, V, table, lens, q, ws),
        lambda: fs.paged_attend(p, q, K.transpose(1, 2), V, table, lens, q, ws),
        lambda: fs.paged_attend(p, q, K, V, table.long(), lens, q, ws),
        lambda: fs.paged_attend(p, q, K, V, table[:, :2], lens, q, ws),
        lambda: fs.paged_attend(p, q, K, V, table, lens, q, ws, lse=torch.zeros((4, 2))),
        lambda: fs.paged_append(p, q, q, K, V, table, lens, ws),                         # 4 heads, not 2
        lambda: fs.paged_append(p, q[:, :2], q[:, :2], K, V, table, lens, ws, Q=q),
        lambda: fs.pages_reserve(p, lens.float(), refs, table, lens, ws),
        lambda: fs.pages_free(p, refs[:4], table, lens, lens, ws),
        lambda: fs.pages_copy(p, K, V, lens, lens[:1], ws),
        lambda: fs.rope(fs.Rotary(64), q, q),
        lambda: fs.rope(fs.Rotary(64), q[None], q[None], q[None]),
        lambda: fs.rope(fs.Rotary(64), q[None], q[None].float()),
        lambda: fs.rope(fs.Rotary(64), q[None].transpose(2, 3), q[None].transpose(2, 3)),
        lambda: fs.rope(fs.Rotary(64), q[None], q[None], positions=torch.zeros(4)),
        lambda: fs.rope(fs.Rotary(64), q[None], q[None], positions=torch.zeros(3, dtype=torch.int32)),
        lambda: fs.rope(fs.Rotary(64), q[None], q[None]),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.code == 1, i


def test_the_forward_pass_refuses_f16():
    with pytest.raises(fs.FsError) as e:
        fs.workspace_size(fs.Params(B=1, H=2, Nq=256, Nk=256, alpha=[0.5, 1.0], dtype="f16"))
    assert e.value.code == 1


def test_position_to_page_arithmetic():
    """The division by a reciprocal that the kernels use, at every page size's borders."""
    for page in list(range(1, 300)) + [511, 512, 513, 4095, 65535, 65536, 65537, (1 << 29) - 1, (1 << 30) - 1]:
        magic = min(0xFFFFFFFF, (1 << 32) // page)
        top = (1 << 30) - 1
        for k in {0, 1, 2, 3, top // page // 2, top // page - 1, top // page}:
            for pos in (k * page - 1, k * page, k * page + 1, k * page + page - 1):
                if not 0 <= pos <= top:
                    continue
                q = pos * magic >> 32
                r = pos - q * page
                if r >= page:
                    q, r = q + 1, r - page
                assert (q, r) == divmod(pos, page)
