"""Refusals of the serving operators at the borders of their ranges (no GPU needed): every call
here is refused before anything is launched."""
import ctypes
import os
import subprocess

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


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def wide(*shape):
    """A tensor of these sizes, its last dimension's elements two apart."""
    return bf(*shape[:-1], 2 * shape[-1])[..., ::2]


def calls():
    """Every serving call with arguments that it takes: name -> (function, arguments)."""
    p, K, V, refs, table, lens, ws = cache()
    rot = fs.Rotary(64)
    base = dict(Kp=K, Vp=V, table=table, lens=lens, ws=ws)
    return {
        "rope": (fs.rope, dict(rotary=rot, Q=bf(2, 4, 8, 64), Qo=bf(2, 4, 8, 64), K=bf(2, 2, 8, 64), Ko=bf(2, 2, 8, 64),
                               positions=i32(2, 8))),
        "rope_backward": (fs.rope_backward, dict(rotary=rot, dQo=bf(2, 4, 8, 64), dQ=bf(2, 4, 8, 64), dKo=bf(2, 2, 8, 64),
                                                 dK=bf(2, 2, 8, 64), positions=i32(8))),
        "append": (fs.paged_append, dict(params=p, K_new=bf(5, 2, 64), V_new=bf(5, 2, 64), cu=i32(3), rotary=rot,
                                         Q=bf(5, 4, 64), Qo=bf(5, 4, 64), **base)),
        "attend": (fs.paged_attend, dict(params=p, Q=bf(2, 4, 64), O=bf(2, 4, 64), lse=torch.zeros(2, 4), **base)),
        "reserve": (fs.pages_reserve, dict(params=p, n_new=i32(2), refs=refs, table=table, lens=lens, ws=ws)),
        "copy": (fs.pages_copy, dict(params=p, Kp=K, Vp=V, src=i32(3), dst=i32(3), ws=ws)),
        "fork": (fs.pages_fork, dict(params=p, refs=refs, src=i32(1), dst=i32(1), **base)),
        "free": (fs.pages_free, dict(params=p, refs=refs, table=table, lens=lens, rows=i32(2), ws=ws)),
        "compact": (fs.pages_compact, dict(params=p, Kp=K, Vp=V, refs=refs, table=table, ws=ws, live=i32(1),
                                           refs_out=i32(8), table_out=i32(2, 4))),
    }


POOL = [bf(7, 2, 16, 64), bf(8, 2, 16, 64).float(), bf(8, 16, 2, 64).transpose(1, 2), wide(8, 2, 16, 64), bf(8, 2, 16, 128)[..., :64]]
TABLE = [i32(2, 3), i32(3, 4), i32(2, 4).long(), i32(2, 8)[:, :4], i32(4, 2).t()]
LENS = [i32(3), i32(2).long(), i32(4)[::2]]
REFS = [i32(7), i32(8).float(), i32(16)[::2]]
ROWS = [bf(4, 2, 64), bf(5, 2, 64).half(), bf(5, 2, 128)[..., :64], wide(5, 2, 64), bf(2, 5, 64).transpose(0, 1), bf(5, 128)]
HEADS = [bf(4, 4, 64), bf(5, 4, 64).float(), bf(5, 4, 128)[..., :64], wide(5, 4, 64), bf(4, 5, 64).transpose(0, 1)]
STEP = [bf(3, 4, 64), bf(2, 2, 64), bf(2, 4, 64).half(), bf(2, 4, 128)[..., :64], wide(2, 4, 64), bf(4, 2, 64).transpose(0, 1)]
LIST = [i32(3).long(), i32(6)[::2], i32(3, 1), i32(2)]
TURNED = [bf(2, 4, 8, 32), bf(2, 4, 7, 64), bf(2, 4, 8, 64).float(), wide(2, 4, 8, 64), bf(2, 4, 64)]
KEYS = [bf(1, 2, 8, 64), bf(2, 2, 7, 64), bf(2, 2, 8, 64).half(), wide(2, 2, 8, 64), bf(2, 8, 64), None]
POS = [i32(7), i32(1, 8), i32(2, 8).long(), i32(2, 16)[:, ::2], torch.zeros(2, 8)]
WRONG = {
    "rope": dict(Q=TURNED, Qo=TURNED, K=KEYS, Ko=KEYS, positions=POS),
    "rope_backward": dict(dQo=TURNED, dQ=TURNED, dKo=KEYS, dK=KEYS, positions=POS),
    "append": dict(K_new=ROWS, V_new=ROWS, Kp=POOL, Vp=POOL, table=TABLE, lens=LENS, cu=[i32(2), i32(4), i32(3).long(), i32(6)[::2]],
                   Q=HEADS + [None], Qo=HEADS + [None]),
    "attend": dict(Q=STEP, O=STEP, Kp=POOL, Vp=POOL, table=TABLE, lens=LENS,
                   lse=[torch.zeros(2, 3), torch.zeros(2, 4).double(), torch.zeros(2, 4).half(), torch.zeros(4, 2).t()]),
    "reserve": dict(n_new=LENS, refs=REFS, table=TABLE, lens=LENS),
    "copy": dict(Kp=POOL, Vp=POOL, src=LIST, dst=LIST),
    "fork": dict(Kp=POOL, Vp=POOL, refs=REFS, table=TABLE, lens=LENS, src=[i32(1).long(), i32(2), i32(1, 1)], dst=[i32(1).long(), i32(2), i32(1, 1)]),
    "free": dict(refs=REFS, table=TABLE, lens=LENS, rows=[i32(2).long(), i32(4)[::2], i32(2, 1)]),
    "compact": dict(Kp=POOL, Vp=POOL, refs=REFS, table=TABLE, refs_out=REFS, table_out=TABLE, live=[i32(2), i32(1).long()]),
}


@pytest.mark.parametrize("name", list(WRONG))
def test_the_binding_takes_what_it_documents(passed, name):
    call, kw = calls()[name]
    with pytest.raises(Seen):
        call(**kw)


@pytest.mark.parametrize("name,arg,i", [(n, a, i) for n, w in WRONG.items() for a, v in w.items() for i in range(len(v))])
def test_the_binding_refuses_each_wrong_tensor(passed, name, arg, i):
    """One argument wrong in its type, sizes or strides, everything else right: refused by the check
    of that argument, since nothing else is there to refuse it."""
    call, kw = calls()[name]
    with pytest.raises(fs.FsError) as e:
        call(**{**kw, arg: WRONG[name][arg][i]})
    assert e.value.code == 1


@pytest.mark.parametrize("name", list(WRONG))
def test_the_binding_refuses_tensors_off_the_gpu(monkeypatch, name):
    """Right in all else."""
    def call(*args):
        raise Seen

    monkeypatch.setattr(fs, "_call", call)
    call, kw = calls()[name]
    with pytest.raises(fs.FsError) as e:
        call(**kw)
    assert e.value.code == 1


def test_a_dimension_of_one_may_have_any_stride(passed):
    p = fs.PagedParams(B=1, H=1, Hkv=1, d=64, page_size=16, num_pages=1, max_pages=4)
    K, V, refs, table, lens = fs.alloc_pages(p, "cpu")
    ws = fs.alloc_paged_workspace(p, "cpu")
    K, V = (x.as_strided((1, 1, 16, 64), (5, 7, 64, 1)) for x in (K, V))
    q = bf(1, 1, 64).as_strided((1, 1, 64), (3, 9, 1))
    with pytest.raises(Seen):
        fs.paged_attend(p, q, K, V, table, lens, q.clone(), ws)
    with pytest.raises(Seen):
        fs.paged_append(p, q, q, K, V, table, lens, ws)
    with pytest.raises(Seen):
        fs.rope(fs.Rotary(64), q.view(1, 1, 1, 64), bf(1, 1, 1, 64), positions=i32(1, 2)[:, ::2])


# ---------------------------------------------------------------- positions to pages
LOCATE = r"""
#include "fs_paged.cuh"
#include <cstdio>
#include <cstdlib>

namespace fs { fs_status paged_dev(const fs_paged_params *p, PagedDev *out); }

int main() {
    const int top = (1 << 30) - 1;
    long long seen = 0, wrong = 0;
    auto check = [&](const fs::PagedDev &P, long long pos) {
        if (pos < 0 || pos > top) return;
        int idx, slot;
        P.locate((int)pos, idx, slot);
        seen++;
        wrong += idx != pos / P.ps || slot != pos % P.ps || P.pages_of((int)pos) != (pos + P.ps - 1) / P.ps;
    };
    auto all = [&](int page) {
        fs_paged_params p = {};
        p.B = p.H = p.Hkv = p.num_pages = p.max_pages = 1;
        p.d = 64;
        p.page_size = page;
        p.token_stride = 64;
        fs::PagedDev P;
        // the head's 2^30 elements limit a page of one head to 2^24 tokens
        if (page > 1 << 24) return;
        if (fs::paged_dev(&p, &P) != FS_OK) exit(2);
        const long long last = top / page;
        for (long long k : {0ll, 1ll, 2ll, 3ll, last / 3, last / 2, last - 1, last})
            for (long long e = -2; e <= 2; e++) check(P, k * page + e), check(P, k * page + page / 2 + e);
        check(P, top);
        unsigned x = 12345u + page;
        for (int i = 0; i < 200; i++) check(P, (x = x * 1664525u + 1013904223u) >> 2);
    };
    for (int page = 1; page <= 20000; page++) all(page);
    for (int bit = 1; bit <= 24; bit++)
        for (int e = -1; e <= 1; e++) all((1 << bit) + e > 0 ? (1 << bit) + e : 1);
    printf("%lld %lld\n", seen, wrong);
    return wrong != 0;
}
"""


def test_position_to_page(tmp_path):
    """The kernels' own division by a reciprocal, compiled for the host, at the borders of every page
    size to 20000 and of the larger powers of two."""
    from long_context_sparse_head_b200 import build
    (tmp_path / "locate.cu").write_text(LOCATE)
    cmd = [build.NVCC] + build.ARCH + build.FLAGS + ["-I", build.CSRC, str(tmp_path / "locate.cu"), fs.LIB_PATH,
                                                     "-o", str(tmp_path / "locate")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(tmp_path / "locate")], capture_output=True, text=True,
                       env={**os.environ, "LD_LIBRARY_PATH": os.path.dirname(fs.LIB_PATH)})
    seen, wrong = (int(x) for x in r.stdout.split())
    assert r.returncode == 0 and wrong == 0 and seen > 4e6
