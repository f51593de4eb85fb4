"""Calls of the serving operators at the borders of what their documentation allows, on the GPU."""
import numpy as np
import pytest
import torch

import long_context_sparse_head_b200 as fs
from tests._paged import DTYPES, HALF_STEP, Book, attend, rotate, rotate_bound, thetas

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 11), (256, 16)])
@pytest.mark.parametrize("gap", [8.0, 12.0, 15.7, 17.5, 20.0])
def test_attend_weighs_a_long_tail_under_one_peak(dtype, d, group, gap):
    """One key `gap` above all others, its value 0: the output is what the others' small
    probabilities add up to.  So many sequences that no row is cut: the peak's warp holds a quarter
    of the tail."""
    n, B, page = 2048, 300, 32
    p = fs.PagedParams(B=B, H=2 * group, Hkv=2, d=d, page_size=page, num_pages=3 * n // page, max_pages=n // page,
                       dtype=dtype)
    K, V, _, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    K.zero_()
    V.copy_(torch.rand(p.shape, generator=torch.Generator().manual_seed(d)) + 0.5)
    lens.fill_(n)
    scale = d ** -0.5
    at = (0, 1000, n - 1)                                    # the peak's place: three kinds of sequence share the pages
    for i, t in enumerate(at):
        pages = np.arange(i * (n // page), (i + 1) * (n // page))
        K[int(pages[t // page]), :, t % page, 0] = gap / scale
        V[int(pages[t // page]), :, t % page] = 0
        table[i::3] = ints(pages)
    q = torch.zeros((B, 2 * group, d), dtype=DTYPES[dtype], device="cuda")
    q[..., 0] = 1
    o, lse = torch.empty_like(q), torch.empty((B, 2 * group), device="cuda")
    fs.paged_attend(p, q, K, V, table, lens, o, ws, lse=lse)
    fs.sync_status(ws)
    for i in range(3):
        for h in range(2):
            k, v = (f64(x[i * (n // page):(i + 1) * (n // page), h].flatten(0, 1)) for x in (K, V))
            want, l, _ = attend(f64(q[i, :1]), k, v, scale)
            # scores have one term: its rounding, the factor's and the exponent's, 2^-22 of the gap in
            # all, and 2^-20 for the exponential; n sums of 2^-23; a probability's two parts lose 2^-16
            # of it, in f16 or 2^-40 of the largest; the output's own rounding
            rel = 2 * (gap * 2.0 ** -22 + 2.0 ** -20) + n * 2.0 ** -23 + (0.0 if dtype == "f32" else 2.0 ** -16)
            bound = np.abs(want) * (rel + HALF_STEP[dtype]) + (n * 2.0 ** -40 * 1.5 + 2.0 ** -25 if dtype == "f16" else 0.0)
            assert (np.abs(f64(o[i::3, h * group:(h + 1) * group]) - want) <= bound).all(), (i, h)
            assert (np.abs(f64(lse[i::3, h * group:(h + 1) * group]) - l) <= rel + gap * 2.0 ** -22).all()


# ---------------------------------------------------------------- writing
def test_append_with_the_most_rows():
    """2^31 - 1 rows, of which five are tokens and the others padding."""
    T = 2 ** 31 - 1
    p = fs.PagedParams(B=1, H=1, Hkv=1, page_size=4, num_pages=3, max_pages=2)
    K, V, _, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    K.fill_(7)
    V.fill_(7)
    table.copy_(ints([[2, 0]]))
    lens.fill_(6)
    k = torch.full((1, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda").expand(T, 1, 64)
    fs.paged_append(p, k, k, K, V, table, lens, ws, cu=ints([0, 5]))
    fs.sync_status(ws)
    for x in (K, V):
        assert x[2, 0, :, 5].tolist() == [7, 3, 3, 3] and x[0, 0, :, 5].tolist() == [3, 3, 7, 7] and (x[1] == 7).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_of_one_token_with_the_most_heads(layout):
    """More rows for a token than a grid's second dimension counts."""
    H = 65535
    p = fs.PagedParams(B=1, H=H, Hkv=H, page_size=2, num_pages=1, max_pages=1)
    K, V, _, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    table.zero_()
    lens.fill_(2)
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((1, H, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    qo = torch.empty_like(q)
    fs.paged_append(p, k, v, K, V, table, lens, ws, rotary=fs.Rotary(64, layout), Q=q, Qo=qo)
    fs.sync_status(ws)
    for x, got in ((q[0], qo[0]), (k[0], K[0, :, 1])):
        a = f64(x)
        want = rotate(a, 1, thetas(64), layout)
        assert (np.abs(f64(got) - want) <= rotate_bound(a, want, 64, layout, "bf16")).all()
    assert torch.equal(V[0, :, 1], v[0])


def test_append_reports_rows_that_are_counted_but_not_given():
    """cu counts nine tokens, the call brings five rows: those are written, and it is reported that
    the others, which lens counts too, were not."""
    p = fs.PagedParams(B=2, H=1, Hkv=1, page_size=4, num_pages=4, max_pages=2)
    K, V, _, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    K.fill_(7)
    V.fill_(7)
    table.copy_(ints([[2, -1], [0, 3]]))
    lens.copy_(ints([3, 6]))
    k = torch.arange(1, 6, device="cuda").to(torch.bfloat16)[:, None, None].expand(5, 1, 64).contiguous()
    fs.paged_append(p, k, -k, K, V, table, lens, ws, cu=ints([0, 3, 9]))
    with pytest.raises(fs.FsError) as e:
        fs.sync_status(ws)
    assert e.value.code == 6
    assert K[2, 0, :, 0].tolist() == [1, 2, 3, 7] and K[0, 0, :, 0].tolist() == [4, 5, 7, 7]
    assert V[2, 0, :, 0].tolist() == [-1, -2, -3, 7] and V[0, 0, :, 0].tolist() == [-4, -5, 7, 7]
    fs.paged_append(p, k, -k, K, V, table, lens, ws, cu=ints([0, 3, 5]))     # exactly as many
    fs.sync_status(ws)


# ---------------------------------------------------------------- rotary positions
def test_rope_of_the_most_tokens():
    """2^31 - 1 tokens: the last block's threads stand past the last of them."""
    T = 2 ** 31 - 1
    x = torch.empty((T, 2), dtype=torch.float16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, -0.5
    a = np.broadcast_to(np.array([1.0, -0.5]), (300, 2)).copy()
    q = x.view(1, 1, T, 2)
    fs.rope(fs.Rotary(2), q, q)
    for first in (0, 2 ** 30 - 150, T - 300):
        want = rotate(a, np.arange(first, first + 300), thetas(2), "interleaved")
        assert (np.abs(f64(x[first:first + 300]) - want) <= rotate_bound(a, want, 2, "interleaved", "f16")).all()


# ---------------------------------------------------------------- several rows a thread, as long prompts take them
def turn64(x, pos, theta, layout, sign=1.0):
    """rotate() on the GPU: x [..., d] in 64 bits, pos broadcastable to x.shape[:-1]."""
    r, x = 2 * len(theta), x.double()
    a = pos.double()[..., None] * torch.tensor(theta, device="cuda")
    c, s = torch.cos(a), torch.sin(a) * sign
    i, j = (slice(0, r, 2), slice(1, r, 2)) if layout == "interleaved" else (slice(0, r // 2), slice(r // 2, r))
    y = x.clone()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def near(got, x, want, r, layout, dtype):
    """rotate_bound() on the GPU."""
    i, j = (slice(0, r, 2), slice(1, r, 2)) if layout == "interleaved" else (slice(0, r // 2), slice(r // 2, r))
    both = torch.zeros_like(want)
    both[..., i] = both[..., j] = x[..., i].double().abs() + x[..., j].double().abs()
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    return bool(((got.double() - want).abs() <= both * 2.0 ** -21 + want.abs() * HALF_STEP[dtype] + tiny).all())


def tokens_for(rows, units, per_thread):
    """As few tokens of `rows` rows of `units` threads each as make a thread take per_thread rows: two
    threads are left for every one of 148 x 2048."""
    return -(-2 * 148 * 2048 // (units * -(-rows // per_thread)))


@pytest.mark.parametrize("dtype,layout,d,r,units", [("bf16", "interleaved", 64, 64, 8), ("bf16", "half", 64, 64, 4),
                                                    ("f32", "half", 128, 64, 24), ("f16", "interleaved", 64, 6, 32)])
@pytest.mark.parametrize("H,Hk,per_thread", [(5, 2, 2), (5, 2, 4), (5, 2, 32), (33, 8, 32)])
def test_rope_with_several_heads_a_thread(dtype, layout, d, r, units, H, Hk, per_thread):
    """Blocks that hold the last of the queries' heads and the first of the keys'; forward, gradient,
    in place."""
    N = tokens_for(H + Hk, units, per_thread) // 2 + 1
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k = (torch.randn((2, N, h, d), generator=g, device="cuda").to(DTYPES[dtype]).transpose(1, 2) for h in (H, Hk))
    pos = torch.randint(0, 1 << 20, (2, N), generator=g, device="cuda", dtype=torch.int32)
    rot, theta = fs.Rotary(r, layout), thetas(r)
    for fn, sign in ((fs.rope, 1.0), (fs.rope_backward, -1.0)):
        qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
        fn(rot, q, qo, k, ko, positions=pos)
        for x, y in ((q, qo), (k, ko)):
            for b in range(2):
                assert near(y[b], x[b], turn64(x[b], pos[b], theta, layout, sign), r, layout, dtype)
    fs.rope_backward(rot, q, q, k, k, positions=pos)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype,layout,d,r,units", [("bf16", "interleaved", 64, 64, 8), ("f16", "half", 64, 64, 4),
                                                    ("f32", "half", 128, 128, 16), ("bf16", "half", 64, 24, 32),
                                                    ("f32", None, 64, 0, 16)])
@pytest.mark.parametrize("per_thread", [2, 4, 8, 32])
@pytest.mark.parametrize("pool", ["heads_first", "tokens_first"])
def test_append_with_several_rows_a_thread(dtype, layout, d, r, units, per_thread, pool):
    """Blocks that hold queries, keys and values of a token; ragged prompts, one behind tokens written
    before, rows of padding."""
    H, Hkv, page, pad = 9, 3, 16, 3
    T = tokens_for((H if r else 0) + 2 * Hkv, units, per_thread) + 1
    new = [T // 2 - 40, 0, 1, 37, T - T // 2 + 2, 0]
    assert sum(new) == T
    old = [0, 5, 16, 3, 0, 0]
    lens = [a + b for a, b in zip(old, new)]
    need = [-(-n // page) for n in lens]
    p = fs.PagedParams(B=6, H=H, Hkv=Hkv, d=d, page_size=page, num_pages=sum(need) + 2, max_pages=max(need), dtype=dtype,
                       layout=pool)
    K, V, refs, table, ln = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    fs.pages_reserve(p, ints(lens), refs, table, ln, ws)
    K.fill_(7)
    V.fill_(7)
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn((T + pad, h, d), generator=g, device="cuda").to(DTYPES[dtype]) for h in (H, Hkv, Hkv))
    qo = torch.full_like(q, 9.0)
    cu = np.concatenate([[0], np.cumsum(new)])
    kw = dict(rotary=fs.Rotary(r, layout), Q=q, Qo=qo) if r else {}
    fs.paged_append(p, k, v, K, V, table, ln, ws, cu=ints(cu), **kw)
    fs.sync_status(ws)
    pos = torch.tensor(np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]), device="cuda")
    seq = torch.tensor(np.repeat(np.arange(6), new), device="cuda")
    at = (table[seq, pos // page].long(), slice(None), pos % page)
    assert torch.equal(V[at], v[:T])
    if r:
        for x, y in ((k[:T], K[at]), (q[:T], qo[:T])):
            assert near(y, x, turn64(x, pos[:, None], thetas(r), layout), r, layout, dtype)
    else:
        assert torch.equal(K[at], k[:T])
    assert (qo[T:] == 9).all()
    for x in (K, V):
        x[at] = 7
        assert (x == 7).all()


# ---------------------------------------------------------------- streams and graphs
def test_two_caches_are_written_and_read_on_two_streams():
    """Appends and attention of two caches, each with its own workspace, side by side on two streams:
    the results of one after the other, bit for bit."""
    def start(seed):
        p = fs.PagedParams(B=3, H=8, Hkv=2, page_size=16, num_pages=400, max_pages=200)
        K, V, refs, table, lens = fs.alloc_pages(p)
        ws = fs.alloc_paged_workspace(p)
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        T = 2500 + 100 + 700
        return dict(p=p, K=K, V=V, refs=refs, table=table, lens=lens, ws=ws, first=ints([2500, 100, 700]), one=ints([1, 1, 1]),
                    cu=ints([0, 2500, 2600, 3300]), k=draw(T, 2, 64), v=draw(T, 2, 64), steps=[
                        (draw(3, 8, 64), draw(3, 2, 64), draw(3, 2, 64)) for _ in range(12)], rot=fs.Rotary(64, "half"), out=[])

    def calls(s):
        """The run's calls, one at a time."""
        p, rest = s["p"], (s["K"], s["V"], s["table"], s["lens"])
        fs.pages_reserve(p, s["first"], s["refs"], s["table"], s["lens"], s["ws"])
        yield
        fs.paged_append(p, s["k"], s["v"], *rest, s["ws"], cu=s["cu"], rotary=s["rot"])
        yield
        for q, k, v in s["steps"]:
            fs.pages_reserve(p, s["one"], s["refs"], s["table"], s["lens"], s["ws"])
            yield
            qr, o = torch.empty_like(q), torch.empty_like(q)
            fs.paged_append(p, k, v, *rest, s["ws"], rotary=s["rot"], Q=q, Qo=qr)
            yield
            fs.paged_attend(p, qr, *rest, o, s["ws"])
            s["out"].append((qr, o))
            yield

    alone, both = [start(1), start(2)], [start(1), start(2)]
    for s in alone:
        for _ in calls(s):
            pass
    torch.cuda.synchronize()
    streams, runs = [torch.cuda.Stream() for _ in both], [calls(s) for s in both]
    more = True
    while more:
        more = False
        for st, r in zip(streams, runs):
            with torch.cuda.stream(st):
                more |= next(r, "done") != "done"
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        fs.sync_status(a["ws"])
        fs.sync_status(b["ws"])
        assert torch.equal(a["table"], b["table"]) and torch.equal(a["lens"], b["lens"]) and torch.equal(a["refs"], b["refs"])
        for (q1, o1), (q2, o2) in zip(a["out"], b["out"]):
            assert torch.equal(q1, q2) and torch.equal(o1, o2) and o1.isfinite().all()


@pytest.mark.parametrize("pages", [200, 5000])
def test_page_calls_captured(pages):
    """A beam step and a packing in one graph: every replay acts on the tables of its time.  One CTA for
    the plans, and a cluster of them."""
    B, page, width = 12, 8, 12
    p = fs.PagedParams(B=B, H=2, Hkv=2, page_size=page, num_pages=pages, max_pages=width, dtype="f32")
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    book, rng = Book(B, pages, width, page), np.random.default_rng(pages)
    n = rng.integers(1, 60, B).tolist()
    assert book.reserve(n)
    fs.pages_reserve(p, ints(n), refs, table, lens, ws)
    K.copy_(torch.arange(K.numel(), device="cuda").view(K.shape) % 8191)
    V.copy_(-K)
    drop, src, dst, new, live = ints([6, 7, 8]), ints([0, 1, 0]), ints([6, 7, 8]), ints([0] * B), ints([0])
    one, two = ints([0]), ints([pages - 1])

    def beam():
        fs.pages_free(p, refs, table, lens, drop, ws)
        fs.pages_fork(p, K, V, refs, table, lens, src, dst, ws)
        fs.pages_reserve(p, new, refs, table, lens, ws)
        fs.pages_compact(p, K, V, refs, table, ws, live=live)
        fs.pages_copy(p, K, V, one, two, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beam()
    for step in range(6):
        rows = rng.permutation(B)
        a, b, m = rows[:3].tolist(), rows[3:6].tolist(), rng.integers(0, 3, B).tolist()
        drop.copy_(ints(b))
        dst.copy_(ints(b))
        src.copy_(ints(a))
        new.copy_(ints(m))
        want = K.clone()
        book.free(b)
        for x, y, t in book.fork(a, b):
            want[y, :, :t] = want[x, :, :t]
        assert book.reserve(m)
        for x, y in book.compact().items():
            want[y] = want[x]
        want[pages - 1] = want[0]
        graph.replay()
        fs.sync_status(ws)
        assert refs.tolist() == book.refs and table.tolist() == book.table and lens.tolist() == book.lens
        assert live.item() == sum(x > 0 for x in book.refs)
        assert torch.equal(K, want) and torch.equal(V, -want)
