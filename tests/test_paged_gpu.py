"""The paged cache on the GPU: writing tokens, attention over the pages, the pages themselves, and
a run of them together, against float64 forms and bookkeeping in Python."""
import numpy as np
import pytest
import torch

import long_context_sparse_head_b200 as fs
from tests._paged import DTYPES, Book, attend, attend_bounds, rotate, rotate_bound, thetas

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """A cache with the given lengths: pages in random order, values from the seed, NaN in every
    slot that holds no token."""

    def __init__(self, lens, *, H, Hkv, d=64, page=16, dtype="bf16", layout="heads_first", seed=0, spare=3, width=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.width = max([1] + need) if width is None else width
        self.p = fs.PagedParams(B=len(lens), H=H, Hkv=Hkv, d=d, page_size=page, num_pages=sum(need) + spare,
                                max_pages=self.width, dtype=dtype, layout=layout)
        self.K, self.V, _, self.table, self.lens = fs.alloc_pages(self.p)
        self.ws = fs.alloc_paged_workspace(self.p)
        g = torch.Generator().manual_seed(seed)
        pages = sum(need) + spare
        for x in (self.K, self.V):
            x.copy_(torch.randn((pages, Hkv, page, d), generator=g).to(DTYPES[dtype]))
        order = rng.permutation(sum(need) + spare)
        table, at, used = np.full((len(lens), self.width), -1), 0, np.zeros((sum(need) + spare, page), bool)
        for b, n in enumerate(lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            for t in range(need[b]):
                used[table[b, t], :max(0, min(page, n - t * page))] = True
        empty = torch.tensor(~used, device="cuda")[:, None, :, None]
        for x in (self.K, self.V):
            x.masked_fill_(empty, float("nan"))
        self.table.copy_(ints(table))
        self.lens.copy_(ints(lens))
        self.n, self.rows, self.dtype = lens, table, dtype
        self.q = torch.randn((len(lens), H, d), generator=g).to(DTYPES[dtype]).cuda()

    def tokens(self, x, b, h, a, n):
        pages = torch.tensor(self.rows[b, :-(-n // self.p.page_size)], device="cuda")
        return f64(x[pages, h].flatten(0, 1)[a:n]) if n else np.zeros((0, self.p.d))

    def run(self, window=-1, scale=None, out=None):
        o = torch.full_like(self.q, float("nan")) if out is None else out
        lse = torch.full((self.p.B, self.p.H), float("nan"), device="cuda")
        fs.paged_attend(self.p, self.q, self.K, self.V, self.table, self.lens, o, self.ws, lse=lse, window=window,
                        scale=scale)
        fs.sync_status(self.ws)
        return o, lse

    def check(self, o, lse, window=-1, scale=None):
        p = self.p
        scale = p.d ** -0.5 if scale is None else scale
        G, got, got_lse = p.H // p.Hkv, f64(o), f64(lse)
        assert np.isfinite(got).all()
        for b, n in enumerate(self.n):
            a = max(0, n - 1 - window) if window >= 0 else 0
            for h in range(p.Hkv):
                q = f64(self.q[b, h * G:(h + 1) * G])
                k, v = self.tokens(self.K, b, h, a, n), self.tokens(self.V, b, h, a, n)
                want, l, av = attend(q, k, v, scale)
                bo, bl = attend_bounds(q, k, want, l, av, scale, self.dtype)
                assert (np.abs(got[b, h * G:(h + 1) * G] - want) <= bo).all(), (b, n, h)
                gl = got_lse[b, h * G:(h + 1) * G]
                if n == 0:
                    assert (gl == -np.inf).all() and (got[b, h * G:(h + 1) * G] == 0).all()
                else:
                    assert (np.abs(gl - l) <= bl).all(), (b, n, h)


# ---------------------------------------------------------------- attention
LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 0, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 11])
def test_attend_lengths_and_groups(dtype, d, group):
    c = Cache(LENS, H=2 * group, Hkv=2, d=d, page=16, dtype=dtype, seed=d + group)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 7, 24, 32, 100, 256])
@pytest.mark.parametrize("layout", ["heads_first", "tokens_first"])
def test_attend_page_sizes_and_layouts(dtype, page, layout):
    """Pages that end inside a tile, pages longer than one."""
    c = Cache(LENS, H=6, Hkv=3, page=page, dtype=dtype, layout=layout, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 1, 31, 64, 100, 512, 5000])
def test_attend_window(dtype, window):
    c = Cache([0, 1, 33, 101, 600, 1111], H=4, Hkv=2, d=128, page=8, dtype=dtype, seed=window)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("dtype,H,Hkv,d", [("bf16", 4, 1, 64), ("f16", 40, 1, 128), ("f32", 20, 2, 64), ("bf16", 1, 1, 256)])
def test_attend_long_sequences_are_split_and_joined(dtype, H, Hkv, d):
    """Rows cut over many CTAs beside short ones; larger groups than one tile of heads."""
    c = Cache([30011, 5, 0, 4096, 1], H=H, Hkv=Hkv, d=d, page=32, dtype=dtype, seed=H)
    o, lse = c.run(scale=0.3)
    c.check(o, lse, scale=0.3)
    again, lse2 = c.run(scale=0.3)
    assert torch.equal(o, again) and torch.equal(lse, lse2)      # joined in a fixed order


def test_attend_many_sequences():
    lens = np.random.default_rng(5).integers(0, 90, 700).tolist()
    c = Cache(lens, H=2, Hkv=1, page=16, seed=5)
    c.check(*c.run())


def test_attend_peaked_scores():
    """One key far above the rest, early and late: the running maximum moves once, or at the end."""
    for at in (0, 700, 1999):
        c = Cache([2000], H=2, Hkv=1, page=16, dtype="f32", seed=at)
        c.K[c.rows[0, at // 16], 0, at % 16] = c.q[0, 0] * 3
        c.check(*c.run())


def test_attend_infinite_and_nan_values():
    """A NaN key reaches every output of its sequence and no other; an infinite value its column (as
    infinity, or as NaN where a probability's two parts differ in sign or one is zero)."""
    c = Cache([100, 100], H=2, Hkv=1, page=16, dtype="bf16", seed=8)
    c.K[c.rows[0, 3], 0, 5, 7] = float("nan")
    c.V[c.rows[1, 3], 0, 5, 7] = float("inf")
    o, _ = c.run()
    assert torch.isnan(o[0]).all()
    assert not torch.isfinite(o[1, :, 7]).any() and torch.isfinite(o[1, :, :7]).all() and torch.isfinite(o[1, :, 8:]).all()


def test_attend_strided_queries_and_outputs():
    """Queries inside a fused projection's rows, outputs inside wider rows, which stay as they were."""
    c = Cache([40, 300, 7], H=4, Hkv=2, seed=9)
    rows = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    c.q = rows[:, :256].view(3, 4, 64)
    wide = torch.full((3, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, 64:].view(3, 4, 64)
    _, lse = c.run(out=o)
    c.check(o, lse)
    assert (wide[:, :64] == 5).all()


def test_attend_workspace_serves_other_batches():
    """One workspace, made for the largest: calls of other sizes and head dims in between."""
    big = Cache([3000, 900, 4000], H=16, Hkv=1, d=256, page=16, seed=10)
    small = Cache([2500, 7], H=2, Hkv=2, d=64, page=16, dtype="f32", seed=11)
    small.ws = big.ws
    for _ in range(3):
        big.check(*big.run())
        small.check(*small.run())


def test_attend_captured_step_follows_lens():
    """One graph of a step serves every length; two graphs share the workspace in turn."""
    c = Cache([900, 40, 0], H=4, Hkv=2, page=16, seed=12)
    o, lse = torch.zeros_like(c.q), torch.zeros((3, 4), device="cuda")
    graphs = []
    for w in (-1, 50):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fs.paged_attend(c.p, c.q, c.K, c.V, c.table, c.lens, o, c.ws, lse=lse, window=w)
        graphs.append(g)
    for n in ([900, 40, 0], [17, 0, 0], [850, 33, 0]):
        c.lens.copy_(ints(n))
        c.n = n
        for g, w in zip(graphs, (-1, 50)):
            g.replay()
            torch.cuda.synchronize()
            c.check(o, lse, window=w)


def test_attend_offsets_past_32_bits():
    """Pages more than 2^32 elements apart."""
    far = (1 << 32) + 1024
    p = fs.PagedParams(B=1, H=2, Hkv=2, page_size=16, num_pages=2, max_pages=2, strides=(far, 1024, 64))
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    x = torch.randn((2, 2, 2, 16, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    K.copy_(x[0])
    V.copy_(x[1])
    fs.pages_copy(p, K, V, ints([0]), ints([1]), ws)
    assert torch.equal(K[1], x[0, 0]) and torch.equal(V[1], x[1, 0])
    K[1].copy_(x[0, 1])
    V[1].copy_(x[1, 1])
    table.copy_(ints([[1, 0]]))
    lens.copy_(ints([30]))
    q = torch.randn((1, 2, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    o = torch.empty_like(q)
    fs.paged_attend(p, q, K, V, table, lens, o, ws)
    fs.sync_status(ws)
    for h in range(2):
        k, v = (f64(t[[1, 0], h].flatten(0, 1)[:30]) for t in (K, V))
        want, l, av = attend(f64(q[0, h:h + 1]), k, v, 0.125)
        assert (np.abs(f64(o[0, h:h + 1]) - want) <= attend_bounds(f64(q[0, h:h + 1]), k, want, l, av, 0.125, "bf16")[0]).all()


def test_attend_reports_bad_pages_and_lengths():
    """The kernel's own checks: an entry outside the pool or a length past the row is reported, the
    other sequences are answered."""
    for bad_page, bad_len in ((-1, None), (1 << 20, None), (None, 10 ** 6), (None, -5)):
        c = Cache([100, 300], H=2, Hkv=1, seed=13)
        if bad_page is not None:
            c.table[0, 2] = bad_page
        if bad_len is not None:
            c.lens[0] = bad_len
        o = torch.empty_like(c.q)
        lse = torch.empty((2, 2), device="cuda")
        fs.paged_attend(c.p, c.q, c.K, c.V, c.table, c.lens, o, c.ws, lse=lse)
        with pytest.raises(fs.FsError) as e:
            fs.sync_status(c.ws)
        assert e.value.code == 6
        fs.sync_status(c.ws)                                 # the flag was cleared
        q, k, v = f64(c.q[1]), c.tokens(c.K, 1, 0, 0, 300), c.tokens(c.V, 1, 0, 0, 300)
        want, l, av = attend(q, k, v, 0.125)
        assert (np.abs(f64(o[1]) - want) <= attend_bounds(q, k, want, l, av, 0.125, "bf16")[0]).all()


def test_attend_is_the_window_branch():
    """Rotated keys in pages and the look-back window: o^sr of eq. (3), as fs_forward with alpha 0
    computes it from the contiguous archive for its newest token."""
    N, H, w = 700, 2, 128
    g = torch.Generator().manual_seed(14)
    Q, K, V = (torch.randn((1, H, n, 64), generator=g).to(torch.bfloat16).cuda() for n in (1, N, N))
    p = fs.Params(B=1, H=H, Nq=1, Nk=N, w=w, K=0, alpha=[0.0] * H)
    O = torch.empty_like(Q)
    ws = fs.alloc_workspace(p)
    fs.forward(p, Q, K, V, O, ws)
    fs.sync_status(ws)
    pp = fs.PagedParams(B=1, H=H, Hkv=H, page_size=32, num_pages=30, max_pages=30)
    Kp, Vp, refs, table, lens = fs.alloc_pages(pp)
    pws = fs.alloc_paged_workspace(pp)
    fs.pages_reserve(pp, ints([N]), refs, table, lens, pws)
    rot, q = fs.Rotary(64), torch.empty((1, H, 64), dtype=Q.dtype, device="cuda")
    fs.paged_append(pp, K[0].transpose(0, 1).contiguous(), V[0].transpose(0, 1).contiguous(), Kp, Vp, table, lens, pws,
                    cu=ints([0, N]), rotary=rot)
    fs.rope(rot, Q, q.view(1, H, 1, 64), pos0=N - 1)
    o = torch.empty_like(q)
    fs.paged_attend(pp, q, Kp, Vp, table, lens, o, pws, window=w)
    fs.sync_status(pws)
    # both round rotated queries, keys and probabilities to bf16 and hold 2e-2 against the formula
    assert (o.float() - O[:, :, 0].float()).abs().max() <= 2e-2


# ---------------------------------------------------------------- writing
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout,r", [("interleaved", 64), ("half", 64), ("half", 24), ("interleaved", 6), (None, 0)])
@pytest.mark.parametrize("pool", ["heads_first", "tokens_first"])
def test_append_ragged(dtype, layout, r, pool):
    lens, new = [5, 0, 40, 33, 100, 7], [5, 0, 1, 20, 64, 0]
    c = Cache(lens, H=4, Hkv=2, page=8, dtype=dtype, layout=pool, seed=r)
    K0, V0 = c.K.clone(), c.V.clone()
    T, pad = sum(new), 5
    g = torch.Generator().manual_seed(1)
    rows = torch.randn((T + pad, 8, 64), generator=g).to(DTYPES[dtype]).cuda()      # a fused projection
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    cu = np.concatenate([[0], np.cumsum(new)])
    rot = fs.Rotary(r, layout) if r else None
    qo = torch.full((T + pad, 4, 64), 9.0, dtype=DTYPES[dtype], device="cuda")
    kw = dict(rotary=rot, Q=q, Qo=qo) if r else {}
    fs.paged_append(c.p, k, v, c.K, c.V, c.table, c.lens, c.ws, cu=ints(cu), **kw)
    fs.sync_status(c.ws)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    seq = np.repeat(np.arange(6), new)
    page, slot = c.rows[seq, pos // 8], pos % 8
    at = (torch.tensor(page, device="cuda"), slice(None), torch.tensor(slot, device="cuda"))
    theta = thetas(r) if r else np.zeros(0)
    lay = layout or "half"
    for x, got in ((k[:T], c.K[at]), (q[:T], qo[:T]))[:2 if r else 1]:
        a = f64(x)
        want = rotate(a, pos[:, None], theta, lay)
        assert (np.abs(f64(got) - want) <= rotate_bound(a, want, r, lay, dtype)).all()
    assert torch.equal(c.V[at], v[:T])
    assert (qo[T:] == 9).all() and (r or (qo == 9).all())
    # every other slot keeps its bytes (NaN among them)
    for x, x0 in ((c.K, K0), (c.V, V0)):
        x[at] = x0[at]
        assert torch.equal(torch.nan_to_num(x, nan=77.0), torch.nan_to_num(x0, nan=77.0))


@pytest.mark.parametrize("B", [1, 3, 300])
def test_append_step_in_place(B):
    lens = np.random.default_rng(B).integers(0, 50, B).tolist()
    c = Cache(lens, H=2, Hkv=1, page=16, dtype="f32", seed=B)
    g = torch.Generator().manual_seed(B)
    k, v = (torch.randn((B, 1, 64), generator=g).cuda() for _ in range(2))
    q = c.q.clone()
    fs.paged_append(c.p, k, v, c.K, c.V, c.table, c.lens, c.ws, rotary=fs.Rotary(64), Q=q, Qo=q)
    fs.sync_status(c.ws)
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.equal(q[b], c.q[b])                 # skipped
            continue
        pi, slot = divmod(n - 1, 16)
        for x, got in ((k[b], c.K[c.rows[b, pi], :, slot]), (c.q[b], q[b])):
            a = f64(x)
            want = rotate(a, n - 1, thetas(64), "interleaved")
            assert (np.abs(f64(got) - want) <= rotate_bound(a, want, 64, "interleaved", "f32")).all()
        assert torch.equal(c.V[c.rows[b, pi], :, slot], v[b])


def test_append_finds_sequences_among_many():
    """More sequences than a block has threads, most of them empty."""
    B = 5000
    lens = np.zeros(B, int)
    lens[[0, 17, 255, 256, 2500, 4999]] = [3, 1, 40, 2, 9, 1]
    c = Cache(lens.tolist(), H=1, Hkv=1, page=16, seed=3)
    T = int(lens.sum())
    k = torch.arange(T, device="cuda").to(torch.bfloat16)[:, None, None].expand(T, 1, 64).contiguous()
    cu = np.concatenate([[0], np.cumsum(lens)])
    fs.paged_append(c.p, k, k, c.K, c.V, c.table, c.lens, c.ws, cu=ints(cu))
    fs.sync_status(c.ws)
    for b in np.nonzero(lens)[0]:
        assert np.array_equal(c.tokens(c.K, b, 0, 0, lens[b])[:, 0], np.arange(cu[b], cu[b + 1]))


def test_append_reports_tokens_without_a_place():
    for what in ("page", "short", "long"):
        c = Cache([20, 30], H=1, Hkv=1, page=16, seed=4)
        K0 = c.K.clone()
        if what == "page":
            c.table[0, 1] = 1 << 25
        c.lens[0] = {"page": 20, "short": 2, "long": 10 ** 6}[what]
        k = torch.ones((4 + 1, 1, 64), dtype=torch.bfloat16, device="cuda")
        fs.paged_append(c.p, k, k, c.K, c.V, c.table, c.lens, c.ws, cu=ints([0, 4, 5]))
        with pytest.raises(fs.FsError) as e:
            fs.sync_status(c.ws)
        assert e.value.code == 6
        assert (c.tokens(c.K, 1, 0, 29, 30) == 1).all()      # the other sequence's token is written
        if what == "page":
            assert torch.equal(torch.nan_to_num(c.K[c.rows[0]]), torch.nan_to_num(K0[c.rows[0]]))


# ---------------------------------------------------------------- pages
def same_book(book, refs, table, lens):
    assert refs.tolist() == book.refs and table.tolist() == book.table and lens.tolist() == book.lens


@pytest.mark.parametrize("pages,page,B", [(64, 16, 24), (20000, 4, 24), (4000, 2, 1300)])
def test_reserve_fork_free_compact_against_the_book(pages, page, B):
    """Random calls; tables, counts and lengths equal the book's after each, the pools' moved
    tokens too, and a refused call changes nothing.  Fewer pages and sequences than a block looks
    at in a step, and more."""
    rng = np.random.default_rng(pages)
    width = max(16, pages // 8)
    p = fs.PagedParams(B=B, H=2, Hkv=2, page_size=page, num_pages=pages, max_pages=width, dtype="f32")
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    K.copy_(torch.arange(K.numel(), device="cuda").view(K.shape) % 8191)
    V.copy_(-K)
    book, refused = Book(B, pages, width, page), 0
    for step in range(60):
        what = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        K0 = K.clone()
        ok = True
        if what == "reserve":
            new = (rng.integers(0, 3 * pages * page // B, B) * (rng.random(B) < 0.4)).tolist()
            ok = book.reserve(new)
            fs.pages_reserve(p, ints(new), refs, table, lens, ws)
        elif what == "fork":
            empty = [b for b in range(B) if book.lens[b] == 0]
            full = [b for b in range(B) if book.lens[b] > 0]
            if not empty or not full:
                continue
            dst = rng.permutation(empty)[:rng.integers(1, len(empty) + 1)].tolist()
            src = rng.choice(full, len(dst)).tolist()
            moved = book.fork(src, dst)
            ok = moved is not None
            fs.pages_fork(p, K, V, refs, table, lens, ints(src), ints(dst), ws)
            for a, b, n in moved or []:
                K0[b, :, :n] = K0[a, :, :n]
        elif what == "free":
            rows = rng.integers(0, B, rng.integers(1, max(10, B // 2))).tolist()     # the same one twice now and then
            book.free(rows)
            fs.pages_free(p, refs, table, lens, ints(rows), ws)
        else:
            to = book.compact()
            live = ints([-1])
            fs.pages_compact(p, K, V, refs, table, ws, live=live)
            assert live.item() == sum(n > 0 for n in book.refs)
            for a, b in to.items():
                K0[b] = K0[a]
        if ok:
            fs.sync_status(ws)
        else:
            refused += 1
            with pytest.raises(fs.FsError) as e:
                fs.sync_status(ws)
            assert e.value.code == 6
        same_book(book, refs, table, lens)
        assert torch.equal(K, K0) and torch.equal(V, -K0)
    assert refused > 0


def test_compact_into_another_table_keeps_the_first():
    c = Cache([70, 0, 33], H=2, Hkv=2, page=16, spare=40, layout="tokens_first", seed=6)
    refs = ints(np.bincount(c.rows[c.rows >= 0], minlength=c.p.num_pages))
    refs0, table0 = refs.clone(), c.table.clone()
    before = [c.tokens(c.K, b, 1, 0, n) for b, n in enumerate(c.n)]
    r2, t2 = torch.empty_like(refs), torch.empty_like(c.table)
    fs.pages_compact(c.p, c.K, c.V, refs, c.table, c.ws, refs_out=r2, table_out=t2)
    fs.sync_status(c.ws)
    assert torch.equal(refs, refs0) and torch.equal(c.table, table0)
    live = int((refs0 > 0).sum())
    assert (r2[:live] == 1).all() and (r2[live:] == 0).all() and int(t2.max()) == live - 1
    c.rows = t2.cpu().numpy()
    for b, n in enumerate(c.n):
        assert np.array_equal(c.tokens(c.K, b, 1, 0, n), before[b])


@pytest.mark.parametrize("src,dst", [([0], [0]), ([0], [2]), ([0, 1], [3, 3]), ([3], [4]), ([0, 3], [3, 4]),
                                     ([0], [9]), ([-1], [3])])
def test_fork_refusals_change_nothing(src, dst):
    """A dst in use, listed twice, a src as well, or outside the table.  (An empty src alone is a
    branch of nothing.)"""
    p = fs.PagedParams(B=5, H=1, Hkv=1, page_size=4, num_pages=30, max_pages=6)
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    fs.pages_reserve(p, ints([5, 8, 3, 0, 0]), refs, table, lens, ws)
    fs.sync_status(ws)
    was = [x.clone() for x in (refs, table, lens)]
    fs.pages_fork(p, K, V, refs, table, lens, ints(src), ints(dst), ws)
    if (src, dst) == ([3], [4]):
        fs.sync_status(ws)
    else:
        with pytest.raises(fs.FsError) as e:
            fs.sync_status(ws)
        assert e.value.code == 6
    assert all(torch.equal(a, b) for a, b in zip(was, (refs, table, lens)))


def test_bad_page_lists_are_reported():
    p = fs.PagedParams(B=2, H=1, Hkv=1, page_size=4, num_pages=8, max_pages=4)
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    K.fill_(1)
    V.fill_(2)
    K[0] = 5

    def reported(call):
        call()
        with pytest.raises(fs.FsError) as e:
            fs.sync_status(ws)
        assert e.value.code == 6

    reported(lambda: fs.pages_copy(p, K, V, ints([0, 0, 8]), ints([-1, 3, 4]), ws))
    assert (K[3] == 5).all() and (K[4] == 1).all()
    reported(lambda: fs.pages_free(p, refs, table, lens, ints([7]), ws))
    reported(lambda: fs.pages_reserve(p, ints([-1, 0]), refs, table, lens, ws))
    reported(lambda: fs.pages_reserve(p, ints([17, 0]), refs, table, lens, ws))      # past max_pages
    reported(lambda: fs.pages_reserve(p, ints([2 ** 31 - 1, 2 ** 31 - 1]), refs, table, lens, ws))
    assert refs.tolist() == [0] * 8 and lens.tolist() == [0, 0]
    # a row that lists a page more often than refs counts
    fs.pages_reserve(p, ints([4, 0]), refs, table, lens, ws)
    fs.sync_status(ws)
    refs[table[0, 0]] = 0
    reported(lambda: fs.pages_free(p, refs, table, lens, ints([0]), ws))
    assert refs.tolist() == [0] * 8


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,page,Hkv,layout", [(64, 1, 1, "heads_first"), (128, 7, 3, "tokens_first"), (256, 33, 5, "heads_first")])
def test_copy_pages(dtype, d, page, Hkv, layout):
    p = fs.PagedParams(B=1, H=Hkv, Hkv=Hkv, d=d, page_size=page, num_pages=90, max_pages=1, dtype=dtype, layout=layout)
    K, V, *_ = fs.alloc_pages(p)
    g = torch.Generator().manual_seed(1)
    K.copy_(torch.randn(p.shape, generator=g))
    V.copy_(torch.randn(p.shape, generator=g))
    order = torch.randperm(90, generator=g).to(torch.int32).cuda()
    src, dst = order[:41].clone(), order[41:82].clone()
    k, v = K.clone(), V.clone()
    k[dst.long()], v[dst.long()] = K[src.long()], V[src.long()]
    ws = fs.alloc_paged_workspace(p)
    fs.pages_copy(p, K, V, src, dst, ws)
    fs.sync_status(ws)
    assert torch.equal(K, k) and torch.equal(V, v)


def test_copy_and_fork_in_a_pool_with_gaps():
    """K and V in one tensor, heads and pages further apart than they are long; the gaps stay."""
    both = torch.randn((12, 2, 3, 5, 80), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    K, V = both[:, 0, :, :, :64], both[:, 1, :, :, :64]
    p = fs.PagedParams(B=2, H=3, Hkv=3, page_size=5, num_pages=12, max_pages=4, strides=K.stride()[:3])
    refs, table, lens = torch.zeros(12, dtype=torch.int32, device="cuda"), ints([[-1] * 4] * 2), ints([0, 0])
    ws = fs.alloc_paged_workspace(p)
    want = both.clone()
    fs.pages_copy(p, K, V, ints([3, 4]), ints([9, 8]), ws)
    want[9, ..., :64], want[8, ..., :64] = want[3, ..., :64], want[4, ..., :64]
    assert torch.equal(both, want)
    fs.pages_reserve(p, ints([8, 0]), refs, table, lens, ws)
    fs.pages_fork(p, K, V, refs, table, lens, ints([0]), ints([1]), ws)
    fs.sync_status(ws)
    want[2, :, :, :3, :64] = want[1, :, :, :3, :64]
    assert torch.equal(both, want) and table.tolist() == [[0, 1, -1, -1], [0, 2, -1, -1]]
    assert refs.tolist()[:4] == [2, 1, 1, 0] and lens.tolist() == [8, 8]


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,layout", [("bf16", "heads_first"), ("f32", "tokens_first")])
def test_serving_run(dtype, layout):
    """Prompts admitted, steps decoded from one captured graph, a beam forked, branches dropped, the
    pool packed, and more steps: every step's outputs against attention over the tokens that each
    sequence was given, rotated in float64."""
    H, Hkv, d, page, B = 4, 2, 64, 8, 6
    rng = torch.Generator().manual_seed(31)
    p = fs.PagedParams(B=B, H=H, Hkv=Hkv, d=d, page_size=page, num_pages=80, max_pages=20, dtype=dtype, layout=layout)
    K, V, refs, table, lens = fs.alloc_pages(p)
    ws = fs.alloc_paged_workspace(p)
    rot, theta = fs.Rotary(d, "half"), thetas(d)
    told = [([], []) for _ in range(B)]                      # each sequence's raw keys and values

    def draw(*shape):
        return torch.randn(shape, generator=rng).to(DTYPES[dtype]).cuda()

    def append(new):
        T = sum(new)
        k, v, cu = draw(T, Hkv, d), draw(T, Hkv, d), np.concatenate([[0], np.cumsum(new)])
        fs.pages_reserve(p, ints(new), refs, table, lens, ws)
        fs.paged_append(p, k, v, K, V, table, lens, ws, cu=ints(cu), rotary=rot)
        for b in range(B):
            told[b][0].extend(f64(k[cu[b]:cu[b + 1]]))
            told[b][1].extend(f64(v[cu[b]:cu[b + 1]]))

    active = ints([0] * B)
    k1, v1, q1 = draw(B, Hkv, d), draw(B, Hkv, d), draw(B, H, d)
    qr, o = torch.zeros_like(q1), torch.zeros_like(q1)

    def step_calls():
        fs.pages_reserve(p, active, refs, table, lens, ws)
        fs.paged_append(p, k1, v1, K, V, table, lens, ws, rotary=rot, Q=q1, Qo=qr)
        fs.paged_attend(p, qr, K, V, table, lens, o, ws)

    graph = torch.cuda.CUDAGraph()
    step_calls()                                             # nothing is active yet
    with torch.cuda.graph(graph):
        step_calls()

    def step():
        for x in (k1, v1, q1):
            x.copy_(draw(*x.shape))
        act = [1 if told[b][0] else 0 for b in range(B)]
        active.copy_(ints(act))
        graph.replay()
        fs.sync_status(ws)
        for b in range(B):
            if not act[b]:
                assert (o[b] == 0).all()
                continue
            told[b][0].append(f64(k1[b]))
            told[b][1].append(f64(v1[b]))
            n = len(told[b][0])
            kk, vv = (np.stack(x) for x in told[b])          # [n, Hkv, d]
            kr = rotate(kk, np.arange(n)[:, None], theta, "half")
            q = rotate(f64(q1[b]), n - 1, theta, "half")
            half = torch.finfo(DTYPES[dtype]).eps / 2
            for h in range(Hkv):
                qh = q[2 * h:2 * h + 2]
                want, l, av = attend(qh, kr[:, h], vv[:, h], d ** -0.5)
                bo, _ = attend_bounds(qh, kr[:, h], want, l, av, d ** -0.5, dtype)
                # the rotated query and keys are rounded once each: two half steps on every product
                extra = 2 * (2 * half + 2.0 ** -20) * (np.abs(qh) @ np.abs(kr[:, h]).T).max(1) * d ** -0.5
                err = np.abs(f64(o[b, 2 * h:2 * h + 2]) - want)
                assert (err <= bo + av * extra[:, None]).all(), (b, n, h)

    append([13, 0, 30, 0, 8, 0])
    for _ in range(4):
        step()
    fs.pages_fork(p, K, V, refs, table, lens, ints([2, 2]), ints([1, 3]), ws)
    for b in (1, 3):
        told[b] = (list(told[2][0]), list(told[2][1]))
    for _ in range(10):
        step()
    fs.pages_free(p, refs, table, lens, ints([2, 0]), ws)
    told[2], told[0] = ([], []), ([], [])
    live = ints([0])
    fs.pages_compact(p, K, V, refs, table, ws, live=live)
    fs.sync_status(ws)
    assert int(table.max()) == live.item() - 1
    for _ in range(3):
        step()
    append([0, 0, 50, 0, 0, 0])
    step()


def test_append_and_attend_on_two_streams_with_their_own_workspaces():
    """Two caches used at once from two streams."""
    caches = [Cache([2000, 100], H=4, Hkv=2, seed=s) for s in (41, 42)]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs = []
        for c, s in zip(caches, streams):
            with torch.cuda.stream(s):
                o, lse = torch.empty_like(c.q), torch.empty((2, 4), device="cuda")
                fs.paged_attend(c.p, c.q, c.K, c.V, c.table, c.lens, o, c.ws, lse=lse)
                outs.append((o, lse))
    torch.cuda.synchronize()
    for c, (o, lse) in zip(caches, outs):
        fs.sync_status(c.ws)
        c.check(o, lse)
