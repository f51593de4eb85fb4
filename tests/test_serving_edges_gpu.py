"""Calls of the serving operators at the borders of what their documentation allows, on the GPU."""
import numpy as np
import pytest
import torch

import long_context_sparse_head_b200 as fs
from tests._paged import DTYPES, HALF_STEP, attend, rotate, rotate_bound, thetas

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
