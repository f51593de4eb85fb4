"""What is measured of the serving operators: rotary positions, the paged key-value cache that takes
the rotated keys, attention of one new token per sequence over its pages, and the management of pages.

`own` false: the operators in elementary torch operations.  `own` true: the calls a user makes of
long_context_sparse_head_b200.  A pool of pages is [pages, kv heads, page size, d] with any strides; a
row of `table` lists a sequence's pages, `lens` its tokens, `refs[page]` how many rows list a page."""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step's queries and keys, as the projection leaves them, far into a long archive
        dict(name="rope_step", op="rope", B=32, N=1, H=16, Hk=4, d=64, r=64, half=False, scaling="none", factor=1.0,
             tokens_first=True, far=262144, back=False, dtype="bf16"),
        # the queries and keys of the 65536-token prefill, positions 0..N-1
        dict(name="rope_prefill", op="rope", B=1, N=65536, H=16, Hk=16, d=64, r=64, half=False, scaling="none",
             factor=1.0, tokens_first=False, far=0, back=False, dtype="bf16"),
        # training: forward and gradients, half the head rotated, context extended four times
        dict(name="rope_train", op="rope", B=4, N=4095, H=16, Hk=4, d=128, r=64, half=True, scaling="by_parts",
             factor=4.0, tokens_first=True, far=0, back=True, dtype="f32"),
        # a decoding step of a batch: rotate, write the new keys and values into their pages
        dict(name="append_step", op="append", B=64, longest=8192, step=True, H=16, Hkv=4, d=128, page=16, r=128,
             half=True, scaling="none", factor=1.0, tokens_first=False, dtype="bf16"),
        # prompts of ragged lengths written in one call, rows of padding behind the last one
        dict(name="append_prompts", op="append", B=12, longest=8191, step=False, H=16, Hkv=8, d=64, page=32, r=64,
             half=False, scaling="linear", factor=2.0, tokens_first=False, dtype="f16"),
        # one short sequence: latency counts
        dict(name="attend_first", op="attend", B=1, longest=77, ragged=False, H=16, Hkv=2, d=64, page=32, window=-1,
             tokens_first=False, dtype="f16"),
        # a served batch of ragged lengths, four query heads on each key-value head
        dict(name="attend_batch", op="attend", B=64, longest=8192, ragged=True, H=16, Hkv=4, d=128, page=16, window=-1,
             tokens_first=False, dtype="bf16"),
        # one new token over the 262144-token archive, every head with keys of its own
        dict(name="attend_archive", op="attend", B=1, longest=262144, ragged=False, H=16, Hkv=16, d=64, page=32,
             window=-1, tokens_first=False, dtype="bf16"),
        # the look-back window of 512 over long sequences, pages with the tokens first
        dict(name="attend_window", op="attend", B=128, longest=16384, ragged=True, H=16, Hkv=16, d=64, page=64,
             window=512, tokens_first=True, dtype="f32"),
        # pages copied within a pool (a shared prefix made private)
        dict(name="pages_copy", op="copy", n=512, pages=2048, Hkv=16, d=64, page=32, tokens_first=False, dtype="bf16"),
        # a beam step: dropped branches are freed, kept ones forked, each branch gets room for a token
        dict(name="pages_beams", op="beams", S=8, F=56, longest=8191, Hkv=8, d=128, page=32, tokens_first=False,
             dtype="bf16"),
        # a pool after many sequences came and went is packed to its front
        dict(name="pages_compact", op="compact", B=64, pages=16384, live=0.6, Hkv=8, d=128, page=16,
             tokens_first=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "attend", "attend", "attend", "copy", "beams", "compact"])
    c = dict(op=op, tokens_first=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    es = 4 if c["dtype"] == "f32" else 2
    if op in ("rope", "append"):
        c["d"] = rng.choice([64, 128, 256])
        c["r"] = rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] // 4])
        c["half"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "by_parts"])
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
        c["H"] = rng.choice([1, 4, 8, 16, 32])
    if op == "rope":
        c["Hk"] = rng.choice([h for h in (1, 2, 4, 8, 16) if h <= c["H"]])
        c["B"] = _log(rng, 1, 16)
        c["back"] = rng.random() < 0.5
        most = 2.5e8 / (c["B"] * (c["H"] + c["Hk"]) * c["d"] * es * (2 if c["back"] else 1))
        c["N"] = _log(rng, 1, max(1, min(65536, most)))
        c["far"] = rng.choice([0, 4096, 262144])
        return c
    c["page"] = rng.choice([1, 8, 16, 24, 32, 64, 128]) if op in ("append", "attend") else rng.choice([8, 16, 24, 32, 64])
    if op == "append":
        c["Hkv"] = c["H"] // rng.choice([g for g in (1, 2, 4, 8) if g <= c["H"]])
        c["step"] = rng.random() < 0.5
        c["B"] = _log(rng, 1, 256) if c["step"] else _log(rng, 1, 16)
        most = 4e8 / (c["B"] * 2 * c["Hkv"] * c["d"] * es)
        c["longest"] = _log(rng, 16, max(17, min(16384 if c["step"] else 4096, most)))
        return c
    if op == "attend":
        c["d"] = rng.choice([64, 64, 128, 256])
        c["Hkv"] = rng.choice([1, 2, 3, 4, 8, 16])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8, 16])
        c["B"] = _log(rng, 1, 128)
        c["window"] = rng.choice([-1, -1, _log(rng, 32, 2048)])
        most = 5e8 / (c["B"] * 2 * c["Hkv"] * c["d"] * es)
        c["longest"] = _log(rng, 1, max(2, min(262144, most)))
        c["ragged"] = rng.random() < 0.7
        return c
    c["d"] = rng.choice([64, 128, 256])
    c["Hkv"] = rng.choice([1, 2, 4, 8, 16])
    size = c["Hkv"] * c["d"] * c["page"] * es
    if op == "copy":
        c["n"] = _log(rng, 1, max(2, min(2048, 1e8 / size)))
        c["pages"] = 2 * c["n"] + rng.randrange(100)
    elif op == "beams":
        c["S"] = _log(rng, 1, 8)
        c["F"] = _log(rng, 1, 60)
        c["longest"] = _log(rng, 16, max(17, min(8192, 8e8 / ((c["S"] + c["F"]) * 2 * c["Hkv"] * c["d"] * es))))
    else:
        c["B"] = _log(rng, 1, 128)
        c["pages"] = _log(rng, 64, max(65, min(16384, 4e8 / size)))
        c["live"] = rng.choice([0.1, 0.35, 0.6, 0.85])
    return c


# ---------------------------------------------------------------- inputs
def _lengths(c, ragged, many):
    """The sequences' lengths: part of the case, the same for every seed (one in eight empty where ragged)."""
    rng = random.Random(1000003 * many + c["longest"])
    if not ragged:
        return [c["longest"]] * many
    lens = [_log(rng, 1, c["longest"]) for _ in range(many)]
    lens[0] = c["longest"]
    return [0 if i % 8 == 5 else n for i, n in enumerate(lens)]


def _up(n, m):
    return -(-n // m)


def _normal(g, dtype, *shape):
    """N(0,1) values; made in parts so that a large pool needs no float32 copy of itself."""
    x = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    flat = x.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        part = flat[a:a + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV))
    return x


def _pool(g, c, pages):
    shape = (pages, c["page"], c["Hkv"], c["d"]) if c["tokens_first"] else (pages, c["Hkv"], c["page"], c["d"])
    x = _normal(g, c["dtype"], *shape)
    return x.transpose(1, 2) if c["tokens_first"] else x


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(g, lens, page, pages, width):
    """Each sequence's pages, drawn without repetition from the pool; -1 behind them."""
    counts = [_up(n, page) for n in lens]
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _frequencies(c):
    """theta_m of the rotated pairs in 64 bits."""
    r, f = c["r"], c["factor"]
    base = 10000.0 * (f ** (r / (r - 2.0)) if c["scaling"] == "ntk" else 1.0)
    theta = base ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r)
    if c["scaling"] == "linear":
        theta = theta / f
    if c["scaling"] == "by_parts":
        turns = 4096 * theta / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        theta = theta * ((1 - keep) / f + keep)
    return theta


def _mscale(c):
    return 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "by_parts" else 1.0


def _rotary(c):
    import long_context_sparse_head_b200 as fs
    return fs.Rotary(c["r"], layout="half" if c["half"] else "interleaved", base=10000.0, scaling=c["scaling"],
                     factor=c["factor"], orig_len=4096, slow=1.0, fast=32.0, mscale=_mscale(c))


def _handles(s, B, H, pages, width):
    """The plan and the workspace that a program keeps beside its cache."""
    import long_context_sparse_head_b200 as fs
    c = s["c"]
    s["p"] = fs.PagedParams(B=B, H=H, Hkv=c["Hkv"], d=c["d"], page_size=c["page"], num_pages=pages, max_pages=width,
                            dtype=c["dtype"], strides=s["K"].stride()[:3])
    s["ws"] = fs.alloc_paged_workspace(s["p"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, s = case, {"c": case}
    if c["op"] == "rope":
        for name, h in (("q", c["H"]), ("k", c["Hk"])):
            for t in (name, "d" + name):
                if t[0] == "d" and not c["back"]:
                    continue
                x = _normal(g, c["dtype"], *((c["B"], c["N"], h, c["d"]) if c["tokens_first"] else (c["B"], h, c["N"], c["d"])))
                s[t] = x.transpose(1, 2) if c["tokens_first"] else x
                s[t + "_out"] = torch.empty_like(s[t])
        first = torch.randint(0, c["far"] or 1, (c["B"], 1), generator=g, device=DEV)
        s["pos"] = (first + torch.arange(c["N"], device=DEV)).to(torch.int32)
        s["theta"] = torch.from_numpy(_frequencies(c)).to(DEV)
        if own:
            s["rotary"] = _rotary(c)
        return s
    if c["op"] == "append":
        lens = _lengths(c, True, c["B"])
        new = [min(1, n) for n in lens] if c["step"] else [_up(n, 1 + b % 2) for b, n in enumerate(lens)]
        if c["step"]:
            lens, new = [max(1, n) for n in lens], [1] * c["B"]
        width = _up(c["longest"], c["page"])
        pages = sum(_up(n, c["page"]) for n in lens) + 5
        s["K"], s["V"] = _pool(g, c, pages), _pool(g, c, pages)
        s["table"], s["lens"] = _tables(g, lens, c["page"], pages, width), _int(lens)
        s["total"] = sum(new)
        rows = s["total"] if c["step"] else s["total"] + 3
        s["cu"] = None if c["step"] else _int([sum(new[:b]) for b in range(c["B"] + 1)])
        for name, h in (("q", c["H"]), ("k", c["Hkv"]), ("v", c["Hkv"])):
            s[name] = _normal(g, c["dtype"], rows, h, c["d"])
        s["q_out"] = torch.zeros_like(s["q"])
        s["theta"] = torch.from_numpy(_frequencies(c)).to(DEV)
        if own:
            s["rotary"] = _rotary(c)
            _handles(s, c["B"], c["H"], pages, width)
        return s
    if c["op"] == "attend":
        lens = _lengths(c, c["ragged"], c["B"])
        width = _up(c["longest"], c["page"])
        pages = sum(_up(n, c["page"]) for n in lens) + 3
        s["K"], s["V"] = _pool(g, c, pages), _pool(g, c, pages)
        s["table"], s["lens"] = _tables(g, lens, c["page"], pages, width), _int(lens)
        s["span"] = max(1, max(_span(c, n) for n in lens))
        s["q"] = _normal(g, c["dtype"], c["B"], c["H"], c["d"])
        # where a page is part filled, what lies behind the last token was never written
        for b, n in enumerate(lens):
            if n % c["page"]:
                for x in (s["K"], s["V"]):
                    x[s["table"][b, n // c["page"]].long(), :, n % c["page"]:] = float("nan")
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["B"], c["H"]), dtype=torch.float32, device=DEV)
        if own:
            _handles(s, c["B"], c["H"], pages, width)
        return s
    if c["op"] == "copy":
        s["K"], s["V"] = _pool(g, c, c["pages"]), _pool(g, c, c["pages"])
        order = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:c["n"]].clone(), order[c["n"]:2 * c["n"]].clone()
        if own:
            _handles(s, 1, c["Hkv"], c["pages"], 1)
        return s
    if c["op"] == "beams":
        many = c["S"] + c["F"]
        lens = [max(1, n) for n in _lengths(c, True, many)]
        width = _up(c["longest"] + 1, c["page"])
        pages = sum(_up(n, c["page"]) for n in lens) + 2 * c["F"] + 7
        s["K"], s["V"] = _pool(g, c, pages), _pool(g, c, pages)
        s["table"], s["lens"] = _tables(g, lens, c["page"], pages, width), _int(lens)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["dst"] = torch.arange(c["S"], many, device=DEV).to(torch.int32)
        s["src"] = torch.randint(0, c["S"], (c["F"],), generator=g, device=DEV).to(torch.int32)
        s["new"] = _int([0] * c["S"] + [1] * c["F"])
        if own:
            _handles(s, many, c["Hkv"], pages, width)
        return s
    s["K"], s["V"] = _pool(g, c, c["pages"]), _pool(g, c, c["pages"])
    n = max(1, int(c["live"] * c["pages"]))
    width = _up(n, c["B"])
    s["table"] = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
    s["table"].view(-1)[:n] = torch.randperm(c["pages"], generator=g, device=DEV)[:n].to(torch.int32)
    if c["B"] > 1:
        s["table"][1, 0] = s["table"][0, 0]  # a page that two sequences share
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0], minlength=c["pages"]).to(torch.int32)
    s["refs_out"], s["table_out"] = torch.empty_like(s["refs"]), torch.empty_like(s["table"])
    s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        _handles(s, c["B"], c["Hkv"], c["pages"], width)
    return s


def _span(c, n):
    """Tokens that a sequence of n attends to."""
    return min(n, c["window"] + 1) if c["window"] >= 0 else n


# ---------------------------------------------------------------- the plain forms
def _turned(x, angle, c, sign):
    """The first r of the last dimension's d turned by `angle` (64 bits, x's shape with r/2 last)."""
    cos, sin = (torch.cos(angle) * _mscale(c)).float(), (torch.sin(angle) * (sign * _mscale(c))).float()
    r = c["r"]
    y = x[..., :r].float()
    if c["half"]:
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((y.to(x.dtype), x[..., r:]), -1)


def _plain_rope(s):
    c = s["c"]
    angle = s["pos"].double()[:, None, :, None] * s["theta"]
    out = [_turned(s["q"], angle, c, 1.0), _turned(s["k"], angle, c, 1.0)]
    if c["back"]:
        out += [_turned(s["dq"], angle, c, -1.0), _turned(s["dk"], angle, c, -1.0)]
    return out


def _plain_append(s):
    c, n = s["c"], s["total"]
    t = torch.arange(n, device=DEV)
    if s["cu"] is None:
        b, pos = t, s["lens"].long() - 1
    else:
        cu = s["cu"].long()
        b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        pos = s["lens"].long()[b] - cu[b + 1] + t
    angle = pos.double()[:, None, None] * s["theta"]
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    s["K"][page, :, slot] = _turned(s["k"][:n], angle, c, 1.0)
    s["V"][page, :, slot] = s["v"][:n]
    s["q_out"][:n] = _turned(s["q"][:n], angle, c, 1.0)
    return s["q_out"], s["K"], s["V"]


def _plain_attend(s):
    c = s["c"]
    n = s["lens"].long()
    start = (n - 1 - c["window"]).clamp(min=0) if c["window"] >= 0 else torch.zeros_like(n)
    pos = start[:, None] + torch.arange(s["span"], device=DEV)
    seen = pos < n[:, None]
    pos = torch.where(seen, pos, 0)
    page = torch.where(seen, s["table"].gather(1, pos // c["page"]), 0).long()
    k = torch.where(seen[..., None, None], s["K"][page, :, pos % c["page"]].float(), 0.0)
    v = torch.where(seen[..., None, None], s["V"][page, :, pos % c["page"]].float(), 0.0)
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    x = torch.einsum("bhgd,bnhd->bhgn", q, k) / math.sqrt(c["d"])
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,bnhd->bhgd", e, v) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).reshape(c["B"], c["H"])
    return o.reshape(c["B"], c["H"], c["d"]).to(s["q"].dtype), lse


def _plain_copy(s):
    s["K"][s["dst"].long()] = s["K"][s["src"].long()]
    s["V"][s["dst"].long()] = s["V"][s["src"].long()]
    return s["K"], s["V"]


def _free_pages(refs):
    """All pages, the free ones first and in their order."""
    return torch.argsort((refs != 0).to(torch.int32), stable=True)


def _plain_beams(s):
    page, table, lens, refs = s["c"]["page"], s["table"], s["lens"], s["refs"]
    at = torch.arange(table.shape[1], device=DEV)
    dst, src = s["dst"].long(), s["src"].long()
    # free
    held = at < ((lens[dst] + page - 1) // page)[:, None]
    old = table[dst]
    refs.index_add_(0, torch.where(held, old, 0).long().view(-1), -held.to(torch.int32).view(-1))
    table[dst] = torch.where(held, -1, old)
    lens[dst] = 0
    # fork: whole pages are shared, the part-filled one is copied into the lowest free page
    n = lens[src]
    whole, part = n // page, n % page
    has = part > 0
    rank = torch.cumsum(has, 0) - 1
    fresh = _free_pages(refs)[rank.clamp(min=0)].to(torch.int32)
    shared = at < whole[:, None]
    tail = (at == whole[:, None]) & has[:, None]
    row = torch.where(shared, table[src], torch.where(tail, fresh[:, None], table[dst]))
    refs.index_add_(0, torch.where(shared, table[src], 0).long().view(-1), shared.to(torch.int32).view(-1))
    refs.index_add_(0, torch.where(has, fresh, 0).long(), has.to(torch.int32))
    old_tail = torch.where(has, table[src].gather(1, whole.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0], 0).long()
    slots = (torch.arange(page, device=DEV) < part[:, None])[:, None, :, None]
    fresh = torch.where(has, fresh, 0).long()
    keep = torch.nonzero(has)[:, 0]
    for_k = torch.where(slots, s["K"][old_tail], s["K"][fresh])
    for_v = torch.where(slots, s["V"][old_tail], s["V"][fresh])
    s["K"][fresh[keep]] = for_k[keep]
    s["V"][fresh[keep]] = for_v[keep]
    table[dst] = row
    lens[dst] = n
    # room for the new tokens, from the lowest free pages
    n, new = lens.clone(), s["new"]
    had, want = (n + page - 1) // page, (n + new + page - 1) // page
    first = torch.cumsum(want - had, 0) - (want - had)
    take = (at >= had[:, None]) & (at < want[:, None])
    fresh = _free_pages(refs)[torch.where(take, first[:, None] + at - had[:, None], 0).long()]
    table.copy_(torch.where(take, fresh.to(torch.int32), table))
    refs.index_add_(0, torch.where(take, fresh, 0).view(-1), take.to(torch.int32).view(-1))
    lens.add_(new)
    return s["K"], s["V"], refs, table, lens


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    used = refs != 0
    live = used.sum()
    at = torch.arange(refs.numel(), device=DEV)
    low = at < live
    moved, hole = torch.nonzero(used & ~low)[:, 0], torch.nonzero(~used & low)[:, 0]
    to = at.clone()
    to[moved] = hole
    s["K"][hole] = s["K"][moved]
    s["V"][hole] = s["V"][moved]
    out = refs.clone()
    out[hole] = refs[moved]
    out[moved] = 0
    return s["K"], s["V"], out, torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table), live.to(torch.int32).view(1)


# ---------------------------------------------------------------- the framework's calls
def _own_rope(s):
    import long_context_sparse_head_b200 as fs
    fs.rope(s["rotary"], s["q"], s["q_out"], s["k"], s["k_out"], positions=s["pos"])
    if not s["c"]["back"]:
        return [s["q_out"], s["k_out"]]
    fs.rope_backward(s["rotary"], s["dq"], s["dq_out"], s["dk"], s["dk_out"], positions=s["pos"])
    return [s["q_out"], s["k_out"], s["dq_out"], s["dk_out"]]


def _own_append(s):
    import long_context_sparse_head_b200 as fs
    fs.paged_append(s["p"], s["k"], s["v"], s["K"], s["V"], s["table"], s["lens"], s["ws"], cu=s["cu"],
                    rotary=s["rotary"], Q=s["q"], Qo=s["q_out"])
    return s["q_out"], s["K"], s["V"]


def _own_attend(s):
    import long_context_sparse_head_b200 as fs
    fs.paged_attend(s["p"], s["q"], s["K"], s["V"], s["table"], s["lens"], s["o"], s["ws"], lse=s["lse"],
                    window=s["c"]["window"])
    return s["o"], s["lse"]


def _own_copy(s):
    import long_context_sparse_head_b200 as fs
    fs.pages_copy(s["p"], s["K"], s["V"], s["src"], s["dst"], s["ws"])
    return s["K"], s["V"]


def _own_beams(s):
    import long_context_sparse_head_b200 as fs
    fs.pages_free(s["p"], s["refs"], s["table"], s["lens"], s["dst"], s["ws"])
    fs.pages_fork(s["p"], s["K"], s["V"], s["refs"], s["table"], s["lens"], s["src"], s["dst"], s["ws"])
    fs.pages_reserve(s["p"], s["new"], s["refs"], s["table"], s["lens"], s["ws"])
    return s["K"], s["V"], s["refs"], s["table"], s["lens"]


def _own_compact(s):
    import long_context_sparse_head_b200 as fs
    fs.pages_compact(s["p"], s["K"], s["V"], s["refs"], s["table"], s["ws"], live=s["live"], refs_out=s["refs_out"],
                     table_out=s["table_out"])
    return s["K"], s["V"], s["refs_out"], s["table_out"], s["live"]


def run(state):
    op = state["c"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "copy": _own_copy, "beams": _own_beams,
                "compact": _own_compact}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "copy": _plain_copy,
            "beams": _plain_beams, "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        n = c["B"] * c["N"] * (c["H"] + c["Hk"]) * (2 if c["back"] else 1)
        return {"bytes": 2 * n * c["d"] * es + 4 * c["B"] * c["N"], "flops": 3 * n * c["r"]}
    if c["op"] == "append":
        lens = _lengths(c, True, c["B"])
        n = c["B"] if c["step"] else sum(_up(n, 1 + b % 2) for b, n in enumerate(lens))
        return {"bytes": 2 * n * (c["H"] + 2 * c["Hkv"]) * c["d"] * es + 8 * c["B"], "flops": 3 * n * (c["H"] + c["Hkv"]) * c["r"]}
    if c["op"] == "attend":
        n = sum(_span(c, x) for x in _lengths(c, c["ragged"], c["B"]))
        pages = sum(_up(_span(c, x), c["page"]) for x in _lengths(c, c["ragged"], c["B"]))
        return {"bytes": 2 * n * c["Hkv"] * c["d"] * es + 2 * c["B"] * c["H"] * c["d"] * es + 4 * c["B"] * (c["H"] + 1) + 4 * pages,
                "flops": 4 * n * c["H"] * c["d"]}
    token = 2 * c["Hkv"] * c["d"] * es
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * c["page"] * token + 8 * c["n"], "flops": 0}
    if c["op"] == "beams":
        lens = [max(1, n) for n in _lengths(c, True, c["S"] + c["F"])]
        mean = sum(n % c["page"] for n in lens[:c["S"]]) / c["S"]
        held = sum(_up(n, c["page"]) for n in lens[:c["S"]]) / c["S"]
        return {"bytes": 2 * c["F"] * mean * token + 28 * c["F"] * held + 24 * c["F"], "flops": 0}
    n = int(c["live"] * c["pages"])
    moved = n * (1 - c["live"])
    return {"bytes": 2 * moved * c["page"] * token + 8 * c["pages"] + 8 * n, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits
def _whirled(x, pos, c, sign):
    """x [.., n, d] in 64 bits as complex pairs times mscale e^(i sign pos theta); pos [.., n]."""
    theta = torch.tensor([_theta(c, m) for m in range(c["r"] // 2)], dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(theta, _mscale(c)).expand(*pos.shape, -1), sign * pos.double()[..., None] * theta)
    x = x.double()
    first, rest = x[..., :c["r"]], x[..., c["r"]:]
    pairs = first.unflatten(-1, (2, -1)).transpose(-1, -2) if c["half"] else first.unflatten(-1, (-1, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = (y.transpose(-1, -2) if c["half"] else y).flatten(-2)
    return torch.cat((y, rest), -1)


def _theta(c, m):
    r, f = c["r"], c["factor"]
    if c["scaling"] == "ntk":
        return math.exp(-2.0 * m / r * (math.log(10000.0) + r / (r - 2) * math.log(f)))
    t = math.exp(-2.0 * m / r * math.log(10000.0))
    if c["scaling"] == "linear":
        return t / f
    if c["scaling"] == "by_parts":
        g = min(1.0, max(0.0, (4096 * t / (2 * math.pi) - 1.0) / 31.0))
        return (1 - g) * t / f + g * t
    return t


def _host_free(refs):
    return [p for p, n in enumerate(refs) if n == 0]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    page = c.get("page")
    if c["op"] == "rope":
        pos = s["pos"][:, None, :]
        out = [_whirled(s[t], pos, c, 1.0) for t in ("q", "k")]
        return out + ([_whirled(s[t], pos, c, -1.0) for t in ("dq", "dk")] if c["back"] else [])
    if c["op"] == "append":
        lens, table = s["lens"].tolist(), s["table"].long().cpu()
        cu = s["cu"].tolist() if s["cu"] is not None else list(range(c["B"] + 1))
        q, K, V = s["q_out"].double(), s["K"].double(), s["V"].double()
        for b in range(c["B"]):
            n = cu[b + 1] - cu[b]
            if not n:
                continue
            pos = torch.arange(lens[b] - n, lens[b])
            at, slot, pos = table[b][pos // page].to(DEV), (pos % page).to(DEV), pos.to(DEV)
            rows = slice(cu[b], cu[b + 1])
            q[rows] = _whirled(s["q"][rows].transpose(0, 1), pos[None], c, 1.0).transpose(0, 1)
            K[at, :, slot] = _whirled(s["k"][rows].transpose(0, 1), pos[None], c, 1.0).transpose(0, 1)
            V[at, :, slot] = s["v"][rows].double()
        return q, K, V
    if c["op"] == "attend":
        o = torch.zeros((c["B"], c["H"], c["d"]), dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)
        group = c["H"] // c["Hkv"]
        for b, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            at = s["table"][b, :_up(n, page)].long()
            a = n - _span(c, n)
            for h in range(c["Hkv"]):
                k = s["K"][at, h].flatten(0, 1)[a:n].double()
                v = s["V"][at, h].flatten(0, 1)[a:n].double()
                q = s["q"][b, h * group:(h + 1) * group].double()
                x = (q @ k.T) * c["d"] ** -0.5
                o[b, h * group:(h + 1) * group] = torch.softmax(x, -1) @ v
                lse[b, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
        return o, lse
    K, V = s["K"].double(), s["V"].double()
    if c["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            K[b], V[b] = K[a], V[a]
        return K, V
    table, refs = s["table"].tolist(), s["refs"].tolist()
    if c["op"] == "beams":
        lens = s["lens"].tolist()
        for b in s["dst"].tolist():
            for i in range(_up(lens[b], page)):
                refs[table[b][i]] -= 1
                table[b][i] = -1
            lens[b] = 0
        free = _host_free(refs)
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            whole, part = divmod(lens[a], page)
            for i in range(whole):
                table[b][i] = table[a][i]
                refs[table[a][i]] += 1
            if part:
                table[b][whole] = free.pop(0)
                refs[table[b][whole]] = 1
                K[table[b][whole], :, :part] = K[table[a][whole], :, :part]
                V[table[b][whole], :, :part] = V[table[a][whole], :, :part]
            lens[b] = lens[a]
        for b, n in enumerate(s["new"].tolist()):
            for i in range(_up(lens[b], page), _up(lens[b] + n, page)):
                table[b][i] = free.pop(0)
                refs[table[b][i]] = 1
            lens[b] += n
        return K, V, _int(refs), _int(table), _int(lens)
    live = sum(n > 0 for n in refs)
    holes = [p for p in range(live) if refs[p] == 0]
    to = {p: holes[i] for i, p in enumerate(p for p in range(live, c["pages"]) if refs[p] > 0)}
    if to:
        a, b = (torch.tensor(list(x), device=DEV) for x in (to.keys(), to.values()))
        K[b], V[b] = K[a], V[a]
    for p, h in to.items():
        refs[h], refs[p] = refs[p], 0
    return K, V, _int(refs), _int([[to.get(p, p) for p in row] for row in table]), _int([live])
