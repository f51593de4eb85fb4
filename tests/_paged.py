"""Plain float64 forms of the serving operators, and the page bookkeeping in Python lists."""
import math

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {t: torch.finfo(x).eps / 2 for t, x in DTYPES.items()}     # one rounding, relative


def thetas(r, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, slow=1.0, fast=32.0):
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    t = base ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r)
    if scaling == "linear":
        t = t / factor
    if scaling == "by_parts":
        g = np.clip((orig_len * t / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        t = t * ((1 - g) / factor + g)
    return t


def rotate(x, pos, theta, layout, mscale=1.0, sign=1.0):
    """x [..., d] float64, pos broadcastable to x.shape[:-1]; the first 2 len(theta) elements turned."""
    r = 2 * len(theta)
    a = np.asarray(pos, np.float64)[..., None] * theta
    c, s = np.cos(a) * mscale, np.sin(a) * mscale * sign
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if layout == "interleaved" else (np.arange(r // 2), np.arange(r // 2, r))
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def rotate_bound(x, y, r, layout, dtype, mscale=1.0):
    """How far a rotated element may be off: its rounding, half a step, and in fp32 the angle (an
    argument of at most pi/4 with a relative error of 2^-24 and 2^-32 turns), sincospi (2 ulp) and
    three roundings of products and sums: under 8 x 2^-24 on each of the two terms."""
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if layout == "interleaved" else (np.arange(r // 2), np.arange(r // 2, r))
    both = np.zeros_like(x)
    both[..., i] = both[..., j] = (np.abs(x[..., i]) + np.abs(x[..., j])) * abs(mscale)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0             # half a step of the subnormals
    return both * 2.0 ** -21 + np.abs(y) * HALF_STEP[dtype] + tiny


def attend(q, k, v, scale):
    """q [G,d], k, v [n,d] float64 -> o [G,d], lse [G], and the mean |v| under the softmax [G,d]."""
    if len(k) == 0:
        return np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf), np.zeros((len(q), v.shape[1]))
    x = q @ k.T * scale
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    l = e.sum(1, keepdims=True)
    return e @ v / l, (m + np.log(l))[:, 0], e @ np.abs(v) / l


def attend_bounds(q, k, o, lse, absv, scale, dtype):
    """Bounds on o and lse.  A score is a sum of d products kept in fp32 (an ulp of the running sum
    at each step: d 2^-23 sum|q k|), and its exponent is rounded at 2^-23 of its size; a
    probability goes into the product in two parts of the type (half a step of half a step, under
    2^-16); sums over n tokens lose at most an ulp each."""
    n, d = k.shape
    if n == 0:
        return np.zeros_like(o), np.zeros_like(lse)
    size = scale * (np.abs(q) @ np.abs(k).T).max(1)
    score = size * (d + 4) * 2.0 ** -23 + 2.0 ** -20
    sums = n * 2.0 ** -23
    half = HALF_STEP[dtype]
    rel = 2 * score + sums + (0.0 if dtype == "f32" else 2.0 ** -16)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    # the second part of an fp16 probability is held in steps of 2^-24: half a step on each
    if dtype == "f16":
        rel = rel + n * 2.0 ** -25
    return absv * rel[:, None] + np.abs(o) * half + tiny, score + sums + np.abs(lse) * 2.0 ** -22


class Book:
    """What the page calls have to do to refs, table and lens."""

    def __init__(self, B, pages, width, page):
        self.refs, self.lens = [0] * pages, [0] * B
        self.table = [[-1] * width for _ in range(B)]
        self.page, self.width = page, width

    def held(self, b):
        return -(-self.lens[b] // self.page)

    def take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def reserve(self, new):
        need = [-(-(n + m) // self.page) - -(-n // self.page) for n, m in zip(self.lens, new)]
        if sum(need) > self.refs.count(0) or any(n + m > self.width * self.page for n, m in zip(self.lens, new)):
            return False
        for b, k in enumerate(need):
            h = self.held(b)
            for i in range(k):
                self.table[b][h + i] = self.take()
            self.lens[b] += new[b]
        return True

    def fork(self, src, dst):
        """Returns [(tail of src, new page, tokens)], or None where it is refused."""
        need = sum(self.lens[a] % self.page > 0 for a in src)
        if need > self.refs.count(0) or any(self.lens[b] for b in dst) or len(set(dst)) < len(dst) or set(src) & set(dst):
            return None
        moved = []
        for a, b in zip(src, dst):
            whole, part = divmod(self.lens[a], self.page)
            for i in range(whole):
                self.table[b][i] = self.table[a][i]
                self.refs[self.table[a][i]] += 1
            if part:
                self.table[b][whole] = self.take()
                moved.append((self.table[a][whole], self.table[b][whole], part))
            self.lens[b] = self.lens[a]
        return moved

    def free(self, rows):
        for b in rows:
            for i in range(self.held(b)):
                self.refs[self.table[b][i]] -= 1
                self.table[b][i] = -1
            self.lens[b] = 0

    def compact(self):
        """Returns {from: to}."""
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip((p for p in range(live, len(self.refs)) if self.refs[p] > 0), holes))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return to
