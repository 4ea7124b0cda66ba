"""A plain fp64 restatement of include/pa_q8.h, row by row, for the tests."""
import numpy as np

# Half a step of rounding, relative to the value, and the least step's half.
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LEAST_HALF = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


E4M3 = _e4m3_values()
_GRID = E4M3[:127]  # the codes 0 .. 126 in ascending order


def e4m3_code(x):
    """Codes of fp64 values, to nearest even, 448 at most; non-finite: NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    i = np.clip(np.searchsorted(_GRID, a, side="right") - 1, 0, 126)
    up = np.minimum(i + 1, 126)
    d0, d1 = a - _GRID[i], _GRID[up] - a
    i = np.where((d1 < d0) | ((d1 == d0) & (i % 2 == 1)), up, i)
    c = np.where(np.isfinite(x), i | np.where(np.signbit(x), 128, 0), 127)
    return c.astype(np.uint8)


def e4m3_step(x):
    """Distance of the codes around fp64 values."""
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))
    return np.ldexp(1.0, e - 1 - 3)


def scale_for(amax):
    e = -120
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def turned(x, w, positions, eps, theta, rot):
    """Heads x [n, heads, D] normalised (w or None) and rotated (theta > 0)."""
    y = np.array(x, np.float64)
    if w is not None:
        y = y * w / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    if theta > 0:
        half = rot // 2
        f = theta ** (-2.0 * np.arange(half) / rot)
        ang = np.asarray(positions, np.float64)[:, None] * f
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[..., :half].copy(), y[..., half:rot].copy()
        y[..., :half], y[..., half:rot] = a * c - b * s, b * c + a * s
    return y


def turned_tolerance(x, w, want, eps, theta, rot, dtype):
    """What fp32 in between and one rounding may do.  The norm: a sum of D squares (each
    rounding at most 2^-24 of it, log-like chains of at most D / 8 + 8), 1 / sqrt within 2
    units, two products: (D / 16 + 16) 2^-24 relative.  The rotation: cosine and sine within
    2^-21 (the angle's top 32 bits to fp32: 2^-26 of a turn, then the function's 2 units),
    three roundings, of the pair's magnitude."""
    y = turned(x, w, None, eps, 0.0, rot)
    D = y.shape[-1]
    rel = (D / 16 + 16) * 2.0 ** -24 if w is not None else 0.0
    mag = np.abs(y)
    tol = rel * np.abs(want)
    if theta > 0:
        half = rot // 2
        pair = mag[..., :half] + mag[..., half:rot]
        tol[..., :half] = tol[..., half:rot] = pair * (rel + 2.0 ** -21 + 3 * 2.0 ** -24)
    return tol + (HALF_STEP[dtype] * (np.abs(want) + tol) + LEAST_HALF[dtype] if dtype else 0.0)


class Cache:
    """One of K and V: codes [pages, H, 16, D] and scales [pages, H]."""

    def __init__(self, pages, H, D):
        self.codes = np.full((pages, H, 16, D), 127, np.uint8)
        self.scales = np.ones((pages, H))

    def append(self, rows, slots):
        """rows fp64 [n, H, D] at slots, runs of a page's rows one after the other."""
        i, n = 0, len(slots)
        while i < n:
            s = slots[i]
            if s < 0 or s >= self.codes.shape[0] * 16:
                i += 1
                continue
            j = i + 1
            while j < n and slots[j] == slots[j - 1] + 1 and slots[j] % 16:
                j += 1
            page, r0 = s // 16, s % 16
            for h in range(rows.shape[1]):
                x = rows[i:j, h]
                fin = np.abs(np.where(np.isfinite(x), x, 0.0))
                new = scale_for(fin.max())
                if r0:
                    old = self.scales[page, h]
                    new = max(new, old)
                    if new != old:
                        kept = E4M3[self.codes[page, h, :r0]] * (old / new)
                        self.codes[page, h, :r0] = e4m3_code(kept)
                self.scales[page, h] = new
                self.codes[page, h, r0:r0 + j - i] = e4m3_code(x / new)
            i = j

    def values(self):
        with np.errstate(invalid="ignore"):
            return E4M3[self.codes] * self.scales[..., None, None]


def decode(q, k, v, bt, lens, starts, scale, window, dtype, pow2=True):
    """Rows out, lse and what the kernel's may differ by, from the values k, v [pages, Hkv, 16, D].

    Weights are rounded to 11 bits and normalised by their rounded sum: the row moves by at most
    2^-11 sum p |v - out| (again as much where scales are no powers of two, whose ratio rounds
    the weights once more).  A score is a sum of D exact products in fp32, its factor and the
    maximum's subtraction: (D + 4) 2^-24 of scale sum |q k| at most, plus 2^-23 of the score in the
    log2 domain and 2^-22 of ex2: a relative error of the weight.  Weights below 2^-32 of the
    greatest may vanish.  Then one rounding to T."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    out = np.full(q.shape, np.nan)
    lse = np.full((n, Hq), np.nan)
    tol, ltol = np.zeros(q.shape), np.zeros((n, Hq))
    for b, L in enumerate(lens):
        r0, r1 = int(starts[b]), int(starts[b + 1])
        pos = np.arange(L)
        ids = bt[b][pos // 16]
        for h in range(Hkv):
            kb, vb = k[ids, h, pos % 16], v[ids, h, pos % 16]
            for r in range(r0, r1):
                end = L - (r1 - r) + 1
                begin = max(0, end - window) if window > 0 else 0
                hs = slice(h * g, (h + 1) * g)
                if end <= begin:
                    out[r, hs], lse[r, hs] = 0.0, -np.inf
                    continue
                kk, vv = kb[begin:end], vb[begin:end]
                qq = q[r, hs]
                s = qq @ kk.T * scale  # [g, tokens]
                mag = np.abs(qq) @ np.abs(kk).T * abs(scale)
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                z = p.sum(-1, keepdims=True)
                p /= z
                o = p @ vv
                out[r, hs] = o
                lse[r, hs] = top[:, 0] + np.log(z[:, 0])
                err = (D + 8) * 2.0 ** -24 * mag.max(-1) + 2.0 ** -22 * np.abs(s - top).max(-1) \
                    + 2.0 ** -21
                far = np.abs(vv[None] - o[:, None])  # [g, tokens, D]
                dev = np.einsum("gt,gtd->gd", p, far)
                rel = (1.0 if pow2 else 2.0) * 2.0 ** -11 + 2 * err
                t = rel[:, None] * dev + (end - begin) * 2.0 ** -32 * np.abs(vv).max(0)
                # sums of the products: fp32, in chains of at most a page count's length
                t += 2.0 ** -24 * (16 + (end - begin) / 8) * (p @ np.abs(vv))
                tol[r, hs] = t + HALF_STEP[dtype] * (np.abs(o) + t) + LEAST_HALF[dtype]
                ltol[r, hs] = err + 2.0 ** -11 + 2.0 ** -22 * np.abs(lse[r, hs])
    return out, lse, tol, ltol


def verify(target, draft, drafts, num, accept, sample):
    """accepted, tokens, whether an error is reported; probabilities fp64 values of fp32."""
    B, T1, V = target.shape
    T = T1 - 1
    accepted, tokens, bad = np.zeros(B, np.int32), np.full((B, T1), -1, np.int32), False

    def lim(x):
        return np.clip(np.where(np.isnan(x), 0.0, x), 0.0, 1.0)

    for b in range(B):
        n = T if num is None else int(num[b])
        if not 0 <= n <= T:
            bad, n = True, min(max(n, 0), T)
        j = 0
        hole = None
        while j < n:
            x = int(drafts[b, j])
            if not 0 <= x < V:
                bad = True
                break
            qx = 1.0 if draft is None else lim(draft[b, j, x])
            if not float(accept[b, j]) * qx < lim(target[b, j, x]):
                hole = x
                break
            j += 1
        p = lim(target[b, j]).astype(np.float32)
        w = p.copy()
        if j < n and draft is not None:
            w = np.maximum(p - lim(draft[b, j]).astype(np.float32), np.float32(0))
        elif j < n and hole is not None:
            w[hole] = 0
        units = np.rint(w.astype(np.float64) * 2.0 ** 44).astype(np.int64)
        if units.sum() == 0:
            units = np.rint(p.astype(np.float64) * 2.0 ** 44).astype(np.int64)
        c = np.cumsum(units)
        accepted[b] = j
        tokens[b, :j] = drafts[b, :j]
        total = int(c[-1])
        if total == 0:
            bad = True
            continue
        u = float(sample[b])
        at = 0 if not u > 0 else min(int(np.floor(u * float(total))), total - 1) if u < 1 else total - 1
        tokens[b, j] = int(np.searchsorted(c, at, side="right"))
    return accepted, tokens, bad
