"""Plain fp64 references of the operators in include/pa_q4.h, on numpy arrays.

Values of T (fp16 or bf16) are handled as float64 numbers that T represents;
`bits` gives their 16-bit patterns.  Written from the header's formulas, token
by token, without the package's code."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
LIMIT = {"f16": 16384.0, "bf16": 2.0 ** 120}
# half a step of rounding to T, relative to the value
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rn(x, dtype):
    """float64 -> nearest value of T, ties to even (one rounding)."""
    x = np.asarray(x, dtype=np.float64)
    if dtype == "f32":
        return x.astype(np.float32).astype(np.float64)
    sig, emin, big = (11, -14, 65504.0) if dtype == "f16" else (8, -126, 3.3895313892515355e38)
    _, e = np.frexp(x)
    ulp = np.ldexp(1.0, np.maximum(e - 1, emin) - (sig - 1))
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(np.isfinite(x), np.rint(x / ulp) * ulp, x)
        return np.where(np.abs(y) > big, np.copysign(np.inf, y), y)


def bits(x, dtype):
    """16-bit patterns of values of T."""
    x = np.asarray(x, dtype=np.float64)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            b = x.astype(np.float16).view(np.uint16)
    else:
        b = (x.astype(np.float32).view(np.uint32) >> np.uint32(16)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), b)


def quantise(row, dtype):
    """(codes [D], scales [D/32], offsets [D/32]) of a row's D values."""
    row = np.asarray(row, dtype=np.float64)
    M = LIMIT[dtype]
    codes = np.zeros(row.size, dtype=np.int64)
    ss, zs = [], []
    for n in range(row.size // 32):
        x = row[32 * n:32 * n + 32]
        if np.isnan(x).any():
            ss.append(0.0)
            zs.append(np.nan)
            continue
        mn, mx = min(max(x.min(), -M), M), min(max(x.max(), -M), M)
        s = float(rn((mx - mn) / 15, dtype))
        z = float(rn(mn - 16 * s, dtype))
        if s != 0:
            with np.errstate(invalid="ignore"):
                codes[32 * n:32 * n + 32] = np.clip(np.rint((x - z) / s - 16), 0, 15).astype(int)
        ss.append(s)
        zs.append(z)
    return codes, np.array(ss), np.array(zs)


def values(codes, s, z, dtype):
    """What codes stand for: RN_T(s (16 + c) + z)."""
    return rn(np.repeat(s, 32) * (16 + codes) + np.repeat(z, 32), dtype)


def k_place(D, r, d):
    W = min(D, 128)
    return (d // W) * 8 * W + r * W // 2 + (d % W) // 2, 4 * (d % 2)


def v_place(D, r, d):
    if D == 96:
        col, w = (d % 32) // 4, d // 32
    else:
        col, w = d // (D // 8), (d % (D // 8)) // 4
    V = {64: 2, 96: 1, 128: 4, 256: 4}[D]
    j = r // 2
    word = 8 * D + (j // 4) * 4 * D + (w // V) * 128 * V + 4 * V * (4 * col + j % 4) + 4 * (w % V)
    return word + 2 * (r % 2) + (d % 4) // 2, 4 * (d % 2)


def k_cell(D, r, n):
    N = min(D, 128) // 32
    at = 16 * D + 4 * (((n // N) * 16 + r) * N + n % N)
    return at, at + 2


def v_cell(D, r, n):
    at = 18 * D + ((r // 2) * (D // 32) + n) * 8 + 2 * (r % 2)
    return at, at + 4


def store_row(block, D, r, row, dtype, is_v):
    """Quantise a row into a page block (uint8 [20 D]); returns what it then stands for."""
    codes, s, z = quantise(row, dtype)
    for d in range(D):
        at, sh = (v_place if is_v else k_place)(D, r, d)
        block[at] = (int(block[at]) & ~(15 << sh) & 255) | (int(codes[d]) << sh)
    sb, zb = bits(s, dtype), bits(z, dtype)
    for n in range(D // 32):
        a, b = (v_cell if is_v else k_cell)(D, r, n)
        block[a:a + 2] = np.array([sb[n]], dtype="<u2").view(np.uint8)
        block[b:b + 2] = np.array([zb[n]], dtype="<u2").view(np.uint8)
    return values(codes, s, z, dtype)


def from_bits(b, dtype):
    b = np.ascontiguousarray(b, dtype=np.uint16)
    if dtype == "f16":
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def unpack(blocks, D, dtype):
    """fp64 K, V [n, 16, D] that page blocks uint8 [n, 20 D] stand for."""
    out = []
    for place, cell in ((k_place, k_cell), (v_place, v_cell)):
        at = np.array([[place(D, r, d)[0] for d in range(D)] for r in range(PAGE)])
        sh = np.array([[place(D, r, d)[1] for d in range(D)] for r in range(PAGE)])
        c = (blocks[:, at] >> sh) & 15
        cs = np.array([[cell(D, r, n) for n in range(D // 32)] for r in range(PAGE)])
        par = [from_bits(blocks[:, cs[..., i]].astype(np.uint16) |
                         (blocks[:, cs[..., i] + 1].astype(np.uint16) << 8), dtype)
               for i in (0, 1)]
        with np.errstate(invalid="ignore", over="ignore"):
            out.append(rn(np.repeat(par[0], 32, -1) * (16 + c) + np.repeat(par[1], 32, -1), dtype))
    return out


def attend(q, k, v, scale, dtype):
    """(out, lse, tolerance of out, of lse) for the query heads q [g, D] over k, v
    [tokens, D]: fp64 results, and what the kernel may be off by.

    Score: D products summed in fp32 (each sum off by at most 2^-23 of the
    magnitudes it adds up), times a scale rounded to fp32, and an exp2 good to
    2^-22: es.  Weights: relative error es, and rounded to T (fp16: 2^-11; bf16:
    a head and a rest, 2^-16); they are normalised by their own rounded sum, so
    an output is off by at most twice that times the largest |v|, plus sums of
    fp32 (2^-23 per token-block, taken as 2^-16 in all) and its own rounding."""
    D = q.shape[1]
    if k.shape[0] == 0:
        return (np.zeros((q.shape[0], D)), np.full(q.shape[0], -np.inf), 0.0,
                np.zeros(q.shape[0]))
    s = scale * (q @ k.T)
    mag = abs(scale) * (np.abs(q) @ np.abs(k).T)
    es = (mag.max(1) * D * 2.0 ** -23 + np.abs(s).max(1) * 2.0 ** -22 + 2.0 ** -21)[:, None]
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    tot = w.sum(1, keepdims=True)
    out = (w @ v) / tot
    wr = 2.0 ** -11 if dtype == "f16" else 2.0 ** -16
    vm = np.abs(v).max(0)[None]
    tol = (2 * (wr + es) + 2.0 ** -16) * vm + HALF_STEP[dtype] * np.abs(out) + (
        2.0 ** -25 if dtype == "f16" else 0.0)
    return out, (m + np.log(tot))[:, 0], tol, es[:, 0] + 2.0 ** -20


def decode(q, cache, bt, lens, scale, window, dtype):
    """pa_q4_decode's result and tolerances.  cache uint8 [pages, Hkv, 20 D]."""
    B, Hq, D = q.shape
    hkv = cache.shape[1]
    g = Hq // hkv
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, ltol = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        L = int(lens[b])
        lo = max(0, L - window) if window > 0 else 0
        if L == 0:
            continue
        p0, p1 = lo // PAGE, -(-L // PAGE)
        for h in range(hkv):
            k, v = unpack(cache[bt[b, p0:p1], h], D, dtype)
            sl = slice(lo - p0 * PAGE, L - p0 * PAGE)
            hs = slice(h * g, h * g + g)
            out[b, hs], lse[b, hs], tol[b, hs], ltol[b, hs] = attend(
                q[b, hs], k.reshape(-1, D)[sl], v.reshape(-1, D)[sl], scale, dtype)
    return out, lse, tol, ltol


def axis_of(half, sections, interleaved):
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    k = len(sections)
    return np.array([i % k if i < k * sections[i % k] else 0 for i in range(half)])


def rope(x, positions, sections, theta, rot, interleaved=False, inverse=False):
    """fp64 rotation of x [n, heads, D], positions [axes, n]."""
    half = rot // 2
    ax = axis_of(half, sections, interleaved)
    freq = np.array([math.pow(theta, -2.0 * i / rot) for i in range(half)])
    ang = positions[ax].T.astype(np.float64) * freq
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1 if inverse else 1)
    y = x.astype(np.float64).copy()
    a, b = x[..., :half].astype(np.float64), x[..., half:rot].astype(np.float64)
    y[..., :half] = a * c - b * s
    y[..., half:rot] = b * c + a * s
    return y


def extend_tables(past, new, free, num_pages, bt, cap):
    """pa_extend_tables on Python integers.  Returns (tables, lens, starts, slots,
    positions, taken, error bits)."""
    bt = bt.copy()
    B, maxp = bt.shape
    slots, positions = np.full(cap, -1, np.int64), np.zeros(cap, np.int32)
    starts, lens, err = [0], [], 0
    used = asked = 0
    for b in range(B):
        p, n = int(past[b]), int(new[b])
        row = starts[-1]
        starts.append(row + max(0, n))
        lens.append(p)
        ok = p >= 0 and n >= 0 and p + n <= maxp * PAGE and starts[-1] <= cap
        served = False
        first = asked
        if not ok:
            err |= 2
        else:
            have, need = -(-p // PAGE), -(-(p + n) // PAGE)
            asked += need - have
            served = need == have or asked <= len(free)
            if not served:
                err |= 16
        if served:
            lens[-1] = p + n
            used += need - have
            for j in range(have, need):
                pid = int(free[first + j - have])
                bt[b, j] = pid if 0 <= pid < num_pages else -1
        for j in range(max(0, n)):
            if row + j >= cap:
                break
            x = p + j
            positions[row + j] = x if p >= 0 and x < maxp * PAGE else 0
            if served:
                pid = int(bt[b, x // PAGE])
                if 0 <= pid < num_pages:
                    slots[row + j] = pid * PAGE + x % PAGE
                else:
                    err |= 1
    return (bt, np.array(lens, np.int32), np.minimum(starts, 2**31 - 1).astype(np.int32), slots, positions, used, err)
