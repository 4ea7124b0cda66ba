"""GPU tests of include/pa_q8.h at what its first tests left open: outputs off by no more than
their own rounding, V scales at the ends of their range, scores that overflow, q beside 8-bit
rows through the rings, verification of more sequences than one wave holds, angles, q_norm
without q and the pages of drafts that were not accepted."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q8_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q4, q8
from paged_kv_gqa_pa_gb300 import build as pa_build
from test_q8_gpu import (DIMS, Decode, Rows, T, check_q8, check_verify, code_bytes, host, i32,
                         i64, page_slots, rounded, run_q8_append, to_t, verify_case)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pa_build.build()
    pa.load()


# ---------------------------------------------------------------- attention: the weights

def half_step(x, dtype):
    """Half the distance of T's values around |x|."""
    _, e = np.frexp(np.abs(x))  # |x| in [2^(e - 1), 2^e)
    bits, least = {"f16": (11, -14), "bf16": (8, -126)}[dtype]
    return np.ldexp(1.0, np.maximum(e - 1, least) - bits)


def one_dim_queries(d, size):
    """q with one element a row that is not 0: a score then is one product, exact in fp32, and
    K's codes of 2^-2 to 3.75, so that several tokens weigh."""
    n, Hq, D = d.q.shape
    q = np.zeros(d.q.shape)
    at = d.g.integers(0, D, (n, Hq, 1))
    np.put_along_axis(q, at, d.g.uniform(0.5, 1.0, at.shape) * size, 2)
    d.q = rounded(q, d.dtype)
    x = d.g.integers(0x28, 0x48, d.codes[0].shape) | (d.codes[0] & 0x80)
    d.codes[0] = np.where(d.codes[0] & 127 == 127, 127, x)


def narrow(d, scale):
    """Rows out and what they may be off by where a score is one product and n tokens are seen.

    A weight: the score's factor (three roundings) and its difference from the maximum (of at most
    2 max |s| + 8 in the log2 domain), ex2 (2^-22) of it and of up to four rescalings and joins, the
    ratio of V's scales (2^-22), and two fp16 numbers (each 2^-11 of what it stands for):
    together 2^-22 (max |s| + 12) relative.  The row moves by at most twice that of sum p |v - out|.
    Sums in fp32 in chains of a page count's length, truncating products, the divisions:
    2^-23 (16 + n / 8) (sum p |v| + |out|)."""
    k, v = d.values()
    n, Hq, D = d.q.shape
    g = Hq // d.Hkv
    out, tol = np.zeros(d.q.shape), np.zeros(d.q.shape)
    for b, L in enumerate(d.lens):
        pos = np.arange(L)
        ids = d.bt[b][pos // 16]
        r0, r1 = d.starts[b], d.starts[b + 1]
        for r in range(r0, r1):
            end = L - (r1 - r) + 1
            for h in range(d.Hkv):
                kk, vv = k[ids, h, pos % 16][:end], v[ids, h, pos % 16][:end]
                s = d.q[r, h * g:(h + 1) * g] @ kk.T * scale
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ vv
                err = 2.0 ** -22 * (np.abs(s).max(-1) + 12)
                dev = np.einsum("gt,gtd->gd", p, np.abs(vv[None] - o[:, None]))
                t = 2 * err[:, None] * dev + 2.0 ** -23 * (16 + end / 8) * (p @ np.abs(vv) + np.abs(o))
                t += end * 2.0 ** -32 * np.abs(vv).max(0)
                out[r, h * g:(h + 1) * g], tol[r, h * g:(h + 1) * g] = o, t
    return out, tol


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("queries", [1, 3, 8])
@pytest.mark.parametrize("cluster", [None, 0])
@pytest.mark.parametrize("spread,pow2", [(0.0, True), (4.0, True), (2.0, False)])
def test_decode_rows_are_off_by_their_own_rounding(D, dtype, queries, cluster, spread, pow2):
    """Weights of 11 bits would move most rows of a few tokens across a rounding's border somewhere."""
    d = Decode([D, queries], [1, 2, 3, 5, 40, 333, 700], 4, 2, D, dtype, T=queries, spread=spread,
               pow2=pow2)
    one_dim_queries(d, 64.0)
    out, _, err = d.run(1.0, cluster=cluster)
    assert err == 0
    want, tol = narrow(d, 1.0)
    over = np.abs(out - want) - tol - half_step(np.abs(want) + tol, dtype)
    assert not (over > 0).any(), f"{np.mean(over > 0):.2e} of the elements"


# ---------------------------------------------------------------- attention: V scales of any size

@pytest.mark.parametrize("form", ["whole", "cut", "merged", "cluster"])
@pytest.mark.parametrize("low,high", [(100, 100), (120, 120), (126, 126), (100, 126), (-120, -120),
                                      (-126, -126), (-140, -128), (-149, -110)])
@pytest.mark.parametrize("queries", [1, 4])
@pytest.mark.parametrize("D", [64, 256])
def test_decode_v_scales_of_any_size(D, queries, low, high, form):
    """Scales of 2^low to 2^high, subnormal ones among them, where every value of V is finite."""
    lens = [40, 300, 1, 17] if form == "whole" else [900, 300, 1500, 20]
    d = Decode([D, queries, high + 200], lens, 4, 2, D, "bf16", T=queries)
    x = d.codes[1]  # codes of at most 1.75 either way
    d.codes[1] = np.where(x & 127 == 127, 127, (x & 0x80) | (0x20 + (x & 0x1F)) - ((x & 0x1F) == 0x1F))
    d.scales[1] = 2.0 ** d.g.integers(low, high + 1, d.scales[1].shape)
    assert (d.scales[1] > 0).all()
    if form == "merged":  # (so many CTAs for the sequences that a kernel of its own merges)
        p = d.plan()
        p.cluster, p.ctas_per_group, p.workspace_bytes = 0, 60, 1 << 27
        ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
        tq = to_t(d.q, "bf16")
        out, lse = torch.full_like(tq, 3.0), torch.empty(tq.shape[0], 4, device="cuda")
        pa.pa_q8_decode(p, tq, i32(d.starts), *d.device(), i32(d.bt), i32(d.lens), 0.1, 0, out, lse, ws)
        got = host(out), host(lse), pa.pa_get_error(ws)
    else:
        p = d.plan()
        assert form != "cluster" or p.cluster > 1
        got = d.run(0.1, **{"whole": dict(cluster=0, ctas=4), "cut": dict(ctas=7), "cluster": {}}[form])
    d.check(got, d.want(0.1, 0))


@pytest.mark.parametrize("first", ["zero", "subnormal", "least", "one"])
@pytest.mark.parametrize("queries", [1, 4])
def test_decode_v_scales_that_rise(first, queries):
    """A page of scale 0, subnormal or least in front of ordinary ones, in every warp."""
    d = Decode([7, queries], [600, 90], 4, 1, 128, "bf16", T=queries)
    for b, n in ((0, 38), (1, 6)):
        d.scales[1, d.bt[b, :n // 2], 0] = {"zero": 0.0, "subnormal": 2.0 ** -140, "least": 2.0 ** -120,
                                           "one": 1.0}[first]
    d.case(0.1)
    d.case(0.1, ctas=1)


# ---------------------------------------------------------------- attention: scores that overflow

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("queries", [1, 4])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_scores_beyond_fp32_by_sign(dtype, queries, cluster):
    """Scores that overflow to -inf weigh nothing, those to +inf make their rows NaN, and the rows of
    the other heads stay what they are."""
    L, Hq, D = 700, 5, 128
    # (the factor of the products, K's scale times the call's in the log2 domain, is finite)
    big, scale, small = (2.0 ** 14, 2.0 ** 8, 0.0) if dtype == "f16" else (2.0 ** 44, 2.0 ** -22, 2.0 ** -77)
    d = Decode([queries, 3], [L, 50], Hq, 1, D, dtype, T=queries, new=[queries, 1])
    k = d.codes[0]
    d.codes[0] = np.where(k & 127 == 127, 127, (k & 0x80) | (0x28 + (k & 7)))  # 0.25 to 0.47 either way
    gone = np.zeros(L, bool)
    gone[d.g.permutation(L)[:300]] = True
    gone[16:16 * 9] = True  # whole pages
    gone[0] = gone[L - queries:] = False
    pos = np.arange(L)
    cells = d.bt[0][pos // 16], 0, pos % 16
    d.codes[0][cells + (5,)] = np.where(gone, 0xFE, 0)  # -448, 0
    d.codes[0][cells + (9,)] = 0xFE
    d.scales[0] = 2.0 ** 100
    d.q[:] = 0.0
    d.q[:, 0, 5] = d.q[:, 2, 9] = big
    d.q[:, 1, 5] = -big
    d.q[:, 3, 3] = small
    out, lse, err = d.run(scale, cluster=cluster)
    assert err == 0
    w, wl, tol, ltol = d.want(scale, 0)
    row = slice(0, queries)
    assert np.isnan(out[row, 1]).all() and np.isnan(lse[row, 1]).all()
    assert (out[row, 2] == 0).all() and np.isneginf(lse[row, 2]).all()
    for h in (3, 4):
        assert (np.abs(out[row, h] - w[row, h]) <= tol[row, h]).all()
        assert (np.abs(lse[row, h] - wl[row, h]) <= ltol[row, h]).all()
    # head 0: equal weights of what is not gone, sums in fp32
    v = d.values()[1][cells]
    for t in range(queries):
        see = ~gone & (pos < L - queries + 1 + t)
        mean, room = v[see].mean(0), 2.0 ** -16 * np.abs(v[see]).mean(0)
        assert (np.abs(out[t, 0] - mean) <= room + half_step(np.abs(mean) + room, dtype)).all()
        assert abs(lse[t, 0] - np.log(see.sum())) <= 2.0 ** -16


# ---------------------------------------------------------------- q beside 8-bit rows, by rings

@pytest.mark.parametrize("D,rot,dtype,hq,n,norm", [(256, 128, "bf16", 32, 3100, True), (256, 256, "f16", 17, 5800, False),
                                                   (128, 64, "f32", 40, 2461, True), (96, 96, "f16", 48, 5470, True),
                                                   (64, 32, "bf16", 65, 6060, True)])
@pytest.mark.parametrize("inplace", [False, True])
def test_q8_append_many_large_q_rows(D, rot, dtype, hq, n, norm, inplace):
    """q of 8 KB a token and more, 48 MB in all: it goes through the rings, by a launch of its own."""
    es = 4 if dtype == "f32" else 2
    assert hq * D * es >= 8 << 10 and n * hq * D * es >= 48 << 20
    hkv, pages = 2, n // 16 + 2
    r = Rows([D, n], n, hq, hkv, D, dtype, norm, 1e4, rot)
    slots = page_slots(r.g, n, pages, 5)
    slots[n // 2] = -1 if slots[n // 2] % 16 == 15 else slots[n // 2]
    caches = pa.new_q8_cache(pages, hkv, D)
    rk, rv = ref.Cache(pages, hkv, D), ref.Cache(pages, hkv, D)
    rk.codes[...] = rv.codes[...] = 0
    q_out = r.tq if inplace else torch.full((n + 2, hq, D), 3.0, dtype=T[dtype], device="cuda")
    run_q8_append(r, slots, caches, q_out if inplace else q_out[1:-1])
    if not inplace:
        assert (q_out[0] == 3).all() and (q_out[-1] == 3).all()
        q_out = q_out[1:-1]
    for lo in range(0, n, 512):  # (the reference's fp64 rows a share at a time)
        x = r.q[lo:lo + 512]
        w = ref.turned(x, r.w[0], r.pos[lo:lo + 512], r.eps, r.theta, rot)
        tol = ref.turned_tolerance(x, r.w[0], w, r.eps, r.theta, rot, dtype)
        assert (np.abs(host(q_out[lo:lo + 512]) - w) <= tol).all()
    np.testing.assert_array_equal(host(r.tv), r.v)
    check_q8(r, slots, caches, rk, rv, exact_k=False)


# ---------------------------------------------------------------- verification of many sequences

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,V,drafts,ctas", [(160, 33000, 1, 640), (80, 70000, 2, 640), (155, 32771, 2, 620),
                                             (310, 20000, 2, 620), (610, 1500, 2, 610)])
def test_verify_more_sequences_than_a_wave(B, V, drafts, ctas, dtype):
    """More CTAs than one wave of 608: rows with few loads in flight, with and without clusters."""
    c = 1
    while c < 8 and V >= c * 2 * 2048:
        c *= 2
    while c > 1 and B * c > 608 and V <= c // 2 * 16384:
        c //= 2
    assert B * c == ctas > 608
    case = verify_case([V, B], B, V, drafts, dtype, ragged=True)
    check_verify(case, dtype)
    check_verify(case, dtype, offset=1)
    case["draft"], case["num"] = None, None
    check_verify(case, dtype)


# ---------------------------------------------------------------- angles

@pytest.mark.parametrize("n,hq,hkv", [(300, 2, 1), (1500, 1, 2), (900, 30, 1)])  # (threads; rings)
@pytest.mark.parametrize("theta,rot,far", [(1e4, 128, False), (1e4, 128, True), (5e5, 64, True)])
def test_append_cosines_and_sines_are_fp32s(n, hq, hkv, theta, rot, far):
    """Rows (1 .. 1, 0 .. 0) become cosines and sines.  Of a position's 64-bit turn the top 32 bits
    count (2^-32 of a turn), at most an eighth of a turn either way goes to fp32 (2^-28 of a turn, half a
    step), and the functions have a unit in the last place next to 1, 2^-24.  (Exactly: the steps
    of an angle x of at most a quarter half turn in fp32 leave the cosine, for z = x^2 <= 2^-4 and
    its series 1 + z Q with 4 <= |Q| < 8, half a step of the sum, 2^-25, of Q and of its constant,
    2^-4 2^-22 and 2^-4 1.5e-7, and of z, 2^-29 |Q|: 6.3e-8, with sin(pi / 4) of the angle's 2.5e-8
    together 8.1e-8 of the 8.4e-8 here; the sine's are smaller.)"""
    g = np.random.default_rng([n, rot])
    pos = (g.integers(-2 ** 31, 2 ** 31 - 1, n) if far else g.integers(0, 100000, n)).astype(np.int32)
    half, pages = rot // 2, n // 16 + 1
    x = torch.zeros(n, hq + 2 * hkv, 128, device="cuda")
    x[..., :half] = 1.0
    q_out = torch.empty(n, hq, 128, device="cuda")
    kc, vc = (torch.zeros(pages, hkv, 16, 128, device="cuda") for _ in range(2))
    pa.pa_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i64(np.arange(n)), i32(pos), kc, vc,
                 q_out=q_out, theta=theta, rotary_dim=rot)
    # (64 bits and more: a position of 2^31 has 31 of a double's 53 in front of the point)
    f = np.longdouble(theta) ** (-2 * np.arange(half, dtype=np.longdouble) / rot)
    ang = pos.astype(np.longdouble)[:, None] * f
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1)[:, None]
    room = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32) + 2.0 ** -24
    k = kc.transpose(1, 2).reshape(-1, hkv, 128)[:n]
    for got in (q_out, k):
        assert np.abs(host(got)[..., :rot] - want).max() <= room
        assert (host(got)[..., rot:] == 0).all()


# ---------------------------------------------------------------- norm weights without q

def test_append_without_q_does_not_use_its_norm():
    """With no q heads q_norm is not used, wherever it points and whatever eps is."""
    n, hkv, D = 20, 2, 64
    r = Rows(3, n, 0, hkv, D, "f16", False, 0.0, D)
    caches = [torch.zeros(2, hkv, 16, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    slots, w = i64(np.arange(n)), torch.ones(D + 1, dtype=torch.float16, device="cuda")
    s = r.tk.stride(0)
    st = q8._lib().pa_append(n, 0, hkv, D, D, 16, 2, 0, 0.0, -1.0, None, 0, r.tk.data_ptr(), s,
                             r.tv.data_ptr(), s, w[1:].data_ptr(), None, None, slots.data_ptr(), None, 0,
                             caches[0].data_ptr(), caches[1].data_ptr(), None,
                             torch.cuda.current_stream().cuda_stream)
    assert st == binding.PA_OK
    for c, want in zip(caches, (r.k, r.v)):
        np.testing.assert_array_equal(host(c).transpose(0, 2, 1, 3).reshape(-1, hkv, D)[:n], want)


# ---------------------------------------------------------------- pages of drafts that were not accepted

def free_list(past_lens, block_tables, num_pages):
    """The pages that no token in past_lens lies in, on the device; behind them ids of no page."""
    held = torch.arange(block_tables.shape[1], device="cuda") < ((past_lens + 15) // 16)[:, None]
    free = torch.ones(num_pages + 1, dtype=torch.bool, device="cuda")
    free[torch.where(held, block_tables, num_pages).long()] = False
    ids = torch.arange(num_pages, dtype=torch.int32, device="cuda")
    return torch.where(free[:-1], ids, num_pages).sort().values.int()


@pytest.mark.parametrize("give_back", [True, False])
def test_pages_of_drafts_that_were_not_accepted(give_back):
    """The loop over tables, rows, attention and verification, drafts mostly not accepted: with the
    pages that only they had begun given back the pool lasts, without them it runs out."""
    g = np.random.default_rng(6)
    B, Hq, Hkv, D, maxp, pages, drafts, V, steps = 4, 4, 2, 64, 8, 36, 4, 60, 100
    scale, n = D ** -0.5, B * (drafts + 1)
    caches = pa.new_q8_cache(pages, Hkv, D)
    plan = pa.pa_q8_plan(B, Hq, Hkv, D, 16, pages, maxp, maxp * 16, max_query_len=drafts + 1)
    ws = pa.new_workspace(plan, "cuda")
    table, past, ctx = i32(np.full((B, maxp), -1)), i32(np.zeros(B)), i32(np.zeros(B))
    new, starts, pos, taken = i32(np.full(B, drafts + 1)), i32(np.zeros(B + 1)), i32(np.zeros(n)), i32([0])
    slots = torch.zeros(n, dtype=torch.int64, device="cuda")
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    err = i32(np.zeros(64))
    accepted, tokens = i32(np.zeros(B)), i32(np.zeros((B, drafts + 1)))
    hp = np.zeros(B, np.int64)
    for step in range(steps):
        if hp.max() + drafts + 1 > maxp * 16:
            break
        r = Rows([5, step], n, Hq, Hkv, D, "f16", False, 0.0, D)
        q, out, lse = r.tq.contiguous(), torch.zeros(n, Hq, D, dtype=T["f16"], device="cuda"), torch.zeros(n, Hq, device="cuda")
        pa.pa_extend_tables(past, new, free, pages, table, ctx, starts, slots, pos, taken, err)
        pa.pa_q8_append(q, r.tk, r.tv, slots, pos, *caches)
        pa.pa_q8_decode(plan, q, starts, *caches, table, ctx, scale, 0, out, lse, ws)
        c = verify_case([8, step], B, V, drafts, "f32", near=3.0)
        args = [to_t(c["target"], "f32"), to_t(c["draft"], "f32"), i32(c["tok"]), None,
                torch.from_numpy(c["accept"]).cuda(), torch.from_numpy(c["sample"]).cuda()]
        pa.pa_verify_drafts(*args, accepted, tokens)
        bad = pa.pa_get_error_ex(err)
        if bad:
            break
        # every token's row is where the table says, and no page belongs to two sequences
        bt = table.cpu().numpy()
        lens = hp + drafts + 1
        np.testing.assert_array_equal(ctx.cpu().numpy(), lens)
        at = (hp[:, None] + np.arange(drafts + 1)).ravel()
        want = bt[np.arange(B).repeat(drafts + 1), at // 16].astype(np.int64) * 16 + at % 16
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
        held = np.concatenate([bt[b, :-(-lens[b] // 16)] for b in range(B)])
        assert len(set(held)) == len(held) and (held >= 0).all() and (held < pages).all()
        k, v = (ref.E4M3[code_bytes(x)] * host(y)[..., None, None] for x, y in ((caches[0], caches[2]), (caches[1], caches[3])))
        w, wl, tol, ltol = ref.decode(host(q), k, v, bt, lens, np.arange(B + 1) * (drafts + 1), scale, 0, "f16")
        assert (np.abs(host(out) - w) <= tol).all() and (np.abs(host(lse) - wl) <= ltol).all()
        past.add_(accepted + 1)
        hp = hp + accepted.cpu().numpy() + 1
        np.testing.assert_array_equal(past.cpu().numpy(), hp)
        free = free_list(past, table, pages) if give_back else free[int(taken):]
    if give_back:
        assert bad == 0 and pa.pa_get_error(ws) == 0 and hp.max() > 100
    else:
        assert bad == q4.PA_DEVERR_NO_PAGES and hp.max() < 100
