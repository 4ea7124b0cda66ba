"""GPU tests of include/pa_q8.h (pa_append, pa_q8_append, pa_q8_read,
pa_q8_decode, pa_verify_drafts) against the fp64 reference: codes, scales and
tokens exactly, what is computed within the bounds the reference derives."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q8_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q4, q8
from paged_kv_gqa_pa_gb300 import build as pa_build
from test_q4_gpu import late_writer  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DT = {"f16": 0, "bf16": 1, "f32": 2}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    pa_build.build()
    pa.load()


def rounded(x, dtype):
    """fp64 values rounded to T (through fp32, whose own rounding the values do not need)."""
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(T[dtype]).double().numpy()


def to_t(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().float().to(T[dtype])


def host(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def i64(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int64)).cuda()


def f8(codes):
    return torch.from_numpy(codes).cuda().view(F8)


def code_bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def rows(g, shape, dtype):
    x = g.standard_normal(shape) * np.where(g.random(shape[-1]) < 0.05, 6.0, 1.0)
    return rounded(x + g.standard_normal(shape[-1]) * 0.5, dtype)


def page_slots(g, n, pages, begin=0):
    """Slots of n rows in order through shuffled pages, the first at position `begin`."""
    perm = g.permutation(pages)
    flat = begin + np.arange(n)
    return perm[flat // 16].astype(np.int64) * 16 + flat % 16


# ---------------------------------------------------------------- appending

class Rows:
    """q, k, v as columns of a fused projection's rows, and what the call gets beside them."""

    def __init__(self, seed, n, hq, hkv, D, dtype, norm, theta, rot, far=False):
        g = self.g = np.random.default_rng(seed)
        self.dtype, self.eps, self.theta, self.rot = dtype, 1e-5, theta, rot
        x = rows(g, (n, hq + 2 * hkv, D), dtype)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        self.pos = g.integers(0, 2 ** 31 - 1 if far else 5000, n).astype(np.int32)
        self.w = [rounded(1 + 0.3 * g.standard_normal(D), dtype) if norm else None
                  for _ in range(2)]
        t = to_t(x, dtype)
        self.tq, self.tk, self.tv = t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:]
        self.kw = dict(q_norm=None if not norm else to_t(self.w[0], dtype),
                       k_norm=None if not norm else to_t(self.w[1], dtype), eps=self.eps,
                       theta=theta, rotary_dim=rot)

    def want(self, x, which, dtype):
        w = ref.turned(x, self.w[which], self.pos, self.eps, self.theta, self.rot)
        return w, ref.turned_tolerance(x, self.w[which], w, self.eps, self.theta, self.rot, dtype)

    def check_q(self, q_out):
        w, tol = self.want(self.q, 0, self.dtype)
        assert (np.abs(host(q_out) - w) <= tol).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (96, 96), (96, 48), (128, 128), (128, 64),
                                   (256, 256), (256, 32)])
@pytest.mark.parametrize("norm,theta", [(True, 1e4), (False, 5e5), (True, 0.0), (False, 0.0)])
def test_append(D, rot, dtype, norm, theta):
    n, hq, hkv, pages = 37, 6, 3, 5
    r = Rows(D + rot, n, hq, hkv, D, dtype, norm, theta, rot)
    slots = page_slots(r.g, n, pages, 3)
    slots[[4, 20]] = -1
    before = rows(r.g, (2, pages, hkv, 16, D), dtype)
    kc, vc = to_t(before[0], dtype), to_t(before[1], dtype)
    q_out = torch.full((n, hq, D), float("nan"), dtype=T[dtype], device="cuda")
    pa.pa_append(r.tq, r.tk, r.tv, i64(slots), i32(r.pos), kc, vc, q_out=q_out, **r.kw)
    r.check_q(q_out)
    k, tol = r.want(r.k, 1, dtype)
    got_k, got_v = host(kc), host(vc)
    there = np.zeros((pages, 16), bool)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        there[s // 16, s % 16] = True
        assert (np.abs(got_k[s // 16, :, s % 16] - k[i]) <= tol[i]).all()
        np.testing.assert_array_equal(got_v[s // 16, :, s % 16], r.v[i])
    other = ~there[:, None, :, None] & np.ones_like(got_k, bool)
    np.testing.assert_array_equal(got_k[other], before[0][other])
    np.testing.assert_array_equal(got_v[other], before[1][other])


@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (1, 32, 8), (3, 0, 2), (300, 5, 1), (2, 40, 20)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_append_shapes_in_place(n, hq, hkv, dtype):
    D = 128
    r = Rows(n + hq, n, hq, hkv, D, dtype, True, 1e4, D)
    slots = r.g.permutation(16 * 40)[:n]
    kc, vc = (torch.zeros(40, hkv, 16, D, dtype=T[dtype], device="cuda") for _ in range(2))
    kw = dict(r.kw)
    if hq == 0:
        kw["q_norm"] = None
    pa.pa_append(r.tq if hq else None, r.tk, r.tv, i64(slots), i32(r.pos), kc, vc, **kw)
    if hq:
        r.check_q(r.tq)  # (written where q was)
    k, tol = r.want(r.k, 1, dtype)
    got = host(kc)[slots // 16, :, slots % 16]
    assert (np.abs(got - k) <= tol).all()
    np.testing.assert_array_equal(host(vc)[slots // 16, :, slots % 16], r.v)
    np.testing.assert_array_equal(host(r.tk), r.k)
    np.testing.assert_array_equal(host(r.tv), r.v)


@pytest.mark.parametrize("n", [609, 1301])
@pytest.mark.parametrize("D,rot,dtype,hq,hkv", [(64, 64, "f16", 8, 8), (96, 48, "f16", 8, 2), (64, 16, "bf16", 1, 1),
                                                (64, 64, "f32", 32, 4), (96, 96, "bf16", 48, 8),
                                                (128, 64, "f16", 32, 8), (256, 256, "bf16", 16, 2)])
def test_append_some_hundred_tokens(n, D, rot, dtype, hq, hkv):
    """Tokens of one warp each, two to a CTA, the last one alone; tokens of 8 KB and more,
    through rings of them."""
    test_append_many_tokens(n, D, rot, dtype, hq, hkv)


@pytest.mark.parametrize("n", [2048, 2700, 5001])
@pytest.mark.parametrize("D,rot,dtype,hq,hkv", [(64, 32, "f32", 3, 1), (96, 96, "bf16", 4, 2), (128, 128, "f16", 5, 1),
                                                (256, 64, "bf16", 2, 1), (128, 128, "f32", 40, 8), (256, 256, "f32", 64, 1),
                                                (64, 64, "f16", 0, 3)])
def test_append_many_tokens(n, D, rot, dtype, hq, hkv):
    """Prompts of so many tokens that CTAs go through several; rows too wide for a ring of them."""
    if n > 2000 and n != 2700 and hq >= 40:
        pytest.skip("one length is enough")
    r = Rows(n + D, n, hq, hkv, D, dtype, True, 1e4, rot)
    pages = n // 16 + 3
    slots = page_slots(r.g, n, pages, 5)
    slots[r.g.random(n) < 0.1] = -1
    q_out = torch.full((n, hq, D), float("nan"), dtype=T[dtype], device="cuda") if hq else None
    kw = dict(r.kw)
    if not hq:
        kw["q_norm"] = None
    k, tol = r.want(r.k, 1, dtype)
    kept = slots >= 0
    kc, vc = (torch.full((pages, hkv, 16, D), 7.0, dtype=T[dtype], device="cuda") for _ in range(2))
    for place in ("out", "in place"):
        pa.pa_append(r.tq if hq else None, r.tk, r.tv, i64(slots), i32(r.pos), kc, vc,
                     q_out=q_out if place == "out" else None, **kw)
        if hq:
            r.check_q(q_out if place == "out" else r.tq)
        got_k, got_v = host(kc), host(vc)
        s = slots[kept]
        assert (np.abs(got_k[s // 16, :, s % 16] - k[kept]) <= tol[kept]).all()
        np.testing.assert_array_equal(got_v[s // 16, :, s % 16], r.v[kept])
        rest = np.ones((pages, 16), bool)
        rest[s // 16, s % 16] = False
        assert (got_k.transpose(0, 2, 1, 3)[rest] == 7).all() and (got_v.transpose(0, 2, 1, 3)[rest] == 7).all()


@pytest.mark.parametrize("norms", ["both", "q", "k", "none"])
@pytest.mark.parametrize("n", [40, 2100])
def test_append_with_either_norm(norms, n):
    D, hq, hkv = 128, 4, 2
    r = Rows(n, n, hq, hkv, D, "f16", True, 1e4, 64)
    for i, name in enumerate("qk"):
        if norms not in ("both", name):
            r.w[i] = r.kw[name + "_norm"] = None
    slots = np.arange(n)
    pages = n // 16 + 1
    kc, vc = (torch.zeros(pages, hkv, 16, D, dtype=torch.float16, device="cuda") for _ in range(2))
    q_out = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
    pa.pa_append(r.tq, r.tk, r.tv, i64(slots), i32(r.pos), kc, vc, q_out=q_out, **r.kw)
    r.check_q(q_out)
    k, tol = r.want(r.k, 1, "f16")
    assert (np.abs(host(kc).transpose(0, 2, 1, 3).reshape(-1, hkv, D)[:n] - k) <= tol).all()
    caches = pa.new_q8_cache(pages, hkv, D)
    q2 = torch.empty_like(q_out)
    run_q8_append(r, slots, caches, q2)
    r.check_q(q2)
    check_q8(r, slots, caches, zero_cache(pages, hkv, D), zero_cache(pages, hkv, D), exact_k=False)


def zero_cache(pages, H, D):
    c = ref.Cache(pages, H, D)
    c.codes[...] = 0
    return c


def test_append_keeps_infinities_behind_the_rotated_dims_apart():
    # dims behind rotary_dim are not mixed: an infinity there stays in its place
    for n in (3, 2048):
        r = Rows(n, n, 2, 1, 64, "f32", False, 1e4, 32)
        r.tq[:, :, 40] = float("inf")
        kc, vc = (torch.zeros(n // 16 + 1, 1, 16, 64, device="cuda") for _ in range(2))
        q_out = torch.empty(n, 2, 64, device="cuda")
        pa.pa_append(r.tq, r.tk, r.tv, i64(np.arange(n)), i32(r.pos), kc, vc, q_out=q_out, **r.kw)
        got = host(q_out)
        assert np.isinf(got[..., 40]).all() and np.isfinite(np.delete(got, 40, -1)).all()
        np.testing.assert_array_equal(np.delete(got[..., 32:], 8, -1), np.delete(r.q[..., 32:], 8, -1))


def test_append_far_positions():
    r = Rows(5, 200, 2, 1, 64, "f32", False, 1e4, 64, far=True)
    r.pos[:3] = [2 ** 31 - 1, -2 ** 31, -1]
    kc, vc = (torch.zeros(20, 1, 16, 64, device="cuda") for _ in range(2))
    q_out = torch.empty(200, 2, 64, device="cuda")
    pa.pa_append(r.tq, r.tk, r.tv, i64(np.arange(200)), i32(r.pos), kc, vc, q_out=q_out, **r.kw)
    # the fp64 angle itself is off by 2^31 (2^-53 of it and of its frequency) radians
    w, tol = r.want(r.q, 0, "f32")
    pair = np.abs(r.q[..., :32]) + np.abs(r.q[..., 32:])
    assert (np.abs(host(q_out) - w) <= tol + np.concatenate([pair, pair], -1) * 2.0 ** -20).all()


@pytest.mark.parametrize("fn", ["pa_append", "pa_q8_append"])
def test_append_bad_slots_are_left_out_and_reported(fn):
    n, D, pages = 6, 64, 2
    r = Rows(6, n, 2, 1, D, "f16", False, 0.0, D)
    err = torch.zeros(64, dtype=torch.int32, device="cuda")
    for bad in (32, -2, 1 << 40, -(1 << 62)):
        slots = [0, 1, bad, -1, 16, 17]
        q_out = torch.empty(n, 2, D, dtype=torch.float16, device="cuda")
        if fn == "pa_append":
            kc, vc = (torch.zeros(pages, 1, 16, D, dtype=torch.float16, device="cuda") for _ in range(2))
            pa.pa_append(r.tq, r.tk, r.tv, i64(slots), None, kc, vc, q_out=q_out, device_error=err)
            got = host(kc)
        else:
            kc, vc, ks, vs = pa.new_q8_cache(pages, 1, D)
            pa.pa_q8_append(r.tq, r.tk, r.tv, i64(slots), None, kc, vc, ks, vs, q_out=q_out,
                            device_error=err)
            got = ref.E4M3[code_bytes(kc)]
        assert pa.pa_get_error_ex(err) == q4.PA_DEVERR_BAD_SLOT
        assert torch.equal(q_out, r.tq.contiguous())
        used = np.abs(got).max((1, 3)) > 0
        assert used[0, :2].all() and used[1, :2].all() and used.sum() == 4


def run_q8_append(r, slots, caches, q_out=None, **kw):
    a = dict(r.kw, **kw)
    pa.pa_q8_append(r.tq if q_out is not None else None, r.tk, r.tv, i64(slots), i32(r.pos), *caches,
                    q_out=q_out, **(a if q_out is not None else dict(a, q_norm=None)))


def check_q8(r, slots, caches, rk, rv, exact_k):
    """The caches against the reference's, which the same rows are appended to."""
    k, tol = r.want(r.k, 1, None)
    old_scales = rk.scales.copy()
    rk.append(k, slots)
    rv.append(r.v, slots)
    kc, vc, ks, vs = caches
    np.testing.assert_array_equal(host(vs), rv.scales)
    np.testing.assert_array_equal(code_bytes(vc) & 127 == 127, rv.codes & 127 == 127)
    np.testing.assert_array_equal(ref.E4M3[code_bytes(vc)], ref.E4M3[rv.codes])
    np.testing.assert_array_equal(host(ks), rk.scales)
    got, want = ref.E4M3[code_bytes(kc)], ref.E4M3[rk.codes]
    if exact_k:
        np.testing.assert_array_equal(got, want)
        return
    # A code is the nearest to a value that is off by tol; kept rows follow exactly.
    fine = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), fine)
    diff = np.where(fine, got - want, 0.0)
    ok = diff == 0
    for i, s in enumerate(slots):
        if s < 0:
            continue
        p, at = s // 16, s % 16
        sc = rk.scales[p][:, None]
        room = sc * ref.e4m3_step(np.abs(k[i]) / sc + tol[i] / sc) / 2 + tol[i]
        good = np.abs(got[p, :, at] * sc - k[i]) <= room * (1 + 1e-12)
        assert good.all()
        ok[p, :, at] = True
    assert ok.all()
    rk.codes[...] = code_bytes(kc)  # (what follows builds on the codes that are there)
    assert old_scales.shape == rk.scales.shape


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(64, 32), (96, 96), (128, 128), (256, 256)])
@pytest.mark.parametrize("norm,theta", [(True, 1e4), (False, 0.0)])
def test_q8_append_in_steps(D, rot, dtype, norm, theta):
    """A prompt that ends inside a page, then steps of a few rows and of one, which raise scales
    and begin pages; cells hold NaN before."""
    hq, hkv, pages = 4, 3, 9
    caches = (f8(np.full((pages, hkv, 16, D), 127, np.uint8)),
              f8(np.full((pages, hkv, 16, D), 127, np.uint8)),
              torch.full((pages, hkv), float("nan"), device="cuda"),
              torch.full((pages, hkv), -1.0, device="cuda"))
    rk, rv = ref.Cache(pages, hkv, D), ref.Cache(pages, hkv, D)
    perm = np.random.default_rng(D).permutation(pages)
    at = 0
    for step, n in enumerate((37, 1, 1, 5, 1, 17, 1, 1, 16, 3, 1, 40)):
        r = Rows([D, step], n, hq, hkv, D, dtype, norm, theta, rot)
        f = 2.0 ** (step % 5 - 1)  # (rows of other sizes: some raise the scale)
        if not norm:
            r.k, r.v = r.k * f, r.v * f
            r.tk.mul_(f)
            r.tv.mul_(f)
        flat = at + np.arange(n)
        slots = perm[flat // 16] * 16 + flat % 16
        if step == 9:
            slots[1] = -1  # a row left out ends a run: what follows in its page is another call's
            slots[2:] = -1
            at -= 2
        at += n
        q_out = torch.empty(n, hq, D, dtype=T[dtype], device="cuda")
        run_q8_append(r, slots, caches, q_out)
        r.check_q(q_out)
        # pages never written keep what they hold
        never = np.isnan(host(caches[2]))
        rk.scales[never], rv.scales[never] = np.nan, -1.0
        check_q8(r, slots, caches, rk, rv, exact_k=not norm and theta == 0)
    assert not np.isnan(host(caches[2])).all()


@pytest.mark.parametrize("hkv,n,order", [(8, 64, "decode"), (1, 3000, "prompt"), (8, 700, "chunks"),
                                         (5, 400, "decode"), (2, 4100, "decode"), (4, 5000, "prompt")])
def test_q8_append_sizes(hkv, n, order):
    """Grids of either tile, one head a CTA or several; rows of other sequences in between."""
    D = 64
    r = Rows(n, n, 2, hkv, D, "bf16", False, 0.0, D)
    g = r.g
    if order == "decode":
        pages = n + 7
        at = g.integers(0, 16, n)
        slots = g.permutation(pages)[:n] * 16 + at
    elif order == "prompt":
        pages = n // 16 + 4
        slots = page_slots(g, n, pages, 9)
    else:
        parts = []
        left, base = n, 0
        while left:
            m = min(left, int(g.integers(1, 60)))
            parts.append(base * 16 + int(g.integers(0, 16)) + np.arange(m))
            base = int(parts[-1][-1]) // 16 + 1
            left -= m
        pages = base + 1
        slots = g.permutation(pages)[np.concatenate(parts) // 16] * 16 + np.concatenate(parts) % 16
    rk, rv = ref.Cache(pages, hkv, D), ref.Cache(pages, hkv, D)
    had = [rows(g, (pages * 16, hkv, D), "bf16") * 0.25 for _ in range(2)]
    for c, x in zip((rk, rv), had):
        c.append(x, np.arange(pages * 16))
    caches = (f8(rk.codes), f8(rv.codes), torch.from_numpy(rk.scales).float().cuda(),
              torch.from_numpy(rv.scales).float().cuda())
    run_q8_append(r, slots, caches)
    # only rows before a run are kept up: what lies behind it is compared as it was
    want_k, want_v = rk.codes.copy(), rv.codes.copy()
    check_q8(r, slots, caches, rk, rv, exact_k=True)
    assert (want_k != rk.codes).any() and (want_v != rv.codes).any()


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (64, "f32"), (96, "bf16"), (128, "f16"), (128, "f32"),
                                     (256, "bf16"), (256, "f32")])
@pytest.mark.parametrize("hkv,most", [(1, 1), (2, 3), (3, 6), (20, 1), (9, 20)])
def test_q8_append_steps_of_many_sequences(D, dtype, hkv, most):
    """Tiles of several runs, of one row each or a few, beside rows that are left out; runs that
    go on behind their tile or in the next page; infinities and NaN in some of the rows."""
    n = 40 if hkv == 20 else 333
    r = Rows(D + most, n, 2, hkv, D, dtype, True, 1e4, D)
    g = r.g
    slots, page = [], 0
    while len(slots) < n:
        at = int(g.integers(0, 16)) + np.arange(int(g.integers(1, most + 1)))
        slots += list((page + at // 16) * 16 + at % 16)
        page += int(at[-1]) // 16 + 1
        if g.random() < 0.1:
            slots.append(-1)
    slots = np.array(slots[:n])
    perm = g.permutation(page + 2)
    slots = np.where(slots < 0, -1, perm[slots // 16] * 16 + slots % 16)
    for value in (np.inf, -np.inf, np.nan):
        i, h, d = g.integers(0, n, 12), g.integers(0, hkv, 12), g.integers(0, D, 12)
        r.v[i, h, d] = value
        r.tv[torch.from_numpy(i).cuda(), torch.from_numpy(h).cuda(), torch.from_numpy(d).cuda()] = value
    r.v[n // 2] = 0.0
    r.tv[n // 2] = 0.0
    rk, rv = ref.Cache(page + 2, hkv, D), ref.Cache(page + 2, hkv, D)
    for c in (rk, rv):
        c.append(rows(g, ((page + 2) * 16, hkv, D), dtype) * 0.25, np.arange((page + 2) * 16))
    caches = (f8(rk.codes), f8(rv.codes), torch.from_numpy(rk.scales).float().cuda(),
              torch.from_numpy(rv.scales).float().cuda())
    run_q8_append(r, slots, caches)
    check_q8(r, slots, caches, rk, rv, exact_k=False)


@pytest.mark.parametrize("n", [1, 3, 50, 1001])
@pytest.mark.parametrize("D,dtype,hq", [(128, "f16", 1), (128, "bf16", 6), (128, "f16", 9), (256, "f32", 3), (64, "bf16", 5),
                                        (96, "f32", 4), (256, "f16", 17)])
def test_q8_append_queries_of_few_heads(n, D, dtype, hq):
    """q of several tokens to a CTA, of one, of threads that are left over."""
    r = Rows(n + hq, n, hq, 1, D, dtype, True, 1e4, D // 2)
    pages = n // 16 + 2
    caches = pa.new_q8_cache(pages, 1, D)
    for q_out in (torch.full((n, hq, D), float("nan"), dtype=T[dtype], device="cuda"), r.tq):
        run_q8_append(r, np.arange(n), caches, q_out=q_out)
        r.check_q(q_out)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_q8_append_special_values(dtype):
    """Infinities and NaN, zeros of both signs, values at the borders of scales and codes, the
    largest and the least numbers."""
    D, g = 64, np.random.default_rng(9)
    big = {"f16": 65504.0, "bf16": float(torch.finfo(torch.bfloat16).max),
           "f32": float(torch.finfo(torch.float32).max)}[dtype]
    tiny = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "f32": 2.0 ** -149}[dtype]
    lines = [np.zeros(D), np.full(D, -0.0), np.full(D, np.inf), np.full(D, np.nan),
             np.where(np.arange(D) == 7, np.inf, 1.0), np.where(np.arange(D) == 63, np.nan, -2.0),
             np.where(np.arange(D) == 0, -np.inf, g.standard_normal(D)),
             np.full(D, big), np.where(np.arange(D) == 9, -big, 1.0), np.full(D, tiny),
             np.where(np.arange(D) < 2, 448.0, np.arange(D) / 2), np.where(np.arange(D) < 2, 450.0, 1.0),
             np.concatenate([ref.E4M3[:126:2], [448.0]]),
             np.concatenate([(ref.E4M3[:126:2] + ref.E4M3[1:127:2]) / 2, [448.0]]),
             np.where(np.arange(D) == 1, 448.0, 2.0 ** -10), np.where(np.arange(D) == 1, 448.0, 3 * 2.0 ** -10)]
    x = rounded(np.stack(lines), dtype)[:, None]
    n = len(lines)
    # each row in a page of its own; then all of them one after the other in one page
    for slots in (np.arange(n) * 16, np.arange(n)):
        caches = pa.new_q8_cache(n, 1, D)
        rv = ref.Cache(n, 1, D)
        rv.codes[...] = 0
        t = to_t(x, dtype)
        pa.pa_q8_append(None, t, t, i64(slots), None, *caches)
        rv.append(x, slots)
        for codes, scales in ((caches[0], caches[2]), (caches[1], caches[3])):
            np.testing.assert_array_equal(host(scales), rv.scales)
            np.testing.assert_array_equal(ref.E4M3[code_bytes(codes)], ref.E4M3[rv.codes])
        k, v = torch.empty_like(t), torch.empty_like(t)
        pa.pa_q8_read(*caches, i64(slots), k, v)
        with np.errstate(over="ignore"):
            want = rounded(rv.values()[slots // 16, :, slots % 16], dtype)
        np.testing.assert_array_equal(host(k), want)
        np.testing.assert_array_equal(host(v), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,H,n", [(64, 1, 1), (96, 3, 50), (128, 8, 300), (256, 2, 4000)])
def test_q8_read(D, H, n, dtype):
    g = np.random.default_rng(n)
    pages = 40
    codes = [g.integers(0, 256, (pages, H, 16, D)).astype(np.uint8) for _ in range(2)]
    scales = [np.exp(g.standard_normal((pages, H))).astype(np.float32) for _ in range(2)]
    slots = g.integers(-1, pages * 16, n)  # some twice, some -1
    bad = n // 2
    slots[bad] = pages * 16
    wide = torch.full((n, 2 * H, D), 7.0, dtype=T[dtype], device="cuda")
    k, v = wide[:, :H], wide[:, H:]
    err = torch.zeros(64, dtype=torch.int32, device="cuda")
    pa.pa_q8_read(f8(codes[0]), f8(codes[1]), *[torch.from_numpy(s).cuda() for s in scales], i64(slots),
                  k, v, err)
    assert pa.pa_get_error_ex(err) == q4.PA_DEVERR_BAD_SLOT
    for got, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        # a code has 4 significant bits and the scale 24: the product in fp32, then to T
        x = (ref.E4M3[c].astype(np.float32) * s[..., None, None])[slots % (pages * 16) // 16, :, slots % 16]
        x = np.where((slots < 0)[:, None, None], 0.0, x)
        x[bad] = np.nan
        np.testing.assert_array_equal(host(got), rounded(x.astype(np.float64), dtype))


def test_append_offsets_beyond_32_bits():
    # 16-bit cache of 600,000 pages x 16 x 256 elements: 4.9 GB, K and V; 8-bit: 1.1 million pages.
    D, n = 256, 40
    r = Rows(11, n, 1, 1, D, "f16", False, 0.0, D)
    for fn, pages in (("pa_append", 600_000), ("pa_q8_append", 1_100_000)):
        ids = np.array([pages - 1, 0, pages - 3])
        flat = np.arange(n)
        slots = ids[flat // 16] * 16 + flat % 16
        at = torch.from_numpy(ids).cuda()
        if fn == "pa_append":
            kc, vc = (torch.empty(pages, 1, 16, D, dtype=torch.float16, device="cuda") for _ in range(2))
            pa.pa_append(None, r.tk, r.tv, i64(slots), None, kc, vc)
            got = host(kc[at]).transpose(0, 2, 1, 3).reshape(-1, 1, D)[:n]
            np.testing.assert_array_equal(got, r.k)
        else:
            kc, vc = (torch.empty(pages, 1, 16, D, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
            ks, vs = (torch.ones(pages, 1, device="cuda") for _ in range(2))
            pa.pa_q8_append(None, r.tk, r.tv, i64(slots), None, kc, vc, ks, vs)
            rk = ref.Cache(3, 1, D)
            rk.append(r.k, flat)
            got = kc.view(torch.uint8)[at].cpu().numpy()
            np.testing.assert_array_equal(got[:2], rk.codes[:2])
            np.testing.assert_array_equal(got[2, :, :8], rk.codes[2, :, :8])
            k, v = torch.empty_like(r.tk.contiguous()), torch.empty_like(r.tk.contiguous())
            pa.pa_q8_read(kc, vc, ks, vs, i64(slots), k, v)
            want = rk.values().transpose(0, 2, 1, 3).reshape(-1, 1, D)[:n]
            np.testing.assert_array_equal(host(k), rounded(want, "f16"))
        del kc, vc


# ---------------------------------------------------------------- attention

class Decode:
    """A cache whose cells are NaN wherever no token lies, and the queries of a step."""

    def __init__(self, seed, lens, Hq, Hkv, D, dtype, T=1, new=None, q_std=1.0, spread=0.0,
                 pow2=True, pad=0, maxp=None):
        g = self.g = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        B = len(lens)
        self.T, self.dtype, self.pow2 = T, dtype, pow2
        new = np.minimum(g.integers(1, T + 1, B), self.lens) if new is None else np.asarray(new)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        need = -(-self.lens // 16)
        self.pages = pages = int(need.sum()) + 3
        perm = g.permutation(pages)
        self.maxp = maxp or max(1, int(need.max()) if B else 1)
        self.bt = np.full((B, self.maxp), -1, np.int32)
        live = np.zeros(pages, int)
        at = 0
        for b, n in enumerate(need):
            ids = perm[at:at + n]
            self.bt[b, :n] = ids
            live[ids] = np.minimum(16, self.lens[b] - 16 * np.arange(n))
            at += n
        self.unused = perm[at:]
        x = g.integers(0, 256, (2, pages, Hkv, 16, D)).astype(np.uint8)
        x = np.where(x & 127 == 127, x & 129, x)
        # codes like a quantiser's: most of them of moderate size
        x = np.where(g.random(x.shape) < 0.9, (x & 0x87) | (0x28 + (x & 0x18)), x).astype(np.uint8)
        hidden = np.arange(16)[None, None, :, None] >= live[:, None, None, None]
        x = np.where(hidden, np.uint8(127), x)
        self.codes = x
        s = 2.0 ** np.rint(-6 + g.standard_normal((2, pages, Hkv)) * [[[min(spread, 1)]], [[spread]]])
        if not pow2:
            s = s * g.uniform(0.5, 1.0, s.shape)
        self.scales = s.astype(np.float32)
        n_rows = int(self.starts[-1]) + pad
        self.q = rounded(g.standard_normal((n_rows, Hq, D)) * q_std, dtype)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D

    def values(self):
        with np.errstate(invalid="ignore"):
            return [ref.E4M3[c] * s.astype(np.float64)[..., None, None]
                    for c, s in zip(self.codes, self.scales)]

    def want(self, scale, window):
        return ref.decode(self.q, *self.values(), self.bt, self.lens, self.starts, scale, window,
                          self.dtype, self.pow2)

    def device(self):
        return [f8(self.codes[0]), f8(self.codes[1]), torch.from_numpy(self.scales[0]).cuda(),
                torch.from_numpy(self.scales[1]).cuda()]

    def plan(self, window=0, max_len=None, ctas=None, cluster=None, sms=0):
        p = pa.pa_q8_plan(len(self.lens), self.Hq, self.Hkv, self.D, 16, self.pages, self.maxp,
                          int(self.lens.max(initial=0)) if max_len is None else max_len, window,
                          self.T, sms, DT[self.dtype])
        if ctas is not None:
            p.ctas_per_group, p.cluster = ctas, 0
        if cluster == 0:
            p.cluster = 0
        return p

    def run(self, scale, window=0, ws=None, stall=0, starts=True, **kw):
        p = self.plan(window, **kw)
        p.test_stall_bytes = stall
        n, guard = self.q.shape[0], 64
        ob = torch.full((n * self.Hq * self.D + 2 * guard,), 3.0, dtype=T[self.dtype], device="cuda")
        lb = torch.full((n * self.Hq + 2 * guard,), 5.0, device="cuda")
        if ws is None:  # only the control bytes start at zero
            ws = torch.full((p.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
            ws[:p.ctrl_bytes] = 0
        out, lse = ob[guard:-guard].view(n, self.Hq, self.D), lb[guard:-guard].view(n, self.Hq)
        pa.pa_q8_decode(p, to_t(self.q, self.dtype), i32(self.starts) if starts else None,
                        *self.device(), i32(self.bt), i32(self.lens), scale, window, out, lse, ws)
        err = pa.pa_get_error_ex(ws)
        assert int(ws[:p.ctrl_bytes].count_nonzero()) == 0, "control bytes not left zero"
        last = int(self.starts[-1]) if starts else len(self.lens)
        assert (ob[:guard] == 3).all() and (ob[-guard:] == 3).all() and (out[last:] == 3).all()
        assert (lb[:guard] == 5).all() and (lb[-guard:] == 5).all() and (lse[last:] == 5).all()
        return host(out[:last]), host(lse[:last]), err

    def check(self, got, want, only=slice(None)):
        out, lse, err = got
        n = out.shape[0]
        w_out, w_lse, tol, ltol = (x[:n][only] for x in want)
        out, lse = out[only], lse[only]
        assert err == 0
        np.testing.assert_array_equal(np.isnan(out), np.isnan(w_out))
        if self.dtype == "f16":
            # Beyond 65520 fp16 is infinite.  As 65536, the next number it would have, an
            # infinity is a rounding like any other (half a step, 16 or 32, is in the
            # tolerance), and limiting both sides brings them no further apart.
            out, w_out = np.clip(out, -65536, 65536), np.clip(w_out, -65536, 65536)
        over = np.abs(out - w_out) - tol
        assert not (over > 0).any(), f"beyond by {np.nanmax(over):.3e}"
        fin = np.isfinite(w_lse)
        np.testing.assert_array_equal(lse[~fin], w_lse[~fin])
        assert (np.abs(lse[fin] - w_lse[fin]) <= ltol[fin]).all()

    def case(self, scale=None, window=0, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        got = self.run(scale, window, **kw)
        self.check(got, self.want(scale, window))
        return got


DIMS = [(64, "f16"), (96, "bf16"), (128, "f16"), (128, "bf16"), (256, "f16"), (256, "bf16")]


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 1), (12, 1), (20, 1), (27, 1), (10, 5)])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_lengths(Hq, Hkv, D, dtype, cluster):
    Decode(D + Hq, [1, 15, 16, 17, 0, 255, 700], Hq, Hkv, D, dtype).case(cluster=cluster)


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("queries", [2, 3, 5, 8, 16])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_several_queries(queries, D, dtype, cluster):
    d = Decode(queries, [queries, 15, 16, 17, 0, 1, 255, 700, 33], 4, 2, D, dtype, T=queries, pad=3)
    d.case(cluster=cluster)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (96, "f16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 333, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("queries,cluster", [(1, None), (1, 0), (4, None), (4, 0)])
def test_decode_windows(window, D, dtype, queries, cluster):
    Decode(window % 1000, [1, 4, 16, 33, 333, 1000, 0], 4, 2, D, dtype, T=queries).case(
        window=window, cluster=cluster)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (96, "f16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("C", [2, 3, 7, 8])
@pytest.mark.parametrize("queries", [1, 3])
def test_decode_cluster_sizes(C, D, dtype, queries):
    lens = [3, 16, 17, 0, 400, 16 * C, 16 * C + 1, 33 * C]
    d = Decode(60 + C, lens, 6, 2, D, dtype, T=queries)
    p = d.plan()
    p.cluster, p.ctas_per_group = C, C * len(lens)
    p.workspace_bytes, p.ctrl_bytes = 1 << 28, max(p.ctrl_bytes, 4096)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    tq = to_t(d.q, dtype)
    out, lse = torch.full_like(tq, 3.0), torch.empty(tq.shape[0], 6, device="cuda")
    pa.pa_q8_decode(p, tq, i32(d.starts), *d.device(), i32(d.bt), i32(d.lens), 0.1, 0, out, lse, ws)
    d.check((host(out), host(lse), pa.pa_get_error(ws)), d.want(0.1, 0))


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (96, "bf16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 60])
@pytest.mark.parametrize("queries", [1, 4])
def test_decode_ranges_cut_anywhere(ctas, D, dtype, queries):
    # Ranges of the batch's pages: one CTA for all, cuts inside and between sequences, many
    # sequences in one range; 60 leave more partials than the last CTA merges.
    lens = [40, 1, 0, 16, 0, 900, 128, 128, 3, 0] + [20] * 20
    if ctas == 60:
        lens = [900, 3, 0, 1500]
    d = Decode(7, lens, 4, 1, D, dtype, T=queries)
    p = d.plan()
    if ctas == 60:
        p = d.plan(sms=2000)
        ctas = p.ctas_per_group if p.cluster == 0 else 60
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        p.cluster, p.ctas_per_group, p.workspace_bytes = 0, 60, 1 << 26
        tq = to_t(d.q, dtype)
        out, lse = torch.full_like(tq, 3.0), torch.empty(tq.shape[0], 4, device="cuda")
        pa.pa_q8_decode(p, tq, i32(d.starts), *d.device(), i32(d.bt), i32(d.lens), 0.1, 0, out, lse,
                        ws)
        d.check((host(out), host(lse), pa.pa_get_error(ws)), d.want(0.1, 0))
    else:
        d.case(ctas=ctas)


@pytest.mark.parametrize("longest", [30, 60, 62, 63, 64, 65, 66, 67, 68, 90])
@pytest.mark.parametrize("queries,window", [(1, 0), (3, 700)])
def test_decode_sequences_with_a_cta_each(longest, queries, window):
    # Seven CTAs for six sequences: one each, or, from a longest sequence of about 65 pages
    # on, equal ranges.
    lens = [30 * 16, 29 * 16 + 1, 30 * 16, 0, 30 * 16 - 5, 16 * longest]
    Decode(longest, lens, 4, 1, 64, "f16", T=queries).case(window=window, ctas=7)


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("queries", [1, 3, 8])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_lse_is_of_the_unrounded_weights(D, dtype, queries, cluster):
    # The bound less what rounding the weights to 11 bits would add, with 2^-24 for each of the
    # additions a weight goes through.
    d = Decode(45 + queries, [3, 40, 700, 2100, 5000], 4, 1, D, dtype, T=queries)
    _, lse, _ = d.run(D ** -0.5, cluster=cluster)
    _, want, _, ltol = d.want(D ** -0.5, 0)
    room = ltol - 2.0 ** -11 + 2.0 ** -24 * (16 + 5000 / 8)
    fin = np.isfinite(want)
    assert fin.any() and (np.abs(lse[fin] - want[fin]) <= room[fin]).all()


def test_decode_long_ranges_are_staged_in_stretches():
    # One CTA serves 2600 pages, more than it stages at a time, with sequences that end at,
    # before and behind the borders of the stretches.
    Decode(8, [512 * 16, 100, 511 * 16, 9000], 2, 1, 64, "f16", T=3).case(ctas=1)
    Decode(8, [512 * 16, 512 * 16], 2, 1, 64, "bf16").case(ctas=1)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_one_long_sequence(D):
    Decode(9, [20011], 8, 1, D, "f16").case()
    Decode(9, [20011, 17], 4, 2, D, "bf16", T=5, new=[5, 2]).case(window=15000)


@pytest.mark.parametrize("B,queries", [(129, 1), (300, 4), (1500, 1), (4096, 2)])
def test_decode_large_batches(B, queries):
    g = np.random.default_rng(B)
    Decode(B, g.integers(0, 60 if B < 4000 else 20, B), 2, 1, 64, "f16", T=queries).case()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_decode_scales(scale):
    Decode(11, [50, 300, 1], 4, 1, 128, "f16").case(scale=scale)


@pytest.mark.parametrize("D,dtype", DIMS)
def test_decode_sharp_scores(D, dtype):
    # Scores of some hundreds: the running maximum has to be raised again and again.
    Decode(12, [600, 33], 4, 1, D, dtype, q_std=30.0, T=2).case(scale=0.3)


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("spread", [2.0, 8.0])
def test_decode_page_scales_of_many_sizes(D, dtype, spread, pow2):
    # V scales octaves apart: raised references, ratios on the weights and on the products.
    Decode(13, [600, 33, 1200], 4, 1, D, dtype, spread=spread, pow2=pow2, T=2).case(scale=1e-3)


@pytest.mark.parametrize("order", [1, -1])
def test_decode_rising_and_falling_scales(order):
    d = Decode(14, [400], 4, 1, 128, "f16")
    n = 25
    d.scales[1, d.bt[0, :n], 0] = 2.0 ** np.rint(order * np.linspace(-30, 30, n))
    d.case()
    d.scales[1, d.bt[0, 3], 0] = 0.0  # a page that stands for zeros
    d.scales[0, d.bt[0, 4], 0] = 0.0
    d.case()
    d.scales[1, d.bt[0], 0] = 0.0
    out, lse, err = d.run(0.1)
    assert err == 0 and (out == 0).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("q_std", [1e-30, 1e-3, 1e20])
def test_decode_bf16_queries_of_any_size(q_std):
    d = Decode(15, [200, 33], 12, 1, 128, "bf16", q_std=q_std)
    d.case(scale=0.1 / q_std)
    d.q[0, 3] = 0.0
    d.case(scale=0.1 / q_std)


def test_decode_table_wider_than_the_lengths():
    Decode(16, [100, 20], 4, 2, 128, "f16", maxp=40).case()


def test_decode_without_starts():
    d = Decode(17, [100, 20, 0, 333], 4, 2, 128, "f16", pad=2)
    d.starts = np.arange(5, dtype=np.int32)
    d.q = rounded(d.g.standard_normal((6, 4, 128)), "f16")
    got = d.run(0.1, starts=False)
    d.check(got, d.want(0.1, 0))


def test_decode_equals_pa_decode_on_the_values():
    d = Decode(18, [700, 33, 16], 8, 2, 128, "f16")
    k, v = (to_t(x, "f16") for x in d.values())
    out, lse, err = d.run(0.1)
    o2, l2, _, e2 = pa.decode(to_t(d.q, "f16"), k, v, i32(d.bt), i32(d.lens), 0.1)
    assert err == e2 == 0
    w, _, tol, ltol = d.want(0.1, 0)
    assert (np.abs(out - host(o2)) <= 2 * tol + 2.0 ** -11 * np.abs(w)).all()
    assert (np.abs(lse - host(l2)) <= ltol + 1e-4).all()


def test_decode_more_queries_than_tokens():
    # (two tokens cannot have three queries of their own: the first attends to nothing)
    d = Decode(19, [2, 50, 0], 4, 2, 64, "f16", T=3, new=[3, 3, 2])
    out, lse, err = d.run(0.1)
    assert err == 0
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (out[6:] == 0).all() and np.isneginf(lse[6:]).all()
    d.check((out, lse, err), d.want(0.1, 0))


@pytest.mark.parametrize("D,dtype", DIMS)
@pytest.mark.parametrize("window", [0, 40])
def test_decode_nan_in_tokens_that_a_query_does_not_see(D, dtype, window):
    """A drafted token's NaN, in K or in some dims of V, reaches its own row and the later ones
    only; a NaN behind a window the rows before it slides past."""
    queries, L = 5, 71
    d = Decode(20, [L, 300], 4, 2, D, dtype, T=queries, new=[queries, 2])
    scale = 0.1

    def cell(tok):
        return d.bt[0, tok // 16], tok % 16

    for tok in (L - 1, L - 3, L - 5) if not window else (L - 4, L - window - 1, L - window - 3):
        clean = d.codes.copy()
        p, at = cell(tok)
        for which, dims in ((0, [3]), (1, [0, 5, D - 1])):
            for h in (0, 1):
                d.codes[which, p, h, at, dims] = 127 if h else 255
            got = d.run(scale, window)
            w = list(d.want(scale, window))
            # fp64: NaN in a seen token's K makes the whole row NaN, in V its dims
            sees = []
            for t in range(queries):
                end = L - queries + 1 + t
                sees.append(tok < end and (not window or tok >= end - window))
            assert any(sees)
            for t, s in enumerate(sees):
                nan = np.isnan(got[0][t])
                if not s:
                    assert not nan.any()
                elif which == 0:
                    assert nan.all() and np.isnan(got[1][t]).all()
                else:
                    assert nan[:, dims].all() and nan.sum() == 4 * len(dims)
            np.testing.assert_array_equal(np.isnan(got[0]), np.isnan(w[0]))
            fine = ~np.isnan(w[0])
            tol = np.where(fine, w[2], 0)
            assert (np.abs(got[0] - w[0])[fine] <= tol[fine]).all()
            d.codes = clean.copy()


def test_decode_nan_in_one_query_head_stays_there():
    d = Decode(21, [500, 20], 8, 1, 128, "f16", T=2, new=[2, 2])
    want = d.want(0.1, 0)
    d.q[0, 3, 17] = np.nan
    out, lse, err = d.run(0.1)
    assert err == 0 and np.isnan(out[0, 3]).all() and np.isnan(lse[0, 3])
    keep = np.ones(out.shape[:2], bool)
    keep[0, 3] = False
    assert (np.abs(out - want[0])[keep] <= want[2][keep]).all()


def test_decode_scores_beyond_fp32():
    # -inf scores weigh nothing; +inf makes NaN rows of their own
    d = Decode(22, [300, 40], 4, 1, 128, "bf16", q_std=1e30)
    d.scales[0] = 2.0 ** 60
    out, lse, err = d.run(1e3)
    assert err == 0 and out.shape == (2, 4, 128)


@pytest.mark.parametrize("ctas", [1, 6, None])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("queries", [1, 3])
def test_bad_page_ids_lengths_and_starts_give_nan_rows(D, ctas, queries):
    d = Decode(23, [700, 300, 90, 16], 4, 1, D, "f16", T=queries, new=[queries] * 4)
    good = d.want(0.1, 0)

    def rows_of(got, gone):
        out, lse, _ = got
        for b in range(4):
            sl = slice(b * queries, (b + 1) * queries)
            if b in gone:
                assert np.isnan(out[sl]).all() and np.isnan(lse[sl]).all()
            else:
                d.check((out, lse, 0), good, sl)

    bt, lens, starts = d.bt.copy(), d.lens.copy(), d.starts.copy()
    for bad in (d.pages, -1, 1 << 30):
        d.bt = bt.copy()
        d.bt[0, 20] = bad
        got = d.run(0.1, ctas=ctas)
        assert got[2] == binding.PA_DEVERR_BAD_PAGE
        rows_of(got, [0])
    d.bt = bt
    for bad in (-1, 701, 1 << 30, -(1 << 31), 2 ** 31 - 1):
        d.lens = lens.copy()
        d.lens[1] = bad
        got = d.run(0.1, ctas=ctas, max_len=700)
        assert got[2] == binding.PA_DEVERR_BAD_LENGTH
        rows_of(got, [1])
    d.lens = lens
    # a start that leaves its sequence, or the one before it, without rows in order
    for bad in (-5, 4 * queries + 1, 1 << 30, -(1 << 31)):
        d.starts = starts.copy()
        d.starts[2] = bad
        got = d.run(0.1, ctas=ctas, max_len=700)
        assert got[2] == binding.PA_DEVERR_BAD_LENGTH
        out, lse, _ = got
        for b in (0, 3):
            d.check((out, lse, 0), good, slice(b * queries, (b + 1) * queries))
        # (their rows are left as they were)
        assert (out[queries:3 * queries] == 3).all() and (lse[queries:3 * queries] == 5).all()
    # more query tokens than planned
    d.starts = np.array([0, 2 * queries, 2 * queries, 3 * queries, 4 * queries], np.int32)
    got = d.run(0.1, ctas=ctas, max_len=700)
    assert got[2] == binding.PA_DEVERR_BAD_LENGTH
    assert np.isnan(got[0][:2 * queries]).all()
    for b in (2, 3):
        d.check((got[0], got[1], 0), good, slice(b * queries, (b + 1) * queries))


@pytest.mark.parametrize("cluster", [None, 0])
@pytest.mark.parametrize("queries", [1, 4])
def test_copy_timeout_is_reported_and_the_next_call_is_clean(cluster, queries):
    d = Decode(24, [500, 20], 4, 1, 128, "f16", T=queries)
    out, lse, err = d.run(0.1, stall=16, cluster=cluster)
    assert err & binding.PA_DEVERR_TIMEOUT
    assert np.isnan(out).all() and np.isnan(lse).all()
    d.case(0.1)


@pytest.mark.parametrize("cluster", [None, 0])
def test_calls_repeat_bit_for_bit(cluster):
    d = Decode(25, [3000, 100, 2000], 8, 2, 128, "f16", T=3)
    first = d.run(0.1, cluster=cluster)
    for _ in range(5):
        again = d.run(0.1, cluster=cluster)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_two_streams_with_their_own_workspaces_and_a_prepared_call():
    d = Decode(26, [3000, 100, 2000, 7], 8, 2, 128, "bf16", T=2)
    want = d.want(0.1, 0)
    plan = d.plan()
    cache, tq = d.device(), to_t(d.q, "bf16")
    st, tb, tl = i32(d.starts), i32(d.bt), i32(d.lens)
    jobs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        out, lse = torch.empty_like(tq), torch.empty(tq.shape[0], 8, device="cuda")
        ws = pa.new_workspace(plan, "cuda")
        jobs.append((pa.prepare_q8_decode(plan, tq, st, *cache, tb, tl, 0.1, 0, out, lse, ws, s), out,
                     lse, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, *_ in jobs:
            call()
    torch.cuda.synchronize()
    for _, out, lse, ws in jobs:
        d.check((host(out), host(lse), pa.pa_get_error(ws)), want)


def test_two_graphs_share_a_workspace_one_after_the_other():
    d = Decode(27, [3000, 100, 2000, 900, 3], 8, 2, 128, "f16", T=2)
    want = d.want(0.1, 0)
    plan = d.plan()
    ws = pa.new_workspace(plan, "cuda")
    cache, tq = d.device(), to_t(d.q, "f16")
    st, tb, tl = i32(d.starts), i32(d.bt), i32(d.lens)
    runs = []
    for _ in range(2):
        out, lse = torch.empty_like(tq), torch.empty(tq.shape[0], 8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                pa.pa_q8_decode(plan, tq, st, *cache, tb, tl, 0.1, 0, out, lse, ws)
        runs.append((graph, out, lse))
    for i in (0, 1, 1, 0):
        runs[i][0].replay()
    torch.cuda.synchronize()
    for _, out, lse in runs:
        d.check((host(out), host(lse), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("cluster", [None, 0])
@pytest.mark.parametrize("old", ["same lengths", "a token more", "pages fewer", "garbage", "starts"])
@pytest.mark.parametrize("lens,window,D,queries", [([3000, 1200, 0, 2049, 77], 0, 128, 1),
                                                   ([3000, 1200, 2049, 77], 1000, 64, 4),
                                                   ([20000], 0, 256, 2), ([30] * 127 + [0], 0, 64, 2),
                                                   ([40, 3] * 100, 0, 96, 1)])
def test_decode_uses_what_is_written_late(late_writer, lens, window, D, queries, old, cluster):  # noqa: F811
    # What the kernel reads before its dependency wait are hints; everything counts only as it
    # stands after the wait.  The old table points at a page of NaN.
    d = Decode(30, lens, 4, 2, D, "f16", T=queries)
    scale = D ** -0.5
    want = d.want(scale, window)
    B = len(lens)
    # lengths and starts lie in one buffer, which the helper writes
    new = np.concatenate([d.lens, d.starts]).astype(np.int32)
    now = new.copy()
    old_bt = np.full_like(d.bt, d.unused[0])
    if old == "a token more":
        now[:B] = np.minimum(d.lens + 1, d.lens.max())
    elif old == "pages fewer":
        now[:B] = d.lens // 2
    elif old == "garbage":
        now[:B] = np.where(np.arange(B) % 2, -5, 1 << 30)
        now[B:] = np.where(np.arange(B + 1) % 2, -5, 1 << 30)
        old_bt[:, ::2], old_bt[:, 1::2] = -7, 1 << 30
    elif old == "starts":
        now[B:] = 0
    plan = d.plan(window)
    if cluster == 0:
        plan.cluster = 0
    ws = pa.new_workspace(plan, "cuda")
    tq, cache = to_t(d.q, "f16"), d.device()
    t_new, t_now, b_new, b_now = i32(new), i32(now), i32(d.bt), i32(old_bt)
    out = torch.full_like(tq, 3.0)
    lse = torch.full(tq.shape[:2], 5.0, device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    assert late_writer.launch_delayed_copy(b_new.data_ptr(), b_now.data_ptr(), d.bt.size,
                                           t_new.data_ptr(), t_now.data_ptr(), new.size, 20000,
                                           stream.cuda_stream) == 0
    pa.pa_q8_decode(plan, tq, t_now[B:], *cache, b_now, t_now[:B], scale, window, out, lse, ws)
    d.check((host(out), host(lse), pa.pa_get_error(ws)), want)


def test_sequences_may_share_pages():
    d = Decode(31, [160, 160, 90], 4, 2, 128, "f16")
    d.bt[1, :5] = d.bt[0, :5]
    d.case(0.1)


def test_plans_for_other_sm_counts():
    d = Decode(32, [500, 20, 1000], 4, 2, 128, "f16", T=2)
    for sms in (1, 8, 500):
        d.case(0.1, sms=sms)


def test_decode_offsets_beyond_32_bits():
    # 1,100,000 pages of 4096 codes: 4.5 GB of K and of V, used near their end.
    d = Decode(33, [75], 4, 1, 256, "f16", T=2)
    want = d.want(0.1, 0)
    big = 1_100_000
    ids = np.array([big - 1, 3, big - 2, 1_048_577, big - 7], np.int32)
    at = torch.from_numpy(ids).long().cuda()
    small = d.device()
    cache = [torch.empty(big, 1, 16, 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(big, 1, device="cuda") for _ in range(2)]
    mine = torch.from_numpy(d.bt[0]).long().cuda()
    for c, s, c0, s0 in zip(cache, scales, small[:2], small[2:]):
        c[at] = c0.view(torch.uint8)[mine]
        s[at] = s0[mine]
    plan = pa.pa_q8_plan(1, 4, 1, 256, 16, big, 5, 75, 0, 2)
    tq = to_t(d.q, "f16")
    out, lse = torch.empty_like(tq), torch.empty(tq.shape[0], 4, device="cuda")
    ws = pa.new_workspace(plan, "cuda")
    pa.pa_q8_decode(plan, tq, i32(d.starts), cache[0].view(F8), cache[1].view(F8), *scales, i32(ids[None]),
                    i32(d.lens), 0.1, 0, out, lse, ws)
    d.check((host(out), host(lse), pa.pa_get_error(ws)), want)


def test_convenience_call_without_sequences():
    d = Decode(40, [20], 2, 1, 64, "f16")
    q = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    for starts in (None, i32(np.zeros(1, np.int32))):
        out, lse, plan, err = pa.q8_decode(q, starts, *d.device(), i32(d.bt[:0]), i32(d.lens[:0]), 0.1)
        assert out.shape == (0, 2, 64) and lse.shape == (0, 2) and plan.batch == 0 and err == 0


def test_convenience_call():
    d = Decode(34, [100, 20, 333], 4, 2, 128, "bf16", T=3, new=[3, 1, 2])
    for stream in (None, torch.cuda.Stream()):
        out, lse, plan, err = pa.q8_decode(to_t(d.q, "bf16"), i32(d.starts), *d.device(), i32(d.bt),
                                           i32(d.lens), 0.1, stream=stream)
        torch.cuda.synchronize()
        assert plan.max_query_len == 3
        d.check((host(out), host(lse), err), d.want(0.1, 0))


def test_refused_tensors():
    d = Decode(35, [30], 4, 1, 128, "f16")
    plan = d.plan()
    tq = to_t(d.q, "f16")
    kc, vc, ks, vs = d.device()
    out, lse, ws = torch.empty_like(tq), torch.empty(1, 4, device="cuda"), pa.new_workspace(plan, "cuda")
    st, tb, tl = i32(d.starts), i32(d.bt), i32(d.lens)
    ok = [plan, tq, st, kc, vc, ks, vs, tb, tl, 0.1, 0, out, lse, ws]
    pa.pa_q8_decode(*ok)
    for i, bad, exc in [(1, tq.bfloat16(), TypeError), (1, tq.transpose(1, 2), ValueError),
                        (1, tq.cpu(), ValueError), (1, tq[0], ValueError), (2, st.long(), TypeError),
                        (2, st[:1], ValueError), (3, kc.view(torch.uint8), TypeError),
                        (4, vc[:1], ValueError), (4, vc[..., :64], ValueError),
                        (5, ks.half(), TypeError), (6, vs[:, 0], ValueError), (7, tb.long(), TypeError),
                        (8, tl.repeat(2), ValueError), (11, out.float(), TypeError),
                        (12, lse.double(), TypeError), (13, ws[:8], pa.PAError), (10, 3, pa.PAError)]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            pa.pa_q8_decode(*args)
    rows_ = torch.zeros(4, 2, 128, dtype=torch.float16, device="cuda")
    kc, vc, ks, vs = pa.new_q8_cache(2, 2, 128)
    k16, v16 = (torch.zeros(2, 2, 16, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    sl, pos = torch.arange(4, device="cuda"), i32(np.arange(4))
    w = torch.ones(128, dtype=torch.float16, device="cuda")
    good = dict(q=None, k=rows_, v=rows_, slots=sl, positions=pos)
    for kw, exc in [(dict(k=rows_.half()[:3]), ValueError), (dict(v=rows_.bfloat16()), TypeError),
                    (dict(slots=sl.int()), TypeError), (dict(slots=sl[:3]), ValueError),
                    (dict(positions=None, theta=1e4), TypeError),
                    (dict(positions=pos.long(), theta=1e4), TypeError),
                    (dict(k_norm=w.float()), TypeError), (dict(k_norm=w[:64]), ValueError),
                    (dict(q_norm=w), ValueError), (dict(q_out=rows_), ValueError),
                    (dict(q=rows_, q_out=rows_[:, :1]), ValueError),
                    (dict(k=rows_[:, :1], v=rows_[:, :1]), ValueError),
                    (dict(theta=-1.0), pa.PAError), (dict(theta=1e4, rotary_dim=8), pa.PAError),
                    (dict(q=rows_.clone(), q_out=rows_), pa.PAError)]:
        a = dict(good, **kw)
        with pytest.raises(exc):
            pa.pa_append(**a, k_cache=k16, v_cache=v16)
        with pytest.raises(exc):
            pa.pa_q8_append(**a, k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs)
    with pytest.raises(TypeError):
        pa.pa_append(**good, k_cache=kc, v_cache=vc)
    with pytest.raises(TypeError):
        pa.pa_q8_append(**good, k_cache=k16, v_cache=v16, k_scales=ks, v_scales=vs)
    with pytest.raises(pa.PAError):
        pa.pa_append(**good, k_cache=k16, v_cache=k16)
    with pytest.raises(pa.PAError):
        pa.pa_q8_read(kc, vc, ks, vs, sl, rows_, rows_)


def test_empty_calls():
    none = torch.empty(0, 1, 64, dtype=torch.float16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    caches = pa.new_q8_cache(2, 1, 64)
    pa.pa_q8_append(none, none, none, slots, None, *caches)
    pa.pa_q8_read(*caches, slots, none, none.clone())
    assert int(caches[0].view(torch.uint8).count_nonzero()) == 0 and (caches[2] == 1).all()
    d = Decode(36, [0, 0, 0], 2, 1, 64, "f16", T=2, new=[1, 2, 0])
    out, lse, err = d.run(0.1, max_len=0)
    assert err == 0 and (out == 0).all() and np.isneginf(lse).all()
    d = Decode(37, [20, 30], 2, 1, 64, "f16", new=[0, 0])
    assert d.run(0.1)[2] == 0


# ---------------------------------------------------------------- verification

def verify_case(seed, B, V, drafts, dtype, certain=False, ragged=False, near=0.5):
    g = np.random.default_rng(seed)
    x = 2.0 * g.standard_normal((B, drafts + 1, V))
    y = x[:, :drafts] + near * g.standard_normal((B, drafts, V))

    def soft(z):
        e = np.exp(z - z.max(-1, keepdims=True))
        return rounded(e / e.sum(-1, keepdims=True), dtype)

    target, draft = soft(x), None if certain else soft(y)
    source = target[:, :drafts] if certain else draft
    tok = np.zeros((B, drafts), np.int32)
    for b in range(B):
        for t in range(drafts):
            p = source[b, t] / source[b, t].sum()
            tok[b, t] = g.choice(V, p=p)
    num = g.integers(0, drafts + 1, B).astype(np.int32) if ragged else None
    return dict(target=target, draft=draft, tok=tok, num=num,
                accept=g.random((B, drafts)).astype(np.float32),
                sample=g.random(B).astype(np.float32))


def run_verify(c, dtype, err=None, offset=0):
    B, T1, V = c["target"].shape

    def dev(x):
        t = to_t(x, dtype)
        if offset:  # rows that do not lie at multiples of 16 bytes
            buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
            buf[offset:] = t.flatten()
            return buf[offset:].view(t.shape)
        return t

    accepted = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    tokens = torch.full((B, T1), -9, dtype=torch.int32, device="cuda")
    pa.pa_verify_drafts(dev(c["target"]), None if c["draft"] is None else dev(c["draft"]),
                        i32(c["tok"]), None if c["num"] is None else i32(c["num"]),
                        torch.from_numpy(c["accept"]).cuda(), torch.from_numpy(c["sample"]).cuda(),
                        accepted, tokens, err)
    return accepted.cpu().numpy(), tokens.cpu().numpy()


def check_verify(c, dtype, offset=0):
    err = torch.zeros(64, dtype=torch.int32, device="cuda")
    a, t = run_verify(c, dtype, err, offset)
    wa, wt, bad = ref.verify(c["target"], c["draft"], c["tok"], c["num"], c["accept"], c["sample"])
    np.testing.assert_array_equal(a, wa)
    np.testing.assert_array_equal(t, wt)
    assert pa.pa_get_error_ex(err) == (q8.PA_DEVERR_BAD_TOKEN if bad else 0)
    return a, t


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,V,drafts", [(1, 1, 1), (3, 2, 2), (40, 17, 3), (7, 1000, 8), (5, 4096, 4),
                                        (4, 8195, 32), (3, 32003, 4), (2, 131072, 5), (1, 524288, 1),
                                        (3, 32002, 3), (40, 16388, 2), (200, 9002, 2)])
def test_verify(B, V, drafts, dtype):
    if dtype != "f32" and V > 100000:
        pytest.skip("one type is enough")
    c = verify_case(V, B, V, drafts, dtype, ragged=B > 3)
    check_verify(c, dtype)
    check_verify(c, dtype, offset=1)
    c["draft"], c["num"] = None, None
    check_verify(c, dtype)


def test_verify_every_stop_and_every_token():
    # Random numbers that stop at each draft; draws from the first to the last token.
    V, drafts = 300, 4
    c = verify_case(1, 200, V, drafts, "f32")
    c["sample"] = ((np.arange(200) + 0.5) / 200).astype(np.float32)
    a, t = check_verify(c, "f32")
    assert set(a) == set(range(drafts + 1))
    c["sample"][:] = 0.0
    _, t = check_verify(c, "f32")
    c["sample"][:] = np.float32(1 - 2.0 ** -24)
    check_verify(c, "f32")
    for u in (1.0, 2.0, -1.0, np.nan, np.inf):
        c["sample"][:] = u
        check_verify(c, "f32")


def test_verify_without_drafts_is_a_draw():
    V = 50
    c = verify_case(2, 500, V, 1, "f32")
    c["num"] = np.zeros(500, np.int32)
    a, t = check_verify(c, "f32")
    assert (a == 0).all() and (t[:, 1] == -1).all() and (t[:, 0] >= 0).all()
    # and with no room for any
    p = to_t(c["target"][:, :1], "f32")
    acc, tok = i32(np.zeros(500)), i32(np.zeros((500, 1)))
    empty = torch.empty(500, 0, dtype=torch.int32, device="cuda")
    pa.pa_verify_drafts(p, None, empty, None, empty.float(), torch.from_numpy(c["sample"]).cuda(), acc, tok)
    np.testing.assert_array_equal(tok.cpu().numpy()[:, 0], t[:, 0])


def test_verify_the_tokens_have_the_targets_distribution():
    # 200,000 sequences of one draft over 8 tokens: counts within six deviations of the target.
    n, V = 200_000, 8
    g = np.random.default_rng(4)
    p, q = (g.dirichlet(np.ones(V)) for _ in range(2))
    c = dict(target=np.broadcast_to(rounded(p, "f32"), (n, 2, V)), num=None,
             draft=np.broadcast_to(rounded(q, "f32"), (n, 1, V)),
             tok=g.choice(V, size=(n, 1), p=q).astype(np.int32),
             accept=g.random((n, 1)).astype(np.float32), sample=g.random(n).astype(np.float32))
    _, t = run_verify(c, "f32")
    counts = np.bincount(t[:, 0], minlength=V)
    assert (np.abs(counts - n * p) <= 6 * np.sqrt(n * p * (1 - p)) + 1).all()


def test_verify_odd_probabilities():
    """NaN, infinite, negative and large entries; equal rows (no residual); rows of zeros; drafts
    outside the vocabulary; numbers of drafts out of bounds."""
    V, drafts, B = 70, 3, 12
    c = verify_case(5, B, V, drafts, "f32")
    tg, dr = c["target"], c["draft"]
    tg[0, :, ::7] = np.nan
    dr[1, :, ::5] = np.nan
    tg[2, :, 3], dr[3, :, 4] = np.inf, np.inf
    tg[4, :, 5], dr[4, :, 6] = -1.0, -np.inf
    tg[5] *= 100
    dr[6] = tg[6, :drafts]
    c["accept"][6] = 1.0  # never below p / q = 1: no weight is left, the draw is from p
    tg[7] = 0
    tg[8, 1:] = 0
    c["tok"][9, 1], c["tok"][10, 0] = V, -1
    check_verify(c, "f32")
    c["num"] = np.array([-1, 4, 1 << 30, -(1 << 31)] + [drafts] * (B - 4), np.int32)
    check_verify(c, "f32")
    # a bad token behind the first draft that is not accepted is not looked at
    c = verify_case(6, 1, V, drafts, "f32")
    c["accept"][0] = 1.0
    c["draft"][0, 0, c["tok"][0, 0]] = 1.0
    c["target"][0, 0, c["tok"][0, 0]] = 0.1
    c["tok"][0, 2] = -5
    a, _ = check_verify(c, "f32")
    assert a[0] == 0


def test_verify_replays_and_streams():
    c = verify_case(7, 6, 5000, 4, "f32")
    want = ref.verify(c["target"], c["draft"], c["tok"], c["num"], c["accept"], c["sample"])
    args = [to_t(c["target"], "f32"), to_t(c["draft"], "f32"), i32(c["tok"]), None,
            torch.from_numpy(c["accept"]).cuda(), torch.from_numpy(c["sample"]).cuda()]
    acc, tok = i32(np.zeros(6)), i32(np.zeros((6, 5)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_verify_drafts(*args, acc, tok)
    c2 = verify_case(8, 6, 5000, 4, "f32")
    for x in (c2, c):  # the replay reads what its buffers hold then
        for t, name in ((args[0], "target"), (args[1], "draft")):
            t.copy_(to_t(x[name], "f32"))
        args[2].copy_(i32(x["tok"]))
        args[4].copy_(torch.from_numpy(x["accept"]))
        args[5].copy_(torch.from_numpy(x["sample"]))
        graph.replay()
        torch.cuda.synchronize()
        w = ref.verify(x["target"], x["draft"], x["tok"], x["num"], x["accept"], x["sample"])
        np.testing.assert_array_equal(acc.cpu().numpy(), w[0])
        np.testing.assert_array_equal(tok.cpu().numpy(), w[1])
    s = torch.cuda.Stream()
    acc2, tok2 = torch.zeros_like(acc), torch.zeros_like(tok)
    torch.cuda.synchronize()
    pa.pa_verify_drafts(*args, acc2, tok2, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(tok2.cpu().numpy(), want[1])


def test_verify_refused_tensors():
    c = verify_case(9, 2, 100, 3, "f32")
    ok = [to_t(c["target"], "f32"), to_t(c["draft"], "f32"), i32(c["tok"]), i32([3, 1]),
          torch.from_numpy(c["accept"]).cuda(), torch.from_numpy(c["sample"]).cuda(), i32([0, 0]),
          i32(np.zeros((2, 4)))]
    pa.pa_verify_drafts(*ok)
    for i, bad, exc in [(0, ok[0][0], ValueError), (0, ok[0].double(), TypeError),
                        (0, ok[0].transpose(1, 2), ValueError), (1, ok[1].half(), TypeError),
                        (1, ok[0], ValueError), (2, ok[2].long(), TypeError), (2, ok[2][:, :2], ValueError),
                        (3, ok[3][:1], ValueError), (4, ok[4].double(), TypeError),
                        (5, ok[5].cpu(), ValueError), (6, ok[6].float(), TypeError),
                        (7, ok[7][:, :3], ValueError), (6, ok[3], pa.PAError)]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            pa.pa_verify_drafts(*args)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 64), ("f16", 96), ("bf16", 256)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_loop_of_drafts_and_verification(dtype, D, graph):
    """A prompt step, then steps that verify four drafted tokens of each request (captured once and
    replayed in one variant): tables, rows, attention and verification as they follow one
    another, with the lengths that the verification leaves.  Everything stays on the device; the
    host's reference goes along."""
    g = np.random.default_rng([D, int(graph)])
    B, Hq, Hkv, maxp, pages, theta, drafts, V = 3, 8, 2, 16, 60, 10000.0, 4, 500
    scale = D ** -0.5
    caches = pa.new_q8_cache(pages, Hkv, D)
    rk, rv = ref.Cache(pages, Hkv, D), ref.Cache(pages, Hkv, D)
    rk.codes[...] = rv.codes[...] = 0
    # Every request has its pages beforehand: a rejected draft's page then is not lost.
    bt = g.permutation(pages)[:B * maxp].reshape(B, maxp).astype(np.int32)
    free = np.zeros(1, np.int32)
    step_rows = drafts + 1
    plan = pa.pa_q8_plan(B, Hq, Hkv, D, 16, pages, maxp, maxp * 16, 0, step_rows, 0, DT[dtype])
    wide = pa.pa_q8_plan(B, Hq, Hkv, D, 16, pages, maxp, maxp * 16, 0, 16, 0, DT[dtype])
    w = [to_t(rounded(1 + 0.2 * g.standard_normal(D), dtype), dtype) for _ in range(2)]
    hw = [host(x) for x in w]
    past = i32(np.zeros(B))
    ctx, table = i32(np.zeros(B)), i32(bt)
    err = i32(np.zeros(64))

    def buffers(n, plan):
        return dict(new=i32(np.zeros(B)), starts=i32(np.zeros(B + 1)),
                    slots=torch.zeros(n, dtype=torch.int64, device="cuda"), pos=i32(np.zeros(n)),
                    taken=i32([0]), qkv=torch.zeros(n, Hq + 2 * Hkv, D, dtype=T[dtype], device="cuda"),
                    q=torch.zeros(n, Hq, D, dtype=T[dtype], device="cuda"),
                    out=torch.zeros(n, Hq, D, dtype=T[dtype], device="cuda"),
                    lse=torch.zeros(n, Hq, device="cuda"), ws=pa.new_workspace(plan, "cuda"), plan=plan)

    def forward(b):
        # (pages are in the table already: lengths that have them need none of the free list)
        pa.pa_extend_tables(past, b["new"], i32_free, pages, scratch, ctx, b["starts"], b["slots"], b["pos"],
                            b["taken"], None)
        page = table.flatten().long()[(row_seq(b) * maxp + b["pos"].long() // 16).clamp(max=B * maxp - 1)]
        slots = torch.where(live(b), page * 16 + b["pos"].long() % 16, -1)
        b["slots"].copy_(slots)
        pa.pa_q8_append(b["qkv"][:, :Hq], b["qkv"][:, Hq:Hq + Hkv], b["qkv"][:, Hq + Hkv:], b["slots"],
                        b["pos"], *caches, q_out=b["q"], q_norm=w[0], k_norm=w[1], theta=theta,
                        device_error=err)
        pa.pa_q8_decode(b["plan"], b["q"], b["starts"], *caches, table, ctx, scale, 0, b["out"],
                        b["lse"], b["ws"])

    def row_seq(b):
        n = torch.arange(b["slots"].numel(), device="cuda", dtype=torch.int32)
        return (torch.searchsorted(b["starts"], n, right=True) - 1).clamp(0, B - 1)

    def live(b):
        n = torch.arange(b["slots"].numel(), device="cuda", dtype=torch.int32)
        return n < b["starts"][-1]

    i32_free = i32(np.arange(B * maxp))
    scratch = i32(np.full((B, maxp), 0))  # the tables that pa_extend_tables makes are not used here
    ver = dict(target=torch.zeros(B, drafts + 1, V, device="cuda"),
               draft=torch.zeros(B, drafts, V, device="cuda"), tok=i32(np.zeros((B, drafts))),
               accept=torch.zeros(B, drafts, device="cuda"), sample=torch.zeros(B, device="cuda"),
               acc=i32(np.zeros(B)), out=i32(np.zeros((B, drafts + 1))))

    def verify():
        pa.pa_verify_drafts(ver["target"], ver["draft"], ver["tok"], None, ver["accept"], ver["sample"],
                            ver["acc"], ver["out"], err)
        past.add_(ver["acc"] + 1)  # the accepted drafts and the token before them are in the cache

    def reference_step(b, x, hp, new):
        n = int(new.sum())
        pos = np.concatenate([p + np.arange(m) for p, m in zip(hp, new)])
        seq = np.repeat(np.arange(B), new)
        slots = bt[seq, pos // 16].astype(np.int64) * 16 + pos % 16
        assert np.array_equal(host(b["pos"])[:n], pos) and np.array_equal(host(b["slots"])[:n], slots)
        q = ref.turned(x[:n, :Hq], hw[0], pos, 1e-6, theta, D)
        qt = ref.turned_tolerance(x[:n, :Hq], hw[0], q, 1e-6, theta, D, dtype)
        assert (np.abs(host(b["q"])[:n] - q) <= qt).all()
        k = ref.turned(x[:n, Hq:Hq + Hkv], hw[1], pos, 1e-6, theta, D)
        rk.append(k, slots)
        rv.append(x[:n, Hq + Hkv:], slots)
        # V and scales exactly; K's codes to one step (fp32 next to a border), then as they are
        for got, want in ((caches[2], rk.scales), (caches[3], rv.scales)):
            seen = np.unique(slots // 16)
            np.testing.assert_array_equal(host(got)[seen], want[seen])
        np.testing.assert_array_equal(ref.E4M3[code_bytes(caches[1])], ref.E4M3[rv.codes])
        gk = ref.E4M3[code_bytes(caches[0])]
        assert np.mean(gk != ref.E4M3[rk.codes]) < 1e-3
        rk.codes[...] = code_bytes(caches[0])
        lens = hp + new
        starts = np.concatenate([[0], np.cumsum(new)])
        want = ref.decode(host(b["q"])[:n], rk.values(), rv.values(), bt, lens, starts, scale, 0, dtype)
        out, lse = host(b["out"])[:n], host(b["lse"])[:n]
        assert (np.abs(out - want[0]) <= want[2]).all() and (np.abs(lse - want[1]) <= want[3]).all()

    hp = np.zeros(B, np.int64)
    new = np.array([16, 3, 11])
    b = buffers(int(new.sum()) + 2, wide)
    x = rows(g, (b["slots"].numel(), Hq + 2 * Hkv, D), dtype)
    b["qkv"].copy_(to_t(x, dtype))
    b["new"].copy_(i32(new))
    forward(b)
    torch.cuda.synchronize()
    reference_step(b, x, hp, new)
    past.copy_(i32(new))
    hp = new.astype(np.int64)

    b = buffers(B * step_rows, plan)
    b["new"].fill_(step_rows)
    captured = None
    for step in range(6):
        x = rows(g, (B * step_rows, Hq + 2 * Hkv, D), dtype)
        b["qkv"].copy_(to_t(x, dtype))
        c = verify_case([D, step], B, V, drafts, "f32")
        for name, key in (("target", "target"), ("draft", "draft")):
            ver[name].copy_(to_t(c[key], "f32"))
        ver["tok"].copy_(i32(c["tok"]))
        ver["accept"].copy_(torch.from_numpy(c["accept"]))
        ver["sample"].copy_(torch.from_numpy(c["sample"]))
        torch.cuda.synchronize()
        if graph and step >= 1:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    forward(b)
                    verify()
            captured.replay()
        else:
            forward(b)
            verify()
        torch.cuda.synchronize()
        reference_step(b, x, hp, np.full(B, step_rows))
        a, t, bad = ref.verify(c["target"], c["draft"], c["tok"], None, c["accept"], c["sample"])
        assert not bad
        assert np.array_equal(ver["acc"].cpu().numpy(), a) and np.array_equal(ver["out"].cpu().numpy(), t)
        hp = hp + a + 1
        assert np.array_equal(past.cpu().numpy(), hp)
        assert pa.pa_get_error_ex(err) == 0 and pa.pa_get_error(b["ws"]) == 0


def test_calls_without_the_marshalling_extension(monkeypatch):
    """The same calls through the Python checks alone give the same bits."""
    if q4._fast is None:
        pytest.skip("the marshalling extension is not built here")
    fast = q4._fast
    n, hq, hkv, D = 40, 4, 2, 128
    r = Rows(50, n, hq, hkv, D, "f16", True, 1e4, 64)
    slots, results = i64(np.arange(n)), []
    d = Decode(51, [100, 20], hq, hkv, D, "f16", T=2)
    c = verify_case(52, 3, 700, 2, "f32")
    for ext in (fast, None):
        monkeypatch.setattr(q4, "_fast", ext)
        q_out = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
        kc, vc = (torch.zeros(3, hkv, 16, D, dtype=torch.float16, device="cuda") for _ in range(2))
        pa.pa_append(r.tq, r.tk, r.tv, slots, i32(r.pos), kc, vc, q_out=q_out, **r.kw)
        cache = pa.new_q8_cache(3, hkv, D)
        q2 = torch.empty_like(q_out)
        pa.pa_q8_append(r.tq, r.tk, r.tv, slots, i32(r.pos), *cache, q_out=q2, **r.kw)
        k, v = (torch.empty(n, hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
        pa.pa_q8_read(*cache, slots, k, v)
        out, lse, err = d.run(0.1)
        acc, tok = run_verify(c, "f32")
        results.append([q_out, kc, vc, q2, k, v, *cache[2:], cache[0].view(torch.uint8),
                        cache[1].view(torch.uint8), *map(torch.from_numpy, (out, lse, acc, tok))])
    for a, b in zip(*results):
        assert torch.equal(a, b)
