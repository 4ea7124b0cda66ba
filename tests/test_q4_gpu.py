"""GPU tests of the 4-bit cache (pa_q4_write, pa_q4_read, pa_q4_decode) against
the fp64 reference: bytes and values exactly, attention within the bounds the
reference derives from the arithmetic."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q4_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q4
from paged_kv_gqa_pa_gb300 import build as pa_build

pytestmark = pytest.mark.gpu

T = {"f16": torch.float16, "bf16": torch.bfloat16}
DT = {"f16": 0, "bf16": 1}


@pytest.fixture(scope="module", autouse=True)
def built():
    pa_build.build()
    pa.load()


def to_t(x, dtype):
    """float64 values of T -> CUDA tensor of T (exact)."""
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().float().to(T[dtype])


def kv_values(g, shape, dtype):
    x = g.standard_normal(shape) * np.where(g.random(shape[-1]) < 0.05, 6.0, 1.0)
    return ref.rn(x + g.standard_normal(shape[-1]) * 0.5, dtype)


def special_rows(g, n, H, D, dtype):
    """Rows with what a quantiser can trip over, group by group."""
    x = kv_values(g, (n, H, D), dtype)
    big = ref.LIMIT[dtype]
    makers = [
        lambda: np.full(32, 1.25), lambda: np.zeros(32), lambda: np.full(32, -0.0),
        lambda: np.where(np.arange(32) == 5, np.nan, 1.0),
        lambda: np.where(np.arange(32) == 31, np.inf, g.standard_normal(32)),
        lambda: np.where(np.arange(32) == 0, -np.inf, g.standard_normal(32)),
        lambda: np.where(np.arange(32) % 2 == 0, np.inf, -np.inf),
        lambda: g.standard_normal(32) * big, lambda: np.full(32, big * 2),
        lambda: np.arange(32) % 16 * 1.0, lambda: np.arange(32) * 0.5 - 8,  # ties
        lambda: np.where(np.arange(32) == 0, 15.0, g.integers(0, 31, 32) / 2),
        lambda: g.standard_normal(32) * 1e-6, lambda: g.standard_normal(32) * 2e-38,
        lambda: 100 + g.standard_normal(32) * 0.01, lambda: np.where(g.random(32) < .5, 1000., 1e-4),
    ]
    for i in range(n):
        for h in range(H):
            for d in range(0, D, 32):
                if g.random() < 0.7:
                    with np.errstate(invalid="ignore"):
                        x[i, h, d:d + 32] = ref.rn(makers[g.integers(len(makers))](), dtype)
    return x


def reference_cache(cache, k, v, slots, D, dtype):
    """Host copy of the cache with the rows stored, and the values they stand for."""
    cache = cache.copy()
    kv = [np.zeros(k.shape), np.zeros(v.shape)]
    for i, s in enumerate(slots):
        if s < 0 or s >= cache.shape[0] * 16:
            continue
        for h in range(k.shape[1]):
            for j, x in enumerate((k, v)):
                kv[j][i, h] = ref.store_row(cache[s // 16, h], D, int(s % 16), x[i, h], dtype, j == 1)
    return cache, kv


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n,H", [(1, 1), (3, 2), (37, 3), (64, 1)])
def test_write_and_read_are_exact(n, H, D, dtype):
    g = np.random.default_rng([n, H, D, DT[dtype]])
    pages = n // 8 + 3
    k, v = special_rows(g, n, H, D, dtype), special_rows(g, n, H, D, dtype)
    slots = g.permutation(pages * 16)[:n]
    if n > 2:
        slots[1] = -1
    start = np.full((pages, H, 20 * D), 0xA5, np.uint8)
    want, kv = reference_cache(start, k, v, slots, D, dtype)
    # rows as columns of a fused projection's, with a column block in front
    fused = torch.zeros(n, 2 + 2 * H, D, dtype=T[dtype], device="cuda")
    fused[:, 2:2 + H] = to_t(k, dtype)
    fused[:, 2 + H:] = to_t(v, dtype)
    cache = torch.from_numpy(start).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    pa.pa_q4_write(fused[:, 2:2 + H], fused[:, 2 + H:], sl, cache, err)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    out = torch.full((2, n, H + 1, D), 7.0, dtype=T[dtype], device="cuda")
    pa.pa_q4_read(cache, sl, out[0, :, :H], out[1, :, :H], err)
    for j in range(2):
        o = out[j].double().cpu().numpy()
        np.testing.assert_array_equal(o[:, :H], kv[j])
        assert (o[:, H] == 7).all()  # the column behind is left alone
    assert int(err) == 0


@pytest.mark.parametrize("D", [64, 256])
def test_random_rows_are_exact_in_bulk(D):
    # Many groups, so that rounding borders are met: compared through the values alone,
    # with the fp64 definition on whole arrays.
    for dtype in ("f16", "bf16"):
        g = np.random.default_rng(D)
        n, H = 4000, 4
        x = ref.rn(g.standard_normal((n, H, D)) * 10.0 ** g.uniform(-3, 2, (n, H, 1)) +
                   g.standard_normal((n, H, 1)), dtype)
        gx = x.reshape(n, H, D // 32, 32)
        mn, mx = gx.min(-1, keepdims=True), gx.max(-1, keepdims=True)
        s = ref.rn((mx - mn) / 15, dtype)
        z = ref.rn(mn - 16 * s, dtype)
        c = np.where(s == 0, 0, np.clip(np.rint((gx - z) / np.where(s == 0, 1, s) - 16), 0, 15))
        want = ref.rn(s * (16 + c) + z, dtype).reshape(x.shape)
        rows = to_t(x, dtype)
        cache = pa.new_q4_cache(n // 16, H, D)
        slots = torch.from_numpy(g.permutation(n).astype(np.int64)).cuda()
        pa.pa_q4_write(rows, rows, slots, cache)
        out = torch.empty_like(rows), torch.empty_like(rows)
        pa.pa_q4_read(cache, slots, *out)
        for o in out:
            np.testing.assert_array_equal(o.double().cpu().numpy(), want)


def test_bad_slots_are_left_out_and_reported():
    g = np.random.default_rng(5)
    D, H, pages = 128, 2, 2
    rows = to_t(kv_values(g, (6, H, D), "f16"), "f16")
    for bad in (32, -2, 1 << 40, -(1 << 40)):
        cache = torch.full((pages, H, 20 * D), 0x33, dtype=torch.uint8, device="cuda")
        slots = torch.tensor([0, 17, bad, -1, 31, 5], device="cuda")
        err = torch.zeros(64, dtype=torch.int32, device="cuda")
        pa.pa_q4_write(rows, rows, slots, cache, err)
        assert pa.pa_get_error_ex(err) == q4.PA_DEVERR_BAD_SLOT
        want, kv = reference_cache(np.full((pages, H, 20 * D), 0x33, np.uint8),
                                   *[rows.double().cpu().numpy()] * 2, slots.tolist(), D, "f16")
        assert np.array_equal(cache.cpu().numpy(), want)
        k, v = torch.empty_like(rows), torch.empty_like(rows)
        pa.pa_q4_read(cache, slots, k, v, err)
        assert pa.pa_get_error_ex(err) == q4.PA_DEVERR_BAD_SLOT
        for o, w in ((k, kv[0]), (v, kv[1])):
            o = o.double().cpu().numpy()
            assert np.isnan(o[2]).all() and (o[3] == 0).all()
            np.testing.assert_array_equal(o[[0, 1, 4, 5]], w[[0, 1, 4, 5]])
        pa.pa_q4_write(rows, rows, slots, cache)  # the error word is optional


# ---------------------------------------------------------------- attention

def make_decode(seed, lens, Hq, Hkv, D, dtype, q_std=1.0, maxp=None):
    """A cache whose cells are 0xFF (NaN scales) wherever no attended token lies."""
    g = np.random.default_rng(seed)
    need = [-(-L // 16) for L in lens]
    pages = sum(need) + 3
    perm = g.permutation(pages)
    maxp = maxp or max(1, max(need))
    bt = np.full((len(lens), maxp), -1, np.int32)
    cache = torch.full((pages, Hkv, 20 * D), 255, dtype=torch.uint8, device="cuda")
    at = 0
    slots = []
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
        pos = np.arange(lens[b])
        slots.append(bt[b][pos // 16].astype(np.int64) * 16 + pos % 16)
    slots = np.concatenate(slots)
    k, v = (to_t(kv_values(g, (slots.size, Hkv, D), dtype), dtype) for _ in range(2))
    if slots.size:
        pa.pa_q4_write(k, v, torch.from_numpy(slots).cuda(), cache)
    q = ref.rn(g.standard_normal((len(lens), Hq, D)) * q_std, dtype)
    return q, cache, bt, np.asarray(lens, np.int32)


def run_decode(q, cache, bt, lens, scale, window, dtype, max_len=None, ctas=None, ws=None,
               stall=0, cluster=None):
    B, Hq, D = q.shape
    plan = pa.pa_q4_plan(B, Hq, cache.shape[1], D, 16, cache.shape[0], bt.shape[1],
                         int(lens.max()) if max_len is None else max_len, window, 0, DT[dtype])
    if ctas is not None:
        plan.ctas_per_group, plan.cluster = ctas, 0
    if cluster == 0:
        plan.cluster = 0
    plan.test_stall_bytes = stall
    guard = 64
    nan = float("nan")
    ob = torch.full((B * Hq * D + 2 * guard,), nan, dtype=T[dtype], device="cuda")
    lb = torch.full((B * Hq + 2 * guard,), nan, dtype=torch.float32, device="cuda")
    if ws is None:  # only the control bytes start at zero
        ws = torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        ws[:plan.ctrl_bytes] = 0
    out, lse = ob[guard:-guard].view(B, Hq, D), lb[guard:-guard].view(B, Hq)
    pa.pa_q4_decode(plan, to_t(q, dtype), cache, torch.from_numpy(bt).cuda(),
                    torch.from_numpy(lens).cuda(), scale, window, out, lse, ws)
    err = pa.pa_get_error_ex(ws)
    assert int(ws[:plan.ctrl_bytes].count_nonzero()) == 0, "control bytes not left zero"
    for buf in (ob, lb):
        assert torch.isnan(buf[:guard]).all() and torch.isnan(buf[-guard:]).all(), "guard"
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), err


def check(got, want):
    out, lse, err = got
    w_out, w_lse, tol, ltol = want
    assert err == 0
    assert np.isfinite(out).all()
    over = np.abs(out - w_out) - tol
    assert (over <= 0).all(), f"out off by {np.abs(out - w_out).max():.3e}, beyond by {over.max():.3e}"
    fin = np.isfinite(w_lse)
    assert np.array_equal(lse[~fin], w_lse[~fin])
    d = np.abs(lse[fin] - w_lse[fin])
    assert (d <= ltol[fin]).all(), d.max()


def decode_case(seed, lens, Hq, Hkv, D, dtype, window=0, scale=None, **kw):
    q, cache, bt, lens = make_decode(seed, lens, Hq, Hkv, D, dtype, kw.pop("q_std", 1.0),
                                     kw.pop("maxp", None))
    scale = D ** -0.5 if scale is None else scale
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, scale, window, dtype)
    got = run_decode(q, cache, bt, lens, scale, window, dtype, **kw)
    check(got, want)
    return got


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (6, 1), (8, 1), (16, 1), (10, 5)])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_lengths(Hq, Hkv, D, dtype, cluster):
    decode_case(D + Hq, [1, 15, 16, 17, 0, 255, 700], Hq, Hkv, D, dtype, cluster=cluster)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (96, "f16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 333, 5000])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_windows(window, D, dtype, cluster):
    decode_case(window, [1, 4, 16, 33, 333, 1000, 0], 4, 2, D, dtype, window=window,
                cluster=cluster)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (96, "f16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("C", [2, 3, 7, 8])
def test_decode_cluster_sizes(C, D, dtype):
    # Shares that end inside a slot, ranks without a page, one page for all of them.
    lens = [1, 16, 17, 0, 400, 16 * C, 16 * C + 1, 33 * C]
    q, cache, bt, lens = make_decode(60 + C, lens, 6, 2, D, dtype)
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, dtype)
    plan = pa.pa_q4_plan(len(lens), 6, 2, D, 16, cache.shape[0], bt.shape[1],
                         int(lens.max()), 0, 0, DT[dtype])
    plan.cluster, plan.ctas_per_group = C, C * len(lens)
    plan.workspace_bytes = 1 << 28
    plan.ctrl_bytes = max(plan.ctrl_bytes, 4096)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    tq = to_t(q, dtype)
    out, lse = torch.full_like(tq, float("nan")), torch.empty(len(lens), 6, device="cuda")
    pa.pa_q4_decode(plan, tq, cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 0.1, 0,
                    out, lse, ws)
    check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (96, "bf16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, None])
def test_decode_ranges_cut_anywhere(ctas, D, dtype):
    # Ranges of the batch's pages: one CTA for all, cuts inside and between sequences, many
    # sequences in one range.
    lens = [40, 1, 0, 16, 0, 900, 128, 128, 3, 0] + [20] * 20
    decode_case(7, lens, 4, 1, D, dtype, ctas=ctas)


def test_decode_long_ranges_are_staged_in_stretches():
    # One CTA serves 2600 pages, more than it stages at a time, with sequences that end at,
    # before and behind the borders of the stretches.
    decode_case(8, [1024 * 16, 100, 1023 * 16, 9000], 2, 1, 64, "f16", ctas=1)
    decode_case(8, [1024 * 16, 1024 * 16], 2, 1, 64, "bf16", ctas=1)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_one_long_sequence(D):
    decode_case(9, [20011], 8, 1, D, "f16")
    decode_case(9, [20011, 17], 4, 2, D, "bf16", window=15000)


@pytest.mark.parametrize("B", [129, 300, 1500])
def test_decode_large_batches(B):
    g = np.random.default_rng(B)
    decode_case(B, g.integers(0, 60, B).tolist(), 2, 1, 64, "f16")


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_decode_scales(scale):
    decode_case(11, [50, 300, 1], 4, 1, 128, "f16", scale=scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_sharp_scores(dtype):
    # Scores of some hundreds: the running maximum has to be raised again and again.
    decode_case(12, [600, 33], 4, 1, 128, dtype, q_std=30.0)


def test_decode_table_wider_than_the_lengths():
    decode_case(13, [5, 100], 4, 1, 128, "f16", maxp=40, max_len=640)


def test_decode_equals_pa_decode_on_the_values():
    D, dtype = 128, "f16"
    q, cache, bt, lens = make_decode(14, [1, 300, 777], 8, 2, D, dtype)
    k, v = ref.unpack(cache.cpu().numpy().reshape(-1, 20 * D), D, dtype)
    k, v = (to_t(np.nan_to_num(x), dtype).view(cache.shape[0], 2, 16, D) for x in (k, v))
    out, lse, _, err = pa.decode(to_t(q, dtype), k, v, torch.from_numpy(bt).cuda(),
                                 torch.from_numpy(lens).cuda(), D ** -0.5)
    o4, l4, _, err4 = pa.q4_decode(to_t(q, dtype), cache, torch.from_numpy(bt).cuda(),
                                   torch.from_numpy(lens).cuda(), D ** -0.5)
    assert err == err4 == 0
    _, _, tol, ltol = ref.decode(q, cache.cpu().numpy(), bt, lens, D ** -0.5, 0, dtype)
    assert (np.abs((out.double() - o4.double()).cpu().numpy()) <= 2 * tol).all()
    assert (np.abs((lse.double() - l4.double()).cpu().numpy()) <= 2 * ltol).all()


def test_decode_carries_nan_values_to_their_rows_only():
    q, cache, bt, lens = make_decode(15, [40, 70], 4, 2, 128, "f16")
    row = torch.full((1, 2, 128), 1.0, dtype=torch.float16, device="cuda")
    bad = row.clone()
    bad[0, 1, 40] = float("nan")  # KV head 1 of one token of sequence 1
    slot = torch.tensor([int(bt[1, 2]) * 16 + 3], device="cuda")
    pa.pa_q4_write(row, bad, slot, cache)  # in V: only the group's dims of head 1
    out, lse, err = run_decode(q, cache, bt, lens, 0.1, 0, "f16")
    assert err == 0 and np.isfinite(lse).all()
    nan = np.isnan(out)
    assert nan[1, 2:, 32:64].all() and nan.sum() == 2 * 32


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (96, "bf16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("ctas", [3, 8, 13, 19, 31, 40])
def test_decode_ranges_within_a_sequences_start(ctas, D, dtype):
    """Ranges shorter than what a start counts for: some CTAs get no page, and borders fall on,
    before and behind the first pages, with empty sequences between; both kinds of merge."""
    lens = [0, 400, 1, 0, 0, 16, 17, 300]
    q, cache, bt, lens = make_decode(80 + ctas, lens, 6, 2, D, dtype)
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, dtype)
    plan = pa.pa_q4_plan(len(lens), 6, 2, D, 16, cache.shape[0], bt.shape[1],
                         int(lens.max()), 0, 0, DT[dtype])
    plan.cluster, plan.ctas_per_group = 0, ctas
    plan.workspace_bytes = 1 << 26
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    tq = to_t(q, dtype)
    args = [tq, cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 0.1, 0]
    for _ in range(2):
        out, lse = torch.full_like(tq, float("nan")), torch.empty(len(lens), 6, device="cuda")
        pa.pa_q4_decode(plan, *args, out, lse, ws)
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("ctas", [1, 6, None])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_page_ids_and_lengths_give_nan_rows(D, ctas):
    q, cache, bt, lens = make_decode(16, [700, 300, 90, 16], 4, 1, D, "f16")
    good = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16")

    def rows(got, keep, gone):
        out, lse, _ = got
        for b in gone:
            assert np.isnan(out[b]).all() and np.isnan(lse[b]).all()
        check((out[keep], lse[keep], 0), [x[keep] for x in good])

    for bad in (cache.shape[0], -1, 1 << 30):
        b2 = bt.copy()
        b2[0, 20] = bad
        got = run_decode(q, cache, b2, lens, 0.1, 0, "f16", ctas=ctas)
        assert got[2] == binding.PA_DEVERR_BAD_PAGE
        rows(got, [1, 2, 3], [0])
    for bad in (-1, 701, 1 << 30, -(1 << 31)):
        l2 = lens.copy()
        l2[1] = bad
        got = run_decode(q, cache, bt, l2, 0.1, 0, "f16", ctas=ctas, max_len=700)
        assert got[2] == binding.PA_DEVERR_BAD_LENGTH
        rows(got, [0, 2, 3], [1])


@pytest.mark.parametrize("cluster", [None, 0])
def test_copy_timeout_is_reported_and_the_next_call_is_clean(cluster):
    q, cache, bt, lens = make_decode(17, [500, 20], 4, 1, 128, "f16")
    out, lse, err = run_decode(q, cache, bt, lens, 0.1, 0, "f16", stall=16, cluster=cluster)
    assert err & binding.PA_DEVERR_TIMEOUT
    assert np.isnan(out).all() and np.isnan(lse).all()
    check(run_decode(q, cache, bt, lens, 0.1, 0, "f16"),
          ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16"))


@pytest.mark.parametrize("cluster", [None, 0])
def test_calls_repeat_bit_for_bit(cluster):
    q, cache, bt, lens = make_decode(18, [3000, 100, 2000], 8, 2, 128, "f16")
    first = run_decode(q, cache, bt, lens, 0.1, 0, "f16", cluster=cluster)
    for _ in range(5):
        again = run_decode(q, cache, bt, lens, 0.1, 0, "f16", cluster=cluster)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_two_streams_with_their_own_workspaces_and_a_prepared_call():
    q, cache, bt, lens = make_decode(19, [3000, 100, 2000, 7], 8, 2, 128, "bf16")
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "bf16")
    plan = pa.pa_q4_plan(4, 8, 2, 128, 16, cache.shape[0], bt.shape[1], 3000, dtype=1)
    tq, tb, tl = to_t(q, "bf16"), torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    jobs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        out = torch.empty_like(tq)
        lse = torch.empty(4, 8, device="cuda")
        ws = pa.new_workspace(plan, "cuda")
        jobs.append((pa.prepare_q4_decode(plan, tq, cache, tb, tl, 0.1, 0, out, lse, ws, s), out,
                     lse, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, *_ in jobs:
            call()
    torch.cuda.synchronize()
    for _, out, lse, ws in jobs:
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


def test_refused_tensors():
    q, cache, bt, lens = make_decode(20, [30], 4, 1, 128, "f16")
    plan = pa.pa_q4_plan(1, 4, 1, 128, 16, cache.shape[0], bt.shape[1], 30)
    tq, tb, tl = to_t(q, "f16"), torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    out, lse, ws = torch.empty_like(tq), torch.empty(1, 4, device="cuda"), pa.new_workspace(plan, "cuda")
    ok = [plan, tq, cache, tb, tl, 0.1, 0, out, lse, ws]
    pa.pa_q4_decode(*ok)
    for i, bad, exc in [(1, tq.bfloat16(), TypeError), (1, tq.transpose(1, 2), ValueError),
                        (1, tq.cpu(), ValueError), (2, cache.view(torch.int8), TypeError),
                        (2, cache[:, :, :1280], ValueError), (2, cache[:1], ValueError),
                        (3, tb.long(), TypeError), (4, tl.repeat(2), ValueError),
                        (7, out.float(), TypeError), (8, lse.double(), TypeError),
                        (9, ws[:8], pa.PAError), (6, 3, pa.PAError)]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            pa.pa_q4_decode(*args)
    rows = torch.zeros(4, 2, 128, dtype=torch.float16, device="cuda")
    c2 = pa.new_q4_cache(2, 2, 128)
    slots = torch.arange(4, device="cuda")
    for args, exc in [((rows.float(), rows.float(), slots, c2), pa.PAError),
                      ((rows, rows[:3], slots, c2), ValueError),
                      ((rows, rows.bfloat16(), slots, c2), TypeError),
                      ((rows, rows, slots.int(), c2), TypeError),
                      ((rows, rows, slots[:3], c2), ValueError),
                      ((rows.transpose(0, 1).contiguous().transpose(0, 1), rows, slots, c2), ValueError),
                      ((rows[:, :1], rows[:, :1], slots, c2), ValueError),
                      ((rows, rows, slots, c2.cpu()), ValueError),
                      ((rows[..., :64], rows[..., :64], slots, c2), ValueError)]:
        with pytest.raises(exc):
            pa.pa_q4_write(*args)


def test_empty_calls():
    c = pa.new_q4_cache(2, 1, 64)
    none = torch.empty(0, 1, 64, dtype=torch.float16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    pa.pa_q4_write(none, none, slots, c)
    pa.pa_q4_read(c, slots, none, none)
    assert int(c.count_nonzero()) == 0
    out, lse, err = decode_case(21, [0, 0, 0], 2, 1, 64, "f16", max_len=0)
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.fixture(scope="module")
def late_writer():
    """tests/cuda/pdl_writer.cu: a kernel that lets the next one start early, waits 20 us and only
    then writes the block table and the lengths."""
    import ctypes
    import os
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    os.makedirs(os.path.join(here, "_build"), exist_ok=True)
    so = os.path.join(here, "_build", "libpdl_writer_q4.so")
    src = os.path.join(here, "cuda", "pdl_writer.cu")
    if not os.path.exists(so) or os.path.getmtime(so) < os.path.getmtime(src):
        subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-shared",
                        "-Xcompiler", "-fPIC", src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    P = ctypes.c_void_p
    lib.launch_delayed_copy.argtypes = [P, P, ctypes.c_int, P, P, ctypes.c_int, ctypes.c_ulonglong,
                                        P]
    return lib


@pytest.mark.parametrize("cluster", [None, 0])
@pytest.mark.parametrize("old", ["same lengths", "a token more", "pages fewer", "garbage"])
@pytest.mark.parametrize("lens,window,D", [([3000, 1200, 0, 2049, 77], 0, 128),
                                           ([3000, 1200, 2049, 77], 1000, 64),
                                           ([20000], 0, 256), ([30] * 127 + [0], 0, 64),
                                           ([40, 3] * 100, 0, 96)])
def test_decode_uses_lengths_and_ids_written_late(late_writer, lens, window, D, old, cluster):
    # What the kernel reads before its dependency wait are hints; everything counts only as it
    # stands after the wait.  The old table points at a page of NaN scales.
    q, cache, bt, lens = make_decode(30, lens, 4, 2, D, "f16")
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, D ** -0.5, window, "f16")
    unused = sorted(set(range(cache.shape[0])) - set(bt.ravel().tolist()))
    old_bt = np.full_like(bt, unused[0])
    old_lens = {"same lengths": lens, "a token more": np.minimum(lens + 1, lens.max()),
                "pages fewer": lens // 2,
                "garbage": np.where(np.arange(lens.size) % 2, -5, 1 << 30)}[old].astype(np.int32)
    if old == "garbage":
        old_bt[:, ::2] = -7
        old_bt[:, 1::2] = 1 << 30
    B, Hq = q.shape[:2]
    plan = pa.pa_q4_plan(B, Hq, 2, D, 16, cache.shape[0], bt.shape[1], int(lens.max()), window)
    if cluster == 0:
        plan.cluster = 0
    ws = pa.new_workspace(plan, "cuda")
    tq = to_t(q, "f16")
    new = torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    now = torch.from_numpy(old_bt).cuda(), torch.from_numpy(old_lens).cuda()
    out = torch.full_like(tq, float("nan"))
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    stream = torch.cuda.current_stream()
    assert late_writer.launch_delayed_copy(new[0].data_ptr(), now[0].data_ptr(), bt.size,
                                           new[1].data_ptr(), now[1].data_ptr(), lens.size, 20000,
                                           stream.cuda_stream) == 0
    pa.pa_q4_decode(plan, tq, cache, now[0], now[1], D ** -0.5, window, out, lse, ws)
    check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("Hq,Hkv", [(12, 1), (24, 1), (21, 3), (64, 2)])
def test_decode_head_chunks(Hq, Hkv):
    # More than 8 query heads per KV head go in equal chunks; 7 of 8 columns used.
    decode_case(Hq, [300, 17, 64], Hq, Hkv, 64, "f16")
    decode_case(Hq, [300, 17, 600], Hq, Hkv, 128, "bf16", window=130)


def test_decode_nan_in_one_query_head_stays_there():
    q, cache, bt, lens = make_decode(40, [500, 20], 8, 1, 128, "f16")
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16")
    q = q.copy()
    q[0, 3, 17] = np.nan
    out, lse, err = run_decode(q, cache, bt, lens, 0.1, 0, "f16")
    assert err == 0 and np.isnan(out[0, 3]).all() and np.isnan(lse[0, 3])
    rest = [0, 1, 2, 4, 5, 6, 7]
    for b in (0, 1):
        hs = rest if b == 0 else list(range(8))
        check((out[b, hs], lse[b, hs], 0), [x[b, hs] for x in want])


def test_sequences_may_share_pages():
    q, cache, bt, lens = make_decode(41, [160, 160, 90], 4, 2, 128, "f16")
    bt[1, :5] = bt[0, :5]
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16")
    check(run_decode(q, cache, bt, lens, 0.1, 0, "f16"), want)


def test_offsets_beyond_32_bits():
    # 900,000 pages of 5120 bytes: 4.6 GB, used near their end.
    pages, D = 900_000, 256
    cache = torch.empty(pages, 1, 20 * D, dtype=torch.uint8, device="cuda")
    ids = np.array([pages - 1, 3, pages - 2, 840_001, pages - 7], np.int32)
    g = np.random.default_rng(42)
    n = 75
    k, v = kv_values(g, (n, 1, D), "f16"), kv_values(g, (n, 1, D), "f16")
    pos = np.arange(n)
    slots = ids[pos // 16].astype(np.int64) * 16 + pos % 16
    small = np.full((5, 1, 20 * D), 255, np.uint8)
    want, kv = reference_cache(small, k, v, (pos // 16) * 16 + pos % 16, D, "f16")
    cache[torch.from_numpy(ids).long().cuda()] = 255
    sl = torch.from_numpy(slots).cuda()
    pa.pa_q4_write(to_t(k, "f16"), to_t(v, "f16"), sl, cache)
    assert np.array_equal(cache[torch.from_numpy(ids).long().cuda()].cpu().numpy(), want)
    out = torch.empty(n, 1, D, dtype=torch.float16, device="cuda"), torch.empty(
        n, 1, D, dtype=torch.float16, device="cuda")
    pa.pa_q4_read(cache, sl, *out)
    for o, w in zip(out, kv):
        np.testing.assert_array_equal(o.double().cpu().numpy(), w)
    q = ref.rn(g.standard_normal((1, 4, D)), "f16")
    lens = np.array([n], np.int32)
    res = run_decode(q, cache, ids[None], lens, 0.1, 0, "f16")
    check(res, ref.decode(q, want, np.arange(5, dtype=np.int32)[None], lens, 0.1, 0, "f16"))


def test_read_takes_slots_twice():
    g = np.random.default_rng(43)
    k = kv_values(g, (4, 2, 96), "bf16")
    cache = pa.new_q4_cache(1, 2, 96)
    pa.pa_q4_write(to_t(k, "bf16"), to_t(k, "bf16"), torch.arange(4, device="cuda"), cache)
    out = torch.empty(6, 2, 96, dtype=torch.bfloat16, device="cuda")
    out2 = torch.empty_like(out)
    pa.pa_q4_read(cache, torch.tensor([2, 2, 0, 3, 2, 15], device="cuda"), out, out2)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[4]) and torch.equal(out, out2)
    assert (out[5] == 0).all()  # an empty cell of a fresh cache


def test_two_graphs_share_a_workspace_one_after_the_other():
    q, cache, bt, lens = make_decode(44, [3000, 100, 2000, 900, 3], 8, 2, 128, "f16")
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16")
    plan = pa.pa_q4_plan(5, 8, 2, 128, 16, cache.shape[0], bt.shape[1], 3000)
    ws = pa.new_workspace(plan, "cuda")
    tq, tb, tl = to_t(q, "f16"), torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    runs = []
    for _ in range(2):
        out, lse = torch.empty_like(tq), torch.empty(5, 8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                pa.pa_q4_decode(plan, tq, cache, tb, tl, 0.1, 0, out, lse, ws)
        runs.append((graph, out, lse))
    for i in (0, 1, 1, 0):
        runs[i][0].replay()
    torch.cuda.synchronize()
    for _, out, lse in runs:
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


def test_the_largest_batch():
    g = np.random.default_rng(45)
    decode_case(45, g.integers(0, 20, 4096).tolist(), 1, 1, 64, "f16")


def test_plans_for_other_sm_counts():
    q, cache, bt, lens = make_decode(46, [500, 20, 1000], 4, 2, 128, "f16")
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, 0, "f16")
    for sms in (1, 8, 500):
        plan = pa.pa_q4_plan(3, 4, 2, 128, 16, cache.shape[0], bt.shape[1], 1000, 0, sms)
        ws = pa.new_workspace(plan, "cuda")
        tq = to_t(q, "f16")
        out, lse = torch.empty_like(tq), torch.empty(3, 4, device="cuda")
        pa.pa_q4_decode(plan, tq, cache, torch.from_numpy(bt).cuda(),
                        torch.from_numpy(lens).cuda(), 0.1, 0, out, lse, ws)
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("short_by,window", [(0, 100), (1, 7), (15, 333), (16, 1), (37, 2)])
def test_windows_at_the_longest_lengths(short_by, window):
    # 2^31 - 16 tokens, a table of 2^27 entries whose last pages are there: the same rows as of a
    # sequence of 400 tokens with these pages.  Both caches.
    D, maxp, small = 128, 1 << 27, 25
    q, cache, bt, lens = make_decode(47, [16 * small], 8, 2, D, "f16")
    lens = lens - short_by
    want = ref.decode(q, cache.cpu().numpy(), bt, lens, 0.1, window, "f16")
    table = torch.zeros(1, maxp, dtype=torch.int32, device="cuda")
    table[0, maxp - 1 - small:maxp - 1] = torch.from_numpy(bt[0]).cuda()
    long = torch.full((1,), 2 ** 31 - 16 - short_by, dtype=torch.int32, device="cuda")
    tq = to_t(q, "f16")
    k, v = ref.unpack(cache.cpu().numpy().reshape(-1, 20 * D), D, "f16")
    k, v = (to_t(np.nan_to_num(x), "f16").view(cache.shape[0], 2, 16, D) for x in (k, v))
    for four in (True, False):
        if four:
            plan = pa.pa_q4_plan(1, 8, 2, D, 16, cache.shape[0], maxp, 2 ** 31 - 16, window)
        else:
            plan = pa.pa_plan(1, 8, 2, D, 16, cache.shape[0], maxp, 2 ** 31 - 16, window)
        ws = pa.new_workspace(plan, "cuda")
        out, lse = torch.full_like(tq, float("nan")), torch.empty(1, 8, device="cuda")
        if four:
            pa.pa_q4_decode(plan, tq, cache, table, long, 0.1, window, out, lse, ws)
        else:
            pa.pa_decode(plan, tq, k, v, table, long, 0.1, window, out, lse, ws)
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), pa.pa_get_error(ws)), want)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [256, 1999])
@pytest.mark.parametrize("where", ["first", "last", "alternate pages", "alternate tokens"])
@pytest.mark.parametrize("cluster", [None, 0])
def test_decode_scores_below_fp32(D, n, where, cluster):
    # q k of some tokens is beyond fp32 (bf16 reaches that): -inf, which weighs nothing, also where
    # it is all that a warp has met so far.  The rest of the row is as without these tokens.
    dtype, g = "bf16", np.random.default_rng(n)
    k, v = kv_values(g, (n, 2, D), dtype), kv_values(g, (n, 2, D), dtype)
    at = np.arange(n)
    low = {"first": at < 128, "last": at >= n - 128, "alternate pages": at // 16 % 2 == 0,
           "alternate tokens": at % 2 == 1}[where]
    k[:, :, :32] = 0
    k[low, :, 0] = 2.0 ** 119
    q = ref.rn(g.standard_normal((1, 8, D)), dtype)
    q[:, :, 0] = -2.0 ** 20
    pages = -(-n // 16)
    cache = torch.full((pages, 2, 20 * D), 255, dtype=torch.uint8, device="cuda")
    pa.pa_q4_write(to_t(k, dtype), to_t(v, dtype), torch.arange(n, device="cuda"), cache)
    bt, lens = np.arange(pages, dtype=np.int32)[None], np.array([n], np.int32)
    kk, vv = (x.reshape(pages, 2, 16, D).transpose(0, 2, 1, 3).reshape(-1, 2, D)[:n][~low]
              for x in ref.unpack(cache.cpu().numpy().reshape(-1, 20 * D), D, dtype))
    want = [ref.attend(q[0, 4 * h:4 * h + 4], kk[:, h], vv[:, h], D ** -0.5, dtype) for h in (0, 1)]
    check(run_decode(q, cache, bt, lens, D ** -0.5, 0, dtype, cluster=cluster),
          [np.concatenate([w[i] for w in want])[None] for i in range(4)])


@pytest.mark.parametrize("Hq,Hkv", [(9, 1), (30, 2), (18, 1), (22, 1), (50, 2)])
def test_decode_head_chunks_of_other_sizes(Hq, Hkv):
    # 3 x 3, 3 x 5, 3 x 6, 11 x 2 and 5 x 5 query heads of a KV head.
    decode_case(Hq, [300, 17, 64, 0], Hq, Hkv, 96, "f16")
    decode_case(Hq, [3000, 17, 600], Hq, Hkv, 128, "bf16", window=2000)
