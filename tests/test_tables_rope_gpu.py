"""GPU tests of pa_extend_tables and pa_rope_axes, and of a serving loop that
uses the operators of include/pa_q4.h together."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q4_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q4
from paged_kv_gqa_pa_gb300 import build as pa_build
from test_q4_gpu import T, check, kv_values, reference_cache, to_t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pa_build.build()
    pa.load()


# ---------------------------------------------------------------- tables

def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def run_tables(past, new, free, num_pages, bt, cap):
    B = len(past)
    dev = "cuda"
    err = torch.zeros(64, dtype=torch.int32, device=dev)
    bt_d = i32(bt)
    lens, starts = i32(np.full(B, -7)), i32(np.full(B + 1, -7))
    slots = torch.full((cap + 8,), -7, dtype=torch.int64, device=dev)
    pos = i32(np.full(cap + 8, -7))
    taken = i32([-7])
    pa.pa_extend_tables(i32(past), i32(new), i32(free), num_pages, bt_d, lens, starts, slots[:cap],
                        pos[:cap], taken, err)
    assert (slots[cap:] == -7).all() and (pos[cap:] == -7).all()
    return (bt_d.cpu().numpy(), lens.cpu().numpy(), starts.cpu().numpy(), slots[:cap].cpu().numpy(),
            pos[:cap].cpu().numpy(), int(taken), pa.pa_get_error_ex(err))


def check_tables(past, new, free, num_pages, bt, cap):
    want = ref.extend_tables(past, new, free, num_pages, bt, cap)
    got = run_tables(past, new, free, num_pages, bt, cap)
    for name, g, w in zip("tables lens starts slots positions taken err".split(), got, want):
        assert np.array_equal(g, w), (name, g, w)
    return got


def requests(seed, B, maxp, past_max, new_max):
    g = np.random.default_rng(seed)
    past = g.integers(0, past_max + 1, B)
    new = g.integers(0, new_max + 1, B)
    new = np.minimum(new, maxp * 16 - past)
    have, need = -(-past // 16), -(-(past + new) // 16)
    pages = int(need.sum()) + 5
    perm = g.permutation(pages)
    bt = np.full((B, maxp), -1, np.int32)
    at = 0
    for b in range(B):
        bt[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    return past, new, perm[at:], pages, bt, int(new.sum())


@pytest.mark.parametrize("B,maxp,past_max,new_max", [
    (1, 1, 0, 1), (1, 4, 63, 1), (1, 200, 0, 3000), (7, 9, 100, 3), (64, 40, 500, 1),
    (255, 20, 200, 40), (256, 20, 200, 40), (257, 20, 0, 300), (1000, 8, 100, 1),
    (8192, 3, 40, 5)])
@pytest.mark.parametrize("pad", [0, 13])
def test_tables(B, maxp, past_max, new_max, pad):
    past, new, free, pages, bt, n = requests(B, B, maxp, past_max, new_max)
    got = check_tables(past, new, free, pages, bt, n + pad)
    assert got[6] == 0


def test_tables_prompt_larger_than_a_grid_row():
    past, new, free, pages, bt, n = requests(3, 3, 5000, 10, 70000)
    check_tables(past, new, free, pages, bt, n)


@pytest.mark.parametrize("B", [6015, 6016, 6135, 6136, 6139, 6143, 6144])
def test_tables_of_a_batch_around_48_kb(B):
    # In a process of its own: the kernel's shared memory limit, once raised, stays raised.
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import test_tables_rope_gpu as t\n"
            "past, new, free, pages, bt, n = t.requests(%d, %d, 3, 40, 2)\n"
            "assert t.check_tables(past, new, free, pages, bt, n)[6] == 0\n"
            % (os.path.dirname(here), here, B, B))
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_tables_refusals():
    past, new, free, pages, bt, n = requests(5, 12, 10, 80, 60)
    # lengths out of bounds: negative ones, and one beyond the row
    for i, (p, m) in enumerate([(-1, 3), (5, -2), (100, 61), (161, 0), (-2**31, 2**31 - 1)]):
        p2, n2 = past.copy(), new.copy()
        p2[4], n2[4] = p, m
        cap = min(int(np.maximum(n2, 0).sum()), n + 64)
        got = check_tables(p2, n2, free, pages, bt, cap)
        assert got[6] & binding.PA_DEVERR_BAD_LENGTH
    # tokens beyond the capacity
    assert check_tables(past, new, free, pages, bt, n - 1)[6] == binding.PA_DEVERR_BAD_LENGTH
    assert check_tables(past, new, free, pages, bt, 0)[6] == binding.PA_DEVERR_BAD_LENGTH
    # the free list ends early, down to nothing
    for short in (1, 7, 15, len(free)):
        got = check_tables(past, new, free[:len(free) - short], pages, bt, n)
    assert got[6] & q4.PA_DEVERR_NO_PAGES and got[5] == 0
    # bad ids in the free list and in a row
    f2 = free.copy()
    f2[1], f2[4] = pages, -1
    assert check_tables(past, new, f2, pages, bt, n)[6] == binding.PA_DEVERR_BAD_PAGE
    b2, p2, n2 = bt.copy(), past.copy(), new.copy()
    p2[3], n2[3] = 24, 4
    b2[3, 1] = pages + 3
    assert check_tables(p2, n2, free, pages, b2, int(n2.sum()))[6] == binding.PA_DEVERR_BAD_PAGE


def test_tables_without_requests():
    got = run_tables([], [], [3, 4], 8, np.zeros((0, 4), np.int32), 5)
    assert got[2].tolist() == [0] and got[3].tolist() == [-1] * 5 and got[4].tolist() == [0] * 5
    assert got[5] == 0 and got[6] == 0


def test_tables_graph_replay_with_new_lengths():
    past, new, free, pages, bt, n = requests(6, 30, 20, 100, 20)
    d = [i32(x) for x in (past, new, free, bt)]
    lens, starts, taken = i32(np.zeros(30)), i32(np.zeros(31)), i32([0])
    cap = 30 * 20
    slots, pos = torch.zeros(cap, dtype=torch.int64, device="cuda"), i32(np.zeros(cap))
    err = torch.zeros(64, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        pa.pa_extend_tables(d[0], d[1], d[2], pages, d[3], lens, starts, slots, pos, taken, err)
    for seed in (7, 8):
        past, new, free, p2, bt, n = requests(seed, 30, 20, 100, 20)
        m = min(pages, p2)
        free = free[free < m]
        bt = np.minimum(bt, m - 1)
        d[0].copy_(i32(past)), d[1].copy_(i32(new)), d[3].copy_(i32(bt))
        f = np.zeros(d[2].numel(), np.int64)
        f[:min(len(f), len(free))] = free[:len(f)]
        d[2].copy_(i32(f))
        g.replay()
        torch.cuda.synchronize()
        want = ref.extend_tables(past, new, f, pages, bt, cap)
        for a, w in zip((d[3], lens, starts, slots, pos), want):
            assert np.array_equal(a.cpu().numpy(), w)
        assert int(taken) == want[5]


# ---------------------------------------------------------------- rotary

RT = dict(T, f32=torch.float32)


def rope_tolerance(x, want, rot, dtype):
    """Two products of fp32 and their sum: each cosine is off by at most 2^-22 (angle 2^-24
    of a turn, sincospif), each operation by 2^-24 of what it makes; then one rounding to T."""
    half = rot // 2
    mag = np.zeros_like(want)
    m = np.abs(x[..., :half]) + np.abs(x[..., half:rot])
    mag[..., :half] = m
    mag[..., half:rot] = m
    return mag * 2.0 ** -20 + ref.HALF_STEP[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)


def rope_case(seed, n, hq, hk, D, rot, sections, dtype, interleaved=False, inverse=False,
              theta=10000.0, top=1 << 17, in_place=False, fused=True):
    g = np.random.default_rng(seed)
    H = hq + hk
    x = ref.rn(g.standard_normal((n, H, D)) * 3, dtype)
    pos = g.integers(-top if top > 1 << 20 else 0, top, (len(sections), n))
    buf = torch.zeros(n, H + 2, D, dtype=RT[dtype], device="cuda")
    buf[:, :H] = torch.from_numpy(x).cuda().to(RT[dtype])
    q, k = buf[:, :hq], buf[:, hq:H]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    before = buf.clone()
    kw = {}
    if not in_place:
        kw = dict(q_out=torch.full_like(q, 9).contiguous(), k_out=torch.full_like(k, 9).contiguous())
        if hk == 0:
            kw.pop("k_out")
        if hq == 0:
            kw.pop("q_out")
    pa.pa_rope_axes(q if hq else None, k if hk else None, i32(pos), sections, theta,
                    rotary_dim=rot, interleaved=interleaved, inverse=inverse, **kw)
    got = [kw.get("q_out", q), kw.get("k_out", k)]
    want = ref.rope(x, pos, sections, theta, rot, interleaved, inverse)
    tol = rope_tolerance(x, want, rot, dtype)
    for o, sl in zip(got, (slice(0, hq), slice(hq, H))):
        o = o.double().cpu().numpy()
        if sl.stop == sl.start:
            continue
        assert (np.abs(o - want[:, sl]) <= tol[:, sl]).all(), np.abs(o - want[:, sl]).max()
        assert np.array_equal(o[..., rot:], x[:, sl, rot:])
    if in_place:
        assert torch.equal(buf[:, H:], before[:, H:])
    else:
        assert torch.equal(buf, before)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,rot,sections,inter", [
    (64, 64, (8, 12, 12), False), (64, 32, (6, 5, 5), True), (96, 96, (16, 16, 16), True),
    (96, 48, (24,), False), (128, 128, (16, 24, 24), False), (128, 128, (24, 20, 20), True),
    (128, 16, (0, 8), False), (256, 256, (44, 42, 42), True), (256, 128, (10, 20, 30, 4), False),
    (256, 256, (35, 31, 31, 31), True), (80, 80, (16, 12, 12), False)])
def test_rope(D, rot, sections, inter, dtype):
    rope_case(D + rot, 5, 6, 2, D, rot, sections, dtype, inter)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (1, 1, 0), (3, 0, 2), (257, 7, 3), (2, 128, 8),
                                     (2, 200, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_shapes(n, hq, hk, in_place, dtype):
    rope_case(n, n, hq, hk, 128, 96, (16, 16, 16), dtype, in_place=in_place, fused=not in_place)
    rope_case(n, n, hq, hk, 128, 96, (16, 16, 16), dtype, in_place=in_place)


@pytest.mark.parametrize("theta", [1.0, 0.5, 500000.0, 1e6])
def test_rope_bases_and_directions(theta):
    rope_case(1, 9, 2, 1, 128, 128, (64,), "f32", theta=theta, top=1 << 14)
    rope_case(2, 9, 2, 1, 128, 128, (64,), "f32", theta=theta, top=1 << 14, inverse=True)


def test_rope_far_positions():
    # Any int32: the angle is reduced in 64-bit integers.  (The fp64 reference itself is off by
    # 2^-53 of the angle, 2^-22 at 2^31.)
    rope_case(3, 50, 2, 1, 128, 128, (20, 22, 22), "f32", top=(1 << 31) - 1)
    rope_case(4, 50, 2, 1, 64, 64, (32,), "f32", top=1 << 24, theta=500000.0)


PI_60 = "3.14159265358979323846264338327950288419716939937510582097494"


@pytest.mark.parametrize("theta,rot", [(10000.0, 128), (500000.0, 128), (1e6, 256), (10000.0, 96),
                                       (2.0, 16)])
@pytest.mark.parametrize("sign", [1, -1])
def test_rope_far_positions_are_turned_to_the_last_bit(theta, rot, sign):
    """For each pair a position near 2^31 whose angle is almost a whole number of turns: its sine is
    small, so fp32 hides nothing of what the angle is off by.  The frequencies are taken from 60
    digits; 2^-65 of a turn of theirs times 2^31 positions, and the angle's 32 bits, are 2^-31.7 of
    a turn; the sine itself is good to 2^-21."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    half = rot // 2
    ln = Decimal(theta).ln()
    freq = [int(((ln * Decimal(-2 * i) / Decimal(rot)).exp() / (2 * Decimal(PI_60)) *
                 Decimal(2) ** 64).to_integral_value()) for i in range(half)]
    near = np.arange(2 ** 31 - 2 ** 23, 2 ** 31, dtype=np.uint64)
    pos, turns = [], []
    for f in freq:
        t = (near * np.uint64(f)).view(np.int64)  # modulo 2^64: signed fractions of a turn
        j = int(np.argmin(np.abs(t)))
        pos.append(int(near[j]))
        turns.append(int(t[j]) / 2.0 ** 64)
    x = torch.zeros(half, 1, rot, device="cuda")
    x[:, :, :half] = torch.eye(half, device="cuda")[:, None]  # token i: only pair i
    pa.pa_rope_axes(x, None, i32([[sign * p for p in pos]]), (half,), theta)
    got = x[torch.arange(half), 0, half + torch.arange(half)].double().cpu().numpy()
    want = np.sin(2 * np.pi * sign * np.array(turns))
    assert np.abs(want).max() < 0.01
    assert (np.abs(got - want) <= 2 * np.pi * 2.0 ** -31.7 + np.abs(want) * 2.0 ** -21).all(), \
        np.abs(got - want).max()


def test_rope_backward_is_the_inverse():
    # A rotation's transpose is its inverse: against the formula and against differences.
    g = np.random.default_rng(9)
    n, H, D, sections = 6, 3, 64, (8, 12, 12)
    x, up = g.standard_normal((n, H, D)), g.standard_normal((n, H, D))
    pos = g.integers(0, 5000, (3, n))
    gx = torch.from_numpy(up).float().cuda()
    pa.pa_rope_axes(gx, None, i32(pos), sections, 10000.0, inverse=True)
    got = gx.double().cpu().numpy()
    step = 1e-6
    for _ in range(40):  # differences of sum(up * rope(x))
        i, h, d = g.integers(n), g.integers(H), g.integers(D)
        e = np.zeros_like(x)
        e[i, h, d] = step
        diff = ((ref.rope(x + e, pos, sections, 10000.0, D) -
                 ref.rope(x - e, pos, sections, 10000.0, D)) * up).sum() / (2 * step)
        assert abs(diff - got[i, h, d]) <= 1e-5
    back = torch.from_numpy(x).float().cuda()
    pa.pa_rope_axes(back, None, i32(pos), sections, 10000.0)
    # <rope(x), up> == <x, back(up)> in the kernel's own arithmetic
    assert abs(float((back.double() * torch.from_numpy(up).cuda()).sum()) - (x * got).sum()) <= 1e-3
    pa.pa_rope_axes(back, None, i32(pos), sections, 10000.0, inverse=True)
    assert np.abs(back.double().cpu().numpy() - x).max() <= 2.0 ** -18


def test_rope_refused_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    p = i32(np.zeros((3, 4)))
    for args, kw, exc in [((q, q.bfloat16(), p, (8, 12, 12), 1e4), {}, TypeError),
                          ((q, q[:3], p, (8, 12, 12), 1e4), {}, ValueError),
                          ((q, q, p[:2], (8, 12, 12), 1e4), {}, ValueError),
                          ((q, q, p.long(), (8, 12, 12), 1e4), {}, TypeError),
                          ((q, q, p, (8, 12, 13), 1e4), {}, pa.PAError),
                          ((q, q, p, (8, 12, 12), 1e4), dict(q_out=q.float()), TypeError),
                          ((q, None, p, (8, 12, 12), 1e4), dict(k_out=q), ValueError),
                          ((q.double(), None, p, (8, 12, 12), 1e4), {}, TypeError),
                          ((q.transpose(0, 1), None, p, (8, 12, 12), 1e4), {}, ValueError),
                          ((q[:, :, ::2], None, p, (8, 4, 4), 1e4), {}, ValueError)]:
        with pytest.raises(exc):
            pa.pa_rope_axes(*args, **kw)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 64), ("f16", 96), ("bf16", 256)])
@pytest.mark.parametrize("graph", [False, True])
def test_prefill_and_decode_steps_together(dtype, D, graph):
    """A prompt step of ragged requests, then single-token steps (captured once and replayed in
    one variant): tables, rotation, cache and attention follow the host's at every step."""
    g = np.random.default_rng([D, int(graph)])
    B, Hq, Hkv, maxp, pages, theta = 4, 8, 2, 12, 40, 10000.0
    sections = (D // 2 - 2 * (D // 6), D // 6, D // 6)
    order = g.permutation(pages)
    lens = np.zeros(B, np.int64)
    bt = np.full((B, maxp), -1, np.int32)
    cache_h = np.zeros((pages, Hkv, 20 * D), np.uint8)
    used = 0
    dev = dict(past=i32(lens), new=i32(lens), free=i32(order), bt=i32(bt), lens=i32(lens),
               starts=i32(np.zeros(B + 1)), taken=i32([0]), err=i32(np.zeros(64)),
               cache=torch.zeros(pages, Hkv, 20 * D, dtype=torch.uint8, device="cuda"))
    plan = pa.pa_q4_plan(B, Hq, Hkv, D, 16, pages, maxp, maxp * 16, dtype=1 if dtype == "bf16" else 0)
    ws = pa.new_workspace(plan, "cuda")
    out, lse = torch.empty(B, Hq, D, dtype=T[dtype], device="cuda"), torch.empty(B, Hq, device="cuda")

    def device_step(b):
        """The whole step on the stream: bufs b of `cap` packed rows."""
        pa.pa_extend_tables(dev["past"], dev["new"], dev["free"], pages, dev["bt"], dev["lens"],
                            dev["starts"], b["slots"], b["pos"], dev["taken"], dev["err"])
        b["pos3"].copy_(b["pos"].expand(3, -1))
        pa.pa_rope_axes(b["qkv"][:, :Hq], b["qkv"][:, Hq:Hq + Hkv], b["pos3"], sections, theta)
        pa.pa_q4_write(b["qkv"][:, Hq:Hq + Hkv], b["qkv"][:, Hq + Hkv:], b["slots"], dev["cache"],
                       dev["err"])
        last = (dev["starts"][1:] - 1).clamp(min=0).long()
        q = b["qkv"][:, :Hq].index_select(0, last)
        pa.pa_q4_decode(plan, q, dev["cache"], dev["bt"], dev["lens"], D ** -0.5, 0, out, lse, ws)
        dev["past"].copy_(dev["lens"])

    def bufs(cap):
        return dict(slots=torch.zeros(cap, dtype=torch.int64, device="cuda"), pos=i32(np.zeros(cap)),
                    pos3=i32(np.zeros((3, cap))),
                    qkv=torch.zeros(cap, Hq + 2 * Hkv, D, dtype=T[dtype], device="cuda"))

    captured = None
    single = bufs(B + 3)
    for step in range(6):
        new = np.array([40, 1, 17, 100]) if step == 0 else np.ones(B, np.int64)
        b = bufs(int(new.sum()) + 5) if step == 0 else single
        cap = b["slots"].numel()
        x = kv_values(g, (cap, Hq + 2 * Hkv, D), dtype)
        b["qkv"].copy_(to_t(x, dtype))
        dev["new"].copy_(i32(new))
        rest = order[used:]
        dev["free"][:len(rest)].copy_(i32(rest))
        torch.cuda.synchronize()
        if graph and step >= 1:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    device_step(b)
            captured.replay()
        else:
            device_step(b)
        torch.cuda.synchronize()
        # the host's step; the rotated rows are taken from the device (T's roundings), after a check
        hbt, hl, starts, slots, pos, taken, err = ref.extend_tables(
            lens, new, np.concatenate([rest, np.zeros(len(order) - len(rest), np.int64)])
            if len(rest) < len(order) else rest, pages, bt, cap)
        assert err == 0 and pa.pa_get_error_ex(dev["err"]) == 0 and pa.pa_get_error_ex(ws) == 0
        assert np.array_equal(dev["bt"].cpu().numpy(), hbt)
        assert np.array_equal(dev["lens"].cpu().numpy(), hl) and int(dev["taken"]) == taken
        assert np.array_equal(b["slots"].cpu().numpy(), slots)
        assert np.array_equal(b["pos"].cpu().numpy(), pos)
        rows = b["qkv"].double().cpu().numpy()
        want = ref.rope(x[:, :Hq + Hkv], np.stack([pos] * 3), sections, theta, D)
        assert (np.abs(rows[:, :Hq + Hkv] - want) <=
                rope_tolerance(x[:, :Hq + Hkv], want, D, dtype)).all()
        cache_h, _ = reference_cache(cache_h, rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], slots, D, dtype)
        assert np.array_equal(dev["cache"].cpu().numpy(), cache_h)
        last = starts[1:] - 1
        check((out.double().cpu().numpy(), lse.double().cpu().numpy(), 0),
              ref.decode(rows[last, :Hq], cache_h, hbt, hl, D ** -0.5, 0, dtype))
        bt, lens, used = hbt, hl.astype(np.int64), used + taken


def test_calls_without_the_marshalling_extension(monkeypatch):
    """The same calls through the Python checks alone give the same bits."""
    if q4._fast is None:
        pytest.skip("the marshalling extension is not built here")
    fast = q4._fast
    g = np.random.default_rng(50)
    D, H, n = 128, 2, 40
    rows = to_t(kv_values(g, (n, 3 * H, D), "f16"), "f16")
    results = []
    for ext in (fast, None):
        monkeypatch.setattr(q4, "_fast", ext)
        past, new = i32([0, 0]), i32([33, 7])
        bt, lens, starts, taken = i32(np.full((2, 4), -1)), i32([0, 0]), i32([0, 0, 0]), i32([0])
        slots, pos = torch.zeros(n, dtype=torch.int64, device="cuda"), i32(np.zeros(n))
        pa.pa_extend_tables(past, new, i32([5, 1, 4, 2]), 6, bt, lens, starts, slots, pos, taken)
        x = rows.clone()
        pa.pa_rope_axes(x[:, :H], x[:, H:2 * H], pos.expand(2, -1).contiguous(), (32, 32), 1e4)
        cache = pa.new_q4_cache(6, H, D)
        pa.pa_q4_write(x[:, H:2 * H], x[:, 2 * H:], slots, cache)
        k, v = torch.empty(n, H, D, dtype=torch.float16, device="cuda"), torch.empty(
            n, H, D, dtype=torch.float16, device="cuda")
        pa.pa_q4_read(cache, slots, k, v)
        plan = pa.pa_q4_plan(2, H, H, D, 16, 6, 4, 64)
        q = x[[32, 39], :H].contiguous()
        out, lse = torch.empty_like(q), torch.empty(2, H, device="cuda")
        pa.pa_q4_decode(plan, q, cache, bt, lens, 0.1, 0, out, lse, pa.new_workspace(plan, "cuda"))
        results.append([t.clone() for t in (bt, lens, starts, slots, pos, taken, x, cache, k, v, out,
                                            lse)])
    assert int(results[0][5]) == 4
    for a, b in zip(*results):
        assert torch.equal(a, b)
