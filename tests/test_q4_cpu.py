"""Host-side tests of include/pa_q4.h (no GPU): the reference the GPU tests use
is checked against properties of the definitions, plans and argument checks
return before anything is launched, and the ctypes mirror follows the header."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q4_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q4
from paged_kv_gqa_pa_gb300 import build as pa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return q4._lib()


def test_plan_struct_layout_matches_header():
    text = open(os.path.join(ROOT, "include", "pa_q4.h")).read()
    body = re.search(r"typedef struct pa_q4_plan \{(.*?)\} pa_q4_plan_t;", text, flags=re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"\b(?:int|size_t|float)\s+([a-z_0-9]+)\s*;", body)
    assert fields == [f for f, _ in q4.pa_q4_plan_t._fields_]
    assert q4.pa_q4_plan_t.workspace_bytes.offset == 56
    assert ctypes.sizeof(q4.pa_q4_plan_t) == 80


def test_page_bytes():
    assert [pa.pa_q4_page_bytes(d) for d in (64, 96, 128, 256)] == [1280, 1920, 2560, 5120]
    assert [pa.pa_q4_page_bytes(d) for d in (0, -64, 32, 80, 512)] == [0] * 5


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_layout_covers_the_block_once_and_tokens_own_their_bytes(D):
    owner = {}
    nib = set()
    for r in range(16):
        for d in range(D):
            for place in (ref.k_place, ref.v_place):
                at, sh = place(D, r, d)
                assert (at, sh) not in nib and 0 <= at < 16 * D
                nib.add((at, sh))
                assert owner.setdefault(at, r) == r
        for n in range(D // 32):
            for cell in (ref.k_cell, ref.v_cell):
                for at in cell(D, r, n):
                    assert at % 2 == 0 and 16 * D <= at < 20 * D
                    assert owner.setdefault(at, r) == r and owner.setdefault(at + 1, r) == r
    assert len(nib) == 32 * D and len(owner) == 20 * D


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantisation_error_is_about_half_a_step(dtype):
    g = np.random.default_rng(1)
    grid = {"f16": 1 / 64, "bf16": 1 / 8}[dtype]
    for _ in range(200):
        x = ref.rn(g.standard_normal(32) * 10.0 ** g.uniform(-2, 2), dtype)
        c, s, z = ref.quantise(x, dtype)
        assert x.min() < 0 < x.max()
        got = ref.values(c, s, z, dtype)
        # half a step, the grid's shift, and the value's rounding
        assert (np.abs(got - x) <= s[0] * (0.5 + grid) + ref.HALF_STEP[dtype] * np.abs(got)).all()


def test_quantisation_corners():
    for dtype in ("f16", "bf16"):
        c, s, z = ref.quantise(np.full(32, 3.5), dtype)       # constant: exact
        assert s[0] == 0 and (ref.values(c, s, z, dtype) == 3.5).all()
        x = np.zeros(32)
        x[3] = np.nan
        assert np.isnan(ref.values(*ref.quantise(x, dtype), dtype)).all()
        x[3] = np.inf                                           # saturates at the limit
        got = ref.values(*ref.quantise(x, dtype), dtype)
        assert np.isfinite(got).all() and got[3] == got.max() > 0.9 * ref.LIMIT[dtype]


def _plan(**kw):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=64,
             max_pages_per_seq=16, max_context_len=256, window=0, num_sms=152, dtype=0)
    a.update(kw)
    return pa.pa_q4_plan(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(num_q_heads=7), binding.PA_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), binding.PA_ERR_INVALID_ARG),
    (dict(batch=-1), binding.PA_ERR_INVALID_ARG),
    (dict(max_context_len=257), binding.PA_ERR_INVALID_ARG),
    (dict(max_context_len=-1), binding.PA_ERR_INVALID_ARG),
    (dict(window=-1), binding.PA_ERR_INVALID_ARG),
    (dict(num_pages=0), binding.PA_ERR_INVALID_ARG),
    (dict(dtype=5), binding.PA_ERR_INVALID_ARG),
    (dict(num_sms=-1), binding.PA_ERR_INVALID_ARG),
    (dict(dtype=binding.PA_DTYPE_F32), binding.PA_ERR_UNSUPPORTED),
    (dict(head_dim=80), binding.PA_ERR_UNSUPPORTED),
    (dict(page_size=32, max_pages_per_seq=8), binding.PA_ERR_UNSUPPORTED),
    (dict(batch=4097), binding.PA_ERR_UNSUPPORTED),
    (dict(num_q_heads=22, num_kv_heads=2), binding.PA_ERR_UNSUPPORTED),  # g = 11
    (dict(batch=4096, max_pages_per_seq=1 << 20, max_context_len=1 << 24),
     binding.PA_ERR_UNSUPPORTED),
])
def test_plan_rejects(kw, status):
    with pytest.raises(pa.PAError) as e:
        _plan(**kw)
    assert e.value.status == status


def test_plan_fields():
    p = _plan(batch=64, num_q_heads=32, num_kv_heads=8, max_context_len=4096,
              max_pages_per_seq=256, num_pages=20000)
    assert p.heads_per_cta == 4 and 152 <= p.ctas == p.ctas_per_group * 8 <= 4 * 152
    # two partials per CTA: o, maximum and sum of up to 8 heads
    assert p.workspace_bytes >= p.ctrl_bytes + p.ctas * 2 * 8 * (128 + 2) * 4
    assert p.ctrl_bytes >= 256 + 8 * 64 * 4
    # sixteen query heads per KV head: two chunks
    p = _plan(num_q_heads=32, num_kv_heads=2)
    assert p.heads_per_cta == 8 and p.ctas == p.ctas_per_group * 4
    # no more CTAs than give each of their four warps two pages
    assert _plan(batch=1, max_context_len=100).ctas_per_group == 1
    assert _plan(batch=0).ctas_per_group >= 1


FAKE = 1 << 20  # aligned, never dereferenced: every call below is refused on the host


def test_decode_checks_return_before_launch(lib):
    plan = _plan()
    base = [ctypes.byref(plan), FAKE, FAKE, FAKE, FAKE, 1.0, 0, FAKE, FAKE, FAKE, None]
    IA, WS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_WORKSPACE

    def call(**at):
        a = list(base)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.pa_q4_decode(*a)

    assert call(_0=None) == IA
    for i in (1, 2, 3, 4, 7, 8):
        assert call(**{f"_{i}": None}) == IA
    for i in (1, 2, 7, 9):
        assert call(**{f"_{i}": FAKE + 8}) == IA
    assert call(_9=None) == WS
    assert call(_6=5) == IA  # another window than the plan's
    for field, value, st in [("heads_per_cta", 3, IA), ("heads_per_cta", 0, IA),
                             ("ctas_per_group", 0, IA), ("workspace_bytes", 256, IA),
                             ("ctrl_bytes", 256, IA), ("test_stall_bytes", 5000, IA),
                             ("num_q_heads", 9, IA), ("head_dim", 100, binding.PA_ERR_UNSUPPORTED),
                             ("max_context_len", 1 << 20, IA),
                             ("ctas_per_group", plan.ctas_per_group + 1, IA),
                             ("cluster", 1, IA), ("cluster", 9, IA), ("cluster", -2, IA),
                             ("cluster", plan.ctas_per_group, IA)]:
        bad = q4.pa_q4_plan_t.from_buffer_copy(plan)
        setattr(bad, field, value)
        assert call(_0=ctypes.byref(bad)) == st, field
    empty = _plan(batch=0)
    assert call(_0=ctypes.byref(empty), _1=None, _2=None) == binding.PA_OK


@pytest.mark.parametrize("fn", ["pa_q4_write", "pa_q4_read"])
def test_cache_call_checks_return_before_launch(lib, fn):
    IA, UN = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED

    def call(n=4, hkv=2, D=128, ps=16, pages=8, dtype=0, k=FAKE, ks=256, v=FAKE, vs=256,
             slots=FAKE, cache=FAKE, err=None):
        if fn == "pa_q4_write":
            return lib.pa_q4_write(n, hkv, D, ps, pages, dtype, k, ks, v, vs, slots, cache, err,
                                   None)
        return lib.pa_q4_read(n, hkv, D, ps, pages, dtype, cache, slots, k, ks, v, vs, err, None)

    assert call(n=0, k=None, v=None, slots=None, cache=None) == binding.PA_OK
    for kw in (dict(n=-1), dict(hkv=0), dict(pages=0), dict(dtype=7), dict(ks=255), dict(vs=260),
               dict(ks=-256), dict(k=None), dict(v=None), dict(slots=None), dict(cache=None),
               dict(k=FAKE + 8), dict(v=FAKE + 2), dict(cache=FAKE + 4), dict(slots=FAKE + 4),
               dict(err=FAKE + 2), dict(ks=1 << 50)):
        assert call(**kw) == IA, kw
    for kw in (dict(dtype=2), dict(D=80), dict(ps=8), dict(hkv=40000, ks=1 << 30, vs=1 << 30)):
        assert call(**kw) == UN, kw


def test_tables_checks_return_before_launch(lib):
    IA, UN = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED
    names = ["past", "new", "free", "bt", "lens", "starts", "slots", "pos", "taken", "err"]
    ptr = {n: FAKE + 64 * i for i, n in enumerate(names)}

    def call(B=2, maxp=4, ps=16, pages=8, nfree=3, cap=5, **kw):
        p = dict(ptr, **kw)
        return lib.pa_extend_tables(B, maxp, ps, pages, nfree, cap, *[p[n] for n in names], None)

    for kw in (dict(B=-1), dict(maxp=0), dict(pages=0), dict(nfree=-1), dict(cap=-1)):
        assert call(**kw) == IA, kw
    for n in names[:-1]:
        assert call(**{n: None}) == IA, n
    for n in names:
        assert call(**{n: FAKE + 2}) == IA, n
    assert call(slots=FAKE + 4) == IA
    assert call(lens=ptr["past"]) == IA and call(starts=ptr["new"]) == IA
    assert call(B=8193) == UN and call(ps=8) == UN and call(maxp=1 << 27) == UN


def test_rope_checks_return_before_launch(lib):
    IA, UN = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED

    def call(n=4, hq=4, hk=2, D=128, R=128, sections=(16, 24, 24), axes=None, inter=0, inv=0,
             theta=1e4, dtype=0, q=FAKE, qs=512, k=FAKE, ks=256, pos=FAKE, qo=FAKE, qos=512,
             ko=FAKE, kos=256):
        arr = (ctypes.c_int * max(1, len(sections)))(*sections)
        return lib.pa_rope_axes(n, hq, hk, D, R, len(sections) if axes is None else axes, arr,
                                inter, inv, theta, dtype, q, qs, k, ks, pos, qo, qos, ko, kos,
                                None)

    assert call(n=0) == binding.PA_OK
    assert call(hq=0, hk=0) == binding.PA_OK
    for kw in (dict(n=-1), dict(hq=-1), dict(R=0), dict(R=144), dict(sections=(64, 1)),
               dict(sections=(65, -1)), dict(axes=0), dict(sections=(13, 13, 13, 13, 12)),
               dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")),
               dict(dtype=3), dict(inter=2), dict(inv=-1), dict(q=None), dict(ko=None),
               dict(pos=None), dict(q=FAKE + 8), dict(ko=FAKE + 2), dict(qs=508), dict(kos=264 - 4),
               dict(pos=FAKE + 2), dict(qos=520),  # in place with another stride
               dict(sections=(10, 44, 10), inter=1)):
        assert call(**kw) == IA, kw
    for kw in (dict(D=120, R=112, sections=(56,)), dict(D=512), dict(R=24, sections=(12,))):
        assert call(**kw) == UN, kw


def test_binding_refuses_host_tensors_and_wrong_arguments():
    k = torch.zeros(2, 1, 64, dtype=torch.float16)
    slots = torch.zeros(2, dtype=torch.int64)
    cache = torch.zeros(1, 1, 1280, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q4_write(k, k, slots, cache)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q4_read(cache, slots, k, k)
    with pytest.raises(TypeError):
        pa.pa_q4_write(None, k, slots, cache)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_axes(k, k, torch.zeros(1, 2, dtype=torch.int32), (32,), 1e4)
    with pytest.raises(ValueError, match="q or k"):
        pa.pa_rope_axes(None, None, None, (32,), 1e4)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_extend_tables(i, i, i, 4, i.view(1, 2), i, i, slots, i, i)
    plan = _plan()
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q4_decode(plan, k, cache, i, i, 1.0, 0, k, k, cache)
    with pytest.raises(ValueError):
        pa.new_q4_cache(1, 1, 80, "cpu")
    assert pa.new_q4_cache(3, 2, 96, "cpu").shape == (3, 2, 1920)


def test_reference_tables_by_hand():
    # 20 tokens held, 13 more: a third page; then an idle request; then a new one.
    bt = np.full((3, 4), -1, np.int32)
    bt[0, :2] = [7, 5]
    bt[1, :1] = [9]
    got = ref.extend_tables([20, 16, 0], [13, 0, 2], [3, 1, 4], 10, bt, 17)
    assert got[0].tolist() == [[7, 5, 3, -1], [9, -1, -1, -1], [1, -1, -1, -1]]
    assert got[1].tolist() == [33, 16, 2] and got[2].tolist() == [0, 13, 13, 15]
    assert got[3].tolist() == [5 * 16 + 4 + i for i in range(12)] + [48, 16, 17, -1, -1]
    assert got[4].tolist() == list(range(20, 33)) + [0, 1, 0, 0] and got[5:] == (2, 0)


def tens(dtype, shape, stride=None):
    """A CPU tensor of this form (its device, -1, is the stand-in's current one)."""
    return torch.empty(shape, dtype=dtype) if stride is None else \
        torch.empty_strided(shape, stride, dtype=dtype)


@pytest.fixture
def marshalled(lib):
    """The extension with recording stand-ins for the five C functions; yields (module, calls)."""
    if q4._fast is None:
        pytest.skip("the marshalling extension is not built here")
    calls = []
    P, i, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    protos = dict(
        write=ctypes.CFUNCTYPE(i, *[i] * 6, P, ll, P, ll, P, P, P, P),
        read=ctypes.CFUNCTYPE(i, *[i] * 6, P, P, P, ll, P, ll, P, P),
        decode=ctypes.CFUNCTYPE(i, P, P, P, P, P, ctypes.c_float, i, P, P, P, P),
        tables=ctypes.CFUNCTYPE(i, *[i] * 6, *[P] * 11),
        rope=ctypes.CFUNCTYPE(i, *[i] * 6, ctypes.POINTER(i), i, i, ctypes.c_float, i, P, ll, P, ll,
                              P, P, ll, P, ll, P))
    keep = []
    for name, proto in protos.items():
        def fn(*a, name=name):
            if name == "rope":
                a = a[:6] + ([a[6][j] for j in range(a[5])],) + a[7:]
            if name == "decode":
                a = (ctypes.string_at(a[0], ctypes.sizeof(q4.pa_q4_plan_t)),) + a[1:]
            calls.append((name, a))
            return 3 if name == "read" else 0
        keep.append(proto(fn))
    q4._fast.setup(tuple(ctypes.cast(f, P).value for f in keep), lambda: -1, lambda d: 4096 + d)
    yield q4._fast, calls
    q4._load_fast(lib)  # the real functions again


def test_marshalling_of_the_usual_calls(marshalled):
    fast, calls = marshalled
    f16, i32, i64 = torch.float16, torch.int32, torch.int64

    def at(*t):
        return tuple(x.data_ptr() for x in t)

    k = tens(f16, (5, 2, 128), (1024, 128, 1))
    v = tens(f16, (5, 2, 128))
    sl, c = tens(i64, (5,)), tens(torch.uint8, (9, 2, 2560))
    kp, vp, slp, cp = at(k, v, sl, c)
    assert fast.q4_write(k, v, sl, c) == 0
    assert calls.pop() == ("write", (5, 2, 128, 16, 9, 0, kp, 1024, vp, 256, slp, cp, None, 4095))
    assert fast.q4_read(c, sl, k, v) == 3  # the status comes back
    assert calls.pop() == ("read", (5, 2, 128, 16, 9, 0, cp, slp, kp, 1024, vp, 256, None, 4095))
    plan = _plan(dtype=1)
    bf = torch.bfloat16
    q, out = tens(bf, (2, 8, 128)), tens(bf, (2, 8, 128))
    bt, cl = tens(i32, (2, 16)), tens(i32, (2,))
    cache = tens(torch.uint8, (64, 2, 2560))
    lse, ws = tens(torch.float32, (2, 8)), tens(torch.uint8, (plan.workspace_bytes,))
    assert fast.q4_decode(plan, q, cache, bt, cl, 0.5, 7, out, lse, ws) == 0
    assert calls.pop() == ("decode", (bytes(plan), *at(q, cache, bt, cl), 0.5, 7,
                                      *at(out, lse, ws), 4095))
    t = [tens(i32, (3,)), tens(i32, (3,)), tens(i32, (11,)), 77, tens(i32, (3, 6)), tens(i32, (3,)),
         tens(i32, (4,)), tens(i64, (20,)), tens(i32, (20,)), tens(i32, (1,))]
    assert fast.extend_tables(*t) == 0
    assert calls.pop() == ("tables", (3, 6, 16, 77, 11, 20, *at(*t[:3], *t[4:]), None, 4095))
    f32 = torch.float32
    q, k = tens(f32, (5, 4, 64)), tens(f32, (5, 2, 64), (512, 64, 1))
    o = tens(f32, (5, 2, 64))
    pos = tens(i32, (3, 5))
    qp, kp, op, pp = at(q, k, o, pos)
    assert fast.rope_axes(q, k, pos, (4, 6, 6), 1e4, None, o, 32, True, False) == 0
    assert calls.pop() == ("rope", (5, 4, 2, 64, 32, 3, [4, 6, 6], 1, 0, 1e4, 2, qp, 256, kp, 512, pp,
                                    qp, 256, op, 128, 4095))
    assert fast.rope_axes(q, k, pos, (4, 6, 6), 1e4, None, None, None, False, True) == 0
    assert calls.pop()[1][4:9] == (64, 3, [4, 6, 6], 0, 1)
    assert not calls
    fast.setup((1, 2, 3, 4, 5), lambda: 0, lambda d: 4096)  # another device is the current one
    assert fast.rope_axes(q, k, pos, (4, 6, 6), 1e4, None, o, 32, True, False) is None


def test_marshalling_leaves_everything_else_alone(marshalled):
    fast, calls = marshalled
    f16, i32, i64 = torch.float16, torch.int32, torch.int64
    ok = dict(k=tens(f16, (5, 2, 128)), v=tens(f16, (5, 2, 128)),
              sl=tens(i64, (5,)), c=tens(torch.uint8, (9, 2, 2560)))
    for name, bad in [("k", None), ("k", 3),
                      ("k", tens(f16, (5, 256))), ("k", tens(i32, (5, 2, 128))),
                      ("k", tens(f16, (5, 2, 128), (256, 1, 2))),
                      ("v", tens(f16, (5, 2, 128), (64, 640, 1))),
                      ("v", tens(torch.bfloat16, (5, 2, 128))),
                      ("v", tens(f16, (4, 2, 128))),
                      ("sl", tens(i32, (5,))), ("sl", tens(i64, (6,))),
                      ("sl", tens(i64, (5,), (2,))), ("v", tens(f16, (5, 2, 128)).to_sparse()),
                      ("v", torch.empty((5, 2, 128), dtype=f16, device="meta")),
                      ("v", np.zeros((5, 2, 128), np.float16)),
                      ("c", tens(torch.uint8, (9, 3, 2560))),
                      ("c", tens(torch.uint8, (9, 2, 1280))),
                      ("c", tens(torch.int8, (9, 2, 2560)))]:
        a = dict(ok, **{name: bad})
        assert fast.q4_write(a["k"], a["v"], a["sl"], a["c"]) is None, (name, bad)
        assert fast.q4_read(a["c"], a["sl"], a["k"], a["v"]) is None, (name, bad)
    plan = _plan()
    base = [plan, tens(f16, (2, 8, 128)), tens(torch.uint8, (64, 2, 2560)),
            tens(i32, (2, 16)), tens(i32, (2,)), 0.5, 0,
            tens(f16, (2, 8, 128)), tens(torch.float32, (2, 8)),
            tens(torch.uint8, (plan.workspace_bytes,))]
    assert fast.q4_decode(*base) == 0
    calls.clear()
    for i, bad in [(0, object()), (0, b"x" * 8), (1, tens(f16, (3, 8, 128))), (5, 1), (5, "a"),
                   (6, 0.0), (6, 1 << 40), (6, True), (8, tens(f16, (2, 8))),
                   (9, tens(torch.uint8, (plan.workspace_bytes - 1,))),
                   (9, tens(torch.uint8, (1, plan.workspace_bytes))),
                   (2, tens(torch.uint8, (63, 2, 2560)))]:
        a = list(base)
        a[i] = bad
        assert fast.q4_decode(*a) is None, (i, bad)
    assert fast.q4_decode(*base[:9]) is None and fast.extend_tables(1, 2) is None
    f32 = torch.float32
    r = [tens(f32, (5, 4, 64)), tens(f32, (5, 2, 64)), tens(i32, (3, 5)),
         (4, 6, 6), 1e4, None, None, None, False, False]
    for i, bad in [(0, None), (1, None), (1, tens(f32, (4, 2, 64))),
                   (1, tens(f16, (5, 2, 64))), (2, tens(i32, (2, 5))),
                   (3, [4, 6, 6]), (3, (1, 2, 3, 4, 5)), (3, (4.0, 6, 6)), (3, ()), (4, 10000),
                   (5, tens(f32, (5, 2, 64))), (7, 32.0), (8, 1), (9, None)]:
        a = list(r)
        a[i] = bad
        assert fast.rope_axes(*a) is None, (i, bad)
    assert not calls


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [0, 1])
def test_plan_clusters(D, dtype):
    """Clusters share sequences of medium length; short, very long and many ones go without."""
    for batch, tokens, want in [(1, 128, False), (1, 1000, True), (4, 1000, True),
                                (2, 100000, False), (400, 1000, False), (0, 1000, False)]:
        plan = q4.pa_q4_plan(batch, 16, 4, D, 16, 1 << 16, 6250, tokens, 0, 152, dtype)
        assert (plan.cluster != 0) == want, (batch, tokens)
        if want:
            assert 2 <= plan.cluster <= 8
            assert plan.ctas_per_group == plan.cluster * batch
            assert plan.ctas == plan.ctas_per_group * 4


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("batch,tokens", [(1, 20), (1, 1000), (4, 4000), (4, 100000), (300, 500)])
def test_plan_with_a_window_that_holds_everything(batch, tokens, D):
    """A window of the longest length or more, up to the largest int, plans like no window."""
    want = _plan(batch=batch, num_q_heads=24, num_kv_heads=4, head_dim=D, max_pages_per_seq=6250,
                 max_context_len=tokens)
    for window in (tokens + 16, 1 << 20, INT_MAX - 15, INT_MAX - 14, INT_MAX):
        got = _plan(batch=batch, num_q_heads=24, num_kv_heads=4, head_dim=D, max_pages_per_seq=6250,
                    max_context_len=tokens, window=window)
        assert (got.ctas_per_group, got.ctas, got.cluster) == (want.ctas_per_group, want.ctas,
                                                               want.cluster), window
        assert got.workspace_bytes == want.workspace_bytes


def test_plan_of_the_longest_lengths(lib):
    # Lengths rounded up to whole pages have to fit an int.
    long = dict(batch=1, max_pages_per_seq=1 << 27)
    whole = _plan(**long, max_context_len=1 << 30)
    assert whole.ctas_per_group > 100
    assert _plan(**long, max_context_len=2 ** 31 - 16).ctas_per_group == whole.ctas_per_group
    few = _plan(**long, max_context_len=2 ** 31 - 16, window=100)
    assert few.ctas_per_group == _plan(max_context_len=256, window=100, batch=1).ctas_per_group
    for tokens in (2 ** 31 - 15, INT_MAX):
        for window in (0, 100):
            with pytest.raises(pa.PAError) as e:
                _plan(**long, max_context_len=tokens, window=window)
            assert e.value.status == binding.PA_ERR_UNSUPPORTED
    few.max_context_len = INT_MAX  # an edited plan
    assert lib.pa_q4_decode(ctypes.byref(few), FAKE, FAKE, FAKE, FAKE, 1.0, 100, FAKE, FAKE, FAKE,
                            None) == binding.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_the_grids_ends_move_no_further_than_the_header_says(dtype):
    text = open(os.path.join(ROOT, "include", "pa_q4.h")).read()
    name = {"f16": "fp16", "bf16": "bf16"}[dtype]
    low, high = re.search(name + r": s / (\d+) at the low end, s / (\d+) at the high end", text).groups()
    g = np.random.default_rng(2)
    worst = [0.0, 0.0]
    for i in range(60000):
        mn, mx = -g.uniform(0.001, 1), g.uniform(0.001, 1)
        if i % 3 == 0:  # a greatest element just above zero: z is largest there
            mx = 10.0 ** g.uniform(-6, -2)
        mn, mx = (float(ref.rn(v * 2.0 ** g.integers(-3, 8), dtype)) for v in (mn, mx))
        s = float(ref.rn((mx - mn) / 15, dtype))
        z = float(ref.rn(mn - 16 * s, dtype))
        if s < 2.0 ** -14:
            continue
        worst = [max(worst[0], abs(z + 16 * s - mn) / s), max(worst[1], abs(z + 31 * s - mx) / s)]
    assert worst[0] <= 1 / int(low) and worst[1] <= 1 / int(high), worst
    # ... and not much less far
    assert worst[0] > 0.7 / int(low) and worst[1] > 0.7 / int(high), worst


@pytest.fixture
def build_tree(tmp_path, monkeypatch):
    """build.py over copies of the extension's sources, a torch of its own and an empty _build."""
    for name in ("pa_pyfast.cpp", "pa.h", "pa_q4.h"):
        (tmp_path / name).write_text("// " + name)
    fake = tmp_path / "torch"
    fake.mkdir()
    (fake / "version.py").write_text("__version__ = '1.0'")
    monkeypatch.setattr(pa_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(pa_build, "PYFAST_SRC", str(tmp_path / "pa_pyfast.cpp"))
    monkeypatch.setattr(pa_build, "PYFAST_HEADERS", [str(tmp_path / "pa.h"), str(tmp_path / "pa_q4.h")])
    monkeypatch.setattr(pa_build, "_torch_dir", lambda: str(fake))
    (tmp_path / "_build").mkdir()
    return tmp_path


def test_an_extension_of_other_sources_or_another_torch_is_not_loaded(build_tree, lib):
    for changed in ("pa_pyfast.cpp", "pa.h", "pa_q4.h", os.path.join("torch", "version.py")):
        there = pa_build.pyfast_path()
        with open(there, "w") as f:  # (loading it would be an error)
            f.write("an extension of the sources as they were")
        with open(build_tree / changed, "a") as f:
            f.write("\n# changed")
        assert pa_build.pyfast_path() != there, changed
        assert q4._load_fast(lib) is None, changed
    os.remove(build_tree / "torch" / "version.py")
    assert pa_build.pyfast_path() is None and q4._load_fast(lib) is None


def test_a_stale_extension_goes_even_where_none_can_be_built(build_tree, monkeypatch):
    old = [build_tree / "_build" / n for n in ("_pa_fast.so", "_pa_fast-0123456789abcdef.so")]
    for path in old:
        path.write_text("")
    current = pa_build.pyfast_path()
    open(current, "w").close()
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(pa_build.shutil, "which", lambda name: None)
    assert pa_build._start_pyfast(False, False) is None
    assert not any(p.exists() for p in old) and os.path.exists(current)


def test_outputs_on_one_another_are_refused(lib):
    IA = binding.PA_ERR_INVALID_ARG
    assert lib.pa_q4_read(4, 2, 128, 16, 8, 0, FAKE, FAKE, FAKE, 256, FAKE, 256, None, None) == IA
    arr = (ctypes.c_int * 1)(64)

    def rope(q, k, qo, ko):
        return lib.pa_rope_axes(4, 2, 2, 128, 128, 1, arr, 0, 0, 1e4, 0, q, 256, k, 256, FAKE, qo, 256,
                                ko, 256, None)

    assert rope(FAKE, FAKE, FAKE, FAKE) == IA  # the same rows as q and as k, in place
    assert rope(FAKE, FAKE + 4096, FAKE + 8192, FAKE + 8192) == IA


def test_plan_cuts_head_groups_into_the_fewest_equal_chunks():
    for g in range(1, 65):
        chunks = [n for n in range(1, g) if g % n == 0 and g // n <= 8] or ([1] if g == 1 else [])
        if chunks:
            assert _plan(num_q_heads=2 * g, num_kv_heads=2).heads_per_cta == g // chunks[0], g
        else:  # 11, 13, 17, ...
            with pytest.raises(pa.PAError) as e:
                _plan(num_q_heads=2 * g, num_kv_heads=2)
            assert e.value.status == binding.PA_ERR_UNSUPPORTED


def test_decode_refuses_words_that_are_not_aligned(lib):
    plan = _plan()
    for i in (3, 4, 8):  # block_tables, context_lens, lse
        for off in (1, 2, 3):
            a = [ctypes.byref(plan), FAKE, FAKE, FAKE, FAKE, 1.0, 0, FAKE, FAKE, FAKE, None]
            a[i] += off
            assert lib.pa_q4_decode(*a) == binding.PA_ERR_INVALID_ARG, i


def test_a_stale_extension_that_another_build_has_removed(build_tree, monkeypatch):
    gone = str(build_tree / "_build" / "_pa_fast-0123456789abcdef.so")
    monkeypatch.setattr(pa_build.glob, "glob", lambda pattern: [gone])
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(pa_build.shutil, "which", lambda name: None)
    assert pa_build._start_pyfast(False, False) is None
