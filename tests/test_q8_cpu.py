"""Host-side tests of include/pa_q8.h (no GPU): the reference the GPU tests use
is checked against properties of the definitions, plans and argument checks
return before anything is launched, and the ctypes mirror follows the header."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
import q8_reference as ref
from paged_kv_gqa_pa_gb300 import binding, q8
from paged_kv_gqa_pa_gb300 import build as pa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
IA, UN, WS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED, binding.PA_ERR_WORKSPACE
FAKE = 1 << 20  # aligned, never dereferenced: every call below is refused on the host


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return q8._lib()


def test_plan_struct_layout_matches_header():
    text = open(os.path.join(ROOT, "include", "pa_q8.h")).read()
    body = re.search(r"typedef struct pa_q8_plan \{(.*?)\} pa_q8_plan_t;", text, flags=re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"\b(?:int|size_t|float)\s+([a-z_0-9]+)\s*;", body)
    assert fields == [f for f, _ in q8.pa_q8_plan_t._fields_]
    assert q8.pa_q8_plan_t.workspace_bytes.offset == 64
    assert ctypes.sizeof(q8.pa_q8_plan_t) == 80
    assert int(re.search(r"PA_DEVERR_BAD_TOKEN (\d+)u", text).group(1)) == q8.PA_DEVERR_BAD_TOKEN
    assert int(re.search(r"PA_VERIFY_MAX_DRAFTS (\d+)", text).group(1)) == q8.PA_VERIFY_MAX_DRAFTS


# ---------------------------------------------------------------- the reference

def test_reference_codes_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes.double().numpy(), ref.E4M3)
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal(4000) * 10.0 ** g.uniform(-4, 2, 4000),
                        ref.E4M3[:127], (ref.E4M3[:126] + ref.E4M3[1:127]) / 2, [-0.0, 448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_code(x), want)
    assert (ref.e4m3_code([np.nan, np.inf, -np.inf]) & 127 == 127).all()


def test_reference_scales_are_the_least_powers_of_two():
    for a in (1.0, 448.0, 448.0001, 449, 1e-30, 3e38, 0.875, 0.8751):
        s = ref.scale_for(a)
        assert a <= 448 * s and (a > 224 * s) and np.log2(s) == round(np.log2(s))
    assert ref.scale_for(0.0) == 2.0 ** -120 == ref.scale_for(1e-38)


def test_reference_append_in_pieces_is_append_at_once():
    # but for values below the raised scale's least normal, which round twice
    g = np.random.default_rng(2)
    rows = g.standard_normal((40, 2, 64)) * np.exp(g.standard_normal((40, 1, 1)))
    whole, pieces = ref.Cache(4, 2, 64), ref.Cache(4, 2, 64)
    slots = np.arange(5, 45)
    first = np.zeros((5, 2, 64))
    for c in (whole, pieces):
        c.append(first, np.arange(5))
    whole.append(rows, slots)
    at = 0
    for n in (1, 3, 7, 1, 1, 16, 11):
        pieces.append(rows[at:at + n], slots[at:at + n])
        at += n
    np.testing.assert_array_equal(whole.scales[:3], pieces.scales[:3])
    a, b = whole.values()[:2], pieces.values()[:2]
    assert (np.abs(a - b) <= whole.scales[:2, :, None, None] * 2.0 ** -10).all()
    err = np.abs(whole.values().transpose(0, 2, 1, 3).reshape(-1, 2, 64)[5:45] - rows)
    sc = np.repeat(whole.scales, 16, 0)[5:45][..., None]
    assert (err <= sc * ref.e4m3_step(rows / sc) / 2 * (1 + 1e-12)).all()


def test_reference_verify_keeps_the_targets_distribution():
    # Over a grid of random numbers the first token out has the target's probabilities.
    g = np.random.default_rng(3)
    V, n = 5, 400
    p = g.dirichlet(np.ones(V)).astype(np.float32)
    q = g.dirichlet(np.ones(V)).astype(np.float32)
    counts = np.zeros(V)
    us = (np.arange(n) + 0.5) / n
    for x in range(V):
        for u in us:
            acc, tok, bad = ref.verify(np.stack([p, p])[None].astype(float), q[None, None].astype(float),
                                       np.array([[x]]), None, np.array([[u]]), np.array([0.5]))
            assert not bad
            if acc[0] == 1:
                counts[tok[0, 0]] += q[x] / n
            else:  # the residual draw, over its own grid
                w = np.maximum(p - q, 0)
                counts += q[x] / n * w / w.sum()
    assert np.abs(counts - p / p.sum()).max() < 2 / n


# ---------------------------------------------------------------- plans

def _plan(**kw):
    a = dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=64,
             max_pages_per_seq=16, max_context_len=256, window=0, max_query_len=1, num_sms=152,
             dtype=0)
    a.update(kw)
    return pa.pa_q8_plan(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), IA), (dict(num_q_heads=0), IA), (dict(num_q_heads=9), IA),
    (dict(num_kv_heads=0), IA), (dict(head_dim=0), IA), (dict(num_pages=0), IA),
    (dict(max_pages_per_seq=0), IA), (dict(max_context_len=257), IA), (dict(window=-1), IA),
    (dict(max_query_len=0), IA), (dict(dtype=3), IA), (dict(num_sms=-1), IA),
    (dict(max_query_len=17), UN), (dict(dtype=2), UN), (dict(head_dim=80), UN),
    (dict(page_size=8, max_context_len=100), UN), (dict(batch=4097), UN),
    (dict(num_pages=1 << 27), UN),
    (dict(max_pages_per_seq=1 << 27, max_context_len=2 ** 31 - 15, batch=1), UN),
    (dict(max_pages_per_seq=1 << 26, max_context_len=1 << 30, batch=32), UN)])
def test_plan_rejects(kw, status):
    with pytest.raises(pa.PAError) as e:
        _plan(**kw)
    assert e.value.status == status


def test_plan_heads_and_tiles():
    for g, T, D, G in [(1, 1, 128, 1), (32, 1, 128, 32), (33, 1, 64, 11), (64, 1, 128, 32),
                       (8, 4, 128, 8), (8, 5, 128, 4), (4, 5, 128, 4), (3, 16, 128, 1),
                       (17, 1, 256, 1), (16, 1, 256, 16), (6, 5, 256, 3), (31, 2, 96, 1)]:
        p = _plan(num_q_heads=g * 2, head_dim=D, max_query_len=T)
        assert p.heads_per_cta == G, (g, T, D)
        assert G * T <= (16 if D == 256 else 32) and g % G == 0
        assert p.ctas == p.ctas_per_group * 2 * (g // G)
    assert _plan(batch=1, max_context_len=100).ctas_per_group == 1
    assert _plan(batch=0).ctas_per_group >= 1


def test_plan_with_a_window_that_holds_everything():
    for w in (1 << 20, 2 ** 31 - 1, 2 ** 31 - 8):
        for T in (1, 5):
            a, b = _plan(window=w, max_query_len=T), _plan(window=0, max_query_len=T)
            assert a.ctas == b.ctas and a.workspace_bytes == b.workspace_bytes


def test_plan_of_the_longest_lengths():
    p = _plan(batch=1, num_pages=1000, max_pages_per_seq=(2 ** 31 - 16) // 16,
              max_context_len=2 ** 31 - 16)
    assert p.ctas_per_group > 1 and p.cluster == 0


# ---------------------------------------------------------------- refusals

def test_decode_checks_return_before_launch(lib):
    plan = _plan()
    base = [ctypes.byref(plan), 4] + [FAKE + 64 * i for i in range(8)] + [1.0, 0, FAKE, FAKE, FAKE,
                                                                         None]

    def call(**at):
        a = list(base)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.pa_q8_decode(*a)

    assert call(_0=None) == IA and call(_1=-1) == IA
    assert call(_1=3, _3=None) == IA  # fewer rows than sequences without starts
    for i in (2, 4, 5, 6, 7, 8, 9, 12, 13):
        assert call(**{f"_{i}": None}) == IA, i
    for i in (2, 4, 5, 12, 14):
        assert call(**{f"_{i}": FAKE + 8}) == IA, i
    for i in (3, 6, 7, 8, 9, 13):
        assert call(**{f"_{i}": FAKE + 2}) == IA, i
    assert call(_14=None) == WS
    assert call(_11=5) == IA  # another window than the plan's
    for field, value, st in [("heads_per_cta", 3, IA), ("heads_per_cta", 0, IA),
                             ("ctas_per_group", 0, IA), ("workspace_bytes", 256, IA),
                             ("ctrl_bytes", 256, IA), ("test_stall_bytes", 5000, IA),
                             ("num_q_heads", 9, IA), ("head_dim", 100, UN),
                             ("max_query_len", 0, IA), ("max_query_len", 16, IA),
                             ("max_query_len", 17, UN), ("max_context_len", 1 << 20, IA),
                             ("ctas_per_group", plan.ctas_per_group + 1, IA),
                             ("cluster", 1, IA), ("cluster", 9, IA), ("cluster", -2, IA),
                             ("cluster", plan.ctas_per_group, IA)]:
        bad = q8.pa_q8_plan_t.from_buffer_copy(plan)
        setattr(bad, field, value)
        assert call(_0=ctypes.byref(bad)) == st, field
    empty = _plan(batch=0)
    assert call(_0=ctypes.byref(empty), _2=None, _4=None) == binding.PA_OK
    assert call(_1=0, _2=None) == binding.PA_OK


@pytest.mark.parametrize("fn", ["pa_append", "pa_q8_append"])
def test_append_checks_return_before_launch(lib, fn):
    names = ["q", "qs", "k", "ks", "v", "vs", "qn", "kn", "pos", "slots", "qo", "qos", "kc", "vc"]
    at = {n: FAKE + 4096 * i for i, n in enumerate(names)}
    at.update(qs=512, ks=256, vs=256, qos=512, qo=FAKE + (1 << 16))

    def call(n=4, hq=4, hkv=2, D=128, R=128, ps=16, pages=8, dtype=0, theta=1e4, eps=1e-6, err=None,
             sc=FAKE, sv=FAKE + 64, **kw):
        a = dict(at, **kw)
        tail = [sc, sv] if fn == "pa_q8_append" else []
        return getattr(lib, fn)(n, hq, hkv, D, R, ps, pages, dtype, theta, eps,
                                *[a[x] for x in names], *tail, err, None)

    none = {x: None for x in ("q", "k", "v", "qn", "kn", "pos", "slots", "qo", "kc", "vc")}
    assert call(n=0, **none) == binding.PA_OK
    for kw in (dict(n=-1), dict(hq=-1), dict(hkv=0), dict(D=0), dict(ps=0), dict(pages=0),
               dict(dtype=7), dict(theta=-1.0), dict(theta=float("nan")), dict(theta=float("inf")),
               dict(R=0), dict(R=144), dict(R=-16), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(ks=255), dict(vs=252), dict(qs=504), dict(qos=516),
               dict(ks=-256), dict(ks=1 << 50), dict(q=None), dict(k=None), dict(v=None),
               dict(slots=None), dict(kc=None), dict(vc=None), dict(qo=None), dict(pos=None),
               dict(k=FAKE + 8), dict(v=FAKE + 2), dict(q=FAKE + 4), dict(qo=FAKE + 8),
               dict(kc=FAKE + 8), dict(vc=FAKE + 1), dict(qn=FAKE + 8), dict(kn=FAKE + 4),
               dict(pos=FAKE + 2), dict(slots=FAKE + 4), dict(err=FAKE + 2),
               dict(kc=at["vc"]), dict(kc=at["k"]), dict(vc=at["k"]), dict(kc=at["v"]),
               dict(qo=at["k"]), dict(qo=at["v"]), dict(qo=at["kc"]), dict(q=at["vc"]),
               dict(qo=at["q"], qos=520)):
        assert call(**kw) == IA, kw
    if fn == "pa_q8_append":
        for kw in (dict(sc=None), dict(sv=None), dict(sc=FAKE + 2), dict(sv=FAKE)):
            assert call(**kw) == IA, kw
    for kw in (dict(D=80, R=80), dict(ps=8), dict(R=24), dict(hkv=40000, ks=1 << 30, vs=1 << 30),
               dict(hq=40000, qs=1 << 30, qos=1 << 30)):
        assert call(**kw) == UN, kw


def test_read_checks_return_before_launch(lib):
    def call(n=4, hkv=2, D=128, ps=16, pages=8, dtype=0, kc=FAKE, vc=FAKE + 4096, ks=FAKE, vs=FAKE,
             slots=FAKE, k=FAKE + (1 << 16), kst=256, v=FAKE + (1 << 17), vst=256, err=None):
        return lib.pa_q8_read(n, hkv, D, ps, pages, dtype, kc, vc, ks, vs, slots, k, kst, v, vst,
                              err, None)

    assert call(n=0, kc=None, k=None) == binding.PA_OK
    for kw in (dict(n=-1), dict(hkv=0), dict(pages=0), dict(dtype=-1), dict(kst=255), dict(vst=260),
               dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None),
               dict(slots=None), dict(k=FAKE + 8), dict(vc=FAKE + 4), dict(ks=FAKE + 1),
               dict(slots=FAKE + 4), dict(err=FAKE + 1), dict(k=FAKE + (1 << 17)), dict(k=FAKE)):
        assert call(**kw) == IA, kw
    for kw in (dict(D=80), dict(ps=32), dict(hkv=40000, kst=1 << 30, vst=1 << 30)):
        assert call(**kw) == UN, kw


def test_verify_checks_return_before_launch(lib):
    names = ["p", "q", "x", "n", "u", "s", "acc", "tok", "err"]
    at = {n: FAKE + 4096 * i for i, n in enumerate(names)}

    def call(B=2, T=3, V=100, dtype=2, **kw):
        a = dict(at, **kw)
        return lib.pa_verify_drafts(B, T, V, dtype, *[a[n] for n in names], None)

    assert call(B=0, p=None) == binding.PA_OK
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(dtype=5), dict(p=None), dict(x=None),
               dict(u=None), dict(s=None), dict(acc=None), dict(tok=None), dict(p=FAKE + 2),
               dict(q=FAKE + 1), dict(x=FAKE + 2), dict(n=FAKE + 1), dict(u=FAKE + 2),
               dict(acc=FAKE + 2), dict(err=FAKE + 3), dict(acc=at["tok"]), dict(acc=at["n"]),
               dict(tok=at["x"]), dict(tok=at["n"])):
        assert call(**kw) == IA, kw
    for kw in (dict(T=33), dict(V=524289)):
        assert call(**kw) == UN, kw
    assert call(dtype=0, p=FAKE + 1) == IA


def test_binding_refuses_host_tensors_and_wrong_arguments():
    k = torch.zeros(2, 1, 64, dtype=torch.float16)
    slots = torch.zeros(2, dtype=torch.int64)
    kc, vc, ks, vs = pa.new_q8_cache(3, 1, 64, "cpu")
    assert kc.shape == (3, 1, 16, 64) and kc.dtype == torch.float8_e4m3fn and ks.shape == (3, 1)
    assert (ks == 1).all() and (kc.float() == 0).all()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="supported"):
        pa.new_q8_cache(1, 1, 80, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_append(k, k, k, slots, i, kc, vc)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q8_append(None, k, k, slots, i, kc, vc, ks, vs)
    with pytest.raises(TypeError):
        pa.pa_q8_append(None, None, k, slots, i, kc, vc, ks, vs)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q8_read(kc, vc, ks, vs, slots, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_q8_decode(_plan(), k, None, kc, vc, ks, vs, i, i, 1.0, 0, k, k, kc)
    with pytest.raises(TypeError):
        pa.q8_decode(k.float(), None, kc, vc, ks, vs, i, i, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_verify_drafts(k.float(), None, i, None, k, k, i, i)


# ---------------------------------------------------------------- the marshalling extension

def tens(dtype, shape, stride=None):
    """A CPU tensor of this form (its device, -1, is the stand-in's current one)."""
    return torch.empty(shape, dtype=dtype) if stride is None else \
        torch.empty_strided(shape, stride, dtype=dtype)


@pytest.fixture
def marshalled(lib):
    """The extension with recording stand-ins for the five C functions; yields (module, calls)."""
    from paged_kv_gqa_pa_gb300 import q4
    if q4._fast is None:
        pytest.skip("the marshalling extension is not built here")
    calls = []
    P, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    rows = [i] * 8 + [f, f] + [P, ll] * 3 + [P] * 5 + [ll, P, P]
    protos = dict(append=ctypes.CFUNCTYPE(i, *rows, P, P), q8_append=ctypes.CFUNCTYPE(i, *rows, *[P] * 4),
                  q8_read=ctypes.CFUNCTYPE(i, *[i] * 6, *[P] * 5, P, ll, P, ll, P, P),
                  q8_decode=ctypes.CFUNCTYPE(i, P, i, *[P] * 8, f, i, *[P] * 4),
                  verify=ctypes.CFUNCTYPE(i, *[i] * 4, *[P] * 10))
    keep = []
    for name, proto in protos.items():
        def fn(*a, name=name):
            if name == "q8_decode":
                a = (ctypes.string_at(a[0], ctypes.sizeof(q8.pa_q8_plan_t)),) + a[1:]
            calls.append((name, a))
            return 4 if name == "q8_read" else 0
        keep.append(proto(fn))
    q4._fast.setup((1, 2, 3, 4, 5), lambda: -1, lambda d: 4096 + d)
    q4._fast.setup_q8(tuple(ctypes.cast(fn, P).value for fn in keep))
    yield q4._fast, calls
    q4._load_fast(lib)  # the real functions again
    q4._fast.setup_q8(tuple(ctypes.cast(getattr(lib, n), P).value for n in
                            ("pa_append", "pa_q8_append", "pa_q8_read", "pa_q8_decode",
                             "pa_verify_drafts")))


def at(*t):
    return tuple(None if x is None else x.data_ptr() for x in t)


F16, F32, I32, I64, F8 = (torch.float16, torch.float32, torch.int32, torch.int64,
                          torch.float8_e4m3fn)


def test_marshalling_of_the_usual_calls(marshalled):
    fast, calls = marshalled
    wide = (8 * 128, 128, 1)
    q, k, v = tens(F16, (5, 4, 128), wide), tens(F16, (5, 2, 128), wide), tens(F16, (5, 2, 128), wide)
    qo, qn, kn = tens(F16, (5, 4, 128)), tens(F16, (128,)), tens(F16, (128,))
    sl, pos = tens(I64, (5,)), tens(I32, (5,))
    k16, v16 = tens(F16, (9, 2, 16, 128)), tens(F16, (9, 2, 16, 128))
    assert fast.append(q, k, v, sl, pos, k16, v16, qo, qn, kn, 0.5, 1e4, 64) == 0
    assert calls.pop() == ("append", (5, 4, 2, 128, 64, 16, 9, 0, 1e4, 0.5, *at(q), 1024, *at(k), 1024,
                                      *at(v), 1024, *at(qn, kn, pos, sl, qo), 512, *at(k16, v16), None,
                                      4095))
    assert fast.append(None, k, v, sl, None, k16, v16, None, None, None, 0.5, 0.0, None) == 0
    assert calls.pop() == ("append", (5, 0, 2, 128, 128, 16, 9, 0, 0.0, 0.5, None, 0, *at(k), 1024,
                                      *at(v), 1024, None, None, None, *at(sl), None, 0,
                                      *at(k16, v16), None, 4095))
    kc, vc = tens(F8, (9, 2, 16, 128)), tens(F8, (9, 2, 16, 128))
    ks, vs = tens(F32, (9, 2)), tens(F32, (9, 2))
    assert fast.q8_append(q, k, v, sl, pos, kc, vc, None, None, kn, 0.5, 1e4, None, ks, vs) == 0
    assert calls.pop() == ("q8_append", (5, 4, 2, 128, 128, 16, 9, 0, 1e4, 0.5, *at(q), 1024, *at(k),
                                         1024, *at(v), 1024, None, *at(kn, pos, sl, q), 1024,
                                         *at(kc, vc, ks, vs), None, 4095))
    assert fast.q8_read(kc, vc, ks, vs, sl, k, v) == 4  # the status comes back
    assert calls.pop() == ("q8_read", (5, 2, 128, 16, 9, 0, *at(kc, vc, ks, vs, sl, k), 1024, *at(v), 1024,
                                       None, 4095))
    plan = _plan(num_pages=9, max_query_len=3)
    dq, do, lse = tens(F16, (7, 8, 128)), tens(F16, (7, 8, 128)), tens(F32, (7, 8))
    st, bt, cl = tens(I32, (5,)), tens(I32, (4, 16)), tens(I32, (4,))
    ws = tens(torch.uint8, (plan.workspace_bytes,))
    for s in (st, None):
        assert fast.q8_decode(plan, dq, s, kc, vc, ks, vs, bt, cl, 0.5, 3, do, lse, ws) == 0
        assert calls.pop() == ("q8_decode", (bytes(plan), 7, *at(dq, s, kc, vc, ks, vs, bt, cl), 0.5, 3,
                                             *at(do, lse, ws), 4095))
    p, d = tens(F32, (2, 4, 50)), tens(F32, (2, 3, 50))
    x, n, u, s = tens(I32, (2, 3)), tens(I32, (2,)), tens(F32, (2, 3)), tens(F32, (2,))
    acc, tok = tens(I32, (2,)), tens(I32, (2, 4))
    for dd, nn in ((d, n), (None, None)):
        assert fast.verify(p, dd, x, nn, u, s, acc, tok) == 0
        assert calls.pop() == ("verify", (2, 3, 50, 2, *at(p, dd, x, nn, u, s, acc, tok), None, 4095))
    assert not calls


def test_marshalling_leaves_everything_else_alone(marshalled):
    fast, calls = marshalled
    k, q = tens(F16, (5, 2, 128)), tens(F16, (5, 4, 128))
    sl, pos, w = tens(I64, (5,)), tens(I32, (5,)), tens(F16, (128,))
    k16, kc, ks = tens(F16, (9, 2, 16, 128)), tens(F8, (9, 2, 16, 128)), tens(F32, (9, 2))
    base = [q, k, k, sl, pos, k16, k16, q, w, w, 0.5, 1e4, 64]
    assert fast.append(*base) == 0
    assert fast.q8_append(*base[:5], kc, kc, *base[7:], ks, ks) == 0
    calls.clear()
    for i, bad in [(0, tens(F16, (4, 4, 128))), (0, tens(F32, (5, 4, 128))), (0, None), (0, 3),
                   (1, tens(F16, (5, 256))), (1, tens(F16, (5, 2, 128), (256, 1, 2))),
                   (2, tens(F16, (5, 3, 128))), (2, tens(torch.bfloat16, (5, 2, 128))),
                   (3, tens(I32, (5,))), (3, tens(I64, (6,))), (4, None), (4, tens(I64, (5,))),
                   (7, tens(F16, (5, 2, 128))), (8, tens(F16, (64,))), (9, tens(F32, (128,))),
                   (10, 1), (11, 10000), (12, 64.0), (12, True)]:
        a = list(base)
        a[i] = bad
        assert fast.append(*a) is None, (i, bad)
        assert fast.q8_append(*a[:5], kc, kc, *a[7:], ks, ks) is None, (i, bad)
    for cache in (kc, tens(F16, (9, 3, 16, 128)), tens(F16, (9, 2, 8, 128)), tens(F16, (9, 2, 16, 64)),
                  tens(F16, (9, 2, 16, 128), (4096, 2048, 1, 16))):
        assert fast.append(*base[:5], cache, k16, *base[7:]) is None
        assert fast.append(*base[:5], k16, cache, *base[7:]) is None
    for a in ((k16, kc, ks, ks), (kc, tens(F8, (8, 2, 16, 128)), ks, ks), (kc, kc, tens(F32, (9, 3)), ks),
              (kc, kc, ks, tens(F16, (9, 2)))):
        assert fast.q8_append(*base[:5], *a[:2], *base[7:], *a[2:]) is None
        assert fast.q8_read(*a, sl, k, k) is None
    assert fast.q8_read(kc, kc, ks, ks, tens(I64, (4,)), k, k) is None
    assert fast.q8_read(kc, kc, ks, ks, sl, k, tens(F32, (5, 2, 128))) is None
    plan = _plan(num_pages=9)
    base = [plan, tens(F16, (7, 8, 128)), tens(I32, (5,)), kc, kc, ks, ks, tens(I32, (4, 16)),
            tens(I32, (4,)), 0.5, 0, tens(F16, (7, 8, 128)), tens(F32, (7, 8)),
            tens(torch.uint8, (plan.workspace_bytes,))]
    assert fast.q8_decode(*base) == 0
    calls.clear()
    for i, bad in [(0, object()), (0, b"x" * 8), (1, tens(F16, (7, 4, 128))), (1, tens(F16, (8, 128))),
                   (2, tens(I32, (4,))), (2, tens(I64, (5,))), (3, k16), (5, tens(F32, (9,))),
                   (7, tens(I32, (4, 15))), (8, tens(I64, (4,))), (9, 1), (10, 0.0),
                   (11, tens(F16, (6, 8, 128))), (12, tens(F32, (7, 4))),
                   (13, tens(torch.uint8, (plan.workspace_bytes - 1,)))]:
        a = list(base)
        a[i] = bad
        assert fast.q8_decode(*a) is None, (i, bad)
    few = [plan, tens(F16, (3, 8, 128)), None, *base[3:11], tens(F16, (3, 8, 128)), tens(F32, (3, 8)), base[13]]
    assert fast.q8_decode(*few) is None  # fewer rows than sequences without starts
    base = [tens(F32, (2, 4, 50)), tens(F32, (2, 3, 50)), tens(I32, (2, 3)), tens(I32, (2,)),
            tens(F32, (2, 3)), tens(F32, (2,)), tens(I32, (2,)), tens(I32, (2, 4))]
    assert fast.verify(*base) == 0
    calls.clear()
    for i, bad in [(0, tens(F32, (2, 50))), (0, tens(I32, (2, 4, 50))), (1, tens(F16, (2, 3, 50))),
                   (1, tens(F32, (2, 4, 50))), (2, None), (2, tens(I64, (2, 3))), (3, tens(I32, (3,))),
                   (4, tens(F32, (2, 4))), (5, None), (6, tens(F32, (2,))), (7, tens(I32, (2, 3)))]:
        a = list(base)
        a[i] = bad
        assert fast.verify(*a) is None, (i, bad)
    assert fast.verify(*base[:7]) is None and fast.q8_read(1) is None
    assert not calls
