"""GPU tests of include/pa_q8.h at what its first tests left open: outputs off by no more than
their own rounding and V scales at the ends of their range."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
from paged_kv_gqa_pa_gb300 import build as pa_build
from test_q8_gpu import DIMS, Decode, T, host, i32, rounded, to_t

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
