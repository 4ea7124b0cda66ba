"""The operators of a step with drafted tokens over an 8-bit paged KV cache, as cases to be measured.

Four operators, each in a plain form (elementary torch operations, the default)
and as calls of this package (``own = True``):

  append   q and k normalised by head and rotated, q written to rows, k and v
           into the paged cache of pa_decode (fp16, bf16, fp32) by slot
  store    the same into a paged cache held in 8 bits, and rows of the pages
           that it touched read back
  decode   one or several query tokens per sequence over the 8-bit paged cache
  verify   drafted tokens accepted or not against the target's probabilities,
           and one more token drawn, from given random numbers

Sizes are the head counts, head dims and lengths of this package's own
workloads and tests, or generic ones around them.

The 8-bit cache.  K and V are e4m3 codes [num_pages, Hkv, 16, D] with fp32
scales [num_pages, Hkv]: a code c stands for scale * c.  Appending makes the
scale of a (page, KV head) the least power of two 2^e, e >= -120, with
|x| <= 448 * 2^e for every element of the page's rows so far: rows at position
0 begin a page anew, later ones raise the scale, and then the rows before them
are rounded to the wider steps.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
EPS = 1e-6
_T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_UNIT = 2.0 ** 44  # weights of a draw are whole multiples of 1 / _UNIT


# ---------------------------------------------------------------- cases

def listed():
    return [
        # The decode step's new rows of 64 sequences, heads normalised and rotated.
        dict(name="append_decode64", op="append", tokens=64, hq=32, hkv=8, dim=128, rot=128,
             norm=True, dtype="f16", theta=500000.0, order="decode", skipped=0.0),
        # A long prompt, heads of the long-context workload.
        dict(name="append_prompt", op="append", tokens=16384, hq=24, hkv=4, dim=256, rot=256,
             norm=True, dtype="bf16", theta=10000.0, order="prompt", skipped=0.0),
        # fp32, an odd number of rows of a padded batch, half of each head rotated, no norms.
        dict(name="append_half_f32", op="append", tokens=2049, hq=8, hkv=4, dim=64, rot=32,
             norm=False, dtype="f32", theta=10000.0, order="prompt", skipped=0.1),
        # The decode step's new rows of 64 sequences: every one joins a page that has rows.
        dict(name="store_decode64", op="store", tokens=64, hq=32, hkv=8, dim=128, rot=128,
             norm=True, dtype="f16", theta=500000.0, order="decode"),
        # A long prompt, heads of the long-context workload.
        dict(name="store_prompt", op="store", tokens=16384, hq=24, hkv=4, dim=256, rot=256,
             norm=True, dtype="bf16", theta=10000.0, order="prompt"),
        # Chunks of prompts that begin and end inside pages, an odd number of rows, no norms.
        dict(name="store_chunks_d96", op="store", tokens=4093, hq=16, hkv=4, dim=96, rot=48,
             norm=False, dtype="f16", theta=10000.0, order="chunks"),
        # The single-sequence latency case of this package's benchmark.
        dict(name="decode_tiny_d64", op="decode", batch=1, hq=4, hkv=1, dim=64, length=256,
             spread="equal", window=0, queries=1, dtype="f16"),
        # A serving batch of ragged lengths, bf16.
        dict(name="decode_ragged64", op="decode", batch=64, hq=32, hkv=8, dim=128, length=4096,
             spread="ragged", window=0, queries=1, dtype="bf16"),
        # Four drafted tokens and the last sampled one of each sequence, behind a window.
        dict(name="decode_drafts5", op="decode", batch=16, hq=32, hkv=8, dim=128, length=8192,
             spread="equal", window=4096, queries=5, dtype="f16"),
        # The long-context workload of this package's benchmark, its cache in 8 bits.
        dict(name="decode_100k", op="decode", batch=4, hq=24, hkv=4, dim=256, length=100000,
             spread="equal", window=0, queries=1, dtype="f16"),
        # One request's four drafted tokens, an odd vocabulary.
        dict(name="verify_1", op="verify", batch=1, drafts=4, vocab=32003, dtype="f32"),
        # A serving batch.
        dict(name="verify_128", op="verify", batch=128, drafts=7, vocab=131072, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "store", "decode", "decode", "verify"])
    if op == "verify":
        vocab = _log(rng, 1000, 200000)
        batch = min(_log(rng, 1, 128), 128 * 131072 // vocab)
        return dict(op=op, batch=batch, drafts=rng.randint(1, 7), vocab=vocab,
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 96, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "decode":
        batch = _log(rng, 1, 128)
        queries = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        length = _log(rng, 1, 100000)
        length = max(queries, min(length, (4 * 4 * 256 * 100000) // (batch * hkv * dim),
                                  (4 * 24 * 256 * 100000) // (batch * hkv * g * dim * queries)))
        return dict(op=op, batch=batch, hq=g * hkv, hkv=hkv, dim=dim, length=length,
                    spread=rng.choice(["equal", "ragged"]),
                    window=rng.choice([0, 0, 0, max(1, length // 3)]), queries=queries,
                    dtype=dtype)
    if op == "append" and rng.random() < 0.25:
        dtype = "f32"
    tokens = min(_log(rng, 1, 16384), (16384 * 32 * 256) // (hkv * (g + 2) * dim *
                                                             (2 if dtype == "f32" else 1)))
    case = dict(op=op, tokens=tokens, hq=g * hkv, hkv=hkv, dim=dim,
                rot=rng.choice([dim, dim, dim // 2]), norm=rng.random() < 0.5, dtype=dtype,
                theta=rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "append":
        case.update(order=rng.choice(["decode", "prompt"]), skipped=rng.choice([0.0, 0.0, 0.3]))
    else:
        case.update(order=rng.choice(["decode", "prompt", "chunks"]))
    return case


# ---------------------------------------------------------------- lengths

def _row_slots(case, seed):
    """(slots, positions, first, pages) of the rows of an append or store case, host arrays:
    `first` lists the slots of the rows that the touched pages held before.  How many rows
    join a page that holds some goes by the case, where the pages lie by the seed."""
    g = np.random.default_rng([seed, 21])
    f = np.random.default_rng(21)
    n, order = case["tokens"], case["order"]
    if order == "decode":  # one new row of each of n sequences
        pages = n + n // 4 + 1
        page = g.permutation(pages)[:n].astype(np.int64)
        at = g.permutation(f.integers(0, PAGE, size=n))
        positions = g.integers(0, 6000, size=n) * PAGE + at
        slots = page * PAGE + at
        runs = [(p, a, 1) for p, a in zip(page, at)]
    else:  # runs of prompts' rows through shuffled pages
        lens = [n]
        if order == "chunks":
            lens = []
            while sum(lens) < n:
                lens.append(min(n - sum(lens), int(f.integers(1, 700))))
        begin = [int(f.integers(0, PAGE)) if order == "chunks" else 0 for _ in lens]
        need = [(b + m + PAGE - 1) // PAGE for b, m in zip(begin, lens)]
        pages = sum(need) + sum(need) // 64 + 1
        perm = g.permutation(pages).astype(np.int64)
        slots, positions, runs, off = [], [], [], 0
        for b, m, k in zip(begin, lens, need):
            flat = b + np.arange(m)
            slots.append(perm[off + flat // PAGE] * PAGE + flat % PAGE)
            positions.append(int(g.integers(0, 2000)) * PAGE + flat)
            runs.append((perm[off], b, min(m, PAGE - b)))
            off += k
        slots, positions = np.concatenate(slots), np.concatenate(positions)
    first = np.concatenate([np.arange(p * PAGE, p * PAGE + a) for p, a, _ in runs])
    if case.get("skipped"):
        slots = np.where(f.random(n) < case["skipped"], -1, slots)
    return slots.astype(np.int64), positions.astype(np.int32), first.astype(np.int64), pages


def _context_lengths(case, seed):
    """(lengths, query tokens) of a decode case's sequences."""
    g = np.random.default_rng([seed, 22])
    f = np.random.default_rng(22)
    B, L, T = case["batch"], case["length"], case["queries"]
    if case["spread"] == "equal":
        return np.full(B, L, dtype=np.int64), np.full(B, T, dtype=np.int64)
    # The lengths and numbers of drafts there are go by the case, whose they are by the seed.
    lens, new = f.integers(1, L + 1, size=B), f.integers(1, T + 1, size=B)
    lens[0], new[0] = L, T
    if B > 2:
        lens[-1], new[-1] = 1, 1
    if B > 4:
        lens[-2], new[-2] = 0, 0  # a request that has nothing yet
    p = g.permutation(B)
    lens, new = lens[p], new[p]
    return lens, np.minimum(new, lens)


def _stops(case):
    """Where the verification of each sequence stops: at a draft that is not accepted, or
    (the number of drafts) behind the last."""
    return np.random.default_rng(23).integers(0, case["drafts"] + 1, size=case["batch"])


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 29)
    return {"append": _prepare_rows, "store": _prepare_rows, "decode": _prepare_decode,
            "verify": _prepare_verify}[case["op"]](case, seed, dev, gen)


def _kv_rows(shape, gen, dev):
    """K- or V-like rows: normal values around a bias of each channel, some channels wide."""
    D = shape[-1]
    wide = 1 + 4 * (torch.rand(D, generator=gen, device=dev) < 0.03).float()
    bias = torch.randn(D, generator=gen, device=dev) * 0.5
    return torch.randn(shape, generator=gen, device=dev) * wide + bias


def _scale_of(amax):
    """The least power of two 2^e, e >= -120, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax.double())  # amax = m 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, -120).clamp(min=-120)
    return ((e.long() + 1023) << 52).view(torch.float64).float()  # 2^e


def _prepare_rows(case, seed, dev, gen):
    n, hq, hkv, D = case["tokens"], case["hq"], case["hkv"], case["dim"]
    dt = _T[case["dtype"]]
    # q, k and v as the columns of a fused projection's rows
    qkv = torch.empty(n, hq + 2 * hkv, D, dtype=dt, device=dev)
    for lo in range(0, n, 4096):
        qkv[lo:lo + 4096] = _kv_rows((min(n, lo + 4096) - lo, hq + 2 * hkv, D), gen, dev).to(dt)
    slots, positions, first, pages = _row_slots(case, seed)
    s = dict(op=case["op"], dtype=dt, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
             slots=torch.from_numpy(slots).to(dev), pos=torch.from_numpy(positions).to(dev),
             theta=case["theta"], rot=case["rot"], q_norm=None, k_norm=None,
             q_out=torch.empty(n, hq, D, dtype=dt, device=dev))
    if case["norm"]:
        s["q_norm"] = (1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt)
        s["k_norm"] = (1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt)
    if case["op"] == "append":
        for name in ("k_cache", "v_cache"):
            s[name] = torch.randn(pages, hkv, PAGE, D, generator=gen, device=dev).to(dt)
        return s
    # The rows that were there before are in the cache, other cells hold what they hold.
    old = torch.from_numpy(first).to(dev)
    for name in ("k", "v"):
        codes = torch.full((pages, hkv, PAGE, D), 0x7F, dtype=torch.uint8, device=dev)
        x = torch.zeros(pages, PAGE, hkv, D, device=dev)
        x.view(-1, hkv, D)[old] = _kv_rows((old.numel(), hkv, D), gen, dev) * 0.5
        x = x.transpose(1, 2)
        scale = _scale_of(x.abs().amax((2, 3)))
        c = (x / scale[..., None, None]).to(_F8).view(torch.uint8)
        had = torch.zeros(pages * PAGE, dtype=torch.bool, device=dev)
        had[old] = True
        codes = torch.where(had.view(pages, 1, PAGE, 1), c, codes)
        s[name + "_cache"], s[name + "_scales"] = codes.contiguous().view(_F8), scale
    rows = np.sort(np.concatenate([first, slots]))
    s["read"] = torch.from_numpy(rows).to(dev)
    s["k_out"] = torch.empty(rows.size, hkv, D, dtype=dt, device=dev)
    s["v_out"] = torch.empty(rows.size, hkv, D, dtype=dt, device=dev)
    return s


def _prepare_decode(case, seed, dev, gen):
    B, hq, hkv, D, T = case["batch"], case["hq"], case["hkv"], case["dim"], case["queries"]
    dt = _T[case["dtype"]]
    lens, new = _context_lengths(case, seed)
    need = -(-lens // PAGE)
    total = int(need.sum())
    pages = total + total // 8 + 1
    perm = np.random.default_rng([seed, 24]).permutation(pages).astype(np.int32)
    maxp = max(1, int(need.max()))
    bt = np.full((B, maxp), -1, dtype=np.int32)
    live = np.zeros(pages, dtype=np.int64)  # rows of each page that its sequence has
    off = 0
    for b in range(B):
        ids = perm[off:off + need[b]]
        bt[b, :need[b]] = ids
        live[ids] = np.minimum(PAGE, lens[b] - PAGE * np.arange(need[b]))
        off += need[b]
    live = torch.from_numpy(live).to(dev)
    st = dict(op="decode", dtype=dt, window=case["window"], scale=1.0 / math.sqrt(D), queries=T)
    row = torch.arange(PAGE, device=dev).view(1, 1, PAGE, 1)
    for name in ("k", "v"):
        # cells that no sequence has hold NaN
        codes = torch.full((pages, hkv, PAGE, D), 0x7F, dtype=torch.uint8, device=dev)
        scales = torch.ones(pages, hkv, device=dev)
        for lo in range(0, pages, 4096):
            have = row < live[lo:lo + 4096].view(-1, 1, 1, 1)
            x = torch.where(have, _kv_rows((have.shape[0], hkv, PAGE, D), gen, dev), 0.0)
            sc = _scale_of(x.abs().amax((2, 3)))
            c = (x / sc[..., None, None]).to(_F8).view(torch.uint8)
            codes[lo:lo + 4096] = torch.where(have, c, codes[lo:lo + 4096])
            scales[lo:lo + 4096] = sc
        st[name + "_cache"], st[name + "_scales"] = codes.view(_F8), scales
    starts = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(max(int(starts[-1]), 1), hq, D, generator=gen, device=dev).to(dt)
    st.update(q=q, bt=torch.from_numpy(bt).to(dev),
              lens=torch.from_numpy(lens.astype(np.int32)).to(dev),
              starts=torch.from_numpy(starts.astype(np.int32)).to(dev),
              out=torch.zeros_like(q),
              lse=torch.zeros(q.shape[0], hq, dtype=torch.float32, device=dev))
    if own:
        import paged_kv_gqa_pa_gb300 as pa
        st["plan"] = pa.pa_q8_plan(B, hq, hkv, D, PAGE, pages, maxp, int(lens.max()),
                                   window=case["window"], max_query_len=T,
                                   dtype=1 if case["dtype"] == "bf16" else 0)
        st["ws"] = pa.new_workspace(st["plan"], dev)
    return st


def _prepare_verify(case, seed, dev, gen):
    B, T, V = case["batch"], case["drafts"], case["vocab"]
    dt = _T[case["dtype"]]
    target = torch.empty(B, T + 1, V, dtype=dt, device=dev)
    draft = torch.empty(B, T, V, dtype=dt, device=dev)
    tokens = torch.empty(B, T, dtype=torch.int32, device=dev)
    accept = torch.rand(B, T, generator=gen, device=dev)
    stops = torch.from_numpy(_stops(case)).to(dev)
    ratio = torch.empty(B, T, device=dev)
    for b in range(B):
        # peaked rows, as a language model's are; the draft's are near the target's
        x = 2.5 * torch.randn(T + 1, V, generator=gen, device=dev)
        y = x[:T] + 0.7 * torch.randn(T, V, generator=gen, device=dev)
        target[b] = torch.softmax(x, -1).to(dt)
        draft[b] = torch.softmax(y, -1).to(dt)
        # drafted tokens: drawn from the draft's, where a sequence stops from those that the
        # target has less of
        p, q = target[b, :T].float(), draft[b].float()
        last = (torch.arange(T, device=dev) == stops[b])[:, None]
        w = torch.where(torch.where(last, p < 0.8 * q, p > 0), q, 0.0)
        c = torch.cumsum(w.double(), -1)
        u = torch.rand(T, 1, generator=gen, device=dev).double() * c[:, -1:]
        x = torch.searchsorted(c, u, right=True).clamp(max=V - 1)
        tokens[b] = x[:, 0].int()
        ratio[b] = torch.clamp(p.gather(1, x)[:, 0] / q.gather(1, x)[:, 0], max=1.0)
    # random numbers below p / q before the stop, above it there
    t = torch.arange(T, device=dev)
    accept = torch.where(t < stops[:, None], accept * ratio * 0.999,
                         torch.where(t == stops[:, None], ratio + accept * (1 - ratio) * 0.999 +
                                     5e-4 * (1 - ratio), accept)).clamp(0, 1 - 2.0 ** -24)
    return dict(op="verify", target=target, draft=draft, draft_tokens=tokens,
                num=torch.full((B,), T, dtype=torch.int32, device=dev), accept=accept,
                sample=torch.rand(B, generator=gen, device=dev),
                accepted=torch.empty(B, dtype=torch.int32, device=dev),
                tokens=torch.empty(B, T + 1, dtype=torch.int32, device=dev))


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_append(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_append(s["q"], s["k"], s["v"], s["slots"], s["pos"], s["k_cache"], s["v_cache"],
                 q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                 theta=s["theta"], rotary_dim=s["rot"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _own_store(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_q8_append(s["q"], s["k"], s["v"], s["slots"], s["pos"], s["k_cache"], s["v_cache"],
                    s["k_scales"], s["v_scales"], q_out=s["q_out"], q_norm=s["q_norm"],
                    k_norm=s["k_norm"], eps=EPS, theta=s["theta"], rotary_dim=s["rot"])
    pa.pa_q8_read(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["read"], s["k_out"],
                  s["v_out"])
    return [s["q_out"], s["k_out"], s["v_out"]]


def _own_decode(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_q8_decode(s["plan"], s["q"], s["starts"], s["k_cache"], s["v_cache"], s["k_scales"],
                    s["v_scales"], s["bt"], s["lens"], s["scale"], s["window"], s["out"],
                    s["lse"], s["ws"])
    return [s["out"], s["lse"]]


def _own_verify(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_verify_drafts(s["target"], s["draft"], s["draft_tokens"], s["num"], s["accept"],
                        s["sample"], s["accepted"], s["tokens"])
    return [s["accepted"], s["tokens"]]


def _turned(x, w, s):
    """Heads normalised (where there are weights) and rotated, fp32."""
    f = x.float()
    if w is not None:
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()
    rot, half = s["rot"], s["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = s["pos"].double()[:, None] * s["theta"] ** (-2.0 * i / rot)  # far positions: 64 bits
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = f[..., :half], f[..., half:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, f[..., rot:]], -1)


def _put(cache, slots, rows):
    """The row of each slot, rows of slot -1 left out."""
    pages, hkv, _, D = cache.shape
    flat = torch.cat([cache.transpose(1, 2).reshape(-1, hkv, D),
                      torch.zeros(1, hkv, D, dtype=cache.dtype, device=cache.device)])
    flat[torch.where(slots >= 0, slots, pages * PAGE)] = rows  # (a spare row takes the left-out ones)
    cache.copy_(flat[:-1].view(pages, PAGE, hkv, D).transpose(1, 2))
    return cache


def _plain_append(s):
    dt = s["dtype"]
    q_out = _turned(s["q"], s["q_norm"], s).to(dt)
    k = _turned(s["k"], s["k_norm"], s).to(dt)
    return [q_out, _put(s["k_cache"], s["slots"], k), _put(s["v_cache"], s["slots"], s["v"])]


def _plain_store_one(s, name, rows):
    """Rows [n, hkv, D] (fp32) quantised into the cache `name`; its rows `read`."""
    cache, scales, slots = s[name + "_cache"], s[name + "_scales"], s["slots"]
    pages, hkv, _, D = cache.shape
    page, at = slots // PAGE, slots % PAGE
    need = torch.zeros(pages, hkv, device=rows.device).index_reduce_(0, page, rows.abs().amax(-1),
                                                                    "amax")
    begin = torch.full((pages,), PAGE, device=rows.device).index_reduce_(0, page, at, "amin")
    touched = (begin < PAGE)[:, None]
    base = torch.where((begin == 0)[:, None], torch.zeros_like(scales), scales)
    new = torch.where(touched, torch.maximum(base, _scale_of(need)), scales)
    kept = cache.float() * (scales / new)[..., None, None]  # (rows that are rewritten among them)
    kept = kept.to(_F8).view(torch.uint8).transpose(1, 2).reshape(-1, hkv, D)
    kept[slots] = (rows / new[page][..., None]).to(_F8).view(torch.uint8)
    scales.copy_(new)
    cache.view(torch.uint8).copy_(kept.view(pages, PAGE, hkv, D).transpose(1, 2))
    vals = kept[s["read"]].view(_F8).float() * new[s["read"] // PAGE][..., None]
    return vals.to(s["dtype"])


def _plain_store(s):
    return [_turned(s["q"], s["q_norm"], s).to(s["dtype"]),
            _plain_store_one(s, "k", _turned(s["k"], s["k_norm"], s)),
            _plain_store_one(s, "v", s["v"].float())]


def _plain_decode(s):
    lens, starts, T = s["lens"].long(), s["starts"].long(), s["queries"]
    N, hq, D = s["q"].shape
    hkv = s["k_cache"].shape[1]
    B, P = s["bt"].shape
    g = hq // hkv
    t = torch.arange(T, device=lens.device)
    new = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + t).clamp(max=N - 1)  # [B, T]
    q = s["q"].float()[row].view(B, T, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * g, D)
    bt = s["bt"].long().clamp(min=0)
    pos = torch.arange(P * PAGE, device=lens.device)
    ends = (lens - new)[:, None] + t + 1  # tokens before this one are seen by query t
    seen = (pos < ends[..., None]) & (t < new[:, None])[..., None]  # [B, T, tokens]
    if s["window"] > 0:
        seen &= pos >= (ends - s["window"])[..., None]
    any_seen = seen.any(1)

    def values(name):
        x = s[name + "_cache"][bt].float() * s[name + "_scales"][bt][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, hkv, P * PAGE, D)

    x = torch.matmul(q, values("k").transpose(2, 3)) * s["scale"]  # [B, hkv, T g, tokens]
    mask = seen[:, None, :, None].expand(B, hkv, T, g, P * PAGE).reshape(x.shape)
    x = torch.where(mask, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    v = torch.where(any_seen[:, None, :, None], values("v"), 0.0)
    out = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)

    n = torch.arange(N, device=lens.device)  # whose row is it, and which of its tokens
    b = (torch.searchsorted(starts, n, right=True) - 1).clamp(0, B - 1)
    at = (n - starts[b]).clamp(0, T - 1)
    out = out.view(B, hkv, T, g, D).transpose(1, 2).reshape(B, T, hq, D)[b, at]
    lse = lse.view(B, hkv, T, g).transpose(1, 2).reshape(B, T, hq)[b, at]
    return [out.to(s["dtype"]), lse]


def _plain_verify(s):
    target, draft, x = s["target"], s["draft"], s["draft_tokens"].long()
    B, T, V = draft.shape
    t = torch.arange(T, device=x.device)
    px = target[:, :T].gather(2, x[..., None])[..., 0].double()  # 64 bits: next to a border
    qx = draft.gather(2, x[..., None])[..., 0].double()
    ok = (s["accept"].double() * qx < px) & (t < s["num"][:, None])
    j = ok.long().cumprod(-1).sum(-1)
    b = torch.arange(B, device=x.device)
    p = target[b, j].float().clamp(0, 1)
    q = draft[b, j.clamp(max=T - 1)].float().clamp(0, 1)
    cut = (j < s["num"])[:, None]
    w = torch.where(cut, (p - q).clamp(min=0), p)
    w = torch.where((w * _UNIT).round().sum(-1, keepdim=True) > 0, w, p)
    c = torch.cumsum((w.double() * _UNIT).round().long(), -1)
    total = c[:, -1:]
    at = torch.minimum(torch.floor(s["sample"].double()[:, None] * total.double()).long(), total - 1)
    y = (c <= at).sum(-1)
    k = torch.arange(T + 1, device=x.device)
    drafted = torch.cat([x, x[:, :1]], 1)
    out = torch.where(k < j[:, None], drafted, torch.where(k == j[:, None], y[:, None], -1))
    return [j.int(), out.int()]


_OWN = {"append": _own_append, "store": _own_store, "decode": _own_decode, "verify": _own_verify}
_PLAIN = {"append": _plain_append, "store": _plain_store, "decode": _plain_decode,
          "verify": _plain_verify}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "verify":
        B, V, es = case["batch"], case["vocab"], _T[case["dtype"]].itemsize
        cut = int((_stops(case) < case["drafts"]).sum())
        # a row of the target's, where a draft was not accepted one of the draft's too
        return {"bytes": (B + cut) * V * es + 16 * B * case["drafts"], "flops": 3 * B * V}
    D = case["dim"]
    if op == "decode":
        lens, new = _context_lengths(case, 0)
        tok = lens if not case["window"] else np.minimum(lens, case["window"] + new - 1)
        read = int(tok.sum()) * case["hkv"] * 2 * D + int((tok // PAGE).sum()) * (8 * case["hkv"] + 4)
        seen = lens if not case["window"] else np.minimum(lens, case["window"])
        return {"bytes": read + int(new.sum()) * case["hq"] * (4 * D + 4),
                "flops": 4 * int((seen * new).sum()) * case["hq"] * D}
    n, hq, hkv, es = case["tokens"], case["hq"], case["hkv"], _T[case["dtype"]].itemsize
    flops = n * (hq + hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))
    if op == "append":
        kept = 1 - case["skipped"]
        return {"bytes": int(2 * n * (hq + 2 * hkv * kept) * D * es) + 12 * n, "flops": int(flops)}
    # rows in, q rows out, codes written; the touched pages' rows read back and written out
    slots, _, first, _ = _row_slots(case, 0)
    back = slots.size + first.size
    return {"bytes": n * (hq + 2 * hkv) * D * es + n * hq * D * es + 2 * n * hkv * D + 12 * n +
            2 * back * hkv * D * (1 + es) + 8 * back,
            "flops": flops + 4 * n * hkv * D}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "store": _exact_store, "decode": _exact_decode,
            "verify": _exact_verify}[case["op"]](case, state)


def _exact_heads(x, w, s):
    y = x.double()
    if w is not None:
        ms = torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / y.shape[-1]
        y = w.double() * y / torch.sqrt(ms + EPS)
    out = y.clone()
    rot = s["rot"]
    for i in range(rot // 2):
        phi = s["pos"].double() * math.pow(s["theta"], -2.0 * i / rot)
        c, sn = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        out[..., i] = c * y[..., i] - sn * y[..., i + rot // 2]
        out[..., i + rot // 2] = sn * y[..., i] + c * y[..., i + rot // 2]
    return out


def _exact_append(case, s):
    k = _exact_heads(s["k"], s["k_norm"], s)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    have = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, at = s["slots"][have] // PAGE, s["slots"][have] % PAGE
    kc[page, :, at] = k[have]
    vc[page, :, at] = s["v"][have].double()
    return [_exact_heads(s["q"], s["q_norm"], s), kc, vc]


def _below(x):
    """The power of two at or below a positive fp64 number: its significand's bits cleared."""
    return (x.contiguous().view(torch.int64) & (0x7FF << 52)).view(torch.float64)


def _e4m3(x):
    """fp64 to the nearest e4m3 value, ties to the even one: steps of 2^(e - 3), 2^-9 at least."""
    step = _below(torch.clamp(x.abs(), min=2.0 ** -6)) / 8
    return torch.round(x / step) * step


def _exact_store_one(s, name, rows):
    cache, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
    pages, hkv, _, D = cache.shape
    vals = torch.zeros(pages * PAGE, hkv, D, dtype=torch.float64, device=rows.device)
    vals[s["slots"]] = rows
    fresh = torch.zeros(pages * PAGE, dtype=torch.bool, device=rows.device)
    fresh[s["slots"]] = True
    vals, fresh = vals.view(pages, PAGE, hkv, D), fresh.view(pages, PAGE)
    amax = vals.abs().amax((1, 3))
    unit = _below(torch.clamp(amax, min=2.0 ** -112))  # 448 = 1.75 * 2^8
    least = torch.clamp(torch.where(amax > 1.75 * unit, 2 * unit, unit) / 256, min=2.0 ** -120)
    fits = torch.where(fresh[:, :1], least, torch.maximum(least, scales))
    fits = torch.where(fresh.any(1, keepdim=True), fits, scales)
    new = fits[:, None, :, None]
    old = cache.transpose(1, 2) * scales[:, None, :, None]
    res = _e4m3(torch.where(fresh[:, :, None, None], vals, old) / new) * new
    return res.reshape(pages * PAGE, hkv, D)[s["read"]]


def _exact_store(case, s):
    return [_exact_heads(s["q"], s["q_norm"], s),
            _exact_store_one(s, "k", _exact_heads(s["k"], s["k_norm"], s)),
            _exact_store_one(s, "v", s["v"].double())]


def _exact_decode(case, s):
    hq, hkv = case["hq"], case["hkv"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    starts = s["starts"].tolist()
    for b, L in enumerate(s["lens"].tolist()):
        r0, r1 = starts[b], starts[b + 1]
        if r0 == r1:
            continue
        ids = s["bt"][b, :(L + 15) // 16].long()
        for h in range(hkv):
            k = (s["k_cache"][ids, h].double() * s["k_scales"][ids, h].double()[:, None, None])
            v = (s["v_cache"][ids, h].double() * s["v_scales"][ids, h].double()[:, None, None])
            k, v = k.flatten(0, 1)[:L], v.flatten(0, 1)[:L]
            for r in range(r0, r1):
                end = L - (r1 - r) + 1
                begin = max(0, end - case["window"]) if case["window"] > 0 else 0
                x = k[begin:end] @ s["q"][r, h * g:(h + 1) * g].double().T * s["scale"]
                z = torch.logsumexp(x, 0)
                lse[r, h * g:(h + 1) * g] = z
                out[r, h * g:(h + 1) * g] = torch.exp(x - z).T @ v[begin:end]
    return [out, lse]


def _exact_verify(case, s):
    accepted, tokens = [], []
    for b, n in enumerate(s["num"].tolist()):
        p, q = s["target"][b].double().cpu().numpy(), s["draft"][b].double().cpu().numpy()
        x, u = s["draft_tokens"][b].tolist(), s["accept"][b].double().tolist()
        j = 0
        while j < n and u[j] * q[j, x[j]] < p[j, x[j]]:
            j += 1
        w = np.maximum(p[j] - q[j], 0) if j < n else p[j]
        c = np.cumsum(w)
        y = int(np.searchsorted(c, float(s["sample"][b]) * c[-1], side="right"))
        accepted.append(j)
        tokens.append(x[:j] + [y] + [-1] * (case["drafts"] - j))
    return [np.asarray(accepted, np.int32), np.asarray(tokens, np.int32)]
