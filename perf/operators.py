"""The operators around a paged KV cache held in 4 bits, as cases to be measured.

Four operators, each in a plain form (elementary torch operations, the default)
and as calls of this package (``own = True``):

  tables   block tables, context lengths, slot map and positions of a step,
           from the requests' lengths and a list of free pages
  rope     rotary embedding of q and k whose pairs take their position from
           one of several axes (time, height, width)
  store    new K/V rows quantised to 4 bits into the paged cache, and the same
           slots read back
  decode   one query token per sequence over the 4-bit paged cache

Sizes are the head counts, head dims and lengths of this package's own
workloads and tests, or generic ones around them.

The 4-bit cache.  uint8 [num_pages, Hkv, 20 D]: a page (16 tokens) of one KV
head is one block of 20 D bytes: K codes (8 D), V codes (8 D), K parameters
(2 D), V parameters (2 D).  32 consecutive dims of one token form a group with
a scale s and an offset z of the element type T (fp16 or bf16); a code c in
0..15 stands for RN_T(s (16 + c) + z).  _places() says where each lies.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
GROUP = 32
_T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_CLAMP = {"f16": 16384.0, "bf16": 2.0 ** 120}
_MANT = {torch.float16: (11, -14), torch.bfloat16: (8, -126)}  # significant bits, least exponent


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One request's decode step: the smallest bookkeeping there is.
        dict(name="tables_1", op="tables", batch=1, new="one", past=255, maxp=64, pad=0),
        # A mixed step of a busy server: mostly decodes, some long prompts.
        dict(name="tables_512_mixed", op="tables", batch=512, new="mixed", past=9000, maxp=1024,
             pad=37),
        # Decode step of 64 sequences, 32 query / 8 KV heads, text and image tokens.
        dict(name="rope_decode64", op="rope", tokens=64, hq=32, hkv=8, dim=128, rot=128,
             sections="16,24,24", interleaved=False, inverse=False, dtype="f16", theta=500000.0),
        # A prompt with images, heads of the long-context workload.
        dict(name="rope_prompt", op="rope", tokens=16384, hq=24, hkv=4, dim=256, rot=256,
             sections="44,42,42", interleaved=True, inverse=False, dtype="bf16", theta=10000.0),
        # fp32, odd token count, half of each head rotated, turned back (a gradient, or keys
        # that are to be moved).
        dict(name="rope_back_f32", op="rope", tokens=2049, hq=8, hkv=4, dim=64, rot=32,
             sections="4,6,6", interleaved=False, inverse=True, dtype="f32", theta=10000.0),
        # The decode step's new rows of 64 sequences.
        dict(name="store_decode64", op="store", tokens=64, hq=32, hkv=8, dim=128, dtype="f16",
             order="decode", skipped=0.0),
        # A long prompt, heads of the long-context workload.
        dict(name="store_prompt", op="store", tokens=16384, hq=24, hkv=4, dim=256, dtype="bf16",
             order="prompt", skipped=0.0),
        # A padded batch of prompts with an odd number of rows, some without a slot.
        dict(name="store_ragged_d96", op="store", tokens=4093, hq=32, hkv=8, dim=96, dtype="f16",
             order="prompt", skipped=0.1),
        # The single-sequence latency case of this package's benchmark.
        dict(name="decode_tiny_d64", op="decode", batch=1, hq=4, hkv=1, dim=64, length=256,
             spread="equal", window=0, dtype="f16"),
        # A serving batch of ragged lengths, bf16.
        dict(name="decode_ragged64", op="decode", batch=64, hq=32, hkv=8, dim=128, length=4096,
             spread="ragged", window=0, dtype="bf16"),
        # A sliding window that starts inside a page.
        dict(name="decode_window", op="decode", batch=4, hq=8, hkv=4, dim=256, length=8191,
             spread="equal", window=4096, dtype="f16"),
        # The long-context workload of this package's benchmark, its cache in 4 bits.
        dict(name="decode_100k", op="decode", batch=4, hq=24, hkv=4, dim=256, length=100000,
             spread="equal", window=0, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "store", "decode", "decode"])
    if op == "tables":
        batch = _log(rng, 1, 1024)
        return dict(op=op, batch=batch, new=rng.choice(["one", "mixed", "few"]),
                    past=_log(rng, 1, 9000), maxp=1024, pad=rng.randrange(0, 100))
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 96, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2])
        interleaved = rng.random() < 0.5
        half = rot // 2
        if interleaved:
            a = rng.randint(1, half // 3)
            b = rng.randint(1, half // 3)
        else:
            a = rng.randint(1, half // 2)
            b = rng.randint(0, half - a - 1)
        if rng.random() < 0.25:
            dtype = "f32"
        tokens = min(_log(rng, 1, 16384), (16384 * 28 * 256) // (hkv * (g + 1) * dim *
                                                                 (2 if dtype == "f32" else 1)))
        return dict(op=op, tokens=tokens, hq=g * hkv, hkv=hkv, dim=dim, rot=rot,
                    sections="%d,%d,%d" % (half - a - b, a, b), interleaved=interleaved,
                    inverse=rng.random() < 0.3, dtype=dtype,
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "store":
        return dict(op=op, tokens=min(_log(rng, 1, 16384), (16384 * 4 * 256) // (hkv * dim)),
                    hq=g * hkv, hkv=hkv, dim=dim, dtype=dtype,
                    order=rng.choice(["decode", "prompt"]), skipped=rng.choice([0.0, 0.0, 0.3]))
    batch = _log(rng, 1, 128)
    length = _log(rng, 1, 100000)
    length = max(1, min(length, (4 * 4 * 256 * 100000 // 4) // (batch * hkv * dim),
                        (4 * 24 * 256 * 100000 // 4) // (batch * hkv * g * dim)))
    return dict(op=op, batch=batch, hq=g * hkv, hkv=hkv, dim=dim, length=length,
                spread=rng.choice(["equal", "ragged"]),
                window=rng.choice([0, 0, 0, max(1, length // 3)]), dtype=dtype)


# ---------------------------------------------------------------- lengths from the seed

def _request_lengths(case, seed):
    """(past, new) of a tables case, host arrays.  How many new tokens there are goes by
    the case, which request has them by the seed."""
    g = np.random.default_rng([seed, 11])
    f = np.random.default_rng(11)
    B = case["batch"]
    past = g.integers(0, case["past"] + 1, size=B)
    if B == 1:
        past[0] = case["past"]
    if case["new"] == "one":
        new = np.ones(B, dtype=np.int64)
    elif case["new"] == "few":  # several tokens of each: verification of drafted ones
        new = g.permutation(f.integers(0, 9, size=B))
    else:  # decodes, a few idle requests, a few prompts
        new = np.ones(B, dtype=np.int64)
        new[f.random(B) < 0.05] = 0
        prompt = f.random(B) < 0.06
        new[prompt] = f.integers(1, 4097, size=int(prompt.sum()))
        new = g.permutation(new)
        past[new > 1] = 0
    return past.astype(np.int64), new.astype(np.int64)


def _context_lengths(case, seed):
    g = np.random.default_rng([seed, 12])
    B, L = case["batch"], case["length"]
    if case["spread"] == "equal":
        return np.full(B, L, dtype=np.int64)
    lens = g.integers(1, L + 1, size=B)
    lens[0] = L
    if B > 2:
        lens[-1] = 1
    if B > 4:
        lens[-2] = 0  # a request that has nothing cached yet
    return lens


# ---------------------------------------------------------------- the cache's layout

def _places(D, device):
    """Where a page block keeps (token r, dim d): byte and shift of K's and V's
    codes [16, D], and byte offsets of (s, z) of K and V [16, D / 32]."""
    r = torch.arange(PAGE, device=device).view(PAGE, 1)
    d = torch.arange(D, device=device).view(1, D)
    # K codes: slices of at most 128 dims; a slice keeps a token's dims in order, two a byte.
    sw = min(D, 128)
    kb = (d // sw) * (8 * sw) + r * (sw // 2) + (d % sw) // 2
    ks = 4 * (d % 2) + 0 * r
    # V codes: 32-bit words, 2 bytes of an even token (4 dims) and 2 of the odd one after it.
    # Word w of lane (g, t) has dims of column g and tokens 2 (4 h + t) and the next.
    vw = 4 if D % 128 == 0 else (2 if D == 64 else 1)
    if D == 96:
        w, g = d // 32, (d % 32) // 4
    else:
        w, g = (d % (D // 8)) // 4, d // (D // 8)
    p = d % 4
    h, t = r // 8, (r // 2) % 4
    vb = (8 * D + h * (4 * D) + (w // vw) * (128 * vw) + (4 * g + t) * (4 * vw) + (w % vw) * 4 +
          (r % 2) * 2 + p // 2)
    vs = 4 * (p % 2) + 0 * r
    n = torch.arange(D // GROUP, device=device).view(1, -1)
    ns = sw // GROUP
    kp = 16 * D + (((n // ns) * PAGE + r) * ns + n % ns) * 4
    vp = 18 * D + ((r // 2) * (D // GROUP) + n) * 8 + (r % 2) * 2
    return kb, ks, vb, vs, (kp, kp + 2), (vp, vp + 4)


def _pair(block, at, dtype):
    """16-bit values whose low byte lies at `at` of each block."""
    lo = block[..., at].to(torch.int32)
    hi = block[..., at + 1].to(torch.int32)
    u = lo | (hi << 8)
    u = torch.where(u >= 32768, u - 65536, u).to(torch.int16)
    return u.view(dtype)


def _unpack(block, D, dtype):
    """K and V that page blocks [..., 20 D] stand for: fp32 [..., 16, D], values of T."""
    kb, ks, vb, vs, kp, vp = _places(D, block.device)
    out = []
    for b, s, (ps, pz) in ((kb, ks, kp), (vb, vs, vp)):
        c = ((block[..., b] >> s) & 15).to(torch.float32)
        sc = _pair(block, ps, dtype).float().repeat_interleave(GROUP, dim=-1)
        ze = _pair(block, pz, dtype).float().repeat_interleave(GROUP, dim=-1)
        # s (16 + c) has at most 16 significant bits: exact in fp32.
        out.append((sc * (16 + c) + ze).to(dtype).float())
    return out


def _pack(k, v, D, dtype):
    """Page blocks [n, 20 D] of K and V [n, 16, D] (fp32 values), for inputs."""
    n = k.shape[0]
    kb, ks, vb, vs, kp, vp = _places(D, k.device)
    block = torch.zeros(n, 20 * D, dtype=torch.uint8, device=k.device)
    for x, b, (ps, pz) in ((k, kb, kp), (v, vb, vp)):
        gx = x.view(n, PAGE, D // GROUP, GROUP)
        mn, mx = gx.amin(-1), gx.amax(-1)
        s = ((mx - mn) / 15).to(dtype)
        z = (mn - 16 * s.float()).to(dtype)
        c = ((gx - z.float()[..., None]) / s.float()[..., None] - 16).round().clamp(0, 15)
        c = c.view(n, PAGE, D).to(torch.uint8)
        # dims d and d + 1 share a byte, the even one in its low half
        block[:, b[:, 0::2]] = c[..., 0::2] | (c[..., 1::2] << 4)
        for val, at in ((s, ps), (z, pz)):
            bits = val.contiguous().view(torch.int16).to(torch.int32) & 0xFFFF
            block[:, at] = (bits & 255).to(torch.uint8)
            block[:, at + 1] = (bits >> 8).to(torch.uint8)
    return block


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    return {"tables": _prepare_tables, "rope": _prepare_rope, "store": _prepare_store,
            "decode": _prepare_decode}[case["op"]](case, seed, dev, gen)


def _prepare_tables(case, seed, dev, gen):
    past, new = _request_lengths(case, seed)
    B, maxp = case["batch"], case["maxp"]
    have = -(-past // PAGE)
    need = -(-(past + new) // PAGE)
    taken = int((need - have).sum())
    pages = int(have.sum()) + taken + 64
    perm = np.random.default_rng([seed, 13]).permutation(pages).astype(np.int32)
    bt = np.full((B, maxp), -1, dtype=np.int32)
    off = 0
    for b in range(B):
        bt[b, :have[b]] = perm[off:off + have[b]]
        off += have[b]
    cap = int(new.sum()) + case["pad"]  # the buffers of a padded step

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    return dict(op="tables", past=i32(past), new=i32(new), free=i32(perm[off:]), num_pages=pages,
                bt=i32(bt), lens=torch.zeros(B, dtype=torch.int32, device=dev),
                starts=torch.zeros(B + 1, dtype=torch.int32, device=dev),
                slots=torch.zeros(max(cap, 1), dtype=torch.int64, device=dev),
                positions=torch.zeros(max(cap, 1), dtype=torch.int32, device=dev),
                taken=torch.zeros(1, dtype=torch.int32, device=dev))


def _axis_positions(tokens, seed):
    """Positions [3, tokens] of prompts of text with images between: along text the
    axes agree, inside an image time stands still and height and width count."""
    g = np.random.default_rng([seed, 14])
    out = np.zeros((3, tokens), dtype=np.int64)
    i, pos = 0, int(g.integers(0, 100000))
    while i < tokens:
        n = min(int(g.integers(1, 400)), tokens - i)
        out[:, i:i + n] = pos + np.arange(n)
        i += n
        pos += n
        hgt, wid = int(g.integers(4, 40)), int(g.integers(4, 40))
        n = min(hgt * wid, tokens - i)
        j = np.arange(n)
        out[0, i:i + n] = pos
        out[1, i:i + n] = pos + j // wid
        out[2, i:i + n] = pos + j % wid
        i += n
        pos += max(hgt, wid)
    return out


def _prepare_rope(case, seed, dev, gen):
    n, hq, hkv, D = case["tokens"], case["hq"], case["hkv"], case["dim"]
    dt = _T[case["dtype"]]
    # q and k as the first columns of a fused projection's rows
    qkv = torch.randn(n, hq + 2 * hkv, D, generator=gen, device=dev).to(dt)
    pos = torch.from_numpy(_axis_positions(n, seed).astype(np.int32)).to(dev)
    return dict(op="rope", q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], pos=pos,
                sections=tuple(int(x) for x in case["sections"].split(",")), rot=case["rot"],
                theta=case["theta"], interleaved=case["interleaved"], inverse=case["inverse"],
                q_out=torch.empty(n, hq, D, dtype=dt, device=dev),
                k_out=torch.empty(n, hkv, D, dtype=dt, device=dev))


def _kv_rows(shape, gen, dev):
    """K- or V-like rows: normal values around a bias of each channel, some channels wide."""
    D = shape[-1]
    wide = 1 + 4 * (torch.rand(D, generator=gen, device=dev) < 0.03).float()
    bias = torch.randn(D, generator=gen, device=dev) * 0.5
    return torch.randn(shape, generator=gen, device=dev) * wide + bias


def _prepare_store(case, seed, dev, gen):
    n, hq, hkv, D = case["tokens"], case["hq"], case["hkv"], case["dim"]
    dt = _T[case["dtype"]]
    qkv = torch.zeros(n, hq + 2 * hkv, D, dtype=dt, device=dev)
    qkv[:, hq:] = _kv_rows((n, 2 * hkv, D), gen, dev).to(dt)
    g = np.random.default_rng([seed, 15])
    if case["order"] == "decode":  # every row in a page of its own sequence
        pages = n + n // 4 + 1
        slots = g.permutation(pages)[:n].astype(np.int64) * PAGE + g.integers(0, PAGE, size=n)
    else:  # runs of a prompt's rows through shuffled pages
        pages = (n + PAGE) // PAGE + 1 + n // 64
        perm = g.permutation(pages)
        flat = int(g.integers(0, PAGE)) + np.arange(n)
        slots = perm[flat // PAGE].astype(np.int64) * PAGE + flat % PAGE
    if case["skipped"]:
        slots[g.random(n) < case["skipped"]] = -1
    return dict(op="store", dtype=dt, k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                slots=torch.from_numpy(slots).to(dev),
                cache=torch.zeros(pages, hkv, 20 * D, dtype=torch.uint8, device=dev),
                k_out=torch.empty(n, hkv, D, dtype=dt, device=dev),
                v_out=torch.empty(n, hkv, D, dtype=dt, device=dev))


def _prepare_decode(case, seed, dev, gen):
    B, hq, hkv, D = case["batch"], case["hq"], case["hkv"], case["dim"]
    dt = _T[case["dtype"]]
    lens = _context_lengths(case, seed)
    need = -(-lens // PAGE)
    total = int(need.sum())
    pages = total + total // 8 + 1
    perm = np.random.default_rng([seed, 16]).permutation(pages).astype(np.int32)
    maxp = max(1, int(need.max()))
    bt = np.full((B, maxp), -1, dtype=np.int32)
    off = 0
    for b in range(B):
        bt[b, :need[b]] = perm[off:off + need[b]]
        off += need[b]
    # pages that no sequence owns hold whatever was there
    cache = torch.full((pages, hkv, 20 * D), 255, dtype=torch.uint8, device=dev)
    owned = torch.from_numpy(perm[:off].astype(np.int64)).to(dev)
    for lo in range(0, off, 2048):
        ids = owned[lo:lo + 2048]
        n = ids.numel() * hkv
        k = _kv_rows((n, PAGE, D), gen, dev).to(dt).float()
        v = _kv_rows((n, PAGE, D), gen, dev).to(dt).float()
        cache[ids] = _pack(k, v, D, dt).view(-1, hkv, 20 * D)
    q = torch.randn(B, hq, D, generator=gen, device=dev).to(dt)
    st = dict(op="decode", dtype=dt, q=q, cache=cache, bt=torch.from_numpy(bt).to(dev),
              lens=torch.from_numpy(lens.astype(np.int32)).to(dev), window=case["window"],
              scale=1.0 / math.sqrt(D), out=torch.empty_like(q),
              lse=torch.empty(B, hq, dtype=torch.float32, device=dev))
    if own:
        import paged_kv_gqa_pa_gb300 as pa
        st["plan"] = pa.pa_q4_plan(B, hq, hkv, D, PAGE, pages, maxp, int(lens.max()),
                                   window=case["window"],
                                   dtype=1 if case["dtype"] == "bf16" else 0)
        st["ws"] = pa.new_workspace(st["plan"], dev)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_tables(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_extend_tables(s["past"], s["new"], s["free"], s["num_pages"], s["bt"], s["lens"],
                        s["starts"], s["slots"], s["positions"], s["taken"])
    return [s["bt"], s["lens"], s["starts"], s["slots"], s["positions"], s["taken"]]


def _own_rope(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_rope_axes(s["q"], s["k"], s["pos"], s["sections"], s["theta"], q_out=s["q_out"],
                    k_out=s["k_out"], rotary_dim=s["rot"], interleaved=s["interleaved"],
                    inverse=s["inverse"])
    return [s["q_out"], s["k_out"]]


def _own_store(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_q4_write(s["k"], s["v"], s["slots"], s["cache"])
    pa.pa_q4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return [s["k_out"], s["v_out"]]


def _own_decode(s):
    import paged_kv_gqa_pa_gb300 as pa
    pa.pa_q4_decode(s["plan"], s["q"], s["cache"], s["bt"], s["lens"], s["scale"], s["window"],
                    s["out"], s["lse"], s["ws"])
    return [s["out"], s["lse"]]


def _plain_tables(s):
    past, new, bt = s["past"].long(), s["new"].long(), s["bt"]
    B, cap = past.numel(), s["slots"].numel()
    lens = past + new
    have, need = (past + PAGE - 1) // PAGE, (lens + PAGE - 1) // PAGE
    add = need - have
    first = torch.cumsum(add, 0) - add
    # new table entries: entry j of a row is new where have <= j < need
    col = torch.arange(bt.shape[1], device=bt.device)
    fresh = (col >= have[:, None]) & (col < need[:, None])
    src = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    bt.copy_(torch.where(fresh, s["free"][src], bt))
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    tok = torch.arange(cap, device=bt.device)
    live = tok < ends[-1]
    b = torch.searchsorted(ends, tok, right=True).clamp(max=B - 1)
    pos = torch.where(live, past[b] + tok - starts[b], 0)
    page = bt[b, (pos // PAGE).clamp(max=bt.shape[1] - 1)].long()
    slots = torch.where(live, page * PAGE + pos % PAGE, -1)
    return [bt, lens.int(), starts.int(), slots, pos.int(), add.sum().int().view(1)]


def _axis_of(half, sections, interleaved):
    """Axis of every pair: sections one after another, or axes taken in turn
    (the first axis has what the others leave)."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    k = len(sections)
    return [i % k if i % k and i < k * sections[i % k] else 0 for i in range(half)]


def _plain_rope(s):
    rot, half = s["rot"], s["rot"] // 2
    axis = torch.tensor(_axis_of(half, s["sections"], s["interleaved"]), device=s["pos"].device)
    i = torch.arange(half, dtype=torch.float64, device=axis.device)
    ang = s["pos"][axis].double().T * s["theta"] ** (-2.0 * i / rot)  # far positions: 64 bits
    if s["inverse"]:
        ang = -ang
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    out = []
    for x in (s["q"], s["k"]):
        f = x.float()
        a, b = f[..., :half], f[..., half:rot]
        out.append(torch.cat([a * cos - b * sin, b * cos + a * sin, f[..., rot:]], -1).to(x.dtype))
    return out


def _rn(x, dtype):
    """fp64 rounded once to T (a cast would go through fp32)."""
    bits, emin = _MANT[dtype]
    _, e = torch.frexp(x)
    e = torch.clamp(e - 1, min=emin) - (bits - 1)
    step = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e
    return torch.round(x / step) * step


def _plain_store(s):
    out = []
    lim = _CLAMP["f16" if s["dtype"] == torch.float16 else "bf16"]
    there = (s["slots"] >= 0)[:, None, None]
    for x in (s["k"], s["v"]):
        n, hkv, D = x.shape
        g = x.double().reshape(n, hkv, D // GROUP, GROUP)  # 64 bits: codes next to a border
        mn, mx = g.amin(-1, keepdim=True).clamp(-lim, lim), g.amax(-1, keepdim=True).clamp(-lim, lim)
        sc = _rn((mx - mn) / g.new_full((1,), 15.0), s["dtype"])  # (a number would be multiplied by 1/15)
        ze = _rn(mn - 16 * sc, s["dtype"])
        c = torch.round((g - ze) / sc - 16).clamp(0, 15)
        c = torch.where(sc == 0, torch.zeros_like(c), c)
        val = _rn(sc * (16 + c) + ze, s["dtype"]).reshape(n, hkv, D)
        out.append(torch.where(there, val, torch.zeros_like(val)).to(s["dtype"]))
    return out


def _plain_decode(s):
    q, lens, dt = s["q"].float(), s["lens"].long(), s["dtype"]
    B, hq, D = q.shape
    pages, hkv, _ = s["cache"].shape
    bt = s["bt"].long().clamp(min=0)
    P = bt.shape[1]
    g = hq // hkv
    window = s["window"]
    pos = torch.arange(P * PAGE, device=q.device)
    lo = (lens - window).clamp(min=0) if window > 0 else torch.zeros_like(lens)
    seen = (pos < lens[:, None]) & (pos >= lo[:, None])
    qg = q.view(B, hkv, g, D)
    scores = torch.empty(B, hkv, g, P * PAGE, device=q.device)
    acc = torch.zeros(B, hkv, g, D, device=q.device)
    step = max(1, (1 << 17) // (B * hkv))  # table columns a block, for the memory of the unpacked values
    vals = []
    for c0 in range(0, P, step):
        k, v = _unpack(s["cache"][bt[:, c0:c0 + step]], D, dt)  # [B, p, hkv, 16, D]
        n = k.shape[1] * PAGE
        k = k.permute(0, 2, 1, 3, 4).reshape(B, hkv, n, D)
        v = v.permute(0, 2, 1, 3, 4).reshape(B, hkv, n, D)
        m = seen[:, c0 * PAGE:c0 * PAGE + n]
        vals.append(torch.where(m[:, None, :, None], v, 0.0))
        scores[..., c0 * PAGE:c0 * PAGE + n] = torch.where(
            m[:, None, None], torch.matmul(qg, k.transpose(2, 3)) * s["scale"], -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    at = 0
    for v in vals:
        acc += torch.matmul(w[..., at:at + v.shape[2]], v)
        at += v.shape[2]
    out = acc / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    return [out.view(B, hq, D).to(dt), lse.view(B, hq)]


_OWN = {"tables": _own_tables, "rope": _own_rope, "store": _own_store, "decode": _own_decode}
_PLAIN = {"tables": _plain_tables, "rope": _plain_rope, "store": _plain_store,
          "decode": _plain_decode}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "tables":
        past, new = _request_lengths(case, 0)
        B, n = case["batch"], int(new.sum())
        add = int((-(-(past + new) // PAGE) + (past // -PAGE)).sum())
        # lengths in and out, starts, free pages read, entries written, the page of each token's
        # slot, slots and positions
        return {"bytes": B * 16 + add * 8 + n * 4 + (n + case["pad"]) * 12, "flops": 0}
    D = case["dim"]
    if op == "rope":
        n, h, es = case["tokens"], case["hq"] + case["hkv"], _T[case["dtype"]].itemsize
        return {"bytes": 2 * n * h * D * es + 12 * n, "flops": 3 * n * h * case["rot"]}
    if op == "store":
        rows = case["tokens"] * case["hkv"]
        kept = rows * (1 - case["skipped"])
        # rows in, their cells written, the cells read back, rows out
        return {"bytes": int(kept * (4 * D + 2.5 * D) + rows * 4 * D + 16 * case["tokens"]),
                "flops": int(12 * 2 * D * kept)}
    lens = _context_lengths(case, 0)
    if case["window"] > 0:
        lens = np.minimum(lens, case["window"])
    tok = int(lens.sum())
    io = case["batch"] * case["hq"] * (4 * D + 4)
    return {"bytes": int(tok * case["hkv"] * 1.25 * D) + io + 4 * (tok // PAGE),
            "flops": 4 * tok * case["hq"] * D}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "store": _exact_store,
            "decode": _exact_decode}[case["op"]](case, state)


def _exact_tables(case, s):
    past, new = s["past"].tolist(), s["new"].tolist()
    free, bt = s["free"].tolist(), s["bt"].cpu().numpy().copy()
    slots = np.full(s["slots"].numel(), -1, dtype=np.int64)
    positions = np.zeros(slots.size, dtype=np.int32)
    starts, lens, used, n = [0], [], 0, 0
    for b, (p, m) in enumerate(zip(past, new)):
        held = (p + 15) // 16
        while held * 16 < p + m:
            bt[b, held] = free[used]
            used += 1
            held += 1
        for x in range(p, p + m):
            slots[n] = int(bt[b, x // 16]) * 16 + x % 16
            positions[n] = x
            n += 1
        lens.append(p + m)
        starts.append(n)
    return [bt, np.asarray(lens, np.int32), np.asarray(starts, np.int32), slots, positions,
            np.asarray([used], np.int32)]


def _exact_rope(case, s):
    rot, k = case["rot"], len(s["sections"])
    half = rot // 2
    pos = s["pos"].double()
    sign = -1.0 if case["inverse"] else 1.0
    turned = []
    for x in (s["q"], s["k"]):
        y = x.double()
        turned.append((y, y.clone()))
    ends = np.cumsum(s["sections"])
    for i in range(half):
        if case["interleaved"]:
            a = i % k
            if a > 0 and i >= k * s["sections"][a]:
                a = 0
        else:
            a = int(np.searchsorted(ends, i, side="right"))
        phi = sign * pos[a] * math.pow(case["theta"], -2.0 * i / rot)
        c, sn = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        for y, o in turned:
            o[..., i] = c * y[..., i] - sn * y[..., i + half]
            o[..., i + half] = sn * y[..., i] + c * y[..., i + half]
    return [o for _, o in turned]


def _nearest(x, dtype):
    """fp64 to the nearest value of T, ties to the even one, by its neighbours."""
    bits, emin = _MANT[dtype]
    mag = torch.clamp(x.abs(), min=2.0 ** emin).contiguous()
    # the power of two below: the significand's bits cleared
    unit = (mag.view(torch.int64) & (0x7FF << 52)).view(torch.float64) * 2.0 ** (1 - bits)
    down = torch.floor(x / unit)
    rest = x / unit - down
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(down, 2) == 1))
    return (down + up.double()) * unit


def _exact_store(case, s):
    out = []
    lim = _CLAMP[case["dtype"]]
    dt = s["dtype"]
    for x in (s["k"], s["v"]):
        y = x.double().contiguous()
        res = torch.zeros_like(y)
        for d0 in range(0, case["dim"], GROUP):
            part = y[..., d0:d0 + GROUP]
            low = part.min(-1).values.clamp(-lim, lim)
            high = part.max(-1).values.clamp(-lim, lim)
            s1 = _nearest((high - low) / torch.full_like(low, 15), dt)
            z1 = _nearest(low - 16 * s1, dt)
            # the code whose 16 + c lies nearest to (x - z) / s, the even one of two
            u = (part - z1[..., None]) / torch.where(s1 == 0, 1.0, s1)[..., None] - 16
            c = torch.floor(u)
            rest = u - c
            c = c + ((rest > 0.5) | ((rest == 0.5) & (torch.remainder(c, 2) == 1))).double()
            c = torch.where((s1 == 0)[..., None], 0.0, torch.clamp(c, 0, 15))
            res[..., d0:d0 + GROUP] = _nearest(s1[..., None] * (16 + c) + z1[..., None], dt)
        res[s["slots"] < 0] = 0
        out.append(res)
    return out


def _nibbles(b):
    """Bytes to codes: the low half first."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _exact_pages(block, D, dtype):
    """fp64 K, V [n, 16, D] of page blocks [n, 20 D], by the blocks' own structure."""
    n = block.shape[0]
    sl = max(1, D // 128)
    sw = D // sl
    kc = _nibbles(block[:, :8 * D].reshape(n, sl, 16, sw // 2)).permute(0, 2, 1, 3).reshape(n, 16, D)
    vw = {64: 2, 96: 1, 128: 4, 256: 4}[D]
    raw = block[:, 8 * D:16 * D].reshape(n, 2, D // 32 // vw, 8, 4, vw, 2, 2)  # h, s, g, t, w, odd, byte
    raw = _nibbles(raw)  # h, s, g, t, w, odd, p
    if D == 96:
        vc = raw.permute(0, 1, 4, 6, 2, 5, 3, 7)  # h, t, odd, s, (w), g, p
    else:
        vc = raw.permute(0, 1, 4, 6, 3, 2, 5, 7)  # h, t, odd, g, s, w, p
    vc = vc.reshape(n, 16, D)
    par = block[:, 16 * D:].contiguous().view(dtype).double()
    kp = par[:, :D].reshape(n, sl, 16, sw // 32, 2).permute(0, 2, 1, 3, 4).reshape(n, 16, D // 32, 2)
    vp = par[:, D:].reshape(n, 8, D // 32, 2, 2).permute(0, 1, 4, 2, 3).reshape(n, 16, D // 32, 2)
    out = []
    for c, p in ((kc, kp), (vc, vp)):
        c = c.reshape(n, 16, D // 32, 32).double()
        out.append(_nearest(p[..., :1] * (16 + c) + p[..., 1:], dtype).reshape(n, 16, D))
    return out


def _exact_decode(case, s):
    B, hq, hkv, D = case["batch"], case["hq"], case["hkv"], case["dim"]
    g = hq // hkv
    out = torch.zeros(B, hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        begin = max(0, L - case["window"]) if case["window"] > 0 else 0
        first = begin // 16
        ids = s["bt"][b, first:(L + 15) // 16].long()
        for h in range(hkv):
            k, v = _exact_pages(s["cache"][ids, h], D, s["dtype"])
            k = k.reshape(-1, D)[begin - first * 16:L - first * 16]
            v = v.reshape(-1, D)[begin - first * 16:L - first * 16]
            x = k @ s["q"][b, h * g:(h + 1) * g].double().T * s["scale"]  # [tokens, g]
            z = torch.logsumexp(x, 0)
            lse[b, h * g:(h + 1) * g] = z
            out[b, h * g:(h + 1) * g] = torch.exp(x - z).T @ v
    return [out, lse]
