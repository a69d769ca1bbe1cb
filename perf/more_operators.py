"""What is measured of the 4-bit paged KV cache and of the page plan: laying out a serving step's pages,
slots and positions, storing rows in the cache, decoding and prefilling over it.

Each case is one call sequence as a serving program makes it. `own = False` computes the operator in
its plain form (elementary torch operations in fp32, angles in fp64); `own = True` calls the library.
`exact` computes the definition in fp64 (whole numbers for the plan) from the same inputs, request by
request, without the byte layouts.

The stored form of a head vector x (fp32), one scale per 32 columns (microscaled 4-bit floating point):
  a = max |x| over the block,  E = floor(log2 a) - 2, one more when a > 7 * 2^E,
  value = the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} * 2^E (ties to the even code, 6 at most),
  scale byte E + 127. A block with a < 2^-77 is zeros, scale 0; E is at most 125; a vector that
  holds an infinity or NaN is NaN throughout (scales 255).
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 16
MAX_POS = 262144
HEADS = 32
WINDOW = 1024
# head dim, turning pairs, KV heads and RoPE base of the two layer kinds
GEOM = {"sliding": dict(d=256, r=128, kv=16, theta=1.0e4), "global": dict(d=512, r=64, kv=4, theta=1.0e6)}
EPS = 1e-6


# ---- the cases -------------------------------------------------------------------------------------

def listed():
    mix = dict(batch=64, len_lo=1024, len_hi=32768, len_seed=7)
    return [
        # One decode step of the ragged serving mix: a token per request, on both layer kinds' pools.
        dict(name="plan 64 decode", op="plan", batch=64, ctx_lo=1024, ctx_hi=32768, rows_hi=1, prompts=0.0, idle=0.0,
             ended=0.0, supply=2.0, evicted=False, groups=2, len_seed=7),
        # Chunked prompts among decoding requests; some requests ended, pages came back from the eviction.
        dict(name="plan 300 mixed", op="plan", batch=300, ctx_lo=1, ctx_hi=16384, rows_hi=2048, prompts=0.1, idle=0.1,
             ended=0.05, supply=1.5, evicted=True, groups=2, len_seed=11),
        # The largest batch, prompts arriving faster than pages free up: some of them have to wait.
        dict(name="plan 4096 short of pages", op="plan", batch=4096, ctx_lo=1, ctx_hi=8192, rows_hi=1024, prompts=0.05,
             idle=0.02, ended=0.05, supply=0.8, evicted=True, groups=2, len_seed=13),
        # Two short prompts admitted together (ragged, below one tile): the smallest store.
        dict(name="store sliding 96+200", op="store", kind="sliding", tp=1, norms=False, batch=2, rows_lo=96,
             rows_hi=200, ctx_lo=0, ctx_hi=0, len_seed=3),
        # The new tokens of one decode step of 64 requests, with the model's q/k/v norms: one row each.
        dict(name="store global 64x1 normed", op="store", kind="global", tp=1, norms=True, batch=64, rows_lo=1,
             rows_hi=1, ctx_lo=1023, ctx_hi=32767, len_seed=7),
        # Four long prompts of a sliding layer stored in one go: bandwidth.
        dict(name="store sliding 4x4096", op="store", kind="sliding", tp=1, norms=False, batch=4, rows_lo=4096,
             rows_hi=4096, ctx_lo=0, ctx_hi=0, len_seed=1),
        # One short request alone on a global layer: latency.
        dict(name="decode global 1x37", op="decode", kind="global", tp=1, norms=False, weights=False, batch=1, len_lo=37,
             len_hi=37, len_seed=1, shift=0),
        # One very long request: its keys split over the whole card; evicted pages before it, weights kept.
        dict(name="decode global 1x131072", op="decode", kind="global", tp=1, norms=False, weights=True, batch=1,
             len_lo=131072, len_hi=131072, len_seed=1, shift=640),
        # The ragged serving mix on a global layer and on a sliding one.
        dict(name="decode global mix 64", op="decode", kind="global", tp=1, norms=False, weights=False, shift=0, **mix),
        dict(name="decode sliding mix 64", op="decode", kind="sliding", tp=1, norms=True, weights=False, shift=0, **mix),
        # Whole prompts over an empty cache.
        dict(name="prefill sliding 4x4096", op="prefill", kind="sliding", tp=1, norms=False, image=False, batch=4,
             rows_lo=4096, rows_hi=4096, ctx_lo=0, ctx_hi=0, len_seed=1),
        # Ragged chunks of long prompts over their cached history, normed, an image in each.
        dict(name="prefill global 3 chunks", op="prefill", kind="global", tp=1, norms=True, image=True, batch=3,
             rows_lo=65, rows_hi=515, ctx_lo=1024, ctx_hi=32768, len_seed=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "decode", "decode", "prefill"])
    if op == "plan":
        batch = _log_int(rng, 1, 4096)
        ctx = _log_int(rng, 1, min(131072, 8192 * 4096 // batch))
        return dict(op=op, batch=batch, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx,
                    rows_hi=_log_int(rng, 1, min(8192, 1024 * 4096 // batch)), prompts=rng.choice([0.0, 0.05, 0.3]),
                    idle=rng.choice([0.0, 0.1]), ended=rng.choice([0.0, 0.05, 0.3]), supply=rng.choice([0.6, 1.2, 3.0]),
                    evicted=rng.random() < 0.5, groups=rng.choice([1, 2, 2]), len_seed=rng.randrange(1 << 20))
    c = dict(op=op, kind=rng.choice(["sliding", "global"]), tp=rng.choice([1, 1, 1, 2, 4, 8]),
             norms=rng.random() < 0.4, len_seed=rng.randrange(1 << 20))
    if op == "decode":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(131072, 32768 * 32 // batch))
        c.update(batch=batch, len_lo=rng.randint(1, hi), len_hi=hi,
                 weights=c["kind"] == "global" and rng.random() < 0.5, shift=rng.choice([0, 0, rng.randint(1, 1000)]))
        return c
    batch = _log_int(rng, 1, 16)
    hi = _log_int(rng, 1, 16384 // batch if op == "store" else min(2048, 8192 // batch))
    ctx = 0 if rng.random() < 0.4 else _log_int(rng, 1, 16384 // batch)
    c.update(batch=batch, rows_lo=rng.randint(1, hi), rows_hi=hi, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    if op == "prefill":
        c["image"] = rng.random() < 0.3
    return c


# ---- sizes -----------------------------------------------------------------------------------------

def _between(lo, hi, n, seed):
    """n whole numbers in [lo, hi]; the first two are the ends."""
    r = random.Random(seed)
    v = [r.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[1] = lo
    return v


def _sizes(case):
    """(rows, ctx) of each sequence; a decode sequence has its length as ctx and no rows."""
    n, seed = case["batch"], case["len_seed"]
    if case["op"] == "decode":
        return [0] * n, _between(case["len_lo"], case["len_hi"], n, seed)
    return _between(case["rows_lo"], case["rows_hi"], n, seed), _between(case["ctx_lo"], case["ctx_hi"], n, seed + 1)


def _requests(case):
    """(tokens held, new tokens) of each request of a plan: 1 decoding, more for a prompt or its chunk, 0
    idle, -1 ended."""
    r = random.Random(case["len_seed"])
    ctx, new = _between(case["ctx_lo"], case["ctx_hi"], case["batch"], case["len_seed"] + 1), []
    for b in range(case["batch"]):
        x = r.random()
        if x < case["prompts"]:
            new.append(r.randint(1, case["rows_hi"]))
            if r.random() < 0.5:
                ctx[b] = 0
        elif x < case["prompts"] + case["idle"]:
            new.append(0)
        elif x < case["prompts"] + case["idle"] + case["ended"]:
            new.append(-1)
        else:
            new.append(1)
    return ctx, new


def _pages_of(tokens):
    return (tokens + PAGE - 1) // PAGE


def _heads(case):
    g = GEOM[case["kind"]]
    return HEADS // case["tp"], max(1, g["kv"] // case["tp"])


def _first_key(case, first_row):
    """The first key that a query at first_row sees."""
    return max(0, first_row - WINDOW + 1) if case["kind"] == "sliding" else 0


def _vector_bytes(case):
    """Bytes of one key of one head: 4-bit with a scale byte per 32 columns, and in bf16."""
    return (256 + 16, 2 * 512) if case["kind"] == "sliding" else (256 + 64 + 20, 2 * 640)


def work(case):
    if case["op"] == "plan":
        ctx, new = _requests(case)
        rows = sum(max(n, 0) for n in new)
        pages = 0
        for c, n in zip(ctx, new):
            pages += _pages_of(c) if n < 0 else _pages_of(c + n) - _pages_of(c)
        g = case["groups"]
        return {"bytes": float(case["batch"] * (24 + 16 * g) + rows * (4 + 8 * g) + 8 * g * pages), "flops": float(rows)}
    rows, ctx = _sizes(case)
    hq, hkv = _heads(case)
    d = GEOM[case["kind"]]["d"]
    b4, b16 = _vector_bytes(case)
    raw = 2 * d * (2 if case["kind"] == "sliding" else 1)   # bf16 bytes of one row's new k (and v) of one head
    if case["op"] == "store":
        return {"bytes": float(sum(rows) * hkv * (raw + b4 + b16)), "flops": 10.0 * sum(rows) * hkv * d}
    if case["op"] == "decode":
        keys = sum(L - _first_key(case, L - 1) for L in ctx)
        qo = 4 * case["batch"] * hq * d
        w = 8 * sum(_pages_of(L) for L in ctx) if case["weights"] else 0
        return {"bytes": float(keys * hkv * b4 + qo + w + 4 * sum(_pages_of(L) for L in ctx)),
                "flops": 4.0 * d * hq * keys}
    pairs, seen, hist = 0, 0, 0
    for n, c in zip(rows, ctx):
        seen += c + n - _first_key(case, c)
        hist += c - _first_key(case, c)
        s0, s1 = _image(case, n, c)
        for i in range(c, c + n):
            lo, hi = _first_key(case, i), i + 1
            if s0 <= i < s1:
                lo, hi = min(lo, s0), max(hi, s1)
            pairs += hi - lo
    bytes_ = sum(rows) * (4 * hq * d + hkv * (raw + b4)) + hist * hkv * b4 + seen * hkv * b16
    return {"bytes": float(bytes_), "flops": 4.0 * d * hq * pairs}


def _image(case, rows, ctx):
    """The positions of a sequence's image: the middle of its new rows; none in very short chunks."""
    if not case["image"] or rows < 3:
        return 0, 0
    return ctx + rows // 4, ctx + rows // 4 + max(1, rows // 2)


# ---- the 4-bit form ----------------------------------------------------------------------------------

STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """fp32 head vectors [..., n] -> codes uint8 [..., n] (sign in bit 3) and scales uint8 [..., n / 32]."""
    blocks = x.unflatten(-1, (-1, 32))
    bits = blocks.abs().amax(-1).view(torch.int32)
    e = ((bits + 0x1FFFFF) >> 23).clamp(max=254)             # the exponent; one more from 1.75 on
    scale = torch.where(e < 50, torch.zeros_like(e), e - 2)
    m = blocks.abs() * ((254 - scale.clamp(min=48)) << 23).view(torch.float32)[..., None]
    step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = torch.where(m <= 2.0, m * 2.0, torch.where(m <= 4.0, m + 2.0, 7.0)) + 8.0 * (blocks < 0)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    code = torch.where((scale == 0)[..., None] | bad[..., None], torch.zeros_like(code), code)
    scale = torch.where(bad, torch.full_like(scale, 255), scale)
    return code.nan_to_num().to(torch.uint8).flatten(-2), scale.to(torch.uint8)


def _values(code, scale, dtype=torch.float32):
    """The values that codes [..., n] with scales [..., n / 32] stand for."""
    table = torch.tensor(STEPS + tuple(-s for s in STEPS), dtype=dtype, device=code.device)
    f = torch.exp2(scale.to(dtype) - 127.0)
    f = torch.where(scale == 255, torch.full_like(f, float("nan")), f)
    return (table[code.int()].unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


# ---- inputs ----------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cos_sin(case, pos):
    g = GEOM[case["kind"]]
    t = torch.arange(g["r"], dtype=torch.float64, device=pos.device)
    a = pos.double()[..., None] * g["theta"] ** (-2.0 * t / g["d"])
    return torch.cos(a), torch.sin(a)


def _rope(case, x, pos):
    """RoPE of fp32 vectors [..., H, d] at positions [...]: pairs (t, t + d/2), t < r, turn."""
    g = GEOM[case["kind"]]
    c, s = (v[..., None, :].to(x.dtype) for v in _cos_sin(case, pos))
    r, h = g["r"], g["d"] // 2
    a, b = x[..., :r], x[..., h:h + r]
    return torch.cat([a * c - b * s, x[..., r:h], b * c + a * s, x[..., h + r:]], -1)


def _turned(case, x):
    """The columns of a head vector that RoPE turns (a global layer keeps only these of K)."""
    g = GEOM[case["kind"]]
    return torch.cat([x[..., :g["r"]], x[..., g["d"] // 2:g["d"] // 2 + g["r"]]], -1)


def _parts(case, k, v, pos, wk):
    """The two tensors a layer stores of its new rows, before the 4-bit cast: K' and V, or S and the
    turned columns of its K."""
    k = k.float()
    normed = (lambda x: x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)) if wk is not None else None
    if case["kind"] == "sliding":
        v = v.float()
        return _rope(case, normed(k) * wk.float() if normed else k, pos), normed(v) if normed else v
    s = normed(k) if normed else k
    return s, _turned(case, _rope(case, s * wk.float() if normed else k, pos))


def _tokens(case, g, n, hkv):
    """n raw key and value rows; the values' sizes differ from token to token, and a few columns of every
    head are larger than the others."""
    d = GEOM[case["kind"]]["d"]
    size = torch.exp2(_normal(g, n, 1, 1))
    size = size * torch.where(torch.arange(d, device=DEV) % 61 == 7, 4.0, 1.0)
    k = _normal(g, n, hkv, d)
    if case["kind"] == "sliding":
        return k.bfloat16(), (_normal(g, n, hkv, d) * size).bfloat16()
    return (k * size).bfloat16(), None


def _inputs(case, seed):
    """Everything a pass reads, in logical order: cached tokens as codes and scales, page plan, rows."""
    if case["op"] == "plan":
        return _plan_inputs(case, seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows, ctx = _sizes(case)
    n = case["batch"]
    held = [_pages_of(r + c) for r, c in zip(rows, ctx)]   # pages of each sequence
    width = max(held)
    # a sliding layer maps the pages of its window only
    first = [_first_key(case, max(c - 1, 0) if case["op"] == "decode" else c) // PAGE for c in ctx]
    pool = sum(h - f for h, f in zip(held, first)) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).int()
    at = torch.arange(width, device=DEV)[None, :]
    mapped = (at >= _i32(first)[:, None]) & (at < _i32(held)[:, None])
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    table[mapped] = perm[:pool - 3]
    s = dict(case=case, rows=rows, ctx=ctx, table=table, pool=pool, ctx_t=_i32(ctx), rows_t=_i32(rows),
             first=first, held=held)
    d, (hq, hkv) = GEOM[case["kind"]]["d"], _heads(case)
    s["wq"] = s["wk"] = None
    if case["norms"]:
        s["wq"], s["wk"] = ((0.5 + torch.rand(d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    # the cached tokens, page by page in the order of `mapped` (slots past the end hold stale bytes)
    own_pos = (at * PAGE + (case["shift"] * PAGE if case["op"] == "decode" else 0))[..., None] + torch.arange(
        PAGE, device=DEV)
    pos = own_pos.expand(n, width, PAGE)[mapped].reshape(-1)                       # [pages * 16]
    codes, scales = [], []
    step = 2048 * PAGE
    for i in range(0, pos.numel(), step):
        p = pos[i:i + step]
        k, v = _tokens(case, g, p.numel(), hkv)
        q = [_quantise(x) for x in _parts(case, k, v, p, s["wk"])]
        codes.append([c for c, _ in q])
        scales.append([e for _, e in q])
    s["codes"] = [torch.cat(c).unflatten(0, (-1, PAGE)) for c in zip(*codes)]      # [pages, 16, H, n]
    s["scales"] = [torch.cat(e).unflatten(0, (-1, PAGE)) for e in zip(*scales)]    # [pages, 16, H, n / 32]
    s["mapped"] = mapped
    if case["op"] == "decode":
        s["q"] = _normal(g, n, hq, d).bfloat16()
        s["pos"] = s["ctx_t"] - 1 + case["shift"] * PAGE
        if case["weights"]:
            s["before"] = torch.rand(n, width, generator=g, device=DEV)   # what earlier steps left
        return s
    # new rows, packed, with a few rows of nobody behind them
    total = sum(rows) + 5
    s["k"], s["v"] = _tokens(case, g, total, hkv)
    s["start"] = [sum(rows[:b]) for b in range(n)]
    s["start_t"] = _i32(s["start"])
    if case["op"] == "prefill":
        s["q"] = _normal(g, total, hq, d).bfloat16()
        s["span"] = None
        if case["image"]:
            spans = [_image(case, r, c) for r, c in zip(rows, ctx)]
            span = torch.zeros(total, 2, dtype=torch.int32, device=DEV)
            for b, (s0, s1) in enumerate(spans):
                span[s["start"][b] + s0 - ctx[b]:s["start"][b] + s1 - ctx[b]] = _i32([s0, s1])
            s["span"] = span
    return s


def _plan_inputs(case, seed):
    """The state that a serving program keeps between steps, for each layer kind a pool of pages: the free
    ones in a ring, the others in the requests' tables or just evicted."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ctx, new = _requests(case)
    n = case["batch"]
    total = sum(max(x, 0) for x in new)
    s = dict(case=case, ctx=_i32(ctx), new=_i32(new), rows=total + 7, groups=[])
    for kind in ("global", "sliding")[:case["groups"]]:
        window = WINDOW if kind == "sliding" else 0
        lost = [0] * n
        if kind == "global" and case["evicted"]:
            r = random.Random(case["len_seed"] + 2)
            lost = [PAGE * r.randint(0, min(40, max(0, c - 1) // (2 * PAGE))) for c in ctx]
        # an earlier step's lost tokens, and the pages that the last eviction took (in `freed`)
        n_freed = [min(4, x // PAGE) for x in lost]
        held = [c - x for c, x in zip(ctx, lost)]
        first = [max(0, h - window) // PAGE if window else 0 for h in held]
        last = [_pages_of(h) for h in held]
        need = sum(_pages_of(h + x) - _pages_of(h) for h, x in zip(held, new) if x > 0)
        spare = max(2, int(case["supply"] * need))
        mapped_n = sum(l - f for l, f in zip(last, first))
        pages = mapped_n + sum(n_freed) + spare
        perm = torch.randperm(pages, generator=g, device=DEV).int()
        width = max(_pages_of(h + max(x, 0)) for h, x in zip(held, new)) + 1
        at = torch.arange(width, device=DEV)[None, :]
        mapped = (at >= _i32(first)[:, None]) & (at < _i32(last)[:, None])
        table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        table[mapped] = perm[:mapped_n]
        gone = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        gone[at < _i32(n_freed)[:, None]] = perm[mapped_n:mapped_n + sum(n_freed)]
        head = int(torch.randint(pages, (1,), generator=g, device=DEV))
        ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(spare, device=DEV)) % pages] = perm[mapped_n + sum(n_freed):]
        s["groups"].append(dict(window=window, pages=pages, width=width, table=table, ring=ring,
                                pool=_i32([head, spare]), first=_i32(first) if window else None,
                                lost=_i32([x - PAGE * f for x, f in zip(lost, n_freed)]) if case["evicted"] and not window else None,
                                freed=gone if case["evicted"] and not window else None,
                                n_freed=_i32(n_freed) if case["evicted"] and not window else None))
    return s


# ---- the byte layout of the pages ------------------------------------------------------------------
# A page-head block: two tiles (K' and V, or S and the turned columns), the scales of each ([16 keys][columns
# / 32]), then each key's largest scale of the tensor that serves as V.
# A tile of 256 or 512 columns: [columns / 256][16 keys][128 bytes], a key's 16-byte piece c at piece
# c ^ ((j & 6) ^ 4 (j & 1)); piece c holds columns 4c .. 4c + 3 of each of the 8 blocks of 32. The tile of the
# 128 turned columns: [16 keys][64 bytes], piece c holding columns 4c .. 4c + 3 and 16 + 4c .. of each of 4 blocks.

def _swizzle(x):
    """Pieces [..., 16 keys, 8, 16] put into, or taken out of, their places."""
    j = torch.arange(PAGE, device=x.device)[:, None]
    c = torch.arange(8, device=x.device)[None, :]
    return x[..., j, c ^ ((j & 6) ^ ((j & 1) << 2)), :]


def _tile(codes):
    """Codes [..., 16, n] -> bytes [..., 8 n]."""
    n = codes.shape[-1]
    byte = codes[..., 0::2] | (codes[..., 1::2] << 4)                                # [..., 16, n / 2]
    if n == 128:   # [block 4][half 2][piece 4][2 bytes] -> [piece][block][half][2]
        b = byte.unflatten(-1, (4, 2, 4, 2)).movedim(-2, -4)
        return b.flatten(-5)
    b = byte.unflatten(-1, (n // 256, 8, 8, 2)).transpose(-3, -2).flatten(-2)        # [..., 16, seg, piece, 16]
    return _swizzle(b.transpose(-4, -3)).flatten(-4)


def _untile(data, n):
    """Bytes [..., 8 n] -> codes [..., 16, n]."""
    if n == 128:
        b = data.unflatten(-1, (PAGE, 4, 4, 2, 2)).movedim(-4, -2).flatten(-4)
    else:
        b = _swizzle(data.unflatten(-1, (n // 256, PAGE, 8, 16))).transpose(-4, -3)
        b = b.unflatten(-1, (8, 2)).transpose(-3, -2).flatten(-4)
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _columns(case):
    d = GEOM[case["kind"]]["d"]
    return (d, d) if case["kind"] == "sliding" else (d, 128)


def _to_bytes(s):
    """All pages of the pool as bytes [pool, H, block]; pages of nobody and stale slots hold anything."""
    codes = [c.transpose(1, 2) for c in s["codes"]]                                   # [pages, H, 16, n]
    scales = [e.transpose(1, 2) for e in s["scales"]]
    top = scales[1 if s["case"]["kind"] == "sliding" else 0].amax(-1)
    data = torch.cat([_tile(c) for c in codes] + [e.flatten(-2) for e in scales] + [top], -1)
    out = torch.full((s["pool"], *data.shape[1:]), 255, dtype=torch.uint8, device=DEV)
    out[s["table"][s["mapped"]].long()] = data
    return out


def _from_bytes(case, data):
    """Bytes [..., H, block] -> the two tensors' values in fp32, [..., 16, H, n]."""
    one, two = _columns(case)
    at = [0, 8 * one, 8 * (one + two)]
    at += [at[2] + one // 2, at[2] + (one + two) // 2]
    got = []
    for i, n in enumerate((one, two)):
        codes = _untile(data[..., at[i]:at[i + 1]], n)
        scale = data[..., at[2 + i]:at[3 + i]].unflatten(-1, (PAGE, n // 32))
        got.append(_values(codes, scale).transpose(-3, -2))
    return got


def _tile16(x, halves):
    """bf16 rows [pages, 16, H, n] as 8x8 core matrices [pages, H, halves, 2, n/halves/8, 8, 8]."""
    p, _, h, n = x.shape
    x = x.bfloat16().transpose(1, 2).reshape(p, h, 2, 8, halves, n // halves // 8, 8)
    return x.permute(0, 1, 4, 2, 5, 3, 6).contiguous()


def _scratch(case, pool, hkv):
    """The tensors of a bf16 paged cache, zeros."""
    z = lambda *s: torch.zeros(pool, hkv, *s, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    if case["kind"] == "sliding":
        return [z(1, 2, 32, 8, 8), z(2, 2, 16, 8, 8)]
    return [z(2, 2, 32, 8, 8), z(2, 2, 8, 8, 8)]


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "plan":
        e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device=DEV)   # noqa: E731
        n = case["batch"]
        s["out"] = dict(ctx_len=e(n), q_start=e(n), q_len=e(n), ctx_start=e(n), positions=e(s["rows"]))
        for g in s["groups"]:
            g["out"] = dict(pool=e(2), seq_len=e(n), slots=e(s["rows"], torch.int64), first=e(n) if g["window"] else None,
                            lost=e(n) if g["lost"] is not None else None)
        return s
    s["pages"] = _to_bytes(s)
    for name in ("codes", "scales", "mapped"):
        del s[name]
    if case["op"] != "decode":
        s["scratch"] = _scratch(case, s["pool"], _heads(case)[1])
    elif case["weights"]:
        s["weights"] = torch.zeros_like(s["before"])
    if "q" in s:
        s["out"] = torch.zeros_like(s["q"])
    return s


# ---- plain forms -----------------------------------------------------------------------------------

def _query(case, q, pos, wq, wk):
    """The query vectors the scores are taken with: normed, turned, cast to bf16 (a decode step of a
    normed layer casts the normed queries to bf16 first)."""
    g = GEOM[case["kind"]]
    x = q.float()
    if wq is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * wq.float()
        if case["kind"] == "global":   # w_k of the columns that are read from S
            t = torch.arange(g["d"], device=q.device) % (g["d"] // 2)
            x = torch.where(t >= g["r"], x * wk.float(), x)
        if case["op"] == "decode":
            x = x.bfloat16().float()
    return _rope(case, x, pos).bfloat16().float()


def _keys(case, one, two):
    """K and V from the two stored tensors: on a global layer V is S, and K is S with its turned columns."""
    if case["kind"] == "sliding":
        return one, two
    g = GEOM[case["kind"]]
    r, h = g["r"], g["d"] // 2
    return torch.cat([two[..., :r], one[..., r:h], two[..., r:], one[..., h + r:]], -1), one


def _attend(case, q, k, v, seen):
    """q [B, n, Hq, d], k and v [B, m, H, d], seen [B, n, m] -> out [B, n, Hq, d], p [B, H, G, n, m]."""
    b, n, hq, d = q.shape
    hkv = k.shape[2]
    q = q.reshape(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)        # [B, H, G n, d]
    v = torch.where(seen.any(1)[..., None, None], v, torch.zeros_like(v))              # stale slots may hold NaN
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d)).unflatten(2, (-1, n))
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (-1, n))
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d), p


def _new_rows(s):
    """(sequence, position) of each packed new row."""
    n = sum(s["rows"])
    b = torch.repeat_interleave(torch.arange(len(s["rows"]), device=DEV), s["rows_t"], output_size=n)
    return b, s["ctx_t"][b] + torch.arange(n, device=DEV) - s["start_t"][b]


def _stored_rows(s):
    """The values that the new rows' 4-bit form stands for."""
    b, pos = _new_rows(s)
    n = pos.numel()
    parts = _parts(s["case"], s["k"][:n], None if s["v"] is None else s["v"][:n], pos, s["wk"])
    return b, pos, [_values(*_quantise(x)) for x in parts]


def _into_pages(s, values, b, pos):
    """The bf16 pages, zeros but for the keys (b, pos)."""
    case, got = s["case"], []
    page, slot = s["table"][b, pos // PAGE].long(), (pos % PAGE).long()
    for i, x in enumerate(values):
        rows = torch.zeros(s["pool"], PAGE, *x.shape[1:], device=DEV, dtype=torch.bfloat16)
        rows[page, slot] = x.bfloat16()
        got.append(_tile16(rows, 1 if case["kind"] == "sliding" and i == 0 else 2))
    return got


def _plain_store(s):
    b, pos, values = _stored_rows(s)
    return _into_pages(s, values, b, pos)


def _plain_decode(s):
    case = s["case"]
    length = s["ctx_t"].long()
    first = (length - WINDOW).clamp(min=0) if case["kind"] == "sliding" else torch.zeros_like(length)
    n_pages = min(s["table"].shape[1], WINDOW // PAGE + 1) if case["kind"] == "sliding" else s["table"].shape[1]
    page = first[:, None] // PAGE + torch.arange(n_pages, device=DEV)                    # [B, pages]
    phys = torch.gather(s["table"], 1, page.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    one, two = (x.flatten(1, 2) for x in _from_bytes(case, s["pages"][phys]))           # [B, keys, H, n]
    key = (page[..., None] * PAGE + torch.arange(PAGE, device=DEV)).flatten(1)
    seen = (key >= first[:, None]) & (key < length[:, None])
    k, v = _keys(case, one, two)
    del one, two
    q = _query(case, s["q"], s["pos"], s["wq"], s["wk"])
    o, p = _attend(case, q[:, None], k, v, seen[:, None])
    if not case["weights"]:
        return o[:, 0].bfloat16()
    return [o[:, 0].bfloat16(), s["before"] + p.sum((1, 2, 3)).unflatten(1, (-1, PAGE)).sum(-1)]


def _plain_prefill(s):
    case = s["case"]
    b, pos, new = _stored_rows(s)
    width = s["table"].shape[1]
    hist = [x.flatten(1, 2) for x in _from_bytes(case, s["pages"][s["table"].clamp(min=0).long()])]
    for x, y in zip(hist, new):
        x[b, pos] = y
    key = torch.arange(width * PAGE, device=DEV)
    ctx, end = s["ctx_t"][:, None], (s["ctx_t"] + s["rows_t"])[:, None]
    lo = (ctx - WINDOW + 1).clamp(min=0) if case["kind"] == "sliding" else torch.zeros_like(ctx)
    kb, kp = torch.nonzero((key >= lo) & (key < end), as_tuple=True)
    pages = _into_pages(s, [x[kb, kp] for x in hist], kb, kp)
    k, v = _keys(case, *hist)
    del hist
    # queries padded to the longest chunk
    n = max(s["rows"])
    at = (pos - s["ctx_t"][b]).long()
    q = torch.zeros(len(s["rows"]), n, *s["q"].shape[1:], device=DEV)
    q[b, at] = _query(case, s["q"][:pos.numel()], pos, s["wq"], s["wk"])
    row = ctx + torch.arange(n, device=DEV)                                              # [B, n]
    seen = (key <= row[..., None]) & (key < end[..., None])
    if case["kind"] == "sliding":
        seen &= row[..., None] - key < WINDOW
    if s["span"] is not None:
        span = torch.zeros(len(s["rows"]), n, 2, device=DEV, dtype=torch.int32)
        span[b, at] = s["span"][:pos.numel()]
        seen |= (key >= span[..., :1]) & (key < span[..., 1:])
    seen &= row[..., None] < end[..., None]
    o, _ = _attend(case, q, k, v, seen)
    out = torch.zeros_like(s["out"])
    out[:pos.numel()] = o[b, at].bfloat16()
    return [out, *pages]


def _plain_plan(s):
    """Who is served: the requests, in order, as long as the rows and every pool's free pages last (a request
    that needs no page of a pool does not wait for one); one that is not still counts for those behind it."""
    ctx, new = s["ctx"].long(), s["new"].long()
    rows = new.clamp(min=0)
    end_row = rows.cumsum(0)
    served = (rows > 0) & (end_row <= s["rows"])
    ended = new < 0
    for g in s["groups"]:
        g["now_lost"] = 0 if g["lost"] is None else g["lost"].long() + PAGE * g["n_freed"].long()
        g["held"] = ctx - g["now_lost"]
        g["last"] = (g["held"] + PAGE - 1) // PAGE
        g["need"] = (g["held"] + rows + PAGE - 1) // PAGE - g["last"]
        served &= (g["need"] == 0) | (g["need"].cumsum(0) <= g["pool"][1])
    q_len = torch.where(served, rows, torch.zeros_like(rows))
    at = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(end_row, at, right=True).clamp(max=len(rows) - 1)
    live = (at < end_row[-1]) & served[b]
    index = at - (end_row - rows)[b]
    position = torch.where(live, ctx[b] + index, torch.full_like(at, -1))
    zero = torch.zeros_like(ctx)
    out = [torch.where(ended, zero, ctx + q_len).int(), (end_row - rows).int(), q_len.int(), ctx.int(), position.int()]
    for g in s["groups"]:
        table, ring, n = g["table"].clone(), g["ring"].clone(), g["pages"]
        col = torch.arange(g["width"], device=DEV)[None]
        first = zero if g["first"] is None else g["first"].long()
        visible = (g["held"] - g["window"] + 1).clamp(min=0) // PAGE if g["window"] else zero
        to = torch.where(ended, g["last"], torch.where(served, torch.maximum(visible, first), first))
        leaving = (col >= first[:, None]) & (col < to[:, None])
        if g["freed"] is None:
            back = table[leaving]
        else:   # a request's evicted pages first
            both = torch.cat([g["freed"], table], 1)
            back = both[torch.cat([col < g["n_freed"][:, None], leaving], 1)]
        got = (col >= g["last"][:, None]) & (col < (g["last"] + g["need"])[:, None]) & served[:, None]
        head, count = g["pool"][0].long(), g["pool"][1].long()
        k = got.sum()
        table[got] = ring[(head + torch.arange(int(k), device=DEV)) % n]
        ring[(head + count + torch.arange(back.numel(), device=DEV)) % n] = back
        slot = table[b, ((g["held"][b] + index) // PAGE).clamp(max=g["width"] - 1)].long() * PAGE + (g["held"][b] + index) % PAGE
        out += [table, ring, torch.stack([(head + k) % n, count - k + back.numel()]).int(),
                torch.where(served, g["held"] + q_len, zero).int(), torch.where(live, slot, torch.full_like(slot, -1))]
        if g["window"]:
            out.append(torch.where(ended, zero, to).int())
        if g["lost"] is not None:
            out.append(torch.where(ended, zero, g["now_lost"]).int())
    return out


# ---- the library's calls -----------------------------------------------------------------------------

def _handle(s):
    """What a program sets up once per layer and batch shape: descriptors and workspace."""
    import invariant_hybrid_attention_gb300 as g4
    case = s["case"]
    h = {"g4": g4}
    if case["op"] == "plan":
        h["groups"] = [g4.make_page_group(g["window"], g["table"], g["ring"], g["pool"], g["out"]["pool"], g["out"]["seq_len"],
                                          g["out"]["slots"], first_page=g["first"], out_first_page=g["out"]["first"],
                                          lost=g["lost"], out_lost=g["out"]["lost"], freed=g["freed"], n_freed=g["n_freed"])
                       for g in s["groups"]]
    else:
        h["layer"] = g4.sliding_layer(WINDOW, tp=case["tp"]) if case["kind"] == "sliding" else g4.global_layer(
            tp=case["tp"])
        h["norms"] = g4.make_norms(s["wq"], s["wk"], True, EPS) if case["norms"] else None
        h["cache"] = g4.make_cache4(s["pages"], s["pool"])
        if case["op"] == "decode":
            size = g4.g4attn_kv4_decode_workspace_bytes(h["layer"], case["batch"], s["table"].shape[1], case["weights"])
            h["work"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        else:
            one, two = s["scratch"]
            h["scratch"] = (g4.make_cache(one, two, s["pool"]) if case["kind"] == "sliding"
                            else g4.make_cache(one, None, s["pool"], two))
            h["end"] = s["ctx_t"] + s["rows_t"]
    s["handle"] = h
    return h


def _own(s):
    h = s.get("handle") or _handle(s)
    g4, case = h["g4"], s["case"]
    if case["op"] == "plan":
        o = s["out"]
        g4.g4attn_plan_pages(s["ctx"], s["new"], h["groups"], o["ctx_len"], o["q_start"], o["q_len"], o["ctx_start"],
                             o["positions"])
        got = [o["ctx_len"], o["q_start"], o["q_len"], o["ctx_start"], o["positions"]]
        for g in s["groups"]:
            x = g["out"]
            got += [g["table"], g["ring"], x["pool"], x["seq_len"], x["slots"]]
            got += [y for y in (x["first"], x["lost"]) if y is not None]
        return got
    if case["op"] == "store":
        g4.g4attn_kv4_append(h["layer"], h["norms"], s["k"], s["v"], s["start_t"], s["rows_t"], s["ctx_t"], h["cache"],
                             s["table"])
        g4.g4attn_kv4_unpack(h["layer"], s["ctx_t"], h["end"], h["cache"], s["table"], h["scratch"], s["table"])
        return s["scratch"]
    if case["op"] == "decode":
        if case["weights"]:
            s["weights"].copy_(s["before"])
        g4.g4attn_kv4_decode(h["layer"], h["norms"], s["q"], None, None, s["ctx_t"], h["cache"], s["table"], s["out"],
                             h["work"], pos=s["pos"] if case["shift"] else None, page_weights=s.get("weights"))
        return [s["out"], s["weights"]] if case["weights"] else s["out"]
    g4.g4attn_kv4_prefill(h["layer"], h["norms"], s["q"], s["k"], s["v"], s["start_t"], s["rows_t"], s["ctx_t"],
                          h["cache"], s["table"], h["scratch"], s["table"], s["out"], span=s["span"])
    return [s["out"], *s["scratch"]]


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "store": _plain_store, "decode": _plain_decode,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _rounded(x):
    """fp64 head vectors -> the fp64 values their 4-bit form stands for."""
    y = x.unflatten(-1, (-1, 32))
    a = y.abs().amax(-1, keepdim=True)
    e = torch.frexp(a.clamp(min=2.0 ** -77)).exponent.double() - 3          # floor(log2 a) - 2
    e = torch.where(a > 7.0 * torch.exp2(e), e + 1, e).clamp(max=125)
    grid = torch.tensor(STEPS, dtype=torch.float64, device=x.device)
    m = y.abs() / torch.exp2(e)
    # the nearest of the eight steps: how many midpoints lie below; a midpoint itself goes to the even index
    mid = (grid[1:] + grid[:-1]) / 2
    index = torch.zeros_like(m, dtype=torch.int64)
    for i in range(7):
        index += (m > mid[i]) if i % 2 == 0 else (m >= mid[i])
    v = grid[index] * torch.sign(y) * torch.exp2(e)
    return torch.where(a < 2.0 ** -77, torch.zeros_like(v), v).flatten(-2)


def _turn64(case, x, pos):
    """RoPE of fp64 vectors [n, H, d] at positions [n], the pairs (t, t + d/2) as complex numbers."""
    g = GEOM[case["kind"]]
    r, h = g["r"], g["d"] // 2
    rate = g["theta"] ** (torch.arange(r, dtype=torch.float64, device=x.device) * (-1.0 / h))
    angle = pos.double()[:, None, None] * rate
    z = torch.complex(x[..., :r], x[..., h:h + r]) * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., :r], y[..., h:h + r] = z.real, z.imag
    return y


def _unit64(x):
    return x * (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()


def _query64(s, q, pos):
    """The query vectors of _core in fp64, with the two casts to bf16 that belong to the definition."""
    case, x = s["case"], q.double()
    if s["wq"] is not None:
        x = _unit64(x) * s["wq"].double()
        if case["kind"] == "global":
            x[..., 64:256] *= s["wk"][64:256].double()
            x[..., 320:] *= s["wk"][320:].double()
        if case["op"] == "decode":
            x = x.bfloat16().double()
    return _turn64(case, x, pos).bfloat16().double()


def _stored64(s, at, pos):
    """The two stored tensors of the new rows `at` (positions pos), as the values of their 4-bit form."""
    case, k = s["case"], s["k"][at].double()
    if case["kind"] == "sliding":
        v = s["v"][at].double()
        if s["wk"] is not None:
            k, v = _unit64(k) * s["wk"].double(), _unit64(v)
        return [_rounded(_turn64(case, k, pos)), _rounded(v)]
    key = k if s["wk"] is None else _unit64(k) * s["wk"].double()
    key = _turn64(case, key, pos)
    return [_rounded(k if s["wk"] is None else _unit64(k)), _rounded(torch.cat([key[..., :64], key[..., 256:320]], -1))]


def _keys64(case, one, two):
    if case["kind"] == "sliding":
        return one, two
    k = one.clone()
    k[..., :64], k[..., 256:320] = two[..., :64], two[..., 64:]
    return k, one


def _core(q, k, v, lo, hi, scale):
    """One KV head: q [G, n, d], k, v [m, d]; row i sees keys lo[i] .. hi[i] - 1. Output [G, n, d], p."""
    key = torch.arange(k.shape[0], device=k.device)
    x = torch.einsum("gnd,md->gnm", q, k) * scale
    x = torch.where((key >= lo[:, None]) & (key < hi[:, None]), x, torch.full_like(x, -math.inf))
    p = torch.softmax(x, -1)
    return torch.einsum("gnm,md->gnd", p, v), p


def _exact_page_order(s, values, where):
    """Values of keys {(page, slot): row} as the bf16 pages hold them, in fp64."""
    case, got = s["case"], []
    for i, x in enumerate(values):
        n = x.shape[-1]
        width = n if case["kind"] == "sliding" and i == 0 else n // 2
        flat = torch.zeros(s["pool"], x.shape[1], PAGE * n, dtype=torch.float64, device=DEV)
        d = torch.arange(n, device=DEV)
        page, slot = where
        place = (((d // width)[None] * 2 + (slot // 8)[:, None]) * (width // 8) + (d % width // 8)[None]) * 64 \
            + (slot % 8)[:, None] * 8 + (d % 8)[None]                                    # [rows, n]
        h = torch.arange(x.shape[1], device=DEV)
        flat[page[:, None, None], h[None, :, None], place[:, None, :]] = x
        halves = n // width
        got.append(flat.reshape(s["pool"], x.shape[1], halves, 2, width // 8, 8, 8))
    return got


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    rows, ctx = s["rows"], s["ctx"]
    d, (hq, hkv) = GEOM[case["kind"]]["d"], _heads(case)
    group, scale = hq // hkv, 1.0 / math.sqrt(d)
    first_page = [sum(h - f for h, f in zip(s["held"][:b], s["first"][:b])) for b in range(case["batch"])]

    def cached(b):
        """The values of sequence b's cached tokens, from the first key of its first page."""
        one = slice(first_page[b], first_page[b] + s["held"][b] - s["first"][b])
        return [_values(c[one].flatten(0, 1), e[one].flatten(0, 1), torch.float64)
                for c, e in zip(s["codes"], s["scales"])]

    if case["op"] == "decode":
        out = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device=DEV)
        weights = s["before"].double() if case["weights"] else None
        for b, length in enumerate(ctx):
            k, v = _keys64(case, *cached(b))
            base = s["first"][b] * PAGE
            lo = torch.tensor([_first_key(case, length - 1) - base], device=DEV)
            hi = torch.tensor([length - base], device=DEV)
            q = _query64(s, s["q"][b:b + 1], s["pos"][b:b + 1])[0]
            for h in range(hkv):
                o, p = _core(q[h * group:(h + 1) * group, None], k[:, h], v[:, h], lo, hi, scale)
                out[b, h * group:(h + 1) * group] = o[:, 0]
                if case["weights"]:
                    weights[b, :k.shape[0] // PAGE] += p.sum((0, 1)).unflatten(0, (-1, PAGE)).sum(-1)
        return [out, weights] if case["weights"] else out

    if case["op"] == "prefill" and 4.0 * sum(r * (r + c) for r, c in zip(rows, ctx)) * hq * d > 1.2e13:
        return None
    out = None if case["op"] == "store" else torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    values, pages, slots = [[], []], [], []
    for b, (n, c) in enumerate(zip(rows, ctx)):
        at = s["start"][b]
        pos = torch.arange(c, c + n, device=DEV)
        new = _stored64(s, slice(at, at + n), pos)
        lo = c
        if case["op"] == "prefill":
            base = s["first"][b] * PAGE
            lo = _first_key(case, c)
            new = [torch.cat([x[lo - base:c - base], y]) for x, y in zip(cached(b), new)]
            k, v = _keys64(case, *new)
            q = _query64(s, s["q"][at:at + n], pos)
            s0, s1 = _image(case, n, c)
            begin = torch.tensor([_first_key(case, i) for i in range(c, c + n)], device=DEV)
            end = pos + 1
            inside = (pos >= s0) & (pos < s1)
            begin = torch.where(inside, begin.clamp(max=s0), begin) - lo
            end = torch.where(inside, end.clamp(min=s1), end) - lo
            for h in range(hkv):
                for i in range(0, n, 512):
                    r = slice(i, min(n, i + 512))
                    m0, m1 = int(begin[r].min()), int(end[r].max())
                    o, _ = _core(q[r, h * group:(h + 1) * group].transpose(0, 1), k[m0:m1, h], v[m0:m1, h], begin[r] - m0,
                                 end[r] - m0, scale)
                    out[at + r.start:at + r.stop, h * group:(h + 1) * group] = o.transpose(0, 1)
        key = torch.arange(lo, c + n, device=DEV)
        pages.append(s["table"][b, key // PAGE].long())
        slots.append(key % PAGE)
        for x, y in zip(values, new):
            x.append(y)
    got = _exact_page_order(s, [torch.cat(x) for x in values], (torch.cat(pages), torch.cat(slots)))
    return got if case["op"] == "store" else [out, *got]


def _exact_plan(s):
    """Request by request, with Python's whole numbers."""
    ctx, new = s["ctx"].tolist(), s["new"].tolist()
    state = []
    for g in s["groups"]:
        n = len(ctx)
        freed = [[] for _ in range(n)] if g["freed"] is None else [
            r[:k] for r, k in zip(g["freed"].tolist(), g["n_freed"].tolist())]
        lost = [0] * n if g["lost"] is None else [x + PAGE * len(f) for x, f in zip(g["lost"].tolist(), freed)]
        head, count = g["pool"].tolist()
        state.append(dict(window=g["window"], table=g["table"].tolist(), ring=g["ring"].tolist(), head=head, free=count,
                          wanted=0, taken=0, back=[], lost=lost, freed=freed, has_lost=g["lost"] is not None,
                          first=[0] * n if g["first"] is None else g["first"].tolist(), seq_len=[], slots=[-1] * s["rows"]))
    after, q_start, q_len, positions, rows = [], [], [], [-1] * s["rows"], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        add = max(n, 0)
        fits = add > 0 and rows + add <= s["rows"]
        for g in state:
            held = c - g["lost"][b]
            need = math.ceil((held + add) / PAGE) - math.ceil(held / PAGE)
            g["wanted"] += need
            fits = fits and (need == 0 or g["wanted"] <= g["free"])
        for g in state:
            held = c - g["lost"][b]
            last = math.ceil(held / PAGE)
            g["back"] += g["freed"][b]
            to = g["first"][b]
            if n < 0:
                to = last
            elif fits and g["window"]:
                to = max(to, max(0, held - g["window"] + 1) // PAGE)
            g["back"] += g["table"][b][g["first"][b]:to]
            g["first"][b] = to
            if fits:
                for page in range(last, math.ceil((held + add) / PAGE)):
                    g["table"][b][page] = g["ring"][(g["head"] + g["taken"]) % len(g["ring"])]
                    g["taken"] += 1
                for i in range(add):
                    at = held + i
                    g["slots"][rows + i] = g["table"][b][at // PAGE] * PAGE + at % PAGE
            g["seq_len"].append(held + add if fits else 0)
            if n < 0:
                g["first"][b] = g["lost"][b] = 0
        if fits:
            positions[rows:rows + add] = range(c, c + add)
        after.append(0 if n < 0 else c + (add if fits else 0))
        q_start.append(rows)
        q_len.append(add if fits else 0)
        rows += add
    out = [_i32(after), _i32(q_start), _i32(q_len), _i32(ctx), _i32(positions)]
    for g in state:
        n = len(g["ring"])
        for i, page in enumerate(g["back"]):
            g["ring"][(g["head"] + g["free"] + i) % n] = page
        pool = [(g["head"] + g["taken"]) % n, g["free"] - g["taken"] + len(g["back"])]
        out += [_i32(g["table"]), _i32(g["ring"]), _i32(pool), _i32(g["seq_len"]),
                torch.tensor(g["slots"], dtype=torch.int64, device=DEV)]
        if g["window"]:
            out.append(_i32(g["first"]))
        if g["has_lost"]:
            out.append(_i32(g["lost"]))
    return out
