"""What is measured of the 8-bit paged KV cache: storing rows in it, decoding and prefilling over it,
and evicting its pages by accumulated attention weight.

Each case is one call sequence as a serving program makes it. `own = False` computes the operator in
its plain form (elementary torch operations in fp32, angles in fp64); `own = True` calls the library.
`exact` computes the definition in fp64 from the same inputs, request by request, without the byte
layouts.

The stored form of a head vector x (fp32, 128 .. 512 columns), one scale per token and head:
  a = max |x|,  E = floor(log2 a) - 6,  code = clamp(round_half_even(x / 2^E), -127, 127),
  the byte code + 128 and the biased exponent of a (E + 133; 0, all zeros, when a < 2^-119; 255 when
  x holds an infinity or NaN). The value it stands for is code * 2^E.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 16
MAX_POS = 262144
HEADS = 32
# head dim, turning pairs, KV heads and RoPE base of the two layer kinds
GEOM = {"sliding": dict(d=256, r=128, kv=16, theta=1.0e4), "global": dict(d=512, r=64, kv=4, theta=1.0e6)}
EPS = 1e-6


# ---- the cases -------------------------------------------------------------------------------------

def listed():
    mix = dict(batch=64, len_lo=1024, len_hi=32768, len_seed=7)
    return [
        # Two short prompts admitted together (ragged, below one tile): the smallest store.
        dict(name="store sliding 96+200", op="store", kind="sliding", tp=1, norms=False, batch=2, rows_lo=96,
             rows_hi=200, ctx_lo=0, ctx_hi=0, len_seed=3),
        # The new tokens of one decode step of 64 requests, with the model's q/k/v norms: one row each.
        dict(name="store sliding 64x1 normed", op="store", kind="sliding", tp=1, norms=True, batch=64, rows_lo=1,
             rows_hi=1, ctx_lo=1023, ctx_hi=32767, len_seed=7),
        # Two long prompts of a global layer stored in one go: bandwidth.
        dict(name="store global 2x8192", op="store", kind="global", tp=1, norms=False, batch=2, rows_lo=8192,
             rows_hi=8192, ctx_lo=0, ctx_hi=0, len_seed=2),
        # One short request alone on a global layer: latency.
        dict(name="decode global 1x37", op="decode", kind="global", tp=1, norms=False, weights=False, batch=1, len_lo=37,
             len_hi=37, len_seed=1, shift=0),
        # One very long request: its keys split over the whole card; evicted pages before it, weights kept.
        dict(name="decode global 1x131072", op="decode", kind="global", tp=1, norms=False, weights=True, batch=1,
             len_lo=131072, len_hi=131072, len_seed=1, shift=640),
        # The ragged serving mix on a global layer and on a sliding one.
        dict(name="decode global mix 64", op="decode", kind="global", tp=1, norms=False, weights=True, shift=0, **mix),
        dict(name="decode sliding mix 64", op="decode", kind="sliding", tp=1, norms=True, weights=False, shift=0, **mix),
        # Whole prompts over an empty cache.
        dict(name="prefill sliding 4x4096", op="prefill", kind="sliding", tp=1, norms=False, image=False, batch=4,
             rows_lo=4096, rows_hi=4096, ctx_lo=0, ctx_hi=0, len_seed=1),
        dict(name="prefill global 2x8192", op="prefill", kind="global", tp=1, norms=False, image=False, batch=2,
             rows_lo=8192, rows_hi=8192, ctx_lo=0, ctx_hi=0, len_seed=2),
        # Ragged chunks of long prompts over their cached history, normed, an image in each.
        dict(name="prefill global 3 chunks", op="prefill", kind="global", tp=1, norms=True, image=True, batch=3,
             rows_lo=65, rows_hi=515, ctx_lo=1024, ctx_hi=32768, len_seed=7),
        # A handful of short global contexts trimmed to half; and long ones of the serving mix.
        dict(name="evict 3x131", op="evict", batch=3, len_lo=1100, len_hi=2085, keep=65, first=1, last=4, len_seed=5),
        dict(name="evict 64x16384", op="evict", batch=64, len_lo=16384, len_hi=262144, keep=1024, first=4, last=64,
             len_seed=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "decode", "prefill", "evict"])
    if op == "evict":
        hi = _log_int(rng, 40, MAX_POS)
        keep = rng.randint(2, max(2, hi // PAGE))
        last = rng.randint(1, keep)
        return dict(op=op, batch=_log_int(rng, 1, 64), len_lo=rng.randint(1, hi), len_hi=hi, keep=keep,
                    first=rng.randint(0, keep - last), last=last, len_seed=rng.randrange(1 << 20))
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
    """(rows, ctx) of each sequence; a decode or evict sequence has its length as ctx and no rows."""
    n, seed = case["batch"], case["len_seed"]
    if case["op"] in ("decode", "evict"):
        return [0] * n, _between(case["len_lo"], case["len_hi"], n, seed)
    return _between(case["rows_lo"], case["rows_hi"], n, seed), _between(case["ctx_lo"], case["ctx_hi"], n, seed + 1)


def _heads(case):
    g = GEOM[case["kind"]]
    return HEADS // case["tp"], max(1, g["kv"] // case["tp"])


WINDOW = 1024


def _first_key(case, first_row):
    """The first key that a query at first_row sees."""
    return max(0, first_row - WINDOW + 1) if case["kind"] == "sliding" else 0


def _vector_bytes(case):
    """Bytes of one key of one head: 8-bit, and in bf16."""
    return (2 * 256 + 2, 2 * 512) if case["kind"] == "sliding" else (512 + 128 + 2, 2 * 640)


def work(case):
    rows, ctx = _sizes(case)
    if case["op"] == "evict":
        pages = sum((L + PAGE - 1) // PAGE for L in ctx)
        width = case["batch"] * ((max(ctx) + PAGE - 1) // PAGE)
        return {"bytes": 8.0 * pages + 12.0 * width, "flops": float(pages)}
    hq, hkv = _heads(case)
    d = GEOM[case["kind"]]["d"]
    b8, b16 = _vector_bytes(case)
    raw = 2 * d * (2 if case["kind"] == "sliding" else 1)   # bf16 bytes of one row's new k (and v) of one head
    if case["op"] == "store":
        return {"bytes": float(sum(rows) * hkv * (raw + b8 + b16)), "flops": 10.0 * sum(rows) * hkv * d}
    if case["op"] == "decode":
        keys = sum(L - _first_key(case, L - 1) for L in ctx)
        qo = 4 * case["batch"] * hq * d
        w = 8 * sum((L + PAGE - 1) // PAGE for L in ctx) if case["weights"] else 0
        return {"bytes": float(keys * hkv * b8 + qo + w + 4 * sum((L + PAGE - 1) // PAGE for L in ctx)),
                "flops": 4.0 * d * hq * keys}
    pairs, seen, hist = 0, 0, 0
    for b, (n, c) in enumerate(zip(rows, ctx)):
        seen += c + n - _first_key(case, c)
        hist += c - _first_key(case, c)
        s0, s1 = _image(case, n, c)
        for i in range(c, c + n):
            lo, hi = _first_key(case, i), i + 1
            if s0 <= i < s1:
                lo, hi = min(lo, s0), max(hi, s1)
            pairs += hi - lo
    bytes_ = sum(rows) * (4 * hq * d + hkv * (raw + b8)) + hist * hkv * b8 + seen * hkv * b16
    return {"bytes": float(bytes_), "flops": 4.0 * d * hq * pairs}


def _image(case, rows, ctx):
    """The positions of a sequence's image: the middle of its new rows; none in very short chunks."""
    if not case["image"] or rows < 3:
        return 0, 0
    return ctx + rows // 4, ctx + rows // 4 + max(1, rows // 2)


# ---- inputs ----------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _factor(biased):
    """2^(biased - 133) as fp32; NaN for 255."""
    bits = (biased.to(torch.int32).clamp(8, 254) - 6) << 23
    return torch.where(biased == 255, torch.full_like(bits, 0x7FC00000), bits).view(torch.float32)


def _quantise(x):
    """fp32 head vectors [..., n] -> codes int8 [..., n] and biased exponents uint8 [...]."""
    a = x.abs().amax(-1)
    biased = (a.view(torch.int32) >> 23) & 255
    biased = torch.where(biased < 8, torch.zeros_like(biased), biased)
    biased = torch.where(torch.isfinite(x).all(-1), biased, torch.full_like(biased, 255))
    inverse = ((260 - biased.clamp(8, 254)) << 23).view(torch.float32)   # 2^(133 - biased)
    code = torch.round(x * inverse[..., None]).clamp(-127, 127)
    code = torch.where(((biased == 0) | (biased == 255))[..., None], torch.zeros_like(code), code)
    return code.to(torch.int8), biased.to(torch.uint8)


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
    """The two tensors a layer stores of its new rows, before the 8-bit cast: K' and V, or S and the
    turned columns of its K."""
    k = k.float()
    normed = (lambda x: x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)) if wk is not None else None
    if case["kind"] == "sliding":
        v = v.float()
        return _rope(case, normed(k) * wk.float() if normed else k, pos), normed(v) if normed else v
    s = normed(k) if normed else k
    return s, _turned(case, _rope(case, s * wk.float() if normed else k, pos))


def _tokens(case, g, n, hkv):
    """n raw key and value rows; the values' sizes differ from token to token."""
    d = GEOM[case["kind"]]["d"]
    size = torch.exp2(_normal(g, n, 1, 1))
    k = _normal(g, n, hkv, d)
    if case["kind"] == "sliding":
        return k.bfloat16(), (_normal(g, n, hkv, d) * size).bfloat16()
    return (k * size).bfloat16(), None


def _inputs(case, seed):
    """Everything a pass reads, in logical order: cached tokens as codes and exponents, page plan, rows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows, ctx = _sizes(case)
    n = case["batch"]
    held = [(r + c + PAGE - 1) // PAGE for r, c in zip(rows, ctx)]   # pages of each sequence
    width = max(held)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    if case["op"] == "evict":
        first, held = [0] * n, held
    else:   # a sliding layer maps the pages of its window only
        first = [_first_key(case, max(c - 1, 0) if case["op"] == "decode" else c) // PAGE for c in ctx]
    pool = sum(h - f for h, f in zip(held, first)) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).int()
    at = torch.arange(width, device=DEV)[None, :]
    lo, hi = i32(first)[:, None], i32(held)[:, None]
    mapped = (at >= lo) & (at < hi)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    table[mapped] = perm[:pool - 3]
    s = dict(case=case, rows=rows, ctx=ctx, table=table, pool=pool, ctx_t=i32(ctx), rows_t=i32(rows),
             first=first, held=held)
    if case["op"] == "evict":
        # weights as decode steps leave them: heavy first and recent pages, a long tail, exact ties at zero
        w = torch.exp(2.0 * _normal(g, n, width)) / (1.0 + 0.01 * (i32(held)[:, None] - at).abs())
        s["weights"] = torch.where(torch.rand(n, width, generator=g, device=DEV) < 0.2, torch.zeros_like(w), w)
        return s
    d, (hq, hkv) = GEOM[case["kind"]]["d"], _heads(case)
    s["wq"] = s["wk"] = None
    if case["norms"]:
        s["wq"], s["wk"] = ((0.5 + torch.rand(d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    # the cached tokens, page by page in the order of `mapped` (slots past the end hold stale bytes)
    own_pos = (at * PAGE + (case["shift"] * PAGE if case["op"] == "decode" else 0))[..., None] + torch.arange(
        PAGE, device=DEV)
    pos = own_pos.expand(n, width, PAGE)[mapped].reshape(-1)                       # [pages * 16]
    codes, exps = [], []
    step = 4096 * PAGE
    for i in range(0, pos.numel(), step):
        p = pos[i:i + step]
        k, v = _tokens(case, g, p.numel(), hkv)
        q = [_quantise(x) for x in _parts(case, k, v, p, s["wk"])]
        codes.append([c for c, _ in q])
        exps.append([e for _, e in q])
    s["codes"] = [torch.cat(c).unflatten(0, (-1, PAGE)) for c in zip(*codes)]      # [pages, 16, H, n]
    s["exps"] = [torch.cat(e).unflatten(0, (-1, PAGE)) for e in zip(*exps)]        # [pages, 16, H]
    s["mapped"] = mapped
    if case["op"] == "decode":
        s["q"] = _normal(g, n, hq, d).bfloat16()
        s["pos"] = s["ctx_t"] - 1 + case["shift"] * PAGE
        if case["weights"]:
            s["weights"] = torch.zeros(n, width, device=DEV)
        return s
    # new rows, packed, with a few rows of nobody behind them
    total = sum(rows) + 5
    s["k"], s["v"] = _tokens(case, g, total, hkv)
    s["start"] = [sum(rows[:b]) for b in range(n)]
    s["start_t"] = i32(s["start"])
    if case["op"] == "prefill":
        s["q"] = _normal(g, total, hq, d).bfloat16()
        s["span"] = None
        if case["image"]:
            spans = [_image(case, r, c) for r, c in zip(rows, ctx)]
            span = torch.zeros(total, 2, dtype=torch.int32, device=DEV)
            for b, (s0, s1) in enumerate(spans):
                span[s["start"][b] + s0 - ctx[b]:s["start"][b] + s1 - ctx[b]] = i32([s0, s1])
            s["span"] = span
    return s


# ---- the byte layout of the pages ------------------------------------------------------------------
# A page-head block: two tiles (K' and V, or S and the turned columns), then the 16 exponents of each.
# A tile: [columns / 128][16 keys][128 bytes], the 16-byte piece c of key j at piece c ^ ((j & 6) ^ 4 (j & 1)).

def _swizzle(x):
    """Pieces [..., 16 keys, 8, 16] put into, or taken out of, their places."""
    j = torch.arange(PAGE, device=x.device)[:, None]
    c = torch.arange(8, device=x.device)[None, :]
    return x[..., j, c ^ ((j & 6) ^ ((j & 1) << 2)), :]


def _to_bytes(s):
    """All pages of the pool as bytes [pool, H, block]; pages of nobody and stale slots hold anything."""
    blocks = []
    for c in s["codes"]:
        u = (c.to(torch.int16) + 128).to(torch.uint8).transpose(1, 2)              # [pages, H, 16, n]
        u = _swizzle(u.unflatten(-1, (-1, 8, 16)).transpose(2, 3))                 # [pages, H, seg, 16, 8, 16]
        blocks.append(u.flatten(2))
    blocks += [e.transpose(1, 2) for e in s["exps"]]
    data = torch.cat(blocks, -1)
    out = torch.full((s["pool"], *data.shape[1:]), 255, dtype=torch.uint8, device=DEV)
    out[s["table"][s["mapped"]].long()] = data
    return out


def _from_bytes(case, data):
    """Bytes [..., H, block] -> the two tensors' values in fp32, [..., 16, H, n]."""
    d = GEOM[case["kind"]]["d"]
    sizes = (d, d) if case["kind"] == "sliding" else (d, 128)
    at, got = 0, []
    for i, n in enumerate(sizes):
        u = data[..., at:at + PAGE * n]
        at += PAGE * n
        u = _swizzle(u.unflatten(-1, (n // 128, PAGE, 8, 16))).transpose(-4, -3).flatten(-3)   # [..., H, 16, n]
        e = data[..., PAGE * sum(sizes) + PAGE * i:PAGE * sum(sizes) + PAGE * (i + 1)]
        got.append(((u.float() - 128.0) * _factor(e)[..., None]).transpose(-3, -2))
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
    if case["op"] == "evict":
        s["out"] = [torch.empty_like(s["ctx_t"]), torch.empty_like(s["table"]), torch.empty_like(s["weights"]),
                    torch.empty_like(s["table"]), torch.empty_like(s["ctx_t"])]
        return s
    s["pages"] = _to_bytes(s)
    for name in ("codes", "exps", "mapped"):
        del s[name]
    if case["op"] != "decode":
        s["scratch"] = _scratch(case, s["pool"], _heads(case)[1])
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
    """The values that the new rows' 8-bit form stands for."""
    b, pos = _new_rows(s)
    n = pos.numel()
    parts = _parts(s["case"], s["k"][:n], None if s["v"] is None else s["v"][:n], pos, s["wk"])
    got = []
    for x in parts:
        code, exp = _quantise(x)
        got.append(code.float() * _factor(exp)[..., None])
    return b, pos, got


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
    s["weights"] += p.sum((1, 2, 3)).unflatten(1, (-1, PAGE)).sum(-1)
    return [o[:, 0].bfloat16(), s["weights"]]


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


def _plain_evict(s):
    case, table, w = s["case"], s["table"], s["weights"]
    width = table.shape[1]
    at = torch.arange(width, device=DEV)[None]
    n = ((s["ctx_t"] + PAGE - 1) // PAGE)[:, None]
    drop = (n - case["keep"]).clamp(min=0)
    free = (at >= case["first"]) & (at < n - case["last"])
    rank = torch.argsort(torch.argsort(torch.where(free, w, torch.full_like(w, float("inf"))), stable=True), stable=True)
    out = free & (rank < drop)
    order = torch.argsort((out | (at >= n)).int(), stable=True)        # the kept pages first, in their order
    kept = at < n - drop
    gone = torch.argsort((~out).int(), stable=True)                    # the evicted ones first
    empty, none = torch.full_like(table, -1), torch.zeros_like(w)
    return [s["ctx_t"] - PAGE * drop[:, 0], torch.where(kept, table.gather(1, order), empty),
            torch.where(kept, w.gather(1, order), none), torch.where(at < drop, table.gather(1, gone), empty),
            drop[:, 0].int()]


# ---- the library's calls -----------------------------------------------------------------------------

def _handle(s):
    """What a program sets up once per layer and batch shape: descriptors and workspace."""
    import invariant_hybrid_attention_gb300 as g4
    case = s["case"]
    h = {"g4": g4}
    if case["op"] != "evict":
        h["layer"] = g4.sliding_layer(WINDOW, tp=case["tp"]) if case["kind"] == "sliding" else g4.global_layer(
            tp=case["tp"])
        h["norms"] = g4.make_norms(s["wq"], s["wk"], True, EPS) if case["norms"] else None
        h["cache"] = g4.make_cache8(s["pages"], s["pool"])
        if case["op"] == "decode":
            size = g4.g4attn_kv8_decode_workspace_bytes(h["layer"], case["batch"], s["table"].shape[1], case["weights"])
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
    if case["op"] == "store":
        g4.g4attn_kv8_append(h["layer"], h["norms"], s["k"], s["v"], s["start_t"], s["rows_t"], s["ctx_t"], h["cache"],
                             s["table"])
        g4.g4attn_kv8_unpack(h["layer"], s["ctx_t"], h["end"], h["cache"], s["table"], h["scratch"], s["table"])
        return s["scratch"]
    if case["op"] == "decode":
        g4.g4attn_kv8_decode(h["layer"], h["norms"], s["q"], None, None, s["ctx_t"], h["cache"], s["table"], s["out"],
                             h["work"], pos=s["pos"] if case["shift"] else None, page_weights=s.get("weights"))
        return [s["out"], s["weights"]] if case["weights"] else s["out"]
    if case["op"] == "prefill":
        g4.g4attn_kv8_prefill(h["layer"], h["norms"], s["q"], s["k"], s["v"], s["start_t"], s["rows_t"], s["ctx_t"],
                              h["cache"], s["table"], h["scratch"], s["table"], s["out"], span=s["span"])
        return [s["out"], *s["scratch"]]
    g4.g4attn_evict_pages(s["ctx_t"], s["table"], s["weights"], case["keep"], case["first"], case["last"], *s["out"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"store": _plain_store, "decode": _plain_decode, "prefill": _plain_prefill,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _rounded(x):
    """fp64 head vectors -> the fp64 values their 8-bit form stands for."""
    a = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -119)))
    e = torch.where(torch.exp2(e) > a, e - 1, e)                       # log2 rounded up to the next whole number
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e)                  # or down
    step = torch.exp2(e - 6)
    return torch.where(a < 2.0 ** -119, torch.zeros_like(x), torch.round(x / step).clamp(-127, 127) * step)


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
    """The two stored tensors of the new rows `at` (positions pos), as the values of their 8-bit form."""
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
    rows, ctx = s["rows"], s["ctx"]
    if case["op"] == "evict":
        return _exact_evict(s)
    d, (hq, hkv) = GEOM[case["kind"]]["d"], _heads(case)
    group, scale = hq // hkv, 1.0 / math.sqrt(d)
    first_page = [sum(h - f for h, f in zip(s["held"][:b], s["first"][:b])) for b in range(case["batch"])]

    def cached(b):
        """The values of sequence b's cached tokens, from the first key of its first page."""
        one = slice(first_page[b], first_page[b] + s["held"][b] - s["first"][b])
        return [c[one].flatten(0, 1).double() * torch.exp2(e[one].flatten(0, 1).double() - 133.0)[..., None]
                for c, e in zip(s["codes"], s["exps"])]

    if case["op"] == "decode":
        out = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device=DEV)
        weights = torch.zeros(s["table"].shape, dtype=torch.float64, device=DEV)
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


def _exact_evict(s):
    case = s["case"]
    table, weights = s["table"].cpu().tolist(), s["weights"].cpu().tolist()
    lengths, tables, kept_w, freed, n_freed = [], [], [], [], []
    for b, length in enumerate(s["ctx"]):
        n, width = s["held"][b], len(table[b])
        may = range(case["first"], n - case["last"])
        out = set(sorted(may, key=lambda i: (weights[b][i], i))[:max(0, n - case["keep"])])
        keep = [i for i in range(n) if i not in out]
        lengths.append(length - PAGE * len(out))
        tables.append([table[b][i] for i in keep] + [-1] * (width - len(keep)))
        kept_w.append([weights[b][i] for i in keep] + [0.0] * (width - len(keep)))
        freed.append([table[b][i] for i in sorted(out)] + [-1] * (width - len(out)))
        n_freed.append(len(out))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    return [i32(lengths), i32(tables), torch.tensor(kept_w, dtype=torch.float64, device=DEV), i32(freed), i32(n_freed)]
