"""Promises of the header that the 8-bit cache's calls share with the bf16 ones, held to the bit."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV8

from gpu_cases import Norms
from test_gpu_kv8 import Rows, Step, i32, make_layers, status_ok
from test_gpu_tp import rank_heads

pytestmark = pytest.mark.gpu


# ---- rank slices ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,weights", [("sliding", False), ("global", False), ("global", True)])
@pytest.mark.parametrize("tp", [2, 4, 8])
def test_decode_rank_slices_are_the_full_call_bit_for_bit(kind, tp, weights):
    """Sharp scores and values whose sizes differ from token to token, so that the running maxima of a
    KV head's query heads move at different pages."""
    r = Rows(kind, [700, 31, 1500, 2600], seed=101, gap=0)
    gen = torch.Generator().manual_seed(2)
    for x in (r.v if kind == "sliding" else r.k):
        x.copy_((x.double() * torch.exp2(torch.randint(-10, 3, (x.shape[0], 1, 1), generator=gen).double())).bfloat16())
    r.fill()
    s = Step(r, weights=weights, q_scale=6.0)
    s.run()
    status_ok()
    for rank in range(tp):
        (q0, q1), (k0, k1) = rank_heads(kind, tp, rank)
        layer, _ = make_layers(kind, tp=tp)
        cache = PagedKV8(layer, r.plan.num_pages)
        cache.pages.copy_(r.cache.pages[:, k0:k1])
        q = s.q[:, q0:q1].contiguous()
        out = torch.full_like(q, float("nan"))
        w = torch.zeros(r.table.shape, device="cuda") if weights else None
        ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, 4, r.table.shape[1], weights), dtype=torch.uint8,
                         device="cuda")
        g4.g4attn_kv8_decode(layer, None, q, None, None, i32(s.lens), cache.desc, r.table, out, ws, page_weights=w)
        status_ok()
        assert torch.equal(out, s.out[:, q0:q1]), (kind, tp, rank)


# ---- refused sequences in staged calls ------------------------------------------------------------------

# A refused sequence (q_start, q_len, ctx_start), listed before the valid one and overlapping its rows.
REFUSED = {"past the rows": lambda T: (T - 9, 60, 0), "before the rows": lambda T: (-4, 60, 0),
           "past the positions": lambda T: (0, 30, 262144 - 20), "negative positions": lambda T: (0, 30, -3)}


class Overlap:
    """One valid sequence, and a refused one listed before it."""

    def __init__(self, kind, refused, normed, image):
        self.r = r = Rows(kind, [70], [40], seed=103, spare=8)
        self.weights = Norms(kind, 7) if normed else None   # (holds the device tensors)
        self.norms = self.weights.arg if normed else None
        bad = REFUSED[refused](r.T)
        used = set(r.table[0].tolist())
        spare = [p for p in range(r.plan.num_pages) if p not in used]
        assert len(spare) >= 4
        width = r.table.shape[1]
        row = torch.tensor([spare[i % len(spare)] for i in range(width)], dtype=torch.int32, device="cuda")
        self.table = torch.stack([row, r.table[0]]).contiguous()
        self.args = [i32([x, y]) for x, y in zip(bad, (r.start[0], 70, 40))]
        self.alone = r.row_args()
        self.span = None
        if image:
            self.span = torch.zeros(r.T, 2, dtype=torch.int32, device="cuda")
            self.span[r.start[0] + 5:r.start[0] + 50] = torch.tensor([45, 90], dtype=torch.int32, device="cuda")
        self.q, self.k = r.pack(r.q), r.pack(r.k)
        self.v = None if r.v is None else r.pack(r.v)
        self.gap = torch.ones(r.T, dtype=torch.bool, device="cuda")
        self.gap[r.start[0]:r.start[0] + 70] = False

    def check(self, call, caches):
        """call(rows, table, out, cache index): the valid sequence alone, then after the refused one."""
        ref, out = torch.full_like(self.q, 5.0), torch.full_like(self.q, 5.0)
        call(self.alone, self.r.table, ref, 0)
        status_ok()
        call(self.args, self.table, out, 1)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert torch.equal(out, ref)                              # gaps included: 5.0 in both
        assert (out[self.gap] == 5.0).all()
        for a, b in zip(*caches):
            assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("normed,image", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("refused", list(REFUSED))
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_staged_prefill_refuses_a_bad_sequence_and_serves_the_others(kind, refused, normed, image):
    o = Overlap(kind, refused, normed, image)
    o.r.append_history(o.norms)
    caches = [PagedKV8(o.r.layer, o.r.plan.num_pages) for _ in range(2)]
    scratch = [PagedKV(o.r.plan.num_pages, o.r.layer.n_kv_heads, o.r.layer.head_dim, kind == "global") for _ in range(2)]
    for c in caches:
        c.pages.copy_(o.r.cache.pages)

    def call(rows, table, out, i):
        g4.g4attn_kv8_prefill(o.r.layer, o.norms, o.q, o.k, o.v, *rows, caches[i].desc, table, scratch[i].desc, table, out,
                              span=o.span)
    o.check(call, [(c.pages, s.k, s.v, s.k_rot) for c, s in zip(caches, scratch)])


@pytest.mark.parametrize("form", ["normed", "vision", "staged"])
@pytest.mark.parametrize("refused", list(REFUSED))
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_staged_bf16_prefill_refuses_a_bad_sequence_and_serves_the_others(kind, refused, form):
    o = Overlap(kind, refused, form != "staged", form == "vision")
    layer, norms = o.r.layer, o.norms
    caches = [PagedKV(o.r.plan.num_pages, layer.n_kv_heads, layer.head_dim, kind == "global") for _ in range(2)]
    hist = (o.r.pack(o.r.k, True), None if o.v is None else o.r.pack(o.r.v, True), i32([0]), i32([40]), i32([0]))
    for c in caches:
        if norms is None:
            g4.g4attn_kv_append(layer, *hist, c.desc, o.r.table)
        else:
            g4.g4attn_kv_append_normed(layer, norms, *hist, c.desc, o.r.table)

    def call(rows, table, out, i):
        c = caches[i].desc
        if form == "normed":
            g4.g4attn_prefill_normed(layer, norms, o.q, o.k, o.v, *rows, c, table, out)
        elif form == "vision":
            g4.g4attn_prefill_vision(layer, norms, o.q, o.k, o.v, *rows, o.span, c, table, out)
        else:
            g4.g4attn_prefill_stage(layer, o.q, o.k, o.v, *rows, c, table, out)
            g4.g4attn_prefill_attend(layer, None, *rows, c, table, out)
    o.check(call, [(c.k, c.v, c.k_rot) for c in caches])


@pytest.mark.parametrize("refused", list(REFUSED))
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_normed_append_refuses_a_bad_sequence_whole(kind, refused):
    o = Overlap(kind, refused, True, False)
    layer = o.r.layer
    caches = [PagedKV(o.r.plan.num_pages, layer.n_kv_heads, layer.head_dim, kind == "global") for _ in range(2)]

    def call(rows, table, out, i):
        g4.g4attn_kv_append_normed(layer, o.norms, o.k, o.v, *rows, caches[i].desc, table)
    o.check(call, [(c.k, c.v, c.k_rot) for c in caches])


# ---- a wait that runs out ---------------------------------------------------------------------------------

def test_decode_wait_that_runs_out_leaves_finite_page_weights():
    """64 requests of 4096 keys with the limit at 0: some waits give up. The accumulators, which live on over steps,
    get what was computed or nothing: at most one unit per query head and request."""
    layer, _ = make_layers("global")
    B, width = 64, 256
    cache = PagedKV8(layer, B * width, fill=None)
    cache.pages.random_(100, 140)                     # exponents too: steps around 2^-13
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    q = gi.bf16_normal((B, 32, 512), 3).cuda()
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, B, width, True), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))

    def run(w):
        g4.g4attn_kv8_decode(layer, None, q, None, None, i32([16 * width] * B), cache.desc, table, out, ws, page_weights=w)
        torch.cuda.synchronize()
        return g4.g4attn_status_sync()
    ref = torch.zeros(B, width, device="cuda")
    assert run(ref) == g4.G4_OK
    good = out.clone()
    for _ in range(5):
        w = torch.ones(B, width, device="cuda")
        ws.fill_(255)                                 # the next kernel's shared memory is not the last call's
        torch.randn(1 << 24, device="cuda").sort()
        g4.g4attn_set_wait_limit_ns(0)
        try:
            st = run(w)
        finally:
            g4.g4attn_set_wait_limit_ns(g4.DEFAULT_WAIT_LIMIT_NS)
        assert st == g4.G4_ERR_TIMEOUT, g4.status_string(st)
        assert w.isfinite().all() and (w >= 1).all() and out.isfinite().all()
        # a request's shares sum to its heads (n_q_heads, fp32 sums of 256 pages: 2^-16), or to less
        assert ((w - 1).double().sum(1) <= 32 * (1 + 2.0 ** -16)).all()
    again = torch.zeros(B, width, device="cuda")
    assert run(again) == g4.G4_OK and torch.equal(again, ref) and torch.equal(out, good)


# ---- image spans --------------------------------------------------------------------------------------------

def agree(x, axis_max):
    """Whether the 8-bit and the bf16 cast of x give one number, both away from their borders by 2% of a step
    (axis_max: largest |x| of the stored vector)."""
    def near(y):
        return np.abs(np.abs(y - np.floor(y)) - 0.5) > 0.02
    top = np.floor(np.log2(np.maximum(axis_max, 1e-30)))
    inside = (axis_max / 2.0 ** top > 1.002) & (axis_max / 2.0 ** top < 127.4 / 64)
    a = x / 2.0 ** (top - 6)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 1e-30))) - 7)
    b = x / step
    return inside & near(a) & near(b) & (np.rint(a) * 2.0 ** (top - 6) == np.rint(b) * step)


def exact_rows(r, norms, seed):
    """Fills a Rows batch with rows whose stored K' and V (or S and its turned columns) are the same numbers in an
    8-bit and in a bf16 cache: values of 7 bits, or signs whose common normed size rounds alike, and keys with one
    turning pair per head, searched so that both casts of its turned value agree."""
    d, pairs = r.layer.head_dim, 64 if r.kind == "global" else 128
    theta = 1e6 if r.kind == "global" else 1e4
    rng = np.random.default_rng(seed)
    plain = np.setdiff1d(np.arange(d), np.concatenate([np.arange(pairs), np.arange(d // 2, d // 2 + pairs)]))
    w = np.ones(d) if norms is None else norms.oracle.k_weight
    fitting = [m for m in range(20, d - 2 * pairs if r.kind == "global" else d)
               if agree(np.array((m / d + 1e-6) ** -0.5), np.array((m / d + 1e-6) ** -0.5))]
    for b, x in enumerate(r.k):
        n, h = x.shape[:2]
        v = np.zeros((n, h, d))
        size = np.ones((n, h))
        if norms is None:
            v[:] = rng.integers(-127, 128, v.shape) / 64.0
            v[..., 3 if r.kind == "sliding" else plain[0]] = 1.5
        else:
            columns = plain if r.kind == "global" else np.arange(d)
            m = rng.choice(fitting, (n, h))
            size = (m / d + 1e-6) ** -0.5
            order = rng.random((n, h, len(columns))).argsort(-1).argsort(-1)
            count = m - (2 if r.kind == "global" else 0)      # a global row's pair is two of the m
            v[..., columns] = np.where(order < count[..., None], rng.choice([-1.0, 1.0], order.shape), 0.0)
        # candidates: a pair t and its two columns
        c = 160
        t = rng.integers(0, pairs, (n, h, c))
        if norms is not None and r.kind == "global":
            lo, hi = (rng.choice([-1.0, 1.0], t.shape) for _ in range(2))
            k_lo, k_hi = lo * size[..., None], hi * size[..., None]
        else:
            lo, hi = (rng.integers(-100, 101, t.shape) / 64.0 for _ in range(2))
            k_lo, k_hi = lo, hi
            if norms is not None:
                root = np.sqrt((lo * lo + hi * hi) / d + 1e-6)
                k_lo, k_hi = lo / root, hi / root
        k_lo, k_hi = k_lo * w[t], k_hi * w[t + d // 2]
        angle = np.arange(n)[:, None, None] * theta ** (-2.0 * t / d)
        u = np.stack([k_lo * np.cos(angle) - k_hi * np.sin(angle), k_hi * np.cos(angle) + k_lo * np.sin(angle)])
        ok = agree(u, np.abs(u).max(0)).all(0)
        pick = ok.argmax(-1)[..., None]
        found = np.take_along_axis(ok, pick, -1)[..., 0]
        t, lo, hi = (np.take_along_axis(y, pick, -1)[..., 0] for y in (t, lo, hi))
        key = np.zeros((n, h, d)) if r.kind == "sliding" else v
        if r.kind == "global":
            key[..., np.setdiff1d(np.arange(d), plain)] = 0.0
        i, j = np.nonzero(found)
        key[i, j, t[i, j]], key[i, j, t[i, j] + d // 2] = lo[i, j], hi[i, j]
        if norms is not None and r.kind == "global":          # a row without its pair has two ones less
            for i, j in zip(*np.nonzero(~found)):
                rest = np.nonzero(v[i, j] == 0)[0]
                rest = rest[np.isin(rest, plain)][:2]
                v[i, j, rest] = 1.0
        assert found.mean() > 0.9
        x.copy_(torch.tensor(key).bfloat16())
        if r.v is not None:
            r.v[b].copy_(torch.tensor(v).bfloat16())


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("kind,window", [("sliding", 1024), ("sliding", 16), ("global", 0)])
def test_prefill_with_image_spans_is_the_bf16_call_bit_for_bit(kind, window, normed):
    """Where both caches hold the same numbers, the two prefills give the same bits: one key more or less at an
    image's end, or a stale key before a window, would show. Images inside a chunk, past a window, and begun before
    the chunk."""
    norms = Norms(kind, 12) if normed else None
    arg = None if norms is None else norms.arg
    r = Rows(kind, [150, 1300, 90, 40], [30, 0, 70, 333], seed=104, gap=1, norms=norms, window=window or 1024)
    exact_rows(r, norms, 5)
    images = [(50, 140), (20, 1200), (33, 71), (0, 0)]
    span = torch.full((r.T, 2), -1, dtype=torch.int32)
    for b, (s0, s1) in enumerate(images):
        first, n = r.start[b], r.rows[b]
        span[first:first + n] = 0
        lo = max(s0, r.ctx[b])
        span[first + lo - r.ctx[b]:first + s1 - r.ctx[b]] = torch.tensor([s0, s1], dtype=torch.int32)
    span = span.cuda()
    r.append_history(arg)
    bf = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    starts = [sum(r.ctx[:b]) for b in range(4)]
    hist = (r.pack(r.k, True), None if r.v is None else r.pack(r.v, True), i32(starts), i32(r.ctx), i32([0] * 4))
    if arg is None:
        g4.g4attn_kv_append(r.layer, *hist, bf.desc, r.table)
    else:
        g4.g4attn_kv_append_normed(r.layer, arg, *hist, bf.desc, r.table)
    q, k, v = r.pack(r.q), r.pack(r.k), None if r.v is None else r.pack(r.v)
    want = torch.full_like(q, 5.0)
    g4.g4attn_prefill_vision(r.layer, arg, q, k, v, *r.row_args(), span, bf.desc, r.table, want)
    status_ok()
    scratch = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    got = torch.full_like(q, 5.0)
    g4.g4attn_kv8_prefill(r.layer, arg, q, k, v, *r.row_args(), r.cache.desc, r.table, scratch.desc, r.table, got, span=span)
    status_ok()
    # both caches hold the same numbers (the read-back of every key against the bf16 pages)
    everything = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    lens = [n + c for n, c in r.pairs()]
    g4.g4attn_kv8_unpack(r.layer, i32([0] * 4), i32(lens), r.cache.desc, r.table, everything.desc, r.table)
    status_ok()
    for a, b in ((everything.k, bf.k), (everything.v, bf.v), (everything.k_rot, bf.k_rot)):
        if a is not None:
            assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
    assert got.isfinite().all() and torch.equal(got, want)


# ---- caches elsewhere ---------------------------------------------------------------------------------------

def test_a_cache_or_scratch_on_another_device_is_refused():
    r = Rows("global", [40], seed=105, gap=0)
    s = Step(r)
    elsewhere = PagedKV8(r.layer, r.plan.num_pages, device="cpu")
    with pytest.raises(ValueError, match="the 8-bit cache is on the CPU"):
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(s.lens), elsewhere.desc, r.table, s.out, s.ws)
    with pytest.raises(ValueError, match="the 8-bit cache is on the CPU"):
        g4.g4attn_kv8_append(r.layer, None, r.pack(r.k), None, *r.row_args(), elsewhere.desc, r.table)
    scratch = PagedKV(r.plan.num_pages, 4, 512, True, device="cpu")
    q = r.pack(r.q)
    with pytest.raises(ValueError, match="the bf16 cache is on the CPU"):
        g4.g4attn_kv8_prefill(r.layer, None, q, r.pack(r.k), None, *r.row_args(), r.cache.desc, r.table, scratch.desc,
                              r.table, q)
    with pytest.raises(ValueError, match="the bf16 cache is on the CPU"):
        g4.g4attn_kv8_unpack(r.layer, i32([0]), i32([40]), r.cache.desc, r.table, scratch.desc, r.table)


# ---- the first call ------------------------------------------------------------------------------------------

FIRST_IN_A_CAPTURE = """
import torch
import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV8, device_int32
for kind in ("sliding", "global"):
    layer = g4.sliding_layer() if kind == "sliding" else g4.global_layer()
    x = gi.bf16_normal((40, layer.n_kv_heads, layer.head_dim), 3).cuda()
    v = x if kind == "sliding" else None
    pos = device_int32(list(range(40)))
    g4.g4attn_rope_apply(layer, x, pos, torch.empty_like(x))          # the library's first call: a bf16 one
    rows = (device_int32([0]), device_int32([40]), device_int32([700]))
    table = torch.arange(47, dtype=torch.int32, device="cuda")[None].contiguous()
    one, two = PagedKV8(layer, 47), PagedKV8(layer, 47)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                                      # the first 8-bit call of the process
        g4.g4attn_kv8_append(layer, None, x, v, *rows, one.desc, table)
    graph.replay()
    torch.cuda.synchronize()
    g4.g4attn_kv8_append(layer, None, x, v, *rows, two.desc, table)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_OK
    assert torch.equal(one.pages, two.pages) and not (one.pages[-1] == 255).all()
print("captured")
"""


FIRST_FROM_THREADS = """
import threading
import torch
import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV8, device_int32
layer = g4.global_layer()
x, q = gi.bf16_normal((1, 4, 512), 3).cuda(), gi.bf16_normal((1, 32, 512), 4).cuda()
table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
ws = [torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, 1, 1), dtype=torch.uint8, device="cuda") for _ in range(8)]
caches, outs = [PagedKV8(layer, 1) for _ in range(8)], [torch.empty_like(q) for _ in range(8)]
streams, one = [torch.cuda.Stream() for _ in range(8)], device_int32([1])
g4.load()
torch.cuda.synchronize()
start = threading.Barrier(8)
def work(i):
    start.wait()
    g4.g4attn_kv8_decode(layer, None, q, x, None, one, caches[i].desc, table, outs[i], ws[i], stream=streams[i])
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert g4.g4attn_status_sync() == g4.G4_OK
assert all(torch.equal(o, outs[0]) and torch.equal(c.pages[:, :, :1], caches[0].pages[:, :, :1]) for o, c in zip(outs, caches))
assert outs[0].isfinite().all()
print("threads")
"""


@pytest.mark.parametrize("script,word", [(FIRST_IN_A_CAPTURE, "captured"), (FIRST_FROM_THREADS, "threads")],
                         ids=["captured", "threads"])
def test_the_first_8_bit_calls_of_a_process(script, word):
    """Captured, after a first bf16 call; and from eight threads at once. Each in a process of its own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and word in p.stdout, p.stderr[-2000:]


# ---- the largest keys -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_of_keys_near_the_largest_bf16(kind):
    """Keys of size 2^113 under queries of size 2^-112: every product q.k, and every sum of them, is far inside
    fp32's range, and so are the outputs."""
    r = Rows(kind, [300, 40, 1100], seed=106, gap=0)
    for x in r.k:
        x.copy_((x.double() * 2.0 ** 113).bfloat16())
    r.fill()
    s = Step(r, weights=kind == "global", q_scale=2.0 ** -112)
    s.run()
    s.check()
