"""The 8-bit paged cache and the page eviction on the GPU, against the fp64 definition (oracle/kv8.py).

Tolerances, derived before the first run:
* Stored values. The kernel's x is fp32: normed, turned (three table factors, five roundings) and at
  most 2^-20 |x| off, so |x| / step < 128 is off by 1.3e-4 steps and the code is within 0.5 + 2e-4
  steps of the exact x (1 step where it clamps). Raw V and S involve no rounding at all: bit-equal.
  The exponent byte differs only when max |x| lies within 2^-20 of a power of two.
* Decode. Queries are turned in fp64 and cast to bf16, as the definition says, and keys are taken from the
  bytes in the cache, so both sides compute from the same numbers, but where a turned query lies so near
  a border between two bf16 numbers (2^-22 of its pair's size: the kernel's fp32 products) that it
  may fall on either side. Such a column, one step u apart, moves a score by at most u max|k| scale, all of
  them together by delta, and a weight by at most exp(2 delta) - 1 of itself. Else left are the weights' cast to fp16 (2^-11 of each weight; below fp16's
  normal range half of its smallest step, 2^-25, where the largest weight p_i 2^e_i of the row is at
  least 2^7: 2^-32 of that one, for each of n keys, times a code of at most 127 < 2 max|v_j| / 2^e_j,
  in all n 2^-31 max_i p_i max|v_i|), fp32 sums (2^-16 covers 2^-24 x the score magnitudes, and the
  sums over up to 2^12 keys) and the cast of the output (bf16, half a step: 2^-8):
  |got - want| <= 2^-8 |want| + (2^-11 + 2^-16) sum p |v| + n 2^-31 max p max|v|.
* Page weights: fp32 throughout; scores of magnitude up to 2^6 in log2 units carry 2^-18, so each
  page's weight is within 2e-5 of itself.
* Prefill: the attention kernel runs on the same bf16 pages as g4attn_prefill_attend: bit-equal to it.
"""
import math

import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
import oracle
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV8, device_int32, tile, tile_v256, untile8
from oracle import kv8

from gpu_cases import Norms, f64

pytestmark = pytest.mark.gpu

GEOM = {"sliding": (16, 256), "global": (4, 512)}


def make_layers(kind, window=1024, tp=1):
    if kind == "sliding":
        layer = g4.sliding_layer(window, tp=tp)
        ol = oracle.with_window(oracle.SLIDING, window)
    else:
        layer, ol = g4.global_layer(tp=tp), oracle.GLOBAL
    return layer, ol


def i32(v):
    return device_int32(v)


def status_ok():
    torch.cuda.synchronize()
    st = g4.g4attn_status_sync()
    assert st == g4.G4_OK, g4.status_string(st)


class Rows:
    """Sequences with new rows at given contexts, in a pool of scattered pages: raw bf16 rows per
    sequence (history first), packed with gaps, and the 8-bit cache."""

    def __init__(self, kind, rows, ctx=None, seed=0, tp=1, scale=1.0, gap=2, norms=None, spare=3, window=1024):
        self.kind, self.rows = kind, list(rows)
        self.ctx = [0] * len(rows) if ctx is None else list(ctx)
        self.layer, self.olayer = make_layers(kind, window, tp)
        hkv, d = self.layer.n_kv_heads, self.layer.head_dim
        self.norms = norms
        self.k = [gi.bf16_normal((c + n, hkv, d), seed * 977 + 3 * b, scale) for b, (n, c) in enumerate(self.pairs())]
        self.v = None if kind == "global" else [gi.bf16_normal((c + n, hkv, d), seed * 977 + 3 * b + 1, scale)
                                                for b, (n, c) in enumerate(self.pairs())]
        self.q = [gi.bf16_normal((n, self.layer.n_q_heads, d), seed * 977 + 3 * b + 2) for b, n in enumerate(self.rows)]
        self.plan = gi.make_page_plan([max(1, c + n) for n, c in self.pairs()], seed=seed + 5, spare_pages=spare)
        self.table = self.plan.table.cuda()
        self.start, at = [], gap
        for n in self.rows:
            self.start.append(at)
            at += n + gap
        self.T = at
        self.cache = PagedKV8(self.layer, self.plan.num_pages)

    def pairs(self):
        return list(zip(self.rows, self.ctx))

    def pack(self, per_seq, history=False):
        """Rows of the call (or the history rows before them) packed [T, H, d]; gaps are NaN."""
        if history:
            return torch.cat([x[:c] for x, c in zip(per_seq, self.ctx)]).cuda()
        h, d = per_seq[0].shape[1:]
        t = torch.full((self.T, h, d), float("nan"), dtype=torch.bfloat16)
        for x, n, s in zip(per_seq, self.rows, self.start):
            t[s:s + n] = x[x.shape[0] - n:]
        return t.cuda()

    def row_args(self):
        return i32(self.start), i32(self.rows), i32(self.ctx)

    def append_history(self, norms=None):
        if max(self.ctx) == 0:
            return
        starts = [sum(self.ctx[:b]) for b in range(len(self.ctx))]
        g4.g4attn_kv8_append(self.layer, norms, self.pack(self.k, True),
                             None if self.v is None else self.pack(self.v, True), i32(starts), i32(self.ctx),
                             i32([0] * len(self.ctx)), self.cache.desc, self.table)

    def append(self, norms=None):
        g4.g4attn_kv8_append(self.layer, norms, self.pack(self.k), None if self.v is None else self.pack(self.v),
                             *self.row_args(), self.cache.desc, self.table)

    def fill(self):
        n = None if self.norms is None else self.norms.arg
        self.append_history(n)
        self.append(n)

    def values(self, b):
        """The stored values of sequence b's keys, fp64 [n, H, cols] twice, from the cache's bytes."""
        one, two = untile8(self.cache.pages, self.layer.head_dim)
        n = self.rows[b] + self.ctx[b]
        pages = self.plan.table[b, :(n + 15) // 16].long()
        return [x[pages.cuda()].transpose(1, 2).flatten(0, 1)[:n].double().cpu().numpy() for x in (one, two)]

    def exact_parts(self, b):
        n = self.rows[b] + self.ctx[b]
        return kv8.parts(self.olayer, self.k[b].double().numpy(), None if self.v is None else self.v[b].double().numpy(),
                         np.arange(n), None if self.norms is None else self.norms.oracle)


def assert_stored(got, exact, rounded):
    """got: stored values of exact vectors; rounded: whether x itself was rounded on the way."""
    if not rounded:
        assert np.array_equal(got, kv8.stored(exact), equal_nan=True)
        return
    a = np.abs(exact).max(-1, keepdims=True)
    step = np.exp2(np.floor(np.log2(a * (1 + 2.0 ** -20))) - 6)      # the larger of the two possible steps
    limit = np.where(np.abs(exact) > 127.4 * step, 1.0, 0.5 + 2e-4) * step
    assert (np.abs(got - exact) <= limit).all(), np.max(np.abs(got - exact) / step)


# ---- append -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("tp", [1, 4, 8])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_stores_the_definition(kind, tp, normed):
    r = Rows(kind, [1, 17, 40, 0, 16], [0, 15, 3, 9, 300], seed=1, tp=tp, norms=Norms(kind, 5) if normed else None)
    r.fill()
    status_ok()
    for b in range(5):
        n = r.rows[b] + r.ctx[b]
        for i, (got, want) in enumerate(zip(r.values(b), r.exact_parts(b))):
            raw = not normed and (i == 1 if kind == "sliding" else i == 0)
            assert_stored(got[:n], want, rounded=not raw)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_norms_by_a_rounded_division(kind):
    """Small whole numbers: their squares' sum is exact in any order, so mean + eps, its root and the quotient
    are one elementary fp32 operation each, and every code is fixed. A mean past fp32's range gives zeros,
    an infinity a NaN vector."""
    r = Rows(kind, [150, 33], seed=3, norms=Norms(kind, 6))
    x = r.k if kind == "global" else r.v
    rng = np.random.default_rng(3)
    for t in x:
        t.copy_(torch.from_numpy(rng.integers(-15, 16, t.shape).astype(np.float32)).bfloat16())
    x[0][5], x[0][6] = x[0][5] * 1e30, x[0][6] * 1e-30
    x[1][7, 0, 9] = float("inf")
    r.fill()
    status_ok()
    for b in range(2):
        a = x[b].float().numpy()
        with np.errstate(over="ignore", invalid="ignore"):
            mean = np.square(a).sum(-1, keepdims=True, dtype=np.float32) / np.float32(a.shape[-1])
            quotient = a / np.sqrt(mean + np.float32(1e-6))
        got = r.values(b)[0 if kind == "global" else 1]
        assert np.array_equal(got, kv8.stored(quotient.astype(np.float64)), equal_nan=True)
    assert (r.values(0)[0 if kind == "global" else 1][5] == 0).all()


def test_append_far_positions():
    """The last usable position, where fp32 angles would be 0.02 rad off."""
    for kind in ("sliding", "global"):
        layer, ol = make_layers(kind)
        hkv, d = GEOM[kind]
        n, ctx = 5, 262144 - 5
        k = gi.bf16_normal((n, hkv, d), 3)
        v = gi.bf16_normal((n, hkv, d), 4) if kind == "sliding" else None
        table = torch.full((1, 16384), -1, dtype=torch.int32)
        table[0, 16383] = 1
        cache = PagedKV8(layer, 2)
        g4.g4attn_kv8_append(layer, None, k.cuda(), None if v is None else v.cuda(), i32([0]), i32([n]), i32([ctx]),
                             cache.desc, table.cuda())
        status_ok()
        got = [x[1].transpose(0, 1)[ctx % 16:].double().cpu().numpy() for x in untile8(cache.pages, d)]
        want = kv8.parts(ol, k.double().numpy(), None if v is None else v.double().numpy(), np.arange(ctx, ctx + n))
        for g, w in zip(got, want):
            assert_stored(g, w, rounded=True)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_sizes_zeros_and_bad_vectors(kind):
    """Vectors from 2^-120 to near the largest bf16, zeros, infinities and NaN; neighbours keep theirs."""
    r = Rows(kind, [24], seed=2)
    x = r.k[0] if kind == "global" else r.v[0]
    scales = [2.0 ** e for e in (-121, -119, -100, -3, 0, 40, 100, 124)]
    for t in range(8):
        x[t] = (x[t].double().clamp(-3, 3) * scales[t]).bfloat16()
    x[8] = 0
    x[9, 0, 7], x[10, 0, 200], x[11, 0, 255] = float("inf"), float("-inf"), float("nan")
    r.append()
    status_ok()
    got, want = r.values(0), r.exact_parts(0)
    raw = 0 if kind == "global" else 1
    assert_stored(got[raw], want[raw], rounded=False)
    assert np.isnan(got[raw][9:12, 0]).all() and np.isfinite(got[raw][9:12, 1]).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_bytes_do_not_depend_on_chunks_or_batch(kind):
    whole = Rows(kind, [77], seed=7)
    whole.append()
    a = whole.values(0)
    for cuts in ([0, 1, 77], [0, 16, 33, 34, 77]):
        cut = Rows(kind, [77], seed=7)
        for lo, hi in zip(cuts, cuts[1:]):
            k = cut.k[0][lo:hi].cuda()
            v = None if cut.v is None else cut.v[0][lo:hi].cuda()
            g4.g4attn_kv8_append(cut.layer, None, k, v, i32([0]), i32([hi - lo]), i32([lo]), cut.cache.desc, cut.table)
        status_ok()
        assert all(np.array_equal(x, y) for x, y in zip(a, cut.values(0)))
        assert torch.equal(whole.cache.pages, cut.cache.pages)


def test_append_refuses_on_the_device_and_writes_nothing_else():
    r = Rows("sliding", [20, 20], seed=3)
    before = r.cache.pages.clone()
    k, v = r.pack(r.k), r.pack(r.v)

    def call(start, rows, ctx, table=r.table):
        g4.g4attn_kv8_append(r.layer, None, k, v, i32(start), i32(rows), i32(ctx), r.cache.desc, table)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert torch.equal(r.cache.pages, before)
    call([r.T - 3, 0], [20, 0], [0, 0])               # rows past T
    call([-1, 0], [20, 0], [0, 0])
    call([0, 0], [20, 0], [-4, 0])
    call([0, 0], [20, 0], [262143, 0])                # positions past the last
    call([0, 0], [20, 0], [2 ** 31 - 10, 0])
    call([0, 0], [5, 0], [16 * r.table.shape[1], 0])  # past the table
    bad = torch.full_like(r.table, r.plan.num_pages)
    call([0, 0], [5, 0], [0, 0], bad)
    call([0, 0], [5, 0], [0, 0], torch.full_like(r.table, -1))


# ---- read-back ----------------------------------------------------------------------------------------

def bf16_pages(layer, pages):
    """The bf16 cache tensors that hold the same values as the 8-bit pages."""
    one, two = untile8(pages, layer.head_dim)
    if layer.kv_shared:
        p, h = two.shape[:2]
        rot = two.bfloat16().reshape(p, h, 2, 8, 2, 8, 8).permute(0, 1, 4, 2, 5, 3, 6).contiguous()
        return tile(one.bfloat16()), rot
    return tile(one.bfloat16()), tile_v256(two.bfloat16())


@pytest.mark.parametrize("tp", [1, 8])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_unpack_is_exact_and_touches_only_its_keys(kind, tp):
    r = Rows(kind, [100, 1, 33, 16], seed=4, tp=tp)
    r.fill()
    out = PagedKV(r.plan.num_pages + 2, r.layer.n_kv_heads, r.layer.head_dim, kind == "global", fill=-7.0)
    lo, hi = [5, 0, 33, 9], [97, 1, 33, 3]            # inside pages, whole, empty, reversed
    g4.g4attn_kv8_unpack(r.layer, i32(lo), i32(hi), r.cache.desc, r.table, out.desc, r.table + 2)
    status_ok()
    want = bf16_pages(r.layer, r.cache.pages)
    got = (out.k, out.k_rot if kind == "global" else out.v)
    touched = torch.zeros(r.plan.num_pages + 2, 16, dtype=torch.bool)
    for b in range(4):
        for i in range(lo[b], hi[b]):
            touched[int(r.plan.table[b, i // 16]) + 2, i % 16] = True
    for g, w in zip(got, want):
        w2 = torch.full_like(g, -7.0)
        w2[2:] = w.reshape(w.shape[0], *g.shape[1:])
        t = touched.cuda()[:, None, None, :].unflatten(-1, (2, 8))[..., None, :, None]     # [p, 1, 1, 2, 1, 8, 1]
        g7, w7 = (x.reshape(x.shape[0], x.shape[1], -1, 2, x.shape[-3], 8, 8) for x in (g, w2))
        assert torch.equal(g7, torch.where(t, w7, torch.full_like(w7, -7.0)))


def test_unpack_refuses_on_the_device():
    r = Rows("global", [40], seed=4)
    r.fill()
    out = PagedKV(r.plan.num_pages, 4, 512, True, fill=-7.0)
    before = out.k.clone()
    for lo, hi, table in ((-1, 5, r.table), (0, 16 * r.table.shape[1] + 1, r.table), (0, 2 ** 31 - 1, r.table),
                          (0, 40, torch.full_like(r.table, -1))):
        g4.g4attn_kv8_unpack(r.layer, i32([lo]), i32([hi]), r.cache.desc, r.table, out.desc, table)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert torch.equal(out.k, before)


# ---- decode -------------------------------------------------------------------------------------------

def turned_queries(olayer, q, pos):
    """The queries q [B, Hq, D] at positions pos [B] as the definition turns and casts them, in fp64, and per
    column the step to the neighbour it may be instead (0: none)."""
    x = f64(q)
    y = oracle.rope(x, np.asarray(pos)[:, None], olayer.rope_theta, olayer.rope_partial)
    half = x.shape[-1] // 2
    size = np.abs(x[..., :half]) + np.abs(x[..., half:])
    turned = np.zeros(x.shape[-1], dtype=bool)
    turned[kv8.turned_columns(olayer)] = True
    near = np.where(turned, 2.0 ** -22 * np.concatenate([size, size], -1), 0.0)
    cast = lambda v: f64(torch.tensor(v).bfloat16())   # noqa: E731
    return cast(y), cast(y + near) - cast(y - near)


def border(step, k, scale):
    """exp(2 delta) - 1 per query head [Hq, 1] for the border steps [Hq, D] and keys [n, H, D]."""
    group = step.shape[0] // k.shape[1]
    largest = np.repeat(np.nanmax(np.abs(k), axis=0), group, axis=0)
    return np.expm1(2 * scale * (step * largest).sum(-1, keepdims=True))


def assert_row(got, want, mag, peak, more=0.0):
    """The tolerance of a decode row, derived above; more: a further share of sum p |v|."""
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16 + more) * mag + 2.0 ** -31 * peak)
    assert (over <= 0).all(), over.max()


class Step:
    """A decode step over the keys of a Rows batch: one query per sequence."""

    def __init__(self, r, seed=11, weights=False, pos=None, q_scale=1.0):
        self.r, self.lens = r, [n + c for n, c in r.pairs()]
        self.q = gi.bf16_normal((len(self.lens), r.layer.n_q_heads, r.layer.head_dim), seed, q_scale).cuda()
        self.pos = [n - 1 for n in self.lens] if pos is None else pos
        self.given_pos = None if pos is None else i32(pos)
        self.weights = torch.zeros(r.table.shape, device="cuda") if weights else None
        self.ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, len(self.lens), r.table.shape[1], weights),
                              dtype=torch.uint8, device="cuda").fill_(255)
        self.out = torch.full_like(self.q, float("nan"))

    def run(self, **kw):
        norms = None if self.r.norms is None else self.r.norms.arg
        a = dict(pos=self.given_pos, page_weights=self.weights)
        a.update(kw)
        return g4.g4attn_kv8_decode(self.r.layer, norms, self.q, None, None, i32(self.lens), self.r.cache.desc,
                                    self.r.table, self.out, self.ws, **a)

    def check(self):
        status_ok()
        q, steps = turned_queries(self.r.olayer, self.q, self.pos)
        scale = self.r.layer.softmax_scale
        got = f64(self.out)
        for b, n in enumerate(self.lens):
            k, v = kv8.keys_values(self.r.olayer, *self.r.values(b))
            lo = max(0, n - self.r.layer.window) if self.r.kind == "sliding" else 0
            want, p, mag, peak = kv8.decode(q[b], k, v, scale, lo)
            more = border(steps[b], k, scale)
            assert_row(got[b], want, mag, peak, more)
            if self.weights is not None:
                w = f64(self.weights[b])
                s = kv8.page_sums(p)
                assert np.allclose(w[:len(s)], s, rtol=2e-5 + more.max(), atol=1e-9), (b, np.abs(w[:len(s)] / s - 1).max())
                assert (w[len(s):] == 0).all()


LENS = [1, 2, 15, 16, 17, 64, 255, 257, 1023, 1024, 1025, 1100, 2300]


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_matches_the_definition(kind):
    r = Rows(kind, LENS, seed=21, gap=0)
    r.fill()
    s = Step(r, weights=kind == "global")
    s.run()
    s.check()


@pytest.mark.parametrize("window", [1, 16, 17, 250, 5000])
def test_decode_windows(window):
    r = Rows("sliding", [1, 16, 33, 700, 6000], seed=22, gap=0, window=window)
    r.fill()
    s = Step(r)
    s.run()
    s.check()


def test_decode_long_context_and_large_scores():
    """Sharp softmaxes (queries of size 6), and keys and values whose sizes differ by 2^20 from token to token."""
    for kind in ("sliding", "global"):
        r = Rows(kind, [5000, 900], seed=23, gap=0)
        g = torch.Generator().manual_seed(1)
        for x in (r.v if kind == "sliding" else r.k):
            x.copy_((x.double() * torch.exp2(torch.randint(-10, 3, (x.shape[0], 1, 1), generator=g).double())).bfloat16())
        r.fill()
        s = Step(r, weights=kind == "global", q_scale=6.0)
        s.run()
        s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_tiny_and_huge_values(kind):
    """Values near both ends of the stored range; queries far from 1."""
    for scale in (2.0 ** -110, 2.0 ** 60):
        r = Rows(kind, [300, 40], seed=24, gap=0)
        for x in (r.v if kind == "sliding" else r.k):
            x.copy_((x.double() * scale).bfloat16())
        r.fill()
        s = Step(r, q_scale=1.0 if kind == "sliding" else 1 / scale)
        s.run()
        s.check()


@pytest.mark.parametrize("tp", [2, 4, 8])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_rank_slices(kind, tp):
    r = Rows(kind, [700, 31, 1500], seed=25, gap=0, tp=tp)
    r.fill()
    s = Step(r, weights=kind == "global")
    s.run()
    s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_appends_the_new_token_like_append(kind):
    """k_new in the call: the same bytes and the same output as an append before it."""
    a = Rows(kind, [1, 1, 1], [0, 16, 1200], seed=26, gap=0)
    b = Rows(kind, [1, 1, 1], [0, 16, 1200], seed=26, gap=0)
    a.fill()
    b.append_history()
    sa, sb = Step(a), Step(b)
    sa.run()
    g4.g4attn_kv8_decode(b.layer, None, sb.q, b.pack(b.k), None if b.v is None else b.pack(b.v), i32(sb.lens),
                         b.cache.desc, b.table, sb.out, sb.ws)
    status_ok()
    assert torch.equal(a.cache.pages, b.cache.pages)
    assert torch.equal(sa.out, sb.out)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_normed(kind):
    """Norms: bit-equal to the un-normed call on queries normed by hand, where that is one cast."""
    norms = Norms(kind, 9)
    r = Rows(kind, [600, 45], seed=27, gap=0, norms=norms)
    r.fill()
    s = Step(r)
    s.run()
    status_ok()
    qn = oracle.normed_q(norms.oracle, s.q.double().cpu().numpy())
    if kind == "global":
        rest = np.setdiff1d(np.arange(512), kv8.turned_columns(r.olayer))
        qn[..., rest] *= norms.oracle.k_weight[rest]
    want = f64(g4.g4attn_rope_apply(r.layer, torch.tensor(qn).bfloat16().cuda(), i32(s.pos)))
    got = f64(s.out)
    for b, n in enumerate(s.lens):
        one, two = r.values(b)
        k, v = kv8.keys_values(r.olayer, one, two)
        o, _, mag, peak = kv8.decode(want[b], k, v, r.layer.softmax_scale, 0)
        # the norm's fp32 result may fall to the other side of a bf16 boundary in a few of 512 columns:
        # one column moves a score by at most 2^-8 |q| |k| scale, a weight by as much
        flip = 4 * 2.0 ** -8 * np.abs(want[b]).max() * np.abs(k).max() * r.layer.softmax_scale
        assert_row(got[b], o, mag, peak, flip)


def test_decode_after_eviction_uses_the_true_position():
    """Held pages with gaps between them: queries turn by pos, the mask goes by the held keys."""
    r = Rows("global", [330, 90], seed=28, gap=0)
    r.fill()
    keep = [[0, 3, 4, 9, 20], [1, 2, 5]]
    table = torch.full_like(r.table, -1)
    for b, pages in enumerate(keep):
        table[b, :len(pages)] = r.table[b, pages]
    lens = [4 * 16 + 330 % 16, 2 * 16 + 90 % 16]
    pos = [329, 89]
    q = gi.bf16_normal((2, 32, 512), 5).cuda()
    out = torch.empty_like(q)
    w = torch.zeros(r.table.shape, device="cuda")
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, 2, table.shape[1], True), dtype=torch.uint8,
                     device="cuda")
    g4.g4attn_kv8_decode(r.layer, None, q, None, None, i32(lens), r.cache.desc, table, out, ws, pos=i32(pos),
                         page_weights=w)
    status_ok()
    roped, steps = turned_queries(r.olayer, q, pos)
    for b, pages in enumerate(keep):
        idx = np.concatenate([np.arange(16 * p, 16 * p + 16) for p in pages])[:lens[b]]
        k, v = kv8.keys_values(r.olayer, *(x[idx] for x in r.values(b)))
        want, p, mag, peak = kv8.decode(roped[b], k, v, r.layer.softmax_scale)
        more = border(steps[b], k, r.layer.softmax_scale)
        assert_row(f64(out[b]), want, mag, peak, more)
        s = kv8.page_sums(p)
        assert np.allclose(f64(w[b])[:len(s)], s, rtol=2e-5 + more.max(), atol=1e-9)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_rows_do_not_depend_on_the_batch(kind):
    lens = [900, 77, 2500, 1, 1024]
    r = Rows(kind, lens, seed=29, gap=0)
    r.fill()
    s = Step(r, weights=kind == "global")
    s.run()
    status_ok()
    for b in range(5):
        wide = torch.full((1, r.table.shape[1] + 40), -1, dtype=torch.int32, device="cuda")
        wide[0, :r.table.shape[1]] = r.table[b]
        out = torch.empty_like(s.out[b:b + 1])
        w = torch.zeros(wide.shape, device="cuda") if kind == "global" else None
        ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, 1, wide.shape[1], kind == "global"),
                         dtype=torch.uint8, device="cuda")
        g4.g4attn_kv8_decode(r.layer, None, s.q[b:b + 1], None, None, i32(lens[b:b + 1]), r.cache.desc, wide, out, ws,
                             page_weights=w)
        status_ok()
        assert torch.equal(out[0], s.out[b])
        if w is not None:
            assert torch.equal(w[0, :r.table.shape[1]], s.weights[b])


def test_decode_page_weights_accumulate_and_do_not_change_the_output():
    r = Rows("global", [300, 1400], seed=30, gap=0)
    r.fill()
    s = Step(r, weights=True)
    s.run()
    one, out = s.weights.clone(), s.out.clone()
    s.run()
    status_ok()
    assert torch.equal(s.weights, one * 2)
    assert np.allclose(f64(one).sum(1), 32.0, rtol=1e-5)          # a step adds one per head
    plain = Step(r)
    plain.run()
    status_ok()
    assert torch.equal(plain.out, out)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_bad_requests_give_zeros_and_an_error(kind):
    r = Rows(kind, [40, 50, 60, 70], seed=31, gap=0)
    r.fill()
    s = Step(r)
    s.run()
    status_ok()
    good = s.out.clone()
    width = 16 * r.table.shape[1]
    for bad_len in (0, -5, width + 1, 2 ** 31 - 1):
        s.out.fill_(float("nan"))
        lens = list(s.lens)
        lens[2] = bad_len
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(lens), r.cache.desc, r.table, s.out, s.ws)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert (s.out[2] == 0).all()
        assert all(torch.equal(s.out[b], good[b]) for b in (0, 1, 3))
    for bad_pos in (58, 262144):                     # before the held keys' end, past the last position
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, r.table, s.out, s.ws,
                             pos=i32([39, 49, bad_pos, 69]))
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert (s.out[2] == 0).all() and torch.equal(s.out[1], good[1])
    for bad_page in (-1, r.plan.num_pages, 2 ** 31 - 1):
        table = r.table.clone()
        table[2, 0:4] = bad_page
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, table, s.out, s.ws)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert (s.out[2] == 0).all()
        assert all(torch.equal(s.out[b], good[b]) for b in (0, 1, 3))


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_bad_vectors_show_only_where_they_are_seen(kind):
    """A NaN key makes the rows of its KV head NaN; stale slots and unseen keys never matter."""
    r = Rows(kind, [50, 2000], seed=32, gap=0)
    (r.v if kind == "sliding" else r.k)[0][7, 1, 3] = float("nan")
    r.k[1][3, 0, 0] = float("inf")                     # outside the window of the sliding layer
    r.fill()
    s = Step(r)
    s.run()
    status_ok()
    group = r.layer.n_q_heads // r.layer.n_kv_heads
    bad = torch.isnan(s.out).all(-1)
    some = torch.isnan(s.out).any(-1)
    assert torch.equal(bad, some)
    want = torch.zeros_like(bad)
    want[0, group:2 * group] = True
    if kind == "global":
        want[1, :group] = True
    assert torch.equal(bad, want)


def test_decode_pool_past_4_gib():
    """Page blocks beyond 2^32 bytes of the pool."""
    layer, ol = make_layers("global")
    num = (2 ** 32) // (4 * 10272) + 50
    r = Rows("global", [100], seed=33, gap=0)
    r.fill()
    big = PagedKV8(layer, num, fill=None)
    table = r.table + (num - r.plan.num_pages)
    big.pages[num - r.plan.num_pages:] = r.cache.pages
    s = Step(r)
    s.run()
    status_ok()
    out = torch.empty_like(s.out)
    g4.g4attn_kv8_decode(layer, None, s.q, None, None, i32([100]), big.desc, table, out, s.ws)
    status_ok()
    assert torch.equal(out, s.out)
    # and appends there
    g4.g4attn_kv8_append(layer, None, r.k[0].cuda(), None, i32([0]), i32([100]), i32([0]), big.desc, table)
    status_ok()
    assert torch.equal(big.pages[num - r.plan.num_pages:][r.table[0].long()][:-1],
                       r.cache.pages[r.table[0].long()][:-1])


@pytest.mark.parametrize("kind,B,length", [("sliding", 96, 1024), ("global", 64, 4096)])
def test_decode_wait_that_runs_out_is_reported_and_the_next_call_is_exact(kind, B, length):
    """Enough requests that the page copies queue up behind one another and some first poll fails."""
    layer, _ = make_layers(kind)
    width = length // 16
    cache = PagedKV8(layer, B * width, fill=None)
    cache.pages.random_(100, 140)                     # exponents too: steps around 2^-13
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    q = gi.bf16_normal((B, 32, layer.head_dim), 3).cuda()
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, B, width), dtype=torch.uint8, device="cuda")

    def run():
        out = torch.full_like(q, float("nan"))
        g4.g4attn_kv8_decode(layer, None, q, None, None, i32([length] * B), cache.desc, table, out, ws)
        torch.cuda.synchronize()
        return out, g4.g4attn_status_sync()
    ref, st = run()
    assert st == g4.G4_OK
    g4.g4attn_set_wait_limit_ns(0)
    try:
        _, st = run()
    finally:
        g4.g4attn_set_wait_limit_ns(g4.DEFAULT_WAIT_LIMIT_NS)
    assert st == g4.G4_ERR_TIMEOUT, g4.status_string(st)
    again, st = run()
    assert st == g4.G4_OK and torch.equal(again, ref)


# ---- prefill ------------------------------------------------------------------------------------------

def prefill(r, norms=None, span=None):
    n = None if norms is None else norms.arg
    r.append_history(n)
    scratch = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, r.kind == "global")
    q = r.pack(r.q)
    out = torch.full_like(q, 5.0)
    g4.g4attn_kv8_prefill(r.layer, n, q, r.pack(r.k), None if r.v is None else r.pack(r.v), *r.row_args(), r.cache.desc,
                          r.table, scratch.desc, r.table, out, span=span)
    status_ok()
    return q, out, scratch


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_prefill_is_the_attention_over_the_stored_values(kind):
    r = Rows(kind, [96, 1, 200, 0, 300], [0, 40, 17, 5, 1500], seed=41)
    q, out, scratch = prefill(r)
    # the same attention kernel on bf16 pages made from the cache's bytes
    k, two = bf16_pages(r.layer, r.cache.pages)
    other = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    other.k.copy_(k.reshape(other.k.shape))
    (other.k_rot if kind == "global" else other.v).copy_(two.reshape((other.k_rot if kind == "global" else other.v).shape))
    ref = torch.full_like(q, 5.0)
    g4.g4attn_prefill_attend(r.layer, q, *r.row_args(), other.desc, r.table, ref)
    status_ok()
    assert torch.equal(out, ref)
    gap = torch.ones(r.T, dtype=torch.bool)
    for s, n in zip(r.start, r.rows):
        gap[s:s + n] = False
    assert (out[gap.cuda()] == 5.0).all() and torch.isfinite(out).all()
    # and near the definition: bf16 outputs of fp32 sums (the library's own bar for the bf16 cache)
    for b in (0, 2):
        kk, vv = kv8.keys_values(r.olayer, *r.values(b))
        n, c = r.rows[b], r.ctx[b]
        roped = f64(g4.g4attn_rope_apply(r.layer, r.q[b].cuda(), i32(list(range(c, c + n)))))
        group = r.layer.n_q_heads // r.layer.n_kv_heads
        for h in (0, 31):
            want = oracle.attention(roped[:, h], kk[:, h // group], vv[:, h // group], np.arange(c, c + n),
                                    np.arange(c + n), r.layer.window, r.layer.softmax_scale)
            err = np.abs(f64(out[r.start[b]:r.start[b] + n, h]) - want)
            assert err.max() <= 2e-2 and err.mean() <= 2e-3


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_prefill_in_chunks_is_bit_identical(kind, normed):
    norms = Norms(kind, 8) if normed else None
    whole = Rows(kind, [1300], seed=42, gap=0)
    _, ref, _ = prefill(whole, norms)
    cut = Rows(kind, [1300], seed=42, gap=0)
    scratch = PagedKV(cut.plan.num_pages, cut.layer.n_kv_heads, cut.layer.head_dim, kind == "global")
    got = torch.empty_like(ref)
    for lo, hi in ((0, 5), (5, 640), (640, 641), (641, 1300)):
        q, k = cut.q[0][lo:hi].cuda(), cut.k[0][lo:hi].cuda()
        v = None if cut.v is None else cut.v[0][lo:hi].cuda()
        got[lo:hi] = g4.g4attn_kv8_prefill(cut.layer, None if norms is None else norms.arg, q, k, v, i32([0]),
                                           i32([hi - lo]), i32([lo]), cut.cache.desc, cut.table, scratch.desc, cut.table,
                                           torch.empty_like(q))
    status_ok()
    assert torch.equal(cut.cache.pages, whole.cache.pages)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_prefill_with_image_spans(kind):
    r = Rows(kind, [150, 1300], [30, 0], seed=43, gap=1)
    span = torch.zeros(r.T, 2, dtype=torch.int32)
    images = [(50, 140), (20, 1200)]
    for b, (s0, s1) in enumerate(images):
        span[r.start[b] + s0 - r.ctx[b]:r.start[b] + s1 - r.ctx[b]] = torch.tensor([s0, s1], dtype=torch.int32)
    q, out, _ = prefill(r, span=span.cuda())
    for b in range(2):
        n, c = r.rows[b], r.ctx[b]
        kk, vv = kv8.keys_values(r.olayer, *r.values(b))
        roped = f64(g4.g4attn_rope_apply(r.layer, r.q[b].cuda(), i32(list(range(c, c + n)))))
        group = r.layer.n_q_heads // r.layer.n_kv_heads
        want = oracle.attention(roped[:, 5], kk[:, 5 // group], vv[:, 5 // group], np.arange(c, c + n), np.arange(c + n),
                                r.layer.window, r.layer.softmax_scale, [images[b]])
        err = np.abs(f64(out[r.start[b]:r.start[b] + n, 5]) - want)
        assert err.max() <= 2e-2 and err.mean() <= 2e-3


def test_prefill_with_an_image_that_began_before_the_chunk():
    """The image starts before the chunk's window does: its keys are read back too."""
    r = Rows("sliding", [150, 90], [60, 70], seed=45, gap=1, window=16)
    span = torch.zeros(r.T, 2, dtype=torch.int32)
    images = [(5, 140), (33, 71)]
    for b, (s0, s1) in enumerate(images):
        span[r.start[b]:r.start[b] + s1 - r.ctx[b]] = torch.tensor([s0, s1], dtype=torch.int32)
    q, out, scratch = prefill(r, span=span.cuda())
    for b, (s0, _) in enumerate(images):
        pages = r.table[b, s0 // 16:(r.ctx[b] + r.rows[b] + 15) // 16].long()
        held = scratch.k[pages].isfinite().flatten(1).all(1)
        assert held[:-1].all()                                  # (the last page's tail holds no key)
    for b in range(2):
        n, c = r.rows[b], r.ctx[b]
        kk, vv = kv8.keys_values(r.olayer, *r.values(b))
        roped = f64(g4.g4attn_rope_apply(r.layer, r.q[b].cuda(), i32(list(range(c, c + n)))))
        group = r.layer.n_q_heads // r.layer.n_kv_heads
        want = oracle.attention(roped[:, 5], kk[:, 5 // group], vv[:, 5 // group], np.arange(c, c + n), np.arange(c + n),
                                16, r.layer.softmax_scale, [images[b]])
        err = np.abs(f64(out[r.start[b]:r.start[b] + n, 5]) - want)
        assert err.max() <= 2e-2 and err.mean() <= 2e-3


def test_prefill_refuses_a_bad_sequence_and_serves_the_others():
    r = Rows("sliding", [60, 70], seed=44)
    _, ref, _ = prefill(r)
    q, k, v = r.pack(r.q), r.pack(r.k), r.pack(r.v)
    scratch = PagedKV(r.plan.num_pages, 16, 256, False)
    out = torch.full_like(q, 5.0)
    g4.g4attn_kv8_prefill(r.layer, None, q, k, v, i32([r.T - 9, r.start[1]]), i32(r.rows), i32(r.ctx), r.cache.desc,
                          r.table, scratch.desc, r.table, out)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    assert torch.equal(out[r.start[1]:r.start[1] + 70], ref[r.start[1]:r.start[1] + 70])
    assert (out[:r.start[1]] == 5.0).all()


# ---- eviction -----------------------------------------------------------------------------------------

def run_evict(lens, table, weights, keep, first, last, in_place=False):
    t, w, n = i32(table), torch.tensor(weights, dtype=torch.float32, device="cuda"), i32(lens)
    if in_place:
        out = [n, t, w]
    else:
        out = [torch.full_like(n, -9), torch.full_like(t, -9), torch.full_like(w, -9)]
    freed, nf = torch.full_like(t, -9), torch.full_like(n, -9)
    g4.g4attn_evict_pages(n, t, w, keep, first, last, *out, freed, nf)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in (*out, freed, nf)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("width,keep,first,last", [(1, 1, 0, 1), (7, 3, 1, 1), (40, 39, 5, 30), (40, 2, 0, 2),
                                                   (1500, 700, 4, 64), (1025, 1, 0, 1), (16384, 1024, 4, 64),
                                                   (16384, 16384, 1, 1), (2050, 1030, 0, 1)])
def test_evict_matches_the_definition(width, keep, first, last, in_place):
    rng = np.random.default_rng(width + keep)
    B = 6
    lens = [16 * width, max(0, 16 * width - 15), int(rng.integers(0, 16 * width + 1)), 0, 1, 16 * min(width, keep)]
    lens = [min(x, 262144) for x in lens]
    table = rng.permutation(B * width).reshape(B, width).tolist()
    w = np.exp(rng.standard_normal((B, width)) * 3).astype(np.float32)
    w[rng.random((B, width)) < 0.3] = 0.0                       # many exact ties
    w[0, ::7] = w[0, 0]
    if width > 6:
        w[1, 3], w[1, 4], w[1, 5] = np.inf, np.nan, -2.5        # a caller's own values
    got = run_evict(lens, table, w.tolist(), keep, first, last, in_place)
    assert g4.g4attn_status_sync() == g4.G4_OK
    for b in range(B):
        n, kept, kw, out = kv8.evict(lens[b], table[b], w[b].tolist(), keep, first, last)
        assert got[0][b] == n and got[4][b] == len(out)
        assert got[1][b] == kept + [-1] * (width - len(kept))
        assert np.array_equal(np.float32(got[2][b]), np.float32(kw + [0.0] * (width - len(kept))), equal_nan=True)
        assert got[3][b] == out + [-1] * (width - len(out))


def test_evict_many_sequences_twice():
    """Weights without ties, so that most searches end early, at every bit: each row against the definition,
    and the same again."""
    rng = np.random.default_rng(91)
    B, width, keep = 400, 2050, 700
    lens = rng.integers(16 * keep, 16 * width + 1, B).tolist()
    table = rng.permutation(B * width).reshape(B, width).tolist()
    w = rng.random((B, width)).astype(np.float32)
    w[::2] = np.exp(20 * w[::2] - 10)
    w = w.tolist()
    first = run_evict(lens, table, w, keep, 2, 3)
    status_ok()
    for b in range(B):
        n, kept, kw, out = kv8.evict(lens[b], table[b], w[b], keep, 2, 3)
        assert first[0][b] == n and first[4][b] == len(out)
        assert first[1][b] == kept + [-1] * (width - len(kept)) and first[3][b] == out + [-1] * (width - len(out))
    for in_place in (False, True):
        assert run_evict(lens, table, w, keep, 2, 3, in_place) == first


def test_evict_passes_a_bad_sequence_on():
    table, w = [[3, 4, 5, 6]] * 3, [[1.0, 2.0, 3.0, 4.0]] * 3
    for bad in (-1, 65, 2 ** 31 - 1):
        got = run_evict([64, bad, 64], table, w, 2, 0, 1)
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert got[0] == [32, bad, 32] and got[1][1] == table[1] and got[2][1] == w[1] and got[4] == [2, 0, 2]
        assert got[1][0] == [5, 6, -1, -1] and got[3][0] == [3, 4, -1, -1]


# ---- larger sizes and other schedules --------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_seventy_sequences(kind):
    """More sequences than a warp looks at at once: append, read-back, prefill and decode."""
    rng = np.random.default_rng(7)
    rows = [int(x) for x in rng.integers(0, 5, 70)]
    rows[3], rows[69] = 40, 33
    ctx = [int(x) for x in rng.integers(0, 40, 70)]
    ctx = [max(c, 1 - n) for c, n in zip(ctx, rows)]
    r = Rows(kind, rows, ctx, seed=71, gap=1)
    q, out, scratch = prefill(r)
    for b in (0, 3, 33, 64, 69):
        n = rows[b] + ctx[b]
        for i, (got, want) in enumerate(zip(r.values(b), r.exact_parts(b))):
            raw = i == 1 if kind == "sliding" else i == 0
            assert_stored(got[:n], want, rounded=not raw)
    k, two = bf16_pages(r.layer, r.cache.pages)
    other = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    other.k.copy_(k.reshape(other.k.shape))
    (other.k_rot if kind == "global" else other.v).copy_(two.reshape((other.k_rot if kind == "global" else other.v).shape))
    ref = torch.full_like(q, 5.0)
    g4.g4attn_prefill_attend(r.layer, q, *r.row_args(), other.desc, r.table, ref)
    status_ok()
    assert torch.equal(out, ref)
    s = Step(r, weights=kind == "global")
    s.run()
    s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_row_does_not_depend_on_the_table_width(kind):
    """Wide page tables take the split merge: the same bits."""
    r = Rows(kind, [3000, 70], seed=72, gap=0, window=30000)
    r.fill()
    s = Step(r, weights=kind == "global")
    s.run()
    s.check()
    wide = torch.full((2, r.table.shape[1] + 5000), -1, dtype=torch.int32, device="cuda")
    wide[:, :r.table.shape[1]] = r.table
    w = torch.zeros(wide.shape, device="cuda") if kind == "global" else None
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, 2, wide.shape[1], kind == "global"), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(s.out)
    g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, wide, out, ws, page_weights=w)
    status_ok()
    assert torch.equal(out, s.out)
    if w is not None:
        assert torch.equal(w[:, :r.table.shape[1]], s.weights) and (w[:, r.table.shape[1]:] == 0).all()


@pytest.mark.parametrize("kind,limit", [("global", 64), ("sliding", 32)])
def test_decode_of_one_chunk_gives_the_merged_bits(kind, limit):
    """Tables of one chunk are served without a merge, into q itself here: the bits of a wider table's call,
    zeros for a request that is refused or has a page outside the pool."""
    r = Rows(kind, [16 * limit, 1, 16, 333, 40, 50], seed=77, gap=0, norms=Norms(kind, 3))
    r.fill()
    wide = r.table.clone()
    wide[4, 1] = r.plan.num_pages
    wide = torch.cat([wide, torch.full((6, limit + 1 - wide.shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    lens = i32([16 * limit, 1, 16, 333, 40, 0])
    q = gi.bf16_normal((6, r.layer.n_q_heads, r.layer.head_dim), 9).cuda()
    got = []
    for width in (limit, limit + 1):
        table, out = wide[:, :width].contiguous(), q.clone()
        ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, 6, width), dtype=torch.uint8, device="cuda")
        g4.g4attn_kv8_decode(r.layer, r.norms.arg, out, None, None, lens, r.cache.desc, table, out, ws)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        got.append(out)
    assert torch.equal(got[0], got[1])
    group = r.layer.n_q_heads // r.layer.n_kv_heads
    assert (got[0][5] == 0).all() and (got[0][4].unflatten(0, (-1, group)) == 0).all()
    assert (got[0][:4] != 0).flatten(1).any(1).all()


def test_decode_table_wider_than_the_longest_sequence():
    """Columns past position 262143 hold no page: they are neither read nor written."""
    r = Rows("global", [3000, 70], seed=72, gap=0)
    r.fill()
    s = Step(r, weights=True)
    s.run()
    s.check()
    wide = torch.full((2, 16384 + 5000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :r.table.shape[1]] = r.table
    w = torch.full(wide.shape, 2.0, device="cuda")
    w[:, :r.table.shape[1]] = 0.0
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, 2, wide.shape[1], True), dtype=torch.uint8,
                     device="cuda").fill_(255)
    out = torch.empty_like(s.out)
    g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, wide, out, ws, page_weights=w)
    status_ok()
    assert torch.equal(out, s.out)
    assert torch.equal(w[:, :r.table.shape[1]], s.weights) and (w[:, r.table.shape[1]:] == 2.0).all()


@pytest.mark.parametrize("kind,window", [("global", 0), ("sliding", 262144)])
def test_decode_longest_context(kind, window):
    """262144 keys, the last usable position, against fp64 on the device. Beyond the tolerance above: the
    sums run over 2^18 keys, in runs of 16 pages per warp and 256 or 512 chunks, each addition off by at
    most 2^-24 of a partial sum that is at most sum p |v|: under 2^-15 of it in all."""
    layer = g4.global_layer() if kind == "global" else g4.sliding_layer(window)
    hkv, d, hq = layer.n_kv_heads, layer.head_dim, 32
    n = 262144
    cache = PagedKV8(layer, n // 16, fill=None)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache.pages.random_(28, 229, generator=g)                       # codes -100 .. 100
    cache.pages[..., -32:].random_(126, 129, generator=g)           # steps 2^-7 .. 2^-5
    table = torch.randperm(n // 16, generator=g, device="cuda").int()[None].contiguous()
    q = gi.bf16_normal((1, hq, d), 9).cuda()
    out = torch.empty_like(q)
    w = torch.zeros(table.shape, device="cuda") if kind == "global" else None
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, 1, n // 16, kind == "global"), dtype=torch.uint8,
                     device="cuda")
    g4.g4attn_kv8_decode(layer, None, q, None, None, i32([n]), cache.desc, table, out, ws, page_weights=w)
    status_ok()
    olayer = oracle.GLOBAL if kind == "global" else oracle.SLIDING
    turned, steps = turned_queries(olayer, q, [n - 1])
    roped = torch.tensor(turned[0], device="cuda")
    one, two = (x[table[0].long()].transpose(1, 2).flatten(0, 1).double() for x in untile8(cache.pages, d))
    cols = torch.tensor(kv8.turned_columns(olayer), device="cuda")
    most = 0.0
    pages = torch.zeros(n // 16, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        k, v = one[:, h], (one if kind == "global" else two)[:, h]
        if kind == "global":
            k = k.clone()
            k[:, cols] = two[:, h]
        group = hq // hkv
        p = torch.softmax(roped[group * h:group * (h + 1)] @ k.T * layer.softmax_scale, -1)
        want, mag = p @ v, p @ v.abs()
        peak = n * (p * v.abs().amax(-1)).amax(-1, keepdim=True)
        got = out[0, group * h:group * (h + 1)].double()
        more = torch.tensor(border(steps[0, group * h:group * (h + 1)], k.abs().amax(0)[None, None].cpu().numpy(),
                                   layer.softmax_scale), device="cuda")
        most = max(most, float(more.max()))
        over = (got - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -14 + more) * mag + 2.0 ** -31 * peak)
        assert (over <= 0).all(), float(over.max())
        pages += p.sum(0).unflatten(0, (-1, 16)).sum(-1)
    if w is not None:
        assert torch.allclose(w[0].double(), pages, rtol=2e-5 + most, atol=1e-9)


def test_two_calls_at_once():
    """Steps of two layers on two streams, each with its own workspace, over one cache."""
    r = Rows("global", [700, 1500, 40], seed=73, gap=0)
    r.fill()
    want = []
    for seed in (1, 2):
        s = Step(r, seed=seed, weights=True)
        for _ in range(20):
            s.run()
        status_ok()
        want.append((s.out.clone(), s.weights.clone()))
    steps = [Step(r, seed=seed, weights=True) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    lens = i32(steps[0].lens)
    for _ in range(20):
        for s, st in zip(steps, streams):
            g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, lens, r.cache.desc, r.table, s.out, s.ws,
                                 page_weights=s.weights, stream=st)
    status_ok()
    for st in streams:
        assert g4.g4attn_status_sync(st) == g4.G4_OK
    for s, (out, w) in zip(steps, want):
        assert torch.equal(s.out, out) and torch.equal(s.weights, w)


def test_wrong_device_and_strides_are_refused():
    r = Rows("global", [40], seed=74, gap=0)
    r.fill()
    s = Step(r)
    with pytest.raises(ValueError, match="current CUDA device"):
        g4.g4attn_kv8_decode(r.layer, None, s.q.cpu(), None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws)
    # one row of two is dense whatever its stride says; every other column is not
    g4.g4attn_kv8_decode(r.layer, None, torch.cat([s.q, s.q])[::2], None, None, i32([40]), r.cache.desc, r.table, s.out,
                         s.ws)
    status_ok()
    with pytest.raises(ValueError, match="strided"):
        g4.g4attn_kv8_decode(r.layer, None, torch.cat([s.q, s.q], -1)[..., ::2], None, None, i32([40]), r.cache.desc,
                             r.table, s.out, s.ws)
    with pytest.raises(g4.G4Error):
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws[:64])


def test_a_workspace_elsewhere_is_refused():
    r = Rows("global", [40], seed=74, gap=0)
    s = Step(r)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws.cpu())


# ---- together -------------------------------------------------------------------------------------------

def test_a_conversation_prefill_decode_evict_decode():
    """Prefill a prompt, decode with weights, trim the cache, decode on: every step against fp64 over the
    keys that are held."""
    r = Rows("global", [150, 420], seed=51, gap=0)
    _, _, _ = prefill(r)
    layer, ol, B, width = r.layer, r.olayer, 2, 64
    lens, pos = [150, 420], [149, 419]
    keys = [[x.copy() for x in r.values(b)] for b in range(B)]           # held keys' stored values
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, :r.plan.max_pages] = r.plan.table
    pool = PagedKV8(layer, r.plan.num_pages + 40)
    pool.pages[:r.plan.num_pages] = r.cache.pages
    free = list(range(r.plan.num_pages, r.plan.num_pages + 40))
    w = torch.zeros(B, width, device="cuda")
    acc, most = [np.zeros(0), np.zeros(0)], [0.0, 0.0]
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(layer, B, width, True), dtype=torch.uint8, device="cuda")
    d_table = table.cuda()
    for step in range(40):
        for b in range(B):
            lens[b] += 1
            pos[b] += 1
            if (lens[b] - 1) % 16 == 0:
                d_table[b, (lens[b] - 1) // 16] = free.pop()
        q, k_new = gi.bf16_normal((B, 32, 512), 900 + step).cuda(), gi.bf16_normal((B, 4, 512), 1900 + step)
        out = torch.empty_like(q)
        g4.g4attn_kv8_decode(layer, None, q, k_new.cuda(), None, i32(lens), pool.desc, d_table, out, ws, pos=i32(pos),
                             page_weights=w)
        status_ok()
        roped, steps = turned_queries(ol, q, pos)
        one, two = untile8(pool.pages, 512)
        for b in range(B):
            page, slot = int(d_table[b, (lens[b] - 1) // 16]), (lens[b] - 1) % 16
            new = [x[page, :, slot].double().cpu().numpy()[None] for x in (one, two)]
            for x, y in zip(new, kv8.parts(ol, k_new[b:b + 1].double().numpy(), None, [pos[b]])):
                assert_stored(x, y, rounded=True)
            keys[b] = [np.concatenate([x, y]) for x, y in zip(keys[b], new)]
            k, v = kv8.keys_values(ol, *keys[b])
            want, p, mag, peak = kv8.decode(roped[b], k, v, layer.softmax_scale)
            more = border(steps[b], k, layer.softmax_scale)
            assert_row(f64(out[b]), want, mag, peak, more)
            s = kv8.page_sums(p)
            acc[b] = np.concatenate([acc[b], np.zeros(len(s) - len(acc[b]))]) + s
            most[b] = max(most[b], more.max())
            assert np.allclose(f64(w[b])[:len(s)], acc[b], rtol=1e-4 + most[b])
        if step in (12, 30):
            n_len, nf = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
            freed = torch.empty_like(d_table)
            before, w_before = d_table.cpu().tolist(), w.cpu().tolist()
            g4.g4attn_evict_pages(i32(lens), d_table, w, 8, 1, 2, n_len, d_table, w, freed, nf)
            status_ok()
            for b in range(B):
                n, kept, kw, out_pages = kv8.evict(lens[b], before[b], w_before[b], 8, 1, 2)
                assert int(n_len[b]) == n and d_table[b, :len(kept)].tolist() == kept
                held = (lens[b] + 15) // 16
                idx = [i for i in range(held) if before[b][i] in kept]
                sel = np.concatenate([np.arange(16 * i, min(16 * i + 16, lens[b])) for i in idx])
                keys[b] = [x[sel] for x in keys[b]]
                acc[b] = acc[b][idx]
                lens[b] = n
                free.extend(int(x) for x in freed[b, :int(nf[b])])


def test_graphs_streams_and_shared_workspace():
    """Two captured steps that share a workspace, replayed in order on another stream; inputs change in place."""
    r = Rows("global", [300, 1100, 40], seed=61, gap=0)
    r.fill()
    a, b = Step(r, seed=1, weights=True), Step(r, seed=2, weights=True)
    ws = torch.empty_like(a.ws)
    lens = i32(a.lens)
    stream = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for s in (a, b):
            def call():
                g4.g4attn_kv8_decode(r.layer, None, s.q, None, None, lens, r.cache.desc, r.table, s.out, ws,
                                     page_weights=s.weights)
            call()
            s.weights.zero_()
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call()
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
        stream.synchronize()
    for s in (a, b):
        want = Step(r, seed=1 if s is a else 2, weights=True)
        for _ in range(3):
            want.run()
        status_ok()
        assert torch.equal(s.out, want.out) and torch.equal(s.weights, want.weights)
    lens.sub_(7)
    graphs[0].replay()
    torch.cuda.synchronize()
    short = Step(r, seed=1)
    g4.g4attn_kv8_decode(r.layer, None, short.q, None, None, lens, r.cache.desc, r.table, short.out, short.ws)
    status_ok()
    assert torch.equal(a.out, short.out)


def test_captured_serving_step_between_copies_and_fills():
    """One graph: inputs copied in, weights set to zero, decode with a new token, eviction into other buffers,
    a copy out. Replayed over changed inputs it gives what the calls give one by one."""
    r = Rows("global", [300, 1100, 40], seed=62, gap=0)
    r.fill()
    B, width = 3, r.table.shape[1] + 1
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, :r.table.shape[1]] = r.table.cpu()
    pool = PagedKV8(r.layer, r.plan.num_pages + B)
    pool.pages[:r.plan.num_pages] = r.cache.pages
    lens = [n + 1 for n in r.rows]
    for b in range(B):
        if r.rows[b] % 16 == 0:
            table[b, r.rows[b] // 16] = r.plan.num_pages + b
    table, lens = table.cuda(), i32(lens)
    ws = torch.empty(g4.g4attn_kv8_decode_workspace_bytes(r.layer, B, width, True), dtype=torch.uint8, device="cuda")

    def buffers():
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")   # noqa: E731
        return dict(q=torch.zeros(B, 32, 512, dtype=torch.bfloat16, device="cuda"),
                    k=torch.zeros(B, 4, 512, dtype=torch.bfloat16, device="cuda"),
                    out=torch.zeros(B, 32, 512, dtype=torch.bfloat16, device="cuda"),
                    w=torch.zeros(B, width, device="cuda"), n_len=z(B), n_table=z(B, width),
                    n_w=torch.zeros(B, width, device="cuda"), freed=z(B, width), nf=z(B), copy=z(B, width))

    def step(x, q, k):
        x["q"].copy_(q)
        x["k"].copy_(k)
        x["w"].zero_()
        g4.g4attn_kv8_decode(r.layer, None, x["q"], x["k"], None, lens, pool.desc, table, x["out"], ws,
                             page_weights=x["w"])
        g4.g4attn_evict_pages(lens, table, x["w"], 10, 1, 2, x["n_len"], x["n_table"], x["n_w"], x["freed"], x["nf"])
        x["copy"].copy_(x["n_table"])

    q_in, k_in = torch.zeros(B, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(
        B, 4, 512, dtype=torch.bfloat16, device="cuda")
    got, want = buffers(), buffers()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(got, q_in, k_in)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(got, q_in, k_in)
    for seed in range(4):
        q, k = gi.bf16_normal((B, 32, 512), 70 + seed).cuda(), gi.bf16_normal((B, 4, 512), 80 + seed).cuda()
        step(want, q, k)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            q_in.copy_(q)
            k_in.copy_(k)
            graph.replay()
            graph.replay()
        status_ok()
        for name in want:
            assert torch.equal(got[name], want[name]), name
