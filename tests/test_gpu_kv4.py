"""The 4-bit paged cache on the GPU, against the fp64 definition (oracle/kv4.py).

Tolerances, derived before the first run:
* Stored values. Raw V and S involve no rounding before the cast: bit-equal. Else the kernel's x is fp32 and at most
  2^-20 a off (a: the block's largest, see test_gpu_kv8.py), so it is stored as one of the two steps around it: the
  error is at most half the gap between steps at |x| (1 + 2^-18), in the larger of the two units that an a within
  2^-20 of a border can have, and 2^-19 a.
* Decode. Both sides compute from the values in the cache and from queries turned and cast alike, but for columns
  next to a border between two bf16 numbers (`border` in test_gpu_kv8.py). Left are the weights' cast to fp16 (2^-11 of
  each; below fp16's normal range half of its smallest step, 2^-25, where the row's largest weight p 2^top is at
  least 2^7), the product of that with a block's power of two (exact, or 2^-25 again), so 2^-24 / 2^7 of
  max p 2^top for each of n keys, times a code of at most 6, where max |v| >= 3.5 * 2^top: under 2^-30 n max p max|v|;
  fp32 sums (2^-16 of sum p |v|) and the cast of the output (2^-8):
  |got - want| <= 2^-8 |want| + (2^-11 + 2^-16) sum p |v| + n 2^-30 max p max|v|.
* Page weights: fp32 throughout, 2e-5 of themselves as over the 8-bit cache.
* Prefill: the attention kernel runs on the same bf16 pages as g4attn_prefill_attend: bit-equal to it.
"""
import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
import oracle
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV4, device_int32, tile, tile_v256, untile4
from oracle import kv4, kv8

from gpu_cases import Norms, f64
from test_gpu_kv8 import Rows, border, make_layers, status_ok, turned_queries
from test_gpu_tp import rank_heads

pytestmark = pytest.mark.gpu
i32 = device_int32


class Rows4(Rows):
    """Rows over a 4-bit cache."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.cache = PagedKV4(self.layer, self.plan.num_pages)

    def append_history(self, norms=None):
        if max(self.ctx) == 0:
            return
        starts = [sum(self.ctx[:b]) for b in range(len(self.ctx))]
        g4.g4attn_kv4_append(self.layer, norms, self.pack(self.k, True),
                             None if self.v is None else self.pack(self.v, True), i32(starts), i32(self.ctx),
                             i32([0] * len(self.ctx)), self.cache.desc, self.table)

    def append(self, norms=None):
        g4.g4attn_kv4_append(self.layer, norms, self.pack(self.k), None if self.v is None else self.pack(self.v),
                             *self.row_args(), self.cache.desc, self.table)

    def values(self, b):
        one, two = untile4(self.cache.pages, self.layer.head_dim)
        n = self.rows[b] + self.ctx[b]
        pages = self.plan.table[b, :(n + 15) // 16].long()
        return [x[pages.cuda()].transpose(1, 2).flatten(0, 1)[:n].double().cpu().numpy() for x in (one, two)]


def workspace(layer, B, width, weights=False):
    return torch.empty(g4.g4attn_kv4_decode_workspace_bytes(layer, B, width, weights), dtype=torch.uint8,
                       device="cuda").fill_(255)


class Step4:
    """A decode step over the keys of a Rows4 batch: one query per sequence."""

    def __init__(self, r, seed=11, weights=False, pos=None, q_scale=1.0):
        self.r, self.lens = r, [n + c for n, c in r.pairs()]
        self.q = gi.bf16_normal((len(self.lens), r.layer.n_q_heads, r.layer.head_dim), seed, q_scale).cuda()
        self.pos = [n - 1 for n in self.lens] if pos is None else pos
        self.given_pos = None if pos is None else i32(pos)
        self.weights = torch.zeros(r.table.shape, device="cuda") if weights else None
        self.ws = workspace(r.layer, len(self.lens), r.table.shape[1], weights)
        self.out = torch.full_like(self.q, float("nan"))

    def run(self, **kw):
        norms = None if self.r.norms is None else self.r.norms.arg
        a = dict(pos=self.given_pos, page_weights=self.weights)
        a.update(kw)
        return g4.g4attn_kv4_decode(self.r.layer, norms, self.q, None, None, i32(self.lens), self.r.cache.desc,
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
                w, s = f64(self.weights[b]), kv8.page_sums(p)
                assert np.allclose(w[:len(s)], s, rtol=2e-5 + more.max(), atol=1e-9), b
                assert (w[len(s):] == 0).all()


def assert_row(got, want, mag, peak, more=0.0):
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16 + more) * mag + 2.0 ** -30 * peak)
    assert (over <= 0).all(), over.max()


def assert_stored(got, exact, rounded):
    if not rounded:
        assert np.array_equal(got, kv4.stored(exact), equal_nan=True)
        return
    a = np.abs(exact).reshape(*exact.shape[:-1], -1, 32).max(-1)
    unit = np.exp2(np.repeat(kv4.exponents(exact * (1 + 2.0 ** -20)), 32, -1))
    m = np.abs(exact) * (1 + 2.0 ** -18) / unit
    limit = np.where(m < 2, 0.25, np.where(m < 4, 0.5, 1.0)) * unit + 2.0 ** -19 * np.repeat(a, 32, -1)
    assert (np.abs(got - exact) <= limit).all(), np.max(np.abs(got - exact) / unit)


# ---- append -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("tp", [1, 2, 8])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_stores_the_definition(kind, tp, normed):
    r = Rows4(kind, [1, 17, 40, 0, 16], [0, 15, 3, 9, 300], seed=1, tp=tp, norms=Norms(kind, 5) if normed else None)
    r.fill()
    status_ok()
    tops = r.cache.pages[..., -16:].cpu().numpy()
    for b in range(5):
        n = r.rows[b] + r.ctx[b]
        values = r.values(b)
        for i, (got, want) in enumerate(zip(values, r.exact_parts(b))):
            raw = not normed and (i == 1 if kind == "sliding" else i == 0)
            assert_stored(got[:n], want, rounded=not raw)
        # the top of a key is its largest scale byte
        v = values[1 if kind == "sliding" else 0]
        pages = r.plan.table[b].numpy()
        scale_at = 8 * (r.layer.head_dim + (256 if kind == "sliding" else 128)) + (128 if kind == "sliding" else 0)
        per = r.layer.head_dim // 32
        raw_pages = r.cache.pages.cpu().numpy()
        for j in range(n):
            at = scale_at + (j % 16) * per
            assert (tops[pages[j // 16], :, j % 16] == raw_pages[pages[j // 16], :, at:at + per].max(-1)).all()
        assert np.isfinite(v).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_sizes_zeros_and_bad_vectors(kind):
    """Blocks from 2^-79 to near the largest bf16 in one vector, borders between two exponents, zeros, infinities and
    NaN; neighbours keep theirs."""
    r = Rows4(kind, [24], seed=2)
    x = r.k[0] if kind == "global" else r.v[0]
    gen = torch.Generator().manual_seed(4)
    for t in range(8):
        e = torch.randint(-79, 124, (x.shape[1], x.shape[2] // 32, 1), generator=gen).double()
        x[t] = (x[t].double().clamp(-3, 3).unflatten(-1, (-1, 32)) * torch.exp2(e)).flatten(-2).bfloat16()
    x[8] = 0
    x[9, 0, 7], x[10, 0, 200], x[11, 0, 255] = float("inf"), float("-inf"), float("nan")
    x[12] = 0
    x[12, :, ::32] = torch.tensor(1.75)          # a = 7 * 2^-2 exactly, and the next bf16 above it
    x[12, :, 1::32], x[12, :, 2::32] = torch.tensor(0.0625), torch.tensor(-0.1875)
    x[13] = x[12]
    x[13, :, ::32] = torch.tensor(1.7578125)
    x[14, :, :] = torch.finfo(torch.bfloat16).max
    r.append()
    status_ok()
    got, want = r.values(0), r.exact_parts(0)
    raw = 0 if kind == "global" else 1
    assert_stored(got[raw], want[raw], rounded=False)
    assert np.isnan(got[raw][9:12, 0]).all() and np.isfinite(got[raw][9:12, 1]).all()
    assert np.isfinite(got[raw][14]).all()


def test_append_far_positions():
    """The last usable position, where fp32 angles would be 0.02 rad off."""
    for kind in ("sliding", "global"):
        layer, ol = make_layers(kind)
        n, ctx = 5, 262144 - 5
        k = gi.bf16_normal((n, layer.n_kv_heads, layer.head_dim), 3)
        v = gi.bf16_normal(tuple(k.shape), 4) if kind == "sliding" else None
        table = torch.full((1, 16384), -1, dtype=torch.int32)
        table[0, 16383] = 1
        cache = PagedKV4(layer, 2)
        g4.g4attn_kv4_append(layer, None, k.cuda(), None if v is None else v.cuda(), i32([0]), i32([n]), i32([ctx]),
                             cache.desc, table.cuda())
        status_ok()
        got = [x[1].transpose(0, 1)[ctx % 16:].double().cpu().numpy() for x in untile4(cache.pages, layer.head_dim)]
        want = kv8.parts(ol, k.double().numpy(), None if v is None else v.double().numpy(), np.arange(ctx, ctx + n))
        for g, w in zip(got, want):
            assert_stored(g, w, rounded=True)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_append_bytes_do_not_depend_on_chunks(kind):
    whole = Rows4(kind, [77], seed=7)
    whole.append()
    for cuts in ([0, 1, 77], [0, 16, 33, 34, 77]):
        cut = Rows4(kind, [77], seed=7)
        for lo, hi in zip(cuts, cuts[1:]):
            g4.g4attn_kv4_append(cut.layer, None, cut.k[0][lo:hi].cuda(), None if cut.v is None else cut.v[0][lo:hi].cuda(),
                                 i32([0]), i32([hi - lo]), i32([lo]), cut.cache.desc, cut.table)
        status_ok()
        assert torch.equal(whole.cache.pages, cut.cache.pages)


def test_append_refuses_on_the_device_and_writes_nothing_else():
    r = Rows4("sliding", [20, 20], seed=3)
    before = r.cache.pages.clone()
    k, v = r.pack(r.k), r.pack(r.v)

    def call(start, rows, ctx, table=r.table):
        g4.g4attn_kv4_append(r.layer, None, k, v, i32(start), i32(rows), i32(ctx), r.cache.desc, table)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert torch.equal(r.cache.pages, before)
    call([r.T - 3, 0], [20, 0], [0, 0])               # rows past T
    call([-1, 0], [20, 0], [0, 0])
    call([0, 0], [20, 0], [-4, 0])
    call([0, 0], [20, 0], [262143, 0])                # positions past the last
    call([0, 0], [5, 0], [16 * r.table.shape[1], 0])  # past the table
    call([0, 0], [5, 0], [0, 0], torch.full_like(r.table, r.plan.num_pages))
    call([0, 0], [5, 0], [0, 0], torch.full_like(r.table, -1))


# ---- read-back ----------------------------------------------------------------------------------------

def bf16_pages(layer, pages):
    """The bf16 cache tensors that hold the same values as the 4-bit pages."""
    one, two = untile4(pages, layer.head_dim)
    if layer.kv_shared:
        p, h = two.shape[:2]
        rot = two.bfloat16().reshape(p, h, 2, 8, 2, 8, 8).permute(0, 1, 4, 2, 5, 3, 6).contiguous()
        return tile(one.bfloat16()), rot
    return tile(one.bfloat16()), tile_v256(two.bfloat16())


@pytest.mark.parametrize("tp", [1, 8])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_unpack_is_exact_and_touches_only_its_keys(kind, tp):
    r = Rows4(kind, [100, 1, 33, 16], seed=4, tp=tp)
    r.fill()
    out = PagedKV(r.plan.num_pages + 2, r.layer.n_kv_heads, r.layer.head_dim, kind == "global", fill=-7.0)
    lo, hi = [5, 0, 33, 9], [97, 1, 33, 3]            # inside pages, whole, empty, reversed
    g4.g4attn_kv4_unpack(r.layer, i32(lo), i32(hi), r.cache.desc, r.table, out.desc, r.table + 2)
    status_ok()
    touched = torch.zeros(r.plan.num_pages + 2, 16, dtype=torch.bool)
    for b in range(4):
        for i in range(lo[b], hi[b]):
            touched[int(r.plan.table[b, i // 16]) + 2, i % 16] = True
    for g, w in zip((out.k, out.k_rot if kind == "global" else out.v), bf16_pages(r.layer, r.cache.pages)):
        w2 = torch.full_like(g, -7.0)
        w2[2:] = w.reshape(w.shape[0], *g.shape[1:])
        t = touched.cuda()[:, None, None, :].unflatten(-1, (2, 8))[..., None, :, None]     # [p, 1, 1, 2, 1, 8, 1]
        g7, w7 = (x.reshape(x.shape[0], x.shape[1], -1, 2, x.shape[-3], 8, 8) for x in (g, w2))
        assert torch.equal(g7, torch.where(t, w7, torch.full_like(w7, -7.0)))
    before = out.k.clone()
    for a, z, table in ((-1, 5, r.table), (0, 16 * r.table.shape[1] + 1, r.table), (0, 33, torch.full_like(r.table, -1))):
        g4.g4attn_kv4_unpack(r.layer, i32([0, 0, a, 0]), i32([0, 0, z, 0]), r.cache.desc, r.table, out.desc, table)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert torch.equal(out.k, before)


# ---- decode -------------------------------------------------------------------------------------------

LENS = [1, 2, 15, 16, 17, 64, 255, 257, 1023, 1024, 1025, 1100, 2300]


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_matches_the_definition(kind):
    r = Rows4(kind, LENS, seed=21, gap=0)
    r.fill()
    s = Step4(r, weights=kind == "global")
    s.run()
    s.check()


@pytest.mark.parametrize("window", [1, 16, 17, 250, 5000])
def test_decode_windows(window):
    r = Rows4("sliding", [1, 16, 33, 700, 6000], seed=22, gap=0, window=window)
    r.fill()
    s = Step4(r)
    s.run()
    s.check()


@pytest.mark.parametrize("kind,window", [("sliding", 1024), ("sliding", 129), ("sliding", 128), ("global", 0)])
def test_decode_around_chunk_ends(kind, window):
    """Lengths on both sides of a chunk's end, windows that begin on both sides of one; the last chunk holds one key."""
    lens = [127, 128, 129, 256, 257, 1023, 1025, 1151, 1152, 1153, 1154, 2049]
    r = Rows4(kind, lens, seed=24, gap=0, **({"window": window} if window else {}))
    r.fill()
    s = Step4(r, weights=kind == "global")
    s.run()
    s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_sharp_scores_and_blocks_of_very_different_sizes(kind):
    """Queries of size 6, values whose sizes differ by 2^13 from token to token and by 2^12 from block to block."""
    r = Rows4(kind, [5000, 900], seed=23, gap=0)
    g = torch.Generator().manual_seed(1)
    for x in (r.v if kind == "sliding" else r.k):
        size = torch.randint(-10, 3, (x.shape[0], 1, 1, 1), generator=g) + torch.randint(-12, 1, (1, 1, x.shape[2] // 32, 1),
                                                                                         generator=g)
        x.copy_((x.double().unflatten(-1, (-1, 32)) * torch.exp2(size.double())).flatten(-2).bfloat16())
    r.fill()
    s = Step4(r, weights=kind == "global", q_scale=6.0)
    s.run()
    s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_tiny_and_huge_values(kind):
    """Values near both ends of the stored range; queries far from 1."""
    for scale in (2.0 ** -70, 2.0 ** 60):
        r = Rows4(kind, [300, 40], seed=24, gap=0)
        for x in (r.v if kind == "sliding" else r.k):
            x.copy_((x.double() * scale).bfloat16())
        r.fill()
        s = Step4(r, q_scale=1.0 if kind == "sliding" else 1 / scale)
        s.run()
        s.check()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_of_keys_near_the_largest_bf16(kind):
    """Keys of size 2^113 under queries of size 2^-112: every product q.k, and every sum of them, is far inside
    fp32's range, and so are the outputs."""
    r = Rows4(kind, [300, 40, 1100], seed=106, gap=0)
    for x in r.k:
        x.copy_((x.double() * 2.0 ** 113).bfloat16())
    r.fill()
    s = Step4(r, weights=kind == "global", q_scale=2.0 ** -112)
    s.run()
    s.check()


@pytest.mark.parametrize("kind,weights", [("sliding", False), ("global", False), ("global", True)])
@pytest.mark.parametrize("tp", [2, 8])
def test_decode_rank_slices_are_the_full_call_bit_for_bit(kind, tp, weights):
    r = Rows4(kind, [700, 31, 1500, 2600], seed=101, gap=0)
    gen = torch.Generator().manual_seed(2)
    for x in (r.v if kind == "sliding" else r.k):
        x.copy_((x.double() * torch.exp2(torch.randint(-10, 3, (x.shape[0], 1, 1), generator=gen).double())).bfloat16())
    r.fill()
    s = Step4(r, weights=weights, q_scale=6.0)
    s.run()
    s.check()
    for rank in range(tp):
        (q0, q1), (k0, k1) = rank_heads(kind, tp, rank)
        layer, _ = make_layers(kind, tp=tp)
        cache = PagedKV4(layer, r.plan.num_pages)
        cache.pages.copy_(r.cache.pages[:, k0:k1])
        q = s.q[:, q0:q1].contiguous()
        out = torch.full_like(q, float("nan"))
        g4.g4attn_kv4_decode(layer, None, q, None, None, i32(s.lens), cache.desc, r.table, out,
                             workspace(layer, 4, r.table.shape[1], weights),
                             page_weights=torch.zeros(r.table.shape, device="cuda") if weights else None)
        status_ok()
        assert torch.equal(out, s.out[:, q0:q1]), (kind, tp, rank)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_appends_the_new_token_like_append(kind):
    """k_new in the call: the same bytes and the same output as an append before it; a request without keys gets none."""
    a = Rows4(kind, [1, 1, 1], [0, 16, 1200], seed=26, gap=0, norms=Norms(kind, 4))
    b = Rows4(kind, [1, 1, 1], [0, 16, 1200], seed=26, gap=0, norms=a.norms)
    a.fill()
    b.append_history(b.norms.arg)
    sa, sb = Step4(a), Step4(b)
    sa.run()
    args = (b.pack(b.k), None if b.v is None else b.pack(b.v))
    before = b.cache.pages.clone()
    g4.g4attn_kv4_decode(b.layer, b.norms.arg, sb.q, *args, i32([0, 0, 0]), b.cache.desc, b.table, sb.out, sb.ws)
    status_ok()
    assert torch.equal(b.cache.pages, before) and (sb.out == 0).all()
    g4.g4attn_kv4_decode(b.layer, b.norms.arg, sb.q, *args, i32(sb.lens), b.cache.desc, b.table, sb.out, sb.ws)
    status_ok()
    assert torch.equal(a.cache.pages, b.cache.pages)
    assert torch.equal(sa.out, sb.out)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_normed(kind):
    norms = Norms(kind, 9)
    r = Rows4(kind, [600, 45], seed=27, gap=0, norms=norms)
    r.fill()
    s = Step4(r)
    s.run()
    status_ok()
    qn = oracle.normed_q(norms.oracle, s.q.double().cpu().numpy())
    if kind == "global":
        rest = np.setdiff1d(np.arange(512), kv8.turned_columns(r.olayer))
        qn[..., rest] *= norms.oracle.k_weight[rest]
    want = f64(g4.g4attn_rope_apply(r.layer, torch.tensor(qn).bfloat16().cuda(), i32(s.pos)))
    got = f64(s.out)
    for b, n in enumerate(s.lens):
        k, v = kv8.keys_values(r.olayer, *r.values(b))
        o, _, mag, peak = kv8.decode(want[b], k, v, r.layer.softmax_scale, 0)
        # the norm's fp32 result may fall to the other side of a bf16 boundary in a few of 512 columns:
        # one column moves a score by at most 2^-8 |q| |k| scale, a weight by as much
        flip = 4 * 2.0 ** -8 * np.abs(want[b]).max() * np.abs(k).max() * r.layer.softmax_scale
        assert_row(got[b], o, mag, peak, flip)


def test_decode_after_eviction_uses_the_true_position():
    """Held pages with gaps between them: queries turn by pos, the mask goes by the held keys."""
    r = Rows4("global", [330, 90], seed=28, gap=0)
    r.fill()
    keep = [[0, 3, 4, 9, 20], [1, 2, 5]]
    table = torch.full_like(r.table, -1)
    for b, pages in enumerate(keep):
        table[b, :len(pages)] = r.table[b, pages]
    lens, pos = [4 * 16 + 330 % 16, 2 * 16 + 90 % 16], [329, 89]
    q = gi.bf16_normal((2, 32, 512), 5).cuda()
    out, w = torch.empty_like(q), torch.zeros(r.table.shape, device="cuda")
    g4.g4attn_kv4_decode(r.layer, None, q, None, None, i32(lens), r.cache.desc, table, out,
                         workspace(r.layer, 2, table.shape[1], True), pos=i32(pos), page_weights=w)
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
def test_decode_rows_do_not_depend_on_the_batch_or_the_table(kind):
    """Alone under a wider table (other merges), and in the batch: the same bits; page weights do not change them."""
    lens = [900, 77, 2500, 1, 1024, 400]
    r = Rows4(kind, lens, seed=29, gap=0)
    r.fill()
    s = Step4(r, weights=kind == "global")
    s.run()
    s.check()
    plain = Step4(r)
    plain.run()
    status_ok()
    assert torch.equal(plain.out, s.out)
    for b in range(6):
        for width in (max(1, (lens[b] + 15) // 16), r.table.shape[1] + 5000):
            table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
            n = min(width, r.table.shape[1])
            table[0, :n] = r.table[b, :n]
            out = torch.empty_like(s.out[b:b + 1])
            g4.g4attn_kv4_decode(r.layer, None, s.q[b:b + 1], None, None, i32(lens[b:b + 1]), r.cache.desc, table, out,
                                 workspace(r.layer, 1, width))
            status_ok()
            assert torch.equal(out[0], s.out[b]), (b, width)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_bad_requests_give_zeros_and_an_error_and_empty_ones_zeros(kind):
    r = Rows4(kind, [40, 50, 60, 70], seed=31, gap=0)
    r.fill()
    s = Step4(r)
    s.run()
    status_ok()
    good = s.out.clone()
    others = lambda: all(torch.equal(s.out[b], good[b]) for b in (0, 1, 3))   # noqa: E731
    for bad_len in (0, -5, 16 * r.table.shape[1] + 1, 2 ** 31 - 1):
        s.out.fill_(float("nan"))
        lens = list(s.lens)
        lens[2] = bad_len
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, i32(lens), r.cache.desc, r.table, s.out, s.ws)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == (g4.G4_OK if bad_len == 0 else g4.G4_ERR_DEVICE)
        assert (s.out[2] == 0).all() and others()
    for bad_pos in (58, 262144):                     # before the held keys' end, past the last position
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, r.table, s.out, s.ws,
                             pos=i32([39, 49, bad_pos, 69]))
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert (s.out[2] == 0).all() and torch.equal(s.out[1], good[1])
    for bad_page in (-1, r.plan.num_pages, 2 ** 31 - 1):
        table = r.table.clone()
        table[2, 0:4] = bad_page
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, i32(s.lens), r.cache.desc, table, s.out, s.ws)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert (s.out[2] == 0).all() and others()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_bad_vectors_and_stale_slots_show_only_where_they_are_seen(kind):
    """A NaN key makes the rows of its KV head NaN; keys behind the end or before the window hold anything."""
    r = Rows4(kind, [50, 2000], seed=32, gap=0)
    (r.v if kind == "sliding" else r.k)[0][7, 1, 3] = float("nan")
    r.k[0][40, 2, 5] = float("inf")
    r.k[1][3, 0, 0] = float("inf")                     # outside the window of the sliding layer
    r.fill()
    for fill in (0, 255, 0x7f):                         # what the slots past the end hold
        for b, n in enumerate((50, 2000)):
            page = int(r.plan.table[b, (n - 1) // 16])
            block = r.cache.pages[page]
            clean = block.clone()
            block.fill_(fill)
            one = 8 * r.layer.head_dim
            cols1 = 256 if kind == "sliding" else 128
            for j in range((n - 1) % 16 + 1):            # put the sequence's own keys back
                for at, size in key_bytes(r.layer.head_dim, cols1, one, j):
                    block[:, at:at + size] = clean[:, at:at + size]
        s = Step4(r)
        s.run()
        status_ok()
        group = r.layer.n_q_heads // r.layer.n_kv_heads
        bad = torch.isnan(s.out).all(-1)
        assert torch.equal(bad, torch.isnan(s.out).any(-1))
        want = torch.zeros_like(bad)
        want[0, group:3 * group] = True
        if kind == "global":
            want[1, :group] = True
        assert torch.equal(bad, want)


def key_bytes(d, cols1, one, j):
    """(offset, length) of every run of bytes that belongs to key j of a page-head block."""
    runs = [(sg * 2048 + j * 128, 128) for sg in range(d // 256)]
    runs += [(one + j * 64, 64)] if cols1 == 128 else [(one + j * 128, 128)]
    s0 = one + 8 * cols1
    return runs + [(s0 + j * d // 32, d // 32), (s0 + 16 * d // 32 + j * cols1 // 32, cols1 // 32),
                   (s0 + 16 * (d + cols1) // 32 + j, 1)]


def test_decode_pool_past_4_gib():
    """Page blocks beyond 2^32 bytes of the pool."""
    layer, _ = make_layers("global")
    num = (2 ** 32) // (4 * 5456) + 50
    r = Rows4("global", [100], seed=33, gap=0)
    r.fill()
    big = PagedKV4(layer, num, fill=None)
    table = r.table + (num - r.plan.num_pages)
    big.pages[num - r.plan.num_pages:] = r.cache.pages
    s = Step4(r)
    s.run()
    out = torch.empty_like(s.out)
    g4.g4attn_kv4_decode(layer, None, s.q, None, None, i32([100]), big.desc, table, out, s.ws)
    status_ok()
    assert torch.equal(out, s.out)
    g4.g4attn_kv4_append(layer, None, r.k[0].cuda(), None, i32([0]), i32([100]), i32([0]), big.desc, table)
    status_ok()
    held = r.table[0].long()
    assert torch.equal(big.pages[num - r.plan.num_pages:][held][:-1], r.cache.pages[held][:-1])


def test_decode_wait_that_runs_out_is_reported_and_the_next_call_is_exact():
    """Enough requests that the page copies queue up behind one another and some first poll fails. (A global step's
    warps take longer over a page than its copy does: with 96 requests of 8192 keys no poll failed there. The
    code is the same.)"""
    kind, B, length = "sliding", 96, 1024
    layer, _ = make_layers(kind)
    width = length // 16
    cache = PagedKV4(layer, B * width, fill=None)
    cache.pages.random_(110, 130)                     # scales too: around 1
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    q = gi.bf16_normal((B, 32, layer.head_dim), 3).cuda()
    ws = workspace(layer, B, width)

    def run():
        out = torch.full_like(q, float("nan"))
        g4.g4attn_kv4_decode(layer, None, q, None, None, i32([length] * B), cache.desc, table, out, ws)
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


@pytest.mark.parametrize("kind,window", [("global", 0), ("sliding", 262144)])
def test_decode_longest_context(kind, window):
    """262144 keys, the last usable position, against fp64 on the device. Beyond the tolerance above: the
    sums run over 2^18 keys, in runs of 8 or 16 pages per warp and 256 or 2048 chunks (in four sums), each addition off by at
    most 2^-24 of a partial sum that is at most sum p |v|: under 2^-15 of it in all."""
    layer = g4.global_layer() if kind == "global" else g4.sliding_layer(window)
    hkv, d, n = layer.n_kv_heads, layer.head_dim, 262144
    cache = PagedKV4(layer, n // 16, fill=None)
    g = torch.Generator(device="cuda").manual_seed(5)
    cols = d + (256 if kind == "sliding" else 128)
    cache.pages.random_(0, 256, generator=g)                                    # any codes
    scales = cache.pages[..., 8 * cols:-16]
    scales.random_(124, 127, generator=g)                                       # units 2^-3 .. 2^-1
    per = d // 32
    value = scales[..., (16 * per if kind == "sliding" else 0):][..., :16 * per]
    cache.pages[..., -16:] = value.unflatten(-1, (16, per)).amax(-1)
    table = torch.randperm(n // 16, generator=g, device="cuda").int()[None].contiguous()
    q = gi.bf16_normal((1, 32, d), 9).cuda()
    out = torch.empty_like(q)
    w = torch.zeros(table.shape, device="cuda") if kind == "global" else None
    g4.g4attn_kv4_decode(layer, None, q, None, None, i32([n]), cache.desc, table, out,
                         workspace(layer, 1, n // 16, kind == "global"), page_weights=w)
    status_ok()
    olayer = oracle.GLOBAL if kind == "global" else oracle.SLIDING
    turned, steps = turned_queries(olayer, q, [n - 1])
    roped = torch.tensor(turned[0], device="cuda")
    one, two = (x[table[0].long()].transpose(1, 2).flatten(0, 1).double() for x in untile4(cache.pages, d))
    turned_cols = torch.tensor(kv8.turned_columns(olayer), device="cuda")
    pages, most = torch.zeros(n // 16, dtype=torch.float64, device="cuda"), 0.0
    group = 32 // hkv
    for h in range(hkv):
        k, v = one[:, h], (one if kind == "global" else two)[:, h]
        if kind == "global":
            k = k.clone()
            k[:, turned_cols] = two[:, h]
        rows = slice(group * h, group * (h + 1))
        p = torch.softmax(roped[rows] @ k.T * layer.softmax_scale, -1)
        want, mag = p @ v, p @ v.abs()
        peak = n * (p * v.abs().amax(-1)).amax(-1, keepdim=True)
        more = torch.tensor(border(steps[0, rows], k.abs().amax(0)[None, None].cpu().numpy(), layer.softmax_scale),
                            device="cuda")
        most = max(most, float(more.max()))
        over = (out[0, rows].double() - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -14 + more) * mag
                                                       + 2.0 ** -30 * peak)
        assert (over <= 0).all(), float(over.max())
        pages += p.sum(0).unflatten(0, (-1, 16)).sum(-1)
    if w is not None:
        assert torch.allclose(w[0].double(), pages, rtol=2e-5 + most, atol=1e-9)


# ---- prefill ------------------------------------------------------------------------------------------

def prefill(r, norms=None, span=None):
    n = None if norms is None else norms.arg
    r.append_history(n)
    scratch = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, r.kind == "global")
    q = r.pack(r.q)
    out = torch.full_like(q, 5.0)
    g4.g4attn_kv4_prefill(r.layer, n, q, r.pack(r.k), None if r.v is None else r.pack(r.v), *r.row_args(), r.cache.desc,
                          r.table, scratch.desc, r.table, out, span=span)
    status_ok()
    return q, out, scratch


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_prefill_is_the_attention_over_the_stored_values(kind):
    r = Rows4(kind, [96, 1, 200, 0, 300], [0, 40, 17, 5, 1500], seed=41)
    q, out, _ = prefill(r)
    k, two = bf16_pages(r.layer, r.cache.pages)      # the same attention kernel on bf16 pages made from the bytes
    other = PagedKV(r.plan.num_pages, r.layer.n_kv_heads, r.layer.head_dim, kind == "global")
    second = other.k_rot if kind == "global" else other.v
    other.k.copy_(k.reshape(other.k.shape))
    second.copy_(two.reshape(second.shape))
    ref = torch.full_like(q, 5.0)
    g4.g4attn_prefill_attend(r.layer, q, *r.row_args(), other.desc, r.table, ref)
    status_ok()
    assert torch.equal(out, ref) and torch.isfinite(out).all()
    for b in (0, 2):   # and near the definition: the library's own bar for the bf16 cache
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
    whole = Rows4(kind, [1300], seed=42, gap=0)
    _, ref, _ = prefill(whole, norms)
    cut = Rows4(kind, [1300], seed=42, gap=0)
    scratch = PagedKV(cut.plan.num_pages, cut.layer.n_kv_heads, cut.layer.head_dim, kind == "global")
    got = torch.empty_like(ref)
    for lo, hi in ((0, 5), (5, 640), (640, 641), (641, 1300)):
        q, k = cut.q[0][lo:hi].cuda(), cut.k[0][lo:hi].cuda()
        v = None if cut.v is None else cut.v[0][lo:hi].cuda()
        got[lo:hi] = g4.g4attn_kv4_prefill(cut.layer, None if norms is None else norms.arg, q, k, v, i32([0]),
                                           i32([hi - lo]), i32([lo]), cut.cache.desc, cut.table, scratch.desc, cut.table,
                                           torch.empty_like(q))
    status_ok()
    assert torch.equal(cut.cache.pages, whole.cache.pages)
    assert torch.equal(got, ref)


def test_prefill_with_image_spans_and_a_refused_sequence():
    r = Rows4("sliding", [150, 90, 60], [60, 70, 0], seed=45, gap=1, window=16)
    span = torch.zeros(r.T, 2, dtype=torch.int32)
    images = [(5, 140), (33, 71)]                                # begun before the chunk's window does
    for b, (s0, s1) in enumerate(images):
        span[r.start[b]:r.start[b] + s1 - r.ctx[b]] = torch.tensor([s0, s1], dtype=torch.int32)
    q, out, scratch = prefill(r, span=span.cuda())
    group = r.layer.n_q_heads // r.layer.n_kv_heads
    for b in range(2):
        n, c = r.rows[b], r.ctx[b]
        kk, vv = kv8.keys_values(r.olayer, *r.values(b))
        roped = f64(g4.g4attn_rope_apply(r.layer, r.q[b].cuda(), i32(list(range(c, c + n)))))
        want = oracle.attention(roped[:, 5], kk[:, 5 // group], vv[:, 5 // group], np.arange(c, c + n), np.arange(c + n),
                                16, r.layer.softmax_scale, [images[b]])
        err = np.abs(f64(out[r.start[b]:r.start[b] + n, 5]) - want)
        assert err.max() <= 2e-2 and err.mean() <= 2e-3
    again = torch.full_like(q, 5.0)
    g4.g4attn_kv4_prefill(r.layer, None, q, r.pack(r.k), r.pack(r.v), i32([r.T - 9, *r.start[1:]]), i32(r.rows),
                          i32(r.ctx), r.cache.desc, r.table, scratch.desc, r.table, again, span=span.cuda())
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    assert torch.equal(again[r.start[1]:], out[r.start[1]:]) and (again[:r.start[1]] == 5.0).all()


# ---- streams, graphs and two calls at once ----------------------------------------------------------------

def test_two_calls_at_once():
    r = Rows4("global", [700, 1500, 40], seed=73, gap=0)
    r.fill()
    want = []
    for seed in (1, 2):
        s = Step4(r, seed=seed, weights=True)
        for _ in range(20):
            s.run()
        status_ok()
        want.append((s.out.clone(), s.weights.clone()))
    steps = [Step4(r, seed=seed, weights=True) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    lens = i32(steps[0].lens)
    for _ in range(20):
        for s, st in zip(steps, streams):
            g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, lens, r.cache.desc, r.table, s.out, s.ws,
                                 page_weights=s.weights, stream=st)
    for st in streams:
        assert g4.g4attn_status_sync(st) == g4.G4_OK
    for s, (out, w) in zip(steps, want):
        assert torch.equal(s.out, out) and torch.equal(s.weights, w)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_two_captured_steps_share_a_workspace(kind):
    """Replayed in order on another stream; the lengths change in place."""
    r = Rows4(kind, [300, 1100, 40], seed=61, gap=0)
    r.fill()
    a, b = Step4(r, seed=1), Step4(r, seed=2)
    ws, lens, stream, graphs = torch.empty_like(a.ws), i32(a.lens), torch.cuda.Stream(), []
    torch.cuda.synchronize()

    def call(s, ws):
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, lens, r.cache.desc, r.table, s.out, ws)
    with torch.cuda.stream(stream):
        for s in (a, b):
            call(s, ws)
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call(s, ws)
            graphs.append(g)
    for less in (0, 7):
        lens.sub_(less)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, seed in ((a, 1), (b, 2)):
            want = Step4(r, seed=seed)
            call(want, want.ws)
            status_ok()
            assert torch.equal(s.out, want.out)


def test_wrong_device_and_strides_are_refused():
    r = Rows4("global", [40], seed=74, gap=0)
    r.fill()
    s = Step4(r)
    with pytest.raises(ValueError, match="current CUDA device"):
        g4.g4attn_kv4_decode(r.layer, None, s.q.cpu(), None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws)
    with pytest.raises(ValueError, match="strided"):
        g4.g4attn_kv4_decode(r.layer, None, torch.cat([s.q, s.q], -1)[..., ::2], None, None, i32([40]), r.cache.desc,
                             r.table, s.out, s.ws)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws.cpu())
    with pytest.raises(g4.G4Error):
        g4.g4attn_kv4_decode(r.layer, None, s.q, None, None, i32([40]), r.cache.desc, r.table, s.out, s.ws[:64])


@pytest.mark.parametrize("power", [8, 12, 20, 24, 26, 32, 40])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_beside_one_key_with_one_large_block(kind, power):
    """A key with a block 2^power larger than all others and zeros elsewhere: what the other blocks' columns keep. The
    limit is the header's, for each of n keys: 2^-31 of the row's largest p 2^E times a code of at most 6, where the
    largest |v| of a key is at least 4 * 2^E. Up to 2^16 every weight, p within 2 of the largest and a block of 32 normal
    numbers within 2^3 of another, is at least 2^-20 of that largest, and only its cast is left (2^-11 of each)."""
    r = Rows4(kind, [300, 1500], seed=35, gap=0)
    for x in (r.v if kind == "sliding" else r.k):
        x[7] = 0
        x[7, :, 128:160] = (r.q[0][0, 0, :32].double() * 2.0 ** power).bfloat16()
    r.fill()
    s = Step4(r, q_scale=2.0 ** -12)                     # scores next to 0: all weights alike
    s.q[..., 128:160] = 0                                # (a global key is its value too)
    s.run()
    status_ok()
    q, steps = turned_queries(r.olayer, s.q, s.pos)
    scale, got = r.layer.softmax_scale, f64(s.out)
    others = np.setdiff1d(np.arange(r.layer.head_dim), np.arange(128, 160))
    for b, n in enumerate(s.lens):
        k, v = kv8.keys_values(r.olayer, *r.values(b))
        lo = max(0, n - r.layer.window) if kind == "sliding" else 0
        want, p, mag, peak = kv8.decode(q[b], k, v, scale, lo)
        assert p[:, lo:].min() * 2 > p.max()
        seen = lo <= 7
        lost = 1.5 * 2.0 ** -31 * peak if seen and power > 16 else 0
        limit = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16 + border(steps[b], k, scale)) * mag + lost
        if seen and 16 < power < 25:                     # the limit says something in these columns
            assert np.median(limit[:, others]) < np.median(mag[:, others])
        over = np.abs(got[b] - want) - limit
        assert (over <= 0).all(), (b, over.max())


def normed_turned_queries(r, q, pos):
    """Normed queries as the definition casts and turns them, in fp64, and per column the step to the neighbour it may be
    instead. Before the first cast the kernel's fp32 x is off by at most 2^-20 of itself (a sum of 512 squares over 32
    lanes, half of whose 21 roundings the root keeps, then the root, a quotient and two products); a column next to a
    border of that cast moves its pair's turned columns by a step too, and plain columns are turned by nothing."""
    norms = r.norms.oracle
    x = oracle.normed_q(norms, q.double().cpu().numpy())
    d, turned = x.shape[-1], kv8.turned_columns(r.olayer)
    plain = np.setdiff1d(np.arange(d), turned)
    if r.kind == "global":
        x[..., plain] *= norms.k_weight[plain]
    cast = lambda v: f64(torch.tensor(v).bfloat16())   # noqa: E731
    near, mid = 2.0 ** -20 * np.abs(x), cast(x)
    step = cast(x + near) - cast(x - near)
    y = oracle.rope(mid, np.asarray(pos)[:, None], r.olayer.rope_theta, r.olayer.rope_partial)
    half = d // 2
    pair = 2.0 ** -22 * (np.abs(mid[..., :half]) + np.abs(mid[..., half:])) + step[..., :half] + step[..., half:]
    near = np.where(np.isin(np.arange(d), turned), np.concatenate([pair, pair], -1), step)
    out = cast(y)
    return out, np.maximum(cast(y + near) - out, out - cast(y - near))


@pytest.mark.parametrize("kind,tp", [("sliding", 1), ("sliding", 8), ("global", 1), ("global", 4)])
def test_decode_normed_against_fp64(kind, tp):
    """Lengths within and beyond the window, page weights on global layers; a row's tolerance grows only by the columns of
    its query that lie next to a border between two bf16 numbers."""
    r = Rows4(kind, [45, 600, 1500, 2300], seed=36, gap=0, tp=tp, norms=Norms(kind, 9))
    r.fill()
    s = Step4(r, weights=kind == "global")
    s.run()
    status_ok()
    q, steps = normed_turned_queries(r, s.q, s.pos)
    scale, got, slack = r.layer.softmax_scale, f64(s.out), []
    for b, n in enumerate(s.lens):
        k, v = kv8.keys_values(r.olayer, *r.values(b))
        lo = max(0, n - r.layer.window) if kind == "sliding" else 0
        want, p, mag, peak = kv8.decode(q[b], k, v, scale, lo)
        more = border(steps[b], k, scale)
        assert_row(got[b], want, mag, peak, more)
        slack += list(more[:, 0])
        if s.weights is not None:
            w, sums = f64(s.weights[b]), kv8.page_sums(p)
            assert np.allclose(w[:len(sums)], sums, rtol=2e-5 + more.max(), atol=1e-9), b
            assert (w[len(sums):] == 0).all()
    assert np.median(slack) < 2.0 ** -9                  # half of the heads are held to the roundings alone


@pytest.mark.parametrize("lens", [[300, 40], [2300, 40, 1025]])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_decode_into_its_queries(kind, lens):
    """out is q: the bits of a call with an output of its own, with one chunk and with several."""
    r = Rows4(kind, lens, seed=37, gap=0, norms=Norms(kind, 6))
    r.fill()
    s = Step4(r, weights=kind == "global")
    s.run()
    status_ok()
    both, weights = s.q.clone(), None if s.weights is None else torch.zeros_like(s.weights)
    g4.g4attn_kv4_decode(r.layer, r.norms.arg, both, None, None, i32(s.lens), r.cache.desc, r.table, both, s.ws,
                         page_weights=weights)
    status_ok()
    assert torch.equal(both, s.out) and (weights is None or torch.equal(weights, s.weights))
    both = s.q.clone()
    g4.g4attn_kv4_decode(r.layer, r.norms.arg, both, None, None, i32(s.lens), r.cache.desc, r.table, both, s.ws)
    status_ok()
    assert torch.equal(both, s.out)
