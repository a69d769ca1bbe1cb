"""Promises of the header that the 8-bit cache's calls share with the bf16 ones, held to the bit."""
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
