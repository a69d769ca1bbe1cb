"""The page plan on the GPU, against its plain definition (oracle/plan.py): whole numbers, equal to the last one; and a
serving loop that runs on it: prefill, decode and eviction over a 4-bit cache of both layer kinds."""
import copy
import random

import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
import oracle
from invariant_hybrid_attention_gb300 import inputs as gi
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV4, device_int32, untile4
from oracle import kv8
from oracle import plan as oplan

from gpu_cases import f64
from test_gpu_kv4 import assert_row, workspace
from test_gpu_kv8 import border, make_layers, status_ok, turned_queries

pytestmark = pytest.mark.gpu
i32 = device_int32


class Plan:
    """A step's state on both sides. ctx, new: of each request; windows: a group each (0: may evict)."""

    def __init__(self, ctx, new, rows, windows=(0, 1024), spare=0, evicted=False, seed=0, width=None):
        r = random.Random(seed)
        self.ctx, self.new, self.rows, self.groups = list(ctx), list(new), rows, []
        for w in windows:
            lost = [0] * len(ctx)
            if w == 0 and evicted:
                lost = [16 * r.randint(0, max(0, c - 1) // 32) for c in ctx]
            freed = [min(3, x // 16) for x in lost]
            held = [c - x for c, x in zip(ctx, lost)]
            first = [max(0, h - w) // 16 if w else 0 for h in held]
            cols = width or max(1, max(oplan.pages(h + max(0, x)) for h, x in zip(held, new)))
            total = sum(oplan.pages(h) - f for h, f in zip(held, first)) + sum(freed) + spare
            order = list(range(total))
            r.shuffle(order)
            table = [[-1] * cols for _ in ctx]
            for b, h in enumerate(held):
                for i in range(first[b], oplan.pages(h)):
                    table[b][i] = order.pop()
            gone = [[order.pop() for _ in range(f)] for f in freed]
            total = max(1, total)
            head = r.randrange(total)
            ring = [-7] * total
            for i, page in enumerate(order):
                ring[(head + i) % total] = page
            self.groups.append(dict(window=w, num_pages=total, table=table, ring=ring, pool=[head, len(order)],
                                    first=first if w else None, lost=[x - 16 * f for x, f in zip(lost, freed)] if not w else None,
                                    freed=gone if evicted and not w else None))

    def device(self, in_place=False):
        n = len(self.ctx)
        z = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")   # noqa: E731
        d = dict(ctx=i32(self.ctx), new=i32(self.new), q_start=z(n), q_len=z(n), ctx_start=z(n), pos=z(self.rows), groups=[])
        d["out_ctx"] = d["ctx"] if in_place else z(n)
        for g in self.groups:
            x = dict(table=i32(g["table"]), ring=i32(g["ring"]), pool=i32(g["pool"]), seq=z(n),
                     slots=torch.full((self.rows,), -99, dtype=torch.int64, device="cuda"), first=None, lost=None, freed=None,
                     n_freed=None)
            for name in ("first", "lost"):
                if g[name] is not None:
                    x[name] = i32(g[name])
            if g["freed"] is not None:
                x["freed"] = torch.full_like(x["table"], -1)
                for b, f in enumerate(g["freed"]):
                    x["freed"][b, :len(f)] = i32(f)
                x["n_freed"] = i32([len(f) for f in g["freed"]])
            for name in ("pool", "first", "lost"):
                x["out_" + name] = None if x[name] is None else x[name] if in_place else torch.full_like(x[name], -99)
            x["group"] = g4.make_page_group(g["window"], x["table"], x["ring"], x["pool"], x["out_pool"], x["seq"],
                                            x["slots"], first_page=x["first"], out_first_page=x["out_first"],
                                            lost=x["lost"], out_lost=x["out_lost"], freed=x["freed"], n_freed=x["n_freed"])
            d["groups"].append(x)
        return d

    @staticmethod
    def call(d):
        g4.g4attn_plan_pages(d["ctx"], d["new"], [x["group"] for x in d["groups"]], d["out_ctx"], d["q_start"], d["q_len"],
                             d["ctx_start"], d["pos"])

    def check(self, d):
        groups = copy.deepcopy(self.groups)
        after, start, length, pos, seq, slots = oplan.plan(self.ctx, self.new, self.rows, groups)
        assert d["out_ctx"].tolist() == after and d["q_start"].tolist() == start and d["q_len"].tolist() == length
        assert d["ctx_start"].tolist() == self.ctx and d["pos"].tolist() == pos
        for x, g, s, sl in zip(d["groups"], groups, seq, slots):
            assert x["table"].tolist() == g["table"] and x["ring"].tolist() == g["ring"]
            assert x["out_pool"].tolist() == g["pool"] and x["seq"].tolist() == s and x["slots"].tolist() == sl
            if g["first"] is not None:
                assert x["out_first"].tolist() == g["first"]
            if g["lost"] is not None:
                assert x["out_lost"].tolist() == g["lost"]
        return length


def run(plan, in_place=False):
    d = plan.device(in_place)
    plan.call(d)
    status_ok()
    return plan.check(d)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n", [1, 7, 256, 257, 1500])
def test_plan_matches_the_definition(n, seed, in_place):
    r = random.Random(100 * n + seed)
    top = r.choice([40, 700, 3000])
    ctx = [r.choice([0, 1, 15, 16, 17, 1023, 1024, 1025, r.randint(0, top), r.randint(0, top)]) for _ in range(n)]
    new = [r.choice([-1, 0, 1, 1, 1, 1, 16, 17, r.randint(1, 300)]) for _ in range(n)]
    rows = sum(max(0, x) for x in new)
    need = sum(oplan.pages(c + max(0, x)) - oplan.pages(c) for c, x in zip(ctx, new))
    spare = r.choice([0, need // 2, need, 2 * need + 3])
    rows = max(0, rows + r.choice([0, 5, -rows // 3]))
    windows = r.choice([(0,), (1024,), (0, 1024), (16, 0), (1, 50)])
    served = run(Plan(ctx, new, rows, windows, spare, evicted=r.random() < 0.5, seed=seed), in_place)
    if n > 7 and spare >= need and rows >= sum(max(0, x) for x in new):
        assert served == [max(0, x) for x in new]


def test_plan_of_the_largest_batch_and_the_longest_request():
    r = random.Random(5)
    ctx = [r.randint(0, 500) for _ in range(4096)]
    new = [r.choice([-1, 0, 1, 1, 1, 40]) for _ in range(4096)]
    run(Plan(ctx, new, sum(max(0, x) for x in new) + 3, spare=9000, evicted=True, seed=3))
    run(Plan([262144 - 5, 0, 262144], [5, 262144, -1], 262149, windows=(0, 1024), spare=17000))


def test_a_request_that_does_not_fit_holds_its_place_in_the_line():
    """Pages are counted in the requests' order whether served or not; who needs no page does not wait."""
    p = Plan([0, 16, 5, 32, 0], [48, 1, 1, 1, 16], 100, windows=(0,), spare=4)
    assert run(p) == [48, 1, 1, 0, 0]             # 3 pages, 1, none, 1 too many, another
    p = Plan([0, 16, 5, 32, 0], [80, 1, 1, 1, 16], 100, windows=(0,), spare=4)
    assert run(p) == [0, 0, 1, 0, 0]
    p = Plan([3, 3, 3, 3], [5, 6, 4, 1], 11, windows=(0,), spare=4)
    assert run(p) == [5, 6, 0, 0]                 # rows past T
    p = Plan([3, 3], [1, 1], 0, windows=(0,), spare=4)
    assert run(p) == [0, 0]


def refused(plan, change, requests):
    """The call with `change` made to the device state: requests are not served and keep their state; the rest as ever."""
    d = plan.device()
    change(d)
    before = {k: d[k].clone() for k in ("ctx", "new")}
    firsts = [(None if x["first"] is None else x["first"].clone(), None if x["lost"] is None else x["lost"].clone())
              for x in d["groups"]]
    plan.call(d)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    for b in requests:
        assert int(d["q_len"][b]) == 0 and int(d["out_ctx"][b]) == int(before["ctx"][b])
        for x, (first, lost) in zip(d["groups"], firsts):
            assert int(x["seq"][b]) == 0
            assert first is None or int(x["out_first"][b]) == int(first[b])
            assert lost is None or int(x["out_lost"][b]) == int(lost[b])
    return d


def test_bad_requests_are_left_as_they_are():
    def plan(**kw):
        return Plan([20, 40, 60, 80], [1, 1, 1, 1], 8, windows=(0, 32), spare=9, seed=1, **kw)

    def set_(name, b, value, group=None):
        def change(d):
            (d if group is None else d["groups"][group])[name][b] = value
        return change
    for change in (set_("ctx", 1, -1), set_("ctx", 1, 262144), set_("ctx", 1, 2 ** 31 - 1), set_("new", 1, -2),
                   set_("new", 1, 262145), set_("new", 1, 2 ** 31 - 1), set_("new", 1, 16 * 6), set_("first", 1, -1, 1),
                   set_("first", 1, 4, 1), set_("lost", 1, -16, 0), set_("lost", 1, 41, 0)):
        d = refused(plan(), change, [1])
        # (96 refused rows keep their place: those of the requests behind them end past T = 8)
        past = int(d["new"][1]) == 96
        assert [int(d["q_len"][b]) for b in (0, 2, 3)] == [1, 0 if past else 1, 0 if past else 1]
    e = Plan([200, 400, 60, 80], [1, 1, 1, 1], 8, windows=(0, 32), spare=9, seed=2, evicted=True)
    for value in (-1, 14, 2 ** 31 - 1):
        # (14 pages are within the table and the 400 tokens: the request is served, and the pages behind its freed
        # ones, -1, are passed on and reported)
        d = refused(e, set_("n_freed", 1, value, 0), [] if value == 14 else [1])
        assert [int(d["q_len"][b]) for b in range(4)] == [1, 1 if value == 14 else 0, 1, 1]


def test_a_pool_that_contradicts_itself_gives_and_takes_nothing():
    for pool in ([-1, 3], [10 ** 9, 3], [0, -1], [0, 10 ** 9]):
        p = Plan([16, 40, 32], [1, 1, -1], 8, windows=(0, 32), spare=4, seed=1)
        d = p.device()
        d["groups"][0]["pool"].copy_(i32(pool))
        ring = d["groups"][0]["ring"].clone()
        p.call(d)
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
        assert d["q_len"].tolist() == [0, 1, 0]            # the first needs a page
        assert d["groups"][0]["out_pool"].tolist() == pool and torch.equal(d["groups"][0]["ring"], ring)
    p = Plan([16, 40, 32], [1, 1, -1], 8, windows=(0,), spare=4, seed=1)
    d = p.device()
    n = p.groups[0]["num_pages"]
    d["groups"][0]["pool"].copy_(i32([0, n - 1]))          # no room for the two pages of the request that ended
    p.call(d)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    assert d["groups"][0]["out_pool"].tolist() == [1, n - 2]


def test_pages_outside_the_pool_are_reported():
    p = Plan([20, 40], [1, 1], 4, windows=(0,), spare=3, seed=1)
    d = p.device()
    d["groups"][0]["table"][1, 2] = 10 ** 6
    p.call(d)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    assert int(d["groups"][0]["slots"][1]) == -1 and int(d["groups"][0]["slots"][0]) >= 0


def test_slots_past_32_bits():
    """Physical pages from 2^27 on: their slots pass 2^31."""
    n = (1 << 27) + 100
    ring = torch.zeros(n, dtype=torch.int32, device="cuda")
    ring[5] = n - 1
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    table, pool = z(1, 4), i32([5, 1])
    group = g4.make_page_group(0, table, ring, pool, pool, z(1), slots)
    g4.g4attn_plan_pages(z(1), i32([3]), [group], z(1), z(1), z(1), z(1), z(3))
    status_ok()
    assert slots.tolist() == [16 * (n - 1) + i for i in range(3)] and int(table[0, 0]) == n - 1
    assert pool.tolist() == [6, 0]


def test_outputs_over_the_inputs_and_groups_without_slots():
    p = Plan([20, 40, 0, 70], [1, 30, 5, -1], 40, windows=(0, 32), spare=9, seed=6)
    want = p.device()
    p.call(want)
    d = p.device(in_place=True)
    for x in d["groups"]:
        t = x["group"].tensors
        x["group"] = g4.make_page_group(x["group"].window, t["page_table"], t["free_pages"], t["pool"], t["out_pool"],
                                        t["seq_len"], None, **{k: t[k] for k in ("first_page", "out_first_page", "lost",
                                                                                 "out_lost", "freed", "n_freed")})
    g4.g4attn_plan_pages(d["ctx"], d["new"], [x["group"] for x in d["groups"]], d["ctx"], d["q_start"], d["new"],
                         d["ctx_start"], d["pos"])
    status_ok()
    assert torch.equal(d["ctx"], want["out_ctx"]) and torch.equal(d["new"], want["q_len"])
    assert torch.equal(d["pos"], want["pos"]) and torch.equal(d["ctx_start"], want["ctx_start"])
    for x, y in zip(d["groups"], want["groups"]):
        assert torch.equal(x["table"], y["table"]) and torch.equal(x["ring"], y["ring"])
        assert torch.equal(x["pool"], y["out_pool"]) and (x["slots"] == -99).all()


def test_two_plans_at_once():
    """Of two batches, on two streams, with states of their own."""
    plans = [Plan([20 + i, 400, 0, 70] * 80, [1, 30, 5, -1] * 80, 4000, spare=500, seed=i) for i in (1, 2)]
    states, streams = [p.device() for p in plans], [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, d, stream in zip(plans, states, streams):
            with torch.cuda.stream(stream):
                p.call(d)
    status_ok()
    for p, d in zip(plans, states):
        p.check(d)


def test_groups_of_other_sizes_are_refused():
    p = Plan([20, 40], [1, 1], 4)
    d, other = p.device(), Plan([20, 40, 1], [1, 1, 1], 4).device()
    d["groups"][1] = other["groups"][1]
    with pytest.raises(ValueError, match="a group of 3 requests"):
        p.call(d)


def test_a_captured_step_replays_over_its_own_state():
    """In place, captured once: every replay plans the step after the last one's."""
    n, width = 6, 40
    p = Plan([0, 3, 15, 30, 100, 250], [7, 1, 1, 1, 1, 1], 12, windows=(0, 32), spare=60, width=width, seed=4)
    d = p.device(in_place=True)
    first = p.device(in_place=True)
    p.call(first)                                           # the library's first call comes before any capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        p.call(d)
    for _ in range(30):
        graph.replay()
        torch.cuda.synchronize()
        assert g4.g4attn_status_sync() == g4.G4_OK
        p.check(d)
        groups = copy.deepcopy(p.groups)
        p.ctx, *_ = oplan.plan(p.ctx, p.new, p.rows, groups)
        p.groups = groups
    assert p.ctx == [210, 33, 45, 60, 130, 280] and all(x >= 0 for x in p.ctx)


# ---- together: a serving loop --------------------------------------------------------------------------

@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_loop_of_plan_prefill_decode_and_eviction(captured):
    """Three request slots of a hybrid model with one layer of each kind over 4-bit caches. Prompts are planned and
    prefilled, decode steps planned and run with page weights, the global table trimmed and its pages returned; a request
    ends and another takes its slot, another waits for pages. Every decode row is checked in fp64 over the keys that the
    request must hold by then (captured: the decode step is one graph, from plan to eviction)."""
    window, n, width = 64, 3, 24
    layers = {k: make_layers(k, window) for k in ("global", "sliding")}
    pools = {"global": 22, "sliding": 20}
    cache = {k: PagedKV4(layers[k][0], pools[k]) for k in pools}
    scratch = {k: PagedKV(pools[k], layers[k][0].n_kv_heads, layers[k][0].head_dim, k == "global") for k in pools}
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    table = {k: torch.full((n, width), -1, dtype=torch.int32, device="cuda") for k in pools}
    ring = {k: torch.randperm(pools[k], device="cuda").int() for k in pools}
    pool = {k: i32([0, pools[k]]) for k in pools}
    first, lost, freed, n_freed = z(n), z(n), z(n, width), z(n)
    seq = {k: z(n) for k in pools}
    ctx, new = z(n), z(n)
    weights = torch.zeros(n, width, device="cuda")
    ws = {k: workspace(layers[k][0], n, width, k == "global") for k in pools}

    def groups(rows, slots):
        return [g4.make_page_group(0, table["global"], ring["global"], pool["global"], pool["global"], seq["global"],
                                   slots["global"], lost=lost, out_lost=lost, freed=freed, n_freed=n_freed),
                g4.make_page_group(window, table["sliding"], ring["sliding"], pool["sliding"], pool["sliding"],
                                   seq["sliding"], slots["sliding"], first_page=first, out_first_page=first)]

    def buffers(rows):
        slots = {k: z(rows, t=torch.int64) for k in pools}
        return dict(pos=z(rows), start=z(n), len=z(n), ctx=z(n), slots=slots, groups=groups(rows, slots))

    def plan(x):
        g4.g4attn_plan_pages(ctx, new, x["groups"], ctx, x["start"], x["len"], x["ctx"], x["pos"])
        n_freed.zero_()

    held = [None] * n                                        # per request: {kind: [stored values of its keys]}, positions

    def read_back(kind, b, slots):
        """The stored values of the keys at these slots, fp64."""
        one, two = untile4(cache[kind].pages, layers[kind][0].head_dim)
        return [v[slots // 16, :, slots % 16].double().cpu().numpy() for v in (one, two)]

    rng = random.Random(3)

    def prompts(lengths, seed):
        """Plans and prefills prompts; returns who was served."""
        rows = sum(max(0, v) for v in lengths) + 2
        new.copy_(i32(lengths))
        x = buffers(rows)
        plan(x)
        status_ok()
        served = x["len"].tolist()
        for k in pools:
            layer = layers[k][0]
            kv = lambda s: gi.bf16_normal((rows, layer.n_kv_heads, layer.head_dim), s).cuda()   # noqa: E731
            q = gi.bf16_normal((rows, 32, layer.head_dim), seed + 5).cuda()
            out = torch.full_like(q, 5.0)
            g4.g4attn_kv4_prefill(layer, None, q, kv(seed), kv(seed + 1) if k == "sliding" else None, x["start"], x["len"],
                                  x["ctx"], cache[k].desc, table[k], scratch[k].desc, table[k], out)
            status_ok()
            live = (x["pos"] >= 0)[:, None, None]
            assert torch.equal(out == 5.0, ~live.expand_as(out)) and torch.isfinite(out).all()
            for b in range(n):
                if lengths[b] < 0:
                    held[b] = None
                if served[b]:
                    s = x["slots"][k][int(x["start"][b]):int(x["start"][b]) + served[b]]
                    held[b] = held[b] or {}
                    held[b][k] = read_back(k, b, s)
        return served

    step_in = {k: dict(q=z(n, 32, layers[k][0].head_dim, t=torch.bfloat16),
                       k=z(n, layers[k][0].n_kv_heads, layers[k][0].head_dim, t=torch.bfloat16),
                       v=z(n, layers[k][0].n_kv_heads, layers[k][0].head_dim, t=torch.bfloat16) if k == "sliding" else None,
                       out=z(n, 32, layers[k][0].head_dim, t=torch.bfloat16)) for k in pools}
    one_row = buffers(n)
    held_len, new_len = z(n), z(n)

    def decode():
        plan(one_row)
        for k in pools:
            s = step_in[k]
            g4.g4attn_kv4_decode(layers[k][0], None, s["q"], s["k"], s["v"], seq[k], cache[k].desc, table[k], s["out"], ws[k],
                                 pos=one_row["pos"].clamp(min=0) if k == "global" else None,
                                 page_weights=weights if k == "global" else None)

    def evict(keep):
        torch.sub(ctx, lost, out=held_len)
        g4.g4attn_evict_pages(held_len, table["global"], weights, keep, 1, 2, new_len, table["global"], weights, freed,
                              n_freed)

    assert prompts([100, 37, 0], 100) == [100, 37, 0]
    assert prompts([0, 0, 250], 200) == [0, 0, 0]            # 16 global pages wanted, 12 free: it waits
    stream, graph = torch.cuda.Stream(), None
    for step in range(60):
        live = [h is not None for h in held]
        new.copy_(i32([1 if v else 0 for v in live]))
        for k in pools:
            for name, t in step_in[k].items():
                if t is not None and name != "out":
                    t.copy_(gi.bf16_normal(tuple(t.shape), 1000 * step + len(name) + ord(name[0]) + (k == "global")))
        # (rows are packed: with an idle slot before a live one, rows and requests part, so idle slots come last here)
        assert live == sorted(live, reverse=True)
        if captured and step == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                decode()
        if graph is not None:
            graph.replay()
        else:
            decode()
        status_ok()
        for b in range(n):
            if not live[b]:
                assert all((step_in[k]["out"][b] == 0).all() for k in pools)
                continue
            assert int(one_row["len"][b]) == 1
            pos = int(one_row["pos"][b])
            for k in pools:
                layer, ol = layers[k]
                new_kv = read_back(k, b, one_row["slots"][k][b:b + 1])
                held[b][k] = [np.concatenate([h, x]) for h, x in zip(held[b][k], new_kv)]
                if k == "sliding":
                    held[b][k] = [h[-window:] for h in held[b][k]]
                kk, vv = kv8.keys_values(ol, *held[b][k])
                roped, steps = turned_queries(ol, step_in[k]["q"][b:b + 1], [pos])
                want, _, mag, peak = kv8.decode(roped[0], kk, vv, layer.softmax_scale)
                assert_row(f64(step_in[k]["out"][b]), want, mag, peak, border(steps[0], kk, layer.softmax_scale))
        if step in (8, 25, 40):                               # trim the global tables to five pages
            before = table["global"].cpu().tolist()
            evict(5)
            status_ok()
            after, cut = table["global"].cpu().tolist(), n_freed.tolist()
            for b in range(n):
                if held[b] is None:
                    continue
                m = held[b]["global"][0].shape[0]
                kept = after[b][:oplan.pages(m) - cut[b]]
                idx = np.concatenate([np.arange(16 * i, min(16 * i + 16, m)) for i in range(oplan.pages(m)) if before[b][i] in kept])
                held[b]["global"] = [h[idx] for h in held[b]["global"]]
        if step == 12:                                        # by now pages came back: the long prompt fits
            assert prompts([0, 0, 150], 300) == [0, 0, 150]
        if step == 30:                                        # the first request ends, another takes its slot
            assert prompts([-1, 0, 0], 400) == [0, 0, 0]
            assert int(ctx[0]) == 0 and int(lost[0]) == 0 and int(first[0]) == 0
            weights[0].zero_()
            assert prompts([60, 0, 0], 500) == [60, 0, 0]
    # nothing got lost: every page is free or held
    for k in pools:
        h, c = pool[k].tolist()
        pages = [int(ring[k][(h + i) % pools[k]]) for i in range(c)]
        for b in range(n):
            m = int(ctx[b]) - (int(lost[b]) if k == "global" else 0)
            pages += table[k][b, (int(first[b]) if k == "sliding" else 0):oplan.pages(m)].tolist()
        if k == "global":
            pages += [p for b in range(n) for p in freed[b, :int(n_freed[b])].tolist()]
        assert sorted(pages) == list(range(pools[k])), k


# ---- evictions between steps -----------------------------------------------------------------------------

def census(d, p):
    """Every physical page of the first group, from where it is: free, held, or evicted and not yet taken back."""
    x, (h, c) = d["groups"][0], d["groups"][0]["out_pool"].tolist()
    n = p.groups[0]["num_pages"]
    pages = [int(x["ring"][(h + i) % n]) for i in range(c)]
    for b, tokens in enumerate(d["out_ctx"].tolist()):
        pages += x["table"][b, :oplan.pages(tokens - int(x["out_lost"][b]))].tolist()
    return sorted(pages)


@pytest.mark.parametrize("captured", [False, True])
def test_pages_of_an_eviction_come_back_once(captured):
    """Steps without an eviction between them, in place: the first takes the evicted pages back, the others none."""
    p = Plan([200, 400, 60, 80], [1, 1, 1, 1], 6, windows=(0,), spare=12, evicted=True, seed=2, width=30)
    assert any(p.groups[0]["freed"])
    d, twin = p.device(in_place=True), p.device(in_place=True)
    p.call(twin)                                             # the library's first call comes before any capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            p.call(d)
    for _ in range(4):
        graph.replay() if captured else p.call(d)
        status_ok()
        p.check(d)
        assert d["groups"][0]["n_freed"].tolist() == [0, 0, 0, 0]
        assert census(d, p) == list(range(p.groups[0]["num_pages"]))
        groups = copy.deepcopy(p.groups)
        p.ctx, *_ = oplan.plan(p.ctx, p.new, p.rows, groups)
        groups[0]["freed"] = [[] for _ in p.ctx]
        p.groups = groups


def test_pages_of_an_eviction_that_a_step_does_not_take_stay_in_their_list():
    """Outputs apart from the inputs; a request that is refused, one that waits, one that ends."""
    p = Plan([200, 400, 160, 280], [1, 1, 300, -1], 400, windows=(0,), spare=8, evicted=True, seed=3, width=60)
    counts = [len(f) for f in p.groups[0]["freed"]]
    assert all(counts)
    d = p.device()
    x = d["groups"][0]
    p.call(d)
    status_ok()
    assert p.check(d)[2] == 0                                  # short of pages: its evicted ones come back all the same
    assert x["n_freed"].tolist() == counts and x["group"].tensors["out_n_freed"].tolist() == [0, 0, 0, 0]
    d = p.device()
    d["ctx"][1] = -1
    x = d["groups"][0]
    p.call(d)
    torch.cuda.synchronize()
    assert g4.g4attn_status_sync() == g4.G4_ERR_DEVICE
    assert x["group"].tensors["out_n_freed"].tolist() == [0, counts[1], 0, 0]
    assert int(x["out_lost"][1]) == int(x["lost"][1])


def test_a_step_of_prompts_decoding_and_idle_requests():
    """Two plans a step, one for the decoding requests and one for the prompts, as the calls that follow want them. Slot 0
    is empty at first, slot 1 decodes and loses pages to evictions, slot 2 gets its prompt in two chunks and then
    decodes, slot 3 decodes in every other step only. Every decode row against fp64 over the keys that the request must
    hold by then, at its own position."""
    window, n, width = 32, 4, 16
    kinds = ("global", "sliding")
    layers = {k: make_layers(k, window) for k in kinds}
    pools = {"global": 40, "sliding": 30}
    cache = {k: PagedKV4(layers[k][0], pools[k]) for k in kinds}
    scratch = {k: PagedKV(pools[k], layers[k][0].n_kv_heads, layers[k][0].head_dim, k == "global") for k in kinds}
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    table = {k: torch.full((n, width), -1, dtype=torch.int32, device="cuda") for k in kinds}
    ring = {k: torch.randperm(pools[k], device="cuda").int() for k in kinds}
    pool = {k: i32([0, pools[k]]) for k in kinds}
    seq = {k: z(n) for k in kinds}
    first, lost, freed, n_freed, ctx = z(n), z(n), z(n, width), z(n), z(n)
    weights = torch.zeros(n, width, device="cuda")
    ws = {k: workspace(layers[k][0], n, width, k == "global") for k in kinds}
    held, seed = [{k: None for k in kinds} for _ in range(n)], [0]

    def normal(*shape):
        seed[0] += 1
        return gi.bf16_normal(shape, seed[0]).cuda()

    def plan(new):
        rows = sum(max(0, x) for x in new)
        x = dict(pos=z(rows), start=z(n), len=z(n), ctx=z(n), slots={k: z(rows, t=torch.int64) for k in kinds})
        g = [g4.make_page_group(0, table["global"], ring["global"], pool["global"], pool["global"], seq["global"],
                                x["slots"]["global"], lost=lost, out_lost=lost, freed=freed, n_freed=n_freed),
             g4.make_page_group(window, table["sliding"], ring["sliding"], pool["sliding"], pool["sliding"],
                                seq["sliding"], x["slots"]["sliding"], first_page=first, out_first_page=first)]
        g4.g4attn_plan_pages(ctx, i32(new), g, ctx, x["start"], x["len"], x["ctx"], x["pos"])
        status_ok()
        assert x["len"].tolist() == [max(0, v) for v in new]
        return x

    def keep(k, b, slots):
        got = [v[slots // 16, :, slots % 16].double().cpu().numpy() for v in untile4(cache[k].pages, layers[k][0].head_dim)]
        old = held[b][k]
        held[b][k] = got if old is None else [np.concatenate([h, x]) for h, x in zip(old, got)]

    def kv(k, rows):
        layer = layers[k][0]
        shape = (rows, layer.n_kv_heads, layer.head_dim)
        return normal(*shape), normal(*shape) if k == "sliding" else None

    def prefill(new):
        x = plan(new)
        for k in kinds:
            layer = layers[k][0]
            q = normal(sum(max(0, v) for v in new), 32, layer.head_dim)
            g4.g4attn_kv4_prefill(layer, None, q, *kv(k, q.shape[0]), x["start"], x["len"], x["ctx"], cache[k].desc, table[k],
                                  scratch[k].desc, table[k], torch.empty_like(q))
            status_ok()
            for b in range(n):
                if new[b] > 0:
                    at = int(x["start"][b])
                    keep(k, b, x["slots"][k][at:at + new[b]])

    def decode(new):
        x = plan(new)
        for k in kinds:
            layer, ol = layers[k]
            q = normal(n, 32, layer.head_dim)
            out = torch.full_like(q, float("nan"))
            g4.g4attn_kv4_decode(layer, None, q, *kv(k, n), seq[k], cache[k].desc, table[k], out, ws[k], pos=x["ctx"] if
                                 k == "global" else None, page_weights=weights if k == "global" else None)
            status_ok()
            for b in range(n):
                if new[b] != 1:
                    assert (out[b] == 0).all()
                    continue
                at = int(x["start"][b])
                keep(k, b, x["slots"][k][at:at + 1])
                position = int(x["ctx"][b])
                assert int(x["pos"][at]) == position
                mine = [h[-window:] for h in held[b][k]] if k == "sliding" else held[b][k]
                kk, vv = kv8.keys_values(ol, *mine)
                roped, steps = turned_queries(ol, q[b:b + 1], [position])
                want, _, mag, peak = kv8.decode(roped[0], kk, vv, layer.softmax_scale)
                assert_row(f64(out[b]), want, mag, peak, border(steps[0], kk, layer.softmax_scale))

    def evict(pages):
        before, length = table["global"].tolist(), ctx - lost
        g4.g4attn_evict_pages(length, table["global"], weights, pages, 1, 1, z(n), table["global"], weights, freed, n_freed)
        status_ok()
        after, cut = table["global"].tolist(), n_freed.tolist()
        for b, m in enumerate(length.tolist()):
            if m:
                kept = after[b][:oplan.pages(m) - cut[b]]
                idx = np.concatenate([np.arange(16 * i, min(16 * i + 16, m)) for i in range(oplan.pages(m))
                                      if before[b][i] in kept])
                held[b]["global"] = [h[idx] for h in held[b]["global"]]
        return cut

    prefill([0, 100, 0, 70])
    for step in range(24):
        decode([1 if step > 15 else 0, 1, 1 if step > 10 else 0, step % 2])
        if step in (4, 10):
            prefill([0, 0, 45 if step == 4 else 20, 0])
        if step == 15:
            prefill([33, 0, 0, 0])
        if step in (6, 17):                                   # slot 3 is idle or not; it keeps its pages either way
            assert evict(4)[1] > 0
    assert int(lost[1]) > 0 and ctx.tolist() == [41, 124, 78, 82]
    for k in kinds:
        h, c = pool[k].tolist()
        pages = [int(ring[k][(h + i) % pools[k]]) for i in range(c)]
        for b in range(n):
            m = int(ctx[b]) - (int(lost[b]) if k == "global" else 0)
            pages += table[k][b, (int(first[b]) if k == "sliding" else 0):oplan.pages(m)].tolist()
        assert sorted(pages) == list(range(pools[k])), k
