"""CPU checks of the page plan: its definition's invariants, and the refusals of host and binding."""
import random

import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300 import build as g4build
from oracle import plan as oplan


@pytest.fixture(scope="module")
def lib():
    g4build.build()
    return g4.load()


def test_the_definition_keeps_every_page_in_one_place():
    """A long run of steps with short pools, windows, evictions and ends: at every step each physical page is free, or
    held by one request in its place, and nobody loses a key that is still visible."""
    for seed in range(6):
        r = random.Random(seed)
        n, width, window = 5, 12, 40
        groups = [dict(window=w, num_pages=23, table=[[-1] * width for _ in range(n)], ring=list(range(23)), pool=[7, 23],
                       first=[0] * n if w else None, lost=None if w else [0] * n, freed=None) for w in (0, window)]
        ctx = [0] * n
        for _ in range(150):
            if r.random() < 0.2 and groups[0]["freed"] is None:   # an eviction closes a table up
                g = groups[0]
                g["freed"] = [[] for _ in range(n)]
                for b in range(n):
                    held = oplan.pages(ctx[b] - g["lost"][b])
                    if held > 3:
                        g["freed"][b] = [g["table"][b].pop(1)]
                        g["table"][b].append(-1)
            evicted = groups[0]["freed"]
            new = [r.choice([0, 1, 1, 1, 16, 25, -1]) for _ in range(n)]
            new = [x if ctx[b] + max(x, 0) <= 16 * width else -1 for b, x in enumerate(new)]
            before = list(ctx)
            ctx, start, length, pos, seq, slots = oplan.plan(ctx, new, 60, groups)
            groups[0]["freed"] = None
            assert evicted is None or groups[0]["lost"] is not None
            for g in groups:
                free = [g["ring"][(g["pool"][0] + i) % 23] for i in range(g["pool"][1])]
                held = []
                for b in range(n):
                    h = ctx[b] - (g["lost"][b] if g["lost"] else 0)
                    held += g["table"][b][g["first"][b] if g["first"] else 0:oplan.pages(h)]
                assert sorted(free + held) == list(range(23))
            for b in range(n):
                if length[b]:
                    assert pos[start[b]:start[b] + length[b]] == list(range(before[b], before[b] + length[b]))
                    assert ctx[b] == before[b] + new[b] == seq[1][b]
                    assert groups[1]["first"][b] * 16 <= max(0, before[b] - window + 1)
                elif new[b] >= 0:
                    assert ctx[b] == before[b] and seq[0][b] == 0


# ---- host refusals ------------------------------------------------------------------------------------

def group(**kw):
    f = dict(window=0, num_pages=4, max_pages=2, free_pages=16, pool=16, out_pool=16, page_table=16, first_page=None,
             out_first_page=None, lost=None, out_lost=None, freed=None, n_freed=None, seq_len=16, slots=None)
    f.update(kw)
    return g4.g4attn_page_group(*f.values())


def test_plan_refusals(lib):
    I = g4.G4_ERR_INVALID

    def call(B=2, T=8, n=1, groups=None, arrays=(16,) * 7):
        gs = groups or [group()]
        a = (g4.g4attn_page_group * len(gs))(*gs)
        return lib.g4attn_plan_pages(arrays[0], arrays[1], B, T, a, n, *arrays[2:], None)
    assert call(B=0) == I and call(B=4097) == I and call(T=-1) == I and call(n=0) == I and call(n=3) == I
    for i in range(6):   # all but positions
        assert call(arrays=(16,) * i + (None,) + (16,) * (6 - i)) == I
    for bad in (dict(window=-1), dict(window=262145, first_page=16, out_first_page=16), dict(num_pages=0), dict(max_pages=0),
                dict(free_pages=None), dict(pool=None), dict(out_pool=None), dict(page_table=None), dict(seq_len=None),
                dict(slots=20), dict(window=8), dict(window=8, first_page=16), dict(first_page=16, out_first_page=16),
                dict(lost=16), dict(out_lost=16), dict(lost=16, out_lost=16, freed=16), dict(freed=16, n_freed=16),
                dict(window=8, first_page=16, out_first_page=16, lost=16, out_lost=16),
                dict(window=8, first_page=16, out_first_page=16, freed=16, n_freed=16)):
        assert call(groups=[group(**bad)]) == I, bad
        assert call(groups=[group(), group(**bad)], n=2) == I, bad


def test_binding_refuses_other_types_shapes_and_sizes(lib):
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)   # noqa: E731
    good = dict(window=0, page_table=z(3, 5), free_pages=z(20), pool=z(2), out_pool=z(2), seq_len=z(3),
                slots=z(9, t=torch.int64))
    for name, bad in (("page_table", z(5, 3).t()), ("free_pages", z(20, t=torch.int64)), ("pool", z(3)),
                      ("seq_len", z(4)), ("slots", z(9)), ("lost", z(2)), ("freed", z(3, 4)), ("n_freed", z(3, 1))):
        with pytest.raises(ValueError, match=name):
            g4.make_page_group(**{**good, name: bad})
    group = g4.make_page_group(**good)
    a = dict(ctx_len=z(3), new_len=z(3), groups=[group], out_ctx_len=z(3), q_start=z(3), q_len=z(3), ctx_start=z(3),
             positions=z(9))
    for name, bad in (("new_len", z(4)), ("q_len", z(3, t=torch.int64)), ("positions", z(18)[::2])):
        with pytest.raises(ValueError, match=name):
            g4.g4attn_plan_pages(**{**a, name: bad})


def test_the_freed_pages_come_with_a_place_for_their_count_after_the_step(lib):
    """A list of evicted pages that no step marks as taken would come back at every step."""
    I = g4.G4_ERR_INVALID
    names = [name for name, _ in g4.g4attn_page_group._fields_]

    def call(**kw):
        g = group()
        for name, value in kw.items():
            assert name in names
            setattr(g, name, value)
        a = (g4.g4attn_page_group * 1)(g)
        return lib.g4attn_plan_pages(16, 16, 2, 8, a, 1, 16, 16, 16, 16, 16, None)
    lost = dict(lost=16, out_lost=16)
    assert call(**lost, freed=16, n_freed=16) == I
    assert call(**lost, out_n_freed=16) == I and call(out_n_freed=16) == I
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)   # noqa: E731
    a = dict(window=0, page_table=z(3, 5), free_pages=z(20), pool=z(2), out_pool=z(2), seq_len=z(3), freed=z(3, 5),
             n_freed=torch.ones(3, dtype=torch.int32), lost=z(3))
    inside = g4.make_page_group(**a, out_lost=a["lost"])
    assert inside.out_n_freed == inside.n_freed == a["n_freed"].data_ptr()
    apart = g4.make_page_group(**a, out_lost=z(3))
    kept = apart.tensors["out_n_freed"]
    assert apart.out_n_freed == kept.data_ptr() != apart.n_freed and kept.shape == (3,)
    given = z(3)
    assert g4.make_page_group(**a, out_lost=z(3), out_n_freed=given).out_n_freed == given.data_ptr()
    with pytest.raises(ValueError, match="out_n_freed"):
        g4.make_page_group(**a, out_lost=z(3), out_n_freed=z(4))
