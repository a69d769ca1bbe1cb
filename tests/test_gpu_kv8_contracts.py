"""Promises of the header that the 8-bit cache's calls share with the bf16 ones, held to the bit."""
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300.paged import PagedKV8

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
