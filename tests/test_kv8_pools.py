"""The binding's 8-bit calls look at the tensors behind a cache: one that does not hold the pages it is said to
have would be read and written past its end. Nothing is launched here; the tensors are the CPU's."""
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV8

KINDS = {"sliding": g4.sliding_layer, "global": g4.global_layer}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return g4.load()


def tensors(layer, rows=5, B=2, width=4):
    bf, h, d = torch.bfloat16, layer.n_kv_heads, layer.head_dim
    k = torch.zeros(rows, h, d, dtype=bf)
    i32 = torch.zeros(B, dtype=torch.int32)
    return dict(q=torch.zeros(rows, layer.n_q_heads, d, dtype=bf), k=k, v=None if layer.kv_shared else k, rows=i32,
                one=torch.zeros(B, layer.n_q_heads, d, dtype=bf), table=torch.zeros(B, width, dtype=torch.int32),
                ws=torch.zeros(64, dtype=torch.uint8))


def calls(layer, cache, scratch):
    a = tensors(layer)
    return {
        "append": lambda: g4.g4attn_kv8_append(layer, None, a["k"], a["v"], *[a["rows"]] * 3, cache, a["table"]),
        "unpack": lambda: g4.g4attn_kv8_unpack(layer, a["rows"], a["rows"], cache, a["table"], scratch, a["table"]),
        "prefill": lambda: g4.g4attn_kv8_prefill(layer, None, a["q"], a["k"], a["v"], *[a["rows"]] * 3, cache,
                                                 a["table"], scratch, a["table"], a["q"]),
        "decode": lambda: g4.g4attn_kv8_decode(layer, None, a["one"], None, None, a["rows"], cache, a["table"],
                                               a["one"], a["ws"])}


@pytest.mark.parametrize("call", ["append", "unpack", "prefill", "decode"])
@pytest.mark.parametrize("tp", [1, 8])
@pytest.mark.parametrize("kind", list(KINDS))
def test_a_cache_larger_than_its_tensor_is_refused(kind, tp, call):
    layer = KINDS[kind](tp=tp)
    pool = PagedKV8(layer, 7, device="cpu")
    scratch = PagedKV(7, layer.n_kv_heads, layer.head_dim, kind == "global", device="cpu")
    with pytest.raises(ValueError, match="the 8-bit cache has .* bytes, its pages take"):
        calls(layer, g4.make_cache8(pool.pages, 8), scratch.desc)[call]()
    with pytest.raises(ValueError, match="the 8-bit cache has .* bytes, its pages take"):
        calls(layer, g4.make_cache8(pool.pages[1:], 7), scratch.desc)[call]()
    with pytest.raises(ValueError, match="not on the current CUDA device"):     # of its own size: the next refusal
        calls(layer, pool.desc, scratch.desc)[call]()
    if call in ("unpack", "prefill"):
        wrong = PagedKV(7, layer.n_kv_heads, layer.head_dim, kind == "global", device="cpu")
        wrong.num_pages = 8
        with pytest.raises(ValueError, match="the bf16 cache has .* bytes, its pages take"):
            calls(layer, pool.desc, wrong.desc)[call]()
        second = "k_rot" if kind == "global" else "v"
        wrong.num_pages = 7
        setattr(wrong, second, getattr(wrong, second)[:6])
        with pytest.raises(ValueError, match="the bf16 cache has .* bytes, its pages take"):
            calls(layer, pool.desc, wrong.desc)[call]()


def test_a_full_layers_cache_under_a_slices_layer_and_the_reverse():
    full, slice_ = g4.sliding_layer(), g4.sliding_layer(tp=2)
    with pytest.raises(ValueError, match="its pages take"):
        calls(full, PagedKV8(slice_, 7, device="cpu").desc, None)["append"]()
    with pytest.raises(ValueError, match="current CUDA device"):                # large enough
        calls(slice_, PagedKV8(full, 7, device="cpu").desc, None)["append"]()


def test_a_strided_pool_is_refused():
    layer = g4.global_layer()
    pool = PagedKV8(layer, 7, device="cpu")
    with pytest.raises(ValueError, match="dense"):
        g4.make_cache8(PagedKV8(layer, 14, device="cpu").pages[::2], 7)
    scratch = PagedKV(14, 4, 512, True, device="cpu")
    scratch.k, scratch.num_pages = scratch.k[::2], 7
    for call in ("unpack", "prefill"):
        with pytest.raises(ValueError, match="dense"):
            calls(layer, pool.desc, scratch.desc)[call]()


def test_a_raw_address_is_passed_on_and_a_descriptor_keeps_its_tensor():
    """Raw addresses alone reach the next refusal; a descriptor's tensors live as long as it does."""
    layer = g4.sliding_layer()
    raw8, raw16 = g4.make_cache8(4096, 1 << 20), g4.make_cache(16, 32, 1 << 20)
    assert raw8.tensor is None
    for call in ("append", "unpack", "prefill", "decode"):
        for scratch in (raw16, g4.g4attn_cache(16, 32, None, 1 << 20, 16)):
            with pytest.raises(ValueError, match="current CUDA device"):
                calls(layer, raw8, scratch)[call]()
    pool = PagedKV8(layer, 3, device="cpu")
    assert pool.desc.tensor is pool.pages and pool.desc.pages == pool.pages.data_ptr()
