"""CPU checks of the 4-bit paged cache: its fp64 definition, its byte layout, and the refusals of host and binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
from invariant_hybrid_attention_gb300 import build as g4build
from invariant_hybrid_attention_gb300.paged import PagedKV, PagedKV4, untile4
from oracle import kv4

L = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    g4build.build()
    return g4.load()


# ---- the definition -----------------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** 90, 3.7e-5])
def test_stored_values_are_the_nearest_step_and_bf16(scale):
    x = np.random.default_rng(3).standard_normal((200, 128)) * scale
    y = kv4.stored(x)
    unit = np.exp2(np.repeat(kv4.exponents(x), 32, -1))
    m = np.abs(x) / unit
    assert (m <= 7.0).all() and (m.reshape(200, 4, 32).max(-1) > 3.5).all()
    # the distance to the nearest step is half of the gap between its neighbours at most
    assert (np.abs(y - x) <= np.where(m < 2, 0.25, np.where(m < 4, 0.5, 1.0)) * unit).all()
    grid = np.concatenate([-kv4.STEPS[::-1], kv4.STEPS])
    nearest = np.abs(x[..., None] / unit[..., None] - grid).min(-1)
    assert np.allclose(np.abs(y - x) / unit, nearest, rtol=0, atol=1e-12)
    assert (torch.tensor(y).bfloat16().double().numpy() == y).all()


def test_stored_ties_and_the_border_between_two_exponents():
    row = np.zeros((1, 64))
    row[0, :10] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.25, -0.75, 3.4999]
    row[0, 32:36] = [7.0, 5.0, 0.25, 1.0]
    want = np.zeros((1, 64))
    want[0, :10] = [4, 0, 1, 1, 2, 2, 4, 0, -1, 3]
    want[0, 32:36] = [6, 4, 0, 1]             # 7 still rounds to 6, a tie of 5 to the even code 4
    assert (kv4.stored(row) == want).all()
    row[0, 32] = 7.0001                       # from here on the unit is 2
    assert kv4.stored(row)[0, 32] == 8.0 and kv4.stored(row)[0, 33] == 4.0 and kv4.stored(row)[0, 35] == 1.0


def test_stored_edge_vectors():
    z = np.zeros((5, 64))
    z[1, 3], z[1, 40] = 2.0 ** -78, 1.0       # below the smallest stored size: zeros, block by block
    z[2, 3] = 2.0 ** -77
    z[3, 0] = 255 * 2.0 ** 120                # near the largest bf16: the largest value is 6 * 2^125
    z[4, 5] = 1e-300
    y = kv4.stored(z)
    assert (y[[0, 4]] == 0).all() and y[1, 3] == 0 and y[1, 40] == 1 and y[2, 3] == 2.0 ** -77
    assert y[3, 0] == 6 * 2.0 ** 125
    for bad in (np.inf, -np.inf, np.nan):
        w = np.ones((1, 64))
        w[0, 2] = bad
        assert np.isnan(kv4.stored(w)).all()


# ---- the byte layout ----------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_byte_layout(lib, kind):
    layer = g4.sliding_layer() if kind == "sliding" else g4.global_layer()
    d, cols1, block = (256, 256, 4368) if kind == "sliding" else (512, 128, 5456)
    assert g4.g4attn_kv4_page_bytes(layer) == layer.n_kv_heads * block
    cache = PagedKV4(layer, 3, device="cpu")
    cache.pages.random_(0, 256, generator=torch.Generator().manual_seed(1))
    one, two = untile4(cache.pages, d)
    assert one.shape == (3, layer.n_kv_heads, 16, d) and two.shape == (3, layer.n_kv_heads, 16, cols1)
    raw, rng = cache.pages.numpy(), np.random.default_rng(0)
    tops = raw[..., -16:]
    assert tops.shape[-1] == 16
    for _ in range(300):
        p, h, j, which = (int(rng.integers(n)) for n in (3, layer.n_kv_heads, 16, 2))
        n, vals = (d, one) if which == 0 else (cols1, two)
        c = int(rng.integers(n))
        at, b, in_b = (8 * d if which else 0), c // 32, c % 32
        if n == 128:
            at += j * 64 + (in_b % 16 // 4) * 16 + b * 4 + in_b // 16 * 2 + in_b % 4 // 2
        else:
            piece = (in_b // 4) ^ (j & 6) ^ ((j & 1) << 2)
            at += c // 256 * 2048 + j * 128 + piece * 16 + b % 8 * 2 + in_b % 4 // 2
        code = (int(raw[p, h, at]) >> (4 * (c & 1))) & 15
        scales = 8 * (d + cols1) + (16 * d // 32 if which else 0) + j * (n // 32)
        s = int(raw[p, h, scales + b])
        got = float(vals[p, h, j, c])
        if s == 255:
            assert math.isnan(got)
        else:
            want = float(kv4.STEPS[code & 7]) * 2.0 ** (s - 127) * (-1 if code & 8 else 1)
            with np.errstate(over="ignore"):
                assert got == float(np.float32(want)) or abs(want) < 2.0 ** -126


def test_page_bytes_of_rank_slices_and_bad_layers(lib):
    for tp in (1, 2, 4, 8):
        assert g4.g4attn_kv4_page_bytes(g4.sliding_layer(tp=tp)) == 16 // tp * 4368
        assert g4.g4attn_kv4_page_bytes(g4.global_layer(tp=tp)) == max(1, 4 // tp) * 5456
    bad = g4.sliding_layer()
    bad.head_dim = 128
    assert g4.g4attn_kv4_page_bytes(bad) == 0
    assert g4.g4attn_kv4_decode_workspace_bytes(bad, 4, 4) == 0


# ---- host refusals: nothing is launched, the fake pointers are never touched ---------------------------

def bad_layer():
    b = g4.sliding_layer()
    b.n_q_heads = 24
    return b


def c4(pages=16, num=4, size=16):
    return g4.g4attn_cache4(pages, num, size)


S, GL = g4.sliding_layer(), g4.global_layer()
C16S, C16G = g4.g4attn_cache(16, 32, None, 4, 16), g4.g4attn_cache(16, None, 48, 4, 16)


def test_append_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED

    def call(layer=S, norms=None, k=16, v=16, T=8, rows=(16, 16, 16), B=1, cache=None, table=16, mp=1):
        return lib.g4attn_kv4_append(L(layer), L(norms) if norms else None, k, v, T, *rows, B, L(cache or c4()), table,
                                     mp, None)
    assert call(layer=bad_layer()) == U
    assert call(k=None) == I and call(k=24) == I and call(v=None) == I and call(v=24) == I
    assert call(layer=GL) == I                             # K==V takes no v
    assert call(T=-1) == I and call(B=0) == I and call(rows=(16, None, 16)) == I
    assert call(cache=c4(pages=None)) == I and call(cache=c4(pages=24)) == I
    assert call(cache=c4(num=0)) == I and call(cache=c4(size=8)) == U
    assert call(table=None) == I and call(mp=0) == I
    assert call(norms=g4.g4attn_norms(16, 16, 1, 0.0)) == I
    assert call(layer=GL, v=None, norms=g4.g4attn_norms(16, 16, 0, 1e-6)) == U
    assert call(T=0) == g4.G4_OK                           # nothing to do


def test_unpack_and_prefill_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED

    def unpack(layer=S, begin=16, end=16, B=1, cache=None, table=16, out=C16S, out_table=16, mp=1):
        return lib.g4attn_kv4_unpack(L(layer), begin, end, B, L(cache or c4()), table, L(out), out_table, mp, None)
    assert unpack(layer=bad_layer()) == U and unpack(begin=None) == I and unpack(end=None) == I and unpack(B=0) == I
    assert unpack(cache=c4(size=32)) == U and unpack(table=None) == I and unpack(out_table=None) == I
    assert unpack(mp=0) == I and unpack(out=C16G) == I and unpack(layer=GL, out=C16S) == I

    def prefill(layer=S, q=16, k=16, v=16, T=8, span=None, cache=None, table=16, scratch=C16S, st=16, mp=1, out=16, B=1):
        return lib.g4attn_kv4_prefill(L(layer), None, q, k, v, T, 16, 16, 16, B, span, L(cache or c4()), table,
                                      L(scratch), st, mp, out, None)
    assert prefill(layer=bad_layer()) == U and prefill(q=None) == I and prefill(q=24) == I and prefill(k=None) == I
    assert prefill(v=None) == I and prefill(out=None) == I and prefill(out=24) == I and prefill(span=20) == I
    assert prefill(scratch=C16G) == I and prefill(st=None) == I and prefill(table=None) == I and prefill(mp=0) == I
    assert prefill(layer=GL, v=16, scratch=C16G) == I and prefill(B=0) == I and prefill(T=-3) == I
    assert prefill(cache=c4(size=8)) == U and prefill(T=0) == g4.G4_OK


def test_decode_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED
    need = {False: lib.g4attn_kv4_decode_workspace_bytes(L(S), 4, 100, 0),
            True: lib.g4attn_kv4_decode_workspace_bytes(L(GL), 4, 100, 1)}
    assert need[True] > lib.g4attn_kv4_decode_workspace_bytes(L(GL), 4, 100, 0) > 0
    assert lib.g4attn_kv4_decode_workspace_bytes(L(S), 4, 100, 1) == 0      # page weights: global layers only
    assert lib.g4attn_kv4_decode_workspace_bytes(L(S), 0, 100, 0) == 0
    assert lib.g4attn_kv4_decode_workspace_bytes(L(S), 4, 0, 0) == 0

    def call(layer=S, q=16, kn=None, vn=None, sl=16, pos=None, B=4, cache=None, table=16, mp=100, pw=None, out=16, ws=16,
             size=None):
        size = need[layer is GL] if size is None else size
        return lib.g4attn_kv4_decode(L(layer), None, q, kn, vn, sl, pos, B, L(cache or c4()), table, mp, pw, out, ws, size,
                                     None)
    assert call(layer=bad_layer()) == U and call(pw=16) == U
    assert call(q=None) == I and call(q=24) == I and call(sl=None) == I and call(out=None) == I and call(out=24) == I
    assert call(ws=None) == I and call(ws=24) == I and call(B=0) == I and call(table=None) == I and call(mp=0) == I
    assert call(kn=16) == I and call(kn=24, vn=16) == I and call(vn=16) == I         # k_new and v_new come together
    assert call(layer=GL, kn=16, vn=16) == I
    assert call(size=need[False] - 1) == I and call(layer=GL, pw=16, size=need[True] - 1) == I
    assert call(cache=c4(size=8)) == U


# ---- the binding: a raw pointer cannot say what it points to ----------------------------------------------

@pytest.mark.parametrize("call", ["append", "unpack", "prefill", "decode"])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_cache_larger_than_its_tensor_is_refused(lib, kind, call):
    layer = S if kind == "sliding" else GL
    bf, h, d = torch.bfloat16, layer.n_kv_heads, layer.head_dim
    k, q = torch.zeros(5, h, d, dtype=bf), torch.zeros(5, 32, d, dtype=bf)
    v, rows, table = None if kind == "global" else k, torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    pool, scratch = PagedKV4(layer, 7, device="cpu"), PagedKV(7, h, d, kind == "global", device="cpu")

    def run(cache):
        if call == "append":
            g4.g4attn_kv4_append(layer, None, k, v, rows, rows, rows, cache, table)
        elif call == "unpack":
            g4.g4attn_kv4_unpack(layer, rows, rows, cache, table, scratch.desc, table)
        elif call == "prefill":
            g4.g4attn_kv4_prefill(layer, None, q, k, v, rows, rows, rows, cache, table, scratch.desc, table, q)
        else:
            g4.g4attn_kv4_decode(layer, None, q[:2], None, None, rows, cache, table, q[:2], torch.zeros(64, dtype=torch.uint8))
    for cache in (g4.make_cache4(pool.pages, 8), g4.make_cache4(pool.pages[1:], 7)):
        with pytest.raises(ValueError, match="the 4-bit cache has .* bytes, its pages take"):
            run(cache)
    with pytest.raises(ValueError, match="not on the current CUDA device"):     # of its own size: the next refusal
        run(pool.desc)


def test_binding_refuses_other_types_shapes_and_strides(lib):
    i32, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    k = torch.zeros(5, 16, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k must"):
        g4.g4attn_kv4_append(S, None, k.half(), k, i32, i32, i32, c4(), table)
    with pytest.raises(ValueError, match="v must"):
        g4.g4attn_kv4_append(S, None, k, k[:4], i32, i32, i32, c4(), table)
    with pytest.raises(ValueError, match="dense"):
        g4.make_cache4(torch.zeros(4, 8, dtype=torch.uint8).t(), 1)
    with pytest.raises(ctypes.ArgumentError):                  # an 8-bit cache is not a 4-bit one
        lib.g4attn_kv4_append(L(S), None, 16, 16, 8, 16, 16, 16, 1, L(g4.g4attn_cache8(16, 4, 16)), 16, 1, None)


@pytest.mark.parametrize("tp", [1, 2])
def test_provenance_names_the_chunks_that_the_workspace_holds(lib, tp):
    """The record's split is the one the decode makes: a state of D + 2 floats per head and chunk slot, in two runs of
    whole 256 bytes."""
    for layer, window in ((g4.sliding_layer(tp=tp), 1024), (g4.sliding_layer(700, tp=tp), 700), (g4.global_layer(tp=tp), 0)):
        chunk = int(g4.g4attn_provenance(layer).split("kv4=")[1].split("split-")[1].split("@")[0])
        d, width = layer.head_dim, 1000
        slots = -(-width * 16 // chunk)
        if window:
            slots = min(slots, (window - 1) // chunk + 2)
        states = 3 * layer.n_q_heads * slots
        want = sum(-(-states * 4 * n // 256) * 256 for n in (2, d))
        assert g4.g4attn_kv4_decode_workspace_bytes(layer, 3, width) == want
