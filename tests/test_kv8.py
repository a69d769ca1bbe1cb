"""CPU checks of the 8-bit paged cache: its fp64 definition, its byte layout and the host refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import invariant_hybrid_attention_gb300 as g4
import oracle
from invariant_hybrid_attention_gb300 import build as g4build
from invariant_hybrid_attention_gb300.paged import PagedKV8, untile8
from oracle import kv8

L = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    g4build.build()
    return g4.load()


# ---- the definition -----------------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 90, 3.7e-5])
def test_stored_values_are_within_half_a_step_and_bf16(scale):
    x = np.random.default_rng(3).standard_normal((200, 128)) * scale
    y = kv8.stored(x)
    a = np.abs(x).max(-1, keepdims=True)
    step = np.exp2(np.floor(np.log2(a)) - 6)
    # |x| / step < 128: every error is at most half a step, but for x beyond 127.5 steps (clamped to 127)
    assert (np.abs(y - x) <= np.where(np.abs(x) > 127.5 * step, 1.0, 0.5) * step).all()
    assert (torch.tensor(y).bfloat16().double().numpy() == y).all()
    assert (np.abs(y / step) <= 127).all()


def test_stored_edge_vectors():
    z = np.zeros((4, 8))
    z[1, 3] = 2.0 ** -120          # below the smallest stored size: zeros
    z[2, 3] = 2.0 ** -119
    z[3, :2] = [1.0, 127.6 / 64]   # a = 1.99: the step is 2^-6, 127.6 steps clamp to 127
    y = kv8.stored(z)
    assert (y[:2] == 0).all() and y[2, 3] == 2.0 ** -119 and y[3, 1] == 127 / 64 and y[3, 0] == 1.0
    for bad in (np.inf, -np.inf, np.nan):
        w = np.ones((1, 8))
        w[0, 2] = bad
        assert np.isnan(kv8.stored(w)).all()


def test_ties_go_to_the_even_code():
    assert (kv8.stored(np.array([[64.0, 0.5, 1.5, 2.5, -0.5, -1.5]])) == [[64, 0, 2, 2, 0, -2]]).all()


def test_turned_columns():
    c = kv8.turned_columns(oracle.GLOBAL)
    assert list(c) == list(range(64)) + list(range(256, 320))
    assert len(kv8.turned_columns(oracle.SLIDING)) == 256


def test_evict_oracle_keeps_the_ends_and_the_heaviest():
    n, keep, table, w = 81, 3, list(range(10, 16)), [0.0, 5.0, 1.0, 1.0, math.nan, 0.0]
    # pages 1 .. 4 may leave (first 1, last 1): the lightest three, ties by index, NaN the heaviest
    assert kv8.evict(n, table, w, keep, 1, 1)[1] == [10, 14, 15]
    assert kv8.evict(n, table, w, keep, 1, 1)[3] == [11, 12, 13]
    assert kv8.evict(n, table, w, keep, 1, 1)[0] == 81 - 48
    assert kv8.evict(n, table, w, 6, 1, 1)[3] == []


# ---- the byte layout ----------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_byte_layout(lib, kind):
    layer = g4.sliding_layer() if kind == "sliding" else g4.global_layer()
    d, cols1 = (256, 256) if kind == "sliding" else (512, 128)
    block = 16 * (d + cols1) + 32
    assert g4.g4attn_kv8_page_bytes(layer) == layer.n_kv_heads * block
    cache = PagedKV8(layer, 3, device="cpu")
    cache.pages.random_(0, 256, generator=torch.Generator().manual_seed(1))
    one, two = untile8(cache.pages, d)
    assert one.shape == (3, layer.n_kv_heads, 16, d) and two.shape == (3, layer.n_kv_heads, 16, cols1)
    raw = cache.pages.numpy()
    rng = np.random.default_rng(0)
    for _ in range(200):
        p, h, j, which = (int(rng.integers(n)) for n in (3, layer.n_kv_heads, 16, 2))
        n, vals = (d, one) if which == 0 else (cols1, two)
        c = int(rng.integers(n))
        piece = ((c >> 4) & 7) ^ (j & 6) ^ ((j & 1) << 2)
        byte = int(raw[p, h, (16 * d if which else 0) + (c >> 7) * 2048 + j * 128 + piece * 16 + (c & 15)])
        e = int(raw[p, h, 16 * (d + cols1) + 16 * which + j])
        got = float(vals[p, h, j, c])
        if e == 255:
            assert math.isnan(got)
        else:
            assert got == (byte - 128) * 2.0 ** (max(e, 8) - 133)


def test_page_bytes_of_rank_slices_and_bad_layers(lib):
    for tp in (1, 2, 4, 8):
        assert g4.g4attn_kv8_page_bytes(g4.sliding_layer(tp=tp)) == 16 // tp * 8224
        assert g4.g4attn_kv8_page_bytes(g4.global_layer(tp=tp)) == max(1, 4 // tp) * 10272
    bad = g4.sliding_layer()
    bad.head_dim = 128
    assert g4.g4attn_kv8_page_bytes(bad) == 0
    assert g4.g4attn_kv8_decode_workspace_bytes(bad, 4, 4) == 0


# ---- host refusals: nothing is launched, the fake pointers are never touched ---------------------------

def bad_layer():
    b = g4.sliding_layer()
    b.n_q_heads = 24
    return b


def c8(pages=16, num=4, size=16):
    return g4.g4attn_cache8(pages, num, size)


S, GL = g4.sliding_layer(), g4.global_layer()
C16S, C16G = g4.g4attn_cache(16, 32, None, 4, 16), g4.g4attn_cache(16, None, 48, 4, 16)


def append(lib, layer=S, norms=None, k=16, v=16, T=8, rows=(16, 16, 16), B=1, cache=None, table=16, mp=1):
    return lib.g4attn_kv8_append(L(layer), L(norms) if norms else None, k, v, T, *rows, B, L(cache or c8()), table, mp,
                                 None)


def test_append_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED
    assert append(lib, layer=bad_layer()) == U
    assert append(lib, k=None) == I and append(lib, k=24) == I and append(lib, v=None) == I and append(lib, v=24) == I
    assert append(lib, layer=GL) == I                      # K==V takes no v
    assert append(lib, T=-1) == I and append(lib, B=0) == I and append(lib, rows=(16, None, 16)) == I
    assert append(lib, cache=c8(pages=None)) == I and append(lib, cache=c8(pages=24)) == I
    assert append(lib, cache=c8(num=0)) == I and append(lib, cache=c8(size=8)) == U
    assert append(lib, table=None) == I and append(lib, mp=0) == I
    assert append(lib, norms=g4.g4attn_norms(16, 16, 1, 0.0)) == I
    assert append(lib, layer=GL, v=None, norms=g4.g4attn_norms(16, 16, 0, 1e-6)) == U
    assert append(lib, T=0) == g4.G4_OK                    # nothing to do


def test_unpack_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED

    def call(layer=S, begin=16, end=16, B=1, cache=None, table=16, out=C16S, out_table=16, mp=1):
        return lib.g4attn_kv8_unpack(L(layer), begin, end, B, L(cache or c8()), table, L(out), out_table, mp, None)
    assert call(layer=bad_layer()) == U and call(begin=None) == I and call(end=None) == I and call(B=0) == I
    assert call(cache=c8(size=32)) == U and call(table=None) == I and call(out_table=None) == I and call(mp=0) == I
    assert call(out=C16G) == I and call(layer=GL, out=C16S) == I
    assert call(out=g4.g4attn_cache(24, 32, None, 4, 16)) == I


def test_prefill_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED

    def call(layer=S, norms=None, q=16, k=16, v=16, T=8, span=None, cache=None, table=16, scratch=C16S, st=16, mp=1,
             out=16, B=1):
        return lib.g4attn_kv8_prefill(L(layer), L(norms) if norms else None, q, k, v, T, 16, 16, 16, B, span,
                                      L(cache or c8()), table, L(scratch), st, mp, out, None)
    assert call(layer=bad_layer()) == U and call(q=None) == I and call(q=24) == I and call(k=None) == I
    assert call(v=None) == I and call(v=24) == I and call(out=None) == I and call(out=24) == I and call(span=20) == I
    assert call(scratch=C16G) == I and call(st=None) == I and call(table=None) == I and call(mp=0) == I
    assert call(layer=GL, v=16, scratch=C16G) == I and call(B=0) == I and call(T=-3) == I
    assert call(norms=g4.g4attn_norms(24, None, 0, 1e-6)) == I
    assert call(cache=c8(size=8)) == U
    assert call(T=0) == g4.G4_OK


def test_decode_refusals(lib):
    I, U = g4.G4_ERR_INVALID, g4.G4_ERR_UNSUPPORTED
    need = {False: lib.g4attn_kv8_decode_workspace_bytes(L(S), 4, 100, 0),
            True: lib.g4attn_kv8_decode_workspace_bytes(L(GL), 4, 100, 1)}
    assert need[True] > lib.g4attn_kv8_decode_workspace_bytes(L(GL), 4, 100, 0) > 0
    assert lib.g4attn_kv8_decode_workspace_bytes(L(S), 4, 100, 1) == 0      # page weights: global layers only
    assert lib.g4attn_kv8_decode_workspace_bytes(L(S), 0, 100, 0) == 0
    assert lib.g4attn_kv8_decode_workspace_bytes(L(S), 4, 0, 0) == 0

    def call(layer=S, norms=None, q=16, kn=None, vn=None, sl=16, pos=None, B=4, cache=None, table=16, mp=100, pw=None,
             out=16, ws=16, size=None):
        size = need[layer is GL] if size is None else size
        return lib.g4attn_kv8_decode(L(layer), L(norms) if norms else None, q, kn, vn, sl, pos, B, L(cache or c8()),
                                     table, mp, pw, out, ws, size, None)
    assert call(layer=bad_layer()) == U and call(pw=16) == U
    assert call(q=None) == I and call(q=24) == I and call(sl=None) == I and call(out=None) == I and call(out=24) == I
    assert call(ws=None) == I and call(ws=24) == I and call(B=0) == I and call(table=None) == I and call(mp=0) == I
    assert call(kn=16) == I and call(kn=24, vn=16) == I and call(vn=16) == I         # k_new and v_new come together
    assert call(layer=GL, kn=16, vn=16) == I
    assert call(size=need[False] - 1) == I and call(layer=GL, pw=16, size=need[True] - 1) == I
    assert call(cache=c8(size=8)) == U and call(norms=g4.g4attn_norms(None, None, 2, 1e-6)) == I


def test_evict_refusals(lib):
    I = g4.G4_ERR_INVALID

    def call(B=1, mp=8, keep=4, first=1, last=1, ptrs=(16,) * 8):
        return lib.g4attn_evict_pages(*ptrs[:3], B, mp, keep, first, last, *ptrs[3:], None)
    assert call(B=0) == I and call(mp=0) == I and call(mp=16385) == I
    assert call(keep=0) == I and call(first=-1) == I and call(last=0) == I
    assert call(first=3, last=2) == I and call(first=2 ** 31 - 1, last=2 ** 31 - 1, keep=4) == I
    for i in range(8):
        assert call(ptrs=(16,) * i + (None,) + (16,) * (7 - i)) == I


def test_binding_refuses_other_types_shapes_and_strides(lib):
    """A raw pointer cannot say what it points to, so the binding looks at the tensors."""
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    w = torch.zeros(2, 4)
    good = dict(seq_len=i32, page_table=table, page_weights=w, keep_pages=2, first_pages=0, last_pages=1,
                out_seq_len=i32, out_table=table, out_weights=w, freed=table, n_freed=i32)
    for name, bad in (("seq_len", i32.long()), ("page_table", torch.zeros(4, 2, dtype=torch.int32).t()),
                      ("page_weights", w.double()), ("out_table", table[:, :3]), ("n_freed", torch.zeros(3).int())):
        with pytest.raises(ValueError, match=name):
            g4.g4attn_evict_pages(**{**good, name: bad})
    k = torch.zeros(5, 16, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k must"):
        g4.g4attn_kv8_append(S, None, k.half(), k, i32, i32, i32, c8(), table)
    with pytest.raises(ValueError, match="v must"):
        g4.g4attn_kv8_append(S, None, k, k[:4], i32, i32, i32, c8(), table)
    q, ws = torch.zeros(2, 32, 256, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must"):      # 2^30 elements on 8 bytes
        g4.g4attn_kv8_decode(S, None, q, None, None, i32, c8(), table, q, ws.expand(2 ** 27, 8))
