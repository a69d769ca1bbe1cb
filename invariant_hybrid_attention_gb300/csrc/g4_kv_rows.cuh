// What the appends and read-backs of the quantised caches (8-bit and 4-bit) have in common: a lane's share of a
// head vector with its norm and its largest magnitude, the place of a row's token, its angles, and the walk over
// a batch's pages.
#pragma once

#include <math.h>

#include "g4_kv8.cuh"

namespace g4 {

// D/16 lanes hold a head vector, 8 half-split pairs each (columns t0 .. t0+7 and D/2 + t0 .. +7), so
// loads are 16 bytes a lane and the vector's largest |x| is one warp reduction.
template <int D>
struct Vec {
  float a[8], b[8];   // columns t0 + i and D/2 + t0 + i
};

struct Raw {   // a lane's columns as bf16, as loaded
  uint4 lo, hi;
};

template <int D>
G4_DEV Raw load_raw(const __nv_bfloat16* __restrict__ src, int t0) {
  return Raw{*reinterpret_cast<const uint4*>(src + t0), *reinterpret_cast<const uint4*>(src + D / 2 + t0)};
}

template <int D>
G4_DEV Vec<D> widen(const Raw& raw) {
  const uint4 lo = raw.lo, hi = raw.hi;
  const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
  Vec<D> v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[2 * i] = bf16_lo(lw[i]);
    v.a[2 * i + 1] = bf16_hi(lw[i]);
    v.b[2 * i] = bf16_lo(hw[i]);
    v.b[2 * i + 1] = bf16_hi(hw[i]);
  }
  return v;
}

// sqrt(mean(x^2) + eps) over the D/16 lanes of the vector, and its reciprocal.
struct Norm {
  float root, inv;
};

template <int D>
G4_DEV Norm norm_of(const Vec<D>& v, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v.a[i], v.a[i], ss);
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v.b[i], v.b[i], ss);
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float root = __fsqrt_rn(__fadd_rn(ss * (1.0f / (float)D), eps));   // ss / D is exact: D is a power of 2
  // an infinite root divides every number to 0: with root 0 the quotient below is x 0
  return Norm{root == INFINITY ? 0.f : root, __frcp_rn(root)};
}

// x / root to the nearest, by Markstein's method: the product with the rounded reciprocal, corrected by its
// exact remainder. What is rounded to a code next then agrees with the definition's division.
G4_DEV float over(float x, Norm n) {
  const float q = x * n.inv;
  return fmaf(fmaf(-q, n.root, x), n.inv, q);
}

template <int D>
G4_DEV void divide(Vec<D>& v, Norm n) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.a[i] = over(v.a[i], n);
    v.b[i] = over(v.b[i], n);
  }
}

template <int D>
G4_DEV void weight(Vec<D>& v, const __nv_bfloat16* __restrict__ w, int t0) {
  const Vec<D> m = widen<D>(load_raw<D>(w, t0));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.a[i] *= m.a[i];
    v.b[i] *= m.b[i];
  }
}

// max(a, |b|), NaN if either is one.
G4_DEV float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The bits of the largest |x| over the lanes of `mask` (all of which call it); a NaN wins.
template <int D>
G4_DEV uint32_t max_bits(const Vec<D>& v, unsigned mask) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    m[0] = max_abs(m[0], v.a[i]);
    m[1] = max_abs(m[1], v.a[i + 1]);
    m[2] = max_abs(m[2], v.b[i]);
    m[3] = max_abs(m[3], v.b[i + 1]);
  }
  return __reduce_max_sync(mask, __float_as_uint(max_abs(max_abs(m[0], m[1]), max_abs(m[2], m[3]))));
}

// Where row r's token goes: its held index, RoPE position and physical page; false (and an error, for a row that
// some sequence owns) when it goes nowhere. MODE 0: the rows of a prefill; MODE 1: one new token per request at
// held index seq_len - 1 (a seq_len of 0 is an error unless empty_ok). The warp of unit 0 (first) looks at every
// sequence of a prefill, for its error.
template <int MODE>
G4_DEV bool token_place(const SeqRows& rows, const int32_t* seq_len, const int32_t* rope_pos, const PagedCache8& cache,
                        uint32_t* err, int r, bool first, int lane, int& idx, int& pos, int& phys, bool empty_ok = false) {
  int b = r;
  if (MODE == 0) {
    int owner = -1;
    for (int b0 = 0; b0 < rows.B; b0 += 32) {
      const int i = b0 + lane;
      bool mine = false;
      if (i < rows.B) {
        const int qs = rows.q_start[i], L = rows.q_len[i];
        if (L > 0) {
          const bool ok = rows_ok(rows, qs, L, rows.ctx_start[i]);
          if (!ok && first) set_error(err, kErrPos);
          mine = ok && r >= qs && r - qs < L;
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, mine);
      if (m && owner < 0) owner = b0 + __ffs(m) - 1;
      if (owner >= 0 && !first) break;
    }
    if (owner < 0) return false;
    b = owner;
    idx = rows.ctx_start[b] + (r - rows.q_start[b]);
    pos = idx;
  } else {
    idx = seq_len[b] - 1;
    if (empty_ok && idx == -1) return false;
    pos = rope_pos ? rope_pos[b] : idx;
  }
  if (idx < 0 || idx >= kMaxPos || (idx >> 4) >= cache.max_pages || pos < idx || pos >= kMaxPos) {
    if (lane == 0) set_error(err, kErrPos);
    return false;
  }
  phys = cache.page_table[(size_t)b * cache.max_pages + (idx >> 4)];
  if (phys < 0 || phys >= cache.num_pages) {
    if (lane == 0) set_error(err, kErrPage);
    return false;
  }
  return true;
}

// The angles of a row at RoPE position pos, for this lane's pairs tr .. tr + 7: pair t by lane t % 32 (whole lines
// of the tables), then to the lanes that turn by them through shared memory (mine: R entries of this warp), two
// pairs to 16 bytes, [i / 2][lane] so that the reads conflict on no bank.
template <int R>
G4_DEV void row_angles(const Kv8Angles& angles, int pos, int lane, float2* mine, int tr, float2 (&cs)[8]) {
  const float4* cx = angles.coarse + (size_t)(pos >> 8) * R;
  const float4* fx = angles.fine + (size_t)(pos & 255) * R;
  float4 c4[R / 32], f4[R / 32];
#pragma unroll
  for (int k = 0; k < R / 32; ++k) {
    c4[k] = __ldg(cx + 32 * k + lane);
    f4[k] = __ldg(fx + 32 * k + lane);
  }
#pragma unroll
  for (int k = 0; k < R / 32; ++k) {
    const int t = 32 * k + lane;
    mine[(((t & 7) >> 1) * (R / 8) + (t >> 3)) * 2 + (t & 1)] = rope_cs_exact(c4[k], f4[k]);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(mine + (i * (R / 8) + (tr >> 3)) * 2);
    cs[2 * i] = make_float2(v.x, v.y);
    cs[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// ---- read-back: which keys, and the walk over their pages ---------------------------------------------
struct UnpackArgs {
  Kv8Range range;
  PagedCache8 src;
  PagedCache dst;   // page_table: the destination pages of the same logical pages
  uint32_t* err;
};

// The key range of sequence b; an impossible one is refused (empty, kErrPos).
G4_DEV void key_range(const UnpackArgs& p, int b, int& lo, int& hi, uint32_t* err) {
  lo = hi = 0;
  if (p.range.key_begin) {
    const int k0 = p.range.key_begin[b], k1 = p.range.key_end[b];
    if (k1 <= k0) return;
    if (k0 < 0 || k1 > kMaxPos || ((k1 - 1) >> 4) >= p.src.max_pages) {
      set_error(err, kErrPos);
      return;
    }
    lo = k0;
    hi = k1;
  } else {
    const int L = p.range.rows.q_len[b], cs = p.range.rows.ctx_start[b];
    if (L <= 0) return;
    if (!rows_ok(p.range.rows, p.range.rows.q_start[b], L, cs) || ((cs + L - 1) >> 4) >= p.src.max_pages) {
      set_error(err, kErrPos);
      return;
    }
    lo = p.range.window > 0 ? max(0, cs - p.range.window + 1) : 0;
    hi = cs + L;
    // An image that began before this chunk holds its first row, whatever other rows it holds.
    if (lo > 0 && p.range.rows.span) {
      const int2 s = reinterpret_cast<const int2*>(p.range.rows.span)[p.range.rows.q_start[b]];
      if (s.x >= 0 && s.x <= cs && cs < s.y && s.y <= hi) lo = min(lo, s.x);
    }
  }
}

// The (page, KV head) of a unit of the batch: its sequence's key range [lo, hi), logical page, head and physical
// pages. Walks on from where the last unit was found: base units before sequence group b0. -1: no such unit; 0: a
// page outside a pool (an error); 1: found.
G4_DEV int find_page(const UnpackArgs& p, long long unit, int lane, long long& base, int& b0, int& lo, int& hi, int& page,
                     int& g, int& from, int& to) {
  const int HKV = p.src.hkv, B = p.range.rows.B;
  int b = -1;
  page = g = 0;
  while (b0 < B) {
    int lo = 0, hi = 0;
    if (b0 + lane < B) key_range(p, b0 + lane, lo, hi, p.err);
    const int n = hi > lo ? (((hi - 1) >> 4) - (lo >> 4) + 1) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const long long first = base + (long long)(incl - n) * HKV, last = base + (long long)incl * HKV;
    const unsigned m = __ballot_sync(0xffffffffu, unit >= first && unit < last);
    if (m) {
      const int s = __ffs(m) - 1;
      const long long off = unit - __shfl_sync(0xffffffffu, first, s);
      b = b0 + s;
      page = (__shfl_sync(0xffffffffu, lo, s) >> 4) + (int)(off / HKV);
      g = (int)(off % HKV);
      break;
    }
    base += (long long)__shfl_sync(0xffffffffu, incl, 31) * HKV;
    b0 += 32;
  }
  if (b < 0) return -1;
  key_range(p, b, lo, hi, p.err);
  from = p.src.page_table[(size_t)b * p.src.max_pages + page];
  to = p.dst.page_table[(size_t)b * p.dst.max_pages + page];
  if (from < 0 || from >= p.src.num_pages || to < 0 || to >= p.dst.num_pages) {
    if (lane == 0) set_error(p.err, kErrPage);
    return 0;
  }
  return 1;
}

}  // namespace g4
