// The 8-bit paged cache's append and read-back, and the page eviction (see g4_kv8.cuh for the layout
// and the cast).
#include "g4_kv8.cuh"

namespace g4 {

namespace {

// ---- append: rows -> 8-bit pages ---------------------------------------------------------------------
// D/16 lanes hold a head vector, 8 half-split pairs each (columns t0 .. t0+7 and D/2 + t0 .. +7), so
// loads are 16 bytes a lane and the vector's largest |x| is one warp reduction.
template <int D>
struct Vec {
  float a[8], b[8];   // columns t0 + i and D/2 + t0 + i
};

template <int D>
G4_DEV Vec<D> load_vec(const __nv_bfloat16* __restrict__ src, int t0) {
  const uint4 lo = *reinterpret_cast<const uint4*>(src + t0);
  const uint4 hi = *reinterpret_cast<const uint4*>(src + D / 2 + t0);
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

// x / sqrt(mean(x^2) + eps), over the D/16 lanes of the vector.
template <int D>
G4_DEV void unit_norm(Vec<D>& v, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v.a[i], v.a[i], ss);
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v.b[i], v.b[i], ss);
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = __frsqrt_rn(fmaf(ss, 1.0f / (float)D, eps));   // ss / D is exact: D is a power of 2
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.a[i] *= inv;
    v.b[i] *= inv;
  }
}

template <int D>
G4_DEV void weight(Vec<D>& v, const __nv_bfloat16* __restrict__ w, int t0) {
  const Vec<D> m = load_vec<D>(w, t0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.a[i] *= m.a[i];
    v.b[i] *= m.b[i];
  }
}

// The largest |x| bits over the lanes of `mask` (all of which call it).
template <int D>
G4_DEV uint32_t max_bits(const Vec<D>& v, unsigned mask) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m = max(m, max(__float_as_uint(v.a[i]) & 0x7fffffffu, __float_as_uint(v.b[i]) & 0x7fffffffu));
  return __reduce_max_sync(mask, m);
}

// Stores the vector as key j of a tile; col_b: the tile column of b[0].
template <int D>
G4_DEV void store_vec(uint8_t* tile, uint8_t* exps, int j, const Vec<D>& v, int t0, int col_b, unsigned mask) {
  const uint32_t e = kv8_exponent(max_bits<D>(v, mask));
  *reinterpret_cast<uint2*>(tile + kv8_offset(j, t0)) = kv8_codes(v.a, e);
  *reinterpret_cast<uint2*>(tile + kv8_offset(j, col_b)) = kv8_codes(v.b, e);
  if (t0 == 0) exps[j] = (uint8_t)e;
}

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  // rows of a prefill (MODE 0), or one new token per request at held index seq_len - 1 (MODE 1)
  SeqRows rows;
  const int32_t* seq_len;
  const int32_t* pos;   // MODE 1: RoPE position of the new token; NULL: its held index
  PagedCache8 cache;
  RopeTables tb;
  uint32_t* err;
  NormArgs nm;
  int parts;   // warps per row
};

// Sequence b of a prefill batch is refused (none of its rows is read or written) when its rows do
// not lie inside the T rows of the call or its positions inside [0, 262144).
G4_DEV bool rows_ok(const SeqRows& r, int qs, int L, int cs) {
  return qs >= 0 && L <= r.T - qs && cs >= 0 && L <= kMaxPos && cs <= kMaxPos - L;
}

// One warp per (row, share of the KV heads). D/16 lanes per vector: two heads at a time when D = 256.
template <bool GLOBAL, bool NORM, int MODE>
__global__ void __launch_bounds__(256) kv8_append_kernel(const AppendArgs p) {
  using Blk = Kv8Block<GLOBAL>;
  constexpr int D = Blk::D, R = Blk::R, LPV = D / 16, VPW = 32 / LPV;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int n_rows = MODE == 0 ? p.rows.T : p.rows.B;
  const long long r64 = unit / p.parts;
  if (r64 >= n_rows) return;
  const int r = (int)r64, part = (int)(unit % p.parts);

  int b = r, idx, pos;   // sequence, held index and RoPE position of the row's token
  if (MODE == 0) {
    int owner = -1;
    for (int b0 = 0; b0 < p.rows.B; b0 += 32) {
      const int i = b0 + lane;
      bool mine = false;
      if (i < p.rows.B) {
        const int qs = p.rows.q_start[i], L = p.rows.q_len[i];
        if (L > 0) {
          const bool ok = rows_ok(p.rows, qs, L, p.rows.ctx_start[i]);
          if (!ok && unit == 0) set_error(p.err, kErrPos);
          mine = ok && r >= qs && r - qs < L;
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, mine);
      if (m && owner < 0) owner = b0 + __ffs(m) - 1;
      if (owner >= 0 && unit != 0) break;   // warp 0 looks at every sequence, for its error
    }
    if (owner < 0) return;
    b = owner;
    idx = p.rows.ctx_start[b] + (r - p.rows.q_start[b]);
    pos = idx;
  } else {
    idx = p.seq_len[b] - 1;
    pos = p.pos ? p.pos[b] : idx;
  }
  if (idx < 0 || idx >= kMaxPos || (idx >> 4) >= p.cache.max_pages || pos < idx || pos >= kMaxPos) {
    if (lane == 0) set_error(p.err, kErrPos);
    return;
  }
  const int phys = p.cache.page_table[(size_t)b * p.cache.max_pages + (idx >> 4)];
  if (phys < 0 || phys >= p.cache.num_pages) {
    if (lane == 0) set_error(p.err, kErrPage);
    return;
  }
  const int j = idx & 15;
  const int t0 = (lane % LPV) * 8;
  float2 cs[8];
  if (t0 < R) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = rope_cs(p.tb, t0 + i, pos);
  }
  const unsigned vec_mask = LPV == 32 ? 0xffffffffu : (0xffffu << (lane & 16));
  const int HKV = p.cache.hkv;
  const int per = (HKV + p.parts - 1) / p.parts;   // parts divides HKV / VPW, so this is exact
  uint8_t* page = p.cache.pages + (size_t)phys * HKV * Blk::kBytes;
#pragma unroll 2
  for (int g0 = part * per; g0 < (part + 1) * per; g0 += VPW) {
    const int g = g0 + lane / LPV;
    uint8_t* blk = page + (size_t)g * Blk::kBytes;
    const size_t src = ((size_t)r * HKV + g) * D;
    Vec<D> k = load_vec<D>(p.k + src, t0);
    if (GLOBAL) {   // S as given (or n(S)), and the turned columns of K
      if (NORM && p.nm.v_norm) unit_norm<D>(k, p.nm.eps);
      store_vec<D>(blk, blk + Blk::kExp0, j, k, t0, D / 2 + t0, 0xffffffffu);
      if (t0 < R) {
        if (NORM && p.nm.wk) weight<D>(k, p.nm.wk, t0);
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_pair(k.a[i], k.b[i], cs[i]);
        store_vec<D>(blk + Blk::kTile1, blk + Blk::kExp1, j, k, t0, R + t0, 0xffu);
      }
      __syncwarp();
    } else {
      Vec<D> v = load_vec<D>(p.v + src, t0);
      if (NORM && p.nm.wk) {
        unit_norm<D>(k, p.nm.eps);
        weight<D>(k, p.nm.wk, t0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_pair(k.a[i], k.b[i], cs[i]);
      store_vec<D>(blk, blk + Blk::kExp0, j, k, t0, D / 2 + t0, vec_mask);
      if (NORM && p.nm.v_norm) unit_norm<D>(v, p.nm.eps);
      store_vec<D>(blk + Blk::kTile1, blk + Blk::kExp1, j, v, t0, D / 2 + t0, vec_mask);
    }
  }
}

// ---- read-back: 8-bit pages -> bf16 pages --------------------------------------------------------------
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
  }
}

// Sixteen stored bytes (one key's piece) as 16 bf16 values, in column order.
G4_DEV void piece_bf16(const uint4& raw, float step, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)   // 2^23 + byte as a float, minus 2^23 + 128
      f[e] = (__uint_as_float(__byte_perm(w[i], 0x4b000000u, 0x7650 + e)) - 8388736.0f) * step;
    o[2 * i] = pack_bf16(f[0], f[1]);
    o[2 * i + 1] = pack_bf16(f[2], f[3]);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One warp per (page, KV head), walking the batch's pages in a grid-sized stride. Lane (key kk = lane
// & 7, piece p = lane >> 3) turns 16 columns into two core-matrix rows, so a warp store fills four
// whole 128-byte core matrices.
template <bool GLOBAL>
__global__ void __launch_bounds__(256) kv8_unpack_kernel(const UnpackArgs p) {
  using Blk = Kv8Block<GLOBAL>;
  constexpr int D = Blk::D;
  const int lane = threadIdx.x & 31;
  const int HKV = p.src.hkv;
  const long long stride = (long long)gridDim.x * 8;
  const int B = p.range.rows.B;
  // A prefill's attention multiplies the slots before a window's first key, in its page, by zero: they
  // are set to zero, since anything else might not be a number.
  const bool zero_before = p.range.key_begin == nullptr;
  long long base = 0;   // units before sequence group b0
  int b0 = 0;
  for (long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);; unit += stride) {
    // find (sequence, logical page, head) of this unit, from where the last one was found
    int b = -1, page = 0, g = 0;
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
    if (b < 0) return;
    int lo, hi;
    key_range(p, b, lo, hi, p.err);
    const int from = p.src.page_table[(size_t)b * p.src.max_pages + page];
    const int to = p.dst.page_table[(size_t)b * p.dst.max_pages + page];
    if (from < 0 || from >= p.src.num_pages || to < 0 || to >= p.dst.num_pages) {
      if (lane == 0) set_error(p.err, kErrPage);
      continue;
    }
    const uint8_t* blk = p.src.pages + ((size_t)from * HKV + g) * Blk::kBytes;
    const size_t out = (size_t)to * HKV + g;
    __nv_bfloat16* k16 = (__nv_bfloat16*)p.dst.k + out * kPage * D;
    __nv_bfloat16* v16 = GLOBAL ? (__nv_bfloat16*)p.dst.krot + out * kRotPageElems
                                : (__nv_bfloat16*)p.dst.v + out * kPage * D;
    const int kk = lane & 7, pc = lane >> 3;
#pragma unroll
    for (int jg = 0; jg < 2; ++jg) {
      const int j = jg * 8 + kk, key = page * kPage + j;
      if (key >= hi || (key < lo && !zero_before)) continue;
      const float s0 = key < lo ? 0.f : kv8_step(blk[Blk::kExp0 + j]);
      const float s1 = key < lo ? 0.f : kv8_step(blk[Blk::kExp1 + j]);
      uint4 raw[D / 64];
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        raw[i] = *reinterpret_cast<const uint4*>(blk + kv8_offset(j, 16 * (pc + 4 * i)));
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int d = 16 * (pc + 4 * i);
        uint4 l, h;
        piece_bf16(raw[i], s0, l, h);
        *reinterpret_cast<uint4*>(k16 + tiled_offset(j, d, D)) = l;
        *reinterpret_cast<uint4*>(k16 + tiled_offset(j, d + 8, D)) = h;
      }
#pragma unroll
      for (int i = 0; i < Blk::kCols1 / 64; ++i)
        raw[i] = *reinterpret_cast<const uint4*>(blk + Blk::kTile1 + kv8_offset(j, 16 * (pc + 4 * i)));
#pragma unroll
      for (int i = 0; i < Blk::kCols1 / 64; ++i) {
        const int d = 16 * (pc + 4 * i);
        uint4 l, h;
        piece_bf16(raw[i], s1, l, h);
        if (GLOBAL) {   // tile 1 holds the turned columns 0 .. 63 and 256 .. 319
          const int col = d < kGlobalR ? d : D / 2 + d - kGlobalR;
          *reinterpret_cast<uint4*>(v16 + rot_offset(j, col)) = l;
          *reinterpret_cast<uint4*>(v16 + rot_offset(j, col + 8)) = h;
        } else {
          *reinterpret_cast<uint4*>(v16 + tiled_offset_v256(j, d)) = l;
          *reinterpret_cast<uint4*>(v16 + tiled_offset_v256(j, d + 8)) = h;
        }
      }
    }
  }
}

// ---- eviction: keep the first, the last and the heaviest pages ------------------------------------------
// One block per sequence; its table row and weights stay in shared memory, so the outputs may be the
// inputs. The n - keep lightest evictable pages leave: a radix select over the weights' ordered bits
// (four passes of 8 bits) finds the weight of the last one to leave, T, and how many pages of weight
// T leave; those are the first ones in index order. A block-wide scan then gives every page its place.
constexpr int kEvictThreads = 1024;

G4_DEV uint32_t ordered_bits(float w) {   // unsigned order = the order of the floats; NaN above all, or below if negative
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of one int per thread; *total gets the sum. sums: 32 ints.
G4_DEV int block_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();   // sums may still be read from an earlier scan
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int s = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += up;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return incl - x + (warp > 0 ? before : 0);
}

struct EvictArgs {
  const int32_t* seq_len;
  const int32_t* table;
  const float* weights;
  int max_pages, keep, first, last;
  int32_t* out_len;
  int32_t* out_table;
  float* out_weights;
  int32_t* freed;
  int32_t* n_freed;
  uint32_t* err;
};

__global__ void __launch_bounds__(kEvictThreads) evict_pages_kernel(const EvictArgs p) {
  extern __shared__ uint8_t smem[];
  float* w = reinterpret_cast<float*>(smem);                   // [max_pages]
  int32_t* tab = reinterpret_cast<int32_t*>(w + p.max_pages);  // [max_pages]
  __shared__ int hist[256];
  __shared__ int sums[32];
  __shared__ uint32_t sel_prefix;
  __shared__ int sel_left;
  const int b = blockIdx.x, tid = threadIdx.x;
  const size_t row = (size_t)b * p.max_pages;
  const int len = p.seq_len[b];
  int n = 0;
  if (len < 0 || len > kMaxPos || ((len + kPage - 1) >> 4) > p.max_pages) {
    if (tid == 0) set_error(p.err, kErrPos);   // the row is passed on as it is
    n = p.max_pages;
  } else {
    n = (len + kPage - 1) >> 4;
  }
  const bool bad = len < 0 || len > kMaxPos || ((len + kPage - 1) >> 4) > p.max_pages;
  const int drop = bad ? 0 : max(0, n - p.keep);
  for (int i = tid; i < n; i += kEvictThreads) {
    w[i] = p.weights[row + i];
    tab[i] = p.table[row + i];
  }
  if (tid == 0) {
    sel_prefix = 0;
    sel_left = drop;
  }
  __syncthreads();
  const int e0 = p.first, e1 = n - p.last;   // evictable pages [e0, e1); drop <= e1 - e0 since keep >= first + last
  if (drop > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = sel_prefix;
      for (int i = e0 + tid; i < e1; i += kEvictThreads) {
        const uint32_t u = ordered_bits(w[i]);
        // counting is exact in any order: these atomics decide nothing
        if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(u >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = sel_left, d = 0;
        while (left > hist[d]) left -= hist[d++];
        sel_left = left;
        sel_prefix = prefix | ((uint32_t)d << shift);
      }
      __syncthreads();
    }
  }
  const uint32_t T = sel_prefix;   // pages below T leave, and the first `ties` of weight T
  const int ties = sel_left;
  int out_base = 0, tie_base = 0, ev_base = 0;
  for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
    const int i = i0 + tid;
    bool lower = false, tie = false;
    if (drop > 0 && i >= e0 && i < e1) {
      const uint32_t u = ordered_bits(w[i]);
      lower = u < T;
      tie = u == T;
    }
    int total;
    const int t = tie_base + block_scan(tie ? 1 : 0, sums, &total);
    tie_base += total;
    const bool leaves = lower || (tie && t < ties);
    const int ev = ev_base + block_scan(leaves ? 1 : 0, sums, &total);
    if (i < n) {
      if (leaves) {
        p.freed[row + ev] = tab[i];
      } else {
        const int to = out_base + tid - (ev - ev_base);
        p.out_table[row + to] = tab[i];
        p.out_weights[row + to] = w[i];
      }
    }
    ev_base += total;
    out_base += min(kEvictThreads, n - i0) - total;
  }
  const int kept = n - drop;
  for (int i = kept + tid; i < p.max_pages; i += kEvictThreads) {
    p.out_table[row + i] = -1;
    p.out_weights[row + i] = 0.f;
  }
  for (int i = drop + tid; i < p.max_pages; i += kEvictThreads) p.freed[row + i] = -1;
  if (tid == 0) {
    p.out_len[b] = bad ? len : len - kPage * drop;
    p.n_freed[b] = drop;
  }
}

// Raises the kernel's dynamic shared-memory limit once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <bool GLOBAL, int MODE>
cudaError_t append(AppendArgs& a, int n_rows, cudaStream_t s) {
  constexpr int VPW = 32 / (Kv8Block<GLOBAL>::D / 16);
  a.parts = a.cache.hkv / VPW;
  const long long blocks = ((long long)n_rows * a.parts + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.nm.any())
    kv8_append_kernel<GLOBAL, true, MODE><<<(unsigned)blocks, 256, 0, s>>>(a);
  else
    kv8_append_kernel<GLOBAL, false, MODE><<<(unsigned)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(bool global, const void* k, const void* v, const SeqRows& rows, const PagedCache8& cache,
                              const NormArgs& nm, const DeviceState& st, cudaStream_t s) {
  if (rows.T <= 0 || rows.B <= 0) return cudaSuccess;
  AppendArgs a{(const __nv_bfloat16*)k, (const __nv_bfloat16*)v, rows, nullptr, nullptr, cache,
               global ? st.global : st.sliding, st.err, nm, 1};
  return global ? append<true, 0>(a, rows.T, s) : append<false, 0>(a, rows.T, s);
}

cudaError_t launch_kv8_append_decode(bool global, const void* k_new, const void* v_new, const int32_t* seq_len,
                                     const int32_t* pos, int B, const PagedCache8& cache, const NormArgs& nm,
                                     const DeviceState& st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  SeqRows rows{nullptr, nullptr, nullptr, B, B};
  AppendArgs a{(const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, rows, seq_len, pos, cache,
               global ? st.global : st.sliding, st.err, nm, 1};
  return global ? append<true, 1>(a, B, s) : append<false, 1>(a, B, s);
}

cudaError_t launch_kv8_unpack(bool global, const Kv8Range& range, const PagedCache8& src, const PagedCache& dst,
                              const DeviceState& st, cudaStream_t s) {
  if (range.rows.B <= 0) return cudaSuccess;
  UnpackArgs a{range, src, dst, st.err};
  const long long units = (long long)range.rows.B * src.max_pages * src.hkv;   // at most
  const unsigned blocks = (unsigned)(units + 7 < 8LL * 152 * 8 ? (units + 7) / 8 : 152 * 8);
  if (global)
    kv8_unpack_kernel<true><<<blocks, 256, 0, s>>>(a);
  else
    kv8_unpack_kernel<false><<<blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict_pages(const int32_t* seq_len, const int32_t* table, const float* weights, int B, int max_pages,
                               int keep, int first, int last, int32_t* out_len, int32_t* out_table, float* out_weights,
                               int32_t* freed, int32_t* n_freed, const DeviceState& st, cudaStream_t s) {
  static bool done[64] = {};
  const int bytes = max_pages * 8;
  cudaError_t e = allow_smem(evict_pages_kernel, kMaxPos / kPage * 8, done);
  if (e != cudaSuccess) return e;
  EvictArgs a{seq_len, table, weights, max_pages, keep, first, last, out_len, out_table, out_weights, freed, n_freed,
              st.err};
  evict_pages_kernel<<<B, kEvictThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace g4
