// The 4-bit paged cache's append and read-back (see g4_kv4.cuh for the layout and the cast).
#include "g4_kv4.cuh"
#include "g4_kv_rows.cuh"

namespace g4 {

namespace {

// ---- append: rows -> 4-bit pages ---------------------------------------------------------------------
// A lane holds 8 + 8 columns of a head vector (Vec); the four lanes of a block agree on its scale by two shuffles.
// Their codes are two bytes of two pieces each, so a vector's line is put together in shared memory and leaves in
// 8-byte stores that fill it whole.

// The largest |x| of eight columns, as bits; a NaN wins.
G4_DEV uint32_t max8(const float (&x)[8]) {
  const float a = max_abs(max_abs(fabsf(x[0]), x[1]), max_abs(fabsf(x[2]), x[3]));
  const float b = max_abs(max_abs(fabsf(x[4]), x[5]), max_abs(fabsf(x[6]), x[7]));
  return __float_as_uint(max_abs(a, b));
}

G4_DEV uint32_t max4lanes(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// One vector's bytes on their way out: its line (128 bytes per 256 columns; 64 of the turned columns), its scales.
struct __align__(16) Line {
  uint8_t bytes[256];
  uint8_t scales[16];
  uint8_t top;
};

// Quantises a vector held by the lanes of `mask` (all lanes of the warp call it, two or four vectors at a time) and
// puts its bytes into `line`. TURNED: 8 lanes hold the 128 turned columns; else D / 16 lanes hold all of them. i: the
// lane within its vector.
template <int D, bool TURNED>
G4_DEV void quantise(const Vec<D>& v, Line* line, int i, unsigned mask) {
  const uint32_t ma = max4lanes(max8(v.a)), mb = max4lanes(max8(v.b));
  const uint32_t m = __reduce_max_sync(mask, max(ma, mb));
  const bool bad = m >= 0x7f800000u;
  const uint32_t sa = bad ? 255u : kv4_scale(ma), sb = bad ? 255u : kv4_scale(mb);
  const uint32_t wa = kv4_codes(v.a, sa), wb = kv4_codes(v.b, sb);
  const int blk = i >> 2, q = i & 3;   // this lane's block of each part, its eight columns there
  int at_a, at_b, n;                   // offsets of the first two bytes; blocks per part
  if (TURNED) {
    n = 2;
    at_a = (2 * (q & 1)) * 16 + blk * 4 + (q >> 1) * 2;
    at_b = at_a + n * 4;
  } else if (D == 256) {
    n = 4;
    at_a = 2 * q * 16 + blk * 2;
    at_b = at_a + n * 2;
  } else {
    n = 8;
    at_a = 2 * q * 16 + blk * 2;
    at_b = at_a + 128;   // the other segment
  }
  *reinterpret_cast<uint16_t*>(line->bytes + at_a) = (uint16_t)wa;
  *reinterpret_cast<uint16_t*>(line->bytes + at_a + 16) = (uint16_t)(wa >> 16);
  *reinterpret_cast<uint16_t*>(line->bytes + at_b) = (uint16_t)wb;
  *reinterpret_cast<uint16_t*>(line->bytes + at_b + 16) = (uint16_t)(wb >> 16);
  if (q == 0) {
    line->scales[blk] = (uint8_t)sa;
    line->scales[n + blk] = (uint8_t)sb;
  }
  if (i == 0) line->top = (uint8_t)(bad ? 255u : kv4_scale(m));
}

// Stores a line as key j of a tile. Every lane of the vector takes eight bytes.
template <int D, bool TURNED>
G4_DEV void store_line(const Line* line, uint8_t* tile, uint8_t* scales, uint8_t* top, int j, int i) {
  constexpr int kScales = TURNED ? 4 : D / 32;
  const int off = TURNED ? kv4_turned_piece(j, i >> 1) + (i & 1) * 8 : kv4_piece(i >> 4, j, (i & 15) >> 1) + (i & 1) * 8;
  *reinterpret_cast<uint2*>(tile + off) = *reinterpret_cast<const uint2*>(line->bytes + i * 8);
  if (i < kScales / 4)
    *reinterpret_cast<uint32_t*>(scales + j * kScales + i * 4) = *reinterpret_cast<const uint32_t*>(line->scales + i * 4);
  if (top && i == 7) top[j] = line->top;
}

// A sliding row's heads arrive through shared memory, two heads of K' and V (64 bytes a lane) to a stage, one stage ahead
// of their use: a warp that held them in registers had its loads in flight for the codes' arithmetic alone, and waited
// for them (4 x 4096 rows: 85 us, 70 so; two stages ahead 2.8 more).
constexpr int kAhead = 1, kAppendStages = kAhead + 1;
// A warp a block: it leaves its place to the next row by itself (96 and 200 rows with their read-back: 10.0 us in a graph,
// blocks of four warps 11.6; 4 x 4096: 120.1 and 122.5; 28 blocks an SM, of 72 registers, 125.6).
constexpr int kAppendWarps = 1, kAppendBlocks = 24;

G4_DEV void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
G4_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
G4_DEV void copies_wait() {   // until all but the latest N groups of this thread have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  // rows of a prefill (MODE 0), or one new token per request at held index seq_len - 1 (MODE 1)
  SeqRows rows;
  const int32_t* seq_len;
  const int32_t* pos;   // MODE 1: RoPE position of the new token; NULL: its held index
  PagedCache4 cache;
  Kv8Angles angles;
  uint32_t* err;
  NormArgs nm;
  int parts;   // warps per row
};

// One warp per (row, share of the KV heads). The row's angles are computed once for its heads, in two-part
// arithmetic. Sliding: half a warp per vector, two heads at a time, K' then V. Global: a warp per head for S, then
// 8 lanes per head for the turned columns of up to four heads at once.
// The 4 x 4096 sliding rows take 70 us with cold caches in blocks of four warps (340 MB, 4.8 TB/s, 72% of the copy rate; the
// ALU pipe 55%, 2.9 instructions a cycle) and 68 in blocks of one; the 2 x 8192 global ones 29 (89 MB, 3.0 TB/s, DRAM 30%
// busy, 2.4 instructions a cycle, long-scoreboard stalls of 1.8 an issue: a row's loads are issued once, before its place is
// known) and 24 with the rows in L2. A decode step's token (one row a request) adds 2.1 us to a lone step of 37 keys.
template <bool GLOBAL, bool NORM, int MODE>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendBlocks) kv4_append_kernel(const AppendArgs p) {
  using Blk = Kv4Block<GLOBAL>;
  constexpr int D = Blk::D, R = Blk::R, LPV = D / 16;
  __shared__ __align__(16) float2 angles[kAppendWarps][R];
  __shared__ Line lines[kAppendWarps][4];
  __shared__ __align__(16) uint8_t staged[GLOBAL ? 16 : kAppendWarps * kAppendStages * 2048];   // [warp][stage][4][32 lanes][16]
  wait_for_grid();
  let_next_grid_start();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int n_rows = MODE == 0 ? p.rows.T : p.rows.B;
  const long long r64 = unit / p.parts;
  if (r64 >= n_rows) return;
  const int r = (int)r64, part = (int)(unit % p.parts);

  const int HKV = p.cache.hkv, per = HKV / p.parts, g_lo = part * per, g_hi = g_lo + per;
  const int t0 = (lane % LPV) * 8;       // this lane's pairs t0 .. t0 + 7
  const int tr = (lane % (R / 8)) * 8;   // and its turning ones (sliding: the same)
  const __nv_bfloat16* k_row = p.k + (size_t)r * HKV * D;
  const __nv_bfloat16* v_row = GLOBAL ? nullptr : p.v + (size_t)r * HKV * D;
  // The row's loads are in flight while its sequence, page and angles are looked up: all of a global row's (four heads
  // at most, and the turned columns again, 8 lanes a head), the first stages of a sliding one.
  Raw raw[4], raw_turned;
  uint8_t* stage = staged + (threadIdx.x >> 5) * kAppendStages * 2048 + lane * 16;   // a lane reads what it copied
  auto fetch = [&](int n) {   // sliding: heads g_lo + 2n + {0, 1}, half a warp each
    const int g = g_lo + 2 * n + lane / LPV;
    if (g < g_hi) {
      const uint32_t to = smem_u32(stage + n % kAppendStages * 2048);
      const __nv_bfloat16 *k = k_row + (size_t)g * D + t0, *v = v_row + (size_t)g * D + t0;
      copy16(to, k);
      copy16(to + 512, k + D / 2);
      copy16(to + 1024, v);
      copy16(to + 1536, v + D / 2);
    }
    copies_commit();
  };
  if (GLOBAL) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) raw[i] = load_raw<D>(k_row + (size_t)(g_lo + i) * D, t0);
    if ((lane >> 3) < per) raw_turned = load_raw<D>(k_row + (size_t)(g_lo + (lane >> 3)) * D, tr);
  } else {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) fetch(n);
  }

  int idx, pos, phys;
  if (!token_place<MODE>(p.rows, p.seq_len, p.pos, p.cache, p.err, r, unit == 0, lane, idx, pos, phys, true)) {
    if (!GLOBAL) copies_wait<0>();
    return;
  }
  const int j = idx & 15;
  uint8_t* page = p.cache.pages + (size_t)phys * HKV * Blk::kBytes;
  float2 cs[8];
  row_angles<R>(p.angles, pos, lane, angles[threadIdx.x >> 5], tr, cs);
  Line* line = lines[threadIdx.x >> 5];
  if (GLOBAL) {
    Norm norm[4];   // of each head
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= per) break;
      Vec<D> k = widen<D>(raw[i]);
      if (NORM && p.nm.v_norm) {
        norm[i] = norm_of<D>(k, p.nm.eps);
        divide<D>(k, norm[i]);
      }
      quantise<D, false>(k, line + i, lane, 0xffffffffu);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= per) break;
      uint8_t* blk = page + (size_t)(g_lo + i) * Blk::kBytes;
      store_line<D, false>(line + i, blk, blk + Blk::kScale0, blk + Blk::kTop, j, lane);
    }
    __syncwarp();
    const int i = lane >> 3;   // the turned columns of head g_lo + i
    Vec<D> k = widen<D>(i < per ? raw_turned : Raw{});
    if (NORM && i < per) {
      if (p.nm.v_norm) divide<D>(k, i == 0 ? norm[0] : i == 1 ? norm[1] : i == 2 ? norm[2] : norm[3]);
      if (p.nm.wk) weight<D>(k, p.nm.wk, tr);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) rope_pair_apart(k.a[e], k.b[e], cs[e]);
    quantise<D, true>(k, line + i, lane & 7, 0xffu << (lane & 24));
    __syncwarp();
    if (i < per) {
      uint8_t* blk = page + (size_t)(g_lo + i) * Blk::kBytes;
      store_line<D, true>(line + i, blk + Blk::kTile1, blk + Blk::kScale1, nullptr, j, lane & 7);
    }
  } else {
    const unsigned mask = 0xffffu << (lane & 16);
    Line* mine = line + 2 * (lane >> 4);
#pragma unroll 1
    for (int n = 0; 2 * n < per; ++n) {
      const int g = g_lo + 2 * n + lane / LPV;
      uint8_t* blk = page + (size_t)g * Blk::kBytes;
      copies_wait<kAhead - 1>();
      const uint4* got = reinterpret_cast<const uint4*>(stage + n % kAppendStages * 2048);
      Vec<D> k = widen<D>(Raw{got[0], got[32]}), v = widen<D>(Raw{got[64], got[96]});
      fetch(n + kAhead);   // (into the stage that was read a turn ago)
      if (NORM && p.nm.wk) {
        divide<D>(k, norm_of<D>(k, p.nm.eps));
        weight<D>(k, p.nm.wk, t0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_pair_apart(k.a[i], k.b[i], cs[i]);
      quantise<D, false>(k, mine, lane & 15, mask);
      if (NORM && p.nm.v_norm) divide<D>(v, norm_of<D>(v, p.nm.eps));
      quantise<D, false>(v, mine + 1, lane & 15, mask);
      __syncwarp();
      store_line<D, false>(mine, blk, blk + Blk::kScale0, nullptr, j, lane & 15);
      store_line<D, false>(mine + 1, blk + Blk::kTile1, blk + Blk::kScale1, blk + Blk::kTop, j, lane & 15);
      __syncwarp();
    }
  }
}

// ---- read-back: 4-bit pages -> bf16 pages --------------------------------------------------------------
// Eight consecutive columns of one block, as two halves of a piece pair, in bf16.
G4_DEV uint4 eight_bf16(uint32_t lo16, uint32_t hi16, float factor) {
  uint32_t h[4], o[4];
  kv4_halves((lo16 & 0xffffu) | (hi16 << 16), h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    o[i] = pack_bf16(f.x * factor, f.y * factor);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Bound by its loads: the 4 x 4096 sliding rows take 54 us (56 with cold caches; 340 MB, 6.1 to 6.3 TB/s), the 2 x 8192
// global ones 17 with the pages in L2 and 19 with cold caches (106 MB, 5.7 TB/s). Blocks of four
// warps, eight an SM and two rounds of them: against blocks of eight warps, 0.5 us less for small calls, the same for large
// ones; blocks of one warp 1 us less for the large call and 6 more for 64 single rows, many warps looking for few pages.
constexpr int kUnpackWarps = 4, kUnpackBlocks = 8;

// One warp per (page, KV head), walking the batch's pages in a grid-sized stride. Lane (key kk = lane & 7, q = lane
// >> 3) turns columns 8q .. 8q + 7 of every block of its key into core-matrix rows, so a warp store fills four whole
// 128-byte core matrices.
template <bool GLOBAL>
__global__ void __launch_bounds__(kUnpackWarps * 32, kUnpackBlocks) kv4_unpack_kernel(const UnpackArgs p) {
  using Blk = Kv4Block<GLOBAL>;
  constexpr int D = Blk::D;
  wait_for_grid();
  let_next_grid_start();
  const int lane = threadIdx.x & 31;
  const int HKV = p.src.hkv;
  const long long stride = (long long)gridDim.x * kUnpackWarps;
  // A prefill's attention multiplies the slots before a window's first key, in its page, by zero: they
  // are set to zero, since anything else might not be a number.
  const bool zero_before = p.range.key_begin == nullptr;
  const int kk = lane & 7, q = lane >> 3;
  long long base = 0;   // units before sequence group b0
  int b0 = 0;
  for (long long unit = (long long)blockIdx.x * kUnpackWarps + (threadIdx.x >> 5);; unit += stride) {
    int lo, hi, page, g, from, to;
    const int found = find_page(p, unit, lane, base, b0, lo, hi, page, g, from, to);
    if (found < 0) return;
    if (found == 0) continue;
    const uint8_t* blk = p.src.pages + ((size_t)from * HKV + g) * Blk::kBytes;
    const size_t out = (size_t)to * HKV + g;
    __nv_bfloat16* k16 = (__nv_bfloat16*)p.dst.k + out * kPage * D;
    __nv_bfloat16* v16 = GLOBAL ? (__nv_bfloat16*)p.dst.krot + out * kRotPageElems
                                : (__nv_bfloat16*)p.dst.v + out * kPage * D;
#pragma unroll
    for (int jg = 0; jg < 2; ++jg) {
      const int j = jg * 8 + kk, key = page * kPage + j;
      if (key >= hi || (key < lo && !zero_before)) continue;
      const bool zero = key < lo;
      constexpr int kWide = GLOBAL ? 1 : 2;   // wide tiles
#pragma unroll
      for (int tile = 0; tile < kWide; ++tile) {
        const uint8_t* src = blk + (tile == 0 ? 0 : Blk::kTile1);
        const uint8_t* sc = blk + (tile == 0 ? Blk::kScale0 + j * Blk::kBlocks0 : Blk::kScale1 + j * Blk::kBlocks1);
#pragma unroll
        for (int sg = 0; sg < D / 256; ++sg) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + kv4_piece(sg, j, 2 * q));
          const uint4 y = *reinterpret_cast<const uint4*>(src + kv4_piece(sg, j, 2 * q + 1));
          const uint2 s8 = *reinterpret_cast<const uint2*>(sc + sg * 8);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t scale = ((b < 4 ? s8.x : s8.y) >> (8 * (b & 3))) & 255u;
            const int d = sg * 256 + b * 32 + q * 8;
            const uint4 o = zero ? make_uint4(0, 0, 0, 0)
                                 : eight_bf16(xw[b >> 1] >> (16 * (b & 1)), yw[b >> 1] >> (16 * (b & 1)), kv4_factor(scale));
            __nv_bfloat16* dst = tile == 0 ? k16 + tiled_offset(j, d, D) : v16 + tiled_offset_v256(j, d);
            *reinterpret_cast<uint4*>(dst) = o;
          }
        }
      }
      if (GLOBAL) {   // the turned columns 0 .. 63 and 256 .. 319
        const uint8_t* src = blk + Blk::kTile1;
        const uint4 x = *reinterpret_cast<const uint4*>(src + kv4_turned_piece(j, 2 * (q & 1)));
        const uint4 y = *reinterpret_cast<const uint4*>(src + kv4_turned_piece(j, 2 * (q & 1) + 1));
        const uint32_t s4 = *reinterpret_cast<const uint32_t*>(blk + Blk::kScale1 + j * 4);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int d = b * 32 + q * 8, col = d < kGlobalR ? d : D / 2 + d - kGlobalR;
          const uint4 o = zero ? make_uint4(0, 0, 0, 0)
                               : eight_bf16(xw[b] >> (16 * (q >> 1)), yw[b] >> (16 * (q >> 1)),
                                            kv4_factor((s4 >> (8 * b)) & 255u));
          *reinterpret_cast<uint4*>(v16 + rot_offset(j, col)) = o;
        }
      }
    }
  }
}

template <bool GLOBAL, int MODE>
cudaError_t append(AppendArgs& a, int n_rows, cudaStream_t s) {
  // One warp per row computes its angles once for all heads; with few rows the heads are shared out
  // so that about 32 warps run per SM (a row's bytes do not depend on it).
  const int most = a.cache.hkv / (GLOBAL ? 1 : 2);
  a.parts = 1;
  while (a.parts < most && (long long)n_rows * a.parts < 152 * 32) a.parts *= 2;
  const long long blocks = ((long long)n_rows * a.parts + kAppendWarps - 1) / kAppendWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.nm.any())
    return launch_early(kv4_append_kernel<GLOBAL, true, MODE>, (unsigned)blocks, kAppendWarps * 32, 0, s, a);
  return launch_early(kv4_append_kernel<GLOBAL, false, MODE>, (unsigned)blocks, kAppendWarps * 32, 0, s, a);
}

}  // namespace

cudaError_t launch_kv4_append(bool global, const void* k, const void* v, const SeqRows& rows, const PagedCache4& cache,
                              const NormArgs& nm, const DeviceState& st, cudaStream_t s) {
  if (rows.T <= 0 || rows.B <= 0) return cudaSuccess;
  AppendArgs a{(const __nv_bfloat16*)k, (const __nv_bfloat16*)v, rows, nullptr, nullptr, cache, {}, st.err, nm, 1};
  const cudaError_t e = kv8_angles(global, &a.angles);
  if (e != cudaSuccess) return e;
  return global ? append<true, 0>(a, rows.T, s) : append<false, 0>(a, rows.T, s);
}

cudaError_t launch_kv4_append_decode(bool global, const void* k_new, const void* v_new, const int32_t* seq_len,
                                     const int32_t* pos, int B, const PagedCache4& cache, const NormArgs& nm,
                                     const DeviceState& st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  SeqRows rows{nullptr, nullptr, nullptr, B, B};
  AppendArgs a{(const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, rows, seq_len, pos, cache, {}, st.err, nm, 1};
  const cudaError_t e = kv8_angles(global, &a.angles);
  if (e != cudaSuccess) return e;
  return global ? append<true, 1>(a, B, s) : append<false, 1>(a, B, s);
}

cudaError_t launch_kv4_unpack(bool global, const Kv8Range& range, const PagedCache4& src, const PagedCache& dst,
                              const DeviceState& st, cudaStream_t s) {
  if (range.rows.B <= 0) return cudaSuccess;
  UnpackArgs a{range, src, dst, st.err};
  const long long units = (long long)range.rows.B * src.max_pages * src.hkv;   // at most
  const long long some = (units + kUnpackWarps - 1) / kUnpackWarps;
  const unsigned blocks = (unsigned)(some < 152 * 2 * kUnpackBlocks ? some : 152 * 2 * kUnpackBlocks);
  return global ? launch_early(kv4_unpack_kernel<true>, blocks, kUnpackWarps * 32, 0, s, a)
                : launch_early(kv4_unpack_kernel<false>, blocks, kUnpackWarps * 32, 0, s, a);
}

}  // namespace g4
