// The 8-bit paged cache's append and read-back, and the page eviction (see g4_kv8.cuh for the layout
// and the cast).
#include <math.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "g4_kv8.cuh"
#include "g4_kv_rows.cuh"

namespace g4 {

static __device__ float4 g_kv8_coarse_sliding[kRopeCoarse * kSlidingR];
static __device__ float4 g_kv8_fine_sliding[256 * kSlidingR];
static __device__ float4 g_kv8_coarse_global[kRopeCoarse * kGlobalR];
static __device__ float4 g_kv8_fine_global[256 * kGlobalR];

namespace {

constexpr int kAngleDevices = 64;
std::mutex g_angles_mutex;
std::atomic<bool> g_angles_ready[kAngleDevices][2];   // per device and layer kind
Kv8Angles g_angles[kAngleDevices][2];

// The table of angles (step i) f_t, i < entries, in two fp32 parts (computed in fp64).
std::vector<float4> angle_table(int entries, double step, int D, int R, double theta) {
  std::vector<float4> h((size_t)entries * R);
  for (int t = 0; t < R; ++t) {
    const double f = pow(theta, -2.0 * t / (double)D);
    for (int i = 0; i < entries; ++i) {
      const double c = cos((step * i) * f), s = sin((step * i) * f);
      const float ch = (float)c, sh = (float)s;
      h[(size_t)i * R + t] = make_float4(ch, sh, (float)(c - ch), (float)(s - sh));
    }
  }
  return h;
}

// Copies a layer kind's tables to the current device, on a stream of its own: the call that needs them may
// be part of a capture, which must neither record the copy nor be broken by it.
cudaError_t copy_tables(const void* coarse_symbol, const std::vector<float4>& coarse, const void* fine_symbol,
                        const std::vector<float4>& fine) {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return e;
  cudaStream_t s = nullptr;
  e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
  if (e == cudaSuccess) {
    e = cudaMemcpyToSymbolAsync(coarse_symbol, coarse.data(), coarse.size() * sizeof(float4), 0,
                                cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess)
      e = cudaMemcpyToSymbolAsync(fine_symbol, fine.data(), fine.size() * sizeof(float4), 0, cudaMemcpyHostToDevice, s);
    const cudaError_t done = cudaStreamSynchronize(s);   // before the host tables go
    if (e == cudaSuccess) e = done;
    cudaStreamDestroy(s);
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  return e;
}

cudaError_t upload_angles(int dev, bool global) {
  const void* coarse = global ? (const void*)g_kv8_coarse_global : (const void*)g_kv8_coarse_sliding;
  const void* fine = global ? (const void*)g_kv8_fine_global : (const void*)g_kv8_fine_sliding;
  const int D = global ? kGlobalD : kSlidingD, R = global ? kGlobalR : kSlidingR;
  const double theta = global ? 1.0e6 : 1.0e4;
  try {   // no exception leaves a C entry point
    const cudaError_t e = copy_tables(coarse, angle_table(kRopeCoarse, 256.0, D, R, theta), fine,
                                      angle_table(256, 1.0, D, R, theta));
    if (e != cudaSuccess) return e;
  } catch (...) {
    return cudaErrorMemoryAllocation;
  }
  void *c = nullptr, *f = nullptr;
  cudaError_t e;
  if ((e = cudaGetSymbolAddress(&c, coarse)) != cudaSuccess) return e;
  if ((e = cudaGetSymbolAddress(&f, fine)) != cudaSuccess) return e;
  g_angles[dev][global] = Kv8Angles{(const float4*)c, (const float4*)f};
  return cudaSuccess;
}

}  // namespace

cudaError_t kv8_angles(bool global, Kv8Angles* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kAngleDevices) return cudaErrorInvalidDevice;
  if (!g_angles_ready[dev][global].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_angles_mutex);
    if (!g_angles_ready[dev][global].load(std::memory_order_relaxed)) {
      if ((e = upload_angles(dev, global)) != cudaSuccess) return e;
      g_angles_ready[dev][global].store(true, std::memory_order_release);
    }
  }
  *out = g_angles[dev][global];
  return cudaSuccess;
}

namespace {

// ---- append: rows -> 8-bit pages ---------------------------------------------------------------------
// Stores the vector as key j of a tile (off_a, off_b: the offsets of columns t0 and of b[0] there); the lane
// of column 0 stores the exponent.
template <int D>
G4_DEV void store_vec(uint8_t* tile, uint32_t off_a, uint32_t off_b, uint8_t* exponent, const Vec<D>& v, bool first,
                      unsigned mask) {
  const uint32_t e = kv8_exponent(max_bits<D>(v, mask));
  *reinterpret_cast<uint2*>(tile + off_a) = kv8_codes(v.a, e);
  *reinterpret_cast<uint2*>(tile + off_b) = kv8_codes(v.b, e);
  if (first) *exponent = (uint8_t)e;
}

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  // rows of a prefill (MODE 0), or one new token per request at held index seq_len - 1 (MODE 1)
  SeqRows rows;
  const int32_t* seq_len;
  const int32_t* pos;   // MODE 1: RoPE position of the new token; NULL: its held index
  PagedCache8 cache;
  Kv8Angles angles;
  uint32_t* err;
  NormArgs nm;
  int parts;   // warps per row
};

// The 4 x 4096 sliding rows take 79 us (402 MB, 5.1 TB/s, 1.33 times the copy's time), the 2 x 8192 global ones
// 27 us (109 MB, 4 TB/s, 1.7 times). Neither memory nor issue (57%; the ALU pipe 55%) is full: 24 warps an SM
// wait for their loads and for each other's results by turns.
// One warp per (row, share of the KV heads). The row's angles are computed once for its heads, in two-part
// arithmetic. Sliding: half a warp per vector, two heads at a time, K' and V together. Global: a warp
// per head for S, then 8 lanes per head for the turned columns of up to four heads at once.
template <bool GLOBAL, bool NORM, int MODE>
__global__ void __launch_bounds__(256, 3) kv8_append_kernel(const AppendArgs p) {
  using Blk = Kv8Block<GLOBAL>;
  constexpr int D = Blk::D, R = Blk::R, LPV = D / 16;
  __shared__ __align__(16) float2 angles[8][R];
  wait_for_grid();
  let_next_grid_start();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int n_rows = MODE == 0 ? p.rows.T : p.rows.B;
  const long long r64 = unit / p.parts;
  if (r64 >= n_rows) return;
  const int r = (int)r64, part = (int)(unit % p.parts);

  const int HKV = p.cache.hkv, per = HKV / p.parts, g_lo = part * per, g_hi = g_lo + per;
  const int t0 = (lane % LPV) * 8;       // this lane's pairs t0 .. t0 + 7
  const int tr = (lane % (R / 8)) * 8;   // and its turning ones (sliding: the same)
  const __nv_bfloat16* k_row = p.k + (size_t)r * HKV * D;
  const __nv_bfloat16* v_row = GLOBAL ? nullptr : p.v + (size_t)r * HKV * D;
  // The row's loads are in flight while its sequence, page and angles are looked up: all of a global
  // row's (four heads at most, and the turned columns again, 8 lanes a head), the first two heads' of a
  // sliding one, whose others follow two heads ahead.
  Raw raw[4], raw_turned, raw_v;
  if (GLOBAL) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) raw[i] = load_raw<D>(k_row + (size_t)(g_lo + i) * D, t0);
    if ((lane >> 3) < per) raw_turned = load_raw<D>(k_row + (size_t)(g_lo + (lane >> 3)) * D, tr);
  } else {
    raw[0] = load_raw<D>(k_row + (size_t)(g_lo + lane / LPV) * D, t0);
    raw_v = load_raw<D>(v_row + (size_t)(g_lo + lane / LPV) * D, t0);
  }

  int idx, pos, phys;
  if (!token_place<MODE>(p.rows, p.seq_len, p.pos, p.cache, p.err, r, unit == 0, lane, idx, pos, phys)) return;
  const int j = idx & 15;
  uint8_t* page = p.cache.pages + (size_t)phys * HKV * Blk::kBytes;
  float2 cs[8];
  row_angles<R>(p.angles, pos, lane, angles[threadIdx.x >> 5], tr, cs);
  const uint32_t off_a = kv8_offset(j, t0), off_b = kv8_offset(j, D / 2 + t0);
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
      uint8_t* blk = page + (size_t)(g_lo + i) * Blk::kBytes;
      store_vec<D>(blk, off_a, off_b, blk + Blk::kExp0 + j, k, lane == 0, 0xffffffffu);
    }
    const int i = lane >> 3;   // the turned columns of head g_lo + i
    if (i < per) {
      Vec<D> k = widen<D>(raw_turned);
      if (NORM) {
        if (p.nm.v_norm) divide<D>(k, i == 0 ? norm[0] : i == 1 ? norm[1] : i == 2 ? norm[2] : norm[3]);
        if (p.nm.wk) weight<D>(k, p.nm.wk, tr);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) rope_pair_apart(k.a[e], k.b[e], cs[e]);
      uint8_t* blk = page + (size_t)(g_lo + i) * Blk::kBytes;
      store_vec<D>(blk + Blk::kTile1, kv8_offset(j, tr), kv8_offset(j, R + tr), blk + Blk::kExp1 + j, k, tr == 0,
                   0xffu << (lane & 24));
    }
  } else {
    const unsigned mask = 0xffffu << (lane & 16);
#pragma unroll 1
    for (int g0 = g_lo; g0 < g_hi; g0 += 2) {
      const int g = g0 + lane / LPV;
      uint8_t* blk = page + (size_t)g * Blk::kBytes;
      Vec<D> k = widen<D>(raw[0]), v = widen<D>(raw_v);
      if (g0 + 2 < g_hi) {
        raw[0] = load_raw<D>(k_row + (size_t)(g + 2) * D, t0);
        raw_v = load_raw<D>(v_row + (size_t)(g + 2) * D, t0);
      }
      if (NORM && p.nm.wk) {
        divide<D>(k, norm_of<D>(k, p.nm.eps));
        weight<D>(k, p.nm.wk, t0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_pair_apart(k.a[i], k.b[i], cs[i]);
      store_vec<D>(blk, off_a, off_b, blk + Blk::kExp0 + j, k, t0 == 0, mask);
      if (NORM && p.nm.v_norm) divide<D>(v, norm_of<D>(v, p.nm.eps));
      store_vec<D>(blk + Blk::kTile1, off_a, off_b, blk + Blk::kExp1 + j, v, t0 == 0, mask);
    }
  }
}

// ---- read-back: 8-bit pages -> bf16 pages --------------------------------------------------------------
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

// Bound by memory: the 4 x 4096 sliding rows take 61 us (403 MB, 6.6 TB/s).
// One warp per (page, KV head), walking the batch's pages in a grid-sized stride. Lane (key kk = lane
// & 7, piece p = lane >> 3) turns 16 columns into two core-matrix rows, so a warp store fills four
// whole 128-byte core matrices.
template <bool GLOBAL>
__global__ void __launch_bounds__(256) kv8_unpack_kernel(const UnpackArgs p) {
  using Blk = Kv8Block<GLOBAL>;
  constexpr int D = Blk::D;
  wait_for_grid();
  let_next_grid_start();
  const int lane = threadIdx.x & 31;
  const int HKV = p.src.hkv;
  const long long stride = (long long)gridDim.x * 8;
  // A prefill's attention multiplies the slots before a window's first key, in its page, by zero: they
  // are set to zero, since anything else might not be a number.
  const bool zero_before = p.range.key_begin == nullptr;
  long long base = 0;   // units before sequence group b0
  int b0 = 0;
  for (long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);; unit += stride) {
    int lo, hi, page, g, from, to;
    const int found = find_page(p, unit, lane, base, b0, lo, hi, page, g, from, to);
    if (found < 0) return;
    if (found == 0) continue;
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
// One block per sequence, warp w and lane l hold pages (w * ITEMS + i) * 32 + l, i < ITEMS, in registers, so
// the outputs may be the inputs. The n - keep lightest evictable pages leave. The weight T of the last
// one to leave is found bit by bit from the top: the number of keys below a candidate is a compare per
// key, a warp sum and one barrier, until it is exact. Of the pages of weight T the first in index order
// leave. Two block-wide scans of per-warp counts then give every page its place. Bound by the rounds of the
// search: 64 rows of up to 16384 pages take 18 us (21 with the search as a loop), 3 of 131 5 us.
G4_DEV uint32_t ordered_bits(float w) {   // unsigned order = the order of the floats; NaN above all
  const uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if ((u & 0x7fffffffu) == 0u) return 0x80000000u;   // -0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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

template <int ITEMS>
__global__ void __launch_bounds__(1024) evict_pages_kernel(const EvictArgs p) {
  __shared__ int counts[4][32];   // by bit parity; the ties; the leaving: none is written while it may be read
  wait_for_grid();
  let_next_grid_start();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const size_t row = (size_t)b * p.max_pages;
  const int base = warp * ITEMS * 32 + lane;
  float w[ITEMS];
  int32_t tab[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {   // of the whole row: entries past the sequence's pages are not used
    const int at = base + 32 * i;
    w[i] = at < p.max_pages ? p.weights[row + at] : 0.f;
    tab[i] = at < p.max_pages ? p.table[row + at] : -1;
  }
  const int len = p.seq_len[b];
  const bool bad = len < 0 || len > kMaxPos || ((len + kPage - 1) >> 4) > p.max_pages;
  const int n = bad ? p.max_pages : (len + kPage - 1) >> 4;   // a bad row is passed on as it is
  const int drop = bad ? 0 : max(0, n - p.keep);
  const int e0 = p.first, e1 = n - p.last;   // evictable pages [e0, e1): at least drop, as keep >= first + last
  // The sum over the block of one count per warp, in every thread.
  auto block_sum = [&](int x, int array) {
    if (lane == 0) counts[array][warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < n_warps ? counts[array][lane] : 0);
  };
  // Exclusive sum over the warps before this one.
  auto before = [&](int x, int array) {
    if (lane == 0) counts[array][warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? counts[array][lane] : 0);
  };
  uint32_t key[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = base + 32 * i;
    key[i] = at >= e0 && at < e1 ? ordered_bits(w[i]) : 0xffffffffu;
  }
  uint32_t T = 0;     // at last the drop-th smallest key, or any value with exactly drop keys below it
  int below = 0;      // keys below T
  if (drop > 0) {
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = T | (1u << bit);
      int x = 0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) x += key[i] < c ? 1 : 0;
      x = block_sum(__reduce_add_sync(0xffffffffu, x), bit & 1);
      if (x <= drop) {
        T = c;
        below = x;
      }
      if (x == drop) break;   // exactly the pages below T leave
    }
  }
  const int ties = drop - below;   // pages of weight T that leave
  unsigned tie_mask[ITEMS];
  int x = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = base + 32 * i;
    tie_mask[i] = __ballot_sync(0xffffffffu, drop > 0 && at >= e0 && at < e1 && key[i] == T);
    x += __popc(tie_mask[i]);
  }
  int tie = before(x, 2);
  const unsigned lower = (1u << lane) - 1u;
  unsigned leave[ITEMS];
  x = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const bool mine = (tie_mask[i] >> lane) & 1u;
    const int at = base + 32 * i;
    const bool out = drop > 0 && at >= e0 && at < e1 && (key[i] < T || (mine && tie + __popc(tie_mask[i] & lower) < ties));
    tie += __popc(tie_mask[i]);
    leave[i] = __ballot_sync(0xffffffffu, out);
    x += __popc(leave[i]);
  }
  int gone = before(x, 3);
  const int kept = n - drop;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = base + 32 * i;
    const int ev = gone + __popc(leave[i] & lower);   // evicted pages before this one
    gone += __popc(leave[i]);
    if (at < n) {
      if ((leave[i] >> lane) & 1u) {
        p.freed[row + ev] = tab[i];
      } else {
        p.out_table[row + at - ev] = tab[i];
        p.out_weights[row + at - ev] = w[i];
      }
    }
    if (at < p.max_pages) {   // what lies behind: none, none, no weight
      if (at >= kept) {
        p.out_table[row + at] = -1;
        p.out_weights[row + at] = 0.f;
      }
      if (at >= drop) p.freed[row + at] = -1;
    }
  }
  if (threadIdx.x == 0) {
    if (bad) set_error(p.err, kErrPos);
    p.out_len[b] = bad ? len : len - kPage * drop;
    p.n_freed[b] = drop;
  }
}

template <bool GLOBAL, int MODE>
cudaError_t append(AppendArgs& a, int n_rows, cudaStream_t s) {
  // One warp per row computes its angles once for all heads; with few rows the heads are shared out
  // so that about 32 warps run per SM (a row's bytes do not depend on it).
  const int most = a.cache.hkv / (GLOBAL ? 1 : 2);
  a.parts = 1;
  while (a.parts < most && (long long)n_rows * a.parts < 152 * 32) a.parts *= 2;
  const long long blocks = ((long long)n_rows * a.parts + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.nm.any())
    return launch_early(kv8_append_kernel<GLOBAL, true, MODE>, (unsigned)blocks, 256, 0, s, a);
  return launch_early(kv8_append_kernel<GLOBAL, false, MODE>, (unsigned)blocks, 256, 0, s, a);
}

}  // namespace

cudaError_t launch_kv8_append(bool global, const void* k, const void* v, const SeqRows& rows, const PagedCache8& cache,
                              const NormArgs& nm, const DeviceState& st, cudaStream_t s) {
  if (rows.T <= 0 || rows.B <= 0) return cudaSuccess;
  AppendArgs a{(const __nv_bfloat16*)k, (const __nv_bfloat16*)v, rows, nullptr, nullptr, cache, {}, st.err, nm, 1};
  const cudaError_t e = kv8_angles(global, &a.angles);
  if (e != cudaSuccess) return e;
  return global ? append<true, 0>(a, rows.T, s) : append<false, 0>(a, rows.T, s);
}

cudaError_t launch_kv8_append_decode(bool global, const void* k_new, const void* v_new, const int32_t* seq_len,
                                     const int32_t* pos, int B, const PagedCache8& cache, const NormArgs& nm,
                                     const DeviceState& st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  SeqRows rows{nullptr, nullptr, nullptr, B, B};
  AppendArgs a{(const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, rows, seq_len, pos, cache, {}, st.err, nm, 1};
  const cudaError_t e = kv8_angles(global, &a.angles);
  if (e != cudaSuccess) return e;
  return global ? append<true, 1>(a, B, s) : append<false, 1>(a, B, s);
}

cudaError_t launch_kv8_unpack(bool global, const Kv8Range& range, const PagedCache8& src, const PagedCache& dst,
                              const DeviceState& st, cudaStream_t s) {
  if (range.rows.B <= 0) return cudaSuccess;
  UnpackArgs a{range, src, dst, st.err};
  const long long units = (long long)range.rows.B * src.max_pages * src.hkv;   // at most
  const unsigned blocks = (unsigned)(units + 7 < 8LL * 152 * 8 ? (units + 7) / 8 : 152 * 8);
  return global ? launch_early(kv8_unpack_kernel<true>, blocks, 256, 0, s, a)
                : launch_early(kv8_unpack_kernel<false>, blocks, 256, 0, s, a);
}

cudaError_t launch_evict_pages(const int32_t* seq_len, const int32_t* table, const float* weights, int B, int max_pages,
                               int keep, int first, int last, int32_t* out_len, int32_t* out_table, float* out_weights,
                               int32_t* freed, int32_t* n_freed, const DeviceState& st, cudaStream_t s) {
  EvictArgs a{seq_len, table, weights, max_pages, keep, first, last, out_len, out_table, out_weights, freed, n_freed,
              st.err};
  // Few pages per thread while that keeps the block small (its barriers are what a short row costs).
  const int items = max_pages <= 1024 ? 2 : max_pages <= 4096 ? 4 : 16;
  const unsigned threads = (unsigned)((max_pages + 32 * items - 1) / (32 * items) * 32);
  return launch_early(items == 2   ? evict_pages_kernel<2>
                      : items == 4 ? evict_pages_kernel<4>
                                   : evict_pages_kernel<16>,
                      (unsigned)B, threads, 0, s, a);
}

}  // namespace g4
