// Decode over the 8-bit paged cache: one query token per request, its keys split into fixed chunks (512
// keys on sliding layers, 1024 on global ones, aligned to key 0); inside a chunk page i goes to warp i % 4
// and the warps' states merge in warp order, and the chunks' states merge by a tree fixed by the chunk
// numbers. Every number a request gets depends on its own position, window and data, and every number of a
// query head on that head alone (a rank's slice gives the full call's bits). Where the page table
// holds one chunk at most (short contexts) the chunk's block writes the output itself, the bits that the
// merge would give: a lone step of 37 keys takes 5.6 us instead of 7.5.
//
// The stored bytes are u = c + 128 for values c 2^e with one exponent e per key and tile (g4_kv8.cuh).
// The matrix instructions (m16n8k16, fp16 operands, fp32 sums) take the bytes as they are: 0x00uu is
// the fp16 subnormal u 2^-24, which they multiply exactly, so one byte permute makes an operand pair.
// The bias of 128 is taken off the sums: 128 sum(q) from the scores, and 128 sum(w) from the value
// sums, where sum(w) is itself a row of that product (a row of constant bytes 128), so that what the
// tensor cores' fp32 sums round away of the common part is rounded away on both sides. The
// powers of two stay outside:
//   scores   x_j = scale log2(e) 2^e_j (c_j . q), with q as fp16 scaled by a power of two per head
//            (the bf16 q' is exact there: its largest magnitude sits at 2^14, and what falls below
//            fp16's smallest step is 2^-38 of that);
//   weights  P.V needs w_j = p_j 2^ev_j c_j: the power joins the exponent of the softmax weight,
//            w_j = 2^(x_j + ev_j - m2 + 7) in fp16, with a running maximum m2 of x_j + ev_j of its
//            own, apart from the maximum m1 that the sum of p_j = 2^(x_j - m1) is kept with. A head's
//            m2 moves only when its own maximum grows by more than 2^8, so w_j <= 2^15, and a weight
//            is lost only below 2^-32 of the largest.
// Declared roundings: roped q to bf16, w to fp16 (2^-11 relative, each weight by itself), the output
// to bf16; all sums are fp32.
//
// What bounds it. With many requests the page stream: 64 requests of 1k to 32k keys take 393 us on a
// global layer (2.3 GB, 5.9 TB/s, 86% of the measured copy rate; its chunks' states, 71 MB written and
// read again, are 5% of that traffic) and 91 us on a sliding one (0.54 GB, 5.9 TB/s). A block's start
// (its queries turned and laid out, 12 us of the 393) and end (the merge of its warps, 8 us besides the
// states' own bytes) are covered only in part by the SM's other block. With few requests a warp's
// chain through a page, about 0.8 us (scores 470 cycles, values 500, weights 440, the refill 150),
// bounds it: a lone request takes 21 us from 1024 keys up to 16384. Chunks of 2048 keys would take 5%
// off the large batch and put 60% on the lone request; chunks of 512 the reverse (15% on, 30% off). A
// quarter of the output per warp with the weights exchanged through shared memory (four blocks an SM,
// no merge), runs of two chunks per block with the pages streaming across, and clusters that merge
// 2 x 1024 keys were built and measured slower (405, 408 and 419 against 399 us).
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "g4_kv8.cuh"

namespace g4 {

namespace {

constexpr int kChunkSliding = 512, kChunkGlobal = kDecodeChunkGlobal;   // keys per chunk
constexpr int kWarps = 4;
constexpr int kStages = 2;             // pages in flight per warp
constexpr float kLazy = 8.0f;          // m2 moves when the maximum grows by more than 2^8
constexpr float kShift = 7.0f;         // the weights' scale: w <= 2^(kLazy + kShift)
constexpr float kNone = -1.0e38f;      // running maximum before the first key (finite: no inf - inf)

template <bool GLOBAL>
struct Shape {
  using Blk = Kv8Block<GLOBAL>;
  static constexpr int D = Blk::D;
  static constexpr int kSegs = D / 128;                  // 128-column segments of V
  static constexpr int kHalves = GLOBAL ? 8 : 4;         // 64-column halves of K: global 6 plain + 2 turned
  static constexpr int kHeads = GLOBAL ? 8 : 2;          // at most; columns beyond the group carry q = 0
  static constexpr int kChunk = GLOBAL ? kChunkGlobal : kChunkSliding;
  static constexpr int kStage = (Blk::kBytes + 127) / 128 * 128;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = kHalves * 1024;              // q fragments: [half][2][32 lanes][16 bytes]
  static constexpr int kPages = (kChunk / kPage) * 8 * 8;   // per page and head: max and sum of the page's weights
  static constexpr int smem(bool pages) { return kRing + kQ + (pages ? kPages : 0); }
  static_assert(kRing >= kWarps * kHeads * D * 4, "the warp merge reuses the ring");
};

struct Decode8Params {
  const __nv_bfloat16* q;
  const int32_t* seq_len;
  const int32_t* pos;   // RoPE position of the query; NULL: seq_len - 1
  int B;
  int window;
  float scale_log2;
  PagedCache8 cache;
  NormArgs nm;          // query norm, and the key norm's weight on a global layer's plain columns
  float* ws_ml;         // [B][hq][NC][2]: running max (log2 units) and sum
  float* ws_o;          // [B][hq][NC][D]: un-normalised output, relative to that max
  float* ws_page;       // [B][hkv][max_pages][8]: each page's weight relative to its chunk's max, or NULL
  int NC;
  __nv_bfloat16* out;   // one chunk slot and no page weights: the output, written without a merge; or NULL
  Kv8Angles angles;
  uint32_t* err;
  unsigned long long wait_ns;
};

constexpr float kUp = 16777216.0f;   // 2^24: undoes the bytes' reading as fp16 subnormals

// Two bytes of `w` as a pair of fp16 subnormals: the bytes at selector digits 0 and 2 (digit 4: zero).
G4_DEV uint32_t codes2(uint32_t w, uint32_t selector) { return __byte_perm(w, 0u, selector); }
// bulk_g2s whose lines are the first to leave L2: the pages stream through once, and the chunks' states,
// written meanwhile, stay there for the merge.
G4_DEV uint64_t evict_first_policy() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
G4_DEV void bulk_g2s_first(void* smem, const void* gmem, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(smem)),
      "l"(gmem), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
G4_DEV uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
G4_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
      "%1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
G4_DEV uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
G4_DEV uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Position checks shared by the two kernels: the held index of request b's token, or -1.
G4_DEV int held_index(const int32_t* seq_len, const int32_t* pos, int b, int max_pages, int& rope_pos) {
  const int idx = seq_len[b] - 1;
  rope_pos = pos ? pos[b] : idx;
  return (idx < 0 || idx >= kMaxPos || (idx >> 4) >= max_pages || rope_pos < idx || rope_pos >= kMaxPos) ? -1 : idx;
}

// Column d of a query head -> which half of the K order it belongs to (see Shape::kHalves).
template <bool GLOBAL>
G4_DEV int half_of(int d) {
  const int sh = d >> 6;
  if (!GLOBAL) return sh;
  return sh == 0 ? 6 : sh == 4 ? 7 : sh < 4 ? sh - 1 : sh - 2;
}

// The norm of a query head held by a warp (lane: columns t0 .. and D/2 + t0 ..), times its weight; on a
// global layer's plain columns also the key norm's weight, which the stored S lacks. The result is cast
// to bf16 (a declared cast), as in the bf16 decode.
template <bool GLOBAL>
G4_DEV void norm_query(const NormArgs& nm, int t0, float (&a)[Shape<GLOBAL>::D / 64], float (&b)[Shape<GLOBAL>::D / 64]) {
  constexpr int D = Shape<GLOBAL>::D, P = D / 64;
  if (nm.wq) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
    // the definition's operations, each rounded by itself: the cast below meets borders too
    const float root = __fsqrt_rn(__fadd_rn(ss * (1.0f / (float)D), nm.eps));   // ss / D is exact: D is a power of 2
#pragma unroll
    for (int i = 0; i < P; ++i) {
      a[i] = __fmul_rn(__fdiv_rn(a[i], root), bf16_to_f(nm.wq[t0 + i]));
      b[i] = __fmul_rn(__fdiv_rn(b[i], root), bf16_to_f(nm.wq[D / 2 + t0 + i]));
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (GLOBAL && nm.wk && t0 >= Shape<GLOBAL>::Blk::R) {
      a[i] *= bf16_to_f(nm.wk[t0 + i]);
      b[i] *= bf16_to_f(nm.wk[D / 2 + t0 + i]);
    }
    a[i] = round_bf16(a[i]);
    b[i] = round_bf16(b[i]);
  }
}

// Zeros to the block's query heads of a request that cannot be served.
template <int D>
G4_DEV void zero_heads(__nv_bfloat16* out, int heads) {
  for (int i = threadIdx.x; i < heads * D / 8; i += kWarps * 32) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
}

template <bool GLOBAL, bool PAGES>
__global__ void __launch_bounds__(kWarps * 32, 2) kv8_decode_kernel(const Decode8Params p) {
  using S = Shape<GLOBAL>;
  using Blk = Kv8Block<GLOBAL>;
  constexpr int D = S::D;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* q_s = smem + S::kRing;
  float2* page_s = reinterpret_cast<float2*>(q_s + S::kQ);   // [page of the chunk][8 heads]
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int abort_flag;
  __shared__ float q_scale[8], q_sum[2][8];   // per head: power of two, 128 x sum of q over the plain and turned columns
  __shared__ float red_m[kWarps][8], red_l[kWarps][8], red_m2[kWarps][8], factor[kWarps][8];
  __shared__ float inv_sum[8];

  wait_for_grid();
  let_next_grid_start();
  const int HKV = p.cache.hkv, G = p.cache.hq / HKV;
  const int cr = blockIdx.x % p.NC;                    // chunk slot, KV head, request
  const int g = (blockIdx.x / p.NC) % HKV;
  const int b = blockIdx.x / p.NC / HKV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, cq = lane & 3;             // matrix fragment coordinates

  // This warp's query heads, warp and warp + 4, in flight while the length and the pages are looked up.
  constexpr int P = D / 64;   // pairs per lane: columns t0 .. t0 + P - 1 and D / 2 + t0 ..
  constexpr int kMine = (S::kHeads + kWarps - 1) / kWarps;
  const int t0 = lane * P;
  uint32_t q_lo[kMine][P / 2], q_hi[kMine][P / 2];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int h = warp + kWarps * i;
    if (h >= G) continue;
    const __nv_bfloat16* src = p.q + ((size_t)b * p.cache.hq + (size_t)G * g + h) * D + t0;
    if (P == 8) {
      *reinterpret_cast<uint4*>(q_lo[i]) = *reinterpret_cast<const uint4*>(src);
      *reinterpret_cast<uint4*>(q_hi[i]) = *reinterpret_cast<const uint4*>(src + D / 2);
    } else {
      *reinterpret_cast<uint2*>(q_lo[i]) = *reinterpret_cast<const uint2*>(src);
      *reinterpret_cast<uint2*>(q_hi[i]) = *reinterpret_cast<const uint2*>(src + D / 2);
    }
  }
  const int32_t* table = p.cache.page_table + (size_t)b * p.cache.max_pages;
  int phys = 0;
  if (GLOBAL) {   // the chunk is known before the length: its table entries load along with it
    const int i = cr * (S::kChunk / kPage) + warp + kWarps * lane;
    if (lane < S::kChunk / kPage / kWarps && i < p.cache.max_pages) phys = table[i];
  }
  int rope_pos;
  const int last = held_index(p.seq_len, p.pos, b, p.cache.max_pages, rope_pos);
  if (last < 0) {
    if (threadIdx.x == 0 && cr == 0 && g == 0) set_error(p.err, kErrPos);
    if (!PAGES && p.out) zero_heads<D>(p.out + ((size_t)b * p.cache.hq + (size_t)G * g) * D, G);
    return;   // else the merge writes zeros for this request
  }
  const int lo = GLOBAL ? 0 : max(0, last - p.window + 1);
  const int c = lo / S::kChunk + cr;
  const int k_begin = max(lo, c * S::kChunk);
  const int k_end = min(last, c * S::kChunk + S::kChunk - 1);   // inclusive
  if (k_begin > k_end) return;                                    // unused slot

  // This warp's pages: warp, warp + 4, ... of the chunk's; lane n keeps the n-th one's physical page. A
  // warp that finds one outside the pool copies none of its pages, and the chunk then adds nothing.
  const int pg0 = k_begin >> 4, n_pages = (k_end >> 4) - pg0 + 1;
  int mine = n_pages > warp ? (n_pages - warp + kWarps - 1) / kWarps : 0;   // at most 32
  if (!GLOBAL && lane < mine) phys = table[pg0 + warp + kWarps * lane];
  const bool bad = __any_sync(0xffffffffu, lane < mine && (phys < 0 || phys >= p.cache.num_pages));
  if (bad) mine = 0;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < kStages) mbar_init(&full[warp][lane], 1);   // a warp's barriers are its own
  fence_mbar_init();
  __syncwarp();
  const size_t slot = ((size_t)b * p.cache.hq + (size_t)G * g) * p.NC + cr;   // head G g + h adds h NC

  uint8_t* ring = smem + warp * kStages * S::kStage;
  const uint64_t policy = evict_first_policy();
  auto issue = [&](int n, int page) {   // lane 0: copy this warp's n-th page
    const int st = n % kStages;
    mbar_arrive_expect_tx(&full[warp][st], Blk::kBytes);
    bulk_g2s_first(ring + st * S::kStage, p.cache.pages + ((size_t)page * HKV + g) * Blk::kBytes, Blk::kBytes,
                   &full[warp][st], policy);
  };
#pragma unroll
  for (int n = 0; n < kStages; ++n) {
    const int page = __shfl_sync(0xffffffffu, phys, n);
    if (lane == 0 && n < mine) issue(n, page);
  }

  // The query heads of this KV head, turned, cast to bf16, scaled by a power of two each and laid out
  // as matrix fragments: lane (head, cc) of half i and step t holds columns 16 cc + 4t + {0, 2} and
  // {1, 3} of the half. One warp per head.
  float2 cs[P];               // (cos, sin) of this lane's pairs, the same for every head
  {
    // Exact to 2^-25, like the append's: a turned query falls on the far side of a border between two bf16
    // numbers as rarely as with exactly rounded angles. Pairs R/32 to a lane; a global layer's eight lanes
    // that turn fetch theirs from four lanes each.
    constexpr int kOwn = Blk::R / 32;
    const float4* cx = p.angles.coarse + (size_t)(rope_pos >> 8) * Blk::R + kOwn * lane;
    const float4* fx = p.angles.fine + (size_t)(rope_pos & 255) * Blk::R + kOwn * lane;
    float2 own[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own[i] = rope_cs_exact(__ldg(cx + i), __ldg(fx + i));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (GLOBAL) {
        const int src = 4 * (lane & 7) + (i >> 1);
        cs[i].x = __shfl_sync(0xffffffffu, own[i & 1].x, src);
        cs[i].y = __shfl_sync(0xffffffffu, own[i & 1].y, src);
      } else {
        cs[i] = own[i % kOwn];
      }
    }
  }
  // Columns of the product beyond the group carry q = 0.
  for (int h = S::kHeads + warp; h < 8; h += kWarps) {   // (a sliding layer's six)
    for (int i = lane; i < S::kHalves * 2 * 4; i += 32)
      *reinterpret_cast<uint4*>(q_s + ((i >> 2) * 32 + h * 4 + (i & 3)) * 16) = make_uint4(0, 0, 0, 0);
    if (lane == 0) q_scale[h] = q_sum[0][h] = q_sum[1][h] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int h = warp + kWarps * k;
    if (h >= S::kHeads) continue;
    float a[P], bb[P];
    if (h < G) {
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        a[i] = bf16_lo(q_lo[k][i / 2]);
        a[i + 1] = bf16_hi(q_lo[k][i / 2]);
        bb[i] = bf16_lo(q_hi[k][i / 2]);
        bb[i + 1] = bf16_hi(q_hi[k][i / 2]);
      }
      if (p.nm.wq || (GLOBAL && p.nm.wk)) norm_query<GLOBAL>(p.nm, t0, a, bb);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (t0 < Blk::R) rope_pair_apart(a[i], bb[i], cs[i]);
        a[i] = round_bf16(a[i]);   // declared cast: roped q in bf16
        bb[i] = round_bf16(bb[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) a[i] = bb[i] = 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      m = max(m, max(__float_as_uint(a[i]) & 0x7fffffffu, __float_as_uint(bb[i]) & 0x7fffffffu));
    m = __reduce_max_sync(0xffffffffu, m);
    // largest |q| = 2^(eb - 127) up to twice that, moved to [2^14, 2^15); an infinity or NaN stays one
    const int eb = max(20, min(254, (int)(m >> 23)));
    const float down = __uint_as_float((uint32_t)(268 - eb) << 23);   // 2^(141 - eb)
    if (lane == 0) q_scale[h] = __uint_as_float((uint32_t)(eb - 14) << 23);   // 2^(eb - 141)
    float sum = 0.f;   // a lane's columns are all plain or all turned
    uint32_t frag[2][P / 4][2];   // per half of the head and group of four columns: {0, 2} and {1, 3}
#pragma unroll
    for (int i = 0; i < P; i += 4) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        frag[0][i / 4][e] = pack_f16(a[i + e] * down, a[i + e + 2] * down);
        frag[1][i / 4][e] = pack_f16(bb[i + e] * down, bb[i + e + 2] * down);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&frag[half][i / 4][e]));
          sum += f.x + f.y;
        }
      }
    }
    const bool turned = GLOBAL && t0 < Blk::R;
    float plain_sum = turned ? 0.f : sum, turned_sum = turned ? sum : 0.f;
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
      plain_sum += __shfl_xor_sync(0xffffffffu, plain_sum, w);
      if (GLOBAL) turned_sum += __shfl_xor_sync(0xffffffffu, turned_sum, w);
    }
    if (lane == 0) {
      q_sum[0][h] = 128.0f * plain_sum;
      q_sum[1][h] = 128.0f * turned_sum;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // a lane's columns are one group of four, or the two of a step pair
      const int d = t0 + half * (D / 2), cc = (d & 63) >> 4, t = (d >> 2) & 3;
      uint8_t* dst = q_s + ((half_of<GLOBAL>(d) * 2 + (t >> 1)) * 32 + h * 4 + cc) * 16 + (t & 1) * 8;
      if (P == 8)
        *reinterpret_cast<uint4*>(dst) = make_uint4(frag[half][0][0], frag[half][0][1], frag[half][P / 4 - 1][0],
                                                    frag[half][P / 4 - 1][1]);
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(frag[half][0][0], frag[half][0][1]);
    }
  }
  const bool void_chunk = __syncthreads_or(bad);
  const float qs[2] = {q_scale[2 * cq], q_scale[2 * cq + 1]};
  const float q0[2] = {q_sum[0][2 * cq], q_sum[0][2 * cq + 1]}, q1[2] = {q_sum[1][2 * cq], q_sum[1][2 * cq + 1]};

  float o[S::kSegs * 8][4];   // O^T: rows = columns of V, columns = heads 2cq, 2cq + 1
#pragma unroll
  for (int i = 0; i < S::kSegs * 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ow[4] = {0.f, 0.f, 0.f, 0.f};   // the row of constant bytes 128
  float m1[2] = {kNone, kNone}, l1[2] = {0.f, 0.f}, m2[2] = {kNone, kNone};   // m1, l1 of this lane's own keys

  const uint32_t q_addr = smem_u32(q_s) + lane * 16;
  const uint32_t k_lane = gq * 128 + ((cq ^ kv8_swizzle(gq)) << 4);          // rows of K: key gq, piece cq (+ 4: ^ 64)
  // columns of V: keys 2cq, 2cq + 1 (and + 8, 1 KB on), piece gq
  const uint32_t v_lane0 = 2 * cq * 128 + ((gq ^ kv8_swizzle(2 * cq)) << 4);
  const uint32_t v_lane1 = (2 * cq + 1) * 128 + ((gq ^ kv8_swizzle(2 * cq + 1)) << 4);

  int n = 0;
  for (; n < mine; ++n) {
    const int st = n % kStages;
    const bool ok = mbar_wait(&full[warp][st], (n / kStages) & 1, &abort_flag, p.err, p.wait_ns);
    if (!__all_sync(0xffffffffu, ok)) break;
    const uint8_t* blk = ring + st * S::kStage;
    const uint32_t base = smem_u32(blk);
    const int key0 = (pg0 + warp + kWarps * n) * kPage;

    // ---- S^T = K q^T: 16 keys x 8 heads, the plain columns (four chains) and the turned ones (two) apart
    float s0[4][4] = {}, s1[2][4] = {};
#pragma unroll
    for (int i = 0; i < S::kHalves; ++i) {
      const bool turned = GLOBAL && i >= 6;
      const int sh = !GLOBAL ? i : i < 3 ? i + 1 : i + 2;   // 64-column half of the tile
      const uint32_t at = turned ? (uint32_t)Blk::kTile1 + (k_lane ^ (i == 7 ? 64u : 0u))
                                 : (uint32_t)(sh >> 1) * 2048 + (k_lane ^ ((sh & 1) ? 64u : 0u));
      const uint4 x = lds128(base + at), y = lds128(base + at + 1024);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint4 qf = lds128(q_addr + (i * 2 + tt) * 512);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = tt * 2 + u;
          const uint32_t a0 = codes2(xw[t], 0x4240), a1 = codes2(yw[t], 0x4240);
          const uint32_t a2 = codes2(xw[t], 0x4341), a3 = codes2(yw[t], 0x4341);
          mma_f16(turned ? s1[u] : s0[t], a0, a1, a2, a3, u ? qf.z : qf.x, u ? qf.w : qf.y);
        }
      }
    }

    // ---- softmax of this lane's keys gq, gq + 8 for heads 2cq, 2cq + 1
    const uint32_t e_lo = blk[Blk::kExp0 + gq], e_hi = blk[Blk::kExp0 + gq + 8];
    const uint32_t f_lo = blk[Blk::kExp1 + gq], f_hi = blk[Blk::kExp1 + gq + 8];
    const uint32_t v_lo = GLOBAL ? e_lo : f_lo, v_hi = GLOBAL ? e_hi : f_hi;
    const float ev_lo = v_lo == 255u ? NAN : (float)((int)v_lo - 133), ev_hi = v_hi == 255u ? NAN : (float)((int)v_hi - 133);
    const bool see_lo = key0 + gq >= k_begin && key0 + gq <= k_end;
    const bool see_hi = key0 + gq + 8 >= k_begin && key0 + gq + 8 <= k_end;
    // the query's and the key's powers of two go together: either alone could leave fp32's range with large keys
    float x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float sum0 = (s0[0][r] + s0[1][r]) + (s0[2][r] + s0[3][r]);
      float s = fmaf(sum0, kUp, -q0[r & 1]) * (qs[r & 1] * kv8_step(r < 2 ? e_lo : e_hi));
      if (GLOBAL) s += fmaf(s1[0][r] + s1[1][r], kUp, -q1[r & 1]) * (qs[r & 1] * kv8_step(r < 2 ? f_lo : f_hi));
      const bool see = r < 2 ? see_lo : see_hi;
      x[r] = see ? s * p.scale_log2 : -INFINITY;
      y[r] = see ? x[r] + (r < 2 ? ev_lo : ev_hi) : -INFINITY;
    }
    float2 page_ms[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mn = fmaxf(m1[j], fmaxf(x[j], x[2 + j]));
      if (PAGES) {   // the page's weight by itself: its maximum and sum over the warp
        float mp = fmaxf(x[j], x[2 + j]);
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, w));
        mp = fmaxf(mp, kNone);
        float ps = ex2(x[j] - mp) + ex2(x[2 + j] - mp);
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
        page_ms[j] = make_float2(mp, ps);
      }
      l1[j] = fmaf(l1[j], ex2(m1[j] - mn), ex2(x[j] - mn) + ex2(x[2 + j] - mn));
      m1[j] = mn;
    }
    if (PAGES && gq == 0)
      *reinterpret_cast<float4*>(page_s + (warp + kWarps * n) * 8 + 2 * cq) =
          make_float4(page_ms[0].x, page_ms[0].y, page_ms[1].x, page_ms[1].y);
    // the weights' reference: a head's moves only when one of its own keys passes it by 2^8, whatever the
    // other columns do (a head's bits are those it gets in a rank's slice); the vote only skips the block
    const bool grow = fmaxf(y[0], y[2]) > m2[0] + kLazy || fmaxf(y[1], y[3]) > m2[1] + kLazy;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mn = fmaxf(y[j], y[2 + j]);
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
        mn = mn > m2[j] + kLazy ? mn : m2[j];
        const float al = ex2(m2[j] - mn);
        m2[j] = mn;
#pragma unroll
        for (int i = 0; i < S::kSegs * 8; ++i) {
          o[i][j] *= al;
          o[i][2 + j] *= al;
        }
        ow[j] *= al;
      }
    }
    float wgt[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) wgt[r] = ex2(y[r] - m2[r & 1] + kShift);
    const uint32_t b0 = transpose8x8(pack_f16(wgt[0], wgt[1]));   // keys 2cq, 2cq + 1 of head gq
    const uint32_t b1 = transpose8x8(pack_f16(wgt[2], wgt[3]));   // keys 2cq + 8, 2cq + 9

    mma_f16(ow, 0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u, b0, b1);

    // ---- O^T += V^T w^T: columns 16 gq .. + 15 of each segment, keys 2cq, 2cq + 1, 2cq + 8, 2cq + 9
#pragma unroll
    for (int sg = 0; sg < S::kSegs; ++sg) {
      const uint32_t at = base + (GLOBAL ? 0u : (uint32_t)Blk::kTile1) + sg * 2048;
      const uint4 k0 = lds128(at + v_lane0), k1 = lds128(at + v_lane1);
      const uint4 k2 = lds128(at + v_lane0 + 1024), k3 = lds128(at + v_lane1 + 1024);
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
      const uint32_t w2[4] = {k2.x, k2.y, k2.z, k2.w}, w3[4] = {k3.x, k3.y, k3.z, k3.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // byte pairs (key, key + 1) of columns 4t, 4t + 1 and of 4t + 2, 4t + 3
        const uint32_t ab = __byte_perm(w0[t], w1[t], 0x5140), cd = __byte_perm(w0[t], w1[t], 0x7362);
        const uint32_t ef = __byte_perm(w2[t], w3[t], 0x5140), gh = __byte_perm(w2[t], w3[t], 0x7362);
        mma_f16(o[sg * 8 + 2 * t], codes2(ab, 0x4140), codes2(ab, 0x4342), codes2(ef, 0x4140), codes2(ef, 0x4342), b0, b1);
        mma_f16(o[sg * 8 + 2 * t + 1], codes2(cd, 0x4140), codes2(cd, 0x4342), codes2(gh, 0x4140), codes2(gh, 0x4342), b0,
                b1);
      }
    }
    __syncwarp();
    const int page = __shfl_sync(0xffffffffu, phys, (n + kStages) & 31);
    if (lane == 0 && n + kStages < mine) {   // every lane has read the stage: refill it
      fence_proxy_async();
      issue(n + kStages, page);
    }
  }
  if (n < mine && lane == 0) {   // a wait ran out: let the copies in flight finish (bounded)
    const unsigned long long t0 = globaltimer();
    for (int i = n; i < min(mine, n + kStages); ++i)
      while (!mbar_try_wait(smem_u32(&full[warp][i % kStages]), (i / kStages) & 1) && globaltimer() - t0 < kWaitLimitNs) {
      }
  }

  // This warp's (m1, l1) per head, over the eight lanes that hold its keys.
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float mw = m1[j];
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, w));
    float lw = l1[j] * ex2(m1[j] - mw);
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, w);
    if (gq == 0) {
      red_m[warp][2 * cq + j] = mw;
      red_l[warp][2 * cq + j] = lw;
      red_m2[warp][2 * cq + j] = m2[j];
    }
  }
  const bool cut = __syncthreads_or(n < mine);   // every stage has been read: reuse the ring for the warp merge
  float* page_out = PAGES ? p.ws_page + (((size_t)b * HKV + g) * p.cache.max_pages + pg0) * 8 : nullptr;
  if (void_chunk || cut) {   // a page outside the pool, or a wait that ran out: a state that adds nothing
    if (threadIdx.x == 0 && void_chunk) set_error(p.err, kErrPage);
    if (!PAGES && p.out) {
      zero_heads<D>(p.out + ((size_t)b * p.cache.hq + (size_t)G * g) * D, G);
      return;
    }
    if ((int)threadIdx.x < G)
      *reinterpret_cast<float2*>(p.ws_ml + (slot + (size_t)threadIdx.x * p.NC) * 2) = make_float2(-INFINITY, 0.f);
    if (PAGES)
      for (int i = threadIdx.x; i < n_pages * 8; i += kWarps * 32) page_out[i] = 0.f;
    return;
  }
  if (PAGES) {   // against the chunk's max: exact differences of maxima, where sums of logarithms would be rounded
    for (int i = threadIdx.x; i < n_pages * 8; i += kWarps * 32) {
      const int h = i & 7;
      float M = red_m[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, red_m[w][h]);
      page_out[i] = page_s[i].y * ex2(page_s[i].x - M);
    }
  }
  // The warps' outputs in fragment order ([warp][row tile][lane][4]: 16 bytes a lane, no bank conflicts);
  // on sliding layers only lanes with heads (cq = 0) hold any.
  constexpr int kTiles = S::kSegs * 8, kLanes = GLOBAL ? 32 : 8;
  float4* red_o = reinterpret_cast<float4*>(smem);
  const int my = GLOBAL ? lane : gq;
  if (GLOBAL || cq == 0) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
      red_o[(warp * kTiles + i) * kLanes + my] = make_float4((o[i][0] - ow[0]) * kUp, (o[i][1] - ow[1]) * kUp,
                                                             (o[i][2] - ow[0]) * kUp, (o[i][3] - ow[1]) * kUp);
  }
  if (threadIdx.x < 8) {   // per head: the chunk's max and sum, and each warp's factor (a product of two: it may lie below 2^-126)
    const int h = threadIdx.x;
    float M = red_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, red_m[w][h]);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      L = fmaf(red_l[w][h], ex2(red_m[w][h] - M), L);
      factor[w][h] = ex2(0.5f * (red_m2[w][h] - kShift - M));
    }
    if (!PAGES && p.out)
      inv_sum[h] = L == 0.f ? 0.f : __frcp_rn(L);
    else if (h < G)
      *reinterpret_cast<float2*>(p.ws_ml + (slot + (size_t)h * p.NC) * 2) = make_float2(L == 0.f ? -INFINITY : M, L);
  }
  __syncthreads();
  // A thread merges, in warp order, four neighbouring row tiles of one lane: eight columns of two heads.
  for (int i = threadIdx.x; i < S::kSegs * 2 * kLanes; i += kWarps * 32) {
    const int ln = i % kLanes, t4 = i / kLanes;
    const int lq = GLOBAL ? ln >> 2 : ln, lc = GLOBAL ? ln & 3 : 0;
    float acc[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f0 = factor[w][2 * lc], f1 = factor[w][2 * lc + 1];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 v = red_o[(w * kTiles + t4 * 4 + u) * kLanes + ln];
        acc[0][2 * u] = fmaf(v.x * f0, f0, acc[0][2 * u]);
        acc[1][2 * u] = fmaf(v.y * f1, f1, acc[1][2 * u]);
        acc[0][2 * u + 1] = fmaf(v.z * f0, f0, acc[0][2 * u + 1]);
        acc[1][2 * u + 1] = fmaf(v.w * f1, f1, acc[1][2 * u + 1]);
      }
    }
    const int d = (t4 >> 1) * 128 + lq * 16 + (t4 & 1) * 8;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (2 * lc + j >= G) continue;
      if (!PAGES && p.out) {   // the bits that the merge of one chunk gives
        const float f = inv_sum[2 * lc + j];
        uint4 pk;
        pk.x = pack_bf16(acc[j][0] * f, acc[j][1] * f);
        pk.y = pack_bf16(acc[j][2] * f, acc[j][3] * f);
        pk.z = pack_bf16(acc[j][4] * f, acc[j][5] * f);
        pk.w = pack_bf16(acc[j][6] * f, acc[j][7] * f);
        *reinterpret_cast<uint4*>(p.out + ((size_t)b * p.cache.hq + (size_t)G * g + 2 * lc + j) * D + d) = pk;
        continue;
      }
      float* dst = p.ws_o + (slot + (size_t)(2 * lc + j) * p.NC) * D + d;
      *reinterpret_cast<float4*>(dst) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
  }
}

// Number of chunk slots that request b fills.
G4_DEV int chunks_of(int last, int window, int chunk) {
  const int lo = window > 0 ? max(0, last - window + 1) : 0;
  return last / chunk - lo / chunk + 1;
}

// ---- ordered merge of the chunks, and the accumulated page weights -----------------------------------------
// Merge units are (request, head, 128 columns). The chunks c = q (mod 4) of a unit are added in ascending
// order, q = 0 .. 3, and the four sums in the order of q: a tree fixed by the chunk numbers. With SPLIT 1 a
// warp does a unit, sixteen loads in flight; with SPLIT 4 (long page tables: few units of many chunks)
// the four warps of a block take one sum each. A refused request gets zeros. The blocks after them add
// page_weights[b][i] += sum over heads of the page's share of the softmax, a thread per page, heads in
// ascending order.
constexpr int kFinishThreads = 128;

template <int D, bool PAGES, int SPLIT>
__global__ void __launch_bounds__(kFinishThreads) kv8_finish_kernel(const Decode8Params p, int chunk, unsigned units,
                                                                    unsigned merge_blocks, int blocks_per_row,
                                                                    __nv_bfloat16* out, float* page_weights) {
  wait_for_grid();
  let_next_grid_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = p.cache.hq;
  if (!PAGES || blockIdx.x < merge_blocks) {
    __shared__ float4 part[3][32];
    constexpr int kCols = D / 128;
    const unsigned unit = SPLIT == 4 ? blockIdx.x : blockIdx.x * 4 + warp;
    if (unit >= units) return;
    const int col = (unit % kCols) * 128 + lane * 4;
    const int h = (unit / kCols) % hq, b = unit / kCols / hq;
    int rope_pos;
    const int last = held_index(p.seq_len, p.pos, b, p.cache.max_pages, rope_pos);
    const int n = last < 0 ? 0 : min(p.NC, chunks_of(last, p.window, chunk));
    const size_t s0 = ((size_t)b * hq + h) * p.NC;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + s0;
    const float* o_src = p.ws_o + s0 * D + col;
    const float2 none = make_float2(-INFINITY, 0.f);
    float2 v = lane < n ? ml[lane] : none;   // lane l: chunk l, later 32 k + l
    float M = v.x;
#pragma unroll 4
    for (int c = 32 + lane; c < n; c += 32) M = fmaxf(M, ml[c].x);
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    float L = 0.f;
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += 32) {
      const float2 next = c0 + 32 + lane < n ? ml[c0 + 32 + lane] : none;
      const bool some = v.x != -INFINITY;   // a chunk that added nothing did not write its output slot
      const float wc = some ? ex2(v.x - M) : 0.f;
      if (some) L = fmaf(v.y, wc, L);
      v = next;
      const unsigned wrote = __ballot_sync(0xffffffffu, some);
#pragma unroll
      for (int half = 0; half < (SPLIT == 4 ? 1 : 2); ++half) {
        constexpr int kLoads = SPLIT == 4 ? 8 : 16;
        if (SPLIT == 1 && c0 + 16 * half >= n) break;
        float4 o[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int c = SPLIT == 4 ? warp + 4 * i : 16 * half + i;
          o[i] = ((wrote >> c) & 1u) ? *reinterpret_cast<const float4*>(o_src + (size_t)(c0 + c) * D)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const float w = __shfl_sync(0xffffffffu, wc, SPLIT == 4 ? warp + 4 * i : 16 * half + i);
          float4& s = acc[SPLIT == 4 ? 0 : i & 3];
          s.x = fmaf(o[i].x, w, s.x);
          s.y = fmaf(o[i].y, w, s.y);
          s.z = fmaf(o[i].z, w, s.z);
          s.w = fmaf(o[i].w, w, s.w);
        }
      }
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
    if (SPLIT == 4) {
      if (warp > 0) part[warp - 1][lane] = acc[0];
      __syncthreads();
      if (warp > 0) return;
#pragma unroll
      for (int i = 1; i < 4; ++i) acc[i] = part[i - 1][lane];
    }
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      acc[0].x += acc[i].x;
      acc[0].y += acc[i].y;
      acc[0].z += acc[i].z;
      acc[0].w += acc[i].w;
    }
    const float inv = L == 0.f ? 0.f : __frcp_rn(L);
    uint2 pk;
    pk.x = pack_bf16(acc[0].x * inv, acc[0].y * inv);
    pk.y = pack_bf16(acc[0].z * inv, acc[0].w * inv);
    *reinterpret_cast<uint2*>(out + ((size_t)b * hq + h) * D + col) = pk;
    return;
  }
  // 128 pages, of kSpan chunks: per head and chunk the factor 2^(chunk's max - M) / L
  constexpr int kSpan = kFinishThreads * kPage / kChunkGlobal;
  static_assert(kSpan * kChunkGlobal == kFinishThreads * kPage, "a block's pages are whole chunks");
  __shared__ float factor[kSpan][kSlidingHq];
  const int unit = blockIdx.x - merge_blocks;
  const int b = unit / blocks_per_row, i0 = (unit % blocks_per_row) * kFinishThreads, i = i0 + threadIdx.x;
  int rope_pos;
  const int last = held_index(p.seq_len, p.pos, b, p.cache.max_pages, rope_pos);
  const int n_pages = (last >> 4) + 1;   // 0 when refused
  if (i0 >= n_pages) return;
  const int HKV = p.cache.hkv, G = hq / HKV;
  const int n = min(p.NC, chunks_of(last, 0, chunk));
  float4 x[2 * kGlobalHkv];   // this page's weights, in flight while the factors are formed
#pragma unroll
  for (int g = 0; g < kGlobalHkv; ++g) {
    if (g >= HKV || i >= n_pages) continue;
    const float4* src = reinterpret_cast<const float4*>(p.ws_page + (((size_t)b * HKV + g) * p.cache.max_pages + i) * 8);
    x[2 * g] = src[0];
    x[2 * g + 1] = src[1];
  }
  {   // four threads a head, chunks q, q + 4, ... each, one pass with a running maximum
    const int h = threadIdx.x >> 2, q = threadIdx.x & 3;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + ((size_t)b * hq + min(h, hq - 1)) * p.NC;
    float M = kNone, L = 0.f;
#pragma unroll 8
    for (int c = q; c < n; c += 4) {
      const float2 v = ml[c];
      const float mn = fmaxf(M, v.x);
      L = fmaf(L, ex2(M - mn), v.x == -INFINITY ? 0.f : v.y * ex2(v.x - mn));
      M = mn;
    }
#pragma unroll
    for (int w = 1; w <= 2; w <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, w), l2 = __shfl_xor_sync(0xffffffffu, L, w);
      const float mn = fmaxf(M, m2);
      L = L * ex2(M - mn) + l2 * ex2(m2 - mn);
      M = mn;
    }
    const int c = i0 / (kChunkGlobal / kPage) + q;
    if (q < kSpan && h < hq) factor[q][h] = c < n && L != 0.f ? ex2(ml[c].x - M) / L : 0.f;   // (a NaN sum stays one)
  }
  __syncthreads();
  if (i >= n_pages) return;
  const float* f = factor[threadIdx.x / (kChunkGlobal / kPage)];
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < kGlobalHkv; ++g) {
    if (g >= HKV) break;
    const float v[8] = {x[2 * g].x, x[2 * g].y, x[2 * g].z, x[2 * g].w, x[2 * g + 1].x, x[2 * g + 1].y, x[2 * g + 1].z,
                        x[2 * g + 1].w};
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < G) sum = fmaf(v[h], f[G * g + h], sum);
  }
  page_weights[(size_t)b * p.cache.max_pages + i] += sum;
}

int chunk_slots(bool global, int max_pages, int window) {
  const long long keys = (long long)max_pages * kPage < kMaxPos ? (long long)max_pages * kPage : kMaxPos;
  if (global) return (int)((keys + kChunkGlobal - 1) / kChunkGlobal);
  const int by_window = (window - 1) / kChunkSliding + 2;
  const int by_table = (int)((keys + kChunkSliding - 1) / kChunkSliding);
  return by_window < by_table ? by_window : by_table;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int D, bool PAGES>
cudaError_t finish(const Decode8Params& p, int chunk, void* out, float* page_weights, cudaStream_t s) {
  const long long units = (long long)p.B * p.cache.hq * (D / 128);
  const bool split = p.NC > 32;   // one warp's sixteen loads at a time would be a long chain
  const long long merge_blocks = split ? units : (units + 3) / 4;
  const int held = p.cache.max_pages < kMaxPos / kPage ? p.cache.max_pages : kMaxPos / kPage;   // pages at most
  const int per_row = (held + kFinishThreads - 1) / kFinishThreads;
  const long long blocks = merge_blocks + (PAGES ? (long long)p.B * per_row : 0);
  if (blocks > 0x7fffffffLL || units > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(split ? kv8_finish_kernel<D, PAGES, 4> : kv8_finish_kernel<D, PAGES, 1>, (unsigned)blocks,
                      kFinishThreads, 0, s, p, chunk, (unsigned)units, (unsigned)merge_blocks, per_row,
                      (__nv_bfloat16*)out, page_weights);
}

template <bool GLOBAL, bool PAGES>
cudaError_t launch(const Decode8Params& p, cudaStream_t s) {
  static std::atomic<bool> done[64];   // per device; two first calls at once both set the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kv8_decode_kernel<GLOBAL, PAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<GLOBAL>::smem(PAGES));
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const long long blocks = (long long)p.NC * p.cache.hkv * p.B;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(kv8_decode_kernel<GLOBAL, PAGES>, (unsigned)blocks, kWarps * 32, Shape<GLOBAL>::smem(PAGES), s, p);
}

}  // namespace

size_t kv8_decode_workspace_bytes(bool global, int B, int max_pages, int window, int hq, int hkv, bool pages) {
  const size_t nc = (size_t)chunk_slots(global, max_pages, window);
  const size_t D = global ? kGlobalD : kSlidingD;
  size_t n = align256((size_t)B * hq * nc * 2 * sizeof(float)) + align256((size_t)B * hq * nc * D * sizeof(float));
  if (pages) n += (size_t)B * hkv * max_pages * 8 * sizeof(float);
  return n;
}

cudaError_t launch_kv8_decode(bool global, const void* q, const int32_t* seq_len, const int32_t* pos, int B, int window,
                              float scale_log2, const PagedCache8& cache, const NormArgs& nm, float* page_weights, void* out,
                              void* ws, const DeviceState& st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  Decode8Params p{};
  p.q = (const __nv_bfloat16*)q;
  p.seq_len = seq_len;
  p.pos = pos;
  p.B = B;
  p.window = global ? 0 : window;
  p.scale_log2 = scale_log2;
  p.cache = cache;
  p.nm = nm;
  p.NC = chunk_slots(global, cache.max_pages, window);
  // A page table of one chunk (1024 keys on a global layer, 512 on a sliding one): nothing to merge.
  p.out = p.NC == 1 && !page_weights ? (__nv_bfloat16*)out : nullptr;
  const size_t D = global ? kGlobalD : kSlidingD;
  const size_t slots = (size_t)B * cache.hq * p.NC;
  uint8_t* w = (uint8_t*)ws;
  p.ws_ml = (float*)w;
  w += align256(slots * 2 * sizeof(float));
  p.ws_o = (float*)w;
  w += align256(slots * D * sizeof(float));
  p.ws_page = page_weights ? (float*)w : nullptr;
  cudaError_t e = kv8_angles(global, &p.angles);
  if (e != cudaSuccess) return e;
  p.err = st.err;
  p.wait_ns = wait_limit_ns();
  if (!global)
    e = launch<false, false>(p, s);
  else
    e = page_weights ? launch<true, true>(p, s) : launch<true, false>(p, s);
  if (e != cudaSuccess || p.out) return e;
  if (!global) return finish<kSlidingD, false>(p, kChunkSliding, out, nullptr, s);
  return page_weights ? finish<kGlobalD, true>(p, kChunkGlobal, out, page_weights, s)
                      : finish<kGlobalD, false>(p, kChunkGlobal, out, nullptr, s);
}

}  // namespace g4
