// Decode over the 4-bit paged cache: one query token per request, its keys split into fixed chunks (128 keys, a warp each,
// on sliding layers; 1024 keys, four warps, on global ones; aligned to key 0); inside a global chunk page i goes to warp
// i % 4 and the warps' states merge in warp order, and the chunks' states merge by a tree fixed by the chunk numbers. Every
// number a request gets depends on its own position, window and data, and every number of a query head on that head alone.
//
// The stored codes are E2M1 with a power of two per block of 32 columns (g4_kv4.cuh). The matrix instructions
// (m16n8k16, fp16 operands, fp32 sums) take them as fp16 numbers, one conversion per byte of two codes; the powers of
// two stay outside:
//   scores   x_j = scale log2(e) sum over blocks 2^s_jb (c_jb . q_b): a block is two matrix steps into sums of their
//            own, which join the score times 2^(s_jb - 167) (the 2^-40 keeps every scale in fp32's range). q is fp16
//            scaled by a power of two per head, its largest magnitude at 2^14: the bf16 q' is exact there down to 2^-31
//            of that magnitude, where fp16's smallest step passes its eighth bit, and at most 2^-39 of it off below;
//   weights  P.V needs w_jb = p_j 2^s_jb for every block b of V's columns. w_j = 2^(x_j + top_j - m2 + 7) in fp16, top_j
//            the key's largest scale, with a running maximum m2 of x_j + top_j of its own, apart from the maximum m1
//            that the sum of p_j = 2^(x_j - m1) is kept with; a block's weight is w_j 2^(s_jb - top_j), an exact fp16
//            product while it does not fall below 2^-14. A head's m2 moves only when its own maximum grows by more than
//            2^8, so the largest w_j so far is between 2^7 and 2^15: weights are exact but for the cast of w_j down to
//            2^-21 of the row's largest p_j 2^top_j (over all its keys), below that each of the two roundings is at
//            most 2^-25 beside 2^7, 2^-32 of the largest, and what is smaller than that is lost.
// Declared roundings: roped q to bf16, w to fp16 (2^-11 relative, each weight by itself), the output to bf16; all sums
// are fp32.
//
// What bounds it. Not the page stream: 64 requests of 1k to 32k keys take 365 us on a global layer (1.23 GB, 3.4 TB/s,
// 50% of the measured copy rate) and 74 us on a sliding one (normed; 0.29 GB, 3.9 TB/s), where the 8-bit cache's decode takes
// 391 and 90 for twice the bytes. A page-head block of 5456 bytes costs its warp about 1000 instructions: 256 are
// conversions of code pairs (every global S value is needed twice, in pairs of columns for the scores and in pairs of keys
// for the values), 64 order the keys' pairs, 64 are matrix instructions. The ALU pipe, which takes one instruction in two
// cycles and gives way to the matrix pipe, is 52% busy, and two warps a scheduler (128 output registers a thread) cover
// the rest of the chain's latency only in part (2.0 instructions a cycle). A lone request of 37 keys takes 5.3 us, of
// 16384 keys 29, of 131072 keys 72 (512 blocks on 304 places).
// Built, measured and not kept (us for the mix; kept: 374 timed alone with cold caches): two warps a page, one per
// 256 columns, with 12 warps an SM: 425; the same with two pages a step and the softmax shared out: 373 to 396; the
// scores of page n + 1 and the values of page n in one stretch of code: 424; two pages a warp together: 414 (the loop
// then outgrows the instruction caches). Shifts as multiplications on the other pipe: 375 to 383. Chunks of 512 keys: 436,
// and 25 instead of 30 for a lone request of 16384.
// Sliding layers see few pages of many chunks' ends, and blocks of several warps wait for their slowest one: a warp a block
// leaves its place to the next chunk by itself. In a graph, us for the normed mix and for a lone request of 4096 keys: 74.3
// and 10.2; four warps to a chunk of 512 keys 80.5 and 11.0; a warp to 256 keys 73.1 and 15.4; three warps with a chunk of
// 128 each and the queries laid out once for them 74.7. Three stages a warp in place of two 1 more; 14 or 16 blocks an SM
// (128 registers, some spilled) no faster. Of the mix's time the copies with the blocks' starts and ends are 54, the
// queries' norm 6 and their angles 3 (once per chunk). Short requests pay for it: 40 keys take 5.0 us, 3.8 with four warps.
// The chunk was chosen at a window of 1024 and is the same for all: of windows far wider a step's states are four times
// those of chunks of 512 (64 requests under a window of 262144: 4.3 GB of workspace, 1.1 over the 8-bit cache).
#include <atomic>

#include "g4_kv4.cuh"
#include "g4_kv_decode.cuh"

namespace g4 {

namespace {

constexpr int kChunkSliding = 128, kChunkGlobal = 1024;   // keys per chunk

template <bool GLOBAL>
struct Shape {
  using Blk = Kv4Block<GLOBAL>;
  static constexpr int D = Blk::D;
  static constexpr int kSegs = D / 256;                  // 256-column segments of V
  static constexpr int kBlocks = D / 32;                 // blocks of V's columns
  static constexpr int kQBlocks = GLOBAL ? 16 : 8;       // blocks of K's: global 12 plain, then 4 turned
  static constexpr int kHeads = GLOBAL ? 8 : 2;          // at most; columns beyond the group carry q = 0
  static constexpr int kChunk = GLOBAL ? kChunkGlobal : kChunkSliding;
  static constexpr int kStages = GLOBAL ? 4 : 2;         // pages in flight per warp
  static constexpr int kWarps = GLOBAL ? 4 : 1;          // of a chunk
  static constexpr int kResident = GLOBAL ? 2 : 12;      // blocks per SM
  static constexpr int kStage = (Blk::kBytes + 127) / 128 * 128;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = kQBlocks * 512;              // q fragments: [block][32 lanes][16 bytes]
  static constexpr int kFactors = kBlocks * 32;          // per warp: [block pair][lane % 4][2 blocks][2 key pairs] fp16x2
  static constexpr int kPages = (kChunk / kPage) * 8 * 8;   // per page and head: max and sum of the page's weights
  static constexpr int smem(bool pages) { return kRing + kQ + kWarps * kFactors + (pages ? kPages : 0); }
  static_assert(kRing >= kWarps * kHeads * D * 4, "the warp merge reuses the ring");
};

constexpr float kDown = 9.094947017729282e-13f;   // 2^-40: keeps every key's powers of two in fp32's range
constexpr float kUp = 1099511627776.0f;           // 2^40

G4_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b.
G4_DEV void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The powers of two of the scale bytes of two neighbouring blocks, the low half of w. A zero byte gives (next to) 0, a
// byte of 255 NaN.
G4_DEV float2 two_powers(uint32_t w) {
  uint32_t u;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(u) : "h"((uint16_t)w));
  return make_float2(bf16_lo(u), bf16_hi(u));
}

// Block of the q fragments that column d of a query head belongs to (see Shape::kQBlocks).
template <bool GLOBAL>
G4_DEV int q_block(int d) {
  const int b = d >> 5;
  if (!GLOBAL) return b;
  const int half = b >> 3, in = b & 7;
  return in < 2 ? 12 + 2 * half + in : 6 * half + in - 2;
}

G4_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
G4_DEV uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Stale scales above their key's top are cut to it (their weights are zeros); a NaN becomes 1.
G4_DEV uint32_t at_most_one(uint32_t a) {
  const __half2 h = __hmin2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(1.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
G4_DEV uint32_t mul_f16(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool GLOBAL, bool PAGES>
__global__ void __launch_bounds__(Shape<GLOBAL>::kWarps * 32, Shape<GLOBAL>::kResident) kv4_decode_kernel(const ChunkParams p) {
  using S = Shape<GLOBAL>;
  using Blk = Kv4Block<GLOBAL>;
  constexpr int D = S::D, kStages = S::kStages, kWarps = S::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* q_s = smem + S::kRing;
  uint32_t* factors = reinterpret_cast<uint32_t*>(q_s + S::kQ + (threadIdx.x >> 5) * S::kFactors);
  float2* page_s = reinterpret_cast<float2*>(q_s + S::kQ + kWarps * S::kFactors);   // [page of the chunk][8 heads]
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int abort_flag;
  __shared__ float q_scale[8];   // per head: power of two
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

  // This warp's query heads, warp and warp + kWarps, in flight while the length and the pages are looked up.
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
    if (threadIdx.x == 0 && cr == 0 && g == 0 && p.seq_len[b] != 0) set_error(p.err, kErrPos);
    if (!PAGES && p.out) zero_heads<D>(p.out + ((size_t)b * p.cache.hq + (size_t)G * g) * D, G);
    return;   // else the merge writes zeros for this request
  }
  const int lo = GLOBAL ? 0 : max(0, last - p.window + 1);
  const int c = lo / S::kChunk + cr;
  const int k_begin = max(lo, c * S::kChunk);
  const int k_end = min(last, c * S::kChunk + S::kChunk - 1);   // inclusive
  if (k_begin > k_end) return;                                    // unused slot

  // This warp's pages: warp, warp + kWarps, ... of the chunk's; lane n keeps the n-th one's physical page. A
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
  // as matrix fragments: lane (head, t) of a block holds its columns 4t .. 4t + 3 and 16 + 4t .. One warp per head.
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
    for (int i = lane; i < S::kQBlocks * 4; i += 32)
      *reinterpret_cast<uint4*>(q_s + ((i >> 2) * 32 + h * 4 + (i & 3)) * 16) = make_uint4(0, 0, 0, 0);
    if (lane == 0) q_scale[h] = 0.f;
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
      if (p.nm.wq || (GLOBAL && p.nm.wk)) norm_query<GLOBAL, D, Blk::R>(p.nm, t0, a, bb);
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
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        const float* x = half ? bb + i : a + i;
        const int d = t0 + half * (D / 2) + i, quad = (d & 31) >> 2;
        *reinterpret_cast<uint2*>(q_s + (q_block<GLOBAL>(d) * 32 + h * 4 + (quad & 3)) * 16 + (quad >> 2) * 8) =
            make_uint2(pack_f16(x[0] * down, x[1] * down), pack_f16(x[2] * down, x[3] * down));
      }
    }
  }
  const bool void_chunk = __syncthreads_or(bad);
  const float qs[2] = {q_scale[2 * cq], q_scale[2 * cq + 1]};

  float o[S::kBlocks * 2][4];   // O^T: rows = columns of V, columns = heads 2cq, 2cq + 1
#pragma unroll
  for (int i = 0; i < S::kBlocks * 2; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m1[2] = {kNone, kNone}, l1[2] = {0.f, 0.f}, m2[2] = {kNone, kNone};   // m1, l1 of this lane's own keys

  const uint32_t q_addr = smem_u32(q_s) + lane * 16;
  const uint32_t k_lane = gq * 128 + ((cq ^ kv8_swizzle(gq)) << 4);          // key gq, piece cq (piece cq + 4: ^ 64)
  // columns of V: keys 2cq, 2cq + 1 (and + 8, 1 KB on), piece gq
  const uint32_t v_lane0 = 2 * cq * 128 + ((gq ^ kv8_swizzle(2 * cq)) << 4);
  const uint32_t v_lane1 = (2 * cq + 1) * 128 + ((gq ^ kv8_swizzle(2 * cq + 1)) << 4);
  constexpr int kVScale = GLOBAL ? Blk::kScale0 : Blk::kScale1;
  const uint32_t f_addr = smem_u32(factors);

  int n = 0;
  for (; n < mine; ++n) {
    const int st = n % kStages;
    const bool ok = mbar_wait(&full[warp][st], (n / kStages) & 1, &abort_flag, p.err, p.wait_ns);
    if (!__all_sync(0xffffffffu, ok)) break;
    const uint8_t* blk = ring + st * S::kStage;
    const uint32_t base = smem_u32(blk);
    const int key0 = (pg0 + warp + kWarps * n) * kPage;

    // ---- the value blocks' powers of two against their key's top, as fp16 pairs: lane (pair of keys, quarter of the
    // blocks) forms them for the warp
    {
      constexpr int kQuarter = S::kBlocks / 4;
      const int pair = lane & 7, quarter = lane >> 3;
      const uint8_t* at = blk + kVScale + 2 * pair * S::kBlocks + quarter * kQuarter;
      const uint32_t tops = *reinterpret_cast<const uint16_t*>(blk + Blk::kTop + 2 * pair);
      const float inv0 = __uint_as_float((uint32_t)max(254 - (int)(tops & 255u), 0) << 23);   // 2^(127 - top)
      const float inv1 = __uint_as_float((uint32_t)max(254 - (int)(tops >> 8), 0) << 23);
#pragma unroll
      for (int i = 0; i < kQuarter; i += 2) {
        const float2 f0 = two_powers(*reinterpret_cast<const uint16_t*>(at + i));
        const float2 f1 = two_powers(*reinterpret_cast<const uint16_t*>(at + S::kBlocks + i));
        const int vb = quarter * kQuarter + i;
        uint32_t* to = factors + ((vb >> 1) * 4 + (pair & 3)) * 4 + (pair >> 2);
        to[0] = at_most_one(pack_f16(f0.x * inv0, f1.x * inv1));
        to[2] = at_most_one(pack_f16(f0.y * inv0, f1.y * inv1));
      }
    }

    // ---- S^T = K q^T: 16 keys x 8 heads, block by block
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float (&t)[4], float f_lo, float f_hi) {   // keys gq, gq + 8
      s[0] = fmaf(t[0], f_lo, s[0]);
      s[1] = fmaf(t[1], f_lo, s[1]);
      s[2] = fmaf(t[2], f_hi, s[2]);
      s[3] = fmaf(t[3], f_hi, s[3]);
    };
    {
      uint32_t sc_lo[S::kBlocks / 4], sc_hi[S::kBlocks / 4];
      if (GLOBAL) {
        *reinterpret_cast<uint4*>(sc_lo) = lds128(base + Blk::kScale0 + gq * 16);
        *reinterpret_cast<uint4*>(sc_hi) = lds128(base + Blk::kScale0 + gq * 16 + 128);
      } else {
        *reinterpret_cast<uint2*>(sc_lo) = lds64(base + Blk::kScale0 + gq * 8);
        *reinterpret_cast<uint2*>(sc_hi) = lds64(base + Blk::kScale0 + gq * 8 + 64);
      }
#pragma unroll
      for (int sg = 0; sg < S::kSegs; ++sg) {
        const uint32_t at = base + sg * 2048 + k_lane;
        const uint4 x0 = lds128(at), x1 = lds128(at ^ 64u), y0 = lds128(at + 1024), y1 = lds128((at ^ 64u) + 1024);
        const uint32_t x0w[4] = {x0.x, x0.y, x0.z, x0.w}, x1w[4] = {x1.x, x1.y, x1.z, x1.w};
        const uint32_t y0w[4] = {y0.x, y0.y, y0.z, y0.w}, y1w[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int w = GLOBAL ? 1 : 0; w < 4; ++w) {   // a global layer's first two blocks turn: they are below
          uint32_t a0[4], a1[4], c0[4], c1[4];
          kv4_halves(x0w[w], a0);
          kv4_halves(y0w[w], a1);
          kv4_halves(x1w[w], c0);
          kv4_halves(y1w[w], c1);
          const int vb = sg * 8 + 2 * w, qb = GLOBAL ? sg * 6 + 2 * w - 2 : vb;
          const float2 f_lo = two_powers(sc_lo[vb / 4] >> (16 * (w & 1))), f_hi = two_powers(sc_hi[vb / 4] >> (16 * (w & 1)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 qf = lds128(q_addr + (qb + u) * 512);
            float t[4];
            mma_first(t, a0[2 * u], a1[2 * u], a0[2 * u + 1], a1[2 * u + 1], qf.x, qf.y);
            mma(t, c0[2 * u], c1[2 * u], c0[2 * u + 1], c1[2 * u + 1], qf.z, qf.w);
            add(t, (u ? f_lo.y : f_lo.x) * kDown, (u ? f_hi.y : f_hi.x) * kDown);
          }
        }
      }
      if (GLOBAL) {
        const uint32_t at = base + Blk::kTile1 + gq * 64 + cq * 16;
        const uint4 x = lds128(at), y = lds128(at + 512);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
        const uint32_t tc_lo = lds32(base + Blk::kScale1 + gq * 4), tc_hi = lds32(base + Blk::kScale1 + gq * 4 + 32);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0[4], a1[4];
          kv4_halves(xw[w], a0);
          kv4_halves(yw[w], a1);
          const float2 f_lo = two_powers(tc_lo >> (8 * (w & 2))), f_hi = two_powers(tc_hi >> (8 * (w & 2)));
          const uint4 qf = lds128(q_addr + (12 + w) * 512);
          float t[4];
          mma_first(t, a0[0], a1[0], a0[1], a1[1], qf.x, qf.y);
          mma(t, a0[2], a1[2], a0[3], a1[3], qf.z, qf.w);
          add(t, (w & 1 ? f_lo.y : f_lo.x) * kDown, (w & 1 ? f_hi.y : f_hi.x) * kDown);
        }
      }
    }

    // ---- softmax of this lane's keys gq, gq + 8 for heads 2cq, 2cq + 1
    const uint32_t v_lo = blk[Blk::kTop + gq], v_hi = blk[Blk::kTop + gq + 8];
    const float ev_lo = v_lo == 255u ? NAN : (float)((int)v_lo - 127);
    const float ev_hi = v_hi == 255u ? NAN : (float)((int)v_hi - 127);
    float x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = (s[r] * qs[r & 1]) * kUp * p.scale_log2;
      y[r] = x[r] + (r < 2 ? ev_lo : ev_hi);
    }
    if (key0 < k_begin || key0 + kPage - 1 > k_end) {   // (the whole warp) keys outside are not seen
      const bool see_lo = key0 + gq >= k_begin && key0 + gq <= k_end;
      const bool see_hi = key0 + gq + 8 >= k_begin && key0 + gq + 8 <= k_end;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!(r < 2 ? see_lo : see_hi)) x[r] = y[r] = -INFINITY;
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
        for (int i = 0; i < S::kBlocks * 2; ++i) {
          o[i][j] *= al;
          o[i][2 + j] *= al;
        }
      }
    }
    float wgt[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) wgt[r] = ex2(y[r] - m2[r & 1] + kShift);
    const uint32_t b0 = transpose8x8(pack_f16(wgt[0], wgt[1]));   // keys 2cq, 2cq + 1 of head gq
    const uint32_t b1 = transpose8x8(pack_f16(wgt[2], wgt[3]));   // keys 2cq + 8, 2cq + 9
    __syncwarp();                                                   // the factors are in place

    // ---- O^T += V^T w^T: columns 4 gq .. + 3 of each block, keys 2cq, 2cq + 1, 2cq + 8, 2cq + 9
#pragma unroll
    for (int sg = 0; sg < S::kSegs; ++sg) {
      const uint32_t at = base + (GLOBAL ? 0u : (uint32_t)Blk::kTile1) + sg * 2048;
      const uint4 k0 = lds128(at + v_lane0), k1 = lds128(at + v_lane1);
      const uint4 k2 = lds128(at + v_lane0 + 1024), k3 = lds128(at + v_lane1 + 1024);
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
      const uint32_t w2[4] = {k2.x, k2.y, k2.z, k2.w}, w3[4] = {k3.x, k3.y, k3.z, k3.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // bytes of (key, key + 1): the even columns' codes, and the odd ones'
        const uint32_t ev0 = (w0[w] & 0x0f0f0f0fu) | ((w1[w] << 4) & 0xf0f0f0f0u);
        const uint32_t od0 = ((w0[w] >> 4) & 0x0f0f0f0fu) | (w1[w] & 0xf0f0f0f0u);
        const uint32_t ev1 = (w2[w] & 0x0f0f0f0fu) | ((w3[w] << 4) & 0xf0f0f0f0u);
        const uint32_t od1 = ((w2[w] >> 4) & 0x0f0f0f0fu) | (w3[w] & 0xf0f0f0f0u);
        uint32_t e0[4], d0[4], e1[4], d1[4];
        kv4_halves(ev0, e0);
        kv4_halves(od0, d0);
        kv4_halves(ev1, e1);
        kv4_halves(od1, d1);
        const uint4 f = lds128(f_addr + ((sg * 4 + w) * 4 + cq) * 16);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t wb0 = mul_f16(b0, u ? f.z : f.x), wb1 = mul_f16(b1, u ? f.w : f.y);
          const int vb = sg * 8 + 2 * w + u;
          mma(o[2 * vb], e0[2 * u], d0[2 * u], e1[2 * u], d1[2 * u], wb0, wb1);
          mma(o[2 * vb + 1], e0[2 * u + 1], d0[2 * u + 1], e1[2 * u + 1], d1[2 * u + 1], wb0, wb1);
        }
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
  constexpr int kTiles = S::kBlocks * 2, kLanes = GLOBAL ? 32 : 8;
  float4* red_o = reinterpret_cast<float4*>(smem);
  const int my = GLOBAL ? lane : gq;
  if (GLOBAL || cq == 0) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) red_o[(warp * kTiles + i) * kLanes + my] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
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
  // A thread merges, in warp order, the two row tiles of a block of one lane: four columns of two heads.
  for (int i = threadIdx.x; i < S::kBlocks * kLanes; i += kWarps * 32) {
    const int ln = i % kLanes, vb = i / kLanes;
    const int lq = GLOBAL ? ln >> 2 : ln, lc = GLOBAL ? ln & 3 : 0;
    float acc[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f0 = factor[w][2 * lc], f1 = factor[w][2 * lc + 1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 v = red_o[(w * kTiles + vb * 2 + u) * kLanes + ln];
        acc[0][2 * u] = fmaf(v.x * f0, f0, acc[0][2 * u]);
        acc[1][2 * u] = fmaf(v.y * f1, f1, acc[1][2 * u]);
        acc[0][2 * u + 1] = fmaf(v.z * f0, f0, acc[0][2 * u + 1]);
        acc[1][2 * u + 1] = fmaf(v.w * f1, f1, acc[1][2 * u + 1]);
      }
    }
    const int d = vb * 32 + lq * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (2 * lc + j >= G) continue;
      if (!PAGES && p.out) {   // the bits that the merge of one chunk gives
        const float f = inv_sum[2 * lc + j];
        *reinterpret_cast<uint2*>(p.out + ((size_t)b * p.cache.hq + (size_t)G * g + 2 * lc + j) * D + d) =
            make_uint2(pack_bf16(acc[j][0] * f, acc[j][1] * f), pack_bf16(acc[j][2] * f, acc[j][3] * f));
        continue;
      }
      *reinterpret_cast<float4*>(p.ws_o + (slot + (size_t)(2 * lc + j) * p.NC) * D + d) =
          make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    }
  }
}

template <bool GLOBAL, bool PAGES>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  static std::atomic<bool> done[64];   // per device; two first calls at once both set the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kv4_decode_kernel<GLOBAL, PAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<GLOBAL>::smem(PAGES));
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const long long blocks = (long long)p.NC * p.cache.hkv * p.B;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(kv4_decode_kernel<GLOBAL, PAGES>, (unsigned)blocks, Shape<GLOBAL>::kWarps * 32, Shape<GLOBAL>::smem(PAGES), s, p);
}

int slots(bool global, int max_pages, int window) {
  return chunk_slots(max_pages, global ? 0 : window, global ? kChunkGlobal : kChunkSliding);
}

}  // namespace

size_t kv4_decode_workspace_bytes(bool global, int B, int max_pages, int window, int hq, int hkv, bool pages) {
  return chunk_workspace_bytes(global, B, max_pages, hq, hkv, slots(global, max_pages, window), pages);
}

cudaError_t launch_kv4_decode(bool global, const void* q, const int32_t* seq_len, const int32_t* pos, int B, int window,
                              float scale_log2, const PagedCache4& cache, const NormArgs& nm, float* page_weights, void* out,
                              void* ws, const DeviceState& st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  ChunkParams p{};
  p.q = (const __nv_bfloat16*)q;
  p.seq_len = seq_len;
  p.pos = pos;
  p.B = B;
  p.window = global ? 0 : window;
  p.scale_log2 = scale_log2;
  p.cache = cache;
  p.nm = nm;
  p.NC = slots(global, cache.max_pages, window);
  // A page table of one chunk: nothing to merge.
  p.out = p.NC == 1 && !page_weights ? (__nv_bfloat16*)out : nullptr;
  place_workspace(p, global, ws, page_weights != nullptr);
  cudaError_t e = kv8_angles(global, &p.angles);
  if (e != cudaSuccess) return e;
  p.err = st.err;
  p.wait_ns = wait_limit_ns();
  if (!global)
    e = launch<false, false>(p, s);
  else
    e = page_weights ? launch<true, true>(p, s) : launch<true, false>(p, s);
  if (e != cudaSuccess || p.out) return e;
  if (!global) return finish<kSlidingD, false, kChunkSliding>(p, out, nullptr, s);
  return page_weights ? finish<kGlobalD, true, kChunkGlobal>(p, out, page_weights, s)
                      : finish<kGlobalD, false, kChunkGlobal>(p, out, nullptr, s);
}

}  // namespace g4
