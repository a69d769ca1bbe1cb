// What the decodes over the quantised caches (8-bit and 4-bit) have in common: a step's parameters and workspace,
// the query norm, small matrix wrappers, and the ordered merge of the chunks with the accumulated page weights.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "g4_kv8.cuh"

namespace g4 {

constexpr float kLazy = 8.0f;          // the weights' reference moves when the maximum grows by more than 2^8
constexpr float kShift = 7.0f;         // the weights' scale: w <= 2^(kLazy + kShift)
constexpr float kNone = -1.0e38f;      // running maximum before the first key (finite: no inf - inf)

struct ChunkParams {
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

// The norm of a query head held by a warp (lane: columns t0 .. and D/2 + t0 ..), times its weight; on a
// global layer's plain columns also the key norm's weight, which the stored S lacks. The result is cast
// to bf16 (a declared cast), as in the bf16 decode.
template <bool GLOBAL, int D, int R>
G4_DEV void norm_query(const NormArgs& nm, int t0, float (&a)[D / 64], float (&b)[D / 64]) {
  constexpr int P = D / 64;
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
    if (GLOBAL && nm.wk && t0 >= R) {
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
  for (int i = threadIdx.x; i < heads * D / 8; i += blockDim.x) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
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

template <int D, bool PAGES, int SPLIT, int CHUNK>
__global__ void __launch_bounds__(kFinishThreads) merge_chunks_kernel(const ChunkParams p, unsigned units,
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
    const int n = last < 0 ? 0 : min(p.NC, chunks_of(last, p.window, CHUNK));
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
  constexpr int kSpan = CHUNK < kFinishThreads * kPage ? kFinishThreads * kPage / CHUNK : 1;
  static_assert(!PAGES || kSpan * CHUNK == kFinishThreads * kPage, "a block's pages are whole chunks");
  __shared__ float factor[kSpan][kSlidingHq];
  const int unit = blockIdx.x - merge_blocks;
  const int b = unit / blocks_per_row, i0 = (unit % blocks_per_row) * kFinishThreads, i = i0 + threadIdx.x;
  int rope_pos;
  const int last = held_index(p.seq_len, p.pos, b, p.cache.max_pages, rope_pos);
  const int n_pages = (last >> 4) + 1;   // 0 when refused
  if (i0 >= n_pages) return;
  const int HKV = p.cache.hkv, G = hq / HKV;
  const int n = min(p.NC, chunks_of(last, 0, CHUNK));
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
    const int c = i0 / (CHUNK / kPage) + q;
    if (q < kSpan && h < hq) factor[q][h] = c < n && L != 0.f ? ex2(ml[c].x - M) / L : 0.f;   // (a NaN sum stays one)
  }
  __syncthreads();
  if (i >= n_pages) return;
  const float* f = factor[threadIdx.x / (CHUNK / kPage)];
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

// Chunk slots of a request at most (window 0: no window).
inline int chunk_slots(int max_pages, int window, int chunk) {
  const long long keys = (long long)max_pages * kPage < kMaxPos ? (long long)max_pages * kPage : kMaxPos;
  const int by_table = (int)((keys + chunk - 1) / chunk);
  if (window == 0) return by_table;
  const int by_window = (window - 1) / chunk + 2;
  return by_window < by_table ? by_window : by_table;
}

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

inline size_t chunk_workspace_bytes(bool global, int B, int max_pages, int hq, int hkv, int slots, bool pages) {
  const size_t nc = (size_t)slots, D = global ? kGlobalD : kSlidingD;
  size_t n = align256((size_t)B * hq * nc * 2 * sizeof(float)) + align256((size_t)B * hq * nc * D * sizeof(float));
  if (pages) n += (size_t)B * hkv * max_pages * 8 * sizeof(float);
  return n;
}

// Lays p's states out in the workspace (B, NC and the cache are set).
inline void place_workspace(ChunkParams& p, bool global, void* ws, bool pages) {
  const size_t D = global ? kGlobalD : kSlidingD;
  const size_t slots = (size_t)p.B * p.cache.hq * p.NC;
  uint8_t* w = (uint8_t*)ws;
  p.ws_ml = (float*)w;
  w += align256(slots * 2 * sizeof(float));
  p.ws_o = (float*)w;
  w += align256(slots * D * sizeof(float));
  p.ws_page = pages ? (float*)w : nullptr;
}

template <int D, bool PAGES, int CHUNK>
cudaError_t finish(const ChunkParams& p, void* out, float* page_weights, cudaStream_t s) {
  const long long units = (long long)p.B * p.cache.hq * (D / 128);
  const bool split = p.NC > 32;   // one warp's sixteen loads at a time would be a long chain
  const long long merge_blocks = split ? units : (units + 3) / 4;
  const int held = p.cache.max_pages < kMaxPos / kPage ? p.cache.max_pages : kMaxPos / kPage;   // pages at most
  const int per_row = (held + kFinishThreads - 1) / kFinishThreads;
  const long long blocks = merge_blocks + (PAGES ? (long long)p.B * per_row : 0);
  if (blocks > 0x7fffffffLL || units > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(split ? merge_chunks_kernel<D, PAGES, 4, CHUNK> : merge_chunks_kernel<D, PAGES, 1, CHUNK>, (unsigned)blocks,
                      kFinishThreads, 0, s, p, (unsigned)units, (unsigned)merge_blocks, per_row,
                      (__nv_bfloat16*)out, page_weights);
}

}  // namespace g4
