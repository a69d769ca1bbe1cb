// The page plan of a serving step: which requests are served, their page tables, slots and positions, and the pages
// that come back, in one launch.
//
// Every block goes through all requests (two scans over them: the rows and pages that each request wants, then the
// pages that the served ones take and give back) and keeps the running sums in shared memory; then the blocks share
// the rows, the taken pages and the returned pages out and find each one's request by bisection. So no sum travels
// between blocks and nothing is kept in a workspace. The blocks are one cluster: its barrier stands between the last
// read of the requests' state and the first write, so that the outputs may be the inputs.
//
// The free pages are a ring: pages are taken at its head and come back behind its tail, so that reads and writes of a
// step never meet, and what comes back can be taken from the next step on. Every place is fixed by the requests'
// order, not by timing.
//
// Bound by latency: a chain of loads, two scans, a search, a load and a store, and in a small step by the instructions
// themselves, which come from memory (a version with its loops unrolled over four items took 10.3 us instead of 3.9 for
// 64 decoding requests). Of 4096 requests' 24 us some 7 are the loads and what is computed of them, 3 the scans, 1 the
// state, 7 the 110 thousand rows and 6 the pages, by leaving parts out; a row costs the same without its loads or its stores, and searching
// on from the last owner in place of a bisection gains nothing.
#include <atomic>

#include "g4_kv8.cuh"
#include "g4_plan.h"

namespace g4 {

namespace {

G4_DEV int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

// Sums over the block before this thread, and of the whole block, of N values. buf: [2][N][32].
template <int N>
G4_DEV void block_scan(const uint32_t (&x)[N], uint32_t (&before)[N], uint32_t (&total)[N], uint32_t* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t v = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += up;
    }
    before[i] = v - x[i];
    if (lane == 31) buf[i * 32 + warp] = v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w = lane < (int)(blockDim.x >> 5) ? buf[i * 32 + lane] : 0u;   // of warp `lane`
    before[i] += __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
    total[i] = __reduce_add_sync(0xffffffffu, w);
  }
  __syncthreads();
}

// The first i < n with end[i] > x (ends ascend; there is one).
G4_DEV int owner_of(const uint32_t* end, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}
G4_DEV uint32_t start_of(const uint32_t* end, int i) { return i ? end[i - 1] : 0u; }

G4_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
G4_DEV uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

// Thread t's K neighbouring values of n.
template <int K>
G4_DEV void get(const int32_t* from, int t, int n, int (&x)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = t * K + k < n ? from[t * K + k] : 0;
}
// To shared memory (16-byte aligned, with room for the last thread's K); four of them in one store, which has no bank
// conflicts (4096 requests: 25.5 -> 24.2 us).
template <int K>
G4_DEV void put(uint32_t* to, int t, const uint32_t (&x)[K]) {
  if (K == 4)
    reinterpret_cast<uint4*>(to)[t] = make_uint4(x[0], x[1 % K], x[2 % K], x[3 % K]);
  else
#pragma unroll
    for (int k = 0; k < K; ++k) to[t * K + k] = x[k];
}

// What the second half needs of a request, in shared memory, [field][request].
enum Field { kRowEnd, kCtx, kTake0, kGive0, kLost0, kFirst0, kTake1, kGive1, kLost1, kFirst1, kFields };

// K requests per thread; a thread handles ITEMS neighbouring rows or pages together.
template <int K, int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) plan_pages_kernel(const PlanArgs p) {
  extern __shared__ __align__(16) uint32_t req[];   // [kFields][B up to K]
  __shared__ uint32_t buf[4 * 32];
  wait_for_grid();
  let_next_grid_start();
  const int B = p.B;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int pad = (B + K - 1) / K * K;
  auto field = [&](int f) { return req + (size_t)f * pad; };
  const bool any = threadIdx.x * K < B;

  // Each group's ring; one that contradicts itself gives and takes nothing.
  uint32_t head[kPlanGroups], count[kPlanGroups];
  bool sound[kPlanGroups];
#pragma unroll
  for (int g = 0; g < kPlanGroups; ++g) {
    head[g] = count[g] = 0;
    sound[g] = false;
    if (g >= p.n_groups) continue;
    const int h = p.group[g].pool[0], c = p.group[g].pool[1], n = p.group[g].num_pages;
    sound[g] = h >= 0 && h < n && c >= 0 && c <= n;
    if (!sound[g]) continue;
    head[g] = (uint32_t)h;
    count[g] = (uint32_t)c;
  }

  // ---- what each request wants: rows, and pages of each group
  int ctx[K], add[K], held[K][kPlanGroups], first[K][kPlanGroups], lost[K][kPlanGroups], back[K][kPlanGroups];
  bool ended[K], valid[K], served[K];
  uint32_t need[K][kPlanGroups];
  uint32_t sum[3] = {0, 0, 0};   // rows, pages
  get<K>(p.ctx_len, threadIdx.x, B, ctx);
  get<K>(p.new_len, threadIdx.x, B, add);
#pragma unroll
  for (int g = 0; g < kPlanGroups; ++g) {
    int x[3][K] = {};
    if (g < p.n_groups) {
      const PlanGroup& q = p.group[g];
      if (q.first_page) get<K>(q.first_page, threadIdx.x, B, x[0]);
      if (q.lost) get<K>(q.lost, threadIdx.x, B, x[1]);
      if (q.n_freed) get<K>(q.n_freed, threadIdx.x, B, x[2]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      first[k][g] = x[0][k];
      lost[k][g] = x[1][k];
      back[k][g] = x[2][k];
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const bool in = (int)threadIdx.x * K + k < B;
    const int n = add[k];
    add[k] = n > 0 && n <= kMaxPos ? n : 0;   // its rows keep their place whether it is served or not
    ended[k] = n == -1;
    valid[k] = n >= -1 && n <= kMaxPos && ctx[k] >= 0 && ctx[k] <= kMaxPos - add[k];
#pragma unroll
    for (int g = 0; g < kPlanGroups; ++g) {
      held[k][g] = 0;
      if (g >= p.n_groups || !in) continue;
      const PlanGroup& q = p.group[g];
      const int f = back[k][g], most = min(q.max_pages, kMaxPos / kPage);
      valid[k] = valid[k] && f >= 0 && f <= most && lost[k][g] >= 0 && lost[k][g] <= ctx[k] - kPage * f;
      held[k][g] = ctx[k] - (lost[k][g] + kPage * f);
      valid[k] = valid[k] && pages_of(held[k][g] + add[k]) <= most && first[k][g] >= 0 && first[k][g] <= pages_of(held[k][g]);
    }
    sum[0] += (uint32_t)add[k];
#pragma unroll
    for (int g = 0; g < kPlanGroups; ++g) {
      need[k][g] = valid[k] && g < p.n_groups ? (uint32_t)(pages_of(held[k][g] + add[k]) - pages_of(held[k][g])) : 0u;
      sum[1 + g] += need[k][g];
    }
  }
  uint32_t at[3], all[3];
  block_scan<3>(sum, at, all, buf);
  const uint32_t rows = all[0];

  // ---- who is served, and what comes back
  uint32_t move[4] = {0, 0, 0, 0};   // pages taken and given back, by group
  uint32_t row_start[K], row_end[K], ctx_served[K], was_first[kPlanGroups][K], is_lost[kPlanGroups][K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    row_start[k] = at[0];
    at[0] += (uint32_t)add[k];
    served[k] = valid[k] && add[k] > 0 && at[0] <= (uint32_t)p.T;
#pragma unroll
    for (int g = 0; g < kPlanGroups; ++g) {
      at[1 + g] += need[k][g];
      if (g < p.n_groups) served[k] = served[k] && (need[k][g] == 0 || at[1 + g] <= count[g]);
    }
    row_end[k] = at[0];
    ctx_served[k] = (uint32_t)ctx[k] * 2u + (served[k] ? 1u : 0u);
#pragma unroll
    for (int g = 0; g < kPlanGroups; ++g) {
      was_first[g][k] = is_lost[g][k] = 0;
      if (g >= p.n_groups) continue;
      const int W = p.group[g].window;
      if (!valid[k]) back[k][g] = 0;
      const int now_lost = lost[k][g] + kPage * back[k][g];
      int to = first[k][g];   // own pages first .. to - 1 go back, after the evicted ones
      if (valid[k] && ended[k])
        to = pages_of(held[k][g]);
      else if (served[k] && W > 0)
        to = max(to, max(0, held[k][g] - W + 1) / kPage);
      is_lost[g][k] = (uint32_t)now_lost;
      was_first[g][k] = (uint32_t)first[k][g] | ((uint32_t)back[k][g] << 16);   // both at most 16384
      lost[k][g] = now_lost;
      back[k][g] += to - first[k][g];
      first[k][g] = to;
      if (!served[k]) need[k][g] = 0;
      move[2 * g] += need[k][g];
      move[2 * g + 1] += (uint32_t)back[k][g];
    }
  }
  if (any) {
    put<K>(field(kRowEnd), threadIdx.x, row_end);
    put<K>(field(kCtx), threadIdx.x, ctx_served);
#pragma unroll
    for (int g = 0; g < kPlanGroups; ++g) {
      if (g >= p.n_groups) continue;
      put<K>(field(kLost0 + 4 * g), threadIdx.x, is_lost[g]);
      put<K>(field(kFirst0 + 4 * g), threadIdx.x, was_first[g]);
    }
  }
  uint32_t at4[4], all4[4];
  block_scan<4>(move, at4, all4, buf);
  bool give[kPlanGroups];
#pragma unroll
  for (int g = 0; g < kPlanGroups; ++g)
    give[g] = g < p.n_groups && sound[g] && all4[2 * g + 1] <= (uint32_t)p.group[g].num_pages - count[g];
#pragma unroll
  for (int g = 0; g < kPlanGroups; ++g) {
    if (g >= p.n_groups || !any) continue;
    uint32_t take[K], given[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      take[k] = at4[2 * g] += need[k][g];
      given[k] = at4[2 * g + 1] += (uint32_t)back[k][g];
    }
    put<K>(field(kTake0 + 4 * g), threadIdx.x, take);
    put<K>(field(kGive0 + 4 * g), threadIdx.x, given);
  }
  __syncthreads();
  cluster_sync();   // every block has read the state: from here on it is written

  // ---- the requests' state, shared out by warps
  if ((threadIdx.x >> 5) % ranks == rank) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = threadIdx.x * K + k;
      if (b >= B) continue;
      if (!valid[k]) set_error(p.err, kErrPos);
      const int rows_of = served[k] ? add[k] : 0;
      const bool gone = valid[k] && ended[k];
      p.out_ctx_len[b] = gone ? 0 : ctx[k] + rows_of;
      p.q_start[b] = (int32_t)row_start[k];
      p.q_len[b] = rows_of;
      p.ctx_start[b] = ctx[k];
#pragma unroll
      for (int g = 0; g < kPlanGroups; ++g) {
        if (g >= p.n_groups) continue;
        const PlanGroup& q = p.group[g];
        q.seq_len[b] = served[k] ? held[k][g] + add[k] : 0;
        if (q.out_first_page) q.out_first_page[b] = gone ? 0 : first[k][g];
        if (q.out_lost) q.out_lost[b] = gone ? 0 : lost[k][g];
        if (q.out_n_freed) q.out_n_freed[b] = valid[k] ? 0 : q.n_freed[b];   // its pages come back once
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kPlanGroups; ++g) {
    if (g >= p.n_groups || rank != 0 || threadIdx.x != 0) continue;
    const PlanGroup& q = p.group[g];
    if (!give[g]) set_error(p.err, kErrPage);
    if (sound[g]) {
      uint32_t h = head[g] + all4[2 * g];
      if (h >= (uint32_t)q.num_pages) h -= (uint32_t)q.num_pages;
      q.out_pool[0] = (int32_t)h;
      q.out_pool[1] = (int32_t)(count[g] - all4[2 * g] + (give[g] ? all4[2 * g + 1] : 0u));
    } else {
      const int h = q.pool[0], c = q.pool[1];   // (only this thread writes out_pool)
      q.out_pool[0] = h;
      q.out_pool[1] = c;
    }
  }

  // ---- rows (positions and slots), pages taken, pages given back: a thread takes ITEMS neighbouring ones at a time,
  // mostly of one request, so that it searches once and has their loads in flight together; the kinds of work follow one
  // another in the threads' numbering, so that in a small step they run side by side.
  auto do_rows = [&](uint32_t r0) {
    int pos[ITEMS], page[ITEMS][kPlanGroups], place[ITEMS][kPlanGroups];
    int b = -1;
    uint32_t end = 0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t r = r0 + i;
      pos[i] = -1;
#pragma unroll
      for (int g = 0; g < kPlanGroups; ++g) page[i][g] = -1;
      if (r >= rows || r >= (uint32_t)p.T) continue;
      if (b < 0 || r >= end) {
        b = owner_of(field(kRowEnd), B, r);
        end = field(kRowEnd)[b];
      }
      const uint32_t c = field(kCtx)[b];
      if (!(c & 1u)) continue;
      const int ctx_b = (int)(c >> 1);
      pos[i] = ctx_b + (int)(r - start_of(field(kRowEnd), b));
#pragma unroll
      for (int g = 0; g < kPlanGroups; ++g) {
        if (g >= p.n_groups) continue;
        const PlanGroup& q = p.group[g];
        const int lost_b = (int)field(kLost0 + 4 * g)[b], key = pos[i] - lost_b;
        const int past = (key >> 4) - pages_of(ctx_b - lost_b);   // >= 0: one of the pages taken now
        uint32_t j = head[g] + start_of(field(kTake0 + 4 * g), b) + (uint32_t)past;
        if (j >= (uint32_t)q.num_pages) j -= (uint32_t)q.num_pages;
        page[i][g] = past >= 0 ? q.free_pages[j] : q.page_table[(size_t)b * q.max_pages + (key >> 4)];
        place[i][g] = key & 15;
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t r = r0 + i;
      if (r >= (uint32_t)p.T) break;
      if (p.positions) p.positions[r] = pos[i];
#pragma unroll
      for (int g = 0; g < kPlanGroups; ++g) {
        if (g >= p.n_groups) continue;
        const bool in = page[i][g] >= 0 && page[i][g] < p.group[g].num_pages;
        if (pos[i] >= 0 && !in) set_error(p.err, kErrPage);
        if (p.group[g].slots) p.group[g].slots[r] = in ? (long long)page[i][g] * kPage + place[i][g] : -1;
      }
    }
  };
  auto do_takes = [&](int g, uint32_t i0, uint32_t total) {
    const PlanGroup& q = p.group[g];
    const uint32_t head_g = g ? head[1] : head[0];
    const uint32_t* ends = field(kTake0 + 4 * g);
    int page[ITEMS];
    int32_t* to[ITEMS];
    int b = -1;
    uint32_t end = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t i = i0 + k;
      to[k] = nullptr;
      if (i >= total) continue;
      if (b < 0 || i >= end) {
        b = owner_of(ends, B, i);
        end = ends[b];
      }
      const int held_b = (int)(field(kCtx)[b] >> 1) - (int)field(kLost0 + 4 * g)[b];
      uint32_t from = head_g + i;
      if (from >= (uint32_t)q.num_pages) from -= (uint32_t)q.num_pages;
      page[k] = q.free_pages[from];
      to[k] = q.page_table + (size_t)b * q.max_pages + pages_of(held_b) + (i - start_of(ends, b));
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (to[k]) *to[k] = page[k];
  };
  auto do_gives = [&](int g, uint32_t i0, uint32_t total) {
    const PlanGroup& q = p.group[g];
    const uint32_t tail = g ? head[1] + count[1] : head[0] + count[0];
    const uint32_t* ends = field(kGive0 + 4 * g);
    int page[ITEMS];
    int b = -1;
    uint32_t end = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t i = i0 + k;
      page[k] = 0;
      if (i >= total) continue;
      if (b < 0 || i >= end) {
        b = owner_of(ends, B, i);
        end = ends[b];
      }
      const uint32_t off = i - start_of(ends, b), f = field(kFirst0 + 4 * g)[b], evicted = f >> 16;
      page[k] = off < evicted ? q.freed[(size_t)b * q.max_pages + off]
                              : q.page_table[(size_t)b * q.max_pages + (f & 0xffffu) + (off - evicted)];
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t i = i0 + k;
      if (i >= total) break;
      if (page[k] < 0 || page[k] >= q.num_pages) set_error(p.err, kErrPage);   // (a call that meets it later refuses it)
      uint32_t to = tail + i;
      if (to >= (uint32_t)q.num_pages) to -= (uint32_t)q.num_pages;
      q.free_pages[to] = page[k];
    }
  };
  auto units = [](uint32_t n) { return (n + ITEMS - 1) / ITEMS; };
  const uint32_t u_rows = units((uint32_t)p.T);
  const uint32_t u_take0 = u_rows + units(all4[0]), u_give0 = u_take0 + (give[0] ? units(all4[1]) : 0u);
  const uint32_t u_take1 = u_give0 + units(all4[2]), u_give1 = u_take1 + (give[1] ? units(all4[3]) : 0u);
  for (uint32_t u = rank * THREADS + threadIdx.x; u < u_give1; u += ranks * THREADS) {
    if (u < u_rows) {
      do_rows(u * ITEMS);
    } else {   // (one copy of the code for both groups: a small step runs it once, from memory)
      const int g = u >= u_give0;
      const uint32_t from = g ? u_give0 : u_rows, mid = g ? u_take1 : u_take0;
      if (u < mid)
        do_takes(g, (u - from) * ITEMS, g ? all4[2] : all4[0]);
      else
        do_gives(g, (u - mid) * ITEMS, g ? all4[3] : all4[1]);
    }
  }
}

template <int K, int THREADS, int ITEMS>
cudaError_t launch(const PlanArgs& p, unsigned blocks, cudaStream_t s) {
  static std::atomic<bool> done[64];   // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(plan_pages_kernel<K, THREADS, ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kFields * K * THREADS * (int)sizeof(uint32_t));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(plan_pages_kernel<K, THREADS, ITEMS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)kFields * ((p.B + K - 1) / K * K) * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;   // (a lone block is a cluster of its own)
  return cudaLaunchKernelEx(&cfg, plan_pages_kernel<K, THREADS, ITEMS>, p);
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs& p, cudaStream_t s) {
  // Few requests: a small block, whose barriers are short, and one of them while its threads can take the rows in a few
  // turns (64 decoding requests take 3.7 us, with 16 blocks 4.1, with the large block 5.2; 300 mixed ones with 32 thousand
  // rows 8.0, with a cluster of 8 11.2). The rule looks at the rows, not at the pages that come back, which the lengths
  // alone tell: a lone block hands them out 256 at a time, so that a step of 64 in which four requests of 32768 keys end
  // takes 26 us, one in which all do 347 (of 300 requests, by the cluster, one of 131072 keys ends in 6.7). Many requests:
  // two rows or pages a thread at a time (4096 requests, 110 thousand rows: 24.2 us; one takes 1.6 more, four 4.5 more),
  // held to 64 registers with 168 bytes spilled.
  if (p.B <= 256) return launch<1, 256, 1>(p, p.T <= 1024 ? 1 : 16, s);
  if (p.B <= 1024) return launch<1, 1024, 1>(p, 16, s);
  return launch<kPlanRequests / 1024, 1024, 2>(p, 16, s);
}

}  // namespace g4
