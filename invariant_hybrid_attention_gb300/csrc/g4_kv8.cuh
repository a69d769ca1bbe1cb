// The 8-bit paged cache: its block layout and the cast between fp32 vectors and stored bytes.
//
// A page-head block holds 16 keys of one KV head as two tiles and the exponents of their vectors:
//   sliding: K' (16 x 256), V (16 x 256);   global: S (16 x 512), the turned columns of K (16 x 128)
//   [tile 0][tile 1][16 exponent bytes of tile 0][16 of tile 1]
// A tile is [columns / 128][16 keys][128 bytes]; the 16-byte piece c of key j's 128-byte line sits at
// piece c ^ kv8_swizzle(j). One key's 128 columns are one line, so an append writes whole lines and
// never reads one back. The swizzle lets the decode kernels read the same bytes from shared memory
// in two orders, each 16 bytes a lane and without bank conflicts: a quarter warp reads 4 pieces of
// two neighbouring keys (rows of K for Q.K^T) or two neighbouring pieces of 4 even (or 4 odd) keys
// (columns of V for P.V).
//
// A head vector x (one token of one head) is stored with one power-of-two step:
//   a = max |x|, E = floor(log2 a) - 6, code = clamp(rne(x / 2^E), -127, 127); byte = code + 128,
//   exponent byte = the biased fp32 exponent of a = E + 133; 0 (all codes 0) when a < 2^-119; 255
//   when x holds an infinity or NaN (the vector then reads as NaN).
// The step is a power of two so that x / 2^E is exact, the one rounding is to the code, and the value
// code * 2^E is itself a bf16 number: reading the cache back loses nothing. One step per token and
// head, not per page: a longer block would make a key's bytes depend on the tokens appended after
// it, and so on how a prompt was cut into chunks; it would save at most 1 byte in 128.
#pragma once

#include "g4_internal.h"

namespace g4 {

template <bool GLOBAL>
struct Kv8Block {
  static constexpr int D = GLOBAL ? kGlobalD : kSlidingD;
  static constexpr int R = GLOBAL ? kGlobalR : kSlidingR;
  static constexpr int kCols1 = GLOBAL ? 2 * kGlobalR : kSlidingD;   // columns of tile 1
  static constexpr int kTile1 = kPage * D;                           // byte offset of tile 1
  static constexpr int kExp0 = kTile1 + kPage * kCols1;              // exponents of tile 0
  static constexpr int kExp1 = kExp0 + kPage;                        // exponents of tile 1
  static constexpr int kBytes = kExp1 + kPage;                       // 8224 sliding, 10272 global
};

// Pieces of key j's line are xored with this: 0, 4, 2, 6, 4, 0, 6, 2 for j = 0 .. 7.
__host__ __device__ constexpr int kv8_swizzle(int j) { return (j & 6) ^ ((j & 1) << 2); }

// Byte offset of column d of key j in a tile.
__host__ __device__ constexpr int kv8_offset(int j, int d) {
  return (d >> 7) * 2048 + j * 128 + ((((d >> 4) & 7) ^ kv8_swizzle(j)) << 4) + (d & 15);
}

// The step 2^(biased - 133) of a stored vector as fp32; NaN for 255.
G4_DEV float kv8_step(uint32_t biased) {
  const uint32_t b = biased < 8u ? 8u : biased;
  return __uint_as_float(biased == 255u ? 0x7fc00000u : (b - 6u) << 23);
}

// The exponent byte of a vector whose largest |x| has these fp32 bits (sign cleared): integer order
// puts NaN above infinity above every number.
G4_DEV uint32_t kv8_exponent(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e < 8u ? 0u : e;
}

// 1 / step for exponents 8 .. 254.
G4_DEV float kv8_inverse_step(uint32_t biased) { return __uint_as_float((260u - biased) << 23); }

// Eight consecutive columns as stored bytes (biased: the vector's exponent byte). x / step is exact;
// adding 1.5 * 2^23 + 128 rounds it to a whole number, half to even, and leaves code + 128 in the
// sum's low byte.
G4_DEV uint2 kv8_codes(const float (&x)[8], uint32_t biased) {
  if (biased == 0u || biased == 255u) return make_uint2(0x80808080u, 0x80808080u);
  const float inv = kv8_inverse_step(biased), mid = 12583040.0f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = __float_as_uint(fminf(fmaxf(fmaf(x[i], inv, mid), mid - 127.0f), mid + 127.0f));
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040),
                       0x5410);
  return make_uint2(w[0], w[1]);
}

// ---- angles ------------------------------------------------------------------------------------------
// Tables of (cos, sin) in two fp32 parts (cos, sin, and what their rounding left), entry-major: coarse[c][t]
// of 256 c f_t, fine[a][t] of a f_t, 0 <= a < 256. Static, each layer kind's filled by its first 8-bit append
// or decode on a device (1.3 or 2.6 MB), which may be part of a capture.
struct Kv8Angles {
  const float4* coarse;   // [kRopeCoarse][R]
  const float4* fine;     // [256][R]
};
cudaError_t kv8_angles(bool global, Kv8Angles* out);   // for the current device

// a b - c d and its kind in two fp32 parts: products exact through fma, the sum's error kept, one rounding
// at the end.
G4_DEV float dot2_exact(float ah, float al, float bh, float bl, float ch, float cl, float dh, float dl) {
  const float p = ah * bh, pe = fmaf(ah, bh, -p);
  const float q = ch * dh, qe = fmaf(ch, dh, -q);
  const float s = p + q, z = s - p;
  const float se = (p - (s - z)) + (q - z);
  float low = fmaf(ah, bl, fmaf(al, bh, fmaf(ch, dl, fmaf(cl, dh, pe + qe))));
  return s + (se + low);
}

// (cos, sin)(pos * f_t) rounded once to fp32 (nearly always to the nearest): the angle-addition formula
// on the two-part tables. Where rope_cs carries the rounding of three table entries and two products
// (a few 2^-24), this leaves 2^-25, so that a value next to a border between two codes falls on the
// border's right side as often as with exactly rounded angles.
G4_DEV float2 rope_cs_exact(float4 a, float4 b) {
  return make_float2(dot2_exact(a.x, a.z, b.x, b.z, -a.y, -a.w, b.y, b.w),
                     dot2_exact(a.y, a.w, b.x, b.z, a.x, a.z, b.y, b.w));
}

// The rotation of one half-split pair with every product and sum rounded by itself. What is rounded again
// next (to bf16, to a code) then agrees with the elementary operations on fp32 angles, border values
// included, so that two programs that follow the definition store and compare the same numbers.
G4_DEV void rope_pair_apart(float& lo, float& hi, float2 cs) {
  const float a = lo, b = hi;
  lo = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  hi = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// ---- launches ----------------------------------------------------------------------------------------
// Programmatic dependent launch. Every kernel of the 8-bit cache waits for the grid before it at its
// first instruction (its end and its writes), and then lets the next grid of the stream start: back to
// back, the launch of one hides behind the other, and nothing is read early.
G4_DEV void wait_for_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
G4_DEV void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t s,
                         const Args&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Paged 8-bit cache of one layer, and the head counts of the call.
struct PagedCache8 {
  uint8_t* pages;
  int32_t num_pages;
  const int32_t* page_table;
  int32_t max_pages;
  int32_t hq;
  int32_t hkv;
};

// Which keys of each sequence g4attn_kv8_unpack or a prefill reads back: key_begin .. key_end - 1, or
// (key_begin NULL) the keys that the rows of a prefill see, new rows included.
struct Kv8Range {
  const int32_t* key_begin;
  const int32_t* key_end;
  SeqRows rows;   // B; the rest when key_begin is NULL
  int window;     // with key_begin NULL: keys before ctx_start - window + 1 (and the first row's image) are not read
                  // (0: all are)
};

// The rows' queries alone, staged into q_out as launch_append_prefill does (normed, turned, bf16); of the
// cache only hq, hkv and max_pages are read.
cudaError_t launch_stage_queries(bool global, const void* q, void* q_out, const SeqRows& rows, const PagedCache& cache,
                                 const DeviceState& st, cudaStream_t s, const NormArgs& nm);

// Writes the rows of a prefill batch into 8-bit pages.
cudaError_t launch_kv8_append(bool global, const void* k, const void* v, const SeqRows& rows, const PagedCache8& cache,
                              const NormArgs& nm, const DeviceState& st, cudaStream_t s);
// Writes one new token per request at held index seq_len - 1, turned by pos (NULL: the held index).
cudaError_t launch_kv8_append_decode(bool global, const void* k_new, const void* v_new, const int32_t* seq_len,
                                     const int32_t* pos, int B, const PagedCache8& cache, const NormArgs& nm,
                                     const DeviceState& st, cudaStream_t s);
// Reads keys of 8-bit pages back into bf16 pages (dst.page_table: the destination's page table).
cudaError_t launch_kv8_unpack(bool global, const Kv8Range& range, const PagedCache8& src, const PagedCache& dst,
                              const DeviceState& st, cudaStream_t s);
size_t kv8_decode_workspace_bytes(bool global, int B, int max_pages, int window, int hq, int hkv, bool pages);
// Decode partials, ordered merge and (page_weights set) the accumulated page weights.
cudaError_t launch_kv8_decode(bool global, const void* q, const int32_t* seq_len, const int32_t* pos, int B, int window,
                              float scale_log2, const PagedCache8& cache, const NormArgs& nm, float* page_weights,
                              void* out, void* ws, const DeviceState& st, cudaStream_t s);
cudaError_t launch_evict_pages(const int32_t* seq_len, const int32_t* table, const float* weights, int B, int max_pages,
                               int keep, int first, int last, int32_t* out_len, int32_t* out_table, float* out_weights,
                               int32_t* freed, int32_t* n_freed, const DeviceState& st, cudaStream_t s);

}  // namespace g4
