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

// Programmatic dependent launch. Every kernel of the 8-bit cache waits for the grid before it at its
// first instruction (its end and its writes), and then lets the next grid of the stream start: back to
// back, the launch of one hides behind the other, and nothing is read early.
G4_DEV void wait_for_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
G4_DEV void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_early_clusters(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem,
                                  unsigned cluster, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t s,
                         const Args&... args) {
  return launch_early_clusters(kernel, blocks, threads, smem, 1, s, args...);
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
  int window;     // with key_begin NULL: keys before ctx_start - window + 1 are not read (0: none)
};

}  // namespace g4
