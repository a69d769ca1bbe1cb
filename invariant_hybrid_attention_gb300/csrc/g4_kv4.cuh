// The 4-bit paged cache: its block layout and the cast between fp32 vectors and stored codes.
//
// A head vector (one token of one head) is stored in microscaled 4-bit floating point: E2M1 codes (sign, then
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one power-of-two scale 2^(s - 127) per block of 32 columns:
//   a = max |x| over the block, E = floor(log2 a) - 2, one more when a > 7 2^E; code = the nearest step of x / 2^E,
//   ties to the even code, 6 at most; s = E + 127.
// E grows at 7 2^E and not at 6 2^E: up to there the largest step, 6, is still within half a step (1) of x, so that
// no column is off by more than 2^E, and the other columns keep the finer scale. x / 2^E is exact, the one rounding
// is to the code, and a value is a bf16 number. A block with a < 2^-77 is zeros, s = 0 (else s >= 48, so that the
// decode's powers of two stay in fp32's range); s is at most 252 (E = 125; 6 2^125 is finite). A vector that holds an
// infinity or NaN has s = 255 and zero codes in all its blocks and reads as NaN.
//
// A page-head block holds 16 keys of one KV head as two tiles, their scales, and each key's largest scale of the
// tensor that serves as V (its "top"; 255 for a NaN vector):
//   sliding: K' (16 x 256), V (16 x 256);   global: S (16 x 512), the turned columns of K (16 x 128)
//   [tile 0][tile 1][16 keys][scales of tile 0][16 keys][scales of tile 1][16 tops]
// A wide tile is [columns / 256][16 keys][128 bytes]; the 16-byte piece c of key j's line sits at piece
// c ^ kv8_swizzle(j), and piece c holds columns 4c .. 4c + 3 of each of the 8 blocks, two bytes a block. So one
// 16-byte read gives a lane four columns of eight blocks, which is what the decode's matrix operands want in both
// orders, without bank conflicts: for Q.K^T lane c takes pieces c and c + 4 of its key (8 columns of every block),
// for P.V lane c takes piece c of four keys (4 columns of every block). The turned columns are only keys:
// [16 keys][64 bytes], piece c holding columns 4c .. and 16 + 4c .. of each of the 4 blocks, four bytes a block.
#pragma once

#include "g4_kv8.cuh"

namespace g4 {

template <bool GLOBAL>
struct Kv4Block {
  static constexpr int D = GLOBAL ? kGlobalD : kSlidingD;
  static constexpr int R = GLOBAL ? kGlobalR : kSlidingR;
  static constexpr int kCols1 = GLOBAL ? 2 * kGlobalR : kSlidingD;   // columns of tile 1
  static constexpr int kBlocks0 = D / 32, kBlocks1 = kCols1 / 32;    // scales per key
  static constexpr int kTile1 = kPage * D / 2;                       // byte offset of tile 1
  static constexpr int kScale0 = kTile1 + kPage * kCols1 / 2;
  static constexpr int kScale1 = kScale0 + kPage * kBlocks0;
  static constexpr int kTop = kScale1 + kPage * kBlocks1;
  static constexpr int kBytes = kTop + kPage;                        // 4368 sliding, 5456 global
  static_assert(kBytes % 16 == 0 && kScale0 % 16 == 0 && kScale1 % 16 == 0 && kTop % 16 == 0, "bulk copies, wide loads");
};

// Byte offset of piece c (0 .. 7) of key j in 256-column segment sg of a wide tile; of piece c (0 .. 3) of key j of
// the turned columns.
__host__ __device__ constexpr int kv4_piece(int sg, int j, int c) { return sg * 2048 + j * 128 + ((c ^ kv8_swizzle(j)) << 4); }
__host__ __device__ constexpr int kv4_turned_piece(int j, int c) { return j * 64 + c * 16; }

// The scale byte of a block whose largest |x| has these fp32 bits (sign cleared, finite): adding 0x1fffff carries
// into the exponent when the mantissa is above 1.75.
G4_DEV uint32_t kv4_scale(uint32_t max_bits) {
  const uint32_t e = min((max_bits + 0x1fffffu) >> 23, 254u);
  return max_bits < (50u << 23) ? 0u : e - 2u;   // below 2^-77: zeros
}

// Eight consecutive columns as codes, column i in bits 4i .. 4i + 3 (scale: their block's byte, 0 and 255: zeros).
G4_DEV uint32_t kv4_codes(const float (&x)[8], uint32_t scale) {
  if (scale == 0u || scale == 255u) return 0u;
  const float inv = __uint_as_float((254u - scale) << 23);   // 2^(127 - s), exact
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv), "f"(x[4] * inv), "f"(x[5] * inv),
        "f"(x[6] * inv), "f"(x[7] * inv));
  return w;
}

// The four bytes of w as pairs of fp16 numbers (h[i]: codes 2i in the low half and 2i + 1), without their scale.
G4_DEV void kv4_halves(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(s - 127) as fp32 for s in 1 .. 254; NaN for 255, 0 for 0 (its codes are zeros).
G4_DEV float kv4_factor(uint32_t scale) { return __uint_as_float(scale == 255u ? 0x7fc00000u : scale << 23); }

using PagedCache4 = PagedCache8;

// Writes the rows of a prefill batch into 4-bit pages.
cudaError_t launch_kv4_append(bool global, const void* k, const void* v, const SeqRows& rows, const PagedCache4& cache,
                              const NormArgs& nm, const DeviceState& st, cudaStream_t s);
// Writes one new token per request at held index seq_len - 1, turned by pos (NULL: the held index); none where
// seq_len is 0.
cudaError_t launch_kv4_append_decode(bool global, const void* k_new, const void* v_new, const int32_t* seq_len,
                                     const int32_t* pos, int B, const PagedCache4& cache, const NormArgs& nm,
                                     const DeviceState& st, cudaStream_t s);
// Reads keys of 4-bit pages back into bf16 pages (dst.page_table: the destination's page table).
cudaError_t launch_kv4_unpack(bool global, const Kv8Range& range, const PagedCache4& src, const PagedCache& dst,
                              const DeviceState& st, cudaStream_t s);
size_t kv4_decode_workspace_bytes(bool global, int B, int max_pages, int window, int hq, int hkv, bool pages);
// Decode partials, ordered merge and (page_weights set) the accumulated page weights.
cudaError_t launch_kv4_decode(bool global, const void* q, const int32_t* seq_len, const int32_t* pos, int B, int window,
                              float scale_log2, const PagedCache4& cache, const NormArgs& nm, float* page_weights,
                              void* out, void* ws, const DeviceState& st, cudaStream_t s);

}  // namespace g4
