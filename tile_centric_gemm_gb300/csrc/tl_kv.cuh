// tl_kv.cuh -- the 8-bit paged key/value cache on the device: its layout, the
// ragged batch's bookkeeping with its checks, and the e4m3 / E8M0 conversions.
#pragma once

#include <cstdint>

#include "tl_ptx.cuh"

namespace tl {

struct KvCacheDev {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  int64_t page_stride, head_stride, token_stride;
  int32_t num_pages, ps, Hkv;
};

// The batch as the caller described it; every value read from it is checked before use.
struct KvBatch {
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  uint32_t* status;
  int32_t B, n_tokens, max_pages;
};

struct KvSeq {
  int32_t row0;  // its first new token's row
  int32_t q;     // new tokens
  int32_t len;   // length with them
};

constexpr uint32_t kKvInvalid = 1u;  // TL_ERR_INVALID

// Sequence s, made safe: rows inside [0, n_tokens), a length that the page table's
// row can hold.  Records TL_ERR_INVALID when something had to be changed.
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int ps, int s) {
  const int c0 = b.cu[s], c1 = b.cu[s + 1], len = b.lens[s];
  KvSeq r{c0, c1 - c0, len};
  const int64_t room = int64_t(b.max_pages) * ps;
  bool bad = false;
  if (c0 < 0 || c1 < c0 || c1 > b.n_tokens) {
    r.row0 = r.q = 0;
    bad = true;
  }
  if (len < 0 || int64_t(len) > room) {
    r.len = len < 0 ? 0 : int(room);
    bad = true;
  }
  if (r.len < r.q) bad = true;
  if (bad) record_error(b.status, kKvInvalid, uint32_t(s), uint32_t(len), uint32_t(c1));
  return r;
}

// Two e4m3 codes (low byte first) as two halves: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t two) {  // the upper 16 bits
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
// Two floats as e4m3 codes in the low 16 bits (lo in the low byte): nearest even,
// above 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, z;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tmov.b16 z, 0;\n\tmov.b32 %0, {a, z};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// 2^e for -127 <= e <= 127 (2^-127 is a subnormal); anything above is NaN (scale byte 255).
__device__ __forceinline__ float pow2f(int e) {
  if (e > 127) return __uint_as_float(0x7FFFFFFFu);
  return e <= -127 ? __uint_as_float(0x00400000u) : __uint_as_float(uint32_t(e + 127) << 23);
}

}  // namespace tl
