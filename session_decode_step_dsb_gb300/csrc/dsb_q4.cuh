// The 4-bit KV row and the page block it lives in, shared by the kernels that
// write and read it.
//
// A head vector x of D values is stored as D codes in 0..15 and two fp16
// numbers, one pair per key and head: d = fp16((max - min) * fl(1/15)),
// z = fp16(min + 8 d), code = clamp(round-half-even((x - z) / d) + 8, 0, 15)
// (8 where d is 0), and stands for z + d (code - 8).  Centring the codes on 8
// lets a matrix product run on small signed integers (exact in fp16) with the
// scale and the offset applied once per key.
//
// A page holds 128 keys.  Per page and kv head one block of 128 (D + 8) bytes:
//   K codes  [128 keys][D/2]: dimension 2i in the low half of byte i
//   K (d, z) [128 keys] half2
//   V codes  [64 key pairs][D/4 words][2 keys] u16: word i of a key holds
//            dimensions 4i .. 4i+3, lowest four bits first.  A 32-bit load
//            gives four dimensions of two neighbouring keys, whose codes sit
//            16 bits apart: the pairs along the keys that the product P V
//            wants as half2, with no shuffling; and a key's own bytes are whole,
//            so that one key can be written without touching its neighbour
//   V (d, z) [128 keys] half2
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace dsbk {

constexpr int kQ4Page = 128;
template <int D>
struct Q4Block {
  static constexpr int kz = kQ4Page * D / 2;          // K (d, z)
  static constexpr int v = kz + kQ4Page * 4;          // V codes
  static constexpr int vz = v + kQ4Page * D / 2;      // V (d, z)
  static constexpr int bytes = vz + kQ4Page * 4;      // 128 (D + 8)
};

// Eight codes of a 32-bit word, less 8, as four half2: h[n] holds nibble n (low
// half) and nibble n + 4 (high half).  A nibble at bits 0..3 of an fp16 with
// exponent bits 0x6400 is 1024 + q; at bits 4..7 it is 1024 + 16 q.  Both steps
// are exact.
// (w & mask) | 0x64006400 in one instruction.
__device__ __forceinline__ uint32_t q4_biased(uint32_t w, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
  return r;
}
__device__ __forceinline__ void q4_unpack(uint32_t w, __half2 (&h)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t a = q4_biased(w, 0x000F000Fu), b = q4_biased(w, 0x00F000F0u);
  const uint32_t c = q4_biased(w8, 0x000F000Fu), d = q4_biased(w8, 0x00F000F0u);
  const __half2 bias = __float2half2_rn(1032.0f), s = __float2half2_rn(0.0625f), o = __float2half2_rn(-72.0f);
  h[0] = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  h[1] = __hfma2(*reinterpret_cast<const __half2*>(&b), s, o);
  h[2] = __hsub2(*reinterpret_cast<const __half2*>(&c), bias);
  h[3] = __hfma2(*reinterpret_cast<const __half2*>(&d), s, o);
}

}  // namespace dsbk
