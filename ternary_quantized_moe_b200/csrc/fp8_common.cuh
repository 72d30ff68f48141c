// fp8_common.cuh -- the 8-bit container of the dense operators: e4m3 codes with one power-of-two
// scale byte per block (include/scion.h, "8-bit dense operators").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace scion {
namespace fp8 {

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// One product call: out = base + W x (w[1] null), or h = silu(W0 x) (W1 x) to bf16 or codes and scales.
struct Call {
  const uint8_t* x;
  const uint8_t* sx;
  const uint8_t* w[2];
  const uint8_t* sw[2];
  const float* base;
  void* out;  // plain: out; gated: bf16 h or null
  uint8_t* codes;
  uint8_t* scales;
  int T, N, K, KB;  // KB = ceil(K / 128)
  int out_bf16, sms;
  int clusters8;  // clusters of 8 CTAs that run at once with one CTA per SM
};

// k_fp8_rows.cu: up to 32 tokens
cudaError_t launch_rows(const Call& c, cudaStream_t s);

// |v| as an unsigned integer: ordered like the magnitudes, infinities and NaN above every number
// (a maximum over these keeps a NaN, which fmaxf would drop).
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale byte of a block whose largest magnitude is `m` (bits of mag()): 2^(b - 127) is the smallest
// power of two s with m / s <= 448 = 1.75 * 2^8.  A mantissa up to 1.75 takes the exponent less 8,
// a larger one the next: adding 0x1fffff carries into the exponent exactly above 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 255u;
  if (m == 0u) return 127u;
  const int b = int((m + 0x1fffffu) >> 23) - 8;
  return b > 0 ? uint32_t(b) : 0u;
}

// 2^(127 - b), the factor onto the codes' range (NaN for b = 255); exact, and so is the product
// with it for every value that does not round to zero.
__device__ __forceinline__ float scale_inverse(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fffffffu : (254u - b) << 23);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

// Four values (already times scale_inverse) to four e4m3 bytes, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Eight consecutive elements (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void unpack_bf16x8(uint4 a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

}  // namespace fp8
}  // namespace scion
