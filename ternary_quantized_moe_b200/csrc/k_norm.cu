// k_norm.cu -- the residual add with its root-mean-square norm, and the float -> e4m3 quantizers
// (rows x 128 for activations, 128 x 128 for weights).  Entry points at the end of the file.
//
// All three are bound by HBM: one read of every input, one write of every output, nothing kept in
// memory in between.  A thread holds 8 consecutive columns (16 bytes of bf16, 32 of fp32 per load
// and lane), so a group of 128 columns is half a warp and its largest magnitude one redux over 16
// lanes; the loads of a warp cover whole 32-byte sectors.  Programmatic dependent launch lets a call's
// blocks start as its predecessor's drain.  Replayed from a graph: the norm of 16384 x 4096 (bf16 + fp32
// in, fp32 + 8 bits out, 738 MB) 106.7 us, 6.9 TB/s, and of one row of 2048 1.8 us; 8192 x 8192 fp32 in
// 128 x 128 blocks 49.4 us, 6.8 TB/s, bf16 33.8 us, 6.0; 16384 x 4096 bf16 by rows 37.3 us, 5.4 TB/s (issue
// slots 84% busy: the conversions of two bytes of source to one).
#include <math.h>

#include <algorithm>
#include <atomic>

#include "fp8_common.cuh"
#include "scion_internal.cuh"

namespace scion {
namespace {

using namespace fp8;
typedef __nv_bfloat16 bf16;

// Largest magnitude of the half warp the lane is in (all 32 lanes take part).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m) {
  const uint32_t mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  return __reduce_max_sync(mask, m);
}
__device__ __forceinline__ uint32_t mag8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag(v[i]));
  return m;
}
__device__ __forceinline__ uint2 code8(const float (&v)[8], float inv) {
  return make_uint2(pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// ------------------------------------------------------------------ norm
struct NormParams {
  const void* x;
  const void* resid;
  const bf16* w;
  void* resid_out;
  bf16* y;
  uint8_t* codes;
  uint8_t* scales;
  float eps;
  int d, groups;
};

// The row of `lanes` threads (a warp, or the whole CTA with kBlock): thread t of them holds the 8-column
// chunks t, t + lanes, ..., so that the row stays in registers between the statistic and the output.
// y = (r w) rms: the products r w and their largest magnitude per group do not wait for the statistic,
// and (rounding is monotonic) max |y| = max |r w| rms to the last bit.
// Squares below 2^-126 lose bits, which matters only where neither eps nor the rest of the sum is far
// above them: with eps < kTiny (kSmallEps) the squares of r kLift are summed beside, and a row whose sum
// is below kTiny (|r| < 2^-30, so that (r kLift)^2 sums to less than 2^120; the least fp32 gives 2^-118)
// takes its statistic from those.  (A variant of its own: as a branch on eps it kept loads apart, 16384 x
// 4096 bf16 without a residual in 55 us, 48 without it.)
constexpr float kTiny = 0x1p-60f, kLift = 0x1p90f;

// Sum over the row's threads, the same in all of them; `part`: 32 floats of shared memory per sum.
template <bool kBlock>
__device__ __forceinline__ float row_sum(float v, int t, int lanes, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (kBlock) {
    const int lane = t & 31;
    if (lane == 0) part[t >> 5] = v;
    __syncthreads();
    v = lane < (lanes >> 5) ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

template <typename X, typename R, int CPT, bool kBlock, bool kSmallEps>
__device__ __forceinline__ void norm_row(const NormParams& p, int64_t r, int t, int lanes, float* part) {
  const int64_t row = r * p.d;
  const int chunks = p.d >> 3;
  float v[CPT][8];
  uint32_t m[CPT];
  float ss = 0.f, lifted = 0.f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * lanes;
    const bool in = c < chunks;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (in) {
      w = __ldg(reinterpret_cast<const uint4*>(p.w + 8 * c));
      load8(static_cast<const X*>(p.x) + row + 8 * c, v[i]);
      if (p.resid) {
        float o[8];
        load8(static_cast<const R*>(p.resid) + row + 8 * c, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += o[j];
      }
      if (p.resid_out) store8(static_cast<R*>(p.resid_out) + row + 8 * c, v[i]);
    }
    float wf[8];
    unpack_bf16x8(w, wf);
    if (kSmallEps) {
#pragma unroll
      for (int j = 0; j < 8; ++j) lifted = fmaf(v[i][j] * kLift, v[i][j] * kLift, lifted);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss), v[i][j] *= wf[j];
    if (p.codes) m[i] = half_warp_max(mag8(v[i]));
  }
  if (!p.y && !p.codes) return;
  ss = row_sum<kBlock>(ss, t, lanes, part);
  // an infinite sum would turn the row's finite elements into zeros: the whole row is NaN instead
  float rms = ss < INFINITY ? rsqrtf(ss / float(p.d) + p.eps) : NAN;
  if (kSmallEps) {
    lifted = row_sum<kBlock>(lifted, t, lanes, part + 32);
    if (ss < kTiny) {  // (a row of zeros without eps: 0 / 0 in every element)
      rms = rsqrtf(lifted / float(p.d) + p.eps * kLift * kLift);
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= kLift;
        if (p.codes) m[i] = mag(__uint_as_float(m[i]) * kLift);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * lanes;
    if (c >= chunks) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rms;
    if (p.codes) {
      // (in two steps: near the smallest numbers rms / s leaves the fp32 range where y / s does not)
      const uint32_t b = scale_byte(mag(__uint_as_float(m[i]) * rms));
      *reinterpret_cast<uint2*>(p.codes + row + 8 * c) = code8(v[i], scale_inverse(b));
      if ((t & 15) == 0) p.scales[r * p.groups + (c >> 4)] = uint8_t(b);
    }
    if (p.y) store8(p.y + row + 8 * c, v[i]);
  }
}

// A CTA per row.
template <typename X, typename R, int CPT, bool kSmallEps>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormParams p) {
  __shared__ float part[64];
  pdl_trigger();
  pdl_wait();
  norm_row<X, R, CPT, true, kSmallEps>(p, blockIdx.x, threadIdx.x, blockDim.x, part);
}

// A warp per row, eight rows per CTA: no barrier.
template <typename X, typename R, int CPT, bool kSmallEps>
__global__ void __launch_bounds__(256) rmsnorm_warp_kernel(const NormParams p, int T) {
  pdl_trigger();
  pdl_wait();
  const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (r < T) norm_row<X, R, CPT, false, kSmallEps>(p, r, threadIdx.x & 31, 32, nullptr);
}

template <typename X, typename R, bool kSmallEps>
cudaError_t launch_norm(const NormParams& p, int T, cudaStream_t s) {
  const int chunks = p.d >> 3;
  // 16384 rows of 128 fp32: 7 us with a warp per row, 17 with a CTA
  if (chunks <= 64) return launch_pdl(rmsnorm_warp_kernel<X, R, 2, kSmallEps>, dim3(unsigned((int64_t(T) + 7) / 8)), dim3(256), 0, s, p, T);
  // One chunk per thread is the quickest for few rows (1 x 4096 fp32: 2.2 us, 2.6 with two) and as good
  // for many, except where a thread would read 16 bytes in all (16384 x 4096 bf16 without a residual: 60
  // us, 48 with two) or the CTA have 1024 threads (8192 x 8192 bf16 with a residual: 84 us, 83).
  const int cpt = chunks > 2048 ? 4 : chunks > 512 || (chunks > 256 && sizeof(X) == 2 && !p.resid) ? 2 : 1;
  const int nt = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
  if (cpt == 1) return launch_pdl(rmsnorm_kernel<X, R, 1, kSmallEps>, dim3(T), dim3(nt), 0, s, p);
  if (cpt == 2) return launch_pdl(rmsnorm_kernel<X, R, 2, kSmallEps>, dim3(T), dim3(nt), 0, s, p);
  return launch_pdl(rmsnorm_kernel<X, R, 4, kSmallEps>, dim3(T), dim3(nt), 0, s, p);
}
template <typename X, typename R>
cudaError_t launch_norm(const NormParams& p, int T, cudaStream_t s) {
  return p.eps < kTiny ? launch_norm<X, R, true>(p, T, s) : launch_norm<X, R, false>(p, T, s);
}

// ------------------------------------------------------------------ quantizers
// Eight source elements as loaded, their largest magnitude (bits of mag()) and their values.
template <typename S>
struct Chunk;
template <>
struct Chunk<float> {
  struct Raw {
    float4 a, b;
  };
  static __device__ __forceinline__ Raw zero() { return {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}; }
  static __device__ __forceinline__ Raw load(const float* p) {
    return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
  }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w, v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
  }
  static __device__ __forceinline__ uint32_t largest(const Raw& r) {
    float v[8];
    values(r, v);
    return mag8(v);
  }
};
template <>
struct Chunk<bf16> {
  typedef uint4 Raw;
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ Raw load(const bf16* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) { unpack_bf16x8(r, v); }
  // two at a time; magnitudes order like their bits, and the maximum that keeps NaN has the largest
  static __device__ __forceinline__ uint32_t largest(const Raw& r) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    return max(w & 0xffff0000u, w << 16);
  }
};

// Activations: a half warp per group of 128 columns of a row, `per` rows per CTA, four groups' loads
// in flight.  (With a division per group to find its row the kernel was bound by its instructions:
// 16384 x 4096 bf16 in 52 us with a 64-bit one, 42 us with a 32-bit one, 37 us without.)
template <typename S>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const S* __restrict__ src, int64_t rows, int cols, int groups,
                                                            int per, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  constexpr int U = 4;
  pdl_trigger();
  pdl_wait();
  const int64_t row0 = int64_t(blockIdx.x) * per;
  const uint32_t n = uint32_t(min(int64_t(per), rows - row0)) * groups;
  src += row0 * cols, codes += row0 * cols, scales += row0 * groups;
  const int lane = threadIdx.x & 15;
  // group i of the CTA's rows, its row and its place there, stepping by 16 groups without a division
  uint32_t i = threadIdx.x >> 4, row = i / uint32_t(groups), g = i - row * groups;
  const uint32_t step_row = 16u / uint32_t(groups), step_g = 16u - step_row * groups;
  const uint32_t end = (n + 1) / 2 * 2;  // whole warps: a warp's two half warps walk neighbouring groups
  while (i < end) {
    typename Chunk<S>::Raw raw[U];
    int64_t at[U];
    uint32_t first = i;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = int(g) * 128 + 8 * lane;
      at[u] = i < n && c < cols ? int64_t(row) * cols + c : -1;
      raw[u] = Chunk<S>::zero();
      if (at[u] >= 0) raw[u] = Chunk<S>::load(src + at[u]);
      i += 16, row += step_row, g += step_g;
      if (g >= uint32_t(groups)) g -= groups, ++row;
    }
#pragma unroll
    for (int u = 0; u < U; ++u, first += 16) {
      if (first >= end) break;
      const uint32_t b = scale_byte(half_warp_max(Chunk<S>::largest(raw[u])));
      float v[8];
      Chunk<S>::values(raw[u], v);
      if (at[u] >= 0) *reinterpret_cast<uint2*>(codes + at[u]) = code8(v, scale_inverse(b));
      if (first < n && lane == 0) scales[first] = uint8_t(b);
    }
  }
}

// Weights: a CTA per 128 x 128 block, 8 x 8 values per thread in registers.
template <typename S>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const S* __restrict__ src, int64_t rows, int cols,
                                                              int groups, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  __shared__ uint32_t part[8];
  pdl_trigger();
  pdl_wait();
  const int64_t rb = blockIdx.x / groups;
  const int g = int(blockIdx.x - rb * groups);
  const int c = g * 128 + 8 * (threadIdx.x & 15);
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && c < cols) {
      load8(src + r * cols + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag8(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  const uint32_t b = scale_byte(m);
  const float inv = scale_inverse(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = code8(v[i], inv);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = uint8_t(b);
}

// SMs of the current device.
int sm_count() {
  static std::atomic<int> known[16];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 16 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
  if (dev < 16) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <typename S>
cudaError_t launch_quantize(const S* src, int64_t rows, int cols, int block_rows, uint8_t* codes, uint8_t* scales,
                            cudaStream_t s) {
  const int groups = (cols + 127) / 128;
  if (block_rows == 1) {
    // 64 groups per CTA where that leaves two CTAs for every SM; the grid stays within 2^31 - 1
    int64_t per = std::max<int64_t>(1, std::min<int64_t>(64 / groups, rows / (2 * sm_count())));
    per = std::max(per, rows >> 30);
    return launch_pdl(quantize_rows_kernel<S>, dim3(unsigned((rows + per - 1) / per)), dim3(256), 0, s, src, rows, cols,
                      groups, int(per), codes, scales);
  }
  return launch_pdl(quantize_blocks_kernel<S>, dim3(unsigned((rows + 127) / 128 * groups)), dim3(256), 0, s, src, rows, cols,
                    groups, codes, scales);
}

}  // namespace
}  // namespace scion

extern "C" int scion_fp8_quantize_device(int src_type, const void* src, int64_t rows, int cols, int block_rows,
                                         uint8_t* codes, uint8_t* scales, void* stream) {
  if ((src_type != SCION_F32 && src_type != SCION_BF16) || (block_rows != 1 && block_rows != 128)) return SCION_EINVAL;
  if (rows < 0 || cols < 16 || cols % 16 || cols > (1 << 20)) return SCION_EINVAL;
  // one CTA per 128 x 128 block: the grid stays within 2^31 - 1
  if (rows > (int64_t(1) << 40) || (block_rows == 128 && (rows + 127) / 128 * ((cols + 127) / 128) > 0x7fffffff))
    return SCION_EINVAL;
  if (rows == 0) return SCION_OK;
  if (!src || !codes || !scales || scion::fp8::misaligned(src, 16) || scion::fp8::misaligned(codes, 16)) return SCION_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      src_type == SCION_F32
          ? scion::launch_quantize(static_cast<const float*>(src), rows, cols, block_rows, codes, scales, s)
          : scion::launch_quantize(static_cast<const __nv_bfloat16*>(src), rows, cols, block_rows, codes, scales, s);
  return e == cudaSuccess ? SCION_OK : SCION_ECUDA;
}

extern "C" int scion_rmsnorm_forward(const void* x, int x_type, const void* resid, int resid_type, const void* weight,
                                     float eps, int T, int d, void* resid_out, void* y_bf16, uint8_t* y_codes,
                                     uint8_t* y_scales, void* stream) {
  if ((x_type != SCION_F32 && x_type != SCION_BF16) || (resid_type != SCION_F32 && resid_type != SCION_BF16))
    return SCION_EINVAL;
  if (T < 0 || d < 16 || d % 16 || d > 32768 || !(eps >= 0.f) || !isfinite(eps)) return SCION_EINVAL;
  if (T == 0) return SCION_OK;  // (empty tensors have null addresses)
  if (!y_codes != !y_scales || (!resid_out && !y_bf16 && !y_codes)) return SCION_EINVAL;
  if (!x || !weight) return SCION_EINVAL;
  for (const void* p : {x, resid, weight, static_cast<const void*>(resid_out), static_cast<const void*>(y_bf16),
                        static_cast<const void*>(y_codes)})
    if (scion::fp8::misaligned(p, 16)) return SCION_EINVAL;
  // in place on x only where an element is as wide (a thread then overwrites what it alone has read)
  if (resid_out == x && resid_type != x_type) return SCION_EINVAL;
  scion::NormParams p{x,       resid,    static_cast<const __nv_bfloat16*>(weight), resid_out, static_cast<__nv_bfloat16*>(y_bf16),
                      y_codes, y_scales, eps, d, (d + 127) / 128};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  scion::count_launch();
  using scion::launch_norm;
  const cudaError_t e = x_type == SCION_F32
                            ? (resid_type == SCION_F32 ? launch_norm<float, float>(p, T, s)
                                                       : launch_norm<float, __nv_bfloat16>(p, T, s))
                            : (resid_type == SCION_F32 ? launch_norm<__nv_bfloat16, float>(p, T, s)
                                                       : launch_norm<__nv_bfloat16, __nv_bfloat16>(p, T, s));
  return e == cudaSuccess ? SCION_OK : SCION_ECUDA;
}
