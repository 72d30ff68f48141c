// k_fp8.cu -- matrix products in e4m3 with one power-of-two scale per 128 columns (activations) or
// 128 x 128 block (weights): the plain layer and the gated layer.
//
// A plain tiled kernel: codes expanded to fp32 times their scale in shared memory, fp32 FMAs.
#include <algorithm>
#include <new>

#include "fp8_common.cuh"
#include "scion_internal.cuh"

struct scion_fp8 {
  scion_fp8_desc desc;
  int* err;  // device status word
  size_t device_bytes;
};

namespace scion {
namespace {

using namespace fp8;
typedef __nv_bfloat16 bf16;

__device__ __forceinline__ float value(uint8_t code) {
  __nv_fp8_e4m3 v;
  v.__x = code;
  return float(v);
}

struct Fp8Params {
  const uint8_t* x;
  const uint8_t* sx;
  const uint8_t* w[2];
  const uint8_t* sw[2];
  const float* base;
  void* out;  // plain: out of out_type; gated: bf16 h
  uint8_t* codes;
  uint8_t* scales;
  int T, N, K, KB, out_bf16;
};

constexpr int kTT = 32, kTK = 32;

template <int NW>
__global__ void __launch_bounds__(256) fp8_simple_kernel(const Fp8Params p) {
  __shared__ float xs[kTT][kTK + 1], ws[NW][128][kTK + 1];
  const int n0 = blockIdx.x * 128, t0 = blockIdx.y * kTT;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[NW][4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kTK) {
    const int kb = k0 / 128;
    for (int i = threadIdx.x; i < kTT * kTK; i += 256) {
      const int t = t0 + i / kTK, k = k0 + i % kTK;
      xs[i / kTK][i % kTK] =
          t < p.T && k < p.K ? value(p.x[int64_t(t) * p.K + k]) * scale_value(p.sx[int64_t(t) * p.KB + kb]) : 0.f;
    }
#pragma unroll
    for (int m = 0; m < NW; ++m)
      for (int i = threadIdx.x; i < 128 * kTK; i += 256) {
        const int n = n0 + i / kTK, k = k0 + i % kTK;
        ws[m][i / kTK][i % kTK] = n < p.N && k < p.K ? value(p.w[m][int64_t(n) * p.K + k]) *
                                                          scale_value(p.sw[m][int64_t(blockIdx.x) * p.KB + kb])
                                                     : 0.f;
      }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kTK; ++k)
#pragma unroll
      for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][i][j] = fmaf(xs[ty + 8 * i][k], ws[m][tx + 32 * j][k], acc[m][i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 8 * i;
    if (t >= p.T) break;  // (whole warps: a warp's tokens are its ty)
    float h[4];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = acc[0][i][j];
      h[j] = NW == 2 ? a / (1.f + __expf(-a)) * acc[NW - 1][i][j] : a;
      if (n0 + tx + 32 * j < p.N) m = max(m, mag(h[j]));
    }
    const uint32_t b = scale_byte(__reduce_max_sync(0xffffffffu, m));
    if (NW == 2 && p.codes && tx == 0) p.scales[int64_t(t) * ((p.N + 127) / 128) + blockIdx.x] = uint8_t(b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 32 * j;
      if (n >= p.N) continue;
      const int64_t at = int64_t(t) * p.N + n;
      if (NW == 2 && p.codes) {
        p.codes[at] = uint8_t(pack4(h[j] * scale_inverse(b), 0.f, 0.f, 0.f));
      } else {
        const float v = NW == 1 && p.base ? p.base[at] + h[j] : h[j];
        if (p.out_bf16) static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.out)[at] = v;
      }
    }
  }
}

cudaError_t launch_fp8(const Fp8Params& p, int gated, cudaStream_t s) {
  const dim3 grid((p.N + 127) / 128, (p.T + kTT - 1) / kTT);
  if (gated) fp8_simple_kernel<2><<<grid, 256, 0, s>>>(p);
  else fp8_simple_kernel<1><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

int status(cudaError_t e) {
  return e == cudaSuccess ? SCION_OK : e == cudaErrorMemoryAllocation ? SCION_ENOMEM : SCION_ECUDA;
}
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

Fp8Params params(const scion_fp8* L, const uint8_t* x, const uint8_t* sx, int T) {
  Fp8Params p{};
  p.x = x, p.sx = sx;
  p.w[0] = L->desc.w_codes, p.sw[0] = L->desc.w_scales;
  p.w[1] = L->desc.up_codes, p.sw[1] = L->desc.up_scales;
  p.T = T, p.N = L->desc.n, p.K = L->desc.k, p.KB = (p.K + 127) / 128;
  return p;
}

}  // namespace
}  // namespace scion

extern "C" int scion_fp8_create(const scion_fp8_desc* D, void* stream, scion_fp8** out) {
  if (!out) return SCION_EINVAL;
  *out = nullptr;
  if (!D || D->n < 1 || D->n > (1 << 20) || D->k < 16 || D->k % 16 || D->k > 65536) return SCION_EINVAL;
  if (!D->w_codes || !D->w_scales || scion::misaligned(D->w_codes, 16)) return SCION_EINVAL;
  if (!D->up_codes != !D->up_scales) return SCION_EINVAL;
  if (D->up_codes && (D->n % 16 || scion::misaligned(D->up_codes, 16))) return SCION_EINVAL;
  scion_fp8* L = new (std::nothrow) scion_fp8;
  if (!L) return SCION_ENOMEM;
  L->desc = *D;
  L->err = nullptr;
  L->device_bytes = sizeof(int);
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&L->err), sizeof(int));
  if (e == cudaSuccess) e = cudaMemsetAsync(L->err, 0, sizeof(int), static_cast<cudaStream_t>(stream));
  // (the word is cleared before a forward on another stream can run)
  if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    scion_fp8_destroy(L);
    return scion::status(e);
  }
  *out = L;
  return SCION_OK;
}

extern "C" void scion_fp8_destroy(scion_fp8* L) {
  if (!L) return;
  if (L->err) cudaFree(L->err);  // waits for the device
  delete L;
}

extern "C" size_t scion_fp8_device_bytes(const scion_fp8* L) { return L ? L->device_bytes : 0; }

extern "C" int scion_fp8_forward(const uint8_t* x_codes, const uint8_t* x_scales, int T, const scion_fp8* L,
                                 const float* base, void* out, int out_type, void* stream) {
  if (!L || L->desc.up_codes || T < 0 || (out_type != SCION_F32 && out_type != SCION_BF16)) return SCION_EINVAL;
  if (T == 0) return SCION_OK;
  if (!x_codes || !x_scales || !out || scion::misaligned(x_codes, 16)) return SCION_EINVAL;
  if (scion::misaligned(base, 4) || scion::misaligned(out, out_type == SCION_F32 ? 4 : 2)) return SCION_EINVAL;
  if (out_type == SCION_BF16 && static_cast<const void*>(base) == out && base) return SCION_EINVAL;
  scion::Fp8Params p = scion::params(L, x_codes, x_scales, T);
  p.base = base, p.out = out, p.out_bf16 = out_type == SCION_BF16;
  return scion::status(scion::launch_fp8(p, 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int scion_fp8_gated_forward(const uint8_t* x_codes, const uint8_t* x_scales, int T, const scion_fp8* L,
                                       void* h_bf16, uint8_t* h_codes, uint8_t* h_scales, void* stream) {
  if (!L || !L->desc.up_codes || T < 0) return SCION_EINVAL;
  if (!h_codes != !h_scales || !h_codes == !h_bf16) return SCION_EINVAL;
  if (T == 0) return SCION_OK;
  if (!x_codes || !x_scales || scion::misaligned(x_codes, 16) || scion::misaligned(h_bf16, 16) ||
      scion::misaligned(h_codes, 16))
    return SCION_EINVAL;
  scion::Fp8Params p = scion::params(L, x_codes, x_scales, T);
  p.out = h_bf16, p.out_bf16 = 1, p.codes = h_codes, p.scales = h_scales;
  return scion::status(scion::launch_fp8(p, 1, static_cast<cudaStream_t>(stream)));
}

extern "C" int scion_fp8_check(const scion_fp8* L, void* stream) {
  if (!L) return SCION_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int err = 0;
  cudaError_t e = cudaMemcpyAsync(&err, L->err, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return SCION_ECUDA;
  if (err != 0) {
    e = cudaMemsetAsync(L->err, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? err : SCION_ECUDA;
  }
  return SCION_OK;
}
