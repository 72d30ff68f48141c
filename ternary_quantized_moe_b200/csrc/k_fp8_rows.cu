// k_fp8_rows.cu -- products in e4m3 with power-of-two block scales for single tokens and small decode
// batches (up to 32 tokens).
//
// Bound by latency and by reading the weights once, so the path from the first load to the result is
// kept short: no ring, no tensor memory, no cluster for a plain layer.  A CTA holds 16 weight rows (of
// each matrix) and its eight warps split K by blocks of 128; a lane loads its share of a block straight
// into mma.sync fragments.  The order of k inside a block is free as long as both operands agree, so a
// lane takes 32 consecutive bytes of its row -- four lanes cover the row's 128 bytes -- and step s of
// the four uses bytes 8 s .. 8 s + 7 of them.  A block's sum is scaled once (both scales are powers of
// two) and added in fp32; the warps' sums meet in shared memory and are added in warp order.
// A gated layer that writes 8 bits needs the largest |h| of 128 features: the eight CTAs of a cluster
// hold them and exchange one magnitude per token.
// Measured (replayed from a graph, one token): 4096 x 2048 2.5 us, 16384 x 8192 25.5 us (5.3 TB/s), gated
// 2 x 512 x 2048 3.1 us; 8 tokens, gated 2 x 2048 x 4096 5.8 us.
#include "fp8_common.cuh"
#include "scion_internal.cuh"

namespace scion {
namespace {

using namespace fp8;
typedef __nv_bfloat16 bf16;

constexpr int kRowsWarps = 8;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Bytes32 {
  uint4 v[2];
};
// 32 bytes at p (16-byte aligned); `n` of them exist (a multiple of 16, or less than 1), the rest are 0.
__device__ __forceinline__ Bytes32 load32(const uint8_t* p, int n) {
  Bytes32 b;
  b.v[0] = b.v[1] = make_uint4(0u, 0u, 0u, 0u);
  if (n > 0) b.v[0] = *reinterpret_cast<const uint4*>(p);
  if (n > 16) b.v[1] = *reinterpret_cast<const uint4*>(p + 16);
  return b;
}
__device__ __forceinline__ uint32_t word(const Bytes32& b, int i) {
  const uint4& v = b.v[i >> 2];
  return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
}

// 2^(a - 127) 2^(b - 127) for scale bytes a and b, as two factors of the same sign of exponent, so that
// nothing between overflows or underflows where the product with a value does not.  Nearly always one
// factor does and the other is 1.
__device__ __forceinline__ float2 scale_factors(uint32_t a, uint32_t b) {
  const int e = int(a + b) - 254;
  if (a != 255u && b != 255u && unsigned(e + 126) <= 253u) return make_float2(__uint_as_float(uint32_t(e + 127) << 23), 1.f);
  if (a == 255u || b == 255u) return make_float2(NAN, 1.f);
  const int e1 = e >> 1, e2 = e - e1;
  return make_float2(__uint_as_float(uint32_t(e1 + 127) << 23), __uint_as_float(uint32_t(e2 + 127) << 23));
}

// Row pointers of a lane: its two weight rows, its token rows (operand rows and the columns of its
// sums), clamped to what exists (a row past the end repeats the last one; its sums are not used).
template <int NW, int NT>
struct Lane {
  const uint8_t* w[NW][2];
  const uint8_t* x[NT];
  const uint8_t* sw[NW];
  const uint8_t* sx[NT][2];
};

// U blocks of K, kRowsWarps apart, from block kb on: loads first, then the products.  kTail: the last
// of a row, where blocks and parts of blocks may be missing.
template <int NW, int NT, int U, bool kTail>
__device__ __forceinline__ void blocks(const Call& p, const Lane<NW, NT>& l, int kb, int c, float (&acc)[NW][NT][4]) {
  Bytes32 w[U][NW][2], x[U][NT];
  uint32_t sw[U][NW], sx[U][NT][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (kb + u * kRowsWarps) * 128 + 32 * c, left = kTail ? p.K - k : 128;
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[u][m][h] = load32(l.w[m][h] + k, left);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int b = kb + u * kRowsWarps, k = b * 128 + 32 * c, left = kTail ? p.K - k : 128;
    const bool in = !kTail || b < p.KB;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      x[u][t] = load32(l.x[t] + k, left);
#pragma unroll
      for (int j = 0; j < 2; ++j) sx[u][t][j] = in ? l.sx[t][j][b] : 127u;
    }
#pragma unroll
    for (int m = 0; m < NW; ++m) sw[u][m] = in ? l.sw[m][b] : 127u;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int m = 0; m < NW; ++m) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_e4m3(d, word(w[u][m][0], 2 * s), word(w[u][m][1], 2 * s), word(w[u][m][0], 2 * s + 1),
                   word(w[u][m][1], 2 * s + 1), word(x[u][t], 2 * s), word(x[u][t], 2 * s + 1));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = scale_factors(sx[u][t][j], sw[u][m]);
          acc[m][t][j] = fmaf(d[j] * f.y, f.x, acc[m][t][j]);
          acc[m][t][j + 2] = fmaf(d[j + 2] * f.y, f.x, acc[m][t][j + 2]);
        }
      }
    }
  }
}

// NW matrices, NT tiles of 8 tokens, U blocks of K per warp with their loads in flight together, G:
// results to 8 bits (gated, clusters of 8 CTAs); PerSm: CTAs whose registers fit an SM.
template <int NW, int NT, int U, bool G, int PerSm>
__global__ void __launch_bounds__(kRowsWarps * 32, PerSm) fp8_rows_kernel(const Call p) {
  __shared__ float part[kRowsWarps][NW][8 * NT][17];  // [warp][matrix][token][row], padded
  __shared__ uint32_t amax[8][8 * NT];                // [CTA of the cluster][token]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * 16;
  // (shared memory of another CTA may be used once all of the cluster run: awaited before the first store)
  if (G) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  Lane<NW, NT> l;
#pragma unroll
  for (int m = 0; m < NW; ++m) {
#pragma unroll
    for (int h = 0; h < 2; ++h) l.w[m][h] = p.w[m] + int64_t(min(row0 + g + 8 * h, p.N - 1)) * p.K;
    l.sw[m] = p.sw[m] + int64_t(min(row0, p.N - 1) / 128) * p.KB;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l.x[t] = p.x + int64_t(min(8 * t + g, p.T - 1)) * p.K;
#pragma unroll
    for (int j = 0; j < 2; ++j) l.sx[t][j] = p.sx + int64_t(min(8 * t + 2 * c + j, p.T - 1)) * p.KB;
  }
  pdl_trigger();
  pdl_wait();
  float acc[NW][NT][4] = {};
  if (row0 < p.N) {  // (a cluster's last CTAs may have no rows)
    int kb = warp;
    for (; (kb + (U - 1) * kRowsWarps + 1) * 128 <= p.K; kb += kRowsWarps * U) blocks<NW, NT, U, false>(p, l, kb, c, acc);
    for (; kb < p.KB; kb += kRowsWarps) blocks<NW, NT, 1, true>(p, l, kb, c, acc);
  }
#pragma unroll
  for (int m = 0; m < NW; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][m][8 * t + 2 * c + (i & 1)][g + 8 * (i >> 1)] = acc[m][t][i];
  __syncthreads();
  if (G) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // thread: row threadIdx % 16 of tokens threadIdx / 16, 16 further, ... (a half warp per token)
  constexpr int kPasses = (NT + 1) / 2;
  const int r = threadIdx.x & 15, tok0 = threadIdx.x >> 4, n = row0 + r;
  const uint32_t half = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  const int rank = blockIdx.x & 7;
  float h[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int tok = tok0 + 16 * i;
    const bool mine = tok < p.T && n < p.N;
    float v[NW];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      v[m] = 0.f;
      if (tok < 8 * NT)
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) v[m] += part[w][m][tok][r];
    }
    const int64_t at = int64_t(tok) * p.N + n;
    if (NW == 1) {
      if (!mine) continue;
      if (p.base) v[0] += p.base[at];
      if (p.out_bf16) static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(v[0]);
      else static_cast<float*>(p.out)[at] = v[0];
      continue;
    }
    h[i] = silu_mul(v[0], v[NW - 1]);
    if (!G) {
      if (mine) static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(h[i]);
      continue;
    }
    const uint32_t m = __reduce_max_sync(half, mine ? mag(h[i]) : 0u);
    if (tok < 8 * NT && r < 8) {  // one magnitude per token to each CTA of the cluster
      const uint32_t dst = map_cluster_rank(smem_addr(&amax[rank][tok]), r);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst), "r"(m) : "memory");
    }
  }
  if (!G) return;
  cluster_sync();
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int tok = tok0 + 16 * i;
    if (tok >= p.T || n >= p.N) return;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, amax[j][tok]);
    const uint32_t b = scale_byte(top);
    p.codes[int64_t(tok) * p.N + n] = uint8_t(pack4(h[i] * scale_inverse(b), 0.f, 0.f, 0.f));
    if (rank == 0 && r == 0) p.scales[int64_t(tok) * ((p.N + 127) / 128) + (blockIdx.x >> 3)] = uint8_t(b);
  }
}

template <int NW, int NT, int U, bool G, int PerSm>
cudaError_t launch(const Call& c, cudaStream_t s) {
  const unsigned ctas = unsigned((c.N + 15) / 16);
  const dim3 block(kRowsWarps * 32);
  if (G) return launch_pdl_cluster(fp8_rows_kernel<NW, NT, U, G, PerSm>, dim3((ctas + 7) / 8 * 8), block, dim3(8), 0, s, c);
  return launch_pdl(fp8_rows_kernel<NW, NT, U, G, PerSm>, dim3(ctas), block, 0, s, c);
}

// Registers against CTAs.  Where every SM has one CTA at most, its warps take the registers to keep a whole
// row's blocks in flight; where there are many, more CTAs per SM keep more loads in flight than deeper ones.
// One token, n x k (us): 2048 x 4096 (128 CTAs) U = 4 with registers for one CTA per SM 2.9, for two 3.9; 4096
// x 4096 (256) 4.8, 4.0, U = 2 3.7; 8192 x 8192 (512) U = 4 for two 15.9, U = 2 for four 13.9.  16 tokens: 2048
// x 4096 U = 2 for one 3.7, for two 4.6; 4096 x 4096 6.6, U = 1 5.4.  32 tokens (U = 1): 2048 x 2048 for one
// 3.7, for two 5.1; 2400 x 1024 4.1, 3.6; 4096 x 512 3.8, 3.0 (24 tokens).  Gated, 16 tokens: registers for two
// CTAs per SM spill (136 bytes), so that even two rounds of one are quicker, 2 x 2048 x 1024 to bf16 2.6
// against 4.1; to 8 bits 2 x 1792 x 1024 3.4, 4.8, but 2 x 2048 x 512, 16 clusters of which 15 run at once with
// one CTA per SM, 5.0, 3.9.
template <int NW, bool G>
cudaError_t launch_tokens(const Call& c, cudaStream_t s) {
  const int ctas = (c.N + 15) / 16;
  if constexpr (NW == 1) {
    const bool few = ctas <= c.sms, longer = c.KB > 2 * kRowsWarps;
    if (c.T > 16) return few ? launch<1, 4, 1, G, 1>(c, s) : launch<1, 4, 1, G, 2>(c, s);
    if (c.T > 8) return few ? launch<1, 2, 2, G, 1>(c, s) : launch<1, 2, 1, G, 2>(c, s);
    if (few && longer) return launch<1, 1, 4, G, 1>(c, s);
    return ctas <= 2 * c.sms ? launch<1, 1, 2, G, 2>(c, s) : launch<1, 1, 2, G, 4>(c, s);
  } else {
    if (c.T > 8) {
      if constexpr (G)
        if ((ctas + 7) / 8 > c.clusters8) return launch<2, 2, 1, G, 2>(c, s);
      return launch<2, 2, 1, G, 1>(c, s);
    }
    return launch<2, 1, 1, G, 2>(c, s);
  }
}

}  // namespace

namespace fp8 {
cudaError_t launch_rows(const Call& c, cudaStream_t s) {
  if (!c.w[1]) return launch_tokens<1, false>(c, s);
  return c.codes ? launch_tokens<2, true>(c, s) : launch_tokens<2, false>(c, s);
}
}  // namespace fp8
}  // namespace scion
