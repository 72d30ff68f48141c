// k_fp8.cu -- matrix products in e4m3 with one power-of-two scale per 128 columns (activations) or
// 128 x 128 block (weights): the plain layer and the gated layer.
//
// Both run on tcgen05.mma kind::mxf8f6f4: the tensor cores multiply e4m3 operands and apply the
// E8M0 scales themselves (a scale byte per row and 32 columns; the four steps of a 128-column block
// use the same byte), so nothing is expanded or promoted outside them.
#include <stddef.h>

#include <algorithm>
#include <new>

#include "fp8_common.cuh"
#include "scion_internal.cuh"
#include "tc_common.cuh"

struct scion_fp8 {
  scion_fp8_desc desc;
  CUtensorMap w[2];
  int sms;
  int clusters[9];  // clusters of 1 .. 8 CTAs that run at once with one CTA per SM
  int* err;         // device status word
  size_t device_bytes;
};

namespace scion {
namespace {

using namespace fp8;
using namespace tc;
typedef __nv_bfloat16 bf16;

// ------------------------------------------------------------------ streaming kernel
// Few tokens: bound by reading the weights once.  The weights are the M side (128 rows per tile),
// the tokens the N side (bn of them, a multiple of 16), and the CTAs of a cluster split K, so that a
// matrix of few tiles still spreads over the SMs.  Partial sums: the tokens of a tile are dealt to
// the CTAs of the cluster; every CTA stores its sums of a token straight into the shared memory of
// the token's owner (counted by a barrier there), and the owner adds them in rank order.  One barrier
// of the cluster, at the start, and none on the way out: an owner leaves when everything sent to it
// has arrived.
// Roles: warp 0 TMA loads through a ring of stages, warp 1 the MMAs, warps 2..9 the epilogue (two per
// lane quarter, alternate 16-token chunks), warps 2..5 also the scale words.  The sums pass through
// shared memory, so that a warp finishes one token at a time with four features per lane: one
// reduction for a token's scale, 128 features in whole sectors.
// Measured (replayed from a graph): 64 tokens, 16384 x 8192, 27.5 us (5.2 TB/s); 2048 x 4096 in clusters of
// 4, 6.0 us, of which the K loop is two: start of the cluster, first copies, exchange and stores are the
// rest.  A block of K of 128 takes 0.27 us with 64 tokens, bound by the MMA warp: 0.25 with the copies left
// out of a copy of the kernel, 0.145 with the MMAs left out and 0.14 with neither (1000 tokens, 1112 rows, K
// = 1024 and 2048; the four MMAs of a block are 0.1, waiting for stages and handing them over the rest).
constexpr int kStreamThreads = 320;
constexpr int kMaxStages = 8;
// K blocks of 128 per stage: waiting for a stage takes as long as four narrow MMAs, so a stage holds
// eight of them (two blocks of one matrix, or one of two).
template <int NW>
constexpr int kStageBlocks = 2 / NW;
constexpr int kSfSlots = 4;  // ring of scale words, each slot for 4 K blocks (one byte each)
constexpr uint32_t kNoScale = 0x7f7f7f7fu;  // words of rows past the end: 2^0
constexpr uint32_t kSmem = 227 * 1024;
constexpr int kMaxTokens = 1 << 21;  // token tiles stay within a grid's z, tiles and scale bytes within 32 bits

struct StreamParams {
  CUtensorMap w[2], x;
  const uint8_t* sw[2];
  const uint8_t* sx;
  const float* base;
  void* out;
  uint8_t* codes;
  uint8_t* scales;
  int* err;
  int T, N, KB;
  int bn, stages, tmem_cols, sf_col, sfb_cols;
  int out_bf16, vec, sf_align;
  int range, longer;  // K blocks of a CTA of the cluster, and how many have one more
  uint32_t inverse;   // 2^16 / splits, rounded up: n inverse >> 16 is n / splits for n < 2^12
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], sf_full[kSfSlots], sf_empty[kSfSlots], acc_full, done, sums;
  uint32_t tmem_slot;
  int abort_flag;
};

// Scale bytes of an array [rows][KB] (fewer than 2^31) as aligned words: byte i of the array is byte
// i + off from `base`, a multiple of 4; words lo .. hi - 1 lie in the array, and what it has of the words
// on either side of them is in head and tail.
struct Scales {
  const uint8_t* base;
  int off, lo, hi;
  uint32_t head, tail;
};

__device__ __forceinline__ Scales scales_of(const uint8_t* first, int n, int align) {
  Scales s;
  s.off = int(reinterpret_cast<uintptr_t>(first) & 3);
  s.base = first - s.off;
  n += s.off;
  s.lo = (s.off + 3) >> 2, s.hi = n >> 2;
  s.head = s.tail = 0;
  if (align == 1) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (j + 1 >= s.off && j + 1 < n && s.lo) s.head |= uint32_t(s.base[j + 1]) << (8 * j + 8);
      if (j < (n & 3) && 4 * s.hi + j >= s.off) s.tail |= uint32_t(s.base[4 * s.hi + j]) << (8 * j);
    }
  }
  return s;
}

// Scale bytes of one row are read 16 K blocks at a time (a "round": four words of four blocks), so
// that the loads of a round overlap and the next round's are in flight while the MMAs use this one.
// `align`: alignment of the row starts (16 or 4).  Bytes of blocks past the row's end are whatever
// follows in the array; no MMA selects them.
__device__ __forceinline__ uint4 scale_round(const Scales& s, int row, int r, int KB, int align) {
  const uint8_t* p = s.base + row * KB + 16 * r;
  if (align == 16) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 16 * r + 4 * i < KB ? *reinterpret_cast<const uint32_t*>(p + 4 * i) : kNoScale;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Row starts of any alignment: five words around the sixteen bytes, all of a round's rows loaded before
// the first is shifted into place (a load and its use row by row made every call 1 to 2 us longer).
struct ScaleWords {
  uint32_t w[5];
};
__device__ __forceinline__ ScaleWords scale_words(const Scales& s, int row, int r, int KB) {
  const int at = (s.off + row * KB + 16 * r) >> 2;
  ScaleWords v;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    v.w[i] = 0;
    if (s.lo < s.hi) v.w[i] = *reinterpret_cast<const uint32_t*>(s.base + 4 * min(max(at + i, s.lo), s.hi - 1));
  }
  return v;
}
__device__ __forceinline__ uint4 scale_round(const Scales& s, int row, int r, int KB, const ScaleWords& v) {
  const int at = s.off + row * KB + 16 * r, shift = 8 * (at & 3);
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (at >> 2) + i < s.lo ? s.head : (at >> 2) + i >= s.hi ? s.tail : v.w[i];
  return make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                    __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Position in a ring of barriers: slot and the parity of its current phase.  (One warp runs each loop
// over K, so every instruction of its iteration counts: no divisions by the ring's size, and nothing
// but straight-line copies, MMAs and commits under elect_one -- with a loop or a branch in there the
// operands leave the uniform registers and an iteration takes five times as long.)
struct RingPos {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int size) {
    if (++slot == size) slot = 0, parity ^= 1;
  }
};

// Four floats into the shared memory of another CTA of the cluster (or this one), counted as 16 bytes
// on a barrier there: the receiver needs no release from the sender, which would wait for its stores.
__device__ __forceinline__ void st_async_f4(uint32_t addr, uint32_t bar, float4 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}

// The base of `count` (at most B) tokens t, t + step, ...: columns n .. n + 3 of this lane, or (p.vec = 0)
// the same four as in store_tokens.
template <bool kLoose, int B>
__device__ __forceinline__ void load_tokens(const StreamParams& p, float4 (&b)[B], int t, int step, int count, int n, int lane) {
#pragma unroll
  for (int i = 0; i < B; ++i) b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!kLoose || p.vec) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < count && n < p.N) b[i] = *reinterpret_cast<const float4*>(p.base + int64_t(t + i * step) * p.N + n);
    return;
  }
  n -= 3 * lane;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    if (i >= count) break;
    const float* at = p.base + int64_t(t + i * step) * p.N + n;
    if (n < p.N) b[i].x = at[0];
    if (n + 32 < p.N) b[i].y = at[32];
    if (n + 64 < p.N) b[i].z = at[64];
    if (n + 96 < p.N) b[i].w = at[96];
  }
}

// The results of those tokens.  Features n .. n + 3 of this lane; where rows cannot be stored in such
// pieces (p.vec = 0, a plain layer) lane, lane + 32, ... of the tile, which keeps a warp's stores
// together.
template <int NW, bool kLoose, int B>
__device__ __forceinline__ void store_tokens(const StreamParams& p, float4 (&v)[B][NW], const float4 (&b)[B], int t, int step,
                                             int count, int n, int lane) {
  if (NW == 1) {
    if (p.base) {
#pragma unroll
      for (int i = 0; i < B; ++i) v[i][0].x += b[i].x, v[i][0].y += b[i].y, v[i][0].z += b[i].z, v[i][0].w += b[i].w;
    }
    if (!kLoose || p.vec) {  // N a multiple of 4, rows aligned: all four or none
      if (n >= p.N) return;
#pragma unroll
      for (int i = 0; i < B; ++i) {
        if (i >= count) break;
        const int64_t at = int64_t(t + i * step) * p.N + n;
        const float4 o = v[i][0];
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<bf16*>(p.out) + at) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
      }
      return;
    }
    const int n0 = n - 3 * lane;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i >= count) break;
      const int64_t at = int64_t(t + i * step) * p.N + n0;
      const float o[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n0 + 32 * j >= p.N) break;
        if (p.out_bf16) static_cast<bf16*>(p.out)[at + 32 * j] = __float2bfloat16_rn(o[j]);
        else static_cast<float*>(p.out)[at + 32 * j] = o[j];
      }
    }
    return;
  }
  uint32_t m[B];
#pragma unroll
  for (int i = 0; i < B; ++i) {
    const float4 g = v[i][0], u = v[i][NW - 1];
    v[i][0] = make_float4(silu_mul(g.x, u.x), silu_mul(g.y, u.y), silu_mul(g.z, u.z), silu_mul(g.w, u.w));
    m[i] = max(max(mag(v[i][0].x), mag(v[i][0].y)), max(mag(v[i][0].z), mag(v[i][0].w)));
  }
  if (p.codes) {
#pragma unroll
    for (int i = 0; i < B; ++i) m[i] = __reduce_max_sync(0xffffffffu, n < p.N ? m[i] : 0u);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i >= count) break;
      const int64_t tok = t + i * step;
      const uint32_t b = scale_byte(m[i]);
      const float inv = scale_inverse(b);
      const float4 h = v[i][0];
      if (n < p.N) *reinterpret_cast<uint32_t*>(p.codes + tok * p.N + n) = pack4(h.x * inv, h.y * inv, h.z * inv, h.w * inv);
      if (lane == 0) p.scales[tok * ((p.N + 127) / 128) + blockIdx.y] = uint8_t(b);
    }
  } else if (n < p.N) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i >= count) break;
      const float4 h = v[i][0];
      *reinterpret_cast<uint2*>(static_cast<bf16*>(p.out) + int64_t(t + i * step) * p.N + n) =
          make_uint2(pack_bf16x2(h.x, h.y), pack_bf16x2(h.z, h.w));
    }
  }
}

// NW = 1: out = base + W x.  NW = 2: h = silu(W0 x) (W1 x), to bf16 or codes and scales.  kSplit: K is split
// over a cluster.  kLoose: rows of outputs, bases and scales of any alignment (p.vec, p.sf_align).  Both are
// there because a launch of few us waits for its instructions, each of which runs once or twice (2048 x
// 4096, 64 tokens: 6.9 us with the code for unaligned rows, 6.4 without).
template <int NW, bool kSplit, bool kLoose>
__global__ void __launch_bounds__(kStreamThreads, 2) fp8_stream_kernel(const __grid_constant__ StreamParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(sizeof(Bars) <= 1024, "shared memory");
  Bars& bars = *reinterpret_cast<Bars*>(smem);
  // 32-bit shared addresses
  const uint32_t smem0 = smem_u32(smem), ring = smem0 + 1024;
  const uint32_t full = smem0 + offsetof(Bars, full), empty = smem0 + offsetof(Bars, empty);
  const uint32_t sf_full = smem0 + offsetof(Bars, sf_full), sf_empty = smem0 + offsetof(Bars, sf_empty);
  const uint32_t acc_full = smem0 + offsetof(Bars, acc_full), done = smem0 + offsetof(Bars, done);
  const uint32_t sums_full = smem0 + offsetof(Bars, sums);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kSplit ? blockIdx.x : 0, splits = kSplit ? gridDim.x : 1;
  const int row0 = blockIdx.y * 128, tok0 = blockIdx.z * p.bn;
  const int kb0 = rank * p.range + min(rank, p.longer), kb1 = kb0 + p.range + (rank < p.longer);
  const uint32_t block_bytes = NW * 16384 + p.bn * 128, stage_bytes = kStageBlocks<NW> * block_bytes;
  const int nt = min(p.bn, p.T - tok0);
  const auto by_splits = [&](int n) { return kSplit ? int(uint32_t(n) * p.inverse >> 16) : n; };  // n / splits
  // this CTA's tokens (rank, rank + splits, ...) and what arrives for them: [token][sender][matrix][feature]
  const int mine = rank < nt ? by_splits(nt - rank + splits - 1) : 0;
  const uint32_t sums = ring + p.stages * stage_bytes;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&p.w[0]), tma_prefetch_map(&p.x);
    if (NW == 2) tma_prefetch_map(&p.w[1]);
    for (int s = 0; s < p.stages; ++s) mbar_init(&bars.full[s], 1), mbar_init(&bars.empty[s], 1);
    for (int s = 0; s < kSfSlots; ++s) mbar_init(&bars.sf_full[s], 128), mbar_init(&bars.sf_empty[s], 1);
    mbar_init(&bars.acc_full, 1), mbar_init(&bars.done, 1), mbar_init(&bars.sums, 1);
    bars.abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(&bars.sums, mine * splits * NW * 512);
  }
  if (warp == 1) tmem_alloc(&bars.tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  // the barriers of the cluster exist before anything is sent (awaited before the first store)
  if (kSplit) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  volatile int* abort_flag = &bars.abort_flag;
  pdl_trigger();

  // (every role that touches global memory waits for the predecessor grid itself, as late as it can)
  bool joined = !kSplit;
  // the loops over K of warps 0 and 1 are run by the whole warp, with one lane (elect_one) issuing
  if (warp == 0) {
    RingPos at;
    int i = 0;
    uint32_t st = ring;
    bool ok = true;
    pdl_wait();
    for (int kb = kb0; kb < kb1; kb += kStageBlocks<NW>, ++i) {
      if (i >= p.stages) ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * at.slot, at.parity ^ 1, abort_flag, p.err));
      if (!ok) break;
      const uint32_t bar = full + 8 * at.slot;
      const bool two = kStageBlocks<NW> == 2 && kb + 1 < kb1;
      const uint32_t bytes = two ? 2 * block_bytes : block_bytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d(st, &p.w[0], kb * 128, row0, bar);
        if (NW == 2) tma_load_2d(st + 16384, &p.w[1], kb * 128, row0, bar);
        tma_load_2d(st + NW * 16384, &p.x, kb * 128, tok0, bar);
      }
      if (two) {
        const uint32_t next = st + block_bytes;
        if (elect_one()) {
          tma_load_2d(next, &p.w[0], kb * 128 + 128, row0, bar);
          tma_load_2d(next + NW * 16384, &p.x, kb * 128 + 128, tok0, bar);
        }
      }
      at.next(p.stages);
      st = at.slot ? st + stage_bytes : ring;
    }
    // copies may still be in flight if the MMA warp gave up
    for (int j = max(0, i - p.stages); j < i; ++j) mbar_drain(full + 8 * (j % p.stages), (j / p.stages) & 1);
  } else if (warp == 1) {
    RingPos at;
    bool ok = true;
    const uint32_t low0 = umma_desc_low(ring), sf_step = 4 * NW + p.sfb_cols;
    uint32_t low = low0, accumulate = 0;
    pdl_wait();  // (so that the limits of the waits below count from the predecessor's end)
    for (int kb = kb0; kb < kb1; kb += kStageBlocks<NW>) {
      ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * at.slot, at.parity, abort_flag, p.err));
#pragma unroll
      for (int j = 0; j < kStageBlocks<NW>; ++j) {
        const int b = kb + j, slot = (b >> 2) % kSfSlots;
        if (b >= kb1) break;
        if (b == kb0 || (b & 3) == 0) {  // (a slot's phase turns over every four words)
          ok = ok && __all_sync(0xffffffffu, mbar_wait(sf_full + 8 * slot, ((b >> 2) - (kb0 >> 2)) / kSfSlots & 1, abort_flag, p.err));
          tc_fence_after();
        }
        if (!ok) break;
        const uint32_t sf = tmem + p.sf_col + slot * sf_step, idesc = umma_idesc_mx8(128, p.bn, b & 3);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int m = 0; m < NW; ++m)
              umma_mx8(tmem + m * p.bn, umma_desc_of(low + m * 1024 + 2 * k), umma_desc_of(low + NW * 1024 + 2 * k), idesc,
                       sf + 4 * m, sf + 4 * NW, k ? 1 : accumulate);
          }
        }
        if ((b & 3) == 3 && elect_one()) umma_commit(sf_empty + 8 * slot);
        accumulate = 1;
        low += block_bytes >> 4;
      }
      if (!ok) break;
      if (elect_one()) umma_commit(empty + 8 * at.slot);
      at.next(p.stages);
      if (at.slot == 0) low = low0;
    }
    if (elect_one()) {
      if (ok) umma_commit(acc_full);
      umma_commit(done);
    }
    // every MMA issued above has finished before tensor memory is released
    mbar_drain(done, 0);
  } else {
    const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
    const int group = (warp - 2) >> 2;
    bool ok = true;
    pdl_wait();
    if (group == 0) {
      // scale words: each of the four warps writes them to its own lane quarter
      const int q0 = kb0 / 4, q1 = (kb1 - 1) / 4;
      constexpr int kCols = kSplit ? 4 : 8;  // (a tile that splits K has up to 128 / NW tokens)
      const int cols = (p.bn + 31) / 32;
      const int align = kLoose ? p.sf_align : 4;
      const Scales sx = scales_of(p.sx, p.T * p.KB, align);
      Scales sw[NW];
#pragma unroll
      for (int m = 0; m < NW; ++m) sw[m] = scales_of(p.sw[m], (p.N + 127) / 128 * p.KB, align);
      uint4 wa[NW], wb[kCols];
      auto load = [&](int r) {
        if (kLoose && p.sf_align == 1) {
          ScaleWords a[NW], b[4];
#pragma unroll
          for (int m = 0; m < NW; ++m) a[m] = scale_words(sw[m], blockIdx.y, r, p.KB);
#pragma unroll
          for (int half = 0; half < kCols; half += 4) {
            if (half && cols <= half) break;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (half + c < cols) b[c] = scale_words(sx, min(tok0 + 32 * (half + c) + lane, p.T - 1), r, p.KB);
            if (half == 0) {
#pragma unroll
              for (int m = 0; m < NW; ++m) wa[m] = scale_round(sw[m], blockIdx.y, r, p.KB, a[m]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int t = tok0 + 32 * (half + c) + lane;
              wb[half + c] = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
              if (half + c < cols && t < p.T) wb[half + c] = scale_round(sx, t, r, p.KB, b[c]);
            }
          }
          return;
        }
#pragma unroll
        for (int m = 0; m < NW; ++m) wa[m] = scale_round(sw[m], blockIdx.y, r, p.KB, p.sf_align);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int t = tok0 + 32 * c + lane;
          wb[c] = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
          if (c < cols && t < p.T) wb[c] = scale_round(sx, t, r, p.KB, p.sf_align);
        }
      };
      load(q0 / 4);
      for (int r = q0 / 4; r <= q1 / 4 && ok; ++r) {
#pragma unroll 1
        for (int slot = 0; slot < kSfSlots; ++slot) {
          const int q = 4 * r + slot, i = q - q0;
          if (i < 0 || q > q1) continue;
          if (i >= kSfSlots) {
            ok = named_bar_and(1, 128, mbar_wait(sf_empty + 8 * slot, (i / kSfSlots - 1) & 1, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t sf = tmem + quarter + p.sf_col + slot * (4 * NW + p.sfb_cols);
#pragma unroll
          for (int m = 0; m < NW; ++m) {
            const uint32_t w = word(wa[m], slot);
            tmem_st4(sf + 4 * m, w, w, w, w);
          }
          tmem_st4(sf + 4 * NW, word(wb[0], slot), word(wb[1], slot), word(wb[2], slot), word(wb[3], slot));
          if (kCols > 4 && p.sfb_cols > 4)
            tmem_st4(sf + 4 * NW + 4, word(wb[4 % kCols], slot), word(wb[5 % kCols], slot), word(wb[6 % kCols], slot), word(wb[7 % kCols], slot));
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars.sf_full[slot]);
        }
        if (r < q1 / 4) load(r + 1);
      }
    }
    ok = named_bar_and(2, 256, ok && mbar_wait(acc_full, 0, abort_flag, p.err));
    if (kSplit) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      joined = true;
    }
    if (ok) {
      tc_fence_after();
      const uint32_t feature = 4 * ((warp & 3) * 32 + lane);
      for (int c = 16 * group; c < nt; c += 32) {
#pragma unroll
        for (int m = 0; m < NW; ++m) {
          float v[16];
          tmem_ld16(tmem + quarter + m * p.bn + c, v);
          if (!kSplit) {
            // (over the ring: every load has been read by an MMA, and every MMA has finished)
            const uint32_t dst = ring + (c * NW + m) * 512 + feature;
#pragma unroll
            for (int i = 0; i < 16; ++i) sts_f32(dst + i * (NW * 512), v[i]);
          } else {
            // the warp's 32 features of 16 tokens, turned through its own part of the (free) ring so
            // that a lane sends four features at once: 8 lanes per token
            const uint32_t turn = ring + (warp - 2) * 2304;
#pragma unroll
            for (int i = 0; i < 16; ++i) sts_f32(turn + i * 144 + lane * 4, v[i]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = 4 * i + (lane >> 3), slot = by_splits(c + t), owner = c + t - slot * splits;
              const float4 o = lds_f4(turn + t * 144 + (lane & 7) * 16);
              if (c + t < nt)
                st_async_f4(map_cluster_rank(sums, owner) + ((slot * splits + rank) * NW + m) * 512 + (warp & 3) * 128 + (lane & 7) * 16,
                            map_cluster_rank(sums_full, owner), o);
            }
            __syncwarp();
          }
        }
      }
    }
    // Tokens per warp at a time: their loads and reductions overlap.  (64 tokens over a cluster leave a warp
    // two, 6.2 us with a batch of four and 5.95 with two; 16384 x 8192 without a split 28.6 with two, 27.5.)
    constexpr int kBatch = kSplit ? 2 : 4;
    const int n = row0 + 4 * lane, first = tok0 + rank;
    const bool read_base = NW == 1 && p.base;
    float4 base[kBatch];
    if (read_base) load_tokens<kLoose>(p, base, first + (warp - 2) * splits, 8 * splits, (mine - (warp - 2) + 7) / 8, n, lane);
    // (an aborted CTA sends nothing: its owners' waits run out, and the status word says so)
    if (!kSplit) asm volatile("bar.sync 2, 256;" ::: "memory");
    else if (mine > 0) ok = named_bar_and(2, 256, mbar_wait_cluster(sums_full, 0, abort_flag, p.err));
    if (ok) {
      const bool spread = kLoose && NW == 1 && !p.vec;
      const uint32_t src = (kSplit ? sums : ring) + (spread ? 4 : 16) * lane;
      for (int j0 = warp - 2; j0 < mine; j0 += 8 * kBatch) {
        const int count = (mine - j0 + 7) / 8;
        if (read_base && j0 != warp - 2) load_tokens<kLoose>(p, base, first + j0 * splits, 8 * splits, count, n, lane);
        float4 v[kBatch][NW];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int m = 0; m < NW; ++m) v[i][m] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int r = 0; r < splits; ++r) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i >= count) break;
#pragma unroll
            for (int m = 0; m < NW; ++m) {
              const uint32_t at = src + (((j0 + 8 * i) * splits + r) * NW + m) * 512;
              const float4 a = spread ? make_float4(lds_f32(at), lds_f32(at + 128), lds_f32(at + 256), lds_f32(at + 384)) : lds_f4(at);
              v[i][m].x += a.x, v[i][m].y += a.y, v[i][m].z += a.z, v[i][m].w += a.w;
            }
          }
        }
        store_tokens<NW, kLoose, kBatch>(p, v, base, first + j0 * splits, 8 * splits, count, n, lane);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (!joined) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  if (kSplit) {
    // an owner that gave up stays until nothing more can be sent to it; the others need not wait
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (*abort_flag) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

// ------------------------------------------------------------------ pair kernel
// Many tokens: bound by the tensor cores.  A pair of CTAs (cta_group::2) computes 256 tokens x 256
// weight rows: tokens are the M side, 128 per CTA, so that a thread of the epilogue holds one token's
// row of consecutive features (a group's largest magnitude needs no exchange beyond two threads), and
// each CTA loads half of the weight rows, which halves the shared-memory traffic of B.  A gated tile
// is 128 gate rows (first CTA) and the 128 up rows of the same features (second CTA).  Persistent:
// the pairs walk the tiles in groups of 8 token tiles, so that the operands in use stay in L2.
// Roles by warpgroup: warp 0 TMA loads and warp 1 the MMAs (first CTA only); warps 4..7 the scale
// words; warps 8..15 the epilogue (two per lane quarter, each half of the 256 columns).  The 256
// accumulator columns are drained into registers (128 per thread) and released before anything is
// computed or stored, so the next tile's MMAs wait for the drain alone; the registers come from the
// other two warpgroups (128 x (48 + 48 + 208 + 208) = the 512 x 128 launched).
// Measured: 8192 x 8192 x 8192 376 us (2.93 PFLOP/s), 8192 x 4096 x 4096 100 us (2.75; tensor pipe 80%
// busy), gated 4096 tokens, 2 x 5504 x 2048, 76 us (2.44; 64%).  A block of K takes 0.33 us where its MMAs
// take 0.28: its operands' way into shared memory and out of it is as wide as the MMAs need, no wider.
// The drain between tiles is 1 us, whatever K is.
constexpr int kPairThreads = 512;
constexpr int kPairStages = 6;
constexpr int kPairStage = 2 * 16384;  // per CTA: 128 token rows, 128 weight rows, 128 columns
constexpr int kPairSfCol = 256;        // scale words behind the accumulators: 4 + 8 columns per slot
constexpr int kPairGroup = 8;

struct PairParams {
  CUtensorMap w[2], x;
  const uint8_t* sw[2];
  const uint8_t* sx;
  const float* base;
  void* out;
  uint8_t* codes;
  uint8_t* scales;
  int* err;
  int T, N, KB;
  int m_tiles, n_tiles;
  int out_bf16, sf_align;  // sf_align: alignment of the scale rows (16, 4, 1)
};

struct PairBars {
  uint64_t full[kPairStages], empty[kPairStages], sf_full[kSfSlots], sf_empty[kSfSlots], acc_full, acc_empty, done;
  uint32_t tmem_slot;
  int abort_flag;
  uint32_t amax[2][2][128];  // [tile parity][column half][token]
};

enum PairEpi { kPairBf16 = 0, kPairF32 = 1, kPairBase = 2, kPairGatedBf16 = 3, kPairGatedCodes = 4, kPairLoose = 5 };

__device__ __forceinline__ void pair_tile(const PairParams& p, int i, int& mt, int& nt) {
  const int per = kPairGroup * p.n_tiles, g = i / per, r = i - g * per;
  const int rows = min(kPairGroup, p.m_tiles - g * kPairGroup);
  nt = r / rows, mt = g * kPairGroup + r - nt * rows;
}

// One warp's 32 token rows x 128 columns, one row per thread in `v`, to global memory.  A chunk of
// 128 bytes per row goes through 4 KB of shared memory (16-byte pieces, XOR-swizzled by row, so both
// sides are conflict-free), and leaves as whole lines: 8 lanes per row, 4 rows per instruction.
// kElem: bytes per staged element (4: fp32, 2: bf16 pairs packed before staging); with a base the
// sums are staged as fp32 and the base is read in the same pattern, one chunk ahead.
struct RowsOut {
  const float* base;
  uint8_t* out;
  int64_t tok;  // first token
  int n0, T, N, out_bf16;
};

// The base of a warp's rows from column `first` of its 128 on, on its way to L2 while the tile's MMAs run (a
// row per lane).
__device__ __forceinline__ void prefetch_base(const RowsOut& o, int first, int lane) {
  const int64_t t = o.tok + lane;
  const float* at = o.base + t * o.N + o.n0;
#pragma unroll
  for (int c = first; c < 128; c += 32)
    if (t < o.T && o.n0 + c < o.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c));
}

template <bool kBase>
__device__ __forceinline__ void load_base(const RowsOut& o, int chunk, int lane, float4 (&b)[8]) {
  if (!kBase) return;
  const int n = o.n0 + chunk * 32 + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t t = o.tok + 4 * i + (lane >> 3);
    b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < o.T && n < o.N) b[i] = *reinterpret_cast<const float4*>(o.base + t * o.N + n);
  }
}

template <int kElem, bool kBase>
__device__ __forceinline__ void store_rows(const RowsOut& o, const uint32_t (&v)[128], uint32_t stage, int lane,
                                           float4 (&b)[8]) {
  constexpr int kCols = 128 / kElem;
#pragma unroll
  for (int c = 0; c < 128 / kCols; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = c * kCols + (4 * i + j) * (4 / kElem);
        w[j] = kElem == 4 ? v[e & 127] : pack_bf16x2(__uint_as_float(v[e & 127]), __uint_as_float(v[(e + 1) & 127]));
      }
      sts_v4(stage + lane * 128 + ((i ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    const int n = o.n0 + c * kCols + (lane & 7) * (16 / kElem);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const int64_t t = o.tok + r;
      float4 x = lds_f4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      if (kBase) x.x += b[i].x, x.y += b[i].y, x.z += b[i].z, x.w += b[i].w;
      if (t < o.T && n < o.N) {
        if (kBase && o.out_bf16)
          *reinterpret_cast<uint2*>(o.out + (t * o.N + n) * 2) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        else
          *reinterpret_cast<float4*>(o.out + (t * o.N + n) * kElem) = x;
      }
    }
    __syncwarp();
    if (c + 1 < 128 / kCols) load_base<kBase>(o, c + 1, lane, b);
  }
}

// The same for rows of any alignment: 32 columns of a row per instruction, one element per lane.  Bound by
// its instructions, so that a row costs a load from shared memory at a constant offset, a pointer's step
// and a store (4096 x 4095 fp32, K = 512: 60 us with pieces that start on a line and indexes per element).
template <typename Out>
__device__ __forceinline__ void store_rows_loose(const RowsOut& o, const uint32_t (&v)[128], uint32_t stage, int lane) {
  constexpr int kRows = 16;
  uint32_t from[8];  // the lane's column of rows r, r + 8, ...
#pragma unroll
  for (int r = 0; r < 8; ++r) from[r] = stage + r * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4;
  const int all = int(min(int64_t(32), o.T - o.tok));
  const int64_t step = o.N;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int n = o.n0 + 32 * c + lane;
    const int rows = n < o.N ? all : 0;
    Out* dst = reinterpret_cast<Out*>(o.out) + o.tok * step + n;
    const float* src = o.base + o.tok * step + n;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sts_v4(stage + lane * 128 + ((i ^ (lane & 7)) << 4), v[32 * c + 4 * i], v[32 * c + 4 * i + 1], v[32 * c + 4 * i + 2],
             v[32 * c + 4 * i + 3]);
    __syncwarp();
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += kRows) {
      float x[kRows];
      if (o.base) {
#pragma unroll
        for (int r = 0; r < kRows; ++r, src += step) x[r] = r0 + r < rows ? *src : 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r] += lds_f32(from[r & 7] + (r0 + r / 8 * 8) * 128);
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r] = lds_f32(from[r & 7] + (r0 + r / 8 * 8) * 128);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r, dst += step)
        if (r0 + r < rows) *dst = Out(x[r]);
    }
    __syncwarp();
  }
}

template <int EPI>
__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const __grid_constant__ PairParams p) {
  constexpr bool kGated = EPI == kPairGatedBf16 || EPI == kPairGatedCodes;
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(kPairStages * kPairStage + 32768 + sizeof(PairBars) <= kSmem, "shared memory");
  // 32-bit shared addresses
  const uint32_t ring = smem_u32(smem), staging = ring + kPairStages * kPairStage, bar0 = staging + 32768;
  const uint32_t full = bar0 + offsetof(PairBars, full), empty = bar0 + offsetof(PairBars, empty);
  const uint32_t sf_full = bar0 + offsetof(PairBars, sf_full), sf_empty = bar0 + offsetof(PairBars, sf_empty);
  const uint32_t acc_full = bar0 + offsetof(PairBars, acc_full), acc_empty = bar0 + offsetof(PairBars, acc_empty);
  const uint32_t done = bar0 + offsetof(PairBars, done);
  PairBars& bars = *reinterpret_cast<PairBars*>(smem + kPairStages * kPairStage + 32768);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int n_tiles = p.m_tiles * p.n_tiles, nq = (p.KB + 3) / 4;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&p.w[kGated ? rank : 0]), tma_prefetch_map(&p.x);
    for (int s = 0; s < kPairStages; ++s) mbar_init(&bars.full[s], 1), mbar_init(&bars.empty[s], 1);
    for (int s = 0; s < kSfSlots; ++s) mbar_init(&bars.sf_full[s], 8), mbar_init(&bars.sf_empty[s], 1);
    mbar_init(&bars.acc_full, 1), mbar_init(&bars.acc_empty, 16), mbar_init(&bars.done, 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&bars.tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  volatile int* abort_flag = &bars.abort_flag;
  pdl_trigger();
  pdl_wait();

  // the loops over K of warps 0 and 1 are run by the whole warp, with one lane (elect_one) issuing
  if (warp < 4) regs_down<48>();
  if (warp == 0) {
    RingPos at;
    int i = 0;
    bool ok = true;
    const uint32_t full0 = map_cluster_rank(full, 0);
    for (int tile = pair; tile < n_tiles && ok; tile += pairs) {
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const int tok = mt * 256 + rank * 128, row = kGated ? nt * 128 : nt * 256 + rank * 128;
      const CUtensorMap* w = &p.w[kGated ? rank : 0];
      for (int kb = 0; kb < p.KB; ++kb, ++i) {
        if (i >= kPairStages)
          ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * at.slot, at.parity ^ 1, abort_flag, p.err));
        if (!ok) break;
        const uint32_t st = ring + at.slot * kPairStage, bar = full0 + 8 * at.slot;
        // both CTAs' copies complete on the first CTA's barrier
        if (rank == 0 && elect_one()) mbar_arrive_expect_tx(full + 8 * at.slot, 2 * kPairStage);
        if (elect_one()) {
          tma_load_2d_pair(st, &p.x, kb * 128, tok, bar);
          tma_load_2d_pair(st + 16384, w, kb * 128, row, bar);
        }
        at.next(kPairStages);
      }
    }
    if (rank == 0) {
      for (int j = max(0, i - kPairStages); j < i; ++j) mbar_drain(full + 8 * (j % kPairStages), (j / kPairStages) & 1);
    } else if (!ok) {
      // given up: the copies complete on the other CTA's barrier; leave them time to land
      for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < 1000000;) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      RingPos at, sf;
      uint32_t acc_parity = 1;
      bool ok = true;
      const uint32_t low0 = umma_desc_low(ring);
      for (int tile = pair; tile < n_tiles && ok; tile += pairs, acc_parity ^= 1) {
        for (int kb = 0; kb < p.KB && ok; ++kb) {
          if ((kb & 3) == 0) {
            ok = mbar_wait_cluster(sf_full + 8 * sf.slot, sf.parity, abort_flag, p.err);
            tc_fence_after();
          }
          ok = __all_sync(0xffffffffu, ok && mbar_wait(full + 8 * at.slot, at.parity, abort_flag, p.err));
          if (kb == 0 && tile != pair) {  // the operands are there; last, the accumulators
            ok = __all_sync(0xffffffffu, ok && mbar_wait_cluster(acc_empty, acc_parity, abort_flag, p.err));
            tc_fence_after();
          }
          if (!ok) break;
          const uint32_t low = low0 + at.slot * (kPairStage >> 4);
          const uint32_t sfa = tmem + kPairSfCol + sf.slot * 12;
          const uint32_t idesc = umma_idesc_mx8(256, 256, kb & 3);
          const bool last = (kb & 3) == 3 || kb == p.KB - 1;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mx8_pair(tmem, umma_desc_of(low + 2 * k), umma_desc_of(low + 1024 + 2 * k), idesc, sfa, sfa + 4,
                            k ? 1 : kb != 0);
            umma_commit_pair(empty + 8 * at.slot);
          }
          at.next(kPairStages);
          if (last) {
            if (elect_one()) umma_commit_pair(sf_empty + 8 * sf.slot);
            sf.next(kSfSlots);
          }
        }
        if (ok && elect_one()) umma_commit_pair(acc_full);
      }
      if (elect_one()) umma_commit_pair(done);
    }
    // the last arrival of a commit on either CTA's barriers
    mbar_drain(done, 0);
  } else if (warp < 4) {
  } else if (warp < 8) {
    regs_down<48>();
    // scale words of this CTA's tokens (4 columns) and of all 256 weight rows (8 columns)
    const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
    const int blocks = (p.N + 127) / 128;
    const Scales sx = scales_of(p.sx, p.T * p.KB, p.sf_align);
    const Scales sw0 = scales_of(p.sw[0], blocks * p.KB, p.sf_align);
    const Scales sw1 = kGated ? scales_of(p.sw[1], blocks * p.KB, p.sf_align) : sw0;
    uint4 a[4], u, v;
    auto load = [&](int tile, int r) {
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const int tok0 = mt * 256 + rank * 128 + lane;
      const int b0 = kGated ? nt : 2 * nt, b1 = kGated ? nt : 2 * nt + 1;
      if (p.sf_align == 1) {
        ScaleWords x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = scale_words(sx, min(tok0 + 32 * c, p.T - 1), r, p.KB);
        const ScaleWords y = scale_words(sw0, b0, r, p.KB), z = scale_words(sw1, min(b1, blocks - 1), r, p.KB);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          a[c] = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
          if (tok0 + 32 * c < p.T) a[c] = scale_round(sx, tok0 + 32 * c, r, p.KB, x[c]);
        }
        u = scale_round(sw0, b0, r, p.KB, y);
        v = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
        if (b1 < blocks) v = scale_round(sw1, b1, r, p.KB, z);
        return;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[c] = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
        if (tok0 + 32 * c < p.T) a[c] = scale_round(sx, tok0 + 32 * c, r, p.KB, p.sf_align);
      }
      u = scale_round(sw0, b0, r, p.KB, p.sf_align);
      v = make_uint4(kNoScale, kNoScale, kNoScale, kNoScale);
      if (b1 < blocks) v = scale_round(sw1, b1, r, p.KB, p.sf_align);
    };
    int sq = 0;
    bool ok = true;
    if (pair < n_tiles) load(pair, 0);
    for (int tile = pair; tile < n_tiles && ok; tile += pairs) {
      for (int q = 0; q < nq && ok; q += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (q + i >= nq) break;
          const int slot = sq % kSfSlots;
          if (sq >= kSfSlots) {
            ok = named_bar_and(1, 128, mbar_wait(sf_empty + 8 * slot, (sq / kSfSlots - 1) & 1, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t sf = tmem + quarter + kPairSfCol + slot * 12;
          const uint32_t uw = word(u, i), vw = word(v, i);
          tmem_st4(sf, word(a[0], i), word(a[1], i), word(a[2], i), word(a[3], i));
          tmem_st4(sf + 4, uw, uw, uw, uw);
          tmem_st4(sf + 8, vw, vw, vw, vw);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(map_cluster_rank(sf_full + 8 * slot, 0));
          ++sq;
        }
        // the next round, or the first of the next tile
        if (q + 4 < nq) load(tile, q / 4 + 1);
        else if (tile + pairs < n_tiles) load(tile + pairs, 0);
      }
    }
  } else {
    regs_up<208>();
    const int quarter = warp & 3, half = (warp - 8) >> 2;
    const int row = quarter * 32 + lane;
    // plain: 128 consecutive columns; gated: 64 gate columns and the up columns of the same features
    const uint32_t acc0 = tmem + (uint32_t(quarter * 32) << 16) + half * (kGated ? 64 : 128);
    const uint32_t acc1 = acc0 + (kGated ? 128 : 64);
    const uint32_t released = map_cluster_rank(acc_empty, 0);
    uint32_t parity = 0;
    for (int tile = pair; tile < n_tiles; tile += pairs, parity ^= 1) {
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const RowsOut rows{p.base, static_cast<uint8_t*>(p.out), int64_t(mt) * 256 + rank * 128 + quarter * 32,
                         nt * 256 + half * 128, p.T, p.N, p.out_bf16};
      float4 base[8];
      load_base<EPI == kPairBase>(rows, 0, lane, base);  // (in flight during the tile's MMAs)
      // (where there is a next tile to overlap with: 4096 x 4096 fp32, K = 512, 43 -> 39 us, but a single
      // round of tiles 14.9 -> 15.3)
      if (EPI == kPairBase && n_tiles > pairs) prefetch_base(rows, 32, lane);
      if (EPI == kPairLoose && p.base && n_tiles > pairs) prefetch_base(rows, 0, lane);
      if (!named_bar_and(2, 256, mbar_wait(acc_full, parity, abort_flag, p.err))) break;
      tc_fence_after();
      uint32_t v[128];
      tmem_ld64x2(acc0, acc1, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(released);
      const int64_t tok = int64_t(mt) * 256 + rank * 128 + row;
      const bool live = tok < p.T;
      if (EPI == kPairLoose) {
        if (p.out_bf16) store_rows_loose<bf16>(rows, v, staging + (warp - 8) * 4096, lane);
        else store_rows_loose<float>(rows, v, staging + (warp - 8) * 4096, lane);
      } else if (!kGated) {
        store_rows<EPI == kPairBf16 ? 2 : 4, EPI == kPairBase>(rows, v, staging + (warp - 8) * 4096, lane, base);
      } else {
        const int f0 = nt * 128 + half * 64;
        float h[64];
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool in = f0 + 16 * c < p.N;  // N is a multiple of 16
#pragma unroll
          for (int j = 16 * c; j < 16 * c + 16; ++j) {
            h[j] = silu_mul(__uint_as_float(v[j]), __uint_as_float(v[64 + j]));
            m = max(m, in ? mag(h[j]) : 0u);
          }
        }
        if (EPI == kPairGatedCodes) {
          // the group's other 64 features are with the thread of the other half
          bars.amax[parity][half][row] = m;
          asm volatile("bar.sync 3, 256;" ::: "memory");
          const uint32_t b = scale_byte(max(m, bars.amax[parity][half ^ 1][row]));
          const float inv = scale_inverse(b);
          if (live) {
            uint8_t* dst = p.codes + tok * p.N + f0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (f0 + 16 * c >= p.N) continue;
              const float* x = h + 16 * c;
              *reinterpret_cast<uint4*>(dst + 16 * c) =
                  make_uint4(pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                             pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv),
                             pack4(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv),
                             pack4(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv));
            }
            if (half == 0) p.scales[tok * ((p.N + 127) / 128) + nt] = uint8_t(b);
          }
        } else if (live) {
          uint8_t* dst = static_cast<uint8_t*>(p.out) + (tok * p.N + f0) * 2;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (f0 + 16 * c >= p.N) continue;
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(h[16 * c + 2 * j], h[16 * c + 2 * j + 1]);
            reinterpret_cast<uint4*>(dst + 32 * c)[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4*>(dst + 32 * c)[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
  }
  __syncthreads();
  cluster_sync();  // no copy, MMA or arrival of the pair is still on its way to either CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
// Tensor map of an e4m3 matrix [rows][K]: boxes of 128 columns x box_rows, 128-byte swizzle.
int make_tmap_codes(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int box_rows) {
  const auto fn = encode_tiled_fn();
  if (!fn) return SCION_ECUDA;
  cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(K)};
  cuuint32_t box[2] = {128, cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SCION_OK : SCION_ECUDA;
}

int status(cudaError_t e) {
  return e == cudaSuccess ? SCION_OK : e == cudaErrorMemoryAllocation ? SCION_ENOMEM : SCION_ECUDA;
}

// Clusters of n CTAs of the stream kernel that are on the current device at once, one CTA per SM.
cudaError_t max_clusters(int n, int* count) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n), cfg.blockDim = dim3(kStreamThreads), cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(count, fp8_stream_kernel<1, true, false>, &cfg);
}

// Shape of a stream launch and what it is expected to take.
struct StreamPlan {
  int bn, t_tiles, n_tiles, splits;
  double us;
};

// Tokens per tile: the accumulators (nw bn columns) and the scale words share 512 columns of tensor
// memory, so 256 at most (208 for two matrices); narrower tiles give more CTAs, and tiles of up to
// 128 / nw tokens can split K over a cluster.  The estimate is a fit to launches of 8 to 128 tiles of
// 32 to 128 tokens, K = 2048 to 8192: a start that grows with the tile's tokens (they pass the epilogue one
// warp each), with the cluster and with the share of the SMs in use (a term without a cause found for it),
// and a time per block of K, which the MMA warp bounds up to 128 tokens; weights that come from HBM are not
// in it.  Clusters that leave next to no SM free start late: 1000 tokens, 1112 x 2048, take 8.6 us as 72
// pairs of CTAs and 7.5 as 144 CTAs.  What it is good for is the choice: over 978 shapes (33 to 4096 tokens,
// K = 256 to 8192, n = 512 to 16384, plain and gated, with and without a base) on both kernels, nine tenths
// of the estimates are 0.71 to 1.17 of the time, and the kernel chosen is more than 5% behind the other in
// 28, more than 10% in 12, 21% at most (gated, 128 tokens, 2 x 8192 x 512: 8.2 us, 6.8 streamed).
StreamPlan plan_stream(const scion_fp8* L, int nw, int T, int N, int KB) {
  StreamPlan best{};
  for (int most : {256, 128, 64}) {
    StreamPlan p;
    if (nw == 2) most = std::min(most, 208);
    p.n_tiles = (N + 127) / 128, p.t_tiles = (T + most - 1) / most;
    p.bn = ((T + p.t_tiles - 1) / p.t_tiles + 15) / 16 * 16;
    const int64_t tiles = int64_t(p.n_tiles) * p.t_tiles;
    // (the sums of a wide tile would leave too little shared memory for the ring)
    for (p.splits = 1; p.splits <= (p.bn > 128 / nw ? 1 : std::min(8, KB)); ++p.splits) {
      // all clusters at once: 16 tiles of 64 tokens, K = 4096, took 6.8 us in clusters of 4 and 12.4 in
      // clusters of 8, of which 15 fit
      if (p.splits > 1 && L->clusters[p.splits] < tiles) break;
      const int range = (KB + p.splits - 1) / p.splits;
      const double waves = double((tiles * p.splits + L->sms - 1) / L->sms);
      const double used = std::min(1.0, double(tiles * p.splits) / L->sms);
      const double wide = std::max(0, p.bn - 128 / nw);
      if (p.splits == 1)
        p.us = waves * ((nw == 1 ? 1.6 + 0.018 * p.bn : 2.0 + 0.045 * p.bn) + used + range * (nw == 1 ? 0.262 + 0.0015 * wide : 0.385 + 0.0012 * wide));
      else
        p.us = (nw == 1 ? 1.6 + 0.018 * p.bn : 1.9 + 0.034 * p.bn) + 0.08 * p.splits + 1.8 * used + (used > 0.9) + range * (nw == 1 ? 0.245 : 0.37);
      if (!best.bn || p.us < best.us) best = p;
    }
  }
  return best;
}

// The same for the pair kernel, fitted the same way (0.76 to 1.07 of the time).  A base costs a round of tiles about 4 us (it passes
// through the shared memory that the next tile's MMAs read from), the streaming kernel less than one.
double pair_us(const scion_fp8* L, int nw, int T, int N, int KB, bool base) {
  const int64_t tiles = int64_t((T + 255) / 256) * (nw == 1 ? (N + 255) / 256 : (N + 127) / 128);
  const int pairs = std::max(1, L->sms / 2);
  return (nw == 1 ? 3.7 : 4.3) + double((tiles + pairs - 1) / pairs) * (1.0 + 0.33 * KB + (base ? 3.5 : 0.0));
}

template <int NW>
int launch_stream(const scion_fp8* L, const StreamPlan& plan, StreamParams& p, const uint8_t* x, int T, cudaStream_t s) {
  p.w[0] = L->w[0], p.w[1] = L->w[NW - 1];
  p.bn = plan.bn;
  const int splits = plan.splits;
  p.range = p.KB / splits, p.longer = p.KB % splits, p.inverse = 65536 / splits + 1;
  p.sfb_cols = p.bn > 128 ? 8 : 4;
  p.sf_col = NW * p.bn;
  p.tmem_cols = int(tmem_cols_pow2(p.sf_col + kSfSlots * (4 * NW + p.sfb_cols)));
  // Shared memory in step with tensor memory: CTAs that fit an SM together by the one then fit by
  // the other too, so no CTA of a cluster can wait for tensor memory held by a CTA that waits for
  // its own cluster.
  const uint32_t share = 228 * 1024 / 512 * p.tmem_cols - 1024;
  const uint32_t stage = kStageBlocks<NW> * (NW * 16384 + p.bn * 128);
  const uint32_t fixed = 2048 + (splits > 1 ? (p.bn + splits - 1) / splits * splits * NW * 512 : 0);
  // Two CTAs per SM where there are more than SMs, unless that leaves one stage to each (tiles of 96 to 208
  // tokens of a plain layer), whose copies would wait for the MMAs and they for them: 20480 x 8192, 96 tokens
  // 53.2 us, 46.7 with one CTA and three stages (the pair kernel 50.9); 128 tokens 54.7, 49.3 (51.6).
  const bool crowded = int64_t(plan.n_tiles) * plan.t_tiles * splits > L->sms;
  const uint32_t half = std::max<uint32_t>(share, 113 * 1024);
  const uint32_t budget = crowded && half >= fixed + 2 * stage ? half : kSmem;
  const int range = (p.KB + splits - 1) / splits;  // K blocks of a CTA, at most
  p.stages = std::max(1, std::min({kMaxStages, int((budget - fixed) / stage), (range + kStageBlocks<NW> - 1) / kStageBlocks<NW>}));
  const uint32_t smem = std::max({fixed + p.stages * stage, uint32_t(2048 + NW * p.bn * 512), share});
  if (smem > kSmem) return SCION_EINVAL;
  int st = make_tmap_codes(&p.x, x, T, L->desc.k, p.bn);
  if (st != SCION_OK) return st;
  const bool loose = p.sf_align == 1 || (NW == 1 && !p.vec);
  const auto kernel = splits > 1 ? loose ? fp8_stream_kernel<NW, true, true> : fp8_stream_kernel<NW, true, false>
                      : loose    ? fp8_stream_kernel<NW, false, true>
                                 : fp8_stream_kernel<NW, false, false>;
  return status(launch_pdl_cluster(kernel,
                                   dim3(splits, plan.n_tiles, plan.t_tiles), dim3(kStreamThreads), dim3(splits, 1, 1), smem, s, p));
}

// Few tokens run on mma.sync (k_fp8_rows.cu) as long as the weights are few: it starts sooner, but reads the
// tokens again for every 16 weight rows, its products are slower (about 50 cycles per step of 8 tokens x 16
// rows x 32 columns), and a second round of its CTAs costs more than the streaming kernel's one.  The bounds
// follow rounds of CTAs (16 weight rows on each of the SMs), from both kernels measured at K = 128 to 8192, n =
// 256 to 65536, 1 to 32 tokens: the kernel taken was at most 11% behind the other.  n x k, us, rows against
// stream.  8 tokens: 4096 x 4096 3.9, 5.8; 16384 x 512 3.6, 3.9; 16384 x 8192 27.5, 28.0; 32768 x 512 6.0, 4.4;
// 65536 x 512 10.6, 12.6 (two rounds of the streaming kernel).  16 tokens: 4096 x 4096 5.3, 5.9; 8192 x 1024
// 4.0, 4.5; 16384 x 512 6.0, 3.9; 8192 x 4096 10.1, 7.7.  32 tokens: 4096 x 1024 3.8, 4.6; 2048 x 2048 3.7,
// 4.8; 8192 x 512 5.1, 3.7; 2048 x 4096 5.7, 5.4.  Gated to 8 bits, 8 tokens: 4096 x 2048 5.1, 5.8; 4096 x 4096
// 6.6, 7.3; 4736 x 1024 5.4, 4.8; 1024 x 8192 7.1, 6.8; to bf16: 8192 x 2048 6.4, 6.9; 8192 x 2560 8.7, 8.0.
// Gated, 16 tokens, to 8 bits: 1920 x 2560 5.2, 5.6; 1024 x 3584 6.0, 5.6; 2368 x 512 4.2, 4.3; 2048 x 1024
// 4.8, 4.7; to bf16: 2368 x 2560 4.4, 5.6; 256 x 3584 5.1, 4.9; 4736 x 1024 4.6, 4.9; 4096 x 2048 6.5, 5.8.
bool use_rows(const Call& c) {
  const int64_t round = 16 * int64_t(c.sms), weights = int64_t(c.N) * c.K;
  if (!c.w[1]) {
    if (c.T <= 8) return c.N <= 8 * round || c.N > 16 * round;
    if (c.T <= 16) return c.N <= 4 * round && weights <= 20 << 20;
    return c.T <= 32 && c.N <= 2 * round && c.K <= 2048 && weights <= 5 << 20;
  }
  if (c.T <= 8) {
    if (c.codes) return c.N <= 4096 && c.K <= 4096;  // (clusters of 8 CTAs, two to an SM)
    return c.N <= 2 * round ? c.K <= 4096 : c.N <= 4 * round && c.K <= 2048;
  }
  if (c.T > 16) return false;
  if (c.codes) return c.N <= 128 * c.clusters8 ? c.K <= 2560 : c.N <= round && c.K <= 768;
  return c.N <= round ? c.K <= 3584 : c.N <= 2 * round && c.K <= 1024;
}

template <int EPI>
int launch_pair(const scion_fp8* L, const StreamParams& q, const uint8_t* x, int T, cudaStream_t s) {
  constexpr bool kGated = EPI == kPairGatedBf16 || EPI == kPairGatedCodes;
  PairParams p{};
  p.w[0] = L->w[0], p.w[1] = L->w[kGated ? 1 : 0];
  p.sw[0] = q.sw[0], p.sw[1] = q.sw[1], p.sx = q.sx, p.base = q.base, p.out = q.out, p.codes = q.codes;
  p.scales = q.scales, p.err = q.err, p.T = T, p.N = q.N, p.KB = q.KB, p.sf_align = q.sf_align;
  p.m_tiles = (T + 255) / 256, p.n_tiles = kGated ? (p.N + 127) / 128 : (p.N + 255) / 256;
  p.out_bf16 = q.out_bf16;
  int st = make_tmap_codes(&p.x, x, T, L->desc.k, 128);
  if (st != SCION_OK) return st;
  const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles;
  const int pairs = int(std::min<int64_t>(tiles, L->sms / 2));
  return status(launch_pdl_cluster(fp8_pair_kernel<EPI>, dim3(2 * pairs), dim3(kPairThreads), dim3(2, 1, 1), kSmem, s, p));
}

Call call(const scion_fp8* L, const uint8_t* x, const uint8_t* sx, int T) {
  Call c{};
  c.x = x, c.sx = sx;
  c.w[0] = L->desc.w_codes, c.sw[0] = L->desc.w_scales, c.w[1] = L->desc.up_codes, c.sw[1] = L->desc.up_scales;
  c.T = T, c.N = L->desc.n, c.K = L->desc.k, c.KB = (c.K + 127) / 128, c.sms = L->sms, c.clusters8 = L->clusters[8];
  return c;
}

StreamParams params(const scion_fp8* L, const uint8_t* sx, int T) {
  StreamParams p{};
  p.sx = sx, p.sw[0] = L->desc.w_scales, p.sw[1] = L->desc.up_scales;
  p.T = T, p.N = L->desc.n, p.KB = (L->desc.k + 127) / 128, p.err = L->err;
  p.sf_align = 1;
  for (int a : {4, 16})
    if (p.KB % a == 0 && !misaligned(sx, a) && !misaligned(p.sw[0], a) && !misaligned(p.sw[1], a)) p.sf_align = a;
  return p;
}

}  // namespace
}  // namespace scion

extern "C" int scion_fp8_create(const scion_fp8_desc* D, void* stream, scion_fp8** out) {
  if (!out) return SCION_EINVAL;
  *out = nullptr;
  if (!D || D->n < 1 || D->n > (1 << 20) || D->k < 16 || D->k % 16 || D->k > 65536) return SCION_EINVAL;
  if (!D->w_codes || !D->w_scales || scion::fp8::misaligned(D->w_codes, 16)) return SCION_EINVAL;
  if (!D->up_codes != !D->up_scales) return SCION_EINVAL;
  if (D->up_codes && (D->n % 16 || scion::fp8::misaligned(D->up_codes, 16))) return SCION_EINVAL;
  scion_fp8* L = new (std::nothrow) scion_fp8;
  if (!L) return SCION_ENOMEM;
  L->desc = *D;
  L->err = nullptr;
  L->device_bytes = sizeof(int);
  int st = scion::make_tmap_codes(&L->w[0], D->w_codes, D->n, D->k, 128);
  if (st == SCION_OK && D->up_codes) st = scion::make_tmap_codes(&L->w[1], D->up_codes, D->n, D->k, 128);
  if (st != SCION_OK) {
    delete L;
    return st;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L->sms, cudaDevAttrMultiProcessorCount, dev);
  // (a function attribute of the current device)
  for (const auto f : {scion::fp8_stream_kernel<1, false, false>, scion::fp8_stream_kernel<1, false, true>,
                       scion::fp8_stream_kernel<1, true, false>, scion::fp8_stream_kernel<1, true, true>,
                       scion::fp8_stream_kernel<2, false, false>, scion::fp8_stream_kernel<2, false, true>,
                       scion::fp8_stream_kernel<2, true, false>, scion::fp8_stream_kernel<2, true, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, scion::kSmem);
  for (const auto f : {scion::fp8_pair_kernel<scion::kPairBf16>, scion::fp8_pair_kernel<scion::kPairF32>,
                       scion::fp8_pair_kernel<scion::kPairBase>, scion::fp8_pair_kernel<scion::kPairLoose>,
                       scion::fp8_pair_kernel<scion::kPairGatedBf16>, scion::fp8_pair_kernel<scion::kPairGatedCodes>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, scion::kSmem);
  for (int n = 1; n <= 8 && e == cudaSuccess; ++n) e = scion::max_clusters(n, &L->clusters[n]);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&L->err), sizeof(int));
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
  if (!L || L->desc.up_codes || T < 0 || T > scion::kMaxTokens || (out_type != SCION_F32 && out_type != SCION_BF16)) return SCION_EINVAL;
  if (T == 0) return SCION_OK;
  if (!x_codes || !x_scales || !out || scion::fp8::misaligned(x_codes, 16)) return SCION_EINVAL;
  if (scion::fp8::misaligned(base, 4) || scion::fp8::misaligned(out, out_type == SCION_F32 ? 4 : 2)) return SCION_EINVAL;
  if (out_type == SCION_BF16 && static_cast<const void*>(base) == out && base) return SCION_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  scion::count_launch();
  scion::fp8::Call c = scion::call(L, x_codes, x_scales, T);
  c.base = base, c.out = out, c.out_bf16 = out_type == SCION_BF16;
  if (scion::use_rows(c)) return scion::status(scion::fp8::launch_rows(c, s));
  scion::StreamParams p = scion::params(L, x_scales, T);
  p.base = base, p.out = out, p.out_bf16 = out_type == SCION_BF16;
  p.vec = p.N % 4 == 0 && !scion::fp8::misaligned(base, 16) && !scion::fp8::misaligned(out, 16);
  const bool rows16 = int64_t(p.N) * (p.out_bf16 ? 2 : 4) % 16 == 0 && p.vec;
  const scion::StreamPlan plan = scion::plan_stream(L, 1, T, p.N, p.KB);
  if (scion::pair_us(L, 1, T, p.N, p.KB, base) < plan.us)
    return !rows16      ? scion::launch_pair<scion::kPairLoose>(L, p, x_codes, T, s)
           : base       ? scion::launch_pair<scion::kPairBase>(L, p, x_codes, T, s)
           : p.out_bf16 ? scion::launch_pair<scion::kPairBf16>(L, p, x_codes, T, s)
                        : scion::launch_pair<scion::kPairF32>(L, p, x_codes, T, s);
  return scion::launch_stream<1>(L, plan, p, x_codes, T, s);
}

extern "C" int scion_fp8_gated_forward(const uint8_t* x_codes, const uint8_t* x_scales, int T, const scion_fp8* L,
                                       void* h_bf16, uint8_t* h_codes, uint8_t* h_scales, void* stream) {
  if (!L || !L->desc.up_codes || T < 0 || T > scion::kMaxTokens) return SCION_EINVAL;
  if (T == 0) return SCION_OK;  // (empty tensors have null addresses)
  if (!h_codes != !h_scales || !h_codes == !h_bf16) return SCION_EINVAL;
  if (!x_codes || !x_scales || scion::fp8::misaligned(x_codes, 16) || scion::fp8::misaligned(h_bf16, 16) ||
      scion::fp8::misaligned(h_codes, 16))
    return SCION_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  scion::count_launch();
  scion::fp8::Call c = scion::call(L, x_codes, x_scales, T);
  c.out = h_bf16, c.codes = h_codes, c.scales = h_scales;
  if (scion::use_rows(c)) return scion::status(scion::fp8::launch_rows(c, s));
  scion::StreamParams p = scion::params(L, x_scales, T);
  p.out = h_bf16, p.codes = h_codes, p.scales = h_scales;
  const scion::StreamPlan plan = scion::plan_stream(L, 2, T, p.N, p.KB);
  if (scion::pair_us(L, 2, T, p.N, p.KB, false) < plan.us)
    return h_codes ? scion::launch_pair<scion::kPairGatedCodes>(L, p, x_codes, T, s)
                   : scion::launch_pair<scion::kPairGatedBf16>(L, p, x_codes, T, s);
  return scion::launch_stream<2>(L, plan, p, x_codes, T, s);
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
