// Weight-only linear for one to a few tokens: int4 weights with a scale per group of
// input channels (weight-only form of the framework's §4.2 / Figure 2 weights, with the
// activations left in bf16).
//   pack_int4_group  offline: W' = W * c -> codes and one bf16 scale per group
//   gemv_w4g         y = x' * W'^T for 1 to 16 tokens, x' = x * cinv
//
// Packed layout: a run of 128 input channels of one output channel is 64 consecutive
// bytes, sixteen 32-bit words.  Word 4t + j (t, j = 0..3) holds channels 32j + 8t .. + 7
// of the run; of those eight, channel 2i is nibble i and channel 2i + 1 nibble i + 4.
// Lane t of a quad therefore gets, with ONE 16-byte load, eight channels of each of the
// run's four 32-channel groups (word j = group j), so the channels that the quad feeds
// into one matrix instruction always share a scale; and (w >> 4i) & 0x000F000F is a
// pair of neighbouring channels, which the instruction wants in one register next to a
// pair of x as it lies in memory.
#pragma once
#include <cuda_bf16.h>

#include "wq_internal.h"
#include "wq_ptx.cuh"
#include "wq_quant.cuh"

namespace wq {
namespace {

// ------------------------------------------------------------ packing (offline)

// Codes of eight channels as one word of the packed layout.
__device__ __forceinline__ uint32_t group_word(const uint32_t (&c)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w |= (c[2 * i] & 0xFu) << (4 * i);
    w |= (c[2 * i + 1] & 0xFu) << (4 * i + 16);
  }
  return w;
}

// Thread = eight channels of one output channel; the G/8 threads of a group are
// neighbours in a warp and share the maximum by shuffles.  W is read and the codes are
// written once.  The scale is rounded to bf16 (2 bytes beside 16 to 64 bytes of codes)
// BEFORE the codes are decided, so the codes belong to the scale that is stored; a
// scale rounded down by at most 2^-9 sends the maximum to 7.03, which clamps to 7.
template <int G>
__global__ void __launch_bounds__(256) pack_int4_group_kernel(
    const uint16_t* __restrict__ W, const float* __restrict__ c, int N, int K,
    uint32_t* __restrict__ qw, uint16_t* __restrict__ s_g) {
  const int chunks = K / 8;  // a multiple of 16
  const size_t total = static_cast<size_t>(N) * chunks;
  const size_t idx = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const bool valid = idx < total;  // threads past the end still take part in the shuffles
  const int n = static_cast<int>(idx / chunks), ch = static_cast<int>(idx % chunks);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (valid) raw = reinterpret_cast<const uint4*>(W)[idx];
  float ci[8], v[8];
  load_cinv8_global(c, ch, ci);
  scale8(raw, ci, v);
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
  for (int o = G / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
  const float s = __bfloat162float(sb);
  const float r = __frcp_rn(s);
  uint32_t q[8];
  if (s > 0.0f && r <= 3.0e38f) {
    quantize8_recip<7>(v, s, r, q);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = static_cast<uint32_t>(quantize<7>(v[e], s));
  }
  if (!valid) return;
  const int at = ch & 15;  // 4 j + t
  qw[idx - at + 4 * (at & 3) + (at >> 2)] = group_word(q);
  if ((ch & (G / 8 - 1)) == 0)
    s_g[static_cast<size_t>(ch / (G / 8)) * N + n] = __bfloat16_as_ushort(sb);
}

// ------------------------------------------------------------ matrix-vector products

// D (16 x 8, fp32) += A (16 x 16, bf16) x B (16 x 8, bf16).
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibble pair i of a packed word as two bf16 codes, exactly: code + 8 placed under the
// exponent of 128 (bf16 holds integers up to 256), then 136 taken off.
template <int I>
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w) {
  const uint32_t u = ((w >> (4 * I)) & 0x000F000Fu) ^ 0x43084308u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                   __floats2bfloat162_rn(136.0f, 136.0f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// x' = x * cinv in two bf16 parts, hi + lo (16 bits of it: an error of at most 2^-17).
__device__ __forceinline__ void fold_pair(uint32_t x, float c0, float c1, uint32_t& hi,
                                          uint32_t& lo) {
  const float a = __fmul_rn(bf16lo(x), c0), b = __fmul_rn(bf16hi(x), c1);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const __nv_bfloat162 l =
      __floats2bfloat162_rn(__fsub_rn(a, __low2float(h)), __fsub_rn(b, __high2float(h)));
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

constexpr int kGemvWarps = 8;

// CTA = 16 MT output channels; its warps take the runs of 128 input channels in turn, so
// that the warps read neighbouring 64-byte pieces of each row at the same time.  Each
// lane keeps PF runs of weights in flight in registers (16 bytes per row and run).  The
// weights are the instruction's A operand (16 output channels x 16 input channels), the
// tokens its 8 columns; sums within a group and across groups are fp32, and a group's
// scale multiplies its fp32 sum.  The warps' sums meet in shared memory, in warp order.
// FOLD: x' = x * cinv enters as two bf16 parts, two instructions instead of one.
template <int G, int MT, int NT, int PF, bool FOLD>
__global__ void __launch_bounds__(32 * kGemvWarps) gemv_w4g_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ cinv,
    const uint8_t* __restrict__ qw, const uint16_t* __restrict__ s_g,
    const float* __restrict__ bias, uint16_t* __restrict__ y, int M, int K, int N) {
  constexpr int R = 16 * MT, C = 8 * NT;
  __shared__ float red[kGemvWarps][C][R + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * R;
  const int runs = K / 128;
  const size_t row_bytes = static_cast<size_t>(K) / 2;

  // rows past N repeat the last one: read in bounds, never written
  const uint8_t* wp[MT][2];
  int row[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row[mt][h] = min(n0 + 16 * mt + 8 * h + g, N - 1);
      wp[mt][h] = qw + row[mt][h] * row_bytes + 16 * t;
    }
  griddep_wait();
  griddep_launch_dependents();

  uint4 w[PF][MT][2];
  uint16_t s[PF][MT][2];
  auto fetch = [&](int p, int run) {
    const size_t gi = (static_cast<size_t>(run) * 128 + 32 * t) / G;  // lane t: the group of word t
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[p][mt][h] = __ldcs(reinterpret_cast<const uint4*>(wp[mt][h] + static_cast<size_t>(run) * 64));
        s[p][mt][h] = __ldg(s_g + gi * N + row[mt][h]);
      }
  };
#pragma unroll
  for (int p = 0; p < PF; ++p) {
    const int run = warp + p * kGemvWarps;
    if (run < runs) fetch(p, run);
  }

  float acc[MT][NT][4] = {};
  for (int base = warp; base < runs; base += PF * kGemvWarps) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      const int run = base + p * kGemvWarps;
      if (run < runs) {
        float sum[MT][NT][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = run * 128 + 32 * j + 8 * t;
          uint32_t b[NT][4], bl[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int m = 8 * nt + g;
            uint4 xv = make_uint4(0, 0, 0, 0);
            if (m < M) xv = __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(m) * K + k));
            b[nt][0] = xv.x; b[nt][1] = xv.y; b[nt][2] = xv.z; b[nt][3] = xv.w;
          }
          if constexpr (FOLD) {
            float ci[8];
            load_cinv8_global(cinv, k / 8, ci);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                fold_pair(b[nt][e], ci[2 * e], ci[2 * e + 1], b[nt][e], bl[nt][e]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t wa = word_of(w[p][mt][0], j), wb = word_of(w[p][mt][1], j);
            const uint32_t a0[4] = {codes_bf16x2<0>(wa), codes_bf16x2<0>(wb),
                                    codes_bf16x2<1>(wa), codes_bf16x2<1>(wb)};
            const uint32_t a1[4] = {codes_bf16x2<2>(wa), codes_bf16x2<2>(wb),
                                    codes_bf16x2<3>(wa), codes_bf16x2<3>(wb)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16(sum[mt][nt], a0, b[nt][0], b[nt][1]);
              mma_bf16(sum[mt][nt], a1, b[nt][2], b[nt][3]);
              if constexpr (FOLD) {
                mma_bf16(sum[mt][nt], a0, bl[nt][0], bl[nt][1]);
                mma_bf16(sum[mt][nt], a1, bl[nt][2], bl[nt][3]);
              }
            }
          }
          if ((j + 1) % (G / 32) == 0) {  // the group ends: scale its sum
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float sc[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = static_cast<uint32_t>(s[p][mt][h]) << 16;
                sc[h] = __uint_as_float(
                    G == 128 ? v : __shfl_sync(0xFFFFFFFFu, v, (lane & 28) | j));
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  acc[mt][nt][e] = fmaf(sum[mt][nt][e], sc[e >> 1], acc[mt][nt][e]);
                  sum[mt][nt][e] = 0.0f;
                }
            }
          }
        }
        const int next = run + PF * kGemvWarps;
        if (next < runs) fetch(p, next);
      }
    }
  }

#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[warp][8 * nt + 2 * t + (e & 1)][16 * mt + 8 * (e >> 1) + g] = acc[mt][nt][e];
  __syncthreads();
  for (int i = threadIdx.x; i < R * M; i += 32 * kGemvWarps) {
    const int r = i % R, m = i / R, n = n0 + r;
    if (n >= N) continue;
    float v = bias ? bias[n] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < kGemvWarps; ++q) sum += red[q][m][r];
    y[static_cast<size_t>(m) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(sum + v));
  }
}

template <int G, int MT, int NT, int PF, bool FOLD>
cudaError_t run_gemv(const uint16_t* x, const float* cinv, const uint8_t* qw, const uint16_t* s_g,
                     const float* bias, uint16_t* y, int M, int K, int N, cudaStream_t st) {
  const int grid = (N + 16 * MT - 1) / (16 * MT);
  return launch_pdl(gemv_w4g_kernel<G, MT, NT, PF, FOLD>, grid, 32 * kGemvWarps, 0, st, 1, x, cinv,
                    qw, s_g, bias, y, M, K, N);
}

template <int G, bool FOLD>
cudaError_t dispatch_gemv(const uint16_t* x, const float* cinv, const uint8_t* qw,
                          const uint16_t* s_g, const float* bias, uint16_t* y, int M, int K, int N,
                          cudaStream_t st) {
  if (M <= 8) return run_gemv<G, 1, 1, 4, FOLD>(x, cinv, qw, s_g, bias, y, M, K, N, st);
  return run_gemv<G, 1, 2, 4, FOLD>(x, cinv, qw, s_g, bias, y, M, K, N, st);
}

}  // namespace

cudaError_t launch_pack_int4_group(const uint16_t* W, const float* c, int N, int K, int group,
                                   uint8_t* qw, uint16_t* s_g, cudaStream_t st) {
  const int grid = static_cast<int>((static_cast<size_t>(N) * (K / 8) + 255) / 256);
  uint32_t* q = reinterpret_cast<uint32_t*>(qw);
  if (group == 32)
    return launch_pdl(pack_int4_group_kernel<32>, grid, 256, 0, st, 1, W, c, N, K, q, s_g);
  if (group == 64)
    return launch_pdl(pack_int4_group_kernel<64>, grid, 256, 0, st, 1, W, c, N, K, q, s_g);
  return launch_pdl(pack_int4_group_kernel<128>, grid, 256, 0, st, 1, W, c, N, K, q, s_g);
}

cudaError_t launch_gemv_w4g(const uint16_t* x, const float* cinv, const uint8_t* qw,
                            const uint16_t* s_g, int group, const float* bias, uint16_t* y, int M,
                            int K, int N, cudaStream_t st) {
#define WQ_GEMV(G_)                                                                       \
  return cinv ? dispatch_gemv<G_, true>(x, cinv, qw, s_g, bias, y, M, K, N, st)           \
              : dispatch_gemv<G_, false>(x, cinv, qw, s_g, bias, y, M, K, N, st)
  if (group == 32) WQ_GEMV(32);
  if (group == 64) WQ_GEMV(64);
  WQ_GEMV(128);
#undef WQ_GEMV
}

}  // namespace wq
