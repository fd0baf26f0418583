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
#include <cuda_fp16.h>

#include "wq_internal.h"
#include "wq_ptx.cuh"
#include "wq_quant.cuh"

namespace wq {
namespace {

// Eight codes rint_half_even(fl(v / s)) for scales of plain_scale(), where no quotient
// rounds beyond the code range, so that nothing has to be clamped; r = 1 / s, correctly
// rounded.  The quotient without a division or a branch, two values at a time: t = v * r,
// improved once with its remainder v - t s, is within one last place; then, by Markstein's
// theorem (Computation of elementary functions on the IBM RISC System/6000 processor, 1990),
// adding its remainder, which is exact, times r gives the correctly rounded fl(v / s).  The low
// bits of a result are the code.  (quantize8_recip's margin around half-integers takes one
// operation less, but sends an eighth of the warps the long way: packing 16384 x 4096 took
// 62.9 us so, 49.3 us this way.)
__device__ __forceinline__ void quantize8_pairs(const float2 (&v)[4], float s, float r,
                                                uint32_t (&c)[8]) {
  const float2 rr = make_float2(r, r), minus_s = make_float2(-s, -s);
  const float2 magic = make_float2(kRoundMagic, kRoundMagic);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 t = __fmul2_rn(v[e], rr);
    t = __ffma2_rn(__ffma2_rn(t, minus_s, v[e]), rr, t);
    t = __ffma2_rn(__ffma2_rn(t, minus_s, v[e]), rr, t);
    const float2 u = __fadd2_rn(t, magic);
    c[2 * e] = __float_as_uint(u.x);
    c[2 * e + 1] = __float_as_uint(u.y);
  }
}

// Scales for which quantize8_pairs holds: 1 / s is normal, a remainder of a quotient that is
// not rounded to 0 is exact, and the scale, a maximum over QMAX, is within 2^-8 of that.
__device__ __forceinline__ bool plain_scale(float s) { return s >= 0x1p-100f && s <= 0x1p120f; }

// The larger one, or NaN if one is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// ------------------------------------------------------------ packing (offline)

// Codes of eight channels (in the low nibbles) as one word of the packed layout.
__device__ __forceinline__ uint32_t group_word(const uint32_t (&c)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (__byte_perm(c[2 * i], c[2 * i + 1], 0x5410) << (4 * i)) & (0x000F000Fu << (4 * i));
  return w;
}

// CTA = 512 input channels of every so many 16 output channels (a tile), the next tile's loads
// in flight while one is packed; four threads to a run of 128 channels.
// Thread t of a run takes channels 32j + 8t .. + 7, j = 0..3 (a quad's loads are 64
// consecutive bytes, all four in flight): they are the words that lie next to each other in
// the packed run, one 16-byte store.  A group is whole in the quad: its maximum is taken
// within the threads, then by two shuffles.  W is read and the codes are written once; the
// scales go through shared memory, so that sixteen rows' leave as one 32-byte piece.  The
// scale is rounded to bf16 (2 bytes beside 16 to 64 bytes of codes) BEFORE the codes are
// decided, so the codes belong to the scale that is stored; a scale rounded down by at most
// 2^-9 sends the maximum to 7.02, which is 7.
// Persistent CTAs that load the next tile while this one is made: the issue of instructions
// (56 % of cycles) and the memory bound it together.  16384 x 4096, groups of 64, with c:
// 36.0 us, 4.7 TB/s read and written (48.0 us with a CTA per tile, nothing loaded ahead);
// 2048 x 2048: 3.6 us.
template <int G, bool SCALED>
__global__ void __launch_bounds__(256, 2) pack_int4_group_kernel(
    const uint16_t* __restrict__ W, const float* __restrict__ c, int N, int K, int strips,
    uint4* __restrict__ qw, uint16_t* __restrict__ s_g) {
  constexpr int GW = G / 32;  // words of a thread in a group
  __shared__ uint16_t scales[2][512 / G][16];
  const int row = threadIdx.x >> 4, t = threadIdx.x & 3;
  const int run0 = blockIdx.x % strips * 4, run = run0 + ((threadIdx.x >> 2) & 3);
  const int tiles = (N + 15) / 16, step = gridDim.x / strips;
  const bool valid = run < K / 128;  // the same for a quad
  const int groups = min(512, K - run0 * 128) / G;
  griddep_wait();
  griddep_launch_dependents();
  uint4 raw[4] = {};
  auto load = [&](int tile) {
    if (!valid || tile >= tiles) return;
    const int n = min(tile * 16 + row, N - 1);  // rows past N repeat the last one, not written
#pragma unroll
    for (int j = 0; j < 4; ++j)
      raw[j] = __ldcs(reinterpret_cast<const uint4*>(W + static_cast<size_t>(n) * K) + run * 16 + 4 * j + t);
  };
  int tile = blockIdx.x / strips;
  load(tile);
  float2 cc[SCALED ? 4 : 1][4];
  if constexpr (SCALED) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4* cp = reinterpret_cast<const float4*>(c) + 2 * (run * 16 + 4 * j + t);
      float4 c0 = make_float4(0, 0, 0, 0), c1 = c0;
      if (valid) {
        c0 = __ldg(cp);
        c1 = __ldg(cp + 1);
      }
      cc[j][0] = make_float2(c0.x, c0.y); cc[j][1] = make_float2(c0.z, c0.w);
      cc[j][2] = make_float2(c1.x, c1.y); cc[j][3] = make_float2(c1.z, c1.w);
    }
  }
  for (int turn = 0; tile < tiles; tile += step, turn ^= 1) {
    const int n0 = tile * 16;
    const uint4 now[4] = {raw[0], raw[1], raw[2], raw[3]};
    load(tile + step);
    uint32_t word[4];
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += GW) {
      float2 v[GW][4];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < GW; ++j) {
        const uint32_t w[4] = {now[j0 + j].x, now[j0 + j].y, now[j0 + j].z, now[j0 + j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = make_float2(bf16lo(w[e]), bf16hi(w[e]));
        if constexpr (SCALED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = __fmul2_rn(v[j][e], cc[j0 + j][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = max_or_nan(amax, max_or_nan(fabsf(v[j][e].x), fabsf(v[j][e].y)));
      }
      amax = max_or_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = max_or_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
      const float s = __bfloat162float(sb);
      const bool plain = plain_scale(s);
      const float r = plain ? __frcp_rn(s) : 0.0f;
#pragma unroll
      for (int j = 0; j < GW; ++j) {
        uint32_t q[8];
        if (plain) {
          quantize8_pairs(v[j], s, r, q);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            q[2 * e] = static_cast<uint32_t>(quantize_exact<7>(v[j][e].x, s));
            q[2 * e + 1] = static_cast<uint32_t>(quantize_exact<7>(v[j][e].y, s));
          }
        }
        word[j0 + j] = group_word(q);
      }
      if (t == 0) scales[turn][(run - run0) * (128 / G) + j0 / GW][row] = __bfloat16_as_ushort(sb);
    }
    if (valid && n0 + row < N)
      qw[static_cast<size_t>(n0 + row) * (K / 32) + run * 4 + t] =
          make_uint4(word[0], word[1], word[2], word[3]);
    __syncthreads();  // (two buffers: the next tile's barrier frees this one's)
    for (int i = threadIdx.x; i < groups * 16; i += 256)
      if (n0 + (i & 15) < N)
        s_g[(static_cast<size_t>(run0) * (128 / G) + (i >> 4)) * N + n0 + (i & 15)] =
            scales[turn][i >> 4][i & 15];
  }
}

// ------------------------------------------------------------ matrix-vector products

// D (16 x 8, int32) = (first ? 0 : D) + A (16 x 32, int8) x B (32 x 8, int8).
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1, bool first) {
  if (first)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D (16 x 8, fp32) += A (16 x 16, f16) x B (16 x 8, f16).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (w & mask) ^ magic, one three-input operation.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t u;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(u) : "r"(w), "r"(mask), "r"(magic));
  return u;
}

// The nibble pairs 0 (I = 0) or 1 (I = 1) of w as two f16 codes, exactly: code + 8 placed
// under the exponent of 1024 (f16 holds integers up to 2048), at bit 0 or bit 4, then 1032
// taken off, or a sixteenth taken and 72 taken off.
template <int I>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
  const uint32_t u = I == 0 ? and_xor(w, 0x000F000Fu, 0x64086408u) : and_xor(w, 0x00F000F0u, 0x64806480u);
  const __half2 h = *reinterpret_cast<const __half2*>(&u);
  const __half2 v = I == 0 ? __hsub2(h, __floats2half2_rn(1032.0f, 1032.0f))
                           : __hfma2(h, __floats2half2_rn(0.0625f, 0.0625f),
                                     __floats2half2_rn(-72.0f, -72.0f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One byte of each of four words -> one word.
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                                 uint32_t byte) {
  const uint32_t sel = byte | (byte + 4) << 4;
  return __byte_perm(__byte_perm(a, b, sel), __byte_perm(c, d, sel), 0x5410);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// The products' sums are held at 2^-12 of their value until bias and rounding: a group's sum of
// x' * code may exceed the largest |x'| 2^10 times, which must not leave fp32's range before
// the weights' scale brings it back.  (The other end has room: bf16's smallest step is 2^-133.)
constexpr float kSumDown = 0x1p-12f, kSumUp = 0x1p12f;

constexpr int kGemvWarps = 16;
constexpr int kGemvMaxSplit = 8;            // CTAs that share K (a portable cluster)
constexpr int kGemvMaxTiles = 512;          // row tiles of a cluster
constexpr int kGemvMaxSmem = 224 * 1024;    // dynamic, beside 2 KB of tables

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// 3-D tiled load global -> shared, completion counted on an mbarrier.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* desc, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

struct GemvArgs {
  const uint16_t* x;     // bf16 [M][K]
  const float* cinv;     // [K] or null
  const uint16_t* s_g;   // bf16 [K / G][N]
  const float* bias;     // [N] or null
  uint16_t* y;           // bf16 [M][N]
  int M, K, N;
  int S;                 // CTAs of a cluster, each with a share of K
  int share;             // runs of 128 channels in a share (the last may have fewer)
  int tiles;             // row tiles of a cluster (the last may have fewer)
};

// MT: 16-channel halves of a row tile; NT: groups of four tokens (1, digits; 2 or 4, f16);
// TINY: one or two tokens, whose lowest digits fill the columns that hi and mid leave free;
// TWO: tokens as two f16 parts, for x * cinv (NT > 1).
template <int MT, int NT, bool TINY, bool TWO>
struct GemvCfg {
  static constexpr int WR = 16 * MT;               // output channels of a row tile
  static constexpr int RPS = MT == 1 ? 2 : 1;      // runs per stage (2 KB tiles)
  static constexpr int STAGES = NT == 4 || TWO ? 2 : 3;
  static constexpr int TILE = RPS * WR * 64;
  static constexpr int RING = kGemvWarps * STAGES * TILE;
  static constexpr bool HALF = NT > 1;             // tokens as f16 instead of digits
  static constexpr int PARTS = TWO ? 2 : 1;
  static constexpr int COLS = HALF ? NT * PARTS : TINY ? 1 : 2;  // KB of staged tokens a run
  static constexpr int TOKENS = TINY ? 2 : 4 * NT;
  static constexpr int SEG = TOKENS * WR;             // floats of a segment's sums
  static constexpr int run_bytes(int group) { return COLS * 1024 + 128 / group * TOKENS * 4; }
  static constexpr int smem(int share, int group, int tiles) {
    return RING + share * run_bytes(group) + (tiles + kGemvWarps - 1) * SEG * 4 + 128;
  }
};

// Weight streaming is the bound, so copies in flight and few instructions per weight are
// what counts.  One CTA per SM; a cluster of S CTAs makes `tiles` row tiles of 16 MT output
// channels, each CTA from its share of K.  The CTA's work, row tile by row tile, is one
// sequence of stages (a row tile x RPS runs of 128 input channels), of which each warp takes
// an equal piece: it has a ring of its own that bulk tensor copies keep full across row
// tiles, and waits for no other warp between its first and last stage.  What a warp sums
// for one row tile is a segment; segments meet in shared memory when all is done, in warp
// order, and the shares through the cluster's shared window, in rank order.
//
// The products run on the integer matrix instructions: a nibble moved to the high half of
// its byte is 16 * code, so eight codes cost one shift and two masks, where making them
// floating-point costs eleven instructions.  The tokens become 22-bit integers relative to
// the largest |x'| of their group (a power-of-two scale: a value is off by at most 2^-22 of
// that maximum, and bf16 values down to 2^-14 of it are exact), split into three signed
// bytes, hi 2^16 + mid 2^8 + lo.  hi and mid of a token are neighbouring columns of one
// column tile, so that a lane holds both sums; the lo fill another (TINY: columns 4 and 6).
// The sums of a group are exact in int32; they are joined, scaled and added over the groups
// in fp32.
//
// Staged layout: column tile c, run r: 1 KB [half][column][t][16 bytes], the 16 bytes of
// half h being the channels of words j = 2h, 2h + 1, in the order 0 4 1 5, 2 6 3 7 in
// which the masks leave the codes.
//
// More than four tokens (HALF) would need three to six column tiles and the joining of as
// many sums, which takes longer than the copies, as does splitting the tokens; they enter as
// f16 instead, over a power-of-two scale per group, against codes made f16 (exact; nine
// instructions for eight codes), in column tiles of eight tokens.  The 11 bits of f16 hold
// bf16 tokens exactly.  x * cinv has 24 bits: it enters as two f16 parts (TWO), the second
// what the first leaves over, which are multiplied by the same codes into the same sums;
// it is then off by at most 2^-22 of itself, or 2^-39 of its group's largest.  Staged run:
// [part] 2 KB per column tile, [word j][column][t][8 channels].
//
// Measured (calls in a graph, nothing in L2): 1 token, 2048 x 2048, groups of 128, 4.1 us;
// 1 token, 4096 -> 12288, 8.2 us, 3.2 TB/s, of which the stream is 4 to 5 us and the rest the
// start (the tokens, the scales, the first stage) and the joining; 8 tokens, 16384 -> 4096,
// groups of 64, cinv, 19.5 us, 1.8 TB/s (18.9 us with 11 bits of x * cinv); 16 tokens,
// 8192 -> 8191, groups of 32, 22.4 us, 1.7 TB/s, with cinv 32.7 us (24.3 us with 11 bits): there the staging of the tokens in every CTA,
// the conversions and the exchange count, not the copies.  Weights loaded straight into
// registers, without the rings, took 2.8 us for the first, whose warps have one stage or two,
// but 12.3 us for the second and 40 and 28 us for the last two.
template <int G, int MT, int NT, bool TINY, bool TWO>
__global__ void __launch_bounds__(32 * kGemvWarps, 1) gemv_w4g_kernel(
    const __grid_constant__ CUtensorMap tm_w, const GemvArgs a) {
  using Cfg = GemvCfg<MT, NT, TINY, TWO>;
  constexpr int WR = Cfg::WR, RPS = Cfg::RPS, STAGES = Cfg::STAGES, SEG = Cfg::SEG;
  constexpr int COLS = Cfg::COLS, TOKENS = Cfg::TOKENS;
  constexpr bool HALF = Cfg::HALF;
  constexpr int CT = NT / 2 > 0 ? NT / 2 : 1;  // HALF: column tiles
  constexpr int THREADS = 32 * kGemvWarps;
  extern __shared__ uint8_t gemv_smem[];
  __shared__ __align__(8) uint64_t full[kGemvWarps][STAGES];
  __shared__ short2 span[kGemvMaxTiles];  // first and last warp with a segment of a row tile
  uint8_t* ring_all = gemv_smem + ((128u - (smem_u32(gemv_smem) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int S = a.S, M = a.M, N = a.N;
  const int rank = blockIdx.x % S, tile0 = blockIdx.x / S * a.tiles;
  const int tiles = min(a.tiles, (N + WR - 1) / WR - tile0);
  const int all = a.K / 128;
  const int r_begin = min(rank * a.share, all), runs = min(a.share, all - r_begin);
  const int per_tile = (runs + RPS - 1) / RPS;                         // stages
  const int total = tiles * per_tile;
  const int u_begin = static_cast<int>(static_cast<long long>(total) * warp / kGemvWarps);
  const int u_end = static_cast<int>(static_cast<long long>(total) * (warp + 1) / kGemvWarps);
  const int count = u_end - u_begin;

  uint8_t* ring = ring_all + warp * STAGES * Cfg::TILE;
  uint8_t* xs = ring_all + Cfg::RING;                                    // [share][COLS] KB
  float* xscale = reinterpret_cast<float*>(xs + a.share * COLS * 1024);  // [group][TOKENS]
  float* segs = xscale + a.share * (128 / G) * TOKENS;

  if (lane == 0) {
    if (warp == 0) tma_prefetch_desc(&tm_w);
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
  }
  // Row tile q's segments are those of the warps whose pieces overlap [q, q + 1) per_tile
  for (int q = threadIdx.x; q < tiles && total > 0; q += THREADS)
    span[q] = make_short2(static_cast<short>((kGemvWarps * q * per_tile + kGemvWarps - 1) / total),
                          static_cast<short>((kGemvWarps * (q + 1) * per_tile - 1) / total));
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  // copies and scales run ahead of the sums: the row tile and the stage within it
  int c_tile = count > 0 ? u_begin / per_tile : 0, c_k = u_begin - c_tile * per_tile;
  int s_tile = c_tile, s_k = c_k;
  const int first_tile = c_tile, first_k = c_k;
  auto issue = [&](int i) {  // copies of my stage i
    if (lane == 0) {
      uint64_t* bar = &full[warp][i % STAGES];
      mbar_arrive_expect_tx(bar, Cfg::TILE);
      tma_load_3d(ring + i % STAGES * Cfg::TILE, &tm_w, bar, 0, (tile0 + c_tile) * WR,
                  r_begin + c_k * RPS);
    }
    if (++c_k == per_tile) {
      c_k = 0;
      ++c_tile;
    }
  };
  for (int i = 0; i < STAGES && i < count; ++i) issue(i);

  // The tokens of this share: a thread takes eight channels, XB times at a time (the loads
  // of a batch are in flight together, the first batch's while the scales are looked up).
  // Columns of tokens past M keep what shared memory held: nothing of them is written.
  constexpr int XB = 4;
  const int pieces = runs * 16, pieces_all = M * pieces;
  const uint32_t inv = pieces > 1 ? 0xFFFFFFFFu / pieces + 1 : 0;  // at / pieces, at < 2^18
  uint4 raw[XB];
  float4 ci[XB][2];
  auto fetch_x = [&](int base) {
#pragma unroll
    for (int e = 0; e < XB; ++e) {
      const int at = base + e * THREADS, m = __umulhi(at, inv), pc = at - m * pieces;
      raw[e] = make_uint4(0, 0, 0, 0);
      ci[e][0] = ci[e][1] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
      if (at >= pieces_all) continue;
      raw[e] = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(m) * a.K) +
                     r_begin * 16 + pc);
      if (a.cinv) {
        const float4* cp = reinterpret_cast<const float4*>(a.cinv) + 2 * (r_begin * 16 + pc);
        ci[e][0] = __ldg(cp);
        ci[e][1] = __ldg(cp + 1);
      }
    }
  };
  fetch_x(threadIdx.x);

  // scales two stages ahead in registers; lane t: the group of word t
  uint16_t sc[2][RPS][MT][2];
  const uint16_t* s_base = a.s_g + static_cast<size_t>(r_begin * 128 + 32 * t) / G * N;
  const size_t run_step = static_cast<size_t>(128 / G) * N;
  const uint16_t* sp[MT][2];
  auto scale_rows = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        sp[mt][h] = s_base + s_k * RPS * run_step +
                    min((tile0 + s_tile) * WR + 16 * mt + 8 * h + g, N - 1);
  };
  auto load_scales = [&](uint16_t (&to)[RPS][MT][2]) {
#pragma unroll
    for (int rr = 0; rr < RPS; ++rr)
      if (s_k * RPS + rr < runs)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            to[rr][mt][h] = __ldg(sp[mt][h]);
            sp[mt][h] += run_step;
          }
    if (++s_k == per_tile) {
      s_k = 0;
      ++s_tile;
      scale_rows();
    }
  };
  if (count > 0) {
    scale_rows();
    load_scales(sc[0]);
    if (count > 1) load_scales(sc[1]);
  }

  // the G / 8 threads of a group are neighbours and share its maximum by shuffles
  {
    for (int base0 = 0; base0 < pieces_all; base0 += XB * THREADS) {
      const int base = base0 + threadIdx.x;
#pragma unroll
      for (int e = 0; e < XB; ++e) {
        if (base0 + e * THREADS >= pieces_all) break;  // uniform
        const int at = base + e * THREADS, m = __umulhi(at, inv), pc = at - m * pieces;
        const bool valid = at < pieces_all;
        const float cf[8] = {ci[e][0].x, ci[e][0].y, ci[e][0].z, ci[e][0].w,
                             ci[e][1].x, ci[e][1].y, ci[e][1].z, ci[e][1].w};
        float v[8];
        scale8(raw[e], cf, v);
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) top = max_or_nan(top, fabsf(v[c]));
#pragma unroll
        for (int o = G / 16; o > 0; o >>= 1)
          top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // digits: 2^(21 - E) with 2^E <= top < 2^(E + 1); f16: 2^(14 - E); at most 2^127
        constexpr uint32_t BITS = HALF ? 14 : 21;
        const uint32_t ex = max(__float_as_uint(top) >> 23, BITS);
        const float up = __uint_as_float((254u + BITS - ex) << 23);
        if (!valid) continue;
        const int run = pc >> 4, j = (pc >> 2) & 3, tt = pc & 3;
        uint8_t* dst = xs + run * (COLS * 1024);
        if constexpr (HALF) {
          dst += (m >> 3) * 2048 + j * 512 + (m & 7) * 64 + tt * 16;
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] *= up;
          const uint32_t h[4] = {pack_half2(v[0], v[1]), pack_half2(v[2], v[3]),
                                 pack_half2(v[4], v[5]), pack_half2(v[6], v[7])};
          *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
          if constexpr (TWO) {  // what is left over: exact, then rounded to 11 bits of its own
            uint32_t rest[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[c]));
              rest[c] = pack_half2(v[2 * c] - f.x, v[2 * c + 1] - f.y);
            }
            *reinterpret_cast<uint4*>(dst + CT * 2048) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
          }
        } else {
          uint32_t d[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)  // rounded to an integer in the low bits, as signed bytes
            d[c] = (__float_as_uint(__fadd_rn(__fmul_rn(v[c], up), kRoundMagic)) -
                    (0x4B400000u - 0x00808080u)) ^ 0x00808080u;
          dst += (j >> 1) * 512 + tt * 16 + (j & 1) * 8;
#pragma unroll
          for (int b = 0; b < 3; ++b) {
            const int tile = !TINY && b == 0 ? 1 : 0;
            const int col = 2 * (m & 3) + (b > 0 ? 2 - b : TINY ? 4 : 0);
            *reinterpret_cast<uint2*>(dst + tile * 1024 + col * 64) =
                make_uint2(gather_bytes(d[0], d[4], d[1], d[5], b),
                           gather_bytes(d[2], d[6], d[3], d[7], b));
          }
        }
        // 2^(E - BITS) * kSumDown, and the digits' 1 / 16 of the codes; digits cannot hold an x' that
        // left fp32's range, so their scale says it (f16 holds infinities itself)
        if (pc % (G / 8) == 0)
          xscale[pc / (G / 8) * TOKENS + m] =
              !HALF && ex == 255u
                  ? __uint_as_float(0x7FC00000u)
                  : __uint_as_float((ex - BITS + 1u) << 23) * (kSumDown * (HALF ? 0.5f : 0.03125f));
      }
      if (base0 + XB * THREADS < pieces_all) fetch_x(base + XB * THREADS);
    }
  }
  __syncthreads();

  // acc[mt][i][h]: row 16 mt + 8 h + g; token 4 i + t, or (HALF) 8 (i / 2) + 2 t + i % 2
  float acc[MT][NT][2] = {};
  bool dead = false;
  int k = first_k, tile_now = first_tile;
  auto take = [&](uint16_t (&scale)[RPS][MT][2], int i) {
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_drain(&full[warp][i % STAGES], (i / STAGES) & 1))) {
      dead = true;
      return;
    }
    const uint8_t* tile = ring + i % STAGES * Cfg::TILE + g * 64 + 16 * t;
#pragma unroll
    for (int rr = 0; rr < RPS; ++rr) {
      const int run = k * RPS + rr;
      if (rr > 0 && run >= runs) break;
      const uint8_t* xp = xs + run * (COLS * 1024) + g * 64 + t * 16;
      const float* xf = xscale + run * (128 / G * TOKENS) + (HALF ? 2 * t : TINY ? t & 1 : t);
      uint4 w[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[mt][h] = *reinterpret_cast<const uint4*>(tile + (rr * WR + 16 * mt + 8 * h) * 64);
      auto row_scale = [&](int mt, int h, int j) {
        const uint32_t v = static_cast<uint32_t>(scale[rr][mt][h]) << 16;
        return __uint_as_float(G == 128 ? v : __shfl_sync(0xFFFFFFFFu, v, (lane & 28) | j));
      };
      if constexpr (HALF) {
        float sum[MT][CT][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 b[Cfg::PARTS * CT];
#pragma unroll
          for (int c = 0; c < Cfg::PARTS * CT; ++c)
            b[c] = *reinterpret_cast<const uint4*>(xp + c * 2048 + j * 512);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t wa = word_of(w[mt][0], j), wb = word_of(w[mt][1], j);
            const uint32_t va = wa >> 8, vb = wb >> 8;
            const uint32_t f[8] = {codes_f16x2<0>(wa), codes_f16x2<0>(wb), codes_f16x2<1>(wa),
                                   codes_f16x2<1>(wb), codes_f16x2<0>(va), codes_f16x2<0>(vb),
                                   codes_f16x2<1>(va), codes_f16x2<1>(vb)};
#pragma unroll
            for (int c = 0; c < Cfg::PARTS * CT; ++c) {
              mma_f16(sum[mt][c % CT], f[0], f[1], f[2], f[3], b[c].x, b[c].y);
              mma_f16(sum[mt][c % CT], f[4], f[5], f[6], f[7], b[c].z, b[c].w);
            }
          }
          if ((j + 1) % (G / 32) == 0) {  // the group ends
            float2 fx[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
              fx[c] = *reinterpret_cast<const float2*>(xf + j / (G / 32) * TOKENS + 8 * c);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float fw = row_scale(mt, h, j);
#pragma unroll
                for (int c = 0; c < CT; ++c) {  // (fw * fx may underflow)
                  float* q = &sum[mt][c][2 * h];
                  acc[mt][2 * c][h] = fmaf(q[0] * fx[c].x, fw, acc[mt][2 * c][h]);
                  acc[mt][2 * c + 1][h] = fmaf(q[1] * fx[c].y, fw, acc[mt][2 * c + 1][h]);
                  q[0] = q[1] = 0.0f;
                }
              }
          }
        }
      } else {
        int sum[MT][COLS][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 b[COLS];
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            b[c] = *reinterpret_cast<const uint4*>(xp + c * 1024 + half * 512);
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int j = 2 * half + jj;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t wa = word_of(w[mt][0], j), wb = word_of(w[mt][1], j);
              const uint32_t f[4] = {(wa << 4) & 0xF0F0F0F0u, (wb << 4) & 0xF0F0F0F0u,
                                     wa & 0xF0F0F0F0u, wb & 0xF0F0F0F0u};
#pragma unroll
              for (int c = 0; c < COLS; ++c)
                mma_s8(sum[mt][c], f, jj ? b[c].z : b[c].x, jj ? b[c].w : b[c].y,
                       j % (G / 32) == 0);
            }
            if ((j + 1) % (G / 32) == 0) {  // the group ends
              const float fx = xf[j / (G / 32) * TOKENS];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float fw = row_scale(mt, h, j);
                  const int* hm = sum[mt][0] + 2 * h;
                  const int low = TINY ? __shfl_xor_sync(0xFFFFFFFFu, hm[0], 2)
                                       : sum[mt][COLS - 1][2 * h];
                  const float v24 = fmaf(static_cast<float>(hm[0]), 65536.0f,
                                         static_cast<float>(hm[1] * 256 + low));
                  // (fw * fx may underflow)
                  acc[mt][0][h] = fmaf(v24 * fx, fw, acc[mt][0][h]);
                }
            }
          }
        }
      }
    }
    __syncwarp();  // the stage has been read
    if (i + STAGES < count) issue(i + STAGES);
    if (i + 2 < count) load_scales(scale);
    if (++k == per_tile || i + 1 == count) {  // the segment ends
      float* seg = segs + (tile_now + warp) * SEG;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int m = HALF ? 8 * (nt >> 1) + 2 * t + (nt & 1) : 4 * nt + t;
            if (!TINY || t < 2) seg[m * WR + 16 * mt + 8 * h + g] = acc[mt][nt][h];
            acc[mt][nt][h] = 0.0f;
          }
      k = 0;
      ++tile_now;
    }
  };
  int i = 0;
  for (; i < count && !dead; i += 2) {
    take(sc[0], i);
    if (i + 1 < count && !dead) take(sc[1], i + 1);
  }
  if (dead && lane == 0)  // a copy did not arrive in time: wait (bounded) for all of them
    for (int q = max(0, i - 2); q < min(count, i + STAGES); ++q)
      mbar_wait_drain(&full[warp][q % STAGES], (q / STAGES) & 1);
  __syncthreads();

  // segment (tile, warp) lies at tile + warp
  auto tile_sum = [&](int q, int at) {
    const short2 w01 = span[q];
    float v = 0.0f;
    for (int w = w01.x; w <= w01.y; ++w)
      if (total >= kGemvWarps || total * w / kGemvWarps < total * (w + 1) / kGemvWarps)
        v += segs[(q + w) * SEG + at];
    return v;
  };
  float* part = reinterpret_cast<float*>(ring_all);  // [tile][token][channel]
  if (S > 1) {
    for (int q = threadIdx.x; q < tiles * SEG; q += THREADS)
      part[q] = total > 0 ? tile_sum(q / SEG, q % SEG) : 0.0f;
    cluster_sync();
  }
  for (int q = threadIdx.x + rank * THREADS; q < tiles * SEG; q += THREADS * S) {
    const int m = q % SEG / WR, n = (tile0 + q / SEG) * WR + q % WR;
    if (m >= M || n >= N) continue;
    float v = 0.0f;
    if (S > 1) {
      float p[kGemvMaxSplit];
#pragma unroll
      for (int c = 0; c < kGemvMaxSplit; ++c) p[c] = c < S ? ld_cluster_f32(mapa_shared(part + q, c)) : 0.0f;
#pragma unroll
      for (int c = 0; c < kGemvMaxSplit; ++c) v += p[c];
    } else {
      v = tile_sum(q / SEG, q % SEG);
    }
    a.y[static_cast<size_t>(m) * N + n] =
        __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(v, kSumUp, a.bias ? a.bias[n] : 0.0f)));
  }
  if (S > 1) cluster_sync();  // nobody leaves while its sums are read
}

bool group_map(CUtensorMap* m, const void* base, int K, int N, int rows, int runs_per_box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(K / 128)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K / 2), 64};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(runs_per_box)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row tiles a cluster may take at most: their joined sums lie over the ring, and their
// segments beside the staged tokens.
template <int G, int MT, int NT, bool TINY, bool TWO>
constexpr int gemv_tiles_limit(int share) {
  using Cfg = GemvCfg<MT, NT, TINY, TWO>;
  const int by_ring = Cfg::RING / (Cfg::SEG * 4);
  const int by_smem = (kGemvMaxSmem - Cfg::smem(share, G, 0)) / (Cfg::SEG * 4);
  const int most = by_ring < by_smem ? by_ring : by_smem;
  return most < kGemvMaxTiles ? most : kGemvMaxTiles;
}

// Clusters of S CTAs, one CTA per SM, that run at the same time on the current device (a
// GPU's SMs come in groups that larger clusters do not fill: 148, 74, 33 and 15 clusters
// of 1, 2, 4 and 8 here).  Asked once per device and instance of the kernel, whose table
// `known` is (all instances have one type).
template <class Kernel>
int gemv_clusters(Kernel kernel, std::atomic<int> (&known)[kAttrDevices][4], int S) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const int at = S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3;
  const bool cached = dev >= 0 && dev < kAttrDevices;
  int n = cached ? known[dev][at].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t q = {};
  q.gridDim = dim3(S);
  q.blockDim = dim3(32 * kGemvWarps);
  q.dynamicSmemBytes = kGemvMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  q.attrs = attr;
  q.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &q) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return sm_count() / S > 0 ? sm_count() / S : 1;  // an estimate, not kept
  }
  if (cached) known[dev][at].store(n, std::memory_order_relaxed);
  return n;
}

template <int G, int MT, int NT, bool TINY, bool TWO>
cudaError_t run_gemv(const uint16_t* x, const float* cinv, const uint8_t* qw, const uint16_t* s_g,
                     const float* bias, uint16_t* y, int M, int K, int N, cudaStream_t st) {
  using Cfg = GemvCfg<MT, NT, TINY, TWO>;
  const int runs = K / 128, tiles = (N + Cfg::WR - 1) / Cfg::WR;
  static std::atomic<bool> done[kAttrDevices];
  static std::atomic<int> known[kAttrDevices][4];
  const cudaError_t e = set_smem_once(gemv_w4g_kernel<G, MT, NT, TINY, TWO>, kGemvMaxSmem, done);
  if (e != cudaSuccess) return e;
  // The split of K, by what an SM has to do, in KB of weights: the tiles of its clusters,
  // staging its share of the tokens (each takes about as long as a quarter of a KB per
  // run), and the exchange of the sums (about 1 us) where there is one.
  int S = 0, per_cluster = 0;
  long long best = 0;
  for (int c = 1; c <= kGemvMaxSplit && c <= runs; c *= 2) {
    const int share = (runs + c - 1) / c;
    const int limit = gemv_tiles_limit<G, MT, NT, TINY, TWO>(share);
    if (limit < 1) continue;
    const int clusters = gemv_clusters(gemv_w4g_kernel<G, MT, NT, TINY, TWO>, known, c);
    int take = (tiles + clusters - 1) / clusters;
    if (take > limit) take = limit;
    const long long waves = ((tiles + take - 1) / take + clusters - 1) / clusters;
    take = static_cast<int>((tiles + clusters * waves - 1) / (clusters * waves));  // even waves
    const long long cost = waves * (4LL * take * share * MT + Cfg::TOKENS * share + (c > 1 ? 184 : 0));
    if (S == 0 || cost < best) {
      best = cost;
      S = c;
      per_cluster = take;
    }
  }
  if (S == 0) return cudaErrorInvalidValue;
  const int share = (runs + S - 1) / S;
  CUtensorMap tm;
  if (!group_map(&tm, qw, K, N, Cfg::WR, Cfg::RPS)) return cudaErrorInvalidValue;
  const GemvArgs a{x, cinv, s_g, bias, y, M, K, N, S, share, per_cluster};
  const int grid = (tiles + per_cluster - 1) / per_cluster * S;
  return launch_pdl(gemv_w4g_kernel<G, MT, NT, TINY, TWO>, grid, 32 * kGemvWarps,
                    Cfg::smem(share, G, per_cluster), st, S, tm, a);
}

template <int G>
cudaError_t dispatch_gemv(const uint16_t* x, const float* cinv, const uint8_t* qw,
                          const uint16_t* s_g, const float* bias, uint16_t* y, int M, int K, int N,
                          cudaStream_t st) {
  // the largest split must hold the staged tokens; where it cannot (more than 8 tokens of
  // long rows), 8 tokens at a time
  const int share = (K / 128 + kGemvMaxSplit - 1) / kGemvMaxSplit;
  const int limit = cinv ? gemv_tiles_limit<G, 2, 4, false, true>(share)
                         : gemv_tiles_limit<G, 2, 4, false, false>(share);
  const int most = M > 8 && limit < 4 ? 8 : M;
  for (int m = 0; m < M; m += most) {
    const int n = M - m < most ? M - m : most;
    const uint16_t* xm = x + static_cast<size_t>(m) * K;
    uint16_t* ym = y + static_cast<size_t>(m) * N;
    const cudaError_t e =
        n <= 2   ? run_gemv<G, 1, 1, true, false>(xm, cinv, qw, s_g, bias, ym, n, K, N, st)
        : n <= 4 ? run_gemv<G, 2, 1, false, false>(xm, cinv, qw, s_g, bias, ym, n, K, N, st)
        : n <= 8 ? (cinv ? run_gemv<G, 2, 2, false, true>(xm, cinv, qw, s_g, bias, ym, n, K, N, st)
                         : run_gemv<G, 2, 2, false, false>(xm, cinv, qw, s_g, bias, ym, n, K, N, st))
        : cinv   ? run_gemv<G, 2, 4, false, true>(xm, cinv, qw, s_g, bias, ym, n, K, N, st)
                 : run_gemv<G, 2, 4, false, false>(xm, cinv, qw, s_g, bias, ym, n, K, N, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_pack_int4_group(const uint16_t* W, const float* c, int N, int K, int group,
                                   uint8_t* qw, uint16_t* s_g, cudaStream_t st) {
  const int strips = (K + 511) / 512, tiles = (N + 15) / 16;
  // two CTAs per SM, a whole number for each strip
  int per_strip = (2 * sm_count() + strips - 1) / strips;
  per_strip = per_strip < tiles ? per_strip : tiles;
  uint4* q = reinterpret_cast<uint4*>(qw);
#define WQ_PACK(G_)                                                                          \
  return c ? launch_pdl(pack_int4_group_kernel<G_, true>, per_strip * strips, 256, 0, st, 1, W, c, \
                        N, K, strips, q, s_g)                                                \
           : launch_pdl(pack_int4_group_kernel<G_, false>, per_strip * strips, 256, 0, st, 1, W, c, \
                        N, K, strips, q, s_g)
  if (group == 32) WQ_PACK(32);
  if (group == 64) WQ_PACK(64);
  WQ_PACK(128);
#undef WQ_PACK
}

cudaError_t launch_gemv_w4g(const uint16_t* x, const float* cinv, const uint8_t* qw,
                            const uint16_t* s_g, int group, const float* bias, uint16_t* y, int M,
                            int K, int N, cudaStream_t st) {
#define WQ_GEMV(G_) return dispatch_gemv<G_>(x, cinv, qw, s_g, bias, y, M, K, N, st)
  if (group == 32) WQ_GEMV(32);
  if (group == 64) WQ_GEMV(64);
  WQ_GEMV(128);
#undef WQ_GEMV
}

}  // namespace wq
