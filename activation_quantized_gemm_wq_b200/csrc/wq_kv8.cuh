// A paged key/value cache in int8 and the attention that reads it (the denoiser keeps
// the keys and values of its context tokens between steps; App. D names the cache).
//   kv8_append  quantizes new keys and values into the cache
//   attn_kv8    softmax(scale q k^T) v over the cached tokens
//
// Cache: codes int8 [pages][kv_heads][page_tokens][D], scales fp32
// [pages][kv_heads][page_tokens / 16]: one scale per head and block of 16 tokens, for
// keys and values each; value = scale * code.  A sequence's token p lies in page
// table[b][p / page_tokens], slot p % page_tokens; blocks never straddle pages.
#pragma once
#include <cuda_fp16.h>

#include "wq_group.cuh"
#include "wq_internal.h"
#include "wq_ptx.cuh"
#include "wq_quant.cuh"

namespace wq {

// Device error bits of the cache operators, in the second error word: the GEMM's waits
// would give up on any bit in the first.
enum : unsigned { kErrCache = 4u };

namespace {

constexpr int kBlockTokens = 16;

__device__ __forceinline__ void raise_cache_error() { atomicOr(&g_error_words[1], kErrCache); }

// The sequence that packed row r belongs to: the last b with start[b] <= r, found 32
// candidates at a time by a whole warp; -1 if r is before the first or behind the last
// sequence.  Stays within start[0..B] whatever the values are.
__device__ __forceinline__ int find_sequence(const int* __restrict__ start, int B, int r) {
  if (r < start[0] || r >= start[B]) return -1;
  const int lane = threadIdx.x & 31;
  int lo = 0, span = B;  // the answer lies in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32;
    const int at = lo + lane * step;
    const bool in = lane * step < span;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, in && start[in ? at : lo] <= r);
    const int k = hit ? 31 - __clz(hit) : 0;
    span = min(step, span - k * step);
    lo += k * step;
  }
  return lo;
}

// ------------------------------------------------------------ append

struct AppendArgs {
  const uint16_t* x[2];  // keys, values: bf16 rows [T], heads x D packed within a row
  long long stride[2];   // elements between rows
  const int* row_start;  // [B + 1]
  const int* past_len;   // [B]
  const int* table;      // [B][max_pages]
  int8_t* codes[2];
  float* scale[2];
  int T, B, max_pages, pages, heads, page_tokens;
  int page_shift;  // log2 of page_tokens
  int window;      // packed rows a warp looks through for the first tokens of blocks
};

// A warp quantizes whole blocks: all new tokens of one block, one head, keys or values.
// It loads them (at most 16 x D bf16, all loads issued together), takes their maximum by
// shuffles, and
//   s_new = max(s_old, max|x| / 127)  (s_old: the block's scale if it has older tokens),
//   new codes  clamp(rint(x / s_new), +-127),
//   old codes  rint(code * (s_old / s_new)) when the scale grew,
// so a block's scale is that of the largest value ever appended to it, however the
// tokens came.  IEEE fp32 throughout: codes and scales are reproducible bit for bit.
// A block is handled by the warp whose window holds its first new token; the window is
// one row for decoding (a warp per new token) and 16 rows for long runs (about one block
// per warp, and no warps that find nothing).  The issue of instructions (54 % of cycles; about
// 650 for a block) and the latency of a block's loads bound it: 3 sequences of up to 4256
// tokens, 32 heads of 128, 55.1 us, 4.2 TB/s read and written; 32 single tokens, 8 heads,
// 3.3 us.  Exact quotients by two remainder steps, without a test for near ties, and 32-bit
// indices within a page took the first from 109 to 60 us, five CTAs to an SM below 55.
template <int D>
__global__ void __launch_bounds__(128, D == 128 ? 5 : 7) kv8_append_kernel(const AppendArgs a) {
  constexpr int TC = D / 8;                        // 8-channel chunks of a token
  constexpr int CPL = kBlockTokens * TC / 32;      // chunks per lane of a full block
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * 4u + (threadIdx.x >> 5);
  const uint32_t windows = (a.T + a.window - 1) / a.window;
  griddep_wait();
  griddep_launch_dependents();
  const long long capacity = static_cast<long long>(a.max_pages) * a.page_tokens;
  if (unit == 0)  // the tables as a whole, once: a sequence may have no row that a warp looks at
    for (int i = lane; i < a.B; i += 32) {
      const long long lo = a.row_start[i], hi = a.row_start[i + 1], past = a.past_len[i];
      if (lo < 0 || hi < lo || hi > a.T || past < 0 || past + (hi - lo) > capacity)
        raise_cache_error();
    }
  if (unit >= windows * a.heads * 2u) return;
  const int which = unit & 1;
  const int head = (unit >> 1) % static_cast<uint32_t>(a.heads);
  const int t0 = (unit >> 1) / static_cast<uint32_t>(a.heads) * a.window;
  const int t_end = min(t0 + a.window, a.T);
  const uint16_t* x = which ? a.x[1] : a.x[0];
  int8_t* codes = which ? a.codes[1] : a.codes[0];
  float* scales = which ? a.scale[1] : a.scale[0];
  const long long stride = which ? a.stride[1] : a.stride[0];

  int t = max(t0, a.row_start[0]), b = -1;
  int first = 0, last = 0, past = 0;  // rows [first, last) of sequence b
  while (t < t_end) {
    if (b < 0 || t >= last) {
      b = find_sequence(a.row_start, a.B, t);
      if (b < 0) return;  // rows outside every sequence are left alone
      first = a.row_start[b];
      const int end = a.row_start[b + 1];
      last = min(end, a.T);
      past = a.past_len[b];
      if (past < 0 || first < 0 || last <= t || end > a.T ||
          static_cast<long long>(past) + (last - first) > capacity) {
        if (lane == 0) raise_cache_error();
        if (last <= t) return;
        t = last;  // the sequence does not fit its table: none of it is written
        continue;
      }
    }
    const int pos = past + (t - first);
    const int in_block = pos & (kBlockTokens - 1);
    const int stop = min(t + kBlockTokens - in_block, last);
    if (in_block != 0 && t != first) {  // a block that an earlier row began
      t = stop;
      continue;
    }
    const int page = a.table[static_cast<long long>(b) * a.max_pages + (pos >> a.page_shift)];
    if (page < 0 || page >= a.pages) {
      if (lane == 0) raise_cache_error();
      t = stop;
      continue;
    }
    const int slot = (pos & (a.page_tokens - 1)) - in_block;  // the block's first slot
    const long long hp = static_cast<long long>(page) * a.heads + head;
    int8_t* blk = codes + (hp * a.page_tokens + slot) * D;
    float* sp = scales + hp * (a.page_tokens / kBlockTokens) + slot / kBlockTokens;
    const int count = stop - t;

    uint4 raw[CPL];
    float amax = 0.0f;
    const float s_old = in_block ? *sp : 0.0f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = lane + 32 * i, tok = c / TC, ch = c % TC;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (tok < count)
        raw[i] = __ldcs(reinterpret_cast<const uint4*>(x + (t + tok) * stride + head * D + 8 * ch));
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        amax = max_or_nan(amax, max_or_nan(fabsf(bf16lo(w[e])), fabsf(bf16hi(w[e]))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      amax = max_or_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    // (a maximum that is not finite gives NaN, and a block that has one keeps it)
    const float s = max_or_nan(s_old, __fdiv_rn(fmaf(amax, 0.0f, amax), 127.0f));
    const bool plain = plain_scale(s);
    const float r = plain ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = lane + 32 * i, tok = c / TC, ch = c % TC;
      if (tok >= count) continue;
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float2 v[4];
      uint32_t q[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = make_float2(bf16lo(w[e]), bf16hi(w[e]));
      if (plain) {
        quantize8_pairs(v, s, r, q);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[2 * e] = static_cast<uint32_t>(quantize_exact<127>(v[e].x, s));
          q[2 * e + 1] = static_cast<uint32_t>(quantize_exact<127>(v[e].y, s));
        }
      }
      *reinterpret_cast<uint2*>(blk + (in_block + tok) * D + 8 * ch) =
          make_uint2(pack_low_bytes(q[0], q[1], q[2], q[3]), pack_low_bytes(q[4], q[5], q[6], q[7]));
    }
    __syncwarp();  // every lane has read the old scale
    if (s > s_old && in_block) {  // the older tokens take the new scale
      const float ratio = __fdiv_rn(s_old, s);
      for (int c = lane; c < in_block * (D / 4); c += 32) {
        uint32_t* p = reinterpret_cast<uint32_t*>(blk) + c;
        const uint32_t w = *p;
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float old = static_cast<float>(static_cast<int8_t>(w >> (8 * e)));
          q[e] = static_cast<uint32_t>(__float2int_rn(__fmul_rn(old, ratio)));
        }
        *p = pack_low_bytes(q[0], q[1], q[2], q[3]);
      }
    }
    if (lane == 0 && (!in_block || !(s <= s_old))) *sp = s;
    t = stop;
  }
}

// ------------------------------------------------------------ attention

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two bytes (code + 128) that `sel` picks out of w, as two f16 codes, exactly: placed
// under the exponent of 1024 (f16 holds integers up to 2048), then 1152 taken off.
__device__ __forceinline__ uint32_t bytes_f16x2(uint32_t w, uint32_t sel) {
  const uint32_t u = __byte_perm(w, 0x64646464u, sel);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __floats2half2_rn(1152.0f, 1152.0f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16-byte chunk `chunk` of row `row` in a tile of D-byte rows as the copy engine's
// 128-byte (D = 128) or 64-byte (D = 64) swizzle leaves it.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4)
                  : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// 2^(e - 127 - bits) times the softmax scale's size, for a row of queries whose largest value has
// the exponent field e >= bits: what turns its sums into scores.  A NaN if that value is not
// finite: digits do not hold one, nor does a maximum or an infinite weight pass it on, but
// scores that are NaN make all of the row's results NaN (of a row that sees any token).
__device__ __forceinline__ float row_factor(uint32_t e, uint32_t bits, float scale) {
  return e == 255u ? __uint_as_float(0x7FC00000u)
                   : __uint_as_float((e - bits + 1u) << 23) * 0.5f * fabsf(scale);
}

constexpr int kAttnWarps = 4;
constexpr int kAttnMinUnits = 16;  // blocks of 16 tokens a CTA takes at least

// Softmax weights p_j times the scale of their values' block enter the second product as two
// f16 parts, the second what the first leaves over, multiplied by the same codes into the same
// sums: one part alone would round them to 11 bits, which is seen where values cancel, and fp32
// weights cannot enter the instruction.  They are 2^kPShift times their value relative to a
// row's reference, which the largest of the row so far may exceed by up to 2^kPSlack before the
// sums are rescaled: at most 2^15 (f16 reaches 65504), off by at most 2^-22 of themselves or
// 2^-36 of the reference.
constexpr float kPShift = 11.0f, kPSlack = 4.0f;

// The sums of p v that leave the matrix instructions' accumulators are held at 2^-14 of their
// value: values near fp32's largest then do not overflow in a sum whose quotient is in range,
// and what is lost at the other end is below half of bf16's smallest step.
constexpr float kSumUnit = 0x1p-14f, kOutUnit = 0x1p25f;  // 2^kPShift / kSumUnit

// What two f16 leave over of two fp32 values, as f16.
__device__ __forceinline__ uint32_t half2_rest(float a, float b, uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_half2(a - f.x, b - f.y);
}

// 2^x down to the smallest subnormal.
__device__ __forceinline__ float exp2_full(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {  // -infinity for subnormals
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's references: weights p_j = 2^(s_j - m), s_j the scores times log2(e); their products
// with the value scales are held relative to 2^e.  Both exponents are whole, so that sums are
// rescaled by powers of two.  e follows the row's own products: a block whose value scale is
// large takes no bits from the others where the row gives it no weight.
struct AttnRow {
  float m, l;   // l: sum of 2^kPShift p_j
  float bound;  // of s_j + log2(scale): m + e + kPSlack
  float inv;    // 2^-e

  __device__ __forceinline__ void start() {
    m = bound = -INFINITY;
    l = 0.0f;
    inv = 0x1p125f;
  }
  // top: of scores, u: of scores + log2(value scale).  Any lane of a row may ask.
  __device__ __forceinline__ bool exceeded(float top, float u) const {
    return top > m + kPSlack || u > bound;
  }
  // The row's own top and u have come: the factor of its sums so far.
  __device__ __forceinline__ float raise(float top, float u) {
    const bool over = exceeded(top, u);
    const float m_new = top > m + kPSlack ? ceilf(top) : m;
    const float back = over ? m - m_new : 0.0f, e = exponent();
    const float e_up = fminf(fmaxf(ceilf(fmaxf(u - m_new, e + back)), -125.0f), 126.0f);
    const float e_new = over ? e_up : e;
    l *= exp2_approx(back);
    m = m_new;
    bound = m_new + e_new + kPSlack;
    inv = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(e_new)) << 23);
    return exp2_approx(back + (e - e_new));
  }
  __device__ __forceinline__ float exponent() const {
    return 127.0f - static_cast<float>(__float_as_uint(inv) >> 23);
  }
  // What turns p_j 2^kPShift into its f16 weight.  (Beyond 2^126 the weights are below 2^-122;
  // an infinity would make a NaN of masked ones.)
  __device__ __forceinline__ float weight(float sv) const {
    float w;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(w) : "f"(sv * inv), "f"(0x1p126f));
    return w;
  }
  __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.0f : m - kPShift; }
};

struct AttnArgs {
  const uint16_t* q;      // bf16 rows [Tq], heads x D packed within a row
  long long q_stride;     // elements between rows
  const int* q_start;     // [B + 1]
  const int* kv_len;      // [B]
  const int* table;       // [B][max_pages]
  const float* k_scale;   // [pages][kv_heads][page_tokens / 16]
  const float* v_scale;
  uint16_t* out;          // bf16 [Tq][q_heads][D]
  float* lse;             // [Tq][q_heads] or null
  struct AttnCut* cuts;   // workspace: [grid], what each CTA's end cuts
  float* partial;         // workspace: [grid][2] partial results
  int Tq, B, q_heads, kv_heads, max_pages, pages, page_tokens, causal;
  int whole;              // items are not cut: a unit is an item
  float scale_log2;       // softmax scale * log2(e)
};

// The item that a CTA's end cuts: parts of it lie at CTA c0, as its second partial result,
// and at c0 + 1 .. c0 + ends, as their first.
struct __align__(16) AttnCut {
  int ends;           // ends of CTAs inside the item; 0: this CTA's end cuts none
  int c0;
  int q0, head;       // the sequence's first query row, the item's cache head
  int r_first, rows;  // the tile's rows
  int unused[2];
};

// What a sequence asks for: the work is cut into units of one block of 16 tokens for one
// item, an item being one cache head and one tile of query rows.  An item without any
// block counts one unit, so that its rows are written.  Where no sequence can be long
// (AttnArgs::whole), a unit is an item: nothing is left to be joined.
struct SeqWork {
  int q0, nq, len;       // query rows [q0, q0 + nq), cached tokens
  int tiles;             // row tiles per cache head
  int blocks;            // of an item
  int item_units;
  long long units;
};

template <int RT>
__device__ __forceinline__ SeqWork sequence_work(const AttnArgs& a, int b, bool report) {
  SeqWork w;
  const long long capacity = static_cast<long long>(a.max_pages) * a.page_tokens;
  const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
  w.q0 = min(max(s0, 0), a.Tq);
  w.nq = max(min(s1, a.Tq) - w.q0, 0);
  const int len = a.kv_len[b];
  w.len = static_cast<int>(min(static_cast<long long>(max(len, 0)), capacity));
  if (report && (len < 0 || len > capacity || s0 < 0 || s1 > a.Tq || s1 < s0)) raise_cache_error();
  const int G = a.q_heads / a.kv_heads;
  w.tiles = static_cast<int>((static_cast<long long>(w.nq) * G + RT - 1) / RT);
  w.blocks = max(1, (w.len + kBlockTokens - 1) / kBlockTokens);
  w.item_units = a.whole ? 1 : w.blocks;
  w.units = static_cast<long long>(w.tiles) * w.item_units * a.kv_heads;
  return w;
}

__device__ __forceinline__ long long units_per_cta(long long total, int grid, int whole) {
  return max(static_cast<long long>(whole ? 1 : kAttnMinUnits), (total + grid - 1) / grid);
}

// Units before every sequence: each thread sums a run of them, then a scan over threads.
// Every CTA finds its share [begin, end) of them and where that starts: sequence b, unit
// rem of it.
struct AttnSched {
  long long scan[kAttnWarps];
  long long rem, end, per;
  int b;
};

struct AttnShare {
  long long begin, end, rem;
  int b;
};

template <int RT>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a, AttnSched& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_thread = (a.B + 32 * kAttnWarps - 1) / (32 * kAttnWarps);
  const int b_lo = min(static_cast<int>(threadIdx.x) * per_thread, a.B);
  const int b_hi = min(b_lo + per_thread, a.B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += sequence_work<RT>(a, b, blockIdx.x == 0).units;
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += up;
  }
  if (lane == 31) sh.scan[warp] = before;
  __syncthreads();
  before -= mine;
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  AttnShare s;
  const long long per = units_per_cta(total, gridDim.x, a.whole);
  s.begin = min(per * blockIdx.x, total);
  s.end = min(s.begin + per, total);
  if (threadIdx.x == 0) {
    sh.end = s.end;
    sh.per = per;
    a.cuts[blockIdx.x].ends = 0;  // until the last segment says otherwise
  }
  if (s.begin >= before && s.begin < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = sequence_work<RT>(a, b, false).units;
      if (s.begin >= at && s.begin < at + n) {
        sh.b = b;
        sh.rem = s.begin - at;
      }
      at += n;
    }
  }
  __syncthreads();
  s.b = sh.b;
  s.rem = sh.rem;
  return s;
}

// A warp's way through a CTA's share: segments, each a part of one item's blocks, of which the
// warp takes every kAttnWarps-th step of two blocks.
template <int RT>
struct AttnSegment {
  SeqWork sw;
  int j0, take;     // the segment: blocks [j0, j0 + take) of the item
  int head, r_first;
  int blocks;       // of those, the ones that some row of the tile sees
  int count;        // my steps

  __device__ __forceinline__ AttnSegment(const AttnArgs& a, const AttnShare& s, int wt, int lane)
      : b_(s.b), rem_(s.rem), left_(s.end - s.begin), wt_(wt), lane_(lane) {
    sw = sequence_work<RT>(a, b_, false);
  }

  __device__ __forceinline__ void begin(const AttnArgs& a) {
    while (rem_ >= sw.units) {  // the next sequence that has any work
      rem_ = 0;
      sw = sequence_work<RT>(a, ++b_, false);
    }
    const long long item = rem_ / sw.item_units;
    const int at = static_cast<int>(rem_ - item * sw.item_units);
    units_ = static_cast<int>(min(static_cast<long long>(sw.item_units - at), left_));
    j0 = a.whole ? 0 : at;
    take = a.whole ? sw.blocks : units_;
    head = static_cast<int>(item / sw.tiles);
    r_first = static_cast<int>(item % sw.tiles) * RT;
    const int G = a.q_heads / a.kv_heads;
    const int r_last = min(r_first + RT, sw.nq * G) - 1;
    // tokens that the tile's last row sees, which no earlier row exceeds
    const int reach = a.causal ? max(0, sw.len - sw.nq + r_last / G + 1) : sw.len;
    blocks = max(0, min(take, (reach + kBlockTokens - 1) / kBlockTokens - j0));
    const int steps = (blocks + 1) / 2;
    count = steps > wt_ ? (steps - wt_ + kAttnWarps - 1) / kAttnWarps : 0;
    look_up(a, 0, row_[0], sk_[0], sv_[0]);
    look_up(a, 1, row_[1], sk_[1], sv_[1]);
  }

  // Whether there is another segment; behind the last one, what the CTA's end cuts.
  __device__ __forceinline__ bool advance(const AttnArgs& a, const AttnSched& sh) {
    if (left_ == units_ && threadIdx.x == 0 && !a.whole && j0 + take < sw.blocks) {
      AttnCut c;
      const long long u0 = sh.end - units_ - j0;  // the item's first unit
      c.c0 = static_cast<int>(u0 / sh.per);
      c.ends = static_cast<int>((u0 + sw.blocks - 1) / sh.per) - c.c0;
      c.q0 = sw.q0;
      c.head = head;
      c.r_first = r_first;
      c.rows = min(RT, sw.nq * (a.q_heads / a.kv_heads) - r_first);
      a.cuts[blockIdx.x] = c;
    }
    rem_ += units_;
    left_ -= units_;
    return left_ > 0;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && take == sw.blocks; }

  // Row of the copy of step i, block lane % 2 (-1: none), while step `now` is looked at.
  __device__ __forceinline__ int copy_row(int i, int now, int lane) const {
    return __shfl_sync(0xFFFFFFFFu, (i >> 4) == (now >> 4) ? row_[0] : row_[1],
                       2 * (i & 15) + (lane & 1));
  }
  __device__ __forceinline__ void scales(int i, int c, float& sk, float& sv) const {
    sk = __shfl_sync(0xFFFFFFFFu, sk_[0], 2 * (i & 15) + c);
    sv = __shfl_sync(0xFFFFFFFFu, sv_[0], 2 * (i & 15) + c);
  }
  // Step i is done.
  __device__ __forceinline__ void next_blocks(int i, const AttnArgs& a) {
    if ((i & 15) != 15) return;
    row_[0] = row_[1];
    sk_[0] = sk_[1];
    sv_[0] = sv_[1];
    look_up(a, (i >> 4) + 2, row_[1], sk_[1], sv_[1]);
  }

 private:
  // Blocks of my steps 16 group .. + 15, one per lane: row of the copy, scales.
  __device__ __forceinline__ void look_up(const AttnArgs& a, int group, int& row, float& sk,
                                          float& sv) const {
    const int i = 16 * group + (lane_ >> 1);
    const int j = 2 * (wt_ + kAttnWarps * i) + (lane_ & 1);  // of the segment's blocks
    row = -1;
    sk = sv = 0.0f;
    if (j >= blocks) return;
    const int pos = (j0 + j) * kBlockTokens;
    int page = a.table[static_cast<long long>(b_) * a.max_pages + pos / a.page_tokens];
    if (page < 0 || page >= a.pages) {
      raise_cache_error();
      page = 0;
    }
    const long long hp = static_cast<long long>(page) * a.kv_heads + head;
    const int slot = pos % a.page_tokens;
    row = static_cast<int>(hp * a.page_tokens + slot);
    const long long at = hp * (a.page_tokens / kBlockTokens) + slot / kBlockTokens;
    // (an infinity becomes a NaN: a score of -infinity would pass for a masked one)
    sk = fmaf(a.k_scale[at], 0.0f, a.k_scale[at]);
    sv = fmaf(a.v_scale[at], 0.0f, a.v_scale[at]);
  }

  int b_;
  long long rem_, left_;  // the unit of sequence b_, units left of the share
  int wt_, lane_, units_;
  int row_[2];            // this and the next sixteen steps' blocks, one per lane
  float sk_[2], sv_[2];
};

// Copies of a step: lanes 0 and 1 fetch the keys and values of a block each (copy_row, -1
// where there is none) into [keys 0, keys 1, values 0, values 1].
template <int TILE>
__device__ __forceinline__ void attn_copy(uint8_t* stage, const void* tm_k, const void* tm_v,
                                          uint64_t* bar, int copy_row, int lane) {
  const int other = __shfl_xor_sync(0xFFFFFFFFu, copy_row, 1);
  if (lane == 0) mbar_arrive_expect_tx(bar, other >= 0 ? 4 * TILE : 2 * TILE);
  __syncwarp();
  if (lane < 2 && copy_row >= 0) {
    tma_load_2d(stage + lane * TILE, tm_k, bar, 0, copy_row);
    tma_load_2d(stage + (2 + lane) * TILE, tm_v, bar, 0, copy_row);
  }
}

// Where the four of channels d .. d + 3 of a row lies in a warp's slab of sums, a whole stage
// of its ring: rows of D floats, the fours of a row swizzled over the banks.
template <int D>
__device__ __forceinline__ int slab_offset(int row, int d) {
  return row * D + (((d >> 2) ^ (row & 7)) << 2);
}

// What the warps leave of a segment in shared memory: their rows' references, sums of
// weights, and exponents of sums of p v.
template <int RT>
struct AttnRows {
  float m[kAttnWarps][RT], l[kAttnWarps][RT], me[kAttnWarps][RT];  // me: m + e
  const float* slab[kAttnWarps];                                  // the sums of p v themselves

  __device__ __forceinline__ void put(int warp, int r, const AttnRow& row, float sum) {
    m[warp][r] = row.m;
    l[warp][r] = sum;
    me[warp][r] = row.m + row.exponent();
  }
};

// The end of a segment: the warps' sums are joined relative to the largest reference, in
// order, and written as the result, or as a partial one where other CTAs have a part of the
// item; rows [row0, row0 + ROWS) of a tile of RT, in PARTS rows of a slab each.
template <int D, int RT, int ROWS, int PARTS>
__device__ __forceinline__ void attn_finish(const AttnArgs& a, const SeqWork& sw,
                                            const AttnRows<RT>& left, int r_first, int row0,
                                            int head, bool whole, bool from_start) {
  constexpr int WT = kAttnWarps;
  const int G = a.q_heads / a.kv_heads, rows = sw.nq * G;
  float* dst = a.partial + (static_cast<long long>(blockIdx.x) * 2 + (from_start ? 1 : 0)) *
                               (RT * (D + 2));
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += 32 * kAttnWarps) {
    const int r = row0 + i / (D / 4), d = 4 * (i % (D / 4));
    if (r_first + r >= rows) break;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < WT; ++k) top = fmaxf(top, left.m[k][r]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < WT; ++k) {
      sum += left.l[k][r] * exp2_approx(left.m[k][r] - ref);  // (a warp without tokens: 0 * 0)
      // (kOutUnit and f one after the other: their quotient may be below the range)
      const float f = exp2_full(left.me[k][r] - ref);
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        const float4 p = *reinterpret_cast<const float4*>(
            left.slab[k] + slab_offset<D>(r - row0 + part * ROWS, d));
        v.x = fmaf(p.x * (1.0f / kOutUnit), f, v.x);
        v.y = fmaf(p.y * (1.0f / kOutUnit), f, v.y);
        v.z = fmaf(p.z * (1.0f / kOutUnit), f, v.z);
        v.w = fmaf(p.w * (1.0f / kOutUnit), f, v.w);
      }
    }
    if (whole) {
      const float inv = sum > 0.0f ? kOutUnit / sum : 0.0f;
      const int qi = (r_first + r) / G, qh = head * G + (r_first + r) % G;
      const long long at = static_cast<long long>(sw.q0 + qi) * a.q_heads + qh;
      const __nv_bfloat162 x0 = __floats2bfloat162_rn(v.x * inv, v.y * inv);
      const __nv_bfloat162 x1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(a.out + at * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1));
      if (a.lse && d == 0)
        a.lse[at] = sum == 0.0f ? -INFINITY : (top - kPShift + log2f(sum)) * 0.69314718055994531f;
    } else {
      *reinterpret_cast<float4*>(dst + r * D + d) = v;
      if (d == 0) {
        dst[RT * D + 2 * r] = top;
        dst[RT * D + 2 * r + 1] = sum;
      }
    }
  }
}

// One CTA of four warps takes an equal share of all units (so ragged batches stay
// balanced and one long sequence fills the GPU), item by item.  An item's steps of two blocks
// are taken by the warps in turn, each with a ring of its own that bulk tensor copies fill, so
// the warps run independently between the ends of segments; the first step of the next
// segment is fetched while a segment's sums are joined.  Codes become f16 in registers,
// exactly (with MT = 2 once for 32 query rows); q enters as f16 after a power-of-two scaling
// per row that keeps all its 8 bits; scores, maxima, sums and the output are fp32.  Block
// scales multiply the scores (keys) and the softmax weights, relative to their row's
// power-of-two reference (values).
// Eight warps to an SM (255 registers) issue in 37 % of all cycles: the chain of copies'
// arrival, conversion, matrix steps and softmax bounds it, not the tensor cores (28 %) nor
// memory (10 %).  2 x 64 queries over up to 8512 tokens, 32 heads of 64: 64.2 us, of 128:
// 100.8 us; 2 x 256 queries, heads of 128: 257 us.  The weights' second parts, half as many
// matrix steps again, are most of what these took less without them (57.3, 84 and 210 us; 55.2,
// 82.2 and 204 us with one reference to a warp).  With one part: 58.1 us for the first with
// MT = 1 (83.5 us the first, simple kernel); codes made f16 once per CTA in shared memory for
// 64 rows were 3 % faster there, but 4 to 7 % slower for heads of 128.
template <int D, int MT>
struct AttnCfg {
  static constexpr int WT = kAttnWarps;
  static constexpr int RT = 16 * MT;           // rows of a tile
  static constexpr int TILE = kBlockTokens * D;
  static constexpr int STEP = 4 * TILE;        // two blocks of keys and values
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr bool QREG = MT * D <= 128;  // q stays in registers, else in shared memory
  static constexpr int RING = WT * STAGES * STEP;
  static constexpr int QBYTES = QREG ? 0 : WT * RT * D * 2;
  static constexpr int SMEM = RING + QBYTES + 1024;  // + alignment
  static constexpr int CTAS = MT == 1 && D == 64 ? 3 : 2;  // per SM
  static_assert(16 * D * 4 <= STEP, "a warp's sums of sixteen rows fit one stage");
};

template <int D, int MT>
__global__ void __launch_bounds__(32 * kAttnWarps, AttnCfg<D, MT>::CTAS) attn_kv8_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const AttnArgs a) {
  using C = AttnCfg<D, MT>;
  constexpr int WT = C::WT, RT = C::RT, STAGES = C::STAGES, TILE = C::TILE, STEP = C::STEP;
  constexpr bool QREG = C::QREG;
  constexpr int KS = D / 16;   // matrix steps over the channels
  constexpr int ND = D / 8;    // 8-channel tiles of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[WT][STAGES];
  __shared__ AttnRows<RT> left;
  __shared__ AttnSched sched;

  const int wt = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.q_heads / a.kv_heads;
  uint8_t* my_ring = ring + wt * STAGES * STEP;
  // [step over the channels][16-row half][lane] operands, a copy per warp
  uint4* q_smem = reinterpret_cast<uint4*>(ring + C::RING) + wt * (QREG ? 0 : KS * MT * 32) + lane;

  if (threadIdx.x == 0) {
    for (int i = 0; i < WT; ++i)
      for (int s = 0; s < STAGES; ++s) mbar_init(&full[i][s], 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();
  griddep_launch_dependents();
  const AttnShare share = attn_share<RT>(a, sched);
  if (share.begin >= share.end) return;

  uint32_t phase = 0;  // steps this warp has taken before this segment (stage and parity)
  AttnSegment<RT> seg(a, share, wt, lane);
  auto issue = [&](int i, int consumed) {  // copies of my step i: two lanes, a block each
    const int copy_row = seg.copy_row(i, consumed, lane);
    const uint32_t st = (phase + i) % STAGES;
    attn_copy<TILE>(my_ring + st * STEP, &tm_k, &tm_v, &full[wt][st], copy_row, lane);
  };
  seg.begin(a);
  if (seg.count > 0) issue(0, 0);

  for (;;) {
    const int count = seg.count, j0 = seg.j0, blocks = seg.blocks, head = seg.head, r_first = seg.r_first;
    const SeqWork sw = seg.sw;
    const int rows = sw.nq * G;
    int issued = min(count, 1);
    for (; issued < min(count, STAGES); ++issued) issue(issued, 0);

    // my rows: g and g + 8 of each sixteen.  q as f16 operands: channel 32t + 16x + 4w + 0..3
    // (D = 128; 16t + 4w for D = 64) of a row is what lane t's word w of its load x holds of
    // a key
    int see[MT][2], see_min = 0x7FFFFFFF;
    float qs[MT][2];  // undoes the rows' power-of-two scaling, times the softmax scale
    uint32_t qf[QREG ? KS : 1][MT][4];
    __syncwarp();  // the last item's operands in shared memory have been read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t f[KS][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r_first + 16 * mt + 8 * h + g;
        const bool valid = r < rows;
        const int qi = valid ? r / G : 0, qh = head * G + (valid ? r % G : 0);
        see[mt][h] = valid && a.causal ? sw.len - sw.nq + qi + 1 : sw.len;
        see_min = min(see_min, see[mt][h]);
        const uint16_t* qp = a.q + (sw.q0 + qi) * a.q_stride + static_cast<long long>(qh) * D + t * (D / 4);
        uint4 raw[D / 32];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          raw[i] = valid ? *reinterpret_cast<const uint4*>(qp + 8 * i) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = max_or_nan(top, max_or_nan(fabsf(bf16lo(w[e])), fabsf(bf16hi(w[e]))));
        }
        top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // the largest value of the row comes to lie in [2^14, 2^15)
        const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
        // (the softmax scale's sign goes to q: factors of scores are not negative)
        const float up = copysignf(__uint_as_float((268u - e) << 23), a.scale_log2);
        qs[mt][h] = row_factor(e, 14u, a.scale_log2);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2)
            f[2 * i + (e2 >> 1)][h + 2 * (e2 & 1)] = pack_half2(bf16lo(w[e2]) * up, bf16hi(w[e2]) * up);
        }
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (QREG) {
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[ks][mt][e] = f[ks][e];
        } else {
          q_smem[(ks * MT + mt) * 32] = make_uint4(f[ks][0], f[ks][1], f[ks][2], f[ks][3]);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int x = 16; x > 2; x >>= 1) see_min = min(see_min, __shfl_xor_sync(0xFFFFFFFFu, see_min, x));

    float o[MT][ND][4] = {};
    AttnRow row[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) row[mt][h].start();
    int dead = -1;  // the step whose copies did not arrive in time
    for (int i = 0; i < count; ++i) {
      const uint32_t n = phase + i, st = n % STAGES;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_drain(&full[wt][st], (n / STAGES) & 1))) {
        dead = i;
        break;
      }
      const uint8_t* kt = my_ring + st * STEP;
      const uint8_t* vt = kt + 2 * TILE;

      // scores of 32 tokens: column tiles 2c, 2c + 1 are tokens 0-7 and 8-15 of block c
      float s[MT][4][4];
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const int chunk = D == 128 ? 2 * t + x : t;
        uint4 kv[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
          kv[nt] = *reinterpret_cast<const uint4*>(kt + (nt >> 1) * TILE +
                                                   tile_offset<D>(8 * (nt & 1) + g, chunk));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 f[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (QREG)
              f[mt] = make_uint4(qf[4 * x + e][mt][0], qf[4 * x + e][mt][1], qf[4 * x + e][mt][2],
                                 qf[4 * x + e][mt][3]);
            else
              f[mt] = q_smem[((4 * x + e) * MT + mt) * 32];
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const uint32_t w = word_of(kv[nt], e) ^ 0x80808080u;
            const uint32_t b0 = bytes_f16x2(w, 0x4140), b1 = bytes_f16x2(w, 0x4342);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if (x == 0 && e == 0) mma_f16_first(s[mt][nt], f[mt].x, f[mt].y, f[mt].z, f[mt].w, b0, b1);
              else mma_f16(s[mt][nt], f[mt].x, f[mt].y, f[mt].z, f[mt].w, b0, b1);
            }
          }
        }
      }

      float sk[2], sv[2], log_sv[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        seg.scales(i, c, sk[c], sv[c]);
        log_sv[c] = log2_approx(sv[c]);
      }
      const int first = (j0 + 2 * (wt + WT * i)) * kBlockTokens;
      const int last = (j0 + blocks) * kBlockTokens;
      const bool cut = first + 2 * kBlockTokens > min(see_min, last);
      // a value scale that is not finite stays with the rows that see its block
      const bool odd = cut && !(sv[0] + sv[1] < INFINITY);
      bool grow = false;
      float top[MT][2], u[MT][2], f[MT][2][2];  // f: from sums of products to scores, for each block
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 0; c < 2; ++c) f[mt][h][c] = qs[mt][h] * sk[c];
          if (cut) {
            const int end = min(see[mt][h], last);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                s[mt][nt][2 * h + e] = first + 8 * nt + 2 * t + e >= end
                                           ? -INFINITY
                                           : s[mt][nt][2 * h + e] * f[mt][h][nt >> 1];
            f[mt][h][0] = f[mt][h][1] = 1.0f;
          }
          float mx[2];
#pragma unroll
          for (int c = 0; c < 2; ++c)  // (no factor is negative)
            mx[c] = fmaxf(fmaxf(s[mt][2 * c][2 * h], s[mt][2 * c][2 * h + 1]),
                          fmaxf(s[mt][2 * c + 1][2 * h], s[mt][2 * c + 1][2 * h + 1])) * f[mt][h][c];
          top[mt][h] = fmaxf(mx[0], mx[1]);  // of my tokens; the row's only where it matters
          u[mt][h] = fmaxf(mx[0] + log_sv[0], mx[1] + log_sv[1]);
          grow |= row[mt][h].exceeded(top[mt][h], u[mt][h]);
        }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int x = 1; x < 4; x *= 2) {
              top[mt][h] = fmaxf(top[mt][h], __shfl_xor_sync(0xFFFFFFFFu, top[mt][h], x));
              u[mt][h] = fmaxf(u[mt][h], __shfl_xor_sync(0xFFFFFFFFu, u[mt][h], x));
            }
            const float fade = row[mt][h].raise(top[mt][h], u[mt][h]);
#pragma unroll
            for (int nd = 0; nd < ND; ++nd) {
              o[mt][nd][2 * h] *= fade;
              o[mt][nd][2 * h + 1] *= fade;
            }
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float base = row[mt][h].base();
          float wvs[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            wvs[c] = row[mt][h].weight(sv[c]);
            if (odd && first + 16 * c >= min(see[mt][h], last)) wvs[c] = 0.0f;
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float wv = wvs[nt >> 1];
            const float p0 = exp2_approx(fmaf(s[mt][nt][2 * h], f[mt][h][nt >> 1], -base));
            const float p1 = exp2_approx(fmaf(s[mt][nt][2 * h + 1], f[mt][h][nt >> 1], -base));
            row[mt][h].l += p0 + p1;
            s[mt][nt][2 * h] = p0 * wv;  // from scores to weights
            s[mt][nt][2 * h + 1] = p1 * wv;
          }
        }
      // o += p v.  Lane (g, t) takes 16 (8) channels of tokens 2t, 2t+1, 2t+8, 2t+9; 4 x 4
      // bytes (four tokens, four channels) give four tiles' operands
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + c * TILE + tile_offset<D>(tok, g));
            vw[k][0] = v.x; vw[k][1] = v.y; vw[k][2] = v.z; vw[k][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(
                vt + c * TILE + tile_offset<D>(tok, g >> 1) + 8 * (g & 1));
            vw[k][0] = v.x; vw[k][1] = v.y;
          }
        }
        uint32_t pf[2][MT][4];  // the weights' two parts
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* w = &s[mt][2 * c + (k >> 1)][2 * (k & 1)];
            pf[0][mt][k] = pack_half2(w[0], w[1]);
            pf[1][mt][k] = half2_rest(w[0], w[1], pf[0][mt][k]);
          }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = vw[k][w] ^ 0x80808080u;
          uint32_t f[4][2];
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              f[x][k] = bytes_f16x2(__byte_perm(v[2 * k], v[2 * k + 1], x >> 1 ? 0x7362 : 0x5140),
                                    x & 1 ? 0x4342 : 0x4140);
#pragma unroll
          for (int part = 0; part < 2; ++part)  // (a sum's two steps lie apart)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma_f16(o[mt][4 * w + x], pf[part][mt][0], pf[part][mt][1], pf[part][mt][2],
                        pf[part][mt][3], f[x][0], f[x][1]);
        }
      }
      __syncwarp();  // the stage has been read
      if (issued < count) {
        issue(issued, i);
        ++issued;
      }
      seg.next_blocks(i, a);
    }
    if (dead >= 0 && lane == 0)  // wait (bounded) for the copies in flight
      for (int i = dead; i < issued; ++i)
        mbar_wait_drain(&full[wt][(phase + i) % STAGES], ((phase + i) / STAGES) & 1);
    phase += count;

#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = row[mt][h].l;
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (t == 0) left.put(wt, 16 * mt + 8 * h + g, row[mt][h], l);
      }
    // on to the next segment: its first copies go to the stage `phase` names, this one's sums
    // to the others of the warp's own ring, whose stages have all been read
    const bool whole = seg.whole(), from_start = j0 == 0;
    const bool more = seg.advance(a, sched) && __all_sync(0xFFFFFFFFu, dead < 0);
    float* slab = reinterpret_cast<float*>(my_ring + (phase + 1) % STAGES * STEP);
    if (lane == 0) left.slab[wt] = slab;
    if (more) {
      seg.begin(a);
      if (seg.count > 0) issue(0, 0);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();  // the slabs have been read
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int nd = 0; nd < ND; nd += 4)
            *reinterpret_cast<float4*>(slab +
                                       slab_offset<D>(8 * h + g, t * (D / 4) + part * ND + nd)) =
                make_float4(o[mt][nd][2 * h + part], o[mt][nd + 1][2 * h + part],
                            o[mt][nd + 2][2 * h + part], o[mt][nd + 3][2 * h + part]);
      __syncthreads();
      attn_finish<D, RT, 16, 1>(a, sw, left, r_first, 16 * mt, head, whole, from_start);
    }
    // the next copies write where the sums were written and read by ordinary accesses
    fence_proxy_async_smem();
    if (__syncthreads_or(dead >= 0)) {  // the error word is set
      if (more && seg.count > 0 && lane == 0)
        mbar_wait_drain(&full[wt][phase % STAGES], (phase / STAGES) & 1);
      return;
    }
    if (!more) return;
  }
}

// Tiles of at most eight query rows (decoding with up to eight query heads to a cache
// head): the same work in fewer instructions, which is what bounds it.
// Scores come from the integer matrix instructions, with the cached codes as they are: q
// becomes 30-bit integers relative to its row's largest value (off by at most 2^-30 of it,
// and exact from 2^-21 of it on), four signed bytes.  For RT = 8, rows 0 to 7 of one operand
// are the highest byte, 8 to 15 the next, so that a lane holds both sums, and a second operand
// has the other two; for RT = 4, one operand has them all (rows 0 to 3 the highest, 8 to 11 the
// third, 4 to 7 the second, 12 to 15 the lowest), and a row's two lanes exchange their halves.
// Sums over the channels are exact and joined in fp32.  A lane then holds the scores of row g
// (RT = 4: g modulo 4) for tokens 2t, 2t + 1, which is the layout that the transposed product
// o^T += v^T p^T wants of p^T: half the instructions and accumulators of o += p v, of whose
// sixteen rows eight would be empty.  For RT = 4 columns 0 to 3 of p^T are the weights' first
// parts and columns 4 to 7 the second ones, at no more matrix steps.
// A step is two blocks (32 tokens): the maxima, the reference and the barrier are looked
// at once for both.  The first step of the next segment is fetched while this one's sums
// are joined (in the other stage of each warp's ring).
// Long contexts are bound by memory, after about 10 us of start, segments' ends and joining:
// one token each, four query heads to a cache head of 128: 32 sequences of up to 8192 tokens
// 61.6 us, 5.1 TB/s; 2 of up to 131072 71.5 us, 5.2 TB/s; 8 of 131072 reach 6.2 TB/s.  A single
// sequence of up to 500 tokens, 16 heads, takes 9.4 us, all of it latency.  (The first, simple
// kernel: 84.0, 87.6 and 11.1 us; before weights had a second part and rows a reference of their
// own: 61.0, 71.3 and 9.0 us.)  Eight query heads to a cache head, 16 sequences of up to 8192
// tokens, four heads of 128: 27.9 us, 2.5 TB/s.
template <int D, int RT_>
struct AttnFewCfg {
  static constexpr int RT = RT_, WT = kAttnWarps, TILE = kBlockTokens * D;
  static constexpr int STEP = 4 * TILE;               // two blocks of keys and values
  static constexpr int STAGES = 2;
  static constexpr int RING = WT * STAGES * STEP;
  static constexpr int SMEM = RING + 1024;            // + alignment
  static constexpr int CTAS = D == 128 ? 3 : 4;
  static_assert(8 * D * 4 <= STEP, "a warp's sums, in eight columns, fit one stage");
};

template <int D, int RT_>
__global__ void __launch_bounds__(32 * kAttnWarps, AttnFewCfg<D, RT_>::CTAS) attn_kv8_few_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const AttnArgs a) {
  using C = AttnFewCfg<D, RT_>;
  constexpr int WT = C::WT, RT = C::RT, STAGES = C::STAGES, TILE = C::TILE, STEP = C::STEP;
  constexpr int KS = D / 32;   // matrix steps over the channels
  constexpr int MD = D / 16;   // 16-channel tiles of the transposed output
  constexpr bool FOUR = RT == 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[WT][STAGES];
  __shared__ AttnRows<RT> left;
  __shared__ AttnSched sched;

  const int wt = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.q_heads / a.kv_heads;
  uint8_t* my_ring = ring + wt * STAGES * STEP;

  if (threadIdx.x == 0) {
    for (int i = 0; i < WT; ++i)
      for (int s = 0; s < STAGES; ++s) mbar_init(&full[i][s], 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();
  griddep_launch_dependents();
  const AttnShare share = attn_share<RT>(a, sched);
  if (share.begin >= share.end) return;

  uint32_t phase = 0;  // steps this warp has taken before this segment (stage and parity)
  AttnSegment<RT> seg(a, share, wt, lane);
  auto issue = [&](int i, int consumed) {  // copies of my step i: two lanes, a block each
    const int copy_row = seg.copy_row(i, consumed, lane);
    const uint32_t st = (phase + i) % STAGES;
    attn_copy<TILE>(my_ring + st * STEP, &tm_k, &tm_v, &full[wt][st], copy_row, lane);
  };
  seg.begin(a);
  if (seg.count > 0) issue(0, 0);

  for (;;) {
    const int count = seg.count, j0 = seg.j0, blocks = seg.blocks, head = seg.head, r_first = seg.r_first;
    const SeqWork sw = seg.sw;
    int issued = min(count, 1);
    for (; issued < min(count, STAGES); ++issued) issue(issued, 0);

    // my row
    const int r = r_first + (FOUR ? g & 3 : g);
    const bool valid = r < sw.nq * G;
    const int qi = valid ? r / G : 0, qh = head * G + (valid ? r % G : 0);
    const int see = valid && a.causal ? sw.len - sw.nq + qi + 1 : sw.len;
    int see_min = see;
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) see_min = min(see_min, __shfl_xor_sync(0xFFFFFFFFu, see_min, o));

    // its q as digits; channel 32t + 8s + 0..7 (D = 128; 16t + 8s for D = 64) of a row is
    // what lane t holds of a key for matrix step s
    uint32_t qa[KS][4], ql[FOUR ? 1 : KS][4];  // RT = 8: bytes 3, 2, 3, 2; 1, 0, 1, 0
    float qs;                                  // undoes the power-of-two scaling, times the softmax scale
    {
      uint4 raw[KS];
#pragma unroll
      for (int i = 0; i < KS; ++i)
        raw[i] = valid ? *reinterpret_cast<const uint4*>(a.q + (sw.q0 + qi) * a.q_stride +
                                                         static_cast<long long>(qh) * D + t * (D / 4) + 8 * i)
                       : make_uint4(0, 0, 0, 0);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = max_or_nan(top, max_or_nan(fabsf(bf16lo(w[e])), fabsf(bf16hi(w[e]))));
      }
      top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const uint32_t ex = max(__float_as_uint(top) >> 23, 29u);
      // 2^(29 - E), 2^E <= top < 2^(E + 1), with the softmax scale's sign
      const float up = copysignf(__uint_as_float((283u - ex) << 23), a.scale_log2);
      qs = row_factor(ex, 29u, a.scale_log2);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = (e & 1 ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1])) * up;
          d[e] = (static_cast<uint32_t>(__float2int_rn(v)) + 0x00808080u) ^ 0x00808080u;
        }
        const uint32_t upper = FOUR && g >= 4 ? 2u : 3u;  // (RT = 4: bytes 3, 1 or 2, 0)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          auto bytes = [&](uint32_t byte) {
            return gather_bytes(d[4 * h], d[4 * h + 1], d[4 * h + 2], d[4 * h + 3], byte);
          };
          qa[i][2 * h] = bytes(upper);
          qa[i][2 * h + 1] = bytes(FOUR ? upper - 2 : 2);
          if constexpr (!FOUR) {
            ql[i][2 * h] = bytes(1);
            ql[i][2 * h + 1] = bytes(0);
          }
        }
      }
    }

    // channels (D / 8) g + 2 i and + 1, queries 2t and 2t + 1; RT = 4: queries modulo 4, from
    // the weights' first parts (columns 0 to 3) and second ones
    float o[MD][4] = {};
    AttnRow row;
    row.start();
    int dead = -1;  // the step whose copies did not arrive in time
    for (int i = 0; i < count; ++i) {
      const uint32_t n = phase + i, st = n % STAGES;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_drain(&full[wt][st], (n / STAGES) & 1))) {
        dead = i;
        break;
      }
      const uint8_t* kt = my_ring + st * STEP;
      const uint8_t* vt = kt + 2 * TILE;
      float sv[2], f[2];  // f: from sums of products to scores, not negative
      float s[2][2][2];   // [block][tile of 8 tokens][token 2t, 2t + 1]
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sk;
        seg.scales(i, c, sk, sv[c]);
        f[c] = qs * sk;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          int hm[4], lo[4];
#pragma unroll
          for (int x = 0; x < KS / 2; ++x) {
            const int chunk = D == 128 ? 2 * t + x : t;
            const uint4 kv =
                *reinterpret_cast<const uint4*>(kt + c * TILE + tile_offset<D>(8 * nt + g, chunk));
            mma_s8(hm, qa[2 * x], kv.x, kv.y, x == 0);
            mma_s8(hm, qa[2 * x + 1], kv.z, kv.w, false);
            if constexpr (!FOUR) {
              mma_s8(lo, ql[2 * x], kv.x, kv.y, x == 0);
              mma_s8(lo, ql[2 * x + 1], kv.z, kv.w, false);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (FOUR) {
              const float half = fmaf(static_cast<float>(hm[e]), 65536.0f,
                                      static_cast<float>(hm[2 + e])) * (g < 4 ? 256.0f : 1.0f);
              s[c][nt][e] = half + __shfl_xor_sync(0xFFFFFFFFu, half, 16);
            } else {
              s[c][nt][e] = fmaf(static_cast<float>(hm[e] * 256 + hm[2 + e]), 65536.0f,
                                 static_cast<float>(lo[e] * 256 + lo[2 + e]));
            }
          }
        }
      }
      const int first = (j0 + 2 * (wt + WT * i)) * kBlockTokens;
      const int end = min(see, (j0 + blocks) * kBlockTokens);
      const bool cut = first + 2 * kBlockTokens > min(see_min, (j0 + blocks) * kBlockTokens);
      // a value scale that is not finite stays with the rows that see its block
      const bool odd = cut && !(sv[0] + sv[1] < INFINITY);
      if (cut) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[c][nt][e] = first + 16 * c + 8 * nt + 2 * t + e >= end ? -INFINITY : s[c][nt][e] * f[c];
        f[0] = f[1] = 1.0f;
      }
      float mx[2];  // of my tokens; the row's only where it matters
#pragma unroll
      for (int c = 0; c < 2; ++c)
        mx[c] = fmaxf(fmaxf(s[c][0][0], s[c][0][1]), fmaxf(s[c][1][0], s[c][1][1])) * f[c];
      float top = fmaxf(mx[0], mx[1]);
      float u = fmaxf(mx[0] + log2_approx(sv[0]), mx[1] + log2_approx(sv[1]));
      if (__any_sync(0xFFFFFFFFu, row.exceeded(top, u))) {
#pragma unroll
        for (int x = 1; x < 4; x *= 2) {
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
          u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, x));
        }
        const float fade = row.raise(top, u);
        if (i > 0) {  // (at the first step nothing has been summed)
          const float f0 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t);
          const float f1 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t + 4);
#pragma unroll
          for (int x = 0; x < MD; ++x) {
            o[x][0] *= f0; o[x][1] *= f1; o[x][2] *= f0; o[x][3] *= f1;
          }
        }
      }
      const float base = row.base();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float wv = row.weight(sv[c]);
        if (odd && first + 16 * c >= end) wv = 0.0f;
        uint32_t pf[2], rest[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float p0 = exp2_approx(fmaf(s[c][nt][0], f[c], -base));
          const float p1 = exp2_approx(fmaf(s[c][nt][1], f[c], -base));
          row.l += p0 + p1;
          const float w0 = p0 * wv, w1 = p1 * wv;
          pf[nt] = pack_half2(w0, w1);
          rest[nt] = half2_rest(w0, w1, pf[nt]);
          if (FOUR && g >= 4) pf[nt] = rest[nt];
        }
        // values: lane (g, t) takes 16 (8) channels of tokens 2t, 2t+1, 2t+8, 2t+9
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + c * TILE + tile_offset<D>(tok, g));
            vw[k][0] = v.x; vw[k][1] = v.y; vw[k][2] = v.z; vw[k][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(
                vt + c * TILE + tile_offset<D>(tok, g >> 1) + 8 * (g & 1));
            vw[k][0] = v.x; vw[k][1] = v.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = vw[k][w] ^ 0x80808080u;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x0 = __byte_perm(v[0], v[1], half ? 0x7362 : 0x5140);
            const uint32_t x1 = __byte_perm(v[2], v[3], half ? 0x7362 : 0x5140);
            const uint32_t f0 = bytes_f16x2(x0, 0x4140), f1 = bytes_f16x2(x0, 0x4342);
            const uint32_t f2 = bytes_f16x2(x1, 0x4140), f3 = bytes_f16x2(x1, 0x4342);
            mma_f16(o[2 * w + half], f0, f1, f2, f3, pf[0], pf[1]);
            if constexpr (!FOUR) mma_f16(o[2 * w + half], f0, f1, f2, f3, rest[0], rest[1]);
          }
        }
      }
      __syncwarp();  // the stage has been read
      if (issued < count) {
        issue(issued, i);
        ++issued;
      }
      seg.next_blocks(i, a);
    }
    if (dead >= 0 && lane == 0)  // wait (bounded) for the copies in flight
      for (int i = dead; i < issued; ++i)
        mbar_wait_drain(&full[wt][(phase + i) % STAGES], ((phase + i) / STAGES) & 1);
    phase += count;

    float l = row.l;
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    if (t == 0 && g < RT) left.put(wt, g, row, l);
    // on to the next segment: its first copies go to the stage `phase` names, this one's
    // sums to the other (of the warp's own ring, whose stages have all been read)
    const bool whole = seg.whole(), from_start = j0 == 0;
    const bool more = seg.advance(a, sched) && __all_sync(0xFFFFFFFFu, dead < 0);
    float* slab = reinterpret_cast<float*>(my_ring + (phase + 1) % STAGES * STEP);
    if (more) {
      seg.begin(a);
      if (seg.count > 0) issue(0, 0);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 0; x < MD; x += 2)
        *reinterpret_cast<float4*>(slab + slab_offset<D>(2 * t + e, g * (D / 8) + 2 * x)) =
            make_float4(o[x][e], o[x][2 + e], o[x + 1][e], o[x + 1][2 + e]);
    if (lane == 0) left.slab[wt] = slab;
    __syncthreads();
    attn_finish<D, RT, RT, FOUR ? 2 : 1>(a, sw, left, r_first, 0, head, whole, from_start);
    // the next copies write where the sums were written and read by ordinary accesses
    fence_proxy_async_smem();
    if (__syncthreads_or(dead >= 0)) {  // the error word is set
      if (more && seg.count > 0 && lane == 0)
        mbar_wait_drain(&full[wt][phase % STAGES], (phase / STAGES) & 1);
      return;
    }
    if (!more) return;
  }
}

// Joins the partial results of items that several CTAs shared.  Such an item has a CTA's
// end inside it: four CTAs of this kernel (twelve for tiles of 32 rows of 128 channels) look
// at the end of each CTA of the first one, and all that look at ends inside one item share its
// outputs among them.  As many lanes as there are parts (a power of two, at most a warp) take
// one four of outputs, so that every load is in flight at once; they are added as a tree, the
// same every time.  Latency bounds it: with one thread to an output, its parts one after the
// other, 2 x 131072 tokens took 83.9 us in all instead of 73.  Sixteen CTAs to an end of tiles
// of 32 rows of 64 channels: 69 us for two chunks of 64 queries instead of 64 with four; four to
// those of 128 channels 104 instead of 101 with twelve.
constexpr int join_split(int RT, int D) { return RT * D >= 4096 ? 12 : 4; }

template <int D>
__global__ void __launch_bounds__(128) attn_kv8_join_kernel(const AttnArgs a, int RT) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, split = join_split(RT, D);
  const AttnCut cut = a.cuts[blockIdx.x / split];
  if (cut.ends == 0) return;
  const int G = a.q_heads / a.kv_heads;
  const int c0 = cut.c0, c1 = c0 + cut.ends;
  const long long size = static_cast<long long>(RT) * (D + 2);
  int lanes = 2;  // to an output
  while (lanes < 32 && lanes <= c1 - c0) lanes *= 2;
  // my piece of the outputs, in fours
  const int all = cut.rows * (D / 4), pieces = cut.ends * split;
  const int my = blockIdx.x - c0 * split, end = all * (my + 1) / pieces;
  for (int base = all * my / pieces; base < end; base += 128 / lanes) {
    const int i = min(base + static_cast<int>(threadIdx.x) / lanes, end - 1);
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    float top = -INFINITY, sum = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
    for (int c = c0 + lane % lanes; c <= c1; c += lanes) {
      const float* p = a.partial + (2LL * c + (c == c0 ? 1 : 0)) * size;
      const float2 ml = *reinterpret_cast<const float2*>(p + RT * D + 2 * r);
      const float4 x = *reinterpret_cast<const float4*>(p + r * D + d);
      if (ml.y == 0.0f) continue;  // an empty part
      const float to = fmaxf(top, ml.x);
      const float f = exp2_approx(top - to), e = exp2_approx(ml.x - to);
      sum = sum * f + ml.y * e;
      v.x = v.x * f + x.x * e; v.y = v.y * f + x.y * e;
      v.z = v.z * f + x.z * e; v.w = v.w * f + x.w * e;
      top = to;
    }
    float all_top = top;
    for (int o = lanes / 2; o > 0; o >>= 1)
      all_top = fmaxf(all_top, __shfl_xor_sync(0xFFFFFFFFu, all_top, o));
    const float f = top == -INFINITY ? 0.0f : exp2_approx(top - all_top);
    top = all_top;
    sum *= f;
    v.x *= f; v.y *= f; v.z *= f; v.w *= f;
    for (int o = lanes / 2; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
      v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
      v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, o);
      v.w += __shfl_xor_sync(0xFFFFFFFFu, v.w, o);
    }
    if (lane % lanes != 0 || base + static_cast<int>(threadIdx.x) / lanes >= end) continue;
    const float inv = sum > 0.0f ? kOutUnit / sum : 0.0f;
    const int qi = (cut.r_first + r) / G, qh = cut.head * G + (cut.r_first + r) % G;
    const long long at = static_cast<long long>(cut.q0 + qi) * a.q_heads + qh;
    const __nv_bfloat162 x0 = __floats2bfloat162_rn(v.x * inv, v.y * inv);
    const __nv_bfloat162 x1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(a.out + at * D + d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1));
    if (a.lse && d == 0)
      a.lse[at] = sum == 0.0f ? -INFINITY : (top - kPShift + log2f(sum)) * 0.69314718055994531f;
  }
}

// ------------------------------------------------------------ host side

// Rows of a tile, by the rows per cache head that an average sequence has: 4 or 8 (their
// own kernel), 16 or 32.  (64 rows on pairs of warps that shared their copies lost to two
// tiles of 32 everywhere: 57.9 / 54.4 us for chunks of 64 over 8512 tokens, heads of 64, with
// weights of one part.)
int attn_tile_rows(int Tq, int B, int q_heads, int kv_heads) {
  const long long rows = static_cast<long long>(Tq) * (q_heads / kv_heads);
  return rows <= 4LL * B ? 4 : rows <= 8LL * B ? 8 : rows <= 16LL * B ? 16 : 32;
}

// Whether items are left whole, one CTA each, and the joining kernel is not launched: where
// the tables have room for few tokens, or for not many and there are items for every SM.
// Measured whole / cut, us: 16 items of at most 512 tokens 9.4 / 9.6, 512 of them 23.1 / 36.1;
// 512 of at most 1024 tokens 33.3 / 37.6, but 8 of them 13.6 / 10.1; 512 of at most 2048,
// heads of 64 28.4 / 37.1, of 128 54.7 / 48.8.
bool attn_whole(const Kv8Cache& c, int Tq, int q_heads, int RT) {
  const long long tokens = static_cast<long long>(c.max_pages) * c.page_tokens;
  const long long rows = static_cast<long long>(Tq) * (q_heads / c.kv_heads);
  return tokens <= 512 || (tokens * c.D <= 131072 && rows / RT * c.kv_heads >= sm_count());
}

constexpr int kAttnMaxCtas = 4;  // per SM, of any instance

size_t attn_cut_bytes(size_t grid) { return (grid * sizeof(AttnCut) + 255) / 256 * 256; }

bool cache_map(CUtensorMap* m, const void* base, int D, long long rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(D), kBlockTokens};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Kernel>
cudaError_t run_attn(Kernel kernel, std::atomic<bool> (&done)[kAttrDevices], int smem, int ctas,
                     const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a, int D,
                     int RT, cudaStream_t st) {
  const cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int grid = sm_count() * ctas;
  const cudaError_t f = launch_pdl(kernel, grid, 32 * kAttnWarps, smem, st, 1, tm_k, tm_v, a);
  if (f != cudaSuccess || a.whole) return f;
  return launch_pdl(D == 128 ? attn_kv8_join_kernel<128> : attn_kv8_join_kernel<64>,
                    (grid - 1) * join_split(RT, D), 128, 0, st, 1, a, RT);
}

template <int D>
cudaError_t dispatch_attn(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a,
                          int RT, cudaStream_t st) {
  static std::atomic<bool> done[4][kAttrDevices];
#define WQ_ATTN(I_, CFG_, KERNEL_) \
  return run_attn(KERNEL_, done[I_], CFG_::SMEM, CFG_::CTAS, tm_k, tm_v, a, D, RT, st)
  using C16 = AttnCfg<D, 1>;
  using C32 = AttnCfg<D, 2>;
  using C4 = AttnFewCfg<D, 4>;
  using C8 = AttnFewCfg<D, 8>;
  if (RT == 4) WQ_ATTN(0, C4, (attn_kv8_few_kernel<D, 4>));
  if (RT == 8) WQ_ATTN(1, C8, (attn_kv8_few_kernel<D, 8>));
  if (RT == 16) WQ_ATTN(2, C16, (attn_kv8_kernel<D, 1>));
  WQ_ATTN(3, C32, (attn_kv8_kernel<D, 2>));
#undef WQ_ATTN
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Append& p, cudaStream_t st) {
  AppendArgs a;
  a.x[0] = p.k; a.x[1] = p.v;
  a.stride[0] = p.k_stride; a.stride[1] = p.v_stride;
  a.row_start = p.row_start; a.past_len = p.past_len; a.table = p.cache.table;
  a.codes[0] = p.cache.k_codes; a.codes[1] = p.cache.v_codes;
  a.scale[0] = p.cache.k_scale; a.scale[1] = p.cache.v_scale;
  a.T = p.T; a.B = p.cache.B; a.max_pages = p.cache.max_pages; a.pages = p.cache.pages;
  a.heads = p.cache.kv_heads; a.page_tokens = p.cache.page_tokens;
  a.page_shift = a.page_tokens == 16 ? 4 : a.page_tokens == 32 ? 5 : a.page_tokens == 64 ? 6 : 7;
  a.window = p.T > 16LL * a.B ? 16 : 1;
  const long long windows = (p.T + a.window - 1) / a.window;
  const int grid = static_cast<int>((windows * a.heads * 2 + 3) / 4);
  return p.cache.D == 128 ? launch_pdl(kv8_append_kernel<128>, grid, 128, 0, st, 1, a)
                          : launch_pdl(kv8_append_kernel<64>, grid, 128, 0, st, 1, a);
}

size_t attn_workspace_bytes(int Tq, int B, int q_heads, int kv_heads, int D) {
  const size_t rt = attn_tile_rows(Tq, B, q_heads, kv_heads);
  const size_t grid = static_cast<size_t>(sm_count()) * kAttnMaxCtas;
  return attn_cut_bytes(grid) + (grid * 2 * rt * (D + 2) * 4 + 255) / 256 * 256;
}

cudaError_t launch_attn_kv8(const Kv8Attn& p, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.cache.pages) * p.cache.kv_heads * p.cache.page_tokens;
  CUtensorMap tm_k, tm_v;
  if (!cache_map(&tm_k, p.cache.k_codes, p.cache.D, rows) ||
      !cache_map(&tm_v, p.cache.v_codes, p.cache.D, rows))
    return cudaErrorInvalidValue;
  AttnArgs a;
  a.q = p.q; a.q_stride = p.q_stride; a.q_start = p.q_start; a.kv_len = p.kv_len;
  a.table = p.cache.table; a.k_scale = p.cache.k_scale; a.v_scale = p.cache.v_scale;
  a.out = p.out; a.lse = p.lse;
  a.cuts = static_cast<AttnCut*>(p.workspace);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) +
                                       attn_cut_bytes(static_cast<size_t>(sm_count()) * kAttnMaxCtas));
  a.Tq = p.Tq; a.B = p.cache.B; a.q_heads = p.q_heads; a.kv_heads = p.cache.kv_heads;
  a.max_pages = p.cache.max_pages; a.pages = p.cache.pages; a.page_tokens = p.cache.page_tokens;
  a.causal = p.causal; a.scale_log2 = p.scale * 1.4426950408889634f;
  const int rt = attn_tile_rows(p.Tq, p.cache.B, p.q_heads, p.cache.kv_heads);
  a.whole = attn_whole(p.cache, p.Tq, p.q_heads, rt);
  return p.cache.D == 128 ? dispatch_attn<128>(tm_k, tm_v, a, rt, st)
                          : dispatch_attn<64>(tm_k, tm_v, a, rt, st);
}

}  // namespace wq
