// moe_decode.cu -- the routed experts of a few tokens on NVFP4 weights: matrix-vector
// products instead of dispatch and padded GEMM tiles.
//
//   h[t,j]  = silu(G) * U,  (G, U) = w13_scale[e] * W13[e] x[t],   e = ids[t,j]
//   y[t]    = sum_j scores[t,j] * w2_scale[e] * W2[e] h[t,j]       (fixed j order)
//
// The weights are the prepared ones of moe_forward_nvfp4 (E2M1 codes, tiled E4M3
// scales per 16 elements); the activations are not quantised: x stays bf16, h is
// kept in fp32 and read by the second product as fp16, all sums are fp32.
//
// Bound by reading each chosen expert once: 3/2 d I codes and 3/16 d I scales.  The work
// is cut into units of 32 rows of one expert's matrix for up to 8 of its tokens:
//   one token (k <= 8)   a W13 unit a CTA, K split over its warps; W2 with a warp an
//                        expert, which adds the experts itself: two launches
//   a few units          a unit a CTA, K split over its warps
//   many units           a unit a warp, weights streamed through a ring in shared memory
// and the last two end with a third launch that adds a token's experts.
// Measured at d=2048, I=768, k=8 (bytes at the rate of a plain copy): 1 token on 128
// experts 12.2 us (3.1), 7 tokens on 16 experts 21.0 (6.2), 64 tokens on 128 experts
// 72.2 (49.4).  Up to the last it is bound by the latency of a launch's start (ids, the
// plan, the tokens' rows, the first weights: some 6 us, twice); the last streams near the
// memory's rate between its two starts.
//
// The product runs on mma.sync m16n8k16 with the weights as the 16-row operand and up to
// 8 tokens as the columns: one token fills one column of eight, but a weight then costs
// half a conversion (cvt.e2m1x2), half a multiplication by its block's scale and no
// accumulation of its own, where per-lane fused multiply-adds cost one and a half
// instructions a weight and token.  (tcgen05 takes its operands from shared memory and
// would need the dequantised weights written there.)  Rounding: E2M1 x E4M3 has at most
// six significant bits and is exact in fp16; a token's x is scaled by a power of two that
// takes its largest element to the top of fp16's range, which is exact down to 2^-31 of
// that element and errs below by at most 2^-39 of it; h, scaled the same way, loses what
// lies beyond fp16's 11 bits, eight times finer than the bf16 h of the other paths.
//
// Operand layout.  Any order of K serves as long as both operands share it: lane
// (g, q) = (lane / 4, lane % 4) loads 16 code bytes (32 elements, two scale blocks)
// of each of its four rows with one instruction, and the eight MMAs of a step take
// four of those elements each.  Rows 8s+g, +32, +64, +96 of a 128-row scale block
// share one 16-byte piece of the tiled scales; for W13 the first two are gate rows
// and the last two the up rows of the same columns, so a lane's accumulators hold
// whole (gate, up) pairs.

#include <climits>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kStep = 128;              // K elements per warp step
constexpr int kCols = 8;                // tokens per pass (MMA columns)
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t word, int byte) {
  uint32_t r;
  switch (byte) {
    case 0:
      asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;}"
          : "=r"(r) : "r"(word));
      break;
    case 1:
      asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;}"
          : "=r"(r) : "r"(word));
      break;
    case 2:
      asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;}"
          : "=r"(r) : "r"(word));
      break;
    default:
      asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;}"
          : "=r"(r) : "r"(word));
  }
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A power of two that takes `amax` (finite) into [2^14, 2^15), as far as fp32
// holds it, and its inverse.
__device__ __forceinline__ void pow2_scale(float amax, float& mul, float& inv) {
  const int e = (int)(__float_as_uint(amax) >> 23);         // amax >= 0
  int s = 268 - e;
  s = s < 1 ? 1 : (s > 254 ? 254 : s);
  mul = __uint_as_float((uint32_t)s << 23);
  inv = s == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - s) << 23);
}

// One lane's operands of a step: 16 code bytes of each of its four rows, and the
// scale words of the four rows (blocks of its half K group).
struct StepA {
  uint4 c[4];
  uint4 s;
};

// Where they are: the lane's bytes of step 0 in its first row, its scales.  The
// second row is `gap` bytes further, the third and fourth `far` beyond those.
struct Rows {
  const uint8_t* code;
  const uint8_t* scale;
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void load_step(const Rows& r, long long gap, long long far, int step,
                                          StepA& a) {
  const uint8_t* p = r.code + step * (kStep / 2);
  a.c[0] = ldg_stream(p);
  a.c[1] = ldg_stream(p + gap);
  a.c[2] = ldg_stream(p + far);
  a.c[3] = ldg_stream(p + far + gap);
  a.s = ldg_stream(r.scale + step * 1024);
}

// acc[..][tile] += (dequantised rows) . (the tokens' step at `xs`, the lane's piece
// of its token; absent tokens are zero).  Two sums per tile: an MMA waits some 50
// cycles for the one before it in its sum.
__device__ __forceinline__ void mma_step(const StepA& a, int half, const uint8_t* xs, bool have,
                                         float (&acc)[2][2][4]) {
  const uint32_t sw[4] = {a.s.x, a.s.y, a.s.z, a.s.w};
  uint32_t code[4][4], s0[4], s1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    code[i][0] = a.c[i].x; code[i][1] = a.c[i].y; code[i][2] = a.c[i].z; code[i][3] = a.c[i].w;
    uint32_t h;
    const uint16_t two = (uint16_t)(sw[i] >> half);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    s0[i] = __byte_perm(h, h, 0x1010);
    s1[i] = __byte_perm(h, h, 0x3232);
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if (have) b = *reinterpret_cast<const uint4*>(xs + w * 64);
    uint32_t f[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        f[i][p] = mul_f16x2(e2m1x2_to_f16x2(code[i][w], p), w < 2 ? s0[i] : s1[i]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mma_f16(acc[0][t], f[2 * t][0], f[2 * t + 1][0], f[2 * t][1], f[2 * t + 1][1], b.x, b.y);
      mma_f16(acc[1][t], f[2 * t][2], f[2 * t + 1][2], f[2 * t][3], f[2 * t + 1][3], b.z, b.w);
    }
  }
}

struct DecodeArgs {
  const uint16_t* x;          // [T, d] bf16
  const int32_t* ids;         // [T, k]
  const float* scores;        // [T, k]
  int T, k, d, I, E;
  int cols;                   // tokens per pass
  float clamp;
  const uint8_t *codes, *sf;  // this launch's matrix
  const float* w_scale;
  float* h;                   // [T*k, I]
  float* ys;                  // [T*k, d]
  uint8_t* keep;              // [T*k] 1: the pair counts (valid id, first in its row)
  uint16_t* y;                // [T, d]
  DevError* err;
};

// A unit is 32 rows of one chosen expert's matrix (a row set) for one pass of its
// tokens (up to a.cols of them); the units are numbered pass by pass, expert by
// expert, and every CTA takes a run of them.  Both are found anew by every CTA from
// the ids alone: a thread per expert counts, and one scan numbers.
struct Plan {
  int2 warp_sums[kThreads / 32];
  int count[kThreads];        // tokens by expert (E <= 256), later the end of its pairs
  int start[kThreads];        // its first pair in the list
  int expert, first, tokens;  // the pass that find_pass() looked for
};

// What a thread keeps: of expert threadIdx.x < 256, and the id of pair threadIdx.x.
struct Mine {
  int passes, before;         // its passes, and those of the experts ahead
  int start, tokens;          // its pairs in the list
  int id;
};

// Bytes of a token's row of K fp16 elements in shared memory: 64 more than the row,
// so that the eight lanes of a quarter-warp load from different banks.
__host__ __device__ constexpr int row_bytes(int K) { return 2 * K + 64; }
// Bytes of the pairs' list and of its unordered form.
__host__ __device__ constexpr int list_bytes(int pairs) { return (4 * pairs + 127) / 128 * 128; }

// True for an id that repeats an earlier one of its row.
__device__ __forceinline__ bool repeated(const DecodeArgs& a, int p) {
  const int e = a.ids[p];
  bool same = false;
#pragma unroll 8
  for (int i = p / a.k * a.k; i < p; ++i) same |= a.ids[i] == e;     // independent loads
  return same;
}

// Counts and numbers; returns the number of passes.  All threads call it; the list is
// complete after fill_list() and a __syncthreads().
__device__ __forceinline__ int make_plan(const DecodeArgs& a, Plan& s, Mine& m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  m = Mine{0, 0, 0, 0, -1};
  for (int p = threadIdx.x; p < a.T * a.k; p += blockDim.x) {
    const int e = a.ids[p];
    if (p == threadIdx.x) m.id = e;
    if (e >= 0 && e < a.E) atomicAdd(&s.count[e], 1);
  }
  __syncthreads();
  int2 sum = make_int2(0, 0);                        // inclusive over the warp's experts
  if (threadIdx.x < kThreads) {
    m.tokens = s.count[threadIdx.x];
    m.passes = (m.tokens + a.cols - 1) / a.cols;
    sum = make_int2(m.passes, m.tokens);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
      if (lane >= o) sum.x += x, sum.y += y;
    }
    if (lane == 31) s.warp_sums[warp] = sum;
  }
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 v = s.warp_sums[w];
    if (w < warp) sum.x += v.x, sum.y += v.y;
    all += v.x;
  }
  if (threadIdx.x < kThreads) {
    m.before = sum.x - m.passes;
    m.start = sum.y - m.tokens;
    s.count[threadIdx.x] = s.start[threadIdx.x] = m.start;
  }
  return all;
}

// The pairs t*k+j by expert, ascending, into `list` (complete after the next
// __syncthreads(); `raw`: as long): every CTA has to come to the same passes.  A pair
// that repeats an id of its row is computed too, and dropped where the tokens'
// experts are added.  All threads call it.
__device__ __forceinline__ void fill_list(const DecodeArgs& a, Plan& s, const Mine& m,
                                          uint16_t* list, uint16_t* raw) {
  for (int p = threadIdx.x; p < a.T * a.k; p += blockDim.x) {
    const int e = p == threadIdx.x ? m.id : a.ids[p];
    if (e >= 0 && e < a.E) raw[atomicAdd(&s.count[e], 1)] = (uint16_t)p;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.T * a.k; p += blockDim.x) {
    const int e = p == threadIdx.x ? m.id : a.ids[p];
    if (e < 0 || e >= a.E) continue;
    int at = s.start[e];
    const int first = at, end = s.count[e];
    for (int i = first; i < end; ++i) at += raw[i] < p;
    list[at] = (uint16_t)p;
  }
}

// The expert of pass `pass`, its first pair in the list and its tokens, for all
// threads after a __syncthreads().
__device__ __forceinline__ void find_pass(const DecodeArgs& a, Plan& s, const Mine& m, int pass) {
  const int n = pass - m.before;
  if (n >= 0 && n < m.passes) {
    s.expert = threadIdx.x;
    s.first = m.start + n * a.cols;
    s.tokens = min(a.cols, m.tokens - n * a.cols);
  }
}

// This CTA's run of `total` units.
__device__ __forceinline__ int2 run_of(int total) {
  const unsigned n = gridDim.x, b = blockIdx.x, q = (unsigned)total / n, r = total - q * n;
  const int from = (int)(b * q + min(b, r));
  return make_int2(from, from + (int)(q + (b < r ? 1u : 0u)));
}

// Eight consecutive activations as they are in memory.
struct PieceX { uint4 v; };
struct PieceH { float4 v[2]; };
__device__ __forceinline__ void load_piece(const uint16_t* p, PieceX& r) {
  r.v = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load_piece(const float* p, PieceH& r) {
  r.v[0] = __ldcg(reinterpret_cast<const float4*>(p));
  r.v[1] = __ldcg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void unpack(const PieceX& r, float (&f)[8]) {
  const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const PieceH& r, float (&f)[8]) {
  f[0] = r.v[0].x; f[1] = r.v[0].y; f[2] = r.v[0].z; f[3] = r.v[0].w;
  f[4] = r.v[1].x; f[5] = r.v[1].y; f[6] = r.v[1].z; f[7] = r.v[1].w;
}

template <bool W13>
struct PieceOf;
template <>
struct PieceOf<true> {
  using type = PieceX;
  static __device__ const uint16_t* row(const DecodeArgs& a, int pair) {
    return a.x + (long long)(pair / a.k) * a.d;
  }
};
template <>
struct PieceOf<false> {
  using type = PieceH;
  static __device__ const float* row(const DecodeArgs& a, int pair) {
    return a.h + (long long)pair * a.I;
  }
};

// The staged tokens of a pass.
struct Tokens {
  unsigned amax[kCols];       // of a token's row, as bits
  float inv[kCols];           // inverse of its scale
  int pair[kCols];
  float score[kCols];
};

// The rows of the pass's `nt` tokens as fp16 scaled by a power of two per token, each
// step's 16 pieces of 8 elements in the order of mma_step: piece 4q+w at 64 w + 16 q.
// Called by all threads; a group of eight warps stages one pass (nt = 0: none), a
// token taking as many warps as there are for it and a lane keeping up to KEPT of its
// pieces between the search for the largest element and the conversion.  The rows are
// complete after the next __syncthreads().
template <bool W13, int KEPT>
__device__ __forceinline__ void stage_tokens(const DecodeArgs& a, Tokens& s, uint8_t* xs,
                                             const uint16_t* list, int nt) {
  using Piece = typename PieceOf<W13>::type;
  const int warp = threadIdx.x >> 5 & 7, lane = threadIdx.x & 31, K = W13 ? a.d : a.I;
  const int share = nt > 4 ? 1 : nt > 2 ? 2 : nt > 1 ? 4 : 8;    // warps of a token
  const int c = warp / share, per = K / 8, hop = 32 * share;
  const int first = lane + 32 * (warp - c * share);
  if ((threadIdx.x & 255) < kCols) s.amax[threadIdx.x & 255] = 0u;
  __syncthreads();
  const bool mine = c < nt;
  const int pair = mine ? list[c] : 0;
  const auto* src = PieceOf<W13>::row(a, pair);
  Piece kept[KEPT];
  float f[8];
  if (mine) {
    float m = 0.f;
    auto largest = [&](const Piece& p) {
      unpack(p, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    };
#pragma unroll
    for (int n = 0; n < KEPT; ++n)
      if (first + n * hop < per) load_piece(src + (first + n * hop) * 8, kept[n]);
    if (first == 0) {
      s.pair[c] = pair;
      if (!W13) s.score[c] = a.scores[pair];
    }
#pragma unroll
    for (int n = 0; n < KEPT; ++n)
      if (first + n * hop < per) largest(kept[n]);
    for (int i = first + KEPT * hop; i < per; i += hop) {
      Piece p;
      load_piece(src + i * 8, p);
      largest(p);
    }
    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (lane == 0) atomicMax(&s.amax[c], top);
  }
  __syncthreads();
  if (!mine) return;
  float mul, inv;
  pow2_scale(__uint_as_float(s.amax[c]), mul, inv);
  if (first == 0) s.inv[c] = inv;
  uint8_t* const to = xs + c * row_bytes(K);
  auto convert = [&](const Piece& p, int i) {
    unpack(p, f);
    *reinterpret_cast<uint4*>(to + (i >> 4) * 256 + (i & 3) * 64 + (i >> 2 & 3) * 16) =
        make_uint4(pack_f16x2(f[0] * mul, f[1] * mul), pack_f16x2(f[2] * mul, f[3] * mul),
                   pack_f16x2(f[4] * mul, f[5] * mul), pack_f16x2(f[6] * mul, f[7] * mul));
  };
#pragma unroll
  for (int n = 0; n < KEPT; ++n)
    if (first + n * hop < per) convert(kept[n], first + n * hop);
  for (int i = first + KEPT * hop; i < per; i += hop) {
    Piece p;
    load_piece(src + i * 8, p);
    convert(p, i);
  }
}

// Where the lane's rows of unit column `sub` of expert e are.
template <bool W13>
__device__ __forceinline__ Rows rows_of(const DecodeArgs& a, int e, int sub) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int K = W13 ? a.d : a.I, blk = sub >> 2, at = (sub & 3) * 8 + g;
  const long long row = W13 ? (long long)e * 2 * a.I + blk * 64 + at : (long long)e * a.d + blk * 128 + at;
  const long long block = W13 ? (long long)e * (a.I / 64) + blk : (long long)e * (a.d / 128) + blk;
  Rows r;
  r.code = a.codes + row * (K / 2) + q * 16;
  r.scale = a.sf + (block * (K / 64) + (q >> 1)) * 512 + at * 16;
  return r;
}

// First of the eight output columns of row i of a unit (rows g = 0..7 follow).
template <bool W13>
__device__ __forceinline__ int out_col(int sub, int i) {
  return W13 ? (sub >> 2) * 64 + i * 32 + (sub & 3) * 8 : (sub >> 2) * 128 + i * 32 + (sub & 3) * 8;
}

__device__ __forceinline__ float swiglu(const DecodeArgs& a, float G, float U) {
  if (a.clamp > 0.f) {                   // by comparisons: fminf and fmaxf drop a NaN
    G = G > a.clamp ? a.clamp : G < -a.clamp ? -a.clamp : G;
    U = U > a.clamp ? a.clamp : U < -a.clamp ? -a.clamp : U;
  }
  return __fdividef(G, 1.f + __expf(-G)) * U;
}

// Which pairs count, and the first bad id into the error word (one CTA calls it).
__device__ __forceinline__ void check_ids(const DecodeArgs& a) {
  for (int p = threadIdx.x; p < a.T * a.k; p += blockDim.x) {
    const int e = a.ids[p];
    const bool ok = e >= 0 && e < a.E && !repeated(a, p);
    a.keep[p] = ok;
    if (!ok) {
      atomicCAS(&a.err->code, 0, MOE_ERR_BAD_IDS);
      atomicMin(&a.err->first_bad, p);
    }
  }
}

// ---- one token ---------------------------------------------------------------------
//
// No list is needed: a pair is an expert of its own.  W13: a unit of one pair a CTA,
// K split over its eight warps as in k_decode_split.  W2: 32 rows a CTA, a warp a pair
// (k <= 8), the first two of its I / 128 steps of weights on their way before h is there,
// and the pairs added in the CTA: no third launch.

// The expert of pair j of the one token; -1 for a bad id or a repeated one.
__device__ __forceinline__ int expert_of(const DecodeArgs& a, int j) {
  const int e = a.ids[j];
  bool ok = e >= 0 && e < a.E;
#pragma unroll 8
  for (int i = 0; i < j; ++i) ok &= a.ids[i] != e;
  return ok ? e : -1;
}

__global__ void __launch_bounds__(kThreads, 3) k_decode_one_w13(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t xs[];         // the token's row
  __shared__ Tokens tok;
  __shared__ uint16_t pair;
  __shared__ float red[kWarps][32][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int per = a.I / 16, steps = a.d / kStep;
  const int j = blockIdx.x / per, sub = blockIdx.x - j * per;
  const long long gap = 32LL * (a.d / 2), far = (long long)a.I * (a.d / 2);
  if (threadIdx.x == 0) pair = (uint16_t)j;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int e = expert_of(a, j);
  StepA w;
  Rows r{nullptr, nullptr};
  if (e >= 0) {
    r = rows_of<true>(a, e, sub);
    if (warp < steps) load_step(r, gap, far, warp, w);
  }
  if (blockIdx.x == 0) check_ids(a);
  if (e < 0) return;
  const float alpha = a.w_scale[e];
  stage_tokens<true, 1>(a, tok, xs, &pair, 1);
  __syncthreads();
  float acc[2][2][4] = {};
  for (int step = warp; step < steps; step += kWarps) {
    StepA cur = w;
    if (step + kWarps < steps) load_step(r, gap, far, step + kWarps, w);
    mma_step(cur, (q & 1) * 16, xs + q * 16 + step * (2 * kStep), g == 0, acc);
  }
  if (q == 0)                            // column 0
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[warp][g][i] = acc[0][i >> 1][(i & 1) * 2] + acc[1][i >> 1][(i & 1) * 2];
  __syncthreads();
  if (threadIdx.x < 16) {
    const int i = threadIdx.x >> 3, gg = threadIdx.x & 7;
    float G = 0.f, U = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      G += red[x][gg][i];
      U += red[x][gg][i + 2];
    }
    const float f = alpha * tok.inv[0];
    a.h[(long long)j * a.I + out_col<true>(sub, i) + gg] = swiglu(a, f * G, f * U);
  }
}

__global__ void __launch_bounds__(kThreads, 2) k_decode_one_w2(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t xs[];         // the pairs' rows of h
  __shared__ Tokens tok;
  __shared__ uint16_t pairs[kCols];
  __shared__ float red[kWarps][32];
  __shared__ float factor[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int sub = blockIdx.x, steps = a.I / kStep;
  const long long gap = 32LL * (a.I / 2), far = 64LL * (a.I / 2);
  if (threadIdx.x < kCols) pairs[threadIdx.x] = (uint16_t)threadIdx.x;
  // weights, ids and scales were there before the W13 kernel started
  const int e = warp < a.k ? expert_of(a, warp) : -1;
  StepA w[2];
  Rows r{nullptr, nullptr};
  if (e >= 0) {
    r = rows_of<false>(a, e, sub);
    load_step(r, gap, far, 0, w[0]);
    load_step(r, gap, far, 1, w[1]);
  }
  const float alpha = e >= 0 ? a.w_scale[e] : 0.f;
  __syncthreads();
  pdl_wait();                            // h is complete
  pdl_trigger();
  stage_tokens<false, 3>(a, tok, xs, pairs, a.k);
  __syncthreads();
  if (e >= 0) {
    float acc[2][2][4] = {};
    const uint8_t* lane_xs = xs + warp * row_bytes(a.I) + q * 16;
    for (int step = 0; step < steps; step += 2) {          // steps is even
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const StepA cur = w[b];
        if (step + b + 2 < steps) load_step(r, gap, far, step + b + 2, w[b]);
        mma_step(cur, (q & 1) * 16, lane_xs + (step + b) * (2 * kStep), g == 0, acc);
      }
    }
    if (q == 0)                          // column 0
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[warp][i * 8 + g] = acc[0][i >> 1][(i & 1) * 2] + acc[1][i >> 1][(i & 1) * 2];
  } else {
    red[warp][lane] = 0.f;
  }
  if (lane == 0) factor[warp] = e >= 0 ? tok.score[warp] * (alpha * tok.inv[warp]) : 0.f;
  __syncthreads();
  if (warp == 0) {
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) y += factor[j] * red[j][lane];
    a.y[out_col<false>(sub, lane >> 3) + (lane & 7)] = f2bf(y);
  }
}

// ---- few units: K split over the warps ------------------------------------------
//
// A CTA of eight warps takes one unit at a time, a warp every eighth step, the sums
// joined in shared memory: a unit is over after d / 1024 steps, and two tokens' experts
// fill the GPU.  Latency bounds it: 8 tokens with all of 8 experts of d=2048, I=768 17.5 us
// with all launches, 1.2 TB/s.
template <bool W13>
__global__ void __launch_bounds__(kThreads, 2) k_decode_split(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];       // the pairs' list, the tokens' rows
  __shared__ Plan s;
  __shared__ Tokens tok;
  __shared__ float red[2][kWarps][32][9];
  uint16_t* const list = reinterpret_cast<uint16_t*>(smem);
  uint8_t* const xs = smem + list_bytes(a.T * a.k);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int K = W13 ? a.d : a.I, per = W13 ? a.I / 16 : a.d / 32;      // units of a pass
  const int steps = K / kStep, half = (q & 1) * 16;
  const long long gap = 32LL * (K / 2), far = (long long)(W13 ? a.I : 64) * (K / 2);
  s.count[threadIdx.x] = 0;
  __syncthreads();
  if (W13) {
    pdl_wait();
    pdl_trigger();        // the W2 kernel may start: before it waits it reads what was
  }                       // there before this one: weights and ids
  Mine m;
  const int passes = make_plan(a, s, m);
  int2 run = run_of(passes * per);
  int pass = run.x / per, sub = run.x - pass * per;
  if (run.x < run.y) find_pass(a, s, m, pass);
  __syncthreads();
  StepA w;
  if (run.x < run.y && warp < steps) load_step(rows_of<W13>(a, s.expert, sub), gap, far, warp, w);
  fill_list(a, s, m, list, list + a.T * a.k);
  if (!W13) {
    pdl_wait();           // h is complete
    pdl_trigger();
  }
  __syncthreads();
  int flip = 0, n = run.y - run.x;
  while (n > 0) {
    const int e = s.expert, nt = s.tokens, stop = min(per, sub + n);
    const float alpha = a.w_scale[e];
    stage_tokens<W13, W13 ? 4 : 2>(a, tok, xs, list + s.first, nt);
    __syncthreads();
    n -= stop - sub;
    for (; sub < stop; ++sub) {
      float acc[2][2][4] = {};
      const Rows r = rows_of<W13>(a, e, sub);
      const uint8_t* lane_xs = xs + g * row_bytes(K) + q * 16;
      for (int step = warp; step < steps; step += kWarps) {
        StepA cur = w;
        if (step + kWarps < steps) load_step(r, gap, far, step + kWarps, w);
        else if (sub + 1 < stop) load_step(rows_of<W13>(a, e, sub + 1), gap, far, warp, w);
        mma_step(cur, half, lane_xs + step * (2 * kStep), g < nt, acc);
      }
      float (*sums)[32][9] = red[flip];
      flip ^= 1;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[warp][lane][t * 4 + j] = acc[0][t][j] + acc[1][t][j];
      __syncthreads();
      // element (row i of four, g; column c), the warps added in order
      auto reduced = [&](int i, int gg, int c) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x)
          v += sums[x][gg * 4 + (c >> 1)][(i >> 1) * 4 + (i & 1) * 2 + (c & 1)];
        return v;
      };
      const int gg = threadIdx.x & 7, c = threadIdx.x >> 3 & 7, i = threadIdx.x >> 6;
      if (c < nt && (!W13 || i < 2)) {
        const float f = alpha * tok.inv[c];
        if (W13)
          a.h[(long long)tok.pair[c] * a.I + out_col<true>(sub, i) + gg] =
              swiglu(a, f * reduced(i, gg, c), f * reduced(i + 2, gg, c));
        else
          a.ys[(long long)tok.pair[c] * a.d + out_col<false>(sub, i) + gg] =
              tok.score[c] * (f * reduced(i, gg, c));
      }
    }
    if (n > 0) {
      pass += 1;
      sub = 0;
      __syncthreads();                   // the pass has been read
      find_pass(a, s, m, pass);
      __syncthreads();
      if (warp < steps) load_step(rows_of<W13>(a, s.expert, 0), gap, far, warp, w);
    }
  }
  if (W13 && blockIdx.x == 0) check_ids(a);
}

// ---- many units: a unit a warp ----------------------------------------------------
//
// One CTA of 16 warps an SM.  It stages the tokens of two passes of its run at once;
// its warps then take the run's units one by one and stream them on their own, each
// through a ring of its own in shared memory filled with cp.async: a stage is 256
// elements (128 bytes) of the unit's 32 rows and their scales, copied as whole lines,
// the next stage (or the next unit's first) on its way while one is read.  Nothing in
// the stream waits for another warp.  Whole lines, because lanes that load 64-byte pieces
// of eight rows stay at 5.1 to 5.8 TB/s where lines reach 6.5.  64 tokens on all of 128
// experts, d=2048, I=768 (335 MB): 72.2 us with all launches, 4.6 TB/s.
constexpr int kStreamWarps = 16;
constexpr int kStages = 2;
constexpr int kStageBytes = 32 * 128 + 512;                 // codes, scales
constexpr int kRingBytes = kStreamWarps * kStages * kStageBytes;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool W13>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) k_decode_stream(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];       // ring, list, two passes' rows
  __shared__ Plan s;
  __shared__ Tokens tok[2];
  __shared__ int two[2][3];                             // expert, first pair, tokens
  __shared__ int taken;
  uint16_t* const list = reinterpret_cast<uint16_t*>(smem + kRingBytes);
  uint8_t* const xs = smem + kRingBytes + list_bytes(a.T * a.k);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int K = W13 ? a.d : a.I, per = W13 ? a.I / 16 : a.d / 32;
  const int steps = K / kStep, half = (q & 1) * 16;
  const long long gap = 32LL * (K / 2), far = (long long)(W13 ? a.I : 64) * (K / 2);
  uint8_t* const ring = smem + warp * (kStages * kStageBytes);
  const int pairs = steps / 2;          // stages of a unit (K is a multiple of 256)
  if (threadIdx.x < kThreads) s.count[threadIdx.x] = 0;
  __syncthreads();
  if (W13) {
    pdl_wait();
    pdl_trigger();        // as in k_decode_split
  }
  Mine m;
  const int passes = make_plan(a, s, m);
  int2 run = run_of(passes * per);
  int pass = run.x / per, sub0 = run.x - pass * per, n = run.y - run.x;
  bool listed = false;
  while (n > 0) {
    // two passes: unit columns [sub0, per) of the first, [0, n - ..) of the second
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
      const int k = pass + i - m.before;
      if (k >= 0 && k < m.passes) {
        two[i][0] = threadIdx.x;
        two[i][1] = m.start + k * a.cols;
        two[i][2] = min(a.cols, m.tokens - k * a.cols);
      }
    }
    const int n0 = min(n, per - sub0), n1 = min(n - n0, per), here = n0 + n1;
    // as many warps as bring whole rounds of units: a last round of a few leaves the
    // memory idle (64 tokens on 128 experts 75.4 us with all warps, 73.6 so; 32: 67.2, 63.2)
    const int rounds = (here + kStreamWarps - 1) / kStreamWarps;
    const int active = (here + rounds - 1) / rounds;
    if (threadIdx.x == 0) taken = active;
    __syncthreads();
    // where the lane copies from: row lane / 8 of a unit, piece lane % 8; and the
    // scales of line lane % 8 in K group lane / 8
    auto rows = [&](int v) {
      const int e = v < n0 ? two[0][0] : two[1][0], sub = v < n0 ? sub0 + v : v - n0;
      const int blk = sub >> 2, at = (sub & 3) * 8;
      const long long row = (W13 ? (long long)e * 2 * a.I + blk * 64 : (long long)e * a.d + blk * 128) +
                            at + (lane >> 3);
      const long long block = W13 ? (long long)e * (a.I / 64) + blk : (long long)e * (a.d / 128) + blk;
      Rows r;
      r.code = a.codes + row * (K / 2) + (lane & 7) * 16;
      r.scale = a.sf + (block * (K / 64) + (lane >> 3)) * 512 + (at + (lane & 7)) * 16;
      return r;
    };
    // The copies are kStages - 1 stages ahead: stage `to` of the rows r comes next, of
    // the warp's unit or (in_next) of the one it takes after that.
    int unit = warp < active ? warp : here, next = here, to = 0, to_slot = 0;
    bool more = unit < here, in_next = false;
    Rows r{nullptr, nullptr};
    if (more) r = rows(unit);
    auto fetch = [&]() {
      if (more) {
        // row 4 n + lane / 8; odd rows have their halves exchanged, so that the reads
        // of two neighbouring rows fall on different banks
        const uint32_t at = smem_u32(ring) + to_slot * kStageBytes + (lane >> 3) * 128 +
                            ((lane & 7) ^ ((lane >> 3 & 1) << 2)) * 16;
        const uint8_t* p = r.code + to * 128;
#pragma unroll
        for (int n = 0; n < 8; ++n)
          cp_async16(at + n * 512, p + (n & 1) * (4 * (K / 2)) + (n >> 1 & 1) * gap + (n >> 2) * far);
        cp_async16(smem_u32(ring) + to_slot * kStageBytes + 4096 + lane * 16, r.scale + to * 2048);
        to_slot = to_slot + 1 == kStages ? 0 : to_slot + 1;
        if (++to == pairs) {
          to = 0;
          more = !in_next && next < here;
          in_next = true;
          if (more) r = rows(next);
        }
      }
      cp_async_commit();
    };
    auto take = [&]() {
      int v = 0;
      if (lane == 0) v = atomicAdd(&taken, 1);
      return __shfl_sync(0xffffffffu, v, 0);
    };
    if (more) next = take();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
    if (!listed) {
      fill_list(a, s, m, list, list + a.T * a.k);
      if (!W13) {
        pdl_wait();                      // h is complete
        pdl_trigger();
      }
      listed = true;
      __syncthreads();
    }
    {
      const int i = (warp >> 3) & 1;     // a third group of warps has nothing to stage
      stage_tokens<W13, W13 ? 8 : 3>(a, tok[i], xs + i * a.cols * row_bytes(K), list + two[i][1],
                                     warp < 8 || (warp < 16 && n1 > 0) ? two[i][2] : 0);
    }
    __syncthreads();
    int stage = 0;
    while (unit < here) {
      const int i = unit < n0 ? 0 : 1, e = two[i][0], nt = two[i][2];
      const int sub = i ? unit - n0 : sub0 + unit;
      const float alpha = a.w_scale[e];
      const uint8_t* lane_xs = xs + (i * a.cols + g) * row_bytes(K) + q * 16;
      float acc[2][2][4] = {};
      for (int j = 0; j < pairs; ++j) {
        cp_async_wait<kStages - 2>();
        __syncwarp();                    // the other lanes' copies are there too, and
        fetch();                         // they have read the stage that this fills
        const uint8_t* at = ring + stage * kStageBytes;
        stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          StepA w;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w.c[i] = *reinterpret_cast<const uint4*>(
                at + (8 * i + g) * 128 + ((4 * b + q) ^ ((g & 1) << 2)) * 16);
          w.s = *reinterpret_cast<const uint4*>(at + 4096 + (2 * b + (q >> 1)) * 128 + g * 16);
          mma_step(w, half, lane_xs + (2 * j + b) * (2 * kStep), g < nt, acc);
        }
      }
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        const int c = 2 * q + c2;
        if (c >= nt) continue;
        const float f = alpha * tok[i].inv[c];
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = f * (acc[0][j >> 1][(j & 1) * 2 + c2] + acc[1][j >> 1][(j & 1) * 2 + c2]);
        if (W13) {
          float* h = a.h + (long long)tok[i].pair[c] * a.I + g;
          h[out_col<true>(sub, 0)] = swiglu(a, v[0], v[2]);
          h[out_col<true>(sub, 1)] = swiglu(a, v[1], v[3]);
        } else {
          float* ys = a.ys + (long long)tok[i].pair[c] * a.d + g;
#pragma unroll
          for (int j = 0; j < 4; ++j) ys[out_col<false>(sub, j)] = tok[i].score[c] * v[j];
        }
      }
      unit = next;                       // its first steps are on their way
      if (unit < here) {
        next = take();
        in_next = !more;                 // all of them are (a row of kStages - 1 stages)
        if (in_next && next < here) {
          more = true;
          r = rows(next);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();
    n -= here;                           // more to do: both passes are over
    pass += 2;
    sub0 = 0;
  }
  if (W13 && blockIdx.x == 0) check_ids(a);
  if (!W13 && !listed) {
    pdl_wait();
    pdl_trigger();
  }
}

// y[t] = the tokens' experts in j order, four columns a thread.
__global__ void __launch_bounds__(kThreads) k_decode_combine(const DecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int per = a.d / 4;
  const long long v = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (v >= (long long)a.T * per) return;
  const int t = (int)(v / per), c = (int)(v - (long long)t * per) * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j;
    const bool on = a.keep[p] != 0;              // a dropped pair's ys is old: not added
    const float4 w = __ldcg(reinterpret_cast<const float4*>(a.ys + (long long)p * a.d + c));
    sum.x += on ? w.x : 0.f;
    sum.y += on ? w.y : 0.f;
    sum.z += on ? w.z : 0.f;
    sum.w += on ? w.w : 0.f;
  }
  *reinterpret_cast<uint2*>(a.y + (long long)t * a.d + c) =
      make_uint2(pack_bf2(sum.x, sum.y), pack_bf2(sum.z, sum.w));
}

// ---- host side -------------------------------------------------------------------

// Dynamic shared memory the kernels may take beside their static.
constexpr int kSplitDynamic = 200 * 1024, kStreamDynamic = 216 * 1024;

// Tokens of a pass: up to 8, fewer where their rows would not fit; two CTAs an SM where
// that leaves room for a row.
int split_cols(int K, int pairs, int T) {
  const int room = kSplitDynamic - list_bytes(pairs), half = room < 88 * 1024 ? room : 88 * 1024;
  const int fit = (half >= row_bytes(K) ? half : room) / row_bytes(K);
  const int most = T < kCols ? T : kCols;
  return fit < most ? fit : most;
}
int stream_cols(int K, int pairs, int T) {
  const int room = kStreamDynamic - kRingBytes - list_bytes(pairs);
  const int fit = room / 2 / row_bytes(K), most = T < kCols ? T : kCols;
  return fit < most ? fit : most;
}

// Units of one launch as far as the host can tell (every pair on an expert of its own
// while there are experts, passes of eight tokens after that; wide rows take fewer at a
// time, and then there are more units than these), and whether it streams: from four
// units an SM on, where passes of four tokens fit.  Measured with K split against a
// unit a warp (us; d=2048, I=768): 1.3 to 1.7 units an SM 11.6 against 14.8, 2.5 to 3.4
// 15.5 against 15.8, 3.8 to 5 19.2 against 18.3, 5 (7 tokens on 16 experts) 23.4 against
// 20.7, 10 (4 on 128) 33.4 against 25.2.
template <bool W13>
long long units_of(const DecodeArgs& a) {
  const int pairs = a.T * a.k, experts = pairs < a.E ? pairs : a.E;
  const int full = (pairs + kCols - 1) / kCols;
  return (long long)(experts > full ? experts : full) * (W13 ? a.I / 16 : a.d / 32);
}
template <bool W13>
bool streams(const DecodeArgs& a) {
  return units_of<W13>(a) >= 4LL * num_sms() &&
         stream_cols(W13 ? a.d : a.I, a.T * a.k, a.T) >= (a.T < 4 ? a.T : 4);
}

cudaError_t launch_one_w13(DecodeArgs a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_decode_one_w13, kSplitDynamic, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_decode_one_w13, dim3(a.k * (a.I / 16)), dim3(kThreads), row_bytes(a.d), st, a);
}

cudaError_t launch_one_w2(DecodeArgs a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_decode_one_w2, kSplitDynamic, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_decode_one_w2, dim3(a.d / 32), dim3(kThreads), a.k * row_bytes(a.I), st, a);
}

template <bool W13>
cudaError_t launch_product(DecodeArgs a, cudaStream_t st) {
  const int pairs = a.T * a.k, K = W13 ? a.d : a.I, sms = num_sms();
  if (streams<W13>(a)) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = smem_optin_once(k_decode_stream<W13>, kStreamDynamic, done);
    if (e != cudaSuccess) return e;
    a.cols = stream_cols(K, pairs, a.T);
    return launch_pdl(k_decode_stream<W13>, dim3(sms), dim3(kStreamWarps * 32),
                      kRingBytes + list_bytes(pairs) + 2 * a.cols * row_bytes(K), st, a);
  }
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_decode_split<W13>, kSplitDynamic, done);
  if (e != cudaSuccess) return e;
  a.cols = split_cols(K, pairs, a.T);
  const long long units = units_of<W13>(a);
  return launch_pdl(k_decode_split<W13>, dim3((unsigned)(units < 2LL * sms ? units : 2LL * sms)),
                    dim3(kThreads), list_bytes(pairs) + a.cols * row_bytes(K), st, a);
}

}  // namespace

bool decode_nvfp4_fits(int d, int I, int pairs) {
  return split_cols(d, pairs, 1) > 0 && split_cols(I, pairs, 1) > 0;
}

cudaError_t launch_decode_nvfp4(const DecodeCall& c, int* launches, cudaStream_t stream) {
  DecodeArgs a = {};
  a.x = static_cast<const uint16_t*>(c.x);
  a.ids = c.ids; a.scores = c.scores;
  a.T = c.T; a.k = c.k; a.d = c.d; a.I = c.I; a.E = c.E;
  a.clamp = c.clamp;
  a.h = c.h; a.ys = c.ys; a.keep = c.keep;
  a.y = static_cast<uint16_t*>(c.y);
  a.err = c.err;
  a.codes = c.w13; a.sf = c.w13_sf; a.w_scale = c.w13_scale;
  // one token of up to eight experts whose rows fit: two launches
  const bool one = c.T == 1 && c.k <= kWarps && row_bytes(c.d) <= kSplitDynamic &&
                   c.k * row_bytes(c.I) <= kSplitDynamic;
  cudaError_t e = one ? launch_one_w13(a, stream) : launch_product<true>(a, stream);
  if (e != cudaSuccess) return e;
  a.codes = c.w2; a.sf = c.w2_sf; a.w_scale = c.w2_scale;
  e = one ? launch_one_w2(a, stream) : launch_product<false>(a, stream);
  *launches = one ? 2 : 3;
  if (e != cudaSuccess || one) return e;
  const long long threads = (long long)c.T * (c.d / 4);
  return launch_pdl(k_decode_combine, dim3((unsigned)((threads + kThreads - 1) / kThreads)),
                    dim3(kThreads), 0, stream, a);
}

}  // namespace moe
