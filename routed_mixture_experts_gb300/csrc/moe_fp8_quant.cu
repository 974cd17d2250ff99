// moe_fp8_quant.cu -- E4M3 codes with one fp32 scale per 128 elements: the operands
// of the 8-bit block products (moe_fp8_gemm.cu).
//
//   top = max(max |v| over the block, 2^-100), scale = top / 448, code = E4M3(v * (448 / top))
//
// (fp32, each step rounded to nearest; scale the next power of two where asked).  A block
// is 128 neighbours of a row, 128 rows of a column (for the products that sum over rows),
// or a 128 x 128 tile (weights).  v is a row of a matrix, gathered through an index or
// not, SwiGLU of a row, or SwiGLU's gradient: nothing is rounded before the codes.
//
// A CTA takes a 128 x 128 tile at a time: warp w rows 8w..8w+7, a lane four neighbouring
// columns, all of it in registers, and copies its share of the next tile into shared memory
// meanwhile.  The eight rows' largest magnitudes go through the lanes together (half the rows
// change lanes at each of the first steps), the columns' through shared memory, as integers
// of the same order in which NaN lies above infinity; a warp then reckons the scales of its
// eight rows and of eight of the columns at once.  Both sets of codes come from the same
// registers, so v is read once whatever is written.  The codes along columns are turned in
// shared memory: eight rows of a column are 8 bytes of one thread, at 16-byte places
// exchanged by the column group, so that neither the writes nor the 16-byte reads meet in a
// bank.
//
// Bound by instructions, some 550 a warp and 1024 elements with both sets, a third of them in
// the ALU at half rate.  65536 rows gathered of 8192 x 2048 in bf16: both 94 us (46 for the
// bytes), by rows 58 (26); SwiGLU of 65536 x 768 65 (46), its gradient 131 (76).

#include <cmath>
#include <type_traits>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_fp8.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr long long kMaxApart = 0x7FFFFFF0;      // elements between rows

struct QuantArgs {
  int M, C, width;             // rows, columns of the source's operand, columns of v
  int E;
  float clamp;
  int pow2;
  const void* x;  int ld_x;  int x_rows;
  const void* dh;  int ld_dh;
  const int32_t* rows;         // source row of each row, or NULL
  const int32_t* offsets;      // [E+1] or NULL
  uint8_t* codes;  int ld_codes;
  float* scales;  long long ld_scales;
  uint8_t* codes_t;  int ld_codes_t;
  float* scales_t;  long long ld_scales_t;
  int row_blocks, row_block0;  // blocks of 128 rows (with offsets: at most); the first one
  int col_blocks;
  int run, runs, run_blocks;   // column blocks of a unit, units and column blocks a row block
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(uint16_t v) { return bf2f(v); }

// Four neighbouring elements, of which `n` are there.
template <bool VEC>
__device__ __forceinline__ void load4(const float* p, int n, float (&v)[4]) {
  if (VEC) {
    if (n > 0) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p));
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? __ldg(p + j) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load4(const uint16_t* p, int n, float (&v)[4]) {
  if (VEC) {
    uint2 q = make_uint2(0u, 0u);
    if (n > 0) q = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xFFFF0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? bf2f(__ldg(p + j)) : 0.f;
  }
}

// Clipped to [-limit, limit] (0: not); a NaN stays.
__device__ __forceinline__ float clip(float v, float limit) {
  if (limit > 0.f) v = v > limit ? limit : v < -limit ? -limit : v;
  return v;
}
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// v[0..3] of columns col.. of source row `row`; `n` of them are there.
template <int SRC, bool VEC, typename T>
__device__ __forceinline__ void source4(const QuantArgs& a, long long row, int col, int n,
                                        float (&v)[4]) {
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  if (SRC == MOE_FP8_ROWS) {
    load4<VEC>(x + col, n, v);
    return;
  }
  if (SRC == MOE_FP8_SWIGLU) {
    float g[4], u[4];
    load4<VEC>(x + col, n, g);
    load4<VEC>(x + a.C + col, n, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float c = clip(g[j], a.clamp);
      v[j] = c * sigmoid(c) * clip(u[j], a.clamp);
    }
    return;
  }
  // SwiGLU's gradient: columns below C at the gate, the others at up.  Four columns lie
  // on one side (C % 4 == 0) or are taken one by one.
  const T* dh = static_cast<const T*>(a.dh) + row * a.ld_dh;
  float g[4], u[4], d[4];
  bool at_up[4];
  if (VEC) {
    const bool second = col >= a.C;
    const int c = second ? col - a.C : col;
    load4<true>(x + c, n, g);
    load4<true>(x + a.C + c, n, u);
    load4<true>(dh + c, n, d);
#pragma unroll
    for (int j = 0; j < 4; ++j) at_up[j] = second;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool second = col + j >= a.C;
      const int c = second ? col + j - a.C : col + j;
      const bool there = j < n;
      at_up[j] = second;
      g[j] = there ? to_f32<T>(__ldg(x + c)) : 0.f;
      u[j] = there ? to_f32<T>(__ldg(x + a.C + c)) : 0.f;
      d[j] = there ? to_f32<T>(__ldg(dh + c)) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float c = clip(g[j], a.clamp), s = sigmoid(c);
    const float r = at_up[j] ? d[j] * c * s
                             : d[j] * clip(u[j], a.clamp) * s * (1.f + c * (1.f - s));
    // no gradient outside the limits; there the factor is 0 and not r (NaN passes)
    const bool out = a.clamp > 0.f && fabsf(at_up[j] ? u[j] : g[j]) > a.clamp;
    v[j] = out ? r * 0.f : r;
  }
}

// scale = top / 448 and factor = 448 / top of a block from the bits of its largest
// magnitude.  On the significand x in [1, 2): a quotient from an approximate reciprocal,
// corrected by its remainder (Markstein's method), which for all 2^23 significands, and a
// reciprocal off by up to two units in the last place before its Newton step, is the
// quotient rounded to nearest.  (Two fp32 divisions took 120 issue slots a warp.)
__device__ __forceinline__ void block_scale(uint32_t bits, int pow2, float& scale, float& factor) {
  const uint32_t b = max(bits, 0x0D800000u), e = b & 0x7F800000u;      // 2^-100 at least
  const float x = __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u);
  float q = x * (1.f / 448.f);
  q = __fmaf_rn(__fmaf_rn(-q, 448.f, x), 1.f / 448.f, q);
  float y = __fdividef(1.f, x);
  y = __fmaf_rn(__fmaf_rn(-x, y, 1.f), y, y);
  float p = 448.f * y;
  p = __fmaf_rn(__fmaf_rn(-p, x, 448.f), y, p);
  uint32_t s = __float_as_uint(q) + (e - 0x3F800000u);
  uint32_t f = __float_as_uint(p) - (e - 0x3F800000u);
  if (pow2) {
    s = (s + 0x7FFFFFu) & 0x7F800000u;                                 // the power at or above
    f = 0x7F000000u - s;                                               // its inverse
  }
  if (e == 0x7F800000u) {                                              // infinity or NaN
    s = b;
    f = b == e ? 0u : b;
  }
  scale = __uint_as_float(s);
  factor = __uint_as_float(f);
}

// Four codes, a in the lowest byte.  (Packed inside the statement: through 16-bit values the
// compiler clears and shifts each half.)
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Up to 16 code bytes at p (16-byte aligned), n of them valid.
__device__ __forceinline__ void store_codes16(uint8_t* p, const uint4& v, int n) {
  if (n >= 16) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// ---- a thread's share of a tile: rows 8 warp .. 8 warp + 7, columns col .. col + 3 ----

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The larger magnitudes of two pairs of bf16 (a NaN stays: all ones below the sign).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  const __nv_bfloat162 v = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Four neighbours as two pairs.
__device__ __forceinline__ void pairs_of(uint2 q, uint64_t (&v)[2]) {
  v[0] = pair(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u));
  v[1] = pair(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
}
__device__ __forceinline__ void load_pairs(const uint16_t* p, uint64_t (&v)[2]) {
  pairs_of(__ldg(reinterpret_cast<const uint2*>(p)), v);
}
__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&v)[2]) {
  const float4 q = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = pair(q.x, q.y);
  v[1] = pair(q.z, q.w);
}
// Sigmoids of two values, as sigmoid() has them.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  float a, b;
  unpair(mul2(g, pair(-1.44269504f, -1.44269504f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  unpair(add2(pair(a, b), pair(1.f, 1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pair(a, b);
}

// SwiGLU's gradient of four neighbours, at up or at the gate.  t = dh s: t c, t u (1 + c (1 - s)),
// whose 1 - s is 0 at large gates (1 + c - c s loses the 1 from c = 2^24 on).
// Outside the limits the factor is 0 and not the gradient, so that a NaN passes.
__device__ __forceinline__ void gradient2(uint64_t (&g)[2], uint64_t (&u)[2], uint64_t (&d)[2],
                                          float clamp, bool at_up, uint64_t (&v)[2]) {
  const uint64_t one = pair(1.f, 1.f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (clamp > 0.f) {
      float x, y, p, q, e, f;
      unpair(g[j], x, y);
      unpair(u[j], p, q);
      unpair(d[j], e, f);
      e = fabsf(at_up ? p : x) > clamp ? e * 0.f : e;
      f = fabsf(at_up ? q : y) > clamp ? f * 0.f : f;
      g[j] = pair(clip(x, clamp), clip(y, clamp));
      u[j] = pair(clip(p, clamp), clip(q, clamp));
      d[j] = pair(e, f);
    }
    const uint64_t s = sigmoid2(g[j]), t = mul2(d[j], s);
    v[j] = at_up ? mul2(t, g[j])
                 : mul2(mul2(t, u[j]),
                        fma2(g[j], add2(one, s ^ 0x8000000080000000ull), one));
  }
}

// Asynchronous copy of BYTES (8 or 16) into shared memory, zeros where `there` is false.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  const int n = there ? BYTES : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
               "r"(n)
               : "memory");
}

// A run of column blocks of one row block, the unit that CTAs take in turn, and the block
// of it that is at hand.
struct Place {
  int unit;
  int cb, cb_end;      // column block, end of the run
  int rb, e;           // row block, matrix or segment
  int row0, rows;      // first row of this warp's eight, how many of them are there
  int source;          // source row of row `lane` of them (-1: none)
};

template <bool BLOCKS>
__device__ __forceinline__ void decode(const QuantArgs& a, const Segments& seg, Place& p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  p.rb = p.unit / a.runs;
  p.cb = (p.unit - p.rb * a.runs) * a.run;
  p.cb_end = min(p.cb + a.run, a.run_blocks);
  p.e = 0;
  int n;
  if (BLOCKS) {
    const int per = (a.M + 127) >> 7;
    p.e = p.rb / per;
    p.row0 = (p.rb - p.e * per) << 7;
    n = a.M - p.row0;
  } else if (a.offsets) {
    p.e = seg.find(p.rb, a.E);
    p.row0 = seg.begin[p.e] + ((p.rb - seg.first[p.e]) << 7);
    n = seg.end[p.e] - p.row0;
  } else {
    p.row0 = p.rb << 7;
    n = a.M - p.row0;
  }
  p.row0 += 8 * warp;
  p.rows = min(max(n - 8 * warp, 0), 8);
  p.source = -1;
  if (lane < p.rows) {
    p.source = p.row0 + lane;
    if (!BLOCKS && a.rows) {
      p.source = __ldg(a.rows + p.source);
      if (p.source >= a.x_rows) p.source = -1;
    }
  }
}

// The next block: of the run, or of this CTA's next unit.
template <bool BLOCKS>
__device__ __forceinline__ void advance(const QuantArgs& a, const Segments& seg, int units,
                                        Place& p) {
  if (++p.cb < p.cb_end) return;
  p.unit += gridDim.x;
  if (p.unit < units) decode<BLOCKS>(a, seg, p);
}

// Operands that v is made of, and whether a thread's share of them is copied ahead into
// shared memory: 64 KB a CTA at most where two are to fit an SM; the gradient's three bf16
// operands take 96 KB and a CTA an SM, whose threads have registers for both its halves
// (65536 x 1536 131 us against 167 without).
template <int SRC, typename T, bool VEC>
struct Share {
  static constexpr int OPS = SRC == MOE_FP8_ROWS ? 1 : SRC + 1;
  static constexpr int PIECE = 4 * (int)sizeof(T);
  static constexpr bool AHEAD = VEC && OPS * sizeof(T) <= 6;
  static constexpr int BYTES = AHEAD ? OPS * 8 * PIECE * kThreads : 0;
  static constexpr int PER_SM = AHEAD && OPS == 3 ? 1 : 2;
};

// SRC: what v is.  COLS: codes along the columns are wanted.  BLOCKS: one scale a tile
// (weights, E matrices of M rows); else one a row and one a column of the tile.
template <int SRC, typename T, bool VEC, bool BLOCKS, bool COLS>
__global__ void __launch_bounds__(kThreads, (Share<SRC, T, VEC>::PER_SM))
    k_fp8_quant(const QuantArgs a) {
  using S = Share<SRC, T, VEC>;
  constexpr bool AHEAD = S::AHEAD;
  constexpr bool PACKED = SRC == MOE_FP8_ROWS && VEC && sizeof(T) == 2;   // v are bf16 words
  constexpr int OPS = S::OPS, PIECE = S::PIECE;
  // the gradient's two halves from one reading, where a block lies on one side
  const int passes = a.run_blocks < a.col_blocks ? 2 : 1;
  constexpr bool GRAD = SRC == MOE_FP8_SWIGLU_GRAD;
  const bool in_ring = AHEAD && (!GRAD || passes == 2);
  extern __shared__ uint4 ring[];                // [row of the warp][operand][thread]
  __shared__ Segments seg;
  // the warps' largest magnitudes of the columns; a row 32 (16) bytes longer than it is
  // wide, so that the eight columns of four rows lie in 32 banks
  constexpr int COLMAX_ROW = PACKED ? 272 : 544;
  __shared__ uint4 colmax[kWarps * COLMAX_ROW / 16];
  __shared__ float4 factors[32];                 // of the columns
  __shared__ uint4 turned[128][8];               // codes of a column, 16 rows a piece
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (!BLOCKS && a.offsets) seg.init<kThreads>(a.offsets, a.E, a.M);
  const int row_blocks =
      !BLOCKS && a.offsets ? min(seg.first[a.E], a.row_blocks) : a.row_blocks;
  const int units = row_blocks * a.runs;         // fits: checked on the host
  const uint32_t my_ring = smem_u32(ring) + threadIdx.x * PIECE;
  auto copy = [&](const Place& p) {
    const int col = (p.cb << 7) + 4 * lane;
    const bool in = col < (GRAD ? a.C : a.width);
    const T* x = static_cast<const T*>(a.x) + (BLOCKS ? (long long)p.e * a.M * a.ld_x : 0LL) +
                 (in ? col : 0);
    const T* const dh = static_cast<const T*>(a.dh) + (in ? col : 0);
    // (all there in all but the last blocks: no tests then)
    if (__all_sync(kAll, in && (lane >= 8 || p.source >= 0))) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const T* q = x + (long long)__shfl_sync(kAll, p.source, i) * a.ld_x;
        copy_async<PIECE>(my_ring + (i * OPS) * (kThreads * PIECE), q);
        if (SRC != MOE_FP8_ROWS)
          copy_async<PIECE>(my_ring + (i * OPS + 1) * (kThreads * PIECE), q + a.C);
        if (GRAD)
          copy_async<PIECE>(my_ring + (i * OPS + 2) * (kThreads * PIECE),
                            dh + (long long)(p.row0 + i) * a.ld_dh);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int src = __shfl_sync(kAll, p.source, i);
        const bool there = in && src >= 0;
        const T* q = x + (long long)max(src, 0) * a.ld_x;
        copy_async<PIECE>(my_ring + (i * OPS) * (kThreads * PIECE), q, there);
        if (SRC != MOE_FP8_ROWS)
          copy_async<PIECE>(my_ring + (i * OPS + 1) * (kThreads * PIECE), q + a.C, there);
        if (GRAD)
          copy_async<PIECE>(my_ring + (i * OPS + 2) * (kThreads * PIECE),
                            dh + (long long)(there ? p.row0 + i : 0) * a.ld_dh, there);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  Place next;
  next.unit = a.row_block0 * a.runs + blockIdx.x;
  if (next.unit < units) {
    decode<BLOCKS>(a, seg, next);
    if (in_ring) copy(next);
  }
  while (next.unit < units) {
    const Place t = next;
    advance<BLOCKS>(a, seg, units, next);
    uint2 held[GRAD && AHEAD ? 8 : 1][3];         // gate, up, dh of both halves
    for (int pass = 0; pass < passes; ++pass) {
      const int cb = t.cb + pass * a.run_blocks;
      const int col = (cb << 7) + 4 * lane;
      const int n = a.width - col;                 // columns of this lane that are there
      uint64_t v[8][2];                            // two neighbours a word
      uint2 raw[PACKED ? 8 : 1];                   // four bf16
      if (GRAD && in_ring) {
        if constexpr (GRAD && AHEAD) {
          if (pass == 0) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < 3; ++j)
                held[i][j] = *reinterpret_cast<const uint2*>(
                    reinterpret_cast<const uint8_t*>(ring) + threadIdx.x * PIECE +
                    (size_t)(i * OPS + j) * (kThreads * PIECE));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint64_t g[2], u[2], d[2];
            pairs_of(held[i][0], g);
            pairs_of(held[i][1], u);
            pairs_of(held[i][2], d);
            gradient2(g, u, d, a.clamp, pass == 1, v[i]);
          }
          // (what was read has been used: the next block's share may take its place)
          if (pass == 0 && next.unit < units) copy(next);
        }
      } else if (in_ring) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint8_t* p = reinterpret_cast<const uint8_t*>(ring) + threadIdx.x * PIECE +
                             (size_t)(i * OPS) * (kThreads * PIECE);
          if (PACKED) {
            raw[i] = *reinterpret_cast<const uint2*>(p);
            pairs_of(raw[i], v[i]);
          } else if (SRC == MOE_FP8_ROWS) {
            const float4 q = *reinterpret_cast<const float4*>(p);
            v[i][0] = pair(q.x, q.y);
            v[i][1] = pair(q.z, q.w);
          } else {
            uint64_t g[2], u[2];
            pairs_of(*reinterpret_cast<const uint2*>(p), g);
            pairs_of(*reinterpret_cast<const uint2*>(p + kThreads * PIECE), u);
            if (a.clamp > 0.f) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x, y;
                unpair(g[j], x, y);
                g[j] = pair(clip(x, a.clamp), clip(y, a.clamp));
                unpair(u[j], x, y);
                u[j] = pair(clip(x, a.clamp), clip(y, a.clamp));
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) v[i][j] = mul2(mul2(g[j], sigmoid2(g[j])), u[j]);
          }
        }
        // the next block's share arrives while this one is worked on
        if (next.unit < units) copy(next);
      } else if (GRAD && VEC && passes == 2) {
        const int c0 = (t.cb << 7) + 4 * lane;       // column of the operands
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i][0] = v[i][1] = 0;
          if (i < t.rows && n > 0) {
            const T* const x = static_cast<const T*>(a.x) + (long long)(t.row0 + i) * a.ld_x + c0;
            uint64_t g[2], u[2], d[2];
            load_pairs(x, g);
            load_pairs(x + a.C, u);
            load_pairs(static_cast<const T*>(a.dh) + (long long)(t.row0 + i) * a.ld_dh + c0, d);
            gradient2(g, u, d, a.clamp, pass == 1, v[i]);
          }
        }
      } else {
        const long long base = BLOCKS ? (long long)t.e * a.M : 0LL;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int src = __shfl_sync(kAll, t.source, i);
          float f[4] = {0.f, 0.f, 0.f, 0.f};
          if (src >= 0 && n > 0) source4<SRC, VEC, T>(a, base + src, col, n, f);
          v[i][0] = pair(f[0], f[1]);
          v[i][1] = pair(f[2], f[3]);
        }
      }
      auto four = [&](int i, float (&f)[4]) {
        unpair(v[i][0], f[0], f[1]);
        unpair(v[i][1], f[2], f[3]);
      };
      // ---- largest magnitudes: of the columns, over this warp's rows; of the rows ----
      uint4 m = make_uint4(0u, 0u, 0u, 0u);         // (PACKED: two 16-bit magnitudes a word)
      uint32_t top;                                 // of row lane / 4
      if (PACKED) {
        uint32_t w[4];                              // two rows a word
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint32_t r[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (COLS) {
              m.x = larger(m.x, raw[i + j].x);
              m.y = larger(m.y, raw[i + j].y);
            }
            r[j] = larger(raw[i + j].x, raw[i + j].y);
          }
          w[i >> 1] = __vmaxu2(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[0], r[1], 0x7632));
        }
        // lanes exchange rows: half of them each time, until a lane has two
        const bool a16 = lane & 16, a8 = lane & 8;
        const uint32_t k0 =
            __vmaxu2(a16 ? w[2] : w[0], __shfl_xor_sync(kAll, a16 ? w[0] : w[2], 16));
        const uint32_t k1 =
            __vmaxu2(a16 ? w[3] : w[1], __shfl_xor_sync(kAll, a16 ? w[1] : w[3], 16));
        uint32_t k = __vmaxu2(a8 ? k1 : k0, __shfl_xor_sync(kAll, a8 ? k0 : k1, 8));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) k = __vmaxu2(k, __shfl_xor_sync(kAll, k, o));
        top = (lane & 4) ? k & 0xFFFF0000u : k << 16;
      } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f[4];
          four(i, f);
          const uint32_t b[4] = {magnitude(f[0]), magnitude(f[1]), magnitude(f[2]),
                                 magnitude(f[3])};
          if (COLS) {
            m.x = max(m.x, b[0]);
            m.y = max(m.y, b[1]);
            m.z = max(m.z, b[2]);
            m.w = max(m.w, b[3]);
          }
          w[i] = max(max(b[0], b[1]), max(b[2], b[3]));
        }
        // lanes exchange rows: half of them each time, until a lane has one
#pragma unroll
        for (int n = 4; n > 0; n >>= 1) {
          const bool hi = lane & (4 * n);
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const uint32_t send = hi ? w[i] : w[i + n], keep = hi ? w[i + n] : w[i];
            w[i] = max(keep, __shfl_xor_sync(kAll, send, 4 * n));
          }
        }
        top = w[0];
        top = max(top, __shfl_xor_sync(kAll, top, 2));
        top = max(top, __shfl_xor_sync(kAll, top, 1));
      }
      float scale = 0.f, factor = 0.f;
      if (BLOCKS) {
        top = __reduce_max_sync(kAll, top);
        if (lane == 0) colmax[warp].x = top;
        __syncthreads();
        top = __reduce_max_sync(kAll, lane < kWarps ? colmax[lane].x : 0u);
        block_scale(top, a.pow2, scale, factor);
        if (threadIdx.x == 0) {
          const int nb = (a.M + 127) >> 7, b = t.rb - t.e * nb;
          if (a.scales) a.scales[((long long)t.e * nb + b) * a.col_blocks + cb] = scale;
          if (a.scales_t) a.scales_t[((long long)t.e * a.col_blocks + cb) * nb + b] = scale;
        }
      } else {
        // one reckoning for both: lanes 4 i take row i, lanes 4 i + 1 this warp's column i
        if (COLS) {
          uint8_t* const at = reinterpret_cast<uint8_t*>(colmax) + warp * COLMAX_ROW;
          if (PACKED)
            reinterpret_cast<uint2*>(at)[lane] = make_uint2(m.x, m.y);
          else
            reinterpret_cast<uint4*>(at)[lane] = m;
          __syncthreads();
          uint32_t c = 0;                           // column 8 warp + lane % 8
#pragma unroll
          for (int j = 0; j < kWarps; j += 4) {
            const uint8_t* const q =
                reinterpret_cast<const uint8_t*>(colmax) + ((lane >> 3) + j) * COLMAX_ROW;
            const int i = 8 * warp + (lane & 7);
            c = max(c, PACKED ? (uint32_t)reinterpret_cast<const uint16_t*>(q)[i] << 16
                              : reinterpret_cast<const uint32_t*>(q)[i]);
          }
          c = max(c, __shfl_xor_sync(kAll, c, 8));
          c = max(c, __shfl_xor_sync(kAll, c, 16));
          c = __shfl_sync(kAll, c, lane >> 2);
          if (lane & 1) top = c;
        }
        block_scale(top, a.pow2, scale, factor);
        const int i = lane >> 2;
        if (a.codes && (lane & 3) == 0 && i < t.rows)
          a.scales[(long long)cb * a.ld_scales + t.row0 + i] = scale;
        if (COLS && (lane & 3) == 1) {
          const int c = (cb << 7) + 8 * warp + i;
          reinterpret_cast<float*>(factors)[8 * warp + i] = factor;
          if (c < a.width) a.scales_t[(long long)t.rb * a.ld_scales_t + c] = scale;
        }
      }
      // ---- codes along the rows ----
      if (a.codes) {
        uint8_t* const p =
            a.codes + ((BLOCKS ? (long long)t.e * a.M : 0LL) + t.row0) * a.ld_codes + col;
        const int rows = n > 0 ? t.rows : 0;
        auto code_rows = [&](auto full) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s = BLOCKS ? factor : __shfl_sync(kAll, factor, 4 * i);
            const uint64_t s2 = pair(s, s);
            float f[4];
            unpair(mul2(v[i][0], s2), f[0], f[1]);
            unpair(mul2(v[i][1], s2), f[2], f[3]);
            const uint32_t w = codes4(f[0], f[1], f[2], f[3]);
            if (decltype(full)::value || i < rows) {
              uint8_t* const q = p + (long long)i * a.ld_codes;
              if (VEC || n >= 4) {
                *reinterpret_cast<uint32_t*>(q) = w;
              } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                  if (j < n) q[j] = (uint8_t)(w >> (8 * j));
              }
            }
          }
        };
        if (VEC && __all_sync(kAll, rows == 8))
          code_rows(std::true_type{});
        else
          code_rows(std::false_type{});
      }
      if (!COLS) {
        if (BLOCKS) __syncthreads();                // colmax has been read
        continue;
      }
      // ---- codes along the columns ----
      float4 f = make_float4(factor, factor, factor, factor);
      if (!BLOCKS) {
        __syncthreads();
        f = factors[lane];
      }
      {
        const uint64_t f2[2] = {pair(f.x, f.y), pair(f.z, f.w)};
        // rows 8 warp.. of a column: half `warp & 1` of piece warp / 2
        const int piece = (warp >> 1) ^ (lane & 7), side = (warp & 1) ^ ((lane >> 3) & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8], y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) unpair(mul2(v[i][h], f2[h]), x[i], y[i]);
          reinterpret_cast<uint2*>(&turned[4 * lane + 2 * h][piece])[side] =
              make_uint2(codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7]));
          reinterpret_cast<uint2*>(&turned[4 * lane + 2 * h + 1][piece])[side] =
              make_uint2(codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7]));
        }
      }
      __syncthreads();
      // first column of codes_t, and how many there are
      const int at_t = BLOCKS ? (t.rb - t.e * ((a.M + 127) >> 7)) << 7 : t.rb << 7;
      const int n_t = BLOCKS ? a.M - at_t : 128;
#pragma unroll
      for (int q = threadIdx.x; q < 1024; q += kThreads) {
        const int c = q >> 3, piece = q & 7, group = c >> 2;
        if ((cb << 7) + c >= a.width || 16 * piece >= n_t) continue;
        uint4 w = turned[c][piece ^ (group & 7)];
        if ((group >> 3) & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        const long long row = (BLOCKS ? (long long)t.e * a.width : 0LL) + (cb << 7) + c;
        uint8_t* p = a.codes_t + row * a.ld_codes_t + at_t + 16 * piece;
        if (BLOCKS)
          store_codes16(p, w, n_t - 16 * piece);
        else
          *reinterpret_cast<uint4*>(p) = w;
      }
      // (between two barriers only: the next block writes colmax before its first, when this
      // one's has been read, factors before its second, turned after that)
      if (BLOCKS) __syncthreads();
    }
  }
  pdl_trigger();
}

template <int SRC, typename T, bool VEC, bool BLOCKS, bool COLS>
cudaError_t launch_one(const QuantArgs& a, dim3 g, dim3 b, cudaStream_t st) {
  constexpr int ring = Share<SRC, T, VEC>::BYTES;
  static std::atomic<unsigned long long> done{0};
  if (ring) {
    const cudaError_t e = smem_optin_once(k_fp8_quant<SRC, T, VEC, BLOCKS, COLS>, ring, done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_fp8_quant<SRC, T, VEC, BLOCKS, COLS>, g, b, ring, st, a);
}

template <int SRC, typename T, bool VEC, bool BLOCKS>
cudaError_t launch_with(const QuantArgs& a, dim3 g, dim3 b, cudaStream_t st) {
  return a.codes_t ? launch_one<SRC, T, VEC, BLOCKS, true>(a, g, b, st)
                   : launch_one<SRC, T, VEC, BLOCKS, false>(a, g, b, st);
}

template <int SRC, typename T, bool BLOCKS>
cudaError_t launch(QuantArgs a, bool vec, cudaStream_t st) {
  const int most = (vec ? Share<SRC, T, true>::PER_SM : 2) * num_sms();
  a.run_blocks = SRC == MOE_FP8_SWIGLU_GRAD && vec && a.C % 128 == 0 ? a.C / 128 : a.col_blocks;
  const int row_blocks = a.row_blocks - a.row_block0;
  // runs as long as leave every CTA some six of them
  const long long each = (long long)row_blocks * a.run_blocks / (6LL * most);
  a.run = (int)(each < 1 ? 1 : each < a.run_blocks ? each : a.run_blocks);
  a.runs = (a.run_blocks + a.run - 1) / a.run;
  const long long units = (long long)row_blocks * a.runs;
  const dim3 g((unsigned)(units < most ? units : most)), b(kThreads);
  return vec ? launch_with<SRC, T, true, BLOCKS>(a, g, b, st)
             : launch_with<SRC, T, false, BLOCKS>(a, g, b, st);
}

bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_quantize(const moe_fp8_quant_desc* s, int M, const void* x, long long ld_x,
                                int x_rows, const void* dh, long long ld_dh, const int32_t* rows,
                                const int32_t* offsets, uint8_t* codes, long long ld_codes,
                                float* scales, long long ld_scales, uint8_t* codes_t,
                                long long ld_codes_t, long long cols_t, float* scales_t,
                                long long ld_scales_t, void* stream) {
  if (!s || s->source < MOE_FP8_ROWS || s->source > MOE_FP8_SWIGLU_GRAD || s->C < 1 ||
      s->C > MOE_FP8_MAX_WIDTH / 2 || s->E < 1 || s->E > kMaxSegments ||
      (s->dtype != MOE_DTYPE_BF16 && s->dtype != MOE_DTYPE_FP32) || !(s->clamp >= 0.f) ||
      !std::isfinite(s->clamp) || (s->flags & ~MOE_FP8_POW2) || M < 0)
    return MOE_ERR_INVALID_ARG;
  const bool grad = s->source == MOE_FP8_SWIGLU_GRAD, plain = s->source == MOE_FP8_ROWS;
  const int width = grad ? 2 * s->C : s->C, in_width = plain ? s->C : 2 * s->C;
  if ((!codes && !codes_t && M > 0) || (s->E > 1 && !offsets) || (rows && !plain) ||
      (rows && x_rows < 0) || (grad != (dh != nullptr) && M > 0) || (plain && s->clamp > 0.f))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const int es = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (ld_x > kMaxApart || ld_dh > kMaxApart || ld_codes > kMaxApart || ld_codes_t > kMaxApart)
    return MOE_ERR_INVALID_ARG;
  if (!x || !aligned(x, es) || ld_x < in_width || (grad && (ld_dh < s->C || !aligned(dh, es))) ||
      !aligned(rows, 4) || !aligned(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (codes && (!scales || !aligned(codes, 16) || ld_codes < width || ld_codes % 16 ||
                !aligned(scales, 4) || ld_scales < M))
    return MOE_ERR_INVALID_ARG;
  long long blocks = ((long long)M + 127) / 128;
  if (codes_t) {
    const long long need = offsets ? 0 : blocks * 128;
    if (!scales_t || !aligned(codes_t, 16) || cols_t < need || cols_t % 128 ||
        ld_codes_t < cols_t || ld_codes_t % 16 || !aligned(scales_t, 4) || ld_scales_t < width ||
        (!offsets && cols_t > 0x7FFFFF80LL))
      return MOE_ERR_INVALID_ARG;
    if (!offsets) blocks = cols_t / 128;         // those beyond the rows are zeros
  }
  // with offsets: every expert's last block may hold as little as one row
  if (offsets) blocks = ((long long)M + 127LL * s->E) / 128;
  const long long all = blocks;
  if (codes_t && offsets && blocks > cols_t / 128) blocks = cols_t / 128;
  QuantArgs a = {};
  a.M = M; a.C = s->C; a.width = width; a.E = s->E; a.clamp = s->clamp;
  a.pow2 = s->flags & MOE_FP8_POW2;
  a.x = x; a.ld_x = (int)ld_x; a.x_rows = x_rows; a.dh = dh; a.ld_dh = (int)ld_dh; a.rows = rows;
  a.offsets = offsets;
  a.codes = codes; a.ld_codes = (int)ld_codes; a.scales = scales; a.ld_scales = ld_scales;
  a.codes_t = codes_t; a.ld_codes_t = (int)ld_codes_t; a.scales_t = scales_t;
  a.ld_scales_t = ld_scales_t;
  a.col_blocks = (width + 127) / 128;
  if ((codes ? all : blocks) * a.col_blocks > (1LL << 30)) return MOE_ERR_INVALID_ARG;
  // four columns at a time: on one side of C, at addresses of their size
  const bool vec = s->C % 4 == 0 && ld_x % 4 == 0 && aligned(x, 4 * es) &&
                   (!grad || (ld_dh % 4 == 0 && aligned(dh, 4 * es)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = s->dtype == MOE_DTYPE_FP32;
  auto run = [&]() {
    switch (s->source) {
      case MOE_FP8_ROWS:
        return f32 ? launch<MOE_FP8_ROWS, float, false>(a, vec, st)
                   : launch<MOE_FP8_ROWS, uint16_t, false>(a, vec, st);
      case MOE_FP8_SWIGLU:
        return f32 ? launch<MOE_FP8_SWIGLU, float, false>(a, vec, st)
                   : launch<MOE_FP8_SWIGLU, uint16_t, false>(a, vec, st);
      default:
        return f32 ? launch<MOE_FP8_SWIGLU_GRAD, float, false>(a, vec, st)
                   : launch<MOE_FP8_SWIGLU_GRAD, uint16_t, false>(a, vec, st);
    }
  };
  cudaError_t e = cudaSuccess;
  a.row_blocks = (int)blocks;
  if (blocks) e = run();
  if (codes && blocks < all && e == cudaSuccess) {
    // Blocks that codes_t may have no room for: by rows alone, in a launch that ends where the
    // segments do.  (Looked at block by block in the one launch, 2 % of the time: 65536 x 2048
    // 96 us against 94.)
    a.row_block0 = (int)blocks;
    a.row_blocks = (int)all;
    a.codes_t = nullptr;
    e = run();
  }
  return cuda_result(e, "moe_fp8_quantize");
}

extern "C" int moe_fp8_quantize_weights(const void* w, int dtype, int E, int N, int K, int flags,
                                        uint8_t* codes, long long ld_codes, float* scales,
                                        uint8_t* codes_t, long long ld_codes_t, float* scales_t,
                                        void* stream) {
  if ((dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) || E < 1 || E > kMaxSegments || N < 1 ||
      K < 1 || N > MOE_FP8_MAX_WIDTH || K > MOE_FP8_MAX_WIDTH || (flags & ~MOE_FP8_POW2) ||
      (!codes && !codes_t))
    return MOE_ERR_INVALID_ARG;
  const int es = dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!w || !aligned(w, es) || ld_codes > kMaxApart || ld_codes_t > kMaxApart)
    return MOE_ERR_INVALID_ARG;
  if (codes && (!scales || !aligned(codes, 16) || ld_codes < K || ld_codes % 16 ||
                !aligned(scales, 4)))
    return MOE_ERR_INVALID_ARG;
  if (codes_t && (!scales_t || !aligned(codes_t, 16) || ld_codes_t < N || ld_codes_t % 16 ||
                  !aligned(scales_t, 4)))
    return MOE_ERR_INVALID_ARG;
  QuantArgs a = {};
  a.M = N; a.C = a.width = K; a.E = E; a.pow2 = flags & MOE_FP8_POW2;
  a.x = w; a.ld_x = K; a.x_rows = 0;
  a.codes = codes; a.ld_codes = (int)ld_codes; a.scales = codes ? scales : nullptr;
  a.codes_t = codes_t; a.ld_codes_t = (int)ld_codes_t; a.scales_t = codes_t ? scales_t : nullptr;
  a.col_blocks = (K + 127) / 128;
  const long long blocks = (long long)E * ((N + 127) / 128);
  if (blocks * a.col_blocks > (1LL << 30)) return MOE_ERR_INVALID_ARG;
  a.row_blocks = (int)blocks;
  const bool vec = K % 4 == 0 && aligned(w, 4 * es);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MOE_DTYPE_FP32
                            ? launch<MOE_FP8_ROWS, float, true>(a, vec, st)
                            : launch<MOE_FP8_ROWS, uint16_t, true>(a, vec, st);
  return cuda_result(e, "moe_fp8_quantize_weights");
}
