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
// columns, all of it in registers.  A row's largest magnitude is one reduction instruction
// on the bits (unsigned order is magnitude order, and NaN is above infinity, so it stays);
// a column's goes through shared memory.  Both sets of codes come from the same registers,
// so v is read once whatever is written.  The codes along columns are turned in shared
// memory: eight rows of a column are 8 bytes of one thread, at 16-byte places exchanged by
// the column group, so that neither the writes nor the 16-byte reads meet in a bank.

#include <cmath>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_fp8.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

struct QuantArgs {
  int M, C, width;             // rows, columns of the source's operand, columns of v
  int E;
  float clamp;
  int pow2;
  const void* x;  long long ld_x;  int x_rows;
  const void* dh;  long long ld_dh;
  const int32_t* rows;         // source row of each row, or NULL
  const int32_t* offsets;      // [E+1] or NULL
  uint8_t* codes;  long long ld_codes;
  float* scales;  long long ld_scales;
  uint8_t* codes_t;  long long ld_codes_t;
  float* scales_t;  long long ld_scales_t;
  int row_blocks;              // blocks of 128 rows (with offsets: at most)
  int col_blocks;
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

// scale and factor of a block from the bits of its largest magnitude
__device__ __forceinline__ void block_scale(uint32_t bits, int pow2, float& scale, float& factor) {
  const float top = __uint_as_float(max(bits, 0x0D800000u));           // 2^-100
  scale = __fdiv_rn(top, 448.f);
  if (pow2 && top <= 3.402823466e38f) {
    const uint32_t b = __float_as_uint(scale);
    const uint32_t up = ((b + 0x7FFFFFu) & 0x7F800000u);               // the power at or above
    scale = __uint_as_float(up);
    factor = __uint_as_float(0x7F000000u - up);                        // 2^-e
  } else {
    factor = __fdiv_rn(448.f, top);
  }
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return (uint32_t)cvt_e4m3x2(a, b) | ((uint32_t)cvt_e4m3x2(c, d) << 16);
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

// SRC: what v is.  BLOCKS: one scale a tile (weights, E matrices of M rows); else one a
// row and one a column of the tile.
template <int SRC, typename T, bool VEC, bool BLOCKS>
__global__ void __launch_bounds__(kThreads, 2) k_fp8_quant(const QuantArgs a) {
  __shared__ Segments seg;
  __shared__ uint4 colmax[kWarps][32];           // [warp][four columns]
  __shared__ float4 factors[32];                 // of the columns
  __shared__ uint4 turned[128][8];               // codes of a column, 16 rows a piece
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (!BLOCKS && a.offsets) seg.init<kThreads>(a.offsets, a.E, a.M);
  const int row_blocks =
      !BLOCKS && a.offsets ? min(seg.first[a.E], a.row_blocks) : a.row_blocks;
  const int tiles = row_blocks * a.col_blocks;   // fits: checked on the host
  const int half = a.C >> 7;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int rb = t / a.col_blocks;
    int cb = t - rb * a.col_blocks;
    // the two tiles that read the same gate, up and dh one after the other
    if (SRC == MOE_FP8_SWIGLU_GRAD && (a.C & 127) == 0) cb = (cb >> 1) + ((cb & 1) ? half : 0);
    int e = 0, row0, n_rows;
    if (BLOCKS) {
      const int per = (a.M + 127) >> 7;
      e = rb / per;
      row0 = (rb - e * per) << 7;
      n_rows = a.M - row0;
    } else if (a.offsets) {
      e = seg.find(rb, a.E);
      row0 = seg.begin[e] + ((rb - seg.first[e]) << 7);
      n_rows = seg.end[e] - row0;
    } else {
      row0 = rb << 7;
      n_rows = a.M - row0;
    }
    const int col = (cb << 7) + 4 * lane;
    const int n = a.width - col;                 // columns of this lane that are there
    float v[8][4];
    const bool direct = BLOCKS || !a.rows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = warp * 8 + i;
      long long src = -1;
      if (r < n_rows) {
        src = BLOCKS ? (long long)e * a.M + row0 + r
                     : direct ? row0 + r : (long long)__ldg(a.rows + row0 + r);
        if (!direct && src >= a.x_rows) src = -1;
      }
      if (src >= 0 && n > 0) {
        source4<SRC, VEC, T>(a, src, col, n, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
      }
    }
    // ---- along the rows ----
    float scale = 0.f, factor = 0.f;
    if (BLOCKS) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, magnitude(v[i][j]));
      m = __reduce_max_sync(kAll, m);
      if (lane == 0) colmax[warp][0].x = m;
      __syncthreads();
      m = __reduce_max_sync(kAll, lane < kWarps ? colmax[lane][0].x : 0u);
      block_scale(m, a.pow2, scale, factor);
      if (threadIdx.x == 0) {
        const int nb = (a.M + 127) >> 7, b = row0 >> 7;
        if (a.scales) a.scales[((long long)e * nb + b) * a.col_blocks + cb] = scale;
        if (a.scales_t) a.scales_t[((long long)e * a.col_blocks + cb) * nb + b] = scale;
      }
    } else if (a.codes) {
      uint32_t mine = 0;                          // lane i: of row i
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = max(max(magnitude(v[i][0]), magnitude(v[i][1])),
                         max(magnitude(v[i][2]), magnitude(v[i][3])));
        m = __reduce_max_sync(kAll, m);
        if (lane == i) mine = m;
      }
      block_scale(mine, a.pow2, scale, factor);
      const int r = warp * 8 + lane;
      if (lane < 8 && r < n_rows) a.scales[(long long)cb * a.ld_scales + row0 + r] = scale;
    }
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = BLOCKS ? factor : __shfl_sync(kAll, factor, i);
        const int r = warp * 8 + i;
        if (r < n_rows && n > 0) {
        const uint32_t w = codes4(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
        const long long at = (BLOCKS ? (long long)e * a.M : 0LL) + row0 + r;
        uint8_t* p = a.codes + at * a.ld_codes + col;
        if (VEC || n >= 4) {
          *reinterpret_cast<uint32_t*>(p) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (j < n) p[j] = (uint8_t)(w >> (8 * j));
        }
        }
      }
    }
    if (!a.codes_t) {
      if (BLOCKS) __syncthreads();                // colmax has been read
      continue;
    }
    // ---- along the columns ----
    float4 f = make_float4(factor, factor, factor, factor);
    if (!BLOCKS) {
      uint4 m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m.x = max(m.x, magnitude(v[i][0]));
        m.y = max(m.y, magnitude(v[i][1]));
        m.z = max(m.z, magnitude(v[i][2]));
        m.w = max(m.w, magnitude(v[i][3]));
      }
      colmax[warp][lane] = m;
      __syncthreads();
      if (threadIdx.x < 128) {
        const uint32_t* all = reinterpret_cast<const uint32_t*>(colmax);
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = max(top, all[w * 128 + threadIdx.x]);
        float s, g;
        block_scale(top, a.pow2, s, g);
        reinterpret_cast<float*>(factors)[threadIdx.x] = g;
        const int c = (cb << 7) + threadIdx.x;
        if (c < a.width) a.scales_t[(long long)rb * a.ld_scales_t + c] = s;
      }
      __syncthreads();
      f = factors[lane];
    }
    {
      const float fj[4] = {f.x, f.y, f.z, f.w};
      // rows 8 warp.. of a column: half `warp & 1` of piece warp / 2
      const int piece = (warp >> 1) ^ (lane & 7), side = (warp & 1) ^ ((lane >> 3) & 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = codes4(v[0][j] * fj[j], v[1][j] * fj[j], v[2][j] * fj[j],
                                   v[3][j] * fj[j]);
        const uint32_t hi = codes4(v[4][j] * fj[j], v[5][j] * fj[j], v[6][j] * fj[j],
                                   v[7][j] * fj[j]);
        reinterpret_cast<uint2*>(&turned[4 * lane + j][piece])[side] = make_uint2(lo, hi);
      }
    }
    __syncthreads();
    const long long at_t = BLOCKS ? row0 : (long long)rb << 7;     // column of codes_t
    const int n_t = BLOCKS ? a.M - row0 : 128;                     // of them there
    for (int q = threadIdx.x; q < 1024; q += kThreads) {
      const int c = q >> 3, piece = q & 7, group = c >> 2;
      if ((cb << 7) + c >= a.width || 16 * piece >= n_t) continue;
      uint4 w = turned[c][piece ^ (group & 7)];
      if ((group >> 3) & 1) w = make_uint4(w.z, w.w, w.x, w.y);
      const long long row = (BLOCKS ? (long long)e * a.width : 0LL) + (cb << 7) + c;
      store_codes16(a.codes_t + row * a.ld_codes_t + at_t + 16 * piece, w, n_t - 16 * piece);
    }
    __syncthreads();                              // before the next tile
  }
  pdl_trigger();
}

template <int SRC, typename T, bool BLOCKS>
cudaError_t launch(const QuantArgs& a, bool vec, cudaStream_t st) {
  const long long tiles = (long long)a.row_blocks * a.col_blocks;
  const long long cap = 2LL * num_sms();
  const dim3 g((unsigned)(tiles < cap ? tiles : cap)), b(kThreads);
  return vec ? launch_pdl(k_fp8_quant<SRC, T, true, BLOCKS>, g, b, 0, st, a)
             : launch_pdl(k_fp8_quant<SRC, T, false, BLOCKS>, g, b, 0, st, a);
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
  if ((!codes && !codes_t) || (s->E > 1 && !offsets) || (rows && !plain) ||
      (rows && x_rows < 0) || (grad != (dh != nullptr) && M > 0) || (plain && s->clamp > 0.f))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const int es = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
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
        ld_codes_t < cols_t || ld_codes_t % 16 || !aligned(scales_t, 4) || ld_scales_t < width)
      return MOE_ERR_INVALID_ARG;
  }
  // with offsets: every expert's last block may hold as little as one row
  if (offsets) blocks = ((long long)M + 127LL * s->E) / 128;
  if (codes_t && offsets && blocks > cols_t / 128) {
    // what does not fit is dropped on both sides, so that they stay in step
    blocks = cols_t / 128;
    if (blocks == 0) return MOE_OK;
  }
  QuantArgs a = {};
  a.M = M; a.C = s->C; a.width = width; a.E = s->E; a.clamp = s->clamp;
  a.pow2 = s->flags & MOE_FP8_POW2;
  a.x = x; a.ld_x = ld_x; a.x_rows = x_rows; a.dh = dh; a.ld_dh = ld_dh; a.rows = rows;
  a.offsets = offsets;
  a.codes = codes; a.ld_codes = ld_codes; a.scales = scales; a.ld_scales = ld_scales;
  a.codes_t = codes_t; a.ld_codes_t = ld_codes_t; a.scales_t = scales_t;
  a.ld_scales_t = ld_scales_t;
  a.col_blocks = (width + 127) / 128;
  if (blocks * a.col_blocks > (1LL << 30)) return MOE_ERR_INVALID_ARG;
  a.row_blocks = (int)blocks;
  // four columns at a time: on one side of C, at addresses of their size
  const bool vec = s->C % 4 == 0 && ld_x % 4 == 0 && aligned(x, 4 * es) &&
                   (!grad || (ld_dh % 4 == 0 && aligned(dh, 4 * es)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = s->dtype == MOE_DTYPE_FP32;
  cudaError_t e;
  switch (s->source) {
    case MOE_FP8_ROWS:
      e = f32 ? launch<MOE_FP8_ROWS, float, false>(a, vec, st)
              : launch<MOE_FP8_ROWS, uint16_t, false>(a, vec, st);
      break;
    case MOE_FP8_SWIGLU:
      e = f32 ? launch<MOE_FP8_SWIGLU, float, false>(a, vec, st)
              : launch<MOE_FP8_SWIGLU, uint16_t, false>(a, vec, st);
      break;
    default:
      e = f32 ? launch<MOE_FP8_SWIGLU_GRAD, float, false>(a, vec, st)
              : launch<MOE_FP8_SWIGLU_GRAD, uint16_t, false>(a, vec, st);
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
  if (!w || !aligned(w, es)) return MOE_ERR_INVALID_ARG;
  if (codes && (!scales || !aligned(codes, 16) || ld_codes < K || ld_codes % 16 ||
                !aligned(scales, 4)))
    return MOE_ERR_INVALID_ARG;
  if (codes_t && (!scales_t || !aligned(codes_t, 16) || ld_codes_t < N || ld_codes_t % 16 ||
                  !aligned(scales_t, 4)))
    return MOE_ERR_INVALID_ARG;
  QuantArgs a = {};
  a.M = N; a.C = a.width = K; a.E = E; a.pow2 = flags & MOE_FP8_POW2;
  a.x = w; a.ld_x = K; a.x_rows = 0;
  a.codes = codes; a.ld_codes = ld_codes; a.scales = codes ? scales : nullptr;
  a.codes_t = codes_t; a.ld_codes_t = ld_codes_t; a.scales_t = codes_t ? scales_t : nullptr;
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
