// moe_decode.cu -- the routed experts of a few tokens on NVFP4 weights: two
// launches of matrix-vector products instead of dispatch and padded GEMM tiles.
//
//   h[t,j]  = silu(G) * U,  (G, U) = w13_scale[e] * W13[e] x[t],   e = ids[t,j]
//   y[t]    = sum_j scores[t,j] * w2_scale[e] * W2[e] h[t,j]       (fixed j order)
//
// The weights are the prepared ones of moe_forward_nvfp4 (E2M1 codes, tiled E4M3
// scales per 16 elements); the activations are not quantised: x stays bf16, h is
// kept in fp32 and read by the second product as fp16, all sums are fp32.
//
// Bound by reading each chosen expert once: 3/2 d I codes and 3/16 d I scales.
// A CTA takes 32 rows of one expert's matrix for all tokens that chose the expert,
// its warps splitting K in steps of 128.  The product runs on mma.sync m16n8k16
// with the weights as the 16-row operand and up to 8 tokens as the columns: one
// token fills one column of eight, but a weight then costs half a conversion
// (cvt.e2m1x2), half a multiplication by its block's scale and no accumulation
// of its own, where per-lane fused multiply-adds cost one and a half instructions
// a weight and token.  (tcgen05 takes its operands from shared memory and would
// need the dequantised weights written there.)  E2M1 x E4M3 has at most six
// significant bits and is exact in fp16, x scaled by a power of two per token and
// K step is exact down to 2^-32 of the step's largest element; h loses what lies
// beyond fp16's 11 bits, eight times finer than the bf16 h of the other paths.
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
constexpr int kMaxWarps = 8;
// shared bytes of a token's step: four 64-byte pieces, and 64 more so that the
// eight lanes of a quarter-warp load from different banks
constexpr int kTokStride = 320;

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

// One lane's operands of a step: 16 code bytes of each of its rows and the scale
// words of the four rows (blocks of its half K group).
struct StepA {
  uint4 c[4];
  uint4 s;
};

struct Rows {
  const uint8_t* code[4];     // the lane's 16 bytes of step 0 in each row
  const uint8_t* scale;       // the lane's 16 scale bytes of step 0
  int half;                   // 16 * (q & 1): which two of a K group's four blocks
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void load_step(const Rows& r, int step, StepA& a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a.c[i] = ldg_stream(r.code[i] + (long long)step * (kStep / 2));
  a.s = *reinterpret_cast<const uint4*>(r.scale + (long long)step * 1024);
}

// acc[tile][..] += (dequantised rows) . (the tokens' step in `xs`), the step's
// token scales (inverse powers of two) applied to the partial sums.
__device__ __forceinline__ void mma_step(const StepA& a, int half, const uint8_t* xs,
                                         const float* inv, int lane, bool have,
                                         float (&acc)[2][4]) {
  const int g = lane >> 2, q = lane & 3;
  const uint32_t sw[4] = {a.s.x, a.s.y, a.s.z, a.s.w};
  uint32_t s0[4], s1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    const uint16_t two = (uint16_t)(sw[i] >> half);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    s0[i] = __byte_perm(h, h, 0x1010);
    s1[i] = __byte_perm(h, h, 0x3232);
  }
  float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if (have) b = *reinterpret_cast<const uint4*>(xs + g * kTokStride + w * 64 + q * 16);
    uint32_t f[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = w == 0 ? a.c[i].x : w == 1 ? a.c[i].y : w == 2 ? a.c[i].z : a.c[i].w;
#pragma unroll
      for (int p = 0; p < 4; ++p) f[i][p] = mul_f16x2(e2m1x2_to_f16x2(word, p), w < 2 ? s0[i] : s1[i]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mma_f16(c[t], f[2 * t][0], f[2 * t + 1][0], f[2 * t][1], f[2 * t + 1][1], b.x, b.y);
      mma_f16(c[t], f[2 * t][2], f[2 * t + 1][2], f[2 * t][3], f[2 * t + 1][3], b.z, b.w);
    }
  }
  const float i0 = inv[2 * q], i1 = inv[2 * q + 1];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    acc[t][0] += c[t][0] * i0;
    acc[t][1] += c[t][1] * i1;
    acc[t][2] += c[t][2] * i0;
    acc[t][3] += c[t][3] * i1;
  }
}

struct DecodeArgs {
  const uint16_t* x;          // [T, d] bf16
  const int32_t* ids;         // [T, k]
  const float* scores;        // [T, k]
  int T, k, d, I, E;
  int slots;                  // gridDim.y: T*k (slot = pair) or E (slot = expert)
  float clamp;
  const uint8_t *codes, *sf;  // this launch's matrix
  const float* w_scale;
  float* h;                   // [T*k, I]
  float* ys;                  // [T*k, d]
  uint8_t* keep;              // [T*k] 1: the pair counts (valid id, first in its row)
  int* arrived;               // [d / 32], zero between calls
  uint16_t* y;                // [T, d]
  DevError* err;
};

struct Shared {
  int list[kDecodeMaxTokens]; // pairs t*k+j of the CTA's expert
  int count, first, last;
  __align__(16) uint8_t xs[kMaxWarps][kCols * kTokStride];
  float inv[kMaxWarps][kCols];
  float red[kMaxWarps][32][9];
};

// The expert of a slot; -1: none.  With a slot per pair the pair's own id.
__device__ __forceinline__ int slot_expert(const DecodeArgs& a, int slot) {
  if (a.slots != a.T * a.k) return slot;
  const int e = a.ids[slot];
  return e >= 0 && e < a.E ? e : -1;
}

// True for an id that repeats an earlier one of its row.
__device__ __forceinline__ bool repeated(const DecodeArgs& a, int p) {
  const int e = a.ids[p], row = p / a.k * a.k;
  for (int i = row; i < p; ++i)
    if (a.ids[i] == e) return true;
  return false;
}

// The pairs that chose expert e, into s.list; false: none, or (a slot per pair)
// another slot has them.  All threads call it.
__device__ __forceinline__ bool collect(const DecodeArgs& a, Shared& s, int slot, int e) {
  if (threadIdx.x == 0) {
    s.count = 0;
    s.first = INT_MAX;
  }
  __syncthreads();
  const int n = a.T * a.k;
  if (e >= 0)
    for (int p = threadIdx.x; p < n; p += blockDim.x)
      if (a.ids[p] == e && !repeated(a, p)) {
        s.list[atomicAdd(&s.count, 1)] = p;
        atomicMin(&s.first, p);
      }
  __syncthreads();
  return s.count > 0 && (a.slots != n || s.first == slot);
}

// Adds the warps' accumulators in order; thread v < 256 returns element
// (row i, g; column c) = (v / 64, v / 8 % 8, v % 8).
__device__ __forceinline__ float reduce_warps(Shared& s, const float (&acc)[2][4], int warp,
                                              int lane, int nw, int v) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) s.red[warp][lane][t * 4 + j] = acc[t][j];
  __syncthreads();
  float r = 0.f;
  if (v < 256) {
    const int i = v >> 6, g = v >> 3 & 7, c = v & 7;
    const int src = g * 4 + (c >> 1), at = (i >> 1) * 4 + (i & 1) * 2 + (c & 1);
    for (int w = 0; w < nw; ++w) r += s.red[w][src][at];
  }
  return r;
}

// W13 x, SwiGLU.  blockIdx.x: 16 columns of h (set s of a 64-column block).
__global__ void __launch_bounds__(256, 3) k_decode_w13(const DecodeArgs a) {
  __shared__ Shared s;
  pdl_wait();
  pdl_trigger();          // the W2 kernel may start: it reads weights and ids before it waits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
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
  const int slot = blockIdx.y, e = slot_expert(a, slot);
  const int blk = blockIdx.x >> 2, set = blockIdx.x & 3;
  const int steps = a.d / kStep;
  Rows r;
  {
    const long long row = (long long)(e < 0 ? 0 : e) * 2 * a.I + blk * 64 + set * 8 + g;
    const uint8_t* base = a.codes + q * 16;
    const long long ld = a.d / 2;
    r.code[0] = base + row * ld;
    r.code[1] = base + (row + 32) * ld;
    r.code[2] = base + (row + a.I) * ld;
    r.code[3] = base + (row + a.I + 32) * ld;
    r.scale = a.sf + (((long long)(e < 0 ? 0 : e) * (a.I / 64) + blk) * (a.d / 64) + (q >> 1)) * 512 +
              (set * 8 + g) * 16;
    r.half = (q & 1) * 16;
  }
  StepA w0;
  if (warp < steps && e >= 0) load_step(r, warp, w0);
  if (!collect(a, s, slot, e)) return;
  const float alpha = a.w_scale[e];
  const int count = s.count;
  for (int t0 = 0; t0 < count; t0 += kCols) {
    const int nt = min(kCols, count - t0);
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int step = warp; step < steps; step += nw) {
      StepA cur;
      if (step == warp && t0 == 0) cur = w0;
      else load_step(r, step, cur);
      // the tokens' 128 elements: 16 lanes a token, 8 elements a lane
      __syncwarp();
      if (lane < kCols) s.inv[warp][lane] = 0.f;
      __syncwarp();
      for (int c = lane >> 4; c < nt; c += 2) {
        const int piece = lane & 15;
        const uint4 v = *reinterpret_cast<const uint4*>(
            a.x + (long long)(s.list[t0 + c] / a.k) * a.d + step * kStep + piece * 8);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float f[8], amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(u[i] << 16);
          f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
        }
        const unsigned half = 0xFFFFu << (lane & 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, o));
        float mul, inv;
        pow2_scale(amax, mul, inv);
        uint4 p;
        p.x = pack_f16x2(f[0] * mul, f[1] * mul);
        p.y = pack_f16x2(f[2] * mul, f[3] * mul);
        p.z = pack_f16x2(f[4] * mul, f[5] * mul);
        p.w = pack_f16x2(f[6] * mul, f[7] * mul);
        *reinterpret_cast<uint4*>(&s.xs[warp][c * kTokStride + (piece & 3) * 64 + (piece >> 2) * 16]) = p;
        if (piece == 0) s.inv[warp][c] = inv;
      }
      __syncwarp();
      mma_step(cur, r.half, s.xs[warp], s.inv[warp], lane, g < nt, acc);
    }
    if (t0) __syncthreads();            // the previous pass's sums have been read
    // gate rows are i = 0, 1, up rows i = 2, 3 of the same column
    const float v = reduce_warps(s, acc, warp, lane, nw, threadIdx.x);
    __shared__ float up[128];
    const int tid = threadIdx.x;
    if (tid >= 128 && tid < 256) up[tid - 128] = v;
    __syncthreads();
    if (tid < 128) {
      const int i = tid >> 6, col = blk * 64 + i * 32 + set * 8 + (tid >> 3 & 7), c = tid & 7;
      if (c < nt) {
        float G = alpha * v, U = alpha * up[tid];
        if (a.clamp > 0.f) {
          G = fminf(fmaxf(G, -a.clamp), a.clamp);
          U = fminf(fmaxf(U, -a.clamp), a.clamp);
        }
        a.h[(long long)s.list[t0 + c] * a.I + col] = G / (1.f + __expf(-G)) * U;
      }
    }
  }
}

// W2 h x score; the CTA that is last of its 32 rows adds the tokens' experts.
__global__ void __launch_bounds__(256, 3) k_decode_w2(const DecodeArgs a) {
  __shared__ Shared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int slot = blockIdx.y, e = slot_expert(a, slot);
  const int blk = blockIdx.x >> 2, set = blockIdx.x & 3;
  const int steps = a.I / kStep;
  Rows r;
  {
    const long long row = (long long)(e < 0 ? 0 : e) * a.d + blk * 128 + set * 8 + g;
    const long long ld = a.I / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.code[i] = a.codes + q * 16 + (row + 32 * i) * ld;
    r.scale = a.sf + (((long long)(e < 0 ? 0 : e) * (a.d / 128) + blk) * (a.I / 64) + (q >> 1)) * 512 +
              (set * 8 + g) * 16;
    r.half = (q & 1) * 16;
  }
  // weights, ids and scales were there before the W13 kernel started
  StepA w0;
  if (warp < steps && e >= 0) load_step(r, warp, w0);
  const bool mine = collect(a, s, slot, e);
  const float alpha = mine ? a.w_scale[e] : 0.f;
  pdl_wait();                            // h is complete
  pdl_trigger();
  const int count = mine ? s.count : 0;
  for (int t0 = 0; t0 < count; t0 += kCols) {
    const int nt = min(kCols, count - t0);
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int step = warp; step < steps; step += nw) {
      StepA cur;
      if (step == warp && t0 == 0) cur = w0;
      else load_step(r, step, cur);
      __syncwarp();
      if (lane < kCols) s.inv[warp][lane] = 0.f;
      __syncwarp();
      // the tokens' 128 elements of h: a warp a token, 4 elements a lane
      for (int c = 0; c < nt; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(
            a.h + (long long)s.list[t0 + c] * a.I + step * kStep + lane * 4);
        float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float mul, inv;
        pow2_scale(amax, mul, inv);
        const uint2 p = make_uint2(pack_f16x2(v.x * mul, v.y * mul), pack_f16x2(v.z * mul, v.w * mul));
        *reinterpret_cast<uint2*>(&s.xs[warp][c * kTokStride + (lane >> 1 & 3) * 64 +
                                              (lane >> 3) * 16 + (lane & 1) * 8]) = p;
        if (lane == 0) s.inv[warp][c] = inv;
      }
      __syncwarp();
      mma_step(cur, r.half, s.xs[warp], s.inv[warp], lane, g < nt, acc);
    }
    if (t0) __syncthreads();
    for (int v0 = threadIdx.x; v0 < 256; v0 += blockDim.x) {
      float v;
      if (v0 == (int)threadIdx.x) {
        v = reduce_warps(s, acc, warp, lane, nw, v0);
      } else {
        const int i = v0 >> 6, gg = v0 >> 3 & 7, c = v0 & 7;
        v = 0.f;
        for (int w = 0; w < nw; ++w)
          v += s.red[w][gg * 4 + (c >> 1)][(i >> 1) * 4 + (i & 1) * 2 + (c & 1)];
      }
      const int i = v0 >> 6, c = v0 & 7;
      if (c < nt) {
        const int p = s.list[t0 + c];
        a.ys[(long long)p * a.d + blk * 128 + i * 32 + set * 8 + (v0 >> 3 & 7)] =
            a.scores[p] * (alpha * v);
      }
    }
  }
  // arrival: the last CTA of these rows sees every other one's ys
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s.last = atomicAdd(&a.arrived[blockIdx.x], 1) == a.slots - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s.last) return;
  for (int v = threadIdx.x; v < a.T * 32; v += blockDim.x) {
    const int t = v >> 5, row = blk * 128 + (v >> 3 & 3) * 32 + set * 8 + (v & 7);
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int p = t * a.k + j;
      if (a.keep[p]) sum += __ldcg(a.ys + (long long)p * a.d + row);
    }
    a.y[(long long)t * a.d + row] = f2bf(sum);
  }
  if (threadIdx.x == 0) a.arrived[blockIdx.x] = 0;
}

int warps_for(int K) {
  const int steps = K / kStep;
  return steps < kMaxWarps ? steps : kMaxWarps;
}

}  // namespace

cudaError_t launch_decode_nvfp4(const DecodeCall& c, cudaStream_t stream) {
  DecodeArgs a = {};
  a.x = static_cast<const uint16_t*>(c.x);
  a.ids = c.ids; a.scores = c.scores;
  a.T = c.T; a.k = c.k; a.d = c.d; a.I = c.I; a.E = c.E;
  a.slots = c.T * c.k < c.E ? c.T * c.k : c.E;
  a.clamp = c.clamp;
  a.h = c.h; a.ys = c.ys; a.keep = c.keep; a.arrived = c.arrived;
  a.y = static_cast<uint16_t*>(c.y);
  a.err = c.err;
  a.codes = c.w13; a.sf = c.w13_sf; a.w_scale = c.w13_scale;
  cudaError_t e = launch_pdl(k_decode_w13, dim3(c.I / 16, a.slots), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  a.codes = c.w2; a.sf = c.w2_sf; a.w_scale = c.w2_scale;
  return launch_pdl(k_decode_w2, dim3(c.d / 32, a.slots), dim3(warps_for(c.I) * 32), 0, stream, a);
}

}  // namespace moe
