// moe_norm.cu -- the norms around a block: the norm after the block with its gate
// and residual scale, joined with the norm before the next block, and the
// gradient of both.
//
//   n    = y * rms(y)^-1 * w_post          (n = y without w_post)
//   out  = residual + alpha * gate * n     (gate: none, [d] or [T])
//   u    = out * rms(out)^-1 * w_pre       rms(v) = sqrt(mean(v^2) + eps)
//
// Everything is computed in fp32 and rounded once, on the way out; u is taken
// from the unrounded out.
//
// Gradient.  With x = out, rs = rms(x)^-1, ry = rms(y)^-1 (1 without w_post),
// t = du * w_pre, q = alpha * gate_c * w_post (the per-channel factors) and g_t
// the token gate:
//   dr  = d_out + rs * t - rs^3 * mean(t x) * x                (also d_residual)
//   dy  = ry * g_t * (q dr - y * ry^2 * mean(q dr y))          (q dr g_t without w_post)
//   dw_pre  = sum_t du x rs         S_c = sum_t g_t dr y ry
//   dw_post = alpha gate_c S        dgate_c = alpha w_post S   dgate_t = ry * sum_c q dr y
// sum_c q dr y splits into sum(q y d_out) + rs sum(q y t) - rs^3 mean(t x) sum(q y x),
// so one reduction over the row gives everything the row needs.
//
// Bound by memory: forward 4, gradient 6 passes over a [T, d] tensor.  At T=8192, d=2048
// in bf16 that is 134 and 201 MB, 19.8 and 29.7 us at the rate of a plain copy; measured
// 22.5 us (6.0 TB/s) and 37.6 us (5.4 TB/s, its second launch included).

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

struct NormArgs {
  int T, d;
  int tpr;                        // threads per row (multiple of 32)
  int gate_kind;                  // MOE_GATE_*
  int param_bf16;                 // w_post, w_pre, gate are bf16 (else fp32)
  float alpha, eps;
  const void* res;  long long ld_res;    // forward: residual; backward: the stream after it
  const void* y;    long long ld_y;
  const void* w_post;
  const void* gate;
  const void* w_pre;
  void* out;        long long ld_out;    // forward: out; backward: d_residual
  void* u;          long long ld_u;      // forward: u; backward: dy
  // backward
  const void* dres; long long ld_dres;
  const void* du;   long long ld_du;
  float* dw_post;
  float* dgate;
  float* dw_pre;
  int accumulate;
  float* partial;                 // [gridDim.x][2][d], NULL: one CTA, final sums directly
  int n_partial;                  // finish kernel
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<uint16_t>(uint16_t v) { return bf2f(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) { return f2bf(v); }

__device__ __forceinline__ void load_vec8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load_vec8(const uint16_t* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_vec8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store_vec8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]),
                                            pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}

// A thread's 8 columns of piece v of a row, W of them next to each other.  Where every
// row is 16-byte aligned and d a multiple of 8, W is 8 if all tensors are bf16 and 4
// if one is fp32 (16 bytes of that one, so that a warp's accesses are whole lines:
// with eight fp32 columns a thread they touch every sector twice: 56 against 39 us for
// the fp32 gradient at T=8192, d=1024).  Else W is 1: a warp's 256
// columns, each 32nd to a lane, so that they lie at constant distances.
template <int W>
__device__ __forceinline__ int col(int v, int e, int li, int tpr) {
  return W == 8 ? (v * tpr + li) * 8 + e
                : W == 4 ? ((2 * v + (e >> 2)) * tpr + li) * 4 + (e & 3)
                         : (v * tpr + (li & ~31)) * 8 + e * 32 + (li & 31);
}

__device__ __forceinline__ void load_vec4(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load_vec4(const uint16_t* p, float* f) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store_vec4(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_vec4(uint16_t* p, const float* f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]));
}

// columns past the row's end read as 0
template <int W, typename T>
__device__ __forceinline__ void load8(const T* p, int v, int li, int tpr, int d, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += W) {
    const int c = col<W>(v, e, li, tpr);
    if (c < d) {
      if constexpr (W == 8) load_vec8(p + c, f);
      else if constexpr (W == 4) load_vec4(p + c, f + e);
      else f[e] = to_f(p[c]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) f[e + i] = 0.f;
    }
  }
}

template <int W, typename T>
__device__ __forceinline__ void store8(T* p, int v, int li, int tpr, int d, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += W) {
    const int c = col<W>(v, e, li, tpr);
    if (c < d) {
      if constexpr (W == 8) store_vec8(p + c, f);
      else if constexpr (W == 4) store_vec4(p + c, f + e);
      else p[c] = from_f<T>(f[e]);
    }
  }
}

__device__ __forceinline__ float param(const void* p, int bf16, long long i) {
  return bf16 ? bf2f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

template <int W, typename P>
__device__ __forceinline__ void load_factors_as(const NormArgs& a, bool y, bool u, int v, int li,
                                                int tpr, float (&q)[8], float (&g)[8],
                                                float (&w)[8]) {
  if (y && a.w_post) load8<W>(static_cast<const P*>(a.w_post), v, li, tpr, a.d, q);
  if (y && a.gate_kind == MOE_GATE_CHANNEL)
    load8<W>(static_cast<const P*>(a.gate), v, li, tpr, a.d, g);
  if (u) load8<W>(static_cast<const P*>(a.w_pre), v, li, tpr, a.d, w);
}
// The row-independent factors of a thread's columns: q = alpha * w_post * channel gate
// (of y) and w_pre (of u; 0 without).  All loads first: one wait instead of three.
template <int W>
__device__ __forceinline__ void load_factors(const NormArgs& a, bool y, bool u, int v, int li,
                                             int tpr, float (&q)[8], float (&w)[8]) {
  float g[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = g[e] = 1.f, w[e] = 0.f;
  if (a.param_bf16)
    load_factors_as<W, uint16_t>(a, y, u, v, li, tpr, q, g, w);
  else
    load_factors_as<W, float>(a, y, u, v, li, tpr, q, g, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = a.alpha * q[e] * g[e];
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sum a value over the tpr threads of a row group of up to WARPS warps (16 or 32): the
// warps' sums in `buf` (one per warp), then every warp adds them in the same order, so
// all threads get the same bits.
template <int WARPS>
__device__ __forceinline__ float group_sum(float s, float* buf, int li, int tpr, int bar) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tpr == 32) return s;
  const int at = li & (WARPS - 1);
  if ((li & 31) == 0) buf[li >> 5] = s;
  group_sync(bar, tpr);
  s = at < tpr / 32 ? buf[at] : 0.f;
#pragma unroll
  for (int o = 1; o < WARPS; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ float inv_rms(float sum_sq, int d, float eps) {
  return rsqrtf(sum_sq * (1.f / (float)d) + eps);
}

// Forward, a row per group of tpr threads and no loop: few rows, and what the stream
// below does not take (d > 8192; tensors that are not 16-byte aligned).  All loads of a
// row are independent; latency bounds it (one row of d=2048 2.3 us, of which a launch is
// most).
template <typename A, typename R, int V, int W>
__global__ void __launch_bounds__(1024) k_block_norm(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  const int tpr = a.tpr, g = threadIdx.x / tpr, li = threadIdx.x - g * tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + g;
  if (row >= a.T) return;                      // whole groups: their barriers are their own
  const int d = a.d;
  float x[V][8], y[V][8], q[V][8], w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load8<W>(static_cast<const R*>(a.res) + row * a.ld_res, v, li, tpr, d, x[v]);
    if (a.y) load8<W>(static_cast<const A*>(a.y) + row * a.ld_y, v, li, tpr, d, y[v]);
    if (V == 1) load_factors<W>(a, a.y, a.u, v, li, tpr, q[v], w[v]);   // else no registers
  }
  if (a.y) {
    float s = 0.f, f = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += y[v][e] * y[v][e];
    if (a.gate_kind == MOE_GATE_TOKEN) f = param(a.gate, a.param_bf16, row);
    if (a.w_post) f *= inv_rms(group_sum<32>(s, &red[0][g * (tpr / 32)], li, tpr, 1 + g), d, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (V > 1) load_factors<W>(a, true, false, v, li, tpr, q[v], w[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] += f * (q[v][e] * y[v][e]);
      store8<W>(static_cast<R*>(a.out) + row * a.ld_out, v, li, tpr, d, x[v]);
    }
  }
  if (a.u) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[v][e] * x[v][e];
    const float rs = inv_rms(group_sum<32>(s, &red[1][g * (tpr / 32)], li, tpr, 1 + g), d, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (V > 1) load_factors<W>(a, false, true, v, li, tpr, q[v], w[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= rs * w[v][e];
      store8<W>(static_cast<A*>(a.u) + row * a.ld_u, v, li, tpr, d, x[v]);
    }
  }
  pdl_trigger();
}


// Pairs of fp32 values and the two-wide arithmetic on them: half the instructions of
// the scalar forms, which is what bounds the row loops.
typedef unsigned long long f2;
__device__ __forceinline__ f2 make_f2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_f2(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum_f2(f2 v) {
  float lo, hi;
  split_f2(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ void to_f2(const float (&f)[8], f2 (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = make_f2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void from_f2(const f2 (&p)[4], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split_f2(p[i], f[2 * i], f[2 * i + 1]);
}

// ---- rows streamed through shared memory ---------------------------------------
//
// Many rows: persistent CTAs of 512 threads, a thread owning 8 V columns of every row
// of its group.  It copies its own pieces of the next rows into its own slots of a
// ring with cp.async and reads them back itself, so a copy in flight costs no register
// and needs no barrier; the parameters of its columns stay in registers.  (One row a
// group without a loop: T=8192, d=2048, bf16: 30.2 us against 22.5.)

constexpr int kStreamThreads = 512;
constexpr int kStreamMaxWidth = kStreamThreads * 8;
constexpr int kStages = 3;

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's slots of one tensor, piece and stage (TH threads): what it copies at a
// time lies TH of them apart, so that a warp reads and writes whole lines.
template <typename T, int TH = kStreamThreads>
__host__ __device__ constexpr int slot_bytes() { return TH * 8 * (int)sizeof(T); }

// Start copying the thread's 8 columns of piece v of the row at `row`.
template <int W, int TH = kStreamThreads, typename T>
__device__ __forceinline__ void slot_copy(uint32_t slot, const T* row, int v, int li, int tpr,
                                          int d) {
  constexpr int bytes = W * (int)sizeof(T);
#pragma unroll
  for (int e = 0; e < 8; e += W) {
    const int c = col<W>(v, e, li, tpr);
    if (c < d) {
      const uint32_t at = slot + (e / W * TH + threadIdx.x) * bytes;
      if constexpr (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(row + c) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(row + c) : "memory");
    }
  }
}
template <int W, int TH = kStreamThreads, typename T>
__device__ __forceinline__ void slot_read(const uint8_t* slot, float (&f)[8], const T*) {
#pragma unroll
  for (int e = 0; e < 8; e += W) {
    const T* p = reinterpret_cast<const T*>(slot) + (e / W * TH + threadIdx.x) * W;
    if constexpr (W == 8) load_vec8(p, f);
    else load_vec4(p, f + e);
  }
}
// A thread's 8 values of a parameter.
template <int TH>
__device__ __forceinline__ void param_read(const uint8_t* slot, float (&f)[8]) {
  load_vec4(reinterpret_cast<const float*>(slot) + threadIdx.x * 4, f);
  load_vec4(reinterpret_cast<const float*>(slot) + (TH + threadIdx.x) * 4, f + 4);
}
template <int TH>
__device__ __forceinline__ void param_write(uint8_t* slot, const float (&f)[8]) {
  *reinterpret_cast<float4*>(slot + threadIdx.x * 16) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(slot + (TH + threadIdx.x) * 16) = make_float4(f[4], f[5], f[6], f[7]);
}

// Rows that are not 16-byte aligned (W = 1; the tensors themselves are): a group copies
// the 16-byte pieces of a row from the one that holds its first element, and reads its
// elements from there after a barrier of the group.  The pieces begin up to 15 bytes
// before the row, in the row before or in what lies between (row 0 is aligned, and rows
// are at least 16 bytes apart: kStagedMinWidth); the last one stops at the row's end.
// Against loads of single elements into registers, one row ahead (us): forward, T=8192,
// d=777, bf16 33.2 -> 25.2; T=8191, d=1023, fp32 36.2 -> 32.3; T=2047, d=8191, bf16
// 85.9 -> 56.2; with the columns of a lane at constant distances 19.9, 26.5 and 43.6.
// Bound by the instructions of single elements (T=8192, d=2047, bf16 39.9); writing whole
// pieces through shared memory too costs more for its barrier than it saves.  (Where the
// rows of a group lie a multiple of 16 bytes apart they all begin at the same offset, and
// columns shifted by it would keep 16-byte accesses: not built.)  The
// gradient of up to 4096 columns keeps its loads (an fp32 residual, T=4099, d=1537: 34.7
// against 39.3 us with copied rows; bf16, T=8192, d=2047: 62.5 against 59.5).
constexpr int kStagedMinWidth = 8;

// A row's slot, and where its first element is in it.
template <typename T>
__host__ __device__ constexpr int row_slot(int d) { return (d * (int)sizeof(T) + 31) / 16 * 16; }
template <typename T>
__device__ __forceinline__ int row_offset(long long row, long long ld) {
  return (int)((unsigned)row * (unsigned)ld * (unsigned)sizeof(T) & 15u);
}
template <typename T>
__device__ __forceinline__ void row_copy(uint32_t slot, const T* row, int li, int tpr, int d) {
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15), bytes = off + d * (int)sizeof(T);
  const uint8_t* const from = reinterpret_cast<const uint8_t*>(row) - off;
  for (int c = li * 16; c < bytes; c += tpr * 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + c), "l"(from + c),
                 "r"(min(16, bytes - c)) : "memory");
}
template <typename T>
__device__ __forceinline__ void row_read(const uint8_t* first, int v, int li, int tpr, int d,
                                         float (&f)[8], const T*) {
  const T* const p = reinterpret_cast<const T*>(first);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = col<1>(v, e, li, tpr);
    f[e] = c < d ? to_f(p[c]) : 0.f;
  }
}
// The copies that a thread has waited for are there for all threads of its group.
__device__ __forceinline__ void group_sees(int bar, int tpr) {
  if (tpr == 32) __syncwarp();
  else group_sync(bar, tpr);
}

// Forward over many rows.
template <typename A, typename R, int V>
__host__ __device__ constexpr int stream_ring_bytes() {
  return kStages * V * (slot_bytes<A>() + slot_bytes<R>());
}
template <typename A, typename R>
__host__ __device__ constexpr int staged_ring_bytes(int d, int groups) {
  return kStages * groups * (row_slot<A>(d) + row_slot<R>(d));
}

template <typename A, typename R, int V, int W>
__global__ void __launch_bounds__(kStreamThreads, V == 1 ? 2 : 1)
    k_block_norm_stream(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][2][kStreamThreads / 32];
  constexpr int kPiece = slot_bytes<A>() + slot_bytes<R>(), kStage = V * kPiece;
  pdl_wait();
  const int tpr = a.tpr, groups = blockDim.x / tpr;
  const int g = threadIdx.x / tpr, li = threadIdx.x - g * tpr, d = a.d;
  const long long first = (long long)blockIdx.x * groups + g;
  const int hop = gridDim.x * groups;
  const uint32_t base = smem_u32(ring);
  const int rows = first < a.T ? (int)((a.T - first + hop - 1) / hop) : 0;   // of the group
  // the rows to fetch next, and the rows to write
  const A* y_in = static_cast<const A*>(a.y) + (a.y ? first * a.ld_y : 0);
  const R* x_in = static_cast<const R*>(a.res) + first * a.ld_res;
  R* out = static_cast<R*>(a.out) + (a.y ? first * a.ld_out : 0);
  A* u_out = static_cast<A*>(a.u) + (a.u ? first * a.ld_u : 0);
  int left = rows;                               // rows not fetched yet
  const int row_bytes = row_slot<A>(d) + row_slot<R>(d);                // W = 1
  auto fetch = [&](int stage) {
    if (left > 0) {
      if constexpr (W > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint32_t at = base + stage * kStage + v * kPiece;
          if (a.y) slot_copy<W>(at, y_in, v, li, tpr, d);
          slot_copy<W>(at + slot_bytes<A>(), x_in, v, li, tpr, d);
        }
      } else {
        const uint32_t at = base + (stage * groups + g) * row_bytes;
        if (a.y) row_copy(at, y_in, li, tpr, d);
        row_copy(at + row_slot<A>(d), x_in, li, tpr, d);
      }
      if (a.y) y_in += hop * a.ld_y;
      x_in += hop * a.ld_res;
      --left;
    }
    cp_async_commit();
  };
  if (W > 1 && (d < 8 * V * tpr || !a.y)) {
    // slots that no copy fills (columns past the row, no y) read as zero
    for (int i = threadIdx.x; i < kStages * kStage / 16; i += blockDim.x)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  f2 q[V][4], w[V][4];         // alpha * w_post * channel gate, w_pre
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float q8[8], w8[8];
    load_factors<W>(a, a.y, a.u, v, li, tpr, q8, w8);
    to_f2(q8, q[v]);
    to_f2(w8, w[v]);
  }
  // the sum of squares of the thread's values
  auto squares = [&](const f2 (&p)[V][4]) {
    f2 s = mul2(p[0][0], p[0][0]);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = v == 0 ? 1 : 0; i < 4; ++i) s = fma2(p[v][i], p[v][i], s);
    return sum_f2(s);
  };
  int stage = 0, flip = 0;
  long long row = first;
  for (int n = 0; n < rows; ++n, row += hop) {
    f2 x[V][4], y[V][4];
    float f = 1.f, t[8];
    if (a.y && a.gate_kind == MOE_GATE_TOKEN) f = param(a.gate, a.param_bf16, row);
    cp_async_wait<kStages - 2>();
    if constexpr (W > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint8_t* at = ring + stage * kStage + v * kPiece;
        slot_read<W>(at, t, y_in);
        to_f2(t, y[v]);
        slot_read<W>(at + slot_bytes<A>(), t, x_in);
        to_f2(t, x[v]);
      }
    } else {
      group_sees(1 + g, tpr);
      const uint8_t* at = ring + (stage * groups + g) * row_bytes;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.y) {
          row_read(at + row_offset<A>(row, a.ld_y), v, li, tpr, d, t, y_in);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = 0.f;
        }
        to_f2(t, y[v]);
        row_read(at + row_slot<A>(d) + row_offset<R>(row, a.ld_res), v, li, tpr, d, t, x_in);
        to_f2(t, x[v]);
      }
    }
    // into the slots read one row ago
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (a.y) {
      if (a.w_post)
        f *= inv_rms(group_sum<16>(squares(y), &red[flip][0][g * (tpr / 32)], li, tpr, 1 + g), d,
                     a.eps);
      const f2 f2x = make_f2(f, f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v][i] = fma2(f2x, mul2(q[v][i], y[v][i]), x[v][i]);
        from_f2(x[v], t);
        store8<W>(out, v, li, tpr, d, t);
      }
    }
    if (a.u) {
      const float rs =
          inv_rms(group_sum<16>(squares(x), &red[flip][1][g * (tpr / 32)], li, tpr, 1 + g), d, a.eps);
      const f2 rs2 = make_f2(rs, rs);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f2 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = mul2(x[v][i], mul2(rs2, w[v][i]));
        from_f2(u, t);
        store8<W>(u_out, v, li, tpr, d, t);
      }
    }
    if (a.y) out += hop * a.ld_out;
    if (a.u) u_out += hop * a.ld_u;
    flip ^= 1;
  }
  pdl_trigger();
}

// The column sums' last step: the parameter gradients of column c from
// P = sum_t du x rs and S = sum_t g_t dr y ry.
__device__ __forceinline__ void put_grad(const NormArgs& a, float* p, int c, float v) {
  p[c] = a.accumulate ? p[c] + v : v;
}
// The factors of S in dw_post and in the channel gate's gradient.
__device__ __forceinline__ float2 gate_factors(const NormArgs& a, int c) {
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  return make_float2(a.dw_post && channel ? param(a.gate, a.param_bf16, c) : 1.f,
                     a.dgate && channel && a.w_post ? param(a.w_post, a.param_bf16, c) : 1.f);
}
__device__ __forceinline__ void gate_grads(const NormArgs& a, int c, float S, float2 f) {
  if (a.dw_post) put_grad(a, a.dw_post, c, a.alpha * S * f.x);
  if (a.dgate && a.gate_kind == MOE_GATE_CHANNEL) put_grad(a, a.dgate, c, a.alpha * S * f.y);
}
__device__ __forceinline__ void param_grads(const NormArgs& a, int c, float P, float S) {
  if (a.dw_pre) put_grad(a, a.dw_pre, c, P);
  gate_grads(a, c, S, gate_factors(a, c));
}

// ---- gradient --------------------------------------------------------------------

// The six row sums over the tpr threads of a group: each exchange halves the values
// a lane still adds (9 shuffles instead of 30), a warp's totals go to buf[warp][8]
// and every warp adds them in the same order.
__device__ __forceinline__ void group_sum6(float (&s)[6], float (*buf)[8], int li, int tpr,
                                           int bar) {
  const int lane = li & 31;
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = s[i], hi = i < 2 ? s[4 + i] : 0.f;
    r[i] = (b4 ? hi : lo) + __shfl_xor_sync(0xffffffffu, b4 ? lo : hi, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r[i] = (b3 ? r[2 + i] : r[i]) + __shfl_xor_sync(0xffffffffu, b3 ? r[i] : r[2 + i], 8);
  float v = (b2 ? r[1] : r[0]) + __shfl_xor_sync(0xffffffffu, b2 ? r[0] : r[1], 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  const int warps = tpr / 32;
  if (warps > 1) {
    if ((lane & 3) == 0) buf[li >> 5][lane >> 2] = v;     // value 4 b4 + 2 b3 + b2
    group_sync(bar, tpr);
    // lane: value lane / 4, of every fourth warp from lane % 4 on
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kStreamThreads / 32; w += 4)
      if (w + (lane & 3) < warps) v += buf[w + (lane & 3)][lane >> 2];
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) s[i] = __shfl_sync(0xffffffffu, v, 4 * i);
}

// What a row's elements need of its six sums.
struct RowFactors {
  float rs, cx;          // 1/rms(x), rs^3 mean(t x)
  float ry, cy, gt;      // 1/rms(y), ry^2 mean(q dr y), token gate
};

// ALL: w_pre and w_post are given.
template <bool ALL>
__device__ __forceinline__ RowFactors row_factors(const NormArgs& a, const float (&s)[6],
                                                  float inv_d, long long row, bool writer) {
  const bool post = ALL || a.w_post;
  RowFactors f;
  f.rs = ALL || a.du ? rsqrtf(s[0] * inv_d + a.eps) : 0.f;
  f.cx = f.rs * (f.rs * (f.rs * (s[1] * inv_d)));      // rs^3 alone leaves fp32's range
  f.ry = post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
  const float D = s[3] + f.rs * s[4] - f.cx * s[5];
  f.gt = 1.f;
  if ((ALL || a.y) && a.gate_kind == MOE_GATE_TOKEN) {
    f.gt = param(a.gate, a.param_bf16, row);
    if (a.dgate && writer) {
      const float v = f.ry * D;
      a.dgate[row] = a.accumulate ? a.dgate[row] + v : v;
    }
  }
  f.cy = post ? f.ry * (f.ry * (D * inv_d)) : 0.f;
  return f;
}

__device__ __forceinline__ void row_sums(float (&s)[6], const float (&x)[8], const float (&y)[8],
                                         const float (&dr)[8], const float (&du)[8],
                                         const float (&wp)[8], const float (&q)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = du[e] * wp[e], qy = q[e] * y[e];
    s[0] += x[e] * x[e];
    s[1] += t * x[e];
    s[2] += y[e] * y[e];
    s[3] += qy * dr[e];
    s[4] += qy * t;
    s[5] += qy * x[e];
  }
}

// dr becomes d_residual, y dy; the column sums take the row's terms.
__device__ __forceinline__ void row_grads(const RowFactors& f, const float (&x)[8], float (&y)[8],
                                          float (&dr)[8], const float (&du)[8],
                                          const float (&wp)[8], const float (&q)[8],
                                          float (&P)[8], float (&S)[8]) {
  const float gy = f.gt * f.ry;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    P[e] += du[e] * (x[e] * f.rs);
    dr[e] += f.rs * (du[e] * wp[e]) - f.cx * x[e];
    S[e] += gy * (dr[e] * y[e]);
    y[e] = gy * (q[e] * dr[e] - f.cy * y[e]);
  }
}

__device__ __forceinline__ bool wants_column_sums(const NormArgs& a) {
  return a.dw_pre || a.dw_post || (a.dgate && a.gate_kind == MOE_GATE_CHANNEL);
}

// The CTA's column sums from sm[2][d]: to `partial`, or (one CTA) to the gradients.
__device__ __forceinline__ void leave_column_sums(const NormArgs& a, const float* sm) {
  const int d = a.d;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    if (a.partial) {
      a.partial[(long long)blockIdx.x * 2 * d + c] = sm[c];
      a.partial[(long long)blockIdx.x * 2 * d + d + c] = sm[d + c];
    } else {
      param_grads(a, c, sm[c], sm[d + c]);
    }
  }
}

// Gradient of rows of up to 4096 columns, up to 8192 with V = 2: row groups walk the
// rows, the next row on its way (through the ring; one piece of unaligned rows in
// registers), the sums of a thread's 8 V columns in registers, its parameters in slots of
// its own.  V = 2 halves what a row costs beside its elements (the reduction, the factors,
// the addresses).
// ALL: every tensor is given.
// Its row loop runs at nine tenths of a copy's rate; the rest of the time are the start,
// the CTAs' column sums and the launch that adds them.  Measured with that launch and a
// channel gate: bf16 T=8192, d=2048 37.7 us, T=4096, d=4096 43, T=2048, d=8192 53 (one row
// at a time: the wait for its sums is not covered), T=2047, d=8191 70, fp32 T=8192, d=1024
// 35; token gate, fp32 residual, T=4099, d=1537 (one piece of single elements) 34.6.
constexpr int kGradThreads = 384;      // with V = 2 and several rows to a CTA
constexpr int kGradStages = 2;

template <int V, int TH>
__host__ __device__ constexpr int grad_param_bytes() { return 2 * V * slot_bytes<float, TH>(); }
template <typename A, typename R, int V, int W, int TH>
__host__ __device__ constexpr int grad_ring_bytes(int d, int groups) {
  return W == 1 && V == 1 ? 0
         : kGradStages * 2 * (W > 1 ? V * (slot_bytes<A, TH>() + slot_bytes<R, TH>())
                                    : groups * (row_slot<A>(d) + row_slot<R>(d)));
}

template <typename A, typename R, int V, int W, int TH, bool ALL>
__global__ void __launch_bounds__(TH, 1) k_block_norm_grad_stream(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];       // ring, then the parameters' slots
  __shared__ __align__(16) float red[2][kStreamThreads / 32][8];
  constexpr int kA = slot_bytes<A, TH>(), kR = slot_bytes<R, TH>(), kF = slot_bytes<float, TH>();
  constexpr int kPiece = 2 * kA + 2 * kR, kStage = V * kPiece;
  constexpr bool kKept = W == 1 && V == 1;       // the next row in registers, not in the ring
  pdl_wait();
  const int tpr = a.tpr, groups = blockDim.x / tpr;
  const int g = threadIdx.x / tpr, li = threadIdx.x - g * tpr, d = a.d;
  uint8_t* const params = kKept ? ring : ring + grad_ring_bytes<A, R, V, W, TH>(d, groups);
  const int slot_a = row_slot<A>(d), slot_r = row_slot<R>(d);            // W = 1
  const bool has_y = ALL || a.y, has_du = ALL || a.du, has_dr = ALL || a.dres;
  const long long first = (long long)blockIdx.x * groups + g;
  const int hop = gridDim.x * groups;
  const int rows = first < a.T ? (int)((a.T - first + hop - 1) / hop) : 0;   // of the group
  // the rows to fetch next, and the rows to write
  const A* y_in = static_cast<const A*>(a.y) + (has_y ? first * a.ld_y : 0);
  const A* du_in = static_cast<const A*>(a.du) + (has_du ? first * a.ld_du : 0);
  const R* x_in = static_cast<const R*>(a.res) + first * a.ld_res;
  const R* dr_in = static_cast<const R*>(a.dres) + (has_dr ? first * a.ld_dres : 0);
  R* dr_out = static_cast<R*>(a.out) + first * a.ld_out;
  A* dy_out = static_cast<A*>(a.u) + (a.u ? first * a.ld_u : 0);
  auto advance = [&]() {
    x_in += hop * a.ld_res;
    if (has_dr) dr_in += hop * a.ld_dres;
    if (has_y) y_in += hop * a.ld_y;
    if (has_du) du_in += hop * a.ld_du;
  };
  int left = rows;                               // rows not fetched yet
  const uint32_t base = smem_u32(ring);
  auto fetch = [&](int stage) {
    if (left > 0) {
      if constexpr (W > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint32_t at = base + stage * kStage + v * kPiece;
          slot_copy<W, TH>(at, x_in, v, li, tpr, d);
          if (has_dr) slot_copy<W, TH>(at + kR, dr_in, v, li, tpr, d);
          if (has_y) slot_copy<W, TH>(at + 2 * kR, y_in, v, li, tpr, d);
          if (has_du) slot_copy<W, TH>(at + 2 * kR + kA, du_in, v, li, tpr, d);
        }
      } else if constexpr (!kKept) {
        const uint32_t at = base + (stage * groups + g) * 2 * (slot_a + slot_r);
        row_copy(at, x_in, li, tpr, d);
        if (has_dr) row_copy(at + slot_r, dr_in, li, tpr, d);
        if (has_y) row_copy(at + 2 * slot_r, y_in, li, tpr, d);
        if (has_du) row_copy(at + 2 * slot_r + slot_a, du_in, li, tpr, d);
      }
      advance();
      --left;
    }
    cp_async_commit();
  };
  // the next row as it is in memory: a conversion would wait for the load
  R nx[8], ndr[8];
  A ny[8], ndu[8];
  auto load = [&]() {
    if (left > 0) {
      auto get = [&](const auto* p, auto (&to)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = col<1>(0, e, li, tpr);
          if (c < d) to[e] = p[c];
        }
      };
      get(x_in, nx);
      if (has_dr) get(dr_in, ndr);
      if (has_y) get(y_in, ny);
      if (has_du) get(du_in, ndu);
      advance();
      --left;
    }
  };
  if (W > 1 && (!ALL || d < 8 * V * tpr)) {
    // slots that no copy fills (columns past the row, absent tensors) read as zero
    for (int i = threadIdx.x; i < kGradStages * kStage / 16; i += blockDim.x)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  if constexpr (kKept) {
#pragma unroll
    for (int e = 0; e < 8; ++e) nx[e] = ndr[e] = 0, ny[e] = ndu[e] = 0;
    load();
  } else {
    fetch(0);
  }
  f2 P[V][4], S[V][4];
  const f2 zero = make_f2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float q8[8], w8[8];
    load_factors<W>(a, has_y, has_du, v, li, tpr, q8, w8);
    param_write<TH>(params + 2 * v * kF, w8);
    param_write<TH>(params + (2 * v + 1) * kF, q8);
#pragma unroll
    for (int i = 0; i < 4; ++i) P[v][i] = S[v][i] = zero;
  }
  const float inv_d = 1.f / (float)d;
  int stage = 0, flip = 0;
  long long row = first;
  for (int n = 0; n < rows; ++n, row += hop) {
    f2 x[4], y[4], dr[4], du[4], wp[4], q[4];
    float f[8];
    // Piece v of the row and of the parameters.  From the ring it is read twice, before
    // and after the reduction: registers that do not hold the row leave room for more
    // rows at a time.
    const uint8_t* const slots =
        ring + (W > 1 ? stage * kStage : (stage * groups + g) * 2 * (slot_a + slot_r));
    int off[4] = {0, 0, 0, 0};
    if constexpr (W == 1 && !kKept) {
      off[0] = row_offset<R>(row, a.ld_res);
      off[1] = slot_r + row_offset<R>(row, a.ld_dres);
      off[2] = 2 * slot_r + row_offset<A>(row, a.ld_y);
      off[3] = 2 * slot_r + slot_a + row_offset<A>(row, a.ld_du);
    }
    auto piece = [&](int v) {
      if constexpr (W > 1) {
        const uint8_t* at = slots + v * kPiece;
        slot_read<W, TH>(at, f, x_in);
        to_f2(f, x);
        slot_read<W, TH>(at + kR, f, x_in);
        to_f2(f, dr);
        slot_read<W, TH>(at + 2 * kR, f, y_in);
        to_f2(f, y);
        slot_read<W, TH>(at + 2 * kR + kA, f, y_in);
        to_f2(f, du);
      } else if constexpr (!kKept) {
        auto get = [&](bool has, int at, const auto* type, f2 (&to)[4]) {
          if (has) row_read(slots + at, v, li, tpr, d, f, type);
          else
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = 0.f;
          to_f2(f, to);
        };
        get(true, off[0], x_in, x);
        get(has_dr, off[1], x_in, dr);
        get(has_y, off[2], y_in, y);
        get(has_du, off[3], y_in, du);
      }
      param_read<TH>(params + 2 * v * kF, f);
      to_f2(f, wp);
      param_read<TH>(params + (2 * v + 1) * kF, f);
      to_f2(f, q);
    };
    if constexpr (kKept) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f(nx[e]);
      to_f2(f, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f(ny[e]);
      to_f2(f, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f(ndr[e]);
      to_f2(f, dr);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f(ndu[e]);
      to_f2(f, du);
      load();
    } else {
      cp_async_wait<0>();
      if (W == 1) group_sees(1 + g, tpr);
      stage ^= 1;
      fetch(stage);                      // into the slots read one row ago
    }
    float s[6];
    {
      f2 z[6] = {zero, zero, zero, zero, zero, zero};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        piece(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 t = mul2(du[i], wp[i]), qy = mul2(q[i], y[i]);
          z[0] = fma2(x[i], x[i], z[0]);
          z[1] = fma2(t, x[i], z[1]);
          z[2] = fma2(y[i], y[i], z[2]);
          z[3] = fma2(qy, dr[i], z[3]);
          z[4] = fma2(qy, t, z[4]);
          z[5] = fma2(qy, x[i], z[5]);
        }
      }
#pragma unroll
      for (int i = 0; i < 6; ++i) s[i] = sum_f2(z[i]);
    }
    group_sum6(s, &red[flip][g * (tpr / 32)], li, tpr, 1 + g);
    flip ^= 1;
    const RowFactors k = row_factors<ALL>(a, s, inv_d, row, li == 0);
    const float gy1 = k.gt * k.ry;
    const f2 rs = make_f2(k.rs, k.rs), ncx = make_f2(-k.cx, -k.cx), gy = make_f2(gy1, gy1),
             ncy = make_f2(-k.cy, -k.cy);
    // dr becomes d_residual, y dy; the column sums take the row's terms
#pragma unroll
    for (int v = 0; v < V; ++v) {
      piece(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        P[v][i] = fma2(du[i], mul2(x[i], rs), P[v][i]);
        dr[i] = fma2(ncx, x[i], fma2(rs, mul2(du[i], wp[i]), dr[i]));
        S[v][i] = fma2(gy, mul2(dr[i], y[i]), S[v][i]);
        y[i] = mul2(gy, fma2(ncy, y[i], mul2(q[i], dr[i])));
      }
      from_f2(dr, f);
      store8<W>(dr_out, v, li, tpr, d, f);
      if (has_y && a.u) {
        from_f2(y, f);
        store8<W>(dy_out, v, li, tpr, d, f);
      }
    }
    dr_out += hop * a.ld_out;
    if (has_y && a.u) dy_out += hop * a.ld_u;
  }
  pdl_trigger();
  if (!wants_column_sums(a)) return;
  cp_async_wait<0>();
  __syncthreads();
  // [group][P, S][d], then the groups in order
  float* const sm = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f[8];
    from_f2(P[v], f);
    store8<W>(sm + (2 * g) * d, v, li, tpr, d, f);
    from_f2(S[v], f);
    store8<W>(sm + (2 * g + 1) * d, v, li, tpr, d, f);
  }
  __syncthreads();
  float* const to = a.partial ? a.partial + (long long)blockIdx.x * 2 * d : sm;
  if (d % 2 == 0) {
    for (int c = 4 * threadIdx.x; c < 2 * d; c += 4 * blockDim.x) {
      float4 v = *reinterpret_cast<const float4*>(sm + c);
      for (int i = 1; i < groups; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(sm + 2 * i * d + c);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      *reinterpret_cast<float4*>(to + c) = v;      // in sm only this thread reads it
    }
  } else {
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
      float v = sm[c];
      for (int i = 1; i < groups; ++i) v += sm[2 * i * d + c];
      to[c] = v;
    }
  }
  if (a.partial) return;
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) param_grads(a, c, sm[c], sm[d + c]);
}

// Gradient of wider rows (d > 8192; d > 4096 with an fp32 tensor or tensors that are not
// 16-byte aligned): a group is the CTA, V pieces of 8 columns a thread, the parameters in
// shared memory.  A row's registers leave no room for the next row, so that its loads are
// waited for: bf16 T=2048, d=8192 took 77 us here when the kernel above took 63; T=2047,
// d=8191 219 against 72.  With a channel gate bf16 T=1000, d=9216 takes 86 us, d=16384 105
// (fp32 131); slowest where four pieces of single elements spill (T=1000, d=9001: 255).
template <typename A, typename R, int V, int W>
__global__ void __launch_bounds__(kStreamThreads, 1) k_block_norm_grad_wide(const NormArgs a) {
  extern __shared__ __align__(16) float wide_sm[];                  // [2][d]: w_pre and q; later P and S
  __shared__ __align__(16) float red[2][kStreamThreads / 32][8];
  pdl_wait();
  const int tpr = a.tpr, li = threadIdx.x, d = a.d;
  float* wpre = wide_sm;
  float* qs = wide_sm + d;
  for (int c = li; c < d; c += tpr) {
    wpre[c] = a.du ? param(a.w_pre, a.param_bf16, c) : 0.f;
    float f = a.alpha;
    if (a.y && a.w_post) f *= param(a.w_post, a.param_bf16, c);
    if (a.y && a.gate_kind == MOE_GATE_CHANNEL) f *= param(a.gate, a.param_bf16, c);
    qs[c] = f;
  }
  __syncthreads();
  float P[V][8], S[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) P[v][e] = S[v][e] = 0.f;
  int flip = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
    // Two pieces of a row are kept over the reduction; four would spill and are read
    // again (without a gate, T=1000, d=16384: bf16 142 -> 90 us, fp32 196 -> 116; with two
    // pieces, d=8192, 95 -> 103).
    constexpr bool kKept = V <= 2;
    float x[kKept ? V : 1][8], y[kKept ? V : 1][8], dr[kKept ? V : 1][8], du[kKept ? V : 1][8];
    float wp[8], q[8];
    auto piece = [&](int v) {
      const int i = kKept ? v : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = dr[i][e] = du[i][e] = 0.f;
      load8<W>(static_cast<const R*>(a.res) + row * a.ld_res, v, li, tpr, d, x[i]);
      if (a.y) load8<W>(static_cast<const A*>(a.y) + row * a.ld_y, v, li, tpr, d, y[i]);
      if (a.dres) load8<W>(static_cast<const R*>(a.dres) + row * a.ld_dres, v, li, tpr, d, dr[i]);
      if (a.du) load8<W>(static_cast<const A*>(a.du) + row * a.ld_du, v, li, tpr, d, du[i]);
    };
    auto factors = [&](int v) {
      load8<W>(wpre, v, li, tpr, d, wp);
      load8<W>(qs, v, li, tpr, d, q);
    };
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (kKept)
#pragma unroll
      for (int v = 0; v < V; ++v) piece(v);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = kKept ? v : 0;
      if (!kKept) piece(v);
      factors(v);
      row_sums(s, x[i], y[i], dr[i], du[i], wp, q);
    }
    group_sum6(s, red[flip], li, tpr, 1);
    const RowFactors f = row_factors<false>(a, s, 1.f / (float)d, row, li == 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = kKept ? v : 0;
      if (!kKept) piece(v);
      factors(v);
      row_grads(f, x[i], y[i], dr[i], du[i], wp, q, P[v], S[v]);
      store8<W>(static_cast<R*>(a.out) + row * a.ld_out, v, li, tpr, d, dr[i]);
      if (a.y && a.u) store8<W>(static_cast<A*>(a.u) + row * a.ld_u, v, li, tpr, d, y[i]);
    }
  }
  pdl_trigger();
  if (!wants_column_sums(a)) return;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    store8<W>(wpre, v, li, tpr, d, P[v]);
    store8<W>(qs, v, li, tpr, d, S[v]);
  }
  __syncthreads();
  leave_column_sums(a, wide_sm);
}

// Adds the CTAs' column sums in order: 32 columns per CTA, 32 slices of the CTAs.  2.5 MB
// at d=2048, from L2: latency (5 us alone, some 3 behind the row kernel's end).
constexpr int kSlices = 32;
__global__ void __launch_bounds__(kSlices * 32) k_block_norm_finish(const NormArgs a) {
  __shared__ float part[32][kSlices + 1];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* const mine = a.partial + (blockIdx.y ? a.d : 0) + c;     // P or S
  const int to = blockIdx.x * 32 + sl;             // the column that this warp's sum is of
  const bool writes = lane == 0 && to < a.d;
  pdl_wait();
  float v = 0.f;
  float2 f = make_float2(0.f, 0.f);
  if (writes && blockIdx.y) f = gate_factors(a, to);
  if (c < a.d)
#pragma unroll 5
    for (int i = sl; i < a.n_partial; i += kSlices) v += mine[(long long)i * 2 * a.d];
  // the slices in order: warp w adds column w's
  part[lane][sl] = v;
  __syncthreads();
  v = part[sl][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (writes) {
    if (blockIdx.y) gate_grads(a, to, v, f);
    else if (a.dw_pre) put_grad(a, a.dw_pre, to, v);
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// host side

// How the rows can be accessed: any rows, rows of aligned tensors (staged), aligned rows
// and parameters.
enum class Access { kAny, kStaged, kVector };

int round32(int n) { return (n + 31) / 32 * 32; }
// ceil(T / n) for T > 0 up to INT_MAX.
int groups_of(int T, int n) { return (T - 1) / n + 1; }

// How the gradient is laid out: pieces of 8 columns a thread, threads of a CTA and of a
// row, rows at a time of a CTA, CTAs.  Two pieces a thread for aligned rows of 1024 to
// 2048 columns with bf16 activations (three rows at a time; T=8192, d=2048: 44 us
// against 49 with one piece) and where one would not do (d=4096: 57 against 46).
struct GradShape {
  int pieces, threads, tpr, groups, grid;
};
GradShape grad_shape(int T, int d, bool vec, bool act_bf16) {
  GradShape s;
  s.pieces = d > 2 * kStreamMaxWidth ? 4 : d > kStreamMaxWidth ? 2 : 1;
  s.threads = kStreamThreads;
  if (vec && act_bf16 && d >= 1024 && d <= 2048) {
    s.pieces = 2;
    s.threads = kGradThreads;
  }
  s.tpr = round32((d + s.pieces * 8 - 1) / (s.pieces * 8));
  s.groups = s.threads / s.tpr;
  // One CTA needs no second launch to add the column sums, but costs more than that as
  // soon as it has a second round of rows: 4 rows, d=2048: 10.3 us against 8.9 on two.
  const int want = T > 0 ? groups_of(T, s.groups) : 1, sms = num_sms();
  s.grid = want < sms ? want : sms;
  return s;
}

// Columns next to each other in a thread's vector accesses (see col()).
template <typename A, typename R>
constexpr int kW = sizeof(A) == 2 && sizeof(R) == 2 ? 8 : 4;

template <typename A, typename R, int V, int W>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t st) {
  const int rows = a.tpr >= 256 ? 1 : 256 / a.tpr;
  return launch_pdl(k_block_norm<A, R, V, W>, dim3(groups_of(a.T, rows)), dim3(rows * a.tpr),
                    0, st, a);
}

template <typename A, typename R, int V, int W>
cudaError_t launch_fwd_stream(NormArgs a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  a.tpr = round32((a.d + 8 * V - 1) / (8 * V));
  const int groups = kStreamThreads / a.tpr, want = groups_of(a.T, groups);
  // the most that a width can take: rows of 4096 V columns' bytes, and 32 more for each row
  constexpr int most =
      W > 1 ? stream_ring_bytes<A, R, V>()
            : kStages * (V * (slot_bytes<A>() + slot_bytes<R>()) + 2 * 16 * 32);
  const int smem = W > 1 ? most : staged_ring_bytes<A, R>(a.d, groups);
  const cudaError_t e = smem_optin_once(k_block_norm_stream<A, R, V, W>, most, done);
  if (e != cudaSuccess) return e;
  const int cap = (V == 1 ? 2 : 1) * num_sms();
  return launch_pdl(k_block_norm_stream<A, R, V, W>, dim3(want < cap ? want : cap),
                    dim3(groups * a.tpr), smem, st, a);
}

template <typename A, typename R>
cudaError_t launch_fwd_types(NormArgs a, Access access, cudaStream_t st) {
  constexpr int W = kW<A, R>;
  const bool vec = access == Access::kVector;
  // More than four rows an SM: the stream (bf16, d=2048, stream against a row a group:
  // 608 rows 3.9 against 3.6 us, 912 rows 5.1 against 6.2).
  if (a.T > 4 * num_sms() && access != Access::kAny) {
    if (a.d <= kStreamMaxWidth)
      return vec ? launch_fwd_stream<A, R, 1, W>(a, st) : launch_fwd_stream<A, R, 1, 1>(a, st);
    if (a.d <= 2 * kStreamMaxWidth)
      return vec ? launch_fwd_stream<A, R, 2, W>(a, st) : launch_fwd_stream<A, R, 2, 1>(a, st);
  }
  // few rows: a row a group, more threads and fewer columns each; d > 8192 needs two
  // pieces
  const bool one = a.d <= 8192;
  a.tpr = round32((a.d + (one ? 7 : 15)) / (one ? 8 : 16));
  if (one) return vec ? launch_fwd<A, R, 1, W>(a, st) : launch_fwd<A, R, 1, 1>(a, st);
  return vec ? launch_fwd<A, R, 2, W>(a, st) : launch_fwd<A, R, 2, 1>(a, st);
}

template <typename... KArgs>
cudaError_t launch_grad(void (*kernel)(KArgs...), std::atomic<unsigned long long>& done,
                        int max_smem, int smem, const NormArgs& a, const GradShape& s,
                        cudaStream_t st) {
  const cudaError_t e = smem_optin_once(kernel, max_smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(s.grid), dim3(s.tpr * s.groups), smem, st, a);
}

template <typename A, typename R, int V, int W, int TH>
cudaError_t launch_grad_stream(const NormArgs& a, const GradShape& s, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0}, done_all{0};
  // the column sums of all groups end up where the ring and the parameters were
  constexpr int sums = 2 * 8 * V * TH * (int)sizeof(float);
  const int rows = grad_ring_bytes<A, R, V, W, TH>(a.d, s.groups) + grad_param_bytes<V, TH>();
  const int smem = rows > sums ? rows : sums;
  // the most that a width can take
  constexpr int stage = 2 * V * (slot_bytes<A, TH>() + slot_bytes<R, TH>()) + 4 * 16 * 32;
  constexpr int most = (W == 1 && V == 1 ? 0 : kGradStages * stage) + grad_param_bytes<V, TH>();
  static_assert(most >= sums, "the column sums fit");
  if (a.y && a.du && a.dres && a.w_post)
    return launch_grad(k_block_norm_grad_stream<A, R, V, W, TH, true>, done_all, most, smem, a, s,
                       st);
  return launch_grad(k_block_norm_grad_stream<A, R, V, W, TH, false>, done, most, smem, a, s, st);
}

template <typename A, typename R, int V, int W>
cudaError_t launch_grad_wide(const NormArgs& a, const GradShape& s, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  return launch_grad(k_block_norm_grad_wide<A, R, V, W>, done,
                     2 * kNormMaxWidth * (int)sizeof(float), 2 * a.d * (int)sizeof(float), a, s,
                     st);
}

template <typename A, typename R>
cudaError_t launch_grad_types(const NormArgs& a, Access access, const GradShape& s,
                              cudaStream_t st) {
  constexpr int W = kW<A, R>;
  const bool vec = access == Access::kVector;
  if (s.pieces == 1)
    return vec ? launch_grad_stream<A, R, 1, W, kStreamThreads>(a, s, st)
               : launch_grad_stream<A, R, 1, 1, kStreamThreads>(a, s, st);
  if constexpr (sizeof(A) == 2)
    if (s.threads == kGradThreads)
      return launch_grad_stream<A, R, 2, W, kGradThreads>(a, s, st);
  if constexpr (sizeof(A) == 2 && sizeof(R) == 2)
    if (s.pieces == 2 && access != Access::kAny)       // fp32 rows would not fit the ring
      return vec ? launch_grad_stream<A, R, 2, W, kStreamThreads>(a, s, st)
                 : launch_grad_stream<A, R, 2, 1, kStreamThreads>(a, s, st);
  if (s.pieces == 4)
    return vec ? launch_grad_wide<A, R, 4, W>(a, s, st) : launch_grad_wide<A, R, 4, 1>(a, s, st);
  return vec ? launch_grad_wide<A, R, 2, W>(a, s, st) : launch_grad_wide<A, R, 2, 1>(a, s, st);
}

int elem(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }
bool known_dtype(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_FP32; }

bool desc_ok(const moe_block_norm_desc* s) {
  return s && s->d >= 1 && s->d <= kNormMaxWidth && known_dtype(s->dtype) &&
         known_dtype(s->residual_dtype) && known_dtype(s->param_dtype) &&
         (s->dtype == MOE_DTYPE_BF16 || s->residual_dtype == MOE_DTYPE_FP32) &&
         s->gate >= MOE_GATE_NONE && s->gate <= MOE_GATE_TOKEN && s->eps >= 0.f;
}

// a [T, d] operand: present, rows at least d apart, aligned to its elements
bool rows_ok(const void* p, long long ld, int d, int dtype) {
  return p && ld >= d && (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem(dtype) - 1)) == 0;
}
bool rows_vec(const void* p, long long ld, int dtype) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * elem(dtype) % 16 == 0);
}
bool base_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool elem_aligned(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem(dtype) - 1)) == 0;
}

NormArgs base_args(const moe_block_norm_desc* s, int T) {
  NormArgs a = {};
  a.T = T;
  a.d = s->d;
  a.gate_kind = s->gate;
  a.param_bf16 = s->param_dtype == MOE_DTYPE_BF16;
  a.alpha = s->alpha;
  a.eps = s->eps;
  return a;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_block_norm_workspace_bytes(const moe_block_norm_desc* s, int T) {
  if (!desc_ok(s) || T < 0) return 0;
  // the widest layout: whether rows are aligned is known with the call
  const bool bf16 = s->dtype == MOE_DTYPE_BF16;
  const int a = grad_shape(T, s->d, true, bf16).grid, b = grad_shape(T, s->d, false, bf16).grid;
  return (size_t)(a > b ? a : b) * 2 * s->d * sizeof(float);
}

extern "C" int moe_block_norm_forward(const moe_block_norm_desc* s, int T, const void* residual,
                                      long long ld_residual, const void* y, long long ld_y,
                                      const void* w_post, const void* gate, const void* w_pre,
                                      void* residual_out, long long ld_out, void* u,
                                      long long ld_u, void* stream) {
  if (!desc_ok(s) || T < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int d = s->d, pt = s->param_dtype;
  if (!rows_ok(residual, ld_residual, d, s->residual_dtype)) return MOE_ERR_INVALID_ARG;
  if (!y && !u) return MOE_ERR_INVALID_ARG;
  if (y && (!rows_ok(y, ld_y, d, s->dtype) ||
            !rows_ok(residual_out, ld_out, d, s->residual_dtype)))
    return MOE_ERR_INVALID_ARG;
  if (!y && (w_post || gate)) return MOE_ERR_INVALID_ARG;
  if (y && (s->gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((u != nullptr) != (w_pre != nullptr)) return MOE_ERR_INVALID_ARG;
  if (u && !rows_ok(u, ld_u, d, s->dtype)) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(w_post, pt) || !elem_aligned(gate, pt) || !elem_aligned(w_pre, pt))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = base_args(s, T);
  a.res = residual; a.ld_res = ld_residual;
  a.y = y; a.ld_y = ld_y;
  a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
  a.out = residual_out; a.ld_out = ld_out;
  a.u = u; a.ld_u = ld_u;
  const bool vec = d % 8 == 0 && rows_vec(residual, ld_residual, s->residual_dtype) &&
                   rows_vec(y, ld_y, s->dtype) && rows_vec(u, ld_u, s->dtype) &&
                   (!y || rows_vec(residual_out, ld_out, s->residual_dtype)) &&
                   base_aligned(w_post) && base_aligned(w_pre) &&
                   (s->gate != MOE_GATE_CHANNEL || base_aligned(gate));
  const Access access = vec ? Access::kVector
                        : d >= kStagedMinWidth && base_aligned(residual) && base_aligned(y)
                            ? Access::kStaged : Access::kAny;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (s->dtype == MOE_DTYPE_FP32)
    e = launch_fwd_types<float, float>(a, access, st);
  else if (s->residual_dtype == MOE_DTYPE_FP32)
    e = launch_fwd_types<uint16_t, float>(a, access, st);
  else
    e = launch_fwd_types<uint16_t, uint16_t>(a, access, st);
  return cuda_result(e, "moe_block_norm_forward");
}

extern "C" int moe_block_norm_backward(
    const moe_block_norm_desc* s, int T, const void* residual_out, long long ld_out, const void* y,
    long long ld_y, const void* d_residual_out, long long ld_dout, const void* d_u,
    long long ld_du, const void* w_post, const void* gate, const void* w_pre, void* d_residual,
    long long ld_dres, void* dy, long long ld_dy, float* dw_post, float* dgate, float* dw_pre,
    int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc_ok(s) || T < 0) return MOE_ERR_INVALID_ARG;
  const int d = s->d, pt = s->param_dtype;
  if ((dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && s->gate == MOE_GATE_NONE) ||
      (dw_post && s->gate == MOE_GATE_CHANNEL && !gate))
    return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(w_post, pt) || !elem_aligned(gate, pt) || !elem_aligned(w_pre, pt) ||
      !elem_aligned(dw_post, MOE_DTYPE_FP32) || !elem_aligned(dgate, MOE_DTYPE_FP32) ||
      !elem_aligned(dw_pre, MOE_DTYPE_FP32))
    return MOE_ERR_INVALID_ARG;
  if (T > 0) {                      // with no rows, tensors of rows may have no address
    if (!y && (!d_u || w_post || gate || dy || dgate)) return MOE_ERR_INVALID_ARG;
    if ((w_pre != nullptr) != (d_u != nullptr)) return MOE_ERR_INVALID_ARG;
    if (y && (s->gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(residual_out, ld_out, d, s->residual_dtype) ||
        !rows_ok(d_residual, ld_dres, d, s->residual_dtype))
      return MOE_ERR_INVALID_ARG;
    if (y && (!rows_ok(y, ld_y, d, s->dtype) || (dy && !rows_ok(dy, ld_dy, d, s->dtype))))
      return MOE_ERR_INVALID_ARG;
    if (d_residual_out && !rows_ok(d_residual_out, ld_dout, d, s->residual_dtype))
      return MOE_ERR_INVALID_ARG;
    if (d_u && !rows_ok(d_u, ld_du, d, s->dtype)) return MOE_ERR_INVALID_ARG;
  } else {
    y = d_u = nullptr;              // the column sums below become 0
  }
  NormArgs a = base_args(s, T);
  a.res = residual_out; a.ld_res = ld_out;
  a.y = y; a.ld_y = ld_y;
  a.dres = d_residual_out; a.ld_dres = ld_dout;
  a.du = d_u; a.ld_du = ld_du;
  a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
  a.out = d_residual; a.ld_out = ld_dres;
  a.u = dy; a.ld_u = ld_dy;
  a.dw_post = dw_post; a.dgate = dgate; a.dw_pre = dw_pre;
  a.accumulate = accumulate ? 1 : 0;
  const bool sums = dw_pre || dw_post || (dgate && s->gate == MOE_GATE_CHANNEL);
  if (T == 0 && (!sums || accumulate)) return MOE_OK;
  const bool vec = d % 8 == 0 && rows_vec(residual_out, ld_out, s->residual_dtype) &&
                   rows_vec(y, ld_y, s->dtype) &&
                   rows_vec(d_residual_out, ld_dout, s->residual_dtype) &&
                   rows_vec(d_u, ld_du, s->dtype) &&
                   rows_vec(d_residual, ld_dres, s->residual_dtype) &&
                   rows_vec(dy, ld_dy, s->dtype) && base_aligned(w_post) && base_aligned(w_pre) &&
                   (s->gate != MOE_GATE_CHANNEL || base_aligned(gate));
  // no rows: one CTA, which writes zero sums
  const Access access = vec ? Access::kVector
                        : d >= kStagedMinWidth && base_aligned(residual_out) && base_aligned(y) &&
                                  base_aligned(d_residual_out) && base_aligned(d_u)
                            ? Access::kStaged : Access::kAny;
  const GradShape shape = grad_shape(T, d, vec, s->dtype == MOE_DTYPE_BF16);
  a.tpr = shape.tpr;
  if (sums && shape.grid > 1) {
    if (!workspace || workspace_bytes < (size_t)shape.grid * 2 * d * sizeof(float))
      return MOE_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return MOE_ERR_INVALID_ARG;
    a.partial = static_cast<float*>(workspace);
  }
  a.n_partial = shape.grid;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (s->dtype == MOE_DTYPE_FP32)
    e = launch_grad_types<float, float>(a, access, shape, st);
  else if (s->residual_dtype == MOE_DTYPE_FP32)
    e = launch_grad_types<uint16_t, float>(a, access, shape, st);
  else
    e = launch_grad_types<uint16_t, uint16_t>(a, access, shape, st);
  if (e == cudaSuccess && a.partial)
    e = launch_pdl(k_block_norm_finish, dim3((d + 31) / 32, 2), dim3(kSlices * 32), 0, st, a);
  return cuda_result(e, "moe_block_norm_backward");
}
