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
// Bound by memory: forward 4, gradient 6 passes over a [T, d] tensor.

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

// A thread's 8 columns of piece v of a row: consecutive ones where every row is
// 16-byte aligned and d a multiple of 8 (VEC), else one of each tpr columns.
template <bool VEC>
__device__ __forceinline__ int col(int v, int e, int li, int tpr) {
  return VEC ? (v * tpr + li) * 8 + e : (v * 8 + e) * tpr + li;
}

// columns past the row's end read as 0
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* p, int v, int li, int tpr, int d, float (&f)[8]) {
  if (VEC) {
    const int c = col<true>(v, 0, li, tpr);
    if (c < d) {
      load_vec8(p + c, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col<false>(v, e, li, tpr);
      f[e] = c < d ? to_f(p[c]) : 0.f;
    }
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int v, int li, int tpr, int d, const float (&f)[8]) {
  if (VEC) {
    const int c = col<true>(v, 0, li, tpr);
    if (c < d) store_vec8(p + c, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col<false>(v, e, li, tpr);
      if (c < d) p[c] = from_f<T>(f[e]);
    }
  }
}

// parameters (fp32 or bf16), at the same columns
template <bool VEC>
__device__ __forceinline__ void load8_param(const void* p, int bf16, int v, int li, int tpr, int d,
                                            float (&f)[8]) {
  if (bf16)
    load8<VEC>(static_cast<const uint16_t*>(p), v, li, tpr, d, f);
  else
    load8<VEC>(static_cast<const float*>(p), v, li, tpr, d, f);
}

__device__ __forceinline__ float param(const void* p, int bf16, long long i) {
  return bf16 ? bf2f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sum N values over the tpr threads of a row group (warps summed in order, so
// every thread of the group gets the same bits).  `buf`: [warps of the group][N].
template <int N>
__device__ __forceinline__ void group_sum(float (&s)[N], float* buf, int li, int tpr, int bar) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (tpr == 32) return;
  if ((li & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[(li >> 5) * N + i] = s[i];
  group_sync(bar, tpr);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  for (int w = 0; w < tpr / 32; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += buf[w * N + i];
}

__device__ __forceinline__ float inv_rms(float sum_sq, int d, float eps) {
  return 1.f / sqrtf(sum_sq / (float)d + eps);
}

// Forward: one row per group of tpr threads, held in registers.
template <typename A, typename R, int V, bool VEC>
__global__ void __launch_bounds__(1024) k_block_norm(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  const int tpr = a.tpr, g = threadIdx.x / tpr, li = threadIdx.x - g * tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + g;
  if (row >= a.T) return;                      // whole groups: their barriers are their own
  const int d = a.d;
  float x[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
    load8<VEC>(static_cast<const R*>(a.res) + row * a.ld_res, v, li, tpr, d, x[v]);
  if (a.y) {
    float y[V][8];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load8<VEC>(static_cast<const A*>(a.y) + row * a.ld_y, v, li, tpr, d, y[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += y[v][e] * y[v][e];
    }
    float f = a.alpha;
    if (a.gate_kind == MOE_GATE_TOKEN) f *= param(a.gate, a.param_bf16, row);
    if (a.w_post) {
      group_sum(s, &red[0][g * (tpr / 32)], li, tpr, 1 + g);
      f *= inv_rms(s[0], d, a.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.w_post) {
        float w[8];
        load8_param<VEC>(a.w_post, a.param_bf16, v, li, tpr, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] *= w[e];
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        float w[8];
        load8_param<VEC>(a.gate, a.param_bf16, v, li, tpr, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] += f * y[v][e];
      store8<VEC>(static_cast<R*>(a.out) + row * a.ld_out, v, li, tpr, d, x[v]);
    }
  }
  if (a.u) {
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[v][e] * x[v][e];
    group_sum(s, &red[1][g * (tpr / 32)], li, tpr, 1 + g);
    const float rs = inv_rms(s[0], d, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[8];
      load8_param<VEC>(a.w_pre, a.param_bf16, v, li, tpr, d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = x[v][e] * rs * w[e];
      store8<VEC>(static_cast<A*>(a.u) + row * a.ld_u, v, li, tpr, d, w);
    }
  }
  pdl_trigger();
}

// The column sums' last step: the parameter gradients of column c from
// P = sum_t du x rs and S = sum_t g_t dr y ry.
__device__ __forceinline__ void param_grads(const NormArgs& a, int c, float P, float S) {
  auto put = [&](float* p, float v) { p[c] = a.accumulate ? p[c] + v : v; };
  if (a.dw_pre) put(a.dw_pre, P);
  if (a.dw_post)
    put(a.dw_post, a.alpha * S *
                       (a.gate_kind == MOE_GATE_CHANNEL ? param(a.gate, a.param_bf16, c) : 1.f));
  if (a.dgate && a.gate_kind == MOE_GATE_CHANNEL)
    put(a.dgate, a.alpha * S * (a.w_post ? param(a.w_post, a.param_bf16, c) : 1.f));
}

constexpr int kGradThreads = 512;

// Gradient: row groups walk the rows; a thread keeps the column sums P and S of
// its columns in registers, the CTA adds its groups' sums in order and leaves
// them in `partial` (k_block_norm_finish adds the CTAs').
template <typename A, typename R, int V, bool VEC>
__global__ void __launch_bounds__(kGradThreads) k_block_norm_grad(const NormArgs a) {
  extern __shared__ float sm[];                // [2][d]: w_pre and q; later P and S
  __shared__ float red[2][kGradThreads / 32 * 6];
  pdl_wait();
  const int tpr = a.tpr, groups = blockDim.x / tpr;
  const int g = threadIdx.x / tpr, li = threadIdx.x - g * tpr;
  const int d = a.d;
  float* wpre = sm;
  float* q = sm + d;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    wpre[c] = a.du ? param(a.w_pre, a.param_bf16, c) : 0.f;
    float f = a.alpha;
    if (a.y && a.w_post) f *= param(a.w_post, a.param_bf16, c);
    if (a.y && a.gate_kind == MOE_GATE_CHANNEL) f *= param(a.gate, a.param_bf16, c);
    q[c] = f;
  }
  __syncthreads();
  float P[V][8], S[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) P[v][e] = S[v][e] = 0.f;
  const float inv_d = 1.f / (float)d;
  int flip = 0;
  for (long long row = (long long)blockIdx.x * groups + g; row < a.T;
       row += (long long)gridDim.x * groups, flip ^= 1) {
    float x[V][8], y[V][8], dr[V][8], du[V][8];
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[v][e] = dr[v][e] = du[v][e] = 0.f;
      load8<VEC>(static_cast<const R*>(a.res) + row * a.ld_res, v, li, tpr, d, x[v]);
      if (a.y) load8<VEC>(static_cast<const A*>(a.y) + row * a.ld_y, v, li, tpr, d, y[v]);
      if (a.dres) load8<VEC>(static_cast<const R*>(a.dres) + row * a.ld_dres, v, li, tpr, d, dr[v]);
      if (a.du) load8<VEC>(static_cast<const A*>(a.du) + row * a.ld_du, v, li, tpr, d, du[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col<VEC>(v, e, li, tpr);
        if (c < d) {
          const float t = du[v][e] * wpre[c], qy = q[c] * y[v][e];
          s[0] += x[v][e] * x[v][e];
          s[1] += t * x[v][e];
          s[2] += y[v][e] * y[v][e];
          s[3] += qy * dr[v][e];
          s[4] += qy * t;
          s[5] += qy * x[v][e];
        }
      }
    group_sum(s, &red[flip][g * (tpr / 32) * 6], li, tpr, 1 + g);
    const float rs = a.du ? inv_rms(s[0], d, a.eps) : 0.f;
    const float cx = rs * rs * rs * (s[1] * inv_d);
    const float ry = a.w_post ? inv_rms(s[2], d, a.eps) : 1.f;
    const float D = s[3] + rs * s[4] - cx * s[5];
    float gt = 1.f;
    if (a.y && a.gate_kind == MOE_GATE_TOKEN) {
      gt = param(a.gate, a.param_bf16, row);
      if (a.dgate && li == 0) {
        const float v = ry * D;
        a.dgate[row] = a.accumulate ? a.dgate[row] + v : v;
      }
    }
    const float cy = a.w_post ? ry * ry * D * inv_d : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col<VEC>(v, e, li, tpr);
        const float wp = c < d ? wpre[c] : 0.f, qc = c < d ? q[c] : 0.f;
        P[v][e] += du[v][e] * x[v][e] * rs;
        dr[v][e] += rs * (du[v][e] * wp) - cx * x[v][e];
        S[v][e] += gt * ry * dr[v][e] * y[v][e];
        o[e] = ry * gt * (qc * dr[v][e] - cy * y[v][e]);
      }
      store8<VEC>(static_cast<R*>(a.out) + row * a.ld_out, v, li, tpr, d, dr[v]);
      if (a.y && a.u) store8<VEC>(static_cast<A*>(a.u) + row * a.ld_u, v, li, tpr, d, o);
    }
  }
  pdl_trigger();
  if (!a.dw_pre && !a.dw_post && !(a.dgate && a.gate_kind == MOE_GATE_CHANNEL)) return;
  for (int i = 0; i < groups; ++i) {
    __syncthreads();
    if (g == i) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = col<VEC>(v, e, li, tpr);
          if (c < d) {
            wpre[c] = (i ? wpre[c] : 0.f) + P[v][e];
            q[c] = (i ? q[c] : 0.f) + S[v][e];
          }
        }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    if (a.partial) {
      a.partial[(long long)blockIdx.x * 2 * d + c] = wpre[c];
      a.partial[(long long)blockIdx.x * 2 * d + d + c] = q[c];
    } else {
      param_grads(a, c, wpre[c], q[c]);
    }
  }
}

// Adds the CTAs' column sums in order: 32 columns per CTA, 8 slices of the CTAs.
__global__ void __launch_bounds__(256) k_block_norm_finish(const NormArgs a) {
  __shared__ float part[2][8][32];
  pdl_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  float P = 0.f, S = 0.f;
  if (c < a.d)
    for (int i = sl; i < a.n_partial; i += 8) {
      P += a.partial[(long long)i * 2 * a.d + c];
      S += a.partial[(long long)i * 2 * a.d + a.d + c];
    }
  part[0][sl][threadIdx.x & 31] = P;
  part[1][sl][threadIdx.x & 31] = S;
  __syncthreads();
  if (sl == 0 && c < a.d) {
    P = S = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      P += part[0][i][threadIdx.x & 31];
      S += part[1][i][threadIdx.x & 31];
    }
    param_grads(a, c, P, S);
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// host side

int round32(int n) { return (n + 31) / 32 * 32; }

int grad_pieces(int d) { return d <= kGradThreads * 16 ? 2 : 4; }
int grad_tpr(int d) { return round32((d + grad_pieces(d) * 8 - 1) / (grad_pieces(d) * 8)); }
int grad_groups(int d) { return kGradThreads / grad_tpr(d); }
int grad_grid(int T, int d) {
  const int per = grad_groups(d), want = (T + per - 1) / per, sms = num_sms();
  return want < sms ? want : sms;
}

template <typename A, typename R, int V, bool VEC>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t st) {
  const int rows = a.tpr >= 256 ? 1 : 256 / a.tpr;
  return launch_pdl(k_block_norm<A, R, V, VEC>, dim3((a.T + rows - 1) / rows), dim3(rows * a.tpr),
                    0, st, a);
}

template <typename A, typename R>
cudaError_t launch_fwd_types(NormArgs a, bool vec, cudaStream_t st) {
  // few rows: more threads and fewer columns each; d > 8192 needs two pieces
  const bool one = a.d <= 8192 && a.T < 4 * num_sms();
  a.tpr = round32((a.d + (one ? 7 : 15)) / (one ? 8 : 16));
  if (one) return vec ? launch_fwd<A, R, 1, true>(a, st) : launch_fwd<A, R, 1, false>(a, st);
  return vec ? launch_fwd<A, R, 2, true>(a, st) : launch_fwd<A, R, 2, false>(a, st);
}

template <typename A, typename R, int V, bool VEC>
cudaError_t launch_grad(const NormArgs& a, int grid, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const int smem = 2 * a.d * (int)sizeof(float);
  cudaError_t e = smem_optin_once(k_block_norm_grad<A, R, V, VEC>, 2 * kNormMaxWidth * 4, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_block_norm_grad<A, R, V, VEC>, dim3(grid),
                    dim3(a.tpr * grad_groups(a.d)), smem, st, a);
}

template <typename A, typename R>
cudaError_t launch_grad_types(const NormArgs& a, bool vec, int grid, cudaStream_t st) {
  if (grad_pieces(a.d) == 2)
    return vec ? launch_grad<A, R, 2, true>(a, grid, st) : launch_grad<A, R, 2, false>(a, grid, st);
  return vec ? launch_grad<A, R, 4, true>(a, grid, st) : launch_grad<A, R, 4, false>(a, grid, st);
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
bool vec_param(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
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
  return (size_t)grad_grid(T > 0 ? T : 1, s->d) * 2 * s->d * sizeof(float);
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
                   vec_param(w_post) && vec_param(w_pre) &&
                   (s->gate != MOE_GATE_CHANNEL || vec_param(gate));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (s->dtype == MOE_DTYPE_FP32)
    e = launch_fwd_types<float, float>(a, vec, st);
  else if (s->residual_dtype == MOE_DTYPE_FP32)
    e = launch_fwd_types<uint16_t, float>(a, vec, st);
  else
    e = launch_fwd_types<uint16_t, uint16_t>(a, vec, st);
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
  a.tpr = grad_tpr(d);
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
  // no rows: one CTA, which writes zero sums
  const int grid = T > 0 ? grad_grid(T, d) : 1;
  if (sums && grid > 1) {
    if (!workspace || workspace_bytes < (size_t)grid * 2 * d * sizeof(float))
      return MOE_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return MOE_ERR_INVALID_ARG;
    a.partial = static_cast<float*>(workspace);
  }
  a.n_partial = grid;
  const bool vec = d % 8 == 0 && rows_vec(residual_out, ld_out, s->residual_dtype) &&
                   rows_vec(y, ld_y, s->dtype) &&
                   rows_vec(d_residual_out, ld_dout, s->residual_dtype) &&
                   rows_vec(d_u, ld_du, s->dtype) &&
                   rows_vec(d_residual, ld_dres, s->residual_dtype) &&
                   rows_vec(dy, ld_dy, s->dtype);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (s->dtype == MOE_DTYPE_FP32)
    e = launch_grad_types<float, float>(a, vec, grid, st);
  else if (s->residual_dtype == MOE_DTYPE_FP32)
    e = launch_grad_types<uint16_t, float>(a, vec, grid, st);
  else
    e = launch_grad_types<uint16_t, uint16_t>(a, vec, grid, st);
  if (e == cudaSuccess && a.partial)
    e = launch_pdl(k_block_norm_finish, dim3((d + 31) / 32), dim3(256), 0, st, a);
  return cuda_result(e, "moe_block_norm_backward");
}
