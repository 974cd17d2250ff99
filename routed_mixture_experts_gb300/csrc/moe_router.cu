// moe_router.cu -- the router: top-k ids and scores from logits, per-expert
// counts, the balance and z losses, and their gradient.
//
//   key = l + bias (selection only); ids = the k largest keys of a row, ties to
//   the lowest index
//   p = softmax(l), or sigmoid(l) / sum sigmoid(l)
//   balance = E/(k N^2) sum_e counts_e P_e, P_e = sum_t p_te, N live tokens
//   z = 1/N sum_t lse_t^2
//
// Gradient.  The counts are constants, so dbalance/dp_te = b_e = E counts_e/(k N^2).
// With v = the gradient at the chosen scores times `scale`:
//   softmax       G = b + v at the chosen; dl = p (G - sum G p) + p 2 lse dz/N
//   softmax_topk  G = b; the same, plus s'_j (v_j - sum v s') at the chosen
//   sigmoid       dl = (1-sigma) (p (b - sum b p) + s'_j (v_j - sum v s') at the chosen)
// (s' the normalised chosen scores).
//
// A warp holds a row: expert e = lane + 32 i in slot i, so loads and stores are
// coalesced and every sum over experts is one warp reduction.

#include <cmath>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxE = 256;
constexpr unsigned kAll = 0xffffffffu;

struct RouterArgs {
  int T, E, k, scoring;
  float scale;
  const void* logits;  long long ld;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* scores;
  int32_t* counts;       // [E+1]
  float* prob_sum;       // [E]
  float* losses;         // [2]
  float* row_stat;       // [T]
  // per-CTA sums (NULL with one CTA): probabilities [n][E], counts [n][E+1], z [n]
  float* part_prob;
  int32_t* part_count;
  float* part_z;
  int n_part;
  // gradient
  const float* d_scores;
  const float* d_losses;
  void* d_logits;  long long ld_d;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = f2bf(v); }

// fp32 to an unsigned integer of the same order; NaN below every number, -0 = +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {      // NaN only if every lane's is
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// A row's weights, before they are divided by their sum: exp(l - top) for the
// softmax, sigmoid(l) * exp(-top) for the sigmoid, with top the largest logit (the
// sigmoid: at most 0), so that the sum neither overflows nor underflows.
__device__ __forceinline__ float weight(float l, float top, bool sig) {
  if (l == -INFINITY) return 0.f;
  if (!sig) return expf(l - top);
  return l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - top) / (1.f + expf(l));
}

// The losses from the whole sums (threads 0..E-1 hold their expert's): one warp
// sum per warp, the warps added in order by thread 0.
__device__ __forceinline__ void write_sums(const RouterArgs& a, int count, float prob, int live,
                                           float z, float* red) {
  const int e = threadIdx.x;
  float v = 0.f;
  if (e < a.E) {
    a.counts[e] = count;
    a.prob_sum[e] = prob;
    v = (float)count * prob;
  }
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += red[w];
    const float n = live > 0 ? (float)live : 1.f;
    a.counts[a.E] = live;
    a.losses[0] = s / n * ((float)a.E / (float)a.k) / n;
    a.losses[1] = z / n;
  }
}

// Forward.  L = logits type, NV = slots of 32 experts.
template <typename L, int NV>
__global__ void __launch_bounds__(1024) k_router(const RouterArgs a) {
  __shared__ int cnt[kMaxE];
  __shared__ float psum[kMaxE];
  __shared__ float zsum[32], red[32];
  __shared__ int nlive;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int E = a.E, k = a.k;
  for (int e = threadIdx.x; e < kMaxE; e += blockDim.x) {
    cnt[e] = 0;
    psum[e] = 0.f;
  }
  if (threadIdx.x == 0) nlive = 0;
  __syncthreads();
  float ps[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) ps[i] = 0.f;
  float z = 0.f;
  int live_rows = 0;
  for (long long t = (long long)blockIdx.x * nw + warp; t < a.T; t += (long long)gridDim.x * nw) {
    const L* row = static_cast<const L*>(a.logits) + t * a.ld;
    int32_t* ids = a.ids + t * k;
    float* scores = a.scores + t * k;
    const bool sig = a.scoring == MOE_ROUTER_SIGMOID;
    if (a.mask && !a.mask[t]) {
      // padding: the row is not read; ids spread over the experts
      for (int j = lane; j < k; j += 32) {
        ids[j] = (int32_t)((t * k + j) % E);
        scores[j] = 0.f;
      }
      if (lane == 0) a.row_stat[t] = -INFINITY;
      continue;
    }
    float l[NV];
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? load_logit(row + e) : -INFINITY;
      key[i] = e < E ? order_key(a.bias ? l[i] + a.bias[e] : l[i]) : 0u;
    }
    // selection; a taken slot's key becomes 0 and its bit in `taken` is set
    uint32_t taken = 0u;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0u;
      int at = kMaxE;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i) {
        const bool open = !(taken >> i & 1u) && lane + 32 * i < E;
        if (open && key[i] >= best) {
          best = key[i];
          at = lane + 32 * i;
        }
      }
      const uint32_t top = __reduce_max_sync(kAll, best);
      const int e = (int)__reduce_min_sync(kAll, best == top ? (unsigned)at : (unsigned)kMaxE);
      if ((e & 31) == lane) taken |= 1u << (e >> 5);
      if (lane == 0) ids[j] = e;
    }
    float mx = l[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      mx = fmaxf(mx, l[i]);
      nan |= l[i] != l[i];
    }
    mx = warp_max(mx);
    nan = __any_sync(kAll, nan);
    const bool live = nan || mx > -INFINITY;
    __syncwarp();                          // lane 0's ids are visible to the warp
    if (!live) {
      for (int j = lane; j < k; j += 32) scores[j] = 0.f;
      if (lane == 0) a.row_stat[t] = -INFINITY;
      continue;
    }
    live_rows += 1;
    const float top = sig ? fminf(mx, 0.f) : mx;
    float p[NV], total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = lane + 32 * i < E ? weight(l[i], top, sig) : 0.f;
      total += p[i];
    }
    total = warp_sum(total);
    const float stat = top + logf(total);
    const float inv = 1.f / total;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] *= inv;
      ps[i] += p[i];
    }
    if (lane == 0) a.row_stat[t] = stat;
    if (!sig) z += stat * stat;
    // the chosen: scores and counts
    float ctop = top, csum = total;
    if (a.scoring != MOE_ROUTER_SOFTMAX) {
      ctop = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (taken >> i & 1u) ctop = fmaxf(ctop, l[i]);
      ctop = warp_max(ctop);
      if (sig) ctop = fminf(ctop, 0.f);
      csum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (taken >> i & 1u) csum += weight(l[i], ctop, sig);
      csum = warp_sum(csum);
    }
    for (int j = lane; j < k; j += 32) {
      const int e = ids[j];
      const float c = load_logit(row + e);
      const float s = csum == 0.f ? 0.f : weight(c, ctop, sig) / csum;
      scores[j] = s * a.scale;
      if (c != -INFINITY) atomicAdd(&cnt[e], 1);
    }
  }
  pdl_trigger();
  // the warps' sums, added in order
  for (int w = 0; w < nw; ++w) {
    __syncthreads();
    if (warp == w) {
#pragma unroll
      for (int i = 0; i < NV; ++i) psum[lane + 32 * i] += ps[i];
      if (lane == 0) {
        zsum[w] = z;
        nlive += live_rows;
      }
    }
  }
  __syncthreads();
  z = 0.f;
  for (int w = 0; w < nw; ++w) z += zsum[w];
  if (a.part_prob) {
    const long long b = blockIdx.x;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      a.part_prob[b * E + e] = psum[e];
      a.part_count[b * (E + 1) + e] = cnt[e];
    }
    if (threadIdx.x == 0) {
      a.part_count[b * (E + 1) + E] = nlive;
      a.part_z[b] = z;
    }
  } else {
    const int e = threadIdx.x < kMaxE ? threadIdx.x : 0;
    write_sums(a, cnt[e], psum[e], nlive, z, red);
  }
}

// Adds the CTAs' sums in order: 4 slices of the CTAs per expert.
__global__ void __launch_bounds__(1024) k_router_finish(const RouterArgs a) {
  __shared__ float sp[4][kMaxE];
  __shared__ int sc[4][kMaxE];
  __shared__ float red[32];
  __shared__ float zs[32];
  __shared__ int ls[32];
  pdl_wait();
  const int e = threadIdx.x & (kMaxE - 1), sl = threadIdx.x / kMaxE;
  float P = 0.f;
  int c = 0;
  if (e < a.E)
    for (int b = sl; b < a.n_part; b += 4) {
      P += a.part_prob[(long long)b * a.E + e];
      c += a.part_count[(long long)b * (a.E + 1) + e];
    }
  sp[sl][e] = P;
  sc[sl][e] = c;
  float z = 0.f;
  int live = 0;
  for (int b = threadIdx.x; b < a.n_part; b += blockDim.x) {
    z += a.part_z[b];
    live += a.part_count[(long long)b * (a.E + 1) + a.E];
  }
  z = warp_sum(z);
  live = __reduce_add_sync(kAll, live);
  if ((threadIdx.x & 31) == 0) {
    zs[threadIdx.x >> 5] = z;
    ls[threadIdx.x >> 5] = live;
  }
  __syncthreads();
  z = 0.f;
  live = 0;
  for (int w = 0; w < 32; ++w) {
    z += zs[w];
    live += ls[w];
  }
  P = 0.f;
  c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    P += sp[i][e];
    c += sc[i][e];
  }
  write_sums(a, c, P, live, z, red);
  pdl_trigger();
}

// Gradient: a warp per row, as the forward.  `extra` holds the chosen experts'
// own terms of the warp's row.
constexpr int kGradWarps = 8;

template <typename L, int NV>
__global__ void __launch_bounds__(kGradWarps * 32) k_router_grad(const RouterArgs a) {
  __shared__ float extra[kGradWarps][kMaxE];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E, k = a.k;
  const bool sig = a.scoring == MOE_ROUTER_SIGMOID;
  float* ex = extra[warp];
#pragma unroll
  for (int i = 0; i < NV; ++i) ex[lane + 32 * i] = 0.f;
  const int live_n = a.counts[E];
  const float n = live_n > 0 ? (float)live_n : 1.f;
  float b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    b[i] = (e < E && a.d_losses)
               ? a.d_losses[0] * ((float)E / (float)k) * (float)a.counts[e] / n / n : 0.f;
  }
  const float dz = (a.d_losses && !sig) ? a.d_losses[1] * 2.f / n : 0.f;
  __syncwarp();
  for (long long t = (long long)blockIdx.x * kGradWarps + warp; t < a.T;
       t += (long long)gridDim.x * kGradWarps) {
    const L* row = static_cast<const L*>(a.logits) + t * a.ld;
    L* out = static_cast<L*>(a.d_logits) + t * a.ld_d;
    const float stat = a.row_stat[t];
    const bool live = stat != -INFINITY;
    if (!live) {                            // padding, or nothing to choose: no gradient
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane + 32 * i < E) store_logit(out + lane + 32 * i, 0.f);
      continue;
    }
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? load_logit(row + e) : -INFINITY;
    }
    if (a.d_scores) {
      const int32_t* ids = a.ids + t * k;
      const float* ds = a.d_scores + t * k;
      // normalised chosen scores s', their sum C and sum v s'
      float ctop = -INFINITY, csum = 0.f, vs = 0.f;
      if (a.scoring != MOE_ROUTER_SOFTMAX) {
        for (int j = lane; j < k; j += 32) {
          const int e = ids[j];
          if (e >= 0 && e < E) ctop = fmaxf(ctop, load_logit(row + e));
        }
        ctop = warp_max(ctop);
        if (sig) ctop = fminf(ctop, 0.f);
        for (int j = lane; j < k; j += 32) {
          const int e = ids[j];
          if (e >= 0 && e < E) csum += weight(load_logit(row + e), ctop, sig);
        }
        csum = warp_sum(csum);
        for (int j = lane; j < k; j += 32) {
          const int e = ids[j];
          if (e >= 0 && e < E && csum != 0.f) {
            const float w = weight(load_logit(row + e), ctop, sig) / csum;
            if (w != 0.f) vs += ds[j] * a.scale * w;
          }
        }
        vs = warp_sum(vs);
      }
      for (int j = lane; j < k; j += 32) {
        const int e = ids[j];
        if (e < 0 || e >= E) continue;
        const float c = load_logit(row + e), v = ds[j] * a.scale;
        float x = 0.f;
        if (c != -INFINITY) {
          if (a.scoring == MOE_ROUTER_SOFTMAX)
            x = v;
          else if (csum != 0.f)
            x = weight(c, ctop, sig) / csum * (v - vs);
        }
        ex[e] = x;
      }
      __syncwarp();
    }
    float p[NV], gp = 0.f;
    const bool in_g = a.scoring == MOE_ROUTER_SOFTMAX;
    // p = weight(l, stat): exp(l - lse), or sigmoid(l) / S (for l > 0 divided by S here)
    const float inv = sig ? expf(-stat) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = lane + 32 * i < E ? weight(l[i], stat, sig) : 0.f;
      if (sig && l[i] > 0.f) p[i] *= inv;
      gp += p[i] * (b[i] + (in_g ? ex[lane + 32 * i] : 0.f));
    }
    gp = warp_sum(gp);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      const float x = ex[e];
      float g = p[i] * (b[i] + (in_g ? x : 0.f) - gp + dz * stat) + (in_g ? 0.f : x);
      if (sig) g *= l[i] > 0.f ? expf(-l[i]) / (1.f + expf(-l[i])) : 1.f / (1.f + expf(l[i]));
      if (e < E) store_logit(out + e, g);
    }
    if (a.d_scores) {                       // clear for the next row
      __syncwarp();
      for (int j = lane; j < k; j += 32) {
        const int e = a.ids[t * k + j];
        if (e >= 0 && e < E) ex[e] = 0.f;
      }
      __syncwarp();
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// host side

// Up to this many rows run on one CTA, which also writes the sums (no second
// launch).
constexpr int kOneCtaRows = 64;
constexpr int kFwdWarps = 16;

int forward_grid(int T) {
  if (T <= kOneCtaRows) return 1;
  const int want = (T + kFwdWarps - 1) / kFwdWarps, cap = num_sms();
  return want < cap ? want : cap;
}

template <typename L>
cudaError_t launch_forward(const RouterArgs& a, int grid, cudaStream_t st) {
  const int warps = grid > 1 ? kFwdWarps : a.T > 8 ? 32 : 8;
  const dim3 g(grid), b(warps * 32);
  switch ((a.E + 31) / 32) {
    case 1: return launch_pdl(k_router<L, 1>, g, b, 0, st, a);
    case 2: return launch_pdl(k_router<L, 2>, g, b, 0, st, a);
    case 3: return launch_pdl(k_router<L, 3>, g, b, 0, st, a);
    case 4: return launch_pdl(k_router<L, 4>, g, b, 0, st, a);
    default: return launch_pdl(k_router<L, 8>, g, b, 0, st, a);
  }
}

template <typename L>
cudaError_t launch_backward(const RouterArgs& a, cudaStream_t st) {
  const int want = (a.T + kGradWarps - 1) / kGradWarps, cap = num_sms() * 6;
  const dim3 g(want < cap ? want : cap), b(kGradWarps * 32);
  switch ((a.E + 31) / 32) {
    case 1: return launch_pdl(k_router_grad<L, 1>, g, b, 0, st, a);
    case 2: return launch_pdl(k_router_grad<L, 2>, g, b, 0, st, a);
    case 3: return launch_pdl(k_router_grad<L, 3>, g, b, 0, st, a);
    case 4: return launch_pdl(k_router_grad<L, 4>, g, b, 0, st, a);
    default: return launch_pdl(k_router_grad<L, 8>, g, b, 0, st, a);
  }
}

bool desc_ok(const moe_router_desc* s) {
  return s && s->E >= 1 && s->E <= kMaxE && s->k >= 1 && s->k <= s->E &&
         (s->dtype == MOE_DTYPE_BF16 || s->dtype == MOE_DTYPE_FP32) &&
         s->scoring >= MOE_ROUTER_SOFTMAX_TOPK && s->scoring <= MOE_ROUTER_SIGMOID &&
         std::isfinite(s->scale);
}

bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

bool sizes_ok(const moe_router_desc* s, int T) {
  return desc_ok(s) && T >= 0 && (long long)T * s->k < (1LL << 31);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_workspace_bytes(const moe_router_desc* s, int T) {
  if (!sizes_ok(s, T)) return 0;
  return (size_t)forward_grid(T) * (2 * s->E + 2) * 4;
}

extern "C" int moe_router_forward(const moe_router_desc* s, int T, const void* logits,
                                  long long ld, const float* bias, const uint8_t* token_mask,
                                  int32_t* ids, float* scores, int32_t* counts, float* prob_sum,
                                  float* losses, float* row_stat, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!sizes_ok(s, T) || !counts || !prob_sum || !losses) return MOE_ERR_INVALID_ARG;
  const int es = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (T > 0 && (!logits || ld < s->E || !ids || !scores || !row_stat || !aligned(logits, es)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(bias, 4) || !aligned(ids, 4) || !aligned(scores, 4) || !aligned(counts, 4) ||
      !aligned(prob_sum, 4) || !aligned(losses, 4) || !aligned(row_stat, 4))
    return MOE_ERR_INVALID_ARG;
  const int grid = forward_grid(T);
  RouterArgs a = {};
  a.T = T; a.E = s->E; a.k = s->k; a.scoring = s->scoring; a.scale = s->scale;
  a.logits = logits; a.ld = ld; a.bias = bias; a.mask = token_mask;
  a.ids = ids; a.scores = scores; a.counts = counts; a.prob_sum = prob_sum; a.losses = losses;
  a.row_stat = row_stat;
  if (grid > 1) {
    if (!workspace || workspace_bytes < moe_router_workspace_bytes(s, T)) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    a.part_prob = static_cast<float*>(workspace);
    a.part_count = reinterpret_cast<int32_t*>(a.part_prob + (size_t)grid * a.E);
    a.part_z = reinterpret_cast<float*>(a.part_count + (size_t)grid * (a.E + 1));
    a.n_part = grid;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = s->dtype == MOE_DTYPE_FP32 ? launch_forward<float>(a, grid, st)
                                             : launch_forward<uint16_t>(a, grid, st);
  if (e == cudaSuccess && a.part_prob)
    e = launch_pdl(k_router_finish, dim3(1), dim3(1024), 0, st, a);
  return cuda_result(e, "moe_router_forward");
}

extern "C" int moe_router_backward(const moe_router_desc* s, int T, const void* logits,
                                   long long ld, const int32_t* ids, const int32_t* counts,
                                   const float* row_stat, const float* d_scores,
                                   const float* d_losses, void* d_logits, long long ld_d,
                                   void* stream) {
  if (!sizes_ok(s, T)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int es = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!logits || ld < s->E || !d_logits || ld_d < s->E || !counts || !row_stat ||
      (d_scores && !ids) || !aligned(logits, es) || !aligned(d_logits, es) || !aligned(ids, 4) ||
      !aligned(counts, 4) || !aligned(row_stat, 4) || !aligned(d_scores, 4) ||
      !aligned(d_losses, 4))
    return MOE_ERR_INVALID_ARG;
  RouterArgs a = {};
  a.T = T; a.E = s->E; a.k = s->k; a.scoring = s->scoring; a.scale = s->scale;
  a.logits = logits; a.ld = ld;
  a.ids = const_cast<int32_t*>(ids);
  a.counts = const_cast<int32_t*>(counts);
  a.row_stat = const_cast<float*>(row_stat);
  a.d_scores = d_scores; a.d_losses = d_losses; a.d_logits = d_logits; a.ld_d = ld_d;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = s->dtype == MOE_DTYPE_FP32 ? launch_backward<float>(a, st)
                                                   : launch_backward<uint16_t>(a, st);
  return cuda_result(e, "moe_router_backward");
}
