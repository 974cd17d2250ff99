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
// coalesced and every sum over experts is one warp reduction.  All arithmetic is fp32;
// the only rounding to fewer bits is that of a bf16 gradient on its way out.

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

// fp32 to an unsigned integer of the same order, above 1; NaN is 1, below every
// number, and 0 stays free for "not there"; -0 = +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return v != v ? 1u : key;
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {      // NaN only if every lane's is
  return order_value(__reduce_max_sync(kAll, order_key(v)));
}

// A row's weights, before they are divided by their sum: exp(l - top) for the
// softmax, sigmoid(l) * exp(-top) for the sigmoid, with top from shift_of() of the
// largest logit, so that the sum neither overflows nor underflows.  The hardware
// exponential errs by a few 2^-23 near the largest logit, where the sum is.
__device__ __forceinline__ float shift_of(float largest, bool sig) {
  return !sig ? largest : largest < -40.f ? largest : 0.f;
}
__device__ __forceinline__ float weight(float l, float top, bool sig) {
  if (!sig) return __expf(l - top);                       // l = -inf: 0 (top is not)
  const float t = __expf(-fabsf(l));
  return __fdividef(l > 0.f ? 1.f : top == 0.f ? t : __expf(l - top), 1.f + t);
}

// Sums over the CTA's warps in a fixed order; all threads call it, warp 0 has the sum.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? buf[threadIdx.x & 31] : 0.f);
}

__device__ __forceinline__ void write_losses(const RouterArgs& a, float balance, float z,
                                             int live) {
  const float n = live > 0 ? (float)live : 1.f;
  a.counts[a.E] = live;
  a.losses[0] = balance / n * ((float)a.E / (float)a.k) / n;
  a.losses[1] = z / n;
}

// Forward.  L = logits type, NV = slots of 32 experts.
//
// One pass over the logits: 4 E bytes a row in, 8 k out, next to nothing for the
// memory (8192 rows of 128 fp32 logits, 4.75 MB: 0.7 us).  What bounds it is the chain of
// the selection, k steps of a warp-wide maximum and a ballot each, and the instructions
// of 32 warps an SM.  A row in one warp keeps that chain free of barriers; integer keys
// of the same order as the logits need one reduction instruction a step, and a ballot
// finds the lowest expert that has the maximum.  The per-expert sums stay in the warps'
// registers over all their rows, so that no atomic adds floating-point values and the
// results do not depend on the order in which warps run.
// Measured, both launches: one token 3.5 us, 8192 rows of 128 experts (k = 8) 11.4, 16411
// rows of 250 bf16 logits (k = 6, sigmoid, bias, 2048 rows masked) 19.6.
template <typename L, int NV>
__global__ void __launch_bounds__(1024) k_router(const RouterArgs a) {
  extern __shared__ float psum[];                 // [warps][NV * 32]
  __shared__ int cnt[kMaxE];
  __shared__ uint8_t sel_id[32][kMaxE];           // a warp's chosen experts, in order
  __shared__ float wz[32];
  __shared__ int wlive[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int E = a.E, k = a.k;
  float* const mine = psum + warp * (NV * 32);    // first the row's logits, by expert
  for (int e = threadIdx.x; e < kMaxE; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  pdl_wait();
  const bool sig = a.scoring == MOE_ROUTER_SIGMOID;
  float ps[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) ps[i] = 0.f;
  float bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bias[i] = a.bias && lane + 32 * i < E ? a.bias[lane + 32 * i] : 0.f;
  float z = 0.f;
  int live_rows = 0;
  for (long long t = (long long)blockIdx.x * nw + warp; t < a.T; t += (long long)gridDim.x * nw) {
    const L* row = static_cast<const L*>(a.logits) + t * a.ld;
    int32_t* ids = a.ids + t * k;
    float* scores = a.scores + t * k;
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
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? load_logit(row + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < E ? order_key(l[i] + bias[i]) : 0u;
      mine[e] = l[i];
      mx = fmaxf(mx, l[i]);
      nan |= l[i] != l[i];
    }
    // the largest key k times; slots are searched in order and lanes within a slot,
    // so equal keys go to the lowest expert.  A chosen key becomes 0.
    for (int j = 0; j < k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) best = max(best, key[i]);
      const uint32_t top = __reduce_max_sync(kAll, best);
      bool open = true;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (open) {
          const unsigned has = __ballot_sync(kAll, key[i] == top);
          if (has) {
            const int at = __ffs(has) - 1;
            if (lane == at) {
              key[i] = 0u;
              sel_id[warp][j] = (uint8_t)(32 * i + at);
            }
            open = false;
          }
        }
    }
    mx = warp_max(mx);
    nan = __any_sync(kAll, nan);
    __syncwarp();                          // sel_id and the row's logits are written
    if (!nan && mx == -INFINITY) {         // nothing to choose
      for (int j = lane; j < k; j += 32) {
        ids[j] = sel_id[warp][j];
        scores[j] = 0.f;
      }
      if (lane == 0) a.row_stat[t] = -INFINITY;
      __syncwarp();
      continue;
    }
    if (mx == -INFINITY) mx = 0.f;         // NaN and -inf only: any shift gives NaN
    live_rows += 1;
    const float top = shift_of(mx, sig);
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      l[i] = lane + 32 * i < E ? weight(l[i], top, sig) : 0.f;
      total += l[i];
    }
    total = warp_sum(total);
    const float inv = 1.f / total;
#pragma unroll
    for (int i = 0; i < NV; ++i) ps[i] += l[i] * inv;
    const float stat = top + logf(total);
    if (lane == 0) a.row_stat[t] = stat;
    if (!sig) z += stat * stat;
    // the chosen: scores and counts.  Without a bias the row's largest logit is among
    // them, and its shift serves.
    float ctop = top, cinv = inv;
    if (a.scoring != MOE_ROUTER_SOFTMAX) {
      if (a.bias) {
        float m = -INFINITY;
        for (int j = lane; j < k; j += 32) m = fmaxf(m, mine[sel_id[warp][j]]);
        ctop = warp_max(m);
        if (ctop != -INFINITY) ctop = shift_of(ctop, sig);
        else if (nan) ctop = top;
      }
      float sum = 0.f;
      if (ctop != -INFINITY)
        for (int j = lane; j < k; j += 32) sum += weight(mine[sel_id[warp][j]], ctop, sig);
      sum = warp_sum(sum);
      cinv = sum == 0.f ? 0.f : 1.f / sum;
    }
    for (int j = lane; j < k; j += 32) {
      const int e = sel_id[warp][j];
      const float c = mine[e];
      ids[j] = e;
      scores[j] = ctop == -INFINITY ? 0.f : weight(c, ctop, sig) * cinv * a.scale;
      if (c != -INFINITY) atomicAdd(&cnt[e], 1);
    }
    __syncwarp();                          // before the next row overwrites them
  }
  pdl_trigger();
  // the warps' sums, added in order
#pragma unroll
  for (int i = 0; i < NV; ++i) mine[lane + 32 * i] = ps[i];
  if (lane == 0) {
    wz[warp] = z;
    wlive[warp] = live_rows;
  }
  __syncthreads();
  float v = 0.f;
  const long long b = blockIdx.x;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float P = 0.f;
    for (int w = 0; w < nw; ++w) P += psum[w * (NV * 32) + e];
    if (a.part_prob) {
      a.part_prob[b * E + e] = P;
      a.part_count[b * (E + 1) + e] = cnt[e];
    } else {
      a.prob_sum[e] = P;
      a.counts[e] = cnt[e];
      v += (float)cnt[e] * P;
    }
  }
  z = warp_sum(lane < nw ? wz[lane] : 0.f);
  const int live = __reduce_add_sync(kAll, lane < nw ? wlive[lane] : 0);
  if (a.part_prob) {
    if (threadIdx.x == 0) {
      a.part_count[b * (E + 1) + E] = live;
      a.part_z[b] = z;
    }
  } else {
    __syncthreads();                       // wz has been read
    v = block_sum(v, wz);
    if (threadIdx.x == 0) write_losses(a, v, z, live);
  }
}

// Adds the CTAs' sums: a cluster of one CTA per 32 experts, warp w of it expert w,
// the balance loss joined through the cluster's shared memory.  Latency: a few dependent
// loads and two cluster barriers, some 4 us beside a launch of its own.
__global__ void __launch_bounds__(1024) k_router_finish(const RouterArgs a) {
  __shared__ float sp[32][33];
  __shared__ int sc[32][33];
  __shared__ float per_warp[32], part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  cluster_sync();                          // every CTA's shared memory is there
  pdl_wait();
  float P = 0.f;
  int c = 0;
  if (e < a.E)
#pragma unroll 4
    for (int b = warp; b < a.n_part; b += 32) {
      P += a.part_prob[(long long)b * a.E + e];
      c += a.part_count[(long long)b * (a.E + 1) + e];
    }
  float z = 0.f;
  int live = 0;
  if (blockIdx.x == 0 && warp == 0)
    for (int b = lane; b < a.n_part; b += 32) {
      z += a.part_z[b];
      live += a.part_count[(long long)b * (a.E + 1) + a.E];
    }
  sp[warp][lane] = P;
  sc[warp][lane] = c;
  __syncthreads();
  P = warp_sum(sp[lane][warp]);            // expert blockIdx.x * 32 + warp
  c = __reduce_add_sync(kAll, sc[lane][warp]);
  if (lane == 0) {
    const int mine = blockIdx.x * 32 + warp;
    if (mine < a.E) {
      a.prob_sum[mine] = P;
      a.counts[mine] = c;
    }
    per_warp[warp] = (float)c * P;
  }
  __syncthreads();
  if (warp == 0) {
    const float v = warp_sum(per_warp[lane]);
    if (lane == 0)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                       mapa_shared(smem_u32(&part[blockIdx.x]), 0)), "f"(v) : "memory");
    __syncwarp();
  }
  cluster_sync();
  if (blockIdx.x == 0 && warp == 0) {
    z = warp_sum(z);
    live = __reduce_add_sync(kAll, live);
    if (lane == 0) {
      float balance = 0.f;
      for (int i = 0; i < (int)gridDim.x; ++i) balance += part[i];
      write_losses(a, balance, z, live);
    }
  }
  pdl_trigger();
}

// Gradient: a warp per row, as the forward.  A warp's shared memory holds the row's
// logits and the chosen experts' own terms.
//
// Reads the logits again and takes the probabilities from row_stat, so that the forward
// leaves 4 bytes a row instead of 4 E.  Bound by latency and instructions (two or
// three exponentials' work a logit): 8192 rows of 128 fp32 logits 5.7 us where the 8.9 MB
// take 1.3; 16411 rows of 250 bf16 logits, 2048 of them masked, 16.3 where they take 2.4.
constexpr int kGradWarps = 8;

template <typename L, int NV>
__global__ void __launch_bounds__(kGradWarps * 32) k_router_grad(const RouterArgs a) {
  __shared__ float logits[kGradWarps][NV * 32], extra[kGradWarps][NV * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E, k = a.k;
  const bool sig = a.scoring == MOE_ROUTER_SIGMOID, in_g = a.scoring == MOE_ROUTER_SOFTMAX;
  float* const lg = logits[warp];
  float* const ex = extra[warp];
#pragma unroll
  for (int i = 0; i < NV; ++i) ex[lane + 32 * i] = 0.f;
  pdl_wait();
  const int live_n = a.counts[E];
  const float inv_n = 1.f / (live_n > 0 ? (float)live_n : 1.f);
  float b[NV], dz = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) b[i] = 0.f;
  if (a.d_losses) {
    const float f = a.d_losses[0] * ((float)E / (float)k) * inv_n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e < E) b[i] = f * ((float)a.counts[e] * inv_n);
    }
    if (!sig) dz = a.d_losses[1] * 2.f * inv_n;
  }
  for (long long t = (long long)blockIdx.x * kGradWarps + warp; t < a.T;
       t += (long long)gridDim.x * kGradWarps) {
    const L* row = static_cast<const L*>(a.logits) + t * a.ld;
    L* out = static_cast<L*>(a.d_logits) + t * a.ld_d;
    const float stat = a.row_stat[t];
    if (stat == -INFINITY) {                // not live: no gradient
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
#pragma unroll
      for (int i = 0; i < NV; ++i) lg[lane + 32 * i] = l[i];
      __syncwarp();
      // normalised chosen scores s' = weight / csum, and sum v s'
      float ctop = -INFINITY, cinv = 0.f, vs = 0.f;
      if (!in_g) {
        for (int j = lane; j < k; j += 32) {
          const int e = ids[j];
          if (e >= 0 && e < E) ctop = fmaxf(ctop, lg[e]);
        }
        ctop = warp_max(ctop);
        if (ctop != -INFINITY) ctop = shift_of(ctop, sig);
        float sum = 0.f;
        if (ctop != -INFINITY)
          for (int j = lane; j < k; j += 32) {
            const int e = ids[j];
            if (e >= 0 && e < E && lg[e] != -INFINITY) {
              const float w = weight(lg[e], ctop, sig);
              sum += w;
              vs += ds[j] * a.scale * w;
            }
          }
        sum = warp_sum(sum);
        cinv = sum == 0.f ? 0.f : 1.f / sum;
        vs = warp_sum(vs) * cinv;
      }
      for (int j = lane; j < k; j += 32) {
        const int e = ids[j];
        if (e < 0 || e >= E) continue;
        const float c = lg[e], v = ds[j] * a.scale;
        float x = 0.f;
        if (c != -INFINITY)
          x = in_g ? v : ctop == -INFINITY ? 0.f : weight(c, ctop, sig) * cinv * (v - vs);
        ex[e] = x;
      }
      __syncwarp();
    }
    // p = exp(l - lse), or sigmoid(l) / S with log S = stat
    float inv = sig ? __expf(-fmaxf(stat, -40.f)) : 1.f;
    const float far = sig && stat < -40.f ? stat + 40.f : 0.f;     // S alone would underflow
    auto probability = [&](float v, float& after) {                // after: 1 - sigmoid
      if (!sig) return __expf(v - stat) * inv;
      const float u = __expf(-fabsf(v)), s = __fdividef(1.f, 1.f + u);
      after = v > 0.f ? u * s : s;
      return (v > 0.f ? s : (far == 0.f ? u : __expf(v - far)) * s) * inv;
    };
    // The rounding of stat, 2^-24 |stat|, is a factor of all of them: divided out, except
    // where it is less than what the exponential errs by (dividing always, with the sum
    // taken beside gp's, 7.1 us against 5.7 at 8192 rows of 128 experts).
    if (fabsf(stat) > 8.f) {
      float sum = 0.f, unused;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += lane + 32 * i < E ? probability(l[i], unused) : 0.f;
      inv *= __fdividef(1.f, warp_sum(sum));
    }
    float gp = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float after = 1.f, p = probability(l[i], after);
      if (lane + 32 * i >= E) p = 0.f;
      const float x = ex[lane + 32 * i];
      const float g = b[i] + (in_g ? x : 0.f);
      gp += p * g;
      // dl = after * (p * (g + dz stat - gp) + own term), without gp for now
      lg[lane + 32 * i] = after * p;
      l[i] = after * (p * (g + dz * stat) + (in_g ? 0.f : x));
    }
    gp = warp_sum(gp);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e < E) store_logit(out + e, l[i] - lg[e] * gp);
      if (a.d_scores) ex[e] = 0.f;          // clear for the next row
    }
    __syncwarp();
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// host side

// Up to a row per warp one CTA does all, the sums too (32 rows of 128 experts 4.8 us).
// More rows are spread, and a second launch adds the sums: 64 rows 6.6 us against 7.8
// on one CTA.
constexpr int kOneCtaRows = 32;

// warps of a CTA: its chosen experts and per-warp sums take shared memory
int forward_warps(int T, int grid) { return grid > 1 ? 32 : T > 8 ? 32 : 8; }

int forward_grid(int T) {
  if (T <= kOneCtaRows) return 1;
  const int want = (T - 1) / 32 + 1, cap = num_sms();      // T + 31 may pass INT_MAX
  return want < cap ? want : cap;
}

template <typename L, int NV>
cudaError_t launch_forward_nv(const RouterArgs& a, int grid, cudaStream_t st) {
  const int warps = forward_warps(a.T, grid), smem = warps * NV * 32 * (int)sizeof(float);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_router<L, NV>, 32 * NV * 32 * (int)sizeof(float), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_router<L, NV>, dim3(grid), dim3(warps * 32), smem, st, a);
}

template <typename L>
cudaError_t launch_forward(const RouterArgs& a, int grid, cudaStream_t st) {
  switch ((a.E + 31) / 32) {
    case 1: return launch_forward_nv<L, 1>(a, grid, st);
    case 2: return launch_forward_nv<L, 2>(a, grid, st);
    case 3: return launch_forward_nv<L, 3>(a, grid, st);
    case 4: return launch_forward_nv<L, 4>(a, grid, st);
    default: return launch_forward_nv<L, 8>(a, grid, st);
  }
}

cudaError_t launch_finish(const RouterArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.E + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cfg.gridDim.x;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_router_finish, a);
}

template <typename L>
cudaError_t launch_backward(const RouterArgs& a, cudaStream_t st) {
  const int want = (a.T - 1) / kGradWarps + 1, cap = num_sms() * 6;
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
  if (e == cudaSuccess && a.part_prob) e = launch_finish(a, st);
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
