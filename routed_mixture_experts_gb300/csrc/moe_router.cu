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
  // choice within groups of neighbouring experts
  int groups, top_groups, group_size, pair;
  int share_log2;        // lanes a group in the search for its largest keys
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

// ---- the choice within groups ---------------------------------------------------
//
// key = s + bias, s = sigmoid(l) or softmax(l); a group's value is the sum of its two
// largest keys (or the largest); the experts of the top_groups best groups compete.  The
// order is that of the exact keys: keys are computed in fp32 with an error below
// key_error(), and where two that the choice separates, or orders, lie closer, the row is
// chosen again on 64-bit keys (choose_slowly).  Without a bias the logits themselves order
// the experts, and the groups too where a group's value is its largest key.

struct GroupRow {
  float* key;                        // [NV * 32] keys by expert, NaN as -inf
  float *value, *second;             // [groups] values, second keys
  uint32_t* kept;                    // [8] bit g: group g competes
};

// How close two fp32 keys, or sums of two, may come without their order being known.  The
// error of s: sigmoid, the exponential's (2 + 1.5 |l|) 2^-23 of e^-l is s (1 - s) times that
// of s, below 2^-23, the sum's rounding and the quotient's 2^-24 + 2^-23; softmax, the same
// relative to s, plus the rounding of l - max (D 2^-24 of a weight e^-D) and the total's,
// together below 2^-20 of the largest s.  Adding biases up to `wide` and two keys: 2^-24 of
// at most twice (1 + wide) each.  Four keys are compared.
__device__ __forceinline__ float key_error(bool sig, float largest, float wide) {
  return (sig ? 0x1p-19f : 0x1p-18f * largest) + 0x1p-20f * wide;
}

__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  const uint64_t key = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
  return v != v ? 1ull : key;
}
__device__ __forceinline__ double order_value64(uint64_t key) {
  return __longlong_as_double(
      (long long)((key >> 63) ? key & 0x7FFFFFFFFFFFFFFFull : ~key));
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// The choice of one row on 64-bit keys, by one warp (logits by expert in shared memory).
template <int NV>
__device__ __forceinline__ void choose_slowly(const RouterArgs& a, const float* logits,
                                              uint32_t* kept, uint8_t* chosen) {
  const int lane = threadIdx.x & 31, E = a.E;
  const bool sig = a.scoring == MOE_ROUTER_SIGMOID;
  float mx = -INFINITY;
  for (int e = lane; e < E; e += 32) mx = fmaxf(mx, logits[e]);
  mx = warp_max(mx);
  double w[NV], total = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    w[i] = 0.0;
    if (e < E) w[i] = sig ? 1.0 / (1.0 + exp(-(double)logits[e])) : exp((double)logits[e] - mx);
    total += w[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  uint64_t key[NV];
  int group[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    group[i] = e < E ? e / a.group_size : -1;
    if (e < E) {
      const double s = sig ? w[i] : w[i] / total;
      const double v = logits[e] == -INFINITY ? -INFINITY : a.bias ? s + (double)a.bias[e] : s;
      key[i] = order_key64(v);
    }
  }
  const uint64_t none = order_key64(-INFINITY);
  if (a.top_groups < a.groups) {
    uint64_t value[8];                       // of group lane + 32 i
#pragma unroll
    for (int i = 0; i < 8; ++i) value[i] = 0;
    for (int g = 0; g < a.groups; ++g) {
      uint64_t best = 0;
      int at = -1;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (group[i] == g && key[i] > best) {
          best = key[i];
          at = i;
        }
      const uint64_t first = warp_max64(best);
      uint64_t v = first < none ? none : first;       // NaN counts as -inf
      if (a.pair) {
        const unsigned has = __ballot_sync(kAll, at >= 0 && best == first);
        const bool mine = has && lane == __ffs(has) - 1;
        best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (group[i] == g && !(mine && i == at)) best = max(best, key[i]);
        const uint64_t second = warp_max64(best);
        if (second > none && v > none)
          v = order_key64(order_value64(v) + order_value64(second));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (g == lane + 32 * i) value[i] = v;
    }
    __syncwarp();
    if (lane < 8) kept[lane] = 0;
    __syncwarp();
    for (int j = 0; j < a.top_groups; ++j) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) best = max(best, value[i]);
      const uint64_t top = warp_max64(best);
      bool open = true;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (open) {
          const unsigned has = __ballot_sync(kAll, value[i] == top);
          if (has) {
            if (lane == __ffs(has) - 1) {
              value[i] = 0;
              kept[i] |= 1u << lane;
            }
            open = false;
          }
        }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (group[i] >= 0 && !((kept[group[i] >> 5] >> (group[i] & 31)) & 1u)) key[i] = 0;
  }
  if (!a.bias)           // the logits have the order, and ties, that their scores round away
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i]) key[i] = order_key(logits[lane + 32 * i]);
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) best = max(best, key[i]);
    const uint64_t top = warp_max64(best);
    bool open = true;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (open) {
        const unsigned has = __ballot_sync(kAll, key[i] == top);
        if (has) {
          if (lane == __ffs(has) - 1) {
            key[i] = 0;
            chosen[j] = (uint8_t)(32 * i + lane);
          }
          open = false;
        }
      }
  }
  __syncwarp();
}

// The choice of one row of sigmoid keys whose groups are known, on the 64-bit keys of the
// experts that come within `error` of the last one chosen, a lane each: an exponential in 64
// bits costs a warp some 1000 cycles, and choose_slowly eight of them.  False where there
// are more of them than lanes.
template <int NV>
__device__ __forceinline__ bool choose_among(const RouterArgs& a, const float* logits,
                                             const float* keys, const uint32_t* kept,
                                             uint8_t* chosen, float error) {
  const int lane = threadIdx.x & 31;
  if (a.k >= 32) return false;
  const float low = keys[chosen[a.k - 1]] - 2.f * error;
  if (!(low > -INFINITY)) return false;
  __syncwarp();
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i, g = e / a.group_size;
    const bool in = e < a.E && keys[e] >= low &&
                    (a.top_groups == a.groups || ((kept[g >> 5] >> (g & 31)) & 1u));
    const unsigned has = __ballot_sync(kAll, in);
    const int at = n + __popc(has & ((1u << lane) - 1u));
    if (in && at < 32) chosen[64 + at] = (uint8_t)e;
    n += __popc(has);
  }
  if (n > 32) return false;
  __syncwarp();
  const int e = lane < n ? chosen[64 + lane] : 0;
  const double key = lane < n ? 1.0 / (1.0 + exp(-(double)logits[e])) + (double)a.bias[e] : 0.0;
  int ahead = 0;                               // the list is in the experts' order
  for (int j = 0; j < n; ++j) {
    const double other = __shfl_sync(kAll, key, j);
    ahead += (other > key || (other == key && j < lane)) ? 1 : 0;
  }
  if (lane < n && ahead < a.k) chosen[ahead] = (uint8_t)e;
  __syncwarp();
  return true;
}

// The values of the groups that fp32 does not tell apart, on the 64-bit keys of the experts
// that make them: those within `error` of a group's second (or largest) key, a lane each.
// Chooses among them so that top_groups compete.  False where there are more than lanes.
// (Sigmoid keys: a softmax key needs the whole row in 64 bits.)
__device__ __forceinline__ bool choose_close_groups(const RouterArgs& a, const GroupRow& row,
                                                    const float* logits, float in, float out,
                                                    float error) {
  const int lane = threadIdx.x & 31, G = a.groups;
  int n = 0, expert = 0, mine = -1;              // list of experts; this lane's and its group
  int open = a.top_groups, close = 0, held = -1; // places left; close groups; this lane's
  for (int g = 0; g < G; ++g) {
    const float v = row.value[g];
    if (v > out + error) open -= 1;
    if (v > out + error || v < in - error) continue;
    if (lane == close) held = g;
    close += 1;
    const float least = (a.pair ? row.second[g] : v) - error;
    for (int i0 = 0; i0 < a.group_size; i0 += 32) {
      const int i = i0 + lane;
      const bool takes = i < a.group_size && row.key[g * a.group_size + i] >= least;
      unsigned has = __ballot_sync(kAll, takes);
      const int m = __popc(has);
      if (n + m > 32) return false;
      if (lane >= n && lane < n + m) {           // the (lane - n)-th of them
        for (int k = lane - n; k > 0; --k) has &= has - 1;
        expert = g * a.group_size + i0 + __ffs(has) - 1;
        mine = g;
      }
      n += m;
    }
  }
  if (close > 32) return false;
  double key = -INFINITY;
  if (mine >= 0 && row.key[expert] > -INFINITY)
    key = 1.0 / (1.0 + exp(-(double)logits[expert])) + (a.bias ? (double)a.bias[expert] : 0.0);
  double value = -INFINITY;                      // of the group that this lane holds
  for (int j = 0; j < n; ++j) {                  // its largest
    const double v = __shfl_sync(kAll, key, j);
    if (__shfl_sync(kAll, mine, j) == held && v > value) value = v;
  }
  if (a.pair) {
    double second = -INFINITY;
    bool met = false;                            // the largest itself, once
    for (int j = 0; j < n; ++j) {
      const double v = __shfl_sync(kAll, key, j);
      if (__shfl_sync(kAll, mine, j) != held) continue;
      if (v == value && !met) met = true;
      else if (v > second) second = v;
    }
    if (second > -INFINITY) value += second;
  }
  int ahead = 0;
  for (int j = 0; j < close; ++j) {
    const double v = __shfl_sync(kAll, value, j);
    ahead += (v > value || (v == value && j < lane)) ? 1 : 0;
  }
  // the bits anew
  for (int g0 = 0; g0 < G; g0 += 32) {
    const int g = g0 + lane;
    const unsigned word = __ballot_sync(kAll, g < G && row.value[g < G ? g : 0] > out + error);
    if (lane == 0) row.kept[g0 >> 5] = word;
  }
  __syncwarp();
  if (held >= 0 && ahead < open) atomicOr(&row.kept[held >> 5], 1u << (held & 31));
  __syncwarp();
  return true;
}

// Which groups compete (row.kept), from the keys in shared memory.  Several lanes share a
// group, from places that differ by group so that they do not meet in a bank.  Returns
// whether the last group in and the first one out are too close to tell.
__device__ __forceinline__ bool choose_groups(const RouterArgs& a, const GroupRow& row,
                                              const float* logits, bool exact, bool sig,
                                              float error) {
  const int lane = threadIdx.x & 31, G = a.groups, size = a.group_size;
  const int share = 1 << a.share_log2, per = (size + share - 1) >> a.share_log2;
  const int q = lane & (share - 1);
  const bool even = size == per << a.share_log2 && (per & (per - 1)) == 0;
  for (int g = lane >> a.share_log2; g - (lane >> a.share_log2) < G; g += 32 >> a.share_log2) {
    float first = -INFINITY, second = -INFINITY;
    if (g < G) {
      const float* const p = row.key + g * size + q;
      if (even && a.pair) {
#pragma unroll 8
        for (int n = 0; n < per; ++n) {
          const float v = p[(n ^ (g & (per - 1))) << a.share_log2];
          second = fmaxf(second, fminf(first, v));
          first = fmaxf(first, v);
        }
      } else if (even) {
#pragma unroll 8
        for (int n = 0; n < per; ++n)
          first = fmaxf(first, p[(n ^ (g & (per - 1))) << a.share_log2]);
      } else {
        int j = g % per;
        for (int n = 0; n < per; ++n) {
          const float v = q + (j << a.share_log2) < size ? p[j << a.share_log2] : -INFINITY;
          second = fmaxf(second, fminf(first, v));
          first = fmaxf(first, v);
          if (++j == per) j = 0;
        }
      }
    }
    for (int o = share >> 1; o > 0; o >>= 1) {
      const float f = __shfl_xor_sync(kAll, first, o), s = __shfl_xor_sync(kAll, second, o);
      second = fmaxf(fminf(first, f), fmaxf(second, s));
      first = fmaxf(first, f);
    }
    if (g < G && q == 0) {
      row.value[g] = a.pair && second > -INFINITY ? first + second : first;
      row.second[g] = second;
    }
  }
  __syncwarp();
  uint32_t low = 0xFFFFFFFFu, high = 0u;     // of those that stay, of those that do not
  for (int g0 = 0; g0 < G; g0 += 32) {
    const int g = g0 + lane;
    bool stays = false;
    if (g < G) {
      const float v = row.value[g];
      int ahead = 0;
#pragma unroll 8
      for (int h = 0; h < G; ++h) {
        const float w = row.value[h];
        ahead += (w > v || (w == v && h < g)) ? 1 : 0;
      }
      stays = ahead < a.top_groups;
      const uint32_t k = order_key(v);
      if (stays) low = min(low, k); else high = max(high, k);
    }
    const unsigned word = __ballot_sync(kAll, stays);
    if (lane == 0) row.kept[g0 >> 5] = word;
  }
  __syncwarp();
  if (exact) return false;
  if (!(error < INFINITY)) return true;
  low = __reduce_min_sync(kAll, low);
  high = __reduce_max_sync(kAll, high);
  const float in = order_value(low), out = order_value(high);
  if (!(in - out <= error)) return false;               // (infinities: NaN, not close)
  return !sig || !choose_close_groups(a, row, logits, in, out, error);
}

// Forward.  L = logits type, NV = slots of 32 experts, GROUPS: the choice within groups.
//
// One pass over the logits: 4 E bytes a row in, 8 k out, next to nothing for the
// memory (8192 rows of 128 fp32 logits, 4.75 MB: 0.7 us).  What bounds it is the chain of
// the selection, k steps of a warp-wide maximum and a ballot each, and the instructions
// of 32 warps an SM.  A row in one warp keeps that chain free of barriers; integer keys
// of the same order as the logits need one reduction instruction a step, and a ballot
// finds the lowest expert that has the maximum.  The per-expert sums stay in the warps'
// registers over all their rows, so that no atomic adds floating-point values and the
// results do not depend on the order in which warps run.
// With groups the chain has the groups' values before it (their largest keys found by up to
// 32 lanes, their places by counting those ahead), and the choice takes the lanes' largest
// keys from lists that each lane has sorted: 8192 rows of 256 experts in 8 groups 24.3 us,
// 16411 rows of 160 experts in 20 (bf16, 2048 rows masked) 23.0, one row 5.3.  The sorted
// lists took 31.1 us, with a search over all slots a step, to 28.5.  The rare choices on
// 64-bit keys are inlined: called, they kept the loop's registers in memory (26.3 us against
// 25.2).  At 28.5 us 56 % of the issue slots and of the integer units' rate were in use.
// Measured, both launches: one token 3.5 us, 8192 rows of 128 experts (k = 8) 11.4, 16411
// rows of 250 bf16 logits (k = 6, sigmoid, bias, 2048 rows masked) 19.6.
template <typename L, int NV, bool GROUPS>
__global__ void __launch_bounds__(GROUPS ? 640 : 1024) k_router(const RouterArgs a) {
  extern __shared__ float psum[];                 // [warps][NV * 32], GROUPS: and the keys
  __shared__ int cnt[kMaxE];
  __shared__ uint8_t sel_id[32][kMaxE];           // a warp's chosen experts, in order
  __shared__ float wz[32];
  __shared__ int wlive[32];
  __shared__ uint32_t kept[GROUPS ? 32 : 1][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int E = a.E, k = a.k;
  // whether slot i of this lane is an expert (with groups NV is the fewest slots)
  auto there = [&](int i) { return (GROUPS && i + 1 < NV) || lane + 32 * i < E; };
  float* const mine = psum + warp * (NV * 32);    // first the row's logits, by expert
  float* const keys = GROUPS ? psum + (nw + warp) * (NV * 32) : nullptr;
  float* const values = GROUPS ? psum + 2 * nw * (NV * 32) + warp * 2 * a.groups : nullptr;
  for (int e = threadIdx.x; e < kMaxE; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  pdl_wait();
  const bool sig = a.scoring == MOE_ROUTER_SIGMOID;
  float ps[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) ps[i] = 0.f;
  float bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bias[i] = a.bias && there(i) ? a.bias[lane + 32 * i] : 0.f;
  float wide = 0.f;                               // the largest bias
  uint64_t group_of = 0;                          // group of the expert in slot i, byte i
  if (GROUPS) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      group_of |= (uint64_t)((lane + 32 * i) / a.group_size) << (8 * i);
#pragma unroll
    for (int i = 0; i < NV; ++i) wide = fmaxf(wide, fabsf(bias[i]));
    wide = warp_max(wide);
    // sums of two such keys are beyond fp32: no comparison of them tells
    if (wide >= 0x1p126f) wide = INFINITY;
  }
  float z = 0.f;
  int live_rows = 0;
  // with groups a row's work is large enough for the last ones to be spread over the SMs
  const long long first = GROUPS ? (long long)warp * gridDim.x + blockIdx.x
                                 : (long long)blockIdx.x * nw + warp;
  for (long long t = first; t < a.T; t += (long long)gridDim.x * nw) {
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
    const bool weighed = GROUPS && (a.bias != nullptr || a.pair);
    float l[NV];
    uint32_t key[NV];
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      l[i] = there(i) ? load_logit(row + lane + 32 * i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!weighed) key[i] = there(i) ? order_key(l[i] + bias[i]) : 0u;
      mine[lane + 32 * i] = l[i];
      mx = fmaxf(mx, l[i]);
      nan |= l[i] != l[i];
    }
    int count = k;
    bool close = false, groups_close = false;
    float error = 0.f;
    if (GROUPS) {
      mx = warp_max(mx);
      float largest = 0.f;
      const bool keyed = a.bias != nullptr;
      if (weighed) {
        // fp32 keys of scores; the weights take the logits' place.  Without a bias the
        // logits order the experts.
        if (!keyed) {
#pragma unroll
          for (int i = 0; i < NV; ++i) key[i] = there(i) ? order_key(l[i]) : 0u;
        }
        uint32_t off = 0;                        // bit i: a logit of -inf
        if (sig) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            off |= (l[i] == -INFINITY ? 1u : 0u) << i;
            l[i] = there(i) ? __fdividef(1.f, 1.f + __expf(-l[i])) : 0.f;
          }
        } else {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            off |= (l[i] == -INFINITY ? 1u : 0u) << i;
            l[i] = there(i) ? __expf(l[i] - mx) : 0.f;
            sum += l[i];
          }
          largest = 1.f / warp_sum(sum);
        }
        const float share = sig ? 1.f : largest;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float v = (off >> i) & 1u ? -INFINITY : fmaf(l[i], share, bias[i]);
          if (keyed) key[i] = there(i) ? order_key(v) : 0u;
          keys[lane + 32 * i] = v == v ? v : -INFINITY;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) keys[lane + 32 * i] = l[i] == l[i] ? l[i] : -INFINITY;
      }
      __syncwarp();
      error = key_error(sig, largest, wide);
      if (a.top_groups < a.groups) {
        const GroupRow row = {keys, values, values + a.groups, kept[warp]};
        close = groups_close = choose_groups(a, row, mine, !keyed && !a.pair, sig, error);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int g = (int)(group_of >> (8 * i)) & 255;
          if (!((kept[warp][g >> 5] >> (g & 31)) & 1u)) key[i] = 0u;
        }
      }
      // the next one too, to see how close it comes
      if (keyed && k < a.top_groups * a.group_size) count = k + 1;
    }
    if (GROUPS) {
      // Each lane sorts its keys (Batcher's network; equal ones by slot), and of the lanes'
      // first ones the largest is taken, of equal ones the lowest expert.
      uint32_t slot[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) slot[i] = i;
      auto order = [&](int i, int j) {
        if (j < NV) {
          const bool swap = key[j] > key[i] || (key[j] == key[i] && slot[j] < slot[i]);
          const uint32_t ki = key[i], si = slot[i];
          key[i] = swap ? key[j] : ki;
          slot[i] = swap ? slot[j] : si;
          key[j] = swap ? ki : key[j];
          slot[j] = swap ? si : slot[j];
        }
      };
      order(0, 1); order(2, 3); order(4, 5); order(6, 7);
      order(0, 2); order(1, 3); order(4, 6); order(5, 7);
      order(1, 2); order(5, 6);
      order(0, 4); order(1, 5); order(2, 6); order(3, 7);
      order(2, 4); order(3, 5);
      order(1, 2); order(3, 4); order(5, 6);
      uint32_t slots = 0;                        // four bits each
#pragma unroll
      for (int i = 0; i < NV; ++i) slots |= slot[i] << (4 * i);
      for (int j = 0; j < count; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, key[0]);
        const uint32_t e = __reduce_min_sync(
            kAll, key[0] == top ? (slots & 15u) * 32u + (uint32_t)lane : 0xFFFFu);
        if (lane == 0) sel_id[warp][j] = (uint8_t)e;
        const bool took = (e & 31u) == (uint32_t)lane;
#pragma unroll
        for (int i = 0; i + 1 < NV; ++i) key[i] = took ? key[i + 1] : key[i];
        key[NV - 1] = took ? 0u : key[NV - 1];
        slots = took ? slots >> 4 : slots;
      }
    } else {
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
    }
    if (GROUPS && !close && a.bias) {
      __syncwarp();
      for (int j = lane; j + 1 < count; j += 32) {
        const int e = sel_id[warp][j], f = sel_id[warp][j + 1];
        // equal logits and biases are a tie in any arithmetic
        if (keys[e] - keys[f] <= error &&
            !(mine[e] == mine[f] && a.bias[e] == a.bias[f]))
          close = true;
      }
      close = __any_sync(kAll, close);
    }
    if (GROUPS && close) {
      __syncwarp();
      if (groups_close || !sig || !choose_among<NV>(a, mine, keys, kept[warp], sel_id[warp], error))
        choose_slowly<NV>(a, mine, kept[warp], sel_id[warp]);
    }
    if (!GROUPS) mx = warp_max(mx);
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
    if (!weighed || (sig && top != 0.f)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        l[i] = there(i) ? weight(weighed ? mine[lane + 32 * i] : l[i], top, sig) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) total += l[i];
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
      if (GROUPS || a.bias) {
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
// on one CTA.  With groups a CTA has 20 warps, whose threads keep all but 156 bytes (of 256
// experts; 76 of 224, and with fewer all) in registers (8192 rows of 256 experts 24.3 us against 25.2 on 16 warps, before the last steps 32.9
// on 32 and 31.5 on 16; 64 rows 10.3 against 9.9).
int most_warps(bool groups) { return groups ? 20 : 32; }

// warps of a CTA: its chosen experts and per-warp sums take shared memory
int forward_warps(int T, int grid, bool groups) {
  return grid > 1 || T > 8 ? most_warps(groups) : 8;
}

int forward_grid(int T, bool groups) {
  const int rows = most_warps(groups);
  if (T <= rows) return 1;
  const int want = (T - 1) / rows + 1, cap = num_sms();      // T + 31 may pass INT_MAX
  return want < cap ? want : cap;
}

size_t workspace_bytes_of(const moe_router_desc* s, int T, bool groups) {
  return (size_t)forward_grid(T, groups) * (2 * s->E + 2) * 4;
}

template <typename L, int NV, bool GROUPS>
cudaError_t launch_forward_nv(const RouterArgs& a, int grid, cudaStream_t st) {
  const int warps = forward_warps(a.T, grid, GROUPS);
  // with groups: the keys too, and the groups' values (256 at most)
  const int a_warp = GROUPS ? 2 * NV * 32 + 2 * a.groups : NV * 32;
  constexpr int most = 32 * (GROUPS ? 2 * NV * 32 + 2 * kMaxE : NV * 32) * (int)sizeof(float);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_router<L, NV, GROUPS>, most, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_router<L, NV, GROUPS>, dim3(grid), dim3(warps * 32),
                    warps * a_warp * (int)sizeof(float), st, a);
}

template <typename L, bool GROUPS>
cudaError_t launch_forward(const RouterArgs& a, int grid, cudaStream_t st) {
  switch ((a.E + 31) / 32) {
    case 1: return launch_forward_nv<L, 1, GROUPS>(a, grid, st);
    case 2: return launch_forward_nv<L, 2, GROUPS>(a, grid, st);
    case 3: return launch_forward_nv<L, 3, GROUPS>(a, grid, st);
    case 4: return launch_forward_nv<L, 4, GROUPS>(a, grid, st);
    case 5: return launch_forward_nv<L, GROUPS ? 5 : 8, GROUPS>(a, grid, st);
    case 6: return launch_forward_nv<L, GROUPS ? 6 : 8, GROUPS>(a, grid, st);
    case 7: return launch_forward_nv<L, GROUPS ? 7 : 8, GROUPS>(a, grid, st);
    default: return launch_forward_nv<L, 8, GROUPS>(a, grid, st);
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
  return workspace_bytes_of(s, T, false);
}

namespace moe {

namespace {

// Both forwards; g: the choice within groups (NULL: among all experts).
int forward(const moe_router_desc* s, const moe_group_router_desc* g, int T, const void* logits,
            long long ld, const float* bias, const uint8_t* token_mask, int32_t* ids, float* scores, int32_t* counts,
            float* prob_sum, float* losses, float* row_stat, void* workspace,
            size_t workspace_bytes, void* stream) {
  if (!sizes_ok(s, T) || !counts || !prob_sum || !losses) return MOE_ERR_INVALID_ARG;
  const int es = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (T > 0 && (!logits || ld < s->E || !ids || !scores || !row_stat || !aligned(logits, es)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(bias, 4) || !aligned(ids, 4) || !aligned(scores, 4) || !aligned(counts, 4) ||
      !aligned(prob_sum, 4) || !aligned(losses, 4) || !aligned(row_stat, 4))
    return MOE_ERR_INVALID_ARG;
  const int grid = forward_grid(T, g != nullptr);
  RouterArgs a = {};
  a.T = T; a.E = s->E; a.k = s->k; a.scoring = s->scoring; a.scale = s->scale;
  a.logits = logits; a.ld = ld; a.bias = bias; a.mask = token_mask;
  a.ids = ids; a.scores = scores; a.counts = counts; a.prob_sum = prob_sum; a.losses = losses;
  a.row_stat = row_stat;
  if (grid > 1) {
    if (!workspace || workspace_bytes < workspace_bytes_of(s, T, g != nullptr))
      return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    a.part_prob = static_cast<float*>(workspace);
    a.part_count = reinterpret_cast<int32_t*>(a.part_prob + (size_t)grid * a.E);
    a.part_z = reinterpret_cast<float*>(a.part_count + (size_t)grid * (a.E + 1));
    a.n_part = grid;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = s->dtype == MOE_DTYPE_FP32;
  cudaError_t e;
  if (g) {
    a.groups = g->groups; a.top_groups = g->top_groups; a.group_size = s->E / g->groups;
    a.pair = g->group_score == MOE_GROUP_TOP2 && a.group_size > 1;
    while ((2 << a.share_log2) * a.groups <= 32 && (2 << a.share_log2) <= a.group_size)
      a.share_log2 += 1;
    e = f32 ? launch_forward<float, true>(a, grid, st)
            : launch_forward<uint16_t, true>(a, grid, st);
  } else {
    e = f32 ? launch_forward<float, false>(a, grid, st)
            : launch_forward<uint16_t, false>(a, grid, st);
  }
  if (e == cudaSuccess && a.part_prob) e = launch_finish(a, st);
  return cuda_result(e, g ? "moe_group_router_forward" : "moe_router_forward");
}

// Adds `rate` to the biases of experts chosen less than the mean, subtracts it from those
// chosen more.  One warp; counts are whole numbers, so the comparison is exact.
__global__ void k_router_bias(float* bias, const int32_t* counts, int E, float rate) {
  pdl_wait();
  const int lane = threadIdx.x;
  long long total = 0;
  for (int e = lane; e < E; e += 32) total += counts[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  for (int e = lane; e < E; e += 32) {
    const long long mine = (long long)counts[e] * E;
    if (mine != total) bias[e] += mine < total ? rate : -rate;
  }
  pdl_trigger();
}

bool group_desc_ok(const moe_group_router_desc* g) {
  return g && desc_ok(&g->router) && g->groups >= 1 && g->router.E % g->groups == 0 &&
         g->top_groups >= 1 && g->top_groups <= g->groups &&
         g->router.k <= g->top_groups * (g->router.E / g->groups) &&
         (g->group_score == MOE_GROUP_MAX || g->group_score == MOE_GROUP_TOP2);
}

}  // namespace

}  // namespace moe

extern "C" int moe_router_forward(const moe_router_desc* s, int T, const void* logits,
                                  long long ld, const float* bias, const uint8_t* token_mask,
                                  int32_t* ids, float* scores, int32_t* counts, float* prob_sum,
                                  float* losses, float* row_stat, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return forward(s, nullptr, T, logits, ld, bias, token_mask, ids, scores, counts, prob_sum,
                 losses, row_stat, workspace, workspace_bytes, stream);
}

extern "C" size_t moe_group_router_workspace_bytes(const moe_group_router_desc* g, int T) {
  return group_desc_ok(g) && sizes_ok(&g->router, T) ? workspace_bytes_of(&g->router, T, true) : 0;
}

extern "C" int moe_group_router_forward(const moe_group_router_desc* g, int T, const void* logits,
                                        long long ld, const float* bias,
                                        const uint8_t* token_mask, int32_t* ids, float* scores,
                                        int32_t* counts, float* prob_sum, float* losses,
                                        float* row_stat, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  if (!group_desc_ok(g)) return MOE_ERR_INVALID_ARG;
  return forward(&g->router, g, T, logits, ld, bias, token_mask, ids, scores, counts, prob_sum,
                 losses, row_stat, workspace, workspace_bytes, stream);
}

extern "C" int moe_router_update_bias(float* bias, const int32_t* counts, int E, float rate,
                                      void* stream) {
  if (!bias || !counts || E < 1 || E > kMaxE || !std::isfinite(rate) || !aligned(bias, 4) ||
      !aligned(counts, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_result(launch_pdl(k_router_bias, dim3(1), dim3(32), 0,
                                static_cast<cudaStream_t>(stream), bias, counts, E, rate),
                     "moe_router_update_bias");
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
