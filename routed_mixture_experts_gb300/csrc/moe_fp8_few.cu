// moe_fp8_few.cu -- the 8-bit block product of a few rows: weights streamed once.
//
//   C[r, n] = sum_b sa[b, r] sb[e, n / 128, b] (A[r, b] . B[e, n, b])
//
// With a row or two an expert the weights' bytes are all that counts, and a 128 x 256 tile
// keeps only as many SMs busy as there are tiles.  Here a CTA has 16 rows of one expert's
// weights and its rows of A, 32 at most; its eight warps take the blocks of 128 along K in
// turn.  Each lane copies its own 16-byte pieces of the blocks to come into a ring (three
// blocks a warp ahead), so that nothing but its own copies is waited for.  The weights are
// the 16-row operand of m16n8k16: the same permutation of K in both operands leaves every
// product where it was, so the pieces are used as they lie.  Codes become fp16, exactly.  The
// other operand's eight columns are eight rows of A; more of them take the weights from the
// registers again.  A block's sum is scaled and added in fp32, the warps' sums are added in
// order through shared memory, which the ring gives up for it: two CTAs fit an SM, and the
// caller has no more of them than fit at once.
//
// Bound by latency: launch, offsets, the first blocks, an exchange.  M = 1, N = K = 4096
// 6.9 us (with one CTA an SM 8.5; on tiles 10.1; the weights' bytes 2.5), N = 300, K = 500 2.0
// (4.2), a row of each of two experts of 2048 x 1024 3.5.

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

// Four codes as two pairs of fp16 (exact).
struct Halves {
  uint32_t lo, hi;
};
__device__ __forceinline__ Halves halves(uint32_t codes) {
  Halves r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.lo), "=r"(r.hi)
      : "r"(codes));
  return r;
}

// c += 16 rows of weights (w0: row lane / 4, w1: eight below) times 8 rows of A, four codes of
// each lane.
__device__ __forceinline__ void mma_codes(float (&c)[4], uint32_t w0, uint32_t w1, uint32_t x) {
  const Halves a = halves(w0), b = halves(w1), v = halves(x);
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.lo), "r"(b.lo), "r"(a.hi), "r"(b.hi), "r"(v.lo), "r"(v.hi));
}

// 16 codes at p, of which n are there (zeros else).
__device__ __forceinline__ uint4 codes16(const uint8_t* p, int n) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (n > 0) {
    v = __ldg(reinterpret_cast<const uint4*>(p));
    if (n < 16) {
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = n - 4 * i;                 // bytes of this word
        w[i] = m >= 4 ? w[i] : m <= 0 ? 0u : w[i] & ((1u << (8 * m)) - 1u);
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return v;
}

// Asynchronous copy of 16 codes of which n (0..16) are there, zeros for the others.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool there) {
  const int n = there ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// A lane's share of a block, and a warp's ring of them.
struct __align__(16) Slot {
  uint4 w[4][32];          // [half of the block, upper or lower eight rows][lane]
  uint4 x[2][32];          // [half]: row lane / 4 of A, the first eight
  float s[3][32];          // scale of the weights' block, of rows 2 (lane % 4) and the next
};
constexpr int kDepth = 4, kGroups = 4;            // groups of eight rows of A
constexpr int kSmem = kWarps * kDepth * (int)sizeof(Slot);

__device__ __forceinline__ int clip16(int n) { return min(max(n, 0), 16); }

__global__ void __launch_bounds__(kWarps * 32, 2) k_fp8_few(const Fp8FewCall a) {
  extern __shared__ Slot ring_all[];
  __shared__ int counts[kWarps], mine_e[3];
  static_assert(2 * (kSmem + (int)sizeof(counts) + (int)sizeof(mine_e) + 1024) <= 228 * 1024,
                "two CTAs an SM");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  // rows [lo, hi) of expert e, the c-th that has some, and weights from n0 on
  const int n_tiles = (a.N + 15) >> 4, c = blockIdx.x / n_tiles;
  const int n0 = (blockIdx.x - c * n_tiles) << 4;
  int e = 0, lo = 0, hi = a.M;
  if (a.offsets) {
    const int i = threadIdx.x;
    int from = 0, to = 0;
    if (i < a.E) {
      from = a.offsets[i];
      to = a.offsets[i + 1];
    }
    if (__syncthreads_or(from < 0 || to < from || to > a.M)) {
      if (blockIdx.x == 0 && i == 0) record_error(a.err, MOE_ERR_INVALID_ARG, 0);
      return;
    }
    const unsigned has = __ballot_sync(kAll, to > from);
    if (lane == 0) counts[warp] = __popc(has);
    if (i == 0) mine_e[0] = -1;
    __syncthreads();
    int place = __popc(has & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) place += counts[w];
    if (to > from && place == c) {
      mine_e[0] = i;
      mine_e[1] = from;
      mine_e[2] = to;
    }
    __syncthreads();
    e = mine_e[0];
    lo = mine_e[1];
    hi = mine_e[2];
    if (e < 0) return;                           // fewer experts have rows
  }
  const int k_blocks = (a.K + 127) >> 7, nb_all = (a.N + 127) >> 7;
  const int mine = (k_blocks - warp + kWarps - 1) / kWarps;      // blocks: warp + 8 j
  Slot* const ring = ring_all + warp * kDepth;
  // the copies, a group a block (an empty one past the end)
  int ahead = 0, in = 0;
  auto copy = [&]() {
    if (ahead < mine) {
      Slot& s = ring[in];
      const int b = warp + kWarps * ahead, k = (b << 7) + 16 * t;
      const int n = a.K - k;
      const uint8_t* const w = a.b + ((long long)e * a.N + n0 + g) * a.ld_b + k;
      const bool in0 = n0 + g < a.N, in1 = n0 + g + 8 < a.N;
      const bool row = lo + g < hi;
      const uint8_t* const x = a.a + (long long)(lo + g) * a.ld_a + k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = clip16(n - 64 * h);
        const int m0 = in0 ? m : 0, m1 = in1 ? m : 0, mx = row ? m : 0;
        copy16(smem_u32(&s.w[2 * h][lane]), m0 ? w + 64 * h : a.b, m0);
        copy16(smem_u32(&s.w[2 * h + 1][lane]), m1 ? w + 8LL * a.ld_b + 64 * h : a.b, m1);
        copy16(smem_u32(&s.x[h][lane]), mx ? x + 64 * h : a.a, mx);
      }
      copy4(smem_u32(&s.s[0][lane]),
            a.sb + ((long long)e * nb_all + (n0 >> 7)) * k_blocks + b, true);
      const int r = lo + 2 * t;
      const float* const sa = a.sa + b * a.ld_sa + r;
      copy4(smem_u32(&s.s[1][lane]), r < hi ? sa : a.sa, r < hi);
      copy4(smem_u32(&s.s[2][lane]), r + 1 < hi ? sa + 1 : a.sa, r + 1 < hi);
      ++ahead;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++in == kDepth) in = 0;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) copy();
  const int groups = (hi - lo + 7) >> 3;
  float sum[kGroups][4];
#pragma unroll
  for (int q = 0; q < kGroups; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[q][i] = 0.f;
  int out = 0;
  for (int j = 0; j < mine; ++j) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    const Slot& s = ring[out];
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = s.w[i][lane];
    const float f = s.s[0][lane];
    auto add = [&](const uint4 (&x)[2], float s0, float s1, float (&to)[4]) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_codes(c, w[2 * h].x, w[2 * h + 1].x, x[h].x);
        mma_codes(c, w[2 * h].y, w[2 * h + 1].y, x[h].y);
        mma_codes(c, w[2 * h].z, w[2 * h + 1].z, x[h].z);
        mma_codes(c, w[2 * h].w, w[2 * h + 1].w, x[h].w);
      }
      to[0] = fmaf(c[0], f * s0, to[0]);
      to[1] = fmaf(c[1], f * s1, to[1]);
      to[2] = fmaf(c[2], f * s0, to[2]);
      to[3] = fmaf(c[3], f * s1, to[3]);
    };
    {
      const uint4 x[2] = {s.x[0][lane], s.x[1][lane]};
      add(x, s.s[1][lane], s.s[2][lane], sum[0]);
    }
    const int b = warp + kWarps * j, k = (b << 7) + 16 * t;
#pragma unroll
    for (int q = 1; q < kGroups; ++q)
      if (q < groups) {                          // rows beyond eight: as they come
        const int r = lo + 8 * q + g, c = lo + 8 * q + 2 * t;
        uint4 x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[h] = codes16(a.a + (long long)r * a.ld_a + k + 64 * h,
                         r < hi ? a.K - k - 64 * h : 0);
        add(x, c < hi ? __ldg(a.sa + b * a.ld_sa + c) : 0.f,
            c + 1 < hi ? __ldg(a.sa + b * a.ld_sa + c + 1) : 0.f, sum[q]);
      }
    if (++out == kDepth) out = 0;
    copy();                                      // into the slot before this one
  }
  // The warps' sums of eight rows at a time, [row of A][row of weights] in the first two slots
  // of each warp's own ring by turns: all that was copied has been waited for and read.
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  typedef float Part[8][17];
  static_assert(sizeof(Part) <= sizeof(Slot), "a slot holds a part");
  for (int q = 0; q < groups; ++q) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q == 0 ? sum[0][i] : q == 1 ? sum[1][i]
                                      : q == 2 ? sum[2][i] : sum[3][i];
    Part& p = *reinterpret_cast<Part*>(ring + (q & 1));
    p[2 * t][g] = v[0];
    p[2 * t + 1][g] = v[1];
    p[2 * t][g + 8] = v[2];
    p[2 * t + 1][g + 8] = v[3];
    __syncthreads();
    const int r = lo + 8 * q + (threadIdx.x >> 4), n = threadIdx.x & 15;
    if (threadIdx.x < 128 && r < hi && n0 + n < a.N) {
      float y = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        y += (*reinterpret_cast<const Part*>(ring_all + i * kDepth + (q & 1)))[threadIdx.x >> 4][n];
      const long long at = (long long)r * a.ld_c + n0 + n;
      if (a.f32)
        static_cast<float*>(a.c)[at] = y;
      else
        static_cast<uint16_t*>(a.c)[at] = f2bf(y);
    }
  }
  pdl_trigger();
}

}  // namespace

cudaError_t launch_fp8_few(const Fp8FewCall& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_fp8_few, kSmem, done);
  if (e != cudaSuccess) return e;
  // a CTA for every 16 rows of weights of every expert that may have rows (M <= 32 of them)
  const int experts = !a.offsets ? 1 : a.M < a.E ? a.M : a.E;
  return launch_pdl(k_fp8_few, dim3((unsigned)(experts * ((a.N + 15) / 16))), dim3(kWarps * 32),
                    kSmem, stream, a);
}

}  // namespace moe
