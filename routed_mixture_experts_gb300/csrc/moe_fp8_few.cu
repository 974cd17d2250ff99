// moe_fp8_few.cu -- the 8-bit block product of a few rows: weights streamed once.
//
//   C[r, n] = sum_b sa[b, r] sb[e, n / 128, b] (A[r, b] . B[e, n, b])
//
// With a row or two an expert the weights' bytes are all that counts, and a 128 x 256 tile
// keeps only as many SMs busy as there are tiles.  Here a unit is 16 rows of one expert's
// weights and up to 32 of its rows of A; a persistent CTA's eight warps take the unit's
// blocks of 128 along K in turn.  Each lane copies its own 16-byte pieces of the blocks to
// come into a ring (three blocks a warp ahead, across units), so that nothing but
// its own copies is waited for.  The weights are the 16-row operand of m16n8k16: the same
// permutation of K in both operands leaves every product where it was, so the pieces are
// used as they lie.  Codes become fp16, exactly.  The other operand's eight columns are
// eight rows of A; more of them take the weights from the registers again.  A block's sum is
// scaled and added in fp32, the warps' sums are added in order through shared memory.
//
// Bound by latency: launch, offsets, the first blocks, an exchange a unit.  M = 1, N = K =
// 4096 8.2 us (10.1 on tiles; the weights' bytes 2.5), N = 300, K = 500 2.0 (4.2).

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_fp8.cuh"
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
constexpr int kDepth = 4, kGroups = 4, kRows = 8 * kGroups;
constexpr int kSmem = kWarps * kDepth * (int)sizeof(Slot);

// Where a CTA is: 16 rows of weights of one expert, and up to 32 of its rows of A.
struct Unit {
  int left;                // units to come, this one included
  int e, lo, hi, n0;       // expert, rows, first row of weights
  int end;                 // end of the expert's rows
};

__device__ __forceinline__ int clip16(int n) { return min(max(n, 0), 16); }

__global__ void __launch_bounds__(kWarps * 32, 2) k_fp8_few(const Fp8FewCall a) {
  extern __shared__ Slot ring_all[];
  __shared__ float part[2][kWarps][8][17];       // [warp][row of A][row of weights]
  __shared__ int first[kMaxSegments + 1], begin[kMaxSegments], end[kMaxSegments];
  __shared__ int sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  // chunks of 32 rows of the experts: chunk c belongs to the e with first[e] <= c < first[e + 1]
  int chunks = (a.M + kRows - 1) / kRows;
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
    const int n = (int)(((unsigned)(to - from) + kRows - 1) / kRows);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sums[w];
    if (i < a.E) {
      first[i + 1] = incl;
      begin[i] = from;
      end[i] = to;
    }
    if (i == 0) first[0] = 0;
    __syncthreads();
    chunks = first[a.E];
  }
  const int n_tiles = (a.N + 15) >> 4, units = chunks * n_tiles;
  const int k_blocks = (a.K + 127) >> 7, nb_all = (a.N + 127) >> 7;
  const int mine = (k_blocks - warp + kWarps - 1) / kWarps;      // blocks of a unit: warp + 8 j
  // a CTA's units follow one another: tiles of a chunk, chunks of an expert, experts
  const int per = units / (int)gridDim.x, more = units % (int)gridDim.x, id = blockIdx.x;
  Unit u;
  u.left = per + (id < more ? 1 : 0);
  if (u.left == 0) return;
  {
    const int at = id * per + min(id, more), c = at / n_tiles;
    u.n0 = (at - c * n_tiles) << 4;
    u.e = 0;
    u.lo = c * kRows;
    u.end = a.M;
    if (a.offsets) {
      int lo = 0, hi = a.E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= c) lo = mid; else hi = mid;
      }
      u.e = lo;
      u.lo = begin[lo] + (c - first[lo]) * kRows;
      u.end = end[lo];
    }
    u.hi = min(u.end, u.lo + kRows);
  }
  auto advance = [&](Unit& v) {
    if (--v.left == 0) return;
    v.n0 += 16;
    if (v.n0 < a.N) return;
    v.n0 = 0;
    v.lo = v.hi;
    if (v.lo == v.end) {
      do ++v.e; while (begin[v.e] == end[v.e]);  // (there is one: units are left)
      v.lo = begin[v.e];
      v.end = end[v.e];
    }
    v.hi = min(v.end, v.lo + kRows);
  };
  Slot* const ring = ring_all + warp * kDepth;
  // the copies: block j of the unit ahead, a group each (an empty one past the end)
  Unit ahead = u;
  int ahead_j = 0, in = 0;
  auto copy = [&]() {
    if (ahead.left > 0 && mine > 0) {
      Slot& s = ring[in];
      const int b = warp + kWarps * ahead_j, k = (b << 7) + 16 * t;
      const int n = a.K - k;
      const uint8_t* const w =
          a.b + ((long long)ahead.e * a.N + ahead.n0 + g) * a.ld_b + k;
      const bool in0 = ahead.n0 + g < a.N, in1 = ahead.n0 + g + 8 < a.N;
      const bool row = ahead.lo + g < ahead.hi;
      const uint8_t* const x = a.a + (long long)(ahead.lo + g) * a.ld_a + k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = clip16(n - 64 * h);
        const int m0 = in0 ? m : 0, m1 = in1 ? m : 0, mx = row ? m : 0;
        copy16(smem_u32(&s.w[2 * h][lane]), m0 ? w + 64 * h : a.b, m0);
        copy16(smem_u32(&s.w[2 * h + 1][lane]), m1 ? w + 8LL * a.ld_b + 64 * h : a.b, m1);
        copy16(smem_u32(&s.x[h][lane]), mx ? x + 64 * h : a.a, mx);
      }
      copy4(smem_u32(&s.s[0][lane]),
            a.sb + ((long long)ahead.e * nb_all + (ahead.n0 >> 7)) * k_blocks + b, true);
      const int c = ahead.lo + 2 * t;
      const float* const sa = a.sa + b * a.ld_sa + c;
      copy4(smem_u32(&s.s[1][lane]), c < ahead.hi ? sa : a.sa, c < ahead.hi);
      copy4(smem_u32(&s.s[2][lane]), c + 1 < ahead.hi ? sa + 1 : a.sa, c + 1 < ahead.hi);
      if (++ahead_j >= mine) {
        ahead_j = 0;
        advance(ahead);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++in == kDepth) in = 0;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) copy();
  int out = 0, buf = 0;
  for (; u.left > 0; advance(u)) {
    const int groups = (u.hi - u.lo + 7) >> 3;
    float sum[kGroups][4];
#pragma unroll
    for (int q = 0; q < kGroups; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[q][i] = 0.f;
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
        if (q < groups) {                        // rows beyond eight: as they come
          const int r = u.lo + 8 * q + g, c = u.lo + 8 * q + 2 * t;
          uint4 x[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[h] = codes16(a.a + (long long)r * a.ld_a + k + 64 * h,
                           r < u.hi ? a.K - k - 64 * h : 0);
          add(x, c < u.hi ? __ldg(a.sa + b * a.ld_sa + c) : 0.f,
              c + 1 < u.hi ? __ldg(a.sa + b * a.ld_sa + c + 1) : 0.f, sum[q]);
        }
      if (++out == kDepth) out = 0;
      copy();                                    // into the slot before this one
    }
    for (int q = 0; q < groups; ++q) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = q == 0 ? sum[0][i] : q == 1 ? sum[1][i]
                                        : q == 2 ? sum[2][i] : sum[3][i];
      float (&p)[8][17] = part[buf][warp];
      p[2 * t][g] = v[0];
      p[2 * t + 1][g] = v[1];
      p[2 * t][g + 8] = v[2];
      p[2 * t + 1][g + 8] = v[3];
      __syncthreads();
      const int r = u.lo + 8 * q + (threadIdx.x >> 4), n = threadIdx.x & 15;
      if (threadIdx.x < 128 && r < u.hi && u.n0 + n < a.N) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) y += part[buf][i][threadIdx.x >> 4][n];
        const long long at = (long long)r * a.ld_c + u.n0 + n;
        if (a.f32)
          static_cast<float*>(a.c)[at] = y;
        else
          static_cast<uint16_t*>(a.c)[at] = f2bf(y);
      }
      buf ^= 1;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_trigger();
}

}  // namespace

cudaError_t launch_fp8_few(const Fp8FewCall& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = smem_optin_once(k_fp8_few, kSmem, done);
  if (e != cudaSuccess) return e;
  // every expert's last chunk may hold as little as one row
  const long long chunks = (a.M - 1LL) / kRows + (a.offsets ? (a.M < a.E ? a.M : a.E) : 1);
  const long long units = chunks * ((a.N + 15) / 16);
  const int sms = num_sms();
  return launch_pdl(k_fp8_few, dim3((unsigned)(units < 2 * sms ? units : 2 * sms)),
                    dim3(kWarps * 32), kSmem, stream, a);
}

}  // namespace moe
