// moe_fp8_gemm.cu -- products of E4M3 codes with one fp32 scale per 128 elements.
//
//   rows      C[r, n] = sum_b sa[b, r] sb[e, n / 128, b] (A[r, b] . B[e, n, b])
//             e the expert of row r, b the blocks of 128 along K
//   weights   dW[e, n, k] (+)= sum_b sy[b, n] sx[b, k] (dYt[n, b] . Xt[k, b])
//             b the blocks of expert e's rows; operands with codes along the rows
//
// The scales change with every block of 128, so the tensor core's sum ends there: the
// 128 products of a block go to tensor memory in fp32 (four K = 32 instructions), are read
// back, and join the running sum in registers with one fused multiply-add an element (two
// multiplications for the weights, whose columns have scales of their own), all fp32.
//
// A tile is 128 x 256: the widest whose sums fit the registers, and a part of tensor memory
// that leaves a second one, which tcgen05.mma writes while the warps read the first; 48 KB
// of codes a block and four of them on their way (weights: three, which leaves room for tiles
// on their way out; before those had any, 4 / 3 / 2 took 302 / 290 / 320 us).  Narrower tiles
// (128 columns, four parts) serve shapes of a single wave.
//
// Bound by the way of the sums: from the last MMA of a block until its part is free again
// some 900 cycles pass a block (barriers, tensor memory loads of 46 cycles and more, additions),
// where its MMAs take 512 and its copies, at the 64 bytes a cycle an SM gets from L2, 768.
// Dense 8192 x 4096 x 4096 106 us (2.6 PFLOP/s), M = 65536, N = 1536, K = 2048 on 128 experts
// 206 (2.0), or up to 242 (1.7) where the power limit lowers the clocks, its weight gradient on
// 32 experts 267 (1.54); 512 rows on the 128 experts 60, the weights' bytes at a copy's rate.

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_fp8.cuh"
#include "moe_gemm_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

struct Fp8GemmArgs {
  int M, N, K, E;                    // rows, columns, depth (weights: dW is [E, N, K])
  const float* sa;  long long ld_sa; // [blocks][rows of A]
  const float* sb;  long long ld_sb; // rows: [E][N blocks][K blocks]; weights: [blocks][K]
  const int32_t* offsets;            // [E+1] or NULL: one segment
  void* c;  long long ld_c;
  int row_blocks;                    // weights: blocks of 128 that the codes have
  int f32, accumulate, wide;         // wide: 16-byte stores (weights: 2, 8-byte; 4, copies)
  DevError* err;
};

// D[tmem] (+)= A B^T, kind::f8f6f4: E4M3 operands, fp32 sums.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: fp32 D (bits 4-5 = 1), E4M3 A and B (format 0 in
// bits 7-9 and 10-12), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 32 lanes x 32 consecutive 32-bit columns of TMEM into 32 registers per thread.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// Waits for this thread's loads; their registers pass through it, so that nothing that uses
// them is scheduled before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 16 lanes x 16 consecutive columns: a thread gets, of each 8 columns, two neighbours
// (2 (lane % 4)) of row lane / 4 and of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8], uint32_t (&q)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]),
                 "+r"(q[4]), "+r"(q[5]), "+r"(q[6]), "+r"(q[7])
               :
               : "memory");
}

// One lane of a converged warp.  Code under it keeps its operands in uniform registers, as
// the tensor core's instructions take them; under a test of the lane each is moved there.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Arrival of lane 0 for its warp, without a branch.  Relaxed: what the warp has read is in
// its registers, and it has written nothing that others wait for.  (An arrival that
// releases took 150 cycles a block.)
__device__ __forceinline__ void arrive_lane0(uint32_t bar, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(lane)
      : "memory");
}

// Asynchronous copy of 4 bytes into shared memory, zero where `there` is false.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool there) {
  const int n = there ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// Warp 0 copies codes, warp 1 issues MMAs, warp 2 copies scales (3 is idle), and from warp 4
// on each adds 32 rows x WIDE columns.  The registers that the first four are launched with
// and do not need go to the others, which hold the sums.
template <int BN, bool WGRAD>
struct Shape {
  static constexpr int SUM_WARPS = WGRAD ? 16 : 8, THREADS = 128 + 32 * SUM_WARPS;
  static constexpr int WIDE = BN / (SUM_WARPS / 4);
  static constexpr int LAUNCH_REGS = WGRAD ? 96 : 168, COPY_REGS = WGRAD ? 56 : 40;
  static constexpr int SUM_REGS = WGRAD ? 104 : 232;
  static_assert(4 * COPY_REGS + SUM_WARPS * SUM_REGS <= (4 + SUM_WARPS) * LAUNCH_REGS,
                "what the first warps give up is all that there is");
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // on the way out: a warp's 32 rows x 64 bytes, 80 apart (weights: x 128)
  static constexpr int TURN = SUM_WARPS * 32 * (WGRAD ? 128 : 80);
  // scales of GROUP blocks: of each its 128 rows', then (weights) BN columns' or the two
  // weight blocks'
  static constexpr int GROUP = 4, SLOTS = WGRAD ? 2 : 4, BLOCK = 512 + (WGRAD ? BN * 4 : 16);
  static constexpr int SLOT = GROUP * BLOCK;
  static constexpr int REST = TURN + SLOTS * SLOT + 512;
  static constexpr int FIT = (226 * 1024 - 3584 - REST) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = STAGES * STAGE + REST + 1024;
  static constexpr int NBUF = 512 / BN;                      // parts of tensor memory
};

// A value that is the same in every lane of a converged warp, in a form that shows it to the
// compiler (what comes from shared memory does not): loops and addresses stay uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

struct Tile {
  int e, m0, m1;       // expert, rows [m0, m1) of C (weights: of dW)
  int n0;
  int b0, b1;          // blocks along the depth
};

// Persistent: tiles in turn over the CTAs, every role walking the same sequence.  Weights' tiles
// are as deep as their expert has rows: the deepest experts come first (order), and the CTAs
// are dealt tiles forwards and backwards by turns (65536 rows on 32 experts, 6 to 56 blocks
// each: the deepest CTA has 340 blocks where the experts' order gives 379, and the mean is
// 333; 302 us against 329, before the tiles left by copies).
template <int BN, bool WGRAD>
__device__ __forceinline__ Tile tile_of(const Fp8GemmArgs& a, const Segments& seg,
                                        const uint8_t* order, int t, int n_tiles) {
  Tile r;
  if (WGRAD) {
    const int m_tiles = (a.N + 127) >> 7, per = m_tiles * n_tiles;
    const int place = t / per;
    const int q = t - place * per;
    r.e = order[place];
    r.m0 = (q / n_tiles) << 7;
    r.m1 = min(r.m0 + 128, a.N);
    r.n0 = (q % n_tiles) * BN;
    r.b0 = a.offsets ? seg.first[r.e] : 0;       // (within row_blocks: checked)
    r.b1 = a.offsets ? seg.first[r.e + 1] : a.row_blocks;
  } else {
    const int b = t / n_tiles;
    r.n0 = (t - b * n_tiles) * BN;
    r.b0 = 0;
    r.b1 = (a.K + 127) >> 7;
    if (a.offsets) {
      r.e = seg.find(b, a.E);
      r.m0 = seg.begin[r.e] + ((b - seg.first[r.e]) << 7);
      r.m1 = min(seg.end[r.e], r.m0 + 128);
    } else {
      r.e = 0;
      r.m0 = b << 7;
      r.m1 = min(a.M, r.m0 + 128);
    }
  }
  return r;
}

// What a summing warp keeps of the rings: the scales' slot, the part of tensor memory, their
// phases.
struct Reader {
  const float* slots;
  uint32_t sfull, sempty, tfull, tempty;         // first barriers
  int slot, buf;
  uint32_t slot_phase, buf_phase;
  bool ok;
  volatile int* abort;
  DevError* err;

  __device__ __forceinline__ void wait_scales() {
    ok = ok && mbar_wait(sfull + 8u * slot, slot_phase, abort, err, 7);
  }
  __device__ __forceinline__ void wait_sums() {
    ok = ok && mbar_wait(tfull + 8u * buf, buf_phase, abort, err, 5);
    __syncwarp();
    tc_fence_after();
  }
  __device__ __forceinline__ void free_scales(int lane) { arrive_lane0(sempty + 8u * slot, lane); }
  __device__ __forceinline__ void free_sums(int lane) {
    tc_fence_before();
    __syncwarp();
    arrive_lane0(tempty + 8u * buf, lane);
  }
  template <int SLOTS>
  __device__ __forceinline__ void next_slot() {
    if (++slot == SLOTS) {
      slot = 0;
      slot_phase ^= 1u;
    }
  }
  template <int NBUF>
  __device__ __forceinline__ void next_buf() {
    if (++buf == NBUF) {
      buf = 0;
      buf_phase ^= 1u;
    }
  }
};

// Rows of C: a thread adds one row x WIDE columns.
template <int BN>
__device__ __forceinline__ void sum_rows(const Fp8GemmArgs& args, const Tile& ti, Reader& rd,
                                         uint32_t lane_base, int quarter, int group, int lane,
                                         uint8_t* turn) {
  using S = Shape<BN, false>;
  constexpr int WIDE = S::WIDE, CH = 32;         // CH: columns a load
  const int row = quarter * 32 + lane, r = ti.m0 + row, c0 = ti.n0 + group * WIDE;
  if (ti.m0 + quarter * 32 >= ti.m1) {           // rows of nobody: only the rings go on
    for (int b = ti.b0; b < ti.b1; ++b) {
      rd.wait_sums();
      rd.free_sums(lane);
      rd.next_buf<S::NBUF>();
      if ((b - ti.b0) % S::GROUP == S::GROUP - 1 || b + 1 == ti.b1) {
        rd.wait_scales();
        rd.free_scales(lane);
        rd.next_slot<S::SLOTS>();
      }
    }
    return;
  }
  uint64_t acc[WIDE / 2];
#pragma unroll
  for (int i = 0; i < WIDE / 2; ++i) acc[i] = 0;
  // The next load is on its way while one is added: of the same block, or the first of the
  // next, whose barrier is looked at before this one's last addition.
  uint32_t d[2][CH];
  float s = 0.f;
  auto start = [&](int b) {
    const int i = (b - ti.b0) % S::GROUP;
    if (i == 0) rd.wait_scales();
    const float* const sc = rd.slots + (rd.slot * S::SLOT + i * S::BLOCK) / 4;
    s = sc[row] * sc[128 + (group * WIDE >> 7)];
    rd.wait_sums();
    tmem_ld(lane_base + (uint32_t)(rd.buf * BN), d[0]);
  };
  if (ti.b0 < ti.b1) start(ti.b0);
  for (int b = ti.b0; b < ti.b1; ++b) {
    const uint32_t tb = lane_base + (uint32_t)(rd.buf * BN);
    const uint64_t s2 = pair(s, s);
    const bool last = (b - ti.b0) % S::GROUP == S::GROUP - 1 || b + 1 == ti.b1;
#pragma unroll
    for (int i = 0; i < WIDE / CH; ++i) {
      tmem_wait(d[i & 1]);
      if (i + 1 < WIDE / CH) {
        tmem_ld(tb + (uint32_t)(CH * (i + 1)), d[(i + 1) & 1]);
      } else {
        rd.free_sums(lane);
        if (last) rd.free_scales(lane);          // of the group's last block
        rd.next_buf<S::NBUF>();
        if (last) rd.next_slot<S::SLOTS>();
        static_assert((WIDE / CH) % 2 == 0, "the next block starts with d[0]");
        if (b + 1 < ti.b1) start(b + 1);
      }
#pragma unroll
      for (int j = 0; j < CH / 2; ++j)
        acc[CH / 2 * i + j] =
            fma2(pair_u(d[i & 1][2 * j], d[i & 1][2 * j + 1]), s2, acc[CH / 2 * i + j]);
    }
  }
  // ---- out ----
  // 64 bytes of each of the warp's rows at a time are turned in shared memory (rows 80 bytes
  // apart, so that neither side meets in a bank), and four lanes write a row's, or all of
  // them its single elements where rows are not aligned (N = 4095 118 us, N = 4096 107).
  const int n_here = min(WIDE, args.N - c0);     // columns of this warp
  if (n_here <= 0) return;
  const int rows_here = min(32, ti.m1 - ti.m0 - quarter * 32);
  const long long row0 = r - lane;               // the warp's first row
  auto put = [&](auto type, const uint32_t (&w)[16], int first) {
    using T = decltype(type);
    constexpr int COLS = 64 / (int)sizeof(T), EACH = 16 / (int)sizeof(T);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(turn + lane * 80 + 16 * q) =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    __syncwarp();
    T* const out = static_cast<T*>(args.c) + row0 * args.ld_c + c0 + first;
    if (args.wide && first + COLS <= n_here) {
      const int q = lane & 3;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 8 * i + (lane >> 2);
        if (k < rows_here)
          *reinterpret_cast<uint4*>(out + k * args.ld_c + EACH * q) =
              *reinterpret_cast<const uint4*>(turn + k * 80 + 16 * q);
      }
    } else {
      constexpr int AT_ONCE = 32 / COLS;         // rows
      const int c = lane % COLS;
      if (first + c < n_here)
        for (int k = lane / COLS; k < rows_here; k += AT_ONCE)
          out[k * args.ld_c + c] = *reinterpret_cast<const T*>(turn + k * 80 + c * sizeof(T));
    }
  };
  if (args.f32) {
#pragma unroll
    for (int i = 0; i < WIDE / 16; ++i) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x, y;
        unpair(acc[8 * i + j], x, y);
        w[2 * j] = __float_as_uint(x);
        w[2 * j + 1] = __float_as_uint(y);
      }
      put(float(), w, 16 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < WIDE / 32; ++i) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float x, y;
        unpair(acc[16 * i + j], x, y);
        w[j] = pack_bf2(x, y);
      }
      put(uint16_t(), w, 32 * i);
    }
  }
  __syncwarp();
}

// Weights: a thread adds four rows (lane / 4 + 8 j) of every fourth pair of columns, the
// 16x256b shape of the tensor memory loads.  With a row a thread, as above, every thread
// would read every column's scale from shared memory: 128 KB a block, twice what the sums'
// additions take; so it is 16 columns a thread, a quarter of that.
template <int BN>
__device__ __forceinline__ void sum_weights(const Fp8GemmArgs& args, const Tile& ti, Reader& rd,
                                            uint32_t lane_base, int quarter, int group,
                                            int lane, uint32_t turn, const CUtensorMap* out_map) {
  using S = Shape<BN, true>;
  constexpr int WIDE = S::WIDE, CH = 16;         // CH: columns a load
  const int row = quarter * 32 + (lane >> 2), pair0 = 2 * (lane & 3);
  uint64_t acc[WIDE / 8][4];                     // [8 columns][row 8 j]
#pragma unroll
  for (int i = 0; i < WIDE / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  for (int b = ti.b0; b < ti.b1; ++b) {
    const int i = (b - ti.b0) % S::GROUP;
    if (i == 0) rd.wait_scales();
    const float* const sc = rd.slots + (rd.slot * S::SLOT + i * S::BLOCK) / 4;
    const float* const cs = sc + 128 + group * WIDE + pair0;
    uint64_t s2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = sc[row + 8 * j];
      s2[j] = pair(s, s);
    }
    const bool last = i == S::GROUP - 1 || b + 1 == ti.b1;
    rd.wait_sums();
#pragma unroll
    for (int c = 0; c < WIDE / CH; ++c) {
      const uint32_t at = lane_base + (uint32_t)(rd.buf * BN + CH * c);
      uint32_t d[2][8];                          // rows 0..15, rows 16..31
      tmem_ld_16x256b_x2(at, d[0]);
      tmem_ld_16x256b_x2(at + (16u << 16), d[1]);
      uint64_t x2[2];                            // (as pairs: put together they are moved)
#pragma unroll
      for (int g = 0; g < 2; ++g) x2[g] = *reinterpret_cast<const uint64_t*>(cs + CH * c + 8 * g);
      tmem_wait(d[0], d[1]);
      if (c + 1 == WIDE / CH) rd.free_sums(lane);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t* const q = d[j >> 1] + 4 * g + 2 * (j & 1);
          acc[2 * c + g][j] = fma2(mul2(pair_u(q[0], q[1]), x2[g]), s2[j], acc[2 * c + g][j]);
        }
      }
    }
    rd.next_buf<S::NBUF>();
    if (last) {
      __syncwarp();
      rd.free_scales(lane);
      rd.next_slot<S::SLOTS>();
    }
  }
  // ---- out ----
  if (args.accumulate && ti.b0 == ti.b1) return;
  float* const out = static_cast<float*>(args.c) + (long long)ti.e * args.N * args.K;
  const int c0 = ti.n0 + group * WIDE + pair0;
  if (args.wide == 4) {
    // 32 x 32 at a time through shared memory, whose copies out go on beside the next tile's
    // sums (279 us; written from registers, a tile of 128 KB kept the warps: 290).
#pragma unroll
    for (int h = 0; h < WIDE / 32; ++h) {
      if (lane == 0) bulk_wait_read<0>();        // of what was there before
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ti.m0 + row + 8 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 32 * h + 8 * i;
          float x, y;
          unpair(acc[4 * h + i][j], x, y);
          if (args.accumulate && r < ti.m1 && c < args.K) {
            const float2 v = *reinterpret_cast<const float2*>(out + (long long)r * args.K + c);
            x += v.x;
            y += v.y;
          }
          // rows of 128 bytes whose 16-byte pieces are turned by the row (lane / 4 of eight)
          const uint32_t piece = (uint32_t)(2 * i + ((lane & 3) >> 1)) ^ (uint32_t)(lane >> 2);
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(
                           turn + (uint32_t)(((lane >> 2) + 8 * j) * 128 + 8 * (lane & 1)) +
                           16u * piece),
                       "f"(x), "f"(y)
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int c = ti.n0 + group * WIDE + 32 * h, r = ti.m0 + quarter * 32;
        if (c < args.K && r < ti.m1) tma_store_3d(out_map, turn, c, r, ti.e);
        bulk_commit();
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = ti.m0 + row + 8 * j;
    if (r >= ti.m1) continue;
    float* const p = out + (long long)r * args.K;
#pragma unroll
    for (int i = 0; i < WIDE / 8; ++i) {
      const int c = c0 + 8 * i;
      float x, y;
      unpair(acc[i][j], x, y);
      if (args.wide) {                           // an even width: both columns or none
        if (c < args.K) {
          float2* const q = reinterpret_cast<float2*>(p + c);
          if (args.accumulate) {
            const float2 v = *q;
            x += v.x;
            y += v.y;
          }
          *q = make_float2(x, y);
        }
      } else {
        if (c < args.K) p[c] = args.accumulate ? p[c] + x : x;
        if (c + 1 < args.K) p[c + 1] = args.accumulate ? p[c + 1] + y : y;
      }
    }
  }
}

template <int BN, bool WGRAD>
__global__ void __launch_bounds__((Shape<BN, WGRAD>::THREADS), 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmC, const Fp8GemmArgs args) {
  using S = Shape<BN, WGRAD>;
  constexpr int STAGES = S::STAGES, NBUF = S::NBUF, SLOTS = S::SLOTS, WIDE = S::WIDE;
  static_assert(S::SMEM + 3584 <= 232448, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint8_t order[WGRAD ? kMaxSegments : 1];
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int abort_s;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* const turn_all = smem + STAGES * S::STAGE;
  float* const slots = reinterpret_cast<float*>(turn_all + S::TURN);
  const uint32_t bar0 = smem_u32(slots + SLOTS * S::SLOT / 4);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + NBUF + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * NBUF);
  auto sfull_bar = [&](int s) { return drain_bar + 8u * (1 + s); };
  auto sempty_bar = [&](int s) { return drain_bar + 8u * (1 + SLOTS + s); };
  static_assert(8 * (2 * STAGES + 2 * NBUF + 1 + 2 * SLOTS) <= 512, "barriers");

  // (read through a shuffle, so that the compiler knows it to be the same in a warp)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), S::SUM_WARPS);
    }
    mbar_init(drain_bar, 1);
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(sfull_bar(s), 32);
      mbar_init(sempty_bar(s), S::SUM_WARPS);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  pdl_wait();                        // the previous kernel of the stream has completed
  bool bad = false;
  if (args.offsets) {
    seg.init<S::THREADS>(args.offsets, args.E, WGRAD ? 0x7FFFFFFF : args.M);
    bad = seg.bad || (WGRAD && seg.first[args.E] > args.row_blocks);   // more than the codes have
    if (bad && blockIdx.x == 0 && threadIdx.x == 0)
      record_error(args.err, MOE_ERR_INVALID_ARG, 0);
  }
  const int n_tiles = ((WGRAD ? args.K : args.N) + BN - 1) / BN;
  const int num_tiles = uniform(
      WGRAD ? args.E * ((args.N + 127) >> 7) * n_tiles
            : (args.offsets ? seg.first[args.E] : (args.M + 127) >> 7) * n_tiles);
  if ((int)blockIdx.x >= num_tiles || (WGRAD && bad)) return;

  // the experts by depth; those as deep as another in their order
  if (WGRAD && threadIdx.x < args.E) {           // (without offsets the one expert)
    const int mine = args.offsets ? seg.first[threadIdx.x + 1] - seg.first[threadIdx.x] : 0;
    int ahead = 0;
    if (args.offsets) {
      int begin = 0;
      for (int f = 0; f < args.E; ++f) {
        const int end = seg.first[f + 1], blocks = end - begin;
        ahead += (blocks > mine || (blocks == mine && f < (int)threadIdx.x)) ? 1 : 0;
        begin = end;
      }
    }
    order[ahead] = (uint8_t)threadIdx.x;
  }
  const int step = WGRAD ? 2 * gridDim.x - 1 - 2 * blockIdx.x : gridDim.x;
  auto next_step = [&](int d) { return WGRAD ? 2 * (int)gridDim.x - d : d; };

  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)tmem_holder);
  const uint32_t stage0 = smem_u32(smem);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::COPY_REGS));
    if (warp == 0) {
      // ---------------- copies ----------------
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0;                         // bit s: stage s has been filled
      uint32_t parity = 0;                         // bit s: in which phase last
      bool ok = true;
      for (int t = blockIdx.x, d = step; t < num_tiles && ok; t += d, d = next_step(d)) {
        const Tile ti = tile_of<BN, WGRAD>(args, seg, order, t, n_tiles);
        for (int b = ti.b0; b < ti.b1; ++b) {
          if (elect_one()) {
            ok = ok && mbar_wait(empty_bar(stage), phase ^ 1u, &abort_s, args.err, 1);
            if (ok) {
              const uint32_t fb = full_bar(stage), sa = stage0 + stage * S::STAGE;
              mbar_arrive_expect_tx(fb, S::STAGE);
              tma_load_2d(sa, &tmA, b << 7, ti.m0, fb);
              if (WGRAD)
                tma_load_2d(sa + S::A_BYTES, &tmB, b << 7, ti.n0, fb);
              else
                tma_load_3d(sa + S::A_BYTES, &tmB, b << 7, ti.n0, ti.e, fb);
              issued |= 1u << stage;
              parity = (parity & ~(1u << stage)) | (phase << stage);
            }
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      for (int s = 0; s < STAGES && ok; ++s) {     // every stage has been released
        if (elect_one()) ok = mbar_wait(empty_bar(stage), phase ^ 1u, &abort_s, args.err, 2);
        ok = __all_sync(0xffffffffu, ok);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (abort_s) {                               // let the copies in flight land
        for (int s = 0; s < STAGES; ++s)
          if ((issued >> s) & 1u) gemm::mbar_wait_drain(full_bar(s), (parity >> s) & 1u);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA: a block of 128 a time ----------------
      // (the whole warp walks the loop, so that its values are uniform; one lane issues)
      {
        const uint64_t a0 = smem_desc_sw128(stage0, 16, 1024);
        const uint64_t b0 = smem_desc_sw128(stage0 + S::A_BYTES, 16, 1024);
        constexpr uint32_t IDESC = idesc_f8(128, BN);
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x, d = step; t < num_tiles && ok; t += d, d = next_step(d)) {
          const Tile ti = tile_of<BN, WGRAD>(args, seg, order, t, n_tiles);
          for (int b = ti.b0; b < ti.b1; ++b) {
            ok = ok && mbar_wait(tempty_bar(buf), buf_phase ^ 1u, &abort_s, args.err, 3) &&
                 mbar_wait(full_bar(stage), phase, &abort_s, args.err, 4);
            __syncwarp();
            if (elect_one()) {
              if (ok) {
                tc_fence_after();
                const uint64_t off = (uint64_t)((uint32_t)(stage * S::STAGE) >> 4);
  #pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_f8(tmem_base + (uint32_t)(buf * BN), a0 + off + 2 * k, b0 + off + 2 * k,
                          IDESC, k != 0);
                umma_commit(empty_bar(stage));
                umma_commit(tfull_bar(buf));
              }
            }
            __syncwarp();
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            if (++buf == NBUF) {
              buf = 0;
              buf_phase ^= 1u;
            }
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        if (abort_s && elect_one()) {
          umma_commit(drain_bar);                  // every MMA issued so far has completed
          gemm::mbar_wait_drain(drain_bar, 0);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- scales of a block, as far ahead as there are slots ----------------
      const int nb_all = (args.N + 127) >> 7, k_blocks = (args.K + 127) >> 7;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x, d = step; t < num_tiles && ok; t += d, d = next_step(d)) {
        const Tile ti = tile_of<BN, WGRAD>(args, seg, order, t, n_tiles);
        const float* const pb =
            WGRAD ? args.sb + ti.n0
                  : args.sb + ((long long)ti.e * nb_all + (ti.n0 >> 7)) * k_blocks;
        for (int g = ti.b0; g < ti.b1; g += S::GROUP) {
          if (lane == 0) ok = mbar_wait(sempty_bar(slot), phase ^ 1u, &abort_s, args.err, 6);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const int end = min(g + S::GROUP, ti.b1);
          for (int b = g; b < end; ++b) {
            const uint32_t to = smem_u32(slots) + slot * S::SLOT + (b - g) * S::BLOCK;
            const float* const pa = args.sa + b * args.ld_sa + ti.m0;
  #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 32 * i + lane;
              const bool there = ti.m0 + r < ti.m1;
              copy4(to + 4 * r, pa + (there ? r : 0), there);
            }
            if (WGRAD) {
  #pragma unroll
              for (int i = 0; i < BN / 32; ++i) {
                const int c = 32 * i + lane;
                const bool there = ti.n0 + c < args.K;
                copy4(to + 512 + 4 * c, pb + b * args.ld_sb + (there ? c : 0), there);
              }
            } else if (lane < BN / 128) {
              const bool there = (ti.n0 >> 7) + lane < nb_all;
              copy4(to + 512 + 4 * lane, pb + b + (there ? lane * k_blocks : 0), there);
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sfull_bar(slot))
                       : "memory");
          if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SUM_REGS));
    // ---------------- sums ----------------
    const int quarter = warp & 3, group = (warp - 4) >> 2;   // of the rows, of the columns
    const uint32_t lane_base =
        tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(group * WIDE);
    Reader rd = {slots, sfull_bar(0), sempty_bar(0), tfull_bar(0), tempty_bar(0), 0, 0, 0u, 0u,
                 true, &abort_s, args.err};
    for (int t = blockIdx.x, d = step; t < num_tiles; t += d, d = next_step(d)) {
      const Tile ti = tile_of<BN, WGRAD>(args, seg, order, t, n_tiles);
      if constexpr (WGRAD)
        sum_weights<BN>(args, ti, rd, lane_base, quarter, group, lane,
                        smem_u32(turn_all) + (uint32_t)(warp - 4) * 4096u, &tmC);
      else
        sum_rows<BN>(args, ti, rd, lane_base, quarter, group, lane,
                     turn_all + (warp - 4) * 32 * 80);
      // after a wait that gave up nothing waits any more, and the tile's end leaves
      rd.ok = __all_sync(0xffffffffu, rd.ok);
      if (!rd.ok) break;
    }
    if (WGRAD && lane == 0) bulk_wait_all();     // the last copies out
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Weight gradient on no columns: 0 (nothing is added), unless some expert has rows.
__global__ void __launch_bounds__(256) k_fp8_no_rows(float* dw, long long n, int accumulate,
                                                     const int32_t* offsets, int E,
                                                     DevError* err) {
  pdl_wait();
  const int t = threadIdx.x;
  if (__syncthreads_or(offsets && t < E && (offsets[t] < 0 || offsets[t + 1] != offsets[t]))) {
    if (blockIdx.x == 0 && t == 0) record_error(err, MOE_ERR_INVALID_ARG, 0);
    return;
  }
  if (!accumulate)
    for (long long i = (long long)blockIdx.x * 256 + t; i < n; i += (long long)gridDim.x * 256)
      dw[i] = 0.f;
  pdl_trigger();
}

template <int BN, bool WGRAD>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                   const Fp8GemmArgs& a, int grid, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e =
      smem_optin_once(k_fp8_gemm<BN, WGRAD>, (Shape<BN, WGRAD>::SMEM), configured);
  if (e != cudaSuccess) return e;
  // the shares above are of what a thread is launched with
  static std::atomic<int> regs{0};
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t q = cudaFuncGetAttributes(&at, k_fp8_gemm<BN, WGRAD>);
    if (q != cudaSuccess) return q;
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != Shape<BN, WGRAD>::LAUNCH_REGS)
    return cudaErrorInvalidConfiguration;
  return launch_pdl(k_fp8_gemm<BN, WGRAD>, dim3(grid), dim3(Shape<BN, WGRAD>::THREADS),
                    (Shape<BN, WGRAD>::SMEM), st, ta, tb, tc, a);
}

bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

bool desc_ok(const moe_fp8_gemm_desc* s) {
  return s && s->N >= 1 && s->N <= MOE_FP8_MAX_WIDTH && s->K >= 1 && s->K <= MOE_FP8_MAX_WIDTH &&
         s->E >= 1 && s->E <= kMaxSegments &&
         (s->out_dtype == MOE_DTYPE_BF16 || s->out_dtype == MOE_DTYPE_FP32);
}

bool codes_ok(const void* p, long long ld, long long width) {
  return p && aligned(p, 16) && ld >= width && ld % 16 == 0 && ld < (1LL << 39);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_gemm(const moe_fp8_gemm_desc* s, int M, const uint8_t* a, long long ld_a,
                            const float* a_scales, long long ld_as, const uint8_t* b,
                            long long ld_b, const float* b_scales, const int32_t* offsets, void* c,
                            long long ld_c, void* status, void* stream) {
  if (!desc_ok(s) || M < 0 || M > 0x7FFFFF80 ||  // (rounded up to blocks: an int)
      (s->E > 1 && !offsets) || !status || !aligned(status, 16))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const int es = s->out_dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!codes_ok(a, ld_a, s->K) || !codes_ok(b, ld_b, s->K) || !a_scales || !b_scales || !c ||
      ld_as < M || ld_c < s->N || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(c, es) || !aligned(offsets, 4) || ld_b >= (1LL << 39) / s->N)
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Few rows, and so few weights that 16 rows of them a CTA are one wave of the streaming
  // kernel (two CTAs an SM; every eight rows of A count, for they take the weights again): M = 1,
  // N = K = 4096 6.9 us against 10.1 on tiles, N = 300, K = 500 2.0 against 4.2.  Beyond a wave
  // neither is always ahead.  In units of 16 rows: 384 of one row each on four experts (K =
  // 4096) 10.4 against 15.5, eight rows on 448 13.6 against 12.3, 32 rows on 320 12.4 against
  // 11.5, one token's eight experts on 768 (K = 2048) 11.5 against 10.0.
  if (M <= 32 && (long long)(M < s->E ? M : s->E) * ((s->N + 15) / 16) * ((M + 7) / 8) <=
                     2 * num_sms()) {
    const Fp8FewCall f = {M, s->N, s->K, s->E, a, ld_a, a_scales, ld_as, b, ld_b, b_scales,
                          offsets, c, ld_c, es == 4, static_cast<DevError*>(status)};
    return cuda_result(launch_fp8_few(f, st), "moe_fp8_gemm");
  }
  Fp8GemmArgs g = {};
  g.M = M; g.N = s->N; g.K = s->K; g.E = s->E;
  g.sa = a_scales; g.ld_sa = ld_as; g.sb = b_scales;
  g.offsets = offsets; g.c = c; g.ld_c = ld_c;
  g.f32 = es == 4;
  g.wide = aligned(c, 16) && ld_c * es % 16 == 0;
  g.err = static_cast<DevError*>(status);
  // 128 columns a tile, and four parts of tensor memory, where 256 leave SMs without a tile
  // (experts count with half a tile each beside their rows).  One wave of M = 1003, N = 1537,
  // K = 2047: 10.0 us against 15.4, M = 16, N = K = 4096 10.2 against 13.9; many waves (M =
  // 65536, N = 1536, K = 2048 on 128 experts) 253 against 205.  A few rows on experts wait for
  // the weights either way, in more and smaller copies with 128 (one token's eight experts
  // 11.6 against 10.3).
  const long long rows = (M + 127) / 128 + (offsets ? (M < s->E ? M : s->E) / 2 : 0);
  const bool narrow = s->N <= 128 || ((!offsets || M >= 128) &&
                                      rows * ((s->N + 255) / 256) <= num_sms());
  const long long n_tiles = (s->N + (narrow ? 127 : 255)) / (narrow ? 128 : 256);
  const long long most = ((M + 127LL * (offsets ? s->E : 1)) / 128) * n_tiles;
  if (most > (1LL << 30)) return MOE_ERR_INVALID_ARG;
  CUtensorMap ta, tb;
  if (encode_tmap_codes(&ta, a, 0, M, s->K, ld_a, 128) != MOE_OK ||
      encode_tmap_codes(&tb, b, s->E, s->N, s->K, ld_b, narrow ? 128 : 256) != MOE_OK)
    return MOE_ERR_CUDA;
  const int grid = (int)(most < num_sms() ? most : num_sms());
  return cuda_result(narrow ? launch<128, false>(ta, tb, ta, g, grid, st)
                            : launch<256, false>(ta, tb, ta, g, grid, st), "moe_fp8_gemm");
}

extern "C" int moe_fp8_gemm_wgrad(const moe_fp8_gemm_desc* s, long long R, const uint8_t* dyt,
                                  long long ld_dyt, const float* dyt_scales, long long ld_dys,
                                  const uint8_t* xt, long long ld_xt, const float* xt_scales,
                                  long long ld_xs, const int32_t* offsets, float* dw,
                                  int accumulate, void* status, void* stream) {
  if (!desc_ok(s) || R < 0 || R % 128 || R > 0x7FFFFF80LL || (s->E > 1 && !offsets) || !dw ||
      !aligned(dw, 4) || !status || !aligned(status, 16))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (R == 0) {
    if (!aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
    if (!offsets && accumulate) return MOE_OK;
    const long long all = (long long)s->E * s->N * s->K, ctas = (all + 1023) / 1024;
    const int most = 8 * num_sms();
    return cuda_result(launch_pdl(k_fp8_no_rows, dim3((unsigned)(ctas < most ? ctas : most)),
                                  dim3(256), 0, st, dw, all, accumulate != 0, offsets, s->E,
                                  static_cast<DevError*>(status)), "moe_fp8_gemm_wgrad");
  }
  if (!codes_ok(dyt, ld_dyt, R) || !codes_ok(xt, ld_xt, R) || !dyt_scales || !xt_scales ||
      ld_dys < s->N || ld_xs < s->K || !aligned(dyt_scales, 4) || !aligned(xt_scales, 4) ||
      !aligned(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  Fp8GemmArgs g = {};
  g.N = s->N; g.K = s->K; g.E = s->E;
  g.sa = dyt_scales; g.ld_sa = ld_dys; g.sb = xt_scales; g.ld_sb = ld_xs;
  g.offsets = offsets; g.c = dw; g.ld_c = s->K;
  g.row_blocks = (int)(R / 128);
  g.f32 = 1;
  g.accumulate = accumulate != 0;
  g.wide = aligned(dw, 16) && s->K % 4 == 0 && (long long)s->N * s->K < (1LL << 37)
               ? 4
               : aligned(dw, 8) && s->K % 2 == 0 ? 2 : 0;
  g.err = static_cast<DevError*>(status);
  // as in moe_fp8_gemm: N = 777, K = 1111 over 1003 rows 10.1 us against 15.4
  const bool narrow = s->K <= 128 || (long long)s->E * ((s->N + 127) / 128) *
                                         ((s->K + 255) / 256) <= num_sms();
  const long long tiles = (long long)s->E * ((s->N + 127) / 128) *
                          ((s->K + (narrow ? 127 : 255)) / (narrow ? 128 : 256));
  if (tiles > (1LL << 30)) return MOE_ERR_INVALID_ARG;
  CUtensorMap ta, tb;
  if (encode_tmap_codes(&ta, dyt, 0, s->N, R, ld_dyt, 128) != MOE_OK ||
      encode_tmap_codes(&tb, xt, 0, s->K, R, ld_xt, narrow ? 128 : 256) != MOE_OK)
    return MOE_ERR_CUDA;
  CUtensorMap tc = ta;                           // (read where rows are aligned)
  if (g.wide == 4 && encode_tmap_f32_weights(&tc, dw, s->E, s->N, s->K) != MOE_OK)
    return MOE_ERR_CUDA;
  const int grid = (int)(tiles < num_sms() ? tiles : num_sms());
  return cuda_result(narrow ? launch<128, true>(ta, tb, tc, g, grid, st)
                            : launch<256, true>(ta, tb, tc, g, grid, st), "moe_fp8_gemm_wgrad");
}

extern "C" int moe_fp8_check(void* status, int* where) {
  if (!status) return MOE_ERR_INVALID_ARG;
  DevError e;
  cudaError_t rc = cudaDeviceSynchronize();
  if (rc == cudaSuccess) rc = cudaMemcpy(&e, status, sizeof e, cudaMemcpyDeviceToHost);
  if (rc == cudaSuccess && e.code) rc = cudaMemset(status, 0, sizeof e);
  if (rc != cudaSuccess) return cuda_result(rc, "moe_fp8_check");
  if (where) *where = e.where;
  return e.code;
}
