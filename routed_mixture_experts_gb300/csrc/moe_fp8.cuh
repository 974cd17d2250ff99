// moe_fp8.cuh -- what the 8-bit block quantiser and products share: the experts'
// segments of rows, read from offsets on the device.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMaxSegments = 256;

// Segments of rows [begin[e], end[e]) and their blocks of 128 rows: block b of all
// belongs to the segment with first[e] <= b < first[e + 1].  Where offsets decrease or
// leave 0..M, `bad` is set and every segment is empty.
struct Segments {
  int begin[kMaxSegments], end[kMaxSegments];
  int first[kMaxSegments + 1];
  int sums[8];
  int bad;

  // All of the CTA's THREADS (256 at least) call it; ends with a barrier.
  template <int THREADS>
  __device__ __forceinline__ void init(const int32_t* offsets, int E, int M) {
    static_assert(THREADS >= kMaxSegments, "a thread a segment");
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int lo = 0, hi = 0;
    if (t < E) {
      lo = offsets[t];
      hi = offsets[t + 1];
    }
    bad = __syncthreads_or(lo < 0 || hi < lo || hi > M);
    int blocks = 0;
    if (t < kMaxSegments) {
      if (bad) hi = lo = 0;
      if (t < E) {
        begin[t] = lo;
        end[t] = hi;
      }
      blocks = (int)(((unsigned)(hi - lo) + 127u) >> 7);
      int incl = blocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sums[warp] = incl;
      blocks = incl - blocks;
    }
    __syncthreads();
    if (t < E) {
      for (int w = 0; w < warp; ++w) blocks += sums[w];
      first[t] = blocks;
      if (t == E - 1) first[E] = blocks + ((int)(((unsigned)(hi - lo) + 127u) >> 7));
    }
    __syncthreads();
  }

  // The segment of block b (b < first[E]).
  __device__ __forceinline__ int find(int b, int E) const {
    int lo = 0, hi = E;                // first[lo] <= b < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= b) lo = mid; else hi = mid;
    }
    return lo;
  }
};

}  // namespace moe
