// slots.cuh - which raster token sits in each slot of a 128-token block.
//
// Shared by the kernels that gather a chunk's tokens into blocks (append,
// query reordering, their rotated and 8-bit forms).
#pragma once

#include "common.cuh"
#include "gilbert.cuh"

namespace bsa {

// Chunks up to this size invert a permutation table per block (a scan).
constexpr int kGatherMaxTokens = 1 << 14;

// The curve walk kept out of line: the kernels' table path stays compact.
static __device__ __noinline__ int curve_token_call(int T, int H, int W, int p) {
  return curve_token(T, H, W, p);
}

// Slot -> token for the 128 curve slots [slot0, slot0 + 128) of one block:
// s_tok[d] is the raster token whose perm entry is slot0 + d, or -1 for a pad
// slot.  With a table, the CTA's NT threads (NT >= 128) scan perm in rounds of
// kScan independent loads per thread (one L2 round trip per round); entries
// outside [0, N) are skipped, and reported when `report_bad`.  Without one
// (perm == NULL), each thread locates its slot on the curve.  Ends with a CTA
// barrier.
template <int NT>
__device__ __forceinline__ void invert_block_slots(const int32_t* perm, int N, int slot0,
                                                   int* s_tok, bool report_bad, int32_t* d_err,
                                                   int T, int H, int W) {
  static_assert(NT >= kBlk, "one thread per slot clears the table");
  if (perm == nullptr) {
    if (threadIdx.x < kBlk) {
      const int p = slot0 + static_cast<int>(threadIdx.x);
      s_tok[threadIdx.x] = p < N ? curve_token_call(T, H, W, p) : -1;
    }
    __syncthreads();
    return;
  }
  if (threadIdx.x < kBlk) s_tok[threadIdx.x] = -1;
  __syncthreads();
  auto take = [&](int r, int p) {
    if (p < 0 || p >= N) {
      if (report_bad) report(d_err, BSA_DEV_BAD_PERM);
      return;
    }
    const unsigned d = static_cast<unsigned>(p - slot0);
    if (d < static_cast<unsigned>(kBlk)) s_tok[d] = r;
  };
  constexpr int kScan = 16;
  // Four entries per load when perm is 16-byte aligned: one round of loads
  // covers 64 * NT tokens, so a chunk's scan costs one memory latency.
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(perm) & 15u) == 0) {
    const int n4 = N / 4;
    const int4* perm4 = reinterpret_cast<const int4*>(perm);
    for (int base = 0; base < n4; base += kScan * NT) {
      int4 pv[kScan];
#pragma unroll
      for (int k = 0; k < kScan; ++k) {
        const int i = base + threadIdx.x + k * NT;
        pv[k] = i < n4 ? __ldg(perm4 + i) : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kScan; ++k) {
        const int i = base + threadIdx.x + k * NT;
        if (i >= n4) break;
        take(4 * i, pv[k].x);
        take(4 * i + 1, pv[k].y);
        take(4 * i + 2, pv[k].z);
        take(4 * i + 3, pv[k].w);
      }
    }
    done = 4 * n4;
  }
  for (int base = done; base < N; base += kScan * NT) {
    int pv[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k) {
      const int r = base + threadIdx.x + k * NT;
      pv[k] = r < N ? __ldg(perm + r) : 0;
    }
#pragma unroll
    for (int k = 0; k < kScan; ++k) {
      const int r = base + threadIdx.x + k * NT;
      if (r >= N) break;
      take(r, pv[k]);
    }
  }
  __syncthreads();
}

// The same for the kernels that turn tokens: CTAs of NT threads start with it
// alone on their SM, so it is kept short (per entry one subtraction, one
// comparison and a predicated store; entries outside [0, N) fall outside the
// block's `valid` slots, and only the CTA that reports looks at them).
template <int NT>
__device__ __forceinline__ void find_block_tokens(const int32_t* perm, int N, int slot0, int valid,
                                                  int* s_tok, bool report_bad, int32_t* d_err,
                                                  int T, int H, int W) {
  static_assert(NT >= kBlk, "one thread per slot clears the table");
  if (perm == nullptr || (reinterpret_cast<uintptr_t>(perm) & 15u) != 0) {
    invert_block_slots<NT>(perm, N, slot0, s_tok, report_bad, d_err, T, H, W);
    return;
  }
  if (threadIdx.x < kBlk) s_tok[threadIdx.x] = -1;
  __syncthreads();
  const int4* perm4 = reinterpret_cast<const int4*>(perm);
  auto take = [&](int r, int p) {
    const unsigned d = static_cast<unsigned>(p - slot0);
    if (d < static_cast<unsigned>(valid)) s_tok[d] = r;
  };
  const int n4 = N / 4;
  constexpr int kScan = 4;
  for (int base = threadIdx.x; base < n4; base += kScan * NT) {
    int4 pv[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k)
      pv[k] = base + k * NT < n4 ? __ldg(perm4 + base + k * NT) : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int k = 0; k < kScan; ++k) {
      const int r = 4 * (base + k * NT);
      take(r, pv[k].x);
      take(r + 1, pv[k].y);
      take(r + 2, pv[k].z);
      take(r + 3, pv[k].w);
    }
  }
  for (int r = 4 * n4 + threadIdx.x; r < N; r += NT) take(r, __ldg(perm + r));
  if (report_bad) {
    for (int r = threadIdx.x; r < N; r += NT)
      if (static_cast<unsigned>(__ldg(perm + r)) >= static_cast<unsigned>(N))
        report(d_err, BSA_DEV_BAD_PERM);
  }
  __syncthreads();
}

}  // namespace bsa
