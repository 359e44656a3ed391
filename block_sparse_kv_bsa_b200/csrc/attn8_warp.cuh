// attn8_warp.cuh - one warp's attention of 16 query rows over keys of the
// 8-bit cache, on mma.sync m16n8k16 (f16 in, fp32 out), K and V from tiles in
// shared memory in TMA's swizzle (16-byte chunk c of row r at chunk c ^ (r % 8)
// of 128-byte rows, c ^ (r / 2 % 4) of 64-byte rows).
//
// Fragment maps (g = lane / 4, t = lane % 4), chosen so that every lane's
// loads are whole 16-byte (V at D = 64: 8-byte) pieces and eight lanes never
// meet in a bank:
//   Q K^T  the k index of step ks is d = (ks / 4) * 64 + t * 16 + (ks % 4) * 4
//          + {0, 1 | 2, 3}: a lane holds 16 consecutive d of key g a load.
//   P V    the n index of tile nt is d = g * (D / 8) + nt: a lane holds D / 8
//          consecutive d of the keys 2t, 2t + 1, 2t + 8, 2t + 9; the bytes of
//          two keys are interleaved before they become f16 pairs.
//
// Scales: with key scale a and value scale v of a block,
//   x = s * (sm_scale * log2 e * a * row scale) + log2 v
// is the exponent of v * softmax weight: the weights p = 2^(x - m) carry v, the
// product with the codes needs no scaling, and the denominator takes
// sum(p) / v.  m is the row's reference, 7 below the running maximum of x when
// set and moved only when a weight would pass 2^15, so f16 weights keep
// 2^-24 / 2^7 of the largest as their smallest step.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "e4m3.cuh"

namespace bsa {

constexpr float kPBias = 7.f;    // log2 of a fresh row maximum's weight
constexpr float kPMaxLog2 = 15.f;  // a larger weight moves the reference

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Loads the compiler keeps in their place among the barrier operations.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}

// 2^e as a float, e within the normal range.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Power-of-two scale of a query row whose largest magnitude is amax: q / scale
// then has its largest magnitude in [2^13, 2^14), and everything down to
// 2^-28 of it is exact in f16.  A row that is zero, or holds an infinity or
// NaN, is not scaled.
__device__ __forceinline__ float q_row_scale(float amax) {
  if (!(amax > 0.f && amax <= 3.402823466e38f)) return 1.f;
  int e = (__float_as_int(amax) >> 23) - 127 - 13;  // subnormal amax: e = -140
  e = e < -126 ? -126 : e;
  return pow2i(e);
}

template <int D>
struct AttnWarp {
  static constexpr int kSteps = D / 16;   // k steps of Q K^T
  static constexpr int kTiles = D / 8;    // n tiles of P V
  static constexpr int kKLoads = D / 64;  // 16-byte pieces of a key per lane
  static constexpr int kVWords = D / 32;  // words of a value row per lane

  uint32_t q[kSteps][4];
  float row_scale[2];  // query row scale * sm_scale * log2 e, rows g and g + 8
  float o[kTiles][4];
  float m[2], l[2];

  static __device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }

  struct Keys {  // 16 keys
    uint4 k[2][kKLoads];         // key g of each half
    uint32_t v[4][kVWords];      // keys 2t, 2t + 1, 2t + 8, 2t + 9
  };

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
      o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // Query rows r0 = g and r1 = g + 8 (null: a row of zeros).
  __device__ __forceinline__ void load_q(const __nv_bfloat16* r0, const __nv_bfloat16* r1,
                                         float scale_log2) {
    const int t = threadIdx.x % 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const __nv_bfloat16* r = half ? r1 : r0;
      uint4 raw[kKLoads][2];
      float amax = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          raw[i][w] = r == nullptr ? make_uint4(0, 0, 0, 0)
                                   : ld_nc_v4(r + i * 64 + t * 16 + w * 8);
          const uint32_t u[4] = {raw[i][w].x, raw[i][w].y, raw[i][w].z, raw[i][w].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = fabsf(bf16lo(u[e])), b = fabsf(bf16hi(u[e]));
            amax = fmaxf(amax, fmaxf(a, b));
            bad |= !(a <= 3.402823466e38f) | !(b <= 3.402823466e38f);
          }
        }
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        bad |= __shfl_xor_sync(0xffffffffu, static_cast<int>(bad), off) != 0;
      }
      const float qs = bad ? 1.f : q_row_scale(amax);
      const float inv = 1.f / qs;  // exact: a power of two
      row_scale[half] = scale_log2 * qs;
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) {
        const uint32_t u[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                               raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          q[i * 4 + w][half] = pack_f16x2(bf16lo(u[2 * w]) * inv, bf16hi(u[2 * w]) * inv);
          q[i * 4 + w][half + 2] =
              pack_f16x2(bf16lo(u[2 * w + 1]) * inv, bf16hi(u[2 * w + 1]) * inv);
        }
      }
    }
  }

  // Keys [first, first + 16) of the tiles at shared addresses kt and vt; values
  // at or past `valid` read as zero (their weights are zero, but a NaN code
  // would survive that).
  __device__ __forceinline__ void load_keys(uint32_t kt, uint32_t vt, int first, int valid,
                                            Keys& x) const {
    if (first >= valid) {
      x = Keys{};
      return;
    }
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int key = first + n * 8 + g;
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) x.k[n][i] = lds128(kt + chunk_at(key, i * 4 + t));
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int key = first + (n / 2) * 8 + 2 * t + (n & 1);
      if (D == 128) {
        const uint4 u = lds128(vt + chunk_at(key, g));
        x.v[n][0] = u.x;
        x.v[n][1] = u.y;
        x.v[n][kVWords - 2] = u.z;
        x.v[n][kVWords - 1] = u.w;
      } else {
        const uint2 u = lds64(vt + chunk_at(key, g >> 1) + (g & 1) * 8);
        x.v[n][0] = u.x;
        x.v[n][1] = u.y;
      }
    }
    if (first + 16 > valid) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (first + (n / 2) * 8 + 2 * t + (n & 1) >= valid) {
#pragma unroll
          for (int w = 0; w < kVWords; ++w) x.v[n][w] = 0;
        }
      }
    }
  }

  // One step: keys [first, first + 16) of G blocks at once (their products and
  // exponentials are independent, one maximum and one rescale serve all).
  // meta[b] = (key scale, log2 v, 1 / v, valid rows as int) of block b; a block
  // with no valid key in the step must hold zeros in x[b].
  template <int G>
  __device__ __forceinline__ void step(const Keys (&x)[G], int first, const uint4 (&meta)[G]) {
    const int t = threadIdx.x % 4;
    float s[2 * G][4];
#pragma unroll
    for (int n = 0; n < 2 * G; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kKLoads; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int n = 0; n < 2 * G; ++n) {
          const uint4& k = x[n / 2].k[n & 1][i];
          const uint32_t w = e == 0 ? k.x : (e == 1 ? k.y : (e == 2 ? k.z : k.w));
          mma_f16(s[n], q[i * 4 + e], e4m3_lo_f16x2(w), e4m3_hi_f16x2(w));
        }
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2 * G; ++n) {
      const float ks = __uint_as_float(meta[n / 2].x), vlog2 = __uint_as_float(meta[n / 2].y);
      const int valid = static_cast<int>(meta[n / 2].w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e / 2;
        const int key = first + (n & 1) * 8 + 2 * t + (e & 1);
        s[n][e] = key < valid ? fmaf(s[n][e], row_scale[r] * ks, vlog2) : -INFINITY;
        mx[r] = fmaxf(mx[r], s[n][e]);
      }
    }
    bool move = false;
    float fix[2] = {1.f, 1.f}, ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      if (mx[r] > m[r] + kPMaxLog2) {
        const float next = mx[r] - kPBias;
        fix[r] = ex2_approx(m[r] - next);
        m[r] = next;
        l[r] *= fix[r];
        move = true;
      }
      ref[r] = m[r] == -INFINITY ? 0.f : m[r];
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        o[i][0] *= fix[0];
        o[i][1] *= fix[0];
        o[i][2] *= fix[1];
        o[i][3] *= fix[1];
      }
    }
#pragma unroll
    for (int b = 0; b < G; ++b) {
      uint32_t p[4];
      const float vinv = __uint_as_float(meta[b].z);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float e0 = ex2_approx(s[2 * b + n][2 * r] - ref[r]);
          const float e1 = ex2_approx(s[2 * b + n][2 * r + 1] - ref[r]);
          sum += e0 + e1;
          p[n * 2 + r] = pack_f16x2(e0, e1);
        }
        l[r] = fmaf(sum, vinv, l[r]);
      }
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        const uint32_t a0 = __byte_perm(x[b].v[0][w], x[b].v[1][w], 0x5140);
        const uint32_t a1 = __byte_perm(x[b].v[0][w], x[b].v[1][w], 0x7362);
        const uint32_t b0 = __byte_perm(x[b].v[2][w], x[b].v[3][w], 0x5140);
        const uint32_t b1 = __byte_perm(x[b].v[2][w], x[b].v[3][w], 0x7362);
        mma_f16(o[4 * w + 0], p, e4m3_lo_f16x2(a0), e4m3_lo_f16x2(b0));
        mma_f16(o[4 * w + 1], p, e4m3_hi_f16x2(a0), e4m3_hi_f16x2(b0));
        mma_f16(o[4 * w + 2], p, e4m3_lo_f16x2(a1), e4m3_lo_f16x2(b1));
        mma_f16(o[4 * w + 3], p, e4m3_hi_f16x2(a1), e4m3_hi_f16x2(b1));
      }
    }
  }

  // Sums over the four lanes of a row.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
  }
};

}  // namespace bsa
