// attn8_warp.cuh - one warp's attention of 16 or 8 query rows over keys of the
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
// Up to 8 rows take the transposed products (S^T = K Q^T, O^T = V^T P^T, the
// rows on the 8-wide side): the same loads and conversions, half the matrix
// instructions and half the registers of O and Q.
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

// The transpose of an 8 x 8 matrix of 16-bit elements, two of row lane / 4 a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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
// 2^-28 of it is exact in f16.  A zero row is not scaled.
__device__ __forceinline__ float q_row_scale(float amax) {
  if (!(amax > 0.f)) return 1.f;
  int e = (__float_as_int(amax) >> 23) - 127 - 13;  // subnormal amax: e = -140
  e = e < -126 ? -126 : e;
  return pow2i(e);
}

// 16 keys of a block as a lane holds them, for both forms.
template <int D>
struct KeyTile {
  static constexpr int kKLoads = D / 64;  // 16-byte pieces of a key per lane
  static constexpr int kVWords = D / 32;  // words of a value row per lane

  struct Keys {
    uint4 k[2][kKLoads];     // key g of each half
    uint32_t v[4][kVWords];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
  };

  static __device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }

  // Keys [first, first + 16) of the tiles at shared addresses kt and vt; values
  // at or past `valid` read as zero (their weights are zero, but a NaN code
  // would survive that).
  static __device__ __forceinline__ void load_keys(uint32_t kt, uint32_t vt, int first, int valid,
                                                   Keys& x) {
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

  // Word w of the values of keys (2t, 2t + 1) and (2t + 8, 2t + 9) as f16 pairs:
  // lo[e], hi[e] for the word's element e.
  static __device__ __forceinline__ void value_pairs(const Keys& x, int w, uint32_t (&lo)[4],
                                                     uint32_t (&hi)[4]) {
    const uint32_t a0 = __byte_perm(x.v[0][w], x.v[1][w], 0x5140);
    const uint32_t a1 = __byte_perm(x.v[0][w], x.v[1][w], 0x7362);
    const uint32_t b0 = __byte_perm(x.v[2][w], x.v[3][w], 0x5140);
    const uint32_t b1 = __byte_perm(x.v[2][w], x.v[3][w], 0x7362);
    lo[0] = e4m3_lo_f16x2(a0);
    lo[1] = e4m3_hi_f16x2(a0);
    lo[2] = e4m3_lo_f16x2(a1);
    lo[3] = e4m3_hi_f16x2(a1);
    hi[0] = e4m3_lo_f16x2(b0);
    hi[1] = e4m3_hi_f16x2(b0);
    hi[2] = e4m3_lo_f16x2(b1);
    hi[3] = e4m3_hi_f16x2(b1);
  }
};

// A lane's part of a query row r (null: zeros) as f16 pairs over the row's
// power-of-two scale, which is returned: lo[ks], hi[ks] are elements {0, 1} and
// {2, 3} of k step ks.  A row with an infinity or a NaN has no softmax: its scale,
// and through it all it leads to, is NaN.
template <int D>
__device__ __forceinline__ float load_query_row(const __nv_bfloat16* r, uint32_t (&lo)[D / 16],
                                                uint32_t (&hi)[D / 16]) {
  constexpr int kLoads = D / 64;
  const int t = threadIdx.x % 4;
  uint4 raw[kLoads][2];
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      raw[i][w] = r == nullptr ? make_uint4(0, 0, 0, 0) : ld_nc_v4(r + i * 64 + t * 16 + w * 8);
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
  const float qs = bad ? __int_as_float(0x7fffffff) : q_row_scale(amax);
  const float inv = 1.f / qs;  // exact: a power of two
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t u[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                           raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      lo[i * 4 + w] = pack_f16x2(bf16lo(u[2 * w]) * inv, bf16hi(u[2 * w]) * inv);
      hi[i * 4 + w] = pack_f16x2(bf16lo(u[2 * w + 1]) * inv, bf16hi(u[2 * w + 1]) * inv);
    }
  }
  return qs;
}

// Moves a row's reference when a weight would pass 2^kPMaxLog2; returns what O
// (and l, done here) must be multiplied by.
__device__ __forceinline__ float move_reference(float mx, float& m, float& l) {
  // The difference of near values is exact; m + 15 rounds to m + 16 from 2^24 on,
  // and a weight of 2^16 is no f16.
  if (!(mx - m > kPMaxLog2)) return 1.f;
  const float next = mx - kPBias;
  const float fix = ex2_approx(m - next);
  m = next;
  l *= fix;
  return fix;
}

// Element of a row at column c of what finish() writes.
template <int D>
__device__ __forceinline__ int out_element(int c) {
  return (c & 7) * (D / 8) + (c >> 3);
}

// 16 query rows: lane (g, t) has rows g and g + 8.
template <int D>
struct AttnWarp16 {
  using Tile = KeyTile<D>;
  using Keys = typename Tile::Keys;
  static constexpr int kRows = 16;
  static constexpr int kSteps = D / 16;   // k steps of Q K^T
  static constexpr int kTiles = D / 8;    // n tiles of P V

  uint32_t q[kSteps][4];
  float row_scale[2];  // query row scale * sm_scale * log2 e
  float o[kTiles][4];
  float m[2], l[2];

  // row(r) is query row r of the tile, or null.
  template <class Row>
  __device__ __forceinline__ void init(Row row, float scale_log2) {
    const int g = threadIdx.x % 32 / 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t lo[kSteps], hi[kSteps];
      row_scale[half] = scale_log2 * load_query_row<D>(row(g + half * 8), lo, hi);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        q[k][half] = lo[k];
        q[k][half + 2] = hi[k];
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // One step: keys [first, first + 16) of a block.
  __device__ __forceinline__ void step(const Keys& x, int first, const uint4& meta) {
    const int t = threadIdx.x % 4;
    const float ks = __uint_as_float(meta.x), vlog2 = __uint_as_float(meta.y);
    const float vinv = __uint_as_float(meta.z);
    const int valid = static_cast<int>(meta.w);
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < Tile::kKLoads; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint4& k = x.k[n][i];
          const uint32_t w = e == 0 ? k.x : (e == 1 ? k.y : (e == 2 ? k.z : k.w));
          mma_f16(s[n], q[i * 4 + e], e4m3_lo_f16x2(w), e4m3_hi_f16x2(w));
        }
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e / 2, key = first + n * 8 + 2 * t + (e & 1);
        s[n][e] = key < valid ? fmaf(s[n][e], row_scale[r] * ks, vlog2) : -INFINITY;
        mx[r] = fmaxf(mx[r], s[n][e]);
      }
    }
    float fix[2], ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      fix[r] = move_reference(mx[r], m[r], l[r]);
      ref[r] = m[r] == -INFINITY ? 0.f : m[r];
    }
    if (__any_sync(0xffffffffu, fix[0] != 1.f || fix[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        o[i][0] *= fix[0];
        o[i][1] *= fix[0];
        o[i][2] *= fix[1];
        o[i][3] *= fix[1];
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float e0 = ex2_approx(s[n][2 * r] - ref[r]);
        const float e1 = ex2_approx(s[n][2 * r + 1] - ref[r]);
        sum += e0 + e1;
        p[n * 2 + r] = pack_f16x2(e0, e1);
      }
      l[r] = fmaf(sum, vinv, l[r]);
    }
#pragma unroll
    for (int w = 0; w < Tile::kVWords; ++w) {
      uint32_t lo[4], hi[4];
      Tile::value_pairs(x, w, lo, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) mma_f16(o[4 * w + e], p, lo[e], hi[e]);
    }
  }

  // Sums over the lanes of a row; O [16][kStride] and (m, l) [16][2] to shared
  // memory.  Element d = n * (D / 8) + i of a row goes to column i * 8 + n
  // (out_element is the way back), and rows are kStride apart: lanes then write
  // different banks, where d as it is would put all 32 into one.
  static constexpr int kStride = D + 8;
  __device__ __forceinline__ void finish(float* s_o, float* s_ml) {
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = g + 8 * r;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        *reinterpret_cast<float2*>(s_o + row * kStride + i * 8 + 2 * t) =
            make_float2(o[i][2 * r], o[i][2 * r + 1]);
      }
      if (t == 0) {
        s_ml[row * 2] = m[r];
        s_ml[row * 2 + 1] = l[r];
      }
    }
  }
};

// 8 query rows: lane (g, t) has rows 2t and 2t + 1, of keys g and g + 8 and of
// elements g * (D / 8) ...
template <int D>
struct AttnWarp8 {
  using Tile = KeyTile<D>;
  using Keys = typename Tile::Keys;
  static constexpr int kRows = 8;
  static constexpr int kSteps = D / 16;
  static constexpr int kTiles = D / 16;  // m tiles of V^T P^T: two elements a lane each

  uint32_t q[kSteps][2];
  float row_scale[2];
  float o[kTiles][4];
  float m[2], l[2];

  template <class Row>
  __device__ __forceinline__ void init(Row row, float scale_log2) {
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    uint32_t lo[kSteps], hi[kSteps];
    const float qs = scale_log2 * load_query_row<D>(row(g), lo, hi);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      q[k][0] = lo[k];
      q[k][1] = hi[k];
    }
    row_scale[0] = __shfl_sync(0xffffffffu, qs, 8 * t);  // lane (2t, 0)
    row_scale[1] = __shfl_sync(0xffffffffu, qs, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  __device__ __forceinline__ void step(const Keys& x, int first, const uint4& meta) {
    const int g = threadIdx.x % 32 / 4;
    const float ks = __uint_as_float(meta.x), vlog2 = __uint_as_float(meta.y);
    const float vinv = __uint_as_float(meta.z);
    const int valid = static_cast<int>(meta.w);
    float s2[2][4];  // two chains
#pragma unroll
    for (int n = 0; n < 2; ++n) s2[n][0] = s2[n][1] = s2[n][2] = s2[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < Tile::kKLoads; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 &k0 = x.k[0][i], &k1 = x.k[1][i];
        const uint32_t w0 = e == 0 ? k0.x : (e == 1 ? k0.y : (e == 2 ? k0.z : k0.w));
        const uint32_t w1 = e == 0 ? k1.x : (e == 1 ? k1.y : (e == 2 ? k1.z : k1.w));
        const uint32_t a[4] = {e4m3_lo_f16x2(w0), e4m3_lo_f16x2(w1), e4m3_hi_f16x2(w0),
                               e4m3_hi_f16x2(w1)};
        mma_f16(s2[e & 1], a, q[i * 4 + e][0], q[i * 4 + e][1]);
      }
    }
    float s[4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e & 1, key = first + g + (e / 2) * 8;
      s[e] = key < valid ? fmaf(s2[0][e] + s2[1][e], row_scale[r] * ks, vlog2) : -INFINITY;
      mx[r] = fmaxf(mx[r], s[e]);
    }
    float fix[2], ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], off));
      fix[r] = move_reference(mx[r], m[r], l[r]);
      ref[r] = m[r] == -INFINITY ? 0.f : m[r];
    }
    if (__any_sync(0xffffffffu, fix[0] != 1.f || fix[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        o[i][0] *= fix[0];
        o[i][1] *= fix[1];
        o[i][2] *= fix[0];
        o[i][3] *= fix[1];
      }
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[e] - ref[e & 1]);
    l[0] = fmaf(p[0] + p[2], vinv, l[0]);
    l[1] = fmaf(p[1] + p[3], vinv, l[1]);
    // (key g, rows 2t, 2t + 1) to (keys 2t, 2t + 1, row g).
    const uint32_t b0 = transpose8x8(pack_f16x2(p[0], p[1]));
    const uint32_t b1 = transpose8x8(pack_f16x2(p[2], p[3]));
#pragma unroll
    for (int w = 0; w < Tile::kVWords; ++w) {
      uint32_t lo[4], hi[4];
      Tile::value_pairs(x, w, lo, hi);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t a[4] = {lo[e], lo[e + 1], hi[e], hi[e + 1]};
        mma_f16(o[2 * w + e / 2], a, b0, b1);
      }
    }
  }

  static constexpr int kStride = D + 4;
  __device__ __forceinline__ void finish(float* s_o, float* s_ml) {
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
      const int row = 2 * t + r;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        s_o[row * kStride + 16 * i + g] = o[i][r];
        s_o[row * kStride + 16 * i + 8 + g] = o[i][2 + r];
      }
      if (g == 0) {
        s_ml[row * 2] = m[r];
        s_ml[row * 2 + 1] = l[r];
      }
    }
  }
};

}  // namespace bsa
