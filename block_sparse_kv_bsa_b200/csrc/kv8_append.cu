// kv8_append.cu - bsa_kv8_append: a chunk into the 8-bit cache.
//
// Per (batch, head, block) and tensor: A = max |r| over the block (r = the
// turned key, or the value), scale = A / 448, code = e4m3(r * (448 / A)).  The
// bytes it cannot do without are 2 read and 1 written per element.  A CTA
// takes one block and a run of heads of one tensor; its 512 threads hold a
// whole 128 x D tile in registers as turned fp32 values (D/16 slots a row,
// rope.cuh), so each element is read and turned once, and load the next
// head's tile while they reduce and round this one.  The angles belong to the
// row and are computed once for all heads of the run (but for kRopeHalfAny, which
// computes them per element and head: 7800 x 24 x 128, 61 pairs, 172 us against
// 49 with 64).
// K (turned, pooled) and V of 6240 x 24 heads x 128: 26.2 us, 4.4 TB/s of the
// least bytes; runs of 8 heads, two waves of one CTA to an SM.  A start costs
// about 3 us and a tile 1.25 us: 4 heads 37 us, 6 heads 32 us, 12 heads 30 us.
#include "common.cuh"
#include "e4m3.cuh"
#include "rope.cuh"
#include "slots.cuh"

namespace bsa {

bsa_status check_rope_chunk(int B, int Hh, int D, int T, int H, int W);

constexpr int kApp8Threads = 512;
constexpr int kApp8Warps = kApp8Threads / 32;

struct Append8Args {
  RopeArgs rope;
  const uint4* src[2];
  uint8_t* dst[2];
  float* scale[2];
  float* kmean;         // optional
  const int32_t* perm;
  int32_t* block_valid;
  int32_t* d_err;
  int N, Hh, nb, B;
  HeadRuns runs;
  int max_blocks, base_block;
  int T, H, W;
};

// Largest of the warps' maxima, over all warps of the CTA.
__device__ __forceinline__ float cta_max(const float* s_red) {
  const float4* v = reinterpret_cast<const float4*>(s_red);
  float m = 0.f;
#pragma unroll
  for (int w = 0; w < kApp8Warps / 4; ++w) {
    const float4 x = v[w];
    m = fmaxf(fmaxf(m, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
  }
  return m;
}

__device__ __forceinline__ float warp_max(float x) {
  // Magnitudes: ordered as their bits.
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

template <int D, int MODE, bool kMean>
__device__ __forceinline__ void append8_heads(const Append8Args& a, int which, int b, int j,
                                              int h0, int h1, const int* s_tok, int valid,
                                              float* s_red, float* s_sum) {
  constexpr int kSlots = D / 16, kVecs = D / 8;
  constexpr int kRowStep = kApp8Threads / kSlots;
  constexpr int kRows = kBlk / kRowStep;  // rows per thread: 2, or 1 for D = 64
  const int slot = threadIdx.x % kSlots;
  const int row0 = threadIdx.x / kSlots;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long bN = static_cast<long long>(b) * a.N;
  int va, vb;
  slot_vectors<D, MODE>(a.rope.P, slot, va, vb);
  SlotTrig g[kRows];
  const uint4* src[kRows];  // the row of head h0; null for a pad row
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int tok = s_tok[row0 + i * kRowStep];
    src[i] = tok < 0 ? nullptr : a.src[which] + ((bN + tok) * a.Hh + h0) * kVecs;
  }
  uint4 x[kRows], y[kRows];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      x[i] = y[i] = make_uint4(0, 0, 0, 0);
      if (MODE != kRopeHalfAny && src[i] != nullptr) {
        x[i] = ld_nc_v4(src[i] + (h - h0) * kVecs + va);
        y[i] = ld_nc_v4(src[i] + (h - h0) * kVecs + vb);
      }
    }
  };
  load(h0);
  if (MODE == kRopeInterleaved || MODE == kRopeHalf) {
    TokenPos pos[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      pos[i] = token_pos(a.rope, bN, max(s_tok[row0 + i * kRowStep], 0));
    slot_trig<MODE, kRows>(a.rope, pos, slot, va, vb, g);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (s_tok[row0 + i * kRowStep] < 0) g[i].n = 0;  // pad rows stay +0
  }
  for (int h = h0; h < h1; ++h) {
    const long long blk = (static_cast<long long>(b) * a.Hh + h) * a.max_blocks + a.base_block + j;
    float p[kRows][8], q[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (MODE == kRopeHalfAny) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[i][e] = q[i][e] = 0.f;
        if (src[i] != nullptr)
          turn_slot_any(a.rope, token_pos(a.rope, bN, s_tok[row0 + i * kRowStep]), slot,
                        reinterpret_cast<const __nv_bfloat16*>(src[i] + (h - h0) * kVecs), p[i],
                        q[i]);
      } else {
        unpack8(x[i], p[i]);
        unpack8(y[i], q[i]);
        if (MODE != kRopeNone) turn_slot<MODE>(g[i], p[i], q[i]);
      }
    }
    if (h + 1 < h1) load(h + 1);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(p[i][e]), fabsf(q[i][e])));
    }
    amax = warp_max(amax);
    // One barrier a head: the buffers alternate, so a head's are written again
    // only after every thread has passed the next head's barrier.
    float* red = s_red + (h & 1) * kApp8Warps;
    float* sums = s_sum + (h & 1) * (kApp8Warps * D);
    if (lane == 0) red[warp] = amax;
    if (kMean) {
      // Lanes with the same slot hold the same columns.
      float sum[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[e] = p[0][e];
        sum[8 + e] = q[0][e];
#pragma unroll
        for (int i = 1; i < kRows; ++i) {
          sum[e] += p[i][e];
          sum[8 + e] += q[i][e];
        }
      }
      // Halve the columns a lane sums with each lane bit it is joined over: a
      // lane ends with 16 / (32 / kSlots) columns.
      int first = 0;
#pragma unroll
      for (int width = 8, off = 16; off >= kSlots; width >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int e = 0; e < width; ++e) {
          const float give = up ? sum[e] : sum[e + width];
          const float keep = up ? sum[e + width] : sum[e];
          sum[e] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
        first += up ? width : 0;
      }
      constexpr int kLeft = 16 * kSlots / 32;
#pragma unroll
      for (int e = 0; e < kLeft; ++e) {
        const int col = first + e;  // 0..7 of vector va, 8..15 of vb
        sums[warp * D + (col < 8 ? va * 8 + col : vb * 8 + col - 8)] = sum[e];
      }
    }
    __syncthreads();
    amax = cta_max(red);
    if (amax > 3.402823466e38f) {
      // An infinity: the scale is that of the largest finite magnitude.
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = fabsf(p[i][e]), v = fabsf(q[i][e]);
          amax = fmaxf(amax, fmaxf(u <= 3.402823466e38f ? u : 0.f, v <= 3.402823466e38f ? v : 0.f));
        }
      }
      amax = warp_max(amax);
      __syncthreads();  // every thread has read the first maxima
      if (lane == 0) red[warp] = amax;
      __syncthreads();
      amax = cta_max(red);
    }
    amax = fmaxf(amax, kAmaxFloor);
    const float mul = kE4m3Max / amax;
    if (threadIdx.x == 0) a.scale[which][blk] = amax / kE4m3Max;
    if (kMean && threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kApp8Warps; ++w) t += sums[w * D + threadIdx.x];
      a.kmean[blk * D + threadIdx.x] = t / static_cast<float>(valid);
    }
    uint8_t* dst = a.dst[which] + blk * (kBlk * D);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[e] = pack_e4m3x2(p[i][4 * e] * mul, p[i][4 * e + 1] * mul) |
               (pack_e4m3x2(p[i][4 * e + 2] * mul, p[i][4 * e + 3] * mul) << 16);
        w[2 + e] = pack_e4m3x2(q[i][4 * e] * mul, q[i][4 * e + 1] * mul) |
                   (pack_e4m3x2(q[i][4 * e + 2] * mul, q[i][4 * e + 3] * mul) << 16);
      }
      uint8_t* row = dst + (row0 + i * kRowStep) * D;
      if (MODE == kRopeInterleaved || MODE == kRopeHalf) {
        *reinterpret_cast<uint2*>(row + va * 8) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + vb * 8) = make_uint2(w[2], w[3]);
      } else {  // the two vectors are neighbours
        st_v4(row + va * 8, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

template <int D, int MODE>
__global__ void __launch_bounds__(kApp8Threads, 1)
append8_kernel(Append8Args a) {
  pdl_wait();     // global memory only after the predecessor grid completed
  pdl_trigger();
  __shared__ int s_tok[kBlk];
  __shared__ __align__(16) float s_red[2 * kApp8Warps];
  __shared__ float s_sum[2 * kApp8Warps * D];
  const RunAt at(a.runs, a.nb, a.B, a.Hh);
  const int slot0 = at.j * kBlk;
  const int valid = min(kBlk, a.N - slot0);
  find_block_tokens<kApp8Threads>(a.perm, a.N, slot0, valid, s_tok, at.j == 0 && at.first, a.d_err,
                                  a.T, a.H, a.W);
  if (at.first && threadIdx.x == 0) a.block_valid[a.base_block + at.j] = valid;
  // A slot of the chunk that no token maps to: perm is not a permutation.
  if (at.first && threadIdx.x < valid && s_tok[threadIdx.x] < 0) report(a.d_err, BSA_DEV_BAD_PERM);
  if (at.which == 1) {
    append8_heads<D, kRopeNone, false>(a, 1, at.b, at.j, at.h0, at.h1, s_tok, valid, s_red, s_sum);
  } else if (a.kmean != nullptr) {
    append8_heads<D, MODE, true>(a, 0, at.b, at.j, at.h0, at.h1, s_tok, valid, s_red, s_sum);
  } else {
    append8_heads<D, MODE, false>(a, 0, at.b, at.j, at.h0, at.h1, s_tok, valid, s_red, s_sum);
  }
}

template <int D>
static bsa_status launch_append8(int mode, Append8Args a, cudaStream_t s) {
  const long long blocks = static_cast<long long>(a.nb) * a.B;
  // K's and V's tiles cost about the same here (both are reduced and rounded):
  // runs of one length, a start counting as one head (8 and 8 heads measured
  // 26.5 us where 12 and 4, which suit rope_blocks_kernel's cost, took 27.6).
  const int heads = heads_per_cta(2 * blocks, a.Hh, 1, 1.0);
  a.runs = HeadRuns{{heads, heads}};
  const dim3 grid(run_ctas(a.runs, blocks, a.Hh, 2)), block(kApp8Threads);
  switch (mode) {
    case kRopeNone: return launch_pdl(append8_kernel<D, kRopeNone>, grid, block, 0, s, a);
    case kRopeInterleaved:
      return launch_pdl(append8_kernel<D, kRopeInterleaved>, grid, block, 0, s, a);
    case kRopeHalf: return launch_pdl(append8_kernel<D, kRopeHalf>, grid, block, 0, s, a);
    default: return launch_pdl(append8_kernel<D, kRopeHalfAny>, grid, block, 0, s, a);
  }
}

}  // namespace bsa

using namespace bsa;

extern "C" bsa_status bsa_kv8_append(bsa_kv_cache8* c, const void* k_tok, const void* v_tok, int T,
                                     int H, int W, const int32_t* d_perm,
                                     const bsa_rope_desc* rope, int32_t* d_err, void* stream) {
  if (c == nullptr || k_tok == nullptr || v_tok == nullptr || c->k == nullptr ||
      c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr ||
      c->block_valid == nullptr)
    return BSA_ERR_INVALID_ARG;
  BSA_TRY(check_rope_chunk(c->B, c->Hh, c->D, T, H, W));
  if (!aligned16(k_tok) || !aligned16(v_tok) || !aligned16(c->k) || !aligned16(c->v) ||
      !aligned16(c->kmean))
    return BSA_ERR_INVALID_ARG;
  if (c->max_blocks <= 0 || c->n_blocks < 0 || c->n_blocks > c->max_blocks)
    return BSA_ERR_INVALID_ARG;
  Append8Args a{};
  int mode = kRopeNone;
  if (rope != nullptr) BSA_TRY(rope_args(rope, c->B, c->D, T, H, W, &a.rope, &mode));
  const int n = T * H * W;
  if (d_perm != nullptr && n > kGatherMaxTokens) return BSA_ERR_UNSUPPORTED;
  const int nb = (n + kBlk - 1) / kBlk;
  if (nb > c->max_blocks - c->n_blocks) return BSA_ERR_CAPACITY;
  a.src[0] = static_cast<const uint4*>(k_tok);
  a.src[1] = static_cast<const uint4*>(v_tok);
  a.dst[0] = static_cast<uint8_t*>(c->k);
  a.dst[1] = static_cast<uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.kmean = c->kmean;
  a.perm = d_perm;
  a.block_valid = c->block_valid;
  a.d_err = d_err;
  a.N = n;
  a.Hh = c->Hh;
  a.nb = nb;
  a.B = c->B;
  a.max_blocks = c->max_blocks;
  a.base_block = c->n_blocks;
  a.T = T;
  a.H = H;
  a.W = W;
  cudaStream_t s = as_stream(stream);
  BSA_TRY(c->D == 128 ? launch_append8<128>(mode, a, s) : launch_append8<64>(mode, a, s));
  c->n_blocks += nb;
  return BSA_OK;
}
