// rope.cu - rotary positions: on raster tokens (bsa_rope, forward and
// gradient) and on the way into 128-token blocks (bsa_tokens_to_blocks_rope,
// bsa_kv_append_rope), with the host tables (bsa_rope_frequencies,
// bsa_rope_phases).
//
// Both kernels are HBM streams: every element is read and written once (4
// bytes).  A thread owns a slot of a token (rope.cuh), computes its eight angles
// once and applies them to a run of heads, so the sines cost nothing per head
// and no table goes through memory.  Not so the half layout with a pair count that
// is no multiple of 8 (kRopeHalfAny): it computes an angle for every element of
// every head and loads elements one by one; 7800 x 24 x 128 with 61 pairs takes
// 125 us, with 56 or 64 pairs 22 to 25.  Means, where asked for, are a second
// kernel over the blocks written (7800 x 24 x 128: 26.6 -> 34.8 us for one
// tensor, 38.9 -> 49.2 us for K and V, cold L2).
//   tokens  40001 x 24 heads x 64, 48 of 64 dimensions: 44.5 us, 5.5 TB/s
//           (runs of 12 heads; runs of 24, one wave and a half of CTAs: 57 us)
//   blocks  K and V of 7800 x 24 heads x 128: 36 us, 5.3 TB/s.  A CTA's start
//           (its tokens, angles and first tiles) costs about 3 us, a head's
//           tile 1.4 us, so K's runs are long (24 heads) and V's shorter ones
//           (6) fill the SMs they leave: 24 heads for both took 39 us, 8 47 us.
#include <math.h>

#include "common.cuh"
#include "rope.cuh"
#include "slots.cuh"

namespace bsa {

bsa_status launch_block_means(const bsa_kv_cache* c, int first, int count, int32_t* d_err,
                              cudaStream_t s);
bsa_status launch_rows_mean(const void* x_blk, float* x_mean, int B, int Hh, int D, int nb, int N,
                            cudaStream_t s);

bsa_status rope_args(const bsa_rope_desc* d, int B, int D, int T, int H, int W, RopeArgs* out,
                     int* mode) {
  if (d == nullptr || d->phase == nullptr) return BSA_ERR_INVALID_ARG;
  if (d->n_axes != 1 && d->n_axes != 3) return BSA_ERR_INVALID_ARG;
  if (d->layout != BSA_ROPE_INTERLEAVED && d->layout != BSA_ROPE_HALF) return BSA_ERR_INVALID_ARG;
  long long P = 0;
  for (int i = 0; i < 3; ++i) {
    if (d->n_pairs[i] < 0 || (d->n_axes == 1 && i > 0 && d->n_pairs[i] != 0))
      return BSA_ERR_INVALID_ARG;
    P += d->n_pairs[i];
  }
  if (P <= 0 || !isfinite(d->amplitude)) return BSA_ERR_INVALID_ARG;
  if (P > D / 2) return BSA_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(d->phase) & 7u) || (reinterpret_cast<uintptr_t>(d->pos) & 3u))
    return BSA_ERR_INVALID_ARG;
  RopeArgs& r = *out;
  r.phase = reinterpret_cast<const uint64_t*>(d->phase);
  r.pos = d->pos;
  r.pos_stride = static_cast<long long>(B) * T * H * W;
  r.P = static_cast<int>(P);
  r.p0 = d->n_pairs[0];
  r.p01 = d->n_pairs[0] + d->n_pairs[1];
  r.n_axes = d->n_axes;
  r.inverse = d->inverse;
  r.H = H;
  r.W = W;
  r.o0 = d->origin[0];
  r.o1 = d->origin[1];
  r.o2 = d->origin[2];
  r.amp = d->amplitude;
  *mode = d->layout == BSA_ROPE_INTERLEAVED ? kRopeInterleaved
                                            : (P % 8 == 0 ? kRopeHalf : kRopeHalfAny);
  return BSA_OK;
}

constexpr int kRopeThreads = 256;
constexpr int kHeadsInFlight = 4;  // heads whose vectors are loaded before any is stored

// Plain 16-byte load (the tensor may be turned in place).
__device__ __forceinline__ uint4 ld_v4(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Turn slot `slot` of heads [h0, h1) of a token, whose heads' rows start at src
// and go to dst.  All of a row's slots are lanes of one warp and the warp has
// read a row before it writes it, so src and dst may be the same; `on` is false
// for a lane without a token.
template <int D, int MODE>
__device__ __forceinline__ void turn_heads(const RopeArgs& r, const TokenPos& pos, int slot,
                                           bool on, const uint4* src, uint4* dst, int h0, int h1) {
  constexpr int kVecs = D / 8;
  SlotTrig g[1];
  int va, vb;
  slot_vectors<D, MODE>(r.P, slot, va, vb);
  if (MODE == kRopeHalfAny) {
    for (int h = h0; h < h1; ++h) {
      float a[8], b[8];
      if (on)
        turn_slot_any(r, pos, slot, reinterpret_cast<const __nv_bfloat16*>(src + h * kVecs), a, b);
      __syncwarp();
      if (on) {
        st_v4(dst + h * kVecs + va, pack8(a));
        st_v4(dst + h * kVecs + vb, pack8(b));
      }
    }
    return;
  }
  if (!on) return;
  const TokenPos at[1] = {pos};
  slot_trig<MODE, 1>(r, at, slot, va, vb, g);
  for (int h = h0; h < h1; h += kHeadsInFlight) {
    uint4 x[kHeadsInFlight], y[kHeadsInFlight];
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < h1) {
        x[u] = ld_v4(src + (h + u) * kVecs + va);
        y[u] = ld_v4(src + (h + u) * kVecs + vb);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u >= h1) break;
      float a[8], b[8];
      unpack8(x[u], a);
      unpack8(y[u], b);
      turn_slot<MODE>(g[0], a, b);
      st_v4(dst + (h + u) * kVecs + va, pack8(a));
      st_v4(dst + (h + u) * kVecs + vb, pack8(b));
    }
  }
}

struct RopeTokensArgs {
  RopeArgs rope;
  const uint4* x;
  uint4* y;
  int N, Hh, heads;  // heads per CTA
};

template <int D, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
rope_tokens_kernel(RopeTokensArgs a) {
  pdl_wait();     // global memory only after the predecessor grid completed
  pdl_trigger();
  constexpr int kSlots = D / 16, kVecs = D / 8;
  const int slot = threadIdx.x % kSlots;
  const int tok = blockIdx.x * (kRopeThreads / kSlots) + threadIdx.x / kSlots;
  const bool on = tok < a.N;
  const long long bN = static_cast<long long>(blockIdx.z) * a.N;
  const TokenPos pos = token_pos(a.rope, bN, on ? tok : 0);
  const long long row = (bN + (on ? tok : 0)) * a.Hh * kVecs;
  const int h0 = blockIdx.y * a.heads;
  const int h1 = min(h0 + a.heads, a.Hh);
  turn_heads<D, MODE>(a.rope, pos, slot, on, a.x + row, a.y + row, h0, h1);
}

// The chunk's tokens into blocks, K (or the one tensor) turned, V as it is:
// one CTA per block and run of heads of one tensor.
struct RopeBlocksArgs {
  RopeArgs rope;
  const uint4* src[2];
  uint4* dst[2];
  const int32_t* perm;
  int32_t* block_valid;  // optional
  int32_t* d_err;
  int N, Hh, nb, B, tensors;
  HeadRuns runs;
  long long blk_stride;
  int base_block;
  int T, H, W;
};

constexpr int kBlocksThreads = 512;

// Heads [h0, h1) of the block's rows.  512 threads hold a whole tile (D/16 slots
// a row, 2 rows a thread, 1 for D = 64), and the tiles of the next two heads
// are on their way while one is turned and written.
template <int D, int MODE>
__device__ __forceinline__ void blocks_heads(const RopeBlocksArgs& a, int which, int b, int j,
                                             int h0, int h1, const int* s_tok) {
  constexpr int kSlots = D / 16, kVecs = D / 8;
  constexpr int kRowStep = kBlocksThreads / kSlots, kRows = kBlk / kRowStep;
  constexpr int kAhead = 2;
  const int slot = threadIdx.x % kSlots, row0 = threadIdx.x / kSlots;
  const long long bN = static_cast<long long>(b) * a.N;
  const long long dst_step = a.blk_stride * kBlk * kVecs;
  uint4* dst = a.dst[which] + (static_cast<long long>(b) * a.Hh + h0) * dst_step +
               (static_cast<long long>(a.base_block + j) * kBlk + row0) * kVecs;
  int va, vb;
  slot_vectors<D, MODE>(a.rope.P, slot, va, vb);
  const uint4* src[kRows];  // the row of head h0; null for a pad row
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int tok = s_tok[row0 + i * kRowStep];
    src[i] = tok < 0 ? nullptr : a.src[which] + ((bN + tok) * a.Hh + h0) * kVecs;
  }
  uint4 x[kAhead][kRows], y[kAhead][kRows];
  auto load = [&](int h, uint4(&u)[kRows], uint4(&v)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      u[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (MODE != kRopeHalfAny && h < h1 && src[i] != nullptr) {
        u[i] = ld_nc_v4(src[i] + (h - h0) * kVecs + va);
        v[i] = ld_nc_v4(src[i] + (h - h0) * kVecs + vb);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(h0 + k, x[k], y[k]);
  SlotTrig g[kRows];
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
  for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (h + k >= h1) break;
      uint4 u[kRows], v[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        u[i] = x[k][i];
        v[i] = y[k][i];
      }
      load(h + k + kAhead, x[k], y[k]);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (MODE != kRopeNone) {
          float p[8], q[8];
          if (MODE == kRopeHalfAny) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = q[e] = 0.f;
            if (src[i] != nullptr)
              turn_slot_any(a.rope, token_pos(a.rope, bN, s_tok[row0 + i * kRowStep]), slot,
                            reinterpret_cast<const __nv_bfloat16*>(src[i] + (h + k - h0) * kVecs),
                            p, q);
          } else {
            unpack8(u[i], p);
            unpack8(v[i], q);
            turn_slot<MODE>(g[i], p, q);
          }
          u[i] = pack8(p);
          v[i] = pack8(q);
        }
        uint4* row = dst + (h + k - h0) * dst_step + i * (kRowStep * kVecs);
        st_v4(row + va, u[i]);
        st_v4(row + vb, v[i]);
      }
    }
  }
}

template <int D, int MODE>
__global__ void __launch_bounds__(kBlocksThreads, 1)
rope_blocks_kernel(RopeBlocksArgs a) {
  pdl_wait();     // global memory only after the predecessor grid completed
  pdl_trigger();
  __shared__ int s_tok[kBlk];
  const RunAt at(a.runs, a.nb, a.B, a.Hh);
  const int slot0 = at.j * kBlk;
  const int valid = min(kBlk, a.N - slot0);
  find_block_tokens<kBlocksThreads>(a.perm, a.N, slot0, valid, s_tok, at.j == 0 && at.first,
                                    a.d_err, a.T, a.H, a.W);
  if (at.first && a.block_valid != nullptr && threadIdx.x == 0)
    a.block_valid[a.base_block + at.j] = valid;
  // A slot of the chunk that no token maps to: perm is not a permutation.
  if (at.first && threadIdx.x < valid && s_tok[threadIdx.x] < 0) report(a.d_err, BSA_DEV_BAD_PERM);
  if (at.which == 0)
    blocks_heads<D, MODE>(a, 0, at.b, at.j, at.h0, at.h1, s_tok);
  else
    blocks_heads<D, kRopeNone>(a, 1, at.b, at.j, at.h0, at.h1, s_tok);
}

template <int D>
static bsa_status launch_tokens(int mode, const RopeTokensArgs& a, int B, cudaStream_t s) {
  constexpr int kToks = kRopeThreads / (D / 16);
  dim3 grid((a.N + kToks - 1) / kToks, (a.Hh + a.heads - 1) / a.heads, B);
  const dim3 block(kRopeThreads);
  if (mode == kRopeInterleaved)
    return launch_pdl(rope_tokens_kernel<D, kRopeInterleaved>, grid, block, 0, s, a);
  if (mode == kRopeHalf) return launch_pdl(rope_tokens_kernel<D, kRopeHalf>, grid, block, 0, s, a);
  return launch_pdl(rope_tokens_kernel<D, kRopeHalfAny>, grid, block, 0, s, a);
}

template <int D>
static bsa_status launch_blocks(int mode, RopeBlocksArgs a, cudaStream_t s) {
  const long long blocks = static_cast<long long>(a.nb) * a.B;
  a.runs = head_runs(blocks, a.Hh, a.tensors);
  const dim3 grid(run_ctas(a.runs, blocks, a.Hh, a.tensors)), block(kBlocksThreads);
  if (mode == kRopeInterleaved)
    return launch_pdl(rope_blocks_kernel<D, kRopeInterleaved>, grid, block, 0, s, a);
  if (mode == kRopeHalf) return launch_pdl(rope_blocks_kernel<D, kRopeHalf>, grid, block, 0, s, a);
  return launch_pdl(rope_blocks_kernel<D, kRopeHalfAny>, grid, block, 0, s, a);
}

// Sizes every rotated call accepts.
bsa_status check_rope_chunk(int B, int Hh, int D, int T, int H, int W) {
  if (B <= 0 || Hh <= 0 || T <= 0 || H <= 0 || W <= 0) return BSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  const long long plane = static_cast<long long>(T) * H;
  if (plane > (1LL << 24) || plane * W > (1LL << 24)) return BSA_ERR_SHAPE;
  if (B > 65535 || Hh > 65535) return BSA_ERR_SHAPE;  // grid limits of the means and bsa_rope
  const long long nb = (plane * W + kBlk - 1) / kBlk;
  if (nb * B * Hh >= (1LL << 31)) return BSA_ERR_SHAPE;  // tiles are counted in 32 bits
  return BSA_OK;
}

}  // namespace bsa

using namespace bsa;

extern "C" bsa_status bsa_rope_frequencies(int n, double base, int scaling, double factor,
                                           double original_length, double beta_fast,
                                           double beta_slow, double* host_freq,
                                           double* host_amplitude) {
  if (host_freq == nullptr || n <= 0 || !(base > 0) || !isfinite(base)) return BSA_ERR_INVALID_ARG;
  if (scaling < BSA_ROPE_SCALE_NONE || scaling > BSA_ROPE_SCALE_BY_PARTS)
    return BSA_ERR_INVALID_ARG;
  if (scaling != BSA_ROPE_SCALE_NONE && (!(factor > 0) || !isfinite(factor)))
    return BSA_ERR_INVALID_ARG;
  if (scaling == BSA_ROPE_SCALE_BY_PARTS &&
      (!(original_length > 0) || !isfinite(original_length) || !(beta_fast > beta_slow) ||
       !isfinite(beta_fast) || !isfinite(beta_slow)))
    return BSA_ERR_INVALID_ARG;
  const double kTwoPi = 2.0 * acos(-1.0);
  double b = base, amp = 1.0;
  if (scaling == BSA_ROPE_SCALE_BASE && n > 1) b *= pow(factor, static_cast<double>(n) / (n - 1));
  if (scaling == BSA_ROPE_SCALE_BY_PARTS && factor > 1.0) amp = 0.1 * log(factor) + 1.0;
  for (int i = 0; i < n; ++i) {
    double f = pow(b, -static_cast<double>(i) / n);
    if (scaling == BSA_ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == BSA_ROPE_SCALE_BY_PARTS) {
      const double turns = original_length * f / kTwoPi;
      double keep = (turns - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    host_freq[i] = f;
  }
  if (host_amplitude != nullptr) *host_amplitude = amp;
  return BSA_OK;
}

extern "C" bsa_status bsa_rope_phases(const double* host_freq, int n, int64_t* host_phase) {
  if (host_freq == nullptr || host_phase == nullptr || n <= 0) return BSA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!isfinite(host_freq[i])) return BSA_ERR_INVALID_ARG;
  const long double two_pi = 2.0L * acosl(-1.0L);
  for (int i = 0; i < n; ++i) {
    const long double turns = static_cast<long double>(host_freq[i]) / two_pi;
    const long double frac = turns - floorl(turns);  // [0, 1)
    // Rounded to 2^64 a fraction just below 1 is a whole turn: phase 0.
    const long double scaled = roundl(ldexpl(frac, 64));
    const uint64_t u = scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
    host_phase[i] = static_cast<int64_t>(u);
  }
  return BSA_OK;
}

extern "C" bsa_status bsa_rope(const void* x_tok, void* y_tok, int B, int Hh, int D, int T, int H,
                               int W, const bsa_rope_desc* rope, void* stream) {
  if (x_tok == nullptr || y_tok == nullptr) return BSA_ERR_INVALID_ARG;
  BSA_TRY(check_rope_chunk(B, Hh, D, T, H, W));
  if (!aligned16(x_tok) || !aligned16(y_tok)) return BSA_ERR_INVALID_ARG;
  RopeTokensArgs a{};
  int mode;
  BSA_TRY(rope_args(rope, B, D, T, H, W, &a.rope, &mode));
  a.x = static_cast<const uint4*>(x_tok);
  a.y = static_cast<uint4*>(y_tok);
  a.N = T * H * W;
  a.Hh = Hh;
  const int toks = kRopeThreads / (D / 16);
  a.heads = heads_per_cta(static_cast<long long>((a.N + toks - 1) / toks) * B, Hh, 3, 2.0);
  return D == 128 ? launch_tokens<128>(mode, a, B, as_stream(stream))
                  : launch_tokens<64>(mode, a, B, as_stream(stream));
}

extern "C" bsa_status bsa_tokens_to_blocks_rope(const void* x_tok, void* x_blk, float* x_mean,
                                                int B, int Hh, int D, int T, int H, int W,
                                                const int32_t* d_perm, const bsa_rope_desc* rope,
                                                int32_t* d_err, void* stream) {
  if (x_tok == nullptr || x_blk == nullptr) return BSA_ERR_INVALID_ARG;
  BSA_TRY(check_rope_chunk(B, Hh, D, T, H, W));
  if (!aligned16(x_tok) || !aligned16(x_blk) || !aligned16(x_mean)) return BSA_ERR_INVALID_ARG;
  RopeBlocksArgs a{};
  int mode;
  BSA_TRY(rope_args(rope, B, D, T, H, W, &a.rope, &mode));
  const int n = T * H * W;
  if (d_perm != nullptr && n > kGatherMaxTokens) return BSA_ERR_UNSUPPORTED;
  const int nb = (n + kBlk - 1) / kBlk;
  a.src[0] = static_cast<const uint4*>(x_tok);
  a.dst[0] = static_cast<uint4*>(x_blk);
  a.perm = d_perm;
  a.d_err = d_err;
  a.N = n;
  a.Hh = Hh;
  a.tensors = 1;
  a.nb = nb;
  a.B = B;
  a.blk_stride = nb;
  a.T = T;
  a.H = H;
  a.W = W;
  cudaStream_t s = as_stream(stream);
  BSA_TRY(D == 128 ? launch_blocks<128>(mode, a, s) : launch_blocks<64>(mode, a, s));
  return x_mean == nullptr ? BSA_OK : launch_rows_mean(x_blk, x_mean, B, Hh, D, nb, n, s);
}

extern "C" bsa_status bsa_kv_append_rope(bsa_kv_cache* c, const void* k_tok, const void* v_tok,
                                         int T, int H, int W, const int32_t* d_perm,
                                         const bsa_rope_desc* rope, int32_t* d_err, void* stream) {
  if (c == nullptr || k_tok == nullptr || v_tok == nullptr || c->k == nullptr ||
      c->v == nullptr || c->block_valid == nullptr)
    return BSA_ERR_INVALID_ARG;
  BSA_TRY(check_rope_chunk(c->B, c->Hh, c->D, T, H, W));
  if (!aligned16(k_tok) || !aligned16(v_tok) || !aligned16(c->k) || !aligned16(c->v) ||
      !aligned16(c->kmean))
    return BSA_ERR_INVALID_ARG;
  if (c->max_blocks <= 0 || c->n_blocks < 0 || c->n_blocks > c->max_blocks)
    return BSA_ERR_INVALID_ARG;
  RopeBlocksArgs a{};
  int mode;
  BSA_TRY(rope_args(rope, c->B, c->D, T, H, W, &a.rope, &mode));
  const int n = T * H * W;
  if (d_perm != nullptr && n > kGatherMaxTokens) return BSA_ERR_UNSUPPORTED;
  const int nb = (n + kBlk - 1) / kBlk;
  if (nb > c->max_blocks - c->n_blocks) return BSA_ERR_CAPACITY;
  a.src[0] = static_cast<const uint4*>(k_tok);
  a.dst[0] = static_cast<uint4*>(c->k);
  a.src[1] = static_cast<const uint4*>(v_tok);
  a.dst[1] = static_cast<uint4*>(c->v);
  a.perm = d_perm;
  a.block_valid = c->block_valid;
  a.d_err = d_err;
  a.N = n;
  a.Hh = c->Hh;
  a.tensors = 2;
  a.nb = nb;
  a.B = c->B;
  a.blk_stride = c->max_blocks;
  a.base_block = c->n_blocks;
  a.T = T;
  a.H = H;
  a.W = W;
  cudaStream_t s = as_stream(stream);
  BSA_TRY(c->D == 128 ? launch_blocks<128>(mode, a, s) : launch_blocks<64>(mode, a, s));
  if (c->kmean != nullptr) BSA_TRY(launch_block_means(c, c->n_blocks, nb, d_err, s));
  c->n_blocks += nb;
  return BSA_OK;
}
