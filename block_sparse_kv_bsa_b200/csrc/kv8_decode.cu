// kv8_decode.cu - bsa_kv8_attn_decode: a few query tokens over the 8-bit
// cache.
//
// The rows of one cache head are its n_tok * group query rows, 16 to a tile, or
// one tile of up to 8 (mma.sync, attn8_warp.cuh).  With so few rows the call is bound by reading
// the cache once (1 byte an element of K and V), so the blocks are split over
// the SMs and each CTA streams its share through a ring of K and V tiles that
// TMA keeps full (192 KB: the 50 KB or so that an SM must have in flight to
// draw its part of the memory rate, several times over).  Eight warps take 16
// keys each of every block; they join through shared memory, and the splits
// through a workspace and a second small kernel, always in the same order.
#include "common.cuh"
#include "attn8_warp.cuh"
#include "tma_host.cuh"

namespace bsa {

constexpr int kDecWarps = 8;                          // consumers: 16 keys of each block
constexpr int kDecThreads = kDecWarps * 32 + 32;      // and one producer warp
constexpr int kDecSlots = 148;     // CTAs resident at once: one on each SM
constexpr int kDecMaxRows = 128;   // query rows of one cache head
constexpr long long kDecWait = 1LL << 31;  // SM clocks (about a second)

template <int D>
struct DecodeLayout {
  static constexpr int kTile = kBlk * D;
  static constexpr int kStages = D == 128 ? 6 : 12;
  static constexpr int kRing = 0;                              // [stage][K, V]
  static constexpr int kBars = kRing + kStages * 2 * kTile;    // full, empty per stage
  static constexpr int kMeta = kBars + kStages * 16;           // float4 per stage
  static constexpr int kMl = kMeta + kStages * 16;             // float [warps][16][2]
  static constexpr int kMisc = kMl + kDecWarps * 16 * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static constexpr int kOut = kRing;                           // float [warps][16][D + 8] at the end
  static_assert(kDecWarps * 16 * (D + 8) * 4 <= kStages * 2 * kTile, "warps' O fits the ring");
  static_assert(kAlloc <= 227 * 1024, "shared memory per CTA");
};

struct Decode8Args {
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_valid;
  const int32_t* idx;
  const int32_t* cnt;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;   // [B*Hh*tiles][n_split][16][D], columns as the warps leave them
  float* part_ml;  // [B*Hh*tiles][n_split][16][2]
  int32_t* d_err;
  int Hq, Hh, group, n_tok, rows, tiles, n_split;
  int n_sel, max_blocks, n_blocks;
  float scale_log2;
};

// Row r (token r / group, head r % group of the group) of cache head bh, as an
// index of [B, n_tok, Hq].
__device__ __forceinline__ long long query_row(const Decode8Args& a, long long bh, int r) {
  const long long b = bh / a.Hh;
  const int h = static_cast<int>(bh % a.Hh);
  return (b * a.n_tok + r / a.group) * a.Hq + h * a.group + r % a.group;
}

// Whether a row saw a key: its sum is zero and its reference unset only without
// one (logits that are all NaN leave the reference unset and the sum NaN).
__device__ __forceinline__ bool row_has_keys(float m, float l) {
  return m > -INFINITY || l != 0.f;
}

// W is AttnWarp16<D>, or AttnWarp8<D> for at most 8 rows in all.
template <int D, class W>
__global__ void __launch_bounds__(kDecThreads, 1)
decode8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               Decode8Args a) {
  using L = DecodeLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(sm);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint64_t* empty = full + L::kStages;
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + L::kMisc);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], kDecWarps);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();     // global memory only after the predecessor grid completed
  pdl_trigger();
  const int split = blockIdx.y;
  const long long item = blockIdx.x;
  const long long bh = item / a.tiles;
  const int tile = static_cast<int>(item % a.tiles);

  int n = a.n_sel;
  const int guess0 = min(n, split * ((n + a.n_split - 1) / a.n_split));
  int guess = -1;
  if (warp == kDecWarps && a.idx != nullptr && guess0 + lane < n)
    guess = a.idx[bh * a.n_sel + guess0 + lane];
  if (a.cnt != nullptr) {
    n = a.cnt[bh];
    if (n < 0 || n > a.n_sel) {
      report(a.d_err, BSA_DEV_BAD_COUNT);
      n = n < 0 ? 0 : a.n_sel;
    }
  }
  const int per = (n + a.n_split - 1) / a.n_split;
  const int e0 = min(n, split * per), count = min(n - e0, per);

  W w;
  bool ok = true;
  if (warp == kDecWarps) {
    // ---------------- producer: 32 blocks at a time, a block's tiles as soon as
    // its index is known, its scales and valid count behind them (a stage is
    // full when both its tiles and its metadata are there)
    int issued = 0;
    for (int c0 = 0; ok && c0 < count; c0 += 32) {
      int blk = e0 + c0 + lane;
      if (a.idx != nullptr && c0 + lane < count) {
        // The first entries were read beside the count, where a full route
        // has them.
        blk = c0 == 0 && e0 == guess0 ? guess : a.idx[bh * a.n_sel + blk];
        if (blk < 0 || blk >= a.n_blocks) {
          report(a.d_err, BSA_DEV_BAD_INDEX);
          blk = 0;
        }
      }
      int valid = kBlk;
      float ks = 1.f, vs = 1.f;
      if (c0 + lane < count) {
        valid = a.block_valid[blk];
        ks = a.k_scale[bh * a.max_blocks + blk];
        vs = a.v_scale[bh * a.max_blocks + blk];
      }
      // The first stages are empty: their copies go out ahead of the loads above.
      auto copy = [&](int u) {
        const int st = u % L::kStages;
        const int row = static_cast<int>((bh * a.max_blocks + blk) * kBlk);
        uint8_t* dst = sm + L::kRing + st * 2 * L::kTile;
        mbar_expect_tx(&full[st], 2 * L::kTile);
        tma_load_2d(dst, &tm_k, 0, row, &full[st]);
        tma_load_2d(dst + L::kTile, &tm_v, 0, row, &full[st]);
      };
      if (c0 == 0 && lane < min(count, L::kStages)) copy(lane);
      if (valid < 1 || valid > kBlk) {
        report(a.d_err, BSA_DEV_BAD_VALID);
        valid = valid < 1 ? 1 : kBlk;
      }
      ks = checked_k_scale(ks, a.d_err);
      vs = checked_v_scale(vs, a.d_err);
      const uint4 meta = make_uint4(__float_as_uint(ks), __float_as_uint(log2f(vs)),
                                    __float_as_uint(1.f / vs), static_cast<uint32_t>(valid));
      for (int i = 0; ok && i < 32 && c0 + i < count; ++i) {
        const int u = c0 + i, st = u % L::kStages;
        if (u >= L::kStages)
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[st], ((u / L::kStages) - 1) & 1,
                                                         s_abort, kDecWait));
        if (!ok) break;
        if (lane == i) {
          reinterpret_cast<uint4*>(sm + L::kMeta)[st] = meta;
          if (u >= L::kStages) copy(u);
          mbar_arrive(&full[st]);
        }
        __syncwarp();
        issued = u + 1;
      }
    }
    if (issued < min(count, L::kStages)) issued = min(count, L::kStages);
    // Copies in flight land before the ring is reused or the CTA exits.
    for (int u = max(0, issued - L::kStages); u < issued; ++u)
      mbar_wait_bounded(&full[u % L::kStages], (u / L::kStages) & 1, nullptr, kDecWait);
  } else {
    w.init(
        [&](int r) {
          r += tile * 16;
          return r < a.rows ? a.q + query_row(a, bh, r) * D : nullptr;
        },
        a.scale_log2);
    for (int u = 0; ok && u < count; ++u) {
      const int st = u % L::kStages;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(&full[st], (u / L::kStages) & 1, s_abort, kDecWait));
      if (!ok) break;
      const uint4 meta = lds128(base + L::kMeta + st * 16);
      const int valid = static_cast<int>(meta.w);
      if (warp * 16 < valid) {
        typename W::Keys x;
        const uint32_t kt = base + L::kRing + st * 2 * L::kTile;
        W::Tile::load_keys(kt, kt + L::kTile, warp * 16, valid, x);
        w.step(x, warp * 16, meta);
      }
      fence_proxy_async_smem();  // these reads before the refill, an async-proxy write
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
  }
  if (!ok && lane == 0) {
    report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
    *s_abort = 1;
  }

  // Join the warps: the ring is empty (every tile issued has been read).
  __syncthreads();
  constexpr int kStride = W::kStride;
  float* s_o = reinterpret_cast<float*>(sm + L::kOut);  // [warp][16][kStride]
  float* s_ml = reinterpret_cast<float*>(sm + L::kMl);  // [warp][16][2]
  if (warp < kDecWarps) w.finish(s_o + warp * 16 * kStride, s_ml + warp * 32);
  __syncthreads();
  const int rows = min(16, a.rows - tile * 16);
  for (int i = threadIdx.x; i < rows * D; i += kDecThreads) {
    const int r = i / D, c = i % D;  // column c as finish() left it
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kDecWarps; ++k) m = fmaxf(m, s_ml[(k * 16 + r) * 2]);
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int k = 0; k < kDecWarps; ++k) {
      const float mk = s_ml[(k * 16 + r) * 2];
      const float f = mk == -INFINITY ? 0.f : ex2_approx(mk - m);
      l = fmaf(s_ml[(k * 16 + r) * 2 + 1], f, l);
      o = fmaf(s_o[(k * 16 + r) * kStride + c], f, o);
    }
    if (a.n_split == 1) {
      const bool have = row_has_keys(m, l);
      const long long out = query_row(a, bh, tile * 16 + r);
      a.o[out * D + out_element<D>(c)] = __float2bfloat16(have ? o / l : 0.f);
      if (c == 0) a.lse[out] = have ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    } else {
      const long long p = (item * a.n_split + split) * 16 + r;
      a.part_o[p * D + c] = o;
      if (c == 0) {
        a.part_ml[p * 2] = m;
        a.part_ml[p * 2 + 1] = l;
      }
    }
  }
}

// Joins the splits of one query row: warp w takes splits w, w + 8, ..., each
// lane D / 32 columns; every warp works out the common maximum and sum for
// itself, so the parts are on their way from the start and one barrier joins
// the warps.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
decode8_join_kernel(Decode8Args a) {
  pdl_wait();     // global memory only after the predecessor grid completed
  pdl_trigger();
  constexpr int kCols = D / 32;
  __shared__ float s_acc[kJoinWarps][D];
  const int row = blockIdx.y;
  const long long bh = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long p0 = (bh * a.tiles + row / 16) * a.n_split * 16 + row % 16;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + p0;
  const float* part = a.part_o + p0 * D + lane * kCols;
  float v[kCols], acc[kCols];
  auto load = [&](int s) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) v[c] = s < a.n_split ? part[s * (16 * D) + c] : 0.f;
  };
  load(warp);
  float m = -INFINITY;
  for (int s = lane; s < a.n_split; s += 32) m = fmaxf(m, ml[s * 16].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float l = 0.f;
  for (int s = lane; s < a.n_split; s += 32) {
    const float2 x = ml[s * 16];
    l = fmaf(x.y, x.x == -INFINITY ? 0.f : ex2_approx(x.x - m), l);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
  for (int s = warp; s < a.n_split; s += kJoinWarps) {
    const float ms = ml[s * 16].x;
    const float f = ms == -INFINITY ? 0.f : ex2_approx(ms - m);
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = fmaf(v[c], f, acc[c]);
    load(s + kJoinWarps);
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) s_acc[warp][lane * kCols + c] = acc[c];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float o = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) o += s_acc[w][threadIdx.x];
  const bool have = row_has_keys(m, l);
  const long long out = query_row(a, bh, row);
  a.o[out * D + out_element<D>(threadIdx.x)] = __float2bfloat16(have ? o / l : 0.f);
  if (threadIdx.x == 0) a.lse[out] = have ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Splits of n_sel blocks: the count whose waves over the resident CTAs leave
// the fewest idle (a split is a wave's share of the blocks; a CTA's start and
// join count as two blocks), fewest first.  Past four items an SM there is one
// split, so that the workspace (16 x D floats an item and split) stays within some
// megabytes; the last wave is then partly empty (one token, 40 blocks: 152 us for
// 592 items, 166 for 608; 196 for 768, whose bytes take 154).
static int most_splits(long long items, int n_sel) {
  long long most = kDecSlots / items;
  if (most < 8) most = items <= 4 * kDecSlots ? 8 : 1;
  return static_cast<int>(most < n_sel ? most : n_sel);
}

static int split_count(long long items, int n_sel) {
  const int most = most_splits(items, n_sel);
  int best = 1;
  double best_cost = 1e30;
  for (int n = 1; n <= most; ++n) {
    const long long waves = (items * n + kDecSlots - 1) / kDecSlots;
    const double cost = static_cast<double>(waves) * ((n_sel + n - 1) / n + 2) * (1.0 + 0.0001 * n);
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

struct DecodeShape {
  int rows, tiles, n_split;
  size_t o_bytes, bytes;
};

static bsa_status decode_shape(int B, int Hq, int Hh, int D, int n_tok, int n_sel,
                               DecodeShape* out) {
  if (B <= 0 || Hq <= 0 || Hh <= 0 || n_tok <= 0 || n_sel < 0) return BSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  if (Hq % Hh != 0) return BSA_ERR_SHAPE;
  const long long rows = static_cast<long long>(n_tok) * (Hq / Hh);
  if (rows > kDecMaxRows) return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hh > (1 << 20)) return BSA_ERR_SHAPE;
  out->rows = static_cast<int>(rows);
  out->tiles = (out->rows + 15) / 16;
  const long long items = static_cast<long long>(B) * Hh * out->tiles;
  out->n_split = n_sel > 0 ? split_count(items, n_sel) : 1;
  // Sized for the most splits of any smaller n_sel: a program sizes the
  // workspace once for the cache it will grow to.
  const int most = most_splits(items, n_sel);
  const size_t parts = most > 1 ? static_cast<size_t>(items) * most * 16 : 0;
  out->o_bytes = (parts * D * sizeof(float) + 255) & ~static_cast<size_t>(255);
  out->bytes = out->o_bytes + ((parts * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255));
  return BSA_OK;
}

template <int D>
static bsa_status launch_decode(const Decode8Args& a, const bsa_kv_cache8* c, cudaStream_t s) {
  CUtensorMap tk, tv;
  const long long bh = static_cast<long long>(c->B) * c->Hh;
  const long long crows = bh * c->max_blocks * kBlk;
  if (!make_map8(&tk, c->k, crows, D) || !make_map8(&tv, c->v, crows, D)) return BSA_ERR_CUDA;
  const int smem = DecodeLayout<D>::kAlloc;
  auto go = [&](void (*kernel)(const CUtensorMap, const CUtensorMap, Decode8Args)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return BSA_ERR_CUDA;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(bh * a.tiles), a.n_split),
                      dim3(kDecThreads), static_cast<size_t>(smem), s, tk, tv, a);
  };
  BSA_TRY(a.rows <= AttnWarp8<D>::kRows ? go(decode8_kernel<D, AttnWarp8<D>>)
                                        : go(decode8_kernel<D, AttnWarp16<D>>));
  if (a.n_split == 1) return BSA_OK;
  return launch_pdl(decode8_join_kernel<D>, dim3(static_cast<unsigned>(bh), a.rows),
                    dim3(kJoinWarps * 32), 0, s, a);
}

}  // namespace bsa

using namespace bsa;

extern "C" bsa_status bsa_kv8_attn_decode_workspace_size(int B, int Hq, int Hh, int D, int n_tok,
                                                         int n_sel, size_t* bytes) {
  if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
  DecodeShape sh;
  BSA_TRY(decode_shape(B, Hq, Hh, D, n_tok, n_sel, &sh));
  *bytes = sh.bytes;
  return BSA_OK;
}

extern "C" bsa_status bsa_kv8_attn_decode(const void* q_tok, const bsa_kv_cache8* c, int Hq,
                                          int n_tok, const int32_t* idx, const int32_t* cnt,
                                          int max_sel, float sm_scale, void* o_tok, float* lse,
                                          void* workspace, size_t ws_bytes, int32_t* d_err,
                                          void* stream) {
  if (q_tok == nullptr || c == nullptr || o_tok == nullptr || lse == nullptr || c->k == nullptr ||
      c->v == nullptr || c->block_valid == nullptr || c->k_scale == nullptr ||
      c->v_scale == nullptr || (idx == nullptr) != (cnt == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (c->B <= 0 || c->Hh <= 0 || c->max_blocks <= 0 || c->n_blocks < 0 ||
      c->n_blocks > c->max_blocks || (idx != nullptr && max_sel <= 0) || !(sm_scale == sm_scale))
    return BSA_ERR_INVALID_ARG;
  if (idx != nullptr && max_sel > (1 << 30)) return BSA_ERR_SHAPE;
  if (!aligned16(q_tok) || !aligned16(c->k) || !aligned16(c->v) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return BSA_ERR_INVALID_ARG;
  const int n_sel = idx != nullptr ? max_sel : c->n_blocks;
  DecodeShape sh;
  BSA_TRY(decode_shape(c->B, Hq, c->Hh, c->D, n_tok, n_sel, &sh));
  const long long crows = static_cast<long long>(c->B) * c->Hh * c->max_blocks * kBlk;
  if (crows >= (1LL << 31)) return BSA_ERR_SHAPE;
  if (sh.bytes > 0 && (workspace == nullptr || ws_bytes < sh.bytes)) return BSA_ERR_CAPACITY;
  if (!device_is_sm100()) return BSA_ERR_UNSUPPORTED;
  Decode8Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q_tok);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.block_valid = c->block_valid;
  a.idx = idx;
  a.cnt = cnt;
  a.o = static_cast<__nv_bfloat16*>(o_tok);
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + sh.o_bytes);
  a.d_err = d_err;
  a.Hq = Hq;
  a.Hh = c->Hh;
  a.group = Hq / c->Hh;
  a.n_tok = n_tok;
  a.rows = sh.rows;
  a.tiles = sh.tiles;
  a.n_split = sh.n_split;
  a.n_sel = n_sel;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  return c->D == 128 ? launch_decode<128>(a, c, as_stream(stream))
                     : launch_decode<64>(a, c, as_stream(stream));
}
