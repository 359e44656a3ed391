// kv8_attn.cu - bsa_kv8_attn: indexed block-sparse attention over the 8-bit
// cache.  One CTA per (batch, query head, query block); each of its eight
// warps owns 16 query rows and walks the route by itself (attn8_warp.cuh).
#include "common.cuh"
#include "attn8_warp.cuh"

namespace bsa {

struct Attn8Args {
  const __nv_bfloat16* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_valid;
  const int32_t* q_valid;
  const int32_t* idx;
  const int32_t* cnt;
  __nv_bfloat16* o;
  float* lse;
  int32_t* d_err;
  int Hq, Hh, group;
  int n_q_blocks, max_sel, max_blocks, n_blocks;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(256)
attn8_simple_kernel(Attn8Args a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const long long item = blockIdx.x;
  const int j = static_cast<int>(item % a.n_q_blocks);
  const long long bq = item / a.n_q_blocks;
  const long long b = bq / a.Hq;
  const long long bh = b * a.Hh + (bq % a.Hq) / a.group;
  const long long route = bh * a.n_q_blocks + j;
  int n = a.cnt[route];
  if (n < 0 || n > a.max_sel) {
    report(a.d_err, BSA_DEV_BAD_COUNT);
    n = n < 0 ? 0 : a.max_sel;
  }
  const long long row = item * kBlk + warp * 16 + g;
  AttnWarp<D> w;
  w.init();
  w.load_q(a.q + row * D, a.q + (row + 8) * D, a.scale_log2);
  for (int i = 0; i < n; ++i) {
    int blk = a.idx[route * a.max_sel + i];
    if (blk < 0 || blk >= a.n_blocks) {
      report(a.d_err, BSA_DEV_BAD_INDEX);
      blk = 0;
    }
    int valid = a.block_valid[blk];
    if (valid < 1 || valid > kBlk) {
      report(a.d_err, BSA_DEV_BAD_VALID);
      valid = valid < 1 ? 1 : kBlk;
    }
    const long long at = bh * a.max_blocks + blk;
    const float ks = checked_scale(a.k_scale[at], a.d_err);
    const float vs = checked_scale(a.v_scale[at], a.d_err);
    const float vlog2 = log2f(vs), vinv = 1.f / vs;
    for (int first = 0; first < valid; first += 16) {
      typename AttnWarp<D>::Keys x;
      w.load_keys(a.k + at * kBlk * D, a.v + at * kBlk * D, first, valid, x);
      w.step(x, first, valid, ks, vlog2, vinv);
    }
  }
  w.finish();
  const int q_valid = a.q_valid != nullptr ? a.q_valid[j] : kBlk;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const bool have = warp * 16 + g + r * 8 < q_valid && w.m[r] > -INFINITY;
    const float inv = have ? 1.f / w.l[r] : 0.f;
    __nv_bfloat16* out = a.o + (row + r * 8) * D;
#pragma unroll
    for (int i = 0; i < AttnWarp<D>::kTiles; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        out[(2 * t + e) * (D / 8) + i] =
            __float2bfloat16(have ? w.o[i][2 * r + e] * inv : 0.f);
    }
    if (t == 0)
      a.lse[row + r * 8] =
          have ? (w.m[r] + log2f(w.l[r])) * 0.6931471805599453f : -INFINITY;
  }
}

bool device_is_sm100();

}  // namespace bsa

using namespace bsa;

extern "C" bsa_status bsa_kv8_attn(const void* q_blk, const bsa_kv_cache8* c, int Hq,
                                   const int32_t* q_valid, const int32_t* idx, const int32_t* cnt,
                                   int n_q_blocks, int max_sel, float sm_scale, void* o_blk,
                                   float* lse, int32_t* d_err, void* stream) {
  if (q_blk == nullptr || c == nullptr || idx == nullptr || cnt == nullptr || o_blk == nullptr ||
      lse == nullptr || c->k == nullptr || c->v == nullptr || c->block_valid == nullptr ||
      c->k_scale == nullptr || c->v_scale == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (c->B <= 0 || c->Hh <= 0 || Hq <= 0 || n_q_blocks <= 0 || max_sel <= 0 ||
      c->max_blocks <= 0 || c->n_blocks < 0 || c->n_blocks > c->max_blocks ||
      !(sm_scale == sm_scale))
    return BSA_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return BSA_ERR_UNSUPPORTED;
  if (Hq % c->Hh != 0) return BSA_ERR_SHAPE;
  if (!aligned16(q_blk) || !aligned16(o_blk) || !aligned16(c->k) || !aligned16(c->v))
    return BSA_ERR_INVALID_ARG;
  const long long items = static_cast<long long>(c->B) * Hq * n_q_blocks;
  const long long crows = static_cast<long long>(c->B) * c->Hh * c->max_blocks * kBlk;
  if (items * kBlk >= (1LL << 31) || crows >= (1LL << 31)) return BSA_ERR_SHAPE;
  if (!device_is_sm100()) return BSA_ERR_UNSUPPORTED;
  Attn8Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q_blk);
  a.k = static_cast<const uint8_t*>(c->k);
  a.v = static_cast<const uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.block_valid = c->block_valid;
  a.q_valid = q_valid;
  a.idx = idx;
  a.cnt = cnt;
  a.o = static_cast<__nv_bfloat16*>(o_blk);
  a.lse = lse;
  a.d_err = d_err;
  a.Hq = Hq;
  a.Hh = c->Hh;
  a.group = Hq / c->Hh;
  a.n_q_blocks = n_q_blocks;
  a.max_sel = max_sel;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  const dim3 grid(static_cast<unsigned>(items));
  cudaStream_t s = as_stream(stream);
  return c->D == 128 ? launch_pdl(attn8_simple_kernel<128>, grid, dim3(256), 0, s, a)
                     : launch_pdl(attn8_simple_kernel<64>, grid, dim3(256), 0, s, a);
}
