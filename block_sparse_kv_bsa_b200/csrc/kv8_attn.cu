// kv8_attn.cu - bsa_kv8_attn: indexed block-sparse attention over the 8-bit
// cache, on tcgen05.
//
// One CTA computes one (batch, query head, query block); a selected block is
// one 128-key tile.  The schedule of the two products and the softmax is
// attn_sm100.cu's; what differs is how 8-bit operands reach the tensor core:
//
//   S = Q K^T  runs on 8-bit operands (kind::f8f6f4), K tiles straight from the
//     cache.  A bf16 has 8 significant bits, an e4m3 code 4 and an e5m2 code 3:
//     with q scaled by a power of two per row, q = q1 + q2 with q1 = e4m3(q) and
//     q2 = e5m2(q - q1) is exact while q1 is a normal e4m3 (the rest of an 8-bit
//     significand after its nearest 4-bit one is at most 8 units, and 0 to 8 all
//     have 3 bits).  The row's largest is scaled to [2^7, 2^8) and e4m3 is normal
//     from 2^-6 on, so that holds for elements down to 2^-13 of the largest;
//     below, q1 has the step 2^-9 and the error is at most 2^-14, 2^-21 of the
//     largest (for rows whose largest is 2^-119 or more: the scale is no
//     subnormal).  Two 8-bit products cost what one bf16 product costs, and K
//     needs no conversion.
//   O += P V  runs on f16 operands: P needs more range than e4m3 has (many
//     small weights beside a large one would be rounded away), so a warpgroup
//     converts each V tile from e4m3 to f16 (exact) in shared memory.
//
// Scales: see attn8_warp.cuh.  The key scale and the row's power of two go into
// the exponent's factor, the value scale into its offset (log2 v), and the row
// sum of a tile is divided by v once.
//
// Tensor memory (512 columns): [0,384) three S buffers, P_t (f16 pairs) over the
// first 64 columns of its S; [384, 384 + D) O.
//
// Warp roles (512 threads; setmaxnreg moves registers to the softmax):
//   warp 0      TMA producer: K tiles (three slots, swizzled) and V tiles (two
//               staging slots, plain bulk copies), V two tiles behind K
//   warp 1      tensor memory; issues O += P_t V_t
//   warp 2      issues S_t = Q K_t^T
//   warp 3      each tile's scales and valid count, 32 tiles at a time, checked
//               and as the other warps use them (read from global memory by
//               every softmax thread they cost 4 % of the call)
//   warps 4-11  softmax: two warpgroups, alternate tiles, a thread per row;
//               before that they split Q into its two 8-bit terms
//   warps 12-15 V tiles from e4m3 to f16 (rows past a block's valid count
//               become zero)
// Every wait is bounded, as in attn_sm100.cu.
#include <cuda_fp16.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "tma_host.cuh"

namespace bsa {

// 2D map over e4m3 [rows, D]: a 128-row tile per box, swizzled over its row.
bool make_map8(CUtensorMap* m, const void* base, long long rows, int D) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(D), kBlk};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kThreads8 = 512;
constexpr int kSoftmax8 = 256;
constexpr int kConvert8 = 128;
constexpr int kK8Slots = 3;
constexpr int kV8Slots = 2;
constexpr int kV16Slots = 3;
constexpr int kS8Bufs = 3;
constexpr int kK8Lead = 2;
constexpr uint32_t kColO8 = 384;
constexpr long long kWait8 = 1LL << 31;  // SM clocks (about a second)
constexpr float kBias = 7.f;       // log2 of the weight of a fresh row maximum
constexpr float kMoveAt = 15.f;    // a weight past 2^15 moves the reference
// Registers per thread of each warpgroup: 64 + 2 * 184 + 80 = 4 * 128, what
// the block is launched with.
constexpr int kRegsIssue = 64, kRegsSoftmax = 184, kRegsConvert = 80;

constexpr int kMetaTiles = 32;  // tiles of a half of the metadata ring

enum {
  A_Q_FULL = 0,                         // Q terms written (256 threads)
  A_K_FULL = 1,                         // + K slot
  A_K_EMPTY = A_K_FULL + kK8Slots,      // + K slot: its Q K^T is done
  A_V8_FULL = A_K_EMPTY + kK8Slots,     // + staging slot: codes landed
  A_V8_EMPTY = A_V8_FULL + kV8Slots,    // + staging slot: converted (128 threads)
  A_V_EMPTY = A_V8_EMPTY + kV8Slots,    // + V slot: its P V is done
  A_PV_READY = A_V_EMPTY + kV16Slots,   // + slot t % 3: P_t stored and V_t converted
  A_S_FULL = A_PV_READY + kV16Slots,    // + S buffer
  A_META_FULL = A_S_FULL + kS8Bufs,     // + half of the ring: 32 tiles' scales (32 threads)
  A_META_EMPTY = A_META_FULL + 2,       // + half: read by all 384 threads
  A_MMA_DONE = A_META_EMPTY + 2,        // + issuer
  A_COUNT = A_MMA_DONE + 2
};

template <int D>
struct Layout8 {
  static constexpr int kTile8 = kBlk * D;        // e4m3 tile
  static constexpr int kTile16 = kBlk * D * 2;   // f16 (bf16) tile
  static constexpr int kQ = 0;                   // the two 8-bit terms
  static constexpr int kK = kQ + 2 * kTile8;
  static constexpr int kV16 = kK + kK8Slots * kTile8;
  static constexpr int kV8 = kV16 + kV16Slots * kTile16;
  static constexpr int kBars = kV8 + kV8Slots * kTile8;
  static constexpr int kMisc = kBars + A_COUNT * 8;
  static constexpr int kTok = (kMisc + 64 + 15) & ~15;  // float [2 warpgroups][128 rows]
  static constexpr int kMeta = kTok + 2 * kBlk * 4;  // Meta [2][32]
  static constexpr int kTotal = kMeta + 2 * kMetaTiles * 16;
  static constexpr int kAlloc = kTotal + 1024;  // room to align to 1024
  static constexpr int kFin = kK;    // the epilogue's [2][2][128] floats: K slot 0
  static constexpr int kStage = kV16;  // and O as bf16: V slot 0
  static_assert(kAlloc <= 227 * 1024, "shared memory per CTA");
  static_assert(kTile8 >= 4 * kBlk * 4, "epilogue scratch fits in one K slot");
};

struct Attn8Args {
  const __nv_bfloat16* q;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_valid;
  const int32_t* q_valid;
  const int32_t* idx;
  const int32_t* cnt;
  float* lse;
  int32_t* d_err;
  int Hq, Hh, group;
  int n_q_blocks, max_sel, max_blocks, n_blocks;
  float scale_log2;  // |sm_scale| * log2 e
  int negate;        // sm_scale < 0: the sign goes into Q
};

__device__ __forceinline__ void bar_sync8(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive8(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// Shared-memory accesses by 32-bit address (the aligned base pointer is a
// generic one to the compiler), kept in their place among the barrier
// operations.
__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ int lds_i(uint32_t addr) {
  int r;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ int meta_half(int t) { return (t / kMetaTiles) & 1; }
__device__ __forceinline__ void sts_f(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// D[tmem] (+)= A[smem] * B[smem]^T on e4m3 operands (K = 32 per instruction).
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor with type codes 0 for both operands (e4m3 for
// kind::f8f6f4, f16 for kind::f16; 1 is e5m2), fp32 out, A K-major.
constexpr uint32_t idesc_0(int M, int N, int b_mn, uint32_t a_type = 0) {
  return (1u << 4) | (a_type << 7) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// K-major e4m3 tile of D bytes a row: 128-byte swizzle, or 64-byte for D = 64.
template <int D>
__device__ __forceinline__ uint64_t e4m3_desc(uint32_t saddr) {
  uint64_t d = smem_desc(saddr, 16, 8 * D);
  if (D == 64) d = (d & ~(7ull << 61)) | (4ull << 61);
  return d;
}

// 16-byte chunk c of row r in that layout.
template <int D>
__device__ __forceinline__ uint32_t e4m3_chunk(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ int clamp_block(const Attn8Args& a, int blk) {
  return static_cast<unsigned>(blk) < static_cast<unsigned>(a.n_blocks) ? blk : 0;
}

// Half a query row (D / 2 elements) as its e4m3 and e5m2 terms in shared
// memory; returns the row's scale.  All 256 softmax threads take part.
template <int D>
__device__ __forceinline__ float split_query(const Attn8Args& a, long long item, int g, int r,
                                             uint8_t* q_terms, uint32_t tok) {
  const __nv_bfloat16* src = a.q + (item * kBlk + r) * D + g * (D / 2);
  uint4 raw[D / 16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    raw[i] = ld_nc_v4(src + i * 8);
    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = fabsf(bf16lo(u[e])), y = fabsf(bf16hi(u[e]));
      // A non-finite element counts as none here and becomes NaN below.
      amax = max3(amax, x <= 3.402823466e38f ? x : 0.f, y <= 3.402823466e38f ? y : 0.f);
    }
  }
  sts_f(tok + (g * kBlk + r) * 4, amax);
  bar_sync8(9, kSoftmax8);
  amax = fmaxf(lds_f(tok + r * 4), lds_f(tok + (kBlk + r) * 4));
  bar_sync8(9, kSoftmax8);  // tok is the softmax's from here on
  // Largest magnitude to [2^7, 2^8); a zero row is not scaled.
  int e = (__float_as_int(amax) >> 23) - 127 - 7;
  e = amax > 0.f ? (e < -126 ? -126 : e) : 0;
  const float scale = __int_as_float((e + 127) << 23);
  float inv = 1.f / scale;  // exact
  if (a.negate) inv = -inv;
  auto value = [&](float x) {
    return fabsf(x) <= 3.402823466e38f ? x * inv : __int_as_float(0x7fffffff);
  };
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {  // 16 elements
    uint32_t w1[4], w2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4& v = raw[2 * c + k / 2];
      const uint32_t lo = k % 2 ? v.z : v.x, hi = k % 2 ? v.w : v.y;
      const float x[4] = {value(bf16lo(lo)), value(bf16hi(lo)), value(bf16lo(hi)),
                          value(bf16hi(hi))};
      w1[k] = pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16);
      const uint32_t f0 = e4m3_lo_f16x2(w1[k]), f1 = e4m3_hi_f16x2(w1[k]);
      const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&f0));
      const float2 y1 = __half22float2(*reinterpret_cast<const __half2*>(&f1));
      w2[k] = pack_e5m2x2(x[0] - y0.x, x[1] - y0.y) |
              (pack_e5m2x2(x[2] - y1.x, x[3] - y1.y) << 16);
    }
    const uint32_t at = e4m3_chunk<D>(r, g * (D / 32) + c);
    *reinterpret_cast<uint4*>(q_terms + at) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    *reinterpret_cast<uint4*>(q_terms + kBlk * D + at) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
  }
  return scale;
}

template <int D>
__global__ void __launch_bounds__(kThreads8, 1)
attn8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_o,
             Attn8Args a) {
  using L = Layout8<D>;
  constexpr int kBoxes = D / 64;  // 64-column boxes of an f16 tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const long long item = blockIdx.x;  // ((b*Hq + hq)*n_q_blocks + j)
  const int j = static_cast<int>(item % a.n_q_blocks);
  const long long bq = item / a.n_q_blocks;
  const long long bh = (bq / a.Hq) * a.Hh + (bq % a.Hq) / a.group;  // cache head
  const long long route_row = bh * a.n_q_blocks + j;

  if (threadIdx.x == 0) {
    for (int i = 0; i < A_COUNT; ++i) {
      uint32_t count = 1;
      if (i == A_Q_FULL) count = kSoftmax8;
      if (i >= A_V8_EMPTY && i < A_V8_EMPTY + kV8Slots) count = kConvert8;
      if (i >= A_META_FULL && i < A_META_FULL + 2) count = 32;
      if (i >= A_META_EMPTY && i < A_META_EMPTY + 2) count = kSoftmax8 + kConvert8;
      if (i >= A_PV_READY && i < A_PV_READY + kV16Slots) count = kSoftmax8 / 2 + kConvert8;
      mbar_init(&bars[i], count);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();  // global memory only after the predecessor grid completed
  pdl_trigger();
  int n = a.cnt[route_row];
  if (n < 0 || n > a.max_sel) {
    report(a.d_err, BSA_DEV_BAD_COUNT);
    n = n < 0 ? 0 : a.max_sel;
  }
  const int32_t* route = a.idx + route_row * a.max_sel;

  if (warp < 4) {
    regs_dec<kRegsIssue>();
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        int k_issued = 0, v_issued = 0;
        bool ok = true;
        auto block_at = [&](int t) {
          const int blk = route[t];
          if (blk < 0 || blk >= a.n_blocks) {
            report(a.d_err, BSA_DEV_BAD_INDEX);
            return 0;
          }
          return blk;
        };
        // Step s issues K_s (while s < n), then V_{s - kK8Lead}.
        for (int step = 0; ok && step < n + kK8Lead; ++step) {
          if (step < n) {
            const int t = step, sl = t % kK8Slots;
            const int row = static_cast<int>((bh * a.max_blocks + block_at(t)) * kBlk);
            if (t >= kK8Slots)
              ok = mbar_wait_bounded(&bars[A_K_EMPTY + sl], ((t / kK8Slots) - 1) & 1, s_abort,
                                     kWait8);
            if (!ok) break;
            mbar_expect_tx(&bars[A_K_FULL + sl], L::kTile8);
            tma_load_2d(sm + L::kK + sl * L::kTile8, &tm_k, 0, row, &bars[A_K_FULL + sl]);
            k_issued = t + 1;
          }
          const int t = step - kK8Lead;
          if (t >= 0 && t < n) {
            const int sl = t % kV8Slots;
            const long long at = (bh * a.max_blocks + block_at(t)) * L::kTile8;
            if (t >= kV8Slots)
              ok = mbar_wait_bounded(&bars[A_V8_EMPTY + sl], ((t / kV8Slots) - 1) & 1, s_abort,
                                     kWait8);
            if (!ok) break;
            mbar_expect_tx(&bars[A_V8_FULL + sl], L::kTile8);
            bulk_load(sm + L::kV8 + sl * L::kTile8, a.v + at, L::kTile8, &bars[A_V8_FULL + sl]);
            v_issued = t + 1;
          }
        }
        if (!ok) {
          report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
          *s_abort = 1;
        }
        // Drain: every copy this warp issued must land before the CTA exits.
        for (int sl = 0; sl < kK8Slots; ++sl) {
          int last = -1;
          for (int t = sl; t < k_issued; t += kK8Slots) last = t;
          if (last >= 0)
            mbar_wait_bounded(&bars[A_K_FULL + sl], (last / kK8Slots) & 1, nullptr, kWait8);
        }
        for (int sl = 0; sl < kV8Slots; ++sl) {
          int last = -1;
          for (int t = sl; t < v_issued; t += kV8Slots) last = t;
          if (last >= 0)
            mbar_wait_bounded(&bars[A_V8_FULL + sl], (last / kV8Slots) & 1, nullptr, kWait8);
        }
      }
    } else if (warp == 3) {
      // ---------------- scales and valid counts ----------------
      bool ok = true;
      for (int b = 0; ok && b * kMetaTiles < n; ++b) {
        const int t = b * kMetaTiles + lane;
        int valid = kBlk;
        float ks = 1.f, vs = 1.f;
        if (t < n) {
          const int blk = clamp_block(a, route[t]);
          valid = a.block_valid[blk];
          ks = checked_k_scale(a.k_scale[bh * a.max_blocks + blk], a.d_err);
          vs = checked_v_scale(a.v_scale[bh * a.max_blocks + blk], a.d_err);
          if (valid < 1 || valid > kBlk) {
            report(a.d_err, BSA_DEV_BAD_VALID);
            valid = valid < 1 ? 1 : kBlk;
          }
        }
        if (b >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_META_EMPTY + (b & 1)],
                                                         ((b >> 1) - 1) & 1, s_abort, kWait8));
        if (!ok) break;
        sts_v4(smem_u32(sm + L::kMeta) + ((b & 1) * kMetaTiles + lane) * 16,
               make_uint4(__float_as_uint(ks), __float_as_uint(log2f(vs)),
                          __float_as_uint(1.f / vs), static_cast<uint32_t>(valid)));
        mbar_arrive(&bars[A_META_FULL + (b & 1)]);
      }
      if (!ok && lane == 0) {
        report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
        *s_abort = 1;
      }
    } else if ((warp == 1 || warp == 2) && n > 0) {
      // ---------------- MMA issuers ----------------
      bool ok = true;
      if (warp == 2) {
        constexpr uint32_t kIdQ1 = idesc_0(128, 128, 0), kIdQ2 = idesc_0(128, 128, 0, 1);
        const uint64_t q_desc = e4m3_desc<D>(smem_u32(sm + L::kQ));
        const uint64_t k_desc0 = e4m3_desc<D>(smem_u32(sm + L::kK));
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_Q_FULL], 0, s_abort, kWait8));
        for (int t = 0; ok && t < n; ++t) {
          const int sl = t % kK8Slots;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_K_FULL + sl], (t / kK8Slots) & 1,
                                                         s_abort, kWait8));
          if (ok && t >= kS8Bufs)  // the P V that read P from this S buffer
            ok = __all_sync(0xffffffffu,
                            mbar_wait_bounded(&bars[A_V_EMPTY + t % kV16Slots],
                                              ((t / kV16Slots) - 1) & 1, s_abort, kWait8));
          if (!ok) break;
          tc_fence_after();
          const uint64_t k_desc = desc_add(k_desc0, sl * (L::kTile8 >> 4));
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 2 * (D / 32); ++i) {
              const int kk = i % (D / 32), term = i / (D / 32);
              mma_f8_ss(tmem + (t % kS8Bufs) * 128,
                        desc_add(q_desc, (term * L::kTile8 + kk * 32) >> 4),
                        desc_add(k_desc, (kk * 32) >> 4), term ? kIdQ2 : kIdQ1, i > 0 ? 1u : 0u);
            }
            tc_commit(&bars[A_K_EMPTY + sl]);
            tc_commit(&bars[A_S_FULL + t % kS8Bufs]);
          }
          __syncwarp();
        }
      } else {
        constexpr uint32_t kIdPV = idesc_0(128, D, 1);
        const uint64_t v_desc0 = smem_desc(smem_u32(sm + L::kV16), kBlk * 128, 1024);
        for (int i = 0; ok && i < n; ++i) {
          const int sl = i % kV16Slots;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_PV_READY + sl],
                                                         (i / kV16Slots) & 1, s_abort, kWait8));
          if (!ok) break;
          tc_fence_after();
          const uint32_t p_col = tmem + (i % kS8Bufs) * 128;
          const uint64_t v_desc = desc_add(v_desc0, sl * (L::kTile16 >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kBlk / 16; ++kk)
              tc_mma_ts(tmem + kColO8, p_col + kk * 8, desc_add(v_desc, (kk * 2048) >> 4), kIdPV,
                        (i > 0 || kk > 0) ? 1u : 0u);
            tc_commit(&bars[A_V_EMPTY + sl]);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) {
        report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
        *s_abort = 1;
      }
      // Drain: all MMAs issued by lane 0 complete before TMEM is freed.
      if (lane == 0) {
        tc_commit(&bars[A_MMA_DONE + (warp - 1)]);
        mbar_wait_bounded(&bars[A_MMA_DONE + (warp - 1)], 0, nullptr, kWait8);
      }
      __syncwarp();
    }
  } else if (warp >= 12) {
    // ---------------- V tiles to f16 ----------------
    // A thread turns 8 codes into one 16-byte chunk of f16 per step: chunk c of
    // row r goes to position c ^ (r % 8) of its 64-column box (128 rows x 128
    // bytes), the swizzled tile the P V reads.  Eight lanes write eight
    // different positions, and a thread's steps are whole multiples of 8
    // rows apart, so its addresses differ by a constant.
    regs_dec<kRegsConvert>();
    const int i0 = threadIdx.x - 384;
    constexpr int kRowChunks = D / 8;
    constexpr int kRowStep = kConvert8 / kRowChunks;
    constexpr int kPer = kBlk / kRowStep;  // chunks per thread
    const int c = i0 & (kRowChunks - 1), r0 = i0 / kRowChunks;
    const uint32_t src0 = smem_u32(sm + L::kV8) + i0 * 8;
    const uint32_t dst0 = smem_u32(sm + L::kV16) + (c >> 3) * (kBlk * 128) + r0 * 128 +
                          (((c & 7) ^ (r0 & 7)) << 4);
    bool ok = true;
    for (int t = 0; ok && t < n; ++t) {
      if (t % kMetaTiles == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_META_FULL + meta_half(t)],
                                                       (t / (2 * kMetaTiles)) & 1, s_abort,
                                                       kWait8));
        if (!ok) break;
      }
      const int valid = lds_i(smem_u32(sm + L::kMeta) + (t % (2 * kMetaTiles)) * 16 + 12);
      if (t % kMetaTiles == kMetaTiles - 1) mbar_arrive(&bars[A_META_EMPTY + meta_half(t)]);
      const int s8 = t % kV8Slots, sl = t % kV16Slots;
      // Three orders keep the staging slot whole.  Every lane waits itself: its
      // acquire makes the copied bytes visible to it.  The loads are volatile, so
      // they stay between the wait and the arrival.  And a proxy fence stands
      // before the arrival: the refill writes the slot through the async proxy,
      // and the arrival alone orders these reads before generic accesses only.
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_V8_FULL + s8], (t / kV8Slots) & 1,
                                                     s_abort, kWait8));
      if (!ok) break;
      const uint32_t src = src0 + s8 * L::kTile8;
      uint2 x[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) x[u] = lds_v2(src + u * (kConvert8 * 8));
      fence_proxy_async_smem();
      mbar_arrive(&bars[A_V8_EMPTY + s8]);
      if (t >= kV16Slots) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_V_EMPTY + sl],
                                                       ((t / kV16Slots) - 1) & 1, s_abort, kWait8));
        if (!ok) break;
      }
      if (valid < kBlk) {
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (r0 + u * kRowStep >= valid) x[u] = make_uint2(0, 0);
      }
      const uint32_t dst = dst0 + sl * L::kTile16;
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        sts_v4(dst + u * (kRowStep * 128),
               make_uint4(e4m3_lo_f16x2(x[u].x), e4m3_hi_f16x2(x[u].x), e4m3_lo_f16x2(x[u].y),
                          e4m3_hi_f16x2(x[u].y)));
      fence_proxy_async_smem();
      mbar_arrive(&bars[A_PV_READY + sl]);
    }
    if (!ok) {
      report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
      *s_abort = 1;
    }
  } else {
    // ---------------- softmax / epilogue (warps 4..11) ----------------
    // The reference exponent of tile t is decided in tile order and handed
    // between the warpgroups as in attn_sm100.cu.
    regs_inc<kRegsSoftmax>();
    const int g = (warp - 4) >> 2;           // warpgroup: 0 or 1
    const int wq = warp & 3;                 // TMEM lane window of this warp
    const int r = wq * 32 + lane;            // query row owned by this thread
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tok = smem_u32(sm + L::kTok);  // float [2 warpgroups][128 rows]
    const uint32_t tok_mine = tok + (g * kBlk + r) * 4, tok_other = tok + ((g ^ 1) * kBlk + r) * 4;
    const int bar_in = 1 + (g ^ 1) * 4 + wq;
    const int bar_out = 1 + g * 4 + wq;

    const float row_scale =
        split_query<D>(a, item, g, r, sm + L::kQ, tok) * a.scale_log2;
    fence_proxy_async_smem();
    mbar_arrive(&bars[A_Q_FULL]);

    float m_last = -INFINITY;  // reference of this warpgroup's running sum
    float l = 0.f;
    bool ok = true;
    for (int t = g; t < n; t += 2) {
      if (t % kMetaTiles == g && ok)
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_META_FULL + meta_half(t)],
                                                       (t / (2 * kMetaTiles)) & 1, s_abort,
                                                       kWait8));
      uint4 meta = make_uint4(__float_as_uint(1.f), 0, __float_as_uint(1.f), kBlk);
      if (ok) meta = lds_v4(smem_u32(sm + L::kMeta) + (t % (2 * kMetaTiles)) * 16);
      if (t % kMetaTiles == kMetaTiles - 2 + g) mbar_arrive(&bars[A_META_EMPTY + meta_half(t)]);
      // Never zero (sm_scale = 0, or underflow): a masked key's -inf stays -inf.
      const float factor = fmaxf(row_scale * __uint_as_float(meta.x), 1.1754944e-38f);
      const float vlog2 = __uint_as_float(meta.y), vinv = __uint_as_float(meta.z);
      const int valid = static_cast<int>(meta.w);
      const uint32_t s_col = static_cast<uint32_t>(t % kS8Bufs) * 128;

      float s[kBlk];
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[A_S_FULL + t % kS8Bufs],
                                                       (t / kS8Bufs) & 1, s_abort, kWait8));
      if (ok) {
        tc_fence_after();
        tmem_ld_cols<kBlk>(tmem + lane_base + s_col, s);
      } else {
#pragma unroll
        for (int c = 0; c < kBlk; ++c) s[c] = 0.f;
      }
      if (valid < kBlk) {  // tail block of a chunk: mask its pad keys
#pragma unroll
        for (int c = 0; c < kBlk; ++c)
          if (c >= valid) s[c] = -INFINITY;
      }
      float mq[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mq[k] = max3(s[k], s[k + 4], s[k + 8]);
#pragma unroll
      for (int c = 12; c + 4 < kBlk; c += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mq[k] = max3(mq[k], s[c + k], s[c + 4 + k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mq[k] = fmaxf(mq[k], s[kBlk - 4 + k]);
      const float mx = fmaf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])), factor, vlog2);

      // Reference of tile t, decided in tile order.
      float m_prev = -INFINITY;
      if (t > 0) {
        bar_sync8(bar_in, 64);
        m_prev = lds_f(tok_other);
      }
      // (the difference, which is exact for near values: m_prev + 15 rounds to
      // m_prev + 16 from 2^24 on, and a weight of 2^16 is no f16)
      const float m_t = (t == 0 || mx - m_prev > kMoveAt) ? mx - kBias : m_prev;
      if (t + 1 < n) {
        sts_f(tok_mine, m_t);
        bar_arrive8(bar_out, 64);
      }

      // P (f16 pairs) overwrites the S buffer it was computed from.
      float mul = factor, off = vlog2 - m_t;
      if (fabsf(mx) > 1048576.f) {
        // The maximum was rounded, the exponents below are not: past 2^20 the
        // difference could overflow a weight, so both take the same rounding.
#pragma unroll
        for (int c = 0; c < kBlk; ++c) s[c] = fmaf(s[c], factor, vlog2);
        mul = 1.f;
        off = -m_t;
      }
      const uint64_t scale2 = f2_pack(mul, mul);
      const uint64_t off2 = f2_pack(off, off);
      uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
      for (int q = 0; q < kBlk / 64; ++q) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[64 * q + 2 * c], s[64 * q + 2 * c + 1]), scale2, off2), x0,
                    x1);
          const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
          acc2[c & 1] = f2_add(acc2[c & 1], f2_pack(e0, e1));
          pk[c] = pack_f16x2(e0, e1);
        }
        if (ok) tmem_st32u(tmem + lane_base + s_col + 32 * q, pk);
      }
      float rq[4];
      f2_unpack(acc2[0], rq[0], rq[1]);
      f2_unpack(acc2[1], rq[2], rq[3]);
      const float rs = (rq[0] + rq[1]) + (rq[2] + rq[3]);
      if (m_t != m_last) {  // m_last = -inf scales the empty sum 0 by 0
        l *= ex2_approx(m_last - m_t);
        m_last = m_t;
      }
      l = fmaf(rs, vinv, l);

      // A row whose reference moved rescales O after the P V of tile t - 1
      // has completed and before this tile's P is released.
      if (ok && t > 0 && __any_sync(0xffffffffu, m_t != m_prev)) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&bars[A_V_EMPTY + (t - 1) % kV16Slots],
                                          ((t - 1) / kV16Slots) & 1, s_abort, kWait8));
        if (ok) {
          tc_fence_after();
          const float alpha = m_t != m_prev ? ex2_approx(m_prev - m_t) : 1.0f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld_cols<32>(tmem + lane_base + kColO8 + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(tmem + lane_base + kColO8 + c * 32, o);
          }
        }
      }
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[A_PV_READY + t % kV16Slots]);
    }
    if (!ok) {
      report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
      *s_abort = 1;
    }
    // Epilogue: merge the two running sums, then each warpgroup normalises
    // D/2 output columns; warpgroup 0 writes the LSE.
    const int q_valid = a.q_valid != nullptr ? a.q_valid[j] : kBlk;
    if (ok && n > 0 && g == ((n - 1) & 1)) {
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(&bars[A_V_EMPTY + (n - 1) % kV16Slots],
                                        ((n - 1) / kV16Slots) & 1, s_abort, kWait8));
      if (!ok) {
        report(a.d_err, BSA_DEV_WAIT_TIMEOUT);
        *s_abort = 1;
      }
    }
    tc_fence_before();
    bar_sync8(9, kSoftmax8);
    float* fin = reinterpret_cast<float*>(sm + L::kFin);  // [m, l][warpgroup][128 rows]
    fin[(0 * 2 + g) * kBlk + r] = m_last;
    fin[(1 * 2 + g) * kBlk + r] = l;
    bar_sync8(9, kSoftmax8);
    tc_fence_after();
    ok = __all_sync(0xffffffffu, ok && *s_abort == 0);
    const float m0 = fin[0 * kBlk + r], m1 = fin[1 * kBlk + r];
    const float m_fin = fmaxf(m0, m1);
    const bool live = ok && n > 0 && r < q_valid;
    float l_tot = 0.f;
    if (live)
      l_tot = fin[2 * kBlk + r] * (m0 == -INFINITY ? 0.f : ex2_approx(m0 - m_fin)) +
              fin[3 * kBlk + r] * (m1 == -INFINITY ? 0.f : ex2_approx(m1 - m_fin));
    const float inv_l = live ? 1.0f / l_tot : 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0.f;
      if (ok && n > 0) tmem_ld_cols<32>(tmem + lane_base + kColO8 + g * (D / 2) + c * 32, o);
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint4 v;
        v.x = pack_bf16x2(live ? o[e + 0] * inv_l : 0.f, live ? o[e + 1] * inv_l : 0.f);
        v.y = pack_bf16x2(live ? o[e + 2] * inv_l : 0.f, live ? o[e + 3] * inv_l : 0.f);
        v.z = pack_bf16x2(live ? o[e + 4] * inv_l : 0.f, live ? o[e + 5] * inv_l : 0.f);
        v.w = pack_bf16x2(live ? o[e + 6] * inv_l : 0.f, live ? o[e + 7] * inv_l : 0.f);
        const int col = g * (D / 2) + c * 32 + e;
        uint8_t* stage = sm + L::kStage + (col / 64) * (kBlk * 128);
        *reinterpret_cast<uint4*>(stage + r * 128 + ((((col % 64) / 8) ^ (r & 7)) * 16)) = v;
      }
    }
    if (g == 0)
      a.lse[item * kBlk + r] = live ? (m_fin + log2f(l_tot)) * 0.6931471805599453f : -INFINITY;
    fence_proxy_async_smem();
    bar_sync8(9, kSoftmax8);
    if (warp == 4 && elect_one()) {
      for (int bx = 0; bx < kBoxes; ++bx)
        tma_store_2d(&tm_o, bx * 64, static_cast<int>(item * kBlk),
                     sm + L::kStage + bx * (kBlk * 128));
      bulk_commit_group();
      bulk_wait_read_all();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// 2D map over bf16 [rows, D]: boxes of 128 rows x 64 columns.
bool make_map_out(CUtensorMap* m, const void* base, long long rows, int D) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
  cuuint32_t box[2] = {64, kBlk};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
bsa_status launch_attn8(const Attn8Args& a, const bsa_kv_cache8* c, void* o, long long items,
                        cudaStream_t s) {
  CUtensorMap tk, to;
  const long long crows = static_cast<long long>(c->B) * c->Hh * c->max_blocks * kBlk;
  if (!make_map8(&tk, c->k, crows, D) || !make_map_out(&to, o, items * kBlk, D))
    return BSA_ERR_CUDA;
  const int smem = Layout8<D>::kAlloc;
  if (cudaFuncSetAttribute(attn8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return BSA_ERR_CUDA;
  return launch_pdl(attn8_kernel<D>, dim3(static_cast<unsigned>(items)), dim3(kThreads8),
                    static_cast<size_t>(smem), s, tk, to, a);
}

}  // namespace

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
  a.v = static_cast<const uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.block_valid = c->block_valid;
  a.q_valid = q_valid;
  a.idx = idx;
  a.cnt = cnt;
  a.lse = lse;
  a.d_err = d_err;
  a.Hq = Hq;
  a.Hh = c->Hh;
  a.group = Hq / c->Hh;
  a.n_q_blocks = n_q_blocks;
  a.max_sel = max_sel;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  a.scale_log2 = (sm_scale < 0.f ? -sm_scale : sm_scale) * 1.4426950408889634f;
  a.negate = sm_scale < 0.f;
  cudaStream_t s = as_stream(stream);
  return c->D == 128 ? launch_attn8<128>(a, c, o_blk, items, s)
                     : launch_attn8<64>(a, c, o_blk, items, s);
}
