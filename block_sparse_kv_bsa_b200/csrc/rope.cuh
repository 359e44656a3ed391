// rope.cuh - rotary positions in registers.
//
// A row of D elements is handled in D/16 slots; a thread owns one slot of a
// row: two 16-byte vectors that hold eight whole pairs (or none), so a pair
// never crosses threads and a row may be turned in place.
//   interleaved   slot s: vectors s and s + D/16, four pairs in each
//   half, P % 8 = 0  slot s < P/8: vectors s and s + P/8, pairs 8s .. 8s + 7;
//                 the vectors past 2P, two a slot, are copied
// (neighbouring lanes take neighbouring vectors: with the two vectors of a slot
// side by side every load and store moved half sectors, 6 % of a rope call)
//   half, any P   the elements of pair i and i + P fall anywhere in their
//                 vectors: slot s owns elements 16s .. 16s + 15 of the output
//                 and fetches each element's partner by itself (kHalfAny)
// The angle is exact: phase[i] is the pair's frequency as a 64-bit fraction
// of a turn, p * phase mod 2^64 the fraction turned, whose top 32 bits (an
// error below 2^-32 turn) give its sine and cosine.
#pragma once

#include "common.cuh"

namespace bsa {

enum RopeMode { kRopeNone = 0, kRopeInterleaved = 1, kRopeHalf = 2, kRopeHalfAny = 3 };

struct RopeArgs {
  const uint64_t* phase;
  const int32_t* pos;   // [n_axes, B, N] or null
  long long pos_stride; // B * N
  int P, p0, p01;       // pairs in all, of axis 0, of axes 0 and 1
  int n_axes, inverse;
  int H, W;
  int o0, o1, o2;       // origin
  float amp;
};

struct TokenPos {
  int p[3];
};

// Positions of raster token `tok` of batch b; bN = b * N.
__device__ __forceinline__ TokenPos token_pos(const RopeArgs& r, long long bN, int tok) {
  TokenPos t;
  if (r.pos != nullptr) {
    const int32_t* q = r.pos + bN + tok;
    t.p[0] = __ldg(q);
    t.p[1] = r.n_axes == 3 ? __ldg(q + r.pos_stride) : 0;
    t.p[2] = r.n_axes == 3 ? __ldg(q + 2 * r.pos_stride) : 0;
  } else if (r.n_axes == 3) {
    const int row = tok / r.W;
    t.p[2] = tok - row * r.W;
    t.p[0] = row / r.H;
    t.p[1] = row - t.p[0] * r.H;
  } else {
    t.p[0] = tok;
    t.p[1] = t.p[2] = 0;
  }
  return t;
}

// cos and sin of a fraction of a turn (its top 32 bits).  The nearest quarter
// turn is split off exactly in integers; what is left, |x| <= pi / 4, goes into
// the Taylor series of sin through x^9 and of cos through x^8 (truncation
// below 2^-25), about 20 instructions.
__device__ __forceinline__ void turn_trig(uint32_t turn, float& c, float& s) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));
  const float x = static_cast<float>(rest) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float ps = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  ps = fmaf(ps, x2, 8.3333333e-3f);
  ps = fmaf(ps, x2, -1.6666667e-1f);
  const float sn = fmaf(ps * x2, x, x);
  float pc = fmaf(x2, 2.4801587e-5f, -1.3888889e-3f);
  pc = fmaf(pc, x2, 4.1666667e-2f);
  pc = fmaf(pc, x2, -0.5f);
  const float cs = fmaf(pc, x2, 1.f);
  const float u = quarter & 1 ? cs : sn, v = quarter & 1 ? sn : cs;
  s = __uint_as_float(__float_as_uint(u) ^ ((quarter & 2) << 30));
  c = __uint_as_float(__float_as_uint(v) ^ (((quarter + 1) & 2) << 30));
}

// A pair's frequency and the position it goes by.
struct PairPhase {
  uint64_t step;
  int axis;
  long long origin;
};
__device__ __forceinline__ PairPhase pair_phase(const RopeArgs& r, int i) {
  PairPhase f;
  f.step = __ldg(r.phase + i);
  f.axis = i < r.p0 ? 0 : (i < r.p01 ? 1 : 2);
  f.origin = f.axis == 0 ? r.o0 : (f.axis == 1 ? r.o1 : r.o2);
  return f;
}

// cos and sin of a pair (amplitude and direction applied).
__device__ __forceinline__ void pair_trig(const RopeArgs& r, const TokenPos& t, const PairPhase& f,
                                          float& c, float& s) {
  const int at = f.axis == 0 ? t.p[0] : (f.axis == 1 ? t.p[1] : t.p[2]);
  const uint64_t turn = static_cast<uint64_t>(at + f.origin) * f.step;
  turn_trig(static_cast<uint32_t>(turn >> 32), c, s);
  c *= r.amp;
  s *= r.inverse ? -r.amp : r.amp;
}

// The eight pairs of a slot; pairs at or past P are left alone.
struct SlotTrig {
  float c[8], s[8];
  int n;  // bit e: pair e of the slot is turned (half layout: all or none)
};

// Pair e of a slot whose vectors are va and vb.
template <int MODE>
__device__ __forceinline__ int slot_pair(int slot, int va, int vb, int e) {
  if (MODE == kRopeInterleaved) return e < 4 ? 4 * va + e : 4 * vb + e - 4;
  return slot * 8 + e;
}

// The angles of a slot for kRows tokens.
template <int MODE, int kRows>
__device__ __forceinline__ void slot_trig(const RopeArgs& r, const TokenPos (&t)[kRows], int slot,
                                          int va, int vb, SlotTrig (&g)[kRows]) {
#pragma unroll
  for (int i = 0; i < kRows; ++i) g[i].n = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pair = slot_pair<MODE>(slot, va, vb, e);
    if (pair < r.P) {
      const PairPhase f = pair_phase(r, pair);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        pair_trig(r, t[i], f, g[i].c[e], g[i].s[e]);
        g[i].n |= 1 << e;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        g[i].c[e] = 1.f;
        g[i].s[e] = 0.f;
      }
    }
  }
}

// The two vectors of a slot of a D-wide row.
template <int D, int MODE>
__device__ __forceinline__ void slot_vectors(int P, int slot, int& va, int& vb) {
  if (MODE == kRopeHalf && slot < P / 8) {
    va = slot;
    vb = slot + P / 8;
  } else if (MODE == kRopeInterleaved) {
    va = slot;
    vb = slot + D / 16;
  } else {
    // Half layout: P/8 slots have taken the first P/4 vectors, so the
    // copied ones are again two a slot, at 2s and 2s + 1.
    va = 2 * slot;
    vb = 2 * slot + 1;
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
  x[4] = bf16lo(v.z); x[5] = bf16hi(v.z); x[6] = bf16lo(v.w); x[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = x * c - y * s;
  y = x * s + y * c;
  x = a;
}

// Turn a slot's sixteen values a (vector va) and b (vector vb).
template <int MODE>
__device__ __forceinline__ void turn_slot(const SlotTrig& g, float (&a)[8], float (&b)[8]) {
  if (MODE == kRopeInterleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (g.n >> e & 1) turn_pair(a[2 * e], a[2 * e + 1], g.c[e], g.s[e]);
      if (g.n >> (e + 4) & 1) turn_pair(b[2 * e], b[2 * e + 1], g.c[e + 4], g.s[e + 4]);
    }
  } else if (MODE == kRopeHalf) {
    if (g.n != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn_pair(a[e], b[e], g.c[e], g.s[e]);
    }
  }
}

// kHalfAny: the output elements 16*slot .. 16*slot + 15 of `row`.
__device__ __forceinline__ void turn_slot_any(const RopeArgs& r, const TokenPos& t, int slot,
                                              const __nv_bfloat16* row, float (&a)[8],
                                              float (&b)[8]) {
#pragma unroll 1
  for (int e = 0; e < 16; ++e) {
    const int el = slot * 16 + e;
    float v = __bfloat162float(row[el]);
    if (el < 2 * r.P) {
      const bool second = el >= r.P;
      const int i = second ? el - r.P : el;
      const float w = __bfloat162float(row[second ? i : i + r.P]);
      float c, s;
      pair_trig(r, t, pair_phase(r, i), c, s);
      v = second ? w * s + v * c : v * c - w * s;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // registers: no indexed store
      if (e == k) a[k] = v;
      if (e == k + 8) b[k] = v;
    }
  }
}

// Heads per CTA for a grid of `others` CTAs per run of heads, `per_sm` of them
// resident on each of 148 SMs: the run whose waves of CTAs take the fewest
// head times, a CTA's start and angles counting as `start` heads.
inline int heads_per_cta(long long others, int Hh, int per_sm, double start) {
  int best = 1;
  double best_cost = -1.0;
  for (int heads = 1; heads <= Hh && heads <= 64; ++heads) {
    const long long ctas = others * ((Hh + heads - 1) / heads);
    const long long waves = (ctas + 148 * per_sm - 1) / (148 * per_sm);
    const double cost = static_cast<double>(waves) * (heads + start);
    if (best_cost < 0.0 || cost < best_cost) {
      best_cost = cost;
      best = heads;
    }
  }
  return best;
}

// The same for a chunk of `blocks` blocks whose K tiles (turned) and V tiles
// (moved; `tensors` = 2) go to CTAs of their own, K's first, one CTA to an SM:
// runs of heads for each, by the sum of the work over the SMs and the longest
// run that may start last.  In head tiles, a K run's start (tokens, angles,
// first loads) counts 2 and a V run's 1; the short V runs fill the SMs that K's
// leave idle.
struct HeadRuns {
  int heads[2];
};
inline HeadRuns head_runs(long long blocks, int Hh, int tensors) {
  HeadRuns best{{1, 1}};
  double best_cost = -1.0;
  for (int gk = 1; gk <= Hh && gk <= 32; ++gk) {
    const int hk = (Hh + gk - 1) / gk;
    const long long nk = blocks * ((Hh + hk - 1) / hk);
    const double k_work = static_cast<double>(blocks) * Hh + 2.0 * nk;
    const double k_time = static_cast<double>((nk + 147) / 148) * (hk + 2.0);
    for (int gv = 1; gv <= (tensors == 2 ? Hh : 1) && gv <= 32; ++gv) {
      const int hv = tensors == 2 ? (Hh + gv - 1) / gv : 0;
      const long long nv = tensors == 2 ? blocks * ((Hh + hv - 1) / hv) : 0;
      const double v_work = tensors == 2 ? static_cast<double>(blocks) * Hh + 1.0 * nv : 0.0;
      const double all = (k_work + v_work) / 148.0 + (tensors == 2 ? 0.5 * (hv + 1.0) : 0.0);
      const double cost = all > k_time ? all : k_time;
      if (best_cost < 0.0 || cost < best_cost) {
        best_cost = cost;
        best.heads[0] = hk;
        best.heads[1] = tensors == 2 ? hv : 1;
      }
    }
  }
  return best;
}

// What a CTA of such a grid works on.
struct RunAt {
  int which, b, j, h0, h1;
  bool first;  // of its block
  __device__ __forceinline__ RunAt(const HeadRuns& r, int nb, int B, int Hh) {
    const int groups0 = (Hh + r.heads[0] - 1) / r.heads[0];
    int x = blockIdx.x;
    const int k_ctas = groups0 * nb * B;
    which = x >= k_ctas;
    if (which) x -= k_ctas;
    j = x % nb;
    x /= nb;
    b = x % B;
    h0 = x / B * r.heads[which];
    h1 = min(h0 + r.heads[which], Hh);
    first = !which && b == 0 && h0 == 0;
  }
};
inline unsigned run_ctas(const HeadRuns& r, long long blocks, int Hh, int tensors) {
  long long n = blocks * ((Hh + r.heads[0] - 1) / r.heads[0]);
  if (tensors == 2) n += blocks * ((Hh + r.heads[1] - 1) / r.heads[1]);
  return static_cast<unsigned>(n);
}

// Checks a descriptor and fills the kernel's arguments; `mode` is how the
// kernels handle its layout.
bsa_status rope_args(const bsa_rope_desc* d, int B, int D, int T, int H, int W, RopeArgs* out,
                     int* mode);

}  // namespace bsa
