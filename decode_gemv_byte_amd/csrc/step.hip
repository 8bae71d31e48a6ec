// HIP kernels of libnwc for what a step does between its blocks and behind the
// last one, for gfx950 (CDNA4), and the C-ABI entry points that launch them:
//
//  * k_residual: the residual sum of a block with the norms before and after it.
//  * k_logprobs, k_logprobs_join: log probabilities of given tokens over a row of
//    logits, its entropy, and its k largest in order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "device_common.hpp"

namespace {

// Eight logits as they are loaded: FP32 rows begin at any multiple of 16 bytes, which is
// less than a vector of 8 floats asks for.
struct F32x8 {
  f32x4_t lo, hi;
};
static_assert(alignof(F32x8) == 16 && alignof(u32x4_t) == 16, "what nwc_token_logprobs checks");

// Sum over the wavefront, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  for (int x = 32; x; x /= 2) v += lane_xor(v, x);
  return v;
}

// -------------------------------------------------------------- k_residual ---

struct ResidualArgs {
  const void* x;
  void* x_out;
  const uint16_t *y, *y_weight, *gate, *weight;
  uint16_t* out;
  uint64_t ld_x, ld_x_out, ld_y, ld_gate, ld_out;
  float scale, eps;
  uint32_t tokens, cols8;  // cols / 8
};

__device__ __forceinline__ void unpack8(u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(v[j]);
    f[2 * j + 1] = bf16_hi(v[j]);
  }
}
__device__ __forceinline__ u32x4_t pack8(const float (&f)[8]) {
  return u32x4_t{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// A token by W wavefronts, P pieces of 8 values a lane, all of a row's values in
// registers between its loads and its stores: each is read once, before any of
// its lane's pieces is written.  Sums of squares are FP32; x', where it is BF16, is
// rounded when it is stored, and the norm takes it as it was before.
// Bound by HBM for a prompt: 16384 tokens of 4096, 537 MB, 102 us, 5.2 TB/s, what a large
// copy and read reach together; by one chain of loads, a sum and a store for a token:
// 2.8 us, of which an empty launch takes 2.5.
template <int W, int P, bool F32>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void k_residual(const ResidualArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;  // tokens that a workgroup has at a time
  __shared__ float sums[W == 1 ? 1 : 4][W];
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave);
  const uint32_t me = W == 1 ? lane : threadIdx.x;
  const float inv = 1.f / (8.f * static_cast<float>(a.cols8));
  int turn = 0;  // of the LDS rows: a sum's is not written again before the next but two
  auto total = [&](float v) {
    v = wave_sum(v);
    if constexpr (W > 1) {
      float(&s)[W] = sums[turn];
      turn = (turn + 1) % 4;
      if (lane == 0) s[wave] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) v += s[i];
    }
    return v;
  };
  // 1 / sqrt(mean(f^2) + eps) for P pieces, which are multiplied by a power of two
  // first where their squares leave FP32's range (or fall below it with no eps
  // beside them)
  auto rms = [&](float (&f)[P][8]) {
    auto squares = [&] {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(f[p][j], f[p][j], s);
      return total(s);
    };
    float sum = squares(), eps = a.eps;
    if (__builtin_expect(!(sum < INFINITY) || (sum < 0x1p-96f && eps < 0x1p-96f), 0)) {
      const float s = sum < 1.f ? 0x1p100f : 0x1p-75f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[p][j] *= s;
      sum = squares();
      eps = eps * s * s;
    }
    return 1.f / sqrtf(fmaf(sum, inv, eps));
  };
  for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * kRows + (W == 1 ? wave : 0); t < a.tokens;
       t += static_cast<uint64_t>(gridDim.x) * kRows) {
    float x[P][8];
    u32x4_t raw[P], gates[P];
    uint32_t at[P];
    bool on[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      at[p] = me + p * (W * kWave);
      on[p] = at[p] < a.cols8;
      raw[p] = gates[p] = u32x4_t{0, 0, 0, 0};
    }
    if constexpr (F32) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
        if (on[p]) {
          const f32x4_t* src = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.x) + t * a.ld_x + 8 * at[p]);
          lo = src[0];
          hi = src[1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[p][j] = lo[j];
          x[p][4 + j] = hi[j];
        }
      }
    } else {
      u32x4_t xr[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        xr[p] = u32x4_t{0, 0, 0, 0};
        if (on[p]) xr[p] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.x) + t * a.ld_x + 8 * at[p]);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) unpack8(xr[p], x[p]);
    }
    if (a.y) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (on[p]) raw[p] = *reinterpret_cast<const u32x4_t*>(a.y + t * a.ld_y + 8 * at[p]);
        if (on[p] && a.gate) gates[p] = *reinterpret_cast<const u32x4_t*>(a.gate + t * a.ld_gate + 8 * at[p]);
      }
      float u[P][8];
#pragma unroll
      for (int p = 0; p < P; ++p) unpack8(raw[p], u[p]);
      if (a.y_weight) {
        u32x4_t w[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          w[p] = u32x4_t{0, 0, 0, 0};
          if (on[p]) w[p] = *reinterpret_cast<const u32x4_t*>(a.y_weight + 8 * at[p]);
        }
        const float r = rms(u);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float g[8];
          unpack8(w[p], g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[p][j] = u[p][j] * r * g[j];
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float g[8];
        unpack8(gates[p], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[p][j] = fmaf(a.gate ? u[p][j] * g[j] : u[p][j], a.scale, x[p][j]);
      }
      if (a.x_out) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (!on[p]) continue;
          if constexpr (F32) {
            f32x4_t* dst = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.x_out) + t * a.ld_x_out + 8 * at[p]);
            dst[0] = f32x4_t{x[p][0], x[p][1], x[p][2], x[p][3]};
            dst[1] = f32x4_t{x[p][4], x[p][5], x[p][6], x[p][7]};
          } else {
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.x_out) + t * a.ld_x_out + 8 * at[p]) = pack8(x[p]);
          }
        }
      }
    }
    if (a.out) {
      u32x4_t w[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        w[p] = u32x4_t{0, 0, 0, 0};
        if (on[p]) w[p] = *reinterpret_cast<const u32x4_t*>(a.weight + 8 * at[p]);
      }
      // a lane without a piece holds zeros, also where x is infinite or NaN elsewhere
      const float r = rms(x);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float g[8];
        unpack8(w[p], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = x[p][j] * r * g[j];
        if (on[p]) *reinterpret_cast<u32x4_t*>(a.out + t * a.ld_out + 8 * at[p]) = pack8(g);
      }
    }
  }
}

// -------------------------------------------------------------- k_logprobs ---
//
// With c = scale log2(e) and M the row's largest logit: e_v = 2^((x_v - M) c), S =
// sum e_v, log p_v = (x_v - M) scale - ln S and the entropy ln S - ln 2 sum e_v
// (x_v - M) c / S, whose two terms are both positive.  One pass: every lane holds
// S and the weighted sum relative to a maximum of its own, which moves only when a
// logit outgrows it by 2^8, so the common piece rescales nothing.
//
// The k largest: each of 64 groups of lanes keeps the largest logit it saw.  The
// k-th largest of those 64 is a bound that at least k logits reach, and only
// lanes whose own largest reaches it look at their logits once more.  What they
// find (little over k for logits in no order; of those equal to the bound each
// wavefront's k lowest) is ranked by counting, each against all.  Where more is
// found than LDS has room for, or NaN stands in the row, k rounds of a largest
// below the last one take its place.
//
// 2048 rows of 128256 BF16 logits, 525 MB, k = 20: 123 us, 4.3 TB/s, bound by vector
// instructions (85 us of them: an exponential, two products and a maximum a logit) beside
// loads that take 85 by themselves; one row of 128256: 8.4 us and 5.4 for the join, both
// one chain of loads, sums over the workgroup and a ranking.

constexpr int kLpThreads = 512, kLpWaves = kLpThreads / kWave;
constexpr uint32_t kLpMaxK = 64, kLpMaxSplit = 32, kLpFound = 2048;
constexpr float kLowest = -3.402823466e+38f, kLowestC = -3e38f;
constexpr float kFar = 0x1p20f;   // maxima, times c, whose product's rounding is off by 2^-4 at most
constexpr float kGrow = 8.f;     // log2 of how far a logit may outgrow its lane's maximum
constexpr float kNoWeight = -16384.f;  // a power of two that is 0 in FP32, and finite: 0 times it is 0

struct LogprobsArgs {
  const void* logits;
  uint64_t ld;
  const int32_t* targets;
  float *logprobs, *entropy, *top_logprobs;
  int32_t* top_ids;
  uint32_t vocab, n_targets, k;
  uint32_t split, chunk;  // workgroups of a row, logits of each (a multiple of 8)
  float scale, c;         // c: scale log2(e)
  float* stats;           // workspace: {largest, S, weighted sum, 0} of each part
  uint64_t* tops;         // k keys of each part, descending
};

// The order of logits: value, the lower index first, NaN above all, -0 as 0.  Every NaN
// counts as the positive quiet one, above +infinity, so that a key is neither 0 nor all
// ones: 0 stands for none, and all ones is above every key.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = x != x ? 0x7FC00000u : __builtin_bit_cast(uint32_t, x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return static_cast<uint64_t>(ordered(x)) << 32 | (0xFFFFFFFFu - index);
}

// The largest of three, as fmaxf, which asks for one instruction more a value (a
// signalling NaN made quiet first).
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}

struct Stats {
  float m, s, a;  // maximum; sum of weights relative to it; sum of weight times log2 weight
  // relative to another maximum, no smaller
  __device__ __forceinline__ void move(float to, float c) {
    const float d = (m - to) * c, f = __builtin_amdgcn_exp2f(d);
    a = f * fmaf(s, fmaxf(d, kNoWeight), a);
    s *= f;
    m = to;
  }
};

// What a row's statistics come to.
struct RowOut {
  float m, log_s;
  bool none;  // no weight at all: every logit -infinity
  __device__ RowOut(const Stats& t) : m(t.m), log_s(logf(t.s)), none(t.s == 0.f) {}
  __device__ __forceinline__ float logprob(float x, float scale) const { return none ? -INFINITY : fmaf(x - m, scale, -log_s); }
};

template <bool F32>
__device__ __forceinline__ float logit(const LogprobsArgs& a, uint64_t row, uint32_t v) {
  return F32 ? static_cast<const float*>(a.logits)[row * a.ld + v]
             : __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[row * a.ld + v]) << 16);
}

template <bool F32>
__device__ void store_targets(const LogprobsArgs& a, uint64_t row, const RowOut& r, uint32_t threads) {
  for (uint32_t i = threadIdx.x; i < a.n_targets; i += threads) {
    const uint64_t at = row * a.n_targets + i;
    const uint32_t v = static_cast<uint32_t>(a.targets[at]);
    if (v < a.vocab) a.logprobs[at] = r.logprob(logit<F32>(a, row, v), a.scale);
  }
}

// Of n keys in LDS the k largest in order, each to put(rank, key): by counting.
template <typename F>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, uint32_t n, uint32_t k, uint32_t threads, F put) {
  for (uint32_t i = threadIdx.x; i < n; i += threads) {
    const uint64_t x = keys[i];
    uint32_t rank = 0;
    for (uint32_t j = 0; j < n; ++j) rank += keys[j] > x;
    if (rank < k) put(rank, x);
  }
}

// Of 64 values, one a lane, the k-th largest.
__device__ __forceinline__ float kth_of_wave(float v, uint32_t k) {
  const uint32_t lane = __lane_id();
  uint32_t rank = 0;
#pragma unroll
  for (int j = 0; j < kWave; ++j) {
    const float y = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), j));
    rank += y > v || (y == v && j < static_cast<int>(lane));
  }
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v),
                                                             __builtin_ctzll(__ballot(rank == k - 1))));
}

template <bool F32>
__global__ __launch_bounds__(kLpThreads) void k_logprobs(const LogprobsArgs a) {
  __shared__ float groups[kWave], shared_bound;
  __shared__ Stats waves[kLpWaves];
  __shared__ uint64_t found[kLpFound];
  __shared__ uint32_t n_found, n_lanes, counts[kLpWaves];
  __shared__ uint16_t lanes[kLpThreads];
  __shared__ uint64_t best[2][kLpWaves];
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave);
  const uint64_t row = blockIdx.x / a.split;
  const uint32_t part = blockIdx.x % a.split;
  const uint32_t v0 = part * a.chunk, v1 = min(v0 + a.chunk, a.vocab);  // this workgroup's logits
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + (row * a.ld + v0) * (F32 ? 4 : 2);
  const uint32_t n = v1 - v0, pieces = (n + 7) / 8;
  if (threadIdx.x == 0) n_found = n_lanes = 0;

  // pieces of 8, the last of which may be short and is filled with -infinity
  const uint32_t full = n / 8;
  typedef std::conditional_t<F32, F32x8, u32x4_t> Raw;
  auto values = [&](const Raw& r, float (&x)[8]) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = r.lo[j];
        x[4 + j] = r.hi[j];
      }
    } else {
      unpack8(r, x);
    }
  };
  auto short_piece = [&](float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 8 * full + j < n ? logit<F32>(a, row, v0 + 8 * full + j) : -INFINITY;
  };
  // f(piece, whether there is one, its values) for the lane's pieces in order
  auto walk = [&](auto f) {
    const Raw* at = reinterpret_cast<const Raw*>(base);
    uint32_t p = threadIdx.x;
    float x[8];
    for (; uniform(p - lane) + kWave <= full; p += kLpThreads) {
      values(at[p], x);
      f(p, true, x);
    }
    if (uniform(p - lane) < full) {
      const bool on = p < full;
      Raw r = {};
      if (on) r = at[p];
      values(r, x);
      f(p, on, x);
    }
    if (full != pieces && wave == full % kLpThreads / kWave) {
      const bool on = threadIdx.x == full % kLpThreads;
      if (on) short_piece(x);
      f(full, on, x);
    }
  };

  // mc: a lane's maximum times c, rounded.  A weight's exponent is x c - mc with one
  // rounding: what mc's rounding moved it by is the same for all, and comes off below
  float mc = kLowestC, sum = 0.f, weighted = 0.f;
  float most = -INFINITY;  // the lane's largest
  walk([&](uint32_t, bool on, const float (&x)[8]) {
    if (!on) return;
    const float pm = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    most = max3(most, pm, pm);
    if (__any(fmaf(pm, a.c, -mc) > kGrow)) {
      const float to = fminf(fmaxf(mc, pm * a.c), -kLowestC), d = mc - to, f = __builtin_amdgcn_exp2f(d);
      weighted = f * fmaf(sum, fmaxf(d, kNoWeight), weighted);
      sum *= f;
      mc = to;
    }
    float s = 0.f, w = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = fmaf(x[j], a.c, -mc), e = __builtin_amdgcn_exp2f(d);
      s += e;
      w = fmaf(e, fmaxf(d, kNoWeight), w);
    }
    sum += s;
    weighted += w;
  });
  // the workgroup's statistics, relative to its largest logit
  {
    float g = most;
    for (int x = 1; x < 8; x *= 2) g = fmaxf(g, lane_xor(g, x));
    if (lane % 8 == 0) groups[wave * 8 + lane / 8] = g;
  }
  __syncthreads();
  float largest = groups[lane];
  for (int x = 32; x; x /= 2) largest = fmaxf(largest, lane_xor(largest, x));
  Stats t = {fmaxf(largest, kLowest), 0.f, 0.f};
  const float top = t.m * a.c;
  if (fabsf(top) <= kFar || largest == -INFINITY) {
    const float to = largest == -INFINITY ? mc : top;  // then all sums are 0
    const float d = mc - to, f = __builtin_amdgcn_exp2f(d);
    t.a = f * fmaf(sum, fmaxf(d, kNoWeight), weighted);
    t.s = sum * f;
  } else {
    // a maximum whose product with c is too coarse: differences first
#pragma unroll 1
    for (uint32_t v = threadIdx.x; v < n; v += kLpThreads) {
      const float d = (logit<F32>(a, row, v0 + v) - t.m) * a.c, e = __builtin_amdgcn_exp2f(d);
      t.s += e;
      t.a = fmaf(e, fmaxf(d, kNoWeight), t.a);
    }
  }
  t.s = wave_sum(t.s);
  t.a = wave_sum(t.a);
  if (lane == 0) waves[wave] = t;
  __syncthreads();
  t.s = t.a = 0.f;
#pragma unroll
  for (int w = 0; w < kLpWaves; ++w) {
    t.s += waves[w].s;
    t.a += waves[w].a;
  }
  if (fabsf(top) <= kFar) {
    const float off = fmaf(t.m, a.c, -top), f = __builtin_amdgcn_exp2f(-off);
    t.a = f * fmaf(t.s, -off, t.a);
    t.s *= f;
  }
  const RowOut out(t);
  const bool whole = a.split == 1;
  if (whole) {
    store_targets<F32>(a, row, out, kLpThreads);
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = out.none ? 0.f : fmaf(-0.69314718055994530942f, t.a / t.s, out.log_s);
  } else if (threadIdx.x == 0) {
    float* st = a.stats + 4 * static_cast<uint64_t>(blockIdx.x);
    st[0] = t.m;
    st[1] = t.s;
    st[2] = t.a;
  }
  const uint32_t k = a.k;
  if (k == 0) return;
  auto put = [&](uint32_t rank, uint64_t key) {
    if (whole) {
      a.top_ids[row * k + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
      a.top_logprobs[row * k + rank] = out.logprob(value_of(static_cast<uint32_t>(key >> 32)), a.scale);
    } else {
      a.tops[static_cast<uint64_t>(blockIdx.x) * k + rank] = key;
    }
  };
  const bool odd = !(t.s < INFINITY);  // NaN or +infinity among them
  if (wave == 0) {
    const float x = kth_of_wave(groups[lane], k);
    if (lane == 0) shared_bound = x;
  }
  __syncthreads();
  const float bound = shared_bound;
  // The logits that reach the bound, then, where there are too many of them for LDS,
  // those above it.  The lanes that have some are listed, and their pieces go round
  // all lanes.
  const uint32_t each = (pieces + kLpThreads - 1) / kLpThreads;  // pieces of a lane at most
  for (uint32_t strict = 0; strict < 2 && !odd; ++strict) {
    if (strict ? most > bound : most >= bound) lanes[atomicAdd(&n_lanes, 1u)] = static_cast<uint16_t>(threadIdx.x);
    __syncthreads();
    const uint32_t listed = n_lanes;
    if (strict || listed <= kLpThreads / 2)  // more: most logits are equal
      for (uint32_t i = threadIdx.x; i < listed * each; i += kLpThreads) {
        const uint32_t p = lanes[i / each] + i % each * kLpThreads;
        if (p >= pieces || *const_cast<volatile uint32_t*>(&n_found) > kLpFound) continue;
        float x[8];
        if (p < full)
          values(reinterpret_cast<const Raw*>(base)[p], x);
        else
          short_piece(x);
        uint32_t hits = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) hits |= ((strict ? x[j] > bound : x[j] >= bound) && 8 * p + j < n ? 1u : 0u) << j;
        if (!hits) continue;
        uint32_t at = atomicAdd(&n_found, static_cast<uint32_t>(__popc(hits)));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (hits >> j & 1) {
            if (at < kLpFound) found[at] = key_of(x[j], v0 + 8 * p + j);
            ++at;
          }
      }
    else if (threadIdx.x == 0)
      n_found = kLpFound + 1;
    __syncthreads();
    uint32_t have = n_found;
    if (have > kLpFound) {
      __syncthreads();  // n_found and the list are read
      if (threadIdx.x == 0) n_found = n_lanes = 0;
      __syncthreads();
      continue;
    }
    // those equal to the bound, from the lowest index on, until there are k
#pragma unroll 1
    for (uint32_t v = 0; strict && have < k && v < n; v += kLpThreads) {
      const uint32_t index = v0 + v + threadIdx.x;
      const bool hit = index < v1 && logit<F32>(a, row, index) == bound;
      const uint64_t which = __ballot(hit);
      if (lane == 0) counts[wave] = __popcll(which);
      __syncthreads();
      uint32_t at = have + __popcll(which & ((uint64_t{1} << lane) - 1));
      for (uint32_t w = 0; w < kLpWaves; ++w) {
        if (w < wave) at += counts[w];
        have += counts[w];
      }
      if (hit && at < k) found[at] = key_of(bound, index);
      __syncthreads();
    }
    have = strict ? min(have, max(k, n_found)) : have;
    rank_keys(found, have, k, kLpThreads, put);
    // a last part with fewer logits than k
    for (uint32_t r = have + threadIdx.x; r < k; r += kLpThreads) put(r, 0);
    return;
  }
  uint64_t last = ~uint64_t{0};
  for (uint32_t r = 0; r < k; ++r) {
    uint64_t top = 0;
#pragma unroll 1
    for (uint32_t v = v0 + threadIdx.x; v < v1; v += kLpThreads) {
      const uint64_t key = key_of(logit<F32>(a, row, v), v);
      if (key < last && key > top) top = key;
    }
    for (int x = 32; x; x /= 2) {
      const uint64_t y = __shfl_xor(top, x, kWave);
      top = y > top ? y : top;
    }
    if (lane == 0) best[r % 2][wave] = top;
    __syncthreads();
    top = 0;
    for (int w = 0; w < kLpWaves; ++w) top = best[r % 2][w] > top ? best[r % 2][w] : top;
    if (threadIdx.x == 0) put(r, top);
    last = top;
  }
}

// The parts of a row, a workgroup each: all that they left is asked for at once.  The
// first few of every part's sorted keys, 64 or more together, give the bound.
constexpr int kJoinThreads = 256;
template <bool F32>
__global__ __launch_bounds__(kJoinThreads) void k_logprobs_join(const LogprobsArgs a) {
  __shared__ uint64_t keys[kLpMaxSplit * kLpMaxK], heads[2 * kWave];
  __shared__ uint64_t bound;
  __shared__ uint32_t n_found;
  __shared__ uint64_t found[kLpMaxSplit * kLpMaxK];
  const uint64_t row = blockIdx.x;
  const uint32_t k = a.k, lane = __lane_id();
  const uint64_t* tops = a.tops + row * a.split * k;
  const f32x4_t* st = reinterpret_cast<const f32x4_t*>(a.stats) + row * a.split;
  if (threadIdx.x == 0) {
    n_found = 0;
    bound = 0;
  }
  f32x4_t part = {kLowest, 0.f, 0.f, 0.f};
  if (lane < a.split) part = st[lane];  // a lane each
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < a.split * k; i += kJoinThreads) keys[i] = tops[i];
  Stats t = {part[0], part[1], part[2]};
  float m = t.m;
  for (int x = 32; x; x /= 2) m = fmaxf(m, lane_xor(m, x));
  t.move(m, a.c);
  t.s = wave_sum(t.s);
  t.a = wave_sum(t.a);
  const RowOut out(t);
  store_targets<F32>(a, row, out, kJoinThreads);
  if (threadIdx.x == 0 && a.entropy) a.entropy[row] = out.none ? 0.f : fmaf(-0.69314718055994530942f, t.a / t.s, out.log_s);
  if (k == 0) return;
  __syncthreads();
  const uint32_t each = min(k, (kWave + a.split - 1) / a.split), n_heads = each * a.split;  // at most 64 + split - 1
  for (uint32_t i = threadIdx.x; i < n_heads; i += kJoinThreads) heads[i] = keys[i / each * k + i % each];
  __syncthreads();
  // fewer heads than k: no bound
  for (uint32_t i = threadIdx.x; i < n_heads; i += kJoinThreads) {
    uint32_t rank = 0;
    for (uint32_t j = 0; j < n_heads; ++j) rank += heads[j] > heads[i] || (heads[j] == heads[i] && j < i);
    if (rank == k - 1) bound = heads[i];
  }
  __syncthreads();
  const uint64_t least = max(bound, uint64_t{1});  // a key of 0 is none
  for (uint32_t i = threadIdx.x; i < a.split * k; i += kJoinThreads) {
    const uint64_t key = keys[i];
    if (key >= least) found[atomicAdd(&n_found, 1u)] = key;
  }
  __syncthreads();
  rank_keys(found, n_found, k, kJoinThreads, [&](uint32_t rank, uint64_t key) {
    a.top_ids[row * k + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
    a.top_logprobs[row * k + rank] = out.logprob(value_of(static_cast<uint32_t>(key >> 32)), a.scale);
  });
}

// ------------------------------------------------------------------- host ---

constexpr uint32_t kMaxCols = 32768;  // 8 wavefronts of 8 pieces a lane

template <bool F32>
nwc_status launch_residual(const ResidualArgs& a, hipStream_t s) {
  // As few wavefronts a token as hold it in 8 pieces a lane where tokens fill the
  // GPU, else as many as have a piece for each lane; past 16384 columns 8, the most
  // whose registers hold 8 pieces.  Us for 4096 columns, few and many wavefronts a token:
  // 256 tokens 6.3 and 3.9, 512 tokens 6.8 and 6.2, 1024 tokens 8.3 and 10.1, 16384 tokens
  // 104 and 169.  At other widths where the rule changes sides, 1023 tokens (many) and 1024
  // (few): 1024 columns 4.2 and 3.8, 2048 4.8 and 5.3, 8192 14.3 and 13.1, 16384 24.8 and 24.2
  const bool many = a.tokens >= 4 * kCus;
  const auto go = [&](auto kernel, uint32_t w) {
    const uint64_t groups = w == 1 ? (static_cast<uint64_t>(a.tokens) + 3) / 4 : a.tokens;
    return launch(kernel, dim3(static_cast<uint32_t>(std::min<uint64_t>(groups, 1u << 20))), dim3(w == 1 ? 256 : w * 64), 0, s, a);
  };
  const uint32_t c = a.cols8;
  if (c > 2048) return go(k_residual<8, 8, F32>, 8);
  if (many) {
    if (c > 1024) return go(k_residual<4, 8, F32>, 4);
    if (c > 512) return go(k_residual<4, 4, F32>, 4);
    if (c > 256) return go(k_residual<1, 8, F32>, 1);
    if (c > 128) return go(k_residual<1, 4, F32>, 1);
    if (c > 64) return go(k_residual<1, 2, F32>, 1);
    return go(k_residual<1, 1, F32>, 1);
  }
  if (c > 1024) return go(k_residual<16, 2, F32>, 16);
  if (c > 256) return go(k_residual<16, 1, F32>, 16);
  if (c > 64) return go(k_residual<4, 1, F32>, 4);
  return go(k_residual<1, 1, F32>, 1);
}

struct LogprobsLayout {
  uint32_t split, chunk;
  uint64_t tops, bytes;
};
LogprobsLayout logprobs_layout(uint32_t rows, uint32_t vocab, uint32_t k) {
  LogprobsLayout L;
  // Two workgroups a compute unit, of 4096 logits at least: us by 2048, 4096 and 8192 at
  // least, 1 row of 32003: 13.6, 13.0, 13.0; 8 rows 14.2, 13.4, 13.9; 16 rows 12.3, 11.6, 11.6
  const uint32_t want = std::min<uint32_t>({(2 * kCus + rows - 1) / rows, (vocab + 4095) / 4096, kLpMaxSplit});
  L.chunk = ((vocab + want - 1) / want + 7) / 8 * 8;
  L.split = (vocab + L.chunk - 1) / L.chunk;
  auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
  // the most parts that as many rows or fewer have, of rows * split < 2 kCus + rows: a
  // workspace for more rows serves fewer
  const uint64_t most = std::min<uint32_t>((vocab + 4095) / 4096, kLpMaxSplit);
  const uint64_t parts = most == 1 ? 0 : std::min<uint64_t>(rows * most, 4 * kCus - 1);
  L.tops = up(parts * 16);
  L.bytes = std::max<uint64_t>(256, L.tops + up(parts * k * 8));
  return L;
}

nwc_status logprobs_shape(uint32_t rows, uint32_t vocab, uint32_t k) {
  if (rows == 0 || vocab == 0 || k > vocab) return NWC_ERR_INVALID_ARG;
  if (k > kLpMaxK || vocab > 0x7FFFFFFF || rows > 1u << 22) return NWC_ERR_UNSUPPORTED;
  return NWC_OK;
}

}  // namespace

extern "C" {

nwc_status nwc_residual_norm(const nwc_residual* r, uint32_t tokens, uint32_t cols, void* stream) {
  if (!r || tokens == 0 || cols == 0 || r->reserved || !r->x || !std::isfinite(r->scale) || !(r->eps >= 0.f) ||
      !std::isfinite(r->eps) || (r->x_type != NWC_OUT_BF16 && r->x_type != NWC_OUT_F32))
    return NWC_ERR_INVALID_ARG;
  if ((!r->out && !r->x_out) || !r->out != !r->weight || (!r->y && (r->x_out || r->y_weight || r->gate))) return NWC_ERR_INVALID_ARG;
  if (cols % 8 || cols > kMaxCols) return NWC_ERR_UNSUPPORTED;
  const bool f32 = r->x_type == NWC_OUT_F32;
  auto bad_ld = [&](const void* p, uint64_t ld) { return p && (ld < cols || ld > kMaxStride); };
  if (bad_ld(r->x, r->ld_x) || bad_ld(r->x_out, r->ld_x_out) || bad_ld(r->y, r->ld_y) || bad_ld(r->out, r->ld_out) ||
      (r->ld_gate && bad_ld(r->gate, r->ld_gate)))
    return NWC_ERR_INVALID_ARG;
  for (const void* p : {r->x, static_cast<const void*>(r->x_out), static_cast<const void*>(r->y), static_cast<const void*>(r->y_weight),
                        static_cast<const void*>(r->gate), static_cast<const void*>(r->weight), static_cast<const void*>(r->out)})
    if (!aligned(p, 16)) return NWC_ERR_ALIGNMENT;
  if (r->ld_x % 8 || (r->x_out && r->ld_x_out % 8) || (r->y && r->ld_y % 8) || (r->gate && r->ld_gate % 8) ||
      (r->out && r->ld_out % 8))
    return NWC_ERR_ALIGNMENT;
  // what may be one buffer: the sum and x, the normed and y, or x of its type that no sum goes to
  if (r->x_out == r->x && r->ld_x_out != r->ld_x) return NWC_ERR_INVALID_ARG;
  if (r->out) {
    const void* o = r->out;
    if (o == r->x_out || o == r->gate || o == r->weight || o == r->y_weight || (o == r->y && r->ld_out != r->ld_y) ||
        (o == r->x && (f32 || r->ld_out != r->ld_x)))
      return NWC_ERR_INVALID_ARG;
  }
  if (r->x_out && (r->x_out == r->y || r->x_out == r->gate || r->x_out == r->weight || r->x_out == r->y_weight))
    return NWC_ERR_INVALID_ARG;
  const ResidualArgs a = {r->x, r->x_out, r->y, r->y_weight, r->gate, r->weight, r->out, r->ld_x, r->ld_x_out, r->ld_y,
                          r->ld_gate, r->ld_out, r->scale, r->eps, tokens, cols / 8};
  return f32 ? launch_residual<true>(a, static_cast<hipStream_t>(stream)) : launch_residual<false>(a, static_cast<hipStream_t>(stream));
}

nwc_status nwc_token_logprobs_workspace_size(uint32_t rows, uint32_t vocab, uint32_t k, size_t* bytes) {
  if (!bytes) return NWC_ERR_INVALID_ARG;
  const nwc_status st = logprobs_shape(rows, vocab, k);
  if (st) return st;
  *bytes = logprobs_layout(rows, vocab, k).bytes;
  return NWC_OK;
}

nwc_status nwc_token_logprobs(const void* logits_dev, uint64_t ld, nwc_out_type type, uint32_t rows, uint32_t vocab, float scale,
                              const int32_t* targets_dev, uint32_t n_targets, float* logprobs_dev, float* entropy_dev, uint32_t k,
                              int32_t* top_ids_dev, float* top_logprobs_dev, void* ws, size_t ws_bytes, void* stream) {
  if (!logits_dev || !ws || !(scale > 0.f) || !std::isfinite(scale * kLog2e) || (type != NWC_OUT_BF16 && type != NWC_OUT_F32))
    return NWC_ERR_INVALID_ARG;
  if (!targets_dev != !logprobs_dev || !targets_dev != !n_targets || !top_ids_dev != !top_logprobs_dev || !top_ids_dev != !k ||
      (!n_targets && !entropy_dev && !k))
    return NWC_ERR_INVALID_ARG;
  const nwc_status st = logprobs_shape(rows, vocab, k);
  if (st) return st;
  if (n_targets > 65536) return NWC_ERR_UNSUPPORTED;
  if (ld < vocab || ld > kMaxStride) return NWC_ERR_INVALID_ARG;
  if (!aligned(logits_dev, 16) || ld % (type == NWC_OUT_F32 ? 4 : 8) || !aligned(targets_dev, 4) || !aligned(logprobs_dev, 4) ||
      !aligned(entropy_dev, 4) || !aligned(top_ids_dev, 4) || !aligned(top_logprobs_dev, 4) || !aligned(ws, 256))
    return NWC_ERR_ALIGNMENT;
  const LogprobsLayout L = logprobs_layout(rows, vocab, k);
  if (ws_bytes < L.bytes) return NWC_ERR_BUFFER_TOO_SMALL;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const LogprobsArgs a = {logits_dev, ld, targets_dev, logprobs_dev, entropy_dev, top_logprobs_dev, top_ids_dev, vocab,
                          n_targets, k, L.split, L.chunk, scale, scale * kLog2e, reinterpret_cast<float*>(w),
                          reinterpret_cast<uint64_t*>(w + L.tops)};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(rows * L.split), block(kLpThreads);
  const nwc_status first = type == NWC_OUT_F32 ? launch(k_logprobs<true>, grid, block, 0, s, a) : launch(k_logprobs<false>, grid, block, 0, s, a);
  if (first || L.split == 1) return first;
  return type == NWC_OUT_F32 ? launch(k_logprobs_join<true>, dim3(rows), dim3(kJoinThreads), 0, s, a)
                             : launch(k_logprobs_join<false>, dim3(rows), dim3(kJoinThreads), 0, s, a);
}

}  // extern "C"
