// HIP kernels of libnwc's attention of a chunk of new tokens per row over the
// paged cache, for gfx950 (CDNA4), and the C-ABI entry points that launch them.
//
//  * k_chunk: all rows, tokens and heads in one grid; see there.
//  * k_chunk_join: adds the partial results of items that several workgroups had.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_common.hpp"

namespace {

typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;

// ---------------------------------------------------------------- k_chunk ---
//
// An item is one key-value head's part of up to kCols columns of a row's tokens
// (column: token * ratio + query head of that key-value head, whole tokens), over
// the positions that its last token sees.  Its positions count in units of kUnit.
// All items in order, heads outermost, make one long stretch of positions, cut
// into equal ranges, one per workgroup: a prompt's triangle, a long context
// behind few tokens and rows of any lengths all end at the same time.  The cuts
// follow from starts and lengths, which every workgroup reads for itself, so a
// captured launch serves any.  An item that is cut leaves partial sums in the
// workspace, which k_chunk_join adds.
//
// A wavefront has 32 columns.  S^T = K Q^T and O^T = V^T P^T on 32 x 32 x 16
// products: a lane's scores are those of one column at positions 8 a + 4 g + j (g =
// lane / 32, a and j = 0 .. 3), which is the order in which the second product
// takes its weights from the lane's own registers, if the values come in the same
// order: two transposing LDS reads of 4 positions each.  Keys and values pass
// through LDS, two units deep, in pieces of 16 bytes placed so that the reads of
// both kinds touch all banks evenly.

constexpr int kChunkThreads = 256;
constexpr uint32_t kCols = 128, kWaveCols = 32, kUnit = 64;
constexpr float kNoMax = -3.402823466e+38f;  // the maximum of nothing: finite, so that exp2(-inf - it) is 0
constexpr float kFinite = 3.0e38f;
// Scaled maxima up to which a weight's exponent, score * scale - maximum * scale
// with the second product rounded, is off by a common 2^5 at most; beyond, a column
// is computed by itself.
constexpr float kFarMax = 0x1p29f;

struct ChunkArgs {
  const uint16_t *k, *v, *q;
  uint16_t* out;
  const int32_t *start, *lengths;
  uint64_t ldq, ldo;
  PageArgs pages;
  uint32_t tokens, hq, hkv, ratio;
  uint32_t tb;       // tokens of an item
  uint32_t cap;      // column slots of a part
  uint32_t workers;  // workgroups that positions are cut for
  float scale, scale2;  // scale * log2(e)
  float* part_o;     // workspace: means over a part of a column's positions [part][column][D]
  float* part_ml;    // their scaled maxima and weight sums
};

// A row's tokens that see something: n tokens from token t0 of q on, the first of
// which has position base, in blocks of tb.
struct RowPart {
  uint32_t t0, n, base, skipped;  // skipped: tokens before t0 that see nothing

  __device__ RowPart(const ChunkArgs& a, uint32_t r) {
    const int32_t most = static_cast<int32_t>(a.tokens);
    const uint32_t s0 = static_cast<uint32_t>(min(max(sload(a.start, r), 0), most));
    const uint32_t s1 = static_cast<uint32_t>(min(max(sload(a.start, r + 1), 0), most));
    const int32_t len = sload(a.lengths, r);
    const uint32_t all = s1 > s0 && len >= 0 ? s1 - s0 : 0;
    const uint32_t end = len < 0 ? 0 : min(static_cast<uint32_t>(len), a.pages.cols << a.pages.shift);
    n = min(all, end);
    skipped = all - n;
    t0 = s0 + skipped;
    base = end - n;
  }
  __device__ uint32_t blocks(uint32_t tb) const { return (n + tb - 1) / tb; }
  // positions that block b sees, and those of all blocks before it
  __device__ uint32_t sees(uint32_t b, uint32_t tb) const { return base + min(n, (b + 1) * tb); }
  __device__ uint64_t before(uint32_t b, uint32_t tb) const {
    return static_cast<uint64_t>(b) * base + static_cast<uint64_t>(tb) * (static_cast<uint64_t>(b) * (b + 1) / 2);
  }
  __device__ uint64_t all(uint32_t tb) const {
    const uint32_t nb = blocks(tb);
    return nb ? before(nb - 1, tb) + sees(nb - 1, tb) : 0;
  }
};

// An item, and where it lies in the stretch of all positions; wave-uniform.
struct Item {
  uint64_t at;  // its first position in the stretch
  uint32_t head, row, block;
  uint32_t units(uint32_t sees) const;
};

// The positions of all rows before each row, in LDS: pre[rows + 1].
__device__ __forceinline__ void make_prefix(const ChunkArgs& a, uint64_t* pre, uint64_t* carry) {
  const uint32_t rows = a.pages.rows, tid = threadIdx.x, lane = __lane_id(), wave = uniform(tid / kWave);
  uint64_t sum = 0;
  if (tid == 0) pre[0] = 0;
  for (uint32_t base = 0; base < rows; base += kChunkThreads) {
    const uint32_t r = base + tid;
    uint64_t x = 0;
    if (r < rows) {
      // as RowPart, by vector loads
      const int32_t most = static_cast<int32_t>(a.tokens), len = a.lengths[r];
      const uint32_t s0 = static_cast<uint32_t>(min(max(a.start[r], 0), most)), s1 = static_cast<uint32_t>(min(max(a.start[r + 1], 0), most));
      const uint32_t all = s1 > s0 && len >= 0 ? s1 - s0 : 0;
      const uint32_t end = len < 0 ? 0 : min(static_cast<uint32_t>(len), a.pages.cols << a.pages.shift);
      const uint32_t n = min(all, end), b = end - n, nb = (n + a.tb - 1) / a.tb;
      if (nb)
        x = static_cast<uint64_t>(nb - 1) * b + static_cast<uint64_t>(a.tb) * (static_cast<uint64_t>(nb - 1) * nb / 2) + b + n;
    }
    for (int d = 1; d < kWave; d *= 2) {
      const uint64_t y = __shfl_up(x, d, kWave);
      if (static_cast<int>(lane) >= d) x += y;
    }
    if (lane == kWave - 1) carry[wave] = x;
    __syncthreads();
    for (uint32_t w = 0; w < 4; ++w) {
      if (w < wave) x += carry[w];
    }
    if (r < rows) pre[r + 1] = sum + x;
    for (uint32_t w = 0; w < 4; ++w) sum += carry[w];
    __syncthreads();
  }
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32 | uniform(static_cast<uint32_t>(v));
}

// Positions per worker: equal ranges, of at least two units.
__device__ __forceinline__ uint64_t quota_of(const ChunkArgs& a, uint64_t total) {
  return max((total + a.workers - 1) / a.workers, uint64_t{2 * kUnit});
}

// The item that position x < hkv * pre[rows] of the stretch belongs to.
__device__ __forceinline__ Item find(const ChunkArgs& a, const uint64_t* pre, uint64_t x) {
  const uint32_t rows = a.pages.rows;
  const uint64_t each = uniform64(pre[rows]);
  Item it;
  it.head = uniform(static_cast<uint32_t>(x / each));
  const uint64_t rem = x - it.head * each;
  uint32_t lo = 0, hi = rows;  // the last row with pre[row] <= rem
  while (lo + 1 < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (uniform64(pre[mid]) <= rem) lo = mid; else hi = mid;
  }
  it.row = lo;
  const uint64_t first = uniform64(pre[lo]);
  const RowPart p(a, lo);
  uint32_t b = 0, end = p.blocks(a.tb);  // the last block with before(b) <= rem - first
  while (b + 1 < end) {
    const uint32_t mid = (b + end) / 2;
    if (p.before(mid, a.tb) <= rem - first) b = mid; else end = mid;
  }
  it.block = b;
  it.at = it.head * each + first + p.before(b, a.tb);
  return it;
}

// LDS places of a tile's pieces of 16 bytes: piece c of row r lies at c ^ key_swap
// (r) of its row, for keys, whose reads take one piece of 32 neighbouring rows, and
// at c ^ value_swap(r) for values, whose reads take 4 pieces of 4 rows.
template <int D>
__device__ __forceinline__ constexpr uint32_t key_swap(uint32_t r) {
  return D == 96 ? r >> 2 & 3 : D == 64 || D == 192 ? r >> 1 & 7 : r & 15;
}
template <int D>
__device__ __forceinline__ constexpr uint32_t value_swap(uint32_t r) {
  return D == 96 ? 0 : D == 64 || D == 192 ? (r >> 1 & 1) << 2 : (r & 3) << 2;
}

// One column once more, by one wavefront, where its sums came out infinite or NaN
// or its maximum passes kFarMax: maximum and sum of the weights first, then the
// values, each with its share of one, in FP32, and nothing that the column does not
// see.  A lane has one position of 64 at a time, then D / 64 components.
template <int D>
__device__ void redo(const ChunkArgs& a, uint32_t row, uint32_t token, uint32_t head, uint32_t sees) {
  constexpr uint32_t kPer = (D + 63) / 64;
  const uint32_t lane = __lane_id(), kvh = head / a.ratio;
  const uint16_t* q = a.q + token * a.ldq + static_cast<uint64_t>(head) * D;
  const int32_t* ids = a.pages.ids + static_cast<uint64_t>(row) * a.pages.ld;
  uint64_t off;  // of the lane's position; all ones: not seen
  auto score = [&](uint32_t pos) {
    off = ~uint64_t{0};
    if (pos >= sees) return -INFINITY;
    const int32_t id = ids[pos >> a.pages.shift];
    if (static_cast<uint32_t>(id) >= a.pages.n_pages) return -INFINITY;
    const uint32_t within = (kvh << a.pages.shift) + (pos & ((1u << a.pages.shift) - 1));
    off = static_cast<uint64_t>(id) * a.pages.stride8 * 8 + static_cast<uint64_t>(within) * D;
    float s = 0.f;
#pragma unroll 1
    for (uint32_t e = 0; e < D; e += 8) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(q + e), y = *reinterpret_cast<const u32x4_t*>(a.k + off + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fmaf(bf16_hi(x[j]), bf16_hi(y[j]), fmaf(bf16_lo(x[j]), bf16_lo(y[j]), s));
    }
    return s;
  };
  float best = kNoMax, total = 0.f, o[kPer];
  for (uint32_t pos = lane; pos < sees; pos += kWave) best = fmaxf(best, score(pos));
  for (int x = 32; x; x /= 2) best = fmaxf(best, lane_xor(best, x));
  auto weight = [&](float s) { return __builtin_amdgcn_exp2f((s - best) * a.scale2); };
  for (uint32_t pos = lane; pos < sees; pos += kWave) total += weight(score(pos));
  for (int x = 32; x; x /= 2) total += lane_xor(total, x);
  const float r = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (uint32_t i = 0; i < kPer; ++i) o[i] = 0.f;
  for (uint32_t pos = 0; pos < sees; pos += kWave) {
    const float s = score(pos + lane), w = weight(s) * r;
    for (uint32_t j = 0; j < kWave; ++j) {
      auto of = [&](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), j)); };
      const float sj = __builtin_bit_cast(float, of(__builtin_bit_cast(uint32_t, s)));
      const float wj = __builtin_bit_cast(float, of(__builtin_bit_cast(uint32_t, w)));
      const uint64_t at = of(static_cast<uint32_t>(off)) | static_cast<uint64_t>(of(off >> 32)) << 32;
      if (at == ~uint64_t{0}) continue;
      const uint16_t* v = a.v + at;
#pragma unroll
      for (uint32_t i = 0; i < kPer; ++i)
        if (D % kWave == 0 || lane + kWave * i < D) {
          const float x = bf16_lo(v[lane + kWave * i]);
          // a weight too small for FP32 is yet above zero
          o[i] += wj == 0.f && sj != -INFINITY && __builtin_isinf(x) ? x : wj * x;
        }
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < kPer; ++i) {
    const uint32_t e = lane + kWave * i;
    if (D % kWave == 0 || e < D)
      a.out[token * a.ldo + static_cast<uint64_t>(head) * D + e] = static_cast<uint16_t>(pack_bf16(o[i], 0.f));
  }
}

template <int D>
struct ChunkShape {
  static constexpr int kKs = D / 16;   // steps of the K Q^T product
  static constexpr int kDt = D / 32;   // 32-row tiles of O^T
  static constexpr uint32_t kTile = kUnit * D * 2;  // bytes of a unit's keys or values
  static constexpr uint32_t kLds = 4 * kTile;       // two units
  static constexpr int kWgs = D <= 128 ? 2 : 1;     // workgroups of a compute unit
};

template <int D>
__device__ __forceinline__ void run_item(const ChunkArgs& a, const Item& it, const RowPart& p, uint32_t u0, uint32_t u1, uint32_t part,
                         uint8_t* lds) {
  using S = ChunkShape<D>;
  constexpr uint32_t kPieces = D / 8;
  constexpr int kLoads = D / 32;  // of a wavefront's 16 rows
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave), n = lane % 32, g = lane / 32;
  const uint32_t sees = p.sees(it.block, a.tb), units = (sees + kUnit - 1) / kUnit;
  const uint32_t tok0 = it.block * a.tb;
  const uint32_t cols = min(a.tb, p.n - tok0) * a.ratio;
  const int32_t* ids = a.pages.ids + static_cast<uint64_t>(it.row) * a.pages.ld;
  // the lane's column
  const uint32_t col = kWaveCols * wave + n, tok = tok0 + col / a.ratio;
  const bool live = col < cols;
  const uint32_t h = it.head * a.ratio + col % a.ratio;
  const uint32_t reach = live ? p.base + tok + 1 : 0;  // positions that it sees
  // what the wavefront's columns see: all of them, and any
  const bool works = kWaveCols * wave < cols;
  const uint32_t all_see = works ? p.base + tok0 + kWaveCols * wave / a.ratio + 1 : 0;
  const uint32_t any_sees = works ? p.base + tok0 + (min(cols, kWaveCols * (wave + 1)) - 1) / a.ratio + 1 : 0;
  const bool full = kWaveCols * (wave + 1) <= cols;

  u32x4_t qf[S::kKs];
  {
    const uint16_t* src = a.q + static_cast<uint64_t>(p.t0 + tok) * a.ldq + static_cast<uint64_t>(h) * D + 8 * g;
#pragma unroll
    for (int k = 0; k < S::kKs; ++k) {
      qf[k] = u32x4_t{0, 0, 0, 0};
      if (live) qf[k] = *reinterpret_cast<const u32x4_t*>(src + 16 * k);
    }
  }
  f32x16_t o[S::kDt];
#pragma unroll
  for (int d = 0; d < S::kDt; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = kNoMax, mc = fmaxf(m * a.scale2, -kFinite), l = 0.f;

  // page numbers of the 16-position quarters of unit u; a quarter past the last
  // position reads that position's
  auto quarter = [&](uint32_t u, uint32_t i) { return min(kUnit * u + 16 * i, (sees - 1) & ~15u); };
  int32_t id[4];
  auto read_ids = [&](uint32_t u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = sload(ids, quarter(u, i) >> a.pages.shift);
  };
  uint32_t known = 0;  // quarters of the unit that have a page
  auto issue = [&](uint32_t u, uint32_t buf) {
    known = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) known |= (static_cast<uint32_t>(id[i]) < a.pages.n_pages ? 1u : 0u) << i;
    const uint32_t q0 = quarter(u, wave), last = min(sees - 1 - q0, 15u);
    const int32_t page = wave == 0 ? id[0] : wave == 1 ? id[1] : wave == 2 ? id[2] : id[3];
    const uint32_t within = (it.head << a.pages.shift) + (q0 & ((1u << a.pages.shift) - 1));
    const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(page) < a.pages.n_pages ? page : 0) * a.pages.stride8 * 8 +
                         static_cast<uint64_t>(within) * D;
    uint8_t* to = lds + buf * (2 * S::kTile) + wave * (16 * D * 2);
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const uint32_t piece = 64 * y + lane, row = piece / kPieces, c = piece % kPieces;
      const uint32_t from = min(row, last) * D + 8 * (c ^ key_swap<D>(row));
      __builtin_amdgcn_global_load_lds(a.k + off + from, to + 1024 * y, 16, 0, 0);
    }
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const uint32_t piece = 64 * y + lane, row = piece / kPieces, c = piece % kPieces;
      const uint32_t from = min(row, last) * D + 8 * (c ^ value_swap<D>(row));
      __builtin_amdgcn_global_load_lds(a.v + off + from, to + S::kTile + 1024 * y, 16, 0, 0);
    }
  };

  read_ids(u0);
  __syncthreads();  // the tiles are free (the plan or the item before lay there)
  issue(u0, 0);
  uint32_t buf = 0;
  for (uint32_t u = u0; u < u1; ++u, buf ^= 1) {
    const uint32_t here = known;
    if (u + 1 < u1) read_ids(u + 1);
    wait_vmem<0>();
    __syncthreads();
    if (u + 1 < u1) issue(u + 1, buf ^ 1);
    if (kUnit * u >= any_sees) continue;
    const uint8_t* kt = lds + buf * (2 * S::kTile);
    f32x16_t sc[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
#pragma unroll
      for (int k = 0; k < S::kKs; ++k) {
        const uint32_t row = 32 * t + n;
        const u32x4_t kf = *reinterpret_cast<const u32x4_t*>(kt + 16 * (row * kPieces + ((2 * k + g) ^ key_swap<D>(row))));
        sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kf), __builtin_bit_cast(bf16x8_t, qf[k]), sc[t], 0, 0, 0);
      }
    }
    if (!full || kUnit * (u + 1) > all_see || here != 15) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t at = 32 * t + 8 * (i / 4) + 4 * g + i % 4;
          if (kUnit * u + at >= reach || !(here >> (2 * t + i / 8) & 1)) sc[t][i] = -INFINITY;
        }
    }
    // weights relative to the maximum so far; it moves only where a lane's sum
    // shows that they outgrew it by 2^11
    float w[32], sum;
    auto weigh = [&] {
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = __builtin_amdgcn_exp2f(fmaf(sc[i / 16][i % 16], a.scale2, -mc));
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i % 4] += w[i];
      sum = (s[0] + s[1]) + (s[2] + s[3]);
      return !(sum <= 2048.f);
    };
    if (__any(weigh())) {
      float x = sc[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) x = fmaxf(x, sc[i / 16][i % 16]);
      x = fmaxf(x, lane_xor(x, 32));
      m = fmaxf(m, x);
      const float to = fminf(fmaxf(m * a.scale2, -kFinite), kFinite);
      const float f = __builtin_amdgcn_exp2f(mc - to);
      mc = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < S::kDt; ++d) o[d] *= f;
      weigh();
    }
    l += sum;
    const uint8_t* vt = kt + S::kTile;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t pf;
#pragma unroll
      for (int j = 0; j < 4; ++j) pf[j] = pack_bf16(w[8 * s + 2 * j], w[8 * s + 2 * j + 1]);
#pragma unroll
      for (int d = 0; d < S::kDt; ++d) {
        // lane: positions 16 s + 4 g + j (and 8 more) of component 32 d + n; it reads
        // 4 components of the position that its place among 16 names
        const uint32_t r0 = 16 * s + 4 * g + (lane % 16) / 4, c = 4 * d + (n / 16) * 2 + (lane % 4) / 2;
        const uint32_t half = 8 * (lane % 2);
        typedef __attribute__((address_space(3))) s16x4_t lds4;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4*)(vt + 16 * (r0 * kPieces + (c ^ value_swap<D>(r0))) + half));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4*)(vt + 16 * ((r0 + 8) * kPieces + (c ^ value_swap<D>(r0 + 8))) + half));
        const u32x2_t a0 = __builtin_bit_cast(u32x2_t, lo), a1 = __builtin_bit_cast(u32x2_t, hi);
        const u32x4_t vf = {a0[0], a0[1], a1[0], a1[1]};
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, vf), __builtin_bit_cast(bf16x8_t, pf), o[d], 0, 0, 0);
      }
    }
  }
  if (!works) return;
  l += lane_xor(l, 32);
  float zero = 0.f;
#pragma unroll
  for (int d = 0; d < S::kDt; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) zero = fmaf(o[d][i], 0.f, zero);
  // columns whose weights are NaN keep it: so does every component
  const bool lost = live && l == l && (!(zero + lane_xor(zero, 32) + l * 0.f == 0.f) || !(fabsf(mc) < kFarMax || m == kNoMax));
  const float r = l == 0.f ? 0.f : 1.f / l;
  const bool direct = u0 == 0 && u1 == units;
  if (live && direct && !lost) {
    uint16_t* dst = a.out + static_cast<uint64_t>(p.t0 + tok) * a.ldo + static_cast<uint64_t>(h) * D + 4 * g;
#pragma unroll
    for (int d = 0; d < S::kDt; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const u32x2_t x = {pack_bf16(o[d][i] * r, o[d][i + 1] * r), pack_bf16(o[d][i + 2] * r, o[d][i + 3] * r)};
        *reinterpret_cast<u32x2_t*>(dst + 32 * d + 2 * i) = x;
      }
  } else if (live && !direct) {
    const uint64_t slot = static_cast<uint64_t>(part) * a.cap + col;
    if (g == 0) {
      a.part_ml[2 * slot] = lost ? INFINITY : mc;  // an infinite maximum: the column is computed by itself
      a.part_ml[2 * slot + 1] = l;
    }
    float* dst = a.part_o + slot * D + 4 * g;
#pragma unroll
    for (int d = 0; d < S::kDt; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4_t*>(dst + 32 * d + 2 * i) = f32x4_t{o[d][i] * r, o[d][i + 1] * r, o[d][i + 2] * r, o[d][i + 3] * r};
  }
  uint64_t again = __ballot(direct && lost) & 0xFFFFFFFFu;
  for (; again; again &= again - 1) {
    const uint32_t c = kWaveCols * wave + __builtin_ctzll(again), t = tok0 + c / a.ratio;
    redo<D>(a, it.row, p.t0 + t, it.head * a.ratio + c % a.ratio, p.base + t + 1);
  }
}

// Workers' order over the grid: neighbours, which share a head's keys and values,
// on one XCD (blocks go round the 8 of them).
__device__ __forceinline__ uint32_t worker_of(uint32_t block, uint32_t workers) { return block % 8 * (workers / 8) + block / 8; }

template <int D>
__global__ __launch_bounds__(kChunkThreads, ChunkShape<D>::kWgs) void k_chunk(const ChunkArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint64_t carry[4];
  uint64_t* pre = reinterpret_cast<uint64_t*>(lds);  // until the first tile arrives
  const uint32_t rows = a.pages.rows;
  make_prefix(a, pre, carry);
  // tokens that see nothing
  for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const RowPart p(a, r);
    const uint32_t per = a.hq * (D / 8);
    for (uint64_t i = threadIdx.x; i < static_cast<uint64_t>(p.skipped) * per; i += kChunkThreads)
      *reinterpret_cast<u32x4_t*>(a.out + (p.t0 - p.skipped + i / per) * a.ldo + i % per * 8) = u32x4_t{0, 0, 0, 0};
  }
  const uint64_t total = uniform64(pre[rows]) * a.hkv, quota = quota_of(a, total);
  const uint32_t w = worker_of(blockIdx.x, a.workers);
  const uint64_t x0 = w * quota, x1 = min(x0 + quota, total);
  if (x0 >= total) return;
  Item it = find(a, pre, x0);
  RowPart p(a, it.row);
  for (;;) {
    const uint32_t sees = p.sees(it.block, a.tb), units = (sees + kUnit - 1) / kUnit;
    const uint32_t u0 = x0 > it.at ? static_cast<uint32_t>((x0 - it.at + kUnit - 1) / kUnit) : 0;
    const uint32_t u1 = static_cast<uint32_t>(min(static_cast<uint64_t>(units), (x1 - it.at + kUnit - 1) / kUnit));
    if (u0 < u1) run_item<D>(a, it, p, u0, u1, 2 * w + (x0 > it.at ? 0 : 1), lds);
    it.at += sees;
    if (it.at >= x1) return;
    if (++it.block == p.blocks(a.tb)) {
      it.block = 0;
      do {
        if (++it.row == rows) {
          it.row = 0;
          ++it.head;
        }
        p = RowPart(a, it.row);
      } while (p.n == 0);
    }
  }
}

// The item that the end of worker blockIdx.x's range cuts first: 8 columns of its
// parts a workgroup, 32 lanes each.
constexpr uint32_t kJoinCols = 8;
template <int D>
__global__ __launch_bounds__(kChunkThreads) void k_chunk_join(const ChunkArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint64_t carry[4];
  uint64_t* pre = reinterpret_cast<uint64_t*>(lds);
  make_prefix(a, pre, carry);
  const uint64_t total = uniform64(pre[a.pages.rows]) * a.hkv, quota = quota_of(a, total);
  const uint32_t w = blockIdx.x;
  const uint64_t x0 = w * quota, x = x0 + quota;
  if (x >= total) return;
  const Item it = find(a, pre, x);
  const RowPart p(a, it.row);
  const uint32_t sees = p.sees(it.block, a.tb), units = (sees + kUnit - 1) / kUnit;
  // began in this range, and goes on behind it
  if (it.at < x0 || it.at >= x || (x - it.at + kUnit - 1) / kUnit >= units) return;
  const uint32_t tok0 = it.block * a.tb, cols = min(a.tb, p.n - tok0) * a.ratio;
  const uint32_t sub = threadIdx.x / 32, lane = threadIdx.x % 32, col = blockIdx.y * kJoinCols + sub;
  if (col - sub % 2 >= cols) return;  // both columns of the wavefront
  const bool live = col < cols;
  // workers after this one that have units of the item
  const uint64_t last = it.at + static_cast<uint64_t>(units - 1) * kUnit;
  const uint32_t more = static_cast<uint32_t>(last / quota) - w;
  auto slot = [&](uint32_t i) { return static_cast<uint64_t>(i ? 2 * (w + i) : 2 * w + 1) * a.cap + (live ? col : cols - 1); };
  float best = -INFINITY, sum = 0.f;
  bool odd = false;
  for (uint32_t i = lane; i <= more; i += 32) {
    const float m = a.part_ml[2 * slot(i)];
    odd |= m == INFINITY;
    best = fmaxf(best, m);
  }
  for (int d = 16; d; d /= 2) best = fmaxf(best, lane_xor(best, d));
  for (uint32_t i = lane; i <= more; i += 32) sum += a.part_ml[2 * slot(i) + 1] * __builtin_amdgcn_exp2f(a.part_ml[2 * slot(i)] - best);
  for (int d = 16; d; d /= 2) sum += lane_xor(sum, d);
  const uint64_t which = __ballot(odd && live);
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  constexpr int kPer = D / 32;
  float o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
#pragma unroll 4
  for (uint32_t i = 0; i <= more; ++i) {
    const uint64_t s = slot(i);
    const float f = a.part_ml[2 * s + 1] * __builtin_amdgcn_exp2f(a.part_ml[2 * s] - best) * r;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = fmaf(f, a.part_o[s * D + lane + 32 * e], o[e]);
  }
  const uint32_t tok = tok0 + col / a.ratio, h = it.head * a.ratio + col % a.ratio;
  if (live && !(which >> (__lane_id() & 32) & 0xFFFFFFFFu)) {
    uint16_t* dst = a.out + static_cast<uint64_t>(p.t0 + tok) * a.ldo + static_cast<uint64_t>(h) * D + lane;
#pragma unroll
    for (int e = 0; e < kPer; ++e) dst[32 * e] = static_cast<uint16_t>(pack_bf16(o[e], 0.f));
  }
  for (uint32_t side = 0; side < 2; ++side) {
    if (!(which >> (32 * side) & 0xFFFFFFFFu)) continue;
    const uint32_t c = uniform(col - sub % 2) + side, t = tok0 + c / a.ratio;
    redo<D>(a, it.row, p.t0 + t, it.head * a.ratio + c % a.ratio, p.base + t + 1);
  }
}

// ------------------------------------------------------------------- host ---

constexpr uint32_t kChunkMaxRows = 4096, kChunkMaxTokens = 1u << 22, kChunkMaxRatio = 64, kChunkMaxLen = 1u << 22;

struct ChunkLayout {
  uint32_t workers, tb, cap;
  uint64_t ml, bytes;
};
ChunkLayout chunk_layout(uint32_t tokens, uint32_t ratio, uint32_t d) {
  ChunkLayout L;
  L.workers = kCus * (d <= 128 ? 2 : 1);
  L.tb = kCols / ratio;
  L.cap = std::min(tokens, L.tb) * ratio;
  const uint64_t slots = 2ull * L.workers * L.cap;
  auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
  L.ml = up(slots * d * 4);
  L.bytes = L.ml + up(slots * 8);
  return L;
}

nwc_status chunk_shape(const nwc_cache* c, uint32_t rows, uint32_t tokens, uint32_t q_heads) {
  if (!c || rows == 0 || tokens == 0 || q_heads == 0 || c->kv_heads == 0) return NWC_ERR_INVALID_ARG;
  const uint32_t d = c->head_dim;
  if (d != 64 && d != 96 && d != 128 && d != 192 && d != 256) return NWC_ERR_UNSUPPORTED;
  if (q_heads % c->kv_heads) return NWC_ERR_INVALID_ARG;
  if (rows > kChunkMaxRows || tokens > kChunkMaxTokens || q_heads / c->kv_heads > kChunkMaxRatio || q_heads > kMaxHeads)
    return NWC_ERR_UNSUPPORTED;
  return NWC_OK;
}

template <int D>
nwc_status launch_chunk(const ChunkArgs& a, hipStream_t s) {
  constexpr size_t lds = std::max<size_t>(ChunkShape<D>::kLds, (kChunkMaxRows + 1) * 8);
  static_assert(lds + 64 <= kMaxLds, "LDS");
  if (lds > 65536 && !allow_lds<k_chunk<D>, lds>()) return NWC_ERR_HIP;
  const nwc_status st = launch(k_chunk<D>, dim3(a.workers), dim3(kChunkThreads), lds, s, a);
  if (st) return st;
  return launch(k_chunk_join<D>, dim3(a.workers, (a.cap + kJoinCols - 1) / kJoinCols), dim3(kChunkThreads),
                (static_cast<size_t>(a.pages.rows) + 1) * 8, s, a);
}

}  // namespace

extern "C" {

nwc_status nwc_attend_chunk_workspace_size(const nwc_cache* cache, uint32_t rows, uint32_t tokens, uint32_t q_heads, size_t* bytes) {
  if (!bytes) return NWC_ERR_INVALID_ARG;
  const nwc_status st = chunk_shape(cache, rows, tokens, q_heads);
  if (st) return st;
  *bytes = chunk_layout(tokens, q_heads / cache->kv_heads, cache->head_dim).bytes;
  return NWC_OK;
}

nwc_status nwc_attend_chunk(const nwc_cache* cache, const nwc_page_table* table, const int32_t* query_start_dev,
                            const int32_t* lengths_dev, const uint16_t* q_dev, uint64_t ldq, uint32_t tokens, uint32_t q_heads,
                            float scale, uint16_t* out_dev, uint64_t ldo, void* ws, size_t ws_bytes, void* stream) {
  if (!cache || !table || !query_start_dev || !lengths_dev || !q_dev || !out_dev || !ws || !std::isfinite(scale * kLog2e) || !(scale > 0.f))
    return NWC_ERR_INVALID_ARG;
  ChunkArgs a = {};
  nwc_status st = chunk_shape(cache, table->rows, tokens, q_heads);
  if (!st) st = check_cache(cache, table, &a.pages);
  if (st) return st;
  const uint32_t d = cache->head_dim;
  const uint64_t row = static_cast<uint64_t>(q_heads) * d;
  if (ldq < row || ldo < row || ldq > kMaxStride || ldo > kMaxStride) return NWC_ERR_INVALID_ARG;
  if ((static_cast<uint64_t>(table->cols) << a.pages.shift) > kChunkMaxLen) return NWC_ERR_UNSUPPORTED;
  if (!aligned(q_dev, 16) || !aligned(out_dev, 16) || ldq % 8 || ldo % 8 || !aligned(lengths_dev, 4) || !aligned(query_start_dev, 4) ||
      !aligned(ws, 256))
    return NWC_ERR_ALIGNMENT;
  a.ratio = q_heads / cache->kv_heads;
  const ChunkLayout L = chunk_layout(tokens, a.ratio, d);
  if (ws_bytes < L.bytes) return NWC_ERR_BUFFER_TOO_SMALL;
  if (out_dev == q_dev) return NWC_ERR_INVALID_ARG;  // workgroups read queries that others have answered
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.k = cache->k;
  a.v = cache->v;
  a.q = q_dev;
  a.out = out_dev;
  a.start = query_start_dev;
  a.lengths = lengths_dev;
  a.ldq = ldq;
  a.ldo = ldo;
  a.tokens = tokens;
  a.hq = q_heads;
  a.hkv = cache->kv_heads;
  a.tb = L.tb;
  a.cap = L.cap;
  a.workers = L.workers;
  a.scale = scale;
  a.scale2 = scale * kLog2e;
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float*>(w + L.ml);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (d) {
    case 64: return launch_chunk<64>(a, s);
    case 96: return launch_chunk<96>(a, s);
    case 128: return launch_chunk<128>(a, s);
    case 192: return launch_chunk<192>(a, s);
    default: return launch_chunk<256>(a, s);
  }
}

}  // extern "C"
