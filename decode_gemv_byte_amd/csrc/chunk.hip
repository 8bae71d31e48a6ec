// HIP kernels of libnwc's attention of a chunk of new tokens per row over the
// paged cache, for gfx950 (CDNA4), and the C-ABI entry points that launch them.
//
//  * k_chunk: all rows, tokens and heads in one grid; see there.
//  * k_chunk_join: adds the partial results of items that several workgroups had.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "device_common.hpp"

namespace {

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
// order: two transposing LDS reads of 4 positions each.  The weights are rounded to
// BF16 for that product, their sum is not: an output is off by half a step of BF16
// (its own rounding) and, from the weights' roundings, which are independent, by less
// than that again (0.0020 to 0.0024 of the norm together, 0.0017 the first alone).
// Keeping their other 16 bits takes a second product, half as much again of all matrix
// work: 4096 tokens behind 28672 positions 2538 us, so 1870; a prompt of 8192 723 and
// 549.  Items of up to 32 columns, which are not bound by the matrix cores, take it, so
// that a token by itself or a few drafted ones come out as by nwc_attend, off by their
// own rounding alone (us with and without: 31 rows of one with heads of 64 47.5 and 44.6,
// of 128 76.7 and 74.7, of 192 70.5 and 69.9, of 256 107 and 92; 8 tokens behind 131007
// positions 111 and 107; 5 behind 507 16.0 and 15.5; 31 of one and one of 512 with heads
// of 64 101 and 96).
//
// Keys and values go straight to a ring of units in LDS, kAhead units before their
// turn, in pieces of 16 bytes placed so that the reads of both kinds touch all banks
// evenly.  Of 8 wavefronts (heads of 128) the two that share a SIMD are half a turn
// apart, so that one's weights are made beside the other's products; 4 wavefronts and
// two or three workgroups a compute unit leave that to chance.
//
// Bound by the matrix cores, whose clock falls under this load: 4096 tokens behind
// 28672 positions, 32 / 8 heads of 128, 1819 to 1886 us by card, 1130 to 1090 TFLOP/s,
// where an 8192^3 product reaches 1250; 8192 tokens of a new prompt 569 to 593 us, 967 to
// 927 TFLOP/s (526 to 553 us a call among others).  With few columns by the loads' and the products'
// turns, which overlap in part, and what an item leaves for the join (64 tokens behind
// 131007 positions: 176 to 179 us and 11 for the join, 3 TB/s and 780 TFLOP/s), with single
// tokens by HBM (31 rows of up to 4001 positions 77 us, 4.2 TB/s), with little work by one
// chain of dependent loads (5 tokens behind 507 positions: 7.7 us).

constexpr int kChunkThreads = 256;
constexpr uint32_t kMaxWorkers = 4 * kCus;
constexpr uint32_t kLeast = 64;     // positions of a worker's range at least
constexpr uint32_t kItemCost = 256;  // what an item's begin and end take, in positions
constexpr float kNoMax = -3.402823466e+38f;  // the maximum of nothing: finite, so that exp2(-inf - it) is 0
constexpr float kFinite = 3.0e38f;
// Scaled maxima up to which a weight's exponent, score * scale - maximum * scale
// with the second product rounded, is off by a common 2^5 at most; beyond, a column
// is computed by itself.
constexpr float kFarMax = 0x1p29f;

// An item that goes on behind the range of the worker that began it, in the ranges
// of `more` others (0: there is none): its key-value head, table row, first token and
// what that one sees, and its columns.
struct Cut {
  uint32_t more, head, cols, token, sees, row, worker, unused;
};

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
  float scale2;      // scale * log2(e)
  float* part_o;     // workspace: means over a part of a column's positions [part][column][D]
  float* part_ml;    // their scaled maxima and weight sums
  Cut* cuts;         // one for each worker
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
  // positions that block b sees, and what the first b < blocks take
  __device__ uint32_t sees(uint32_t b, uint32_t tb) const { return base + min(n, (b + 1) * tb); }
  __device__ uint64_t first(uint32_t b, uint32_t tb) const {
    return static_cast<uint64_t>(b) * (base + kItemCost) + static_cast<uint64_t>(tb) * (static_cast<uint64_t>(b) * (b + 1) / 2);
  }
  // A row's blocks in order: the first, the last, the second, the last but one, ..: two
  // together take the same, so the ranges of a long prompt end where items do (in plain
  // order 4096 tokens behind 28672 positions took 1905 us, so 1790; 8192 tokens 558 and
  // 526; seven short prompts 124 and 126).  The i-th of them, and what all before it take.
  __device__ static uint32_t block(uint32_t i, uint32_t blocks) { return i % 2 ? blocks - 1 - i / 2 : i / 2; }
  __device__ uint64_t before(uint32_t i, uint32_t tb) const {
    uint64_t x = first((i + 1) / 2, tb);
    if (i >= 2) {
      const uint32_t nb = blocks(tb);
      x += first(nb - 1, tb) + base + n + kItemCost - first(nb - i / 2, tb);
    }
    return x;
  }
};

// An item, and where it lies in the stretch of all positions; wave-uniform.
struct Item {
  uint64_t at;  // its first position in the stretch
  uint32_t head, row, order, block;  // order: among the row's blocks
};

// The positions of all rows before each row, in LDS: pre[rows + 1]; carry: W more.
template <int W>
__device__ __forceinline__ void make_prefix(const ChunkArgs& a, uint64_t* pre, uint64_t* carry) {
  const uint32_t rows = a.pages.rows, tid = threadIdx.x, lane = __lane_id(), wave = uniform(tid / kWave);
  uint64_t sum = 0;
  if (tid == 0) pre[0] = 0;
  for (uint32_t base = 0; base < rows; base += W * kWave) {
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
        x = static_cast<uint64_t>(nb - 1) * (b + kItemCost) + static_cast<uint64_t>(a.tb) * (static_cast<uint64_t>(nb - 1) * nb / 2) + b + n + kItemCost;
    }
    if (rows == 1) {
      if (tid == 0) pre[1] = x;
      __syncthreads();
      return;
    }
    for (int d = 1; d < kWave; d *= 2) {
      const uint64_t y = __shfl_up(x, d, kWave);
      if (static_cast<int>(lane) >= d) x += y;
    }
    if (lane == kWave - 1) carry[wave] = x;
    __syncthreads();
    for (uint32_t w = 0; w < W; ++w) {
      if (w < wave) x += carry[w];
    }
    if (r < rows) pre[r + 1] = sum + x;
    for (uint32_t w = 0; w < W; ++w) sum += carry[w];
    __syncthreads();
  }
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32 | uniform(static_cast<uint32_t>(v));
}

// Equal ranges of the stretch for the first n workers: worker w's begins at begin(w).
struct Ranges {
  uint64_t total, each;
  uint32_t n, rest, near;  // near: see unit_of
  __device__ Ranges(const ChunkArgs& a, uint64_t all) : total(all) {
    n = static_cast<uint32_t>(min(static_cast<uint64_t>(a.workers), max(all / kLeast, uint64_t{1})));
    each = all / n;
    rest = static_cast<uint32_t>(all - each * n);
    near = static_cast<uint32_t>(min(each / 8, static_cast<uint64_t>(kItemCost)));
  }
  __device__ uint64_t begin(uint32_t w) const {  // total w / n
    w = min(w, n);
    return each * w + rest * w / n;
  }
  __device__ uint32_t worker(uint64_t x) const { return static_cast<uint32_t>(((x + 1) * n - 1) / total); }  // of position x
  // The unit of an item that a range's bound falls on: none of it where it is that near to
  // its begin, since a cut takes what kItemCost positions take (and near its end, where
  // kItemCost lies).  With it 4 rows of 512 tokens behind 3000 positions take 116 us,
  // without 126; two of 1024 with heads of 256 64.5 and 62.7.
  template <uint32_t kUnit>
  __device__ uint32_t unit_of(uint64_t x, uint64_t at, uint32_t units) const {
    return x <= at + near ? 0 : static_cast<uint32_t>(min(static_cast<uint64_t>(units), (x - at + kUnit - 1) / kUnit));
  }
};

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
  uint32_t b = 0, end = p.blocks(a.tb);  // the last one with before(b) <= rem - first
  while (b + 1 < end) {
    const uint32_t mid = (b + end) / 2;
    if (p.before(mid, a.tb) <= rem - first) b = mid; else end = mid;
  }
  it.order = b;
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

template <int D, int W>
struct ChunkShape {
  static constexpr int kKs = D / 16;   // steps of the K Q^T product
  static constexpr int kDt = D / 32;   // 32-row tiles of O^T
  static constexpr uint32_t kCols = 32 * W;               // columns of an item
  static constexpr uint32_t kUnit = D <= 128 ? 64 : 32;  // positions of a unit
  static constexpr int kKt = kUnit / 32;                  // 32-position tiles of it
  static constexpr uint32_t kTile = kUnit * D * 2;        // bytes of a unit's keys or values
  static constexpr int kRing = W == 8 ? 4 : D <= 96 ? 3 : D <= 128 ? 2 : D <= 192 ? 3 : 4;  // units of each in LDS
  static constexpr uint32_t kLds = 2 * kRing * kTile;
  static constexpr int kLag = W == 8;                     // turns that the slower half is behind
  static constexpr int kAhead = kRing - 1 - kLag;         // units asked for before their turn
  static constexpr int kWgs = W == 8 ? 1 : D <= 64 ? 3 : D <= 192 ? 2 : 1;  // workgroups of a compute unit
  static constexpr int kRows = kUnit / W;                 // rows of a tile that a wavefront loads
  static constexpr int kLoads = kRows * D * 2 / 1024;     // and its loads for them
  static_assert(kRows * D * 2 % 1024 == 0 && 16 % kRows == 0 && kAhead > 0, "rows of a wavefront");
};

// 16 bytes a lane from base + off (bytes) to 1024 bytes of LDS.  In assembly, since
// the compiler lets every transposing LDS read wait for all of them; nothing is
// returned to registers, and wait_vmem counts them.
__device__ __forceinline__ void load_lds(const void* base, uint32_t off, uint32_t to) {
  // five wait states: base may come from a vector instruction, as a scalar register
  // restored from a lane does
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "memory");
}

template <int D, int W>
__device__ __forceinline__ void run_item(const ChunkArgs& a, const Item& it, const RowPart& p, uint32_t u0, uint32_t u1, uint32_t part,
                                         uint8_t* lds) {
  using S = ChunkShape<D, W>;
  constexpr uint32_t kPieces = D / 8, kUnit = S::kUnit;
  constexpr int kKt = S::kKt, kKs = S::kKs, kDt = S::kDt;
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave), n = lane % 32, g = lane / 32;
  const uint32_t sees = p.sees(it.block, a.tb), units = (sees + kUnit - 1) / kUnit;
  const uint32_t tok0 = it.block * a.tb;
  const uint32_t cols = min(a.tb, p.n - tok0) * a.ratio;
  const int32_t* ids = a.pages.ids + static_cast<uint64_t>(it.row) * a.pages.ld;
  // the wavefront's columns and what they see: all of them, and any
  const uint32_t col0 = 32 * wave;
  const bool works = col0 < cols, full = col0 + 32 <= cols;
  const uint32_t all_see = full ? p.base + tok0 + col0 / a.ratio + 1 : 0;
  const uint32_t any_sees = works ? p.base + tok0 + (min(cols, col0 + 32) - 1) / a.ratio + 1 : 0;
  const uint32_t uw = min(u1, (any_sees + kUnit - 1) / kUnit);  // the wavefront's units end here
  // the lane's column
  const uint32_t col = col0 + n, tok = tok0 + col / a.ratio, h = it.head * a.ratio + col % a.ratio;
  const bool live = col < cols;
  const uint32_t reach = live ? p.base + tok + 1 : 0;  // positions that it sees

  u32x4_t qf[kKs];
  const uint16_t* src = a.q + static_cast<uint64_t>(p.t0 + tok) * a.ldq + static_cast<uint64_t>(h) * D + 8 * g;
#pragma unroll
  for (int k = 0; k < kKs; ++k) {
    qf[k] = u32x4_t{0, 0, 0, 0};
    if (live) qf[k] = *reinterpret_cast<const u32x4_t*>(src + 16 * k);
  }

  bool missing = false;  // a page of the range that does not exist
  bool far = false;      // a maximum of the column passed kFarMax
  f32x16_t o[kDt];
  // the maximum so far, and times scale2, which weights are relative to; their sum
  float m = kNoMax, mc = fmaxf(kNoMax * a.scale2, -kFinite), l = 0.f;
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

  typedef __attribute__((address_space(3))) uint8_t lds1;
  typedef const __attribute__((address_space(3))) u32x4_t lds16;
  typedef __attribute__((address_space(3))) s16x4_t lds8;
  const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds1*)lds));
  // The wavefront's rows of a tile come from one page; a row past the last position is
  // that position's.
  auto first_row = [&](uint32_t u) { return min(kUnit * u + S::kRows * wave, (sees - 1) & ~(S::kRows - 1u)); };
  auto page_of = [&](uint32_t u) { return sload(ids, first_row(min(u, u1 - 1)) >> a.pages.shift); };
  uint32_t from[2][S::kLoads];  // byte offsets of the lane's pieces
#pragma unroll
  for (int y = 0; y < S::kLoads; ++y) {
    const uint32_t piece = 64 * y + lane, row = piece / kPieces, c = piece % kPieces, at = S::kRows * wave + row;
    from[0][y] = 2 * (row * D + 8 * (c ^ key_swap<D>(at)));
    from[1][y] = 2 * (row * D + 8 * (c ^ value_swap<D>(at)));
  }
  auto load_rows = [&](const uint16_t* pages, int which, uint32_t u, int32_t page, uint32_t to) {
    const uint32_t r0 = first_row(u), last = sees - 1 - r0;
    const uint32_t within = (it.head << a.pages.shift) + (r0 & ((1u << a.pages.shift) - 1));
    const uint16_t* base = pages + static_cast<uint64_t>(static_cast<uint32_t>(page) < a.pages.n_pages ? page : 0) * a.pages.stride8 * 8 +
                           static_cast<uint64_t>(within) * D;
    to += S::kRows * wave * D * 2;
    if (last >= S::kRows - 1u) {
#pragma unroll
      for (int y = 0; y < S::kLoads; ++y) load_lds(base, from[which][y], to + 1024 * y);
    } else {
#pragma unroll
      for (int y = 0; y < S::kLoads; ++y) {
        const uint32_t row = (64 * y + lane) / kPieces;
        load_lds(base, from[which][y] - (row - min(row, last)) * (2 * D), to + 1024 * y);
      }
    }
  };
  int32_t page = page_of(u0);  // of the next unit to be asked for
  auto issue = [&](uint32_t i, uint32_t place) {
    load_rows(a.k, 0, i, page, place);
    load_rows(a.v, 1, i, page, place + S::kTile);
    page = page_of(i + 1);
  };
  // Operand addresses in a tile: the swap makes the step k (or d) a bit pattern to
  // be turned, kKx (kDx) of them, the rest an offset.
  constexpr int kKx = D == 96 ? 2 : D == 192 ? 4 : kKs, kDx = D == 96 ? 1 : D == 192 ? 2 : kDt;
  const uint32_t key_at = 16 * (n * kPieces + (g ^ key_swap<D>(n)));
  // a lane's positions are 16 s + 4 g + j (and 8 more) of component 32 d + n; it reads 4
  // components of the position that its place among 16 names
  const uint32_t vr = 4 * g + (lane % 16) / 4;
  const uint32_t value_at = 16 * (vr * kPieces + ((n / 16 * 2 + lane % 4 / 2) ^ value_swap<D>(vr))) + 8 * (lane % 2);
  auto scores = [&](uint32_t kt, f32x16_t (&sc)[kKt]) {
    const uint32_t at = kt + key_at;
    constexpr int kReads = kKt * kKs, kHeld = kReads < (D == 192 ? 3 : 6) ? kReads : D == 192 ? 3 : 6;
    u32x4_t kf[kReads];
    auto read = [&](int i) {
      const int k = i / kKt, t = i % kKt;
      kf[i] = *((lds16*)static_cast<uintptr_t>((at ^ (k % kKx * 32)) + (32 * t * D * 2 + k / kKx * (kKx * 32))));
    };
    // kHeld keys on their way from LDS before the first product, one more with each: left
    // alone, the compiler waits for every key by itself
#pragma unroll
    for (int i = 0; i < kHeld; ++i) read(i);
#pragma unroll
    for (int t = 0; t < kKt; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      sc[i % kKt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kf[i]),
                                                            __builtin_bit_cast(bf16x8_t, qf[i / kKt]), sc[i % kKt], 0, 0, 0);
      if (i + kHeld < kReads) {
        read(i + kHeld);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // scores of unit u that are not seen, and the maximum, which weights are relative
  // to: it moves where a score outgrows it by 2^11
  auto settle = [&](uint32_t u, f32x16_t (&sc)[kKt]) {
    if (kUnit * (u + 1) > all_see || missing) {
      uint32_t known = 0;
#pragma unroll
      for (uint32_t i = 0; i < kUnit / 16; ++i) {
        const uint32_t at = min((kUnit * u + 16 * i) >> a.pages.shift, a.pages.cols - 1);
        known |= (static_cast<uint32_t>(sload(ids, at)) < a.pages.n_pages ? 1u : 0u) << i;
      }
#pragma unroll
      for (int t = 0; t < kKt; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t at = 32 * t + 8 * (i / 4) + 4 * g + i % 4;
          if (kUnit * u + at >= reach || !(known >> (2 * t + i / 8) & 1)) sc[t][i] = -INFINITY;
        }
    }
    float x = sc[0][0];
#pragma unroll
    for (int t = 0; t < kKt; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) x = fmaxf(x, sc[t][i]);
    if (__any(fmaf(x, a.scale2, -mc) > 11.f)) {
      m = fmaxf(m, fmaxf(x, lane_xor(x, 32)));
      const float to = fminf(fmaxf(m * a.scale2, -kFinite), kFinite);
      const float f = __builtin_amdgcn_exp2f(mc - to);
      far |= !(fabsf(to) < kFarMax) && m != kNoMax;
      mc = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[d] *= f;
    }
  };
  // the weights of 16 positions at a time, and their products with the values
  auto weigh = [&](uint32_t vt, const f32x16_t (&sc)[kKt]) {
    const uint32_t at = vt + value_at;
    constexpr int kSteps = 2 * kKt, kSets = D == 192 ? 1 : 2;  // a second set of values there would spill
    u32x2_t vf[kSets][kDt][2];
    auto read = [&](int s) {
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        const uint32_t to = (at ^ (d % kDx * 64)) + (16 * s * D * 2 + d / kDx * (kDx * 64));
        vf[s % kSets][d][0] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds8*)static_cast<uintptr_t>(to)));
        vf[s % kSets][d][1] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds8*)static_cast<uintptr_t>(to + 8 * D * 2)));
      }
    };
    float sum[2] = {0.f, 0.f};
    u32x4_t pf[2];
    auto two = [&](int s, int j) {  // weights 2 j and 2 j + 1 of step s
      const float x = __builtin_amdgcn_exp2f(fmaf(sc[s / 2][8 * (s % 2) + 2 * j], a.scale2, -mc));
      const float y = __builtin_amdgcn_exp2f(fmaf(sc[s / 2][8 * (s % 2) + 2 * j + 1], a.scale2, -mc));
      sum[0] += x;
      sum[1] += y;
      pf[s % 2][j] = pack_bf16(x, y);
    };
    // the next step's values come from LDS, and its weights are made, beside the
    // products of this one, in this order
    read(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) two(0, j);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (kSets == 2 && s + 1 < kSteps) read(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        const u32x4_t v = {vf[s % kSets][d][0][0], vf[s % kSets][d][0][1], vf[s % kSets][d][1][0], vf[s % kSets][d][1][1]};
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, pf[s % 2]), o[d],
                                                       0, 0, 0);
        if (s + 1 < kSteps) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j * kDt / 4 == d) two(s + 1, j);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (kSets == 1 && s + 1 < kSteps) read(s + 1);
    }
    l += sum[0] + sum[1];
  };

  // The same with the weights' lower 16 bits by a second product, one step's values on
  // their way beside its weights: few registers, for items that one wavefront has alone.
  auto weigh_fine = [&](uint32_t vt, const f32x16_t (&sc)[kKt]) {
    const uint32_t at = vt + value_at;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 2 * kKt; ++s) {
      u32x4_t hi, lo;
      u32x2_t vf[kDt][2];
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        const uint32_t to = (at ^ (d % kDx * 64)) + (16 * s * D * 2 + d / kDx * (kDx * 64));
        vf[d][0] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds8*)static_cast<uintptr_t>(to)));
        vf[d][1] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds8*)static_cast<uintptr_t>(to + 8 * D * 2)));
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __builtin_amdgcn_exp2f(fmaf(sc[s / 2][8 * (s % 2) + 2 * j], a.scale2, -mc));
        const float y = __builtin_amdgcn_exp2f(fmaf(sc[s / 2][8 * (s % 2) + 2 * j + 1], a.scale2, -mc));
        sum[0] += x;
        sum[1] += y;
        hi[j] = pack_bf16(x, y);
        lo[j] = pack_bf16(x - bf16_lo(hi[j]), y - bf16_hi(hi[j]));
      }
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        const u32x4_t v = {vf[d][0][0], vf[d][0][1], vf[d][1][0], vf[d][1][1]};
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, hi), o[d], 0, 0, 0);
      }
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        const u32x4_t v = {vf[d][0][0], vf[d][0][1], vf[d][1][0], vf[d][1][1]};
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, lo), o[d], 0, 0, 0);
      }
    }
    l += sum[0] + sum[1];
  };

  __syncthreads();  // the ring is free (the plan or the item before lay there)
#pragma unroll
  for (uint32_t i = 0; i < S::kAhead; ++i)
    if (u0 + i < u1) issue(u0 + i, ring + i * (2 * S::kTile));
  // pages that do not exist are looked for once
  for (uint32_t at = kUnit * u0 >> a.pages.shift, end = (min(kUnit * u1, sees) - 1) >> a.pages.shift; at <= end; at += kWave)
    missing |= static_cast<uint32_t>(ids[min(at + lane, end)]) >= a.pages.n_pages;
  missing = __any(missing);
  // the queries have to be there before the loads in flight are counted
#pragma unroll
  for (int k = 0; k < kKs; ++k) asm volatile("" : "+v"(qf[k]));
  // Of 8 wavefronts those that share a SIMD with an earlier one are a barrier, half a
  // turn, behind: one's first product runs beside the other's weights.
  const bool behind = W == 8 && wave >= 4;
  constexpr uint32_t kGroup = 2 * S::kTile, kEnd = S::kRing * kGroup;
  auto arrived = [&](uint32_t u) {  // the wavefront's rows of unit u, kAhead of which are on their way at most
    if (u + S::kAhead - 1 < u1)
      wait_vmem<2 * S::kLoads*(S::kAhead - 1)>();
    else
      wait_vmem<0>();
  };
  auto walk = [&](auto fine) __attribute__((always_inline)) {
    uint32_t place = 0;  // of unit u in the ring
    if (behind) {
      arrived(u0);
      __syncthreads();
    }
    for (uint32_t u = u0; u < u1; ++u) {
      if (!behind) arrived(u);
      __syncthreads();
      if (u + S::kAhead < u1) issue(u + S::kAhead, ring + (place + S::kAhead * kGroup) % kEnd);
      f32x16_t sc[kKt];
      if (u < uw) {
        scores(ring + place, sc);
        settle(u, sc);
      }
      if constexpr (W == 8) {
        if (behind && u + 1 < u1) arrived(u + 1);
        __syncthreads();
      }
      if (u < uw) {
        if constexpr (decltype(fine)::value)
          weigh_fine(ring + place + S::kTile, sc);
        else
          weigh(ring + place + S::kTile, sc);
      }
      place = (place + kGroup) % kEnd;
    }
  };
  if (cols <= 32)  // tokens by themselves or a few together: see above
    walk(std::true_type{});
  else
    walk(std::false_type{});
  if (W == 8 && !behind) __syncthreads();
  if (!works) return;
  const bool direct = u0 == 0 && u1 == units;
  l += lane_xor(l, 32);
  float zero = 0.f;
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) zero = fmaf(o[d][i], 0.f, zero);
  // a column whose weights are NaN keeps it: so does every component
  const bool lost = live && (far || (l == l && !(zero + lane_xor(zero, 32) + l * 0.f == 0.f)));
  const float r = l == 0.f ? 0.f : 1.f / l;
  if (live && direct && !lost) {
    uint16_t* dst = a.out + static_cast<uint64_t>(p.t0 + tok) * a.ldo + static_cast<uint64_t>(h) * D + 4 * g;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<u32x2_t*>(dst + 32 * d + 2 * i) =
            u32x2_t{pack_bf16(o[d][i] * r, o[d][i + 1] * r), pack_bf16(o[d][i + 2] * r, o[d][i + 3] * r)};
  } else if (live && !direct) {
    const uint64_t at = static_cast<uint64_t>(part) * a.cap + col;
    if (g == 0) {
      a.part_ml[2 * at] = lost ? INFINITY : mc;  // an infinite maximum: the column is computed by itself
      a.part_ml[2 * at + 1] = l;
    }
    float* dst = a.part_o + at * D + 4 * g;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4_t*>(dst + 32 * d + 2 * i) = f32x4_t{o[d][i] * r, o[d][i + 1] * r, o[d][i + 2] * r, o[d][i + 3] * r};
  }
  for (uint64_t again = __ballot(direct && lost) & 0xFFFFFFFFu; again; again &= again - 1) {
    const uint32_t x = col0 + __builtin_ctzll(again), t = tok0 + x / a.ratio;
    redo<D>(a, it.row, p.t0 + t, it.head * a.ratio + x % a.ratio, p.base + t + 1);
  }
}

// Workers' order over the grid: neighbours, which share a head's keys and values,
// on one XCD (blocks go round the 8 of them).
__device__ __forceinline__ uint32_t worker_of(uint32_t block, uint32_t workers) { return block % 8 * (workers / 8) + block / 8; }

template <int D, int W>
__global__ __launch_bounds__(W * kWave, (ChunkShape<D, W>::kWgs * W / 4)) void k_chunk(const ChunkArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];  // from LDS address 0 on: there is no other
  uint64_t* pre = reinterpret_cast<uint64_t*>(lds);  // until the first tile arrives
  const uint32_t rows = a.pages.rows;
  constexpr uint32_t kUnit = ChunkShape<D, W>::kUnit;
  make_prefix<W>(a, pre, pre + rows + 1);
  // tokens that see nothing
  for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const RowPart p(a, r);
    const uint32_t per = a.hq * (D / 8);
    for (uint64_t i = threadIdx.x; i < static_cast<uint64_t>(p.skipped) * per; i += W * kWave)
      *reinterpret_cast<u32x4_t*>(a.out + (p.t0 - p.skipped + i / per) * a.ldo + i % per * 8) = u32x4_t{0, 0, 0, 0};
  }
  const uint64_t total = uniform64(pre[rows]) * a.hkv;
  const Ranges ranges(a, total);
  const uint32_t w = worker_of(blockIdx.x, a.workers);
  const uint64_t x0 = ranges.begin(w), x1 = ranges.begin(w + 1);
  Cut cut = {};
  if (x0 < x1) {
    Item it = find(a, pre, x0);
    RowPart p(a, it.row);
    for (;;) {
      it.block = RowPart::block(it.order, p.blocks(a.tb));
      const uint32_t sees = p.sees(it.block, a.tb), units = (sees + kUnit - 1) / kUnit;
      const uint32_t u0 = ranges.unit_of<kUnit>(x0, it.at, units), u1 = ranges.unit_of<kUnit>(x1, it.at, units);
      if (u0 == 0 && u1 != 0 && u1 < units) {  // the last one, which goes on in the next workers' ranges
        const uint64_t last = it.at + static_cast<uint64_t>(units - 1) * kUnit;
        const uint32_t tok0 = it.block * a.tb;
        cut = Cut{ranges.worker(last) - w, it.head, min(a.tb, p.n - tok0) * a.ratio, p.t0 + tok0, p.base + tok0 + 1, it.row, w, 0};
      }
      if (u0 < u1) run_item<D, W>(a, it, p, u0, u1, 2 * w + (u0 ? 0 : 1), lds);
      it.at += sees + kItemCost;
      if (it.at >= x1) break;
      if (++it.order == p.blocks(a.tb)) {
        it.order = 0;
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
  if (threadIdx.x == 0) a.cuts[w] = cut;
}

// Items that several workers had.  The cuts are few beside the workers, so every
// workgroup lists them, and all take (cut, some of its columns) in turn.  A group of
// 32 lanes adds the parts of a column four at a time, relative to their maximum so
// far.  Cuts of up to kJoinFew parts, the ends of most ranges, go by kJoinWide columns a
// workgroup, a group each; those of more by kJoinCols, a column by kJoinSplit groups,
// each with every kJoinSplit-th part, whose sums meet in LDS.
constexpr uint32_t kJoinCols = 2, kJoinSplit = 4, kJoinGroups = 1024, kJoinFew = 16, kJoinWide = 16;
static_assert(kJoinCols * kJoinSplit * 32 == kChunkThreads, "lanes");
template <int D>
__global__ __launch_bounds__(kChunkThreads) void k_chunk_join(const ChunkArgs a) {
  constexpr int kPer = D / 32;
  __shared__ uint32_t list[kMaxWorkers];  // cuts of few parts from its begin on, of many from its end
  __shared__ uint32_t counts[kMaxWorkers / kChunkThreads][kChunkThreads / kWave];
  __shared__ float sums[kJoinCols][kJoinSplit][D], maxima[kJoinCols][kJoinSplit], totals[kJoinCols][kJoinSplit];
  const uint32_t wave = uniform(threadIdx.x / kWave);
  constexpr int kSteps = kMaxWorkers / kChunkThreads;
  uint32_t more[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t w = i * kChunkThreads + threadIdx.x;
    more[i] = w < a.workers ? a.cuts[w].more : 0;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint64_t any = __ballot(more[i] != 0), many = __ballot(more[i] >= kJoinFew);
    if (__lane_id() == 0) counts[i][wave] = __popcll(any & ~many) | __popcll(many) << 16;
  }
  __syncthreads();
  uint32_t n[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const bool kind = more[i] >= kJoinFew;
    const uint64_t many = __ballot(kind), which = kind ? many : __ballot(more[i] != 0) & ~many;
    uint32_t at = __popcll(which & ((uint64_t{1} << __lane_id()) - 1));
#pragma unroll
    for (uint32_t v = 0; v < kChunkThreads / kWave; ++v) {
      const uint32_t x = counts[i][v];
      if (v == wave) at += kind ? n[1] : n[0];
      n[0] += x & 0xFFFF;
      n[1] += x >> 16;
    }
    if (more[i]) list[kind ? kMaxWorkers - 1 - at : at] = i * kChunkThreads + threadIdx.x;
  }
  __syncthreads();
  const uint32_t lane = threadIdx.x % 32, group = threadIdx.x / 32;
  float m, l, o[kPer];  // of a group's parts: maximum, weight sum, weighted sum of means; m infinite where one is computed by itself
  auto add = [&](const Cut& cut, uint32_t col, bool live, uint32_t first, uint32_t step) __attribute__((always_inline)) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = 0.f;
    for (uint32_t i0 = first; i0 <= cut.more; i0 += 4 * step) {
      float mi[4], li[4], x[4][kPer];
#pragma unroll
      for (uint32_t y = 0; y < 4; ++y) {
        const uint32_t i = i0 + y * step;
        const uint64_t s = static_cast<uint64_t>(i ? 2 * (cut.worker + i) : 2 * cut.worker + 1) * a.cap + col;
        mi[y] = -INFINITY;
        li[y] = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[y][e] = 0.f;
        if (i <= cut.more && live) {
          mi[y] = a.part_ml[2 * s];
          li[y] = a.part_ml[2 * s + 1];
#pragma unroll
          for (int e = 0; e < kPer; ++e) x[y][e] = a.part_o[s * D + lane + 32 * e];
        }
      }
      const float to = fmaxf(m, fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])));
      // weights of 0 relative to a maximum that is none yet
      const float f = m == to ? 1.f : __builtin_amdgcn_exp2f(m - to);
      l *= f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] *= f;
#pragma unroll
      for (uint32_t y = 0; y < 4; ++y) {
        const float w = mi[y] == -INFINITY ? 0.f : li[y] * __builtin_amdgcn_exp2f(mi[y] - to);
        l += w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, x[y][e], o[e]);
      }
      m = to;
    }
  };
  auto once_more = [&](const Cut& cut, uint32_t col) __attribute__((always_inline)) {
    const uint32_t t = col / a.ratio;
    redo<D>(a, uniform(cut.row), uniform(cut.token) + t, uniform(cut.head) * a.ratio + col % a.ratio, uniform(cut.sees) + t);
  };
  auto row_of = [&](const Cut& cut, uint32_t col) {
    return a.out + static_cast<uint64_t>(cut.token + col / a.ratio) * a.ldo + static_cast<uint64_t>(cut.head * a.ratio + col % a.ratio) * D;
  };
  const uint32_t wide = (a.cap + kJoinWide - 1) / kJoinWide, narrow = (a.cap + kJoinCols - 1) / kJoinCols;
  const uint32_t few = uniform(n[0]) * wide, tasks = few + uniform(n[1]) * narrow;
  for (uint32_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    if (task < few) {
      const Cut cut = a.cuts[uniform(list[task / wide])];
#pragma unroll
      for (uint32_t y = 0; y < kJoinWide / 8; ++y) {
        const uint32_t col = task % wide * kJoinWide + 8 * y + group;
        const bool live = col < cut.cols;
        add(cut, col, live, 0, 1);
        const bool odd = m == INFINITY;
        const float r = l == 0.f ? 0.f : 1.f / l;
        if (live && !odd) {
          uint16_t* dst = row_of(cut, col) + lane;
#pragma unroll
          for (int e = 0; e < kPer; ++e) dst[32 * e] = static_cast<uint16_t>(pack_bf16(o[e] * r, 0.f));
        }
        const uint64_t again = __ballot(live && odd);
        for (uint32_t side = 0; side < 2; ++side)
          if (again >> (32 * side) & 0xFFFFFFFFu) once_more(cut, uniform(col) + side);
      }
    } else {
      const Cut cut = a.cuts[uniform(list[kMaxWorkers - 1 - (task - few) / narrow])];
      const uint32_t c = group / kJoinSplit, split = group % kJoinSplit, col = (task - few) % narrow * kJoinCols + c;
      const bool live = col < cut.cols;
      add(cut, col, live, split, kJoinSplit);
#pragma unroll
      for (int e = 0; e < kPer; ++e) sums[c][split][lane + 32 * e] = o[e];
      if (lane == 0) {
        maxima[c][split] = m;
        totals[c][split] = l;
      }
      __syncthreads();
      float best = -INFINITY, total = 0.f, f[kJoinSplit];
#pragma unroll
      for (uint32_t i = 0; i < kJoinSplit; ++i) best = fmaxf(best, maxima[c][i]);
#pragma unroll
      for (uint32_t i = 0; i < kJoinSplit; ++i) {
        f[i] = maxima[c][i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(maxima[c][i] - best);
        total = fmaf(f[i], totals[c][i], total);
      }
      const bool odd = best == INFINITY;
      const float r = total == 0.f ? 0.f : 1.f / total;
      if (live && !odd) {
        uint16_t* dst = row_of(cut, col);
        for (uint32_t e = threadIdx.x % (32 * kJoinSplit); e < D; e += 32 * kJoinSplit) {
          float x = 0.f;
#pragma unroll
          for (uint32_t i = 0; i < kJoinSplit; ++i) x = fmaf(f[i] * r, sums[c][i][e], x);
          dst[e] = static_cast<uint16_t>(pack_bf16(x, 0.f));
        }
      }
      if (wave % (kJoinSplit / 2) == 0 && __any(live && odd)) once_more(cut, uniform(col));
      __syncthreads();  // the sums are read
    }
  }
}

// ------------------------------------------------------------------- host ---

constexpr uint32_t kChunkMaxRows = 4096, kChunkMaxTokens = 1u << 22, kChunkMaxRatio = 64, kChunkMaxLen = 1u << 22;

struct ChunkLayout {
  uint32_t waves, workers, tb, cap;
  uint64_t ml, cuts, bytes;
};
ChunkLayout chunk_layout(uint32_t rows, uint32_t tokens, uint32_t ratio, uint32_t kv_heads, uint32_t d) {
  ChunkLayout L;
  // 8 wavefronts a workgroup for long prompts, whose tiles then serve twice as many
  // columns, and where items are so few that all are cut, into half as many parts then.  Us
  // by 4 and by 8, 32 / 8 heads: 1 row of 4096 tokens behind 28672 positions 1874 and 1792, 16
  // rows of 512 behind 3000 455 and 430, of 256 222 and 226, 9 rows with a prompt of 1000
  // among them 109 and 114, 20 prompts of 400 at most 45 and 48, 64 rows of 32 114 and 122; 4
  // rows of 16 behind 3000 33 and 28, of 32 36 and 30, 1 row of 32 behind 100000 105 and 92,
  // of 8 86 and 84, of 4 (16 columns) 87 and 95; 31 rows of one 73 and 88.  28 / 4, 16 / 8, 16
  // / 1 and 8 / 8 heads: 16 rows of 8192 behind 1000 12222 and 11272, 6288 and 5843, 5531 and
  // 5103, 3112 and 2968; 4 rows of 128 behind 3000 56 and 55, 40 and 42, 41 and 42, 37 and 32;
  // 20 prompts of 400 at most 42 and 52, 32 and 41, 34 and 35, 28 and 34; 31 rows of one
  // beside 512 tokens 86 and 115, 89 and 109, 48 and 54, 84 and 103, of which the rule takes
  // the slower side for 28 / 4 and 16 / 1, whose items are few by the mean row.
  const uint64_t columns = static_cast<uint64_t>(tokens) * ratio;
  const bool few = (rows + columns / 128) * kv_heads < kCus && columns >= 32ull * rows;
  const bool wide = d == 128 && (few || columns >= 1536ull * rows);
  auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
  auto by = [&](bool w8) {
    L.waves = w8 ? 8 : 4;
    L.workers = kCus * (w8 ? 1 : d <= 64 ? 3 : d <= 192 ? 2 : 1);  // ChunkShape's workgroups
    L.tb = 32 * L.waves / ratio;
    L.cap = std::min(tokens, L.tb) * ratio;
    const uint64_t slots = 2ull * L.workers * L.cap;
    L.ml = up(slots * d * 4);
    L.cuts = L.ml + up(slots * 8);
    return L.cuts + up(L.workers * sizeof(Cut));
  };
  // what either takes: a workspace for more tokens serves fewer, by however many wavefronts
  const uint64_t other = d == 128 ? by(!wide) : 0;
  L.bytes = by(wide);
  L.bytes = std::max(L.bytes, other);
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

template <int D, int W>
nwc_status launch_chunk(const ChunkArgs& a, hipStream_t s) {
  using S = ChunkShape<D, W>;
  constexpr size_t lds = std::max<size_t>(S::kLds, (kChunkMaxRows + 1 + W) * 8);
  static_assert(lds <= kMaxLds, "LDS");
  if (a.tb != S::kCols / a.ratio) return NWC_ERR_UNSUPPORTED;  // never: the layout's columns are the kernel's
  if (lds > 65536 && !allow_lds<k_chunk<D, W>, lds>()) return NWC_ERR_HIP;
  const nwc_status st = launch(k_chunk<D, W>, dim3(a.workers), dim3(W * kWave), lds, s, a);
  if (st) return st;
  const uint32_t groups = (a.cap + kJoinCols - 1) / kJoinCols;
  return launch(k_chunk_join<D>, dim3(std::min(kJoinGroups, a.workers * groups)), dim3(kChunkThreads), 0, s, a);
}

}  // namespace

extern "C" {

nwc_status nwc_attend_chunk_workspace_size(const nwc_cache* cache, uint32_t rows, uint32_t tokens, uint32_t q_heads, size_t* bytes) {
  if (!bytes) return NWC_ERR_INVALID_ARG;
  const nwc_status st = chunk_shape(cache, rows, tokens, q_heads);
  if (st) return st;
  *bytes = chunk_layout(rows, tokens, q_heads / cache->kv_heads, cache->kv_heads, cache->head_dim).bytes;
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
  const ChunkLayout L = chunk_layout(table->rows, tokens, a.ratio, cache->kv_heads, d);
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
  // no more workers than a call of full tables has work for
  const uint64_t items = std::min<uint64_t>(tokens, table->rows + tokens / L.tb) * a.hkv;
  const uint64_t most = items * ((static_cast<uint64_t>(table->cols) << a.pages.shift) + kItemCost) / kLeast + 1;
  a.workers = static_cast<uint32_t>(std::min<uint64_t>(L.workers, (most + 7) / 8 * 8));
  a.scale2 = scale * kLog2e;
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float*>(w + L.ml);
  a.cuts = reinterpret_cast<Cut*>(w + L.cuts);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (d) {
    case 64: return launch_chunk<64, 4>(a, s);
    case 96: return launch_chunk<96, 4>(a, s);
    case 128: return L.waves == 8 ? launch_chunk<128, 8>(a, s) : launch_chunk<128, 4>(a, s);
    case 192: return launch_chunk<192, 4>(a, s);
    default: return launch_chunk<256, 4>(a, s);
  }
}

}  // extern "C"
