// HIP kernels of libnwc's attention side for gfx950 (CDNA4) and the C-ABI entry
// points that launch them: norm and rotation of query and key heads, the append
// to a paged key-value cache, attention over that cache with shared prefixes
// read once.
//
//  * k_heads: a head is head_dim / 8 lanes of 8 components, both of a rotated
//    pair in one lane.  The result goes to a row or to a slot of a page.  Bound
//    by HBM for long inputs, by one chain of dependent loads for a single token.
//  * k_attend: attention of all rows in one grid; see there.
//  * k_attend_join: adds the partial results of rows whose positions several
//    workgroups had.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "device_common.hpp"

namespace {

// ---------------------------------------------------------------- k_heads ---

struct HeadsArgs {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out, *v_out;  // k_out, v_out: rows, or with pages.ids the cache
  const uint16_t *q_weight, *k_weight;
  const float* freqs;
  const int32_t *positions, *rows;
  PageArgs pages;
  uint32_t ld_q, ld_k, ld_v, ld_q_out, ld_k_out;  // elements / 8
  uint32_t tokens, split;                         // split: wavefronts that share a token's passes
  float eps;
  uint16_t hq, hk, hv, d, half, style;            // half: dims / 2 (0: no rotation)
};

// Sum over the G lanes of a head, in each of them (DPP: swaps within four lanes,
// then mirrors of 8 and 16 whose halves are equal by then).
template <int G>
__device__ __forceinline__ float head_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    const int y = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, y, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
  v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
  if (G >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});  // row_mirror
  if (G >= 32) v += lane_xor(v, 16);
  return v;
}

// A pass takes 64 / G heads of one token (queries, then keys, then values), G
// lanes each, of which head_dim / 8 hold two pieces of 4 components, a and b.
// With halves a lane turns the pairs (a_j, b_j) of components 4 c + j and half +
// 4 c + j, with pairs (a_0, a_1), (a_2, a_3), .. of 8 neighbouring ones; the
// components past `dims` go to the lanes after. So a pair never leaves its lane,
// a lane needs 4 angles, and those serve all heads of the token. A wavefront
// takes U passes at a time, their loads together; `split` wavefronts share a
// token, so that few tokens still fill the GPU.
// 16384 tokens of 32 + 8 heads of 128, 336 MB read and written: 70 us, 4.8 TB/s
// of the 4.9 that a large copy moves; one token: 2.6 us.  (With 8 neighbouring
// components a lane, their partners by a lane permute and 8 angles: 94 and 3.7.)
template <int G, int U>
__global__ __launch_bounds__(256) void k_heads(const HeadsArgs a) {
  constexpr uint32_t kHeads = kWave / G;  // heads of a pass
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave);
  const uint32_t all = a.hq + a.hk + a.hv;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const uint64_t n = static_cast<uint64_t>(a.tokens) * a.split;
  const uint32_t c = lane % G, sub = lane / G;
  const bool on = 8 * c < a.d;
  const bool pairs = a.style == NWC_ROPE_PAIRS;
  const bool turned = 8 * c < 2 * a.half;
  const uint32_t at_a = turned && !pairs ? 4 * c : 8 * c, at_b = turned && !pairs ? a.half + 4 * c : 8 * c + 4;
  float freq[4] = {0.f, 0.f, 0.f, 0.f};
  if (turned)
#pragma unroll
    for (int j = 0; j < 4; ++j) freq[j] = a.freqs[4 * c + j];
  for (uint64_t w = static_cast<uint64_t>(blockIdx.x) * 4 + wave; w < n; w += static_cast<uint64_t>(gridDim.x) * 4) {
    const uint32_t t = static_cast<uint32_t>(w / a.split);
    const int32_t pos = a.positions[t];
    const uint32_t row = a.rows ? static_cast<uint32_t>(a.rows[t]) : t;
    auto row_of = [&](uint32_t ld) { return static_cast<uint64_t>(t) * ld * 8; };  // the token's first element
    float cs[4], sn[4];
    uint64_t slot = 0;  // element offset of the token's slot, less the head's part
    bool stored = true;
    bool first = true;
    for (uint32_t part = static_cast<uint32_t>(w % a.split); part * U * kHeads < all; part += a.split) {
      u32x2_t xa[U], xb[U], wa[U], wb[U];
      uint32_t head[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        head[u] = (part * U + u) * kHeads + sub;
        const bool live = on && head[u] < all;
        const bool is_q = head[u] < a.hq, is_k = !is_q && head[u] < a.hq + a.hk;
        const uint16_t* src = is_q ? a.q + row_of(a.ld_q) + (head[u]) * a.d
                              : is_k ? a.k + row_of(a.ld_k) + (head[u] - a.hq) * a.d
                                     : a.v + row_of(a.ld_v) + (head[u] - a.hq - a.hk) * a.d;
        const uint16_t* wsrc = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
        xa[u] = xb[u] = wa[u] = wb[u] = u32x2_t{0, 0};
        if (live) {
          xa[u] = *reinterpret_cast<const u32x2_t*>(src + at_a);
          xb[u] = *reinterpret_cast<const u32x2_t*>(src + at_b);
        }
        if (live && wsrc) {
          wa[u] = *reinterpret_cast<const u32x2_t*>(wsrc + at_a);
          wb[u] = *reinterpret_cast<const u32x2_t*>(wsrc + at_b);
        }
      }
      if (first) {
        first = false;
        if (pos < 0) break;  // a padding token
        // angles in turns, reduced in FP64: three roundings of 2^-53 (1 / (2 pi),
        // and two products), so 3 2^-53 |position freq| / (2 pi) turns are lost at
        // most: 1.1e-7 for the farthest position at a frequency of one radian
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double turns = static_cast<double>(pos) * (static_cast<double>(freq[j]) * 0.15915494309189533577);
          const float r = static_cast<float>(turns - __builtin_rint(turns));
          cs[j] = __builtin_amdgcn_cosf(r);  // the hardware's sine and cosine take turns
          sn[j] = __builtin_amdgcn_sinf(r);
        }
        if (a.pages.ids) {
          const uint32_t at = static_cast<uint32_t>(pos) >> a.pages.shift;
          stored = row < a.pages.rows && at < a.pages.cols;
          const int32_t id = stored ? a.pages.ids[static_cast<uint64_t>(row) * a.pages.ld + at] : -1;
          stored = static_cast<uint32_t>(id) < a.pages.n_pages;
          if (stored)
            slot = static_cast<uint64_t>(id) * a.pages.stride8 * 8 +
                   static_cast<uint64_t>(static_cast<uint32_t>(pos) & ((1u << a.pages.shift) - 1)) * a.d;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool is_q = head[u] < a.hq, is_k = !is_q && head[u] < a.hq + a.hk;
        float y[8] = {bf16_lo(xa[u][0]), bf16_hi(xa[u][0]), bf16_lo(xa[u][1]), bf16_hi(xa[u][1]),
                      bf16_lo(xb[u][0]), bf16_hi(xb[u][0]), bf16_lo(xb[u][1]), bf16_hi(xb[u][1])};
        auto squares = [&] {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
          return head_sum<G>(sum);
        };
        float sum = squares(), eps = a.eps;
        if (is_q ? a.q_weight != nullptr : is_k && a.k_weight != nullptr) {
          // squares past FP32's range, or below it with no eps beside them: the
          // head first times a power of two, which leaves its direction
          if (__builtin_expect(!(sum < INFINITY) || (sum < 0x1p-96f && eps < 0x1p-96f), 0)) {
            const float s = sum < 1.f ? 0x1p100f : 0x1p-70f;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= s;
            sum = squares();
            eps = eps * s * s;
          }
          const float r = 1.f / sqrtf(fmaf(sum, inv_d, eps));
          const float g[8] = {bf16_lo(wa[u][0]), bf16_hi(wa[u][0]), bf16_lo(wa[u][1]), bf16_hi(wa[u][1]),
                              bf16_lo(wb[u][0]), bf16_hi(wb[u][0]), bf16_lo(wb[u][1]), bf16_hi(wb[u][1])};
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= r * g[j];
        }
        if (turned) {
          float z[8];
          if (pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[2 * j] = fmaf(y[2 * j], cs[j], -y[2 * j + 1] * sn[j]);
              z[2 * j + 1] = fmaf(y[2 * j + 1], cs[j], y[2 * j] * sn[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[j] = fmaf(y[j], cs[j], -y[j + 4] * sn[j]);
              z[j + 4] = fmaf(y[j + 4], cs[j], y[j] * sn[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = z[j];
        }
        u32x2_t ra = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])}, rb = {pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])};
        if (!is_q && !is_k) {  // values as they are
          ra = xa[u];
          rb = xb[u];
        }
        if (!on || head[u] >= all || !(is_q || stored)) continue;
        uint16_t* dst;
        if (is_q) {
          dst = a.q_out + row_of(a.ld_q_out) + head[u] * a.d;
        } else {
          const uint32_t h = is_k ? head[u] - a.hq : head[u] - a.hq - a.hk;
          dst = (is_k ? a.k_out : a.v_out) + (a.pages.ids ? slot + (static_cast<uint64_t>(h) << a.pages.shift) * a.d
                                                          : row_of(a.ld_k_out) + h * a.d);
        }
        *reinterpret_cast<u32x2_t*>(dst + at_a) = ra;
        *reinterpret_cast<u32x2_t*>(dst + at_b) = rb;
      }
    }
  }
}

// --------------------------------------------------------------- k_attend ---
//
// Work: an item is one key-value head's part of either a group's shared prefix
// (columns: the group's rows times the query heads of that key-value head, in
// blocks of at most kCap) or one row's own positions (columns: its query heads).
// An item's positions count in units of 32.  All units of all prefixes in
// order, heads outermost, are cut into equal ranges, one per workgroup; so are
// the units of all own positions, one range per wavefront (per workgroup when
// a key-value head has more than 32 query heads).  The split needs only the
// lengths, which every workgroup reads for itself, so a captured launch serves
// any lengths.  An item cut between ranges, or a row with both kinds, leaves
// partial sums in the workspace, which k_attend_join adds.
//
// A unit is computed by one wavefront.  S^T = K Q^T on the matrix cores (a lane's
// keys: one position, 8 components); with the positions of the two 16-row tiles
// interleaved (tile t, row m is position 8 (m / 4) + 4 t + m % 4) the result
// leaves each lane the 8 neighbouring positions 8 g .. 8 g + 7 of one column, g = lane / 16, which is
// just the operand that O^T = V^T P^T takes.  Of the values a lane takes D / 16
// neighbouring components of its 8 positions and turns that block by one byte
// permute per operand register.  No value crosses lanes in the loop but the
// column's maximum, and that only when the weights have outgrown it by 2^11.
//
// What bounds it, 32 / 8 heads of 128 on one MI355X (large copies move 4.9 TB/s,
// large reads 6.2 TB/s):
//  * own positions: HBM.  131071 positions of one row, 537 MB: 97 us, 5.5 TB/s;
//    the wavefronts' ranges are equal but end some 20 us apart.
//  * a prefix of 128 columns: a wavefront's chain of LDS reads, products, weights
//    and products, 1.1 us a unit (64 rows behind 16384 and 32768 positions: 53
//    and 87 us, 32 units a workgroup apart), and its loads wait behind those of
//    the own positions (64 rows behind 16384 and up to 1024 of their own, 202 MB:
//    60 us).
//  * short calls: launch, the lengths, page numbers, keys and values one after
//    the other (512 positions of one row: 6.0 us a call in a graph).

constexpr uint32_t kCap = 128;        // columns of a prefix block: 4 wavefronts of 2 16-column tiles
constexpr uint32_t kWaveRatio = 32;   // most query heads per key-value head that one wavefront takes
constexpr int kAttendThreads = 256;
constexpr float kNoMax = -3.402823466e+38f;  // the maximum of nothing, no greater than any score and finite, so that exp2(-inf - it) is 0

template <int D>
struct AttendShape {
  static constexpr int kDt = D / 16;   // 16-row tiles of O^T = components of a lane
  static constexpr int kKs = D / 32;   // steps of the K Q^T product
  static constexpr int kJLd = D + 4;   // padded LDS rows (banks)
  static constexpr int kRowWaves = D <= 128 ? 8 : 4;  // of k_attend_rows: as many as their registers allow
  static constexpr int kRing = D <= 128 ? 4 : 3;  // units in the LDS ring (64 KB at 128: two workgroups fit a compute unit)
};

struct AttendArgs {
  const uint16_t *k, *v, *q;
  uint16_t* out;
  const int32_t *lengths, *group_start, *group_len;
  uint64_t ldq, ldo;
  PageArgs pages;
  uint32_t hq, hkv, ratio, n_groups;
  float scale2;             // scale * log2(e)
  float* part_o;            // workspace: means over a part of a column's positions [column slot][D]
  float* part_ml;           // their maxima and weight sums
  uint32_t* plan;           // the plan for k_attend_join
  uint64_t own_slot;        // first column slot of the own positions' parts
  uint32_t cap_p, cap_o;    // column slots of a worker's part: prefixes, own positions
  uint32_t own_wgs;         // workgroups for own positions, the last of the grid
};

// The split of a call, made in LDS by every workgroup, u32 words:
//   row_pre[rows + 1]   units of own positions before the row
//   row_end[rows]       its length, cut to what the table covers; -1 for padding
//   row_group[rows]     the group whose prefix it shares, or the number of groups
//   g_start[groups + 1], g_pre[groups + 1] (units before the group), g_len[groups + 1] (positions; 0 for no group),
//   g_row[groups] (whose table row is read)
// and for k_attend_join in the workspace, four words each: {units per head of
// prefixes, of own positions, 0, 0}, {units per worker: of prefixes, of own
// positions, two words each}, then per row {row_pre, units, group, length},
// then per group {start, pre, len, 0}.
struct Plan {
  uint32_t *row_pre, *row_end, *row_group, *g_start, *g_pre, *g_len, *g_row;
  __host__ __device__ static constexpr uint32_t words(uint32_t rows, uint32_t groups) { return 3 * rows + 1 + 4 * groups + 3; }
  __host__ __device__ static constexpr uint64_t record_words(uint32_t rows, uint32_t groups) { return 8 + 4 * (uint64_t{rows} + groups); }
  __device__ Plan(uint32_t* p, uint32_t rows, uint32_t groups) {
    row_pre = p;
    row_end = row_pre + rows + 1;
    row_group = row_end + rows;
    g_start = row_group + rows;
    g_pre = g_start + groups + 1;
    g_len = g_pre + groups + 1;
    g_row = g_len + groups + 1;
  }
  __device__ uint32_t base(uint32_t r) const { return g_len[row_group[r]]; }  // the row's first own position
};
// What it comes to, wave-uniform.
struct Split {
  uint32_t prefix_units, own_units;  // per head
  uint32_t prefix_wgs;               // workgroups that prefixes are cut for, the first of the grid
  uint64_t prefix_quota, own_quota;  // units per workgroup; per wavefront (or workgroup)
};

// Inclusive scan (sum or maximum of unsigned values) over the wavefront: shifts
// within rows of 16 lanes, then the rows' last lanes.
template <bool MAX>
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(v), decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
    v = MAX ? max(v, y) : v + y;
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});  // row_shr 1, 2, 4, 8
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast 15 to rows 1 and 3
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast 31 to rows 2 and 3
  return v;
}

// In-place inclusive scan of n words in LDS by the workgroup; carry: 8 words of LDS.
template <bool MAX>
__device__ void block_scan(uint32_t* v, uint32_t n, uint32_t* carry) {
  const uint32_t lane = __lane_id(), wave = threadIdx.x / kWave;
  uint32_t before = 0;
  for (uint32_t base = 0; base < n; base += kAttendThreads) {
    const uint32_t i = base + threadIdx.x;
    uint32_t x = wave_scan<MAX>(i < n ? v[i] : 0);
    if (lane == kWave - 1) carry[wave] = x;
    __syncthreads();
    for (uint32_t w = 0; w < 4; ++w) {
      const uint32_t y = carry[w];
      if (w < wave) x = MAX ? max(x, y) : x + y;
    }
    x = MAX ? max(x, before) : x + before;
    if (i < n) v[i] = x;
    for (uint32_t w = 0; w < 4; ++w) before = MAX ? max(before, carry[w]) : before + carry[w];
    __syncthreads();
  }
}

// Lengths and groups (whatever they hold) into a plan whose ranges are all in
// bounds: starts made ascending within 0..rows, lengths within 0..capacity.
// Up to 64 rows and 63 groups one wavefront scans each list in registers, with
// three barriers in all (8 rows in one group: 3.2 us with the scans by the
// workgroup).
__device__ Split make_plan(const AttendArgs& a, const Plan& p, uint32_t* carry) {
  const uint32_t rows = a.pages.rows, G = a.n_groups, tid = threadIdx.x, lane = __lane_id(), wave = uniform(tid / kWave);
  const int32_t most = static_cast<int32_t>(a.pages.cols << a.pages.shift);
  const bool small = rows <= kWave && G < kWave;
  int32_t len = tid < rows ? a.lengths[tid] : -1;  // asked for before the groups are looked at
  auto start_of = [&](uint32_t i) { return static_cast<uint32_t>(min(max(a.group_start[i], 0), static_cast<int32_t>(rows))); };
  auto length_of = [&](uint32_t i) { return static_cast<uint32_t>(min(max(a.group_len[i], 0), most)); };
  if (small && G) {
    if (wave == 0) {
      const uint32_t x = wave_scan<true>(lane <= G ? start_of(lane) : 0);
      if (lane <= G) p.g_start[lane] = x;
    } else if (wave == 1 && lane <= G) {
      p.g_len[lane] = lane < G ? length_of(lane) : 0;
      if (lane < G) p.g_row[lane] = rows;
    }
  } else {
    for (uint32_t i = tid; i < G; i += kAttendThreads) {
      p.g_start[i] = start_of(i);
      p.g_len[i] = length_of(i);
      p.g_row[i] = rows;
    }
    if (tid == 0) {
      p.g_len[G] = 0;
      p.g_start[G] = G ? start_of(G) : 0;
    }
  }
  if (tid == 0) p.row_pre[0] = p.g_pre[0] = 0;
  __syncthreads();
  if (G && !small) block_scan<true>(p.g_start, G + 1, carry);
  uint32_t units = 0;  // of this thread's (last) row, then of its group
  for (uint32_t r = tid; r < rows; r += kAttendThreads) {
    if (r != tid) len = a.lengths[r];
    const uint32_t end = static_cast<uint32_t>(min(len, most));
    uint32_t g = 0, hi = G + 1;  // the last start <= r
    while (G && g + 1 < hi) {
      const uint32_t mid = (g + hi) / 2;
      if (p.g_start[mid] <= r) g = mid; else hi = mid;
    }
    const bool in = G && g < G && p.g_start[g] <= r;
    const uint32_t s = in ? p.g_len[g] : 0;
    const bool shares = s > 0 && len > 0 && end >= s;
    const uint32_t base = shares ? s : 0;
    p.row_end[r] = len < 0 ? 0xFFFFFFFFu : end;
    p.row_group[r] = shares ? g : G;
    units = len > 0 && end > base ? (end + 31) / 32 - base / 32 : 0;
    p.row_pre[r + 1] = units;
    if (shares) atomicMin(&p.g_row[g], r);
  }
  if (small && wave == 0) {
    units = wave_scan<false>(units);
    if (lane < rows) p.row_pre[lane + 1] = units;
  }
  if (G || !small) __syncthreads();
  auto units_of = [&](uint32_t i) {
    const uint32_t cols = (p.g_start[i + 1] - p.g_start[i]) * a.ratio;
    return p.g_row[i] < rows ? (p.g_len[i] + 31) / 32 * ((cols + kCap - 1) / kCap) : 0;
  };
  if (small) {
    if (G && wave == 1) {
      units = wave_scan<false>(lane < G ? units_of(lane) : 0);
      if (lane < G) p.g_pre[lane + 1] = units;
    }
    __syncthreads();
  } else {
    for (uint32_t i = tid; i < G; i += kAttendThreads) p.g_pre[i + 1] = units_of(i);
    block_scan<false>(p.row_pre + 1, rows, carry);  // its barriers serve g_pre too
    if (G) block_scan<false>(p.g_pre + 1, G, carry);
  }
  Split s;
  s.prefix_units = uniform(p.g_pre[G]);
  s.own_units = uniform(p.row_pre[rows]);
  const uint64_t prefix = static_cast<uint64_t>(s.prefix_units) * a.hkv, own = static_cast<uint64_t>(s.own_units) * a.hkv;
  // prefixes to the first half of the workgroups, own positions to the second:
  // one of each per compute unit.  (Prefixes on both halves, where there is
  // little else, were slower: more partial sums, and no faster a unit; 16 rows
  // behind 16384 positions 29.2 us against 24.7, 64 rows 49.7 against 46.7.)  At
  // least four units, one per wavefront, for a workgroup's part of a prefix.
  s.prefix_wgs = gridDim.x - a.own_wgs;
  const uint32_t owners = a.own_wgs * (a.ratio <= kWaveRatio ? 4 : 1);
  s.prefix_quota = s.prefix_wgs ? max((prefix + s.prefix_wgs - 1) / s.prefix_wgs, uint64_t{4}) : 4;
  s.own_quota = max((own + owners - 1) / owners, uint64_t{1});
  if (blockIdx.x == 0) {
    u32x4_t* rec = reinterpret_cast<u32x4_t*>(a.plan);
    if (tid == 0) {
      rec[0] = u32x4_t{s.prefix_units, s.own_units, 0, 0};
      rec[1] = u32x4_t{static_cast<uint32_t>(s.prefix_quota), static_cast<uint32_t>(s.prefix_quota >> 32),
                       static_cast<uint32_t>(s.own_quota), static_cast<uint32_t>(s.own_quota >> 32)};
    }
    for (uint32_t r = tid; r < rows; r += kAttendThreads)
      rec[2 + r] = u32x4_t{p.row_pre[r], p.row_pre[r + 1] - p.row_pre[r], p.row_group[r], p.row_end[r]};
    for (uint32_t i = tid; i < G; i += kAttendThreads) rec[2 + rows + i] = u32x4_t{p.g_start[i], p.g_pre[i], p.g_len[i], 0};
  }
  return s;
}

// A worker's part of one item; all fields wave-uniform.
struct Segment {
  const int32_t* ids;   // the page table row
  uint32_t head;        // key-value head
  uint32_t row0;        // first row of the item's columns
  uint32_t col0, cols;  // columns: (row - row0) * ratio + query head of the key-value head
  uint32_t u0, u1;      // units (position / 32)
  uint32_t p0, p1;      // positions that the item sees
  bool direct;          // the whole of its row's positions: the output itself, no partial sums
  bool prefix;          // a group's: of its rows those count that share it, where groups[row] == group
  uint32_t group;
  const uint32_t* groups;
  uint64_t slot;        // first column slot of the partial sums
};

// Column slot of a worker's partial sums of an item: the columns of all items
// before it, and a full part for each worker before this one.  Items and
// workers that meet follow each other (either the item or the worker steps
// on), so no two overlap.
__device__ __forceinline__ uint64_t part_slot(const AttendArgs& a, bool prefix, uint32_t head, uint32_t row, uint32_t col0,
                                              uint64_t worker) {
  return (prefix ? 0 : a.own_slot) + (static_cast<uint64_t>(head) * a.pages.rows + row) * a.ratio + col0 +
         worker * (prefix ? a.cap_p : a.cap_o);
}

// Whether a column is one of the item's, of a row that takes part in it.
__device__ __forceinline__ bool counts(const AttendArgs& a, const Segment& it, uint32_t col) {
  return col < it.cols && (!it.prefix || it.groups[it.row0 + (it.col0 + col) / a.ratio] == it.group);
}

// The page that holds a position (8 or 16 positions from it on share it), read
// ahead of its use, and then that position's element offset for a head.  A page
// that does not exist reads page 0 and is not seen.
__device__ __forceinline__ int32_t page_id(const AttendArgs& a, const Segment& it, uint32_t pos) {
  return sload(it.ids, min(pos >> a.pages.shift, a.pages.cols - 1));
}
struct PagePart {
  uint64_t off;
  bool known;
};
__device__ __forceinline__ PagePart page_part(const AttendArgs& a, const Segment& it, int32_t id, uint32_t pos, uint32_t d) {
  // in pieces of 8 elements, of which a page has less than 2^32: few scalar
  // instructions, which are what a wavefront waits for here
  PagePart p;
  p.known = static_cast<uint32_t>(id) < a.pages.n_pages && pos >> a.pages.shift < a.pages.cols;
  const uint32_t within = ((it.head << a.pages.shift) + (pos & ((1u << a.pages.shift) - 1))) * (d / 8);
  p.off = (static_cast<uint64_t>(p.known ? id : 0) * a.pages.stride8 + within) << 3;
  return p;
}

// The queries of NT tiles of 16 columns from col on: lane (n, g) has column n,
// components 32 k + 8 g .. of step k; zeros past the item's last column and for
// rows that take no part (a padding row's may be anything).
template <int D, int NT>
__device__ __forceinline__ void load_queries(const AttendArgs& a, const Segment& it, uint32_t col,
                                             u32x4_t (&qf)[AttendShape<D>::kKs][NT]) {
  const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const uint32_t x = col + 16 * c + n;
    const bool live = counts(a, it, x);
    const uint32_t at = it.col0 + (live ? x : 0), row = it.row0 + at / a.ratio, h = it.head * a.ratio + at % a.ratio;
    const uint16_t* p = a.q + row * a.ldq + static_cast<uint64_t>(h) * D + 8 * g;
#pragma unroll
    for (int k = 0; k < AttendShape<D>::kKs; ++k) {
      qf[k][c] = u32x4_t{0, 0, 0, 0};
      if (live) qf[k][c] = *reinterpret_cast<const u32x4_t*>(p + 32 * k);
    }
  }
}

// A wavefront's running sums for NT tiles of 16 columns: lane (n, g) holds column
// n, components kDt (4 g + i) + t of O (tile t, i = 0 .. 3), the maximum of the
// scores so far (as the product gives them, the same in a column's four lanes)
// and its own part of the sum of the weights.  A weight is exp2((score - maximum)
// scale2): the difference first, since a scaled maximum's rounding alone would
// pass 2^7, FP32's largest exponent, where it stands at 2^31 and beyond.  (An
// instruction more a score: 64 rows behind 16384 positions 64.2 -> 65.2 us.)
template <int D, int NT>
struct Sums {
  static constexpr int kDt = AttendShape<D>::kDt;
  f32x4_t o[kDt][NT];
  float m[NT], l[NT];

  __device__ Sums() {
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      m[c] = kNoMax;
      l[c] = 0.f;
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[d][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }

  // One unit: sc are its scores (lane: positions 8 g .. 8 g + 7 of its column,
  // tile t the positions 4 t ..), vr[j] the lane's components of position 8 g +
  // j, first its first position, good whether the lane's positions have a page.
  __device__ __forceinline__ void take(f32x4_t (&sc)[2][NT], uint32_t (&vr)[8][kDt / 2], const Segment& it, uint32_t first,
                                       bool good, float scale2) {
    if (first < it.p0 || first + 32 > it.p1 || !__all(good)) {  // an edge of the item, or a page that is none
      const uint32_t g = __lane_id() / 16;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t pos = first + 8 * g + j;
        const bool seen = good && pos >= it.p0 && pos < it.p1;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (!seen) sc[j / 4][c][j % 4] = -INFINITY;
        // a slot that is not seen may hold anything, and 0 times NaN is NaN
#pragma unroll
        for (int d = 0; d < kDt / 2; ++d)
          if (!seen) vr[j][d] = 0;
      }
    }
    // Weights relative to the maximum so far.  They may grow to 2^11 before the
    // maximum moves (BF16 and FP32 keep their relative precision), so the common
    // unit looks at no maximum at all: a lane's sum of 8 says whether one grew.
    // The matrix cores take them as BF16, and what that rounding leaves goes
    // through a second product, so the weights keep 16 bits: the error against 64
    // bits is the output's own rounding alone, with one product 1.3 to 1.4 times
    // that.  (512 positions of one row 5.9 -> 6.2 us, 64 rows behind 16384 61 ->
    // 64, six groups of 16 49 -> 50, 32 rows behind 4096 with heads of 256 32 ->
    // 33, long rows the same; where a prefix of 128 columns is all there is it
    // shows most, 64 rows behind 16384 with one position each 48 -> 53.)
    float p[NT][8], sum[NT];
    auto weigh = [&] {
      bool grown = false;
#pragma unroll
      for (int c = 0; c < NT; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[c][j] = __builtin_amdgcn_exp2f((sc[j / 4][c][j % 4] - m[c]) * scale2);
        sum[c] = ((p[c][0] + p[c][1]) + (p[c][2] + p[c][3])) + ((p[c][4] + p[c][5]) + (p[c][6] + p[c][7]));
        grown |= !(sum[c] <= 2048.f);
      }
      return grown;
    };
    if (__any(weigh())) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        float x = fmaxf(fmaxf(sc[0][c][0], sc[0][c][1]), fmaxf(sc[0][c][2], sc[0][c][3]));
        x = fmaxf(x, fmaxf(fmaxf(sc[1][c][0], sc[1][c][1]), fmaxf(sc[1][c][2], sc[1][c][3])));
        x = fmaxf(x, lane_xor(x, 16));
        x = fmaxf(x, lane_xor(x, 32));
        x = fmaxf(x, m[c]);
        const float f = __builtin_amdgcn_exp2f((m[c] - x) * scale2);
        m[c] = x;
        l[c] *= f;
#pragma unroll
        for (int d = 0; d < kDt; ++d) o[d][c] *= f;
      }
      weigh();
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) l[c] += sum[c];
    u32x4_t w[NT], rest[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[c][j] = pack_bf16(p[c][2 * j], p[c][2 * j + 1]);
        rest[c][j] = pack_bf16(p[c][2 * j] - bf16_lo(w[c][j]), p[c][2 * j + 1] - bf16_hi(w[c][j]));
      }
    auto add = [&](int d, int c, u32x4_t v, u32x4_t y) {
      o[d][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, y),
                                                        o[d][c], 0, 0, 0);
    };
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __builtin_amdgcn_perm(vr[2 * j + 1][d / 2], vr[2 * j][d / 2], d % 2 ? 0x07060302 : 0x05040100);
#pragma unroll
      for (int c = 0; c < NT; ++c) add(d, c, v, w[c]);
#pragma unroll
      for (int c = 0; c < NT; ++c) add(d, c, v, rest[c]);
    }
  }

  // Which of the wavefront's columns, that count, from col on have a sum that is
  // no finite number (0 times an infinity or a NaN is NaN): a bit each.  Not those
  // whose weights are NaN already, and every output with them.
  __device__ __forceinline__ uint32_t lost(const AttendArgs& a, const Segment& it, uint32_t col) const {
    bool bad[NT], any = false;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      f32x4_t t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = fmaf(o[d][c][i], 0.f, t[i]);
      any |= bad[c] = !((t[0] + t[1]) + (t[2] + t[3]) == 0.f);
    }
    if (__builtin_expect(!__any(any), 1)) return 0;
    uint32_t which = 0;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      auto columns = [](uint64_t lanes) {
        lanes |= lanes >> 32;
        return static_cast<uint32_t>((lanes | lanes >> 16) & 0xFFFF);
      };
      const uint32_t here = columns(__ballot(bad[c] && counts(a, it, col + 16 * c + __lane_id() % 16)));
      which |= (here & ~columns(__ballot(l[c] != l[c]))) << (16 * c);
    }
    return which;
  }

  // The columns' weight sums complete in all four lanes.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      l[c] += lane_xor(l[c], 16);
      l[c] += lane_xor(l[c], 32);
    }
  }

  // The wavefront's columns from col on but those in skip, complete: outputs or
  // partial sums.
  __device__ __forceinline__ void store(const AttendArgs& a, const Segment& it, uint32_t col, uint32_t skip) const {
    const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const uint32_t cc = col + 16 * c + n;
      if (cc >= it.cols || skip >> (16 * c + n) & 1) continue;
      const float r = l[c] == 0.f ? 0.f : 1.f / l[c];
      const uint32_t cl = it.col0 + cc, row = it.row0 + cl / a.ratio, h = it.head * a.ratio + cl % a.ratio;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = kDt * (4 * g + i);
        static_assert(kDt % 2 == 0, "pairs");
        if (it.direct) {
          uint32_t w[kDt / 2];
#pragma unroll
          for (int d = 0; d < kDt; d += 2) w[d / 2] = pack_bf16(o[d][c][i] * r, o[d + 1][c][i] * r);
          __builtin_memcpy(a.out + row * a.ldo + static_cast<uint64_t>(h) * D + e, w, 2 * kDt);
        } else {
          float x[kDt];
#pragma unroll
          for (int d = 0; d < kDt; ++d) x[d] = o[d][c][i] * r;
          __builtin_memcpy(a.part_o + (it.slot + cc) * D + e, x, 4 * kDt);
        }
      }
      if (!it.direct && g == 0) {
        a.part_ml[2 * (it.slot + cc)] = m[c];
        a.part_ml[2 * (it.slot + cc) + 1] = l[c];
      }
    }
  }
};

// Columns of an item once more, those with a bit in `which` (of column col), by
// one wavefront, for sums that came out infinite or NaN: weights of up to 2^11,
// and many of them, take finite values past FP32's range, and the products with
// both parts of a weight lose an infinite value's place, since the second part
// may be zero or negative.  Here the maximum and the sum of the weights come
// first, then the values, each once with its share of one, in FP32, so that an
// infinite value gives its infinity (NaN where two signs meet).  A lane has one
// position of 64 at a time, then D / 64 components.  (Asking for it costs the
// others at most 0.4 us a call, and 1.5 of 34 where heads of 256 spill; with an
// infinite value in every row 512 positions of one row take 160 us, 131071 1.9
// ms, 64 rows behind 16384 10 ms.  One pass for both maximum and sum, and four of
// a position's key pieces at a time, were no faster.)
template <int D>
__device__ void redo(const AttendArgs& a, const Segment& it, uint32_t col, uint32_t which) {
  constexpr uint32_t kPer = (D + 63) / 64;
  const uint32_t lane = __lane_id();
  const uint32_t first = max(32 * it.u0, it.p0), last = min(32 * it.u1, it.p1);
  for (; which; ++col, which >>= 1) {
    if (!(which & 1)) continue;
    const uint32_t cl = it.col0 + col, row = it.row0 + cl / a.ratio, h = it.head * a.ratio + cl % a.ratio;
    const uint16_t* q = a.q + row * a.ldq + static_cast<uint64_t>(h) * D;
    uint64_t off;  // of the lane's position; all ones: not seen
    auto score = [&](uint32_t pos) {
      const int32_t id = pos < last ? it.ids[pos >> a.pages.shift] : -1;
      const PagePart p = page_part(a, it, id, pos, D);
      off = p.known ? p.off : ~uint64_t{0};
      if (!p.known) return -INFINITY;
      float s = 0.f;
#pragma unroll 1
      for (uint32_t e = 0; e < D; e += 8) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(q + e), y = *reinterpret_cast<const u32x4_t*>(a.k + p.off + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(bf16_hi(x[j]), bf16_hi(y[j]), fmaf(bf16_lo(x[j]), bf16_lo(y[j]), s));
      }
      return s;
    };
    float best = kNoMax, total = 0.f, o[kPer];
    for (uint32_t pos = first + lane; pos < last; pos += kWave) best = fmaxf(best, score(pos));
    for (int x = 32; x; x /= 2) best = fmaxf(best, lane_xor(best, x));
    auto weight = [&](float s) { return __builtin_amdgcn_exp2f((s - best) * a.scale2); };
    for (uint32_t pos = first + lane; pos < last; pos += kWave) total += weight(score(pos));
    for (int x = 32; x; x /= 2) total += lane_xor(total, x);
    const float r = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) o[i] = 0.f;
    for (uint32_t pos = first; pos < last; pos += kWave) {
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
      if (D % kWave && e >= D) continue;
      if (it.direct)
        a.out[row * a.ldo + static_cast<uint64_t>(h) * D + e] = static_cast<uint16_t>(pack_bf16(o[i], 0.f));
      else
        a.part_o[(it.slot + col) * D + e] = o[i];
    }
    if (!it.direct && lane == 0) {
      a.part_ml[2 * (it.slot + col)] = best;
      a.part_ml[2 * (it.slot + col) + 1] = total;
    }
  }
}

// Where piece c of key row `row` (0 .. 31 of a unit) lies in its slot row, and
// (INVERSE) which piece lies at c.  An operand read takes one piece of the rows
// 8 (n / 4) + n % 4, n = 0 .. 15, which a slot row of D = 64, 96, 128, 192, 256
// puts on 2, 4, 1, 2, 1 different groups of banks by itself.
template <int D, bool INVERSE>
__device__ __forceinline__ uint32_t key_piece(uint32_t row, uint32_t c) {
  constexpr uint32_t kPieces = D / 8;
  if (D == 128 || D == 256) return c ^ ((row & 3) | (row >> 3) << 2);
  const uint32_t by = D == 96 ? row >> 3 : (row >> 1 & 1) | (row >> 3) << 1;
  if (D == 64) return c ^ by;
  const uint32_t x = INVERSE ? c + kPieces - by : c + by;
  return x >= kPieces ? x - kPieces : x;
}

// One wavefront's loads of a unit and the two products.
template <int D, int NT>
struct Unit {
  static constexpr int kDt = AttendShape<D>::kDt, kKs = AttendShape<D>::kKs;
  u32x4_t kf[2][kKs];
  uint32_t vr[8][kDt / 2];
  __device__ __forceinline__ void load_k(const AttendArgs& a, const PagePart& lo, const PagePart& hi) {
    const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
    const uint16_t* p = a.k + (n < 8 ? lo.off : hi.off) + (n / 4 % 2 * 8 + n % 4) * D + 8 * g;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < kKs; ++k) kf[t][k] = *reinterpret_cast<const u32x4_t*>(p + 4 * t * D + 32 * k);
  }
  // The keys from a slot of LDS (32 rows, pieces as key_piece puts them).  A
  // typed read, never memcpy: a read that may alias the loads in flight makes
  // the compiler wait for all of them.
  __device__ __forceinline__ void read_k(const uint8_t* ks) {
    const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
#pragma unroll
    for (int k = 0; k < kKs; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t row = 8 * (n / 4) + n % 4 + 4 * t;
        kf[t][k] = *reinterpret_cast<const u32x4_t*>(ks + 16 * (row * (D / 8) + key_piece<D, false>(row, 4 * k + g)));
      }
  }
  __device__ __forceinline__ void load_v(const AttendArgs& a, const PagePart& lo, const PagePart& hi) {
    const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
    const uint16_t* p = a.v + (g < 2 ? lo.off : hi.off) + g % 2 * (8 * D) + kDt * n;
#pragma unroll
    for (int j = 0; j < 8; ++j) __builtin_memcpy(vr[j], p + j * D, 2 * kDt);
  }
  __device__ __forceinline__ void scores(const u32x4_t (&qf)[kKs][NT], f32x4_t (&sc)[2][NT]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < NT; ++c) sc[t][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kKs; ++k)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          sc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kf[t][k]),
                                                             __builtin_bit_cast(bf16x8_t, qf[k][c]), sc[t][c], 0, 0, 0);
  }
};

// Units u, u + step, .. of a segment by one wavefront: a unit's keys are asked for
// when the keys before them are used up, and its values likewise (a second set
// of registers, with two units in flight, was no faster: 99.0 and 98.7 us for
// 131071 positions, 84.9 and 86.2 us for 48 ragged rows).  Page numbers come by
// scalar loads a unit before their use, so that waiting for them waits for no
// vector load.
template <int D, int NT>
__device__ __forceinline__ void walk(const AttendArgs& a, const Segment& it, uint32_t u, uint32_t step, Sums<D, NT>& acc) {
  if (u >= it.u1) return;
  const bool upper = __lane_id() / 16 >= 2;
  u32x4_t qf[AttendShape<D>::kKs][NT];
  Unit<D, NT> x;
  int32_t id0 = page_id(a, it, 32 * u), id1 = page_id(a, it, 32 * u + 16);
  PagePart lo, hi;
  auto part = [&](uint32_t unit) {  // of the page numbers read last; then the next unit's
    lo = page_part(a, it, id0, 32 * unit, D);
    hi = page_part(a, it, id1, 32 * unit + 16, D);
    id0 = page_id(a, it, 32 * (unit + step));
    id1 = page_id(a, it, 32 * (unit + step) + 16);
  };
  part(u);
  x.load_k(a, lo, hi);
  x.load_v(a, lo, hi);
  load_queries<D, NT>(a, it, 0, qf);
  for (;;) {
    const bool good = upper ? hi.known : lo.known;
    const uint32_t next = u + step;
    const bool more = next < it.u1;
    f32x4_t sc[2][NT];
    x.scores(qf, sc);
    if (more) {
      part(next);
      x.load_k(a, lo, hi);
    }
    acc.take(sc, x.vr, it, 32 * u, good, a.scale2);
    if (!more) break;
    x.load_v(a, lo, hi);
    u = next;
  }
}

// The same with the keys by way of LDS: two slots of the wavefront's own, filled
// straight from the pages, whole rows at a time, two units ahead.  Read into
// registers as the product wants them, the lanes of a load touch 64 cache lines
// for 16 bytes each, and a compute unit gets 25 B a clock of them.
template <int D, int NT>
__device__ __forceinline__ void walk_lds(const AttendArgs& a, const Segment& it, uint32_t u, uint32_t step, uint8_t* slots,
                                         Sums<D, NT>& acc) {
  if (u >= it.u1) return;
  constexpr int kLoads = D / 16, kSlot = 64 * D;
  constexpr uint32_t kPieces = D / 8;
  const uint32_t lane = __lane_id();
  const bool upper = lane / 16 >= 2;
  u32x4_t qf[AttendShape<D>::kKs][NT];
  load_queries<D, NT>(a, it, 0, qf);
  int32_t id0 = page_id(a, it, 32 * u), id1 = page_id(a, it, 32 * u + 16);
  PagePart lo = page_part(a, it, id0, 32 * u, D), hi = page_part(a, it, id1, 32 * u + 16, D);
  uint32_t ahead = u + step;  // the unit whose keys are asked for next
  id0 = page_id(a, it, 32 * ahead);
  id1 = page_id(a, it, 32 * ahead + 16);
  auto keys = [&](const PagePart& l, const PagePart& h, uint8_t* to) {
    asm volatile("" ::: "memory");  // in the order that the waits count
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const uint32_t piece = 64 * y + lane, row = piece / kPieces, c = piece % kPieces;
      const uint32_t from = (row % 16) * D + 8 * key_piece<D, true>(row, c);
      __builtin_amdgcn_global_load_lds(a.k + (y < kLoads / 2 ? l.off : h.off) + from, to + 1024 * y, 16, 0, 0);
    }
    asm volatile("" ::: "memory");
  };
  // the queries have to be there before the loads in flight are counted
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int k = 0; k < AttendShape<D>::kKs; ++k) asm volatile("" : "+v"(qf[k][c]));
  Unit<D, NT> x;
  bool good = upper ? hi.known : lo.known;
  keys(lo, hi, slots);
  x.load_v(a, lo, hi);
  if (ahead < it.u1) {
    lo = page_part(a, it, id0, 32 * ahead, D);
    hi = page_part(a, it, id1, 32 * ahead + 16, D);
    keys(lo, hi, slots + kSlot);
    id0 = page_id(a, it, 32 * (ahead + step));
    id1 = page_id(a, it, 32 * (ahead + step) + 16);
  }
  uint32_t slot = 0;
  for (;;) {
    // lo, hi: the pages of the next unit, whose keys are in flight or here
    const uint32_t next = u + step;
    const bool more = next < it.u1;
    // behind this unit's keys: a unit's values (8 loads at least), and the next unit's keys
    if (more)
      wait_vmem<8 + kLoads>();
    else
      wait_vmem<8>();
    x.read_k(slots + slot);
    f32x4_t sc[2][NT];
    x.scores(qf, sc);
    const PagePart vlo = lo, vhi = hi;
    ahead = next + step;
    if (ahead < it.u1) {
      lo = page_part(a, it, id0, 32 * ahead, D);
      hi = page_part(a, it, id1, 32 * ahead + 16, D);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot's reads are done
      keys(lo, hi, slots + slot);
      id0 = page_id(a, it, 32 * (ahead + step));
      id1 = page_id(a, it, 32 * (ahead + step) + 16);
    }
    acc.take(sc, x.vr, it, 32 * u, good, a.scale2);
    if (!more) return;
    x.load_v(a, vlo, vhi);
    good = upper ? vhi.known : vlo.known;
    u = next;
    slot ^= kSlot;
  }
}

// Bytes of a wavefront's two key slots.
constexpr uint32_t key_slots(int d) { return 2 * 64 * d; }
// Whether W wavefronts' slots fit beside what else lies in LDS.
constexpr bool keys_fit(int d, int waves) { return waves * key_slots(d) <= (waves == 4 ? 96u : 128u) * 1024; }

template <int D, int NT, int W>
__device__ __forceinline__ void walk_units(const AttendArgs& a, const Segment& it, uint32_t u, uint32_t step, uint8_t* slots,
                                           Sums<D, NT>& acc) {
  if constexpr (keys_fit(D, W))
    walk_lds<D, NT>(a, it, u, step, slots, acc);
  else
    walk<D, NT>(a, it, u, step, acc);
}

// A wavefront's part of an item of at most 16 NT columns.
template <int D, int NT>
__device__ __forceinline__ void attend_alone(const AttendArgs& a, const Segment& it, uint8_t* slots) {
  Sums<D, NT> acc;
  walk_units<D, NT, 4>(a, it, it.u0, 1, slots, acc);
  const uint32_t lost = acc.lost(a, it, 0);
  acc.finish();
  if (__builtin_expect(lost == 0, 1)) return acc.store(a, it, 0, 0);
  acc.store(a, it, 0, lost);
  redo<D>(a, it, 0, lost);
}

// LDS of a workgroup: the fixed part, then the plan, then the ring of slots or
// the sums that the wavefronts exchange (never both).
struct LdsFixed {
  float m[8][32], l[8][32];  // [wavefront][column]
  uint32_t carry[8], lost[8];
};
template <int D, int W>
using Join = float[W][16][AttendShape<D>::kJLd];

// An item of at most 16 NT columns by a workgroup of W wavefronts, which take its
// units in turn; their sums are divided by the whole of the weights, at one
// maximum, and then added in order, so that finite values never pass FP32's range
// on the way.
template <int D, int NT, int W>
__device__ __forceinline__ void attend_turns(const AttendArgs& a, const Segment& it, LdsFixed& s, uint8_t* big) {
  constexpr int kDt = AttendShape<D>::kDt;
  Join<D, W>& join = *reinterpret_cast<Join<D, W>*>(big);  // in the place of the key slots
  const uint32_t wave = uniform(threadIdx.x / kWave), tid = threadIdx.x;
  const uint32_t n = __lane_id() % 16, g = __lane_id() / 16;
  Sums<D, NT> acc;
  __syncthreads();  // the last readers of what lies there are done
  walk_units<D, NT, W>(a, it, it.u0 + wave, W, big + wave * key_slots(D), acc);
  const uint32_t lost = acc.lost(a, it, 0);
  if (__lane_id() == 0) s.lost[wave] = lost;
  acc.finish();
  if (g == 0)
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      s.m[wave][16 * c + n] = acc.m[c];
      s.l[wave][16 * c + n] = acc.l[c];
    }
  __syncthreads();
  uint32_t any = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) any |= s.lost[w];
  any = uniform(any);
  auto whole = [&](uint32_t col, float& best, float& total) {  // a column's maximum and sum of the weights
    best = s.m[0][col];
#pragma unroll
    for (int w = 1; w < W; ++w) best = fmaxf(best, s.m[w][col]);
    total = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) total += s.l[w][col] * __builtin_amdgcn_exp2f((s.m[w][col] - best) * a.scale2);
  };
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    float best, total;
    whole(16 * c + n, best, total);
    const float f = total == 0.f ? 0.f : __builtin_amdgcn_exp2f((acc.m[c] - best) * a.scale2) / total;
    if (c) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* dst = &join[wave][n][kDt * (4 * g + i)];
#pragma unroll
      for (int d = 0; d < kDt; ++d) dst[d] = acc.o[d][c][i] * f;
    }
    __syncthreads();
    for (uint32_t i = tid; i < 16 * (D / 4); i += W * kWave) {
      const uint32_t col = i / (D / 4), e = i % (D / 4) * 4, cc = 16 * c + col;
      if (cc >= it.cols || any >> cc & 1) continue;
      f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const f32x4_t*>(&join[w][col][e]);
      if (it.direct) {
        const uint32_t cl = it.col0 + cc, row = it.row0 + cl / a.ratio, h = it.head * a.ratio + cl % a.ratio;
        const u32x2_t w = {pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
        *reinterpret_cast<u32x2_t*>(a.out + row * a.ldo + static_cast<uint64_t>(h) * D + e) = w;
        continue;
      }
      *reinterpret_cast<f32x4_t*>(a.part_o + (it.slot + cc) * D + e) = sum;
      if (e == 0) {
        float best, total;
        whole(cc, best, total);
        a.part_ml[2 * (it.slot + cc)] = best;
        a.part_ml[2 * (it.slot + cc) + 1] = total;
      }
    }
  }
  static_assert(W == 4 || W == 8, "the wavefronts' bits");
  if (__builtin_expect(any != 0, 0)) redo<D>(a, it, 0, any & (W == 4 ? 0x11111111u : 0x01010101u) << wave);
}

// Wait until at most N of this wavefront's vector memory operations are left
// and all its LDS operations are done, then for the other wavefronts.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 0xF) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The workgroup's part of an item of more than 16 columns: the wavefronts take
// 16 NT columns each of the same units, which pass through a ring of slots in
// LDS, loaded straight from the pages (a quarter of a unit's rows per
// wavefront, kRing - 1 units ahead), so a unit is read once per workgroup.
// One barrier per unit i: behind it unit i + 1 has landed for all, so that its
// keys can be read while unit i is weighed, and the slot of unit i - 1 is free.
// A slot holds 32 rows of keys, then of values; the 16-byte pieces of a key row
// are permuted by the row, so that the 16 rows that one operand read touches lie
// in 64 different banks.
template <int D, int NT>
__device__ __forceinline__ void attend_shared(const AttendArgs& a, const Segment& it, uint8_t* slots) {
  using S = AttendShape<D>;
  constexpr int kDt = S::kDt, kKs = S::kKs, kLoads = (D + 63) / 64;
  constexpr uint32_t kPieces = D / 8, kSlotBytes = 128 * D, kRing = S::kRing, kAhead = kRing - 1;
  const uint32_t lane = __lane_id(), wave = uniform(threadIdx.x / kWave);
  const uint32_t n = lane % 16, g = lane / 16, units = it.u1 - it.u0;
  uint32_t seen = 0;  // two bits a unit, the last 16 units: the pages of its halves exist
  int32_t id0 = 0, id1 = 0;
  auto ask = [&](uint32_t i) {  // page numbers of unit i, a unit ahead of their use
    id0 = page_id(a, it, 32 * (it.u0 + i));
    id1 = page_id(a, it, 32 * (it.u0 + i) + 16);
  };
  auto issue = [&](uint32_t i, uint32_t at) {  // this wavefront's 8 rows of unit i into slot `at`
    const uint32_t pos = 32 * (it.u0 + i);
    const PagePart lo = page_part(a, it, id0, pos, D), hi = page_part(a, it, id1, pos + 16, D);
    const uint64_t off = (wave < 2 ? lo.off : hi.off) + wave % 2 * (8 * D);
    uint8_t* to = slots + at * kSlotBytes + wave * (16 * D);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const uint32_t piece = 64 * x + lane, row = piece / kPieces, c = piece % kPieces;
      if (64 * (x + 1) <= 8 * kPieces || piece < 8 * kPieces) {  // D = 96: the second load is half a wavefront
        __builtin_amdgcn_global_load_lds(a.k + off + row * D + 8 * key_piece<D, true>(8 * wave + row, c), to + 1024 * x, 16, 0, 0);
        __builtin_amdgcn_global_load_lds(a.v + off + row * D + 8 * c, to + 64 * D + 1024 * x, 16, 0, 0);
      }
    }
    const uint32_t sh = 2 * (i % 16);
    seen = (seen & ~(3u << sh)) | ((lo.known ? 1u : 0u) | (hi.known ? 2u : 0u)) << sh;
  };

  u32x4_t qf[kKs][NT];
  load_queries<D, NT>(a, it, wave * (16 * NT), qf);
  // the queries have to be there before the loads in flight are counted
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int k = 0; k < kKs; ++k) asm volatile("" : "+v"(qf[k][c]));
  __syncthreads();  // the slots' last readers are done
  ask(0);
  for (uint32_t i = 0; i < kAhead && i < units; ++i) {
    issue(i, i);
    ask(i + 1);
  }
  Sums<D, NT> acc;
  Unit<D, NT> x;
  // unit 0 has landed when at most the kAhead - 1 units behind it are in flight
  if (units >= kAhead)
    wait_and_meet<2 * kLoads*(kAhead - 1)>();
  else
    wait_and_meet<0>();
  x.read_k(slots);
  uint32_t at = 0;  // slot of unit i
  for (uint32_t i = 0; i < units; ++i) {
    // unit i + 1 has landed when at most the kAhead - 2 units behind it are in flight
    if (i + kAhead <= units)
      wait_and_meet<2 * kLoads*(kAhead - 2)>();
    else
      wait_and_meet<0>();
    const uint32_t after = at + 1 == kRing ? 0 : at + 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* v = slots + at * kSlotBytes + 64 * D + 2 * ((8 * g + j) * D + kDt * n);
      if constexpr (kDt % 8 == 0) {
#pragma unroll
        for (int e = 0; e < kDt / 8; ++e) {
          const u32x4_t y = reinterpret_cast<const u32x4_t*>(v)[e];
#pragma unroll
          for (int q = 0; q < 4; ++q) x.vr[j][4 * e + q] = y[q];
        }
      } else if constexpr (kDt % 4 == 0) {
#pragma unroll
        for (int e = 0; e < kDt / 4; ++e) {
          const u32x2_t y = reinterpret_cast<const u32x2_t*>(v)[e];
          x.vr[j][2 * e] = y[0];
          x.vr[j][2 * e + 1] = y[1];
        }
      } else {
#pragma unroll
        for (int e = 0; e < kDt / 2; ++e) x.vr[j][e] = reinterpret_cast<const uint32_t*>(v)[e];
      }
    }
    f32x4_t sc[2][NT];
    x.scores(qf, sc);
    if (i + 1 < units) x.read_k(slots + after * kSlotBytes);
    if (i + kAhead < units) {
      issue(i + kAhead, at == 0 ? kRing - 1 : at - 1);
      ask(i + kAhead + 1);
    }
    acc.take(sc, x.vr, it, 32 * (it.u0 + i), (seen >> (2 * (i % 16) + g / 2) & 1) != 0, a.scale2);
    at = after;
  }
  const uint32_t col = wave * (16 * NT);
  const uint32_t lost = acc.lost(a, it, col);
  acc.finish();
  if (__builtin_expect(lost == 0, 1)) return acc.store(a, it, col, 0);
  acc.store(a, it, col, lost);
  redo<D>(a, it, col, lost);
}

// Largest i in [0, n) with pre[i] <= x (pre ascending, pre[0] = 0).
__device__ __forceinline__ uint32_t find_last(const uint32_t* pre, uint32_t n, uint32_t x) {
  uint32_t lo = 0, hi = n;
  while (lo + 1 < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The item of own positions that unit `rem` of a head belongs to, and the part
// of it from there on, at most `left` units.
__device__ __forceinline__ Segment own_segment(const AttendArgs& a, const Plan& p, uint32_t head, uint32_t rem, uint64_t left,
                                               uint64_t worker) {
  const uint32_t r = uniform(find_last(p.row_pre, a.pages.rows, rem));
  const uint32_t done = rem - uniform(p.row_pre[r]);
  Segment it;
  it.head = head;
  it.row0 = r;
  it.col0 = 0;
  it.cols = a.ratio;
  it.ids = a.pages.ids + static_cast<uint64_t>(r) * a.pages.ld;
  it.p0 = uniform(p.base(r));
  it.p1 = uniform(p.row_end[r]);
  const uint32_t first = it.p0 / 32, units = (it.p1 + 31) / 32 - first;
  it.u0 = first + done;
  it.u1 = it.u0 + static_cast<uint32_t>(min(static_cast<uint64_t>(units - done), left));
  it.direct = it.p0 == 0 && it.u1 - it.u0 == units;
  it.prefix = false;
  it.slot = part_slot(a, false, head, r, 0, worker);
  return it;
}

// The same for prefixes.
__device__ __forceinline__ Segment prefix_segment(const AttendArgs& a, const Plan& p, uint32_t head, uint32_t rem, uint64_t left,
                                                  uint64_t worker) {
  const uint32_t i = uniform(find_last(p.g_pre, a.n_groups, rem));
  const uint32_t len = uniform(p.g_len[i]), units = (len + 31) / 32, in = rem - uniform(p.g_pre[i]);
  const uint32_t block = in / units, done = in - block * units;
  const uint32_t r = uniform(p.g_row[i]);
  Segment it;
  it.head = head;
  it.row0 = uniform(p.g_start[i]);
  it.col0 = block * kCap;
  it.cols = min((uniform(p.g_start[i + 1]) - it.row0) * a.ratio - it.col0, kCap);
  it.ids = a.pages.ids + static_cast<uint64_t>(r) * a.pages.ld;
  it.p0 = 0;
  it.p1 = len;
  it.u0 = done;
  it.u1 = done + static_cast<uint32_t>(min(static_cast<uint64_t>(units - done), left));
  it.direct = false;
  it.prefix = true;
  it.group = i;
  it.groups = p.row_group;
  it.slot = part_slot(a, true, head, it.row0, it.col0, worker);
  return it;
}

template <int D>
__global__ __launch_bounds__(kAttendThreads, D <= 128 ? 2 : 1) void k_attend(const AttendArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  LdsFixed& s = *reinterpret_cast<LdsFixed*>(lds);
  const uint32_t rows = a.pages.rows, G = a.n_groups;
  const Plan p(reinterpret_cast<uint32_t*>(lds + sizeof(LdsFixed)), rows, G);
  uint8_t* big = lds + sizeof(LdsFixed) + (Plan::words(rows, G) * 4 + 15) / 16 * 16;
  const Split split = make_plan(a, p, s.carry);
  const uint32_t prefix_units = split.prefix_units, own_units = split.own_units;
  if (prefix_units) {
    const uint64_t quota = split.prefix_quota;
    const uint64_t total = static_cast<uint64_t>(prefix_units) * a.hkv;
    // workgroups go round the 8 XCDs in turn: neighbours in the order of the
    // units, which share a head's pages, on one XCD if all have work
    const uint32_t wp = split.prefix_wgs;
    const bool near = wp % 8 == 0 && blockIdx.x < wp && total > quota * (wp / 2);
    const uint64_t wg = near ? blockIdx.x % 8 * (wp / 8) + blockIdx.x / 8 : blockIdx.x;
    const uint64_t end = min(wg * quota + quota, total);
    for (uint64_t at = wg * quota; at < end;) {
      const uint32_t head = static_cast<uint32_t>(at / prefix_units);
      const Segment it = prefix_segment(a, p, head, static_cast<uint32_t>(at % prefix_units), end - at, wg);
      if (it.cols <= 16)
        attend_turns<D, 1, 4>(a, it, s, big);
      else if (it.cols <= 64)
        attend_shared<D, 1>(a, it, big);
      else
        attend_shared<D, 2>(a, it, big);
      at += it.u1 - it.u0;
    }
  }
  if (own_units) {
    const uint64_t quota = split.own_quota;
    const uint64_t total = static_cast<uint64_t>(own_units) * a.hkv;
    // from the last workgroup down
    const uint32_t wg = gridDim.x - 1 - blockIdx.x;
    if (wg >= a.own_wgs) return;
    __syncthreads();  // the prefixes' last readers of LDS are done
    uint8_t* slots = big + uniform(threadIdx.x / kWave) * key_slots(D);
    const uint64_t worker = a.ratio <= kWaveRatio ? static_cast<uint64_t>(uniform(threadIdx.x / kWave)) * a.own_wgs + wg : wg;
    const uint64_t end = min(worker * quota + quota, total);
    for (uint64_t at = worker * quota; at < end;) {
      const uint32_t head = static_cast<uint32_t>(at / own_units);
      const Segment it = own_segment(a, p, head, static_cast<uint32_t>(at % own_units), end - at, worker);
      if (a.ratio <= 16) {
        attend_alone<D, 1>(a, it, slots);
      } else if (a.ratio <= kWaveRatio) {
        attend_alone<D, 2>(a, it, slots);
      } else {
        attend_shared<D, 1>(a, it, big);
      }
      at += it.u1 - it.u0;
    }
  }
}

// Short tables: one workgroup per row, key-value head and 32 query heads of it
// takes all of the row's positions, its wavefronts in turn.  One launch, no plan
// and no partial sums.
template <int D>
__global__ __launch_bounds__(AttendShape<D>::kRowWaves * kWave) void k_attend_rows(const AttendArgs a) {
  constexpr int kRowWaves = AttendShape<D>::kRowWaves;
  __shared__ LdsFixed s;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t r = blockIdx.x / a.hkv;
  const int32_t len = sload(a.lengths, r);
  if (len < 0) return;  // padding
  Segment it;
  it.head = blockIdx.x % a.hkv;
  it.row0 = r;
  it.col0 = blockIdx.y * kWaveRatio;
  it.cols = min(a.ratio - it.col0, kWaveRatio);
  it.ids = a.pages.ids + static_cast<uint64_t>(r) * a.pages.ld;
  it.p0 = 0;
  it.p1 = min(static_cast<uint32_t>(len), a.pages.cols << a.pages.shift);
  it.u0 = 0;
  it.u1 = (it.p1 + 31) / 32;
  it.direct = true;
  it.prefix = false;
  it.slot = 0;
  if (it.cols <= 16)
    attend_turns<D, 1, kRowWaves>(a, it, s, lds);
  else
    attend_turns<D, 2, kRowWaves>(a, it, s, lds);
}

// One workgroup per row and query head: the parts of its column, prefix first,
// each the mean of its values, its maximum and the sum of its weights.  D / 4
// threads hold a column's components; the parts go round kLines such lines, each
// keeps a running maximum, and the lines are added in order.  Sums that come out
// infinite or NaN are taken once more by each part's share of one, which keeps
// means of finite values in their range and an infinity what it is, however small
// its weight.  (A running mean from the start, a division a part: 5000 positions of
// one row with heads of 256 18 -> 30 us.)
template <int D>
__global__ __launch_bounds__(kAttendThreads) void k_attend_join(const AttendArgs a) {
  constexpr uint32_t kLine = D / 4, kLines = kAttendThreads / kLine;
  __shared__ f32x4_t sums[kLines][kLine];
  __shared__ float ms[kLines], ls[kLines];
  const uint32_t rows = a.pages.rows, r = blockIdx.x / a.hq, h = blockIdx.x % a.hq, head = h / a.ratio, j = h % a.ratio;
  const u32x4_t* rec = reinterpret_cast<const u32x4_t*>(a.plan);
  const u32x4_t h0 = rec[0], h1 = rec[1], row = rec[2 + r];
  const uint32_t prefix_units = h0[0], own_units = h0[1], pre = row[0], units = row[1], g = row[2];
  const uint64_t quota_p = h1[0] | static_cast<uint64_t>(h1[1]) << 32, quota_o = h1[2] | static_cast<uint64_t>(h1[3]) << 32;
  if (static_cast<int32_t>(row[3]) < 0) return;  // padding
  const bool shares = g < a.n_groups;
  // the worker that has a unit (32-bit division where the numbers allow)
  auto owner = [](uint64_t x, uint64_t quota) -> uint32_t {
    return static_cast<uint32_t>((x | quota) >> 32 ? x / quota : static_cast<uint32_t>(x) / static_cast<uint32_t>(quota));
  };
  uint32_t n0 = 0, n1 = 0;  // parts of the prefix, of the own positions
  uint64_t slot0 = 0, slot1 = 0;
  if (shares) {
    const u32x4_t group = rec[2 + rows + g];
    const uint32_t first_row = group[0], col = (r - first_row) * a.ratio + j, block = col / kCap, n = (group[2] + 31) / 32;
    const uint64_t first = static_cast<uint64_t>(prefix_units) * head + group[1] + static_cast<uint64_t>(block) * n;
    const uint32_t w = owner(first, quota_p);
    n0 = owner(first + n - 1, quota_p) - w + 1;
    slot0 = part_slot(a, true, head, first_row, block * kCap, w) + col % kCap;
  }
  if (units) {
    const uint64_t first = static_cast<uint64_t>(own_units) * head + pre;
    const uint32_t w = owner(first, quota_o);
    n1 = owner(first + units - 1, quota_o) - w + 1;
    slot1 = part_slot(a, false, head, r, 0, w) + j;
    if (!shares && n1 == 1) return;  // k_attend wrote the output itself
  }
  const uint32_t line = threadIdx.x / kLine, e = threadIdx.x % kLine * 4, parts = n0 + n1;
  auto load = [&](uint32_t i, float2& ml) {
    const uint64_t at = i < n0 ? slot0 + static_cast<uint64_t>(i) * a.cap_p : slot1 + static_cast<uint64_t>(i - n0) * a.cap_o;
    ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
    return *reinterpret_cast<const f32x4_t*>(a.part_o + at * D + e);
  };
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  float best = kNoMax, total = 0.f;
  if (line < kLines) {
#pragma unroll 4
    for (uint32_t i = line; i < parts; i += kLines) {
      float2 ml;
      const f32x4_t x = load(i, ml);
      const float top = fmaxf(best, ml.x);
      const float f = __builtin_amdgcn_exp2f((best - top) * a.scale2), f2 = ml.y * __builtin_amdgcn_exp2f((ml.x - top) * a.scale2);
      sum = sum * f + x * f2;
      total = total * f + f2;
      best = top;
    }
    sums[line][e / 4] = sum;
    if (e == 0) {
      ms[line] = best;
      ls[line] = total;
    }
  }
  __syncthreads();
  if (line != 0) return;
  for (uint32_t i = 1; i < kLines; ++i) best = fmaxf(best, ms[i]);
  sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
  total = 0.f;
#pragma unroll
  for (uint32_t i = 0; i < kLines; ++i) {
    const float f = __builtin_amdgcn_exp2f((ms[i] - best) * a.scale2);
    sum += sums[i][e / 4] * f;
    total += ls[i] * f;
  }
  const float f = total == 0.f ? 0.f : 1.f / total;
  const float zero = (sum[0] * 0.f + sum[1] * 0.f) + (sum[2] * 0.f + sum[3] * 0.f);
  sum *= f;
  if (__builtin_expect(!(zero == 0.f), 0) && total == total) {
    sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (uint32_t i = 0; i < parts; ++i) {
      float2 ml;
      const f32x4_t x = load(i, ml);
      const float w = ml.y * __builtin_amdgcn_exp2f((ml.x - best) * a.scale2) * f;
      for (int j = 0; j < 4; ++j) sum[j] += w == 0.f && __builtin_isinf(x[j]) ? x[j] : x[j] * w;
    }
  }
  uint2 w;
  w.x = pack_bf16(sum[0], sum[1]);
  w.y = pack_bf16(sum[2], sum[3]);
  *reinterpret_cast<uint2*>(a.out + r * a.ldo + static_cast<uint64_t>(h) * D + e) = w;
}

// ------------------------------------------------------------------- host ---

nwc_status check_rope(const nwc_rope* rope, uint32_t d) {
  if (!rope || rope->dims == 0) return NWC_OK;
  if (!rope->freqs || rope->dims > d || rope->style > NWC_ROPE_PAIRS) return NWC_ERR_INVALID_ARG;
  if (rope->dims % 8) return NWC_ERR_UNSUPPORTED;
  return aligned(rope->freqs, 4) ? NWC_OK : NWC_ERR_ALIGNMENT;
}

nwc_status check_heads(const nwc_heads* h, uint32_t d, bool to_rows) {
  if (!h->src || h->heads == 0 || h->heads > kMaxHeads || h->reserved || (to_rows && !h->dst)) return NWC_ERR_INVALID_ARG;
  const uint64_t row = static_cast<uint64_t>(h->heads) * d;
  if (h->ld_src < row || h->ld_src > kMaxStride || (to_rows && (h->ld_dst < row || h->ld_dst > kMaxStride)))
    return NWC_ERR_INVALID_ARG;
  if (!aligned(h->src, 16) || !aligned(h->weight, 16) || h->ld_src % 8) return NWC_ERR_ALIGNMENT;
  if (to_rows && (!aligned(h->dst, 16) || h->ld_dst % 8)) return NWC_ERR_ALIGNMENT;
  if (to_rows && h->dst == h->src && h->ld_dst != h->ld_src) return NWC_ERR_INVALID_ARG;
  return NWC_OK;
}

nwc_status launch_heads(HeadsArgs& a, hipStream_t s) {
  const uint32_t all = a.hq + a.hk + a.hv, lanes = a.d / 8u;
  const uint32_t g = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const uint32_t passes = (all + kWave / g - 1) / (kWave / g);
  // one pass per wavefront while that leaves compute units idle, else four at a
  // time, a token's passes over as many wavefronts as it takes to have 16 per
  // compute unit
  const uint32_t want = kCus * 16;
  const bool few = static_cast<uint64_t>(a.tokens) * passes < want;
  a.split = few ? passes : std::min((passes + 3) / 4, std::max(1u, want / a.tokens));
  const uint64_t waves = static_cast<uint64_t>(a.tokens) * a.split;
  // a launch holds fewer than 2^32 threads; more tokens go round
  const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>((waves + 3) / 4, uint64_t{1} << 22));
  auto go = [&](auto one, auto four) { return launch(few ? one : four, dim3(grid), dim3(256), 0, s, a); };
  if (g == 8) return go(k_heads<8, 1>, k_heads<8, 4>);
  if (g == 16) return go(k_heads<16, 1>, k_heads<16, 4>);
  return go(k_heads<32, 1>, k_heads<32, 4>);
}

bool heads_dim_ok(uint32_t d) { return d >= 8 && d <= 256 && d % 8 == 0; }

void set_rope(HeadsArgs* a, const nwc_rope* rope) {
  if (rope && rope->dims) {
    a->freqs = rope->freqs;
    a->half = static_cast<uint16_t>(rope->dims / 2);
    a->style = static_cast<uint16_t>(rope->style);
  }
}

// Workspace of nwc_attend: partial sums, maxima and sums, the plan.
constexpr uint32_t kAttendMaxRows = 4096, kAttendMaxGroups = 512, kAttendMaxRatio = 64, kAttendMaxLen = 1u << 22;
constexpr uint64_t kAttendMaxCols = 1u << 22;  // rows times query heads: a workgroup each, of 2^32 - 1 threads a launch
struct AttendLayout {
  uint64_t own_slot, ml, plan, bytes;
  uint32_t cap_p, cap_o;
};
AttendLayout attend_layout(uint32_t rows, uint32_t q_heads, uint32_t ratio, uint32_t groups, uint32_t d) {
  AttendLayout L;
  const uint64_t cols = static_cast<uint64_t>(rows) * q_heads;
  L.cap_p = groups ? std::min(kCap, rows * ratio) : 0;
  L.cap_o = ratio;
  L.own_slot = groups ? cols + uint64_t{kCus} * L.cap_p : 0;
  const uint64_t slots = L.own_slot + cols + uint64_t{kCus} * (ratio <= kWaveRatio ? 4 : 1) * L.cap_o;
  auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
  L.ml = up(slots * d * 4);
  L.plan = L.ml + up(slots * 8);
  L.bytes = L.plan + up(Plan::record_words(rows, groups) * 4);
  return L;
}

nwc_status attend_shape(const nwc_cache* c, uint32_t rows, uint32_t q_heads, uint32_t groups) {
  if (!c || rows == 0 || q_heads == 0 || c->kv_heads == 0) return NWC_ERR_INVALID_ARG;
  const uint32_t d = c->head_dim;
  if (d != 64 && d != 96 && d != 128 && d != 192 && d != 256) return NWC_ERR_UNSUPPORTED;
  if (q_heads % c->kv_heads) return NWC_ERR_INVALID_ARG;
  if (rows > kAttendMaxRows || groups > kAttendMaxGroups || q_heads / c->kv_heads > kAttendMaxRatio || q_heads > kMaxHeads ||
      static_cast<uint64_t>(rows) * q_heads > kAttendMaxCols)
    return NWC_ERR_UNSUPPORTED;
  return NWC_OK;
}

// Positions that a table may cover for k_attend_rows to take it, by the number of
// its workgroups (rows times key-value heads) against the compute units.
// Measured (32 / 8 heads of 128, us a call in a graph, k_attend_rows and k_attend
// + k_attend_join): 1 row of 512: 6.1 and 8.1, 1024: 8.3 and 8.1; 4 rows of 1024:
// 9.7 and 11.3, 2048: 15.0 and 12.9; 16 rows of 2048: 28.7 and 31.6, ragged to
// 2048: 16.5 and 19.1, to 4096: 44.8 and 33.1; 64 rows of 2048: 92.5 and 98.4.
// Heads of 256, whose keys have no room in LDS, gain less: 1 row of 256 positions
// (8 / 4 heads) 9.0 and 10.8, of 512 13.4 and 10.7; 32 rows of 1024 37.6 and 40.6.
// Rows that share a prefix read it each for itself here, from the caches, which
// is faster while that is little: 16 rows behind 384 positions with 100 of their
// own 7.0 and 13.8, 64 rows behind 896 19.4 and 23.1.
bool by_rows(uint32_t d, uint64_t groups, uint32_t covers, bool shared) {
  const bool many = 2 * groups >= kCus;
  if (shared) return covers <= (d == 256 ? 256 : 1024) && groups * covers * d <= 1 << 26;
  if (d == 256) return covers <= (many ? 1024 : 256);
  return covers <= (many ? 2048 : 8 * groups >= kCus ? 1024 : 512);
}

template <int D>
nwc_status launch_attend(AttendArgs& a, uint32_t grid, hipStream_t s) {
  const uint64_t items = static_cast<uint64_t>(a.pages.rows) * a.hkv;
  if (by_rows(D, items, a.pages.cols << a.pages.shift, a.n_groups != 0)) {
    constexpr int kRowWaves = AttendShape<D>::kRowWaves;
    constexpr size_t lds = std::max(sizeof(Join<D, kRowWaves>), keys_fit(D, kRowWaves) ? size_t{kRowWaves * key_slots(D)} : 0);
    static_assert(sizeof(LdsFixed) + lds <= kMaxLds, "LDS");
    if (lds + sizeof(LdsFixed) > 65536 && !allow_lds<k_attend_rows<D>, lds>()) return NWC_ERR_HIP;
    return launch(k_attend_rows<D>, dim3(a.pages.rows * a.hkv, (a.ratio + kWaveRatio - 1) / kWaveRatio),
                  dim3(kRowWaves * kWave), lds, s, a);
  }
  const size_t fixed = sizeof(LdsFixed) + (static_cast<size_t>(Plan::words(a.pages.rows, a.n_groups)) * 4 + 15) / 16 * 16;
  constexpr size_t big = std::max({sizeof(Join<D, 4>), size_t{AttendShape<D>::kRing * 128 * D}, keys_fit(D, 4) ? size_t{4 * key_slots(D)} : 0});
  constexpr size_t most = sizeof(LdsFixed) + 4 * Plan::words(kAttendMaxRows, kAttendMaxGroups) + 16 + big;
  static_assert(most <= kMaxLds, "LDS");
  const size_t lds = fixed + big;
  if (lds > 65536 && !allow_lds<k_attend<D>, most>()) return NWC_ERR_HIP;
  const nwc_status st = launch(k_attend<D>, dim3(grid), dim3(kAttendThreads), lds, s, a);
  if (st) return st;
  return launch(k_attend_join<D>, dim3(a.pages.rows * a.hq), dim3(kAttendThreads), 0, s, a);
}

}  // namespace

extern "C" {

nwc_status nwc_qk_norm_rope(const nwc_heads* q, const nwc_heads* k, uint32_t tokens, uint32_t head_dim, float eps,
                            const nwc_rope* rope, const int32_t* positions_dev, void* stream) {
  if ((!q && !k) || tokens == 0 || !positions_dev || !(eps >= 0.f) || !std::isfinite(eps) || head_dim == 0)
    return NWC_ERR_INVALID_ARG;
  if (!heads_dim_ok(head_dim)) return NWC_ERR_UNSUPPORTED;
  if (!aligned(positions_dev, 4)) return NWC_ERR_ALIGNMENT;
  nwc_status st = check_rope(rope, head_dim);
  if (!st && q) st = check_heads(q, head_dim, true);
  if (!st && k) st = check_heads(k, head_dim, true);
  if (st) return st;
  HeadsArgs a = {};
  if (q) {
    a.q = q->src; a.q_out = q->dst; a.q_weight = q->weight; a.ld_q = pieces(q->ld_src); a.ld_q_out = pieces(q->ld_dst); a.hq = static_cast<uint16_t>(q->heads);
  }
  if (k) {
    a.k = k->src; a.k_out = k->dst; a.k_weight = k->weight; a.ld_k = pieces(k->ld_src); a.ld_k_out = pieces(k->ld_dst); a.hk = static_cast<uint16_t>(k->heads);
  }
  set_rope(&a, rope);
  a.positions = positions_dev;
  a.tokens = tokens;
  a.d = static_cast<uint16_t>(head_dim);
  a.eps = eps;
  return launch_heads(a, static_cast<hipStream_t>(stream));
}

nwc_status nwc_kv_append(const nwc_cache* cache, const nwc_page_table* table, const nwc_heads* k, const uint16_t* v_dev,
                         uint64_t ld_v, const nwc_heads* q, uint32_t tokens, float eps, const nwc_rope* rope,
                         const int32_t* positions_dev, const int32_t* rows_dev, void* stream) {
  if (!cache || !table || !k || !v_dev || tokens == 0 || !positions_dev || !(eps >= 0.f) || !std::isfinite(eps) ||
      cache->head_dim == 0)
    return NWC_ERR_INVALID_ARG;
  const uint32_t d = cache->head_dim;
  if (!heads_dim_ok(d)) return NWC_ERR_UNSUPPORTED;
  HeadsArgs a = {};
  nwc_status st = check_cache(cache, table, &a.pages);
  if (!st) st = check_rope(rope, d);
  if (!st) st = check_heads(k, d, false);
  if (!st && q) st = check_heads(q, d, true);
  if (st) return st;
  if (k->heads != cache->kv_heads || ld_v < static_cast<uint64_t>(k->heads) * d || ld_v > kMaxStride) return NWC_ERR_INVALID_ARG;
  if (!rows_dev && tokens > table->rows) return NWC_ERR_INVALID_ARG;  // token t is row t
  if (!aligned(v_dev, 16) || ld_v % 8 || !aligned(positions_dev, 4) || !aligned(rows_dev, 4)) return NWC_ERR_ALIGNMENT;
  if (q) {
    a.q = q->src; a.q_out = q->dst; a.q_weight = q->weight; a.ld_q = pieces(q->ld_src); a.ld_q_out = pieces(q->ld_dst); a.hq = static_cast<uint16_t>(q->heads);
  }
  a.k = k->src; a.k_out = cache->k; a.k_weight = k->weight; a.ld_k = pieces(k->ld_src); a.hk = static_cast<uint16_t>(k->heads);
  a.v = v_dev; a.v_out = cache->v; a.ld_v = pieces(ld_v); a.hv = a.hk;
  set_rope(&a, rope);
  a.positions = positions_dev;
  a.rows = rows_dev;
  a.tokens = tokens;
  a.d = static_cast<uint16_t>(d);
  a.eps = eps;
  return launch_heads(a, static_cast<hipStream_t>(stream));
}

nwc_status nwc_attend_workspace_size(const nwc_cache* cache, uint32_t rows, uint32_t q_heads, uint32_t n_groups, size_t* bytes) {
  if (!bytes) return NWC_ERR_INVALID_ARG;
  const nwc_status st = attend_shape(cache, rows, q_heads, n_groups);
  if (st) return st;
  *bytes = attend_layout(rows, q_heads, q_heads / cache->kv_heads, n_groups, cache->head_dim).bytes;
  return NWC_OK;
}

nwc_status nwc_attend(const nwc_cache* cache, const nwc_page_table* table, const nwc_groups* groups, const int32_t* lengths_dev,
                      const uint16_t* q_dev, uint64_t ldq, uint32_t q_heads, float scale, uint16_t* out_dev, uint64_t ldo,
                      void* ws, size_t ws_bytes, void* stream) {
  if (!cache || !table || !lengths_dev || !q_dev || !out_dev || !ws || !std::isfinite(scale * kLog2e) || !(scale > 0.f))
    return NWC_ERR_INVALID_ARG;
  const uint32_t n_groups = groups ? groups->count : 0;
  if (groups && (groups->reserved || (n_groups && (!groups->start || !groups->len)))) return NWC_ERR_INVALID_ARG;
  AttendArgs a = {};
  nwc_status st = attend_shape(cache, table->rows, q_heads, n_groups);
  if (!st) st = check_cache(cache, table, &a.pages);
  if (st) return st;
  const uint32_t d = cache->head_dim, rows = table->rows;
  const uint64_t row = static_cast<uint64_t>(q_heads) * d;
  if (ldq < row || ldo < row || ldq > kMaxStride || ldo > kMaxStride) return NWC_ERR_INVALID_ARG;
  if ((static_cast<uint64_t>(table->cols) << a.pages.shift) > kAttendMaxLen) return NWC_ERR_UNSUPPORTED;
  if (!aligned(q_dev, 16) || !aligned(out_dev, 16) || ldq % 8 || ldo % 8 || !aligned(lengths_dev, 4) || !aligned(ws, 256) ||
      (n_groups && (!aligned(groups->start, 4) || !aligned(groups->len, 4))))
    return NWC_ERR_ALIGNMENT;
  const AttendLayout L = attend_layout(rows, q_heads, q_heads / cache->kv_heads, n_groups, d);
  if (ws_bytes < L.bytes) return NWC_ERR_BUFFER_TOO_SMALL;
  if (out_dev == q_dev) return NWC_ERR_INVALID_ARG;  // workgroups read queries that others have answered
  const uint32_t grid = n_groups ? 2 * kCus : kCus;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.k = cache->k;
  a.v = cache->v;
  a.q = q_dev;
  a.out = out_dev;
  a.lengths = lengths_dev;
  if (n_groups) {
    a.group_start = groups->start;
    a.group_len = groups->len;
  }
  a.ldq = ldq;
  a.ldo = ldo;
  a.hq = q_heads;
  a.hkv = cache->kv_heads;
  a.ratio = q_heads / cache->kv_heads;
  a.n_groups = n_groups;
  a.scale2 = scale * kLog2e;
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float*>(w + L.ml);
  a.plan = reinterpret_cast<uint32_t*>(w + L.plan);
  a.own_slot = L.own_slot;
  a.own_wgs = kCus;
  a.cap_p = L.cap_p;
  a.cap_o = L.cap_o;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (d) {
    case 64: return launch_attend<64>(a, grid, s);
    case 96: return launch_attend<96>(a, grid, s);
    case 128: return launch_attend<128>(a, grid, s);
    case 192: return launch_attend<192>(a, grid, s);
    default: return launch_attend<256>(a, grid, s);
  }
}

}  // extern "C"
