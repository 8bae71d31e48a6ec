// What the HIP sources of the attention side and of the step's other parts share:
// vector types and BF16 conversions on the device; on the host the launch, the
// LDS allowance and the checks of a paged cache.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <tuple>

#include "nwc.h"

namespace {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

constexpr int kWave = 64;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Two floats rounded to BF16 (nearest even), packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __builtin_bit_cast(float, v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __builtin_bit_cast(float, v & 0xFFFF0000u); }

__device__ __forceinline__ float lane_xor(float v, int mask) {
  return __builtin_bit_cast(float, __shfl_xor(__builtin_bit_cast(int, v), mask, kWave));
}

struct PageArgs {
  const int32_t* ids;
  uint32_t ld;
  uint32_t n_pages, stride8;   // pages; elements / 8 from page to page
  uint32_t rows, cols, shift;  // page_len = 1 << shift
};

// A wave-uniform read of an array that this grid does not write (scalar load).
__device__ __forceinline__ int32_t sload(const int32_t* p, uint64_t i) {
  typedef const __attribute__((address_space(4))) int32_t ci32;
  return ((ci32*)(reinterpret_cast<uintptr_t>(p)))[i];
}

// Wait until at most N of this wavefront's vector memory operations are left.
template <int N>
__device__ __forceinline__ void wait_vmem() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 0xF) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

// ------------------------------------------------------------------- host ---

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Launch a kernel and report that launch's own status.
template <typename... P, typename... A>
inline nwc_status launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t s, const A&... a) {
  static_assert(sizeof...(P) == sizeof...(A), "argument count");
  std::tuple<P...> args{static_cast<P>(a)...};
  void* argv[sizeof...(P)];
  std::apply([&](auto&... e) {
    int i = 0;
    ((argv[i++] = const_cast<void*>(static_cast<const void*>(&e))), ...);
  }, args);
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, argv, lds, s) == hipSuccess
             ? NWC_OK
             : NWC_ERR_HIP;
}

// Lets a kernel take up to MOST bytes of dynamic LDS on the current device.  What
// is allowed belongs to the kernel, for all threads: so the most that it ever
// takes, once, and never less for another call.
template <auto KERNEL, size_t MOST>
inline bool allow_lds() {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return false;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(MOST)) != hipSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// Compute units of an MI355X.  Launches are cut for them; nothing needs them to
// be there, so they are not asked for (two runtime calls less in a call of 4 us).
constexpr uint32_t kCus = 256;

// Most heads of one tensor, and strides that fit 32 bits in pieces of 8 elements.
constexpr uint32_t kMaxHeads = 65535;
constexpr size_t kMaxLds = 160 * 1024;
constexpr uint64_t kMaxStride = uint64_t{0xFFFFFFFF} * 8;
inline uint32_t pieces(uint64_t ld) { return static_cast<uint32_t>(ld / 8); }

inline nwc_status check_cache(const nwc_cache* c, const nwc_page_table* t, PageArgs* p) {
  if (!c || !c->k || !c->v || c->n_pages == 0 || c->n_pages > 0x7FFFFFFF || c->kv_heads == 0 || c->kv_heads > kMaxHeads ||
      c->page_len == 0 || c->reserved)
    return NWC_ERR_INVALID_ARG;
  if (c->page_len < 16 || c->page_len > 1024 || (c->page_len & (c->page_len - 1))) return NWC_ERR_UNSUPPORTED;
  if (c->page_stride < static_cast<uint64_t>(c->kv_heads) * c->page_len * c->head_dim || c->page_stride > kMaxStride)
    return NWC_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % 8) return NWC_ERR_ALIGNMENT;
  p->n_pages = static_cast<uint32_t>(c->n_pages);
  p->stride8 = pieces(c->page_stride);
  p->shift = static_cast<uint32_t>(__builtin_ctz(c->page_len));
  if (t) {
    if (!t->ids || t->rows == 0 || t->cols == 0 || t->ld < t->cols || t->ld > 0xFFFFFFFF) return NWC_ERR_INVALID_ARG;
    if (!aligned(t->ids, 4)) return NWC_ERR_ALIGNMENT;
    p->ids = t->ids;
    p->ld = static_cast<uint32_t>(t->ld);
    p->rows = t->rows;
    p->cols = t->cols;
  }
  return NWC_OK;
}

}  // namespace
