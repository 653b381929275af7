// Shared by the kernels of the paged K+V cache (slim_mha_paged_*): the cache as
// the kernels see it, the checks of a sequence's lengths, e4m3 conversions and
// the scale rule.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace slim {

// Exponent range of a page's scale. 448·2^120 covers every finite bf16; below 2^-100 nothing is
// left of a value that shares a row with ordinary ones.
constexpr int kScaleExpMin = -100;
constexpr int kScaleExpMax = 120;
// Softmax weights over e4m3 are held in f16, at 2^7 times their size relative to the row's running maximum of
// weight times value scale. That maximum may be 2^8 behind, so that they end at 2^15; upwards f16 has
// no other use, and downwards a page may then hold its full 11 bits at a scale 2^21 below the largest one that
// the row attends (one huge value row makes its page's scale so, whatever its own weight), and some at 2^31.
// The sum of weights, which holds 2^-lv of scales from 2^-100 to 2^120, stays without that factor; the
// output loses it with its last product.
constexpr float kWeightLog2 = 7.f, kWeightInv = 0.0078125f;
constexpr int kPagedMaxB = 4096;  // the decode plan holds one line offset per sequence in shared memory

// Plain loads for everything an earlier kernel of the stream may have written (lengths, page tables,
// scales, queries): these kernels are launched while that one may still run and wait for it inside, so
// nothing is constant for their whole lifetime as the read-only path requires.
template <typename T>
__device__ __forceinline__ T ld_plain(const T* p) {
  return *p;
}

struct PagedView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;
  int64_t num_pages;
  int B, Hkv, dh, page, max_pages;
  int page_shift;       // page = 1 << page_shift
  int64_t cap;          // max_pages * page
  int64_t head_bytes;   // bytes of one head of a page
  int64_t page_bytes;   // bytes of a page of one pool

  // page number of row t, or -1 where it is outside the pool
  __device__ __forceinline__ int page_of(int b, int64_t t) const {
    const int id = ld_plain(table + static_cast<int64_t>(b) * max_pages + (t >> page_shift));
    return id >= 0 && id < num_pages ? id : -1;
  }
};

struct PagedRows {
  int row0;  // first packed row
  int n;     // rows of the sequence
  int len;   // rows before them
  int bits;  // SLIM_DEV_* bits; non-zero: skip
  bool span; // starts[] themselves are valid: rows row0 .. row0+n-1 may be written
};

// Rows of sequence b and whether they may be used; limit is the number of positions there are.
__device__ __forceinline__ PagedRows paged_rows(const int32_t* starts, const int32_t* lens, int b, int64_t rows,
                                                int64_t max_new, int64_t cap, int64_t limit) {
  PagedRows r;
  const int s0 = ld_plain(starts + b), s1 = ld_plain(starts + b + 1);
  r.len = ld_plain(lens + b);
  r.row0 = s0;
  r.bits = 0;
  r.span = s0 >= 0 && s1 >= s0 && s1 <= rows;
  r.n = r.span ? s1 - s0 : 0;
  if (!r.span || r.n > max_new || r.len < 0 || r.len > cap)
    r.bits = SLIM_DEV_BADLEN;
  else if (static_cast<int64_t>(r.len) + r.n > (cap < limit ? cap : limit) && r.n > 0)
    r.bits = SLIM_DEV_OVERFLOW;
  return r;
}

// Least e with amax <= 448·2^e = 1.75·2^(8+e), from the bits of a finite amax >= 0.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kScaleExpMin, min(kScaleExpMax, e));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Exponent of a scale (a power of two); NaN for a poisoned page.
__device__ __forceinline__ float scale_log2(float s) {
  return s != s ? s : static_cast<float>(static_cast<int>(__float_as_uint(s) >> 23) - 127);
}

// Two e4m3 codes (lo in the low byte), rounded to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}
// e4m3 codes as f16 pairs (exact: f16 holds every e4m3 value); lo from the low two bytes, hi from the
// high two. In PTX so that each pair is one instruction, without the moves that put the CUDA
// function's two halves together again.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two floats rounded to a bf16 or f16 pair, lo in the low half: one instruction.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t round_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Host: raises a kernel's dynamic shared memory limit on the current device, once per device (the
// call costs about as much as a launch's argument setup). `done` belongs to the kernel.
inline cudaError_t allow_smem(const void* kern, uint32_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Host: the view of a checked cache.
inline PagedView paged_view(const slim_paged_cache& c) {
  PagedView v;
  v.k = static_cast<uint8_t*>(c.kpages);
  v.v = static_cast<uint8_t*>(c.vpages);
  v.ks = c.kscale;
  v.vs = c.vscale;
  v.table = c.table;
  v.num_pages = c.num_pages;
  v.B = c.B;
  v.Hkv = c.Hkv;
  v.dh = c.dh;
  v.page = c.page;
  v.max_pages = c.max_pages;
  v.page_shift = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
  v.cap = static_cast<int64_t>(c.max_pages) * c.page;
  v.head_bytes = static_cast<int64_t>(c.page) * c.dh * (c.dtype == SLIM_BF16 ? 2 : 1);
  v.page_bytes = v.head_bytes * c.Hkv;
  return v;
}

}  // namespace slim
