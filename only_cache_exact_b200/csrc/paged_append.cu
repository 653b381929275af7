// slim_mha_paged_append and slim_mha_paged_gather: rows of keys and values into
// the pages of a K+V cache, with the position rotation applied on the way, and
// rows read back.
//
// Mathematics. A rotated pair at position p with angle number i is
//     y = x·cos[p][i] - x'·sin[p][i],   y' = x'·cos[p][i] + x·sin[p][i],
// in fp32 (one product, one fused multiply-add), rounded once to what is
// stored. For e4m3 the stored code is y / 2^e, where 2^e is the scale of the
// page and head. A power of two makes the division exact, and a code that is
// carried over to a larger scale stays exact until it becomes subnormal, so
// appending token by token gives the values of appending all at once up to
// that.
//
// Bound: memory. An element is read in 2 bytes and written in 1 or 2; the angle
// tables add 8 bytes per pair and position, but they are shared by all heads,
// which is why one CTA takes several heads of the same rows.
//
// Layout of work. The unit is 16 elements of one row and head in two 16-byte loads:
// for the split style 8 columns and their 8 partners rot/2 further, for the
// interleaved one 16 neighbours, so that both elements of every pair are in one
// thread. append_rows_kernel gives a CTA one page of one sequence
// (the rows of it that are new) and a range of heads of K, V or q; with e4m3
// the rotated values of a head wait in registers for the page's largest
// magnitude, so the input is read once. append_token_kernel is the form for
// one row per sequence: the dh/16 threads of a row find its largest magnitude
// by shuffles, and a warp re-rounds a page together where a scale has grown.
#include <algorithm>

#include "paged.cuh"

namespace slim {

namespace {

constexpr int kAppThreads = 256;

struct AppendParams {
  PagedView c;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  const float* cosines;
  const float* sines;
  int rot;
  int64_t n_pos;
  const int32_t* starts;
  const int32_t* lens;
  int64_t rows, max_new;
  int Hq;
  __nv_bfloat16* q_out;
  int32_t* status;
  int heads_per_cta, kv_chunks, q_chunks;
};

// Column offsets of a unit's two 8-element vectors. Without rotation the halves of a row, so that
// neighbouring threads take neighbouring 16 bytes.
template <bool kPairs, int DH>
__device__ __forceinline__ void unit_columns(int i, int rot, int& e0, int& e1) {
  const int half = rot == 0 ? DH / 2 : rot / 2;
  const bool split = rot == 0 || (!kPairs && i * 16 < rot);
  e0 = split ? 8 * i : 16 * i;
  e1 = split ? half + 8 * i : 16 * i + 8;
}

struct RawUnit {
  uint4 a, b;
};
__device__ __forceinline__ RawUnit load_raw(const __nv_bfloat16* src, int e0, int e1) {
  RawUnit r;
  r.a = *reinterpret_cast<const uint4*>(src + e0);  // plain loads: q_out may be q
  r.b = *reinterpret_cast<const uint4*>(src + e1);
  return r;
}
// The 16 elements of a unit in fp32, rotated where `turn` is set; x[0..7] belong to e0, x[8..15] to e1.
template <bool kPairs>
__device__ __forceinline__ void rotate_unit(const RawUnit& raw, bool turn, const float* cs, const float* sn,
                                            float (&x)[16]) {
  const uint32_t w[8] = {raw.a.x, raw.a.y, raw.a.z, raw.a.w, raw.b.x, raw.b.y, raw.b.z, raw.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
  if (!turn) return;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 cv = ld_plain(reinterpret_cast<const float4*>(cs) + i);
    const float4 sv = ld_plain(reinterpret_cast<const float4*>(sn) + i);
    c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
    s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int lo = kPairs ? 2 * i : i, hi = kPairs ? 2 * i + 1 : i + 8;
    const float p = x[lo], r = x[hi];
    x[lo] = fmaf(p, c[i], -(r * s[i]));
    x[hi] = fmaf(r, c[i], p * s[i]);
  }
}

__device__ __forceinline__ uint4 pack8_bf16(const float* x) {
  return make_uint4(round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3]), round_bf16x2(x[4], x[5]),
                    round_bf16x2(x[6], x[7]));
}
// Codes of 8 values; zeros under a NaN scale, so that only the scale carries it. Under the largest scale
// they stop at 240: the next code, 256, would stand for 2^128, which neither fp32 nor bf16 holds.
// bf16's largest value, 255·2^120, stays within 2^-4 of its code (15/255).
__device__ __forceinline__ uint2 pack8_e4m3(const float* x, float inv) {
  if (inv != inv) return make_uint2(0u, 0u);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  if (inv == exp2_int(-kScaleExpMax)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -240.f), 240.f);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_e4m3x2(y[2 * i], y[2 * i + 1]);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// 16 codes carried over to a scale that is larger by 1 / ratio.
__device__ __forceinline__ uint4 rescale16(uint4 w, float ratio) {
  uint32_t in[4] = {w.x, w.y, w.z, w.w}, out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(in[i], lo, hi);
    const float2 a = f16x2_to_float2(lo), b = f16x2_to_float2(hi);
    out[i] = to_e4m3x2(a.x * ratio, a.y * ratio) | (to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The scale after this call, from the largest magnitude of the new rows (its bits: NaN and infinity
// are the largest of all) and the scale of the page's older rows (has_old).
__device__ __forceinline__ float next_scale(uint32_t amax_bits, bool has_old, float old) {
  const float need = amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : exp2_int(scale_exponent(amax_bits));
  if (!has_old) return need;
  return need != need || old != old ? __uint_as_float(0x7fc00000u) : fmaxf(need, old);
}

// Threads of a CTA of append_rows_kernel: one per unit of a page and head, 256 at least.
__host__ __device__ constexpr int rows_threads(int dh, int page) { return page * dh / 16 > 256 ? page * dh / 16 : 256; }

// One page of one sequence (its new rows), heads_per_cta heads of K, V (or q: no page is involved,
// the same rows). HP heads are worked on at once where a head of a page has fewer units than the CTA
// threads. The next heads' rows are loaded before these are worked on:
// the loop is bound by the loads in flight (two units a thread and no prefetch: 181 us, this 128, for
// chunks of 5 sequences with 32 query heads over 8, e4m3, with their read back).
template <bool kE4M3, bool kPairs, int DH, int PAGE>
__global__ void __launch_bounds__(rows_threads(DH, PAGE), 1024 / rows_threads(DH, PAGE))
    append_rows_kernel(const AppendParams p) {
  constexpr int NT = rows_threads(DH, PAGE);
  constexpr int UR = DH / 16;        // units of a row
  constexpr int U = PAGE * UR;       // units of a page and head
  constexpr int HP = NT / U;         // heads at once
  constexpr int GT = U;              // threads of a head
  __shared__ uint32_t s_amax[3][HP];
  pdl_launch_dependents();
  pdl_wait_primary();

  const int b = blockIdx.z;
  const PagedRows r = paged_rows(p.starts, p.lens, b, p.rows, p.max_new, p.c.cap, p.rot ? p.n_pos : p.c.cap);
  if (r.bits) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, r.bits);
    // a skipped sequence's rotated queries are zero
    const int chunk_q = static_cast<int>(blockIdx.y) - 2 * p.kv_chunks;
    if (chunk_q == 0 && r.span && p.q_out)
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
           i < static_cast<int64_t>(r.n) * p.Hq * DH / 8; i += static_cast<int64_t>(gridDim.x) * NT)
        reinterpret_cast<uint4*>(p.q_out + static_cast<int64_t>(r.row0) * p.Hq * DH)[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int64_t slot = (r.len >> p.c.page_shift) + static_cast<int64_t>(blockIdx.x);
  const int64_t page0 = slot * PAGE;
  if (r.n == 0 || page0 >= static_cast<int64_t>(r.len) + r.n) return;
  const int lo = max(0, static_cast<int>(r.len - page0));                           // first new row of the page
  const int hi = static_cast<int>(min(static_cast<int64_t>(PAGE), r.len + static_cast<int64_t>(r.n) - page0));
  const int src0 = r.row0 + static_cast<int>(page0 - r.len);                        // packed row of page row 0

  const int y = blockIdx.y;
  const int which = y < p.kv_chunks ? 0 : y < 2 * p.kv_chunks ? 1 : 2;
  const int chunk = which == 2 ? y - 2 * p.kv_chunks : y - which * p.kv_chunks;
  const int heads = which == 2 ? p.Hq : p.c.Hkv;
  const int h0 = chunk * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, heads);
  const int id = which == 2 ? 0 : p.c.page_of(b, page0);
  if (id < 0) {
    if (threadIdx.x == 0) atomicOr(p.status, SLIM_DEV_BADPAGE);
    return;
  }
  const __nv_bfloat16* src = which == 0 ? p.k : which == 1 ? p.v : p.q;
  const int64_t stride = which == 0 ? p.k_stride : which == 1 ? p.v_stride : p.q_stride;
  uint8_t* dst = (which == 0 ? p.c.k : p.c.v) + id * p.c.page_bytes;
  float* scales = (which == 0 ? p.c.ks : p.c.vs);
  const int rot = which == 1 ? 0 : p.rot;
  const int g = threadIdx.x / GT, gt = threadIdx.x - g * GT;
  if (kE4M3 && threadIdx.x < 3 * HP) s_amax[threadIdx.x / HP][threadIdx.x % HP] = 0u;
  if (kE4M3) __syncthreads();

  // this thread's unit: its columns and source row do not change from head to head
  const int row = gt / UR, i = gt % UR;
  const bool use = row >= lo && row < hi, turn = i * 16 < rot;
  int e0, e1;
  unit_columns<kPairs, DH>(i, rot, e0, e1);
  const __nv_bfloat16* from = src + (src0 + row) * stride;
  const int64_t at = (page0 + row) * (p.rot / 2) + 8 * i;
  RawUnit raw{};
  if (use && h0 + g < h1) raw = load_raw(from + static_cast<int64_t>(h0 + g) * DH, e0, e1);
  int it = 0;
  for (int hb = h0; hb < h1; hb += HP, it = it == 2 ? 0 : it + 1) {
    const int h = hb + g;
    const bool on = h < h1;
    const RawUnit cur = raw;
    if (use && h + HP < h1) raw = load_raw(from + static_cast<int64_t>(h + HP) * DH, e0, e1);
    float x[16];
    uint32_t amax = 0u;
    if (on && use) {
      rotate_unit<kPairs>(cur, turn, p.cosines + at, p.sines + at, x);
      if (kE4M3 && which != 2) {
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
      }
    }
    float inv = 0.f;
    if (kE4M3 && which != 2) {
      const float old = on && lo > 0 ? scales[static_cast<int64_t>(id) * p.c.Hkv + h] : 0.f;
      amax = __reduce_max_sync(0xffffffffu, amax);
      if ((threadIdx.x & 31) == 0) atomicMax(&s_amax[it][g], amax);
      __syncthreads();  // also: every thread has read the old scale
      const float sc = next_scale(s_amax[it][g], lo > 0, old);
      if (threadIdx.x < HP) s_amax[it == 0 ? 2 : it - 1][threadIdx.x] = 0u;  // last read before this barrier
      inv = 1.f / sc;  // a power of two, or NaN
      if (on) {
        if (gt == 0) scales[static_cast<int64_t>(id) * p.c.Hkv + h] = sc;
        if (lo > 0 && sc > old) {
          uint4* rows = reinterpret_cast<uint4*>(dst + h * p.c.head_bytes);
          for (int v = gt; v < lo * UR; v += GT) rows[v] = rescale16(rows[v], old * inv);
        }
      }
    }
    if (!(on && use)) continue;
    if (which == 2) {
      __nv_bfloat16* o = p.q_out + ((static_cast<int64_t>(src0) + row) * p.Hq + h) * DH;
      *reinterpret_cast<uint4*>(o + e0) = pack8_bf16(x);
      *reinterpret_cast<uint4*>(o + e1) = pack8_bf16(x + 8);
    } else if (kE4M3) {
      uint8_t* o = dst + h * p.c.head_bytes + row * DH;
      *reinterpret_cast<uint2*>(o + e0) = pack8_e4m3(x, inv);
      *reinterpret_cast<uint2*>(o + e1) = pack8_e4m3(x + 8, inv);
    } else {
      uint8_t* o = dst + h * p.c.head_bytes + row * DH * 2;
      *reinterpret_cast<uint4*>(o + e0 * 2) = pack8_bf16(x);
      *reinterpret_cast<uint4*>(o + e1 * 2) = pack8_bf16(x + 8);
    }
  }
}

// One row per sequence at most. Thread groups of dh/16 take (sequence, head) pairs, K heads first,
// then V, then q.
template <bool kE4M3, bool kPairs, int DH>
__global__ void __launch_bounds__(kAppThreads) append_token_kernel(const AppendParams p) {
  constexpr int UR = DH / 16;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int per_seq = 2 * p.c.Hkv + (p.q_out ? p.Hq : 0);
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x) / UR;
  const int lane = threadIdx.x & 31;
  const int i = threadIdx.x % UR;
  const int b = static_cast<int>(item / per_seq);
  const int hh = static_cast<int>(item - static_cast<int64_t>(b) * per_seq);
  const int which = hh < p.c.Hkv ? 0 : hh < 2 * p.c.Hkv ? 1 : 2;
  const int h = hh - which * p.c.Hkv;
  bool on = b < p.c.B;
  PagedRows r{};
  if (on) {
    r = paged_rows(p.starts, p.lens, b, p.rows, p.max_new, p.c.cap, p.rot ? p.n_pos : p.c.cap);
    if (r.bits) {
      if (hh == 0 && i == 0) atomicOr(p.status, r.bits);
      if (which == 2 && r.span)
        for (int j = 0; j < r.n; ++j) {
          uint4* o = reinterpret_cast<uint4*>(p.q_out + ((static_cast<int64_t>(r.row0) + j) * p.Hq + h) * DH) + 2 * i;
          o[0] = o[1] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    on = r.bits == 0 && r.n == 1;
  }
  int id = 0;
  if (on && which != 2) {
    id = p.c.page_of(b, r.len);
    if (id < 0) {
      if (i == 0) atomicOr(p.status, SLIM_DEV_BADPAGE);
      on = false;
    }
  }
  const int row = r.len & ((1 << p.c.page_shift) - 1);
  const int rot = which == 1 ? 0 : p.rot;
  int e0 = 0, e1 = 0;
  unit_columns<kPairs, DH>(i, rot, e0, e1);
  uint8_t* dst = (which == 0 ? p.c.k : p.c.v) + id * p.c.page_bytes + h * p.c.head_bytes;
  float* scale = (which == 0 ? p.c.ks : p.c.vs) + static_cast<int64_t>(id) * p.c.Hkv + h;
  float x[16];
  uint32_t amax = 0u;
  float old = 0.f;
  if (on) {
    const __nv_bfloat16* src = which == 0 ? p.k : which == 1 ? p.v : p.q;
    const int64_t stride = which == 0 ? p.k_stride : which == 1 ? p.v_stride : p.q_stride;
    const int64_t at = static_cast<int64_t>(r.len) * (p.rot / 2) + 8 * i;
    rotate_unit<kPairs>(load_raw(src + r.row0 * stride + static_cast<int64_t>(h) * DH, e0, e1), i * 16 < rot,
                        p.cosines + at, p.sines + at, x);
    if (which == 2) {
      __nv_bfloat16* o = p.q_out + (static_cast<int64_t>(r.row0) * p.Hq + h) * DH;
      *reinterpret_cast<uint4*>(o + e0) = pack8_bf16(x);
      *reinterpret_cast<uint4*>(o + e1) = pack8_bf16(x + 8);
    } else if (!kE4M3) {
      uint8_t* o = dst + row * DH * 2;
      *reinterpret_cast<uint4*>(o + e0 * 2) = pack8_bf16(x);
      *reinterpret_cast<uint4*>(o + e1 * 2) = pack8_bf16(x + 8);
    } else {
      if (row > 0) old = *scale;
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
    }
  }
  if (!kE4M3) return;
  const bool store = on && which != 2;
#pragma unroll
  for (int o = 1; o < UR; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float sc = 1.f, inv = 1.f;
  if (store) {
    sc = next_scale(amax, row > 0, old);
    inv = 1.f / sc;
    uint8_t* o = dst + row * DH;
    *reinterpret_cast<uint2*>(o + e0) = pack8_e4m3(x, inv);
    *reinterpret_cast<uint2*>(o + e1) = pack8_e4m3(x + 8, inv);
  }
  // the whole warp re-rounds, one after another, the pages whose scale has grown
  __syncwarp();  // every lane of a row has read the old scale
  if (store && i == 0 && !(row > 0 && sc == old)) *scale = sc;
  uint32_t grown = __ballot_sync(0xffffffffu, store && i == 0 && row > 0 && sc > old);
  while (grown) {
    const int from = __ffs(static_cast<int>(grown)) - 1;
    grown &= grown - 1;
    uint4* rows = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), from));
    const int n = __shfl_sync(0xffffffffu, row, from) * UR;
    const float ratio = __shfl_sync(0xffffffffu, old * inv, from);
    for (int v = lane; v < n; v += 128) {  // four loads in flight for each lane
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (v + 32 * k < n) w[k] = rows[v + 32 * k];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (v + 32 * k < n) rows[v + 32 * k] = rescale16(w[k], ratio);
    }
  }
}

struct GatherParams {
  PagedView c;
  const int32_t* starts;
  const int32_t* first;
  int64_t rows, max_new;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* status;
  int heads_per_cta, chunks;
};

// The rows of one page that a sequence asks for, heads_per_cta heads of K or V.
template <bool kE4M3, int DH>
__global__ void __launch_bounds__(kAppThreads) gather_kernel(const GatherParams p) {
  constexpr int UR = DH / 16;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.z;
  const PagedRows r = paged_rows(p.starts, p.first, b, p.rows, p.max_new, p.c.cap, p.c.cap);
  const int which = blockIdx.y < static_cast<unsigned>(p.chunks) ? 0 : 1;
  const int h0 = (blockIdx.y - which * p.chunks) * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.c.Hkv);
  __nv_bfloat16* out = which == 0 ? p.k_out : p.v_out;
  if (r.bits) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, r.bits);
    if (h0 == 0 && r.span)  // a skipped sequence's rows are zero
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x;
           i < static_cast<int64_t>(r.n) * p.c.Hkv * DH / 8; i += static_cast<int64_t>(gridDim.x) * kAppThreads)
        reinterpret_cast<uint4*>(out + static_cast<int64_t>(r.row0) * p.c.Hkv * DH)[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int page = 1 << p.c.page_shift;
  const int64_t page0 = ((r.len >> p.c.page_shift) + static_cast<int64_t>(blockIdx.x)) << p.c.page_shift;
  if (r.n == 0 || page0 >= static_cast<int64_t>(r.len) + r.n) return;
  const int lo = max(0, static_cast<int>(r.len - page0));
  const int hi = static_cast<int>(min(static_cast<int64_t>(page), r.len + static_cast<int64_t>(r.n) - page0));
  const int64_t dst0 = r.row0 + (page0 - r.len);
  const int id = p.c.page_of(b, page0);
  if (id < 0 && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, SLIM_DEV_BADPAGE);
  const uint8_t* src = (which == 0 ? p.c.k : p.c.v) + (id < 0 ? 0 : id) * p.c.page_bytes;
  const float* scales = (which == 0 ? p.c.ks : p.c.vs) + static_cast<int64_t>(id < 0 ? 0 : id) * p.c.Hkv;
  // a thread takes one unit of 16 elements of a row for every head of the range: independent loads
  // (8 elements, whose stores would be whole lines: 61 us instead of 56 for 16 sequences of 1000 to 6000
  // rows, 8 heads of 128)
  for (int v = threadIdx.x; v < (hi - lo) * UR; v += kAppThreads) {
    const int row = lo + v / UR, i = v % UR;
    const uint8_t* at = src + (static_cast<int64_t>(row) * UR + i) * (kE4M3 ? 16 : 32);
    uint4* to = reinterpret_cast<uint4*>(out + ((dst0 + row) * p.c.Hkv) * DH) + 2 * i;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
      if (id >= 0) {
        o0 = ld_plain(reinterpret_cast<const uint4*>(at + h * p.c.head_bytes));
        if (kE4M3) {
          const float s = ld_plain(scales + h);
          uint32_t y[8];
          e4m3x4_to_f16(o0.x, y[0], y[1]);
          e4m3x4_to_f16(o0.y, y[2], y[3]);
          e4m3x4_to_f16(o0.z, y[4], y[5]);
          e4m3x4_to_f16(o0.w, y[6], y[7]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 a = f16x2_to_float2(y[e]);
            y[e] = round_bf16x2(a.x * s, a.y * s);
          }
          o0 = make_uint4(y[0], y[1], y[2], y[3]);
          o1 = make_uint4(y[4], y[5], y[6], y[7]);
        } else {
          o1 = ld_plain(reinterpret_cast<const uint4*>(at + h * p.c.head_bytes) + 1);
        }
      }
      to[h * (DH / 8)] = o0;
      to[h * (DH / 8) + 1] = o1;
    }
  }
}

cudaError_t launch(const void* kern, dim3 grid, int threads, void** args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kern, args);
}

template <bool E, bool P>
const void* rows_kernel(int dh, int page) {
  if (dh == 64)
    return page == 16   ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 64, 16>)
           : page == 32 ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 64, 32>)
           : page == 64 ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 64, 64>)
                        : reinterpret_cast<const void*>(append_rows_kernel<E, P, 64, 128>);
  return page == 16   ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 128, 16>)
         : page == 32 ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 128, 32>)
         : page == 64 ? reinterpret_cast<const void*>(append_rows_kernel<E, P, 128, 64>)
                      : reinterpret_cast<const void*>(append_rows_kernel<E, P, 128, 128>);
}
template <bool E, bool P>
const void* token_kernel(int dh) {
  return dh == 64 ? reinterpret_cast<const void*>(append_token_kernel<E, P, 64>)
                  : reinterpret_cast<const void*>(append_token_kernel<E, P, 128>);
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st, int* launches) {
  const slim_paged_cache& c = *a.cache;
  AppendParams p;
  p.c = paged_view(c);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.cosines = a.cosines;
  p.sines = a.sines;
  p.rot = a.rot;
  p.n_pos = a.n_pos;
  p.starts = a.starts;
  p.lens = a.lens;
  p.rows = a.rows;
  p.max_new = a.max_new;
  p.Hq = a.q ? a.Hq : 0;
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.status = a.status;
  const bool e4m3 = c.dtype == SLIM_E4M3, pairs = a.interleaved != 0;
  void* args[] = {&p};
  cudaError_t e;
  if (a.max_new == 1) {
    p.heads_per_cta = p.kv_chunks = p.q_chunks = 0;
    const int64_t threads = static_cast<int64_t>(c.B) * (2 * c.Hkv + p.Hq) * (c.dh / 16);
    const void* kern = e4m3 ? (pairs ? token_kernel<true, true>(c.dh) : token_kernel<true, false>(c.dh))
                            : (pairs ? token_kernel<false, true>(c.dh) : token_kernel<false, false>(c.dh));
    e = launch(kern, dim3(static_cast<unsigned>(ceil_div(threads, kAppThreads))), kAppThreads, args, st);
  } else {
    // heads of a CTA: up to eight times what it works on at once, as many as leave about eight CTAs per SM (they
    // share the angles of their rows, and the next heads' loads run under these heads' work). 8 prompts of 2000
    // rows, 32 query heads over 8 of 128: 71 us in bf16, 72 in e4m3; without more heads than at once 98 and 113.
    // 16 CTAs per SM: 76 in e4m3; one per SM is the same there, but 10.3 us against 8.3 for 2 prompts of 500.
    const int slots = ceil_div(a.max_new - 1, c.page) + 1;
    const int threads = rows_threads(c.dh, c.page);
    const int at_once = std::max(1, threads / (c.page * c.dh / 16));
    const int64_t units = (a.rows / c.page + c.B) * (2ll * c.Hkv + p.Hq);
    const int64_t per = units / (8ll * num_sms() * at_once);
    p.heads_per_cta = at_once * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(per, 8)));
    p.kv_chunks = ceil_div(c.Hkv, p.heads_per_cta);
    p.q_chunks = ceil_div(p.Hq, p.heads_per_cta);
    const void* kern = e4m3 ? (pairs ? rows_kernel<true, true>(c.dh, c.page) : rows_kernel<true, false>(c.dh, c.page))
                            : (pairs ? rows_kernel<false, true>(c.dh, c.page) : rows_kernel<false, false>(c.dh, c.page));
    e = launch(kern, dim3(static_cast<unsigned>(slots), static_cast<unsigned>(2 * p.kv_chunks + p.q_chunks),
                          static_cast<unsigned>(c.B)),
               threads, args, st);
  }
  if (e == cudaSuccess && launches) ++*launches;
  return e;
}

cudaError_t launch_paged_gather(const slim_paged_cache& c, const int32_t* starts, const int32_t* first, int64_t rows,
                                int64_t max_new, void* k_out, void* v_out, int32_t* status, cudaStream_t st,
                                int* launches) {
  GatherParams p;
  p.c = paged_view(c);
  p.starts = starts;
  p.first = first;
  p.rows = rows;
  p.max_new = max_new;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.status = status;
  const int slots = ceil_div(max_new - 1, c.page) + 1;
  // heads of a CTA: as many as leave 32 CTAs per SM (8: 64 us, 32: 52 us for 16 sequences of 1000 to 6000 rows)
  const int64_t units = (rows / c.page + c.B) * 2ll * c.Hkv;
  p.heads_per_cta = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(units / (32ll * num_sms()), 8)));
  p.chunks = ceil_div(c.Hkv, p.heads_per_cta);
  const void* kern = c.dtype == SLIM_E4M3 ? (c.dh == 64 ? reinterpret_cast<const void*>(gather_kernel<true, 64>)
                                                        : reinterpret_cast<const void*>(gather_kernel<true, 128>))
                                          : (c.dh == 64 ? reinterpret_cast<const void*>(gather_kernel<false, 64>)
                                                        : reinterpret_cast<const void*>(gather_kernel<false, 128>));
  void* args[] = {&p};
  const cudaError_t e = launch(kern, dim3(static_cast<unsigned>(slots), static_cast<unsigned>(2 * p.chunks),
                                          static_cast<unsigned>(c.B)),
                               kAppThreads, args, st);
  if (e == cudaSuccess && launches) ++*launches;
  return e;
}

}  // namespace slim
