// slim_mha_paged_prefill: causal attention of several new rows per sequence over
// a paged K+V cache in bf16 or e4m3, on tcgen05 tensor cores.
//
// Mathematics: row j of sequence b (position lens[b] + j) and query head i give
//     o = softmax(q·K_{<= position}^T / sqrt(dh)) · V_{<= position},
// as a running (m, l, O) over key tiles: P = 2^(s - m), l = Σ P, O = Σ P·V.
//
// A CTA owns two 128-row tiles of one (sequence, key head): a row is a (query,
// head) pair, the G query heads that share the key head side by side, so that a
// tile holds 128/G queries and every K and V tile it loads serves all of them.
// It walks the 128-key tiles up to its last query's position.
//   warp 0        loads K and V, page by page, by TMA straight into the MMAs' swizzled layouts;
//                 e4m3 values as bulk copies of whole page heads into a raw ring
//   warps 1, 2    issue tcgen05.mma for one row tile each: S_t = Q_t·K^T into the tile's
//                 TMEM S region, O_t += P_t·V with P_t read from tensor memory, in the
//                 order P_t(j)·V_j, S_t(j+1)
//   warps 4..7, 8..11  softmax of tile 0 and 1, one row per thread: causal mask,
//                 lazy running maximum (O is rescaled only when a maximum grows by
//                 more than 2^8), P over the S region, row sums in fp32
//   warps 12..15  (e4m3) value codes to f16 in the MMA's layout
// An e4m3 cache is used as it is stored. S runs in e4m3 on the key codes, with the query in two
// e4m3 parts (high and low) that together hold a bf16 exactly: twice the products at twice the
// rate of f16, and no key is converted. Value codes are exact in f16, and P·V runs in f16. The
// key scale of a page multiplies its scores, the value scale 2^lv its probabilities,
// P = 2^(s + lv - m + kWeightLog2) with m the running maximum of s + lv. P is rounded to f16 (2^-11)
// there; over bf16 values it is rounded to bf16 (2^-8), the type the MMA wants beside them.
// Key rows at or past the sequence's end are zeroed in V before the first MMA
// that reads them: a masked P = 0 never meets what a page held before.
//
// Few rows behind a long cache leave most SMs without a CTA: the key tiles are
// then cut into `splits` ranges, each CTA leaves (m, l, O), and
// merge_prefill_kernel joins them. Where all queries of a sequence fit one row
// tile, an e4m3 cache's keys are divided between the two row tiles as well.
#include <algorithm>

#include "paged.cuh"

namespace slim {

namespace {

constexpr int kFQ = 128;  // rows of a tile
constexpr int kFK = 128;  // keys of a tile
constexpr uint32_t kFTmemPerTile = 256;  // S (and P over it) at columns 0..127, O at 128
constexpr float kFLazyLog2 = 8.f;
constexpr int kScaleSlot = 24;  // floats of a key tile's scales
constexpr int kFSetup = 4;  // a CTA's fixed time (query, first S, output) in key tiles of about 2.2 us

struct PagedPrefillParams {
  PagedView c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* starts;
  const int32_t* lens;
  int64_t rows, max_new;
  int Hq, G, QPT;  // QPT = 128 / G queries of a tile
  uint32_t g_inv;  // ceil(2^16 / G): row / G = row * g_inv >> 16 for row < 128
  int pairs, splits;
  int parts;     // partial results of a row: splits, twice as many with kTwo; 1: none
  __nv_bfloat16* out;
  float* ws_o;   // [part][rows][Hq][dh], parts > 1
  float* ws_ml;  // [part][rows][Hq][2]
  int32_t* status;
  float scale_log2;
};

template <bool E, int DHB>
struct PfCfg {
  // Keys of a step, the unit of S, softmax and P·V. Halves of a key tile (e4m3) have a TMEM region each, so
  // that S of the next tile's half runs under the softmax of this one's other half: 522 us against 553 with
  // whole tiles (4 chunks of 400 rows behind 16000, 32 query heads over 8 of 128). In bf16 the 64-key S MMAs
  // cost as much shared-memory bandwidth as 128-key ones (their A operand is read either way) and the whole
  // tile is faster: 504 us against 523 (a prompt of 8192 rows, 32 heads of 128).
  static constexpr int FH = E ? 64 : 128;
  static constexpr int HV = kFK / FH;                          // steps of a key tile
  static constexpr int kPart1 = FH == 128 ? 96 : 64;           // keys of P that are handed over first
  static constexpr int kParts = FH == 128 ? 2 : 1;
  static constexpr int DH = 64 * DHB;
  static constexpr int NK = E ? 3 : DHB == 2 ? 2 : 4;          // stages of the K ring
  static constexpr int NV = DHB == 2 ? 2 : 4;                  // stages of the V ring the MMAs read
  static constexpr int NR = 2;                                 // stages of the raw V ring (e4m3)
  static constexpr uint32_t kTile = kFK * DH * 2u;             // bytes of a V tile, and of a Q tile (e4m3: two parts)
  static constexpr uint32_t kKTile = E ? kFK * DH : kTile;     // bytes of a K tile
  static constexpr uint32_t kRaw = E ? kFK * DH : 0u;          // bytes of a raw V tile
  static constexpr int kThreads = E ? 512 : 384;
  static constexpr uint32_t kSmem = 2u * kTile + NK * kKTile + NV * kTile + NR * kRaw + 512u + 1024u + 1024u;
};

__device__ __forceinline__ float pf_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void pf_tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// D (TMEM) (+)= A · B, A in tensor memory (row i in lane i, two 16-bit elements per column).
__device__ __forceinline__ void pf_umma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D (TMEM) (+)= A · B, e4m3 operands from shared memory, 32 columns of the contraction.
__device__ __forceinline__ void pf_umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor with both operand type fields 0 (f16 for kind::f16, e4m3 for kind::f8f6f4), fp32 D.
__host__ __device__ constexpr uint32_t idesc_zero_f32(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
constexpr uint32_t kLayoutSW64 = 4;  // 64-byte swizzle in a shared-memory descriptor
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// mbar_wait by a whole warp, one decision for it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// kTwo (e4m3): no sequence has more queries than a row tile. Both row tiles then hold them, and take the CTA's
// even and odd key tiles; their (m, l, O) are joined like those of splits. One row tile alone waits on its own
// chain of S, softmax and P·V: 8 queries of 64 heads over 8 of 128 in 8 sequences of 8000 rows 78 us, this 60;
// 16 sequences of 3000, 32 heads, 57 and 48. Over bf16 the rings have two stages at dh = 128, one for each row
// tile here, and the next load is always waited for: 76 us, and 81 with this.
template <bool E, int DHB, bool kTwo>
__global__ void __launch_bounds__(PfCfg<E, DHB>::kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const PagedPrefillParams p) {
  using C = PfCfg<E, DHB>;
  constexpr int DH = C::DH, NK = C::NK, NV = C::NV, NR = C::NR, FH = C::FH, HV = C::HV;
  constexpr uint32_t T = C::kTile, TK = C::kKTile;
  extern __shared__ uint8_t pf_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pf_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = sm;              // bf16: [row tile][DHB boxes][128 rows][128 B]; e4m3: [row tile][high, low][128 rows][DH]
  uint8_t* ks = qs + 2 * T;      // [stage] bf16: [DHB boxes][128 rows][128 B]; e4m3: [128 rows][DH]
  uint8_t* vs = ks + NK * TK;    // [stage][DHB boxes][128 rows][128 B]
  uint8_t* rv = vs + NV * T;     // [stage][128 rows][DH] raw V (e4m3)
  uint64_t* bars = reinterpret_cast<uint64_t*>(rv + NR * C::kRaw);
  uint64_t* qbar = bars;           // Q written by the softmax warps
  uint64_t* kfull = bars + 1;      // [NK]
  uint64_t* kempty = kfull + NK;   // [NK]
  uint64_t* vfull = kempty + NK;   // [NV]
  uint64_t* vempty = vfull + NV;   // [NV]
  uint64_t* sfull = vempty + NV;   // [row tile][half] S written (e4m3, first half: and the tile's scales)
  uint64_t* pready = sfull + 4;    // [row tile][half or part] P written over S (and O rescaled)
  uint64_t* pvdone = pready + 4;   // [row tile] a P·V completed
  uint64_t* ofull = pvdone + 2;    // [row tile] the tile's last P·V completed
  uint64_t* vfixed = ofull + 2;    // [NV] bf16: V rows past the end are zeroed
  uint64_t* rfull = vfixed + NV;     // [NR] raw V landed
  uint64_t* rempty = rfull + NR;   // [NR] raw V converted
  uint64_t* turn = rempty + NR;    // [row tile][warp of it] the other row tile's exponentials of a step are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(turn + 8);
  int* s_bad = reinterpret_cast<int*>(tmem_slot + 1);  // first position whose page is outside the pool
  // e4m3: [key tile mod 8] for either half of the keys the scale of its pages if they share one (key scale,
  // value exponent, whether), then key scale and value exponent of each page. Written by the K producer before
  // it arrives on the tile's kfull; the MMA warp that has waited for that arrives on the tile's first sfull
  // beside the products, and so passes them on to the softmax warps (a commit alone orders the products, not
  // what threads wrote. A barrier of their own for the scales took 4 % longer: one more wait in every tile).
  // A slot is written again eight tiles later. No reader is that far behind: the rings are shorter, and a V
  // stage comes free only with the P·V of every row tile that attends it, for which all its warps have read
  // the scales and handed P over.
  float* s_scale = reinterpret_cast<float*>(bars + 64);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  pdl_launch_dependents();
  pdl_wait_primary();
  // heaviest pairs (the last rows) first
  const int bh = blockIdx.x % (p.c.B * p.c.Hkv);
  const int rest = blockIdx.x / (p.c.B * p.c.Hkv);
  const int pair = rest / p.splits, split = rest - pair * p.splits;
  const int b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const PagedRows r = paged_rows(p.starts, p.lens, b, p.rows, p.max_new, p.c.cap, p.c.cap);
  if (r.bits) {
    if (threadIdx.x == 0 && h == 0 && rest == 0) atomicOr(p.status, r.bits);
    if (rest == 0 && r.span)  // a skipped sequence's rows are zero: this CTA's heads
      for (int64_t i = threadIdx.x; i < static_cast<int64_t>(r.n) * p.G * (DH / 8); i += C::kThreads) {
        const int64_t row = i / (p.G * (DH / 8)), k = i - row * (p.G * (DH / 8));
        reinterpret_cast<uint4*>(p.out + ((r.row0 + row) * p.Hq + static_cast<int64_t>(h) * p.G) * DH)[k] =
            make_uint4(0u, 0u, 0u, 0u);
      }
    return;
  }
  const int n = r.n, len = r.len, L = len + n;
  const int nqt = (n + p.QPT - 1) / p.QPT;
  if (2 * pair >= nqt) return;
  // tile t of the pair holds queries q0 .. q0 + QPT - 1; a negative q0 is an absent tile
  auto tile_q0 = [&](int t) { return kTwo ? 0 : (nqt - 2 * (pair + 1) + t) * p.QPT; };
  auto tile_keys = [&](int t) {  // key tiles that tile t attends
    const int q0 = tile_q0(t);
    return q0 < 0 ? 0 : (len + min(q0 + p.QPT, n) - 1) / kFK + 1;
  };
  const int nk_all = tile_keys(1);
  const int kt0 = static_cast<int>(static_cast<int64_t>(split) * nk_all / p.splits);
  const int kt1 = static_cast<int>(static_cast<int64_t>(split + 1) * nk_all / p.splits);
  const int nkt = kt1 - kt0;
  // key tile of the CTA that is tile t's j-th
  auto key_tile = [](int t, int j) { return kTwo ? 2 * j + t : j; };
  // steps of this split that tile t attends
  auto tile_steps = [&](int t) {
    const int q0 = tile_q0(t);
    const int all = q0 < 0 ? 0 : (len + min(q0 + p.QPT, n) - 1) / FH + 1;
    const int steps = max(0, min(HV * kt1, all) - HV * kt0);
    // the last key tile, which may have one step only, is that of tile (nkt - 1) & 1
    return !kTwo ? steps : HV * ((nkt + 1 - t) >> 1) - (((nkt - 1) & 1) == t ? HV * nkt - steps : 0);
  };

  if (warp == 0 && lane == 0) {
    mbar_init(qbar, 8);
    for (int s = 0; s < NK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 2);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&vfull[s], E ? 4 : 1);
      mbar_init(&vempty[s], 2);
      mbar_init(&vfixed[s], 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], 4);
    }
    for (int t = 0; t < 4; ++t) {
      mbar_init(&sfull[t], E && (t & 1) == 0 ? 2 : 1);
      mbar_init(&pready[t], 4);
    }
    for (int t = 0; t < 8; ++t) mbar_init(&turn[t], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&pvdone[t], 1);
      mbar_init(&ofull[t], 1);
    }
    *s_bad = 0x7fffffff;
    fence_barrier_init();
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kFTmemPerTile);
    tmem_relinquish();
  }
  const int32_t* table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
  const int psh = p.c.page_shift, ppt = kFK >> psh;  // pages of a key tile
  const int page_lo = kt0 * ppt, page_hi = min(kt1 * ppt, ((L - 1) >> psh) + 1);
  int first_bad = 0x7fffffff;
  for (int i = page_lo + static_cast<int>(threadIdx.x); i < page_hi; i += C::kThreads) {
    const int id = ld_plain(table + i);
    if (id < 0 || id >= p.c.num_pages) first_bad = min(first_bad, i << psh);
  }
  tc_fence_before();
  if (__syncthreads_or(first_bad != 0x7fffffff)) {
    if (first_bad != 0x7fffffff) atomicMin(s_bad, first_bad);
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // keys from here on are not used: the sequence's end, or a page outside the pool (whose place page 0
  // takes in the loads)
  const int Lz = min(L, *s_bad);

  // page number of page i of the sequence for the loads: page 0 where it is outside the pool
  auto page_id = [&](int i) {
    const int id = ld_plain(table + i);
    return id >= 0 && id < p.c.num_pages ? id : 0;
  };
  // pages of key tile j that hold rows of the sequence
  auto pages_of = [&](int j) { return min(ppt, ((L - 1 - j * kFK) >> psh) + 1); };

  if (warp < 4) {
    reg_dec<E ? 64 : 72>();
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      int nk_issued = 0, nv_issued = 0;
      // page numbers two key tiles ahead and, for e4m3, their scales one ahead
      auto page_ahead = [&](int i) { return i < nkt && lane < pages_of(kt0 + i) ? page_id((kt0 + i) * ppt + lane) : -1; };
      auto scale_of = [&](const float* pool, int id) {
        return E && id >= 0 ? ld_plain(pool + static_cast<int64_t>(id) * p.c.Hkv + h) : 1.f;
      };
      int id = page_ahead(0), id_next = page_ahead(1);
      float ks_l = scale_of(p.c.ks, id), vs_l = scale_of(p.c.vs, id);
      for (int i = 0; i < nkt; ++i) {
        const int npg = pages_of(kt0 + i);
        const uint32_t bytes = static_cast<uint32_t>(npg << psh) * DH * (E ? 1u : 2u);
        const int y = (id * p.c.Hkv + h) << psh;  // first line of the page's head
        const uint32_t line = static_cast<uint32_t>(lane << psh);
        const int sk = i % NK;
        if (i >= NK && !warp_wait(&kempty[sk], static_cast<uint32_t>(i / NK - 1) & 1u, p.status)) break;
        if (E) {
          const float lv_l = scale_log2(vs_l);
          float* sc = s_scale + (i & 7) * kScaleSlot;
          if (lane < 8) {
            sc[8 + 2 * lane] = ks_l;
            sc[9 + 2 * lane] = lv_l;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int first = half * (ppt >> 1), last = ppt == 1 ? 1 : first + (ppt >> 1);  // pages of the half
            const float ks0 = __shfl_sync(0xffffffffu, ks_l, first), lv0 = __shfl_sync(0xffffffffu, lv_l, first);
            const bool one = __all_sync(0xffffffffu, lane < first || lane >= min(last, npg) ||
                                                         (ks_l == ks0 && lv_l == lv0));
            if (lane == 0) *reinterpret_cast<float4*>(sc + 4 * half) = make_float4(ks0, lv0, one ? 1.f : 0.f, 0.f);
          }
          ks_l = scale_of(p.c.ks, id_next);
          vs_l = scale_of(p.c.vs, id_next);
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&kfull[sk], bytes);
        __syncwarp();
        if (lane < npg) {
          if (E) {
            tma_load_2d(ks + sk * TK + line * DH, &kmap, 0, y, &kfull[sk], l2_policy_evict_last());
          } else {
#pragma unroll
            for (int k = 0; k < DHB; ++k)
              tma_load_2d(ks + sk * TK + k * 16384 + line * 128u, &kmap, 64 * k, y, &kfull[sk], l2_policy_evict_last());
          }
        }
        ++nk_issued;
        constexpr int N = E ? NR : NV;
        const int sv = i % N;
        uint64_t* full = E ? &rfull[sv] : &vfull[sv];
        if (i >= N && !warp_wait(E ? &rempty[sv] : &vempty[sv], static_cast<uint32_t>(i / N - 1) & 1u, p.status)) break;
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (lane < npg) {
          if (E) {
            bulk_load_g2s(rv + sv * C::kRaw + line * DH, p.c.v + id * p.c.page_bytes + h * p.c.head_bytes,
                          static_cast<uint32_t>(p.c.head_bytes), full);
          } else {
#pragma unroll
            for (int k = 0; k < DHB; ++k)
              tma_load_2d(vs + sv * T + k * 16384 + line * 128u, &vmap, 64 * k, y, full, l2_policy_evict_last());
          }
        }
        ++nv_issued;
        id = id_next;
        id_next = page_ahead(i + 2);
      }
      // every issued copy lands before the CTA exits
      constexpr int N = E ? NR : NV;
      for (int u = max(0, nk_issued - NK); u < nk_issued; ++u)
        mbar_wait(&kfull[u % NK], static_cast<uint32_t>(u / NK) & 1u, p.status);
      for (int u = max(0, nv_issued - N); u < nv_issued; ++u)
        mbar_wait(E ? &rfull[u % N] : &vfull[u % N], static_cast<uint32_t>(u / N) & 1u, p.status);
    } else if (warp <= 2) {
      // ------------------------------------------------------------ MMA issuer of row tile t
      // One warp per row tile: a wait takes about 120 cycles and a commit 100 where an MMA takes 64, and
      // one warp for both tiles spent its whole time on them. The whole warp walks the loop and one elected
      // lane issues, so that descriptors stay in uniform registers: issued from a branch on the lane
      // number, an MMA took 96 cycles.
      const int t = warp - 1;
      const uint32_t idesc_s = E ? idesc_zero_f32(kFQ, FH, 0u, 0u) : idesc_bf16_f32(kFQ, FH, 0u, 0u);
      const uint32_t idesc_o = E ? idesc_zero_f32(kFQ, DH, 0u, 1u) : idesc_bf16_f32(kFQ, DH, 0u, 1u);
      // e4m3 rows of 64 bytes use the 64-byte swizzle, all others the 128-byte one
      constexpr uint32_t kLay = E && DH == 64 ? kLayoutSW64 : kLayoutSW128, kSbo = E && DH == 64 ? 512u : 1024u;
      const uint64_t qdesc = smem_desc(smem_u32(qs) + t * T, 16, kSbo, kLay);
      const uint64_t kdesc = smem_desc(smem_u32(ks), 16, kSbo, kLay);
      const uint64_t vdesc = smem_desc(smem_u32(vs), 16384, 1024, kLayoutSW128);
      const uint32_t tmem_t = tmem + t * kFTmemPerTile;
      const int steps = tile_steps(t);
      // key tiles that only this row tile reads: it releases them for both
      const int alone = kTwo ? 0 : t == 1 ? (tile_steps(0) + HV - 1) / HV : 0x7fffffff;
      const int first_fix = E ? 0x7fffffff : max(0, Lz / kFK - kt0);  // first key tile with rows past Lz
      const bool lead = elect_one();
      bool ok = warp_wait(qbar, 0u, p.status);
      auto release = [&](uint64_t* bar, int i) {
        umma_commit(bar);
        if (i >= alone) umma_commit(bar);
      };
      // S(u) = Q·K^T of the step's keys, stage s; the caller has waited for it
      auto issue_s = [&](int u, int s) {
        const int hf = HV == 2 ? u & 1 : 0;
        tc_fence_after();
        if (lead) {
          const uint32_t d = tmem_t + hf * FH;
          const uint64_t kd = kdesc + static_cast<uint32_t>(s) * (TK >> 4) + static_cast<uint32_t>(hf) * (E ? FH * DH >> 4 : FH * 8);
          if (E) {
#pragma unroll
            for (int kk = 0; kk < DH / 32; ++kk)  // high and low part of Q on the same K columns
#pragma unroll
              for (int part = 0; part < 2; ++part)
                pf_umma_f8(d, qdesc + part * (T >> 5) + kk * 2u, kd + kk * 2u, idesc_s, kk + part > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
              umma_f16(d, qdesc + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
            }
          }
          if (E && hf == 0) mbar_arrive(&sfull[2 * t]);  // passes the tile's scales on
          umma_commit(&sfull[2 * t + hf]);
          if (hf == HV - 1 || u == steps - 1) release(&kempty[s], u / HV);
        }
      };
      // O += P(u)·V of the step's keys; of a whole tile the first part starts while the softmax works on
      // the rest
      auto issue_pv = [&](int u, int s) {
        const int hf = HV == 2 ? u & 1 : 0;
        const uint32_t par = static_cast<uint32_t>(u / HV) & 1u;
        const uint32_t o = tmem_t + 128u, pt = tmem_t + hf * FH;
        const uint64_t vd = vdesc + static_cast<uint32_t>(s) * (T >> 4) + static_cast<uint32_t>(hf) * (FH / 16 * 128);
#pragma unroll
        for (int part = 0; part < C::kParts; ++part) {
          if (!warp_wait(&pready[2 * t + (HV == 2 ? hf : part)], par, p.status)) return false;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int kk = part ? C::kPart1 / 16 : 0; kk < (part + 1 == C::kParts ? FH : C::kPart1) / 16; ++kk)
              pf_umma_tmem_a(o, pt + static_cast<uint32_t>(kk * 8), vd + static_cast<uint32_t>(kk * 128), idesc_o,
                             (u > 0 || kk > 0) ? 1u : 0u);
          }
        }
        if (lead) {
          if (HV == 2) umma_commit(&pvdone[t]);
          if (hf == HV - 1 || u == steps - 1) release(&vempty[s], u / HV);
        }
        return true;
      };
      constexpr int kStep = kTwo ? 2 : 1;  // from one of its key tiles to the next
      int sv = kTwo ? t : 0, sk = sv;      // V stage of the key tile, K stage of the next one
      uint32_t phv = 0u, phk = 0u;
      auto next_stage = [](int& s, uint32_t& ph, int ring) {
        s += kStep;
        if (s >= ring) {
          s -= ring;
          ph ^= 1u;
        }
      };
      if (ok && steps > 0) {
        ok = warp_wait(&kfull[sk], 0u, p.status);
        for (int u = 0; ok && u < min(HV, steps); ++u) issue_s(u, sk);
      }
      next_stage(sk, phk, NK);
      for (int u = 0; ok && u < steps; ++u) {
        const int hf = HV == 2 ? u & 1 : 0, i = key_tile(t, u / HV);
        if (hf == 0) {
          ok = warp_wait(&vfull[sv], phv, p.status) && (u + HV >= steps || warp_wait(&kfull[sk], phk, p.status));
          if (!ok) break;
          // bf16: key rows from Lz on are zeroed in V by tile 1's warp (it attends every key tile of the CTA)
          // before either tile's first P·V that reads them
          if (i >= first_fix) {
            if (t == 1) {
              for (int k = max(0, Lz - (kt0 + i) * kFK) * 8 + lane; k < kFK * 8; k += 32)
#pragma unroll
                for (int box = 0; box < DHB; ++box)
                  *reinterpret_cast<uint4*>(vs + sv * T + box * 16384 + k * 16) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&vfixed[sv]);
            } else if (!(ok = warp_wait(&vfixed[sv], static_cast<uint32_t>((i - first_fix) / NV) & 1u, p.status))) {
              break;
            }
          }
        }
        if (!(ok = issue_pv(u, sv))) break;
        if (u + HV < steps) issue_s(u + HV, sk);  // overwrites the P that the P·V above reads: issued after it
        if (hf == HV - 1) {
          next_stage(sv, phv, NV);
          next_stage(sk, phk, NK);
        }
      }
      // also after a failure: the output barrier covers every MMA issued
      if (lead) umma_commit(&ofull[t]);
      warp_wait(&ofull[t], 0u, p.status);
    }
  } else if (E && warp >= 12) {
    // ------------------------------------------------------------ codes to f16
    reg_dec<64>();
    const int tid = threadIdx.x - 384;
    constexpr int CPR = DH / 16;        // 16-code chunks of a row
    constexpr int RS = 128 / CPR;       // rows that the four warps take at a time
    // At dh = 128 eight lanes read four chunks of one row and the other four of the next, and write two
    // rows of different swizzle parity: every phase of the read and of both writes meets eight different
    // 16-byte banks. RS is a multiple of 8, so that the swizzle stays the same from turn to turn.
    const int row0 = CPR == 8 ? (tid >> 4) * 2 + ((tid >> 2) & 1) : tid / CPR;
    const int cc = CPR == 8 ? (tid & 3) + 4 * (((tid >> 2) ^ (tid >> 3)) & 1) : tid % CPR;
    const int src0 = row0 * DH + cc * 16, box0 = (cc >> 2) * 16384 + row0 * 128;
    const int dst0 = box0 + ((((2 * cc) & 7) ^ (row0 & 7)) << 4), dst1 = box0 + ((((2 * cc + 1) & 7) ^ (row0 & 7)) << 4);
    auto convert = [&](const uint8_t* raw, uint8_t* dst, int valid) {
#pragma unroll
      for (int k = 0; k < kFK / RS; ++k) {
        uint4 w = *reinterpret_cast<const uint4*>(raw + src0 + k * RS * DH);
        if (valid < kFK && row0 + k * RS >= valid) w = make_uint4(0u, 0u, 0u, 0u);
        uint32_t y[8];
        e4m3x4_to_f16(w.x, y[0], y[1]);
        e4m3x4_to_f16(w.y, y[2], y[3]);
        e4m3x4_to_f16(w.z, y[4], y[5]);
        e4m3x4_to_f16(w.w, y[6], y[7]);
        *reinterpret_cast<uint4*>(dst + dst0 + k * RS * 128) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(dst + dst1 + k * RS * 128) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    };
    for (int i = 0; i < nkt; ++i) {
      const int s = i % NV, sr = i % NR;
      if (!warp_wait(&rfull[sr], static_cast<uint32_t>(i / NR) & 1u, p.status) ||
          (i >= NV && !warp_wait(&vempty[s], static_cast<uint32_t>(i / NV - 1) & 1u, p.status)))
        break;
      const int valid = Lz - (kt0 + i) * kFK;
      if (valid >= kFK)
        convert(rv + sr * C::kRaw, vs + s * T, kFK);
      else
        convert(rv + sr * C::kRaw, vs + s * T, valid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&rempty[sr]);
        mbar_arrive(&vfull[s]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax of row tile t
    reg_inc<E ? 192 : 216>();
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lrow = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + t * kFTmemPerTile, tmem_o = ts + 128u;
    const int q0 = tile_q0(t), steps = tile_steps(t), steps_other = tile_steps(1 - t);
    auto div_g = [&](int x) { return static_cast<int>((static_cast<uint32_t>(x) * p.g_inv) >> 16); };
    const int qi = q0 + div_g(row), head = h * p.G + row - div_g(row) * p.G;
    const bool live = q0 >= 0 && row < p.QPT * p.G && qi < n;
    const int pos = live ? len + qi : -1;  // a row without a query attends nothing
    float fq = p.scale_log2;
    // The warp's 32 query rows into the Q tile, zeros where there is none: LR lanes read one row, so that
    // a load takes whole lines (1,500 cycles at dh = 128; a row per thread took 7,000).
    {
      constexpr int LR = DH / 8, RI = 32 / LR;  // lanes of a row, rows of a load
      const int c = lane % LR;
      uint4 wv[32 / RI];
#pragma unroll
      for (int k = 0; k < 32; k += RI) {
        const int rr = quarter * 32 + k + lane / LR, qd = div_g(rr), rq = q0 + qd;
        wv[k / RI] = make_uint4(0u, 0u, 0u, 0u);
        if (q0 >= 0 && rr < p.QPT * p.G && rq < n)
          wv[k / RI] = ld_plain(reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(r.row0) + rq) * p.q_stride +
                                                            (static_cast<int64_t>(h) * p.G + rr - qd * p.G) * DH) + c);
      }
      if (!E) {
#pragma unroll
        for (int k = 0; k < 32; k += RI) {
          const int rr = quarter * 32 + k + lane / LR;
          *reinterpret_cast<uint4*>(qs + t * T + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = wv[k / RI];
        }
      } else {
        // In units that bring the row's largest magnitude to [128, 256): a high and a low e4m3 part hold
        // the 8 bits of a bf16 exactly down to 2^-10 of it, and 2^-17 of it is the error below. The
        // maxima of all rows first, so that their shuffles overlap.
        uint32_t amax[32 / RI];
#pragma unroll
        for (int k = 0; k < 32 / RI; ++k) {
          const uint32_t x[4] = {wv[k].x & 0x7fff7fffu, wv[k].y & 0x7fff7fffu, wv[k].z & 0x7fff7fffu, wv[k].w & 0x7fff7fffu};
          const uint32_t y = __vmaxu2(__vmaxu2(x[0], x[1]), __vmaxu2(x[2], x[3]));
          amax[k] = max(y & 0xffffu, y >> 16);
        }
#pragma unroll
        for (int o = 1; o < LR; o <<= 1)
#pragma unroll
          for (int k = 0; k < 32 / RI; ++k) amax[k] = max(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
#pragma unroll
        for (int k = 0; k < 32; k += RI) {
          const int rr = quarter * 32 + k + lane / LR;
          const uint32_t x[4] = {wv[k / RI].x, wv[k / RI].y, wv[k / RI].z, wv[k / RI].w}, am = amax[k / RI];
          const int e = max(-118, min(126, static_cast<int>(am >> 7) - 127));
          const float inv = exp2_int(7 - e);
          float f = exp2_int(e) * 0.0078125f * p.scale_log2;
          if (am >= 0x7f80u) f = __uint_as_float(0x7fc00000u);  // e4m3 has no infinity
          f = __shfl_sync(0xffffffffu, f, (lane % RI) * LR);
          if (lane / RI == k / RI) fq = f;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float y0 = bf16lo(x[u]) * inv, y1 = bf16hi(x[u]) * inv;
            hi[u] = to_e4m3x2(y0, y1);
            uint32_t back, none;
            e4m3x4_to_f16(hi[u], back, none);
            const float2 g = f16x2_to_float2(back);
            lo[u] = to_e4m3x2(y0 - g.x, y1 - g.y);
          }
          uint8_t* at = qs + t * T + rr * DH + (((c >> 1) ^ (DH == 128 ? rr & 7 : (rr >> 1) & 3)) << 4) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(at + T / 2) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qbar);
    }
    float m = -INFINITY, l = 0.f;
    float ksu = 1.f, lvu = 0.f;
    bool uniform = true;  // one scale pair for all pages of the step
    bool ok = true;
#pragma unroll 1
    for (int u = 0; u < steps; ++u) {
      const int i = key_tile(t, u / HV), hf = HV == 2 ? u & 1 : 0;
      const uint32_t ph = static_cast<uint32_t>(u / HV) & 1u, tsh = ts + lrow + static_cast<uint32_t>(hf * FH);
      const int k0 = (kt0 + i) * kFK + hf * FH;
      if (!warp_wait(&sfull[2 * t + hf], ph, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sc[FH];
#pragma unroll
      for (int c = 0; c < FH / 16; ++c)
        tmem_ld16(tsh + static_cast<uint32_t>(16 * c), *reinterpret_cast<float(*)[16]>(sc + 16 * c));
      tmem_wait_ld();
      // Running maximum of the weights' exponents: of the scores in log2 units, for e4m3 plus the value
      // scale's exponent lv, so that P stays in f16's range whatever the pages' scales are. P of key t
      // is 2^(s_t + e), e = lv - ref, and l adds P·2^-lv/2^kWeightLog2. Where a group's largest P is below 2^-60 (its
      // f16 is zero) e is raised to keep the fp32 sum from underflowing.
      auto ref = [&]() { return m == -INFINITY ? 0.f : E ? m - kWeightLog2 : m; };
      auto advance = [&](float mt) {
        float alpha = 1.f;
        if (m == -INFINITY) {
          m = mt;
        } else if (mt > m + kFLazyLog2) {
          alpha = pf_ex2(m - mt);
          m = mt;
          l *= alpha;
        }
        // O is rescaled before P is handed over, once the step before's P·V is done with it (a whole
        // tile's S was issued after it)
        if (u >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (HV == 2) ok = warp_wait(&pvdone[t], static_cast<uint32_t>(u - 1) & 1u, p.status);
          tc_fence_after();
          for (int c = 0; c < DH; c += 16) {
            float v[16];
            tmem_ld16(tmem_o + lrow + static_cast<uint32_t>(c), v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] *= alpha;
            tmem_st16(tmem_o + lrow + static_cast<uint32_t>(c), v);
          }
        }
      };
      // The two row tiles' warps on one scheduler take turns at the exponentials: while one has the unit to
      // itself, the other does the rest of its step. Left alone they fall into step, both waiting for the unit
      // and then both leaving it idle. Without and with turns: 595 and 561 us (e4m3, a prompt of 8192 rows, 32
      // heads of 128), 536 and 523 (4 chunks of 400 behind 16000, 32 over 8 heads), bf16 507 and 488 (the same
      // chunks), 54 and 51 (a prompt of 2048); the 8192 rows in bf16 run at the power limit either way, 505.
      auto take_turn = [&]() {
        if (t == 0 ? u >= 1 && u - 1 < steps_other : u < steps_other)
          ok = ok && warp_wait(&turn[t * 4 + quarter], static_cast<uint32_t>(t == 0 ? u - 1 : u) & 1u, p.status);
      };
      auto pass_turn = [&]() {
        if (lane == 0) mbar_arrive(&turn[(1 - t) * 4 + quarter]);
      };
      // P of keys 32 q .. 32 q + 31 of the step to tensor memory; the sums of either half of them
      auto weights = [&](int q, float f0, float f1, float e0, float e1, float& sum0, float& sum1) {
        uint32_t pk[16];
        uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float f = c < 8 ? f0 : f1, e = c < 8 ? e0 : e1;
          float x0, x1;
          unpack2(ffma2(pack2(sc[32 * q + 2 * c], sc[32 * q + 2 * c + 1]), pack2(f, f), pack2(e, e)), x0, x1);
          const float a = pf_ex2(x0), bb = pf_ex2(x1);
          s2[c >> 3] = fadd2(s2[c >> 3], pack2(a, bb));
          pk[c] = E ? round_f16x2(a, bb) : round_bf16x2(a, bb);
        }
        pf_tmem_st16(tsh + static_cast<uint32_t>(16 * q), pk);
        sum0 = unpack_sum(s2[0]);
        sum1 = unpack_sum(s2[1]);
      };
      // hands P (and, before its first part, O) to the MMA warp
      auto hand_over = [&](int k) {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * t + k]);
      };
      const float* sc_scale = s_scale + (i & 7) * kScaleSlot;
      if (E) {
        const float4 w = *reinterpret_cast<const float4*>(sc_scale + 4 * hf);
        ksu = w.x;
        lvu = w.y;
        uniform = w.z != 0.f;
      }
      if (uniform) {
        // below fp32's range the scores are zero either way, but the mask's -inf must not meet a zero factor
        float f = E ? fq * ksu : p.scale_log2;
        if (E && f < 1.2e-38f) f = 1.2e-38f;  // a NaN scale stays
        if (k0 + FH - 1 > pos) {
#pragma unroll
          for (int c = 0; c < FH; ++c) sc[c] = (k0 + c <= pos) ? sc[c] : -INFINITY;
        }
        float mx[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
        for (int c = 4; c + 8 <= FH; c += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmax3(mx[k], sc[c + k], sc[c + 4 + k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], sc[FH - 4 + k]);
        const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * f;
        advance(mt + lvu);
        take_turn();
        const float mm = ref();
        float e = lvu - mm;
        if (E && mt != -INFINITY && e < -60.f - mt) e = -60.f - mt;
        float total = 0.f;
#pragma unroll
        for (int q = 0; q < FH / 32; ++q) {
          float s0, s1;
          weights(q, f, f, e, e, s0, s1);
          total += s0 + s1;
          if (C::kParts == 2 && 32 * (q + 1) == C::kPart1) hand_over(0);
        }
        pass_turn();
        l += E ? total * (pf_ex2(-mm - e) * kWeightInv) : total;
      } else {
        float fg[FH / 16], lv[FH / 16], mg[FH / 16], top = -INFINITY;
        const bool masked = __any_sync(0xffffffffu, k0 + FH - 1 > pos);
#pragma unroll
        for (int g = 0; g < FH / 16; ++g) {
          const int pg = (hf * FH + g * 16) >> psh;
          fg[g] = sc_scale[8 + 2 * pg] * fq;
          lv[g] = sc_scale[9 + 2 * pg];
        }
        if (masked) {  // scaled first: a masked score is -inf also beside a NaN scale
#pragma unroll
          for (int g = 0; g < FH / 16; ++g) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              sc[16 * g + c] = k0 + 16 * g + c <= pos ? sc[16 * g + c] * fg[g] : -INFINITY;
            fg[g] = 1.f;
          }
        }
#pragma unroll
        for (int g = 0; g < FH / 16; ++g) {
          float mx = fmax3(sc[16 * g], sc[16 * g + 1], sc[16 * g + 2]);
#pragma unroll
          for (int c = 3; c < 15; c += 2) mx = fmax3(mx, sc[16 * g + c], sc[16 * g + c + 1]);
          mg[g] = fmaxf(mx, sc[16 * g + 15]) * fg[g];
          top = fmaxf(top, mg[g] + lv[g]);
        }
        advance(top);
        take_turn();
        const float mm = ref();
#pragma unroll
        for (int q = 0; q < FH / 32; ++q) {
          float e[2], s2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float x = mg[2 * q + k];
            e[k] = x == -INFINITY ? 0.f : lv[2 * q + k] - mm;
            if (e[k] < -60.f - x && x != -INFINITY) e[k] = -60.f - x;  // a NaN scale stays
          }
          weights(q, fg[2 * q], fg[2 * q + 1], e[0], e[1], s2[0], s2[1]);
          l += s2[0] * (pf_ex2(-mm - e[0]) * kWeightInv) + s2[1] * (pf_ex2(-mm - e[1]) * kWeightInv);
          if (C::kParts == 2 && 32 * (q + 1) == C::kPart1) hand_over(0);
        }
        pass_turn();
      }
      if (!ok) break;
      hand_over(HV == 2 ? hf : C::kParts - 1);
    }
    tmem_wait_st();
    // ------------------------------------------------------------ o = O / l, or the split's partial
    bool got = ok;
    if (steps > 0) got = ok && __all_sync(0xffffffffu, mbar_wait(&ofull[t], 0u, p.status));
    tc_fence_after();
    const bool broken = pos >= *s_bad;
    // 128 bytes of every row at a time go through the warp's part of the Q tile (no MMA reads it any
    // more), so that eight lanes store one whole line
    uint8_t* stage = qs + t * T + quarter * 4096;
    auto put_lines = [&](const uint4 (&w)[8], uint8_t* base, int64_t row_bytes) {
#pragma unroll
      for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = w[c];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const int rl = k + (lane >> 3), rr = quarter * 32 + rl, qd = div_g(rr), rq = q0 + qd;
        const uint4 y = *reinterpret_cast<const uint4*>(stage + rl * 128 + (((lane & 7) ^ (rl & 7)) << 4));
        if (rr < p.QPT * p.G && rq < n)
          *reinterpret_cast<uint4*>(base + ((static_cast<int64_t>(r.row0) + rq) * p.Hq + h * p.G + rr - qd * p.G) * row_bytes +
                                    (lane & 7) * 16) = y;
      }
      __syncwarp();
    };
    if (!kTwo && p.splits == 1) {
      if (q0 >= 0) {
        const float inv = !got || broken || l == 0.f ? 0.f : (E ? kWeightInv : 1.f) / l;
#pragma unroll 1
        for (int c = 0; c < DH; c += 64) {
          uint4 w[8];
          float v[64];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            tmem_ld16(tmem_o + lrow + static_cast<uint32_t>(c + 16 * g), *reinterpret_cast<float(*)[16]>(v + 16 * g));
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              y[k] = broken ? 0u : round_bf16x2(v[16 * g + 2 * k] * inv, v[16 * g + 2 * k + 1] * inv);
            w[2 * g] = make_uint4(y[0], y[1], y[2], y[3]);
            w[2 * g + 1] = make_uint4(y[4], y[5], y[6], y[7]);
          }
          put_lines(w, reinterpret_cast<uint8_t*>(p.out + c), DH * 2);
        }
      }
    } else if (q0 >= 0) {
      const int64_t first = static_cast<int64_t>(kTwo ? 2 * split + t : split) * p.rows * p.Hq;
      if (live) {
        const int64_t prow = first + (static_cast<int64_t>(r.row0) + qi) * p.Hq + head;
        p.ws_ml[prow * 2] = steps > 0 && got ? m : -INFINITY;
        p.ws_ml[prow * 2 + 1] = broken ? -1.f : steps > 0 && got ? l : 0.f;
      }
      if (steps > 0) {
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          uint4 w[8];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float v[16];
            tmem_ld16(tmem_o + lrow + static_cast<uint32_t>(c + 16 * g), v);
            tmem_wait_ld();
            if (E) {
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] *= kWeightInv;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[4 * g + k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                                        __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
          }
          put_lines(w, reinterpret_cast<uint8_t*>(p.ws_o + first * DH + c), DH * 4);
        }
      }
    }
    if (*s_bad != 0x7fffffff && threadIdx.x == 128) atomicOr(p.status, SLIM_DEV_BADPAGE);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kFTmemPerTile);
  }
}

// Joins the parts of each (row, head): one warp each.
template <int DH>
__global__ void __launch_bounds__(256) merge_prefill_kernel(const PagedPrefillParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const PagedRows r = paged_rows(p.starts, p.lens, b, p.rows, p.max_new, p.c.cap, p.c.cap);
  if (r.bits) return;  // zeroed by the first kernel
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(r.n) * p.Hq) return;
  const int64_t row = static_cast<int64_t>(r.row0) * p.Hq + item, step = p.rows * p.Hq;
  float M = -INFINITY;
  bool broken = false;
  for (int s = 0; s < p.parts; ++s) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + s * step + row);
    M = fmaxf(M, ml.x);
    broken |= ml.y < 0.f;
  }
  constexpr int PL = DH / 32;  // columns of a lane
  float o[PL] = {}, L = 0.f;
  for (int s = 0; s < p.parts; ++s) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + s * step + row);
    // nothing attended in this part, whose O was not written then; a part over poisoned pages alone has no
    // maximum either, but its l is NaN and stays
    if (ml.x == -INFINITY && ml.y <= 0.f) continue;
    const float f = pf_ex2(ml.x - M);
    L = fmaf(f, ml.y, L);
    const float* src = p.ws_o + (s * step + row) * DH + lane * PL;
#pragma unroll
    for (int k = 0; k < PL; k += 2) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src + k));
      o[k] = fmaf(f, v.x, o[k]);
      o[k + 1] = fmaf(f, v.y, o[k + 1]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * DH + lane * PL);
#pragma unroll
  for (int k = 0; k < PL; k += 2) dst[k / 2] = broken ? 0u : round_bf16x2(o[k] * inv, o[k + 1] * inv);
}

// Rows of a (sequence, key head) up to which the kernel of paged_decode.cu is taken: it streams the cache
// near memory speed, where a 128-row tile here would be mostly empty. Its work grows with every 8 rows, here
// it does not. 8 sequences of 8000 rows, 8 key heads, there and here. 16 rows: dh = 128 58 and 77 us (bf16), 46
// and 60 (e4m3); dh = 64 34 and 65, 37 and 53. 32 rows: dh = 128 88 and 75, 87 and 60; dh = 64 52 and 64, 57
// and 54 (e4m3, 64 sequences of 500: 45 and 58).
bool pf_few(const slim_paged_cache& c, int Hq, int64_t max_new) {
  return max_new * (Hq / c.Hkv) <= (c.dh == 64 ? 32 : 16);
}

struct PfPlan {
  int G, QPT, pairs, splits;
  bool two;
  size_t o_bytes, ml_bytes;
};
size_t pf_up256(size_t x) { return (x + 255) & ~size_t(255); }
PfPlan pf_plan(const slim_paged_cache& c, int Hq, int64_t rows, int64_t max_new, int64_t t_hint) {
  PfPlan f;
  f.G = Hq / c.Hkv;
  f.QPT = kFQ / f.G;
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page;
  const int64_t hint = t_hint > 0 ? std::min(t_hint, cap) : cap;
  f.pairs = static_cast<int>((max_new + 2 * f.QPT - 1) / (2 * f.QPT));
  // Ranges of keys: as many as make the waves of CTAs end together soonest. A CTA's time is its key tiles
  // and about kFSetup tiles more (query, first S, output); how many pairs of row tiles there are follows
  // from the rows up to half a pair per sequence.
  const int sms = num_sms();
  const int64_t nk = (hint + kFK - 1) / kFK;
  const int64_t some = std::min<int64_t>(static_cast<int64_t>(c.B) * f.pairs,
                                         std::max(rows / (2 * f.QPT) + (c.B + 1) / 2, rows / max_new * f.pairs));
  const int64_t ctas = std::max<int64_t>(1, some) * c.Hkv;
  double best = 0;
  f.splits = 1;
  f.two = false;
  for (int two = 0; two <= (c.dtype == SLIM_E4M3 && max_new <= f.QPT ? 1 : 0); ++two)
    for (int64_t s = 1; s <= std::min<int64_t>(64, std::max<int64_t>(1, nk / 4)); ++s) {
      const double waves = static_cast<double>((ctas * s + sms - 1) / sms);
      const double cost = waves * (static_cast<double>(nk) / (s * (two ? 2 : 1)) + kFSetup + (s > 1 || two ? 2 : 0));
      if ((s == 1 && !two) || cost < 0.95 * best) {
        best = cost;
        f.splits = static_cast<int>(s);
        f.two = two != 0;
      }
    }
  const int parts = f.splits * (f.two ? 2 : 1);
  const size_t items = parts > 1 ? static_cast<size_t>(parts) * rows * Hq : 0;
  f.o_bytes = pf_up256(items * c.dh * 4);
  f.ml_bytes = pf_up256(items * 8);
  return f;
}

template <bool E, int DHB, bool kTwo>
cudaError_t launch_pf(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedPrefillParams& p, cudaStream_t st,
                      int* launches) {
  using C = PfCfg<E, DHB>;
  auto kern = paged_prefill_kernel<E, DHB, kTwo>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.c.B * p.c.Hkv) * p.pairs * p.splits, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  if (launches) ++*launches;
  if (p.parts == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg2 = cfg;
  cfg2.gridDim = dim3(static_cast<unsigned>((p.max_new * p.Hq + 7) / 8), static_cast<unsigned>(p.c.B), 1);
  cfg2.blockDim = dim3(256, 1, 1);
  cfg2.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg2, merge_prefill_kernel<C::DH>, p);
  if (e == cudaSuccess && launches) ++*launches;
  return e;
}

}  // namespace

bool paged_prefill_fits(const slim_paged_cache& c, int Hq, int64_t rows, int64_t max_new, int64_t t_hint) {
  if (pf_few(c, Hq, max_new)) return true;
  const PfPlan f = pf_plan(c, Hq, rows, max_new, t_hint);
  return static_cast<int64_t>(c.B) * c.Hkv * f.pairs * f.splits < (int64_t(1) << 31);
}

size_t paged_prefill_ws_bytes(const slim_paged_cache& c, int Hq, int64_t rows, int64_t max_new, int64_t t_hint) {
  if (pf_few(c, Hq, max_new)) return paged_rows_ws_bytes(c, static_cast<int>(max_new) * (Hq / c.Hkv));
  const PfPlan f = pf_plan(c, Hq, rows, max_new, t_hint);
  return f.o_bytes + f.ml_bytes;
}

cudaError_t launch_paged_prefill(const slim_paged_cache& c, const void* q, int64_t q_stride, const int32_t* starts,
                                 const int32_t* lens, int64_t rows, int64_t max_new, int Hq, int64_t t_hint,
                                 void* out, void* workspace, int32_t* status, cudaStream_t st, int* launches) {
  if (pf_few(c, Hq, max_new))
    return launch_paged_rows(c, q, q_stride, starts, lens, rows, max_new, 0, Hq, t_hint, out, workspace, status, st,
                             launches);
  const PfPlan f = pf_plan(c, Hq, rows, max_new, t_hint);
  PagedPrefillParams p;
  p.c = paged_view(c);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.starts = starts;
  p.lens = lens;
  p.rows = rows;
  p.max_new = max_new;
  p.Hq = Hq;
  p.G = f.G;
  p.QPT = f.QPT;
  p.g_inv = (65536u + static_cast<uint32_t>(f.G) - 1u) / static_cast<uint32_t>(f.G);
  p.pairs = f.pairs;
  p.splits = f.splits;
  p.parts = f.splits * (f.two ? 2 : 1);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + f.o_bytes);
  p.status = status;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(c.dh));
  CUtensorMap kmap = {}, vmap = {};
  if (c.dtype == SLIM_BF16) {
    const uint64_t lines = static_cast<uint64_t>(c.num_pages) * c.Hkv * c.page;
    if (!encode_tmap_2d_bf16(&kmap, c.kpages, c.dh, lines, static_cast<uint64_t>(c.dh) * 2u, 64, c.page, true) ||
        !encode_tmap_2d_bf16(&vmap, c.vpages, c.dh, lines, static_cast<uint64_t>(c.dh) * 2u, 64, c.page, true))
      return cudaErrorInvalidValue;
    return c.dh == 64 ? launch_pf<false, 1, false>(kmap, vmap, p, st, launches)
                      : launch_pf<false, 2, false>(kmap, vmap, p, st, launches);
  }
  // e4m3 keys go to the MMA as they are: whole rows, in the swizzle of their length
  if (!encode_tmap_2d_u8(&kmap, c.kpages, c.dh, static_cast<uint64_t>(c.num_pages) * c.Hkv * c.page, c.dh, c.page))
    return cudaErrorInvalidValue;
  if (f.two)
    return c.dh == 64 ? launch_pf<true, 1, true>(kmap, vmap, p, st, launches)
                      : launch_pf<true, 2, true>(kmap, vmap, p, st, launches);
  return c.dh == 64 ? launch_pf<true, 1, false>(kmap, vmap, p, st, launches)
                    : launch_pf<true, 2, false>(kmap, vmap, p, st, launches);
}

}  // namespace slim
