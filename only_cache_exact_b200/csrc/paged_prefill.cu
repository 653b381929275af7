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
//   warp 0        loads K and V, page by page: bf16 by TMA straight into the MMA's
//                 128-byte swizzle (rings of 2 (dh = 128) or 4 tiles); e4m3 by bulk
//                 copies of whole page heads into one raw K and one raw V tile
//   warp 1        issues tcgen05.mma: S_t = Q_t·K^T into the tile's TMEM S region,
//                 O_t += P_t·V with P_t read from tensor memory, in the order
//                 P_0(j)·V_j, S_0(j+1), P_1(j)·V_j, S_1(j+1)
//   warps 4..7, 8..11  softmax of tile 0 and 1, one row per thread: causal mask,
//                 lazy running maximum (O is rescaled only when a maximum grows by
//                 more than 2^8), P over the S region, row sums in fp32
//   warps 12..15  (e4m3) codes to f16 in the MMA's layout
// e4m3 codes are exact in f16, so the MMAs of an e4m3 cache run in f16 on the bare
// codes: the key scale of a page multiplies its scores, the value scale 2^lv its
// probabilities, P = 2^(s + lv - m) with m the running maximum of s + lv, and
// the query is brought into f16's range by a power of two per row. P is rounded
// to f16 (2^-11) there; over bf16 values it is rounded to bf16 (2^-8), the type
// the MMA wants beside them.
// Key rows at or past the sequence's end are zeroed in V before the first MMA
// that reads them: a masked P = 0 never meets what a page held before.
//
// Few rows behind a long cache leave most SMs without a CTA: the key tiles are
// then cut into `splits` ranges, each CTA leaves (m, l, O), and
// merge_prefill_kernel joins them.
#include <algorithm>

#include "paged.cuh"

namespace slim {

namespace {

constexpr int kFQ = 128;  // rows of a tile
constexpr int kFK = 128;  // keys of a tile
constexpr uint32_t kFTmemPerTile = 256;  // S (and P over it) at columns 0..127, O at 128
constexpr float kFLazyLog2 = 8.f;

struct PagedPrefillParams {
  PagedView c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* starts;
  const int32_t* lens;
  int64_t rows, max_new;
  int Hq, G, QPT;  // QPT = 128 / G queries of a tile
  int pairs, splits;
  __nv_bfloat16* out;
  float* ws_o;   // [split][rows][Hq][dh], splits > 1
  float* ws_ml;  // [split][rows][Hq][2]
  int32_t* status;
  float scale_log2;
};

template <bool E, int DHB>
struct PfCfg {
  static constexpr int DH = 64 * DHB;
  static constexpr int NS = DHB == 2 ? 2 : 4;                  // tiles of a K and a V ring
  static constexpr uint32_t kTile = kFK * DH * 2u;             // bytes of a 16-bit K, V or Q tile
  static constexpr uint32_t kRaw = E ? kFK * DH : 0u;          // bytes of a raw e4m3 tile
  static constexpr int kThreads = E ? 512 : 384;
  static constexpr uint32_t kSmem = 2u * kTile + 2u * NS * kTile + 2u * kRaw + 512u + 1024u;
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
// kind::f16 instruction descriptor with f16 A and B, fp32 D (both type fields 0).
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool E, int DHB>
__global__ void __launch_bounds__(PfCfg<E, DHB>::kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const PagedPrefillParams p) {
  using C = PfCfg<E, DHB>;
  constexpr int DH = C::DH, NS = C::NS;
  constexpr uint32_t T = C::kTile;
  extern __shared__ uint8_t pf_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pf_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = sm;              // [row tile][DHB boxes][128 rows][128 B]
  uint8_t* ks = qs + 2 * T;      // [stage][DHB boxes][128 rows][128 B]
  uint8_t* vs = ks + NS * T;
  uint8_t* rk = vs + NS * T;     // raw K, raw V tile (e4m3)
  uint8_t* rv = rk + C::kRaw;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rv + C::kRaw);
  uint64_t* qbar = bars;           // Q written by the softmax warps
  uint64_t* kfull = bars + 1;      // [NS]
  uint64_t* kempty = kfull + NS;   // [NS]
  uint64_t* vfull = kempty + NS;   // [NS]
  uint64_t* vempty = vfull + NS;   // [NS]
  uint64_t* sfull = vempty + NS;   // [2] S written
  uint64_t* pready = sfull + 2;    // [2] P written over S (and O rescaled)
  uint64_t* pfree = pready + 2;    // [2] the P·V MMA completed
  uint64_t* ofull = pfree + 2;     // [2] the tile's last P·V MMA completed
  uint64_t* rfull = ofull + 2;     // [2] raw K, raw V landed
  uint64_t* rempty = rfull + 2;    // [2] raw K, raw V converted
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rempty + 2);
  int* s_bad = reinterpret_cast<int*>(tmem_slot + 1);  // first position whose page is outside the pool
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
  auto tile_q0 = [&](int t) { return (nqt - 2 * (pair + 1) + t) * p.QPT; };
  auto tile_keys = [&](int t) {  // key tiles that tile t attends
    const int q0 = tile_q0(t);
    return q0 < 0 ? 0 : (len + min(q0 + p.QPT, n) - 1) / kFK + 1;
  };
  const int nk_all = tile_keys(1);
  const int kt0 = static_cast<int>(static_cast<int64_t>(split) * nk_all / p.splits);
  const int kt1 = static_cast<int>(static_cast<int64_t>(split + 1) * nk_all / p.splits);
  auto tile_end = [&](int t) { return max(kt0, min(kt1, tile_keys(t))); };
  const int nkt = kt1 - kt0;

  if (warp == 0 && lane == 0) {
    mbar_init(qbar, 8);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], E ? 4 : 1);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], E ? 4 : 1);
      mbar_init(&vempty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[t], 4);
      mbar_init(&pfree[t], 1);
      mbar_init(&ofull[t], 1);
      mbar_init(&rfull[t], 1);
      mbar_init(&rempty[t], 4);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  for (int i = page_lo + static_cast<int>(threadIdx.x); i < page_hi; i += C::kThreads) {
    const int id = __ldg(table + i);
    if (id < 0 || id >= p.c.num_pages) atomicMin(s_bad, i << psh);
  }
  __syncthreads();
  // keys from here on are not used: the sequence's end, or a page outside the pool (whose place page 0
  // takes in the loads)
  const int Lz = min(L, *s_bad);

  // page number of page i of the sequence for the loads: page 0 where it is outside the pool
  auto page_id = [&](int i) {
    const int id = __ldg(table + i);
    return id >= 0 && id < p.c.num_pages ? id : 0;
  };
  // pages of key tile j that hold rows of the sequence
  auto pages_of = [&](int j) { return min(ppt, ((L - 1 - j * kFK) >> psh) + 1); };

  if (warp < 4) {
    reg_dec<48>();
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      int nk_issued = 0, nv_issued = 0;
      int id_next = nkt > 0 && lane < pages_of(kt0) ? page_id(kt0 * ppt + lane) : 0;
      for (int i = 0; i < nkt; ++i) {
        const int j = kt0 + i, npg = pages_of(j), id = id_next;
        if (i + 1 < nkt) id_next = lane < pages_of(j + 1) ? page_id((j + 1) * ppt + lane) : 0;
        const uint32_t bytes = static_cast<uint32_t>(npg << psh) * DH * (E ? 1u : 2u);
        if (E) {
          const uint32_t ph = static_cast<uint32_t>(i & 1);
          const int64_t src = id * p.c.page_bytes + h * p.c.head_bytes;
          const uint32_t hb = static_cast<uint32_t>(p.c.head_bytes);
          if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(&rempty[0], ph ^ 1u, p.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(&rfull[0], bytes);
          __syncwarp();
          if (lane < npg) bulk_load_g2s(rk + lane * hb, p.c.k + src, hb, &rfull[0]);
          ++nk_issued;
          if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(&rempty[1], ph ^ 1u, p.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(&rfull[1], bytes);
          __syncwarp();
          if (lane < npg) bulk_load_g2s(rv + lane * hb, p.c.v + src, hb, &rfull[1]);
          ++nv_issued;
        } else {
          const int s = i % NS;
          const uint32_t ph = static_cast<uint32_t>((i / NS) & 1);
          const int y = (id * p.c.Hkv + h) << psh;
          const uint32_t off = static_cast<uint32_t>(lane << psh) * 128u;
          if (i >= NS && !__all_sync(0xffffffffu, mbar_wait(&kempty[s], ph ^ 1u, p.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(&kfull[s], bytes);
          __syncwarp();
          if (lane < npg) {
#pragma unroll
            for (int k = 0; k < DHB; ++k)
              tma_load_2d(ks + s * T + k * 16384 + off, &kmap, 64 * k, y, &kfull[s], l2_policy_evict_last());
          }
          ++nk_issued;
          if (i >= NS && !__all_sync(0xffffffffu, mbar_wait(&vempty[s], ph ^ 1u, p.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(&vfull[s], bytes);
          __syncwarp();
          if (lane < npg) {
#pragma unroll
            for (int k = 0; k < DHB; ++k)
              tma_load_2d(vs + s * T + k * 16384 + off, &vmap, 64 * k, y, &vfull[s], l2_policy_evict_last());
          }
          ++nv_issued;
        }
      }
      // every issued copy lands before the CTA exits
      if (E) {
        if (nk_issued > 0) mbar_wait(&rfull[0], static_cast<uint32_t>(nk_issued - 1) & 1u, p.status);
        if (nv_issued > 0) mbar_wait(&rfull[1], static_cast<uint32_t>(nv_issued - 1) & 1u, p.status);
      } else {
        for (int u = max(0, nk_issued - NS); u < nk_issued; ++u)
          mbar_wait(&kfull[u % NS], static_cast<uint32_t>(u / NS) & 1u, p.status);
        for (int u = max(0, nv_issued - NS); u < nv_issued; ++u)
          mbar_wait(&vfull[u % NS], static_cast<uint32_t>(u / NS) & 1u, p.status);
      }
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc_s = E ? idesc_f16_f32(kFQ, kFK, 0u, 0u) : idesc_bf16_f32(kFQ, kFK, 0u, 0u);
      const uint32_t idesc_o = E ? idesc_f16_f32(kFQ, DH, 0u, 1u) : idesc_bf16_f32(kFQ, DH, 0u, 1u);
      const uint32_t qb = smem_u32(qs), kb0 = smem_u32(ks), vb0 = smem_u32(vs);
      int nk[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) nk[t] = tile_end(t) - kt0;
      bool ok = mbar_wait(qbar, 0u, p.status);
      auto issue_s = [&](int t, int i) {
        const int s = i % NS;
        if (!mbar_wait(&kfull[s], static_cast<uint32_t>(i / NS) & 1u, p.status)) return false;
        tc_fence_after();
        const uint32_t kb = kb0 + s * T, qtb = qb + t * T;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384u + (kk & 3) * 32u;
          umma_f16(tmem + t * kFTmemPerTile, smem_desc(qtb + off, 16, 1024, kLayoutSW128),
                   smem_desc(kb + off, 16, 1024, kLayoutSW128), idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&sfull[t]);
        if (t == 1) umma_commit(&kempty[s]);
        return true;
      };
      auto issue_pv = [&](int t, int i) {
        const int s = i % NS;
        if (!mbar_wait(&pready[t], static_cast<uint32_t>(i) & 1u, p.status) ||
            !mbar_wait(&vfull[s], static_cast<uint32_t>(i / NS) & 1u, p.status))
          return false;
        tc_fence_after();
        const uint32_t vb = vb0 + s * T, pt = tmem + t * kFTmemPerTile;
#pragma unroll
        for (int kk = 0; kk < kFK / 16; ++kk) {
          pf_umma_tmem_a(tmem + t * kFTmemPerTile + 128u, pt + static_cast<uint32_t>(kk * 8),
                         smem_desc(vb + kk * 2048u, 16384, 1024, kLayoutSW128), idesc_o,
                         (i > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(&pfree[t]);
        if (t == 1) umma_commit(&vempty[s]);
        return true;
      };
      bool committed[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        committed[t] = false;
        if (ok && nk[t] > 0) ok = issue_s(t, 0);
      }
      for (int i = 0; ok && i < nk[1]; ++i) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || i >= nk[t]) continue;
          if (!issue_pv(t, i)) ok = false;
          if (ok && i == nk[t] - 1) {
            umma_commit(&ofull[t]);
            committed[t] = true;
          }
          // S_t(i+1) overwrites the P that the P·V above reads: issued after it
          if (ok && i + 1 < nk[t] && !issue_s(t, i + 1)) ok = false;
        }
      }
      // also after a failure: each output barrier covers every MMA issued
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (!committed[t]) umma_commit(&ofull[t]);
#pragma unroll
      for (int t = 0; t < 2; ++t) mbar_wait(&ofull[t], 0u, p.status);
    }
  } else if (E && warp >= 12) {
    // ------------------------------------------------------------ codes to f16
    reg_dec<80>();
    const int tid = threadIdx.x - 384;
    constexpr int CPR = DH / 16;  // 16-code chunks of a row
    auto convert = [&](const uint8_t* raw, uint8_t* dst, int valid) {
#pragma unroll 4
      for (int u = tid; u < kFK * CPR; u += 128) {
        const int row = u / CPR, cc = u - row * CPR;
        uint4 w = *reinterpret_cast<const uint4*>(raw + u * 16);
        if (row >= valid) w = make_uint4(0u, 0u, 0u, 0u);
        const uint4 a = make_uint4(e4m3x2_to_f16x2(w.x & 0xffffu), e4m3x2_to_f16x2(w.x >> 16),
                                   e4m3x2_to_f16x2(w.y & 0xffffu), e4m3x2_to_f16x2(w.y >> 16));
        const uint4 d = make_uint4(e4m3x2_to_f16x2(w.z & 0xffffu), e4m3x2_to_f16x2(w.z >> 16),
                                   e4m3x2_to_f16x2(w.w & 0xffffu), e4m3x2_to_f16x2(w.w >> 16));
        uint8_t* box = dst + (cc >> 2) * 16384 + row * 128;
        const int c0 = (2 * cc) & 7, sw = row & 7;
        // lanes of the second box write their odd chunk first: eight lanes, eight banks
        const bool odd = (cc >> 2) != 0;
        *reinterpret_cast<uint4*>(box + (((c0 + (odd ? 1 : 0)) ^ sw) << 4)) = odd ? d : a;
        *reinterpret_cast<uint4*>(box + (((c0 + (odd ? 0 : 1)) ^ sw) << 4)) = odd ? a : d;
      }
    };
    for (int i = 0; i < nkt; ++i) {
      const int s = i % NS, valid = Lz - (kt0 + i) * kFK;
      const uint32_t ph = static_cast<uint32_t>((i / NS) & 1), rph = static_cast<uint32_t>(i & 1);
      bool got = mbar_wait(&rfull[0], rph, p.status) && (i < NS || mbar_wait(&kempty[s], ph ^ 1u, p.status));
      if (!__all_sync(0xffffffffu, got)) break;
      convert(rk, ks + s * T, valid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&rempty[0]);
        mbar_arrive(&kfull[s]);
      }
      got = mbar_wait(&rfull[1], rph, p.status) && (i < NS || mbar_wait(&vempty[s], ph ^ 1u, p.status));
      if (!__all_sync(0xffffffffu, got)) break;
      convert(rv, vs + s * T, valid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&rempty[1]);
        mbar_arrive(&vfull[s]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax of row tile t
    reg_inc<E ? 192 : 224>();
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lrow = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + t * kFTmemPerTile, tmem_o = ts + 128u;
    const int q0 = tile_q0(t), nkt_t = tile_end(t) - kt0;
    const int nkt_below = t > 0 ? tile_end(0) - kt0 : 0;  // key tiles that the lower tile attends too
    const int qi = q0 + row / p.G, head = h * p.G + row % p.G;
    const bool live = q0 >= 0 && row < p.QPT * p.G && qi < n;
    const int pos = live ? len + qi : -1;  // a row without a query attends nothing
    float fq = p.scale_log2;
    // this thread's query row into the Q tile (zeros where there is none)
    {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(r.row0) + (live ? qi : 0)) * p.q_stride +
                                                        static_cast<int64_t>(head) * DH);
      uint4 w[DH / 8];
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) w[c] = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      if (E) {
        uint32_t amax = 0u;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) amax = max(amax, max(x[k] & 0x7fffu, (x[k] >> 16) & 0x7fffu));
        }
        const int e = max(-126, min(126, static_cast<int>(amax >> 7) - 127));
        const float inv = exp2_int(-e);
        fq *= exp2_int(e);
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {
          uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 hv = __floats2half2_rn(bf16lo(x[k]) * inv, bf16hi(x[k]) * inv);
            x[k] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          w[c] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
#pragma unroll
      for (int c = 0; c < DH / 8; ++c)
        *reinterpret_cast<uint4*>(qs + t * T + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = w[c];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qbar);
    }
    // e4m3: scales of a key tile's pages, one page per lane, fetched a tile ahead
    auto fetch = [&](int i, float& ksc, float& vsc) {  // key scale and the value scale's exponent
      ksc = 1.f;
      vsc = 0.f;
      const int j = kt0 + i;
      if (i < nkt_t && lane < pages_of(j)) {
        const int64_t at = static_cast<int64_t>(page_id(j * ppt + lane)) * p.c.Hkv + h;
        ksc = __ldg(p.c.ks + at);
        vsc = scale_log2(__ldg(p.c.vs + at));
      }
    };
    float ks_next = 1.f, lv_next = 0.f;
    if (E) fetch(0, ks_next, lv_next);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < nkt_t; ++i) {
      const int s = i % NS;
      const float ks_lane = ks_next, lv_lane = lv_next;
      if (E) fetch(i + 1, ks_next, lv_next);
      if (!__all_sync(0xffffffffu, mbar_wait(&sfull[t], static_cast<uint32_t>(i) & 1u, p.status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sc[kFK];
#pragma unroll
      for (int c = 0; c < kFK / 16; ++c)
        tmem_ld16(ts + lrow + static_cast<uint32_t>(16 * c), *reinterpret_cast<float(*)[16]>(sc + 16 * c));
      tmem_wait_ld();
      const int k0 = (kt0 + i) * kFK;
      // Running maximum of the weights' exponents: of the scores in log2 units, for e4m3 plus the value
      // scale's exponent lv, so that P stays in f16's range whatever the pages' scales are. P of key t
      // is 2^(s_t + e), e = lv - m, and l adds P·2^-lv. Where a group's largest P is below 2^-60 (its
      // f16 is zero) e is raised to keep the fp32 sum from underflowing.
      float alpha = 1.f;
      auto advance = [&](float mt) {
        if (m == -INFINITY) {
          m = mt;
        } else if (mt > m + kFLazyLog2) {
          alpha = pf_ex2(m - mt);
          m = mt;
          l *= alpha;
        }
      };
      // P of keys 32 q .. 32 q + 31 to tensor memory; returns their sum
      auto weights = [&](int q, float f, float e0, float e1, float& sum0, float& sum1) {
        uint32_t pk[16];
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float e = c < 8 ? e0 : e1;
          const float a = pf_ex2(fmaf(sc[32 * q + 2 * c], f, e));
          const float bb = pf_ex2(fmaf(sc[32 * q + 2 * c + 1], f, e));
          s4[(c & 1) + (c < 8 ? 0 : 2)] += a + bb;
          if (E) {
            const __half2 hv = __floats2half2_rn(a, bb);
            pk[c] = *reinterpret_cast<const uint32_t*>(&hv);
          } else {
            const __nv_bfloat162 hv = __floats2bfloat162_rn(a, bb);
            pk[c] = *reinterpret_cast<const uint32_t*>(&hv);
          }
        }
        pf_tmem_st16(ts + lrow + static_cast<uint32_t>(16 * q), pk);
        sum0 = s4[0] + s4[1];
        sum1 = s4[2] + s4[3];
      };
      float ksu = 1.f, lvu = 0.f;
      bool uniform = true;  // one scale pair for all pages of the tile
      if (E) {
        ksu = __shfl_sync(0xffffffffu, ks_lane, 0);
        lvu = __shfl_sync(0xffffffffu, lv_lane, 0);
        uniform = __all_sync(0xffffffffu, lane >= pages_of(kt0 + i) || (ks_lane == ksu && lv_lane == lvu));
      }
      if (uniform) {
        const float f = E ? fq * ksu : p.scale_log2;
        if (k0 + kFK - 1 > pos) {
#pragma unroll
          for (int c = 0; c < kFK; ++c) sc[c] = (k0 + c <= pos) ? sc[c] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kFK; ++c) mx[c & 3] = fmaxf(mx[c & 3], sc[c]);
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
        advance(mt + lvu);
        const float mm = m == -INFINITY ? 0.f : m;
        float e = lvu - mm;
        if (E && mt != -INFINITY && e < -60.f - mt) e = -60.f - mt;
        float total = 0.f;
#pragma unroll
        for (int q = 0; q < kFK / 32; ++q) {
          float s0, s1;
          weights(q, f, e, e, s0, s1);
          total += s0 + s1;
        }
        l += E ? total * pf_ex2(-mm - e) : total;
      } else {
        float lv[kFK / 16], mg[kFK / 16], top = -INFINITY;
#pragma unroll
        for (int g = 0; g < kFK / 16; ++g) {
          const float f = __shfl_sync(0xffffffffu, ks_lane, (g * 16) >> psh) * fq;
          lv[g] = __shfl_sync(0xffffffffu, lv_lane, (g * 16) >> psh);
          mg[g] = -INFINITY;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            sc[16 * g + c] = k0 + 16 * g + c <= pos ? sc[16 * g + c] * f : -INFINITY;  // after a NaN scale
            mg[g] = fmaxf(mg[g], sc[16 * g + c]);
          }
          top = fmaxf(top, mg[g] + lv[g]);
        }
        advance(top);
        const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int q = 0; q < kFK / 32; ++q) {
          float e[2], s2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float x = mg[2 * q + k];
            e[k] = x == -INFINITY ? 0.f : lv[2 * q + k] - mm;
            if (e[k] < -60.f - x && x != -INFINITY) e[k] = -60.f - x;  // a NaN scale stays
          }
          weights(q, 1.f, e[0], e[1], s2[0], s2[1]);
          l += s2[0] * pf_ex2(-mm - e[0]) + s2[1] * pf_ex2(-mm - e[1]);
        }
      }
      if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O is rescaled once the previous key tile's P·V has completed
        if (!__all_sync(0xffffffffu, mbar_wait(&pfree[t], static_cast<uint32_t>(i - 1) & 1u, p.status))) {
          tmem_wait_st();
          ok = false;
          break;
        }
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
      tmem_wait_st();
      // bf16: key rows from Lz on are zeroed in V (thread r takes key row r, once
      // the tile's V has landed) by the lowest tile that attends this key tile
      if (!E && k0 + kFK > Lz && i >= nkt_below && k0 + row >= Lz) {
        if (mbar_wait(&vfull[s], static_cast<uint32_t>(i / NS) & 1u, p.status)) {
          uint8_t* vrow = vs + s * T + row * 128;
#pragma unroll
          for (int k = 0; k < DHB; ++k)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vrow + k * 16384 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (!E) fence_proxy_async_smem();  // zeroed V rows are read by the tensor cores
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pready[t]);
    }
    // ------------------------------------------------------------ o = O / l, or the split's partial
    bool got = ok;
    if (nkt_t > 0) got = ok && __all_sync(0xffffffffu, mbar_wait(&ofull[t], 0u, p.status));
    tc_fence_after();
    const bool broken = pos >= *s_bad;
    const int64_t orow = (static_cast<int64_t>(r.row0) + (live ? qi : 0)) * p.Hq + head;
    if (p.splits == 1) {
      if (q0 >= 0) {
        const float inv = !got || broken || l == 0.f ? 0.f : 1.f / l;
        for (int c = 0; c < DH; c += 16) {
          float v[16];
          tmem_ld16(tmem_o + lrow + static_cast<uint32_t>(c), v);
          tmem_wait_ld();
          if (live) {
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = broken ? 0u : pack_bf16x2(v[2 * k] * inv, v[2 * k + 1] * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * DH + c);
            dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
            dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      }
    } else if (q0 >= 0) {
      const int64_t prow = static_cast<int64_t>(split) * p.rows * p.Hq + orow;
      if (live) {
        p.ws_ml[prow * 2] = nkt_t > 0 && got ? m : -INFINITY;
        p.ws_ml[prow * 2 + 1] = broken ? -1.f : nkt_t > 0 && got ? l : 0.f;
      }
      if (nkt_t > 0) {
        for (int c = 0; c < DH; c += 16) {
          float v[16];
          tmem_ld16(tmem_o + lrow + static_cast<uint32_t>(c), v);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(p.ws_o + prow * DH + c + k) =
                  make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
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

// Joins the splits of each (row, head): one warp each.
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
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + s * step + row);
    M = fmaxf(M, ml.x);
    broken |= ml.y < 0.f;
  }
  constexpr int PL = DH / 32;  // columns of a lane
  float o[PL] = {}, L = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + s * step + row);
    if (ml.x == -INFINITY) continue;
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
  for (int k = 0; k < PL; k += 2) dst[k / 2] = broken ? 0u : pack_bf16x2(o[k] * inv, o[k + 1] * inv);
}

struct PfPlan {
  int G, QPT, pairs, splits;
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
  // as many ranges of keys as there are SMs for, of four key tiles at least
  const int64_t ctas = static_cast<int64_t>(c.B) * c.Hkv * f.pairs;
  const int64_t by_sms = num_sms() / std::max<int64_t>(ctas, 1), by_keys = hint / (4 * kFK);
  f.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(by_sms, by_keys), 64)));
  const size_t items = f.splits > 1 ? static_cast<size_t>(f.splits) * rows * Hq : 0;
  f.o_bytes = pf_up256(items * c.dh * 4);
  f.ml_bytes = pf_up256(items * 8);
  return f;
}

template <bool E, int DHB>
cudaError_t launch_pf(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedPrefillParams& p, cudaStream_t st,
                      int* launches) {
  using C = PfCfg<E, DHB>;
  auto kern = paged_prefill_kernel<E, DHB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
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
  if (p.splits == 1) return cudaSuccess;
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
  const PfPlan f = pf_plan(c, Hq, rows, max_new, t_hint);
  return static_cast<int64_t>(c.B) * c.Hkv * f.pairs * f.splits < (int64_t(1) << 31);
}

size_t paged_prefill_ws_bytes(const slim_paged_cache& c, int Hq, int64_t rows, int64_t max_new, int64_t t_hint) {
  const PfPlan f = pf_plan(c, Hq, rows, max_new, t_hint);
  return f.o_bytes + f.ml_bytes;
}

cudaError_t launch_paged_prefill(const slim_paged_cache& c, const void* q, int64_t q_stride, const int32_t* starts,
                                 const int32_t* lens, int64_t rows, int64_t max_new, int Hq, int64_t t_hint,
                                 void* out, void* workspace, int32_t* status, cudaStream_t st, int* launches) {
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
  p.pairs = f.pairs;
  p.splits = f.splits;
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
    return c.dh == 64 ? launch_pf<false, 1>(kmap, vmap, p, st, launches)
                      : launch_pf<false, 2>(kmap, vmap, p, st, launches);
  }
  return c.dh == 64 ? launch_pf<true, 1>(kmap, vmap, p, st, launches)
                    : launch_pf<true, 2>(kmap, vmap, p, st, launches);
}

}  // namespace slim
