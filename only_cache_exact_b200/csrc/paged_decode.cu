// Attention of a few query rows per sequence over a paged K+V cache in bf16 or
// e4m3: slim_mha_paged_decode (one row), and slim_mha_paged_prefill where the
// rows that share a key head are at most 32 (a few proposed tokens).
//
// Mathematics, per sequence and key/value head, for the G query heads that
// share it: s_t = q·K_t·log2(e)/sqrt(dh), m = max s, p_t = 2^(s_t - m),
// o = Σ p_t V_t / Σ p_t, kept as a running (m, l, o) per warp and joined by
// 2^(m_i - m). In e4m3 K_t = ks·k8_t and V_t = 2^lv·v8_t with scales of the page
// and head: ks multiplies the score, and the weights of the sum over v8 are
// P_t = 2^(s_t + lv - m) with m the running maximum of s + lv, which keeps them
// in f16's range whatever the pages' scales are; l adds P_t·2^-lv.
//
// Bound: memory. Each cached element is read once and meets 4 flops per row (a
// query and head) for its 2 or 1 bytes; the row count of every matrix product
// is 8 to 32, so the warp-level MMA is ample and needs no tile to be filled. Rows
// are its N and keys its M (S^T = K·q^T) and then columns its M (O^T = V^T·p^T),
// so that up to 8 rows cost half of what 16-row tiles of them would: K and V
// are the A operands straight from shared memory by ldmatrix, and the
// probabilities go from the result's layout to the operand's by movmatrix,
// without shared memory. e4m3 codes become f16 pairs exactly (one cvt per
// pair), with the query scaled into f16's range by a power of two per head.
// Probabilities are rounded to f16 (2^-11) for e4m3; for bf16 values they are
// split in two bf16 parts (2^-16), since one part (2^-8) would be the largest
// error of the whole step.
//
// Work split: 16-row tiles of all (sequence, head group) pairs on one line, cut
// in equal shares for the CTAs and, inside, for their 8 warps; a warp streams
// its tiles through its own ring in shared memory (cp.async, no barrier with
// other warps), three stages deep: 24 KB a warp, 128 KB and more in flight per
// SM. Partials of warps that end in one sequence are joined in the CTA; what a
// sequence has in other CTAs is joined by merge_paged_kernel. Small calls take
// one CTA per (sequence, head group) instead and need no merge.
#include <algorithm>

#include "paged.cuh"

namespace slim {

namespace {

constexpr int kDW = 8;                 // warps of a CTA
constexpr int kDThreads = kDW * 32;
constexpr int kDRing = 24 * 1024;      // bytes of a warp's ring
constexpr int kDSlots = 2 * kDW;       // partials a CTA can leave: kDW of warps' ends, kDW of sequences that end inside a warp's share

struct PagedDecodeParams {
  PagedView c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* lens;
  const int32_t* starts;  // packed query rows of each sequence; nullptr: row b of sequence b
  int64_t rows, max_new;
  int extra;      // rows that lens does not count (starts == nullptr)
  int Hq, G, NG;  // G query heads per key head; rows of a (sequence, key head) in NG groups
  int HG;         // Hkv * NG work sequences per cache sequence
  __nv_bfloat16* out;
  float* ws_o;     // [ctas][kDSlots][heads][dh]
  float* ws_ml;    // [ctas][kDSlots][heads][2]
  uint32_t* ws_pre;  // [B + 1] tiles before each sequence
  int32_t* status;
  int split;
  float scale_log2;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A sequence's query rows and keys. Row j (of n) sits at position len + j - n and attends the keys
// up to its own; keys is 0 where there is nothing to do or the sequence is skipped (bits says why).
struct DecSeq {
  int row0, n, keys, bits;
  bool span;  // rows row0 .. row0+n-1 may be written
};
__device__ __forceinline__ DecSeq dec_seq(const PagedDecodeParams& p, int b) {
  DecSeq s;
  if (p.starts) {
    const PagedRows r = paged_rows(p.starts, p.lens, b, p.rows, p.max_new, p.c.cap, p.c.cap);
    s.row0 = r.row0;
    s.n = r.n;
    s.bits = r.bits;
    s.span = r.span;
    s.keys = r.bits || r.n == 0 ? 0 : r.len + r.n;
    return s;
  }
  const int L = __ldg(p.lens + b);
  s.row0 = b;
  s.n = 1;
  s.span = true;
  s.bits = L < 0 || static_cast<int64_t>(L) > p.c.cap                ? SLIM_DEV_BADLEN
           : static_cast<int64_t>(L) + p.extra > p.c.cap ? SLIM_DEV_OVERFLOW
                                                                     : 0;
  s.keys = s.bits ? 0 : L + p.extra;
  return s;
}

// CTA c of A owns line tiles [c·X/A, (c+1)·X/A); inside it warp w owns `chunk` tiles from w·chunk.
__device__ __forceinline__ int64_t cta_start(int64_t c, int64_t X, int64_t A) { return c * X / A; }
__device__ __forceinline__ int64_t cta_of(int64_t x, int64_t X, int64_t A) { return ((x + 1) * A - 1) / X; }
__device__ __forceinline__ int64_t active_ctas(int64_t X, int64_t grid) {
  return max(int64_t(1), min(grid, X / kDW));
}

// A stretch of tiles of one (sequence, head group).
struct DecSeg {
  int b, hg, T;      // T tiles in the whole sequence
  int tile, end;     // [tile, end)
};
// Walks the line from a starting point over `left` tiles.
struct DecCursor {
  int b, hg, tile, T;
  int64_t left;
  __device__ __forceinline__ bool next(DecSeg& s, const uint32_t* pre, int HG) {
    if (left <= 0) return false;
    s.b = b;
    s.hg = hg;
    s.T = T;
    s.tile = tile;
    const int n = static_cast<int>(min(static_cast<int64_t>(T - tile), left));
    s.end = tile + n;
    left -= n;
    tile = 0;
    if (++hg == HG && left > 0) {
      hg = 0;
      do {
        ++b;
        T = static_cast<int>(pre[b + 1] - pre[b]);
      } while (T == 0);
    }
    return true;
  }
};

template <bool E, int DH, int NT>
struct DecCfg {
  static constexpr int kRowB = DH * (E ? 1 : 2);           // bytes of a row
  static constexpr int kTileB = 16 * kRowB;                // K (or V) of a tile
  static constexpr int kTT = kTileB >= 4096 || NT == 4 ? 1 : 2;  // tiles of a stage (32 rows: registers)
  static constexpr int kStageB = 2 * kTT * kTileB;
  static constexpr int kStages = kDRing / kStageB;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPartB = kHeads * DH * 4;           // a partial's O in the ring
  static_assert(kPartB <= kDRing, "a partial fits the warp's ring");
  // byte offset of 16-byte chunk c of row r: eight rows at one chunk (an ldmatrix phase) meet eight
  // different 16-byte banks
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    return static_cast<uint32_t>(r * kRowB + ((kRowB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  }
};

template <bool E, int DH, int NT>
__global__ void __launch_bounds__(kDThreads, 1) paged_decode_kernel(const PagedDecodeParams p) {
  using C = DecCfg<E, DH, NT>;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  float* s_scale = reinterpret_cast<float*>(dec_smem + kDW * kDRing);  // [warp][stage][tile][k, v]
  float* s_ml = s_scale + kDW * C::kStages * C::kTT * 2;               // [warp][head][m, l]
  int64_t* s_seq = reinterpret_cast<int64_t*>(s_ml + kDW * C::kHeads * 2);  // [warp] sequence of its end partial, -1: none
  int* s_seg = reinterpret_cast<int*>(s_seq + kDW);                    // [warp][tile, end, T]
  uint32_t* s_pre = reinterpret_cast<uint32_t*>(s_seg + kDW * 4);      // [B + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = lane >> 2, lq = lane & 3;
  pdl_launch_dependents();
  pdl_wait_primary();

  // ---------------------------------------------------------------- this warp's share
  auto zero_rows = [&](const DecSeq& q) {
    if (!q.span) return;
    const int64_t n = static_cast<int64_t>(q.n) * p.Hq * DH / 8;
    for (int64_t i = threadIdx.x; i < n; i += kDThreads)
      reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(q.row0) * p.Hq * DH)[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  DecCursor cur;
  if (p.split) {
    if (warp == 0) {
      uint32_t carry = 0;
      int bits = 0;
      for (int base = 0; base < p.c.B; base += 32) {
        const int b = base + lane;
        uint32_t t = 0u;
        if (b < p.c.B) {
          const DecSeq q = dec_seq(p, b);
          bits |= q.bits;
          t = static_cast<uint32_t>((q.keys + 15) >> 4);
        }
        uint32_t x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (b < p.c.B) s_pre[b] = carry + x - t;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) s_pre[p.c.B] = carry;
      bits = __reduce_or_sync(0xffffffffu, bits);
      if (blockIdx.x == 0 && lane == 0 && bits) atomicOr(p.status, bits);
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= p.c.B; b += kDThreads) p.ws_pre[b] = s_pre[b];
    const int64_t X = static_cast<int64_t>(s_pre[p.c.B]) * p.HG;
    const int64_t A = active_ctas(X, gridDim.x);
    cur.left = 0;
    if (X > 0 && blockIdx.x < A) {
      const int64_t c0 = cta_start(blockIdx.x, X, A), c1 = cta_start(blockIdx.x + 1, X, A);
      const int64_t chunk = (c1 - c0 + kDW - 1) / kDW;
      const int64_t x = c0 + warp * chunk;
      cur.left = min(chunk, c1 - x);
      if (cur.left > 0) {
        int lo = 0, hi = p.c.B;  // the last b with s_pre[b]·HG <= x that has tiles
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (static_cast<int64_t>(s_pre[mid]) * p.HG <= x) lo = mid; else hi = mid;
        }
        cur.b = lo;
        cur.T = static_cast<int>(s_pre[lo + 1] - s_pre[lo]);
        const int64_t rem = x - static_cast<int64_t>(s_pre[lo]) * p.HG;
        cur.hg = static_cast<int>(rem / cur.T);
        cur.tile = static_cast<int>(rem - static_cast<int64_t>(cur.hg) * cur.T);
      }
    }
    // nothing to attend to: zero rows, dealt to the CTAs
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x)
      if (s_pre[b + 1] == s_pre[b]) zero_rows(dec_seq(p, b));
  } else {
    cur.b = blockIdx.x / p.HG;
    cur.hg = blockIdx.x - cur.b * p.HG;
    const DecSeq q = dec_seq(p, cur.b);
    cur.T = (q.keys + 15) >> 4;
    if (q.bits && cur.hg == 0 && threadIdx.x == 0) atomicOr(p.status, q.bits);
    const int chunk = (cur.T + kDW - 1) / kDW;
    cur.tile = warp * chunk;
    cur.left = min(chunk, cur.T - cur.tile);
    if (cur.T == 0 && cur.hg == 0) zero_rows(q);
  }

  uint8_t* ring = dec_smem + warp * kDRing;
  const uint32_t ring_u = smem_u32(ring);
  float* my_scale = s_scale + warp * C::kStages * C::kTT * 2;

  // ---------------------------------------------------------------- loads
  // The load side runs kStages - 1 stages ahead, across segments. Page numbers of 32 tiles at a time
  // are held one per lane.
  DecCursor ldc = cur;
  DecSeg ls;
  bool l_more = ldc.next(ls, s_pre, p.HG);
  int l_tile = l_more ? ls.tile : 0, l_win = 0, l_id = 0, l_nb = 0;
  int64_t l_head = 0;
  int l_h = 0;
  auto window = [&]() {  // page numbers of tiles l_tile .. l_tile + 31
    l_win = l_tile;
    const int t = l_tile + lane;
    l_id = t < ls.end ? __ldg(p.c.table + static_cast<int64_t>(ls.b) * p.c.max_pages +
                              ((static_cast<int64_t>(t) * 16) >> p.c.page_shift))
                      : 0;
  };
  auto seg_start = [&]() {
    l_tile = ls.tile;
    l_nb = dec_seq(p, ls.b).keys;
    l_h = ls.hg / p.NG;
    l_head = l_h * p.c.head_bytes;
    window();
  };
  if (l_more) seg_start();
  uint32_t bad_mask = 0u;  // bit stage * kTT + k: that tile's page is outside the pool; it is all zeros
  auto issue = [&](int stage) {
    if (l_more) {
      if (l_tile - l_win > 32 - C::kTT) window();
#pragma unroll
      for (int k = 0; k < C::kTT; ++k) {
        const int t = l_tile + k;
        if (t >= ls.end) break;
        int id = __shfl_sync(0xffffffffu, l_id, t - l_win);
        const bool page_bad = id < 0 || id >= p.c.num_pages;
        if (page_bad) id = 0;
        const uint32_t bit = 1u << (stage * C::kTT + k);
        bad_mask = page_bad ? bad_mask | bit : bad_mask & ~bit;
        const int64_t row = (static_cast<int64_t>(t) * 16) & ((1 << p.c.page_shift) - 1);
        const int64_t off = id * p.c.page_bytes + l_head + row * C::kRowB;
        const uint32_t dst = ring_u + stage * C::kStageB + k * 2 * C::kTileB;
        // rows of the tile that exist; the others are filled with zeros
        const int valid = page_bad ? 0 : l_nb - t * 16;
#pragma unroll
        for (int i = 0; i < C::kTileB / 512; ++i) {
          const int ch = i * 32 + lane, r = ch / (C::kRowB / 16), c = ch % (C::kRowB / 16);
          const uint32_t d = C::at(r, c), n = r < valid ? 16u : 0u;
          cp_async16(dst + d, p.c.k + off + ch * 16, n);
          cp_async16(dst + C::kTileB + d, p.c.v + off + ch * 16, n);
        }
        if (E && lane < 2) {
          const float* sc = (lane == 0 ? p.c.ks : p.c.vs) + static_cast<int64_t>(id) * p.c.Hkv + l_h;
          cp_async4(smem_u32(my_scale + (stage * C::kTT + k) * 2 + lane), sc);
        }
      }
      l_tile += C::kTT;
      if (l_tile >= ls.end) {
        l_more = ldc.next(ls, s_pre, p.HG);
        if (l_more) seg_start();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s);

  // ---------------------------------------------------------------- compute
  if (lane == 0) s_seq[warp] = -1;
  DecSeg sg;
  int stage = 0;
  while (cur.next(sg, s_pre, p.HG)) {
    const int kvh = sg.hg / p.NG, r0g = (sg.hg - kvh * p.NG) * C::kHeads;  // first row of the group
    const DecSeq sq = dec_seq(p, sg.b);
    const int nh = min(C::kHeads, sq.n * p.G - r0g);
    // row rr of the (sequence, key head) is query rr / G of the sequence and head rr % G of the key head
    auto row_of = [&](int rr, int& j) {
      j = rr / p.G;
      return (static_cast<int64_t>(sq.row0) + j) * p.Hq + static_cast<int64_t>(kvh) * p.G + (rr - j * p.G);
    };
    // the query as the B operand: head lg of each group of 8, zero past the group's heads
    uint32_t qf[NT][DH / 16][2];
    float hs[NT][2];  // score factor of heads 2 lq and 2 lq + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int hd = n * 8 + lg;
      const int rr = r0g + (hd < nh ? hd : 0), j = rr / p.G;
      const __nv_bfloat16* src = p.q + (static_cast<int64_t>(sq.row0) + j) * p.q_stride +
                                 (static_cast<int64_t>(kvh) * p.G + (rr - j * p.G)) * DH;
      if (E) {
        uint2 w[DH / 16];
        uint32_t amax = 0u;
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          w[j] = hd < nh ? __ldg(reinterpret_cast<const uint2*>(src + 16 * j + 4 * lq)) : make_uint2(0u, 0u);
          amax = max(max(amax, w[j].x & 0x7fffu), max((w[j].x >> 16) & 0x7fffu, w[j].y & 0x7fffu));
          amax = max(amax, (w[j].y >> 16) & 0x7fffu);
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = max(-126, min(126, static_cast<int>(amax >> 7) - 127));  // bf16 exponent
        const float inv = exp2_int(-e), f = exp2_int(e) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          qf[n][j][0] = pack_f16x2(bf16lo(w[j].x) * inv, bf16hi(w[j].x) * inv);
          qf[n][j][1] = pack_f16x2(bf16lo(w[j].y) * inv, bf16hi(w[j].y) * inv);
        }
        hs[n][0] = __shfl_sync(0xffffffffu, f, lq * 8);
        hs[n][1] = __shfl_sync(0xffffffffu, f, lq * 8 + 4);
      } else {
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          qf[n][j][0] = hd < nh ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * j + 2 * lq)) : 0u;
          qf[n][j][1] = hd < nh ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * j + 8 + 2 * lq)) : 0u;
        }
        hs[n][0] = hs[n][1] = p.scale_log2;
      }
    }
    float o[DH / 16][NT][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
    int bad_pos = 0x7fffffff;  // first key of the segment whose page is outside the pool
    int lim[NT][2];            // keys that rows 2 lq and 2 lq + 1 attend
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) lim[n][i] = sq.keys - sq.n + 1 + min(r0g + n * 8 + 2 * lq + i, sq.n * p.G - 1) / p.G;

    for (int t = sg.tile; t < sg.end; t += C::kTT) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();  // also: every lane is done with the stage before this one, which is filled next
#pragma unroll
      for (int k = 0; k < C::kTT; ++k)
        if (t + k < sg.end && ((bad_mask >> (stage * C::kTT + k)) & 1u)) bad_pos = min(bad_pos, (t + k) * 16);
      issue(stage == 0 ? C::kStages - 1 : stage - 1);
      const uint32_t kb = ring_u + stage * C::kStageB;
      const int tiles = min(C::kTT, sg.end - t);
      float s[C::kTT][NT][4];
#pragma unroll
      for (int k = 0; k < C::kTT; ++k) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
        if (k < tiles) {
          const uint32_t base = kb + k * 2 * C::kTileB;
          if (E) {
#pragma unroll
            for (int j = 0; j < DH / 16; j += 2) {
              uint32_t r[4];
              ldsm4(base + C::at((lane & 7) + ((lane >> 3) & 1) * 8, j + (lane >> 4)), r);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a[4] = {e4m3x2_to_f16x2(r[2 * i] & 0xffffu), e4m3x2_to_f16x2(r[2 * i + 1] & 0xffffu),
                                       e4m3x2_to_f16x2(r[2 * i] >> 16), e4m3x2_to_f16x2(r[2 * i + 1] >> 16)};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816_f16(s[k][n], a, qf[n][j + i][0], qf[n][j + i][1]);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < DH / 16; ++j) {
              uint32_t a[4];
              ldsm4(base + C::at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), a);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816_bf16(s[k][n], a, qf[n][j][0], qf[n][j][1]);
            }
          }
        }
      }
      // scores in log2 units, rows past the length masked; rows lg and lg + 8 of the tile
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
      float lv[C::kTT];
#pragma unroll
      for (int k = 0; k < C::kTT; ++k) {
        const float ks = E && k < tiles ? my_scale[(stage * C::kTT + k) * 2] : 1.f;
        lv[k] = E && k < tiles ? scale_log2(my_scale[(stage * C::kTT + k) * 2 + 1]) : 0.f;
        const int r0 = (t + k) * 16 + lg;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = E ? hs[n][i & 1] * ks : hs[n][i & 1];
            s[k][n][i] = k < tiles && r0 + (i >> 1) * 8 < lim[n][i & 1] ? s[k][n][i] * f : -INFINITY;
            mx[n][i & 1] = fmaxf(mx[n][i & 1], E ? s[k][n][i] + lv[k] : s[k][n][i]);
          }
        }
      }
      bool same = true;
      float alpha[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = mx[n][i];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
          const float mn = fmaxf(m[n][i], x);
          alpha[n][i] = mn == -INFINITY ? 1.f : ex2(m[n][i] - mn);
          m[n][i] = mn;
          l[n][i] *= alpha[n][i];
          same = same && alpha[n][i] == 1.f;
        }
      }
      if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][n][i] *= alpha[n][i & 1];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < C::kTT; ++k) {
        if (k >= tiles) break;
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mm = m[n][i] == -INFINITY ? 0.f : m[n][i];
            float add = lv[k] - mm;
            if (E) {  // weights below 2^-60 are zero in f16; raised, their fp32 sum does not underflow
              const float top = fmaxf(s[k][n][i], s[k][n][i + 2]);
              if (top != -INFINITY && add < -60.f - top) add = -60.f - top;  // a NaN scale stays
            }
            e[i] = ex2(s[k][n][i] + add);
            e[i + 2] = ex2(s[k][n][i + 2] + add);
            l[n][i] += E ? (e[i] + e[i + 2]) * ex2(-mm - add) : e[i] + e[i + 2];
          }
          if (E) {
            ph[n][0] = movmatrix(pack_f16x2(e[0], e[1]));
            ph[n][1] = movmatrix(pack_f16x2(e[2], e[3]));
          } else {
            const uint32_t h0 = pack_bf16x2(e[0], e[1]), h1 = pack_bf16x2(e[2], e[3]);
            ph[n][0] = movmatrix(h0);
            ph[n][1] = movmatrix(h1);
            pl[n][0] = movmatrix(pack_bf16x2(e[0] - bf16lo(h0), e[1] - bf16hi(h0)));
            pl[n][1] = movmatrix(pack_bf16x2(e[2] - bf16lo(h1), e[3] - bf16hi(h1)));
          }
        }
        const uint32_t base = kb + k * 2 * C::kTileB + C::kTileB;
        if (E) {
          // a 16-bit unit of the transposed load is two columns: rows lg of the operand are the even
          // ones, rows lg + 8 the odd ones
#pragma unroll
          for (int j = 0; j < DH / 16; j += 2) {
            uint32_t r[4];
            ldsm4_trans(base + C::at((lane & 7) + ((lane >> 3) & 1) * 8, j + (lane >> 4)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = __byte_perm(r[2 * i], 0u, 0x3120), y = __byte_perm(r[2 * i + 1], 0u, 0x3120);
              const uint32_t a[4] = {e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(x >> 16),
                                     e4m3x2_to_f16x2(y & 0xffffu), e4m3x2_to_f16x2(y >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816_f16(o[j + i][n], a, ph[n][0], ph[n][1]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            uint32_t a[4];
            ldsm4_trans(base + C::at((lane & 7) + (lane >> 4) * 8, 2 * c + ((lane >> 3) & 1)), a);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_16816_bf16(o[c][n], a, ph[n][0], ph[n][1]);
              mma_16816_bf16(o[c][n], a, pl[n][0], pl[n][1]);
            }
          }
        }
      }
      stage = stage == C::kStages - 1 ? 0 : stage + 1;
    }

    // ---------------------------------------------------------------- end of a segment
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], sh);
        if (bad_pos < lim[n][i]) l[n][i] = -1.f;
      }
    if (bad_pos != 0x7fffffff && lane == 0) atomicOr(p.status, SLIM_DEV_BADPAGE);
    const bool whole = sg.tile == 0 && sg.end == sg.T;
    const bool last = cur.left <= 0;
    if (whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hd = n * 8 + 2 * lq + (i & 1);
          if (hd >= nh) continue;
          const float f = l[n][i & 1] > 0.f || l[n][i & 1] != l[n][i & 1] ? 1.f / l[n][i & 1] : 0.f;
          int j;
          __nv_bfloat16* dst = p.out + row_of(r0g + hd, j) * DH;
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            const int col = 16 * c + (E ? 2 * lg + (i >> 1) : lg + (i >> 1) * 8);
            dst[col] = __float2bfloat16_rn(l[n][i & 1] < 0.f ? 0.f : o[c][n][i] * f);
          }
        }
    } else {
      // a partial: in the ring where it is the warp's last segment (every load has landed by then),
      // else in the workspace
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * kDSlots + kDW + warp;
      if (last) {
        cp_async_wait<0>();
        __syncwarp();
      }
      float* po = last ? reinterpret_cast<float*>(ring) : p.ws_o + slot * C::kHeads * DH;
      float* pm = last ? s_ml + warp * C::kHeads * 2 : p.ws_ml + slot * C::kHeads * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hd = n * 8 + 2 * lq + (i & 1);
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            const int col = 16 * c + (E ? 2 * lg + (i >> 1) : lg + (i >> 1) * 8);
            po[hd * DH + col] = o[c][n][i];
          }
          if (lg == 0 && i < 2) {
            pm[hd * 2] = m[n][i];
            pm[hd * 2 + 1] = l[n][i];
          }
        }
      if (last && lane == 0) {
        s_seq[warp] = static_cast<int64_t>(sg.b) * p.HG + sg.hg;
        s_seg[warp * 4] = sg.tile;
        s_seg[warp * 4 + 1] = sg.end;
        s_seg[warp * 4 + 2] = sg.T;
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---------------------------------------------------------------- joining the warps' last partials
  for (int w0 = 0; w0 < kDW;) {
    const int64_t seq = s_seq[w0];
    int w1 = w0 + 1;
    if (seq < 0) {
      w0 = w1;
      continue;
    }
    while (w1 < kDW && s_seq[w1] == seq) ++w1;
    const bool whole = s_seg[w0 * 4] == 0 && s_seg[(w1 - 1) * 4 + 1] == s_seg[w0 * 4 + 2];
    const int b = static_cast<int>(seq / p.HG), hg = static_cast<int>(seq - static_cast<int64_t>(b) * p.HG);
    const int kvh = hg / p.NG, r0g = (hg - kvh * p.NG) * C::kHeads;
    const DecSeq sq = dec_seq(p, b);
    const int nh = min(C::kHeads, sq.n * p.G - r0g);
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * kDSlots + w0;
    for (int i = threadIdx.x; i < nh * DH; i += kDThreads) {
      const int hd = i / DH;
      float M = -INFINITY, L = 0.f, O = 0.f;
      bool broken = false;
      for (int w = w0; w < w1; ++w) M = fmaxf(M, s_ml[(w * C::kHeads + hd) * 2]);
      const float Mf = M == -INFINITY ? 0.f : M;
      for (int w = w0; w < w1; ++w) {
        const float f = ex2(s_ml[(w * C::kHeads + hd) * 2] - Mf), lw = s_ml[(w * C::kHeads + hd) * 2 + 1];
        broken |= lw < 0.f;
        L = fmaf(f, lw, L);
        O = fmaf(f, reinterpret_cast<const float*>(dec_smem + w * kDRing)[i], O);
      }
      if (whole) {
        const int rr = r0g + hd, j = rr / p.G;
        p.out[((static_cast<int64_t>(sq.row0) + j) * p.Hq + static_cast<int64_t>(kvh) * p.G + (rr - j * p.G)) * DH +
              i % DH] = __float2bfloat16_rn(broken || L == 0.f ? 0.f : O / L);
      } else {
        p.ws_o[slot * C::kHeads * DH + i] = O;
        if (i % DH == 0) {
          p.ws_ml[(slot * C::kHeads + hd) * 2] = M;
          p.ws_ml[(slot * C::kHeads + hd) * 2 + 1] = broken ? -1.f : L;
        }
      }
    }
    w0 = w1;
  }
}

// Joins the partials of one (sequence, head group) that more than one CTA (or a CTA's join and a
// warp in whose share it ends) holds. Which slots those are follows from the plan alone.
template <int DH, int NT>
__global__ void __launch_bounds__(256) merge_paged_kernel(const PagedDecodeParams p, int64_t grid) {
  constexpr int kHeads = 8 * NT;
  __shared__ int64_t s_range[4];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.x / p.HG, hg = blockIdx.x - b * p.HG;
  if (threadIdx.x == 0) {
    const int64_t q0 = __ldcg(p.ws_pre + b), q1 = __ldcg(p.ws_pre + b + 1);
    const int64_t X = static_cast<int64_t>(__ldcg(p.ws_pre + p.c.B)) * p.HG;
    const int64_t T = q1 - q0, x0 = q0 * p.HG + hg * T, x1 = x0 + T;
    s_range[0] = 0;
    s_range[1] = -1;
    s_range[2] = 0;
    s_range[3] = -1;
    if (T > 0) {
      const int64_t A = active_ctas(X, grid);
      const int64_t c0 = cta_of(x0, X, A), c1 = cta_of(x1 - 1, X, A);
      auto chunk_of = [&](int64_t c) {
        return (cta_start(c + 1, X, A) - cta_start(c, X, A) + kDW - 1) / kDW;
      };
      const int64_t s0 = cta_start(c0, X, A), s1 = cta_start(c1, X, A), e1 = cta_start(c1 + 1, X, A);
      const int64_t w0 = (x0 - s0) / chunk_of(c0), w1 = (x1 - 1 - s1) / chunk_of(c1);
      const int64_t end_w1 = min(s1 + (w1 + 1) * chunk_of(c1), e1);
      const bool inside = x1 < end_w1;                       // it ends inside the share of warp w1 ..
      const bool own = inside && !(c0 == c1 && w0 == w1);    // .. with a slot of its own there
      const int64_t first_w_last = c0 == c1 ? w0 : 0;        // first warp of the sequence in CTA c1
      const bool joined_last = !inside || w1 > first_w_last; // CTA c1 also has a joined slot
      // joined slots: (c0, w0), (c, 0) for the CTAs between, and c1's where there is one
      s_range[0] = c0;
      s_range[1] = joined_last ? c1 : c1 - 1;
      s_range[2] = w0;
      s_range[3] = own ? c1 * kDSlots + kDW + w1 : -1;
      if (c0 == c1 && !own) s_range[1] = c0 - 1;  // written whole by its CTA or warp
    }
  }
  __syncthreads();
  const int64_t c0 = s_range[0], c1 = s_range[1], w0 = s_range[2], own = s_range[3];
  const int n = static_cast<int>(c1 - c0 + 1), total = n + (own >= 0 ? 1 : 0);
  if (total == 0) return;
  auto slot = [&](int i) { return i == n ? own : (c0 + i) * kDSlots + (i == 0 ? w0 : 0); };
  const int kvh = hg / p.NG, r0g = (hg - kvh * p.NG) * kHeads;
  const DecSeq sq = dec_seq(p, b);
  const int nh = min(kHeads, sq.n * p.G - r0g);
  for (int i = threadIdx.x; i < nh * DH / 4; i += 256) {
    const int hd = i / (DH / 4);
    float M = -INFINITY;
    bool broken = false;
#pragma unroll 4
    for (int k = 0; k < total; ++k) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot(k) * kHeads + hd);
      M = fmaxf(M, ml.x);
      broken |= ml.y < 0.f;
    }
    const float Mf = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < total; ++k) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot(k) * kHeads + hd);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot(k) * kHeads * DH) + i);
      const float f = ex2(ml.x - Mf);
      L = fmaf(f, ml.y, L);
      O.x = fmaf(f, v.x, O.x);
      O.y = fmaf(f, v.y, O.y);
      O.z = fmaf(f, v.z, O.z);
      O.w = fmaf(f, v.w, O.w);
    }
    const float r = broken || L == 0.f ? 0.f : 1.f / L;
    const uint2 y = broken ? make_uint2(0u, 0u)
                           : make_uint2(pack_bf16x2(O.x * r, O.y * r), pack_bf16x2(O.z * r, O.w * r));
    const int rr = r0g + hd, j = rr / p.G;
    reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(sq.row0) + j) * p.Hq + static_cast<int64_t>(kvh) * p.G +
                                      (rr - j * p.G)) * DH)[i - hd * (DH / 4)] = y;
  }
}

struct DecPlan {
  int NT, NG, HG;
  size_t o_bytes, ml_bytes, pre_bytes;
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
// R query rows at most share a (sequence, key head)'s keys.
DecPlan dec_plan(const slim_paged_cache& c, int R) {
  DecPlan d;
  d.NT = R <= 8 ? 1 : R <= 16 ? 2 : 4;
  d.NG = (R + 8 * d.NT - 1) / (8 * d.NT);
  d.HG = c.Hkv * d.NG;
  const size_t slots = static_cast<size_t>(num_sms()) * kDSlots;
  d.o_bytes = up256(slots * 8 * d.NT * c.dh * 4);
  d.ml_bytes = up256(slots * 8 * d.NT * 2 * 4);
  d.pre_bytes = up256((static_cast<size_t>(c.B) + 1) * 4);
  return d;
}

template <bool E, int DH, int NT>
uint32_t dec_smem_bytes(int B, bool split) {
  using C = DecCfg<E, DH, NT>;
  return static_cast<uint32_t>(kDW * kDRing + kDW * C::kStages * C::kTT * 2 * 4 + kDW * C::kHeads * 2 * 4 + kDW * 8 +
                               kDW * 16 + (split ? (B + 1) * 4 : 0));
}

template <bool E, int DH, int NT>
cudaError_t launch_dec(const PagedDecodeParams& p, cudaStream_t st, int* launches) {
  const uint32_t smem = dec_smem_bytes<E, DH, NT>(p.c.B, p.split != 0);
  auto kern = paged_decode_kernel<E, DH, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = p.split ? num_sms() : p.c.B * p.HG;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kDThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  if (launches) ++*launches;
  if (!p.split) return cudaSuccess;
  cudaLaunchConfig_t cfg2 = {};
  cfg2.gridDim = dim3(static_cast<unsigned>(p.c.B * p.HG), 1, 1);
  cfg2.blockDim = dim3(256, 1, 1);
  cfg2.stream = st;
  cfg2.attrs = attr;
  cfg2.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg2, merge_paged_kernel<DH, NT>, p, static_cast<int64_t>(grid));
  if (e == cudaSuccess && launches) ++*launches;
  return e;
}

}  // namespace

size_t paged_rows_ws_bytes(const slim_paged_cache& c, int R) {
  const DecPlan d = dec_plan(c, R);
  return d.o_bytes + d.ml_bytes + d.pre_bytes;
}

template <bool E, int DH>
static cudaError_t launch_dec_nt(const PagedDecodeParams& p, int NT, cudaStream_t st, int* launches) {
  return NT == 1   ? launch_dec<E, DH, 1>(p, st, launches)
         : NT == 2 ? launch_dec<E, DH, 2>(p, st, launches)
                   : launch_dec<E, DH, 4>(p, st, launches);
}

// starts == nullptr: one row per sequence, attending lens[b] + rows_extra keys; else the packed rows,
// at most max_new of a sequence, each attending the keys up to its own.
cudaError_t launch_paged_rows(const slim_paged_cache& c, const void* q, int64_t q_stride, const int32_t* starts,
                              const int32_t* lens, int64_t rows, int64_t max_new, int rows_extra, int Hq,
                              int64_t t_hint, void* out, void* workspace, int32_t* status, cudaStream_t st,
                              int* launches) {
  const int G = Hq / c.Hkv;
  const DecPlan d = dec_plan(c, starts ? static_cast<int>(max_new) * G : G);
  PagedDecodeParams p;
  p.c = paged_view(c);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.lens = lens;
  p.starts = starts;
  p.rows = rows;
  p.max_new = max_new;
  p.extra = rows_extra;
  p.Hq = Hq;
  p.G = G;
  p.NG = d.NG;
  p.HG = d.HG;
  p.out = static_cast<__nv_bfloat16*>(out);
  char* w = static_cast<char*>(workspace);
  p.ws_o = reinterpret_cast<float*>(w);
  p.ws_ml = reinterpret_cast<float*>(w + d.o_bytes);
  p.ws_pre = reinterpret_cast<uint32_t*>(w + d.o_bytes + d.ml_bytes);
  p.status = status;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(c.dh));
  const int64_t hint = t_hint > 0 ? std::min(t_hint, p.c.cap) : p.c.cap;
  // one CTA per work sequence, no merge, where that is one wave and a warp's share stays short
  p.split = !(static_cast<int64_t>(c.B) * d.HG <= num_sms() && hint <= 1024);
  if (c.dtype == SLIM_E4M3)
    return c.dh == 64 ? launch_dec_nt<true, 64>(p, d.NT, st, launches) : launch_dec_nt<true, 128>(p, d.NT, st, launches);
  return c.dh == 64 ? launch_dec_nt<false, 64>(p, d.NT, st, launches) : launch_dec_nt<false, 128>(p, d.NT, st, launches);
}

}  // namespace slim
