// Attention of a few query rows per sequence over a paged K+V cache in bf16 or
// e4m3: slim_mha_paged_decode (one row), and slim_mha_paged_prefill where the
// rows that share a key head are at most 16, 32 at dh = 64 (a few proposed tokens).
//
// Mathematics, per sequence and key/value head, for the G query heads that
// share it: s_t = q·K_t·log2(e)/sqrt(dh), m = max s, p_t = 2^(s_t - m),
// o = Σ p_t V_t / Σ p_t, kept as a running (m, l, o) per warp and joined by
// 2^(m_i - m). In e4m3 K_t = ks·k8_t and V_t = 2^lv·v8_t with scales of the page
// and head: ks multiplies the score, and the weights of the sum over v8 are
// P_t = 2^(s_t + lv - m + kWeightLog2) with m the running maximum of s + lv, which keeps
// them in f16's range whatever the pages' scales are; l adds P_t·2^-(lv + kWeightLog2).
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
// in equal shares for the CTAs and, inside, for their warps; a warp streams its
// tiles through its own ring in shared memory (cp.async, no barrier with other
// warps): 192 KB of rings per SM. All stages but the one being worked on are in flight: two thirds of
// the ring or more, but half with 8 rows over e4m3 at dh = 128 (12 warps, two stages each). Partials of
// warps that end in one sequence are joined in the CTA; what a sequence has in
// other CTAs is joined by merge_paged_kernel. Small calls take one CTA per
// (sequence, head group) instead and need no merge.
#include <algorithm>

#include "paged.cuh"

namespace slim {

namespace {

constexpr int kDRings = 192 * 1024;    // bytes of a CTA's rings
constexpr int kDMergeScan = 256;       // sequences up to which the merge kernel takes the line's offsets from lens
constexpr int kDWide = 3;              // CTAs per (sequence, head group) from which the wide merge is taken
constexpr float kDLazyLog2 = 8.f;      // a row's maximum follows once a score exceeds it by this much

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
  float* ws_o;     // [ctas][kSlots][rows][dh]
  float* ws_ml;    // [ctas][kSlots][rows][2]
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
  const int L = ld_plain(p.lens + b);
  s.row0 = b;
  s.n = 1;
  s.span = true;
  s.bits = 0;
  if (L < 0 || static_cast<int64_t>(L) > p.c.cap)
    s.bits = SLIM_DEV_BADLEN;
  else if (static_cast<int64_t>(L) + p.extra > p.c.cap)
    s.bits = SLIM_DEV_OVERFLOW;
  s.keys = s.bits ? 0 : L + p.extra;
  return s;
}

// Warps of a CTA, each with its part of the rings. Over e4m3 the work is bound by instructions, so more
// warps hide more: 64 sequences of 1000 to 1500 rows, 20 heads of 64: 8 warps 71, 12 61, 16 58 us; 16K to 32K
// rows, heads of 128: 12 warps 137, 16 (registers spill) 141 us. bf16 streams at memory speed with 8. More
// rows need the registers.
__host__ __device__ constexpr int dec_warps(bool e4m3, int dh, int NT) {
  return NT > 1 || !e4m3 ? 8 : dh == 64 ? 16 : 12;
}

// The line has X tiles. CTA c of A owns [c·X/A, (c+1)·X/A), its warp w `chunk` tiles from w·chunk on.
// I is int where c·X fits (64-bit divisions took 0.5 us of a call), int64_t else.
template <typename I>
__device__ __forceinline__ I active_ctas(I X, I grid, int warps) {
  return max(I(1), min(grid, X / warps));
}
template <typename I, int W>
__device__ __forceinline__ void warp_share(I X, I grid, int cta, int warp, I& x, int& left) {
  const I A = active_ctas<I>(X, grid, W);
  x = 0;
  left = 0;
  if (cta >= A) return;
  const I c0 = cta * X / A, c1 = (cta + 1) * X / A, chunk = (c1 - c0 + W - 1) / W;
  x = c0 + warp * chunk;
  left = static_cast<int>(min(chunk, c1 - x));
}
__device__ __forceinline__ bool line_fits_int(int64_t X, int grid) { return X < ((int64_t(1) << 31) - 1) / (grid + 1); }

// A stretch of tiles of one (sequence, head group).
struct DecSeg {
  int b, hg, T;      // T tiles in the whole sequence
  int tile, end;     // [tile, end)
};
// A warp's partial at the end of its share: its stretch, and the sequence's query rows.
struct DecEnd {
  DecSeg s;
  int row0, n;
};
// Walks the line from a starting point over `left` tiles.
struct DecCursor {
  int b, hg, tile, T, left;
  __device__ __forceinline__ bool next(DecSeg& s, const uint32_t* pre, int HG) {
    if (left <= 0) return false;
    s.b = b;
    s.hg = hg;
    s.T = T;
    s.tile = tile;
    const int n = min(T - tile, left);
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
  static constexpr int kWarps = dec_warps(E, DH, NT);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRing = kDRings / kWarps;           // bytes of a warp's ring
  // partials a CTA can leave: of its warps' ends, and of sequences that end inside a warp's share
  static constexpr int kSlots = 2 * kWarps;
  static constexpr int kRowB = DH * (E ? 1 : 2);           // bytes of a row
  static constexpr int kTileB = 16 * kRowB;                // K (or V) of a tile
  static constexpr int kTT = kTileB >= 4096 || NT == 4 ? 1 : 2;  // tiles of a stage (32 rows: registers)
  static constexpr int kStageB = 2 * kTT * kTileB;
  static constexpr int kStages = kRing / kStageB;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPartB = kHeads * DH * 4;           // a partial's O in the ring
  static_assert(kPartB <= kRing, "a partial fits the warp's ring");
  // byte offset of 16-byte chunk c of row r: eight rows at one chunk (an ldmatrix phase) meet eight
  // different 16-byte banks
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    return static_cast<uint32_t>(r * kRowB + ((kRowB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  }
};

template <bool E, int DH, int NT>
__global__ void __launch_bounds__(DecCfg<E, DH, NT>::kThreads, 1) paged_decode_kernel(const PagedDecodeParams p) {
  using C = DecCfg<E, DH, NT>;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  float* s_scale = reinterpret_cast<float*>(dec_smem + C::kWarps * C::kRing);  // [warp][stage][tile][k, v]
  float* s_ml = s_scale + C::kWarps * C::kStages * C::kTT * 2;               // [warp][head][m, l]
  DecEnd* s_end = reinterpret_cast<DecEnd*>(s_ml + C::kWarps * C::kHeads * 2);  // [warp] its end partial, b = -1: none
  uint32_t* s_pre = reinterpret_cast<uint32_t*>(s_end + C::kWarps);             // [B + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = lane >> 2, lq = lane & 3;
  // the merge kernel may start once every CTA is past this wait: what came before is complete then,
  // so that it may read lens and starts at once
  pdl_wait_primary();
  pdl_launch_dependents();

  // ---------------------------------------------------------------- this warp's share
  auto zero_rows = [&](const DecSeq& q) {
    if (!q.span) return;
    const int64_t n = static_cast<int64_t>(q.n) * p.Hq * DH / 8;
    for (int64_t i = threadIdx.x; i < n; i += C::kThreads)
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
    if (blockIdx.x == 0 && p.c.B > kDMergeScan)
      for (int b = threadIdx.x; b <= p.c.B; b += C::kThreads) p.ws_pre[b] = s_pre[b];
    const int64_t X = static_cast<int64_t>(s_pre[p.c.B]) * p.HG;
    const int grid = static_cast<int>(gridDim.x);
    cur.left = 0;
    if (X > 0) {
      int64_t x;
      if (line_fits_int(X, grid)) {
        int xi;
        warp_share<int, C::kWarps>(static_cast<int>(X), grid, blockIdx.x, warp, xi, cur.left);
        x = xi;
      } else {
        warp_share<int64_t, C::kWarps>(X, grid, blockIdx.x, warp, x, cur.left);
      }
      if (cur.left > 0) {
        int lo = 0, hi = p.c.B;  // the last b with s_pre[b]·HG <= x: it has tiles
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (static_cast<int64_t>(s_pre[mid]) * p.HG <= x) lo = mid; else hi = mid;
        }
        cur.b = lo;
        cur.T = static_cast<int>(s_pre[lo + 1] - s_pre[lo]);
        const int64_t rem = x - static_cast<int64_t>(s_pre[lo]) * p.HG;
        cur.hg = rem < (int64_t(1) << 31) ? static_cast<int>(rem) / cur.T : static_cast<int>(rem / cur.T);
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
    const int chunk = (cur.T + C::kWarps - 1) / C::kWarps;
    cur.tile = warp * chunk;
    cur.left = min(chunk, cur.T - cur.tile);
    if (cur.T == 0 && cur.hg == 0) zero_rows(q);
  }

  uint8_t* ring = dec_smem + warp * C::kRing;
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
    l_id = t < ls.end ? ld_plain(p.c.table + static_cast<int64_t>(ls.b) * p.c.max_pages +
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
  if (lane == 0) s_end[warp].s.b = -1;
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
          w[j] = hd < nh ? ld_plain(reinterpret_cast<const uint2*>(src + 16 * j + 4 * lq)) : make_uint2(0u, 0u);
          amax = max(max(amax, w[j].x & 0x7fffu), max((w[j].x >> 16) & 0x7fffu, w[j].y & 0x7fffu));
          amax = max(amax, (w[j].y >> 16) & 0x7fffu);
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = max(-126, min(126, static_cast<int>(amax >> 7) - 127));  // bf16 exponent
        const float inv = exp2_int(-e), f = exp2_int(e) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          qf[n][j][0] = round_f16x2(bf16lo(w[j].x) * inv, bf16hi(w[j].x) * inv);
          qf[n][j][1] = round_f16x2(bf16lo(w[j].y) * inv, bf16hi(w[j].y) * inv);
        }
        hs[n][0] = __shfl_sync(0xffffffffu, f, lq * 8);
        hs[n][1] = __shfl_sync(0xffffffffu, f, lq * 8 + 4);
      } else {
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          qf[n][j][0] = hd < nh ? ld_plain(reinterpret_cast<const uint32_t*>(src + 16 * j + 2 * lq)) : 0u;
          qf[n][j][1] = hd < nh ? ld_plain(reinterpret_cast<const uint32_t*>(src + 16 * j + 8 + 2 * lq)) : 0u;
        }
        hs[n][0] = hs[n][1] = p.scale_log2;
      }
    }
    float o[DH / 16][NT][4] = {};
    float m[NT][2], neg_m[NT][2], l[NT][2];  // neg_m: -m (e4m3: kWeightLog2 - m), 0 while there is none
#pragma unroll
    for (int n = 0; n < NT; ++n)
      m[n][0] = m[n][1] = -INFINITY, neg_m[n][0] = neg_m[n][1] = 0.f, l[n][0] = l[n][1] = 0.f;
    int bad_pos = 0x7fffffff;  // first key of the segment whose page is outside the pool
    int lim[NT][2];            // keys that rows 2 lq and 2 lq + 1 attend
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) lim[n][i] = sq.keys - sq.n + 1 + min(r0g + n * 8 + 2 * lq + i, sq.n * p.G - 1) / p.G;

    const int lim_all = sq.keys - sq.n + 1 + r0g / p.G;  // keys that every row of the group attends

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
                uint32_t a[4];
                e4m3x4_to_f16(r[2 * i], a[0], a[2]);
                e4m3x4_to_f16(r[2 * i + 1], a[1], a[3]);
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
      // Exponent of a weight: s·f + add, f the factor to log2 units, add = lv + neg_m. Tiles that some row
      // does not attend whole (the last ones) are scaled and masked here, with f = 1 from then on.
      float f[C::kTT][NT][2], lv[C::kTT], fac[C::kTT];
      const bool full = (t + C::kTT) * 16 <= lim_all && tiles == C::kTT;
#pragma unroll
      for (int k = 0; k < C::kTT; ++k) {
        const float ks = E && k < tiles ? my_scale[(stage * C::kTT + k) * 2] : 1.f;
        lv[k] = E && k < tiles ? scale_log2(my_scale[(stage * C::kTT + k) * 2 + 1]) : 0.f;
        fac[k] = E ? ex2(-lv[k]) * kWeightInv : 1.f;  // subnormal for the largest scale: exact
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) f[k][n][i] = E ? hs[n][i] * ks : hs[n][i];
      }
      if (!full) {
#pragma unroll
        for (int k = 0; k < C::kTT; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[k][n][i] = k < tiles && (t + k) * 16 + lg + (i >> 1) * 8 < lim[n][i & 1] ? s[k][n][i] * f[k][n][i & 1]
                                                                                        : -INFINITY;
            f[k][n][0] = f[k][n][1] = 1.f;
          }
      }
      // A lane looks at its own scores only; the warp's maximum is taken when one of them exceeds the
      // row's by more than 2^8 (weights up to that fit f16, with 2^kWeightLog2, and bf16).
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[n][i] = -INFINITY;
#pragma unroll
          for (int k = 0; k < C::kTT; ++k)
            mx[n][i] = fmaxf(mx[n][i], fmaf(fmaxf(s[k][n][i], s[k][n][i + 2]), f[k][n][i], lv[k]));
          grow = grow || mx[n][i] > m[n][i] + kDLazyLog2;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = mx[n][i];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
            const float mn = fmaxf(m[n][i], x);
            const float alpha = mn == -INFINITY ? 1.f : ex2(m[n][i] - mn);
            m[n][i] = mn;
            neg_m[n][i] = mn == -INFINITY ? 0.f : E ? kWeightLog2 - mn : -mn;
            l[n][i] *= alpha;
#pragma unroll
            for (int c = 0; c < DH / 16; ++c) {
              o[c][n][i] *= alpha;
              o[c][n][i + 2] *= alpha;
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
          bool low = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float add = lv[k] + neg_m[n][i];
            float x0 = fmaf(s[k][n][i], f[k][n][i], add), x1 = fmaf(s[k][n][i + 2], f[k][n][i], add);
            if (E && !full) {  // a masked weight is zero also beside a NaN scale
              if (s[k][n][i] == -INFINITY) x0 = -INFINITY;
              if (s[k][n][i + 2] == -INFINITY) x1 = -INFINITY;
            }
            e[i] = ex2(x0);
            e[i + 2] = ex2(x1);
            if (!E) l[n][i] += e[i] + e[i + 2];
            if (E) low = low || fminf(x0, x1) < -60.f;
          }
          if (E) {
            // the sum of p itself is that of P·2^-lv/2^kWeightLog2; taken from the scores where P may have underflowed
            if (__any_sync(0xffffffffu, low)) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float z = fac[k] != fac[k] ? fac[k] : 0.f;  // a NaN scale stays
                l[n][i] += (ex2(fmaf(s[k][n][i], f[k][n][i], neg_m[n][i])) +
                            ex2(fmaf(s[k][n][i + 2], f[k][n][i], neg_m[n][i]))) * kWeightInv +
                           (e[i] != 0.f ? e[i] * z : 0.f) + (e[i + 2] != 0.f ? e[i + 2] * z : 0.f);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) l[n][i] = fmaf(e[i] + e[i + 2], fac[k], l[n][i]);
            }
            ph[n][0] = movmatrix(round_f16x2(e[0], e[1]));
            ph[n][1] = movmatrix(round_f16x2(e[2], e[3]));
          } else {
            const uint32_t h0 = round_bf16x2(e[0], e[1]), h1 = round_bf16x2(e[2], e[3]);
            ph[n][0] = movmatrix(h0);
            ph[n][1] = movmatrix(h1);
            pl[n][0] = movmatrix(round_bf16x2(e[0] - bf16lo(h0), e[1] - bf16hi(h0)));
            pl[n][1] = movmatrix(round_bf16x2(e[2] - bf16lo(h1), e[3] - bf16hi(h1)));
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
              uint32_t a[4];
              e4m3x4_to_f16(__byte_perm(r[2 * i], 0u, 0x3120), a[0], a[1]);
              e4m3x4_to_f16(__byte_perm(r[2 * i + 1], 0u, 0x3120), a[2], a[3]);
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
          const float f = l[n][i & 1] > 0.f || l[n][i & 1] != l[n][i & 1] ? (E ? kWeightInv : 1.f) / l[n][i & 1] : 0.f;
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
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * C::kSlots + C::kWarps + warp;
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
            po[hd * DH + col] = E ? o[c][n][i] * kWeightInv : o[c][n][i];
          }
          if (lg == 0 && i < 2) {
            pm[hd * 2] = m[n][i];
            pm[hd * 2 + 1] = l[n][i];
          }
        }
      if (last && lane == 0) s_end[warp] = DecEnd{sg, sq.row0, sq.n};
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---------------------------------------------------------------- joining the warps' last partials
  // The warps [w0, w1) that end in one sequence share its rows; every group is joined at once.
  const int b = s_end[warp].s.b, hg = s_end[warp].s.hg;
  if (b < 0) return;
  auto same = [&](int w) { return s_end[w].s.b == b && s_end[w].s.hg == hg; };
  int w0 = warp, w1 = warp + 1;
  while (w0 > 0 && same(w0 - 1)) --w0;
  while (w1 < C::kWarps && same(w1)) ++w1;
  const bool whole = s_end[w0].s.tile == 0 && s_end[w1 - 1].s.end == s_end[w0].s.T;
  const int row0 = s_end[warp].row0;
  const int kvh = hg / p.NG, r0g = (hg - kvh * p.NG) * C::kHeads;
  const int nh = min(C::kHeads, s_end[warp].n * p.G - r0g);
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * C::kSlots + w0;
  for (int hd = warp - w0; hd < nh; hd += w1 - w0) {
    float M = -INFINITY, L = 0.f;
    bool broken = false;
    for (int w = w0; w < w1; ++w) M = fmaxf(M, s_ml[(w * C::kHeads + hd) * 2]);
    const float Mf = M == -INFINITY ? 0.f : M;
    constexpr int PL = DH / 32;  // columns of a lane
    float O[PL] = {};
    for (int w = w0; w < w1; ++w) {
      const float f = ex2(s_ml[(w * C::kHeads + hd) * 2] - Mf), lw = s_ml[(w * C::kHeads + hd) * 2 + 1];
      broken |= lw < 0.f;
      L = fmaf(f, lw, L);
      const float* src = reinterpret_cast<const float*>(dec_smem + w * C::kRing) + hd * DH + lane * PL;
#pragma unroll
      for (int k = 0; k < PL; ++k) O[k] = fmaf(f, src[k], O[k]);
    }
    if (whole) {
      const int rr = r0g + hd, j = rr / p.G;
      const float r = broken || L == 0.f ? 0.f : 1.f / L;
      uint32_t* dst = reinterpret_cast<uint32_t*>(
          p.out + ((static_cast<int64_t>(row0) + j) * p.Hq + static_cast<int64_t>(kvh) * p.G + (rr - j * p.G)) * DH +
          lane * PL);
#pragma unroll
      for (int k = 0; k < PL; k += 2) dst[k / 2] = broken ? 0u : round_bf16x2(O[k] * r, O[k + 1] * r);
    } else {
      float* dst = p.ws_o + (slot * C::kHeads + hd) * DH + lane * PL;
#pragma unroll
      for (int k = 0; k < PL; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(O[k], O[k + 1]);
      if (lane == 0) {
        p.ws_ml[(slot * C::kHeads + hd) * 2] = M;
        p.ws_ml[(slot * C::kHeads + hd) * 2 + 1] = broken ? -1.f : L;
      }
    }
  }
}

// Slots that hold the partials of line stretch [x0, x1): joined ones of CTAs c0 .. c0+n-1 (of warp w0 in
// the first, of warp 0 in the others), then `own`, a warp's, or -1. None: written whole by the split kernel.
struct DecSlots {
  int c0, n, w0, own;
};
template <typename I, int W>
__device__ __forceinline__ DecSlots dec_slots(I x0, I x1, I X, I grid) {
  const I A = active_ctas<I>(X, grid, W);
  auto start = [&](I c) { return c * X / A; };
  const I c0 = ((x0 + 1) * A - 1) / X, c1 = (x1 * A - 1) / X;
  const I s0 = start(c0), e0 = start(c0 + 1), s1 = c1 == c0 ? s0 : start(c1), e1 = c1 == c0 ? e0 : start(c1 + 1);
  const I k0 = (e0 - s0 + W - 1) / W, k1 = c1 == c0 ? k0 : (e1 - s1 + W - 1) / W;  // tiles of a warp
  const I w0 = (x0 - s0) / k0, w1 = (x1 - 1 - s1) / k1;
  const bool inside = x1 < min(s1 + (w1 + 1) * k1, e1);   // it ends inside the share of warp w1 ..
  const bool own = inside && !(c0 == c1 && w0 == w1);     // .. with a slot of its own there
  const bool joined = !inside || w1 > (c0 == c1 ? w0 : I(0));  // CTA c1 has a joined slot
  DecSlots s;
  s.c0 = static_cast<int>(c0);
  s.w0 = static_cast<int>(w0);
  s.own = own ? static_cast<int>(c1) * 2 * W + W + static_cast<int>(w1) : -1;
  s.n = c0 == c1 && !own ? 0 : static_cast<int>(c1 - c0) + (joined ? 1 : 0);
  return s;
}

// Joins the partials of one (sequence, head group) that more than one CTA (or a CTA's join and a
// warp in whose share it ends) holds. Which slots those are follows from the plan alone; the loads of
// a slot's maximum, sum and output go out together.
//
// kWide: a CTA takes one row and its threads are 1024 / DH groups, each with a share of the slots, for calls
// with many slots of few sequences. Whole decode calls without and with it, bf16, T = 16384, dh = 128: one
// sequence of one key head and 8 query heads (148 CTAs each) 42 and 15 us, one of 8 key heads (18) 25 and 21;
// 4 of 8000 rows (4.6) 31 and 30, 9 of 4000 (2) 32.3 and 32.5.
template <int DH, int NT, int W, bool kWide>
__global__ void __launch_bounds__(256) merge_paged_kernel(const PagedDecodeParams p, int grid) {
  constexpr int kHeads = 8 * NT;
  pdl_launch_dependents();
  const int b = blockIdx.x / p.HG, hg = blockIdx.x - b * p.HG;
  const DecSeq sq = dec_seq(p, b);  // lens and starts do not change in this call
  const int T = (sq.keys + 15) >> 4;
  uint32_t q0, qn;
  if (p.c.B <= kDMergeScan) {
    __shared__ uint32_t s_sum[2];
    if (threadIdx.x < 2) s_sum[threadIdx.x] = 0u;
    __syncthreads();
    const int i = static_cast<int>(threadIdx.x);
    const uint32_t tiles = i < p.c.B ? static_cast<uint32_t>((dec_seq(p, i).keys + 15) >> 4) : 0u;
    const uint32_t below = __reduce_add_sync(0xffffffffu, i < b ? tiles : 0u);
    const uint32_t all = __reduce_add_sync(0xffffffffu, tiles);
    if ((i & 31) == 0) {
      atomicAdd(&s_sum[0], below);
      atomicAdd(&s_sum[1], all);
    }
    __syncthreads();
    q0 = s_sum[0];
    qn = s_sum[1];
    pdl_wait_primary();
  } else {
    pdl_wait_primary();
    q0 = __ldcg(p.ws_pre + b);
    qn = __ldcg(p.ws_pre + p.c.B);
  }
  if (T == 0) return;
  const int64_t X = static_cast<int64_t>(qn) * p.HG, x0 = static_cast<int64_t>(q0) * p.HG + static_cast<int64_t>(hg) * T;
  const DecSlots sl = line_fits_int(X, grid)
                          ? dec_slots<int, W>(static_cast<int>(x0), static_cast<int>(x0 + T), static_cast<int>(X), grid)
                          : dec_slots<int64_t, W>(x0, x0 + T, X, grid);
  const int total = sl.n + (sl.own >= 0 ? 1 : 0);
  if (total == 0) return;
  auto slot = [&](int i) {
    return static_cast<int64_t>(i == sl.n ? sl.own : (sl.c0 + i) * 2 * W + (i == 0 ? sl.w0 : 0));
  };
  const int kvh = hg / p.NG, r0g = (hg - kvh * p.NG) * kHeads;
  const int nh = min(kHeads, sq.n * p.G - r0g);
  constexpr int kQuads = DH / 4, kGroups = kWide ? 256 / kQuads : 1;
  const int first = kWide ? static_cast<int>(blockIdx.y) * kQuads + static_cast<int>(threadIdx.x) % kQuads : threadIdx.x;
  const int g = kWide ? static_cast<int>(threadIdx.x) / kQuads : 0;
  for (int i = first; i < nh * kQuads; i += kWide ? nh * kQuads : 256) {
    const int hd = i / kQuads;
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    bool broken = false;
    auto join = [&](const float2 ml, const float4 v) {
      broken |= ml.y < 0.f;
      const float Mn = fmaxf(M, ml.x), ref = Mn == -INFINITY ? 0.f : Mn;
      const float a = ex2(M - ref), f = ex2(ml.x - ref);
      M = Mn;
      L = fmaf(L, a, f * ml.y);
      O.x = fmaf(O.x, a, f * v.x);
      O.y = fmaf(O.y, a, f * v.y);
      O.z = fmaf(O.z, a, f * v.z);
      O.w = fmaf(O.w, a, f * v.w);
    };
#pragma unroll 4
    for (int k = g; k < total; k += kGroups)
      join(__ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot(k) * kHeads + hd),
           __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot(k) * kHeads * DH) + i));
    if (kWide) {
      __shared__ float4 s_o[256];
      __shared__ float2 s_ml[256];
      s_o[threadIdx.x] = O;
      s_ml[threadIdx.x] = make_float2(M, broken ? -1.f : L);
      __syncthreads();
      if (g > 0) return;
      for (int k = 1; k < kGroups; ++k) join(s_ml[k * kQuads + threadIdx.x], s_o[k * kQuads + threadIdx.x]);
    }
    const float r = broken || L == 0.f ? 0.f : 1.f / L;
    const uint2 y = broken ? make_uint2(0u, 0u)
                           : make_uint2(round_bf16x2(O.x * r, O.y * r), round_bf16x2(O.z * r, O.w * r));
    const int rr = r0g + hd, j = rr / p.G;
    reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(sq.row0) + j) * p.Hq + static_cast<int64_t>(kvh) * p.G +
                                      (rr - j * p.G)) * DH)[i - hd * kQuads] = y;
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
  // A group of 8, 16 or 32 rows; more groups read the cache again (from L2, mostly). 32 rows at dh = 128 want more
  // registers than there are: groups of 16 and 32, e4m3: 68 and 87 us (64 sequences of 8000 rows, one key head,
  // 32 query heads), 17 and 23 (2 of 1000); bf16 92 and 89, 16 and 21. At dh = 64 32 rows pay: 155 and 114 us (64
  // sequences of 1250, 20 key heads, 32 query heads each).
  d.NT = R <= 8 ? 1 : R <= 16 || c.dh == 128 ? 2 : 4;
  d.NG = (R + 8 * d.NT - 1) / (8 * d.NT);
  d.HG = c.Hkv * d.NG;
  const size_t slots = static_cast<size_t>(num_sms()) * 2 * dec_warps(c.dtype == SLIM_E4M3, c.dh, d.NT);
  d.o_bytes = up256(slots * 8 * d.NT * c.dh * 4);
  d.ml_bytes = up256(slots * 8 * d.NT * 2 * 4);
  d.pre_bytes = up256((static_cast<size_t>(c.B) + 1) * 4);
  return d;
}

template <bool E, int DH, int NT>
uint32_t dec_smem_bytes(int B, bool split) {
  using C = DecCfg<E, DH, NT>;
  constexpr int W = C::kWarps;
  return static_cast<uint32_t>(W * C::kRing + W * C::kStages * C::kTT * 2 * 4 + W * C::kHeads * 2 * 4 +
                               W * sizeof(DecEnd) + (split ? (B + 1) * 4 : 0));
}

template <bool E, int DH, int NT>
cudaError_t launch_dec(const PagedDecodeParams& p, cudaStream_t st, int* launches) {
  using C = DecCfg<E, DH, NT>;
  const uint32_t smem = dec_smem_bytes<E, DH, NT>(p.c.B, p.split != 0);
  auto kern = paged_decode_kernel<E, DH, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), static_cast<uint32_t>(max_smem_optin()), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = p.split ? num_sms() : p.c.B * p.HG;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
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
  const bool wide = p.c.B * p.HG * kDWide <= grid;
  cfg2.gridDim = dim3(static_cast<unsigned>(p.c.B * p.HG), wide ? 8 * NT : 1, 1);
  cfg2.blockDim = dim3(256, 1, 1);
  cfg2.stream = st;
  cfg2.attrs = attr;
  cfg2.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg2, merge_paged_kernel<DH, NT, C::kWarps, true>, p, grid)
           : cudaLaunchKernelEx(&cfg2, merge_paged_kernel<DH, NT, C::kWarps, false>, p, grid);
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
  if (NT == 1) return launch_dec<E, DH, 1>(p, st, launches);
  if (DH == 128 || NT == 2) return launch_dec<E, DH, 2>(p, st, launches);
  return launch_dec<E, DH, DH == 64 ? 4 : 2>(p, st, launches);
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
  // One CTA per work sequence, no merge, where that is one wave and the longest sequence, which the call then
  // waits for, is short. bf16, dh = 128, whole and split: one sequence of 8 key heads (4 query heads each), 512
  // rows 7.9 and 10.1 us, 1024 10.6 and 10.4, 1536 13.4 and 11.1; 8 such sequences of 1024 rows 11.8 and 15.0, of
  // 1536 14.7 and 18.6 where all are that long. More rows a group: two sequences of one key head with 32 query
  // heads, 512 rows 10.6 and 12.3, 768 12.5 and 12.5, 1024 14.2 and 12.6.
  p.split = !(static_cast<int64_t>(c.B) * d.HG <= num_sms() && hint <= (d.NT == 1 ? 1024 : 768));
  if (c.dtype == SLIM_E4M3)
    return c.dh == 64 ? launch_dec_nt<true, 64>(p, d.NT, st, launches) : launch_dec_nt<true, 128>(p, d.NT, st, launches);
  return c.dh == 64 ? launch_dec_nt<false, 64>(p, d.NT, st, launches) : launch_dec_nt<false, 128>(p, d.NT, st, launches);
}

}  // namespace slim
