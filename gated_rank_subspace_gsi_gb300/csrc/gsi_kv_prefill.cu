// gsi_kv_prefill.cu -- attention of many rows (prompts, chunks of them) over
// the 8-bit cache, on the tcgen05 tensor cores.
//
// A CTA takes one (D = 256) or two tiles of 128 rows of a key/value head (new
// rows x query heads of its group, which share keys and values) and walks the
// pages they see:
//   S = Q C_k^T (128 x 64), P = 2^(S 2^e q + f - m + 11), O += P C_v
// with the codes C, K's scale 2^e, V's 2^f joined to the exponent, m a running
// maximum of S 2^e q + f and the divisor sum P 2^(-f), as for few rows.  Codes
// are exact in fp16; P is fp16, accumulators fp32.
//
// The tensor cores would bound it (4 D flops a row and token); exponentials (16
// a clock and SM) take as long at D = 128, and codes have to become fp16 tiles
// on the way.  So the roles run side by side: one warp keeps a ring of code tiles
// filled by TMA; converter warps turn them into both operands, 128-byte-swizzled
// K-major tiles (V transposed by byte permutes), without bank conflicts; one lane
// issues the MMAs; eight warps turn S into P inside TMEM, a row per thread (two tiles)
// or half a row (D = 256, whose O leaves TMEM no room for a second tile).  S is
// double-buffered, so the product of page j + 1 runs under the softmax of page
// j.  O stays in TMEM; it is rescaled only when a row's maximum has grown by
// more than 4 (a factor of 16), which P's range allows for.
//
// Measured: 2000 rows over 2049 tokens and themselves, 16 heads of 256: 129 us,
// 775 TFLOP/s (40% of the bf16 rate measured for a large product; the tensor pipe is
// busy 40% of the time, issue slots 51%: softmax and conversion pace it); four
// prompts of 301 to 1023, 12 heads of 64: 22 us.
//
// Few rows of few heads over a long cache would leave most SMs idle: the pages
// are then split over CTAs, and a second launch joins their outputs (fp32, each
// over its own sum) by the logarithms of their sums.  130 rows over 16000 tokens,
// 16 heads of 256: 90 us, unsplit 279.
#include <cuda.h>

#include <algorithm>

#include "gsi_internal.h"
#include "gsi_kv.cuh"
#include "gsi_kv_codes.cuh"
#include "gsi_tcgen05.cuh"

namespace gsi {
namespace {

constexpr int kRows = 128;      // of a tile
constexpr int kSoft = 8;        // softmax warps
constexpr int kLeast = 8;       // pages of a CTA's share, where a group's are split
constexpr int kScales = 16;     // pages whose scales are kept; the ring is shorter
constexpr float kGrow = 4.f;    // growth of a maximum that is let stand
constexpr float kLift = 11.f;   // P <= 2^(kGrow + kLift) = 2^15
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int HL>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr bool kQTmem = D == 256;  // Q's fp16 tile in TMEM, else in shared memory
  static constexpr int kConv = D == 256 ? 8 : 4;      // converter warps: half K, half V
  static constexpr int kPieces = D / 8 / (kConv / 2); // of 8 tokens x 64 dims, a K warp's of a page
  static constexpr int kWords = D / 16 / (kConv / 2); // 64 tokens x 16 dims times this are a V warp's
  static constexpr int kWarps = kSoft + kConv + 1 + kTiles;  // the ring's, the tiles' MMAs
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSlot = kPage * D;   // bytes of a page's codes of K or of V
  static constexpr int kSlots = D == 256 ? (HL ? 1 : 2) : HL ? 2 : 3;  // of each ring, K's and V's
  static constexpr int kTile = 2 * kPage * D;     // fp16 K or V^T of a page
  static constexpr int kStages = D == 256 || HL ? 2 : 3;
  static constexpr int kStagesV = D == 256 && HL ? 1 : kStages;
  static constexpr int kQTile = 2 * kRows * D;
  static constexpr int kQBytes = kTiles * kQTile;  // of the high or the low parts
  static constexpr int kQParts = (kQTmem ? 0 : 1) + HL;  // in shared memory: high part, low part
  static constexpr size_t kSmem =
      1024 + size_t(kQParts) * kQBytes + size_t(kStages + kStagesV) * kTile + size_t(2 * kSlots) * kSlot;
  // TMEM columns: S of each tile (2 x 64, P in its first half), O of each (D), Q (D / 2)
  static constexpr int kColO = kTiles * 2 * kPage, kColQ = kColO + kTiles * D;
  static constexpr int kCols = 512;
  static constexpr int kColsS = kTiles == 1 ? kPage / 2 : kPage;  // of a thread
};

struct PreMaps {
  CUtensorMap k, v;  // boxes of 64 tokens x 128 bytes
};
struct PreArgs {
  KvAttnArgs a;
  int tiles;   // groups of tiles (CTAs) of the longest sequence
  int splits;  // CTAs that share a group's pages, if there are enough
  float* part;      // [CTAs][rows of a group][D] outputs of shares
  float* part_lse;  // [CTAs][rows of a group] log2 of their sums
};

// Rows of a group, and the pages that they see, in shares.
struct Group {
  int64_t row0;
  int rows, total, all, share;
};
__device__ __forceinline__ Group group_of(const PreArgs& p, const SeqRows& sq, int group, int most) {
  Group g;
  const int G = p.a.c.group;
  g.row0 = int64_t(group) * most;
  g.rows = int(min(int64_t(most), int64_t(sq.count) * G - g.row0));
  g.total = min(sq.len + sq.count, p.a.c.max_pages * kPage);
  const int last_row = int((g.row0 + g.rows - 1) / G);
  g.all = (min(sq.len + last_row + 1, g.total) + kPage - 1) / kPage;
  g.share = max((g.all + p.splits - 1) / p.splits, kLeast);
  return g;
}

// Two fp32 values in a register pair, and their product and sum (one instruction).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Column k of S and P, and row k of the K tile, is token k / 8 + 8 (k % 8) of the
// page: eight neighbouring columns are tokens eight apart, which is what lets the
// converters read staged codes without bank conflicts.
__device__ __forceinline__ constexpr int token_of(int k) { return (k >> 3) + 8 * (k & 7); }

// Offset of row r, 16-byte chunk c (8 fp16) of a K-major tile with 128-byte rows.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <int FMT, int D, int HL>
__global__ void __launch_bounds__(Shape<D, HL>::kThreads, 1)
    prefill_kernel(const __grid_constant__ PreMaps maps, const __grid_constant__ PreArgs p) {
  using Sh = Shape<D, HL>;
  constexpr int kConv = Sh::kConv, kStages = Sh::kStages, kStagesV = Sh::kStagesV, kSlots = Sh::kSlots;
  constexpr int kTiles = Sh::kTiles, kN = Sh::kColsS;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t raw_full[2][kSlots], raw_empty[2][kSlots], q_full, x_full[4];
  __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStagesV], v_empty[kStagesV];
  __shared__ uint64_t s_full[kTiles][2], p_full[kTiles][2], o_done[kTiles][2];
  __shared__ uint64_t sc_full[kScales];
  __shared__ float2 s_scale[kScales];  // K's and V's scale of a page; K's 0: out of range
  __shared__ float s_qs[kTiles * kRows];
  __shared__ float s_x[2][2][kRows];   // halves of a row: maxima, at the end sums
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  // (a shuffle: the warp's number is uniform)
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int H = p.a.c.heads, G = p.a.c.group;
  // rows that see most first, of all heads: the last CTAs to start are short
  const int h = blockIdx.x % H, b = blockIdx.z, rest = blockIdx.x / H, split = rest % p.splits;
  const int group = p.tiles - 1 - rest / p.splits;
  pdl_launch_dependents();
  pdl_wait();
  const SeqRows sq = seq_rows(p.a.r, p.a.c, b);
  const Group gr = group_of(p, sq, group, kTiles * kRows);
  const int rows = gr.rows, first = split * gr.share;  // first: page
  if (rows <= 0 || (split > 0 && first >= gr.all)) return;
  const int64_t row0 = gr.row0;
  const int total = gr.total, pages = min(gr.share, gr.all - first);
  const int whole = total / kPage - first;             // counted from first, as j
  const bool shared = gr.share < gr.all;
  const size_t slot = ((size_t(b) * p.tiles + group) * H + h) * p.splits + split;
  const int tiles = rows > kRows ? kTiles : 1;  // that have rows

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
  // Q's parts, K tiles, V^T tiles, code ring
  constexpr uint32_t kAtK = Sh::kQParts * Sh::kQBytes, kAtV = kAtK + kStages * Sh::kTile,
                     kAtRaw = kAtV + kStagesV * Sh::kTile;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], kConv / 2);
      mbar_init(&k_empty[i], tiles);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(&v_full[i], kConv / 2);
      mbar_init(&v_empty[i], tiles);
    }
    for (int i = 0; i < kSlots; ++i)
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&raw_full[kv][i], 1);
        mbar_init(&raw_empty[kv][i], kConv / 2);
      }
    for (int t = 0; t < kTiles; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[t][i], 1);
        mbar_init(&p_full[t][i], kSoft / kTiles);
        mbar_init(&o_done[t][i], 1);
      }
    for (int i = 0; i < kScales; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&x_full[i], 2);
    mbar_init(&q_full, kSoft);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&s_tmem, Sh::kCols);

  // Q: a row per D / 8 lanes, scaled so that its largest lies in [2^13, 2^14)
  // (as for few rows), high parts and low parts as K-major tiles.  High parts
  // that belong in TMEM pass through the K tiles.
  {
    constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes of a row, rows of a warp at a time
    unsigned char* hi_to = smem + (Sh::kQTmem ? kAtK : 0);
    unsigned char* lo_to = smem + (Sh::kQTmem ? 0 : Sh::kQBytes);
    const int c = lane % kLanes;
    constexpr int kUn = 4;
    for (int r0 = warp * kAt; r0 < tiles * kRows; r0 += Sh::kWarps * kAt * kUn) {
      float x[kUn][8];
#pragma unroll
      for (int u = 0; u < kUn; ++u) {
        const int r = r0 + u * Sh::kWarps * kAt + lane / kLanes;
        const int64_t rr = row0 + r;
        const int64_t at = (sq.first + rr / G) * p.a.ldq + (int64_t(h) * G + rr % G) * D + c * 8;
        if (r >= rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
        } else if (p.a.bf16) {
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) + at), x[u]);
        } else {
          const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(p.a.q) + at);
          const float4 y = v[0], z = v[1];
          x[u][0] = y.x; x[u][1] = y.y; x[u][2] = y.z; x[u][3] = y.w;
          x[u][4] = z.x; x[u][5] = z.y; x[u][6] = z.z; x[u][7] = z.w;
        }
      }
#pragma unroll
      for (int u = 0; u < kUn; ++u) {
        const int r = r0 + u * Sh::kWarps * kAt + lane / kLanes;
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[u][e]));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (r >= tiles * kRows) continue;
        const int ex = int(__float_as_uint(top) >> 23) - 126;
        const int sh = top > 0.f && ex < 129 ? min(14 - ex, 100) : 0;
        // the sign of the logits' factor goes to q: a maximum of S is one of S q
        const float up = p.a.qscale < 0.f ? -exp2_int(sh) : exp2_int(sh);
        if (c == 0) s_qs[r] = fabsf(p.a.qscale) * exp2_int(-sh);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y0 = x[u][2 * e] * up, y1 = x[u][2 * e + 1] * up;
          hi[e] = pack_f16(y0, y1);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
          lo[e] = pack_f16(y0 - back.x, y1 - back.y);
        }
        const int at = (r / kRows) * Sh::kQTile + (c >> 3) * (kRows * 128) + swz(r % kRows, c & 7);
        *reinterpret_cast<uint4*>(hi_to + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (HL) *reinterpret_cast<uint4*>(lo_to + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  uint32_t* status = p.a.c.status;

  if (warp < kSoft) {
    // ---- softmax ---------------------------------------------------------------
    const int quarter = warp & 3, part = warp >> 2;   // part: the tile, or half of a row
    const int tile = kTiles == 1 ? 0 : part, half = kTiles == 1 ? part : 0;
    const int r = quarter * 32 + lane;                // in the tile
    const int rt = tile * kRows + r;
    const int64_t rr = row0 + rt;
    const int i = int(rr / G), hq = h * G + int(rr % G);
    const bool real = rt < rows;
    const int see = real ? min(sq.len + i + 1, total) - first * kPage : 0;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t col_o = tmem + lanes + Sh::kColO + tile * D + half * (D / 2);
    constexpr int kOut = kTiles == 1 ? D / 2 : D;     // columns of O of a thread
    const float qs = s_qs[rt];
    if (Sh::kQTmem) {
      // half a row of the high part: 64 columns
#pragma unroll
      for (int c0 = 0; c0 < D / 16; c0 += 8) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = half * (D / 16) + c0 + e;
          const uint4 w = *reinterpret_cast<const uint4*>(smem + kAtK + (c >> 3) * (kRows * 128) + swz(r, c & 7));
          v[4 * e] = w.x;
          v[4 * e + 1] = w.y;
          v[4 * e + 2] = w.z;
          v[4 * e + 3] = w.w;
        }
        tmem_st_32x32b_x32(tmem + lanes + Sh::kColQ + half * (D / 4) + c0 * 4, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&q_full);
    }
    // Warps wait for o_done only when they touch O.  Two barriers, of even and of
    // odd pages: the product of page j + 1 needs this warp's P, so a barrier is
    // never a phase ahead of a wait, and the one of page j - 3 ended before S of
    // page j - 1 began, so it is never a phase behind.
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; tile < tiles && j < pages; ++j) {
      // (not k_full: K tiles are reused as soon as S is done, so their barriers may be
      // two phases ahead of a warp that waits here)
      ok = wait_often(&sc_full[j % kScales], (j / kScales) & 1, status, &s_abort) &&
           wait_often(&s_full[tile][j & 1], (j >> 1) & 1, status, &s_abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      const float2 sc = s_scale[j % kScales];
      // not 0 (a factor of 0, a page out of range): times -inf that is NaN
      const float k = fmaxf(sc.x * qs, 1e-37f);
      const float f = float(int(__float_as_uint(sc.y) >> 23) - 127);
      const float inv_vs = __uint_as_float((254u << 23) - __float_as_uint(sc.y));
      const int limit = sc.x > 0.f ? see - j * kPage : 0;  // tokens of the page that the row sees
      const uint32_t col = tmem + lanes + uint32_t((tile * 2 + (j & 1)) * kPage);
      uint32_t s[kN];
#pragma unroll
      for (int e = 0; e < kN; e += 32)
        tmem_ld_32x32b_x32_nowait(col + half * kN + e, *reinterpret_cast<uint32_t(*)[32]>(&s[e]));
      tmem_wait_ld();
      if (!__all_sync(0xFFFFFFFFu, limit >= kPage)) {
        const int lim = limit - half * (kN / 8);  // token_of(half kN + e) = half kN / 8 + token_of(e)
#pragma unroll
        for (int e = 0; e < kN; ++e) s[e] = token_of(e) < lim ? s[e] : 0xFF800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < kN; e += 2)
        mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
      float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      if (kTiles == 1) {
        // the other half's maximum; it has read its S by then, so P may go there
        s_x[j & 1][half][r] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&x_full[quarter]);
        ok = wait_often(&x_full[quarter], j & 1, status, &s_abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        top = fmaxf(top, s_x[j & 1][half ^ 1][r]);
      }
      top = top == -INFINITY ? -INFINITY : fmaf(top, k, f);
      const bool grow = top > m + kGrow || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float hs = ex2_half(grow ? m - top : 0.f), scale = hs * hs;  // (0 where m is -inf)
        if (grow) m = top;
        l = l * hs * hs;
        if (j > 0) {
          ok = wait_often(&o_done[tile][(j - 1) & 1], ((j - 1) >> 1) & 1, status, &s_abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kOut; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16_nowait(col_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
            tmem_st_32x32b_x16(col_o + c, o);
          }
        }
      }
      const float off = m == -INFINITY ? 0.f : f - m + kLift;
      const uint64_t k2 = pair(k, k), off2 = pair(off, off);
      uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) {
        const float2 x = unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), k2, off2));
        const float a0 = ex2(x.x), a1 = ex2(x.y);
        sum[e & 1] = add2(sum[e & 1], pair(a0, a1));
        s[e] = pack_f16(a0, a1);
      }
      const float2 sums = unpair(add2(sum[0], sum[1]));
      l = fmaf(sums.x + sums.y, inv_vs, l);
      if (kN == 64)
        tmem_st_32x32b_x32(col, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      else
        tmem_st_32x32b_x16(col + half * 16, *reinterpret_cast<uint32_t(*)[16]>(&s[0]));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&p_full[tile][j & 1]);
    }
    if (tile < tiles) {
      if (ok) {
        ok = wait_often(&o_done[tile][(pages - 1) & 1], ((pages - 1) >> 1) & 1, status, &s_abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
      }
      if (kTiles == 1 && ok) {
        // the other half's sum; page `pages` of the exchange
        s_x[pages & 1][half][r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&x_full[quarter]);
        ok = wait_often(&x_full[quarter], pages & 1, status, &s_abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) l = s_x[pages & 1][0][r] + s_x[pages & 1][1][r];
      }
      if (ok && shared) {
        // this share's rows as they are, over their sum
        const float inv = l != 0.f ? 1.f / l : 0.f;
        float* to = p.part + (slot * (kTiles * kRows) + rt) * D + half * (D / 2);
        for (int c = 0; c < kOut; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32_nowait(col_o + c, o);
          tmem_wait_ld();
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(to + c + e) =
                  make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                              __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
          }
        }
        if (real && half == 0)
          p.part_lse[slot * (kTiles * kRows) + rt] = l != 0.f ? m - kLift + log2f(l) : -INFINITY;
      } else if (ok) {
        // O to shared memory as bf16 (Q's, or the stages': every product is done)
        const float inv = l != 0.f ? 1.f / l : 0.f;
        unsigned char* to = smem + rt * (2 * D);
        for (int c = 0; c < kOut; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32_nowait(col_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 v;
            v.x = pack_bf16(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
            v.y = pack_bf16(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            v.z = pack_bf16(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
            v.w = pack_bf16(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
            const int ch = (half * (D / 2) + c + e) / 8;
            *reinterpret_cast<uint4*>(to + ((ch ^ (r & 7)) << 4)) = v;
          }
        }
        if (real && half == 0 && p.a.lse)
          p.a.lse[int64_t(sq.first + i) * (int64_t(H) * G) + hq] =
              l != 0.f ? (m - kLift + log2f(l)) * kLn2 : -INFINITY;
      }
    }
  } else if (warp < kSoft + kConv) {
    // ---- codes to fp16 tiles -----------------------------------------------
    // Half of the warps take K, half V, of every page.  K in pieces of 8 tokens x 64
    // dims (lane: 16 dims of a token); V 64 tokens x 16 dims and more (lane: 4 dims
    // and more of 8 tokens, those eight apart).
    constexpr int kHalf = kConv / 2, kP = Sh::kPieces, kW = Sh::kWords;
    const bool is_v = warp >= kSoft + kHalf;
    const int cw = (warp - kSoft) % kHalf;
    // where byte `dim` (a multiple of 4) of a token lies in a slot
    auto raw_at = [&](int t, int dim) {
      if (D == 64) {
        const int line = t >> 1, c = (t & 1) * 4 + (dim >> 4);
        return line * 128 + ((c ^ (line & 7)) << 4) + (dim & 15);
      }
      return (dim >> 7) * (kPage * 128) + t * 128 + ((((dim & 127) >> 4) ^ (t & 7)) << 4) + (dim & 15);
    };
    const size_t tail_at = (size_t(b) * H + h) * kPage * D;
    const int held = total % kPage;
    auto inverse = [&](float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); };
    bool ok = true;
    auto arrived = [&](uint64_t* bar, int n) {
      return __all_sync(0xFFFFFFFFu, wait_often(bar, n & 1, status, &s_abort));
    };
    auto hand_over = [&](uint64_t* empty, uint64_t* full) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cta(empty);
        mbar_arrive_cta(full);
      }
    };
    if (!is_v) {
      // piece u: tokens 8 ((i + u) % 8) + i, i = 0 .. 7 -- a diagonal of the page, so
      // that neither the staged rows (token % 8) nor the tile's (token / 8) collide --
      // and 64 dims u / 8
      const int ki = lane & 7, kc = lane >> 3;
      auto k_token = [&](int u) { return 8 * ((ki + u) & 7) + ki; };
      auto k_row = [&](int u) { return 8 * ki + ((ki + u) & 7); };
      auto k_dim = [&](int u) { return (u >> 3) * 64 + kc * 16; };
      if (Sh::kQTmem) ok = arrived(&q_full, 0);  // Q passes through the K tiles
#pragma unroll 1
      for (int j = 0; ok && j < pages; ++j) {
        const int st = j % kStages, sl = j % kSlots;
        ok = arrived(&raw_full[0][sl], j / kSlots) && (j < kStages || arrived(&k_empty[st], j / kStages - 1));
        if (!ok) break;
        const float ks = s_scale[j % kScales].x;
        const unsigned char* raw = smem + kAtRaw + sl * Sh::kSlot;
        unsigned char* t = smem + kAtK + st * Sh::kTile;
        if (ks > 0.f && j < whole) {
          uint4 x[kP];
#pragma unroll
          for (int e = 0; e < kP; ++e) {
            const int u = cw * kP + e;
            x[e] = *reinterpret_cast<const uint4*>(raw + raw_at(k_token(u), k_dim(u)));
          }
#pragma unroll
          for (int e = 0; e < kP; ++e) {
            const int u = cw * kP + e;
            uint4 a, c;
            codes_f16<FMT>(x[e].x, a.x, a.y);
            codes_f16<FMT>(x[e].y, a.z, a.w);
            codes_f16<FMT>(x[e].z, c.x, c.y);
            codes_f16<FMT>(x[e].w, c.z, c.w);
            *reinterpret_cast<uint4*>(t + (u >> 3) * (kPage * 128) + swz(k_row(u), 2 * kc)) = a;
            *reinterpret_cast<uint4*>(t + (u >> 3) * (kPage * 128) + swz(k_row(u), 2 * kc + 1)) = c;
          }
        } else {
          // the tail, values over the scale; or a page out of range, zeros
          const float inv = inverse(ks > 0.f ? ks : 1.f);
#pragma unroll 1
          for (int e = 0; e < 2 * kP; ++e) {
            const int u = cw * kP + (e >> 1), tok = k_token(u);
            uint4 y = make_uint4(0, 0, 0, 0);
            if (ks > 0.f && tok < held)
              y = *reinterpret_cast<const uint4*>(p.a.c.tail[0] + tail_at + tok * D + k_dim(u) + (e & 1) * 8);
            *reinterpret_cast<uint4*>(t + (u >> 3) * (kPage * 128) + swz(k_row(u), 2 * kc + (e & 1))) =
                make_uint4(bf16_f16(y.x, inv), bf16_f16(y.y, inv), bf16_f16(y.z, inv), bf16_f16(y.w, inv));
          }
        }
        hand_over(&raw_empty[0][sl], &k_full[st]);
      }
    } else {
      const int vc = lane & 7, dim = cw * (16 * kW) + (lane >> 3) * (4 * kW);
#pragma unroll 1
      for (int j = 0; ok && j < pages; ++j) {
        const int st = j % kStagesV, sl = j % kSlots;
        ok = arrived(&raw_full[1][sl], j / kSlots) && (j < kStagesV || arrived(&v_empty[st], j / kStagesV - 1));
        if (!ok) break;
        const float2 sc = s_scale[j % kScales];
        const unsigned char* raw = smem + kAtRaw + (kSlots + sl) * Sh::kSlot;
        unsigned char* t = smem + kAtV + st * Sh::kTile;
        if (sc.x > 0.f && j < whole) {
          uint32_t x[8][kW];  // of tokens vc + 8 e
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const unsigned char* at = raw + raw_at(vc + 8 * e, dim);
            if (kW == 4) {
              const uint4 w = *reinterpret_cast<const uint4*>(at);
              x[e][0] = w.x;
              x[e][kW > 1 ? 1 : 0] = w.y;
              x[e][kW > 2 ? 2 : 0] = w.z;
              x[e][kW > 3 ? 3 : 0] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(at);
              x[e][0] = w.x;
              x[e][kW > 1 ? 1 : 0] = w.y;
            }
          }
#pragma unroll
          for (int q = 0; q < kW; ++q) {
            uint32_t o[4][4];  // [dim of the four][token pair]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              codes_f16<FMT>(__byte_perm(x[2 * e][q], x[2 * e + 1][q], 0x5140), o[0][e], o[1][e]);
              codes_f16<FMT>(__byte_perm(x[2 * e][q], x[2 * e + 1][q], 0x7362), o[2][e], o[3][e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(t + swz(dim + q * 4 + e, vc)) = make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]);
          }
        } else {
          const float inv = inverse(sc.y);
#pragma unroll 1
          for (int q = 0; q < 2 * kW; ++q) {
            uint32_t o[2][4];  // [dim of two][token pair]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t y[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int tok = vc + 8 * (2 * e + k);
                y[k] = sc.x > 0.f && tok < held
                           ? *reinterpret_cast<const uint32_t*>(p.a.c.tail[1] + tail_at + tok * D + dim + 2 * q)
                           : 0u;
                y[k] = bf16_f16(y[k], inv);
              }
              o[0][e] = __byte_perm(y[0], y[1], 0x5410);
              o[1][e] = __byte_perm(y[0], y[1], 0x7632);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<uint4*>(t + swz(dim + 2 * q + k, vc)) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
          }
        }
        hand_over(&raw_empty[1][sl], &v_full[st]);
      }
    }
  } else if (warp == kSoft + kConv) {
    // ---- the rings of codes ---------------------------------------------------
    // pages and scales of 32 blocks at a time, one per lane
    int page = -1, j = 0, vs_top = 0;
    float2 sc = make_float2(0.f, 1.f);
    bool ok = true;
    for (; ok && j < pages; ++j) {
      if (j % 32 == 0) {
        page = -1;
        sc = make_float2(0.f, 1.f);
        if (j + lane < pages) {
          page = page_of(p.a.c, b, first + j + lane);
          if (page >= 0) sc = make_float2(p.a.c.scale[0][size_t(page) * H + h], p.a.c.scale[1][size_t(page) * H + h]);
        }
      }
      const int pg = __shfl_sync(0xFFFFFFFFu, page, j % 32), sl = j % kSlots;
      const bool codes = pg >= 0 && j < whole;
      const int line = (pg * H + h) * (D == 64 ? kPage / 2 : kPage);
      // (the scales of page j - 16 are out of use: the rings are that short)
      const int vs = clip_scale(__shfl_sync(0xFFFFFFFFu, __float_as_int(sc.y), j % 32), vs_top);
      if (lane == j % 32) {
        s_scale[j % kScales] = make_float2(sc.x, __int_as_float(vs));
        mbar_arrive_cta(&sc_full[j % kScales]);
      }
      __syncwarp();
      for (int kv = 0; kv < 2; ++kv) {
        if (j >= kSlots) ok = ok && wait_often(&raw_empty[kv][sl], (j / kSlots - 1) & 1, status, &s_abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane == 0) {
          if (codes) {
            unsigned char* dst = smem + kAtRaw + (kv * kSlots + sl) * Sh::kSlot;
            mbar_arrive_expect_tx(&raw_full[kv][sl], Sh::kSlot);
#pragma unroll
            for (int f = 0; f < (D + 127) / 128; ++f)
              tma_load_2d(dst + f * (kPage * 128), kv ? &maps.v : &maps.k, 64 * f, line, &raw_full[kv][sl]);
          } else {
            mbar_arrive_cta(&raw_full[kv][sl]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      // no copy may still be writing when the CTA ends
      for (int i = max(0, j - kSlots); i < j; ++i)
        for (int kv = 0; kv < 2; ++kv) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&raw_full[kv][i % kSlots], (i / kSlots) & 1) &&
                 globaltimer_ns() - t0 < kWaitLimitNs / 100) {
          }
        }
    }
  } else {
    // ---- the MMAs ------------------------------------------------------------
    // A warp per tile.  The whole warp walks the loop, so that addresses stay in
    // uniform registers; one elected lane issues.
    const int t = warp - (kSoft + kConv + 1);
    const uint32_t id_s = idesc_f16_f32(kRows, kPage), id_o = idesc_f16_f32(kRows, D);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t q_lo = sw128_desc_lo(base + t * Sh::kQTile);
    bool ok = t < tiles && (!Sh::kQTmem || wait_often(&q_full, 0, status, &s_abort));
    ok = __all_sync(0xFFFFFFFFu, ok);
    tc_fence_after();
    auto arrived = [&](uint64_t* bar, uint32_t parity) {
      const bool in = __all_sync(0xFFFFFFFFu, wait_often(bar, parity, status, &s_abort));
      tc_fence_after();
      return in;
    };
    auto logits = [&](int j) {
      const uint32_t k_lo = sw128_desc_lo(base + kAtK + uint32_t(j % kStages) * Sh::kTile);
      const uint32_t acc = tm + uint32_t((t * 2 + (j & 1)) * kPage);
      if (elect_one()) {
#pragma unroll
        for (int d = 0; d < D; d += 16) {
          const uint64_t bd = sw128_desc(k_lo + ((d >> 6) * (kPage * 128) + (d & 63) * 2) / 16);
          const uint32_t q_at = ((d >> 6) * (kRows * 128) + (d & 63) * 2) / 16;
          if (Sh::kQTmem)
            tc_mma_f16_ts(acc, tm + Sh::kColQ + d / 2, bd, id_s, d != 0);
          else
            tc_mma_f16_ss(acc, sw128_desc(q_lo + q_at), bd, id_s, d != 0);
          if (HL)
            tc_mma_f16_ss(acc, sw128_desc(q_lo + (Sh::kQTmem ? 0 : Sh::kQBytes / 16) + q_at), bd, id_s, 1);
        }
        tc_commit(&s_full[t][j & 1]);
        tc_commit(&k_empty[j % kStages]);
      }
      __syncwarp();
    };
    if (ok) ok = arrived(&k_full[0], 0);
    if (ok) logits(0);
    for (int j = 0; ok && j < pages; ++j) {
      const int st = j % kStagesV;
      if (j + 1 < pages) {
        if (!arrived(&k_full[(j + 1) % kStages], ((j + 1) / kStages) & 1)) break;
        logits(j + 1);
      }
      ok = arrived(&v_full[st], (j / kStagesV) & 1) && arrived(&p_full[t][j & 1], (j >> 1) & 1);
      const uint32_t v_lo = sw128_desc_lo(base + kAtV + uint32_t(st) * Sh::kTile);
      const uint32_t pa = tm + uint32_t((t * 2 + (j & 1)) * kPage);
      if (ok && elect_one()) {
#pragma unroll
        for (int k = 0; k < kPage; k += 16)
          tc_mma_f16_ts(tm + Sh::kColO + t * D, pa + k / 2, sw128_desc(v_lo + k * 2 / 16), id_o, j != 0 || k != 0);
        tc_commit(&o_done[t][j & 1]);
        tc_commit(&v_empty[st]);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (s_abort == 0 && !shared) {
    // the rows, 16 bytes a lane
    constexpr int kVec = D / 8;
    for (int x = threadIdx.x; x < rows * kVec; x += Sh::kThreads) {
      const int rt = x / kVec, ch = x % kVec;
      const int64_t rr = row0 + rt;
      const uint4 v = *reinterpret_cast<const uint4*>(smem + rt * (2 * D) + ((ch ^ (rt & 7)) << 4));
      *reinterpret_cast<uint4*>(p.a.out + (sq.first + rr / G) * p.a.ldo + (int64_t(h) * G + rr % G) * D + ch * 8) = v;
    }
  }
  if (warp == 0) {
    if (s_abort) {
      // the products in flight end before their memory is given back
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < kWaitLimitNs / 1000) {
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kCols);
  }
}

// The rows of groups whose pages were shared: a warp per row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ PreArgs p) {
  constexpr int kMost = (D == 256 ? 1 : 2) * kRows, kE = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int H = p.a.c.heads, G = p.a.c.group, h = blockIdx.y % H, group = blockIdx.y / H, b = blockIdx.z;
  const SeqRows sq = seq_rows(p.a.r, p.a.c, b);
  const Group gr = group_of(p, sq, group, kMost);
  const int rt = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (rt >= gr.rows || gr.share >= gr.all) return;
  const int n = (gr.all + gr.share - 1) / gr.share;
  const size_t at = ((size_t(b) * p.tiles + group) * H + h) * p.splits * kMost + rt;  // of the first share
  float top = -INFINITY;
  for (int s = lane; s < n; s += 32) top = fmaxf(top, p.part_lse[at + size_t(s) * kMost]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (top == -INFINITY) top = 0.f;  // nothing seen: weights of 0
  float sum = 0.f, o[kE] = {};
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float w = ex2(p.part_lse[at + size_t(s) * kMost] - top);
    const float* x = p.part + (at + size_t(s) * kMost) * D + lane * kE;
    sum += w;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const float2 y = *reinterpret_cast<const float2*>(x + e);
      o[e] = fmaf(w, y.x, o[e]);
      o[e + 1] = fmaf(w, y.y, o[e + 1]);
    }
  }
  const int64_t rr = gr.row0 + rt, row = sq.first + rr / G;
  const int hq = h * G + int(rr % G);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.a.out + row * p.a.ldo + int64_t(hq) * D) + lane * (kE / 2);
#pragma unroll
  for (int e = 0; e < kE; e += 2) to[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
  if (lane == 0 && p.a.lse)
    p.a.lse[row * (int64_t(H) * G) + hq] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

template <int FMT, int D, int HL>
gsi_status_t launch(gsi_kv* kv, const KvAttnArgs& a, int64_t max_rows, cudaStream_t s) {
  using Sh = Shape<D, HL>;
  PreMaps maps;
  maps.k = *reinterpret_cast<const CUtensorMap*>(kv->tmaps[4]);
  maps.v = *reinterpret_cast<const CUtensorMap*>(kv->tmaps[5]);
  PreArgs p;
  p.a = a;
  p.tiles = int((max_rows * a.c.group + Sh::kTiles * kRows - 1) / (Sh::kTiles * kRows));
  auto kernel = prefill_kernel<FMT, D, HL>;
  static std::atomic<uint64_t> ready{0};  // devices that allow the kernel its shared memory
  if (!allow_smem(kernel, Sh::kSmem, kv->device, ready)) return GSI_ERR_CUDA;
  // one wave of CTAs, so that is as many shares as part has room for
  const int64_t groups = int64_t(a.c.heads) * p.tiles * a.c.seqs;
  p.splits = int(std::max<int64_t>(1, std::min<int64_t>(kv->num_sms / groups, a.c.max_pages / kLeast)));
  p.part_lse = kv->pre_part;
  p.part = kv->pre_part + size_t(kv->num_sms) * Sh::kTiles * kRows;
  if (int64_t(a.c.heads) * p.tiles * p.splits >= (int64_t(1) << 31)) return GSI_ERR_UNSUPPORTED_SHAPE;
  const unsigned ctas = unsigned(a.c.heads) * p.tiles, seqs = unsigned(a.c.seqs);
  if (launch_pdl(kernel, dim3(ctas * p.splits, 1, seqs), dim3(Sh::kThreads), Sh::kSmem, s, maps, p) != cudaSuccess)
    return GSI_ERR_CUDA;
  if (p.splits == 1) return GSI_OK;
  const unsigned rows8 = unsigned(std::min<int64_t>(Sh::kTiles * kRows, max_rows * a.c.group) + 7) / 8;
  return launch_pdl(join_kernel<D>, dim3(rows8, ctas, seqs), dim3(256), 0, s, p) == cudaSuccess ? GSI_OK
                                                                                                     : GSI_ERR_CUDA;
}

template <int FMT, int HL>
gsi_status_t launch_dim(gsi_kv* kv, const KvAttnArgs& a, int64_t max_rows, cudaStream_t s) {
  switch (kv->b.head_dim) {
    case 64: return launch<FMT, 64, HL>(kv, a, max_rows, s);
    case 128: return launch<FMT, 128, HL>(kv, a, max_rows, s);
    default: return launch<FMT, 256, HL>(kv, a, max_rows, s);
  }
}

}  // namespace

// Outputs of shares and the logarithms of their sums; a cache whose sequences are
// too short to be split needs none.
size_t kv_prefill_part_bytes(const gsi_kv* kv) {
  if (kv->b.max_pages < 2 * kLeast) return 0;
  return size_t(kv->num_sms) * (kv->b.head_dim == 256 ? 1 : 2) * kRows * (kv->b.head_dim + 1) * 4;
}

gsi_status_t kv_prefill_launch(gsi_kv* kv, const KvAttnArgs& a, int64_t max_rows, cudaStream_t s) {
  if (kv->b.format == kInt8)
    return a.lse ? launch_dim<kInt8, 1>(kv, a, max_rows, s) : launch_dim<kInt8, 0>(kv, a, max_rows, s);
  return a.lse ? launch_dim<kE4m3, 1>(kv, a, max_rows, s) : launch_dim<kE4m3, 0>(kv, a, max_rows, s);
}

}  // namespace gsi
