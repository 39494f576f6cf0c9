// gsi_kv_decode.cu -- attention of few rows (a token, a handful of drafted
// tokens) over the 8-bit cache.
//
// For the R = T x group query rows of a key/value head, with codes c and scales
// 2^e of K and 2^f of V:  s = q . c_k 2^e (log2 units, the logits' factor is in
// q), out = sum_j 2^(s_j) 2^(f_j) c_v,j / sum_j 2^(s_j).  The V scale joins the
// exponent: with t_j = s_j + f_j and m the running maximum of t, the weights
// w_j = 2^(t_j - m + 15) lie in (0, 2^15] whatever the scales, go to the second
// product as fp16, and the divisor sums w_j 2^(-f_j) in fp32.
//
// Each key and value is read once and used by R rows only, so HBM bandwidth
// bounds it: 2 D bytes a token and head.  The grid is one wave, and every warp
// is on its own: it takes an equal share of all units (16 to 64 tokens of a
// page of a head) of all sequences and heads, in order, so ragged lengths
// balance and no warp waits for another while data streams.  Its lane 0 keeps a
// private ring of units filled by TMA (128-byte swizzle: the fragment loads
// below are free of bank conflicts at D >= 128).  The products are warp-level
// MMAs (m16n8k16, fp16 operands -- codes of both formats are exact in fp16 --
// fp32 accumulators): the query side fills 8 columns, which a tcgen05 tile of
// 128 rows would waste.  A head that lies in one warp's share is finished
// there; pieces of the others are joined by the CTA, and what several CTAs
// share by the last of them to arrive.
//
// Measured, one token a sequence: 16 sequences of 1000 to 16001 tokens, 8 heads
// of 128, 4 query heads to each: 56 us, 5.0 TB/s (75% of a copy); two of 100003
// and 131071, 8 query heads: 86 us, 5.5 TB/s; one of 2047, 16 heads of 256: 12.4
// us, of which about 10 are a chain that does not depend on the bytes (share of
// the units, page, codes, join of the warps, arrival, join of the CTAs).  Five
// rows of 4 sequences of 4000 to 9000, 8 heads of 128, 2 query heads: 30 us.
#include <cuda.h>

#include <algorithm>

#include "gsi_internal.h"
#include "gsi_kv.cuh"
#include "gsi_kv_codes.cuh"
#include "gsi_tc_gemm.h"

namespace gsi {
namespace {

constexpr int kMostWarps = 12;  // of a CTA
constexpr int kStages = 8;      // most stages of a warp's ring
constexpr int kSeqChunk = 1024;  // sequences whose unit counts shared memory holds at a time

// Warps of a CTA (one CTA per SM), and MT x 16 tokens of a page for a unit.
template <int D, int NT>
struct Shape {
  static constexpr int kMT = D == 256 ? 1 : D == 64 && NT == 1 ? 4 : 2;
  static constexpr int kWarps = D == 256 || (D == 128 && NT == 2) ? 8 : 12;  // as registers allow
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = 16 * kMT;            // tokens
  static constexpr int kPer = kPage / kUnit;        // units of a page
  static constexpr int kBytes = 2 * kUnit * D;      // codes of a unit, K and V
};
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

struct DecMaps {
  CUtensorMap k, v;
};

struct DecArgs {
  KvAttnArgs a;
  int R;            // rows of a head: at most 8 NT
  int stages;       // of a warp's ring
  float* piece;     // [grid][warps][R][D]: output of a warp's first piece, if its share has two
  float* part;      // [grid][2][R][D]: a CTA's pieces of heads that it shares
  float* part_ml;   // [grid][2][R][2]: their maxima and sums
  uint32_t* count;  // [seqs][heads] CTAs arrived; zero between launches
  float* logits;    // [seqs][heads][R][max_pages * 64] s, or null
};

// A head as its units are numbered among all.
struct Head {
  int64_t unit0;  // its first unit
  int units, b, h;
  int first, count;  // its sequence's new rows
};

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Token (0 .. 7) of row g of an MMA's upper or lower half.  Together with the
// 128-byte swizzle this order lets eight lanes that load 16 bytes each, of two
// rows (K) or of four (V), touch every bank once.
__device__ __forceinline__ int tok(int g) { return (g & 1) ? ((g ^ 4) | 1) : g; }

// Offset of 16-byte chunk `ch` of token `t` in a staged unit of U tokens.
template <int D, int U>
__device__ __forceinline__ int chunk_at(int t, int ch) {
  if (D == 64) {
    const int line = t >> 1, c = (t & 1) * 4 + ch;
    return line * 128 + ((c ^ (line & 7)) << 4);
  }
  return (ch >> 3) * (U * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4);
}

// Rows of sequence b, its tokens with them, and its units per head (0 if it has
// no new rows): U tokens each in whole pages, fewer in the tail (bf16 takes
// twice the room; one MMA tile at most).
__host__ __device__ constexpr int tail_tokens(int U) { return U < 32 ? U / 2 : 16; }
template <int U>
__device__ __forceinline__ int units_of(const KvAttnArgs& a, int b, SeqRows& s, int& total) {
  s = seq_rows(a.r, a.c, b);
  total = min(s.len + s.count, a.c.max_pages * kPage);
  return s.count > 0 ? total / kPage * (kPage / U) + (total % kPage + tail_tokens(U) - 1) / tail_tokens(U) : 0;
}

// Lane offsets of a staged unit's fragments, in bytes.
template <int D, int U>
struct Offsets {
  int k[2][2];  // K: row g and g + 8; even and odd 64 dims
  int v[4];     // V: tokens of k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9
  __device__ __forceinline__ explicit Offsets(int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) k[i][c] = chunk_at<D, U>(tok(g) + 8 * i, D == 64 ? t : 4 * c + t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tt = tok(2 * t + (i & 1)) + (i & 2) * 4;
      v[i] = D == 64 ? chunk_at<D, U>(tt, g >> 1) + (g & 1) * 8 : chunk_at<D, U>(tt, g);
    }
  }
};

// What a warp that computes holds of a share: MT x 16 tokens of a page at a
// time against NT x 8 query rows.  HL: the query has a low part.
template <int FMT, int D, int NT, int MT, int HL>
struct Warp {
  static constexpr int kSteps = D / 16;  // MMA steps of a logit; row tiles of an output
  // the query's fragments stay in registers where there are few
  static constexpr bool kQRegs = NT == 1;
  float o[kSteps][NT][4];
  float m[NT][2], l[NT][2];
  static constexpr int U = 16 * MT;
  float qs[NT][2];       // factors of this lane's two columns' logits
  int see[NT][2];        // tokens they see
  uint2 q[kQRegs ? kSteps : 1], q_lo[kQRegs && HL ? kSteps : 1];

  // Start of a head: query fragments (in registers, or in the warp's shared
  // memory qf), factors, empty sums.  Lane (g, t) holds of row 8 n + g the dims
  // 64 c + 16 t .. + 15, as the pairs that four MMA steps take.
  __device__ __forceinline__ void begin(const DecArgs& p, const SeqRows& sq, int total, int h,
                                        unsigned char* qf, int lane) {
    const int g = lane >> 2, t = lane & 3, G = p.a.c.group;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][n][c] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + g, i = row / G;
      const bool real = row < p.R && i < sq.count;
      const int64_t at = int64_t(sq.first + i) * p.a.ldq + int64_t(h * G + row % G) * D + 16 * t;
      auto load = [&](int c16, float (&x)[16]) {
        if (!real) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        } else if (p.a.bf16) {
          const uint4* v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) + at + 64 * c16);
          float y[8];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (e % 8 == 0) bf16x8_to_f32(v[e / 8], y);
            x[e] = y[e % 8];
          }
        } else {
          const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(p.a.q) + at + 64 * c16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 y = v[e];
            x[4 * e] = y.x;
            x[4 * e + 1] = y.y;
            x[4 * e + 2] = y.z;
            x[4 * e + 3] = y.w;
          }
        }
      };
      float x[16], top = 0.f;
#pragma unroll
      for (int c16 = 0; c16 < D / 64; ++c16) {
        load(c16, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // a power of two that brings the largest to [2^13, 2^14): the high part
      // has 11 bits, the low part the next ones down to 2^-24.  Zero and
      // non-finite rows are left as they are
      const int ex = int(__float_as_uint(top) >> 23) - 126;
      const int sh = top > 0.f && ex < 129 ? min(14 - ex, 100) : 0;
      const float up = exp2_int(sh);
      const float fac = p.a.qscale * exp2_int(-sh);
      const int sees = real ? min(sq.len + i + 1, total) : 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // column 2 t + c of the logits is row 8 n + 2 t + c: lane 4 (2 t + c)
        m[n][c] = -INFINITY;
        l[n][c] = 0.f;
        qs[n][c] = __shfl_sync(0xFFFFFFFFu, fac, 4 * (2 * t + c));
        see[n][c] = __shfl_sync(0xFFFFFFFFu, sees, 4 * (2 * t + c));
      }
#pragma unroll
      for (int c16 = 0; c16 < D / 64; ++c16) {
        load(c16, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = x[4 * j + e] * up;
            hi[e] = __half2float(__float2half_rn(y));
            lo[e] = y - hi[e];
          }
          const int step = c16 * 4 + j;
          const uint2 h2 = make_uint2(pack_f16(hi[0], hi[1]), pack_f16(hi[2], hi[3]));
          const uint2 l2 = make_uint2(pack_f16(lo[0], lo[1]), pack_f16(lo[2], lo[3]));
          if (kQRegs) {
            q[kQRegs ? step : 0] = h2;
            if (HL) q_lo[kQRegs && HL ? step : 0] = l2;
          } else if (HL) {
            reinterpret_cast<uint4*>(qf)[(step * NT + n) * 32 + lane] = make_uint4(h2.x, h2.y, l2.x, l2.y);
          } else {
            reinterpret_cast<uint2*>(qf)[(step * NT + n) * 32 + lane] = h2;
          }
        }
      }
    }
  }

  // logits of one step of 16 dims
  __device__ __forceinline__ void logit_step(float (&s)[NT][4], float (&s2)[NT][4], const unsigned char* qf,
                                             int step, int lane, uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (HL) {
        uint4 x;
        if (kQRegs) {
          const uint2 h = q[kQRegs ? step : 0], l_ = q_lo[kQRegs && HL ? step : 0];
          x = make_uint4(h.x, h.y, l_.x, l_.y);
        } else {
          x = reinterpret_cast<const uint4*>(qf)[(step * NT + n) * 32 + lane];
        }
        mma_f16(s[n], a0, a1, a2, a3, x.x, x.y);
        mma_f16(s2[n], a0, a1, a2, a3, x.z, x.w);
      } else {
        const uint2 x = kQRegs ? q[kQRegs ? step : 0] : reinterpret_cast<const uint2*>(qf)[(step * NT + n) * 32 + lane];
        // two accumulators: half the chain
        if (step & 1) mma_f16(s2[n], a0, a1, a2, a3, x.x, x.y);
        else mma_f16(s[n], a0, a1, a2, a3, x.x, x.y);
      }
    }
  }

  // s (rows: tokens t_first + 16 i + tok(g), and 8 further; columns: this
  // lane's query rows) to weights: running maximum, rescale, sum; b: the
  // weights as the second product's operand.
  template <bool TAIL>
  __device__ __forceinline__ void weights(float (&s)[MT][NT][4], int t_first, float ks, float vs, int lane,
                                          float* logits, size_t lstride, uint32_t (&b)[MT][NT][2]) {
    const int t = lane & 3, at = t_first + tok(lane >> 2);
    // vs is a power of two: its exponent, and its inverse
    const float f = float(int(__float_as_uint(vs) >> 23) - 127);
    const float inv_vs = __uint_as_float((254u << 23) - __float_as_uint(vs));
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float k = ks * qs[n][c];
        // the next unit's tokens are not this one's
        const int end = TAIL ? min(see[n][c], t_first + tail_tokens(U)) : see[n][c];
        mx[n][c] = -INFINITY;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          s[i][n][c] *= k;
          s[i][n][c + 2] *= k;
          if (logits && see[n][c] > 0 && (!TAIL || i == 0)) {
            float* to = logits + (8 * n + 2 * t + c) * lstride + at + 16 * i;
            to[0] = s[i][n][c];
            if (!TAIL || tail_tokens(U) > 8) to[8] = s[i][n][c + 2];
          }
          if (at + 16 * i >= end) s[i][n][c] = -INFINITY;
          if (at + 16 * i + 8 >= end) s[i][n][c + 2] = -INFINITY;
          mx[n][c] = fmaxf(mx[n][c], fmaxf(s[i][n][c], s[i][n][c + 2]));
        }
      }
#pragma unroll
    for (int o_ = 4; o_ < 32; o_ <<= 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) mx[n][c] = fmaxf(mx[n][c], __shfl_xor_sync(0xFFFFFFFFu, mx[n][c], o_));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[n][c] = fmaxf(m[n][c], mx[n][c] + f);
        grow |= mx[n][c] > m[n][c];
      }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float hr = m[n][c] == -INFINITY ? 0.f : ex2_half(m[n][c] - mx[n][c]), r = hr * hr;
          m[n][c] = mx[n][c];
          l[n][c] = l[n][c] * hr * hr;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            o[i][n][c] *= r;
            o[i][n][c + 2] *= r;
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // a row that has seen nothing yet has m = -inf and only -inf logits
      const float off0 = m[n][0] == -INFINITY ? 0.f : f - m[n][0] + 15.f;
      const float off1 = m[n][1] == -INFINITY ? 0.f : f - m[n][1] + 15.f;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float w0 = ex2(s[i][n][0] + off0), w1 = ex2(s[i][n][1] + off1);
        const float w2 = ex2(s[i][n][2] + off0), w3 = ex2(s[i][n][3] + off1);
        sum0 += w0 + w2;
        sum1 += w1 + w3;
        b[i][n][0] = transpose_8x8(pack_f16(w0, w1));
        b[i][n][1] = transpose_8x8(pack_f16(w2, w3));
      }
      l[n][0] = fmaf(sum0, inv_vs, l[n][0]);
      l[n][1] = fmaf(sum1, inv_vs, l[n][1]);
    }
  }

  // A staged unit of codes; t_first: its first token in the sequence.
  __device__ __forceinline__ void codes(const unsigned char* kp, const Offsets<D, U>& off, const unsigned char* qf,
                                        int t_first, float ks, float vs, int lane, float* logits,
                                        size_t lstride) {
    const unsigned char* vp = kp + U * D;
    constexpr int kRow16 = 16 * (D == 64 ? 64 : 128);
    float s[MT][NT][4];
    {
      float s2[MT][NT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][n][c] = s2[i][n][c] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 r[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            r[i][e] = *reinterpret_cast<const uint4*>(kp + off.k[e][c & 1] + i * kRow16 + (c >> 1) * U * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t a0, a1, a2, a3;
            codes_f16<FMT>(j == 0 ? r[i][0].x : j == 1 ? r[i][0].y : j == 2 ? r[i][0].z : r[i][0].w, a0, a2);
            codes_f16<FMT>(j == 0 ? r[i][1].x : j == 1 ? r[i][1].y : j == 2 ? r[i][1].z : r[i][1].w, a1, a3);
            logit_step(s[i], s2[i], qf, 4 * c + j, lane, a0, a1, a2, a3);
          }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][n][c] += s2[i][n][c];
    }
    uint32_t b[MT][NT][2];
    weights<false>(s, t_first, ks, vs, lane, logits, lstride, b);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (D == 64) {
        // lane g: dims 8 g .. 8 g + 7
        uint2 r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = *reinterpret_cast<const uint2*>(vp + off.v[e] + i * kRow16);
        out_step(0, r[0].x, r[1].x, r[2].x, r[3].x, b[i]);
        out_step(2, r[0].y, r[1].y, r[2].y, r[3].y, b[i]);
      } else {
        // lane g: dims 128 hf + 16 g .. + 15
#pragma unroll
        for (int hf = 0; hf < D / 128; ++hf) {
          uint4 r[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            r[e] = *reinterpret_cast<const uint4*>(vp + off.v[e] + i * kRow16 + hf * U * 128);
          out_step(hf * 8, r[0].x, r[1].x, r[2].x, r[3].x, b[i]);
          out_step(hf * 8 + 2, r[0].y, r[1].y, r[2].y, r[3].y, b[i]);
          out_step(hf * 8 + 4, r[0].z, r[1].z, r[2].z, r[3].z, b[i]);
          out_step(hf * 8 + 6, r[0].w, r[1].w, r[2].w, r[3].w, b[i]);
        }
      }
    }
  }

  // Four dims of four tokens (a, b its neighbour in k; c, d 8 further): output
  // tiles i (dims 0, 1 of the four in rows g, g + 8) and i + 1 (2, 3).
  __device__ __forceinline__ void out_step(int i, uint32_t wa, uint32_t wb, uint32_t wc, uint32_t wd,
                                           const uint32_t (&b)[NT][2]) {
    uint32_t p0, p1, p2, p3, q0, q1, q2, q3;
    codes_f16<FMT>(__byte_perm(wa, wb, 0x5140), p0, p1);
    codes_f16<FMT>(__byte_perm(wa, wb, 0x7362), p2, p3);
    codes_f16<FMT>(__byte_perm(wc, wd, 0x5140), q0, q1);
    codes_f16<FMT>(__byte_perm(wc, wd, 0x7362), q2, q3);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma_f16(o[i][n], p0, p1, q0, q1, b[n][0], b[n][1]);
      mma_f16(o[i + 1][n], p2, p3, q2, q3, b[n][0], b[n][1]);
    }
  }

  // A staged unit of the tail: tail_tokens(U) rows of bf16, `held` of them (the others are
  // not looked at).  It fills the first tile of 16 tokens, or half of it.
  __device__ __forceinline__ void tail(const unsigned char* stage, int held, const unsigned char* qf, int t_first,
                                       float ks, float vs, int lane, float* logits, size_t lstride) {
    const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(stage);
    const __nv_bfloat16* vp = kp + tail_tokens(U) * D;
    const int g = lane >> 2, t = lane & 3;
    const float ki = __uint_as_float((254u << 23) - __float_as_uint(ks));
    const float vi = __uint_as_float((254u << 23) - __float_as_uint(vs));
    float s[MT][NT][4], s2[NT][4];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s2[n][c] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) s[i][n][c] = 0.f;
      }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 r[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int tt = tok(g) + 8 * e;
          r[e][j] = tt < held ? *reinterpret_cast<const uint4*>(kp + tt * D + 64 * c + 16 * t + 8 * j) : zero;
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 ua = r[0][j >> 1], ub = r[1][j >> 1];
        logit_step(s[0], s2, qf, 4 * c + j, lane, bf16_f16((j & 1) ? ua.z : ua.x, ki),
                   bf16_f16((j & 1) ? ub.z : ub.x, ki), bf16_f16((j & 1) ? ua.w : ua.y, ki),
                   bf16_f16((j & 1) ? ub.w : ub.y, ki));
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[0][n][c] += s2[n][c];
    uint32_t b[MT][NT][2];
    weights<true>(s, t_first, ks, vs, lane, logits, lstride, b);
    // dims as in codes(): 8 g (D = 64) or 128 hf + 16 g, eight at a time
    constexpr int kVecs = D == 64 ? 1 : D / 64;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int d0 = D == 64 ? 8 * g : 128 * (v >> 1) + 16 * g + 8 * (v & 1);
      const int i0 = D == 64 ? 0 : 8 * (v >> 1) + 4 * (v & 1);
      uint32_t w[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tt = tok(2 * t + (e & 1)) + (e & 2) * 4;
        const uint4 r = tt < held ? *reinterpret_cast<const uint4*>(vp + tt * D + d0) : zero;
        w[e][0] = bf16_f16(r.x, vi);
        w[e][1] = bf16_f16(r.y, vi);
        w[e][2] = bf16_f16(r.z, vi);
        w[e][3] = bf16_f16(r.w, vi);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5410), a1 = __byte_perm(w[0][j], w[1][j], 0x7632);
        const uint32_t a2 = __byte_perm(w[2][j], w[3][j], 0x5410), a3 = __byte_perm(w[2][j], w[3][j], 0x7632);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(o[i0 + j][n], a0, a1, a2, a3, b[0][n][0], b[0][n][1]);
      }
    }
  }

  // Dim of output tile i, row g (half 0) or g + 8 (half 1).
  static __device__ __forceinline__ int dim_of(int i, int g, int half) {
    return D == 64 ? 8 * g + 2 * i + half : 128 * (i >> 3) + 16 * g + 2 * (i & 7) + half;
  }
};

// Four dims of a row's outcome: o weighted sum and l divisor, both 2^(15 - top)
// larger.
__device__ __forceinline__ void put4(const KvAttnArgs& a, int64_t n, int hq, int D, int d, const float4& o,
                                     float l, float top) {
  const float inv = l != 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(a.out + n * a.ldo + int64_t(hq) * D + d) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (d == 0 && a.lse)
    a.lse[n * (int64_t(a.c.heads) * a.c.group) + hq] = l != 0.f ? (top - 15.f + log2f(l)) * kLn2 : -INFINITY;
}

template <int FMT, int D, int NT, int HL>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1)
    decode_kernel(const __grid_constant__ DecMaps maps, const __grid_constant__ DecArgs p) {
  using Sh = Shape<D, NT>;
  constexpr int kWarps = Sh::kWarps, kThreads = Sh::kThreads, kMT = Sh::kMT, U = Sh::kUnit, kTail = tail_tokens(U);
  constexpr int kHalf = D >= 128 ? D / 128 : 1;  // TMA boxes of a unit of K or V
  constexpr int kBox = U * D / kHalf;            // bytes of one
  constexpr bool kQRegs = Warp<FMT, D, NT, kMT, HL>::kQRegs;
  constexpr int kQ = kQRegs ? 0 : D / 16 * NT * 32 * (HL ? 16 : 8);  // bytes of a warp's query fragments
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ int s_units[kSeqChunk];
  __shared__ float s_ml[2 * kWarps][8 * NT][2];  // maximum and sum of each piece
  __shared__ Head s_head[2 * kWarps];
  __shared__ int s_place[2 * kWarps];            // a piece's place: 1 the warp's ring, 2 p.piece; 0: none
  __shared__ int s_last[2], s_first[2], s_slot[2], s_groups;
  __shared__ int s_list[2 * kWarps], s_group_of[2 * kWarps], s_start[2 * kWarps + 1];
  __shared__ float s_f[2 * kWarps][8 * NT], s_top[2 * kWarps][8 * NT];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.stages, R = p.R, H = p.a.c.heads, G = p.a.c.group, seqs = p.a.c.seqs;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* all = smem_raw + (base - smem_addr(smem_raw));
  unsigned char* ring = all + size_t(warp) * S * Sh::kBytes;
  unsigned char* qf = all + size_t(kWarps) * S * Sh::kBytes + size_t(warp) * kQ;
  uint64_t* bar = bars[warp];

  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(&bar[s], 1);
  if (lane < 2) s_place[2 * warp + lane] = 0;
  fence_mbar_init();
  pdl_launch_dependents();
  pdl_wait();

  // all units, and where this warp's share [u0, u1) begins
  int64_t n_all = 0, u0 = 0, u1 = 0, cta0 = 0, cta1 = 0, shares = 0;
  Head hd = {};
  SeqRows sq = {};
  int total = 0, blk = 0;  // blk: unit within the head
  auto split = [&]() {
    // as many shares as units if there are fewer than warps, whole CTAs
    shares = min(int64_t(gridDim.x) * kWarps, (n_all + kWarps - 1) / kWarps * kWarps);
    const int64_t w = int64_t(blockIdx.x) * kWarps + warp;
    if (w >= shares) return;
    u0 = n_all * w / shares;
    u1 = n_all * (w + 1) / shares;
    cta0 = n_all * (int64_t(blockIdx.x) * kWarps) / shares;
    cta1 = n_all * (int64_t(blockIdx.x + 1) * kWarps) / shares;
  };
  // units of sequences b0 + lane (one per lane), `at` units before them: finds u0's
  auto locate = [&](int mine, int b0, int64_t at, int64_t& next) {
    int64_t x = int64_t(mine) * H;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    next = at + __shfl_sync(0xFFFFFFFFu, x, 31);
    if (!(u0 < u1 && u0 < next)) return false;
    const int64_t end = at + x, first = end - int64_t(mine) * H;
    const int who = __ffs(__ballot_sync(0xFFFFFFFFu, first <= u0 && u0 < end)) - 1;
    const int64_t unit_b = __shfl_sync(0xFFFFFFFFu, first, who);
    hd.units = __shfl_sync(0xFFFFFFFFu, mine, who);
    hd.b = b0 + who;
    hd.h = int((u0 - unit_b) / hd.units);
    hd.unit0 = unit_b + int64_t(hd.h) * hd.units;
    blk = int(u0 - hd.unit0);
    return true;
  };
  if (seqs <= 32) {
    // every warp for itself
    SeqRows s;
    int t;
    const int mine = lane < seqs ? units_of<U>(p.a, lane, s, t) : 0;
    n_all = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) n_all += __shfl_xor_sync(0xFFFFFFFFu, n_all, o);
    n_all *= H;
    split();
    if (int64_t(blockIdx.x) * kWarps >= shares) return;
    int64_t next;
    locate(mine, 0, 0, next);
    __syncwarp();
  } else {
    for (int pass = 0; pass < 2; ++pass) {
      int64_t at = 0;
      bool found = false;
      for (int b0 = 0; b0 < seqs; b0 += kSeqChunk) {
        if (pass == 0 || seqs > kSeqChunk) {
          __syncthreads();
          for (int i = threadIdx.x; i < kSeqChunk && b0 + i < seqs; i += kThreads) {
            SeqRows s;
            int t;
            s_units[i] = units_of<U>(p.a, b0 + i, s, t);
          }
          __syncthreads();
        }
        const int n = min(kSeqChunk, seqs - b0);
        for (int i = 0; i < n && !found; i += 32) {
          int64_t next = 0;
          found = locate(i + lane < n ? s_units[i + lane] : 0, b0 + i, at, next);
          at = next;
        }
      }
      if (pass == 0) {
        n_all = at;
        split();
        if (int64_t(blockIdx.x) * kWarps >= shares) return;
      }
    }
  }

  if (u0 < u1) {
    Warp<FMT, D, NT, kMT, HL> w;
    const Offsets<D, U> off(lane);
    const size_t lstride = size_t(p.a.c.max_pages) * kPage;
    units_of<U>(p.a, hd.b, sq, total);
    // the cursor that fetches runs S units ahead of the one that computes
    int64_t fu = u0;
    Head fh = hd;
    int fblk = blk, ftotal = total, fit = 0;
    auto block_of = [&](int unit, int tot) {
      const int in_pages = tot / kPage * Sh::kPer;
      return unit < in_pages ? unit / Sh::kPer : tot / kPage;
    };
    // pages and scales of the fetching cursor's next pages, one per lane: lane i
    // has block fb0 + i of its head
    int fb0 = 0, fb1 = 0, page = -1;
    float ks = 1.f, vs = 1.f;
    // what the computing cursor needs of the units in the ring: lane s has
    // stage s's
    float r_ks = 1.f, r_vs = 1.f;
    int vs_top = 0;  // the largest of V's scales of the head so far
    int r_kind = 2;  // 0: codes, 1: tail, 2: nothing (its page is out of range)
    auto fetch = [&]() {
      if (fu >= u1) return;
      const int pb = block_of(fblk, ftotal);
      if (pb >= fb1) {
        fb0 = pb;
        const int last = block_of(int(min(int64_t(fh.units), int64_t(fblk) + (u1 - fu)) - 1), ftotal) + 1;
        fb1 = min(fb0 + 32, last);
        page = -1;
        if (fb0 + lane < fb1) {
          page = p.a.c.page_table[size_t(fh.b) * p.a.c.max_pages + fb0 + lane];
          if (page < 0 || page >= p.a.c.pages) {
            page = -1;
            atomicOr(p.a.c.status, kStatusBadPage);
          } else {
            ks = p.a.c.scale[0][size_t(page) * H + fh.h];
            vs = p.a.c.scale[1][size_t(page) * H + fh.h];
          }
        }
      }
      const int pg = __shfl_sync(0xFFFFFFFFu, page, pb - fb0);
      const bool in_pages = pb < ftotal / kPage;
      const int s = fit % S;
      if (lane == 0 && pg >= 0) {
        unsigned char* dst = ring + size_t(s) * Sh::kBytes;
        mbar_arrive_expect_tx(&bar[s], in_pages ? Sh::kBytes : kTail * D * 4);
        if (in_pages) {
          // in 128-byte lines for D = 64, else in tokens
          const int line = (pg * H + fh.h) * (D == 64 ? kPage / 2 : kPage) + (fblk % Sh::kPer) * (D == 64 ? U / 2 : U);
#pragma unroll
          for (int f = 0; f < kHalf; ++f) {
            tma_load_2d(dst + f * kBox, &maps.k, 64 * f, line, &bar[s]);
            tma_load_2d(dst + U * D + f * kBox, &maps.v, 64 * f, line, &bar[s]);
          }
        } else {
          const int row = (fblk - ftotal / kPage * Sh::kPer) * kTail;
          const size_t at = ((size_t(fh.b) * H + fh.h) * kPage + row) * D;
          bulk_g2s(dst, p.a.c.tail[0] + at, kTail * D * 2, &bar[s]);
          bulk_g2s(dst + kTail * D * 2, p.a.c.tail[1] + at, kTail * D * 2, &bar[s]);
        }
      }
      const float sk = __shfl_sync(0xFFFFFFFFu, ks, pb - fb0), sv = __shfl_sync(0xFFFFFFFFu, vs, pb - fb0);
      if (fblk == 0) vs_top = 0;
      const int vs_bits = pg < 0 ? 0 : clip_scale(__float_as_int(sv), vs_top);
      if (lane == s) {
        r_ks = sk;
        r_vs = __int_as_float(vs_bits);
        r_kind = pg < 0 ? 2 : in_pages ? 0 : 1;
      }
      if (fblk == 0 || fu == u0) {
        // the head's query rows are wanted S units from now
        SeqRows s2;
        int t2;
        units_of<U>(p.a, fh.b, s2, t2);
        const int line = (p.a.bf16 ? 64 : 32) * lane, row = line / D;  // 128-byte lines of the rows
        for (int r = row, d = line % D; r < R && r / G < s2.count; r += (p.a.bf16 ? 2048 : 1024) / D) {
          const int64_t at = int64_t(s2.first + r / G) * p.a.ldq + int64_t(fh.h * G + r % G) * D + d;
          asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const char*>(p.a.q) + at * (p.a.bf16 ? 2 : 4)));
        }
      }
      ++fit;
      ++fu;
      if (++fblk == fh.units && fu < u1) {
        fblk = 0;
        fb0 = fb1 = 0;
        fh.unit0 += fh.units;
        if (++fh.h == H) {
          fh.h = 0;
          SeqRows s2;
          do {
            ++fh.b;
            fh.units = units_of<U>(p.a, fh.b, s2, ftotal);
          } while (fh.units == 0 && fh.b + 1 < seqs);
        }
      }
    };
    for (int i = 0; i < S; ++i) fetch();

    // a stage's barrier completes a phase only where there is data: bit s of `phase` is
    // the parity that stage s waits for next
    uint32_t phase = 0;
    int it = 0, pieces = 0;
    bool ok = true;
    for (int64_t u = u0; ok && u < u1;) {
      const int cnt = int(min(u1 - u, int64_t(hd.units - blk)));
      w.begin(p, sq, total, hd.h, qf, lane);
      __syncwarp();
      float* logits = p.logits ? p.logits + (size_t(hd.b) * H + hd.h) * R * lstride : nullptr;
      for (int i = 0; i < cnt; ++i, ++it) {
        const int s = it % S;
        const int kind = __shfl_sync(0xFFFFFFFFu, r_kind, s);
        const float k0 = __shfl_sync(0xFFFFFFFFu, r_ks, s), v0 = __shfl_sync(0xFFFFFFFFu, r_vs, s);
        if (kind < 2) {
          ok = mbar_wait_bounded(&bar[s], (phase >> s) & 1, p.a.c.status);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          phase ^= 1u << s;
        }
        const unsigned char* stage = ring + size_t(s) * Sh::kBytes;
        if (kind == 0) {
          w.codes(stage, off, qf, (blk + i) * U, k0, v0, lane, logits, lstride);
        } else if (kind == 1) {
          const int row = (blk + i - total / kPage * Sh::kPer) * kTail;
          w.tail(stage, min(kTail, total % kPage - row), qf, total / kPage * kPage + row, k0, v0, lane, logits,
                 lstride);
        }
        __syncwarp();  // the stage is read
        fetch();
      }
      if (!ok) break;
      // a whole head is finished here; a piece is left for the join.  Two at
      // most are: the share's first and last
      const bool whole = cnt == hd.units;
      const int slot = 2 * warp + pieces;
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = w.l[n][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
          const int row = 8 * n + 2 * t + e, i = row / G;
          if (row >= R || i >= sq.count) continue;
          if (whole) {
            const int64_t r = sq.first + i;
            const int hq = hd.h * G + row % G;
            const float inv = l != 0.f ? 1.f / l : 0.f;
            __nv_bfloat16* out = p.a.out + r * p.a.ldo + int64_t(hq) * D;
#pragma unroll
            for (int k = 0; k < w.kSteps; ++k)
              *reinterpret_cast<uint32_t*>(out + w.dim_of(k, g, 0)) =
                  pack_bf16(w.o[k][n][e] * inv, w.o[k][n][e + 2] * inv);
            if (g == 0 && p.a.lse)
              p.a.lse[r * (int64_t(H) * G) + hq] =
                  l != 0.f ? (w.m[n][e] - 15.f + log2f(l)) * kLn2 : -INFINITY;
          } else {
            // the share's last piece in the warp's own ring, which is read and
            // idle by then; a first one in global memory
            float* to = u + cnt == u1 ? reinterpret_cast<float*>(ring) + row * D
                                      : p.piece + ((size_t(blockIdx.x) * kWarps + warp) * R + row) * D;
#pragma unroll
            for (int k = 0; k < w.kSteps; ++k)
              *reinterpret_cast<float2*>(to + w.dim_of(k, g, 0)) = make_float2(w.o[k][n][e], w.o[k][n][e + 2]);
            if (g == 0) {
              s_ml[slot][row][0] = w.m[n][e];
              s_ml[slot][row][1] = l;
            }
          }
        }
      if (!whole) {
        if (lane == 0) {
          hd.first = sq.first;
          hd.count = sq.count;
          s_head[slot] = hd;
          s_place[slot] = u + cnt == u1 ? 1 : 2;
        }
        ++pieces;
      }
      u += cnt;
      blk = 0;
      if (u < u1) {
        hd.unit0 += hd.units;
        if (++hd.h == H) {
          hd.h = 0;
          do {
            ++hd.b;
            hd.units = units_of<U>(p.a, hd.b, sq, total);
          } while (hd.units == 0 && hd.b + 1 < seqs);
        }
      }
    }
    if (!ok && lane == 0) {
      // no copy may still be writing when the CTA ends
      for (int j = it; j < fit; ++j) {
        const int s = j % S;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&bar[s], (phase >> s) & 1) && globaltimer_ns() - t0 < kWaitLimitNs / 100) {
        }
      }
    }
  }

  // ---- join ------------------------------------------------------------------
  // The list of pieces, in order of units: those of one head are neighbours, a
  // group.  Warp 0 lists the groups, lane j from piece j; then a thread per piece
  // and row finds its factor, and one per group, row and four dims the sums.
  __syncthreads();
  const int tid = threadIdx.x;
  if (warp == 0) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const int64_t unit0 = lane < 2 * kWarps && s_place[lane] ? s_head[lane].unit0 : -1;
    const uint32_t valid = __ballot_sync(kAll, unit0 >= 0);
    const uint32_t below = valid & ((1u << lane) - 1);
    const int64_t prev = __shfl_sync(kAll, unit0, below ? 31 - __clz(below) : 0);
    const bool starts = unit0 >= 0 && (below == 0 || prev != unit0);
    const uint32_t all_starts = __ballot_sync(kAll, starts);
    const int at = __popc(below);  // place in the list without gaps
    if (unit0 >= 0) s_list[at] = lane;
    const int gi = __popc(all_starts & ((2u << lane) - 1)) - 1;
    if (unit0 >= 0) s_group_of[at] = gi;
    if (starts) s_start[gi] = at;
    if (lane == 0) {
      s_groups = __popc(all_starts);
      s_start[__popc(all_starts)] = __popc(valid);
    }
  }
  __syncthreads();
  const int groups = s_groups;
  if (groups == 0) return;
  const int pieces = s_start[groups];
  for (int x = tid; x < pieces * R; x += kThreads) {
    const int at = x / R, row = x % R, gi = s_group_of[at];
    float top = -INFINITY;
    for (int k = s_start[gi]; k < s_start[gi + 1]; ++k) top = fmaxf(top, s_ml[s_list[k]][row][0]);
    const float m = s_ml[s_list[at]][row][0];
    const float hf = m == -INFINITY ? 0.f : ex2_half(m - top);
    s_f[at][row] = hf * hf;
    s_ml[s_list[at]][row][1] = s_ml[s_list[at]][row][1] * hf * hf;
    if (at == s_start[gi]) s_top[gi][row] = top;
  }
  __syncthreads();
  // a head that reaches beyond this CTA: its first group, or its last
  auto shared_head = [&](const Head& h) { return h.unit0 < cta0 || h.unit0 + h.units > cta1; };
  constexpr int kD4 = D / 4;
  for (int x = tid; x < groups * R * kD4; x += kThreads) {
    const int d = x % kD4, row = x / kD4 % R, gi = x / (kD4 * R);
    const int k0 = s_start[gi], k1 = s_start[gi + 1], last = s_list[k1 - 1];
    const Head h = s_head[last];
    const int i = row / G;
    if (i >= h.count) continue;
    // only a group's last piece may lie in global memory: the first of two of
    // its warp's.  The others are in their warps' rings
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool far = s_place[last] == 2;
    if (far)
      o = __ldcg(reinterpret_cast<const float4*>(
                     p.piece + ((size_t(blockIdx.x) * kWarps + last / 2) * R + row) * D) + d);
    float l = far ? s_ml[last][row][1] : 0.f;
    const float fl = far ? s_f[k1 - 1][row] : 0.f;
    o.x *= fl; o.y *= fl; o.z *= fl; o.w *= fl;
    for (int k = k0; k < k1 - far; ++k) {
      const int pc = s_list[k];
      const float f = s_f[k][row];
      const float4 v = reinterpret_cast<const float4*>(all + size_t(pc / 2) * S * Sh::kBytes)[row * kD4 + d];
      l += s_ml[pc][row][1];
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    const float top = s_top[gi][row];
    if (!shared_head(h)) {
      put4(p.a, h.first + i, h.h * G + row % G, D, 4 * d, o, l, top);
    } else {
      // slot 0: the head lies at the CTA's start; 1: it begins later
      const size_t at = (size_t(blockIdx.x) * 2 + (h.unit0 > cta0 ? 1 : 0)) * R + row;
      reinterpret_cast<float4*>(p.part + at * D)[d] = o;
      if (d == 0) {
        p.part_ml[2 * at] = top;
        p.part_ml[2 * at + 1] = l;
      }
    }
  }
  // heads shared with other CTAs: the last CTA to arrive finishes them
  if (tid < 2) {
    // the first group's head and the last one's
    const Head h = s_head[s_list[tid == 0 ? 0 : s_start[groups - 1]]];
    s_last[tid] = 0;
    if ((tid == 0 || groups > 1) && shared_head(h)) {
      const int c0 = int(((h.unit0 + 1) * shares - 1) / n_all / kWarps);
      s_last[tid] = int(((h.unit0 + h.units) * shares - 1) / n_all / kWarps) - c0 + 1;
      s_first[tid] = c0;
      // the first CTA may have it as its last piece; every other as its first
      s_slot[tid] = n_all * (int64_t(c0) * kWarps) / shares < h.unit0 ? 1 : 0;
    }
  }
  // (the barrier and the release of the atomic order every thread's stores before
  // it; its acquire and the barrier order them before every thread's loads)
  __syncthreads();
  if (tid < 2 && s_last[tid]) {
    const Head& h = s_head[s_list[tid == 0 ? 0 : s_start[groups - 1]]];
    uint32_t* cnt = p.count + size_t(h.b) * H + h.h;
    if (atom_add_acqrel_gpu(cnt, 1u) == uint32_t(s_last[tid] - 1)) *cnt = 0;
    else s_last[tid] = 0;
  }
  __syncthreads();
  // (both heads in one loop: a CTA is often the last of two)
  const int k_lo = s_last[0] ? 0 : 1, k_hi = s_last[1] ? 2 : 1;
  for (int x = tid; x < (k_hi - k_lo) * R * kD4; x += kThreads) {
    const int rk = x / kD4, d = x % kD4, k = k_lo + (rk >= R ? 1 : 0), row = rk - (k - k_lo) * R, i = row / G;
    const int n = s_last[k], c0 = s_first[k], slot0 = s_slot[k];
    const Head& h = s_head[s_list[k == 0 ? 0 : s_start[groups - 1]]];
    if (i >= h.count) continue;
    float top = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kN = 10;  // CTAs at a time: their loads are in flight together
    for (int e0 = 0; e0 < n; e0 += kN) {
      float2 ml[kN];
      float4 v[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int c = e0 + e;
        const size_t at = (size_t(c0 + c) * 2 + (c == 0 ? slot0 : 0)) * R + row;
        ml[e] = c < n ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at) : make_float2(-INFINITY, 0.f);
        v[e] = c < n ? __ldcg(reinterpret_cast<const float4*>(p.part + at * D) + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mx = top;
#pragma unroll
      for (int e = 0; e < kN; ++e) mx = fmaxf(mx, ml[e].x);
      const float h0 = top == -INFINITY ? 0.f : ex2_half(top - mx), f0 = h0 * h0;
      l = l * h0 * h0;
      o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
      top = mx;
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float hf = ml[e].x == -INFINITY ? 0.f : ex2_half(ml[e].x - mx), f = hf * hf;
        l = fmaf(ml[e].y * hf, hf, l);
        o.x = fmaf(v[e].x, f, o.x);
        o.y = fmaf(v[e].y, f, o.y);
        o.z = fmaf(v[e].z, f, o.z);
        o.w = fmaf(v[e].w, f, o.w);
      }
    }
    put4(p.a, h.first + i, h.h * G + row % G, D, 4 * d, o, l, top);
  }
}

// score[token] += sum over a head's rows of 2^(s - lse), rows in order; four
// neighbouring tokens a thread.  Bound by the logits and scores it reads and
// writes (in L2, the logits just written).
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(KvAttnArgs a, const float* logits, int R) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, H = a.c.heads, G = a.c.group;
  const SeqRows sq = seq_rows(a.r, a.c, b);
  if (sq.count == 0) return;
  const int total = min(sq.len + sq.count, a.c.max_pages * kPage);
  const size_t stride = size_t(a.c.max_pages) * kPage;
  const float* from = logits + (size_t(b) * H + h) * R * stride;
  for (int t = (blockIdx.x * kWeightThreads + threadIdx.x) * 4; t < total; t += gridDim.x * kWeightThreads * 4) {
    const int p = page_of(a.c, b, t / kPage);
    if (p < 0) continue;
    float4* score = reinterpret_cast<float4*>(a.c.score + (size_t(p) * H + h) * kPage + t % kPage);
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int row = 0; row < R; ++row) {
      const int i = row / G;
      if (i >= sq.count) break;
      const float4 s = *reinterpret_cast<const float4*>(from + row * stride + t);
      const float lse = a.lse[size_t(sq.first + i) * (H * G) + h * G + row % G] * kLog2e;
      const int see = min(sq.len + i + 1, total) - t;
      if (see > 0) w.x += ex2(s.x - lse);
      if (see > 1) w.y += ex2(s.y - lse);
      if (see > 2) w.z += ex2(s.z - lse);
      if (see > 3) w.w += ex2(s.w - lse);
    }
    const float4 old = *score;
    const int n = total - t;  // slots beyond the sequence's end keep what they hold
    *score = make_float4(old.x + w.x, n > 1 ? old.y + w.y : old.y, n > 2 ? old.z + w.z : old.z,
                         n > 3 ? old.w + w.w : old.w);
  }
}

template <int FMT, int D, int NT, int HL>
gsi_status_t launch_as(gsi_kv* kv, DecArgs p, cudaStream_t s) {
  using Sh = Shape<D, NT>;
  using W = Warp<FMT, D, NT, Sh::kMT, HL>;
  const size_t q = W::kQRegs ? 0 : size_t(D / 16) * NT * 32 * (HL ? 16 : 8) * Sh::kWarps;
  const size_t room = 212 * 1024 - 1024 - q;  // static shared memory takes up to 13 KB
  p.stages = int(std::min<size_t>(kStages, room / (size_t(Sh::kWarps) * Sh::kBytes)));
  const size_t smem = 1024 + q + size_t(p.stages) * Sh::kWarps * Sh::kBytes;
  auto kernel = decode_kernel<FMT, D, NT, HL>;
  static std::atomic<uint64_t> ready{0};  // devices that allow the kernel its shared memory
  if (!allow_smem(kernel, smem, kv->device, ready)) return GSI_ERR_CUDA;
  DecMaps maps;
  const int map = Sh::kMT == 4 ? 4 : Sh::kMT == 2 ? 2 : 0;
  maps.k = *reinterpret_cast<const CUtensorMap*>(kv->tmaps[map]);
  maps.v = *reinterpret_cast<const CUtensorMap*>(kv->tmaps[map + 1]);
  return launch_pdl(kernel, dim3(unsigned(kv->num_sms)), dim3(Sh::kThreads), smem, s, maps, p) == cudaSuccess
             ? GSI_OK
             : GSI_ERR_CUDA;
}

template <int FMT, int D, int NT>
gsi_status_t launch(gsi_kv* kv, const DecArgs& p, cudaStream_t s) {
  return p.a.lse ? launch_as<FMT, D, NT, 1>(kv, p, s) : launch_as<FMT, D, NT, 0>(kv, p, s);
}

template <int FMT>
gsi_status_t launch_dim(gsi_kv* kv, const DecArgs& p, cudaStream_t s) {
  switch (kv->b.head_dim) {
    case 64: return p.R <= 8 ? launch<FMT, 64, 1>(kv, p, s) : launch<FMT, 64, 2>(kv, p, s);
    case 128: return p.R <= 8 ? launch<FMT, 128, 1>(kv, p, s) : launch<FMT, 128, 2>(kv, p, s);
    default: return launch<FMT, 256, 1>(kv, p, s);
  }
}

}  // namespace

bool kv_decode_maps(gsi_kv* kv) {
  const int D = kv->b.head_dim;
  const uint64_t lines = uint64_t(kv->b.pages) * kv->b.heads * (D == 64 ? kPage / 2 : kPage);
  // codes as 2-byte elements, 128-byte boxes of 16, 32 or 64 tokens
  for (int i = 0; i < 6; ++i)
    if (!tma_encode_bf16_2d(kv->tmaps[i], i & 1 ? kv->b.v_pages : kv->b.k_pages, lines,
                            uint64_t(std::max(D, 128) / 2), (16u << (i / 2)) / (D == 64 ? 2 : 1), 64))
      return false;
  return true;
}

// Two column tiles of an output of 256 dims do not fit a thread's registers.
int kv_decode_rows(const gsi_kv* kv) { return kv->b.head_dim == 256 ? 8 : kDecodeRows; }

// Outputs of pieces: one per warp, and two per CTA with their maxima and sums.
size_t kv_decode_part_bytes(const gsi_kv* kv) {
  const size_t rows = size_t(kv->num_sms) * kv_decode_rows(kv);
  return rows * 4 * (kMostWarps * kv->b.head_dim + 2 * (kv->b.head_dim + 2));
}

gsi_status_t kv_decode_launch(gsi_kv* kv, const KvAttnArgs& a, int R, int accumulate, cudaStream_t s) {
  DecArgs p;
  p.a = a;
  p.R = R;
  p.stages = 0;
  p.piece = kv->part;
  p.part = p.piece + size_t(kv->num_sms) * kMostWarps * R * kv->b.head_dim;
  p.part_ml = p.part + size_t(kv->num_sms) * 2 * R * kv->b.head_dim;
  p.count = kv->count;
  p.logits = accumulate ? kv->logits : nullptr;
  const gsi_status_t st = kv->b.format == kInt8 ? launch_dim<kInt8>(kv, p, s) : launch_dim<kE4m3>(kv, p, s);
  if (st != GSI_OK || !accumulate) return st;
  const int gx = std::min((a.c.max_pages * kPage + 4 * kWeightThreads - 1) / (4 * kWeightThreads), 1024);
  return launch_pdl(weights_kernel, dim3(unsigned(gx), unsigned(a.c.heads), unsigned(a.c.seqs)), dim3(kWeightThreads), 0,
                    s, a, kv->logits, R) == cudaSuccess ? GSI_OK : GSI_ERR_CUDA;
}

}  // namespace gsi
