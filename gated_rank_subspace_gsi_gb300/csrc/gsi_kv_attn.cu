// gsi_kv_attn.cu -- which kernel takes a call of gsi_kv_attention (gsi.h), and the
// accumulation of each token's weight over many rows.
//
// score[token] += sum over rows of 2^(s - lse), s the logits, which are computed
// again: S^T = C_k Q^T by warp-level MMAs.  A warp keeps the fp16 fragments of its
// 16 or 32 tokens in registers and meets all rows that see them, 64 at a time,
// which the CTA lays out as fragments of a high and a low fp16 part (the logits
// have to be as exact as fp32's: their errors are not averaged out where one row
// weighs most).  Rows in order: the sums do not depend on timing.  Bound by the
// warp-level MMAs (4 D flops a row and token for the two parts).  Measured: 2000
// rows over 4049 tokens, 16 heads of 256: 542 us (beside 187 of the attention with
// both parts of q), their pipe busy 74% on the fullest SM, 47% on average; a thread
// per token in fp32 took 2.2 ms.
//
// Few heads with many rows would leave most SMs idle: the rows are then shared by
// CTAs, whose sums a second launch adds in order (3 sequences of 958 to 1210 rows,
// one head of 256, 7 query heads: 136 us with the attention, with neither pass shared
// 1125).  Blocks are counted over max_pages: a cache with far more room than tokens
// launches CTAs that find nothing to do, and shares no rows.
#include <algorithm>

#include "gsi_kv.cuh"
#include "gsi_kv_codes.cuh"

namespace gsi {
namespace {

constexpr int kTiles = 8, kRowsAt = 8 * kTiles;  // rows at a time, by 8

// 256 tokens to a CTA: 16 a warp at D = 256, whose fragments take 64 registers
template <int D>
constexpr int weight_warps() { return D == 256 ? 16 : 8; }

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int FMT, int D>
__global__ void __launch_bounds__(32 * weight_warps<D>(), D == 256 ? 1 : 2) weight_kernel(KvAttnArgs a, int splits, float* part) {
  constexpr int kWarps = weight_warps<D>(), kMT = D == 256 ? 1 : 2, kSteps = D / 16, kTok = 16 * kMT;
  constexpr int kLog = D == 64 ? 6 : D == 128 ? 7 : 8;
  extern __shared__ uint4 s_frag[];  // [kSteps][kTiles][32], then the next rows as they are
  __shared__ float s_k[kRowsAt], s_lse[kRowsAt];
  __shared__ int s_see[kRowsAt];
  // of the rows that follow
  __shared__ int64_t s_at[kRowsAt];
  __shared__ float s_next_lse[kRowsAt];
  __shared__ int s_next_see[kRowsAt];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, H = a.c.heads, G = a.c.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const SeqRows sq = seq_rows(a.r, a.c, b);
  const int total = min(sq.len + sq.count, a.c.max_pages * kPage), whole = total / kPage;
  const int all = min(sq.count, a.r.max_rows) * G;
  // with splits, a CTA takes a share of the rows that see its block of tokens
  const int split = blockIdx.x % splits, blocks = gridDim.x / splits;
  for (int base = blockIdx.x / splits * (kWarps * kTok); base < total && all > 0; base += blocks * (kWarps * kTok)) {
    const int r_first = max(0, base - sq.len) * G / 8 * 8;
    const int share = (max(0, all - r_first + kRowsAt - 1) / kRowsAt + splits - 1) / splits * kRowsAt;
    const int R = min(all, r_first + (split + 1) * share);
    // this warp's tokens, all in one page
    const int t0 = base + warp * kTok, blk = t0 / kPage;
    const int page = t0 < total ? page_of(a.c, b, blk) : -1;
    float ks = 1.f, w[kMT][2] = {};
    uint32_t k[kMT][kSteps][4];
    if (page >= 0) {
      const size_t ph = size_t(page) * H + h;
      ks = a.c.scale[0][ph];
      const float inv = __uint_as_float((254u << 23) - __float_as_uint(ks));
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int row = t0 % kPage + 16 * i + g;  // and 8 further
          if (blk < whole) {
            const uint8_t* src = a.c.codes[0] + (ph * kPage + row) * D + 64 * c + 16 * t;
            const uint4 x = ld_once_v4(src), y = ld_once_v4(src + 8 * D);
            const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              codes_f16<FMT>(wx[j], k[i][4 * c + j][0], k[i][4 * c + j][2]);
              codes_f16<FMT>(wy[j], k[i][4 * c + j][1], k[i][4 * c + j][3]);
            }
          } else {
            const __nv_bfloat16* src = a.c.tail[0] + ((size_t(b) * H + h) * kPage + row) * D + 64 * c + 16 * t;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool held = row + 8 * e < total - whole * kPage;
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (held) x = reinterpret_cast<const uint4*>(src + 8 * e * D)[v];
                k[i][4 * c + 2 * v][e] = bf16_f16(x.x, inv);
                k[i][4 * c + 2 * v][e + 2] = bf16_f16(x.y, inv);
                k[i][4 * c + 2 * v + 1][e] = bf16_f16(x.z, inv);
                k[i][4 * c + 2 * v + 1][e + 2] = bf16_f16(x.w, inv);
              }
            }
          }
        }
    }
    // Rows from the first that sees a token of the CTA.  The next 64 are on their
    // way while the MMAs of these run; a row takes 16 bytes more than it has, so
    // that the eight rows a warp reads at once lie in different banks.
    const int es = a.bf16 ? 2 : 4, pitch = D * es + 16, shift = a.bf16 ? kLog - 3 : kLog - 2;
    char* raw = reinterpret_cast<char*>(s_frag + kSteps * kTiles * 32);
    auto place = [&](int r0) {  // where the rows from r0 on lie, and up to which token they see
      const int row = r0 + int(threadIdx.x), i = row / G, hq = h * G + row - i * G;
      if (threadIdx.x < kRowsAt) {
        s_at[threadIdx.x] = row < R ? (int64_t(sq.first + i) * a.ldq + int64_t(hq) * D) * es : -1;
        s_next_see[threadIdx.x] = row < R ? min(sq.len + i + 1, total) : 0;
        if (row < R) cp_async_4(&s_next_lse[threadIdx.x], a.lse + size_t(sq.first + i) * (H * G) + hq);
      }
    };
    auto fetch = [&] {
      for (int x = threadIdx.x; x < kRowsAt << shift; x += 32 * kWarps) {
        const int n = x >> shift, part = x - (n << shift);
        const int64_t at = s_at[n];
        if (at >= 0) cp_async_16(raw + n * pitch + 16 * part, static_cast<const char*>(a.q) + at + 16 * part);
      }
      cp_async_commit();
    };
    __syncthreads();  // the last block's reads
    int r0 = r_first + split * share;
    place(r0);
    __syncthreads();
    fetch();
    for (; r0 < R; r0 += kRowsAt) {
      cp_async_wait();
      __syncthreads();
      {
        // fragments of row 8 n + g: lane (g, t) holds dims 64 c + 16 t .. + 15
        const int n = warp % kTiles;
        const bool real = r0 + 8 * n + g < R;
        const char* src = raw + (8 * n + g) * pitch + 16 * t * es;
        auto load = [&](int c, float (&x)[16]) {
          if (!real) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
          } else if (a.bf16) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (e % 8 == 0) bf16x8_to_f32(reinterpret_cast<const uint4*>(src + 128 * c)[e / 8], y);
              x[e] = y[e % 8];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 y = reinterpret_cast<const float4*>(src + 256 * c)[e];
              x[4 * e] = y.x;
              x[4 * e + 1] = y.y;
              x[4 * e + 2] = y.z;
              x[4 * e + 3] = y.w;
            }
          }
        };
        float x[16], top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          load(c, x);
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // the largest in [2^13, 2^14), as in the attention itself
        const int ex = int(__float_as_uint(top) >> 23) - 126;
        const int sh = top > 0.f && ex < 129 ? min(14 - ex, 100) : 0;
        const float up = exp2_int(sh);
        if (t == 0 && warp < kTiles) {
          s_k[8 * n + g] = a.qscale * exp2_int(-sh);
          s_lse[8 * n + g] = real ? s_next_lse[8 * n + g] * 1.4426950408889634f : 0.f;
          s_see[8 * n + g] = s_next_see[8 * n + g];
        }
        constexpr int kHalves = kWarps / kTiles;  // warps that share the dims of a row
#pragma unroll
        for (int cc = 0; cc < D / 64 / kHalves; ++cc) {
          const int c = warp / kTiles * (D / 64 / kHalves) + cc;
          load(c, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = x[4 * j + e] * up;
              hi[e] = __half2float(__float2half_rn(y));
              lo[e] = y - hi[e];
            }
            s_frag[((4 * c + j) * kTiles + n) * 32 + lane] =
                make_uint4(pack_f16(hi[0], hi[1]), pack_f16(hi[2], hi[3]), pack_f16(lo[0], lo[1]),
                           pack_f16(lo[2], lo[3]));
          }
        }
      }
      __syncthreads();
      place(r0 + kRowsAt);
      __syncthreads();
      fetch();
      if (page < 0) continue;
#pragma unroll 1
      for (int n = 0; n < kTiles && r0 + 8 * n < R; ++n) {
        // the last row sees most
        if (s_see[min(8 * n + 7, R - 1 - r0)] <= t0) continue;
        float hi[kMT][4] = {}, lo[kMT][4] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint4 q = s_frag[(s * kTiles + n) * 32 + lane];
#pragma unroll
          for (int i = 0; i < kMT; ++i) {
            mma_f16(hi[i], k[i][s][0], k[i][s][1], k[i][s][2], k[i][s][3], q.x, q.y);
            mma_f16(lo[i], k[i][s][0], k[i][s][1], k[i][s][2], k[i][s][3], q.z, q.w);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = 8 * n + 2 * t + c;
          const float f = ks * s_k[row], lse = s_lse[row];
          const int see = s_see[row] - t0 - g;
#pragma unroll
          for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (16 * i + 8 * e < see) w[i][e] += ex2((hi[i][c + 2 * e] + lo[i][c + 2 * e]) * f - lse);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = w[i][e];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
        const int tok = t0 + 16 * i + 8 * e + g;
        if (t != 0 || tok >= total) continue;
        if (splits > 1)
          part[((size_t(b) * H + h) * splits + split) * (size_t(blocks) * (kWarps * kTok)) + tok] = x;
        else if (page >= 0)
          a.c.score[(size_t(page) * H + h) * kPage + tok % kPage] += x;
      }
    cp_async_wait();
  }
}

// The shares' sums, in order.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) share_sum_kernel(KvAttnArgs a, int splits, int room, const float* part) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, tok = blockIdx.x * kSumThreads + threadIdx.x;
  const SeqRows sq = seq_rows(a.r, a.c, b);
  if (sq.count == 0 || tok >= min(sq.len + sq.count, a.c.max_pages * kPage)) return;
  const int page = page_of(a.c, b, tok / kPage);
  if (page < 0) return;
  const float* from = part + (size_t(b) * a.c.heads + h) * splits * room + tok;
  float x = 0.f;
#pragma unroll 8
  for (int s = 0; s < splits; ++s) x += from[size_t(s) * room];
  a.c.score[(size_t(page) * a.c.heads + h) * kPage + tok % kPage] += x;
}

template <int FMT, int D>
gsi_status_t launch_weights(gsi_kv* kv, const KvAttnArgs& a, cudaStream_t s) {
  constexpr int kWarps = weight_warps<D>(), kTokens = kWarps * (D == 256 ? 16 : 32);
  constexpr int kFrag = D / 16 * kTiles * 32 * 16;
  const size_t smem = kFrag + kRowsAt * (D * (a.bf16 ? 2 : 4) + 16);
  static std::atomic<uint64_t> ready{0};  // devices that allow the kernel its shared memory
  if (!allow_smem(weight_kernel<FMT, D>, kFrag + kRowsAt * (D * 4 + 16), kv->device, ready)) return GSI_ERR_CUDA;
  const int64_t gx = (int64_t(a.c.max_pages) * kPage + kTokens - 1) / kTokens;
  // Few blocks of tokens with many rows: the rows are shared by CTAs too, two to an
  // SM in all (their sums take kTokens floats each: less than the decode kernel's part)
  const int64_t ctas = gx * a.c.heads * a.c.seqs, chunks = (int64_t(a.r.max_rows) * a.c.group + kRowsAt - 1) / kRowsAt;
  const int64_t most = std::min<int64_t>(2 * kv->num_sms / ctas, chunks / 2);
  const int splits = int(std::max<int64_t>(1, most));
  const unsigned blocks = unsigned(std::min<int64_t>(gx, 2048)), H = unsigned(a.c.heads), seqs = unsigned(a.c.seqs);
  if (launch_pdl(weight_kernel<FMT, D>, dim3(blocks * splits, H, seqs), dim3(32 * kWarps), smem, s, a, splits,
                 kv->part) != cudaSuccess)
    return GSI_ERR_CUDA;
  if (splits == 1) return GSI_OK;
  static_assert(kTokens == kSumThreads, "a CTA of the sums per block of tokens");
  return launch_pdl(share_sum_kernel, dim3(blocks, H, seqs), dim3(kSumThreads), 0, s, a, splits, int(blocks) * kTokens,
                    static_cast<const float*>(kv->part)) == cudaSuccess ? GSI_OK : GSI_ERR_CUDA;
}

}  // namespace

gsi_status_t kv_attn_launch(gsi_kv* kv, const KvAttnArgs& a, int64_t max_rows, int accumulate,
                            cudaStream_t s) {
  // few rows: the cache's bytes bound the call, and the kernel made for that
  // reads them once (its logits for the weights have room for one new row)
  const int64_t R = max_rows * a.c.group;
  const bool few = R <= kv_decode_rows(kv);
  if (few && (!accumulate || max_rows <= 1)) return kv_decode_launch(kv, a, int(R), accumulate, s);
  const gsi_status_t st =
      few ? kv_decode_launch(kv, a, int(R), 0, s) : kv_prefill_launch(kv, a, max_rows, s);
  if (st != GSI_OK || !accumulate) return st;
  const bool i8 = kv->b.format == kInt8;
  switch (kv->b.head_dim) {
    case 64: return i8 ? launch_weights<kInt8, 64>(kv, a, s) : launch_weights<kE4m3, 64>(kv, a, s);
    case 128: return i8 ? launch_weights<kInt8, 128>(kv, a, s) : launch_weights<kE4m3, 128>(kv, a, s);
    default: return i8 ? launch_weights<kInt8, 256>(kv, a, s) : launch_weights<kE4m3, 256>(kv, a, s);
  }
}

}  // namespace gsi
