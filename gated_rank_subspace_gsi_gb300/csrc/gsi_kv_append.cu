// gsi_kv_append.cu -- new rows into the 8-bit key/value cache.
//
// A block of 64 tokens of one head takes the scale 2^e that covers its rows
// (gsi.h) and its codes x 2^-e.  The rows of the block still filling stay in
// bf16 in the tail, and its scale is kept current: e is a maximum over rows, so
// adding rows needs the old e only.  Work is bound by the bytes of the new
// rows; a CTA takes one block of one head of K or of V, holds its 64 x D values
// in registers between the maximum and the codes, and so reads each once.
// Measured: three prompts of 701 to 4096 rows, 32 heads of 128, fp32: 54 us,
// 5.5 TB/s (82% of a copy); one row of 128 sequences, 8 heads of 128: 5.5 us, which
// is launch and the chain length, page, scale.
#include "gsi_kv.cuh"

namespace gsi {
namespace {

struct AppendArgs {
  KvView c;
  KvRows r;
  const void* x[2];  // K, V rows
  int64_t ld[2];
  int bf16;
};

// Maximum of v over the CTA, in every thread.
template <int kThreads>
__device__ __forceinline__ float cta_max(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = fmaxf(v, s_red[w]);
  return v;
}

template <int FMT, int D, int kThreads>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  constexpr int kV = D / 8;                       // 16-byte vectors of a row of bf16
  constexpr int kPer = kPage * kV / kThreads;     // vectors of a block per thread
  __shared__ float s_red[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, b = blockIdx.z;
  const SeqRows q = seq_rows(a.r, a.c, b);
  if (q.count == 0) return;
  const int r0 = q.len % kPage, end = r0 + q.count;
  const int blk0 = q.len / kPage;
  const int f0 = r0 > 0 ? 1 : 0;
  const int full = max(0, end / kPage - f0);  // blocks made of new rows only
  const size_t sh = size_t(b) * a.c.heads + h;
  __nv_bfloat16* tail = a.c.tail[kv] + sh * kPage * D;
  bool bad = false;

  // new row i of this sequence and head, vector v
  auto fresh = [&](int i, int v) {
    return load8_bf16(a.x[kv], int64_t(q.first + i) * a.ld[kv] + int64_t(h) * D + v * 8, a.bf16, bad);
  };
  // a whole block: rows below `old` from the tail, the others new rows from `i0`
  auto close_block = [&](int blk, int old, int i0) {
    uint4 v[kPer];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = threadIdx.x + i * kThreads, row = at / kV, c = at % kV;
      v[i] = row < old ? reinterpret_cast<const uint4*>(tail)[row * kV + c] : fresh(i0 + row - old, c);
      m = max8(v[i], m);
    }
    m = cta_max<kThreads>(m, s_red);
    const int e = scale_exp<FMT>(m);
    const int p = page_of(a.c, b, blk);
    if (p < 0) return;
    uint2* out = reinterpret_cast<uint2*>(a.c.codes[kv] + (size_t(p) * a.c.heads + h) * kPage * D);
    const float inv = exp2_int(-e);
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[threadIdx.x + i * kThreads] = encode8<FMT>(v[i], inv);
    if (threadIdx.x == 0) a.c.scale[kv][size_t(p) * a.c.heads + h] = exp2_int(e);
    if (kv == 0 && a.c.score)
      for (int i = old + threadIdx.x; i < kPage; i += kThreads)
        a.c.score[(size_t(p) * a.c.heads + h) * kPage + i] = 0.f;
  };
  // rows [old, old + n) of a block that stays open, from new rows `i0` on
  auto fill_block = [&](int blk, int old, int n, int i0) {
    const int p = page_of(a.c, b, blk);
    if (p < 0) return;
    float m = 0.f;
    for (int at = threadIdx.x; at < n * kV; at += kThreads) {
      const uint4 v = fresh(i0 + at / kV, at % kV);
      reinterpret_cast<uint4*>(tail)[old * kV + at] = v;
      m = max8(v, m);
    }
    m = cta_max<kThreads>(m, s_red);
    if (threadIdx.x == 0) {
      float* sc = a.c.scale[kv] + size_t(p) * a.c.heads + h;
      const float s = exp2_int(scale_exp<FMT>(m));
      *sc = old > 0 ? fmaxf(*sc, s) : s;
    }
    if (kv == 0 && a.c.score)
      for (int i = threadIdx.x; i < n; i += kThreads) a.c.score[(size_t(p) * a.c.heads + h) * kPage + old + i] = 0.f;
  };

  for (int j = blockIdx.x; j <= full; j += gridDim.x) {
    if (j > 0) {
      const int blk = f0 + j - 1;
      close_block(blk0 + blk, 0, blk * kPage - r0);
    } else {
      // the first block with the old tail and the last one, in this order: both
      // use the tail, so one CTA takes both
      const bool closes = r0 > 0 && end >= kPage;
      if (closes) close_block(blk0, r0, 0);
      __syncthreads();  // the old tail is read
      const int last = end / kPage, n = end % kPage;
      if (n > 0) {
        const int old = last == 0 ? r0 : 0;
        fill_block(blk0 + last, old, n - old, last * kPage + old - r0);
      }
    }
  }
  if (bad) atomicOr(a.c.status, kStatusNonFinite);
}

template <int FMT, int D>
gsi_status_t launch(const gsi_kv* kv, const AppendArgs& a, int64_t max_rows, cudaStream_t s) {
  const dim3 grid(unsigned(1 + max_rows / kPage), unsigned(2 * a.c.heads), unsigned(a.c.seqs));
  // One or two new rows keep few threads busy but when they close a block: small
  // CTAs, all resident at once.  128 sequences, 8 heads of 128, K and V, with small
  // CTAs and with 256 threads: one row 5.5 and 6.8 us, two 6.3 and 7.0, three 6.3 and
  // 7.2, five 8.3 and 7.9, sixteen 26 and 17; one sequence, 16 heads of 256: one row
  // and two 2.1 either way, five 2.4 and 2.2.
  constexpr int kFew = D == 256 ? 128 : 64;
  const cudaError_t e = max_rows <= 2 ? launch_pdl(append_kernel<FMT, D, kFew>, grid, dim3(kFew), 0, s, a)
                                      : launch_pdl(append_kernel<FMT, D, 256>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? GSI_OK : GSI_ERR_CUDA;
}

}  // namespace

gsi_status_t kv_append_launch(gsi_kv* kv, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              int bf16, const KvRows& r, int64_t max_rows, cudaStream_t s) {
  AppendArgs a;
  a.c = kv->view;
  a.r = r;
  a.x[0] = k;
  a.x[1] = v;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.bf16 = bf16;
  const bool i8 = kv->b.format == kInt8;
  switch (kv->b.head_dim) {
    case 64: return i8 ? launch<kInt8, 64>(kv, a, max_rows, s) : launch<kE4m3, 64>(kv, a, max_rows, s);
    case 128: return i8 ? launch<kInt8, 128>(kv, a, max_rows, s) : launch<kE4m3, 128>(kv, a, max_rows, s);
    default: return i8 ? launch<kInt8, 256>(kv, a, max_rows, s) : launch<kE4m3, 256>(kv, a, max_rows, s);
  }
}

}  // namespace gsi
