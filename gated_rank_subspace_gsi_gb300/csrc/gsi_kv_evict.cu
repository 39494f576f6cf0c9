// gsi_kv_evict.cu -- eviction from the 8-bit key/value cache by accumulated
// attention weight (gsi_kv_evict in gsi.h).
//
// Two launches.  The selection takes one CTA per sequence and head: the
// (budget - recent)-th largest score is found digit by digit (radix selection
// over the ordered bits of the scores, which are read once into shared memory as
// far as they fit), and the kept rows are written in token order.  The move takes
// one CTA per new block of a head: it gathers 64 kept rows, finds their scales
// and writes them as codes, or as bf16 into the tail.  Sources are the old pages
// and the old tail (a copy, if a new tail is written), destinations are spare
// pages, so blocks move in any order.
//
// The kept rows' bytes would bound it; what does is the chain of a selection
// (length, pages, scores, three digits, kept rows) and then of a block (row,
// scale and codes, maximum, codes).  Measured: one sequence of 2303 tokens cut
// to 2048, 16 heads of 256: 21 us; 16 of 3900 to 12001 cut to 4001, 8 heads of
// 128: 79 us, 3.2 TB/s, the selection a third of it; one of 106105 cut to 1000, 2
// heads of 128: 250 us, nearly all of it two CTAs' selection.
#include "gsi_kv.cuh"
#include "gsi_kv_codes.cuh"

namespace gsi {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kKeyRoom = 44 * 1024;  // keys in shared memory; later ones are read again for each digit
constexpr int kPageRoom = 4096;      // page numbers in shared memory; later ones are read again
constexpr int kNoRow = 0x7FFFFFFF;  // a kept token whose page is out of range: reads as zero

struct EvictArgs {
  KvView c;
  const int32_t* len;
  int budget, recent;
  int32_t* spare;
  int32_t* len_out;
  int32_t* keep;       // [seqs][heads][max_pages * 64]: page * 64 + row, or -1 - row of the old tail
  int32_t* dst;        // [seqs][max_pages] destination pages
  int key_room;        // keys that the selection's shared memory holds
  int32_t* was;        // [seqs][2] tokens held, page of the open block
  __nv_bfloat16* old;  // [2][seqs][heads][64][D]
};

// Bits whose unsigned order is the order of the floats, NaN largest.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (u == 0x80000000u) return 0x80000000u;  // -0 equals 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums over the CTA of v before this thread (exclusive).
__device__ __forceinline__ int cta_scan(int v, int* s_scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_scan[warp] = x;
  __syncthreads();
  int before = lane < warp ? s_scan[lane] : 0;  // 32 warps
#pragma unroll
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
  return before + x - v;
}

// Digits of the keys, from the top: 11, 11 and 10 bits.
constexpr int kBins = 2048;

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(EvictArgs a) {
  extern __shared__ uint32_t s_keys[];  // of the candidates, as far as they fit (a.key_room), then pages
  __shared__ int s_hist[kBins];
  __shared__ int s_scan[kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y;
  const int cap = a.c.max_pages * kPage;
  const int raw = a.len[b], n = min(max(raw, 0), cap);
  if (threadIdx.x == 0) {
    if (raw != n) atomicOr(a.c.status, kStatusBadPage);
    s_prefix = 0;
    s_need = a.budget - a.recent;
  }
  if (h == 0 && threadIdx.x == 0) {
    // the move reads the lengths from here: len_out may be len
    a.was[2 * b] = n;
    a.was[2 * b + 1] = n < cap ? a.c.page_table[size_t(b) * a.c.max_pages + n / kPage] : -1;
  }
  if (n <= a.budget) return;
  const size_t sh = size_t(b) * a.c.heads + h;
  const int32_t* table = a.c.page_table + size_t(b) * a.c.max_pages;
  const int old = n - a.recent;  // candidates: tokens 0 .. old - 1
  const int n_pages = (n + kPage - 1) / kPage;
  int32_t* s_page = reinterpret_cast<int32_t*>(s_keys + a.key_room);
  for (int i = threadIdx.x; i < min(n_pages, kPageRoom); i += kSelThreads) s_page[i] = table[i];
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) s_hist[i] = 0;
  __syncthreads();
  auto page_at = [&](int blk) { return blk < kPageRoom ? s_page[blk] : table[blk]; };
  auto load_key = [&](int t) {
    const int p = page_at(t / kPage);
    if (p < 0 || p >= a.c.pages) return 0u;
    return ordered(a.c.score[(size_t(p) * a.c.heads + h) * kPage + t % kPage]);
  };
  auto key = [&](int t) { return t < a.key_room ? s_keys[t] : load_key(t); };
  const bool any = a.budget > a.recent;
  // many scores share a digit: one addition for the lanes that do
  auto count = [&](int bin) {
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, bin);
    if (bin >= 0 && (threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&s_hist[bin], __popc(same));
  };
  if (any)
    for (int t0 = 0; t0 < old; t0 += 8 * kSelThreads) {
      uint32_t k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + e * kSelThreads + int(threadIdx.x);
        k[e] = t < old ? load_key(t) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + e * kSelThreads + int(threadIdx.x);
        if (t < min(old, a.key_room)) s_keys[t] = k[e];
        if (t0 + e * kSelThreads < old) count(t < old ? int(k[e] >> 21) : -1);
      }
    }
  // the tail as it is now, if the move writes to it, and the destination pages
  const int left = n % kPage;
  for (int kv = 0; a.budget % kPage != 0 && kv < 2; ++kv) {
    const uint4* src = reinterpret_cast<const uint4*>(a.c.tail[kv] + sh * kPage * D);
    uint4* out = reinterpret_cast<uint4*>(a.old + (size_t(kv) * a.c.seqs * a.c.heads + sh) * kPage * D);
    for (int i = threadIdx.x; i < left * D / 8; i += kSelThreads) out[i] = src[i];
  }
  if (h == 0)
    for (int j = threadIdx.x; j * kPage < a.budget; j += kSelThreads)
      a.dst[size_t(b) * a.c.max_pages + j] = a.spare[size_t(b) * a.c.max_pages + j];

  // the threshold, from the top digit down: s_prefix holds the digits found,
  // s_need how many of the keys that share them are kept
  for (int pass = 0; any && pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    if (pass > 0) {
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
    }
    const uint32_t prefix = s_prefix;
    const int need = s_need;
    const int top = pass == 1 ? 21 : 10;  // bits above are settled
    for (int t0 = 0; pass > 0 && t0 < old; t0 += kSelThreads) {
      const int t = t0 + threadIdx.x;
      const uint32_t k = t < old ? key(t) : 0u;
      count(t < old && (k >> top) == (prefix >> top) ? int((k >> shift) & uint32_t(bins - 1)) : -1);
    }
    __syncthreads();
    // thread i: the two digits bins - 1 - 2 i and one below
    const int hi = bins - 1 - 2 * int(threadIdx.x), c0 = hi > 0 ? s_hist[hi] : 0, c1 = hi > 0 ? s_hist[hi - 1] : 0;
    const int above = cta_scan(c0 + c1, s_scan);
    if (hi > 0) {
      if (above < need && above + c0 >= need) {
        s_prefix = prefix | (uint32_t(hi) << shift);
        s_need = need - above;
      } else if (above + c0 < need && above + c0 + c1 >= need) {
        s_prefix = prefix | (uint32_t(hi - 1) << shift);
        s_need = need - above - c0;
      }
    }
    __syncthreads();
  }
  const uint32_t thr = s_prefix;
  const int ties = s_need;  // keys equal to thr that are kept, earliest first

  // the kept rows in token order: a run of tokens per thread.  Counted first;
  // keys equal to the threshold count as far as there is room for them
  int32_t* keep = a.keep + sh * size_t(cap);
  const int run = (n + kSelThreads - 1) / kSelThreads, lo = min(n, int(threadIdx.x) * run), end = min(n, lo + run);
  int eq = 0, more = 0;
  for (int t = lo; t < end; ++t) {
    const uint32_t k = any && t < old ? key(t) : 0u;
    eq += any && t < old && k == thr;
    more += t >= old || (any && k > thr);
  }
  const int eq0 = cta_scan(eq, s_scan);
  int pos = cta_scan(more + min(max(ties - eq0, 0), eq), s_scan);
  int room = ties - eq0, p = -1, blk = -1;
  for (int t = lo; t < end; ++t) {
    const uint32_t k = any && t < old ? key(t) : 0u;
    bool stays = t >= old || (any && k > thr);
    if (any && t < old && k == thr) stays = room-- > 0;
    if (!stays) continue;
    if (pos < cap) {
      if (t / kPage != blk) {
        blk = t / kPage;
        p = page_at(blk);
      }
      const bool ok = p >= 0 && p < a.c.pages;
      if (!ok) atomicOr(a.c.status, kStatusBadPage);
      keep[pos] = t >= n - left ? -1 - t % kPage : ok ? p * kPage + t % kPage : kNoRow;
    }
    ++pos;
  }
}

// Sixteen codes as fp16, and back: times 2^k (exact, or below half a code's step)
// and rounded to nearest even.  int8: 1536 + v has v's two's complement in the low
// byte of an fp16, whose step is 1 there.  k is the old scale's exponent less the
// new one's.  No value of a block is above Q times its new scale, so a code that is
// not zero has 2^k <= Q / code: k is at most 6 for int8 (least code 1) and 17 for
// e4m3 (2^-9), where 2^k is no fp16 number beyond 2^15.
constexpr int kMostUp = 17, kFp16Up = 15;
template <int FMT>
__device__ __forceinline__ void codes16_f16(const uint4& w, uint32_t (&f)[8]) {
  codes_f16<FMT>(w.x, f[0], f[1]);
  codes_f16<FMT>(w.y, f[2], f[3]);
  codes_f16<FMT>(w.z, f[4], f[5]);
  codes_f16<FMT>(w.w, f[6], f[7]);
}
template <int FMT>
__device__ __forceinline__ uint32_t f16_codes(uint32_t lo, uint32_t hi, __half2 by) {
  const __half2 l = *reinterpret_cast<const __half2*>(&lo), h = *reinterpret_cast<const __half2*>(&hi);
  if (FMT == kInt8) {
    const uint32_t magic = 0x66006600u;
    const __half2 m = *reinterpret_cast<const __half2*>(&magic);
    const __half2 a = __hfma2(l, by, m), b = __hfma2(h, by, m);
    return __byte_perm(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b), 0x6420);
  }
  const __half2 a = __hmul2(l, by), b = __hmul2(h, by);
  uint32_t r;
  asm("{\n\t.reg .b16 p, q;\n\tcvt.rn.satfinite.e4m3x2.f16x2 p, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, %2;\n\t"
      "mov.b32 %0, {p, q};\n\t}"
      : "=r"(r) : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
  return r;
}

// One new block of a head: K by the first half of the CTA, V by the second.  A
// block whose rows all come from pages, and which stays in pages, is moved in
// fp16 (codes of both formats are exact there, about 3 instructions a code); one with
// rows from or for the tail in fp32.  CTAs on an SM count for more than registers.
// Evictions of 16 sequences of 3900 to 12001 tokens to 4001, 8 heads, selection and
// all: at D = 256 four, with a few spills, 127 us (e4m3) and 130 (int8), three 125 and
// 132, five 179 and 167 (one sequence of 16 heads, 2303 to 2048: four 21, three 24,
// five 25); at D = 128 five 82, four 87, eight, with spills, 97; at D = 64 six 63,
// four 64.
template <int FMT, int D>
__global__ void __launch_bounds__(kMoveThreads, D == 256 ? 4 : D == 128 ? 5 : 6) move_kernel(EvictArgs a) {
  constexpr int kHalf = kMoveThreads / 2;
  __shared__ float s_red[kMoveThreads / 32];
  __shared__ int s_row[kPage];
  __shared__ float s_scale[2][kPage];
  pdl_launch_dependents();
  pdl_wait();
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int cap = a.c.max_pages * kPage;
  const size_t sh = size_t(b) * a.c.heads + h;
  const int rows = min(kPage, a.budget - j * kPage);
  const int kv = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
  // (read before it is known to be used: one round trip less)
  const int src = tid < rows ? a.keep[sh * size_t(cap) + j * kPage + tid] : kNoRow;
  const int p = a.dst[size_t(b) * a.c.max_pages + j];
  const int n = a.was[2 * b], open = a.was[2 * b + 1];
  if (j == 0 && h == 0 && threadIdx.x == 0) a.len_out[b] = min(n, a.budget);
  if (n <= a.budget) return;
  if (p < 0 || p >= a.c.pages) {
    if (threadIdx.x == 0) atomicOr(a.c.status, kStatusBadPage);
    return;
  }
  if (h == 0 && threadIdx.x == 0) {
    // swap the table entries: no CTA of this launch reads either table
    // (sources are in keep, destinations in dst)
    const size_t i = size_t(b) * a.c.max_pages + j;
    a.spare[i] = a.c.page_table[i];
    a.c.page_table[i] = p;
  }
  if (kv == 0 && tid < kPage) s_row[tid] = src;
  const bool tailed = __syncthreads_or(rows < kPage || (tid < rows && src < 0));
  const size_t ph = size_t(p) * a.c.heads + h;
  float scale = 0.f;
  if (tid < rows && src >= 0 && src / kPage < a.c.pages) scale = a.c.scale[kv][size_t(src / kPage) * a.c.heads + h];
  if (kv == 1 && tid < rows) {
    // the tail's scores are in the page of the open block
    const int lp = src < 0 ? open : src / kPage, at = src < 0 ? -1 - src : src % kPage;
    a.c.score[ph * kPage + tid] =
        lp >= 0 && lp < a.c.pages ? a.c.score[(size_t(lp) * a.c.heads + h) * kPage + at] : 0.f;
  }
  // the largest magnitude of each half of the CTA
  auto half_max = [&](float m) {
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kHalf / 32; ++w) m = fmaxf(m, s_red[kv * (kHalf / 32) + w]);
    return m;
  };
  if (!tailed) {
    constexpr int kV = D / 16, kPer = kPage * kV / kHalf;  // vectors of 16 codes: of a row, of a thread
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = tid + i * kHalf, row = at / kV, src = s_row[row];
      const size_t sph = size_t(src / kPage) * a.c.heads + h;
      v[i] = make_uint4(0, 0, 0, 0);
      if (src / kPage < a.c.pages)
        v[i] = reinterpret_cast<const uint4*>(a.c.codes[kv] + (sph * kPage + src % kPage) * D)[at % kV];
    }
    if (tid < kPage) s_scale[kv][tid] = scale;
    __syncthreads();
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint32_t f[8];
      codes16_f16<FMT>(v[i], f);
      __half2 t = __float2half2_rn(0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) t = __hmax2(t, __habs2(*reinterpret_cast<const __half2*>(&f[e])));
      m = fmaxf(m, __half2float(__hmax(__low2half(t), __high2half(t))) * s_scale[kv][(tid + i * kHalf) / kV]);
    }
    const int e = scale_exp<FMT>(half_max(m));
    if (tid == 0) a.c.scale[kv][ph] = exp2_int(e);
    const float inv = exp2_int(-e);
    uint4* out = reinterpret_cast<uint4*>(a.c.codes[kv] + ph * kPage * D);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint32_t f[8];
      codes16_f16<FMT>(v[i], f);
      // (beyond the most only for rows of zeros)
      const float up = fminf(s_scale[kv][(tid + i * kHalf) / kV] * inv, float(1 << kMostUp));
      const float low = fminf(up, float(1 << kFp16Up));
      const __half2 by = __float2half2_rn(low);
      if (FMT == kE4m3) {
        // what is beyond 2^15 (1 but for codes of at most 2^-7) as a factor of its own
        const __half2 rest = __float2half2_rn(up > low ? up * (1.f / (1 << kFp16Up)) : 1.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&f[e]), rest);
          f[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
      }
      out[tid + i * kHalf] = make_uint4(f16_codes<FMT>(f[0], f[1], by), f16_codes<FMT>(f[2], f[3], by),
                                        f16_codes<FMT>(f[4], f[5], by), f16_codes<FMT>(f[6], f[7], by));
    }
    return;
  }
  if (tid < kPage) s_scale[kv][tid] = scale;
  __syncthreads();
  constexpr int kV = D / 8, kPer = kPage * kV / kHalf;  // vectors of 8 values: of a row, of a thread
  constexpr int kUn = kPer < 16 ? 4 : 8;               // read at a time (the second reading is from L2)
  const __nv_bfloat16* old = a.budget % kPage == 0 ? a.c.tail[kv] : a.old + size_t(kv) * a.c.seqs * a.c.heads * kPage * D;
  old += sh * kPage * D;
  auto read = [&](int i0, uint4 (&v)[kUn]) {
#pragma unroll
    for (int i = 0; i < kUn; ++i) {
      const int at = tid + (i0 + i) * kHalf, row = at / kV, c = at % kV, src = s_row[row];
      v[i] = make_uint4(0, 0, 0, 0);
      if (src < 0) {
        v[i] = reinterpret_cast<const uint4*>(old)[(-1 - src) * kV + c];
      } else if (src / kPage < a.c.pages) {
        const size_t sph = size_t(src / kPage) * a.c.heads + h;
        const uint2 w = reinterpret_cast<const uint2*>(a.c.codes[kv] + (sph * kPage + src % kPage) * D)[c];
        v[i].x = w.x;
        v[i].y = w.y;
      }
    }
  };
  // as bf16: a code times a power of two is a bf16 number
  auto value = [&](int at, const uint4& v) {
    const int row = at / kV;
    if (s_row[row] < 0) return v;
    const float s = s_scale[kv][row];
    const float2 f0 = decode2<FMT>(v.x), f1 = decode2<FMT>(v.x >> 16);
    const float2 f2 = decode2<FMT>(v.y), f3 = decode2<FMT>(v.y >> 16);
    return make_uint4(pack_bf16(f0.x * s, f0.y * s), pack_bf16(f1.x * s, f1.y * s), pack_bf16(f2.x * s, f2.y * s),
                      pack_bf16(f3.x * s, f3.y * s));
  };
  float m = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < kPer; i0 += kUn) {
    uint4 v[kUn];
    read(i0, v);
#pragma unroll
    for (int i = 0; i < kUn; ++i) m = max8(value(tid + (i0 + i) * kHalf, v[i]), m);
  }
  const int e = scale_exp<FMT>(half_max(m));
  if (tid == 0) a.c.scale[kv][ph] = exp2_int(e);
  uint2* codes = reinterpret_cast<uint2*>(a.c.codes[kv] + ph * kPage * D);
  uint4* tail = reinterpret_cast<uint4*>(a.c.tail[kv] + sh * kPage * D);
#pragma unroll 1
  for (int i0 = 0; i0 < kPer; i0 += kUn) {
    uint4 v[kUn];
    read(i0, v);
#pragma unroll
    for (int i = 0; i < kUn; ++i) {
      const int at = tid + (i0 + i) * kHalf;
      const uint4 x = value(at, v[i]);
      if (rows == kPage) codes[at] = encode8<FMT>(x, exp2_int(-e));
      else if (at < rows * kV) tail[at] = x;
    }
  }
}

template <int FMT, int D>
gsi_status_t launch(const EvictArgs& a, int device, cudaStream_t s) {
  const size_t smem = size_t(a.key_room + kPageRoom) * 4;
  static std::atomic<uint64_t> ready{0};  // devices that allow the kernel its shared memory
  if (!allow_smem(select_kernel<D>, size_t(kKeyRoom + kPageRoom) * 4, device, ready)) return GSI_ERR_CUDA;
  if (launch_pdl(select_kernel<D>, dim3(unsigned(a.c.heads), unsigned(a.c.seqs)), dim3(kSelThreads), smem, s, a) !=
      cudaSuccess)
    return GSI_ERR_CUDA;
  const dim3 grid(unsigned((a.budget + kPage - 1) / kPage), unsigned(a.c.heads), unsigned(a.c.seqs));
  return launch_pdl(move_kernel<FMT, D>, grid, dim3(kMoveThreads), 0, s, a) == cudaSuccess ? GSI_OK : GSI_ERR_CUDA;
}

}  // namespace

gsi_status_t kv_evict_launch(gsi_kv* kv, const int32_t* len, int budget, int recent,
                             int32_t* spare, int32_t* len_out, cudaStream_t s) {
  EvictArgs a;
  a.c = kv->view;
  a.len = len;
  a.budget = budget;
  a.recent = recent;
  a.spare = spare;
  a.len_out = len_out;
  a.keep = kv->keep;
  a.dst = kv->dst_pages;
  a.was = kv->was;
  const int64_t cap = int64_t(kv->b.max_pages) * kPage;
  a.key_room = int(cap < kKeyRoom ? cap : kKeyRoom);
  a.old = kv->old_tail;
  const bool i8 = kv->b.format == kInt8;
  switch (kv->b.head_dim) {
    case 64: return i8 ? launch<kInt8, 64>(a, kv->device, s) : launch<kE4m3, 64>(a, kv->device, s);
    case 128: return i8 ? launch<kInt8, 128>(a, kv->device, s) : launch<kE4m3, 128>(a, kv->device, s);
    default: return i8 ? launch<kInt8, 256>(a, kv->device, s) : launch<kE4m3, 256>(a, kv->device, s);
  }
}

}  // namespace gsi
