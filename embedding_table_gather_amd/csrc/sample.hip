// Sampling of one token per row of logits with temperature, top-k, top-p and min-p
// from given random numbers (the sampling that ADR-0008 "POST /v1/logits" leaves to
// the caller of its raw logits mode), without the logits leaving the device.
#include <algorithm>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

// Candidates are the allowed tokens whose logit is neither NaN nor -inf.  With M the
// largest candidate logit and T the temperature, candidate v weighs
//   w_v = exp((l_v - M) / T), 1 where l_v == M (an infinite M included),
// in 64 bits.  The order of a row is logit descending, then id ascending; each filter
// keeps a prefix of it, so the kept set is given by its last element (key, id):
//   top-k  the first k;
//   top-p  the shortest prefix whose mass reaches p times the mass of the first k;
//   min-p  every candidate with w_v >= min_p.
// The sampled id is the first kept one, in id order, whose running sum of weights
// exceeds u times the kept mass.
//
// Masses are sums of weights in unsigned fixed point, 2^-shift each: integer sums do
// not depend on the order in which threads add, so a call repeats bitwise, and tokens
// with equal logits weigh exactly the same.  With vocab <= 2^b the sum is at most
// 2^(b + shift) <= 2^63: shift = min(45, 63 - b).  A weight is off by at most half a
// unit, a total (at least 2^shift) by 2^(b - shift - 1) of itself: 2^-28 at 2^18 tokens
// and 2^-24 at the largest vocabulary, 2^20.
//
// Kernels:
//  1. sample_chunk_kernel streams the logits once, a workgroup per 4,096 tokens: the
//     maximum of every small group of tokens and of the chunk and, for rows whose
//     filters need it, the chunk's mass.
//  2. sample_row_kernel, a workgroup per row.  A row without filters picks a chunk by
//     the chunk masses and a token in it.  Otherwise the group maxima give a lower bound
//     of the cut: if the k largest maxima reach a value, so do k tokens, and if the
//     maxima above a value weigh p times the total, so does the nucleus.  Only the groups
//     that reach the bound are read again, and their tokens at or above it (a few more
//     than are kept) are sorted in LDS.
//  3. Rows that keep more than the list holds (flat distributions) go on to
//     sample_hist_kernel, which counts and weighs every token in 1,024 bins per slice
//     of 32,768 tokens, and sample_heavy_kernel, which finds the cut's bin, reads the
//     tokens of that bin and narrows it to the cut.

struct SampleRow {
  float T, p, minp, u;
  int32_t k;    // 0: no top-k
  bool ok;
};

__device__ __forceinline__ SampleRow sample_row(const Sample& s, int64_t row) {
  SampleRow r;
  r.T = s.d_temperature ? s.d_temperature[row] : s.temperature;
  r.k = s.d_top_k ? s.d_top_k[row] : s.top_k;
  r.p = s.d_top_p ? s.d_top_p[row] : s.top_p;
  r.minp = s.d_min_p ? s.d_min_p[row] : s.min_p;
  r.u = s.uniform[row];
  // comparisons that a NaN fails
  r.ok = r.T >= 0.f && r.T < __builtin_inff() && r.k >= 0 && r.p > 0.f && r.p <= 1.f && r.minp >= 0.f &&
         r.minp <= 1.f && r.u >= 0.f && r.u < 1.f;
  if (r.T == 0.f) {  // greedy: the first of the order, with probability 1
    r.T = 1.f;
    r.k = 1;
    r.p = 1.f;
    r.minp = 0.f;
  }
  if (r.k >= s.vocab) r.k = 0;
  return r;
}

static constexpr int kSampleThreads = 1024;
static constexpr int kSampleWaves = kSampleThreads / 64;
static constexpr int kSampleBins = 1024;         // one per thread
static constexpr int kChunk = 4096;              // tokens of a chunk
static constexpr int kChunkThreads = 256;
static constexpr int kSlice = 32768;             // tokens of a histogram slice
static constexpr int kMaxSlices = (1 << 20) / kSlice;
static constexpr int kList = 2048;               // tokens sorted in LDS by the row kernel
static constexpr int kHeavyList = 8192;          // tokens of one bin in the heavy kernel
static constexpr int kMaxGroups = 4096;          // groups per row up to 2^18 tokens
static constexpr int64_t kHeavySlots = 512;      // rows of one call with histograms

// Workspace of a call, from its sizes alone.
struct SampleWs {
  int chunks, slices, group_log2, groups, slots;
  size_t gmax, cmax, csum, flag, nheavy, hcount, hmass, bytes;
};

static SampleWs sample_ws(int64_t rows, int64_t vocab, int32_t dtype) {
  SampleWs w;
  w.chunks = (int)cdiv(vocab, kChunk);
  w.slices = (int)cdiv(vocab, kSlice);
  // groups of one 16-byte load (4 or 8 tokens) to 64 tokens, at most kMaxGroups up to 2^18
  w.group_log2 = dtype == DT_F32 ? 2 : 3;
  while (w.group_log2 < 6 && cdiv(vocab, 1ll << w.group_log2) > kMaxGroups) w.group_log2++;
  w.groups = (int)cdiv(vocab, 1ll << w.group_log2);
  w.slots = (int)std::min(rows, kHeavySlots);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at = align_up(at + n, 256);
    return o;
  };
  w.gmax = take((size_t)rows * w.groups * 4);
  w.cmax = take((size_t)rows * w.chunks * 4);
  w.csum = take((size_t)rows * w.chunks * 8);
  w.flag = take((size_t)rows * 4);
  w.nheavy = take(4);
  w.hcount = take((size_t)w.slots * w.slices * kSampleBins * 4);
  w.hmass = take((size_t)w.slots * w.slices * kSampleBins * 8);
  w.bytes = at;
  return w;
}

struct SamplePtrs {
  float* gmax;       // [rows][groups] largest candidate logit, -inf for none
  float* cmax;       // [rows][chunks]
  uint64_t* csum;    // [rows][chunks] mass relative to the chunk's own maximum
  int32_t* flag;     // [rows] -1: done, else the histogram slot
  uint32_t* nheavy;  // slots taken
  uint32_t* hcount;  // [slots][slices][bins]
  uint64_t* hmass;
  int chunks, slices, group_log2, groups, slots, shift;
};

// ---------------------------------------------------------------------------
// Weights
// ---------------------------------------------------------------------------
// 2^y * 2^e for y <= 0: y = n + f with f in [-1/2, 1/2], 2^f = exp(f ln 2) by its
// series up to the 12th power (truncated at 2e-16), scaled by n + e.
__device__ __forceinline__ double scaled_exp2(double y, int e) {
  const double n = rint(y);
  const double z = (y - n) * 0.693147180559945309417;
  double p = 1.0 / 479001600.0;
  p = fma(p, z, 1.0 / 39916800.0);
  p = fma(p, z, 1.0 / 3628800.0);
  p = fma(p, z, 1.0 / 362880.0);
  p = fma(p, z, 1.0 / 40320.0);
  p = fma(p, z, 1.0 / 5040.0);
  p = fma(p, z, 1.0 / 720.0);
  p = fma(p, z, 1.0 / 120.0);
  p = fma(p, z, 1.0 / 24.0);
  p = fma(p, z, 1.0 / 6.0);
  p = fma(p, z, 0.5);
  p = fma(p, z, 1.0);
  p = fma(p, z, 1.0);
  return ldexp(p, (int)n + e);
}

struct SampleWeight {
  double M, c;  // the largest logit, log2(e) / T
  int shift;
  __device__ __forceinline__ SampleWeight(float top, float T, int shift_)
      : M((double)top), c(1.4426950408889634074 / (double)T), shift(shift_) {}
  // exponents below -1200 give 0 whatever they are (infinite ones included)
  __device__ __forceinline__ double power(float l) const { return fmax(((double)l - M) * c, -1200.0); }
  __device__ __forceinline__ double weight(float l) const {
    return (double)l == M ? 1.0 : scaled_exp2(power(l), 0);
  }
  // rint(weight * 2^shift): at most 2^45, so adding 2^52 leaves it in the low bits
  __device__ __forceinline__ uint64_t fixed(float l) const {
    const double x = ((double)l == M ? ldexp(1.0, shift) : scaled_exp2(power(l), shift)) + 4503599627370496.0;
    return (uint64_t)__double_as_longlong(x) & 0xfffffffffffffull;
  }
};

// floor or ceil of f * m for a float f in [0, 1] and an integer m, exactly: f is a
// 24-bit integer times a power of two, the product 88 bits.
__device__ __forceinline__ uint64_t scaled(float f, uint64_t m, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int e = max((int)(b >> 23), 1);  // f = mant * 2^(e - 150)
  const uint64_t mant = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  const unsigned __int128 x = (unsigned __int128)mant * m;
  const int right = 150 - e;             // at least 23, as f <= 1
  if (right >= 100) return up && x != 0 ? 1 : 0;
  const unsigned __int128 q = x >> right;
  return (uint64_t)q + (up && (q << right) != x);
}
__device__ __forceinline__ uint64_t scaled_floor(float f, uint64_t m) { return scaled(f, m, false); }
__device__ __forceinline__ uint64_t scaled_ceil(float f, uint64_t m) { return scaled(f, m, true); }

// ---------------------------------------------------------------------------
// One row's logits
// ---------------------------------------------------------------------------
template <int DT>
struct SampleSource {
  const uint8_t* base;
  const uint32_t* allowed;
  int V;
  __device__ __forceinline__ SampleSource(const Sample& s, int64_t row)
      : base((const uint8_t*)s.logits + row * s.stride * (DT == DT_F32 ? 4 : 2)),
        allowed(s.allowed ? s.allowed + row * s.allowed_stride : nullptr), V((int)s.vocab) {}
  // the logit of token v, -inf where it is no candidate (v < V)
  __device__ __forceinline__ float logit(int v) const {
    float l;
    if constexpr (DT == DT_F32) l = ((const float*)base)[v];
    else if constexpr (DT == DT_BF16) l = __uint_as_float((uint32_t)((const uint16_t*)base)[v] << 16);
    else l = f16_bits_to_f32(((const uint16_t*)base)[v]);
    const bool live = l > -__builtin_inff() && (allowed == nullptr || ((allowed[v >> 5] >> (v & 31)) & 1u));
    return live ? l : -__builtin_inff();
  }
  // tokens [v, v + N) (v a multiple of N, N = 4 or 8 by type), -inf past the vocabulary:
  // one 16-byte load at any alignment of the value
  static constexpr int N = DT == DT_F32 ? 4 : 8;
  __device__ __forceinline__ void load(int v, float (&l)[N]) const {
    if (v + N <= V) {
      u32x4 w;
      __builtin_memcpy(&w, base + (size_t)v * (16 / N), 16);
#pragma unroll
      for (int j = 0; j < N; j++) {
        if constexpr (DT == DT_F32) l[j] = __uint_as_float(w[j]);
        else if constexpr (DT == DT_BF16) l[j] = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
        else l[j] = f16_bits_to_f32(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
      }
      const uint32_t ok = allowed ? allowed[v >> 5] >> (v & 31) : 0xffffffffu;
#pragma unroll
      for (int j = 0; j < N; j++)
        if (!(l[j] > -__builtin_inff()) || !((ok >> j) & 1u)) l[j] = -__builtin_inff();
    } else {
#pragma unroll
      for (int j = 0; j < N; j++) l[j] = v + j < V ? logit(v + j) : -__builtin_inff();
    }
  }
};

// Order key of a logit, 0 for -inf (every candidate's is larger).
__device__ __forceinline__ uint32_t sample_key(float l) { return l > -__builtin_inff() ? score_ord(l) : 0u; }

// Bin of a logit: logarithmic in its distance to the largest one, 64 bins per octave
// from 2^-8 to 2^8 (nearer ones in bin 0, farther ones in the last).  It never falls
// as the logit falls.
__device__ __forceinline__ int sample_bin(float l, float top) {
  const uint32_t d = l == top ? 0u : __float_as_uint(top - l) & 0x7fffffffu;
  return min(max((int)(d >> 17) - (119 << 6), 0), kSampleBins - 1);
}

// The smallest key whose bin is at most b.
__device__ __forceinline__ uint32_t sample_bin_floor(int b, float top) {
  if (b >= kSampleBins - 1) return 1;
  uint32_t lo = 0, hi = score_ord(top);  // hi's bin is 0
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (sample_bin(ord_score(mid), top) <= b) hi = mid;  // keys below -inf's decode to NaN: the last bin
    else lo = mid;
  }
  return hi;
}

// The smallest key whose weight reaches minp (weights do not fall as keys grow).
__device__ __forceinline__ uint32_t sample_minp_key(const SampleWeight& w, float top, float minp) {
  uint32_t lo = 0, hi = score_ord(top);  // keys above lo are undecided, hi's weight reaches it
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (w.weight(ord_score(mid)) >= (double)minp) hi = mid;
    else lo = mid;
  }
  return hi;
}

// ---------------------------------------------------------------------------
// Workgroup primitives (1,024 threads); every one begins and ends with the shared
// scratch free to reuse.
// ---------------------------------------------------------------------------
struct SampleScratch {
  uint64_t part[kSampleWaves];
  uint64_t value[2];
  uint32_t index[2];
};

__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint64_t o = (uint64_t)__shfl_up((unsigned long long)v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

// Inclusive prefix sum over the threads; *total receives the sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* total, SampleScratch& sc) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  v = wave_scan_u64(v);
  __syncthreads();
  if (lane == 63) sc.part[wv] = v;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSampleWaves; i++) {
    if (i < wv) before += sc.part[i];
    all += sc.part[i];
  }
  *total = all;
  __syncthreads();
  return before + v;
}

// The first thread with `hit`, and the two values it holds, to every thread; -1 for none.
__device__ __forceinline__ int block_first(bool hit, uint64_t a, uint64_t b, uint64_t* oa, uint64_t* ob,
                                           SampleScratch& sc) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint64_t m = __ballot(hit);
  __syncthreads();
  if (lane == 0) sc.part[wv] = m;
  __syncthreads();
  int first = -1;
#pragma unroll
  for (int i = kSampleWaves - 1; i >= 0; i--)
    if (sc.part[i] != 0) first = 64 * i + __ffsll((unsigned long long)sc.part[i]) - 1;
  if ((int)threadIdx.x == first) {
    sc.value[0] = a;
    sc.value[1] = b;
  }
  __syncthreads();
  if (first >= 0) {
    *oa = sc.value[0];
    *ob = sc.value[1];
  }
  __syncthreads();
  return first;
}

// The token of [lo, hi) (lo a multiple of 4) in which the running mass first exceeds
// target; weigh(v) is a token's mass.  The range's mass exceeds target.
template <typename F>
__device__ __forceinline__ int block_pick(int lo, int hi, uint64_t target, F weigh, SampleScratch& sc) {
  int last = lo;
  for (int at = lo; at < hi; at += 4 * kSampleThreads) {
    const int v = at + 4 * (int)threadIdx.x;
    uint64_t w[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      w[j] = v + j < hi ? weigh(v + j) : 0;
      sum += w[j];
    }
    uint64_t total;
    const uint64_t upto = block_scan(sum, &total, sc);
    if (total > target) {
      uint64_t run = upto - sum;
      int id = v;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (run <= target) id = v + j;  // the last token that begins at or below the target
        run += w[j];
      }
      uint64_t got, unused;
      block_first(upto > target, (uint64_t)id, 0, &got, &unused, sc);
      return (int)got;
    }
    target -= total;
    last = at;
  }
  return last;  // not reached
}

// ---------------------------------------------------------------------------
// 1. Chunks
// ---------------------------------------------------------------------------
// Max over the 2^steps-lane groups of a 16-lane row (DPP), to every lane of the group.
__device__ __forceinline__ float group_max(float m, int steps) {
  auto dpp = [&](auto ctrl) {
    return fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), decltype(ctrl)::value, 0xf, 0xf,
                                                               true)));
  };
  if (steps > 0) m = dpp(std::integral_constant<int, 0xb1>{});   // quad_perm 1,0,3,2
  if (steps > 1) m = dpp(std::integral_constant<int, 0x4e>{});   // quad_perm 2,3,0,1
  if (steps > 2) m = dpp(std::integral_constant<int, 0x141>{});  // row_half_mirror
  if (steps > 3) m = dpp(std::integral_constant<int, 0x140>{});  // row_mirror
  return m;
}

// Bound by the logits' bytes (one 16-byte load per 4 or 8 tokens) where no mass is
// needed, else by about 30 f64 operations per token.
template <int DT>
__global__ void __launch_bounds__(kChunkThreads) sample_chunk_kernel(Sample s, SamplePtrs ws) {
  using Src = SampleSource<DT>;
  constexpr int N = Src::N, NV = kChunk / (kChunkThreads * N);
  __shared__ float pmax[kChunkThreads / 64];
  __shared__ uint64_t psum[kChunkThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, c = blockIdx.x;
  const int steps = ws.group_log2 - (DT == DT_F32 ? 2 : 3);
  if (c == 0 && blockIdx.y == 0 && tid == 0) *ws.nheavy = 0;
  for (int64_t row = blockIdx.y; row < s.rows; row += gridDim.y) {
    const Src src(s, row);
    float l[NV][N];
#pragma unroll
    for (int j = 0; j < NV; j++) src.load(c * kChunk + (j * kChunkThreads + tid) * N, l[j]);
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float g = l[j][0];
#pragma unroll
      for (int e = 1; e < N; e++) g = fmaxf(g, l[j][e]);
      g = group_max(g, steps);
      const int v = c * kChunk + (j * kChunkThreads + tid) * N;
      if ((lane & ((1 << steps) - 1)) == 0 && v < src.V) ws.gmax[row * ws.groups + (v >> ws.group_log2)] = g;
      m = fmaxf(m, g);
    }
    m = wave_max_f32(m);
    __syncthreads();
    if (lane == 0) pmax[wv] = m;
    __syncthreads();
    m = fmaxf(fmaxf(pmax[0], pmax[1]), fmaxf(pmax[2], pmax[3]));
    if (tid == 0) ws.cmax[row * ws.chunks + c] = m;
    const SampleRow r = sample_row(s, row);
    if (r.k != 0 || !(r.p < 1.f || r.minp == 0.f) || !r.ok) continue;  // no filter of this row needs the mass
    uint64_t sum = 0;
    if (m > -__builtin_inff()) {
      const SampleWeight w(m, r.T, ws.shift);
#pragma unroll
      for (int j = 0; j < NV; j++)
#pragma unroll
        for (int e = 0; e < N; e++) sum += l[j][e] > -__builtin_inff() ? w.fixed(l[j][e]) : 0;
    }
    sum = wave_scan_u64(sum);
    if (lane == 63) psum[wv] = sum;
    __syncthreads();
    if (tid == 0) ws.csum[row * ws.chunks + c] = psum[0] + psum[1] + psum[2] + psum[3];
  }
}

// ---------------------------------------------------------------------------
// Search for a cut
// ---------------------------------------------------------------------------
// The kept prefix of a row: keys above `key`, and ids up to `id` at `key`.
struct SampleCut {
  uint32_t key = 1, id = 0xffffffffu;
  __device__ __forceinline__ bool keeps(uint32_t k, uint32_t v) const { return k > key || (k == key && v <= id); }
};

struct SampleHist {
  uint32_t count[kSampleBins];
  uint64_t mass[kSampleBins];
};

// Narrows *cut to the element at which the prefix of its kept elements first holds
// `count` of them (by_count) or `mass`; returns the prefix's mass.  That element's key
// lies in [klo, khi]; before_count and before_mass are those of the keys above khi.
// each(f) calls f(key, id) for every element with a key in [klo, khi] at least, each by
// one thread.  1,024 bins per round, then the same on the ids of the last key.
template <typename E>
__device__ __forceinline__ uint64_t sample_find(E each, const SampleWeight& w, int V, SampleCut* cut, uint32_t klo,
                                                uint32_t khi, bool by_count, uint64_t count, uint64_t mass,
                                                uint64_t before_count, uint64_t before_mass, SampleHist& h,
                                                SampleScratch& sc) {
  const int tid = threadIdx.x;
  const SampleCut old = *cut;
  while (klo < khi) {
    const int sh = max(0, 22 - __clz((int)(khi - klo)));  // (khi - klo) >> sh < 1024
    h.count[tid] = 0;
    h.mass[tid] = 0;
    __syncthreads();
    each([&](uint32_t key, uint32_t id) {
      if (key >= klo && key <= khi && old.keeps(key, id)) {
        const int b = (int)((key - klo) >> sh);
        atomicAdd(&h.count[b], 1u);
        atomicAdd((unsigned long long*)&h.mass[b], (unsigned long long)w.fixed(ord_score(key)));
      }
    });
    __syncthreads();
    const uint64_t c = h.count[kSampleBins - 1 - tid], m = h.mass[kSampleBins - 1 - tid];
    uint64_t tc, tm, bc, bm;
    const uint64_t ic = before_count + block_scan(c, &tc, sc), im = before_mass + block_scan(m, &tm, sc);
    // the first bin from the top that reaches the target, else the last that holds any
    int t = block_first(c != 0 && (by_count ? ic >= count : im >= mass), ic - c, im - m, &bc, &bm, sc);
    if (t < 0) t = block_first(c != 0 && ic == before_count + tc, ic - c, im - m, &bc, &bm, sc);
    before_count = bc;
    before_mass = bm;
    klo += (uint32_t)(kSampleBins - 1 - t) << sh;
    khi = min(khi, klo + ((1u << sh) - 1));
    __syncthreads();
  }
  const uint64_t wk = w.fixed(ord_score(klo));
  uint64_t ties = by_count ? count - before_count : wk != 0 ? (mass - before_mass + wk - 1) / wk : ~0ull >> 1;
  // the id of the last of `ties` elements with the key
  uint32_t ilo = 0, ihi = (uint32_t)V - 1;
  uint64_t passed = 0;
  do {
    const int sh = max(0, 22 - __clz((int)(ihi - ilo)));
    h.count[tid] = 0;
    __syncthreads();
    each([&](uint32_t key, uint32_t id) {
      if (key == klo && id >= ilo && id <= ihi && old.keeps(key, id)) atomicAdd(&h.count[(id - ilo) >> sh], 1u);
    });
    __syncthreads();
    const uint64_t c = h.count[tid];
    uint64_t tc, bc, unused;
    const uint64_t ic = passed + block_scan(c, &tc, sc);
    ties = min(ties, passed + tc);
    const int t = block_first(c != 0 && ic >= ties, ic - c, 0, &bc, &unused, sc);
    passed = bc;
    ilo += (uint32_t)t << sh;
    ihi = min(ihi, ilo + ((1u << sh) - 1));
    __syncthreads();
  } while (ilo < ihi);
  cut->key = klo;
  cut->id = ilo;
  return before_mass + ties * wk;
}

// f(key, id) for every candidate of a row, the vocabulary dealt to the threads.
template <int DT, typename F>
__device__ __forceinline__ void sample_each(const SampleSource<DT>& src, F f) {
  constexpr int N = SampleSource<DT>::N;
  for (int v = (int)threadIdx.x * N; v < src.V; v += kSampleThreads * N) {
    float l[N];
    src.load(v, l);
#pragma unroll
    for (int j = 0; j < N; j++)
      if (l[j] > -__builtin_inff()) f(score_ord(l[j]), (uint32_t)(v + j));
  }
}

__device__ __forceinline__ void sample_store(const Sample& s, int64_t row, int id, double w, uint64_t total, int shift) {
  if (threadIdx.x == 0) {
    s.ids[row] = id;
    s.probs[row] = (float)(ldexp(w, shift) / (double)total);
  }
}

// A row by nothing but passes over its logits: for rows past the histogram slots and
// for lists that do not fit.
template <int DT>
__device__ __attribute__((noinline)) void sample_by_passes(const Sample& s, int64_t row, float top, int shift,
                                                           SampleHist& h, SampleScratch& sc) {
  const SampleSource<DT> src(s, row);
  const SampleRow r = sample_row(s, row);
  const SampleWeight w(top, r.T, shift);
  auto each = [&](auto f) { sample_each<DT>(src, f); };
  SampleCut cut;
  auto kept_mass = [&]() {
    uint64_t m = 0, total;
    each([&](uint32_t key, uint32_t id) { m += cut.keeps(key, id) ? w.fixed(ord_score(key)) : 0; });
    block_scan(m, &total, sc);
    return total;
  };
  const uint32_t top_key = score_ord(top);
  uint64_t mass = 0;
  if (r.k > 0) mass = sample_find(each, w, src.V, &cut, 1u, top_key, true, (uint64_t)r.k, 0, 0, 0, h, sc);
  if (r.p < 1.f) {
    if (r.k == 0) mass = kept_mass();
    sample_find(each, w, src.V, &cut, 1u, top_key, false, 0, scaled_ceil(r.p, mass), 0, 0, h, sc);
  }
  if (r.minp > 0.f) {
    const uint32_t key = sample_minp_key(w, top, r.minp);
    if (key > cut.key) cut.key = key, cut.id = 0xffffffffu;
  }
  const uint64_t total = kept_mass();
  const int id = block_pick(0, src.V, scaled_floor(r.u, total), [&](int v) {
    const float l = src.logit(v);
    const uint32_t key = sample_key(l);
    return key != 0 && cut.keeps(key, (uint32_t)v) ? w.fixed(l) : 0ull;
  }, sc);
  sample_store(s, row, id, w.weight(src.logit(id)), total, shift);
}

// ---------------------------------------------------------------------------
// 2. Rows
// ---------------------------------------------------------------------------
struct SampleRowShared {
  SampleScratch sc;
  SampleHist h;
  uint64_t list[kList];    // the tokens at or above the bound in id order: key << 32 | ~id
  uint64_t sorted[kList];  // the same in the row's order
  uint32_t groups[kList];  // groups that reach the bound, in order
  uint32_t wave_count[kSampleWaves];
};

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_row_kernel(Sample s, SamplePtrs ws, int heavy) {
  __shared__ SampleRowShared sh;
  SampleScratch& sc = sh.sc;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const SampleSource<DT> src(s, row);
  const SampleRow r = sample_row(s, row);
  const int V = src.V;
  if (tid == 0 && heavy) ws.flag[row] = -1;

  // the row's largest logit and, where the chunks have masses, their sum
  float cm = -__builtin_inff();
  if (tid < ws.chunks) cm = ws.cmax[row * ws.chunks + tid];
  float top = wave_max_f32(cm);
  if (lane == 0) sc.part[wv] = __float_as_uint(top);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSampleWaves; i++) top = fmaxf(top, __uint_as_float((uint32_t)sc.part[i]));
  __syncthreads();
  if (!(top > -__builtin_inff()) || !r.ok) {  // whole workgroup
    if (tid == 0) {
      s.ids[row] = -1;
      s.probs[row] = 0.f;
    }
    return;
  }
  const SampleWeight w(top, r.T, ws.shift);
  uint64_t total = 0;
  if (r.k == 0 && (r.p < 1.f || r.minp == 0.f)) {
    // chunk masses to the row's maximum: a chunk at it keeps its integer sum
    uint64_t z = 0;
    if (cm > -__builtin_inff()) {
      z = ws.csum[row * ws.chunks + tid];
      if (cm != top) z = (uint64_t)rint((double)z * w.weight(cm));
    }
    const uint64_t upto = block_scan(z, &total, sc);
    if (r.p == 1.f) {  // no filter: the chunk, then the token by weights relative to the chunk's maximum
      const uint64_t target = scaled_floor(r.u, total);
      uint64_t left, cbits;
      const int c = block_first(upto > target, target - (upto - z), (uint64_t)__float_as_uint(cm), &left, &cbits, sc);
      const float m = __uint_as_float((uint32_t)cbits);
      const SampleWeight wc(m, r.T, ws.shift);
      if (m != top) {
        const uint64_t all = ws.csum[row * ws.chunks + c];
        left = min((uint64_t)((double)left / w.weight(m)), all - 1);
      }
      const int id = block_pick(c * kChunk, min(V, (c + 1) * kChunk), left, [&](int v) {
        const float l = src.logit(v);
        return l > -__builtin_inff() ? wc.fixed(l) : 0ull;
      }, sc);
      sample_store(s, row, id, w.weight(src.logit(id)), total, ws.shift);
      return;
    }
  }

  // A key that every kept token (for top-p after top-k: every one of the first k)
  // reaches; 0: none found.
  const float* gmax = ws.gmax + row * ws.groups;
  uint32_t bound = 0;
  const uint64_t p_mass = r.p < 1.f && r.k == 0 ? scaled_ceil(r.p, total) : 0;
  if (r.k > 0 || p_mass > 0) {
    sh.h.count[tid] = 0;
    sh.h.mass[tid] = 0;
    __syncthreads();
    for (int g = tid; g < ws.groups; g += kSampleThreads) {
      const float m = gmax[g];
      if (m > -__builtin_inff()) {
        const int b = sample_bin(m, top);
        atomicAdd(&sh.h.count[b], 1u);
        if (p_mass > 0) atomicAdd((unsigned long long*)&sh.h.mass[b], (unsigned long long)w.fixed(m));
      }
    }
    __syncthreads();
    uint64_t all, unused1, unused2;
    const uint64_t upto = block_scan(r.k > 0 ? (uint64_t)sh.h.count[tid] : sh.h.mass[tid], &all, sc);
    const int b = block_first(upto >= (r.k > 0 ? (uint64_t)r.k : p_mass), 0, 0, &unused1, &unused2, sc);
    if (b >= 0) bound = sample_bin_floor(b, top);
  }
  uint32_t minp_key = 1;
  if (r.minp > 0.f) {
    minp_key = sample_minp_key(w, top, r.minp);
    // top-p after top-k needs the mass of all of the first k
    if (!(r.k > 0 && r.p < 1.f)) bound = max(bound, minp_key);
  }
  if (bound == 0 && V <= kList) bound = 1;

  // the groups that reach the bound, then their tokens that do, both in id order
  int n = -1;
  if (bound != 0) {
    const int per = (ws.groups + kSampleThreads - 1) / kSampleThreads;
    const int g0 = tid * per, g1 = min(g0 + per, ws.groups);
    uint32_t mine = 0;
    for (int g = g0; g < g1; g++) mine += sample_key(gmax[g]) >= bound;
    uint64_t ng;
    uint32_t at = (uint32_t)block_scan(mine, &ng, sc) - mine;
    if (ng <= kList) {
      for (int g = g0; g < g1; g++)
        if (sample_key(gmax[g]) >= bound) sh.groups[at++] = (uint32_t)g;
      __syncthreads();
      const int items = (int)ng << ws.group_log2;
      const int seg = ((items + kSampleThreads - 1) / kSampleThreads) * 64;  // per wave, whole wave steps
      const int i0 = wv * seg, i1 = min(i0 + seg, items);
      auto key_at = [&](int i, int* v) {
        *v = (int)(sh.groups[i >> ws.group_log2] << ws.group_log2) + (i & ((1 << ws.group_log2) - 1));
        return *v < V ? sample_key(src.logit(*v)) : 0u;
      };
      uint32_t hits = 0;
      for (int i = i0; i < i1; i += 64) {
        int v;
        const bool hit = i + lane < i1 && key_at(i + lane, &v) >= bound;
        hits += (uint32_t)__popcll(__ballot(hit));
      }
      if (lane == 0) sh.wave_count[wv] = hits;
      __syncthreads();
      uint32_t base = 0, sum = 0;
#pragma unroll
      for (int i = 0; i < kSampleWaves; i++) {
        if (i < wv) base += sh.wave_count[i];
        sum += sh.wave_count[i];
      }
      if (sum <= kList) {
        n = (int)sum;
        for (int i = i0; i < i1; i += 64) {
          int v = 0;
          const uint32_t key = i + lane < i1 ? key_at(i + lane, &v) : 0u;
          const uint64_t m = __ballot(key >= bound);
          if (key >= bound) {
            const uint64_t x = ((uint64_t)key << 32) | (uint32_t)~(uint32_t)v;
            const uint32_t to = base + (uint32_t)__popcll(m & ((1ull << lane) - 1));
            sh.list[to] = x;
            sh.sorted[to] = x;
          }
          base += (uint32_t)__popcll(m);
        }
      }
    }
  }
  if (n < 0) {  // too many tokens for the list
    if (heavy) {
      if (tid == 0) sc.index[0] = atomicAdd(ws.nheavy, 1u);
      __syncthreads();
      const uint32_t slot = sc.index[0];
      if (slot < (uint32_t)ws.slots) {
        if (tid == 0) ws.flag[row] = (int32_t)slot;
        return;
      }
    }
    __syncthreads();
    sample_by_passes<DT>(s, row, top, ws.shift, sh.h, sc);
    return;
  }

  // sort descending (bitonic, empty entries 0 last)
  int size = 64;
  while (size < n) size <<= 1;
  for (int i = n + tid; i < size; i += kSampleThreads) {
    sh.sorted[i] = 0;
    sh.list[i] = 0;
  }
  __syncthreads();
  for (int len = 2; len <= size; len <<= 1) {
    for (int step = len >> 1; step > 0; step >>= 1) {
      for (int i = tid; i < size / 2; i += kSampleThreads) {
        const int a = 2 * step * (i / step) + i % step, b = a + step;
        const uint64_t x = sh.sorted[a], y = sh.sorted[b];
        if ((x < y) == ((a & len) == 0)) {
          sh.sorted[a] = y;
          sh.sorted[b] = x;
        }
      }
      __syncthreads();
    }
  }

  // prefix masses in the row's order, two tokens per thread; the number kept
  static_assert(kList == 2 * kSampleThreads, "two tokens per thread");
  const uint64_t x0 = sh.sorted[min(2 * tid, size - 1)], x1 = sh.sorted[min(2 * tid + 1, size - 1)];
  const bool have0 = 2 * tid < n, have1 = 2 * tid + 1 < n;
  const float l0 = ord_score((uint32_t)(x0 >> 32)), l1 = ord_score((uint32_t)(x1 >> 32));
  const uint64_t m0 = have0 ? w.fixed(l0) : 0, m1 = have1 ? w.fixed(l1) : 0;
  uint64_t all;
  const uint64_t upto1 = block_scan(m0 + m1, &all, sc), upto0 = upto1 - m1;
  uint64_t n_keep = (uint64_t)n, unused;
  if (r.k > 0) n_keep = min(n_keep, (uint64_t)r.k);
  uint64_t goal = p_mass;
  if (r.p < 1.f && r.k > 0) {  // mass of the first k
    uint64_t mass = 0;
    const uint64_t last = n_keep - 1;
    block_first((uint64_t)tid == last / 2, last & 1 ? upto1 : upto0, 0, &mass, &unused, sc);
    goal = scaled_ceil(r.p, mass);
  }
  if (goal > 0) {
    uint64_t len = 0;
    const bool in0 = have0 && upto0 >= goal, in1 = have1 && upto1 >= goal;
    if (block_first(in0 || in1, (uint64_t)(2 * tid + (in0 ? 1 : 2)), 0, &len, &unused, sc) >= 0)
      n_keep = min(n_keep, len);
  }
  if (r.minp > 0.f) {
    uint64_t reach;
    block_scan((uint64_t)(have0 && (uint32_t)(x0 >> 32) >= minp_key) + (have1 && (uint32_t)(x1 >> 32) >= minp_key), &reach,
               sc);
    n_keep = min(n_keep, reach);
  }
  const uint64_t last = sh.sorted[n_keep - 1];

  // the pick, in id order
  const uint64_t y0 = sh.list[min(2 * tid, size - 1)], y1 = sh.list[min(2 * tid + 1, size - 1)];
  const uint64_t k0 = have0 && y0 >= last ? w.fixed(ord_score((uint32_t)(y0 >> 32))) : 0;
  const uint64_t k1 = have1 && y1 >= last ? w.fixed(ord_score((uint32_t)(y1 >> 32))) : 0;
  const uint64_t sum1 = block_scan(k0 + k1, &total, sc);
  const uint64_t target = scaled_floor(r.u, total);
  uint64_t got = 0;
  block_first(sum1 > target, sum1 - k1 > target ? y0 : y1, 0, &got, &unused, sc);
  sample_store(s, row, (int)~(uint32_t)got, w.weight(ord_score((uint32_t)(got >> 32))), total, ws.shift);
}

// ---------------------------------------------------------------------------
// 3. Heavy rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sample_top(const SamplePtrs& ws, int64_t row) {
  float m = -__builtin_inff();
  for (int c = threadIdx.x & 63; c < ws.chunks; c += 64) m = fmaxf(m, ws.cmax[row * ws.chunks + c]);
  return wave_max_f32(m);
}

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_hist_kernel(Sample s, SamplePtrs ws) {
  constexpr int N = SampleSource<DT>::N;
  __shared__ SampleHist h;
  const int tid = threadIdx.x, c = blockIdx.x;
  for (int64_t row = blockIdx.y; row < s.rows; row += gridDim.y) {
    const int slot = ws.flag[row];
    if (slot < 0) continue;  // whole workgroup
    const SampleSource<DT> src(s, row);
    const SampleRow r = sample_row(s, row);
    const float top = sample_top(ws, row);
    const SampleWeight w(top, r.T, ws.shift);
    h.count[tid] = 0;
    h.mass[tid] = 0;
    __syncthreads();
    const int end = min(src.V, (c + 1) * kSlice);
    for (int v = c * kSlice + tid * N; v < end; v += kSampleThreads * N) {
      float l[N];
      src.load(v, l);
#pragma unroll
      for (int j = 0; j < N; j++)
        if (l[j] > -__builtin_inff()) {
          const int b = sample_bin(l[j], top);
          atomicAdd(&h.count[b], 1u);
          atomicAdd((unsigned long long*)&h.mass[b], (unsigned long long)w.fixed(l[j]));
        }
    }
    __syncthreads();
    const size_t at = ((size_t)slot * ws.slices + c) * kSampleBins + tid;
    ws.hcount[at] = h.count[tid];
    ws.hmass[at] = h.mass[tid];
    __syncthreads();
  }
}

struct SampleHeavyShared {
  SampleScratch sc;
  SampleHist h;
  uint64_t list[kHeavyList];
  uint64_t slice[kMaxSlices];
  uint32_t n;
};

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_heavy_kernel(Sample s, SamplePtrs ws) {
  __shared__ SampleHeavyShared sh;
  SampleScratch& sc = sh.sc;
  const int64_t row = blockIdx.x;
  const int slot = ws.flag[row];
  if (slot < 0) return;  // whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const SampleSource<DT> src(s, row);
  const SampleRow r = sample_row(s, row);
  const float top = sample_top(ws, row);
  const SampleWeight w(top, r.T, ws.shift);
  const uint32_t* hcount = ws.hcount + (size_t)slot * ws.slices * kSampleBins;
  const uint64_t* hmass = ws.hmass + (size_t)slot * ws.slices * kSampleBins;

  // the row's histogram, bin 0 (the largest logits) first
  uint64_t c = 0, m = 0, tc, tm;
  for (int i = 0; i < ws.slices; i++) {
    c += hcount[i * kSampleBins + tid];
    m += hmass[i * kSampleBins + tid];
  }
  const uint64_t ic = block_scan(c, &tc, sc), im = block_scan(m, &tm, sc);

  // f over the tokens of one bin: from the list if they fit there, else by a pass over the row
  int listed = -1;
  uint32_t klo = 1, khi = 0;
  int n = -1;
  auto bin_open = [&](int b) {
    if (listed == b) return;
    listed = b;
    klo = sample_bin_floor(b, top);
    khi = b == 0 ? score_ord(top) : sample_bin_floor(b - 1, top) - 1;
    uint64_t in_bin, unused;
    block_first(tid == b, c, 0, &in_bin, &unused, sc);
    n = -1;
    if (in_bin > kHeavyList) return;
    if (tid == 0) sh.n = 0;
    __syncthreads();
    sample_each<DT>(src, [&](uint32_t key, uint32_t id) {
      if (key >= klo && key <= khi) sh.list[atomicAdd(&sh.n, 1u)] = ((uint64_t)key << 32) | id;
    });
    __syncthreads();
    n = (int)sh.n;
  };
  auto each = [&](auto f) {
    if (n >= 0) {
      for (int i = tid; i < n; i += kSampleThreads) f((uint32_t)(sh.list[i] >> 32), (uint32_t)sh.list[i]);
    } else {
      sample_each<DT>(src, f);
    }
  };
  SampleCut cut;
  uint64_t mass = tm, bc, bm;
  if (r.k > 0) {
    const int b = block_first(ic >= (uint64_t)r.k, ic - c, im - m, &bc, &bm, sc);
    if (b >= 0) {  // else there are fewer candidates than k
      bin_open(b);
      mass = sample_find(each, w, src.V, &cut, klo, khi, true, (uint64_t)r.k, 0, bc, bm, sh.h, sc);
    }
  }
  if (r.p < 1.f) {
    const uint64_t goal = scaled_ceil(r.p, mass);
    const int b = block_first(im >= goal, ic - c, im - m, &bc, &bm, sc);
    bin_open(b);
    sample_find(each, w, src.V, &cut, klo, khi, false, 0, goal, bc, bm, sh.h, sc);
  }
  if (r.minp > 0.f) {
    const uint32_t key = sample_minp_key(w, top, r.minp);
    if (key > cut.key) cut.key = key, cut.id = 0xffffffffu;
  }

  // the kept mass of each slice: whole bins above the cut's, the kept tokens of that one
  const int b = sample_bin(ord_score(cut.key), top);
  bin_open(b);
  if (tid < ws.slices) sh.slice[tid] = 0;
  __syncthreads();
  for (int i = wv; i < ws.slices; i += kSampleWaves) {
    uint64_t z = 0;
    for (int j = lane; j < b; j += 64) z += hmass[i * kSampleBins + j];
    z = wave_scan_u64(z);
    if (lane == 63) atomicAdd((unsigned long long*)&sh.slice[i], (unsigned long long)z);
  }
  each([&](uint32_t key, uint32_t id) {
    if (key >= klo && key <= khi && cut.keeps(key, id))
      atomicAdd((unsigned long long*)&sh.slice[id / kSlice], (unsigned long long)w.fixed(ord_score(key)));
  });
  __syncthreads();
  uint64_t total, left, unused;
  const uint64_t z = tid < ws.slices ? sh.slice[tid] : 0;
  const uint64_t upto = block_scan(z, &total, sc);
  const uint64_t target = scaled_floor(r.u, total);
  const int i = block_first(upto > target, target - (upto - z), 0, &left, &unused, sc);
  const int id = block_pick(i * kSlice, min(src.V, (i + 1) * kSlice), left, [&](int v) {
    const float l = src.logit(v);
    const uint32_t key = sample_key(l);
    return key != 0 && cut.keeps(key, (uint32_t)v) ? w.fixed(l) : 0ull;
  }, sc);
  sample_store(s, row, id, w.weight(src.logit(id)), total, ws.shift);
}

size_t sample_workspace(int64_t rows, int64_t vocab) {
  if (rows == 0) return 0;
  // 16-bit logits have no more groups than f32 ones
  return sample_ws(rows, vocab, DT_F32).bytes;
}

template <int DT>
static hipError_t launch_sample_dt(const Sample& s, const SamplePtrs& ws, bool heavy, hipStream_t stream) {
  const unsigned y = (unsigned)std::min<int64_t>(s.rows, 32768);
  hipLaunchKernelGGL((sample_chunk_kernel<DT>), dim3((unsigned)ws.chunks, y), dim3(kChunkThreads), 0, stream, s, ws);
  hipLaunchKernelGGL((sample_row_kernel<DT>), dim3((unsigned)s.rows), dim3(kSampleThreads), 0, stream, s, ws,
                     (int)heavy);
  if (heavy) {
    hipLaunchKernelGGL((sample_hist_kernel<DT>), dim3((unsigned)ws.slices, y), dim3(kSampleThreads), 0, stream, s, ws);
    hipLaunchKernelGGL((sample_heavy_kernel<DT>), dim3((unsigned)s.rows), dim3(kSampleThreads), 0, stream, s, ws);
  }
  return hipGetLastError();
}

hipError_t launch_sample(const Sample& s, void* space, hipStream_t stream) {
  const SampleWs w = sample_ws(s.rows, s.vocab, s.dtype);
  uint8_t* base = (uint8_t*)space;
  SamplePtrs p;
  p.gmax = (float*)(base + w.gmax);
  p.cmax = (float*)(base + w.cmax);
  p.csum = (uint64_t*)(base + w.csum);
  p.flag = (int32_t*)(base + w.flag);
  p.nheavy = (uint32_t*)(base + w.nheavy);
  p.hcount = (uint32_t*)(base + w.hcount);
  p.hmass = (uint64_t*)(base + w.hmass);
  p.chunks = w.chunks;
  p.slices = w.slices;
  p.group_log2 = w.group_log2;
  p.groups = w.groups;
  p.slots = w.slots;
  int bits = 0;
  while ((1ll << bits) < s.vocab) bits++;
  p.shift = std::min(45, 63 - bits);
  // Rows whose settings may keep more than the list holds: the histogram kernels are
  // launched for them.  With one small k for all rows only ties can overflow the list,
  // which the row kernel then sorts out by itself.
  const bool small_k = s.d_top_k == nullptr && s.top_k > 0 && s.top_k <= kList / 2;
  const bool no_filter = s.d_top_k == nullptr && s.top_k == 0 && s.d_top_p == nullptr && s.top_p == 1.f &&
                         s.d_min_p == nullptr && s.min_p == 0.f;
  const bool heavy = s.vocab > kList && !small_k && !no_filter;
  if (s.dtype == DT_F32) return launch_sample_dt<DT_F32>(s, p, heavy, stream);
  if (s.dtype == DT_BF16) return launch_sample_dt<DT_BF16>(s, p, heavy, stream);
  return launch_sample_dt<DT_F16>(s, p, heavy, stream);
}

}  // namespace etg
