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
// not depend on the order in which threads add, so a call repeats bitwise, and the kept
// tokens of a row with filters weigh exactly the same where their logits are equal.  With
// vocab <= 2^b the sum is at most 2^(b + shift) <= 2^63: shift = min(45, 63 - b).  A weight
// is off by at most half a unit, a total (at least 2^shift) by 2^(b - shift - 1) of itself:
// 2^-28 at 2^18 tokens and 2^-24 at the largest vocabulary, 2^20.  The chunk masses of kernel
// 1 are relative to each chunk's own largest logit and are rounded again when they are
// brought to the row's, by half a unit and about 2^-47 of themselves (the exponent of what
// they are multiplied with, below 46 where it counts, carries roundings of 2^-53): a draw
// without filters, and the total that top-p alone goes by, are that near.
//
// Kernels:
//  1. sample_chunk_kernel streams the logits once, a wave per 2,048 tokens: the
//     maximum of every small group of tokens and of the chunk and, for rows whose
//     filters need it, the chunk's mass.
//  2. sample_row_kernel, a workgroup per row.  A row without filters picks a chunk by
//     the chunk masses and a token in it.  Otherwise the group maxima give a lower bound
//     of the cut: if the k largest maxima reach a value, so do k tokens, and if the
//     maxima above a value weigh p times the total, so does the nucleus.  Only the groups
//     that reach the bound are read again, and their tokens at or above it (a few more
//     than are kept) are sorted in LDS.
//  3. Rows with more tokens at the bound than the list holds (flat distributions, and close
//     logits: bin 0 of the bound's bins is all that lies within 1/8 of the largest logit,
//     whatever the temperature) go on to sample_hist_kernel, which counts and weighs every
//     token in 1,024 bins per slice of 16,384 tokens, sample_gather_kernel, which lists the
//     tokens of the bin that holds the cut, and sample_heavy_kernel, which narrows the list
//     to the cut.

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
static constexpr int kChunk = 2048;              // tokens of a chunk (a wave's)
static constexpr int kChunkThreads = 256;
static constexpr int kSlice = 16384;             // tokens of a histogram slice
static constexpr int kMaxSlices = (1 << 20) / kSlice;
// Tokens sorted in LDS by the row kernel.  1,024 x 151,936 bf16 rows of mixed settings: 2,048
// 250 us, 1,024 357 (more heavy rows), 4,096 276 (one workgroup less per CU).
static constexpr int kList = 2048;
static constexpr int kHeavyList = 8192;          // tokens of one bin in the heavy kernel
static constexpr int kMaxGroups = 4096;          // groups per row
// Most workspace for heavy rows, a slot each; the rest go by passes over their logits (1,024
// x 262,144 f32 rows, all heavy: 256 MiB 1,490 us, 128 MiB 2,358).
static constexpr size_t kHeavyBytes = 256 << 20;

// Where the first cut of a heavy row lies.
struct SampleState {
  int32_t filter;  // which filter makes it: 0 min-p or none, 1 top-k, 2 top-p
  int32_t bin;     // the bin that holds it
  int32_t listed;  // whether the bin's tokens are in the slot's list
  int32_t pad;
  uint64_t goal;                        // top-p's mass
  uint64_t before_count, before_mass;   // of the bins before it
};

// Workspace of a call, from its sizes alone.
struct SampleWs {
  int chunks, slices, group_log2, groups, slots;
  size_t gmax, cmax, csum, heavy, nheavy, hcount, hmass, hlist, hlisted, hstate, bytes;
};

static SampleWs sample_ws(int64_t rows, int64_t vocab, int32_t dtype) {
  SampleWs w;
  w.chunks = (int)cdiv(vocab, kChunk);
  w.slices = (int)cdiv(vocab, kSlice);
  // groups of one 16-byte load (4 or 8 tokens) or more (256 at 2^20 tokens)
  w.group_log2 = dtype == DT_F32 ? 2 : 3;
  while (cdiv(vocab, 1ll << w.group_log2) > kMaxGroups) w.group_log2++;
  w.groups = (int)cdiv(vocab, 1ll << w.group_log2);
  const size_t slot = (size_t)w.slices * kSampleBins * 12 + kHeavyList * 8;
  w.slots = (int)std::min<int64_t>(rows, (int64_t)(kHeavyBytes / slot));
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at = align_up(at + n, 256);
    return o;
  };
  w.gmax = take((size_t)rows * w.groups * 4);
  w.cmax = take((size_t)rows * w.chunks * 4);
  w.csum = take((size_t)rows * w.chunks * 8);
  w.heavy = take((size_t)rows * 4);
  w.nheavy = take(4);
  w.hcount = take((size_t)w.slots * w.slices * kSampleBins * 4);
  w.hmass = take((size_t)w.slots * w.slices * kSampleBins * 8);
  w.hlist = take((size_t)w.slots * kHeavyList * 8);
  w.hlisted = take((size_t)w.slots * 4);
  w.hstate = take((size_t)w.slots * sizeof(SampleState));
  w.bytes = at;
  return w;
}

struct SamplePtrs {
  float* gmax;       // [rows][groups] largest candidate logit, -inf for none
  float* cmax;       // [rows][chunks]
  uint64_t* csum;    // [rows][chunks] mass relative to the chunk's own maximum
  uint32_t* nheavy;  // how many heavy rows there are
  int32_t* heavy;    // [rows] which; the first `slots` of them have histograms
  uint32_t* hcount;  // [slots][slices][bins]
  uint64_t* hmass;
  uint64_t* hlist;    // [slots][kHeavyList] tokens of the bin that holds the cut, key << 32 | id
  uint32_t* hlisted;  // [slots] how many there are
  SampleState* hstate;  // [slots]
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
  // rint(weight * 2^shift): at most 2^45, so adding 2^52 leaves it in the low bits.  0 for
  // -inf and NaN (the maximum of NaN and a number is the number).
  __device__ __forceinline__ uint64_t fixed(float l) const {
    const double y = (double)l == M ? 0.0 : power(l);
    const double x = scaled_exp2(y, shift) + 4503599627370496.0;
    return (uint64_t)__double_as_longlong(x) & 0xfffffffffffffull;
  }
};

// floor or ceil of f * m for a float f in [0, 1] (-0 included) and an integer m, exactly: f is
// a 24-bit integer times a power of two, the product 88 bits.
__device__ __forceinline__ uint64_t scaled(float f, uint64_t m, bool up) {
  const uint32_t b = __float_as_uint(f) & 0x7fffffffu;
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
  // tokens [v, v + N) (v a multiple of N, N = 4 or 8 by type), -inf past the vocabulary and
  // where barred: one 16-byte load at any alignment of the value.  A NaN logit is left as it is.
  static constexpr int N = DT == DT_F32 ? 4 : 8;
  __device__ __forceinline__ u32x4 vec(int v) const {  // v + N <= V
    u32x4 w;
    __builtin_memcpy(&w, base + (size_t)v * (16 / N), 16);
    return w;
  }
  __device__ __forceinline__ void unpack(const u32x4& w, int v, float (&l)[N]) const {
#pragma unroll
    for (int j = 0; j < N; j++) {
      if constexpr (DT == DT_F32) l[j] = __uint_as_float(w[j]);
      else if constexpr (DT == DT_BF16) l[j] = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
      else l[j] = f16_bits_to_f32(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
    }
    if (allowed != nullptr) {
      const uint32_t ok = allowed[v >> 5] >> (v & 31);
#pragma unroll
      for (int j = 0; j < N; j++)
        if (!((ok >> j) & 1u)) l[j] = -__builtin_inff();
    }
  }
  __device__ __forceinline__ void load_raw(int v, float (&l)[N]) const {
    if (v + N <= V) {
      unpack(vec(v), v, l);
    } else {
#pragma unroll
      for (int j = 0; j < N; j++) l[j] = v + j < V ? logit(v + j) : -__builtin_inff();
    }
  }
  // M vectors STRIDE tokens apart from v, the lane's; `end` bounds the whole workgroup's or
  // wave's tokens: where all are in the row the loads are issued together.
  template <int M, int STRIDE>
  __device__ __forceinline__ void load_many(int v, int end, float (&l)[M][N]) const {
    if (end <= V) {
      u32x4 w[M];
#pragma unroll
      for (int i = 0; i < M; i++) w[i] = vec(v + i * STRIDE);
#pragma unroll
      for (int i = 0; i < M; i++) unpack(w[i], v + i * STRIDE, l[i]);
    } else {
#pragma unroll
      for (int i = 0; i < M; i++) load_raw(v + i * STRIDE, l[i]);
    }
  }
  __device__ __forceinline__ void load(int v, float (&l)[N]) const {
    load_raw(v, l);
#pragma unroll
    for (int j = 0; j < N; j++) l[j] = l[j] > -__builtin_inff() ? l[j] : -__builtin_inff();
  }
};

// Order key of a logit, 0 for -inf (every candidate's is larger).
__device__ __forceinline__ uint32_t sample_key(float l) { return l > -__builtin_inff() ? score_ord(l) : 0u; }

// What bounds and bins go by: the f32 distance of a logit to the row's largest one, as
// bits (which order as it does).  It never falls as the logit falls.
__device__ __forceinline__ uint32_t sample_dist(float l, float top) {
  return l == top ? 0u : __float_as_uint(top - l) & 0x7fffffffu;
}

// Bin of a logit: logarithmic in the distance, 128 bins per octave from 2^-3 to 2^5
// (nearer ones in bin 0, farther ones in the last).
static constexpr int kBinShift = 16, kBinBase = 124 << 7;
__device__ __forceinline__ int sample_bin(float l, float top) {
  return min(max((int)(sample_dist(l, top) >> kBinShift) - kBinBase, 0), kSampleBins - 1);
}
// Distances below this are those of bins up to b.
__device__ __forceinline__ uint32_t sample_bin_limit(int b) {
  return b >= kSampleBins - 1 ? 0xffffffffu : (uint32_t)(b + 1 + kBinBase) << kBinShift;
}

// The smallest key for which reaches(logit) holds, given that it holds for `hi` and goes on
// holding as keys grow: every lane tries a key of its own, 6 rounds.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t hi, F reaches) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0;  // does not reach it, or is no candidate's key
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo - 1) / 64 + 1;  // lane i: lo + (i + 1) step, at most hi
    const uint32_t mine = step <= (hi - lo) / (lane + 1) ? lo + (lane + 1) * step : hi;
    const uint64_t m = __ballot(reaches(ord_score(mine)));  // never 0: the last lane's is hi, as 64 step >= hi - lo
    const uint32_t i = (uint32_t)__ffsll((unsigned long long)m) - 1;
    const uint32_t to = step <= (hi - lo) / (i + 1) ? lo + (i + 1) * step : hi;
    lo += i * step;
    hi = to;
  }
  return hi;
}

// The smallest key whose bin is at most b (keys below -inf's decode to NaN: the last bin).
__device__ __forceinline__ uint32_t sample_bin_floor(int b, float top) {
  if (b >= kSampleBins - 1) return 1;
  return first_key(score_ord(top), [&](float l) { return sample_bin(l, top) <= b; });
}

// The smallest key whose weight reaches minp (weights do not fall as keys grow).
__device__ __forceinline__ uint32_t sample_minp_key(const SampleWeight& w, float top, float minp) {
  return first_key(score_ord(top), [&](float l) { return w.weight(l) >= (double)minp; });
}

// ---------------------------------------------------------------------------
// Workgroup primitives (NW waves); every one begins and ends with the shared scratch
// free to reuse.
// ---------------------------------------------------------------------------
template <int NW>
struct SampleScratch {
  uint64_t part[NW];
  uint64_t value[2];
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

__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {  // lane uniform
  return ((uint64_t)__builtin_amdgcn_readlane((uint32_t)(v >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((uint32_t)v, lane);
}

// Inclusive prefix sum over the threads; *total receives the sum.  Every wave sums the
// waves' parts by itself, a part per lane.
template <int NW>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* total, SampleScratch<NW>& sc) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  v = wave_scan_u64(v);
  __syncthreads();
  if (lane == 63) sc.part[wv] = v;
  __syncthreads();
  uint64_t p = lane < NW ? sc.part[lane] : 0;
#pragma unroll
  for (int off = 1; off < NW; off <<= 1) {
    const uint64_t o = (uint64_t)__shfl_up((unsigned long long)p, off, 64);
    if (lane >= off) p += o;
  }
  *total = lane_u64(p, NW - 1);
  if (wv > 0) v += lane_u64(p, wv - 1);
  __syncthreads();
  return v;
}

// The first thread with `hit`, and the two values it holds, to every thread; -1 for none.
template <int NW>
__device__ __forceinline__ int block_first(bool hit, uint64_t a, uint64_t b, uint64_t* oa, uint64_t* ob,
                                           SampleScratch<NW>& sc) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint64_t m = __ballot(hit);
  __syncthreads();
  if (lane == 0) sc.part[wv] = m;
  __syncthreads();
  const uint64_t p = lane < NW ? sc.part[lane] : 0;
  const uint64_t waves = __ballot(p != 0);
  int first = -1;
  if (waves != 0) {
    const int w = __ffsll((unsigned long long)waves) - 1;
    first = 64 * w + __ffsll((unsigned long long)lane_u64(p, w)) - 1;
    if ((int)threadIdx.x == first) {
      sc.value[0] = a;
      sc.value[1] = b;
    }
  }
  __syncthreads();
  if (first >= 0) {
    *oa = sc.value[0];
    *ob = sc.value[1];
  }
  __syncthreads();
  return first;
}

// The token of [lo, hi) (lo a multiple of 8) in which the running mass first exceeds
// target, which the range's mass exceeds; weigh(l, v) is the mass of token v with logit l.
template <int NW, int DT, typename F>
__device__ __forceinline__ int block_pick(const SampleSource<DT>& src, int lo, int hi, uint64_t target, F weigh,
                                          SampleScratch<NW>& sc) {
  constexpr int N = SampleSource<DT>::N;
  for (int at = lo; at < hi; at += N * 64 * NW) {
    const int v = at + N * (int)threadIdx.x;
    float l[N];
#pragma unroll
    for (int j = 0; j < N; j++) l[j] = -__builtin_inff();
    if (v < hi) src.load(v, l);
    uint64_t w[N], sum = 0;
#pragma unroll
    for (int j = 0; j < N; j++) {
      w[j] = l[j] > -__builtin_inff() && v + j < hi ? weigh(l[j], v + j) : 0;
      sum += w[j];
    }
    uint64_t total;
    const uint64_t upto = block_scan(sum, &total, sc);
    if (total > target) {
      uint64_t run = upto - sum;
      int id = v;
#pragma unroll
      for (int j = 0; j < N; j++) {
        if (run <= target) id = v + j;  // the last token that begins at or below the target
        run += w[j];
      }
      uint64_t got, unused;
      block_first(upto > target, (uint64_t)id, 0, &got, &unused, sc);
      return (int)got;
    }
    target -= total;
  }
  return lo;  // not reached
}

// ---------------------------------------------------------------------------
// 1. Chunks
// ---------------------------------------------------------------------------
// The larger of a maximum and a logit, which may be any NaN.  v_max_f32 passes over a quiet NaN,
// but makes a signaling one its (quiet) result and so loses m: the logit is quieted first.
__device__ __forceinline__ float max_logit(float m, float l) { return fmaxf(m, __builtin_canonicalizef(l)); }

// Max over groups of 2^steps lanes (DPP within 16-lane rows), to every lane of the group.
__device__ __forceinline__ float group_max(float m, int steps) {
  auto dpp = [&](auto ctrl) {
    return fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), decltype(ctrl)::value, 0xf, 0xf,
                                                               true)));
  };
  if (steps > 0) m = dpp(std::integral_constant<int, 0xb1>{});   // quad_perm 1,0,3,2
  if (steps > 1) m = dpp(std::integral_constant<int, 0x4e>{});   // quad_perm 2,3,0,1
  if (steps > 2) m = dpp(std::integral_constant<int, 0x141>{});  // row_half_mirror
  if (steps > 3) m = dpp(std::integral_constant<int, 0x140>{});  // row_mirror
  if (steps > 4) m = fmaxf(m, __shfl_xor(m, 16, 64));
  if (steps > 5) m = fmaxf(m, __shfl_xor(m, 32, 64));
  return m;
}

// A wave per chunk, no workgroup synchronisation: bound by the logits' bytes (8 or 4
// 16-byte loads in flight per lane) where no mass is needed, else by about 25 f64
// operations per token.  64 x 262,144 f32 of mixed settings: 19 us; 1,024 x 151,936
// bf16: 82 us, 3.8 TB/s; 1 row 4.5 us.  (Each token weighed against its chunk's maximum: the
// row's is not known yet, and the row kernel rescales one sum per chunk.)
template <int DT>
__global__ void __launch_bounds__(kChunkThreads) sample_chunk_kernel(Sample s, SamplePtrs ws) {
  using Src = SampleSource<DT>;
  constexpr int N = Src::N, NV = kChunk / (64 * N);
  const int lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * (kChunkThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit == 0 && lane == 0) *ws.nheavy = 0;
  const int64_t row = unit / (uint32_t)ws.chunks;  // units: at most 2^16 rows of 2^9 chunks
  const int c = (int)(unit % (uint32_t)ws.chunks);
  if (row >= s.rows) return;  // whole wave, no barrier
  const int steps = ws.group_log2 - (DT == DT_F32 ? 2 : 3);
  const Src src(s, row);
  float l[NV][N];
  src.template load_many<NV, 64 * N>(c * kChunk + lane * N, (c + 1) * kChunk, l);
  const SampleRow r = sample_row(s, row);
  float m = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < NV; j++) {
    float g = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < N; e++) g = max_logit(g, l[j][e]);
    g = group_max(g, steps);
    const int v = c * kChunk + (j * 64 + lane) * N;
    if ((lane & ((1 << steps) - 1)) == 0 && v < src.V) ws.gmax[row * ws.groups + (v >> ws.group_log2)] = g;
    m = fmaxf(m, g);
  }
  m = wave_max_f32(m);
  if (lane == 0) ws.cmax[unit] = m;
  if (r.k != 0 || !(r.p < 1.f || r.minp == 0.f) || !r.ok) return;  // no filter of this row needs the mass
  uint64_t sum = 0;
  if (m > -__builtin_inff()) {
    const SampleWeight w(m, r.T, ws.shift);
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int e = 0; e < N; e++) sum += w.fixed(l[j][e]);
  }
  sum = wave_scan_u64(sum);
  if (lane == 63) ws.csum[unit] = sum;
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

// f(key, id) for every candidate of a row, the vocabulary dealt to the threads, four
// loads in flight each (one workgroup reads a whole row: latency is what it waits for).
template <int NT, int DT, typename F>
__device__ __forceinline__ void sample_each(const SampleSource<DT>& src, F f) {
  constexpr int N = SampleSource<DT>::N, U = 16 / N;
  for (int at = 0; at < src.V; at += NT * N * U) {
    float l[U][N];
    src.template load_many<U, NT * N>(at + (int)threadIdx.x * N, at + NT * N * U, l);
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int j = 0; j < N; j++)
        if (l[u][j] > -__builtin_inff()) f(score_ord(l[u][j]), (uint32_t)(at + (u * NT + (int)threadIdx.x) * N + j));
  }
}

// Tokens of one row between two keys: in an LDS list where they fit, else the row itself.
template <int NT, int DT>
struct SampleRange {
  const SampleSource<DT>& src;
  const SampleWeight& w;
  uint64_t* list;  // key << 32 | id, in no order
  uint64_t* mass;  // of the list's tokens
  uint32_t* size;
  int n = -1;      // entries of the list; -1: the row
  __device__ __forceinline__ SampleRange(const SampleSource<DT>& s_, const SampleWeight& w_, uint64_t* l_, uint64_t* m_,
                                         uint32_t* n_)
      : src(s_), w(w_), list(l_), mass(m_), size(n_) {}
  // f(key, id, mass()) for its tokens
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (n >= 0) {
      for (int i = threadIdx.x; i < n; i += NT) f((uint32_t)(list[i] >> 32), (uint32_t)list[i], [&] { return mass[i]; });
    } else {
      sample_each<NT>(src, [&](uint32_t key, uint32_t id) { f(key, id, [&] { return w.fixed(ord_score(key)); }); });
    }
  }
  // after the list was filled: weighs it (each thread the entries that it visits)
  __device__ __forceinline__ void weigh() {
    for (int i = threadIdx.x; i < n; i += NT) mass[i] = w.fixed(ord_score((uint32_t)(list[i] >> 32)));
  }
  // lists the row's candidates with keys in [klo, khi] if they fit
  __device__ __forceinline__ void gather(uint32_t klo, uint32_t khi) {
    if (threadIdx.x == 0) *size = 0;
    __syncthreads();
    sample_each<NT>(src, [&](uint32_t key, uint32_t id) {
      if (key >= klo && key <= khi) {
        const uint32_t i = atomicAdd(size, 1u);
        if (i < kHeavyList) list[i] = ((uint64_t)key << 32) | id;
      }
    });
    __syncthreads();
    n = *size <= kHeavyList ? (int)*size : -1;
    weigh();
    __syncthreads();
  }
};

// Narrows *cut to the element at which the prefix of its kept elements first holds
// `count` of them (by_count) or `mass`; returns the prefix's mass.  That element's key
// lies in [klo, khi], whose tokens `range` holds; before_count and before_mass are those
// of the keys above khi.  1,024 bins per round (a bin per thread), then the same on the
// ids of the last key.
template <int DT>
__device__ __forceinline__ uint64_t sample_find(SampleRange<kSampleThreads, DT>& range, const SampleWeight& w,
                                                SampleCut* cut, uint32_t klo, uint32_t khi, bool by_count,
                                                uint64_t count, uint64_t mass, uint64_t before_count,
                                                uint64_t before_mass, SampleHist& h,
                                                SampleScratch<kSampleWaves>& sc) {
  const int tid = threadIdx.x;
  const SampleCut old = *cut;
  uint64_t of_key = ~0ull;  // kept elements with the last key, where known
  while (klo < khi) {
    const int sh = max(0, 22 - __clz((int)(khi - klo)));  // (khi - klo) >> sh < 1024
    h.count[tid] = 0;
    h.mass[tid] = 0;
    __syncthreads();
    range.each([&](uint32_t key, uint32_t id, auto mass_of) {
      if (key >= klo && key <= khi && old.keeps(key, id)) {
        const int b = (int)((key - klo) >> sh);
        atomicAdd(&h.count[b], 1u);
        atomicAdd((unsigned long long*)&h.mass[b], (unsigned long long)mass_of());
      }
    });
    __syncthreads();
    const uint64_t c = h.count[kSampleBins - 1 - tid], m = h.mass[kSampleBins - 1 - tid];
    uint64_t tc, tm, bc, bm;
    const uint64_t ic = before_count + block_scan(c, &tc, sc), im = before_mass + block_scan(m, &tm, sc);
    const uint64_t counts = (ic - c) << 32 | c;  // each at most the vocabulary
    // the first bin from the top that reaches the target, else the last that holds any
    int t = block_first(c != 0 && (by_count ? ic >= count : im >= mass), counts, im - m, &bc, &bm, sc);
    if (t < 0) t = block_first(c != 0 && ic == before_count + tc, counts, im - m, &bc, &bm, sc);
    const int bin = kSampleBins - 1 - t;
    before_count = bc >> 32;
    before_mass = bm;
    if (sh == 0) of_key = (uint32_t)bc;
    klo += (uint32_t)bin << sh;
    khi = min(khi, klo + ((1u << sh) - 1));
    __syncthreads();
    if (range.n < 0 && sh > 0) range.gather(klo, khi);
  }
  const uint64_t wk = w.fixed(ord_score(klo));
  uint64_t ties = by_count ? count - before_count : wk != 0 ? (mass - before_mass + wk - 1) / wk : ~0ull >> 1;
  if (ties >= of_key) {  // all elements with the key, as where there is one
    cut->id = old.key == klo ? old.id : 0xffffffffu;
    cut->key = klo;
    return before_mass + of_key * wk;
  }
  // the id of the last of `ties` elements with the key
  uint32_t ilo = 0, ihi = (uint32_t)range.src.V - 1;
  uint64_t passed = 0;
  do {
    const int sh = max(0, 22 - __clz((int)(ihi - ilo)));
    h.count[tid] = 0;
    __syncthreads();
    range.each([&](uint32_t key, uint32_t id, auto) {
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

__device__ __forceinline__ void sample_store(const Sample& s, int64_t row, int id, double w, uint64_t total, int shift) {
  if (threadIdx.x == 0) {
    s.ids[row] = id;
    s.probs[row] = (float)(ldexp(w, shift) / (double)total);
  }
}

// ---------------------------------------------------------------------------
// 2. Rows
// ---------------------------------------------------------------------------
static constexpr int kRowThreads = 512;
static constexpr int kRowWaves = kRowThreads / 64;

struct SampleRowShared {
  SampleScratch<kRowWaves> sc;
  uint64_t list[kList];  // the tokens at or above the bound in id order: key << 32 | ~id
  union {
    struct {
      SampleHist h;
      uint32_t groups[kList];  // groups that reach the bound, in order
    };
    struct {
      uint64_t sorted[kList];  // the list in the row's order
      uint64_t mass[kList];
    };
  };
  uint32_t wave_count[kRowWaves];
  uint32_t bin_end[kSampleBins];
};

// A row is a chain of short dependent steps (1 row 17 us, 64 rows 40 us, 1,024 rows 78 us):
// bound by latency, its barriers and LDS searches.  512 threads: 1,024 synchronise more
// slowly (one row, top-k of 50: 27.6 us per call against 23.7), 256 read a long list's
// groups more slowly (64 rows, top-k of 1,000: 73.9 against 57.7, while the short lists of
// 1,024 rows gain a little, 89.3 against 97.0).
template <int DT>
__global__ void __launch_bounds__(kRowThreads) sample_row_kernel(Sample s, SamplePtrs ws) {
  __shared__ SampleRowShared sh;
  SampleScratch<kRowWaves>& sc = sh.sc;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const SampleSource<DT> src(s, row);
  const SampleRow r = sample_row(s, row);
  const int V = src.V;

  // loaded before anything waits
  constexpr int G = kMaxGroups / kRowThreads;  // consecutive groups of a thread, kept in registers
  float gm[G];
#pragma unroll
  for (int q = 0; q < G; q++) {
    const int g = G * tid + q;
    gm[q] = g < ws.groups ? ws.gmax[row * ws.groups + g] : -__builtin_inff();
  }

  // the row's largest logit
  const float* cmax = ws.cmax + row * ws.chunks;
  float top = -__builtin_inff();
  for (int c = tid; c < ws.chunks; c += kRowThreads) top = fmaxf(top, cmax[c]);
  top = wave_max_f32(top);
  if (lane == 0) sc.part[wv] = __float_as_uint(top);
  for (int i = tid; i < kSampleBins; i += kRowThreads) {
    sh.h.count[i] = 0;
    sh.h.mass[i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowWaves; i++) top = fmaxf(top, __uint_as_float((uint32_t)sc.part[i]));
  if (!(top > -__builtin_inff()) || !r.ok) {  // whole workgroup
    if (tid == 0) {
      s.ids[row] = -1;
      s.probs[row] = 0.f;
    }
    return;
  }
  const SampleWeight w(top, r.T, ws.shift);
  uint64_t total = 0, unused, unused2;
  if (r.k == 0 && (r.p < 1.f || r.minp == 0.f)) {
    // chunk masses to the row's maximum: a chunk at it keeps its integer sum
    const uint64_t* csum = ws.csum + row * ws.chunks;
    const int per = (ws.chunks + kRowThreads - 1) / kRowThreads, c0 = tid * per, c1 = min(c0 + per, ws.chunks);
    auto chunk_mass = [&](int c) -> uint64_t {
      const float m = cmax[c];
      if (!(m > -__builtin_inff())) return 0;
      return m == top ? csum[c] : (uint64_t)rint((double)csum[c] * w.weight(m));
    };
    uint64_t z = 0;
    for (int c = c0; c < c1; c++) z += chunk_mass(c);
    const uint64_t upto = block_scan(z, &total, sc);
    if (r.p == 1.f) {  // no filter: the chunk, then the token by weights relative to the chunk's maximum
      const uint64_t target = scaled_floor(r.u, total);
      uint64_t left = target - (upto - z), mine = (uint64_t)c0, chunk;
      if (upto > target && upto - z <= target)
        for (int c = c0; c < c1; c++) {
          const uint64_t x = chunk_mass(c);
          mine = (uint64_t)c;
          if (x > left) break;
          left -= x;
        }
      block_first(upto > target, left, mine, &left, &chunk, sc);
      const int c = (int)chunk;
      const float m = cmax[c];
      if (m != top) left = min((uint64_t)((double)left / w.weight(m)), csum[c] - 1);
      const SampleWeight wc(m, r.T, ws.shift);
      const int id = block_pick(src, c * kChunk, min(V, (c + 1) * kChunk), left,
                                [&](float l, int) { return wc.fixed(l); }, sc);
      sample_store(s, row, id, w.weight(src.logit(id)), total, ws.shift);
      return;
    }
  }

  // Tokens nearer to the largest logit than `limit` are gathered: among them is every
  // kept token (for top-p after top-k: every one of the first k).
  uint32_t limit = 0xffffffffu;
  const uint64_t p_mass = r.p < 1.f && r.k == 0 ? scaled_ceil(r.p, total) : 0;
  if (r.k > 0 || p_mass > 0) {
#pragma unroll
    for (int q = 0; q < G; q++)
      if (gm[q] > -__builtin_inff()) {
        const int b = sample_bin(gm[q], top);
        atomicAdd(&sh.h.count[b], 1u);
        if (p_mass > 0) atomicAdd((unsigned long long*)&sh.h.mass[b], (unsigned long long)w.fixed(gm[q]));
      }
    __syncthreads();
    constexpr int Q = kSampleBins / kRowThreads;
    uint64_t x[Q], sum = 0, all, bin;
#pragma unroll
    for (int q = 0; q < Q; q++) {
      x[q] = r.k > 0 ? (uint64_t)sh.h.count[Q * tid + q] : sh.h.mass[Q * tid + q];
      sum += x[q];
    }
    const uint64_t goal = r.k > 0 ? (uint64_t)r.k : p_mass, upto = block_scan(sum, &all, sc);
    uint64_t run = upto;
    int mine = Q * tid;
#pragma unroll
    for (int q = Q - 1; q >= 0; q--) {
      if (run >= goal) mine = Q * tid + q;  // the first bin that reaches the goal
      run -= x[q];
    }
    if (block_first(upto >= goal, (uint64_t)mine, 0, &bin, &unused, sc) >= 0) limit = sample_bin_limit((int)bin);
  }
  if (r.minp > 0.f && !(r.k > 0 && r.p < 1.f)) {  // top-p after top-k needs the mass of all of the first k
    // w >= minp means a distance of at most -T ln(minp); 2^-16 of it and 1e-14 T cover
    // the rounding of this product, of the distances and of the weights
    const float most = r.T * (-logf(r.minp) * (1.f + 1.52587890625e-5f) + 1e-14f) + 1.17549435e-38f;
    const uint32_t lim = most < __builtin_inff() ? __float_as_uint(most) + 1 : 0xffffffffu;
    limit = min(limit, lim);
  }

  // the groups within the limit, then their tokens that are, both in id order
  int n = -1;
  {
    // the smallest logit within the limit: one comparison per token, which NaN and -inf fail
    const float least = limit == 0xffffffffu ? -3.40282347e38f : ord_score(first_key(score_ord(top), [&](float l) {
      return sample_dist(l, top) < limit;
    }));
    auto near = [&](float l) { return l >= least; };
    uint32_t mine = 0;
#pragma unroll
    for (int q = 0; q < G; q++) mine += near(gm[q]);
    uint64_t ng;
    uint32_t at = (uint32_t)block_scan((uint64_t)mine, &ng, sc) - mine;
    if (ng <= kList) {
#pragma unroll
      for (int q = 0; q < G; q++)
        if (near(gm[q])) sh.groups[at++] = (uint32_t)(G * tid + q);
      __syncthreads();
      // rounds of U loads per lane, a wave's loads consecutive
      constexpr int N = SampleSource<DT>::N, U = 32 / N;
      const int items = (int)ng << ws.group_log2;
      uint32_t base = 0;
      n = 0;
      for (int r0 = 0; r0 < items && n >= 0; r0 += kRowThreads * N * U) {
        float l[U][N];
        int v[U];
        uint32_t hits = 0;
        bool whole = V >= N;
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int i = r0 + ((wv * U + u) * 64 + lane) * N;
          const int g = (int)(sh.groups[min(i, items - 1) >> ws.group_log2] << ws.group_log2);
          v[u] = i < items ? g + (i & ((1 << ws.group_log2) - 1)) : V;
          whole = whole && (v[u] == V || v[u] + N <= V);
        }
        if (__all(whole)) {  // the loads of all steps together
          u32x4 w4[U];
#pragma unroll
          for (int u = 0; u < U; u++) w4[u] = src.vec(v[u] < V ? v[u] : 0);
#pragma unroll
          for (int u = 0; u < U; u++) {
            src.unpack(w4[u], v[u] < V ? v[u] : 0, l[u]);
#pragma unroll
            for (int j = 0; j < N; j++) l[u][j] = v[u] < V ? l[u][j] : -__builtin_inff();
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; u++) src.load(v[u], l[u]);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
          for (int j = 0; j < N; j++) hits += near(l[u][j]);
        // places in (wave, u, lane, j) order
        uint32_t wave_hits = hits;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) wave_hits += __shfl_xor(wave_hits, off, 64);
        if (lane == 0) sh.wave_count[wv] = wave_hits;
        __syncthreads();
        uint32_t to = base, sum = 0;
#pragma unroll
        for (int i = 0; i < kRowWaves; i++) {
          const uint32_t x = sh.wave_count[i];
          if (i < wv) to += x;
          sum += x;
        }
        if (base + sum > kList) {
          n = -1;  // whole workgroup
        } else if (wave_hits != 0) {
#pragma unroll
          for (int u = 0; u < U; u++) {
            uint32_t place = to, hits_u = 0;
#pragma unroll
            for (int j = 0; j < N; j++) {
              const uint64_t m = __ballot(near(l[u][j]));
              place += __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
              hits_u += (uint32_t)__popcll(m);
            }
            if (hits_u == 0) continue;
#pragma unroll
            for (int j = 0; j < N; j++)
              if (near(l[u][j]))
                sh.list[place++] = ((uint64_t)score_ord(l[u][j]) << 32) | (uint32_t)~(uint32_t)(v[u] + j);
            to += hits_u;
          }
        }
        base += sum;
        if (n >= 0) n = (int)base;
        __syncthreads();
      }
    }
  }
  if (n < 0) {  // too many tokens for the list: a heavy row
    if (tid == 0) {
      const uint32_t i = atomicAdd(ws.nheavy, 1u);
      ws.heavy[i] = (int32_t)row;
      if (i < (uint32_t)ws.slots) ws.hlisted[i] = 0;
    }
    return;
  }
  __syncthreads();

  // Sort descending.  Short lists: a token's place is the number of larger ones.  Longer ones:
  // by bins first (a scan of their counts), where a token's place in its bin is counted the
  // same way; where a bin holds many, the whole list bitonically, empty entries 0 last.
  int size = kRowThreads;
  while (size < n) size <<= 1;
  bool done = size == kRowThreads;
  if (done) {
    const uint64_t x = tid < n ? sh.list[tid] : 0;
    int rank = 0;
    for (int i = 0; i < n; i++) rank += sh.list[i] > x;
    if (tid < n) sh.sorted[rank] = x;
    __syncthreads();
  } else {
    constexpr int Q = kSampleBins / kRowThreads, MANY = 128;
    uint64_t* binned = sh.mass;
    float low = top;  // the smallest logit of the list
    for (int i = tid; i < kSampleBins; i += kRowThreads) sh.bin_end[i] = 0;
    for (int i = tid; i < n; i += kRowThreads) low = fminf(low, ord_score((uint32_t)(sh.list[i] >> 32)));
    low = -wave_max_f32(-low);
    if (lane == 0) sc.part[wv] = __float_as_uint(low);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowWaves; i++) low = fminf(low, __uint_as_float((uint32_t)sc.part[i]));
    // equal bins from the largest to the smallest; logits too far apart or equal fall into one
    const float per_bin = fminf((float)(kSampleBins - 1) / (top - low), 3e38f);
    auto bin_of = [&](uint64_t x) {
      return (int)fminf(fmaxf((top - ord_score((uint32_t)(x >> 32))) * per_bin, 0.f), (float)(kSampleBins - 1));
    };
    for (int i = tid; i < n; i += kRowThreads) atomicAdd(&sh.bin_end[bin_of(sh.list[i])], 1u);
    __syncthreads();
    uint32_t count[Q], sum = 0;
    bool many = false;
#pragma unroll
    for (int q = 0; q < Q; q++) {
      count[q] = sh.bin_end[Q * tid + q];
      many |= count[q] > MANY;
      sum += count[q];
    }
    uint64_t all;
    uint32_t start = (uint32_t)block_scan((uint64_t)sum, &all, sc) - sum;
    if (block_first(many, 0, 0, &unused, &unused2, sc) < 0) {
#pragma unroll
      for (int q = 0; q < Q; q++) {  // each bin's start, which the placing turns into its end
        sh.bin_end[Q * tid + q] = start;
        start += count[q];
      }
      __syncthreads();
      for (int i = tid; i < n; i += kRowThreads) {
        const uint64_t x = sh.list[i];
        binned[atomicAdd(&sh.bin_end[bin_of(x)], 1u)] = x;
      }
      __syncthreads();
      for (int i = tid; i < n; i += kRowThreads) {
        const uint64_t x = sh.list[i];
        const int b = bin_of(x), from = b == 0 ? 0 : (int)sh.bin_end[b - 1], to = (int)sh.bin_end[b];
        int rank = from;
        for (int j = from; j < to; j++) rank += binned[j] > x;
        sh.sorted[rank] = x;
      }
      __syncthreads();
      done = true;
    }
  }
  if (!done) {
    for (int i = tid; i < size; i += kRowThreads) sh.sorted[i] = i < n ? sh.list[i] : 0;
    __syncthreads();
    for (int len = 2; len <= size; len <<= 1) {
      for (int step = len >> 1; step > 0; step >>= 1) {
        for (int i = tid; i < size / 2; i += kRowThreads) {
          const int a = ((i & -step) << 1) | (i & (step - 1)), b = a + step;
          const uint64_t x = sh.sorted[a], y = sh.sorted[b];
          if ((x < y) == ((a & len) == 0)) {
            sh.sorted[a] = y;
            sh.sorted[b] = x;
          }
        }
        __syncthreads();
      }
    }
  }

  // prefix masses in the row's order, `per` tokens per thread; the number kept
  const int per = size / kRowThreads, e0 = tid * per, e1 = min(e0 + per, n);
  auto logit_of = [](uint64_t x) { return ord_score((uint32_t)(x >> 32)); };
  uint64_t sum = 0, reach = 0, all;
  for (int e = e0; e < e1; e++) {
    const uint64_t m = w.fixed(logit_of(sh.sorted[e]));
    sh.mass[e] = m;
    sum += m;
    if (r.minp > 0.f) reach += w.weight(logit_of(sh.sorted[e])) >= (double)r.minp;
  }
  const uint64_t upto = block_scan(sum, &all, sc);
  int n_keep = n;
  if (r.k > 0) n_keep = min(n_keep, r.k);
  uint64_t goal = p_mass;
  if (r.p < 1.f && r.k > 0) {  // mass of the first k
    uint64_t run = upto - sum, mass = 0;
    for (int e = e0; e < min(e1, n_keep); e++) run += sh.mass[e];
    block_first(e0 <= n_keep - 1 && n_keep - 1 < e0 + per, run, 0, &mass, &unused, sc);
    goal = scaled_ceil(r.p, mass);
  }
  if (goal > 0) {
    uint64_t run = upto - sum, len = 0;
    int mine = e0;
    while (mine < e1 && run < goal) run += sh.mass[mine++];
    if (block_first(upto >= goal && e0 < e1, (uint64_t)mine, 0, &len, &unused, sc) >= 0) n_keep = min(n_keep, (int)len);
  }
  if (r.minp > 0.f) {
    uint64_t reached;
    block_scan(reach, &reached, sc);
    n_keep = min(n_keep, (int)reached);
  }
  const uint64_t last = sh.sorted[n_keep - 1];

  // the pick, in id order
  sum = 0;
  for (int e = e0; e < e1; e++) {
    const uint64_t x = sh.list[e];
    sum += x >= last ? w.fixed(logit_of(x)) : 0;
  }
  const uint64_t to = block_scan(sum, &total, sc);
  const uint64_t target = scaled_floor(r.u, total);
  uint64_t run = to - sum, mine = 0, got = 0;
  if (to > target && run <= target)
    for (int e = e0; e < e1; e++) {
      const uint64_t x = sh.list[e];
      mine = x;
      run += x >= last ? w.fixed(logit_of(x)) : 0;
      if (run > target) break;
    }
  block_first(to > target, mine, 0, &got, &unused2, sc);
  sample_store(s, row, (int)~(uint32_t)got, w.weight(logit_of(got)), total, ws.shift);
}

// ---------------------------------------------------------------------------
// 3. Heavy rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sample_top(const SamplePtrs& ws, int64_t row) {
  float m = -__builtin_inff();
  for (int c = threadIdx.x & 63; c < ws.chunks; c += 64) m = fmaxf(m, ws.cmax[row * ws.chunks + c]);
  return wave_max_f32(m);
}

// A workgroup per slice of a heavy row, few of them as calls of mixed settings have few heavy
// rows: bound by the f64 weights and the LDS additions (64 rows of 262,144 of mixed settings
// 10 us).  Whole batches of heavy rows (1,024 x 151,936 bf16, T = 1.5, top-p 0.95: the call
// 1,211 us) read and weigh every token here a second time.
template <int DT>
__global__ void __launch_bounds__(kSampleThreads, 4) sample_hist_kernel(Sample s, SamplePtrs ws) {
  constexpr int N = SampleSource<DT>::N;
  __shared__ SampleHist h;
  const int tid = threadIdx.x, c = blockIdx.x, n = (int)min(*ws.nheavy, (uint32_t)ws.slots);
  for (int slot = blockIdx.y; slot < n; slot += gridDim.y) {
    const int64_t row = ws.heavy[slot];
    const SampleSource<DT> src(s, row);
    constexpr int U = kSlice / (kSampleThreads * N);
    float l[U][N];
    src.template load_many<U, kSampleThreads * N>(c * kSlice + tid * N, (c + 1) * kSlice, l);
    const SampleRow r = sample_row(s, row);
    const float top = sample_top(ws, row);
    const SampleWeight w(top, r.T, ws.shift);
    h.count[tid] = 0;
    h.mass[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int j = 0; j < N; j++)
        if (l[u][j] > -__builtin_inff()) {
          const int b = sample_bin(l[u][j], top);
          atomicAdd(&h.count[b], 1u);
          atomicAdd((unsigned long long*)&h.mass[b], (unsigned long long)w.fixed(l[u][j]));
        }
    __syncthreads();
    const size_t at = ((size_t)slot * ws.slices + c) * kSampleBins + tid;
    ws.hcount[at] = h.count[tid];
    ws.hmass[at] = h.mass[tid];
    __syncthreads();
  }
}

// The row's histogram, one bin per thread (bin 0, the largest logits, first): the bin's
// count and mass, and their sums up to and including it.
struct SampleRowHist {
  uint64_t c, m, tc, tm, ic, im;
  __device__ __forceinline__ SampleRowHist(const SamplePtrs& ws, int slot, SampleScratch<kSampleWaves>& sc)
      : c(0), m(0) {
    const size_t at = (size_t)slot * ws.slices * kSampleBins + threadIdx.x;
#pragma unroll 4
    for (int i = 0; i < ws.slices; i++) {
      c += ws.hcount[at + (size_t)i * kSampleBins];
      m += ws.hmass[at + (size_t)i * kSampleBins];
    }
    ic = block_scan(c, &tc, sc);
    im = block_scan(m, &tm, sc);
  }
};

// A workgroup per heavy row, so that many slices do not each search the histogram (10 us).
// Where the first cut of each heavy row lies: the bin in which the first k end, else that in
// which the nucleus ends, or that of min-p's bound if it comes first.
__global__ void __launch_bounds__(kSampleThreads, 4) sample_bin_kernel(Sample s, SamplePtrs ws) {
  __shared__ SampleScratch<kSampleWaves> sc;
  const int tid = threadIdx.x, count = (int)min(*ws.nheavy, (uint32_t)ws.slots);
  for (int slot = blockIdx.x; slot < count; slot += gridDim.x) {
    const int64_t row = ws.heavy[slot];
    const SampleRow r = sample_row(s, row);
    const float top = sample_top(ws, row);
    const SampleRowHist h(ws, slot, sc);
    SampleState st = {};
    st.bin = kSampleBins - 1;
    uint64_t in_bin = 0, unused;
    if (r.k > 0 && h.tc >= (uint64_t)r.k) {  // else there are fewer candidates than k
      st.filter = 1;
      st.bin = block_first(h.ic >= (uint64_t)r.k, h.ic - h.c, h.im - h.m, &st.before_count, &st.before_mass, sc);
    } else {
      if (r.p < 1.f) {
        st.filter = 2;
        st.goal = scaled_ceil(r.p, h.tm);
        st.bin = block_first(h.im >= st.goal, h.ic - h.c, h.im - h.m, &st.before_count, &st.before_mass, sc);
      }
      if (r.minp > 0.f) {
        const SampleWeight w(top, r.T, ws.shift);
        const int b = sample_bin(ord_score(sample_minp_key(w, top, r.minp)), top);
        if (b < st.bin) st.filter = 0, st.bin = b;  // the nucleus ends in a later bin
      }
    }
    block_first(tid == st.bin, h.c, 0, &in_bin, &unused, sc);
    st.listed = in_bin <= kHeavyList;  // else the heavy kernel narrows the bin by a pass first
    if (tid == 0) ws.hstate[slot] = st;
  }
}

// Lists the tokens of those bins: one workgroup per slice (64 rows of 262,144 of mixed
// settings 8 us; with an addition per wave to the list's size, instead of one per
// workgroup, 14).
template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_gather_kernel(Sample s, SamplePtrs ws) {
  constexpr int N = SampleSource<DT>::N, U = kSlice / (kSampleThreads * N);
  __shared__ SampleScratch<kSampleWaves> sc;
  const int tid = threadIdx.x, count = (int)min(*ws.nheavy, (uint32_t)ws.slots);
  for (int slot = blockIdx.y; slot < count; slot += gridDim.y) {
    const int64_t row = ws.heavy[slot];
    const int b = ws.hstate[slot].listed ? ws.hstate[slot].bin : -1;
    if (b < 0) continue;  // whole workgroup
    const SampleSource<DT> src(s, row);
    float l[U][N];
    src.template load_many<U, kSampleThreads * N>(blockIdx.x * kSlice + tid * N, (blockIdx.x + 1) * kSlice, l);
    const float top = sample_top(ws, row);
    uint32_t n = 0;
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int j = 0; j < N; j++) n += l[u][j] > -__builtin_inff() && sample_bin(l[u][j], top) == b;
    // the order of the list does not matter: one addition per workgroup places its tokens
    uint64_t all, base = 0, unused;
    const uint64_t upto = block_scan((uint64_t)n, &all, sc);
    if (all == 0) continue;  // whole workgroup
    if (tid == 0) base = atomicAdd(&ws.hlisted[slot], (uint32_t)all);
    block_first(tid == 0, base, 0, &base, &unused, sc);
    uint32_t place = (uint32_t)(base + upto - n);
    uint64_t* list = ws.hlist + (size_t)slot * kHeavyList;
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int j = 0; j < N; j++)
        if (l[u][j] > -__builtin_inff() && sample_bin(l[u][j], top) == b)
          list[place++] = ((uint64_t)score_ord(l[u][j]) << 32) |
                          (uint32_t)(blockIdx.x * kSlice + (u * kSampleThreads + tid) * N + j);
  }
}

struct SampleHeavyShared {
  SampleScratch<kSampleWaves> sc;
  SampleHist h;
  uint64_t list[kHeavyList];
  uint64_t mass[kHeavyList];
  uint64_t slice[kMaxSlices];
  uint32_t n;
};

// A workgroup per heavy row, bound by latency as the row kernel is (64 rows of 262,144 of
// mixed settings 34 us; 4 us where there is none).
// Heavy row `row`, with the histograms and the list of `slot`, or (slot -1) by passes over it.
template <int DT>
__device__ __forceinline__ void sample_heavy_row(const Sample& s, const SamplePtrs& ws, int64_t row, int slot,
                                                 SampleHeavyShared& sh) {
  SampleScratch<kSampleWaves>& sc = sh.sc;
  const bool hist = slot >= 0;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const SampleSource<DT> src(s, row);
  const SampleRow r = sample_row(s, row);
  const float top = sample_top(ws, row);
  const uint32_t top_key = score_ord(top);
  const SampleWeight w(top, r.T, ws.shift);
  const uint64_t* hmass = ws.hmass + (size_t)(hist ? slot : 0) * ws.slices * kSampleBins;

  const SampleState st = hist ? ws.hstate[slot] : SampleState{};

  // the tokens of one bin
  SampleRange<kSampleThreads, DT> range(src, w, sh.list, sh.mass, &sh.n);
  int listed = -1;
  uint32_t klo = 1, khi = top_key;
  auto bin_open = [&](int b) {
    if (listed == b) return;
    listed = b;
    klo = sample_bin_floor(b, top);
    khi = b == 0 ? top_key : sample_bin_floor(b - 1, top) - 1;
    if (b == st.bin && st.listed) {  // the gather kernel has listed them
      range.n = (int)ws.hlisted[slot];
      for (int i = tid; i < range.n; i += kSampleThreads) sh.list[i] = ws.hlist[(size_t)slot * kHeavyList + i];
      range.weigh();
      __syncthreads();
    } else {
      range.gather(klo, khi);
    }
  };
  SampleCut cut;
  auto kept = [&](float l, int v) {
    const uint32_t key = score_ord(l);
    return cut.keeps(key, (uint32_t)v) ? w.fixed(l) : 0ull;
  };
  auto kept_mass = [&]() {  // by a pass over the row
    uint64_t z = 0, all;
    sample_each<kSampleThreads>(src, [&](uint32_t key, uint32_t id) { z += kept(ord_score(key), (int)id); });
    block_scan(z, &all, sc);
    return all;
  };
  auto find = [&](bool by_count, uint64_t goal, uint64_t bc, uint64_t bm) {
    const bool whole = range.n >= 0;
    const uint64_t mass =
        sample_find(range, w, &cut, klo, khi, by_count, by_count ? goal : 0, by_count ? 0 : goal, bc, bm, sh.h, sc);
    if (!whole) listed = -1, range.n = -1;  // the search may have listed a part of the range
    return mass;
  };
  if (hist) {
    if (st.filter != 0) {
      bin_open(st.bin);
      const uint64_t mass =
          find(st.filter == 1, st.filter == 1 ? (uint64_t)r.k : st.goal, st.before_count, st.before_mass);
      if (st.filter == 1 && r.p < 1.f) {
        uint64_t bc, bm;
        const uint64_t goal = scaled_ceil(r.p, mass);
        const SampleRowHist h(ws, slot, sc);
        const int b = block_first(h.im >= goal, h.ic - h.c, h.im - h.m, &bc, &bm, sc);
        bin_open(b);
        find(false, goal, bc, bm);
      }
    }
  } else {
    uint64_t mass = 0;
    if (r.k > 0) mass = find(true, (uint64_t)r.k, 0, 0);
    else if (r.p < 1.f) mass = kept_mass();
    if (r.p < 1.f) find(false, scaled_ceil(r.p, mass), 0, 0);
  }
  if (r.minp > 0.f) {
    const uint32_t key = sample_minp_key(w, top, r.minp);
    if (key > cut.key) cut.key = key, cut.id = 0xffffffffu;
  }
  int first = 0, end = src.V;
  uint64_t total, left, unused;
  if (hist) {
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
    range.each([&](uint32_t key, uint32_t id, auto mass_of) {
      if (key >= klo && key <= khi && cut.keeps(key, id))
        atomicAdd((unsigned long long*)&sh.slice[id / kSlice], (unsigned long long)mass_of());
    });
    __syncthreads();
    const uint64_t z = tid < ws.slices ? sh.slice[tid] : 0;
    const uint64_t upto = block_scan(z, &total, sc);
    left = scaled_floor(r.u, total);
    const int i = block_first(upto > left, left - (upto - z), 0, &left, &unused, sc);
    first = i * kSlice;
    end = min(src.V, first + kSlice);
  } else {
    total = kept_mass();
    left = scaled_floor(r.u, total);
  }
  const int id = block_pick(src, first, end, left, kept, sc);
  sample_store(s, row, id, w.weight(src.logit(id)), total, ws.shift);
}

template <int DT>
__global__ void __launch_bounds__(kSampleThreads, 4) sample_heavy_kernel(Sample s, SamplePtrs ws) {
  __shared__ SampleHeavyShared sh;
  const int n = (int)*ws.nheavy;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    sample_heavy_row<DT>(s, ws, ws.heavy[i], i < ws.slots ? i : -1, sh);
    __syncthreads();
  }
}

size_t sample_workspace(int64_t rows, int64_t vocab) {
  if (rows == 0) return 0;
  // 16-bit logits have no more groups than f32 ones
  return sample_ws(rows, vocab, DT_F32).bytes;
}

template <int DT>
static hipError_t launch_sample_dt(const Sample& s, const SamplePtrs& ws, bool filtered, bool flat, hipStream_t stream) {
  const int64_t units = s.rows * ws.chunks;
  hipLaunchKernelGGL((sample_chunk_kernel<DT>), dim3((unsigned)cdiv(units, kChunkThreads / 64)), dim3(kChunkThreads), 0,
                     stream, s, ws);
  hipLaunchKernelGGL((sample_row_kernel<DT>), dim3((unsigned)s.rows), dim3(kRowThreads), 0, stream, s, ws);
  if (flat) {
    // few workgroups, as there are few heavy rows as a rule and none often (10,240 workgroups that
    // found nothing to do took 40 us)
    const dim3 grid((unsigned)ws.slices, (unsigned)std::min<int64_t>(s.rows, cdiv(2 * kTargetBlocks, ws.slices)));
    hipLaunchKernelGGL((sample_hist_kernel<DT>), grid, dim3(kSampleThreads), 0, stream, s, ws);
    hipLaunchKernelGGL(sample_bin_kernel, dim3((unsigned)std::min<int64_t>(s.rows, kTargetBlocks)), dim3(kSampleThreads), 0,
                       stream, s, ws);
    hipLaunchKernelGGL((sample_gather_kernel<DT>), grid, dim3(kSampleThreads), 0, stream, s, ws);
  }
  if (filtered)
    hipLaunchKernelGGL((sample_heavy_kernel<DT>), dim3((unsigned)std::min<int64_t>(s.rows, kTargetBlocks)),
                       dim3(kSampleThreads), 0, stream, s, ws);
  return hipGetLastError();
}

hipError_t launch_sample(const Sample& s, void* space, hipStream_t stream) {
  const SampleWs w = sample_ws(s.rows, s.vocab, s.dtype);
  uint8_t* base = (uint8_t*)space;
  SamplePtrs p;
  p.gmax = (float*)(base + w.gmax);
  p.cmax = (float*)(base + w.cmax);
  p.csum = (uint64_t*)(base + w.csum);
  p.heavy = (int32_t*)(base + w.heavy);
  p.nheavy = (uint32_t*)(base + w.nheavy);
  p.hcount = (uint32_t*)(base + w.hcount);
  p.hmass = (uint64_t*)(base + w.hmass);
  p.hlist = (uint64_t*)(base + w.hlist);
  p.hlisted = (uint32_t*)(base + w.hlisted);
  p.hstate = (SampleState*)(base + w.hstate);
  p.chunks = w.chunks;
  p.slices = w.slices;
  p.group_log2 = w.group_log2;
  p.groups = w.groups;
  p.slots = w.slots;
  int bits = 0;
  while ((1ll << bits) < s.vocab) bits++;
  p.shift = std::min(45, 63 - bits);
  // Rows with more tokens at the bound than the list holds are left to the heavy kernel, with
  // the histograms where their settings may ask for it.  With one small k for all rows the list
  // overflows where thousands of tokens are equal to or within 1/8 of the largest, or where the
  // first k lie in few groups of large tokens (sorted logits): the heavy kernel does without
  // histograms then (no slots), by passes of one workgroup.  262,144 f32 tokens, top-k of 50, 1
  // row / 64: spread 0.01 232 / 351 us, sorted 537 / 554, integers from 0 to 3 848 / 883; a
  // Gaussian of spread 2.5 22 / 32.
  const bool greedy = s.d_temperature == nullptr && s.temperature == 0.f;
  const bool small_k = greedy || (s.d_top_k == nullptr && s.top_k > 0 && s.top_k <= kList / 2);
  const bool no_filter = s.temperature > 0.f && s.d_temperature == nullptr && s.d_top_k == nullptr && s.top_k == 0 &&
                         s.d_top_p == nullptr && s.top_p == 1.f && s.d_min_p == nullptr && s.min_p == 0.f;
  const bool filtered = s.vocab > kList && !no_filter, flat = filtered && !small_k;
  if (!flat) p.slots = 0;
  if (s.dtype == DT_F32) return launch_sample_dt<DT_F32>(s, p, filtered, flat, stream);
  if (s.dtype == DT_BF16) return launch_sample_dt<DT_BF16>(s, p, filtered, flat, stream);
  return launch_sample_dt<DT_F16>(s, p, filtered, flat, stream);
}

}  // namespace etg
