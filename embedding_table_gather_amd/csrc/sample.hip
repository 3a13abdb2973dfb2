// Sampling of one token per row of logits with temperature, top-k, top-p and min-p
// from given random numbers (the sampling that ADR-0008 "POST /v1/logits" leaves to
// the caller of its raw logits mode), without the logits leaving the device.
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
// 2^(b + shift) = 2^63, so shift = 63 - b.  A weight is off by at most half a unit:
// a total (at least 2^shift) by 2^(2 b - 64) of itself, 2^-28 at 2^18 tokens and 2^-24
// at the largest vocabulary, 2^20.

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
  return r;
}

// Order key of a row's logit v, 0 where it is no candidate (every candidate's is larger).
template <int DT>
__device__ __forceinline__ uint32_t sample_key(const void* logits, const uint32_t* allowed, int v) {
  float l;
  if constexpr (DT == DT_F32) l = ((const float*)logits)[v];
  else if constexpr (DT == DT_BF16) l = __uint_as_float((uint32_t)((const uint16_t*)logits)[v] << 16);
  else l = f16_bits_to_f32(((const uint16_t*)logits)[v]);
  const bool live = l > -__builtin_inff() && (allowed == nullptr || ((allowed[v >> 5] >> (v & 31)) & 1u));
  return live ? score_ord(l) : 0u;
}

__device__ __forceinline__ double sample_weight(uint32_t key, uint32_t top, double M, double T) {
  return key == top ? 1.0 : exp(((double)ord_score(key) - M) / T);
}

static constexpr int kSampleThreads = 1024;
static constexpr int kSampleWaves = kSampleThreads / 64;
static constexpr int kSampleBins = 2048;

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor((unsigned long long)v, off, 64);
  return v;
}

// floor(f * m) and ceil(f * m) of a float f in [0, 1] and an integer m, exactly: f is a
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

// The element at which a prefix of the order reaches a target: key, how many of the
// elements with that key belong to the prefix, and the prefix's mass.
struct SampleCut {
  uint32_t key;
  uint32_t ties;
  uint64_t mass;
};

struct SampleShared {
  uint32_t count[kSampleBins];
  uint64_t mass[kSampleBins];
  uint64_t part_mass[kSampleWaves];
  uint32_t part[kSampleWaves];
  uint32_t bin, bin_count;
  uint64_t before_mass;
  uint32_t before_count;
  uint32_t id;
};

// One workgroup per row.  A cut is found by a radix search over the 32-bit keys, 11,
// 11 and 10 bits at a time from the top.
template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(Sample s, int shift) {
  __shared__ SampleShared sh;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, V = (int)s.vocab;
  const uint8_t* base = (const uint8_t*)s.logits + row * s.stride * (DT == DT_F32 ? 4 : 2);
  const uint32_t* allowed = s.allowed ? s.allowed + row * s.allowed_stride : nullptr;
  const SampleRow r = sample_row(s, row);

  uint32_t top = 0;
  for (int v = tid; v < V; v += kSampleThreads) top = max(top, sample_key<DT>(base, allowed, v));
  top = wave_minmax_u32<true>(top);
  if (lane == 0) sh.part[wv] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSampleWaves; i++) top = max(top, sh.part[i]);
  if (top == 0 || !r.ok) {  // whole workgroup
    if (tid == 0) {
      s.ids[row] = -1;
      s.probs[row] = 0.f;
    }
    return;
  }
  const double M = (double)ord_score(top), T = (double)r.T;
  const double unit = (double)(1ull << shift);
  auto fixed = [&](uint32_t key) { return (uint64_t)rint(sample_weight(key, top, M, T) * unit); };

  // the kept prefix so far: keys above cut_key, and ids up to cut_id at cut_key
  uint32_t cut_key = 1, cut_id = 0xffffffffu;
  auto kept = [&](uint32_t key, int v) { return key > cut_key || (key == cut_key && (uint32_t)v <= cut_id); };

  // the prefix of the kept elements that first holds `count` elements or `mass`
  auto find = [&](bool by_count, uint32_t count, uint64_t mass) {
    uint32_t prefix = 0;
    uint32_t before_count = 0;
    uint64_t before_mass = 0;
    uint32_t last_count = 0;
    for (int level = 0; level < 3; level++) {
      const int low = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      __syncthreads();
      for (int i = tid; i < kSampleBins; i += kSampleThreads) {
        sh.count[i] = 0;
        sh.mass[i] = 0;
      }
      __syncthreads();
      for (int v = tid; v < V; v += kSampleThreads) {
        const uint32_t key = sample_key<DT>(base, allowed, v);
        if (key != 0 && kept(key, v) && (level == 0 || (key >> (low + bits)) == prefix)) {
          const int bin = (int)((key >> low) & ((1u << bits) - 1));
          atomicAdd(&sh.count[bin], 1u);
          atomicAdd((unsigned long long*)&sh.mass[bin], (unsigned long long)fixed(key));
        }
      }
      __syncthreads();
      if (tid == 0) {
        // the first bin from the top that reaches the target, else the last one that holds any
        uint32_t c = before_count;
        uint64_t m = before_mass;
        int found = -1;
        uint32_t fc = c;
        uint64_t fm = m;
        for (int b = (1 << bits) - 1; b >= 0; b--) {
          if (sh.count[b] == 0) continue;
          found = b, fc = c, fm = m;
          c += sh.count[b];
          m += sh.mass[b];
          if (by_count ? c >= count : m >= mass) break;
        }
        sh.bin = (uint32_t)found;
        sh.before_count = fc;
        sh.before_mass = fm;
        sh.bin_count = sh.count[found];
      }
      __syncthreads();
      prefix = (prefix << bits) | sh.bin;
      before_count = sh.before_count;
      before_mass = sh.before_mass;
      last_count = sh.bin_count;
    }
    SampleCut c;
    c.key = prefix;
    const uint64_t w = fixed(prefix);
    uint64_t ties = by_count ? (uint64_t)count - before_count
                             : w != 0 ? (mass - before_mass + w - 1) / w : (uint64_t)last_count;
    if (ties > last_count) ties = last_count;
    c.ties = (uint32_t)ties;
    c.mass = before_mass + ties * w;
    // the id of the last of them: counts per wave segment, in id order
    uint32_t want = c.ties;
    int lo = 0, hi = V;
    while (hi - lo > 64) {
      const int seg = (hi - lo + kSampleWaves - 1) / kSampleWaves;
      const int a = min(lo + wv * seg, hi), b = min(a + seg, hi);
      uint32_t n = 0;
      for (int v = a + lane; v < b; v += 64) n += sample_key<DT>(base, allowed, v) == prefix;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, 64);
      __syncthreads();
      if (lane == 0) sh.part[wv] = n;
      __syncthreads();
      int i = 0;
      while (i < kSampleWaves - 1 && sh.part[i] < want) want -= sh.part[i++];
      const int at = min(lo + i * seg, hi);
      hi = min(at + seg, hi);
      lo = at;
    }
    __syncthreads();
    if (wv == 0) {
      const int v = lo + lane;
      const bool hit = v < hi && sample_key<DT>(base, allowed, v) == prefix;
      const uint64_t hits = __ballot(hit);
      const uint32_t rank = __popcll(hits & ((2ull << lane) - 1));
      if (hit && rank == want) sh.id = (uint32_t)v;
    }
    __syncthreads();
    cut_key = c.key;
    cut_id = sh.id;
    return c.mass;
  };

  uint64_t mass = 0;
  const bool by_k = r.k > 0 && r.k < V;
  if (by_k) mass = find(true, (uint32_t)r.k, 0);
  if (r.p < 1.f) {
    if (!by_k) {
      uint64_t m = 0;
      for (int v = tid; v < V; v += kSampleThreads) {
        const uint32_t key = sample_key<DT>(base, allowed, v);
        if (key != 0) m += fixed(key);
      }
      m = wave_sum_u64(m);
      __syncthreads();
      if (lane == 0) sh.part_mass[wv] = m;
      __syncthreads();
      for (int i = 0; i < kSampleWaves; i++) mass += sh.part_mass[i];
    }
    find(false, 0, scaled_ceil(r.p, mass));
  }
  if (r.minp > 0.f) {
    // the smallest key whose weight reaches min_p (weights do not fall as keys grow):
    // keys in (lo, hi] are undecided, hi's weight reaches it
    uint32_t lo = 0, hi = top;
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (sample_weight(mid, top, M, T) >= (double)r.minp) hi = mid;
      else lo = mid;
    }
    if (hi > cut_key) cut_key = hi, cut_id = 0xffffffffu;
  }

  // The pick: per-wave masses of segments of the ids in order, narrowed to 64 ids.
  auto mass_of = [&](int v) {
    const uint32_t key = sample_key<DT>(base, allowed, v);
    return key != 0 && kept(key, v) ? fixed(key) : 0ull;
  };
  int lo = 0, hi = V;
  uint64_t total = 0, target = 0;
  bool first = true;
  while (first || hi - lo > 64) {
    const int seg = (hi - lo + kSampleWaves - 1) / kSampleWaves;
    const int a = min(lo + wv * seg, hi), b = min(a + seg, hi);
    uint64_t m = 0;
    for (int v = a + lane; v < b; v += 64) m += mass_of(v);
    m = wave_sum_u64(m);
    __syncthreads();
    if (lane == 0) sh.part_mass[wv] = m;
    __syncthreads();
    if (first) {
      for (int i = 0; i < kSampleWaves; i++) total += sh.part_mass[i];
      target = scaled_floor(r.u, total);  // < total, as u < 1
      first = false;
    }
    // the segment in which the running mass first exceeds the target
    int at = 0;
    while (at < kSampleWaves - 1 && sh.part_mass[at] <= target) target -= sh.part_mass[at++];
    lo = min(lo + at * seg, hi);
    hi = min(lo + seg, hi);
  }
  if (tid == 0) {
    int v = lo;
    while (v < hi - 1) {
      const uint64_t w = mass_of(v);
      if (w > target) break;
      target -= w;
      v++;
    }
    s.ids[row] = v;
    s.probs[row] = (float)(sample_weight(sample_key<DT>(base, allowed, v), top, M, T) * unit / (double)total);
  }
}

size_t sample_workspace(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const Sample& s, void*, hipStream_t stream) {
  int bits = 0;
  while ((1ll << bits) < s.vocab) bits++;
  const int shift = 63 - bits;
#define ETG_SAMPLE(DT) \
  hipLaunchKernelGGL((sample_kernel<DT>), dim3((unsigned)s.rows), dim3(kSampleThreads), 0, stream, s, shift)
  if (s.dtype == DT_F32) ETG_SAMPLE(DT_F32);
  else if (s.dtype == DT_BF16) ETG_SAMPLE(DT_BF16);
  else ETG_SAMPLE(DT_F16);
#undef ETG_SAMPLE
  return hipGetLastError();
}

}  // namespace etg
