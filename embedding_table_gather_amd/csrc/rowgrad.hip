// Gradient of the row gather with respect to the table:
//   out[v][c] = [out[v][c] +] scale * sum over the positions i with ids[i] = v of grad[i][c]
// The positions are sorted by token (stably), and a token's gradient rows are added in an order
// that depends on the sizes and their places alone, in 32 bits, without atomics: results repeat
// bitwise.
//
// A wave takes a piece of consecutive sorted positions and a chunk of columns, and writes the
// sum of each run of equal tokens that lies inside its piece.  Runs that cross a piece's
// border leave their partial sums, which rowgrad_join_kernel adds, sixteen at a time as a tree.
#include <algorithm>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

constexpr int kSortWaves = 4;
constexpr int kMaxDigits = 1024;  // 10 bits

// Zeros for the output, written by the workgroups behind those that sort: the sort's short
// kernels leave the chip idle, and the fill has to be over before the sums are written anyway.
// 16,384 ids into 262,144 x 768 f32 rows: 259 us with a fill of its own, 175 so.
struct Fill {
  u32x4* at;
  int64_t n16;  // 16-byte pieces
  static constexpr int kPieces = 8192;  // of one workgroup: 128 KiB
  int64_t workgroups() const { return cdiv(n16, kPieces); }
  // the g-th workgroup's part
  __device__ __forceinline__ void run(int64_t g, int threads) const {
    const u32x4 zero = {0, 0, 0, 0};
    const int64_t end = min((g + 1) * kPieces, n16);
#pragma unroll 4
    for (int64_t i = g * kPieces + threadIdx.x; i < end; i += threads) at[i] = zero;
  }
};

__global__ void __launch_bounds__(256) rowgrad_fill_kernel(Fill fill) { fill.run(blockIdx.x, 256); }

// Bad ids sort behind every token.
__device__ __forceinline__ uint32_t token_key(int32_t id, uint32_t V) { return min((uint32_t)id, V); }

// ---------------------------------------------------------------------------
// Few ids: each one's place is the number of ids that sort before it, counted by comparing it
// with all others (two vector instructions per 64 comparisons).  A workgroup places 64 ids;
// its 16 waves count a sixteenth of the others each.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) rowgrad_rank_kernel(const int32_t* __restrict__ ids, int n, uint32_t V,
                                                            uint32_t* __restrict__ keys,
                                                            uint32_t* __restrict__ order, int work, Fill fill) {
  __shared__ uint32_t count[16][64];
  if ((int)blockIdx.x >= work) {  // whole workgroup
    fill.run((int)blockIdx.x - work, 1024);
    return;
  }
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x * 64, i = i0 + lane;
  const uint32_t key = i < n ? token_key(ids[i], V) : 0xffffffffu;
  const int each = (n + 16 * 64 - 1) / (16 * 64) * 64;  // whole blocks of 64
  uint32_t before = 0;
  for (int j0 = wv * each; j0 < min((wv + 1) * each, n); j0 += 64) {
    // past the last id: larger than every key
    const uint32_t other = j0 + lane < n ? token_key(ids[j0 + lane], V) : 0xffffffffu;
    if (j0 != i0) {  // equal ids keep their order: those of an earlier block come before
      const uint32_t limit = key + (j0 < i0 && i < n ? 1u : 0u);
#pragma unroll 16
      for (int j = 0; j < 64; j++) before += (uint32_t)__builtin_amdgcn_readlane(other, j) < limit ? 1u : 0u;
    } else {
#pragma unroll 16
      for (int j = 0; j < 64; j++) {
        const uint32_t o = __builtin_amdgcn_readlane(other, j);
        before += o < key || (o == key && j < lane) ? 1u : 0u;
      }
    }
  }
  count[wv][lane] = before;
  __syncthreads();
  if (wv != 0 || i >= n) return;
#pragma unroll
  for (int w = 1; w < 16; w++) before += count[w][lane];
  keys[before] = key;
  order[before] = (uint32_t)i;
}

// ---------------------------------------------------------------------------
// More ids: a stable radix sort, least significant digit first.  Per pass: the digits'
// counts of every tile of keys, their running sum over (digit, tile), and the keys' move.
// Up to kFewTiles tiles a workgroup of the move adds up what it needs of the counts itself;
// more have a kernel for it.
// ---------------------------------------------------------------------------
constexpr int kFewTiles = 64;

struct SortPass {
  const int32_t* ids;        // the first pass: the ids themselves, positions 0, 1, ..
  const uint32_t *key, *pos;
  int64_t n;
  uint32_t V;
  int shift, bits, tiles, tile;  // tile: keys of one, a multiple of 256
  __device__ __forceinline__ uint32_t load_key(int64_t i) const { return ids != nullptr ? token_key(ids[i], V) : key[i]; }
  __device__ __forceinline__ uint32_t digit(uint32_t k) const { return (k >> shift) & ((1u << bits) - 1); }
};

// counts [tiles][kMaxDigits]
__global__ void __launch_bounds__(64 * kSortWaves) rowgrad_count_kernel(SortPass p, uint32_t* __restrict__ counts,
                                                                        Fill fill) {
  __shared__ uint32_t hist[kMaxDigits];
  if ((int)blockIdx.x >= p.tiles) {  // whole workgroup
    fill.run((int)blockIdx.x - p.tiles, 64 * kSortWaves);
    return;
  }
  for (int d = threadIdx.x; d < kMaxDigits; d += 64 * kSortWaves) hist[d] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.tile;
#pragma unroll 4
  for (int j = threadIdx.x; j < p.tile; j += 64 * kSortWaves)
    if (i0 + j < p.n) atomicAdd(&hist[p.digit(p.load_key(i0 + j))], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < kMaxDigits; d += 64 * kSortWaves) counts[(int64_t)blockIdx.x * kMaxDigits + d] = hist[d];
}

// Exclusive running sum of one value per thread over a workgroup of 64 W threads; the total too.
template <int W>
__device__ __forceinline__ uint32_t workgroup_scan(uint32_t v, uint32_t (&sums)[W], uint32_t* total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  if (lane == 63) sums[wv] = incl;
  __syncthreads();
  uint32_t run = incl - v, all = 0;
#pragma unroll
  for (int w = 0; w < W; w++) {
    if (w < wv) run += sums[w];
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return run;
}

// counts -> where a tile's first key of each digit goes, in place.  One workgroup, a thread per
// digit.
__global__ void __launch_bounds__(kMaxDigits) rowgrad_scan_kernel(uint32_t* __restrict__ counts, int tiles, Fill fill) {
  __shared__ uint32_t sums[kMaxDigits / 64];
  if (blockIdx.x > 0) {  // whole workgroup
    fill.run((int)blockIdx.x - 1, kMaxDigits);
    return;
  }
  uint32_t own = 0, total;
#pragma unroll 8
  for (int t = 0; t < tiles; t++) own += counts[(int64_t)t * kMaxDigits + threadIdx.x];
  uint32_t run = workgroup_scan(own, sums, &total);
#pragma unroll 8
  for (int t = 0; t < tiles; t++) {
    const uint32_t c = counts[(int64_t)t * kMaxDigits + threadIdx.x];
    counts[(int64_t)t * kMaxDigits + threadIdx.x] = run;
    run += c;
  }
}

// FEW: counts as the count kernel left them, else as the scan kernel did.
template <bool FEW>
__global__ void __launch_bounds__(64 * kSortWaves) rowgrad_move_kernel(SortPass p, const uint32_t* __restrict__ counts,
                                                                       uint32_t* __restrict__ key_out,
                                                                       uint32_t* __restrict__ pos_out, Fill fill) {
  __shared__ uint32_t next[kSortWaves][kMaxDigits];  // where a wave's next key of a digit goes
  __shared__ uint32_t sums[kSortWaves];
  constexpr int DPT = kMaxDigits / (64 * kSortWaves);  // digits of a thread, side by side
  static_assert(DPT == 4, "16-byte loads of the counts");
  if ((int)blockIdx.x >= p.tiles) {  // whole workgroup
    fill.run((int)blockIdx.x - p.tiles, 64 * kSortWaves);
    return;
  }
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, share = p.tile / kSortWaves;
  for (int d = threadIdx.x; d < kSortWaves * kMaxDigits; d += 64 * kSortWaves) ((uint32_t*)next)[d] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.tile + wv * share;
#pragma unroll 4
  for (int j = lane; j < share; j += 64)
    if (i0 + j < p.n) atomicAdd(&next[wv][p.digit(p.load_key(i0 + j))], 1u);
  u32x4 at = {0, 0, 0, 0};
  const int d0 = DPT * threadIdx.x;
  if constexpr (FEW) {
    u32x4 all = {0, 0, 0, 0};
#pragma unroll 8
    for (int t = 0; t < p.tiles; t++) {
      const u32x4 c = *(const u32x4*)(counts + (int64_t)t * kMaxDigits + d0);
      all += c;
      if (t < (int)blockIdx.x) at += c;
    }
    uint32_t total, run = workgroup_scan(all[0] + all[1] + all[2] + all[3], sums, &total);
#pragma unroll
    for (int q = 0; q < DPT; q++) {
      at[q] += run;
      run += all[q];
    }
  } else {
    at = *(const u32x4*)(counts + (int64_t)blockIdx.x * kMaxDigits + d0);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < DPT; q++)
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) {
      const uint32_t c = next[w][d0 + q];
      next[w][d0 + q] = at[q];
      at[q] += c;
    }
  __syncthreads();
  // the wave's keys in order, 64 at a time: a key's place among them is the number of lanes
  // below with its digit
  for (int j = 0; j < share && i0 + j < p.n; j += 64) {
    const int64_t i = i0 + j + lane;
    const bool some = i < p.n;
    const uint32_t k = some ? p.load_key(i) : 0u;
    const uint32_t pos = some && p.ids == nullptr ? p.pos[i] : (uint32_t)i;
    const uint32_t d = p.digit(k);
    uint64_t same = __ballot(some);
    for (int b = 0; b < p.bits; b++) {
      const uint64_t ones = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? ones : ~ones;
    }
    const uint32_t below = (uint32_t)__builtin_popcountll(same & ((1ull << lane) - 1));
    const uint32_t to = some ? next[wv][d] + below : 0u;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has read its counter before it moves on
    if (some && below == 0) next[wv][d] = to + (uint32_t)__builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (some) {
      key_out[to] = k;
      pos_out[to] = pos;
    }
  }
}

// ---------------------------------------------------------------------------
// Sums of the sorted rows.
// ---------------------------------------------------------------------------
struct RowSums {
  const uint32_t *keys, *order;
  int64_t n;
  uint32_t V;
  const uint8_t* grad;
  int64_t pitch;   // bytes
  int hidden, piece;
  float scale;
  void* out;
  float* part;     // [pieces][2][hidden]: the run that enters a piece, the one that only leaves it
};

template <int E>
struct Vec {
  float x[E];
};

// E values as they are stored, at any address of the type, and their values.
template <int DT, int E>
struct Raw {
  static constexpr int WORDS = E * (DT == DT_F32 ? 4 : 2) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const uint8_t* at) {
    if constexpr (WORDS % 4 == 0) {
      typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
      for (int q = 0; q < WORDS / 4; q++) {
        const u32x4u v = ((const u32x4u*)at)[q];
#pragma unroll
        for (int i = 0; i < 4; i++) w[4 * q + i] = v[i];
      }
    } else {
      static_assert(WORDS == 2, "four 16-bit values");
      typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
      const u32x2u v = *(const u32x2u*)at;
      w[0] = v[0], w[1] = v[1];
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == DT_F32) return __uint_as_float(w[i]);
    else if constexpr (DT == DT_BF16) return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else return f16_bits_to_f32(w[i / 2] >> 16 * (i % 2) & 0xffffu);
  }
};

template <int DT>
__device__ __forceinline__ uint8_t* out_row(const RowSums& p, uint32_t v, int c) {
  return (uint8_t*)p.out + ((int64_t)v * p.hidden + c) * (DT == DT_F32 ? 4 : 2);
}

// out row = type([old +] scale * sum): the product and the sum rounded to f32, then to the type
template <int DT, int E, bool ADD>
__device__ __forceinline__ void write_row(const RowSums& p, uint32_t v, int c, const Vec<E>& sum,
                                          const Raw<DT, E>& old) {
  uint8_t* at = out_row<DT>(p, v, c);
  Vec<E> x;
#pragma unroll
  for (int i = 0; i < E; i++) x.x[i] = ADD ? old.value(i) + sum.x[i] * p.scale : sum.x[i] * p.scale;
#pragma unroll
  for (int q = 0; q < E / 4; q++) {
    const f32x4 w = {x.x[4 * q], x.x[4 * q + 1], x.x[4 * q + 2], x.x[4 * q + 3]};
    if constexpr (DT == DT_F32) {
      ((f32x4*)at)[q] = w;
    } else if constexpr (DT == DT_BF16) {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      ((bf16x4*)at)[q] = __builtin_convertvector(w, bf16x4);
    } else {
      typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
      ((f16x4*)at)[q] = __builtin_convertvector(w, f16x4);
    }
  }
}

template <int E>
__device__ __forceinline__ void write_part(float* at, const Vec<E>& sum) {
#pragma unroll
  for (int q = 0; q < E / 4; q++)
    ((f32x4*)at)[q] = f32x4{sum.x[4 * q], sum.x[4 * q + 1], sum.x[4 * q + 2], sum.x[4 * q + 3]};
}

// A wave per piece and 64 E columns; U rows, and the output rows that their runs' sums are added
// to, are loaded before the first is used.
template <int GDT, int ODT, int E, bool ADD>
__global__ void __launch_bounds__(256) rowgrad_sum_kernel(RowSums p) {
  constexpr int U = 8, ES = GDT == DT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = ((int)blockIdx.y * 4 + wv) * 64 * E + lane * E;
  if (((int)blockIdx.y * 4 + wv) * 64 * E >= p.hidden) return;  // whole wave
  const bool live = c < p.hidden;
  const int cl = live ? c : 0;
  const int64_t q = blockIdx.x, begin = q * p.piece, end = min(begin + p.piece, p.n);
  bool entered = begin > 0 && p.keys[begin - 1] == p.keys[begin];
  Vec<E> acc = {};
  for (int64_t b = begin; b < end; b += 64) {
    const int m = (int)min((int64_t)64, end - b);
    // the key behind the last one ends its run there; none: 0xffffffff
    const uint32_t key64 = lane < m ? p.keys[b + lane] : 0xffffffffu, pos64 = lane < m ? p.order[b + lane] : 0u;
    const uint32_t behind = b + m < p.n ? p.keys[b + m] : 0xffffffffu;
    auto load = [&](int j, Raw<GDT, E> (&row)[U]) {  // past the last: the last again
#pragma unroll
      for (int u = 0; u < U; u++) {
        const uint32_t pos = __builtin_amdgcn_readlane(pos64, min(j + u, m - 1));
        row[u].load(p.grad + (int64_t)pos * p.pitch + (int64_t)cl * ES);
      }
    };
    Raw<GDT, E> ahead[U];
    load(0, ahead);
    for (int j = 0; j < m; j += U) {
      Raw<GDT, E> row[U];
      Raw<ODT, E> old[U];
      uint32_t key[U + 1];
#pragma unroll
      for (int u = 0; u <= U; u++) key[u] = j + u < m ? __builtin_amdgcn_readlane(key64, (j + u) & 63) : behind;
      if (key[0] >= p.V) return;  // bad ids from here on; the run before them has been written
#pragma unroll
      for (int u = 0; u < U; u++) {
        row[u] = ahead[u];
        // all of them here: the compiler would move each load to its use
#pragma unroll
        for (int i = 0; i < Raw<GDT, E>::WORDS; i++) asm volatile("" : "+v"(row[u].w[i]));
      }
      if (j + U < m) load(j + U, ahead);
      if constexpr (ADD) {
#pragma unroll
        for (int u = 0; u < U; u++)  // (a row within the table where no run ends: not used)
          old[u].load(out_row<ODT>(p, key[u] != key[u + 1] && key[u] < p.V ? key[u] : key[0], cl));
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        if (j + u >= m || key[u] >= p.V) break;  // uniform
#pragma unroll
        for (int i = 0; i < E; i++) acc.x[i] += row[u].value(i);
        const bool last = b + j + u + 1 == end, leaves = last && key[u] == key[u + 1];
        if (!last && key[u] == key[u + 1]) continue;
        if (live) {
          if (entered || leaves) write_part<E>(p.part + (2 * q + (entered ? 0 : 1)) * p.hidden + c, acc);
          else write_row<ODT, E, ADD>(p, key[u], c, acc, old[u]);
        }
        entered = false;
#pragma unroll
        for (int i = 0; i < E; i++) acc.x[i] = 0.f;
      }
    }
  }
}

// A wave per piece and 256 columns, four of them to a workgroup.  If a run begins in the piece and
// leaves it: its partial sums, in order.
template <int ODT, bool ADD>
__global__ void __launch_bounds__(256) rowgrad_join_kernel(RowSums p) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t q = blockIdx.x, begin = q * p.piece, end = begin + p.piece;
  if (end >= p.n) return;
  const uint32_t before = begin > 0 ? p.keys[begin - 1] : 0xffffffffu;
  const uint32_t first = p.keys[begin], cur = p.keys[end - 1], after = p.keys[end];
  if (cur >= p.V || after != cur) return;        // nothing leaves
  if (first == cur && before == cur) return;     // it began before
  const int c = (((int)blockIdx.y * 4 + wv) * 64 + lane) * 4;
  if (c >= p.hidden) return;
  int64_t lo = end, hi = p.n;  // the first position behind the run
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.keys[mid] == cur) lo = mid + 1;
    else hi = mid;
  }
  const int64_t pieces = (lo - 1) / p.piece - q;  // after this one
  Raw<ODT, 4> old;
  if constexpr (ADD) old.load(out_row<ODT>(p, cur, c));
  f32x4 acc = *(const f32x4*)(p.part + (2 * q + 1) * p.hidden + c);
  const float* at = p.part + 2 * (q + 1) * p.hidden + c;
  int64_t i = 0;
  for (; i + 16 <= pieces; i += 16) {
    f32x4 x[16];
#pragma unroll
    for (int u = 0; u < 16; u++) x[u] = *(const f32x4*)(at + 2 * (i + u) * p.hidden);
#pragma unroll
    for (int o = 1; o < 16; o *= 2)
#pragma unroll
      for (int u = 0; u < 16; u += 2 * o) x[u] += x[u + o];
    acc += x[0];
  }
  for (; i < pieces; i++) acc += *(const f32x4*)(at + 2 * i * p.hidden);
  write_row<ODT, 4, ADD>(p, cur, c, Vec<4>{{acc[0], acc[1], acc[2], acc[3]}}, old);
}

namespace {

// Most ids placed by comparison.  Added to 151,936 x 896 bf16 rows, by it / by radix sort: 1,024 ids 14.7 /
// 26.1 us, 4,096 25.2 / 34.0, 8,192 41.3 / 41.5, 16,384 65.5 / 49.5.
constexpr int64_t kRankIds = 8192;
constexpr int64_t kPartialBytes = (int64_t)256 << 20;

struct RowGradWs {
  int64_t piece;
  int passes, bits, tiles, tile;
  size_t keys[2], pos[2], counts, part, bytes;
};
RowGradWs rowgrad_ws(int64_t n, int64_t V, int64_t hidden) {
  RowGradWs w = {};
  // 8 positions to a piece where there are few, so that many waves share them, up to 64; more where
  // the partial sums would not fit.  Added to 151,936 x 896 bf16 rows, ids as words are (of one token
  // alone): 628 ids by 8 13.7 us (17.2), by 16 14.5 (16.0), by 32 17.8 (16.6); 1,000 ids 15.1 (19.7),
  // 15.7 (18.8), 19.0 (20.0); 4,096 ids 24.8 (46.1), 25.3 (35.2), 29.2 (31.6).
  w.piece = n <= 1024 ? 8 : n <= 4096 ? 16 : n <= 32768 ? 32 : 64;
  if (cdiv(n, w.piece) * hidden * 8 > kPartialBytes)
    w.piece = (int64_t)align_up(cdiv(n * hidden * 8, kPartialBytes), 32);
  const bool ranked = n <= kRankIds;
  if (!ranked) {
    int bits = 1;
    while (((uint64_t)V >> bits) != 0) bits++;  // keys 0 .. V
    w.passes = (bits + 9) / 10;
    w.bits = (bits + w.passes - 1) / w.passes;
    w.tile = n <= 1024 * kFewTiles ? 1024 : 4096;
    w.tiles = (int)cdiv(n, w.tile);
  }
  size_t at = 0;
  for (int i = 0; i < (ranked ? 1 : 2); i++) {
    w.keys[i] = at;
    at += align_up((size_t)n * 4, 256);
    w.pos[i] = at;
    at += align_up((size_t)n * 4, 256);
  }
  w.counts = at;
  if (!ranked) at += align_up((size_t)w.tiles * kMaxDigits * 4, 256);
  w.part = at;
  w.bytes = at + align_up((size_t)(cdiv(n, w.piece) * 2 * hidden * 4), 256);
  return w;
}

// Hands out the output's zeros over the launches of the sort.
struct FillShares {
  Fill rest;
  int launches;
  // the next launch's share
  Fill next() {
    Fill f = rest;
    f.n16 = std::min(rest.n16, cdiv(cdiv(rest.n16, Fill::kPieces), std::max(launches, 1)) * Fill::kPieces);
    rest.at += f.n16, rest.n16 -= f.n16, launches--;
    return f;
  }
};

template <int GDT, int ODT, bool ADD>
hipError_t launch_sums(const RowSums& p, hipStream_t stream) {
  const int64_t pieces = cdiv(p.n, p.piece);
  // 16-byte loads of the gradient rows
  constexpr int E = GDT == DT_F32 ? 4 : 8;
  if (p.hidden % E == 0)
    hipLaunchKernelGGL((rowgrad_sum_kernel<GDT, ODT, E, ADD>),
                       dim3((unsigned)pieces, (unsigned)cdiv(p.hidden, 4 * 64 * E)), dim3(256), 0, stream, p);
  else  // 16-bit gradients of a f32 table
    hipLaunchKernelGGL((rowgrad_sum_kernel<GDT, ODT, 4, ADD>),
                       dim3((unsigned)pieces, (unsigned)cdiv(p.hidden, 4 * 64 * 4)), dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pieces == 1) return e;
  hipLaunchKernelGGL((rowgrad_join_kernel<ODT, ADD>), dim3((unsigned)(pieces - 1), (unsigned)cdiv(p.hidden, 1024)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int GDT>
hipError_t launch_sums_to(const RowSums& p, int32_t out_dtype, bool add, hipStream_t stream) {
  switch (out_dtype) {
    case DT_F32: return add ? launch_sums<GDT, DT_F32, true>(p, stream) : launch_sums<GDT, DT_F32, false>(p, stream);
    case DT_BF16: return add ? launch_sums<GDT, DT_BF16, true>(p, stream) : launch_sums<GDT, DT_BF16, false>(p, stream);
    default: return add ? launch_sums<GDT, DT_F16, true>(p, stream) : launch_sums<GDT, DT_F16, false>(p, stream);
  }
}

}  // namespace

size_t rowgrad_workspace(int64_t n, int64_t V, int64_t hidden) { return n == 0 ? 0 : rowgrad_ws(n, V, hidden).bytes; }

// One launch writes at most so many 16-byte pieces of zeros (128 GiB).
constexpr int64_t kFillMost = ((int64_t)1 << 20) * Fill::kPieces;

hipError_t launch_zeros(void* at, int64_t bytes, hipStream_t stream) {
  for (Fill all = {(u32x4*)at, bytes / 16}; all.n16 > 0;) {
    const Fill f = {all.at, std::min(all.n16, kFillMost)};
    hipLaunchKernelGGL(rowgrad_fill_kernel, dim3((unsigned)f.workgroups()), dim3(256), 0, stream, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    all.at += f.n16, all.n16 -= f.n16;
  }
  return hipSuccess;
}

hipError_t launch_rowgrad(const RowGrad& g, void* ws, hipStream_t stream) {
  hipError_t e;
  // whole rows of 16 bytes
  Fill all = {(u32x4*)g.out, g.add ? 0 : g.V * g.hidden * (g.out_dtype == DT_F32 ? 4 : 2) / 16};
  // what the sort's launches cannot take goes first
  const int64_t ahead = g.n == 0 ? all.n16 : std::max<int64_t>(0, all.n16 - kFillMost);
  if ((e = launch_zeros(all.at, ahead * 16, stream)) != hipSuccess) return e;
  all.at += ahead, all.n16 -= ahead;
  if (g.n == 0) return hipSuccess;
  const RowGradWs w = rowgrad_ws(g.n, g.V, g.hidden);
  uint8_t* base = (uint8_t*)ws;
  uint32_t *keys = (uint32_t*)(base + w.keys[0]), *order = (uint32_t*)(base + w.pos[0]);
  if (w.passes == 0) {
    const int work = (int)cdiv(g.n, 64);
    hipLaunchKernelGGL(rowgrad_rank_kernel, dim3((unsigned)(work + all.workgroups())), dim3(1024), 0, stream, g.ids,
                       (int)g.n, (uint32_t)g.V, keys, order, work, all);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool few = w.tiles <= kFewTiles;
  FillShares shares = {all, w.passes * (few ? 2 : 3)};
  for (int i = 0; i < w.passes; i++) {
    SortPass p = {};
    p.ids = i == 0 ? g.ids : nullptr;
    p.key = (uint32_t*)(base + w.keys[(i + 1) % 2]), p.pos = (uint32_t*)(base + w.pos[(i + 1) % 2]);
    p.n = g.n, p.V = (uint32_t)g.V, p.shift = i * w.bits, p.bits = w.bits, p.tiles = w.tiles, p.tile = w.tile;
    keys = (uint32_t*)(base + w.keys[i % 2]), order = (uint32_t*)(base + w.pos[i % 2]);
    uint32_t* counts = (uint32_t*)(base + w.counts);
    Fill f = shares.next();
    hipLaunchKernelGGL(rowgrad_count_kernel, dim3((unsigned)(w.tiles + f.workgroups())), dim3(64 * kSortWaves), 0,
                       stream, p, counts, f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (!few) {
      f = shares.next();
      hipLaunchKernelGGL(rowgrad_scan_kernel, dim3((unsigned)(1 + f.workgroups())), dim3(kMaxDigits), 0, stream,
                         counts, w.tiles, f);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    f = shares.next();
    hipLaunchKernelGGL(few ? rowgrad_move_kernel<true> : rowgrad_move_kernel<false>,
                       dim3((unsigned)(w.tiles + f.workgroups())), dim3(64 * kSortWaves), 0, stream, p, counts, keys,
                       order, f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  RowSums p = {};
  p.keys = keys, p.order = order, p.n = g.n, p.V = (uint32_t)g.V;
  p.grad = (const uint8_t*)g.grad, p.pitch = g.pitch, p.hidden = (int)g.hidden, p.piece = (int)w.piece;
  p.scale = g.scale, p.out = g.out, p.part = (float*)(base + w.part);
  switch (g.grad_dtype) {
    case DT_F32: return launch_sums_to<DT_F32>(p, g.out_dtype, g.add, stream);
    case DT_BF16: return launch_sums_to<DT_BF16>(p, g.out_dtype, g.add, stream);
    default: return launch_sums_to<DT_F16>(p, g.out_dtype, g.add, stream);
  }
}

}  // namespace etg
