// Gradient of the row gather with respect to the table:
//   out[v][c] = [out[v][c] +] scale * sum over the positions i with ids[i] = v of grad[i][c]
// The positions are sorted by token (stably), so that a token's gradient rows are added in
// their order in 32 bits, without atomics: results repeat bitwise.
//
// A wave takes a piece of consecutive sorted positions and a chunk of columns, and writes the
// sum of each run of equal tokens that lies inside its piece.  Runs that cross a piece's
// border leave their partial sums, which rowgrad_join_kernel adds in order.
#include <algorithm>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

constexpr int kTileKeys = 4096;   // keys of one workgroup of the radix sort
constexpr int kSortWaves = 4;
constexpr int kMaxDigits = 512;   // 9 bits

// Bad ids sort behind every token.
__device__ __forceinline__ uint32_t token_key(int32_t id, uint32_t V) { return min((uint32_t)id, V); }

// ---------------------------------------------------------------------------
// Few ids: each one's place is the number of ids that sort before it, counted by comparing it
// with all others (two vector instructions per 64 comparisons).  A workgroup places 64 ids;
// its 16 waves count a sixteenth of the others each.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) rowgrad_rank_kernel(const int32_t* __restrict__ ids, int n, uint32_t V,
                                                            uint32_t* __restrict__ keys,
                                                            uint32_t* __restrict__ order) {
  __shared__ uint32_t count[16][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x * 64, i = i0 + lane;
  const uint32_t key = i < n ? token_key(ids[i], V) : 0xffffffffu;
  const int each = (n + 16 * 64 - 1) / (16 * 64) * 64;  // whole blocks of 64
  uint32_t before = 0;
  for (int j0 = wv * each; j0 < min((wv + 1) * each, n); j0 += 64) {
    const int m = min(64, n - j0);
    const uint32_t other = j0 + lane < n ? token_key(ids[j0 + lane], V) : 0xffffffffu;
    for (int j = 0; j < m; j++) {  // equal ids keep their order
      const uint32_t o = __builtin_amdgcn_readlane(other, j);
      before += o < key || (o == key && j0 + j < i) ? 1u : 0u;
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
// counts of every tile of 4,096 keys, their running sum over (digit, tile), and the keys' move.
// ---------------------------------------------------------------------------
struct SortPass {
  const int32_t* ids;        // the first pass: the ids themselves, positions 0, 1, ..
  const uint32_t *key, *pos;
  int64_t n;
  uint32_t V;
  int shift, bits, tiles;
  __device__ __forceinline__ uint32_t load_key(int64_t i) const { return ids != nullptr ? token_key(ids[i], V) : key[i]; }
  __device__ __forceinline__ uint32_t digit(uint32_t k) const { return (k >> shift) & ((1u << bits) - 1); }
};

__global__ void __launch_bounds__(64 * kSortWaves) rowgrad_count_kernel(SortPass p, uint32_t* __restrict__ counts) {
  __shared__ uint32_t hist[kMaxDigits];
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += 64 * kSortWaves) hist[d] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kTileKeys;
  for (int j = threadIdx.x; j < kTileKeys && i0 + j < p.n; j += 64 * kSortWaves)
    atomicAdd(&hist[p.digit(p.load_key(i0 + j))], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += 64 * kSortWaves) counts[(int64_t)d * p.tiles + blockIdx.x] = hist[d];
}

// counts -> their exclusive running sum, in place.  One workgroup, a contiguous share per thread.
__global__ void __launch_bounds__(1024) rowgrad_scan_kernel(uint32_t* __restrict__ counts, int64_t n) {
  __shared__ uint32_t sums[16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint32_t base = 0;
  for (int64_t c0 = 0; c0 < n; c0 += 8 * 1024) {
    const int64_t at = c0 + 8 * (int64_t)threadIdx.x;
    uint32_t v[8], total = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[j] = at + j < n ? counts[at + j] : 0u;
      total += v[j];
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    if (lane == 63) sums[wv] = incl;
    __syncthreads();
    uint32_t run = base + incl - total, all = 0;
#pragma unroll
    for (int w = 0; w < 16; w++) {
      if (w < wv) run += sums[w];
      all += sums[w];
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (at + j < n) counts[at + j] = run;
      run += v[j];
    }
    base += all;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(64 * kSortWaves) rowgrad_move_kernel(SortPass p,
                                                                       const uint32_t* __restrict__ offsets,
                                                                       uint32_t* __restrict__ key_out,
                                                                       uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t next[kSortWaves][kMaxDigits];  // where a wave's next key of a digit goes
  constexpr int SHARE = kTileKeys / kSortWaves;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < kSortWaves * kMaxDigits; d += 64 * kSortWaves) ((uint32_t*)next)[d] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kTileKeys + wv * SHARE;
  for (int j = lane; j < SHARE && i0 + j < p.n; j += 64) atomicAdd(&next[wv][p.digit(p.load_key(i0 + j))], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += 64 * kSortWaves) {
    uint32_t at = offsets[(int64_t)d * p.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) {
      const uint32_t c = next[w][d];
      next[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
  // the wave's keys in order, 64 at a time: a key's place among them is the number of lanes
  // below with its digit
  for (int j = 0; j < SHARE && i0 + j < p.n; j += 64) {
    const int64_t i = i0 + j + lane;
    const bool some = i < p.n;
    const uint32_t k = some ? p.load_key(i) : 0u;
    const uint32_t d = p.digit(k);
    uint64_t same = __ballot(some);
    for (int b = 0; b < p.bits; b++) {
      const uint64_t ones = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? ones : ~ones;
    }
    const uint32_t below = (uint32_t)__builtin_popcountll(same & ((1ull << lane) - 1));
    const uint32_t at = some ? next[wv][d] + below : 0u;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has read its counter before it moves on
    if (some && below == 0) next[wv][d] = at + (uint32_t)__builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (some) {
      key_out[at] = k;
      pos_out[at] = p.ids != nullptr ? (uint32_t)i : p.pos[i];
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
  int32_t add;
  float* part;     // [pieces][2][hidden]: the run that enters a piece, the one that only leaves it
};

template <int E>
struct Vec {
  float x[E];
};

template <int DT, int E>
__device__ __forceinline__ Vec<E> load_vec(const uint8_t* at) {
  Vec<E> v;
  if constexpr (DT == DT_F32) {
    typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int q = 0; q < E / 4; q++) {
      const f32x4u w = ((const f32x4u*)at)[q];
#pragma unroll
      for (int i = 0; i < 4; i++) v.x[4 * q + i] = w[i];
    }
  } else {
    typedef uint16_t u16xEu __attribute__((ext_vector_type(E), aligned(2)));
    const u16xEu w = *(const u16xEu*)at;
#pragma unroll
    for (int i = 0; i < E; i++)
      v.x[i] = DT == DT_BF16 ? __uint_as_float((uint32_t)w[i] << 16) : f16_bits_to_f32(w[i]);
  }
  return v;
}

// out row = type([out row +] scale * sum): the product and the sum rounded to f32, then to the type
template <int DT, int E>
__device__ __forceinline__ void write_row(const RowSums& p, uint32_t v, int c, const Vec<E>& sum) {
  constexpr int ES = DT == DT_F32 ? 4 : 2;
  uint8_t* at = (uint8_t*)p.out + ((int64_t)v * p.hidden + c) * ES;
  Vec<E> x;
#pragma unroll
  for (int i = 0; i < E; i++) x.x[i] = sum.x[i] * p.scale;
  if (p.add) {
    const Vec<E> old = load_vec<DT, E>(at);
#pragma unroll
    for (int i = 0; i < E; i++) x.x[i] += old.x[i];
  }
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

// A wave per piece and 64 E columns; U rows are loaded before the first is added.
template <int GDT, int ODT, int E>
__global__ void __launch_bounds__(256) rowgrad_sum_kernel(RowSums p) {
  constexpr int U = 8, ES = GDT == DT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = ((int)blockIdx.y * 4 + wv) * 64 * E + lane * E;
  if (((int)blockIdx.y * 4 + wv) * 64 * E >= p.hidden) return;  // whole wave
  const bool live = c < p.hidden;
  const int cl = live ? c : 0;
  const int64_t q = blockIdx.x, begin = q * p.piece, end = min(begin + p.piece, p.n);
  uint32_t cur = p.keys[begin];
  bool entered = begin > 0 && p.keys[begin - 1] == cur;
  Vec<E> acc = {};
  auto flush = [&](bool leaves) {
    if (cur >= p.V || !live) return;
    if (entered || leaves) write_part<E>(p.part + (2 * q + (entered ? 0 : 1)) * p.hidden + c, acc);
    else write_row<ODT, E>(p, cur, c, acc);
  };
  for (int64_t b = begin; b < end && cur < p.V; b += 64) {
    const int m = (int)min((int64_t)64, end - b);
    const uint32_t key64 = lane < m ? p.keys[b + lane] : 0xffffffffu, pos64 = lane < m ? p.order[b + lane] : 0u;
    for (int j = 0; j < m && cur < p.V; j += U) {
      Vec<E> row[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const uint32_t pos = __builtin_amdgcn_readlane(pos64, min(j + u, m - 1));
        row[u] = load_vec<GDT, E>(p.grad + (int64_t)pos * p.pitch + (int64_t)cl * ES);
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        if (j + u >= m || cur >= p.V) break;  // uniform
        const uint32_t k = __builtin_amdgcn_readlane(key64, j + u);
        if (k != cur) {
          flush(false);
          cur = k;
          entered = false;
          if (k >= p.V) break;
#pragma unroll
          for (int i = 0; i < E; i++) acc.x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < E; i++) acc.x[i] += row[u].x[i];
      }
    }
  }
  flush(end < p.n && p.keys[end] == cur);
}

// A workgroup per piece and 256 columns.  If a run begins in the piece and leaves it: its
// partial sums, a contiguous share of them per wave.
template <int ODT>
__global__ void __launch_bounds__(256) rowgrad_join_kernel(RowSums p) {
  __shared__ f32x4 sums[4][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t q = blockIdx.x, begin = q * p.piece, end = begin + p.piece;
  if (end >= p.n) return;
  const uint32_t cur = p.keys[end - 1];
  if (cur >= p.V || p.keys[end] != cur) return;                                        // nothing leaves
  if (p.keys[begin] == cur && begin > 0 && p.keys[begin - 1] == cur) return;           // it began before
  int64_t lo = end, hi = p.n;  // the first position behind the run
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.keys[mid] == cur) lo = mid + 1;
    else hi = mid;
  }
  const int64_t pieces = (lo - 1) / p.piece - q;  // after this one
  const int c = ((int)blockIdx.y * 64 + lane) * 4;
  const bool live = c < p.hidden;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const int64_t each = (pieces + 3) / 4;
    const float* at = p.part + 2 * (q + 1) * p.hidden + c;
    if (wv == 0) acc = *(const f32x4*)(p.part + (2 * q + 1) * p.hidden + c);
#pragma unroll 8
    for (int64_t i = wv * each; i < min((wv + 1) * each, pieces); i++) acc += *(const f32x4*)(at + 2 * i * p.hidden);
  }
  sums[wv][lane] = acc;
  __syncthreads();
  if (wv != 0 || !live) return;
#pragma unroll
  for (int w = 1; w < 4; w++) acc += sums[w][lane];
  const Vec<4> x = {{acc[0], acc[1], acc[2], acc[3]}};
  write_row<ODT, 4>(p, cur, c, x);
}

namespace {

constexpr int64_t kRankIds = 8192;                 // most ids placed by comparison
constexpr int64_t kPartialBytes = (int64_t)256 << 20;

struct RowGradWs {
  int64_t piece;
  int passes, bits, tiles;
  size_t keys[2], pos[2], counts, part, bytes;
};
RowGradWs rowgrad_ws(int64_t n, int64_t V, int64_t hidden) {
  RowGradWs w = {};
  // 32 positions to a piece, 8 where there are few; more where the partial sums would not fit
  w.piece = n <= 4096 ? 8 : 32;
  w.piece = std::max<int64_t>(w.piece, (int64_t)align_up(cdiv(n * hidden * 8, kPartialBytes), 32));
  const bool ranked = n <= kRankIds;
  if (!ranked) {
    int bits = 1;
    while (((uint64_t)V >> bits) != 0) bits++;  // keys 0 .. V
    w.passes = (bits + 8) / 9;
    w.bits = (bits + w.passes - 1) / w.passes;
    w.tiles = (int)cdiv(n, kTileKeys);
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

template <int GDT, int ODT>
hipError_t launch_sums(const RowSums& p, hipStream_t stream) {
  const int64_t pieces = cdiv(p.n, p.piece);
  // 16-byte loads of the gradient rows
  if (GDT != DT_F32 && p.hidden % 8 == 0) {
    hipLaunchKernelGGL((rowgrad_sum_kernel<GDT, ODT, GDT == DT_F32 ? 4 : 8>),
                       dim3((unsigned)pieces, (unsigned)cdiv(p.hidden, 4 * 64 * 8)), dim3(256), 0, stream, p);
  } else {
    hipLaunchKernelGGL((rowgrad_sum_kernel<GDT, ODT, 4>), dim3((unsigned)pieces, (unsigned)cdiv(p.hidden, 4 * 64 * 4)),
                       dim3(256), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pieces == 1) return e;
  hipLaunchKernelGGL(rowgrad_join_kernel<ODT>, dim3((unsigned)(pieces - 1), (unsigned)cdiv(p.hidden, 256)), dim3(256),
                     0, stream, p);
  return hipGetLastError();
}

template <int GDT>
hipError_t launch_sums_to(const RowSums& p, int32_t out_dtype, hipStream_t stream) {
  switch (out_dtype) {
    case DT_F32: return launch_sums<GDT, DT_F32>(p, stream);
    case DT_BF16: return launch_sums<GDT, DT_BF16>(p, stream);
    default: return launch_sums<GDT, DT_F16>(p, stream);
  }
}

}  // namespace

size_t rowgrad_workspace(int64_t n, int64_t V, int64_t hidden) { return n == 0 ? 0 : rowgrad_ws(n, V, hidden).bytes; }

hipError_t launch_rowgrad(const RowGrad& g, void* ws, hipStream_t stream) {
  hipError_t e;
  if (!g.add) {
    const int64_t bytes = g.V * g.hidden * (g.out_dtype == DT_F32 ? 4 : 2);  // whole rows of 16 bytes
    if ((e = launch_write_probe(g.out, bytes, 0, stream)) != hipSuccess) return e;
  }
  if (g.n == 0) return hipSuccess;
  const RowGradWs w = rowgrad_ws(g.n, g.V, g.hidden);
  uint8_t* base = (uint8_t*)ws;
  uint32_t *keys = (uint32_t*)(base + w.keys[0]), *order = (uint32_t*)(base + w.pos[0]);
  if (w.passes == 0) {
    hipLaunchKernelGGL(rowgrad_rank_kernel, dim3((unsigned)cdiv(g.n, 64)), dim3(1024), 0, stream, g.ids, (int)g.n,
                       (uint32_t)g.V, keys, order);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int i = 0; i < w.passes; i++) {
    SortPass p = {};
    p.ids = i == 0 ? g.ids : nullptr;
    p.key = (uint32_t*)(base + w.keys[(i + 1) % 2]), p.pos = (uint32_t*)(base + w.pos[(i + 1) % 2]);
    p.n = g.n, p.V = (uint32_t)g.V, p.shift = i * w.bits, p.bits = w.bits, p.tiles = w.tiles;
    keys = (uint32_t*)(base + w.keys[i % 2]), order = (uint32_t*)(base + w.pos[i % 2]);
    uint32_t* counts = (uint32_t*)(base + w.counts);
    hipLaunchKernelGGL(rowgrad_count_kernel, dim3((unsigned)w.tiles), dim3(64 * kSortWaves), 0, stream, p, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(rowgrad_scan_kernel, dim3(1), dim3(1024), 0, stream, counts, (int64_t)w.tiles << w.bits);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(rowgrad_move_kernel, dim3((unsigned)w.tiles), dim3(64 * kSortWaves), 0, stream, p, counts, keys,
                       order);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  RowSums p = {};
  p.keys = keys, p.order = order, p.n = g.n, p.V = (uint32_t)g.V;
  p.grad = (const uint8_t*)g.grad, p.pitch = g.pitch, p.hidden = (int)g.hidden, p.piece = (int)w.piece;
  p.scale = g.scale, p.out = g.out, p.add = g.add, p.part = (float*)(base + w.part);
  switch (g.grad_dtype) {
    case DT_F32: return launch_sums_to<DT_F32>(p, g.out_dtype, stream);
    case DT_BF16: return launch_sums_to<DT_BF16>(p, g.out_dtype, stream);
    default: return launch_sums_to<DT_F16>(p, g.out_dtype, stream);
  }
}

}  // namespace etg
