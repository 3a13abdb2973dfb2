// Softmax cross entropy of residual rows over the whole vocabulary of a tied lm_head, and
// its gradients, without the logits in memory:
//   L[b][v] = sum_i x[b][i] E[v][i],  lse[b] = ln sum_v exp(L[b][v]),  loss[b] = lse[b] - L[b][label b]
//   D[b][v] = (g_b + h_b) exp(L[b][v] - lse[b]) - g_b [v = label b]
//   dx = D E,  dE = D^T x
// with g and h the gradients that reach loss and lse.  The forward pass is one product whose
// tiles leave a (maximum, sum of exponentials) per residual row.  The backward pass takes the
// vocabulary in pieces: the product again, with D (rounded to the table's type, the operand
// of the two other products) as its result, then the piece's share of dx and its rows of dE.
#include <algorithm>
#include <type_traits>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kXWaves = 8;
constexpr int kGroup = 4;  // tiles along n that neighbouring workgroups share
constexpr uint32_t kOutside = 0x80000000u;  // a copy's offset past its descriptor: zeros arrive

template <int DT>
constexpr int kValue = DT == DT_F32 ? 4 : 2;  // bytes

// acc += a b over one fragment each: 16 bytes per lane, lane l holding K values of row l % 16
// of its operand.  16-bit types: K values 8 (l / 16) + 0 .. 7 in one v_mfma_f32_16x16x32;
// f32: K values 4 (l / 16) + i in the i-th of four v_mfma_f32_16x16x4 (the sum is over all
// of them in either case).  Result register i of lane l: row 4 (l / 16) + i of a, row l % 16 of b.
template <int DT>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 acc) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc,
                                                   0, 0, 0);
  } else if constexpr (DT == DT_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0,
                                                  0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
    return acc;
  }
}

// 1 KiB from memory to LDS: lane l's 16 bytes at base + offset to lds + 16 l (base and lds
// uniform).  An offset at or past 2^31 - 1 is outside the descriptor: no memory is read and
// zeros are written.  In assembly because the compiler would wait for every such copy before
// any LDS read; load_wait waits for the one that is due.  No register is written.
__device__ __forceinline__ void copy_1k(uint64_t base, uint32_t offset, uint32_t lds) {
  const u32x4 rsrc = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
  uint32_t m0;  // the LDS base register, left as it was
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(m0)
      : "v"(offset), "s"(rsrc), "s"(lds)
      : "memory");
}

// Waits until at most N copies of this wave are in flight and its LDS reads are done.
template <int N>
__device__ __forceinline__ void load_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}
// A workgroup barrier that no memory access crosses (the compiler's own also waits for copies).
__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" ::: "memory"); }

// One operand of a product, R rows of it per tile and 128 bytes of K values per stage (KS of
// them).  TR false: rows of K values in memory, pitch bytes apart.  TR true: the K values of
// one row are pitch bytes apart, its neighbours side by side (the operand's transpose is
// what memory holds).
//
// LDS image of a stage, in 16-byte pieces (64 banks of 4 bytes):
//   TR false  row r at 128 r, piece p at p ^ ((r / 2) % 8): the 16 rows that 16 lanes read one
//             piece of lie on 16 different piece columns of the 256-byte bank row.
//   TR true   blocks of 128 rows (16 KiB); K value k at 128 ES k, piece p at p ^ swizzle(k), so
//             that the K values that one transposing read takes lie on different banks.
template <int DT, bool TR, int R>
struct Operand {
  static constexpr int ES = kValue<DT>, KS = 128 / ES, BYTES = R * 128, COPIES = BYTES / 1024 / kXWaves;
  static constexpr int LINE = 128 * ES;  // TR: bytes of one K value's 128 rows
  static_assert(COPIES >= 1 && (!TR || R % 128 == 0), "tile rows");
  uint64_t base;            // first byte of the tile: row row0 (TR: K value k0, row row0)
  int64_t pitch;
  uint32_t off[COPIES];     // this lane's piece of each of the wave's copies, or kOutside
  int k_of[COPIES];         // TR: its K value within the stage; else its first byte within the stage
  int k_end;                // K values (TR) or bytes of K values in the slice

  static __device__ __forceinline__ int swizzle(int k) {
    return ES == 2 ? 2 * (((k >> 3) & 1) * 4 + (k & 3)) : 4 * ((k >> 2) & 3);
  }
  // rows [row0, rows) of the operand, K values [k0, k0 + kn)
  __device__ __forceinline__ Operand(const uint8_t* p, int64_t pitch_, int64_t row0, int64_t rows, int64_t k0, int kn,
                                     int wv, int lane) {
    pitch = pitch_;
    const int left = (int)min(rows - row0, (int64_t)R);
    if constexpr (TR) {
      base = (uint64_t)p + (uint64_t)(k0 * pitch + row0 * ES);
      k_end = kn;
    } else {
      base = (uint64_t)p + (uint64_t)(row0 * pitch + k0 * ES);
      k_end = kn * ES;
    }
#pragma unroll
    for (int j = 0; j < COPIES; j++) {
      const int q = place(wv, j);
      if constexpr (TR) {
        const int at = q % 16 * 1024 + lane * 16, k = at / LINE, piece = at % LINE / 16 ^ swizzle(k);
        const int row = q / 16 * 128 + piece * (16 / ES);  // rows are whole pieces: the pitch and their number are
        k_of[j] = k;
        off[j] = row < left ? (uint32_t)(k * pitch) + (uint32_t)(row * ES) : kOutside;
      } else {
        const int row = 8 * q + (lane >> 3);
        const int piece = (lane & 7) ^ (4 * (COPIES == 1 ? q & 1 : j & 1) + (lane >> 4));  // (row / 2) % 8
        k_of[j] = 16 * piece;
        off[j] = row < left ? (uint32_t)(row * pitch) + (uint32_t)(16 * piece) : kOutside;
      }
    }
  }
  // the wave's j-th copy of stage s to the image at lds (copies of 128 rows of a tile are
  // side by side: j of R / 64)
  __device__ __forceinline__ void copy(int s, int j, int wv, uint32_t lds) const {
    const int step = TR ? s * KS : s * 128;
    // a lane outside stays outside: 2^31 plus at most 2^30 bytes of K values
    const uint32_t at = k_of[j] + step < k_end ? off[j] + (TR ? 0u : (uint32_t)step) : kOutside;
    copy_1k(TR ? base + (uint64_t)step * (uint64_t)pitch : base, at, lds + (uint32_t)place(wv, j) * 1024);
  }
  // which KiB of the image a copy fills: with 256 rows, the wave's first half of copies lies in
  // rows 0 .. 127 and the second in the others
  static __device__ __forceinline__ int place(int wv, int j) {
    return COPIES == 4 ? j / 2 * 16 + wv * 2 + j % 2 : wv * COPIES + j;
  }
  // Fragment of rows [row, row + 16) (row a multiple of 16) and K half kk of the stage at img.
  static __device__ __forceinline__ u32x4 read(const unsigned char* img, int row, int kk, int lane) {
    const int g = lane >> 4;
    if constexpr (!TR) {
      return *(const u32x4*)(img + row * 128 + (lane & 15) * 128 + 16 * ((4 * kk + g) ^ ((lane >> 1) & 7)));
    } else if constexpr (ES == 2) {
      // ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block, lane i K value i / 4 of it and rows
      // 4 (i % 4) .. + 3, and receive row i's four K values
      const unsigned char* blk = img + (row >> 7) * 16384;
      const int kl = 8 * g + ((lane & 15) >> 2);
      const int piece = (((row & 127) >> 3) + ((lane & 3) >> 1)) ^ swizzle(kl);
      const unsigned char* at = blk + (32 * kk + kl) * LINE + 16 * piece + 8 * (lane & 1);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * LINE));
      const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
      return u32x4{l2.x, l2.y, h2.x, h2.y};
    } else {
      const unsigned char* blk = img + (row >> 7) * 16384;
      const int col = (row & 127) + (lane & 15);
      const unsigned char* at = blk + (16 * kk + 4 * g) * LINE + 16 * ((col >> 2) ^ swizzle(4 * g)) + 4 * (col & 3);
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = *(const uint32_t*)(at + i * LINE);
      return v;
    }
  }
};

// One product C[m][n] = sum_k A[m][k] B[n][k].
enum { X_STATS, X_DLOGIT, X_PART, X_OUT };
struct XentProduct {
  const uint8_t *a, *b;
  int64_t a_pitch, b_pitch;  // bytes
  int64_t m, n, k;
  int32_t mt, nt;            // tiles
  int32_t splits;            // K slices of kslice values (a multiple of a stage)
  int32_t kslice;
  // X_STATS: part [n][mt], target [n]; X_DLOGIT: D [n][out_pitch bytes]
  // X_PART: f32 [splits][n][m]; X_OUT: values of the type, [n][m]
  void* out;
  int64_t out_pitch;
  int32_t add;               // X_PART, X_OUT: to what is there
  const int32_t* labels;     // [n]
  int64_t v0, vocab;         // the piece's first table row
  float* target;
  const float *lse, *grad_loss, *grad_lse;
  float grad_loss_all;       // where grad_loss is NULL
  const float* scale;        // X_DLOGIT: factor [0] of D; X_OUT: factor [1] of the product (NULL: 1)
};

// four values rounded to the type (to nearest even; f16 past 65504: infinity)
template <int DT>
__device__ __forceinline__ auto round4(f32x4 x) {
  if constexpr (DT == DT_F32) return x;
  else if constexpr (DT == DT_BF16) return __builtin_convertvector(x, bf16x4);
  else return __builtin_convertvector(x, f16x4);
}
template <int DT>
__device__ __forceinline__ void store4(void* at, f32x4 x) {
  *(decltype(round4<DT>(x))*)at = round4<DT>(x);
}
template <int DT>
__device__ __forceinline__ f32x4 load4(const void* at) {
  if constexpr (DT == DT_F32) {
    return *(const f32x4*)at;
  } else if constexpr (DT == DT_BF16) {
    return __builtin_convertvector(*(const bf16x4*)at, f32x4);
  } else {
    return __builtin_convertvector(*(const f16x4*)at, f32x4);
  }
}

// (maximum, sum of exp relative to it) of the union of two sets; (-inf, 0) is the empty one.
// A NaN in either sum stays.
__device__ __forceinline__ float2 stats_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), at = m == -__builtin_inff() ? 0.f : m;
  return make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - at) * kLog2e) +
                            b.y * __builtin_amdgcn_exp2f((b.x - at) * kLog2e));
}

// What a wave does with its MT x NT tiles of 16 x 16: registers i of tile (a, t) are rows
// m0 + row(a) + 4 (lane / 16) + i and column n0 + col(t) + lane % 16 of the product, where the
// first AH (TH) tiles along a direction are neighbours and the others lie 128 further.
// smem: the LDS of the finished K loop, all of it free.
template <int DT, int MODE, int MT, int NT, int AH, int TH, int WM, int BN>
__device__ __forceinline__ void finish(const XentProduct& p, f32x4 (&acc)[MT][NT], int64_t m0, int64_t n0, int mrow,
                                       int ncol, int mtile, int split, int wm, int lane, unsigned char* smem) {
  const int g = lane >> 4;
  auto row_of = [&](int a) { return m0 + mrow + a / AH * 128 + a % AH * 16 + 4 * g; };
  auto col_of = [&](int t) { return n0 + ncol + t / TH * 128 + t % TH * 16 + (lane & 15); };
  if constexpr (MODE == X_STATS) {
    float2* red = (float2*)smem;  // [WM][BN]
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int64_t n = col_of(t);
      const int64_t label = n < p.n ? (int64_t)(uint32_t)p.labels[n] - p.v0 : -1;  // its row in the piece
      float m = -__builtin_inff(), s = 0.f;
#pragma unroll
      for (int a = 0; a < MT; a++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int64_t v = row_of(a) + i;
          if (v < p.m) m = fmaxf(m, acc[a][t][i]);
          if (v == label && v < p.m) p.target[n] = acc[a][t][i];
        }
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      // all -inf (or no row): exp2(-inf) = 0 for each, a NaN stays one
      const float at = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
      for (int a = 0; a < MT; a++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int64_t v = row_of(a) + i;
          if (v < p.m) s += __builtin_amdgcn_exp2f((acc[a][t][i] - at) * kLog2e);
        }
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (g == 0) red[wm * BN + (int)(n - n0)] = make_float2(m, s);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < BN; c += 64 * kXWaves) {
      float2 r = red[c];
      for (int w = 1; w < WM; w++) r = stats_join(r, red[w * BN + c]);
      if (n0 + c < p.n) ((float2*)p.out)[(n0 + c) * p.mt + mtile] = r;
    }
  } else if constexpr (MODE == X_DLOGIT) {
    const float scale = p.scale != nullptr ? p.scale[0] : 1.f;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int64_t n = col_of(t);
      if (n >= p.n) continue;
      const uint32_t token = (uint32_t)p.labels[n];
      const float gl = token < (uint64_t)p.vocab ? (p.grad_loss != nullptr ? p.grad_loss[n] : p.grad_loss_all) : 0.f;
      const float both = p.grad_lse != nullptr ? gl + p.grad_lse[n] : gl;
      const int64_t label = (int64_t)token - p.v0;
      const float lse = p.lse[n];
      unsigned char* row = (unsigned char*)p.out + n * p.out_pitch;
#pragma unroll
      for (int a = 0; a < MT; a++) {
        const int64_t v = row_of(a);
        f32x4 d;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float e = __builtin_amdgcn_exp2f((acc[a][t][i] - lse) * kLog2e);
          // a row that nothing reaches has no gradient, whatever its logits are
          const float x = both == 0.f ? 0.f : both * e;
          d[i] = v + i < p.m ? (x - (v + i == label ? gl : 0.f)) * scale : 0.f;
        }
        store4<DT>(row + v * kValue<DT>, d);
      }
    }
  } else {
    const float scale = MODE == X_OUT && p.scale != nullptr ? p.scale[1] : 1.f;
    constexpr int ODT = MODE == X_PART ? DT_F32 : DT;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int64_t n = col_of(t);
      if (n >= p.n) continue;
      unsigned char* row = (unsigned char*)p.out + ((int64_t)split * p.n + n) * p.m * kValue<ODT>;
#pragma unroll
      for (int a = 0; a < MT; a++) {
        const int64_t m = row_of(a);
        if (m >= p.m) continue;  // m is a multiple of 4
        f32x4 x = acc[a][t] * scale;
        if (p.add) x += load4<ODT>(row + m * kValue<ODT>);
        store4<ODT>(row + m * kValue<ODT>, x);
      }
    }
  }
}

// Tile and K slice of a workgroup.  Ids {x, x + 8, ...} run on XCD x: each XCD takes a
// contiguous share of the tiles, in blocks of kGroup tiles along n by all along m: its 32
// CUs work on about kGroup x 32 / kGroup tiles, which share their operands' slices in its L2.
struct XentPlace {
  int mtile, ntile, split;
  bool some;
  __device__ __forceinline__ XentPlace(const XentProduct& p) {
    const int per = (int)(gridDim.x / 8), id = (int)blockIdx.x;
    int tile = id % 8 * per + id / 8;
    const int each = p.mt * p.nt;
    some = tile < each * p.splits;
    split = __builtin_amdgcn_readfirstlane(tile / each);
    tile -= split * each;
    const int block = __builtin_amdgcn_readfirstlane(tile / (kGroup * p.mt));
    tile -= block * kGroup * p.mt;
    const int wide = min(kGroup, p.nt - block * kGroup);
    mtile = __builtin_amdgcn_readfirstlane(tile / wide);
    ntile = block * kGroup + tile - mtile * wide;
  }
};

// Tiles of BM x BN, K through a ring of RING LDS images, RING - 1 stages ahead: one barrier
// per stage.
template <int DT, bool TA, bool TB, int MODE, int BM, int BN, int WM, int RING>
__global__ void __launch_bounds__(64 * kXWaves) ring_kernel(XentProduct p) {
  using A = Operand<DT, TA, BM>;
  using B = Operand<DT, TB, BN>;
  constexpr int WN = kXWaves / WM, MT = BM / WM / 16, NT = BN / WN / 16, IMG = A::BYTES + B::BYTES;
  static_assert(RING * IMG <= (int)kMaxLds, "LDS");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const XentPlace at(p);
  if (!at.some) return;  // whole workgroup
  const int64_t m0 = (int64_t)at.mtile * BM, n0 = (int64_t)at.ntile * BN, k0 = (int64_t)at.split * p.kslice;
  const int kn = (int)min((int64_t)p.kslice, p.k - k0), stages = (kn + A::KS - 1) / A::KS;
  const A oa(p.a, p.a_pitch, m0, p.m, k0, kn, wv, lane);
  const B ob(p.b, p.b_pitch, n0, p.n, k0, kn, wv, lane);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  auto copy = [&](int s) {  // past the last stage: zeros that nothing reads
    const uint32_t to = lds + (uint32_t)(s % RING) * IMG;
#pragma unroll
    for (int j = 0; j < A::COPIES; j++) oa.copy(s, j, wv, to);
#pragma unroll
    for (int j = 0; j < B::COPIES; j++) ob.copy(s, j, wv, to + A::BYTES);
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; a++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < RING - 1; s++) copy(s);
  for (int s = 0; s < stages; s++) {
    // stage s has landed, and every wave has read the image that the next copies refill
    load_wait<(RING - 2) * (A::COPIES + B::COPIES)>();
    bare_barrier();
    copy(s + RING - 1);
    const unsigned char* img = smem + s % RING * IMG;
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
      u32x4 fa[MT], fb[NT];
#pragma unroll
      for (int t = 0; t < NT; t++) fb[t] = B::read(img + A::BYTES, wn * (BN / WN) + 16 * t, kk, lane);
#pragma unroll
      for (int a = 0; a < MT; a++) fa[a] = A::read(img, wm * (BM / WM) + 16 * a, kk, lane);
#pragma unroll
      for (int a = 0; a < MT; a++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[a][t] = mma<DT>(fa[a], fb[t], acc[a][t]);
    }
  }
  load_wait<0>();
  bare_barrier();
  finish<DT, MODE, MT, NT, MT, NT, WM, BN>(p, acc, m0, n0, wm * (BM / WM), wn * (BN / WN), at.mtile, at.split, wm, lane,
                                           smem);
}

// Tiles of 256 x 256, bound by the matrix cores.  Two LDS images of a stage; 2 x 4 waves, two
// per SIMD, each with 64 rows of either half of A's tile and 32 of either half of B's.  A
// stage is four steps, one for each pair of halves: a step reads one half's fragments, issues
// two copies, then runs its 16 fragment products.  The waves of the second row of waves are
// one barrier behind the first, so that on every SIMD one wave's products run while the
// other reads.  B's halves are taken in turn, so that the one a stage begins with is read in
// the last step before it.  A half of an image is free once the second row of waves has read
// it, a step after the first, and is refilled in that step: every copy has six steps, one
// and a half stages, until it is waited for.
template <int DT, bool TA, bool TB, int MODE>
__global__ void __launch_bounds__(64 * kXWaves, 2) tile_kernel(XentProduct p) {
  using A = Operand<DT, TA, 256>;
  using B = Operand<DT, TB, 256>;
  constexpr int IMG = A::BYTES + B::BYTES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // [2][IMG]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / 4, wn = wv % 4;
  const XentPlace at(p);
  if (!at.some) return;  // whole workgroup
  const int64_t m0 = (int64_t)at.mtile * 256, n0 = (int64_t)at.ntile * 256, k0 = (int64_t)at.split * p.kslice;
  const int kn = (int)min((int64_t)p.kslice, p.k - k0), stages = (kn + A::KS - 1) / A::KS;
  const A oa(p.a, p.a_pitch, m0, p.m, k0, kn, wv, lane);
  const B ob(p.b, p.b_pitch, n0, p.n, k0, kn, wv, lane);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  // half h of stage s (past the last stage: zeros that nothing reads)
  auto copy_a = [&](int s, int h) {
    oa.copy(s, 2 * h, wv, lds + (uint32_t)(s & 1) * IMG);
    oa.copy(s, 2 * h + 1, wv, lds + (uint32_t)(s & 1) * IMG);
  };
  auto copy_b = [&](int s, int h) {
    ob.copy(s, 2 * h, wv, lds + (uint32_t)(s & 1) * IMG + A::BYTES);
    ob.copy(s, 2 * h + 1, wv, lds + (uint32_t)(s & 1) * IMG + A::BYTES);
  };
  f32x4 acc[8][4];
#pragma unroll
  for (int a = 0; a < 8; a++)
#pragma unroll
    for (int t = 0; t < 4; t++) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 fa[4][2], fb[2][2][2];
  auto read_a = [&](int s, int h) {
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++) fa[a][kk] = A::read(smem + (s & 1) * IMG, 128 * h + 64 * wm + 16 * a, kk, lane);
  };
  auto read_b = [&](int s, int h) {
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++)
        fb[h][t][kk] = B::read(smem + (s & 1) * IMG + A::BYTES, 128 * h + 32 * wn + 16 * t, kk, lane);
  };
  auto products = [&](int ha, int hb) {
    load_wait<12>();  // the fragments are read; the half that the next step reads has landed
    __builtin_amdgcn_sched_barrier(0);
    bare_barrier();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; kk++)
#pragma unroll
      for (int a = 0; a < 4; a++)
#pragma unroll
        for (int t = 0; t < 2; t++)
          acc[4 * ha + a][2 * hb + t] = mma<DT>(fa[a][kk], fb[hb][t][kk], acc[4 * ha + a][2 * hb + t]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    bare_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage s, half F of B first (its fragments are there).
  auto stage = [&](int s, auto first) {
    constexpr int F = decltype(first)::value, L = 1 - F;
    copy_b(s + 2, F);
    read_a(s, 0);
    products(0, F);
    copy_a(s + 2, 0);
    read_b(s, L);
    products(0, L);
    copy_b(s + 2, L);
    read_a(s, 1);
    products(1, L);
    copy_a(s + 2, 1);
    read_b(s + 1, L);
    products(1, F);
  };
  copy_b(0, 0), copy_a(0, 0), copy_b(0, 1), copy_a(0, 1);
  copy_b(1, 1), copy_a(1, 0), copy_b(1, 0), copy_a(1, 1);
  load_wait<12>();
  bare_barrier();
  read_b(0, 0);
  load_wait<12>();
  bare_barrier();  // the first step refills what was read here
  if (wm == 1) bare_barrier();
  int s = 0;
  for (; s + 1 < stages; s += 2) {
    stage(s, std::integral_constant<int, 0>{});
    stage(s + 1, std::integral_constant<int, 1>{});
  }
  if (s < stages) stage(s, std::integral_constant<int, 0>{});
  if (wm == 0) bare_barrier();
  load_wait<0>();
  bare_barrier();
  finish<DT, MODE, 8, 4, 4, 2, 2, 256>(p, acc, m0, n0, 64 * wm, 32 * wn, at.mtile, at.split, wm, lane, smem);
}

// Joins a piece's statistics [n][mt] into run [n]; the last piece writes lse and loss.  One
// wave per residual row.
__global__ void __launch_bounds__(256) xent_join_kernel(const float2* __restrict__ part, int mt, int64_t n, bool first,
                                                        bool last, float2* __restrict__ run,
                                                        const float* __restrict__ target,
                                                        const int32_t* __restrict__ labels, int64_t vocab,
                                                        float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (b >= n) return;  // whole wave
  float2 r = make_float2(-__builtin_inff(), 0.f);
  for (int i = lane; i < mt; i += 64) r = stats_join(r, part[b * mt + i]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    r = stats_join(r, make_float2(__shfl_xor(r.x, o, 64), __shfl_xor(r.y, o, 64)));
  if (lane != 0) return;
  if (!first) r = stats_join(run[b], r);
  if (!last) {
    run[b] = r;
    return;
  }
  // ln s in 64 bits: one rounding of the sum of both terms
  const float total = (float)((double)r.x + log((double)r.y));
  lse[b] = total;
  loss[b] = (uint32_t)labels[b] < (uint64_t)vocab ? (float)((double)r.x - (double)target[b] + log((double)r.y)) : 0.f;
}

// scale[0] = 2^e with the largest |g| + |h| times it in [2^13, 2^14), scale[1] = 2^-e: D in f16
// keeps 11 bits of probabilities down to 2^-27 of the largest coefficient instead of
// losing those below 2^-14 of 1.  One workgroup.
__global__ void __launch_bounds__(1024) xent_scale_kernel(const int32_t* __restrict__ labels, int64_t n, int64_t vocab,
                                                          const float* __restrict__ grad_loss, float grad_loss_all,
                                                          const float* __restrict__ grad_lse,
                                                          float* __restrict__ scale) {
  __shared__ float red[16];
  float m = 0.f;
  for (int64_t b = threadIdx.x; b < n; b += 1024) {
    const float gl =
        (uint32_t)labels[b] < (uint64_t)vocab ? (grad_loss != nullptr ? grad_loss[b] : grad_loss_all) : 0.f;
    const float both = grad_lse != nullptr ? gl + grad_lse[b] : gl;
    m = fmaxf(m, fmaxf(fabsf(gl), fabsf(both)));  // NaN is passed over
  }
  m = wave_max_f32(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 16; i++) m = fmaxf(m, red[i]);
  const int e = m > 0.f && m < __builtin_inff() ? 13 - ilogbf(m) : 0;
  scale[0] = ldexpf(1.f, min(max(e, -126), 126));
  scale[1] = ldexpf(1.f, -min(max(e, -126), 126));
}

// out = type(sum of the K slices' partial sums, times the factor)
template <int DT>
__global__ void __launch_bounds__(256) xent_sum_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                       int64_t hidden, void* __restrict__ out, int64_t out_pitch,
                                                       const float* __restrict__ scale) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x, each = hidden / 4;
  if (q >= n * each) return;
  const int64_t b = q / each, c = q % each * 4;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; s++) x += *(const f32x4*)(part + ((int64_t)s * n + b) * hidden + c);
  x *= scale != nullptr ? scale[1] : 1.f;
  // rows at any address of the type
  typedef decltype(round4<DT>(x)) V;
  typedef V Vu __attribute__((aligned(kValue<DT>)));
  *(Vu*)((unsigned char*)out + b * out_pitch + c * kValue<DT>) = round4<DT>(x);
}

// Rows of `bytes` (a multiple of 16) bytes, pitch bytes apart at any alignment, side by side.
__global__ void __launch_bounds__(256) xent_pack_kernel(const uint8_t* __restrict__ src, int64_t pitch, int64_t n,
                                                        int64_t bytes, uint8_t* __restrict__ dst) {
  typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x, each = bytes / 16;
  if (q >= n * each) return;
  *(u32x4*)(dst + q * 16) = *(const u32x4u*)(src + q / each * pitch + q % each * 16);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
namespace {

constexpr int kXcdCount = 8;

// Tile columns for n residual rows.
int rows_tile(int64_t n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }

template <int DT, bool TA, bool TB, int MODE, int BM, int BN, int WM, int RING>
hipError_t launch_ring(const XentProduct& p, hipStream_t stream) {
  const void* fn = (const void*)ring_kernel<DT, TA, TB, MODE, BM, BN, WM, RING>;
  const size_t lds = (size_t)RING * (BM + BN) * 128;
  hipError_t e = set_dynamic_lds(fn, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = (int64_t)p.mt * p.nt * p.splits;
  hipLaunchKernelGGL((ring_kernel<DT, TA, TB, MODE, BM, BN, WM, RING>), dim3((unsigned)(cdiv(tiles, kXcdCount) * kXcdCount)),
                     dim3(64 * kXWaves), lds, stream, p);
  return hipGetLastError();
}

template <int DT, bool TA, bool TB, int MODE>
hipError_t launch_tile(const XentProduct& p, hipStream_t stream) {
  const void* fn = (const void*)tile_kernel<DT, TA, TB, MODE>;
  const size_t lds = 2 * 512 * 128;
  hipError_t e = set_dynamic_lds(fn, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = (int64_t)p.mt * p.nt * p.splits;
  hipLaunchKernelGGL((tile_kernel<DT, TA, TB, MODE>), dim3((unsigned)(cdiv(tiles, kXcdCount) * kXcdCount)),
                     dim3(64 * kXWaves), lds, stream, p);
  return hipGetLastError();
}

// A product whose columns are residual rows.
template <int DT, bool TA, int MODE>
hipError_t launch_by_rows(const XentProduct& p, int bn, hipStream_t stream) {
  if (bn == 64) return launch_ring<DT, TA, false, MODE, 256, 64, 8, 4>(p, stream);
  if (bn == 128) return launch_ring<DT, TA, false, MODE, 256, 128, 4, 3>(p, stream);
  return launch_tile<DT, TA, false, MODE>(p, stream);
}

constexpr int64_t kMaxTiles = 1 << 20;             // of one launch
constexpr int64_t kPartBytes = (int64_t)256 << 20;  // statistics, or D, of one piece

// Pieces of at most `most` tiles of 256 table rows, as even as they get; in rows.
int64_t even_piece(int64_t vocab, int64_t most) {
  const int64_t tiles = cdiv(vocab, 256);
  return cdiv(tiles, cdiv(tiles, std::max<int64_t>(1, most))) * 256;
}
// Forward: the piece's statistics stay within kPartBytes.
int64_t forward_piece(int64_t vocab, int64_t n) {
  return even_piece(vocab, std::min(kMaxTiles / cdiv(n, rows_tile(n)), kPartBytes / (n * 8)));
}
// Backward: D of a piece stays within kPartBytes and its rows within 4 MiB.
int64_t backward_piece(int64_t vocab, int64_t n, int size) {
  return even_piece(vocab, std::min(std::min(kMaxTiles / cdiv(n, rows_tile(n)), (int64_t)4096),
                                    kPartBytes / (n * size * 256)));
}
// K slices of dx = D E: the fewest rounds of one workgroup per CU, times the stages of one and
// what its start and end cost (about 24 stages); at least 512 table rows each.
int64_t backward_splits(int64_t piece, int64_t n, int64_t hidden) {
  const int64_t tiles = cdiv(hidden, 256) * cdiv(n, rows_tile(n));
  int64_t best = 1, least = INT64_MAX;
  for (int64_t s = 1; s <= std::max<int64_t>(1, piece / 512) && s <= 2 * kTargetBlocks; s++) {
    const int64_t cost = cdiv(tiles * s, kTargetBlocks) * (cdiv(piece, 64 * s) + 24);
    if (cost < least) least = cost, best = s;
    if (tiles * s >= 8 * kTargetBlocks) break;
  }
  return best;
}
int64_t backward_slice(int64_t piece, int64_t splits) { return (int64_t)align_up(cdiv(piece, splits), 64); }

// The residual rows as the copies need them: 16-byte aligned, rows less than 8 MiB apart.
bool rows_direct(const void* x, int64_t pitch) { return ((uintptr_t)x | (uint64_t)pitch) % 16 == 0 && pitch < (8 << 20); }

struct BackwardWs {
  int64_t piece, splits, slice;
  size_t x, d, sums, bytes;
};
BackwardWs backward_ws(const TableDesc& t, int64_t n) {
  const int size = t.dtype == DT_F32 ? 4 : 2;
  BackwardWs w;
  w.piece = backward_piece(t.V, n, size);
  w.splits = backward_splits(w.piece, n, t.hidden);
  w.slice = backward_slice(w.piece, w.splits);
  w.splits = cdiv(w.piece, w.slice);
  w.x = 256;  // the two factors before it
  w.d = w.x + align_up((size_t)(n * t.row_bytes), 256);
  w.sums = w.d + align_up((size_t)(n * w.piece * size), 256);
  w.bytes = w.sums + align_up((size_t)(w.splits * n * t.hidden * 4), 256);
  return w;
}

hipError_t pack_rows(const XentCall& c, const TableDesc& t, uint8_t* to, hipStream_t stream) {
  const int64_t pieces = c.n * (t.row_bytes / 16);
  hipLaunchKernelGGL(xent_pack_kernel, dim3((unsigned)cdiv(pieces, 256)), dim3(256), 0, stream, (const uint8_t*)c.x,
                     c.x_pitch, c.n, t.row_bytes, to);
  return hipGetLastError();
}

template <int DT>
hipError_t forward(const TableDesc& t, const XentCall& c, uint8_t* ws, hipStream_t stream) {
  const int64_t piece = forward_piece(t.V, c.n);
  hipError_t e;
  // workspace: running statistics, targets, packed residual rows, the piece's statistics
  float2* run = (float2*)ws;
  float* target = (float*)(ws + align_up((size_t)c.n * 8, 256));
  uint8_t* packed = (uint8_t*)target + align_up((size_t)c.n * 4, 256);
  float2* part = (float2*)(packed + align_up((size_t)(c.n * t.row_bytes), 256));
  const bool direct = rows_direct(c.x, c.x_pitch);
  if (!direct && (e = pack_rows(c, t, packed, stream)) != hipSuccess) return e;
  const int bn = rows_tile(c.n);
  for (int64_t v0 = 0; v0 < t.V; v0 += piece) {
    XentProduct p = {};
    p.m = std::min(piece, t.V - v0), p.n = c.n, p.k = t.hidden;
    p.a = t.rows + v0 * t.row_bytes, p.a_pitch = t.row_bytes;
    p.b = direct ? (const uint8_t*)c.x : packed, p.b_pitch = direct ? c.x_pitch : t.row_bytes;
    p.mt = (int32_t)cdiv(p.m, 256), p.nt = (int32_t)cdiv(p.n, bn), p.splits = 1, p.kslice = (int32_t)t.hidden;
    p.out = part, p.labels = c.labels, p.v0 = v0, p.target = target;
    if ((e = launch_by_rows<DT, false, X_STATS>(p, bn, stream)) != hipSuccess) return e;
    hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)cdiv(c.n, 4)), dim3(256), 0, stream, part, p.mt, c.n, v0 == 0,
                       v0 + piece >= t.V, run, target, c.labels, t.V, c.loss, c.lse_out);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t backward(const TableDesc& t, const XentCall& c, uint8_t* ws, hipStream_t stream) {
  if (c.n == 0)  // a sum of nothing
    return c.d_rows == nullptr || c.add ? hipSuccess : launch_write_probe(c.d_rows, t.V * t.row_bytes, 0, stream);
  const BackwardWs w = backward_ws(t, c.n);
  hipError_t e;
  float* scale = DT == DT_F16 ? (float*)ws : nullptr;
  uint8_t *packed = ws + w.x, *d = ws + w.d;
  float* sums = (float*)(ws + w.sums);
  if (scale != nullptr) {
    hipLaunchKernelGGL(xent_scale_kernel, dim3(1), dim3(1024), 0, stream, c.labels, c.n, t.V, c.grad_loss,
                       c.grad_loss_all, c.grad_lse, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool direct = rows_direct(c.x, c.x_pitch);
  if (!direct && (e = pack_rows(c, t, packed, stream)) != hipSuccess) return e;
  const uint8_t* x = direct ? (const uint8_t*)c.x : packed;
  const int64_t x_pitch = direct ? c.x_pitch : t.row_bytes;
  const int bn = rows_tile(c.n);
  for (int64_t v0 = 0; v0 < t.V; v0 += w.piece) {
    const int64_t rows = std::min(w.piece, t.V - v0);
    const uint8_t* E = t.rows + v0 * t.row_bytes;
    {
      XentProduct p = {};
      p.m = rows, p.n = c.n, p.k = t.hidden;
      p.a = E, p.a_pitch = t.row_bytes, p.b = x, p.b_pitch = x_pitch;
      p.mt = (int32_t)cdiv(rows, 256), p.nt = (int32_t)cdiv(c.n, bn), p.splits = 1, p.kslice = (int32_t)t.hidden;
      p.out = d, p.out_pitch = w.piece * kValue<DT>;
      p.labels = c.labels, p.v0 = v0, p.vocab = t.V, p.lse = c.lse, p.grad_loss = c.grad_loss;
      p.grad_loss_all = c.grad_loss_all, p.grad_lse = c.grad_lse, p.scale = scale;
      if ((e = launch_by_rows<DT, false, X_DLOGIT>(p, bn, stream)) != hipSuccess) return e;
    }
    if (c.d_x != nullptr) {
      XentProduct p = {};
      p.m = t.hidden, p.n = c.n, p.k = rows;
      p.a = E, p.a_pitch = t.row_bytes, p.b = d, p.b_pitch = w.piece * kValue<DT>;
      p.mt = (int32_t)cdiv(t.hidden, 256), p.nt = (int32_t)cdiv(c.n, bn);
      p.splits = (int32_t)cdiv(rows, w.slice), p.kslice = (int32_t)w.slice;
      p.out = sums, p.add = v0 != 0;
      if ((e = launch_by_rows<DT, true, X_PART>(p, bn, stream)) != hipSuccess) return e;
    }
    if (c.d_rows != nullptr) {
      XentProduct p = {};
      p.m = t.hidden, p.n = rows, p.k = c.n;
      p.a = x, p.a_pitch = x_pitch, p.b = d, p.b_pitch = w.piece * kValue<DT>;
      p.mt = (int32_t)cdiv(t.hidden, 256), p.nt = (int32_t)cdiv(rows, 256);
      p.splits = 1, p.kslice = (int32_t)align_up((size_t)c.n, 64);
      p.out = (uint8_t*)c.d_rows + v0 * t.row_bytes, p.add = c.add, p.scale = scale;
      if ((e = launch_tile<DT, true, true, X_OUT>(p, stream)) != hipSuccess) return e;
    }
  }
  if (c.d_x != nullptr) {
    const int splits = (int)cdiv(std::min(w.piece, t.V), w.slice);  // of the first piece, the fullest
    hipLaunchKernelGGL(xent_sum_kernel<DT>, dim3((unsigned)cdiv(c.n * (t.hidden / 4), 256)), dim3(256), 0, stream,
                       sums, splits, c.n, t.hidden, c.d_x, c.d_x_pitch, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t xent_workspace(const TableDesc& t, int64_t n) {
  if (n == 0) return 0;
  const int64_t piece = forward_piece(t.V, n);
  return align_up((size_t)n * 8, 256) + align_up((size_t)n * 4, 256) + align_up((size_t)(n * t.row_bytes), 256) +
         align_up((size_t)(n * (piece / 256) * 8), 256);
}

size_t xent_grad_workspace(const TableDesc& t, int64_t n) { return n == 0 ? 0 : backward_ws(t, n).bytes; }

hipError_t launch_xent(const TableDesc& t, const XentCall& c, void* ws, hipStream_t stream) {
  switch (t.dtype) {
    case DT_F32: return forward<DT_F32>(t, c, (uint8_t*)ws, stream);
    case DT_BF16: return forward<DT_BF16>(t, c, (uint8_t*)ws, stream);
    default: return forward<DT_F16>(t, c, (uint8_t*)ws, stream);
  }
}

hipError_t launch_xent_grad(const TableDesc& t, const XentCall& c, void* ws, hipStream_t stream) {
  switch (t.dtype) {
    case DT_F32: return backward<DT_F32>(t, c, (uint8_t*)ws, stream);
    case DT_BF16: return backward<DT_BF16>(t, c, (uint8_t*)ws, stream);
    default: return backward<DT_F16>(t, c, (uint8_t*)ws, stream);
  }
}

}  // namespace etg
