// Softmax cross entropy of residual rows over the whole vocabulary of a tied lm_head, and
// its gradients, without the logits in memory:
//   L[b][v] = sum_i x[b][i] E[v][i],  lse[b] = ln sum_v exp(L[b][v]),  loss[b] = lse[b] - L[b][label b]
//   D[b][v] = (g_b + h_b) exp(L[b][v] - lse[b]) - g_b [v = label b]
//   dx = D E,  dE = D^T x
// with g and h the gradients that reach loss and lse.  The forward pass is one product whose
// tiles leave a (maximum, sum of exponentials) per residual row.  The backward pass takes the
// vocabulary in pieces: the product again, with D (rounded to the table's type, the operand
// of the two other products) as its result, then the piece's share of dx and its rows of dE.
//
// D's entry at a label, g (p - 1) + h p, is most of what a row contributes, and is near 0 where
// p is near 1.  There it is about g (L - lse), and an f32 logit of 17 is off by 1e-6: a label's
// logit is summed again, in 64 bits, for loss and lse (xent_join_kernel) and for the entry, which
// is formed by expm1 of its distance to lse and so has f32's relative accuracy for the given lse
// (label_entry).  What its rounding to 16 bits takes away (its "rest") is added to dx, and up to
// 128 residual rows to dE.  Up to 8 residual rows of small tables D is f32 (vector_rows).
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
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kXWaves = 8;
constexpr int kGroup = 4;  // tiles along n that neighbouring workgroups share
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every descriptor: zeros arrive

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

// A buffer descriptor of `valid` bytes (at most 2^31) at base, an address below 2^48.
__device__ __forceinline__ u32x4 descriptor(uint64_t base, int64_t valid) {
  return u32x4{(uint32_t)base, (uint32_t)(base >> 32), (uint32_t)min(max(valid, (int64_t)0), (int64_t)kOutside),
               0x00020000u};
}

// 1 KiB from memory to LDS: lane l's 16 bytes at the descriptor's base + offset to lds + 16 l
// (descriptor and lds uniform).  A lane whose offset is outside the descriptor reads no
// memory: zeros are written for it.  In assembly because the compiler would wait for every
// such copy before any LDS read; load_wait waits for the one that is due.  No register is
// written.
__device__ __forceinline__ void copy_1k(u32x4 rsrc, uint32_t offset, uint32_t lds) {
  uint32_t m0;  // the LDS base register, left as it was
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(m0)
      : "v"(offset), "s"(rsrc), "s"(lds)
      : "memory");
}

// Waits for this wave's LDS accesses alone.
__device__ __forceinline__ void load_wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }

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
//
// BLK: D, which is kept in blocks of 256 table rows, each [residual row][256]: what a tile writes
// and reads of it is one range of memory (64 x 262,144 x 5,376: 1,595 us with rows as long as the
// vocabulary, 1,538 so; 160 rows' table gradient 1,464 and 1,246).
constexpr int kBlock = 256;
template <int DT, bool TR, int R, bool BLK = false>
struct Operand {
  static constexpr int ES = kValue<DT>, KS = 128 / ES, BYTES = R * 128, COPIES = BYTES / 1024 / kXWaves;
  static constexpr int LINE = 128 * ES;  // TR: bytes of one K value's 128 rows
  static_assert(COPIES >= 1 && (!TR || (R % 128 == 0 && COPIES >= 2)), "tile rows");
  // of the stage that is copied from
  u32x4 rsrc;            // from the tile's first row (TR: and the stage's first K value) to the end of what may be read
  uint64_t base;         // its address
  int64_t valid;         // TR: its bytes
  int32_t k_left, far;   // TR false: bytes of K values left in a row; those before the stage (BLK: in the block)
  // always
  int64_t pitch, block;  // block: bytes of one (BLK)
  uint32_t off[TR ? 1 : 2];  // this lane's piece of the wave's first copy (TR false: and of one an odd number of copies on)
  uint32_t k_first;          // TR false: the former's first byte within the stage

  static __device__ __forceinline__ int swizzle(int k) {
    return ES == 2 ? 2 * (((k >> 3) & 1) * 4 + (k & 3)) : 4 * ((k >> 2) & 3);
  }
  // Rows [row0, rows) of the operand, K values [k0, k0 + kn).  BLK: pitch_ are a block's bytes;
  // k0 begins a block, and a tile's rows lie in one (TR).  TR: rows past the last one of a K value
  // are the next one's first: the products of such rows are not stored.
  __device__ __forceinline__ Operand(const uint8_t* p, int64_t pitch_, int64_t row0, int64_t rows, int64_t k0, int kn,
                                     int wv, int lane) {
    pitch = BLK ? kBlock * ES : pitch_;
    block = BLK ? pitch_ : 0;
    const int q = place(wv, 0);
    if constexpr (TR) {
      const int64_t first = (BLK ? row0 % kBlock : row0) * ES;
      base = (uint64_t)p + (uint64_t)((BLK ? row0 / kBlock * block : 0) + k0 * pitch + first);
      valid = rows > row0 ? (BLK ? (int64_t)kn * pitch - first : (int64_t)(kn - 1) * pitch + (rows - row0) * ES) : 0;
      const int at = q % 16 * 1024 + lane * 16, k = at / LINE;
      off[0] = (uint32_t)(k * (int)pitch) + (uint32_t)((at % LINE / 16 ^ swizzle(k)) * 16);
    } else {
      base = (uint64_t)p + (uint64_t)(BLK ? k0 / kBlock * block + row0 * pitch : row0 * pitch + k0 * ES);
      valid = min(rows - row0, (int64_t)R) * pitch;
      k_left = kn * ES, far = 0;
      k_first = 16u * ((lane & 7) ^ (4 * (q & 1) + (lane >> 4)));  // piece by (row / 2) % 8
      off[0] = (uint32_t)((8 * q + (lane >> 3)) * (int)pitch) + k_first;
      off[1] = off[0] - k_first + (k_first ^ 64u) + 8u * (uint32_t)pitch;
    }
    rsrc = descriptor(base, valid);
  }
  // The wave's j-th copy of the stage to the image at lds.  Its place differs from the first
  // one's by whole rows (TR: K values of the same swizzle; and 128 rows), and TR false by the
  // piece's third bit, as rows 8 apart have it.
  __device__ __forceinline__ void copy(int j, int wv, uint32_t lds) const {
    const int q = place(wv, j), d = q - place(wv, 0);  // d: 0, 1, 16 or 17
    uint32_t at;
    if constexpr (TR) {
      at = off[0] + (uint32_t)(d % 16 * (1024 / LINE) * (int)pitch + d / 16 * LINE);
    } else {
      at = off[d & 1] + (uint32_t)(far + d / 16 * 128 * (int)pitch);
      at = (int)(k_first ^ (d & 1 ? 64u : 0u)) < k_left ? at : kOutside;
    }
    copy_1k(rsrc, at, lds + (uint32_t)q * 1024);
  }
  // BLK, TR: to the first stage of the tile of kn K values at row0 (none: zeros)
  __device__ __forceinline__ void restart(const uint8_t* p, int64_t row0, int kn) {
    const int first = (int)(row0 % kBlock) * ES;
    base = (uint64_t)p + (uint64_t)(row0 / kBlock * block + first);
    valid = kn == 0 ? 0 : kn * pitch - first;
    rsrc = descriptor(base, valid);
  }
  // on to the next stage
  __device__ __forceinline__ void advance() {
    if constexpr (TR) {
      base += (uint64_t)(KS * pitch);
      valid -= KS * pitch;
      rsrc = descriptor(base, valid);
    } else {
      k_left -= 128, far += 128;
      if (BLK && far == kBlock * ES) {
        far = 0;
        base += (uint64_t)block;
        rsrc[0] = (uint32_t)base, rsrc[1] = (uint32_t)(base >> 32);
      }
    }
  }
  // which KiB of the image a copy fills: with 256 rows, the wave's first half of copies lies in
  // rows 0 .. 127 and the second in the others
  static __device__ __forceinline__ int place(int wv, int j) {
    return COPIES == 4 ? j / 2 * 16 + wv * 2 + j % 2 : wv * COPIES + j;
  }
  // Fragment of rows [row, row + 16) (row a multiple of 16) and K half kk of the stage at img.
  static __device__ __forceinline__ u32x4 read(const unsigned char* img, int row, int kk, int lane) {
    const uint32_t at = (uint32_t)(uintptr_t)(const lds_u32*)img;
    return TR ? read_at(at + lane_at(row & 127, 0, lane), (row >> 7) * 16384 + kk * HALF)
              : read_at(at + lane_at(0, kk, lane), row * 128);
  }
  // Where the lane's values of rows [row, row + 16) begin in an image, by K half (TR: the second half
  // lies HALF bytes on, and row < 128; else row r lies 128 r bytes on).
  static constexpr int HALF = 64 / ES * LINE;
  static __device__ __forceinline__ uint32_t lane_at(int row, int kk, int lane) {
    const int g = lane >> 4;
    if constexpr (!TR) {
      return row * 128 + (lane & 15) * 128 + 16 * ((4 * kk + g) ^ ((lane >> 1) & 7));
    } else if constexpr (ES == 2) {
      // ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block, lane i K value i / 4 of it and rows
      // 4 (i % 4) .. + 3, and receive row i's four K values
      const int kl = 8 * g + ((lane & 15) >> 2);
      return kl * LINE + 16 * (((row >> 3) + ((lane & 3) >> 1)) ^ swizzle(kl)) + 8 * (lane & 1);
    } else {
      const int col = row + (lane & 15);
      return 4 * g * LINE + 16 * ((col >> 2) ^ swizzle(4 * g)) + 4 * (col & 3);
    }
  }
  // The fragment that begins `more` (a constant) bytes behind a lane_at of the LDS address of an image.
  static __device__ __forceinline__ u32x4 read_at(uint32_t at, int more) {
    at += (uint32_t)more;
    if constexpr (!TR) {
      return *(const lds_u32x4*)(uintptr_t)at;
    } else if constexpr (ES == 2) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 4 * LINE));
      const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
      return u32x4{l2.x, l2.y, h2.x, h2.y};
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = *(const lds_u32*)(uintptr_t)(at + i * LINE);
      return v;
    }
  }
};

// The lane_at of T neighbouring tiles of 16 rows from `row`, in as many registers as it takes: left to
// itself the compiler keeps one for nearly every fragment of both images, and spilled in f32.  (In 16
// bits, too, the products gain: 1,024 x 262,144 x 5,120 bf16 statistics 2,056 us, 1,969 so.  f32 is bound
// elsewhere: 2,000 x 30,000 x 1,024 dx 2,026 us with 26 spilled registers, 2,077 so, dE 2,044 and 2,035.)
template <typename Op, bool TR, int T>
struct LaneAt {
  uint32_t at[TR ? T : 2];
  __device__ __forceinline__ LaneAt(uint32_t lds, int row, int lane) {
#pragma unroll
    for (int i = 0; i < (TR ? T : 2); i++) {
      at[i] = lds + (TR ? Op::lane_at(row + 16 * i, 0, lane) : Op::lane_at(row, i, lane));
      asm volatile("" : "+v"(at[i]));
    }
  }
  __device__ __forceinline__ u32x4 read(int tile, int kk, int more) const {
    return TR ? Op::read_at(at[tile], more + kk * Op::HALF) : Op::read_at(at[kk], more + tile * 16 * 128);
  }
};

// One product C[m][n] = sum_k A[m][k] B[n][k].
enum { X_STATS, X_DLOGIT, X_DLOGIT32, X_PART, X_OUT };
struct XentProduct {
  const uint8_t *a, *b;
  int64_t a_pitch, b_pitch;  // bytes (X_PART, X_OUT: b is D, b_pitch a block's bytes)
  int64_t m, n, k;
  int32_t mt, nt;            // tiles
  int32_t splits;            // K slices of kslice values (a multiple of a stage)
  int32_t kslice;
  // X_STATS: part [n][mt], target [n]; X_DLOGIT: D [m / 256][n][256]; X_DLOGIT32: f32 D [m][8]
  // X_PART: f32 [splits][n][m]; X_OUT: values of the type, [n][m]
  void* out;
  const float* entry;        // X_DLOGIT, X_DLOGIT32, but for direct_kernel: [n], D's entries at the labels
  float* rest;               // 16-bit types: [n], what D's rounding takes away from them
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
__device__ __forceinline__ auto round1(float x) {
  if constexpr (DT == DT_F32) return x;
  else if constexpr (DT == DT_BF16) return (__bf16)x;
  else return (_Float16)x;
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

// Stores a wave's 16 rows of 16 AH values: x[a][i] of lane l is value 16 a + 4 (l / 16) + i of row
// l % 16.  The first value of row 0 goes to `at`, rows are pitch bytes apart; `rows` of them
// and `most` values (a multiple of 4, 8 for 16-bit types) are stored.  16-bit types exchange
// them between the lanes first, so that a store writes whole lines (128 bytes of each of
// eight rows); stores of 8 bytes in every 32 took 1,076 us for 2.8 GB, of half lines 631, of
// whole ones 562.
template <int DT, int AH>
__device__ __forceinline__ void store_rows(unsigned char* at, int64_t pitch, const f32x4 (&x)[AH], int lane,
                                           int64_t rows, int most) {
  const int g = lane >> 4, r = lane & 15;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int a = 0; a < AH; a++)
      if (r < rows && 16 * a + 4 * g < most) *(f32x4*)(at + r * pitch + (16 * a + 4 * g) * 4) = x[a];
  } else {
    static_assert(AH == 4, "four tiles are exchanged");
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x4 w[2];  // of tiles (0, 1) and (2, 3): lane row g has values 8 g .. 8 g + 7 of 32
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const u32x2 lo = __builtin_bit_cast(u32x2, round4<DT>(x[2 * q]));
      const u32x2 hi = __builtin_bit_cast(u32x2, round4<DT>(x[2 * q + 1]));
#pragma unroll
      for (int i = 0; i < 2; i++) {
        // lane rows (0, 1, 2, 3) of tiles a, b -> (a0, a1, b0, b1), (a2, a3, b2, b3)
        const u32x2 s = __builtin_amdgcn_permlane32_swap(lo[i], hi[i], false, false);
        // -> (a0, a2, b0, b2), (a1, a3, b1, b3)
        const u32x2 t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
        w[q][i] = t[0], w[q][2 + i] = t[1];
      }
    }
    // lanes r and r ^ 8 exchange a half: the lower eight keep values 0 .. 31, of rows r and
    // r + 8, the upper eight values 32 .. 63 of rows r - 8 and r
    const bool upper = r >= 8;
    u32x4 first, second;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t got = __builtin_amdgcn_update_dpp(0u, upper ? w[0][i] : w[1][i], 0x128, 0xf, 0xf, false);  // row_ror:8
      first[i] = upper ? got : w[0][i];
      second[i] = upper ? w[1][i] : got;
    }
    // a uniform address and 32 bits of the lane's own
    const int value = (upper ? 32 : 0) + 8 * g;
    const uint32_t mine = (uint32_t)((r & 7) * (int)pitch) + (uint32_t)(value * 2);
    unsigned char* at8 = at + 8 * pitch;
    if (rows >= 16 && most >= 64) {  // uniform
      *(u32x4*)(at + mine) = first;
      *(u32x4*)(at8 + mine) = second;
    } else {
      if ((r & 7) < rows && value < most) *(u32x4*)(at + mine) = first;
      if ((r & 7) + 8 < rows && value < most) *(u32x4*)(at8 + mine) = second;
    }
  }
}

// The gradients that reach a residual row's loss and lse.
struct RowGrads {
  const int32_t* labels;
  int64_t vocab;
  const float *grad_loss, *grad_lse;
  float grad_loss_all;  // where grad_loss is NULL
  // Neither does: the row adds nothing to dE, whatever it holds (0 times a NaN would).
  __device__ __forceinline__ bool none(int64_t b) const {
    const float h = grad_lse != nullptr ? grad_lse[b] : 0.f, g = grad_loss != nullptr ? grad_loss[b] : grad_loss_all;
    return (g == 0.f || (uint32_t)labels[b] >= (uint64_t)vocab) && h == 0.f;
  }
};

// What D's entries (and the loss: the label alone) of one residual row need.
struct DRow {
  float both, lse, entry;
  int64_t label;  // the label's row in the piece; negative where there is none
  DRow() = default;
  template <int MODE>
  __device__ __forceinline__ void load(const XentProduct& p, int64_t n) {
    const uint32_t token = (uint32_t)p.labels[n];
    if constexpr (MODE == X_STATS) {
      label = (int64_t)token - p.v0;
      return;
    }
    both = token < (uint64_t)p.vocab ? (p.grad_loss != nullptr ? p.grad_loss[n] : p.grad_loss_all) : 0.f;
    if (p.grad_lse != nullptr) both += p.grad_lse[n];
    label = token < (uint64_t)p.vocab ? (int64_t)token - p.v0 : -1;
    lse = p.lse[n];
    entry = p.entry != nullptr ? p.entry[n] : 0.f;
  }
  // A row that nothing reaches has no gradient, whatever its logits are.
  __device__ __forceinline__ float other(float l) const {
    return both == 0.f ? 0.f : both * __builtin_amdgcn_exp2f((l - lse) * kLog2e);
  }
};

// Waits for what they loaded.
template <int MODE, int N>
__device__ __forceinline__ void here(DRow (&r)[N]) {
#pragma unroll
  for (int t = 0; t < N; t++) {
    asm volatile("" : "+v"(r[t].label));
    if constexpr (MODE != X_STATS) asm volatile("" : "+v"(r[t].both), "+v"(r[t].lse), "+v"(r[t].entry));
  }
}

// The 16 bytes' values.
template <int DT>
__device__ __forceinline__ void unpack(u32x4 w, float (&x)[16 / kValue<DT>]) {
#pragma unroll
  for (int i = 0; i < 16 / kValue<DT>; i++) {
    if constexpr (DT == DT_F32) x[i] = __uint_as_float(w[i]);
    else if constexpr (DT == DT_BF16) x[i] = i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else x[i] = f16_bits_to_f32(w[i / 2] >> 16 * (i % 2) & 0xffffu);
  }
}

// sum + a b over 16 bytes each; a product of two f32 values is exact in 64 bits
template <int DT>
__device__ __forceinline__ double dot64(u32x4 a, u32x4 b, double sum) {
  float x[16 / kValue<DT>], y[16 / kValue<DT>];
  unpack<DT>(a, x);
  unpack<DT>(b, y);
#pragma unroll
  for (int i = 0; i < 16 / kValue<DT>; i++) sum = fma((double)x[i], (double)y[i], sum);
  return sum;
}

// The logit of a residual row and a table row, in 64 bits, by one wave.
template <int DT>
__device__ __forceinline__ double wave_dot64(const uint8_t* x, const uint8_t* row, int64_t row_bytes, int lane) {
  double sum = 0.;
#pragma unroll 4
  for (int64_t at = lane * 16; at < row_bytes; at += 1024)
    sum = dot64<DT>(*(const u32x4*)(x + at), *(const u32x4*)(row + at), sum);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  return sum;
}

// (g + h) p - g at the label, from its logit's distance to lse: rounded once to f32, where expm1
// keeps its relative accuracy near p = 1.  A row that nothing reaches: 0.
__device__ __forceinline__ float label_entry(const RowGrads& grads, int64_t b, double logit, float lse) {
  const float g = grads.grad_loss != nullptr ? grads.grad_loss[b] : grads.grad_loss_all;
  const float h = grads.grad_lse != nullptr ? grads.grad_lse[b] : 0.f;
  const float t = (float)(logit - (double)lse);
  return g == 0.f && h == 0.f ? 0.f : g * expm1f(t) + h * __builtin_amdgcn_exp2f(t * kLog2e);
}

// (maximum, sum of exp relative to it) of the union of two sets; (-inf, 0) is the empty one.
// A NaN in either sum stays.
__device__ __forceinline__ float2 stats_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), at = m == -__builtin_inff() ? 0.f : m;
  return make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - at) * kLog2e) +
                            b.y * __builtin_amdgcn_exp2f((b.x - at) * kLog2e));
}

// What a wave does with its MT x NT tiles of 16 x 16: registers i of tile (a, t) are rows
// m0 + mrow + off(a) + 4 (lane / 16) + i and column n0 + ncol + off(t) + lane % 16 of the product,
// where the first AH (TH) tiles along a direction are neighbours and the others lie 128 further.
// smem: LDS that is free.
// drow(t): of column tile t (X_STATS, X_DLOGIT, X_DLOGIT32)
template <int DT, int MODE, int MT, int NT, int AH, int TH, int WM, int BN, typename Rows>
__device__ __forceinline__ void finish(const XentProduct& p, f32x4 (&acc)[MT][NT], int64_t m0, int64_t n0, int mrow,
                                       int ncol, int mtile, int split, int wm, int lane, Rows drow,
                                       unsigned char* smem) {
  const int g = lane >> 4;
  // rows in 32 bits, from this lane's first one
  auto off = [](int a) { return a / AH * 128 + a % AH * 16; };
  auto col0 = [&](int t) { return n0 + ncol + t / TH * 128 + t % TH * 16; };
  auto col_of = [&](int t) { return col0(t) + (lane & 15); };
  const int first = mrow + 4 * g, rows = (int)min(p.m - m0, (int64_t)256) - first;
  auto place = [&](int64_t row) {  // of a row of the piece; negative where the tile lacks it
    return row >= m0 && row < m0 + 256 && row < p.m ? (int)(row - m0) - first : -1024;
  };
  if constexpr (MODE == X_STATS) {
    float2* red = (float2*)smem;  // [WM][BN]
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int64_t n = col_of(t);
      const DRow row = drow(t);
      const int label = n < p.n ? place(row.label) : -1024;
      float m = -__builtin_inff(), s = 0.f;
#pragma unroll
      for (int a = 0; a < MT; a++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (off(a) + i < rows) m = fmaxf(m, acc[a][t][i]);
      if (__ballot(label >= 0) != 0) {
        float l = 0.f;
        bool here = false;
#pragma unroll
        for (int a = 0; a < MT; a++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (off(a) + i == label) l = acc[a][t][i], here = true;
        if (here) p.target[n] = l;
      }
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      // all -inf (or no row): exp2(-inf) = 0 for each, a NaN stays one
      const float at = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
      for (int a = 0; a < MT; a++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (off(a) + i < rows) s += __builtin_amdgcn_exp2f((acc[a][t][i] - at) * kLog2e);
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (g == 0) red[wm * BN + (int)(n - n0)] = make_float2(m, s);
    }
    // twice: a row of waves may be one barrier behind
    load_wait_lds();
    bare_barrier();
    bare_barrier();
    for (int c = threadIdx.x; c < BN; c += 64 * kXWaves) {
      float2 r = red[c];
      for (int w = 1; w < WM; w++) r = stats_join(r, red[w * BN + c]);
      if (n0 + c < p.n) ((float2*)p.out)[(n0 + c) * p.mt + mtile] = r;
    }
  } else if constexpr (MODE == X_DLOGIT || MODE == X_DLOGIT32) {
    const float scale = p.scale != nullptr ? p.scale[0] : 1.f;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int64_t n = col_of(t);
      if (MODE == X_DLOGIT32 && n >= p.n) continue;
      const DRow row = drow(t);
      const int label = n < p.n ? place(row.label) : -1024;
#pragma unroll
      for (int a0 = 0; a0 < MT; a0 += AH) {
        f32x4 d[AH];
#pragma unroll
        for (int a = 0; a < AH; a++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            d[a][i] = off(a0 + a) + i < rows ? row.other(acc[a0 + a][t][i]) * scale : 0.f;
        const bool hit = label >= off(a0) && label < off(a0) + 16 * AH;
        if (__ballot(hit) != 0) {
#pragma unroll
          for (int a = 0; a < AH; a++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (off(a0 + a) + i == label) d[a][i] = row.entry;
        }
        if constexpr (MODE == X_DLOGIT32) {
#pragma unroll
          for (int a = 0; a < AH; a++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (off(a0 + a) + i < rows) ((float*)p.out)[(m0 + first + off(a0 + a) + i) * 8 + n] = d[a][i];
        } else {
          constexpr int64_t pitch = kBlock * kValue<DT>;
          const int64_t at = (m0 / kBlock * p.n + col0(t)) * pitch + (mrow + off(a0)) * kValue<DT>;
          store_rows<DT, AH>((unsigned char*)p.out + at, pitch, d, lane, p.n - col0(t), 16 * AH);
        }
      }
    }
  } else {
    const float scale = MODE == X_OUT && DT == DT_F16 && p.scale != nullptr ? p.scale[1] : 1.f;
    constexpr int ODT = MODE == X_PART ? DT_F32 : DT;
    const int64_t pitch = p.m * kValue<ODT>;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      unsigned char* row = (unsigned char*)p.out + ((int64_t)split * p.n + col0(t)) * pitch + (m0 + mrow) * kValue<ODT>;
#pragma unroll
      for (int a0 = 0; a0 < MT; a0 += AH) {
        f32x4 x[AH];
#pragma unroll
        for (int a = 0; a < AH; a++) {
          x[a] = acc[a0 + a][t];
          if constexpr (DT == DT_F16 && MODE == X_OUT) x[a] *= scale;
        }
        if (p.add) {  // the number of rows is a multiple of 4
#pragma unroll
          for (int a = 0; a < AH; a++)
            if (col_of(t) < p.n && off(a0 + a) < rows)
              x[a] += load4<ODT>(row + (lane & 15) * pitch + (off(a0 + a) + 4 * g) * kValue<ODT>);
        }
        store_rows<ODT, AH>(row + off(a0) * kValue<ODT>, pitch, x, lane, p.n - col0(t),
                             (int)min(p.m - m0, (int64_t)256) - mrow - off(a0));
      }
    }
  }
}

// Tiles and K slices.  Workgroups {x, x + 8, ...} run on XCD x: each XCD takes a contiguous
// share of the tiles, in blocks of kGroup tiles along n by all along m: its 32 CUs work on about
// kGroup x 32 / kGroup tiles, which share their operands' slices in its L2 (4,096 x 32,768 x
// 5,120 D: 1,004 us, tile rows in turn 1,080).
struct XentPlace {
  int mtile, ntile, split;
  bool some;
  // the i-th tile of an XCD's share
  __device__ __forceinline__ XentPlace(const XentProduct& p, int xcd, int i) {
    const int each = p.mt * p.nt, all = each * p.splits, per = (all + 7) / 8;
    int tile = xcd * per + i;
    some = i < per && tile < all;
    split = __builtin_amdgcn_readfirstlane(tile / each);
    tile -= split * each;
    const int block = __builtin_amdgcn_readfirstlane(tile / (kGroup * p.mt));
    tile -= block * kGroup * p.mt;
    const int wide = max(1, min(kGroup, p.nt - block * kGroup));
    mtile = __builtin_amdgcn_readfirstlane(tile / wide);
    ntile = block * kGroup + tile - mtile * wide;
  }
};

// Tiles of BM x BN, K through a ring of RING LDS images, RING - 1 stages ahead: one barrier
// per stage.  For few residual rows, where reading the table is the bound: 64 x 262,144 x 5,376
// statistics 465 us (6.1 TB/s; a kernel that only reads reaches 6.9), dx from D 459 us.
template <int DT, bool TA, bool TB, int MODE, int BM, int BN, int WM, int RING>
__global__ void __launch_bounds__(64 * kXWaves) ring_kernel(XentProduct p) {
  using A = Operand<DT, TA, BM>;
  using B = Operand<DT, TB, BN, MODE == X_PART || MODE == X_OUT>;
  constexpr int WN = kXWaves / WM, MT = BM / WM / 16, NT = BN / WN / 16, IMG = A::BYTES + B::BYTES;
  static_assert(RING * IMG <= (int)kMaxLds, "LDS");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const XentPlace at(p, (int)blockIdx.x % 8, (int)blockIdx.x / 8);
  if (!at.some) return;  // whole workgroup
  const int64_t m0 = (int64_t)at.mtile * BM, n0 = (int64_t)at.ntile * BN, k0 = (int64_t)at.split * p.kslice;
  const int kn = (int)min((int64_t)p.kslice, p.k - k0), stages = (kn + A::KS - 1) / A::KS;
  A oa(p.a, p.a_pitch, m0, p.m, k0, kn, wv, lane);
  B ob(p.b, p.b_pitch, n0, p.n, k0, kn, wv, lane);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  auto copy = [&](int s) {  // stage after stage; past the last one: zeros that nothing reads
    const uint32_t to = lds + (uint32_t)(s % RING) * IMG;
#pragma unroll
    for (int j = 0; j < A::COPIES; j++) oa.copy(j, wv, to);
#pragma unroll
    for (int j = 0; j < B::COPIES; j++) ob.copy(j, wv, to + A::BYTES);
    oa.advance();
    ob.advance();
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; a++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < RING - 1; s++) copy(s);
  // the end's few values now, beside the first copies
  DRow drow[NT];
  if constexpr (MODE == X_STATS || MODE == X_DLOGIT || MODE == X_DLOGIT32) {
#pragma unroll
    for (int t = 0; t < NT; t++) drow[t].template load<MODE>(p, min(n0 + wn * (BN / WN) + 16 * t + (lane & 15), p.n - 1));
    here<MODE>(drow);
  }
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
                                           [&](int t) { return drow[t]; }, smem);
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
//
// One workgroup per CU takes tile after tile: the copies run two stages ahead, into the next
// tile, whose first stages thus arrive while this one's end is computed and stored.  A tile
// has an even number of stages (zeros behind an odd one), so that each begins alike.
//
// 4,096 x 32,768 x 5,120 bf16, a launch each, on two cards: D 1,004 to 1,066 us (1.3 PF/s), dx 1,102 to
// 1,181, dE 1,070 to 1,154; the library's plain products take 964, 1,410 and 1,184.  What bounds it are
// the matrix cores at the clock that their load leaves (1.8 GHz): they are busy 72, 62 and 67% of the
// time, LDS is read in 23 to 27% of it, without bank conflicts.  At 14 stages the end of a tile weighs
// most: 2,048 x 151,936 x 896 keeps them busy 37% in D, 54% in dx.
template <int DT, bool TA, bool TB, int MODE>
__global__ void __launch_bounds__(64 * kXWaves, 2) tile_kernel(XentProduct p) {
  using A = Operand<DT, TA, 256>;
  using B = Operand<DT, TB, 256, MODE == X_PART || MODE == X_OUT>;
  constexpr int IMG = A::BYTES + B::BYTES;
  // what finish stores in a whole tile, for each wave
  constexpr int STORES = MODE == X_STATS || MODE == X_DLOGIT ? 0 : DT == DT_F32 || MODE == X_PART ? 32 : 16;
  // A's two images, B's two (64 KiB either: a lane's address and immediate offsets), then what finish needs
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / 4, wn = wv % 4;
  const int xcd = (int)blockIdx.x % 8, step = (int)gridDim.x / 8;
  int i = (int)blockIdx.x / 8;
  XentPlace at(p, xcd, i);
  if (!at.some) return;  // whole workgroup
  auto stages_of = [&](const XentPlace& t) {
    const int kn = (int)min((int64_t)p.kslice, p.k - (int64_t)t.split * p.kslice);
    return (kn + 2 * A::KS - 1) / (2 * A::KS) * 2;
  };
  // of the tile that is copied from; past the last tile: no rows, so zeros that nothing reads
  auto side_a = [&](const XentPlace& t) {
    const int64_t k0 = (int64_t)t.split * p.kslice, m0 = t.some ? (int64_t)t.mtile * 256 : 0;
    return A(p.a, p.a_pitch, m0, t.some ? p.m : 0, t.some ? k0 : 0, (int)min((int64_t)p.kslice, p.k - k0), wv, lane);
  };
  auto side_b = [&](const XentPlace& t) {
    const int64_t k0 = (int64_t)t.split * p.kslice, n0 = t.some ? (int64_t)t.ntile * 256 : 0;
    return B(p.b, p.b_pitch, n0, t.some ? p.n : 0, t.some ? k0 : 0, (int)min((int64_t)p.kslice, p.k - k0), wv, lane);
  };
  A oa = side_a(at);
  B ob = side_b(at);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  // half h of the stage, to image img
  auto copy_a = [&](int img, int h) {
    oa.copy(2 * h, wv, lds + (uint32_t)img * A::BYTES);
    oa.copy(2 * h + 1, wv, lds + (uint32_t)img * A::BYTES);
  };
  auto copy_b = [&](int img, int h) {
    ob.copy(2 * h, wv, lds + 2 * A::BYTES + (uint32_t)img * B::BYTES);
    ob.copy(2 * h + 1, wv, lds + 2 * A::BYTES + (uint32_t)img * B::BYTES);
  };
  f32x4 acc[8][4];
  u32x4 fa[4][2], fb[2][2][2];
  const LaneAt<A, TA, 4> la(lds, 64 * wm, lane);
  const LaneAt<B, TB, 2> lb(lds + 2 * A::BYTES, 32 * wn, lane);
  auto read_a = [&](int img, int h) {
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++) fa[a][kk] = la.read(a, kk, img * A::BYTES + 16384 * h);
  };
  auto read_b = [&](int img, int h) {
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++) fb[h][t][kk] = lb.read(t, kk, img * B::BYTES + 16384 * h);
  };
  // behind: the six steps after a tile's end, in which its stores are newer than the copies that
  // are waited for
  auto products = [&](int ha, int hb, bool behind) {
    // the fragments are read; the half that the next step reads has landed
    if (STORES > 0 && behind) load_wait<12 + STORES>();
    else load_wait<12>();
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
    if constexpr (DT == DT_F32) {  // keeps the accumulators where they are: moved about, some spill
#pragma unroll
      for (int a = 0; a < 4; a++)
#pragma unroll
        for (int t = 0; t < 2; t++) asm volatile("" : "+v"(acc[4 * ha + a][2 * hb + t]));
    }
    __builtin_amdgcn_sched_barrier(0);
    bare_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // The stage in image F, half F of B first (its fragments are there).
  auto stage = [&](auto first, bool behind) {
    constexpr int F = decltype(first)::value, L = 1 - F;
    copy_b(F, F);
    read_a(F, 0);
    products(0, F, behind);
    copy_a(F, 0);
    read_b(F, L);
    products(0, L, behind);
    copy_b(F, L);
    read_a(F, 1);
    products(1, L, behind && F == 0);
    copy_a(F, 1);
    read_b(L, L);
    oa.advance();
    ob.advance();
    products(1, F, behind && F == 0);
  };
  copy_b(0, 0), copy_a(0, 0), copy_b(0, 1), copy_a(0, 1);
  oa.advance();
  ob.advance();
  copy_b(1, 1), copy_a(1, 0), copy_b(1, 0), copy_a(1, 1);
  oa.advance();
  ob.advance();
  load_wait<12>();
  bare_barrier();
  read_b(0, 0);
  load_wait<12>();
  bare_barrier();  // the first step refills what was read here
  if (wm == 1) bare_barrier();
  bool behind = false;
  for (;;) {
    const int stages = stages_of(at);
    const XentPlace next(p, xcd, i + step);
#pragma unroll
    for (int a = 0; a < 8; a++)
#pragma unroll
      for (int t = 0; t < 4; t++) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < stages; s += 2) {
      if (s + 2 == stages) {  // the copies, two stages ahead, go on to the next tile
        oa = side_a(next);
        ob = side_b(next);
      }
      stage(std::integral_constant<int, 0>{}, behind && s == 0);
      stage(std::integral_constant<int, 1>{}, behind && s == 0);
    }
    if (wm == 0) bare_barrier();  // both rows of waves at once, or the ends would follow each other
    const int64_t m0 = (int64_t)at.mtile * 256, n0 = (int64_t)at.ntile * 256;
    // opaque copies: what the end needs of the arguments, and derives from the lane, is not kept
    // through the K loop
    int xl = lane;
    asm volatile("" : "+v"(xl));
    const auto* args = (const __attribute__((address_space(4))) XentProduct*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    const XentProduct q = *(const XentProduct*)args;
    // a column tile's as it is its turn: four at once would spill into the K loop
    auto drow = [&](int t) {
      DRow r[1];
      if constexpr (MODE == X_STATS || MODE == X_DLOGIT) {
        r[0].template load<MODE>(q, min(n0 + 32 * wn + t / 2 * 128 + t % 2 * 16 + (xl & 15), q.n - 1));
        here<MODE>(r);  // a load that some path leaves unread would be waited for there
      }
      return r[0];
    };
    finish<DT, MODE, 8, 4, 4, 2, 2, 256>(q, acc, m0, n0, 64 * wm, 32 * wn, at.mtile, at.split, wm, xl, drow,
                                         smem + 2 * IMG);
    // every store of a whole tile was issued
    behind = STORES > 0 && m0 + 256 <= p.m && n0 + 256 <= p.n && !p.add;
    if (!next.some) break;
    at = next;
    i += step;
    if (wm == 1) bare_barrier();  // one behind again
  }
  load_wait<0>();  // nothing of this workgroup is in flight when its LDS is given away
}

// dE = D^T x for up to 128 residual rows (f32: 64), bound by its stores: a workgroup keeps 256
// columns of x as fragments in registers (64 for each of 4 waves, twice) and walks a range of
// table rows, 128 at a time (64 for each half of the waves), D's tiles RING - 1 steps ahead in
// a ring of LDS images: 64 x 262,144 x 5,376 bf16 646 us (4.4 TB/s), 128 rows 836; tiles as the
// other products have them keep too few stores in flight.  A tile that holds a label has the rest of its entry of D added,
// as a second operand built in registers.
template <int DT, int KT>
constexpr int kOuterRing = DT == DT_F32 ? 4 : KT == 1 ? 7 : 5;  // as deep as the count of a wait and LDS allow

template <int DT, int KT>  // KT: stages of K
__global__ void __launch_bounds__(64 * kXWaves, 2) outer_kernel(XentProduct p) {
  using A = Operand<DT, true, 256>;
  using B = Operand<DT, true, 128, true>;
  constexpr int RING = kOuterRing<DT, KT>, IMG = KT * B::BYTES, COPIES = KT * B::COPIES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // first A's images, then [RING][IMG]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 3, wn = wv >> 2;
  const XentPlace at(p, (int)blockIdx.x % 8, (int)blockIdx.x / 8);  // ntile: a range of kslice table rows (a multiple of 128)
  if (!at.some) return;   // whole workgroup
  const int64_t m0 = (int64_t)at.mtile * 256, n0 = (int64_t)at.ntile * p.kslice, n1 = min(n0 + p.kslice, p.n);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  u32x4 fa[KT][4][2];
  {
    A oa(p.a, p.a_pitch, m0, p.m, 0, (int)p.k, wv, lane);
#pragma unroll
    for (int s = 0; s < KT; s++) {
#pragma unroll
      for (int j = 0; j < A::COPIES; j++) oa.copy(j, wv, lds + s * A::BYTES);
      oa.advance();
    }
    load_wait<0>();
    bare_barrier();
#pragma unroll
    for (int s = 0; s < KT; s++)
#pragma unroll
      for (int a = 0; a < 4; a++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) fa[s][a][kk] = A::read(smem + s * A::BYTES, 64 * wm + 16 * a, kk, lane);
    load_wait<0>();
    bare_barrier();  // the images are free
  }
  // this lane's residual rows' labels (no token: none) and what D lacks there
  uint32_t token[KT];
  float rest[KT];
#pragma unroll
  for (int s = 0; s < KT; s++) {
    const int b = 64 * s + lane;
    const bool some = DT != DT_F32 && b < p.k;
    token[s] = some ? (uint32_t)p.labels[b] : 0xffffffffu;
    rest[s] = some && token[s] < (uint64_t)p.vocab ? p.rest[b] : 0.f;
    asm volatile("" : "+v"(token[s]), "+v"(rest[s]));  // here, not where a copy would be waited for
  }
  const int steps = (int)((n1 - n0 + 127) / 128);
  B ob(p.b, p.b_pitch, n0, p.n, 0, (int)p.k, wv, lane);
  auto copy = [&](int i) {  // D's tile of step i (past the last: zeros that nothing reads)
    ob.restart(p.b, n0 + (int64_t)i * 128, i < steps ? (int)p.k : 0);
#pragma unroll
    for (int s = 0; s < KT; s++) {
#pragma unroll
      for (int j = 0; j < B::COPIES; j++) ob.copy(j, wv, lds + (uint32_t)(i % RING) * IMG + s * B::BYTES);
      ob.advance();
    }
  };
  // Copies and stores complete in order: behind a step's copies are those of the RING - 2 steps
  // after it and the stores of RING - 1 steps, whose number is known where none is left out.
  constexpr int STORES = DT == DT_F32 ? 16 : 8;
  const bool whole = m0 + 256 <= p.m && !p.add;
  for (int i = 0; i < RING - 1; i++) copy(i);
  for (int i = 0; i < steps; i++) {
    if (whole && i >= RING - 1) load_wait<(RING - 2) * COPIES + (RING - 1) * STORES>();
    else load_wait<(RING - 2) * COPIES>();
    bare_barrier();
    copy(i + RING - 1);
    const unsigned char* img = smem + i % RING * IMG;
    const int64_t first = n0 + (int64_t)i * 128;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      f32x4 acc[4][2];
#pragma unroll
      for (int a = 0; a < 4; a++)
#pragma unroll
        for (int t = 0; t < 2; t++) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KT; s++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
          u32x4 fb[2];
#pragma unroll
          for (int t = 0; t < 2; t++) fb[t] = B::read(img + s * B::BYTES, 64 * wn + 32 * h + 16 * t, kk, lane);
#pragma unroll
          for (int a = 0; a < 4; a++)
#pragma unroll
            for (int t = 0; t < 2; t++) acc[a][t] = mma<DT>(fa[s][a][kk], fb[t], acc[a][t]);
        }
      if constexpr (DT != DT_F32) {
        const uint32_t token0 = (uint32_t)(p.v0 + first);
        bool hit = false;
#pragma unroll
        for (int s = 0; s < KT; s++) hit |= token[s] - token0 < 128u;
        if (__ballot(hit) != 0) {  // few tiles
#pragma unroll
          for (int s = 0; s < KT; s++)
#pragma unroll
            for (int kk = 0; kk < 2; kk++) {
              uint32_t w[2][4] = {};
#pragma unroll
              for (int j = 0; j < 8; j++) {
                const int from = 32 * kk + 8 * (lane >> 4) + j;
                const uint32_t column = __shfl(token[s], from, 64) - token0 - (64 * wn + 32 * h);
                const uint32_t value = __builtin_bit_cast(uint16_t, round1<DT>(__shfl(rest[s], from, 64)));
#pragma unroll
                for (int t = 0; t < 2; t++)
                  if (column == 16u * t + (lane & 15)) w[t][j / 2] |= value << 16 * (j % 2);
              }
#pragma unroll
              for (int t = 0; t < 2; t++)
#pragma unroll
                for (int a = 0; a < 4; a++)
                  acc[a][t] = mma<DT>(fa[s][a][kk], u32x4{w[t][0], w[t][1], w[t][2], w[t][3]}, acc[a][t]);
            }
        }
      }
      finish<DT, X_OUT, 4, 2, 4, 2, 1, 128>(p, acc, m0, first, 64 * wm, 64 * wn + 32 * h, 0, 0, 0, lane,
                                            [](int) { return DRow(); }, smem);
    }
  }
  load_wait<0>();  // nothing of this workgroup is in flight when its LDS is given away
}

// Few table rows for few residual rows, bound by latency: a workgroup per 16 x 16 logits, its
// four waves a quarter of K each, straight from memory.
template <int DT, int MODE>
__global__ void __launch_bounds__(256) direct_kernel(XentProduct p) {
  constexpr int U = 4;
  __shared__ float sums[4][16][17];  // [wave][residual row][table row]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x % p.mt) * 16, n0 = (int64_t)(blockIdx.x / p.mt) * 16;
  const int bytes = (int)p.k * kValue<DT>, steps = (bytes + 63) / 64;
  const int c0 = steps * wv / 4, c1 = steps * (wv + 1) / 4;
  const uint8_t* ar = p.a + min(m0 + (lane & 15), p.m - 1) * p.a_pitch;
  const uint8_t* br = p.b + min(n0 + (lane & 15), p.n - 1) * p.b_pitch;
  f32x4 part[U];  // short sums: logits near their log-partition lose little
#pragma unroll
  for (int u = 0; u < U; u++) part[u] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; c += U) {
    u32x4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int at = 64 * (c + u) + 16 * g;
      const bool in = c + u < c1 && at < bytes;  // rows are whole 16-byte pieces
      a[u] = in ? *(const u32x4*)(ar + at) : u32x4{0, 0, 0, 0};
      b[u] = in ? *(const u32x4*)(br + at) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; u++) part[u] = mma<DT>(a[u], b[u], part[u]);
  }
  const f32x4 acc = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
  for (int i = 0; i < 4; i++) sums[wv][lane & 15][4 * g + i] = acc[i];
  __syncthreads();
  // thread: residual row threadIdx / 16, table row threadIdx % 16
  const int r = threadIdx.x & 15, c = threadIdx.x >> 4;
  const float l = (sums[0][c][r] + sums[1][c][r]) + (sums[2][c][r] + sums[3][c][r]);
  const int64_t v = m0 + r, n = n0 + c;
  if constexpr (MODE == X_STATS) {
    const bool some = v < p.m;
    float m = some ? l : -__builtin_inff();
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    const float at = m == -__builtin_inff() ? 0.f : m;
    float s = some ? __builtin_amdgcn_exp2f((l - at) * kLog2e) : 0.f;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) s += __shfl_xor(s, o, 64);
    if (n >= p.n) return;
    if (some && v == (int64_t)(uint32_t)p.labels[n] - p.v0) p.target[n] = l;
    if (r == 0) ((float2*)p.out)[n * p.mt + blockIdx.x % p.mt] = make_float2(m, s);
  } else {
    // past the last residual row: the last again
    const int64_t nc = min(n, p.n - 1);
    DRow row;
    row.load<MODE>(p, nc);
    float x = row.other(l);
    const bool hit = row.label >= m0 && row.label < min(m0 + 16, p.m);
    if (__ballot(hit) != 0) {  // a row's 16 threads sum its label's logit
      const uint8_t* at = p.a + (hit ? row.label : (int64_t)0) * p.a_pitch;
      const uint8_t* xr = p.b + nc * p.b_pitch;
      double sum = 0.;
      for (int o = 16 * r; o < bytes; o += 256) sum = dot64<DT>(*(const u32x4*)(xr + o), *(const u32x4*)(at + o), sum);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor(sum, o, 64);
      if (v == row.label) x = label_entry({p.labels, p.vocab, p.grad_loss, p.grad_lse, p.grad_loss_all}, nc, sum, row.lse);
    }
    if (n >= p.n || (MODE == X_DLOGIT32 && v >= p.m)) return;
    if constexpr (MODE == X_DLOGIT32) {
      ((float*)p.out)[v * 8 + n] = x;
    } else {
      const float scaled = v < p.m ? x * (p.scale != nullptr ? p.scale[0] : 1.f) : 0.f;
      const auto d = round1<DT>(scaled);
      ((decltype(round1<DT>(x))*)p.out)[(v / kBlock * p.n + n) * kBlock + v % kBlock] = d;
      if (DT != DT_F32 && v == row.label) p.rest[n] = scaled - (float)d;
    }
  }
}

// Up to 8 residual rows: both gradients in one pass over the table, with vector FMAs and D in
// f32.  A wave takes 64 pieces of 16 bytes of some consecutive table rows: their share of
// dx stays in its registers, their rows of dE are written as they come: 1 x 4,096 x 256 f32 15.8 us
// with the launches before and after.
struct XentRows {
  const uint8_t *table, *x;
  int64_t row_bytes, x_pitch, m, per;  // per: table rows of a wave
  int hidden, n, chunks, slices;
  const float* d;                      // [m][8]
  uint8_t* rows;                       // dE of the first table row, or NULL
  int32_t add;
  RowGrads grads;
  float* part;                         // [slices][n][hidden], or NULL
};

template <int DT, int NB>
__global__ void __launch_bounds__(256) xent_rows_kernel(XentRows p) {
  constexpr int E = 16 / kValue<DT>, U = 8;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = (int)blockIdx.x * 4 + wv, chunk = w % p.chunks, slice = w / p.chunks;
  if (slice >= p.slices) return;  // whole wave
  const int c = (chunk * 64 + lane) * E;
  const bool live = c < p.hidden;
  const int64_t at = (int64_t)(live ? c : 0) * kValue<DT>;
  const int64_t begin = slice * p.per, end = min(begin + p.per, p.m);
  float x[NB][E], acc[NB][E];
#pragma unroll
  for (int b = 0; b < NB; b++) {
    // past the last row: the last again, as zeros
    const int64_t row = min(b, p.n - 1);
    const uint32_t keep = b < p.n && !p.grads.none(row) ? ~0u : 0u;
    u32x4 w = *(const u32x4*)(p.x + row * p.x_pitch + at);
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] &= keep;
    unpack<DT>(w, x[b]);
#pragma unroll
    for (int i = 0; i < E; i++) acc[b][i] = 0.f;
  }
  // U table rows, their values of D (lane 8 u + b: residual row b; zeros where there is none) and
  // what their gradients are added to, one batch ahead; past the last row: the last again
  struct Batch {
    u32x4 row[U], old[U];
    float d;
  };
  const bool read = p.part != nullptr, add = p.rows != nullptr && p.add;
  auto load = [&](int64_t v, Batch& t) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t r = min(v + u, end - 1) * p.row_bytes + at;
      if (read) t.row[u] = *(const u32x4*)(p.table + r);
      if (add) t.old[u] = *(const u32x4*)(p.rows + r);
    }
    t.d = (lane & 7) < p.n ? p.d[min(v + (lane >> 3), end - 1) * 8 + (lane & 7)] : 0.f;
  };
  Batch ahead = {};
  load(begin, ahead);
  for (int64_t v = begin; v < end; v += U) {
    Batch t = ahead;
#pragma unroll
    for (int u = 0; u < U; u++) asm volatile("" : "+v"(t.row[u]), "+v"(t.old[u]));  // all of them here
    if (v + U < end) load(v + U, ahead);
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (v + u >= end) break;
      float d[NB];
#pragma unroll
      for (int b = 0; b < NB; b++) d[b] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(t.d), 8 * u + b));
      if (read) {
        float e[E];
        unpack<DT>(t.row[u], e);
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
          for (int i = 0; i < E; i++) acc[b][i] = fmaf(d[b], e[i], acc[b][i]);
      }
      if (p.rows != nullptr) {
        float o[E];
        if (add) unpack<DT>(t.old[u], o);
#pragma unroll
        for (int i = 0; i < E; i++) {
          float sum = d[0] * x[0][i];
#pragma unroll
          for (int b = 1; b < NB; b++) sum = fmaf(d[b], x[b][i], sum);
          o[i] = add ? o[i] + sum : sum;
        }
        u32x4 out;
#pragma unroll
        for (int q = 0; q < E / 4; q++) {
          const f32x4 four = {o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]};
          if constexpr (DT == DT_F32) {
            out = __builtin_bit_cast(u32x4, four);
          } else {
            const uint2 two = __builtin_bit_cast(uint2, round4<DT>(four));
            out[2 * q] = two.x, out[2 * q + 1] = two.y;
          }
        }
        if (live) *(u32x4*)(p.rows + (v + u) * p.row_bytes + at) = out;
      }
    }
  }
  if (p.part == nullptr || !live) return;
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (b >= p.n) break;
    float* to = p.part + ((int64_t)slice * p.n + b) * p.hidden + c;
#pragma unroll
    for (int q = 0; q < E / 4; q++)
      ((f32x4*)to)[q] = f32x4{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
  }
}

// D's entries at the labels, in 64 bits up to the distance of a label's logit to lse, times scale[0]
// (NULL: 1), and their rests: one wave per residual row, bound by the latency of its loads (64 x
// 262,144 x 5,376 bf16 5 us, 4,096 rows of 5,120 13).
template <int DT>
__global__ void __launch_bounds__(256) xent_label_kernel(const uint8_t* __restrict__ x, int64_t x_pitch,
                                                         const uint8_t* __restrict__ table, int64_t row_bytes,
                                                         int64_t n, RowGrads grads, const float* __restrict__ lse,
                                                         const float* __restrict__ scale, float* __restrict__ entry,
                                                         float* __restrict__ rest) {
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (b >= n) return;  // whole wave
  const uint32_t token = (uint32_t)grads.labels[b];
  if (token >= (uint64_t)grads.vocab) return;  // no entry
  const double sum = wave_dot64<DT>(x + b * x_pitch, table + (int64_t)token * row_bytes, row_bytes, lane);
  if (lane != 0) return;
  const float d = label_entry(grads, b, sum, lse[b]) * (scale != nullptr ? scale[0] : 1.f);
  entry[b] = d;
  if (DT != DT_F32 && rest != nullptr) rest[b] = d - (float)round1<DT>(d);
}

// Joins a piece's statistics [n][mt] into run [n]; the last piece writes lse and loss.  Two waves
// per residual row: one joins, beside it the other sums the label's logit (one after the other took 5 us
// more at 64 x 262,144 x 5,376).
//
// The statistics hold the label's logit as the product left it, off by c.  With that logit in 64
// bits, exp(lse) grows by p (exp(c) - 1) of itself, and the loss is the distance to the logit that
// the gradients take: where p is near 1, neither error is left in lse - logit.
template <int DT>
__global__ void __launch_bounds__(256) xent_join_kernel(const float2* __restrict__ part, int mt, int64_t n, bool first,
                                                        bool last, float2* __restrict__ run,
                                                        const float* __restrict__ target,
                                                        const int32_t* __restrict__ labels, int64_t vocab,
                                                        const uint8_t* __restrict__ x, int64_t x_pitch,
                                                        const uint8_t* __restrict__ table, int64_t row_bytes,
                                                        float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ double logits[2];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t b = (int64_t)blockIdx.x * 2 + (wv >> 1);
  const uint32_t token = b < n ? (uint32_t)labels[b] : 0xffffffffu;
  const bool has = token < (uint64_t)vocab;
  float2 r = make_float2(-__builtin_inff(), 0.f);
  if (wv & 1) {
    if (last && has) {
      const double sum = wave_dot64<DT>(x + b * x_pitch, table + (int64_t)token * row_bytes, row_bytes, lane);
      if (lane == 0) logits[wv >> 1] = sum;
    }
  } else if (b < n) {
    for (int i = lane; i < mt; i += 64) r = stats_join(r, part[b * mt + i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
      r = stats_join(r, make_float2(__shfl_xor(r.x, o, 64), __shfl_xor(r.y, o, 64)));
  }
  __syncthreads();
  if ((wv & 1) != 0 || b >= n || lane != 0) return;
  if (!first) r = stats_join(run[b], r);
  if (!last) {
    run[b] = r;
    return;
  }
  // ln s in 64 bits: one rounding of the sum of both terms
  const double s = log((double)r.y);
  double more = 0., at = has ? (double)target[b] : 0.;
  if (has && __builtin_isfinite(target[b])) {  // (an infinite or NaN logit stays what it is)
    const double logit = logits[wv >> 1];
    const float p = expf((float)(at - (double)r.x - s));
    more = log1pf(fmaxf(p * expm1f((float)(logit - at)), -0.99999994f));
    at = logit;
  }
  lse[b] = (float)((double)r.x + s + more);
  const double l = (double)r.x - at + s + more;
  loss[b] = !has || l < 0. ? 0.f : (float)l;  // (p rounds to 1: the terms cancel to 2^-24 of c; a NaN stays)
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

// dx row b = type(scale * (sum of the slices' partial sums + rest[b] * the label's table row)).
// SG slices at a time, joined in LDS.
template <int DT, int SG>
__global__ void __launch_bounds__(256) xent_sum_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                       int64_t hidden, void* __restrict__ out,
                                                       int64_t out_pitch, const float* __restrict__ scale,
                                                       const float* __restrict__ rest,
                                                       const int32_t* __restrict__ labels, int64_t vocab,
                                                       const uint8_t* __restrict__ table) {
  __shared__ f32x4 sums[SG][256 / SG];
  const int64_t each = hidden / 4, q = (int64_t)blockIdx.x * (256 / SG) + threadIdx.x % (256 / SG);
  const int sg = threadIdx.x / (256 / SG);
  const bool live = q < n * each;
  const int64_t b = live ? q / each : 0, c = live ? q % each * 4 : 0;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (live) {
#pragma unroll 4
    for (int s = sg; s < splits; s += SG) x += *(const f32x4*)(part + ((int64_t)s * n + b) * hidden + c);
  }
  if constexpr (SG > 1) {
    sums[sg][threadIdx.x % (256 / SG)] = x;
    __syncthreads();
    if (sg != 0) return;
#pragma unroll
    for (int i = 1; i < SG; i++) x += sums[i][threadIdx.x];
  }
  if (!live) return;
  if (rest != nullptr && (uint32_t)labels[b] < (uint64_t)vocab)
    x += rest[b] * load4<DT>(table + ((int64_t)labels[b] * hidden + c) * kValue<DT>);
  x *= scale != nullptr ? scale[1] : 1.f;
  // rows at any address of the type
  typedef decltype(round4<DT>(x)) V;
  typedef V Vu __attribute__((aligned(kValue<DT>)));
  *(Vu*)((unsigned char*)out + b * out_pitch + c * kValue<DT>) = round4<DT>(x);
}

// Rows of `bytes` (a multiple of 16) bytes, pitch bytes apart at any alignment, side by side; for
// the gradients, zeros in the place of those that nothing reaches.
__global__ void __launch_bounds__(256) xent_pack_kernel(const uint8_t* __restrict__ src, int64_t pitch, int64_t n,
                                                        int64_t bytes, uint8_t* __restrict__ dst, RowGrads grads) {
  typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x, each = bytes / 16, b = q / each;
  if (b >= n) return;
  const uint32_t keep = grads.labels != nullptr && grads.none(b) ? 0u : ~0u;
  u32x4 w = *(const u32x4u*)(src + b * pitch + q % each * 16);
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] &= keep;
  *(u32x4*)(dst + q * 16) = w;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
namespace {

constexpr int kXcdCount = 8;

// Columns of a product's tiles for n residual rows, and what the product then takes: rounds of
// one workgroup per CU, times its columns and stages.  16-bit products of 256 columns keep
// the matrix cores busier than those of 128 (1,024 x 262,144 x 5,120: 1,994 us, by 128 columns
// 2,893); in f32, where they are slow enough for either, the choice is about rounds alone (300
// x 20,000 x 600 gradients: 296 us, 425 by 256 columns throughout).
struct Tiling {
  int columns;
  int64_t cost;
};
Tiling tiling(int64_t m, int64_t n, int64_t k, int64_t splits, int size) {
  Tiling best = {0, INT64_MAX};
  for (int c = n <= 64 || size == 4 ? 64 : 128; c <= 256; c *= 2) {
    const int64_t percent = size == 4 ? 100 : c == 256 ? 100 : 140;  // time of a column
    // and a start and an end (5 to 6 stages' time: statistics of 2,048 x 131,072 take 441, 784 and
    // 1,421 us at 14, 28 and 56 stages), and in dx the partial sums that one more K slice leaves: with 24
    // dx of 1,500 x 5,000 x 640 bf16 takes 54 us, with 6 59; most choices are the same
    const int64_t stages = cdiv(cdiv(k, splits), 128 / size) + (size == 4 ? 6 : 24);
    const int64_t cost = cdiv(cdiv(m, 256) * cdiv(n, c) * splits, kTargetBlocks) * c * percent * stages;
    if (cost < best.cost) best = {c, cost};
    if (c >= n) break;
  }
  return best;
}

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
  const size_t lds = 2 * 512 * 128 + (MODE == X_STATS ? 2 * 256 * 8 : 0);
  hipError_t e = set_dynamic_lds(fn, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = (int64_t)p.mt * p.nt * p.splits;
  hipLaunchKernelGGL((tile_kernel<DT, TA, TB, MODE>),
                     dim3((unsigned)std::min<int64_t>(cdiv(tiles, kXcdCount) * kXcdCount, kTargetBlocks)),
                     dim3(64 * kXWaves), lds, stream, p);
  return hipGetLastError();
}

// A product with at most two stages of K.
template <int DT>
hipError_t launch_outer(XentProduct p, hipStream_t stream) {
  const bool two = p.k > 128 / kValue<DT>;
  const void* fn = two ? (const void*)outer_kernel<DT, 2> : (const void*)outer_kernel<DT, 1>;
  const size_t lds = two ? kOuterRing<DT, 2> * 32768 : kOuterRing<DT, 1> * 16384;
  hipError_t e = set_dynamic_lds(fn, lds);
  if (e != hipSuccess) return e;
  // one workgroup per CU
  p.mt = (int32_t)cdiv(p.m, 256);
  const int64_t ranges = std::max<int64_t>(1, kTargetBlocks / p.mt);
  p.kslice = (int32_t)align_up(cdiv(p.n, ranges), 128);
  p.nt = (int32_t)cdiv(p.n, p.kslice);
  const dim3 grid((unsigned)(cdiv((int64_t)p.mt * p.nt, kXcdCount) * kXcdCount));
  if (two) hipLaunchKernelGGL((outer_kernel<DT, 2>), grid, dim3(64 * kXWaves), lds, stream, p);
  else hipLaunchKernelGGL((outer_kernel<DT, 1>), grid, dim3(64 * kXWaves), lds, stream, p);
  return hipGetLastError();
}

// A product whose columns are p.n residual rows.
template <int DT, bool TA, int MODE>
hipError_t launch_by_rows(XentProduct p, hipStream_t stream) {
  const int bn = tiling(p.m, p.n, p.k, p.splits, kValue<DT>).columns;
  p.mt = (int32_t)cdiv(p.m, 256), p.nt = (int32_t)cdiv(p.n, bn);
  if (bn == 64) return launch_ring<DT, TA, false, MODE, 256, 64, 4, 4>(p, stream);
  if constexpr (MODE != X_DLOGIT32) {
    if (bn == 128) return launch_ring<DT, TA, false, MODE, 256, 128, 4, 3>(p, stream);
    return launch_tile<DT, TA, false, MODE>(p, stream);
  }
  return hipErrorInvalidValue;  // X_DLOGIT32: up to 8 rows
}

constexpr int64_t kMaxTiles = 1 << 20;              // of one launch
constexpr int64_t kPartBytes = (int64_t)256 << 20;  // statistics, or D, of one piece

// The 16 x 16 kernel instead of tiles of 256 table rows.  Loss by it / by the tiles: 4 x 4,096 x 256 f32
// 10.3 / 27.0 us, 16 x 32,768 x 256 27.0 / 28.9, 1 x 16,384 x 1,024 bf16 17.4 / 20.1, 64 x 4,096 x 1,024 17.0 /
// 20.0, 16 x 16,384 x 1,024 21.2 / 21.0, and past the border 16 x 32,768 x 1,024 32.6 / 22.2.
bool direct_tiles(int64_t vocab, int64_t n, int dtype) {
  return n <= 64 && cdiv(vocab, 16) * cdiv(n, 16) <= (dtype == DT_F32 ? 4096 : 1024);
}

template <int DT, int MODE>
hipError_t launch_direct(XentProduct p, hipStream_t stream) {
  // D's last block is written whole
  p.mt = (int32_t)(MODE == X_DLOGIT ? cdiv(p.m, kBlock) * (kBlock / 16) : cdiv(p.m, 16));
  p.nt = (int32_t)cdiv(p.n, 16);
  hipLaunchKernelGGL((direct_kernel<DT, MODE>), dim3((unsigned)(p.mt * p.nt)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

// Pieces of at most `most` tiles of 256 table rows, as even as they get; in rows.
int64_t even_piece(int64_t vocab, int64_t most) {
  const int64_t tiles = cdiv(vocab, 256);
  return cdiv(tiles, cdiv(tiles, std::max<int64_t>(1, most))) * 256;
}
// Forward: the piece's statistics stay within kPartBytes.
int64_t forward_piece(int64_t vocab, int64_t n) {
  return even_piece(vocab, std::min(kMaxTiles / cdiv(n, 64), kPartBytes / (n * 8)));
}

struct ForwardWs {
  int64_t piece;
  int32_t mt;        // statistics per residual row of a whole piece
  bool direct;
  size_t target, x, part, bytes;
};
ForwardWs forward_ws(const TableDesc& t, int64_t n) {
  ForwardWs w;
  w.direct = direct_tiles(t.V, n, t.dtype);
  w.piece = forward_piece(t.V, n);
  w.mt = (int32_t)(w.direct ? cdiv(t.V, 16) : w.piece / 256);
  w.target = align_up((size_t)n * 8, 256);  // after the running statistics
  w.x = w.target + align_up((size_t)n * 4, 256);
  w.part = w.x + align_up((size_t)(n * t.row_bytes), 256);
  w.bytes = w.part + align_up((size_t)(n * w.mt * 8), 256);
  return w;
}

// Few residual rows and a small table: D in f32 and one kernel of vector FMAs for both
// gradients, three launches where the products take five.  In a graph of calls, by it / by
// products: 1 x 4,096 x 256 f32 15.8 / 40.5 us, 8 x 4,096 x 256 19.8 / 41.2, 1 x 32,768 x 256 38 / 51,
// 3 x 3,000 x 136 bf16 17.6 / 23.1, 1 x 16,384 x 1,024 34 / 38; from there on they are even (4 x 32,768 x
// 1,024 56.4 / 55.8, f32 8 x 32,768 x 256 52.9 / 51.8).  dx alone costs it more than the products take
// in 16 bits (2 x 32,768 x 1,024 44 / 34), the table's gradient alone less (37 / 40); one rule serves
// all, so that a gradient is the same alone.  A large table takes longer that way: its reads and writes
// alternate (1 x 262,144 x 5,376: 1,668 / 1,554).
constexpr int64_t kVectorBytes = (int64_t)128 << 20;
bool vector_rows(const TableDesc& t, int64_t n) { return n <= 8 && n * t.V * t.row_bytes <= kVectorBytes; }

struct BackwardWs {
  int64_t piece, splits, slice;
  int chunks;
  int64_t block;  // bytes of a block of D
  size_t rest, entry, x, d, sums, bytes;
};
// K slices of dx = D E, at least 256 table rows each.
int64_t backward_splits(int64_t piece, int64_t n, int64_t hidden, int size) {
  int64_t best = 1, least = INT64_MAX;
  for (int64_t s = 1; s <= std::max<int64_t>(1, piece / 256) && s <= kTargetBlocks; s++) {
    const int64_t cost = tiling(hidden, n, piece, s, size).cost;
    if (cost < least) least = cost, best = s;
    if (cdiv(hidden, 256) * cdiv(n, 256) * s >= 8 * kTargetBlocks) break;
  }
  return best;
}
BackwardWs backward_ws(const TableDesc& t, int64_t n) {
  const int size = t.dtype == DT_F32 ? 4 : 2;
  BackwardWs w = {};
  size_t d_bytes;
  if (vector_rows(t, n)) {
    // about eight waves per CU, each with 16 table rows at least
    w.chunks = (int)cdiv(t.row_bytes, 1024);
    w.piece = t.V;
    w.slice = std::max<int64_t>(16, cdiv(w.piece, std::max<int64_t>(1, 8 * kTargetBlocks / w.chunks)));
    w.splits = cdiv(w.piece, w.slice);
    d_bytes = (size_t)w.piece * 32;
  } else {
    // D of a piece stays within kPartBytes, and a piece's K values within 2^28
    w.piece = even_piece(t.V, std::min(std::min(kMaxTiles / cdiv(n, 64), (int64_t)1 << 20),
                                       kPartBytes / (n * size * 256)));
    w.slice = (int64_t)align_up(cdiv(w.piece, backward_splits(w.piece, n, t.hidden, size)), kBlock);
    w.splits = cdiv(std::min(w.piece, t.V), w.slice);  // of the first piece, the fullest
    w.block = n * kBlock * size;
    d_bytes = (size_t)(n * w.piece * size);
  }
  w.rest = 256;  // after the two factors
  w.entry = w.rest + align_up((size_t)n * 4, 256);
  w.x = w.entry + align_up((size_t)n * 4, 256);
  w.d = w.x + align_up((size_t)(n * t.row_bytes), 256);
  w.sums = w.d + align_up(d_bytes, 256);
  w.bytes = w.sums + align_up((size_t)(w.splits * n * t.hidden * 4), 256);
  return w;
}

// The residual rows as the kernels read them: 16-byte aligned, rows less than 8 MiB apart.
bool rows_direct(const void* x, int64_t pitch) { return ((uintptr_t)x | (uint64_t)pitch) % 16 == 0 && pitch < (8 << 20); }

hipError_t pack_rows(const XentCall& c, const TableDesc& t, uint8_t* to, const RowGrads& grads, hipStream_t stream) {
  const int64_t pieces = c.n * (t.row_bytes / 16);
  hipLaunchKernelGGL(xent_pack_kernel, dim3((unsigned)cdiv(pieces, 256)), dim3(256), 0, stream, (const uint8_t*)c.x,
                     c.x_pitch, c.n, t.row_bytes, to, grads);
  return hipGetLastError();
}

template <int DT>
hipError_t forward(const TableDesc& t, const XentCall& c, uint8_t* ws, hipStream_t stream) {
  if (c.n == 0) return hipSuccess;
  const ForwardWs w = forward_ws(t, c.n);
  hipError_t e;
  float2 *run = (float2*)ws, *part = (float2*)(ws + w.part);
  float* target = (float*)(ws + w.target);
  const bool direct = rows_direct(c.x, c.x_pitch);
  if (!direct && (e = pack_rows(c, t, ws + w.x, {}, stream)) != hipSuccess) return e;
  const int64_t piece = w.direct ? t.V : w.piece;
  for (int64_t v0 = 0; v0 < t.V; v0 += piece) {
    XentProduct p = {};
    p.m = std::min(piece, t.V - v0), p.n = c.n, p.k = t.hidden;
    p.a = t.rows + v0 * t.row_bytes, p.a_pitch = t.row_bytes;
    p.b = direct ? (const uint8_t*)c.x : ws + w.x, p.b_pitch = direct ? c.x_pitch : t.row_bytes;
    p.splits = 1, p.kslice = (int32_t)t.hidden;
    p.out = part, p.labels = c.labels, p.v0 = v0, p.target = target;
    e = w.direct ? launch_direct<DT, X_STATS>(p, stream) : launch_by_rows<DT, false, X_STATS>(p, stream);
    if (e != hipSuccess) return e;
    const int mt = (int)(w.direct ? w.mt : cdiv(p.m, 256));
    hipLaunchKernelGGL(xent_join_kernel<DT>, dim3((unsigned)cdiv(c.n, 2)), dim3(256), 0, stream, part, mt, c.n,
                       v0 == 0, v0 + piece >= t.V, run, target, c.labels, t.V, p.b, p.b_pitch, t.rows, t.row_bytes,
                       c.loss, c.lse_out);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int NB>
hipError_t launch_rows(const XentRows& p, hipStream_t stream) {
  hipLaunchKernelGGL((xent_rows_kernel<DT, NB>), dim3((unsigned)cdiv((int64_t)p.chunks * p.slices, 4)), dim3(256), 0,
                     stream, p);
  return hipGetLastError();
}

template <int DT>
hipError_t sum_slices(const TableDesc& t, const XentCall& c, const BackwardWs& w, const float* sums,
                      const float* scale, const float* rest, hipStream_t stream) {
  const int64_t quads = c.n * (t.hidden / 4);
  // few values of many slices: 16 threads to a value's slices
  const auto kernel = w.splits >= 16 ? xent_sum_kernel<DT, 16> : xent_sum_kernel<DT, 1>;
  const int each = w.splits >= 16 ? 16 : 256;
  hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(quads, each)), dim3(256), 0, stream, sums, (int)w.splits, c.n,
                     t.hidden, c.d_x, c.d_x_pitch, scale, rest, c.labels, t.V, t.rows);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_labels(const TableDesc& t, const XentProduct& logits, const RowGrads& grads, float* entry,
                         hipStream_t stream) {
  hipLaunchKernelGGL(xent_label_kernel<DT>, dim3((unsigned)cdiv(logits.n, 4)), dim3(256), 0, stream, logits.b,
                     logits.b_pitch, t.rows, t.row_bytes, logits.n, grads, logits.lse, logits.scale, entry, logits.rest);
  return hipGetLastError();
}

template <int DT>
hipError_t backward(const TableDesc& t, const XentCall& c, uint8_t* ws, hipStream_t stream) {
  if (c.n == 0)  // a sum of nothing
    return c.d_rows == nullptr || c.add ? hipSuccess : launch_zeros(c.d_rows, t.V * t.row_bytes, stream);
  const BackwardWs w = backward_ws(t, c.n);
  hipError_t e;
  uint8_t *packed = ws + w.x, *d = ws + w.d;
  float *sums = (float*)(ws + w.sums), *entry = (float*)(ws + w.entry);
  const RowGrads grads = {c.labels, t.V, c.grad_loss, c.grad_lse, c.grad_loss_all};
  // the products of dE take a copy without the rows that nothing reaches
  const bool direct = rows_direct(c.x, c.x_pitch) && (vector_rows(t, c.n) || c.d_rows == nullptr);
  if (!direct && (e = pack_rows(c, t, packed, grads, stream)) != hipSuccess) return e;
  XentProduct logits = {};  // of a piece, to D
  logits.n = c.n, logits.k = t.hidden, logits.a_pitch = t.row_bytes;
  logits.b = direct ? (const uint8_t*)c.x : packed, logits.b_pitch = direct ? c.x_pitch : t.row_bytes;
  logits.splits = 1, logits.kslice = (int32_t)t.hidden;
  logits.out = d;
  logits.labels = c.labels, logits.vocab = t.V, logits.lse = c.lse, logits.grad_loss = c.grad_loss;
  logits.grad_loss_all = c.grad_loss_all, logits.grad_lse = c.grad_lse;
  if (vector_rows(t, c.n)) {
    XentRows p = {};
    logits.a = p.table = t.rows, logits.m = p.m = t.V;
    p.x = logits.b, p.row_bytes = t.row_bytes, p.x_pitch = logits.b_pitch, p.per = w.slice;
    p.hidden = (int)t.hidden, p.n = (int)c.n, p.chunks = w.chunks, p.slices = (int)w.splits;
    p.d = (const float*)d, p.rows = (uint8_t*)c.d_rows, p.add = c.add, p.grads = grads, p.part = c.d_x != nullptr ? sums : nullptr;
    const bool small = direct_tiles(t.V, c.n, DT);
    logits.entry = entry;
    if (!small && (e = launch_labels<DT>(t, logits, grads, entry, stream)) != hipSuccess) return e;
    e = small ? launch_direct<DT, X_DLOGIT32>(logits, stream)
                                   : launch_by_rows<DT, false, X_DLOGIT32>(logits, stream);
    if (e != hipSuccess) return e;
    e = c.n <= 2   ? launch_rows<DT, 2>(p, stream)
        : c.n <= 4 ? launch_rows<DT, 4>(p, stream)
                   : launch_rows<DT, 8>(p, stream);
    if (e != hipSuccess) return e;
    if (c.d_x == nullptr) return hipSuccess;
    return sum_slices<DT>(t, c, w, sums, nullptr, nullptr, stream);
  }
  float* scale = DT == DT_F16 ? (float*)ws : nullptr;
  float* rest = DT != DT_F32 ? (float*)(ws + w.rest) : nullptr;
  if (scale != nullptr) {
    hipLaunchKernelGGL(xent_scale_kernel, dim3(1), dim3(1024), 0, stream, c.labels, c.n, t.V, c.grad_loss,
                       c.grad_loss_all, c.grad_lse, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  logits.scale = scale, logits.rest = rest;
  const bool small = direct_tiles(t.V, c.n, DT);  // (one piece then)
  if (!small) {
    logits.entry = entry;
    if ((e = launch_labels<DT>(t, logits, grads, entry, stream)) != hipSuccess) return e;
  }
  for (int64_t v0 = 0; v0 < t.V; v0 += w.piece) {
    const int64_t rows = std::min(w.piece, t.V - v0);
    logits.a = t.rows + v0 * t.row_bytes, logits.m = rows, logits.v0 = v0;
    e = small ? launch_direct<DT, X_DLOGIT>(logits, stream) : launch_by_rows<DT, false, X_DLOGIT>(logits, stream);
    if (e != hipSuccess) return e;
    if (c.d_x != nullptr) {
      XentProduct p = {};
      p.m = t.hidden, p.n = c.n, p.k = rows;
      p.a = logits.a, p.a_pitch = t.row_bytes, p.b = d, p.b_pitch = w.block;
      p.splits = (int32_t)cdiv(rows, w.slice), p.kslice = (int32_t)w.slice;
      p.out = sums, p.add = v0 != 0;
      if ((e = launch_by_rows<DT, true, X_PART>(p, stream)) != hipSuccess) return e;
    }
    if (c.d_rows != nullptr) {
      XentProduct p = {};
      p.m = t.hidden, p.n = rows, p.k = c.n;
      p.a = logits.b, p.a_pitch = logits.b_pitch, p.b = d, p.b_pitch = w.block;
      p.splits = 1, p.kslice = (int32_t)align_up((size_t)c.n, 64);
      p.out = (uint8_t*)c.d_rows + v0 * t.row_bytes, p.add = c.add, p.scale = scale;
      p.labels = c.labels, p.v0 = v0, p.vocab = t.V, p.rest = rest;
      if (c.n <= 2 * (128 / kValue<DT>)) {
        e = launch_outer<DT>(p, stream);
      } else {
        p.mt = (int32_t)cdiv(p.m, 256), p.nt = (int32_t)cdiv(p.n, 256);
        e = launch_tile<DT, true, true, X_OUT>(p, stream);
      }
      if (e != hipSuccess) return e;
    }
  }
  return c.d_x == nullptr ? hipSuccess : sum_slices<DT>(t, c, w, sums, scale, rest, stream);
}

}  // namespace

size_t xent_workspace(const TableDesc& t, int64_t n) { return n == 0 ? 0 : forward_ws(t, n).bytes; }

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
