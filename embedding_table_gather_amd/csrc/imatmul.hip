// Matrix product in 8-bit integers with a scale per row of each operand (per token
// and per channel): out[m][n] = T( f32(sum_k a[m][k] w[n][k]) * sa[m] * sw[n] ).
// The sum is exact: |sum| <= 65536 * 128 * 128 = 2^30 fits the int32 accumulators.
// Its conversion to f32 and the two multiplications round to nearest (relative
// error at most 3 * 2^-24), the store in T once more.
#include <algorithm>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Bytes [k, k + 16) of a code row of K bytes at any address, zero past the row.
__device__ __forceinline__ i32x4 load_codes16(const int8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 16; j++)
      if (k + j < K) v[j >> 2] |= (int)((uint32_t)(uint8_t)row[k + j] << (8 * (j & 3)));
  }
  return v;
}

template <int DT>
__device__ __forceinline__ void store_out(void* out, int64_t i, float x) {
  if constexpr (DT == DT_F32) {
    ((float*)out)[i] = x;
  } else if constexpr (DT == DT_BF16) {
    ((__bf16*)out)[i] = (__bf16)x;
  } else {
    // opaque: the compiler would fold the last multiplication into the conversion
    // (one rounding where the definition has two)
    asm volatile("" : "+v"(x));
    ((_Float16*)out)[i] = (_Float16)x;  // past 65504: infinity, as the rounding has it
  }
}

// One wave per tile of 16 w rows x 16 a rows (v_mfma_i32_16x16x64_i8, the w rows as
// the A operand: lane l holds bytes 16 (l / 16) .. + 15 of row l % 16, and result
// register i is w row 4 (l / 16) + i of a row l % 16).  Rows past the end are read
// from the last row and not stored.
template <int DT>
__global__ void __launch_bounds__(256) matmul_i8_kernel(
    const int8_t* __restrict__ a, int64_t a_stride, const float* __restrict__ sa, int64_t sa_stride,
    const int8_t* __restrict__ w, int64_t w_stride, const float* __restrict__ sw, int64_t sw_stride, int64_t M,
    int64_t N, int K, void* __restrict__ out, int64_t out_stride) {
  const int lane = threadIdx.x & 63;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 16, m0 = (int64_t)blockIdx.y * 16;
  if (n0 >= N) return;  // whole wave, no barrier below
  const int8_t* wr = w + min(n0 + (lane & 15), N - 1) * w_stride;
  const int8_t* ar = a + min(m0 + (lane & 15), M - 1) * a_stride;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 16 * (lane >> 4); k - 16 * (lane >> 4) < K; k += 64)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_codes16(wr, k, K), load_codes16(ar, k, K), acc, 0, 0, 0);
  const int64_t m = m0 + (lane & 15);
  if (m >= M) return;
  const float s = sa[m * sa_stride];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t n = n0 + 4 * (lane >> 4) + i;
    if (n < N) store_out<DT>(out, m * out_stride + n, (float)acc[i] * s * sw[n * sw_stride]);
  }
}

// ---------------------------------------------------------------------------
// Streaming kernels: few a rows, bound by reading w once.
//
// The a rows are the B operand of v_mfma_i32_16x16x64_i8, kept as an image in the order
// in which the lanes read it: 1 KiB per K step of 64 and tile of 16 a rows, lane l's 16
// bytes at 16 l (a row 16 t + l % 16, bytes of K slot 4 step + l / 16).  K slot j stands
// for the 16 bytes at k = min(16 j, K - 16): where K is no multiple of 16 the last slot
// overlaps the one before, and the image holds zeros for the bytes that are covered
// twice and for slots and rows past the end.  So w rows of any length are read by
// 16-byte loads that stay inside the row.
// ---------------------------------------------------------------------------
// The image's 16 bytes for a row `row` (nullptr: past the end) and slot j.
__device__ __forceinline__ i32x4 image_slot(const int8_t* row, int j, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (row == nullptr || 16 * j >= K) return v;
  const int k = min(16 * j, K - 16), twice = 16 * j - k;  // bytes of the slot before
  __builtin_memcpy(&v, row + k, 16);
  if (twice != 0) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int cut = min(max(twice - 4 * i, 0), 4);
      v[i] = cut == 4 ? 0 : (int)((uint32_t)v[i] & (0xffffffffu << (8 * cut)));
    }
  }
  return v;
}

// Stores of one 16 x 16 tile: lane l has w rows n0 .. n0 + 3 of a row m (values acc).
template <int DT>
__device__ __forceinline__ void store_tile4(void* out, int64_t out_stride, int64_t m, int64_t n0, int64_t N, i32x4 acc,
                                            float s, const float (&w4)[4], bool vec) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; i++) x[i] = (float)acc[i] * s * w4[i];
  const int64_t at = m * out_stride + n0;
  if (vec && n0 + 4 <= N) {  // rows of the output start at multiples of four values
    if constexpr (DT == DT_F32) {
      *(f32x4*)((float*)out + at) = f32x4{x[0], x[1], x[2], x[3]};
    } else {
      typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
      u16x4 v;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if constexpr (DT == DT_BF16) {
          v[i] = __builtin_bit_cast(unsigned short, (__bf16)x[i]);
        } else {
          asm volatile("" : "+v"(x[i]));  // as in store_out
          v[i] = __builtin_bit_cast(unsigned short, (_Float16)x[i]);
        }
      }
      *(u16x4*)((uint16_t*)out + at) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (n0 + i < N) store_out<DT>(out, at + i, x[i]);
  }
}

typedef i32x4 i32x4u __attribute__((aligned(1)));

// Up to 8 IMG a rows: the whole image in LDS, a persistent grid, each wave a contiguous
// run of tiles of 8 w rows.
//
// One load instruction reads 8 rows x 128 bytes (full lines): lane l row l % 8, slot l / 8
// of the step.  As the A operand of the MFMA that is w row m % 8 at slots 2 g + m / 8 in A
// row m and lane group g; the image's column n holds a row n % 8 at the same slots
// 2 g + n / 8, so the sum for (w row r, a row b) is D[r][b] + D[r + 8][b + 8] and the other
// half of D is unused: the matrix cores idle anyway (16 rows: a second image).
//
// Two groups of four steps (8 KiB a wave) are always in flight, in two register sets used
// in turn, across tiles too; a tile's scales are loaded with its groups.
static constexpr int kStreamSteps = 4;  // steps of 128 bytes per group

template <int DT, int IMG>
__global__ void __launch_bounds__(1024) stream_i8_kernel(MatmulI8 p, int64_t ntiles, int steps, int vec) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  i32x4* img = (i32x4*)smem;  // [steps][IMG][64]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6, K = (int)p.k;
  const int64_t wave = (int64_t)blockIdx.x * nw + wv, waves = (int64_t)gridDim.x * nw;
  const int64_t t0 = wave * ntiles / waves, t1 = (wave + 1) * ntiles / waves;

  struct Set {
    i32x4 v[kStreamSteps];
    float scale;  // of w row lane % 8
  } set[2];
  // The group that is loaded next.  Every call loads (past the last tile that one again):
  // with a fixed number of loads the wait for one set leaves the other's in flight.
  int64_t lt = t0;
  int ls = 0;
  auto load = [&](Set& x) {
    const int64_t r = min(max(min(lt, t1 - 1), (int64_t)0) * 8 + (lane & 7), p.n - 1);
    const int8_t* row = p.w + r * p.w_stride;
    x.scale = p.w_scale[r * p.w_scale_stride];
#pragma unroll
    for (int q = 0; q < kStreamSteps; q++)
      x.v[q] = __builtin_nontemporal_load((const i32x4u*)(row + min(128 * (ls + q) + 16 * (lane >> 3), K - 16)));
    ls += kStreamSteps;
    if (ls >= steps) ls = 0, lt++;
  };
  load(set[0]);
  load(set[1]);
  for (int i = threadIdx.x; i < steps * IMG * 64; i += blockDim.x) {
    const int l = i & 63, im = IMG == 1 ? 0 : (i >> 6) & 1, st = (i >> 6) / IMG;
    const int m = 8 * im + (l & 7);
    img[i] = image_slot(m < p.m ? p.a + m * p.a_stride : nullptr, 8 * st + 2 * (l >> 4) + ((l >> 3) & 1), K);
  }
  __syncthreads();
  const int b = lane & 7;
  const bool holder = (lane & 40) == 0;  // lanes with the first half of a useful sum
  float s[IMG];
#pragma unroll
  for (int im = 0; im < IMG; im++) s[im] = 8 * im + b < p.m ? p.a_scale[(8 * im + b) * p.a_scale_stride] : 0.f;
  i32x4 acc[IMG];
#pragma unroll
  for (int im = 0; im < IMG; im++) acc[im] = i32x4{0, 0, 0, 0};
  int64_t t = t0;
  int st = 0;
  auto compute = [&](const Set& x) {
#pragma unroll
    for (int q = 0; q < kStreamSteps; q++)
#pragma unroll
      for (int im = 0; im < IMG; im++)
        acc[im] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x.v[q], img[((st + q) * IMG + im) * 64 + lane], acc[im], 0, 0, 0);
    st += kStreamSteps;
    if (st < steps || t >= t1) return;
    // holder lane l: w rows 4 (l / 16) + i of the tile, a row 8 im + l % 8
    const int64_t n = t * 8 + 4 * (lane >> 4);
    float w4[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w4[i] = __shfl(x.scale, 4 * ((lane >> 4) & 1) + i, 64);
#pragma unroll
    for (int im = 0; im < IMG; im++) {
      i32x4 sum;
#pragma unroll
      for (int i = 0; i < 4; i++) sum[i] = acc[im][i] + __shfl(acc[im][i], (lane + 40) & 63, 64);
      if (holder && 8 * im + b < p.m) store_tile4<DT>(p.out, p.out_stride, 8 * im + b, n, p.n, sum, s[im], w4, vec);
      acc[im] = i32x4{0, 0, 0, 0};
    }
    st = 0;
    t++;
  };
  const int64_t groups = (t1 - t0) * (steps / kStreamSteps);
  for (int64_t g = 0; g < groups; g += 2) {  // an odd number: the last half has no tile to store
    compute(set[0]);
    load(set[0]);
    compute(set[1]);
    load(set[1]);
  }
}

// Image of all a rows, lane l's 16 bytes being a row l % 16 of its tile:
//  wide kernel  [pass][step of 128][tile of the pass][even, odd][64 lanes], slot 8 step + 2 (l / 16) + odd
//  tile kernel  [pass][step of 128][half][tile of the pass][64 lanes], slot 8 step + 4 half + l / 16
__global__ void __launch_bounds__(256) i8_image_kernel(MatmulI8 p, int nt, int steps, int wide,
                                                       i32x4* __restrict__ img, uint32_t total) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int lane = (int)(i & 63);
  const uint32_t frag = i >> 6, r = frag / (2 * nt);
  const int f = (int)(frag % (2 * nt)), step = (int)(r % steps);
  const int t = wide ? f >> 1 : f % nt, part = wide ? f & 1 : f / nt;
  const int64_t m = (int64_t)(r / steps * nt + t) * 16 + (lane & 15);
  const int slot = 8 * step + (wide ? 2 * (lane >> 4) + part : 4 * part + (lane >> 4));
  img[i] = image_slot(m < p.m ? p.a + m * p.a_stride : nullptr, slot, (int)p.k);
}

// Passes of up to 16 NT a rows: WAVES x MT tiles of 16 w rows per workgroup.  A load reads
// 8 w rows x 128 bytes as in the stream kernel (X: rows 0 - 7 of a tile, Y: rows 8 - 15); two
// DPP moves per register swap the odd half of X with the even half of Y, which leaves the
// 16-row A operands of the even and of the odd slots.  The image
// passes through three LDS buffers of one K step each, copied by global_load_lds two
// chunks ahead; the w rows are loaded up to two chunks ahead into two register sets used in
// turn.  One barrier per chunk.
//
// Template: NT tiles of 16 a rows and MT of 16 w rows per wave, WAVES per workgroup, SETS
// register sets of w rows (the chunk multiplied and those loaded ahead), MINW waves per
// SIMD.

// 1 KiB from memory to LDS: lane l's 16 bytes at src to lds + 16 l.  In assembly because the
// compiler would wait for every such copy before any LDS read; wide_barrier waits for the one
// that is due.  No register is written.
__device__ __forceinline__ void lds_copy_1k(const void* src, uint32_t lds) {
  uint32_t m0;  // the LDS base register, left as it was
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

// vmcnt(N) lgkmcnt(0), then a workgroup barrier that no memory access crosses.
template <int N>
__device__ __forceinline__ void wide_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("s_barrier" ::: "memory");
}

template <int DT, int NT, int MT, int WAVES, int SETS, int MINW>
__global__ void __launch_bounds__(64 * WAVES, MINW) wide_i8_kernel(MatmulI8 p, const unsigned char* __restrict__ img,
                                                                   int chunks, int passes, int nblk, int vec) {
  constexpr int CHUNK = NT * 2048, DMA = (CHUNK / 1024 + WAVES - 1) / WAVES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // [3][CHUNK]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = (int)p.k;
  // Workgroup ids {x, x + 8, ...} run on XCD x: the passes of one block of w rows follow each
  // other there, and find its rows in that XCD's L2.
  const int id = blockIdx.x, pass = id / 8 % passes, blk = id % 8 + 8 * (id / 8 / passes);
  if (blk >= nblk) return;  // whole workgroup
  const int64_t n0 = ((int64_t)blk * WAVES + wv) * MT * 16;
  const unsigned char* src = img + (size_t)pass * chunks * CHUNK;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  auto copy = [&](int c) {
#pragma unroll
    for (int d = 0; d < DMA; d++) {
      const int at = (wv * DMA + d) * 1024;
      if (at < CHUNK) lds_copy_1k(src + (size_t)c * CHUNK + at + lane * 16, lds + c % 3 * CHUNK + at);  // uniform
    }
  };
  const int8_t* row[2 * MT];  // X and Y rows of each tile
#pragma unroll
  for (int t = 0; t < 2 * MT; t++) row[t] = p.w + min(n0 + 8 * t + (lane & 7), p.n - 1) * p.w_stride;
  // w rows of the chunk that is multiplied and of the next, in turn
  i32x4 set[SETS][2 * MT];
  auto load = [&](int c, i32x4 (&v)[2 * MT]) {
    const int off = min(128 * c + 16 * (lane >> 3), K - 16);
#pragma unroll
    for (int t = 0; t < 2 * MT; t++) v[t] = __builtin_nontemporal_load((const i32x4u*)(row[t] + off));
  };
  i32x4 acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[t][j] = i32x4{0, 0, 0, 0};
  auto chunk = [&](int c, i32x4 (&v)[2 * MT]) {
    // Chunk c and its w rows have landed, and this wave has read the buffer that the copy below
    // refills.  Loads complete in order: the w rows of the SETS - 1 chunks after c stay in flight,
    // all loaded after the copy of chunk c, which was started two chunks ago.
    static_assert(SETS == 2 || SETS == 3, "the wait below");
    wide_barrier<(SETS - 1) * 2 * MT>();
    if (c + 2 < chunks) copy(c + 2);  // uniform
    const i32x4* b = (const i32x4*)(smem + c % 3 * CHUNK);
    i32x4 even[MT], odd[MT];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int x = v[2 * t][e], y = v[2 * t + 1][e];
        even[t][e] = __builtin_amdgcn_update_dpp(x, y, 0x118, 0xf, 0xc, false);  // row_shr:8 into lanes 8 - 15
        odd[t][e] = __builtin_amdgcn_update_dpp(y, x, 0x108, 0xf, 0x3, false);   // row_shl:8 into lanes 0 - 7
      }
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const i32x4 f0 = b[j * 128 + lane], f1 = b[j * 128 + 64 + lane];
#pragma unroll
      for (int t = 0; t < MT; t++) acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(even[t], f0, acc[t][j], 0, 0, 0);
#pragma unroll
      for (int t = 0; t < MT; t++) acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(odd[t], f1, acc[t][j], 0, 0, 0);
    }
    load(min(c + SETS, chunks - 1), v);  // always the same number of loads in flight
  };
  copy(0);
  copy(1);
#pragma unroll
  for (int i = 0; i < SETS; i++) load(min(i, chunks - 1), set[i]);
  for (int c = 0; c < chunks; c += SETS) {  // a multiple of SETS
#pragma unroll
    for (int i = 0; i < SETS; i++) chunk(c + i, set[i]);
  }
  wide_barrier<0>();  // the last (repeated) loads
#pragma unroll
  for (int t = 0; t < MT; t++) {
    const int64_t n = n0 + 16 * t + 4 * (lane >> 4);
    float w4[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w4[i] = p.w_scale[min(n + i, p.n - 1) * p.w_scale_stride];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int64_t m = ((int64_t)pass * NT + j) * 16 + (lane & 15);
      if (m < p.m) store_tile4<DT>(p.out, p.out_stride, m, n, p.n, acc[t][j], p.a_scale[m * p.a_scale_stride], w4, vec);
    }
  }
}

// ---------------------------------------------------------------------------
// Tile kernel: many a rows, bound by the matrix cores.
//
// 8 waves x 64 w rows by 128 a rows per workgroup: a wave holds 4 x 8 tiles of 16 x 16
// (128 accumulator registers), so one 1 KiB fragment of the image read from LDS serves
// four MFMAs (64 B / clock per CU of LDS reads at the full MFMA rate), and its own w rows
// come straight from memory into the A operand (lane l: row l % 16, 16 bytes at
// 16 (l / 16) of each half step), two steps ahead.
// ---------------------------------------------------------------------------
static constexpr int kTileWaves = 8, kTileMT = 4, kTileNT = 8;

// acc += a b, in assembly so that the accumulators stay where they are: with 128 of them the
// compiler rotates them through other registers, and copies and spills what no longer fits.
// A product's accumulator is used again 32 MFMAs later, and read otherwise only after
// mfma_settle.
__device__ __forceinline__ void mfma_in_place(i32x4& acc, const i32x4& a, const i32x4& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int DT>
__global__ void __launch_bounds__(64 * kTileWaves, 2) tile_i8_kernel(MatmulI8 p, const unsigned char* __restrict__ img,
                                                                     int chunks, int passes, int nblk, int vec) {
  constexpr int MT = kTileMT, NT = kTileNT, CHUNK = NT * 2048, DMA = CHUNK / 1024 / kTileWaves, F = 2 * NT;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // [3][CHUNK]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = (int)p.k;
  // passes of one block of w rows follow each other on one XCD, as in the wide kernel
  const int id = blockIdx.x, pass = id / 8 % passes, blk = id % 8 + 8 * (id / 8 / passes);
  if (blk >= nblk) return;  // whole workgroup
  const int64_t n0 = ((int64_t)blk * kTileWaves + wv) * MT * 16;
  const unsigned char* src = img + (size_t)pass * chunks * CHUNK;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  auto copy = [&](int c) {
#pragma unroll
    for (int d = 0; d < DMA; d++) {
      const int at = (wv * DMA + d) * 1024;
      lds_copy_1k(src + (size_t)c * CHUNK + at + lane * 16, lds + c % 3 * CHUNK + at);
    }
  };
  const int8_t* row[MT];
#pragma unroll
  for (int t = 0; t < MT; t++) row[t] = p.w + min(n0 + 16 * t + (lane & 15), p.n - 1) * p.w_stride;
  i32x4 set[2][2][MT];
  auto load = [&](int c, i32x4 (&v)[2][MT]) {
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int off = min(128 * c + 64 * q + 16 * (lane >> 4), K - 16);
#pragma unroll
      for (int t = 0; t < MT; t++) v[q][t] = *(const i32x4u*)(row[t] + off);
    }
  };
  i32x4 acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[t][j] = i32x4{0, 0, 0, 0};
  auto chunk = [&](int c, i32x4 (&v)[2][MT]) {
    wide_barrier<2 * MT>();  // as in the wide kernel
    if (c + 2 < chunks) copy(c + 2);
    const i32x4* b = (const i32x4*)(smem + c % 3 * CHUNK) + lane;
    i32x4 f[3];  // fragments read two ahead of their MFMAs
    f[0] = b[0];
    f[1] = b[64];
#pragma unroll
    for (int i = 0; i < F; i++) {
      if (i + 2 < F) f[(i + 2) % 3] = b[(i + 2) * 64];
#pragma unroll
      for (int t = 0; t < MT; t++) mfma_in_place(acc[t][i % NT], v[i / NT][t], f[i % 3]);
    }
    load(min(c + 2, chunks - 1), v);
  };
  copy(0);
  copy(1);
  load(0, set[0]);
  load(1, set[1]);
  mfma_settle();
  for (int c = 0; c < chunks; c += 2) {  // an even number
    chunk(c, set[0]);
    chunk(c + 1, set[1]);
  }
  wide_barrier<0>();  // the last (repeated) loads
  mfma_settle();
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) asm volatile("" : "+a"(acc[t][j]));  // read after the wait
#pragma unroll
  for (int t = 0; t < MT; t++) {
    const int64_t n = n0 + 16 * t + 4 * (lane >> 4);
    float w4[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w4[i] = p.w_scale[min(n + i, p.n - 1) * p.w_scale_stride];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int64_t m = ((int64_t)pass * NT + j) * 16 + (lane & 15);
      if (m < p.m) store_tile4<DT>(p.out, p.out_stride, m, n, p.n, acc[t][j], p.a_scale[m * p.a_scale_stride], w4, vec);
    }
  }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
enum { I8_SIMPLE, I8_STREAM, I8_WIDE, I8_TILE };
struct I8Plan {
  int kind, nt, steps;  // wide: K steps of 128, a multiple of any number of sets
  int64_t passes;
  size_t img_bytes;
};

static I8Plan i8_plan(int64_t m, int64_t n, int64_t k) {
  I8Plan p = {};
  p.steps = (int)cdiv(k, 128 * 6) * 6;
  if (k < 16 || n > ((int64_t)1 << 30)) {
    p.kind = I8_SIMPLE;
  } else if (m <= 16 && (size_t)cdiv(k, 512) * 4 * (m <= 8 ? 1024 : 2048) <= kMaxLds) {
    p.kind = I8_STREAM;
    p.steps = (int)cdiv(k, 128 * kStreamSteps) * kStreamSteps;  // steps of 128
  } else {
    p.kind = m <= 128 ? I8_WIDE : I8_TILE;
    p.nt = m <= 32 ? 2 : m <= 64 ? 4 : 8;
    p.passes = cdiv(m, 16 * p.nt);
    p.img_bytes = (size_t)p.passes * p.nt * p.steps * 2048;
  }
  return p;
}

size_t matmul_i8_workspace(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0) return 0;
  return i8_plan(m, n, k).img_bytes;
}

template <int DT, int IMG>
static hipError_t launch_stream_i8(const MatmulI8& p, const I8Plan& pl, int vec, hipStream_t stream) {
  const size_t lds = (size_t)pl.steps * IMG * 1024;
  hipError_t e = set_dynamic_lds((const void*)stream_i8_kernel<DT, IMG>, lds);
  if (e != hipSuccess) return e;
  const int64_t ntiles = cdiv(p.n, 8);
  // one 16-wave workgroup per CU, or small ones where there are fewer tiles than waves
  const int nw = ntiles >= 16 * kTargetBlocks ? 16 : 4;
  const int64_t blocks = std::min<int64_t>(cdiv(ntiles, nw), nw == 16 ? kTargetBlocks : 4 * kTargetBlocks);
  hipLaunchKernelGGL((stream_i8_kernel<DT, IMG>), dim3((unsigned)blocks), dim3(64 * nw), lds, stream, p, ntiles, pl.steps,
                     vec);
  return hipGetLastError();
}

template <int DT, int NT, int MT, int WAVES, int SETS, int MINW>
static hipError_t launch_wide_i8(const MatmulI8& p, const I8Plan& pl, const void* img, int vec, hipStream_t stream) {
  auto kernel = wide_i8_kernel<DT, NT, MT, WAVES, SETS, MINW>;
  const size_t lds = (size_t)3 * NT * 2048;
  hipError_t e = set_dynamic_lds((const void*)kernel, lds);
  if (e != hipSuccess) return e;
  const int64_t nblk = cdiv(p.n, WAVES * MT * 16);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(align_up((size_t)nblk, 8) * pl.passes)), dim3(64 * WAVES), lds, stream, p,
                     (const unsigned char*)img, pl.steps, (int)pl.passes, (int)nblk, vec);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_matmul_dt(const MatmulI8& p, void* ws, hipStream_t stream) {
  const I8Plan pl = i8_plan(p.m, p.n, p.k);
  // four-value stores of an output whose rows all start at a multiple of four values
  const int vec = (uintptr_t)p.out % (DT == DT_F32 ? 16 : 8) == 0 && p.out_stride % 4 == 0;
  if (pl.kind == I8_SIMPLE) {
    hipLaunchKernelGGL((matmul_i8_kernel<DT>), dim3((unsigned)cdiv(p.n, 64), (unsigned)cdiv(p.m, 16)), dim3(256), 0,
                       stream, p.a, p.a_stride, p.a_scale, p.a_scale_stride, p.w, p.w_stride, p.w_scale,
                       p.w_scale_stride, p.m, p.n, (int)p.k, p.out, p.out_stride);
    return hipGetLastError();
  }
  if (pl.kind == I8_STREAM)
    return p.m <= 8 ? launch_stream_i8<DT, 1>(p, pl, vec, stream) : launch_stream_i8<DT, 2>(p, pl, vec, stream);
  const uint32_t total = (uint32_t)(pl.img_bytes / 16);  // at most 65536 x 65792 bytes
  hipLaunchKernelGGL(i8_image_kernel, dim3((unsigned)cdiv(total, 256)), dim3(256), 0, stream, p, pl.nt, pl.steps,
                     (int)(pl.kind == I8_WIDE), (i32x4*)ws, total);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pl.kind == I8_TILE) {
    const size_t lds = (size_t)3 * kTileNT * 2048;
    e = set_dynamic_lds((const void*)tile_i8_kernel<DT>, lds);
    if (e != hipSuccess) return e;
    const int64_t nblk = cdiv(p.n, kTileWaves * kTileMT * 16);
    hipLaunchKernelGGL((tile_i8_kernel<DT>), dim3((unsigned)(align_up((size_t)nblk, 8) * pl.passes)),
                       dim3(64 * kTileWaves), lds, stream, p, (const unsigned char*)ws, pl.steps, (int)pl.passes, (int)nblk,
                       vec);
    return hipGetLastError();
  }
  if (pl.nt == 2) return launch_wide_i8<DT, 2, 2, 8, 3, 4>(p, pl, ws, vec, stream);
  if (pl.nt == 4) return launch_wide_i8<DT, 4, 2, 8, 3, 4>(p, pl, ws, vec, stream);
  return launch_wide_i8<DT, 8, 2, 8, 3, 2>(p, pl, ws, vec, stream);
}

hipError_t launch_matmul_i8(const MatmulI8& p, void* ws, hipStream_t stream) {
  if (p.out_dtype == DT_F32) return launch_matmul_dt<DT_F32>(p, ws, stream);
  if (p.out_dtype == DT_BF16) return launch_matmul_dt<DT_BF16>(p, ws, stream);
  return launch_matmul_dt<DT_F16>(p, ws, stream);
}

}  // namespace etg
