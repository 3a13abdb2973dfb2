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

// Bytes [k, k + 16) of a code row of K < 16 bytes, zero past the row.
__device__ __forceinline__ i32x4 load_codes16(const int8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; j++)
    if (k + j < K) v[j >> 2] |= (int)((uint32_t)(uint8_t)row[k + j] << (8 * (j & 3)));
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

// K below 16, where a row has no whole 16-byte load: bound by the loads of single bytes and by
// the stores (K = 8, 262,144 w rows: 1 row 9.4 us, 256 rows 184 us).
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
  const int k = 16 * (lane >> 4);
  const i32x4 acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_codes16(wr, k, K), load_codes16(ar, k, K),
                                                          i32x4{0, 0, 0, 0}, 0, 0, 0);
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
// Operands of v_mfma_i32_16x16x64_i8: lane l of the A operand holds 16 bytes of row l % 16,
// of the B operand of column l % 16, both of K group l / 16; result register i is row
// 4 (l / 16) + i of column l % 16.  Here w rows are A rows and a rows are B columns, and a
// K step of 256 bytes is four MFMAs: MFMA i takes slot 4 g + i of the step for K group g.
//
// K slot j stands for the 16 bytes at k = min(16 j, K - 16): where K is no multiple of 16 the
// last slot overlaps the one before, and the a rows' image below holds zeros for the bytes
// that are covered twice and for slots and rows past the end.  So w rows of any length are
// read by 16-byte loads that stay inside the row.
//
// The a rows are kept as an image in fragment order, 1 KiB per (step, i, tile of 16 a rows)
// with lane l's 16 bytes at 16 l: reads of it are free of LDS bank conflicts.
//
// w rows go straight from memory to registers, in four loads per 16 rows and step: lane l of
// load q reads slot 4 (l / 16) + l % 4 of row 4 (l / 4 % 4) + q, so the four lanes of a quad
// read 64 contiguous bytes and an instruction four rows of 256.  (With lane l at row l % 16
// every lane of a quad is in another line: 77 x 50,001 x 1,001 took 40 us against 30.)  A 4 x 4
// transposition over the quad's lanes and the four loads, two DPP selects per register, then
// leaves row l % 16 and slot 4 (l / 16) + i in register set i.  Rows at odd addresses cost a
// third more than aligned ones (K = 1,001 against 1,024), as their lines are read twice.
// ---------------------------------------------------------------------------
typedef i32x4 i32x4u __attribute__((aligned(1)));
typedef u32x4 u32x4u __attribute__((aligned(1)));

// The image's 16 bytes for a row (nullptr: past the end) and slot j.
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

// Row of the tile that a lane's load q reads, and the slot of the step.
__device__ __forceinline__ int load_row(int lane, int q) { return 4 * ((lane >> 2) & 3) + q; }
__device__ __forceinline__ int load_slot(int lane) { return 4 * (lane >> 4) + (lane & 3); }

// v[i] of lane (quad, j) <- v[j] of lane (quad, i).
__device__ __forceinline__ void quad_transpose(i32x4 (&v)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    int r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {  // exchange bit 0 of the lane and of the register
      const int o = __builtin_amdgcn_mov_dpp(v[i ^ 1][e], 0xb1, 0xf, 0xf, true);  // quad_perm 1,0,3,2
      r[i] = b0 == (bool)(i & 1) ? v[i][e] : o;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {  // bit 1
      const int o = __builtin_amdgcn_mov_dpp(r[i ^ 2], 0x4e, 0xf, 0xf, true);  // quad_perm 2,3,0,1
      v[i][e] = b1 == (bool)(i & 2) ? r[i] : o;
    }
  }
}

// Four f32 values rounded to 16-bit ones.
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
template <int DT>
__device__ __forceinline__ u16x4 round4(float (&x)[4]) {
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
  return v;
}

// Stores of one 16 x 16 tile: lane l has w rows n0 .. n0 + 3 of a row m (values acc).
template <int DT>
__device__ __forceinline__ void store_tile4(void* out, int64_t out_stride, int64_t m, int64_t n0, int64_t N, i32x4 acc,
                                            float s, const float (&w4)[4]) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; i++) x[i] = (float)acc[i] * s * w4[i];
  const int64_t at = m * out_stride + n0;
  if (n0 + 4 <= N) {  // one store at any alignment
    if constexpr (DT == DT_F32) {
      const f32x4 v = {x[0], x[1], x[2], x[3]};
      __builtin_memcpy((float*)out + at, &v, 16);
    } else {
      const u16x4 v = round4<DT>(x);
      __builtin_memcpy((uint16_t*)out + at, &v, 8);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (n0 + i < N) store_out<DT>(out, at + i, x[i]);
  }
}

// ---------------------------------------------------------------------------
// Up to 16 a rows, bound by reading w once: the whole image in LDS, a persistent grid, each
// wave a contiguous run of tiles of 16 w rows.  Two steps (8 KiB a wave) are always in
// flight, in two register sets used in turn, across tiles too; a tile's scales are loaded
// with its steps.  262,144 w rows x 5,376, 1 row: 217 us, 6.5 TB/s, where a plain read stream
// reaches 6.8 (a tile at a time, without the second set: 274 us per call against 221).
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(1024) stream_i8_kernel(MatmulI8 p, int64_t ntiles, int steps) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  i32x4* img = (i32x4*)smem;  // [steps][4][64]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6, K = (int)p.k;
  const int64_t wave = (int64_t)blockIdx.x * nw + wv, waves = (int64_t)gridDim.x * nw;
  const int64_t t0 = wave * ntiles / waves, t1 = (wave + 1) * ntiles / waves;

  struct Set {
    i32x4 v[4];
    float scale;  // of w row lane % 16
  } set[2];
  // The step that is loaded next.  Every call loads (past the last tile that one again):
  // with a fixed number of loads the wait for one set leaves the other's in flight.
  int64_t lt = t0;
  int ls = 0;
  auto load = [&](Set& x) {
    const int64_t t = max(min(lt, t1 - 1), (int64_t)0) * 16;
    x.scale = p.w_scale[min(t + (lane & 15), p.n - 1) * p.w_scale_stride];
    const int off = min(256 * ls + 16 * load_slot(lane), K - 16);
#pragma unroll
    for (int q = 0; q < 4; q++)
      x.v[q] = __builtin_nontemporal_load(
          (const i32x4u*)(p.w + min(t + load_row(lane, q), p.n - 1) * p.w_stride + off));
    if (++ls == steps) ls = 0, lt++;
  };
  load(set[0]);
  load(set[1]);
  for (int i = threadIdx.x; i < steps * 256; i += blockDim.x) {
    const int m = i & 15;
    img[i] = image_slot(m < p.m ? p.a + m * p.a_stride : nullptr, 16 * (i >> 8) + 4 * ((i >> 4) & 3) + ((i >> 6) & 3), K);
  }
  __syncthreads();
  const int m = lane & 15;
  const float s = m < p.m ? p.a_scale[m * p.a_scale_stride] : 0.f;
  i32x4 acc = {0, 0, 0, 0};
  int64_t t = t0;
  int st = 0;
  auto compute = [&](Set& x) {
    quad_transpose(x.v, lane);
#pragma unroll
    for (int i = 0; i < 4; i++)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x.v[i], img[(st * 4 + i) * 64 + lane], acc, 0, 0, 0);
    if (++st < steps || t >= t1) return;
    float w4[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w4[i] = __shfl(x.scale, 4 * (lane >> 4) + i, 64);
    if (m < p.m) store_tile4<DT>(p.out, p.out_stride, m, t * 16 + 4 * (lane >> 4), p.n, acc, s, w4);
    acc = i32x4{0, 0, 0, 0};
    st = 0;
    t++;
  };
  const int64_t total = (t1 - t0) * steps;
  for (int64_t g = 0; g < total; g += 2) {  // an odd number: the last half has no tile to store
    compute(set[0]);
    load(set[0]);
    compute(set[1]);
    load(set[1]);
  }
}

// Image of all a rows for the kernels below (5 us): [pass][step][i][tile of the pass][64 lanes].
__global__ void __launch_bounds__(256) i8_image_kernel(MatmulI8 p, int nt, int steps, i32x4* __restrict__ img,
                                                       uint32_t total) {
  const uint32_t x = blockIdx.x * 256 + threadIdx.x;
  if (x >= total) return;
  const int lane = (int)(x & 63);
  const uint32_t frag = x >> 6, r = frag / (4 * nt);
  const int t = (int)(frag % nt), i = (int)(frag / nt & 3), step = (int)(r % steps);
  const int64_t m = (int64_t)(r / steps * nt + t) * 16 + (lane & 15);
  img[x] = image_slot(m < p.m ? p.a + m * p.a_stride : nullptr, 16 * step + 4 * (lane >> 4) + i, (int)p.k);
}

// 1 KiB from memory to LDS: lane l's 16 bytes at src + offset (16 l) to lds + 16 l (src and lds uniform).  In
// assembly because the compiler would wait for every such copy before any LDS read;
// load_barrier waits for the one that is due.  No register is written.
__device__ __forceinline__ void lds_copy_1k(const void* src, uint32_t offset, uint32_t lds) {
  uint32_t m0;  // the LDS base register, left as it was
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "v"(offset), "s"(src), "s"(lds)
               : "memory");
}

// What the two kernels below share: the place of a workgroup, its w rows and its part of the
// image.  Workgroup ids {x, x + 8, ...} run on XCD x: the passes of one block of w rows
// follow each other there, and find its rows in that XCD's L2.
template <int NT, int MT, int WAVES>
struct I8Block {
  static constexpr int CHUNK = NT * 4096, DMA = (CHUNK / 1024 + WAVES - 1) / WAVES;
  int lane, wv, pass, blk, K;
  int64_t n0;
  const unsigned char* src;
  const int8_t* base;   // w row n0 of the block
  uint32_t row[MT][4];  // offsets of the lane's rows from it (at most 256 rows of 2^22 bytes)
  __device__ __forceinline__ I8Block(const MatmulI8& p, const unsigned char* img, int steps, int passes) {
    lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = blockIdx.x;
    // uniform, but divided in vector registers
    const int group = __builtin_amdgcn_readfirstlane(id / 8 / passes);
    pass = id / 8 - group * passes;
    blk = id % 8 + 8 * group;
    K = (int)p.k;
    const int64_t b0 = (int64_t)blk * WAVES * MT * 16;
    n0 = b0 + wv * MT * 16;
    base = p.w + b0 * p.w_stride;
    src = img + (size_t)pass * steps * CHUNK;
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int q = 0; q < 4; q++)
        row[t][q] = (uint32_t)max(min(n0 + 16 * t + load_row(lane, q), p.n - 1) - b0, (int64_t)0) * (uint32_t)p.w_stride;
  }
  // this wave's part of the image of step c to the buffer at lds, and its d-th KiB
  __device__ __forceinline__ void copy_part(int c, uint32_t lds, int d) const {
    const int at = (wv * DMA + d) * 1024;
    if (CHUNK % (1024 * WAVES) == 0 || at < CHUNK)  // uniform
      lds_copy_1k(src + (size_t)c * CHUNK + at, (uint32_t)lane * 16, lds + at);
  }
  __device__ __forceinline__ void copy(int c, uint32_t lds) const {
#pragma unroll
    for (int d = 0; d < DMA; d++) copy_part(c, lds, d);
  }
  // w rows of step c; ONCE: no other pass reads them
  __device__ __forceinline__ uint32_t load_offset(int c) const {
    return (uint32_t)min(256 * c + 16 * load_slot(lane), K - 16);
  }
  template <bool ONCE>
  __device__ __forceinline__ i32x4 load_part(uint32_t off, int t, int q) const {
    const i32x4u* at = (const i32x4u*)(base + (row[t][q] + off));
    if constexpr (ONCE) return __builtin_nontemporal_load(at);
    return *at;
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(int c, i32x4 (&v)[MT][4]) const {
    const uint32_t off = load_offset(c);
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int q = 0; q < 4; q++) v[t][q] = load_part<ONCE>(off, t, q);
  }
  // The output passes through LDS, JT a row tiles at a time, so that a store instruction
  // writes whole lines of one or two output rows (a tile's own registers hold 16 rows of a
  // few values).  16-byte stores at any alignment.  Every scale is loaded before the first
  // store: a load after it would wait for it.
  static constexpr int ROWS = WAVES * MT * 16;  // w rows of the workgroup
  template <int DT>
  static constexpr int JT = DT == DT_F32 ? (NT < 4 ? NT : NT == 6 ? 3 : 4) : (NT < 8 ? NT : NT == 12 ? 6 : 8);
  template <int DT>
  static constexpr int PITCH = ROWS * (DT == DT_F32 ? 4 : 2) + 16;  // bytes of an LDS row
  template <int DT>
  static constexpr size_t STORE_LDS = (size_t)16 * JT<DT> * PITCH<DT>;
  template <int DT>
  __device__ __forceinline__ void store(const MatmulI8& p, const i32x4 (&acc)[MT][NT], unsigned char* smem) const {
    constexpr int ES = DT == DT_F32 ? 4 : 2, VN = 16 / ES, LPR = ROWS / VN;  // values per store, lanes per row
    static_assert(LPR <= 64 && 64 % LPR == 0, "whole rows per store instruction");
    float w4[MT][4], s[NT];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        w4[t][i] = p.w_scale[min(n0 + 16 * t + 4 * (lane >> 4) + i, p.n - 1) * p.w_scale_stride];
    const int64_t m0 = (int64_t)pass * NT * 16;
#pragma unroll
    for (int j = 0; j < NT; j++) s[j] = p.a_scale[min(m0 + 16 * j + (lane & 15), p.m - 1) * p.a_scale_stride];
    const int64_t b0 = (int64_t)blk * ROWS;
#pragma unroll
    for (int j0 = 0; j0 < NT; j0 += JT<DT>) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < JT<DT>; j++)
#pragma unroll
        for (int t = 0; t < MT; t++) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; i++) x[i] = (float)acc[t][j0 + j][i] * s[j0 + j] * w4[t][i];
          unsigned char* to = smem + (16 * j + (lane & 15)) * PITCH<DT> + ((wv * MT + t) * 16 + 4 * (lane >> 4)) * ES;
          if constexpr (DT == DT_F32) *(f32x4*)to = f32x4{x[0], x[1], x[2], x[3]};
          else *(u16x4*)to = round4<DT>(x);
        }
      __syncthreads();
      const int r0 = wv * (64 / LPR) + lane / LPR, col = lane % LPR * VN;
      for (int r = r0; r < 16 * JT<DT>; r += WAVES * (64 / LPR)) {
        const int64_t m = m0 + 16 * j0 + r, n = b0 + col;
        if (m >= p.m) break;
        const unsigned char* from = smem + r * PITCH<DT> + col * ES;
        if (n + VN <= p.n) {
          // non-temporal: 64 rows x 262,144 f32 logits 257 us, with plain stores 278
          __builtin_nontemporal_store(*(const u32x4*)from,
                                      (u32x4u*)((unsigned char*)p.out + (m * p.out_stride + n) * ES));
        } else {
          for (int i = 0; i < VN; i++)
            if (n + i < p.n) {
              if constexpr (ES == 4) ((uint32_t*)p.out)[m * p.out_stride + n + i] = ((const uint32_t*)from)[i];
              else ((uint16_t*)p.out)[m * p.out_stride + n + i] = ((const uint16_t*)from)[i];
            }
        }
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Passes of up to 16 NT a rows, bound by reading w: WAVES x MT tiles of 16 w rows per
// workgroup.  The image passes through three LDS buffers of one step each, copied by
// global_load_lds two steps ahead; the w rows are loaded up to two steps ahead into two
// register sets used in turn.  One barrier per step.  262,144 w rows x 5,376, 64 rows to f32:
// 233 us, 6.3 TB/s of w rows and outputs.  The least NT that holds the rows, as the image's
// copies and reads grow with it (K = 16,384, 48 rows 700 us, 128 rows 784); at 128 rows two
// tiles of w rows per wave share an image fragment, which halves the reads from LDS.  At 192
// rows two no longer fit the registers (spills: 683 us against 294 at 160 rows, K = 5,120).
// w is read by one pass only (non-temporal loads): two passes of 128 rows would read it twice.
// ---------------------------------------------------------------------------
template <int DT, int NT, int MT, int WAVES, int MINW>
__global__ void __launch_bounds__(64 * WAVES, MINW) wide_i8_kernel(MatmulI8 p, const unsigned char* __restrict__ img,
                                                                   int steps, int passes, int nblk) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // [3][CHUNK]
  using B = I8Block<NT, MT, WAVES>;
  const B blk(p, img, steps, passes);
  if (blk.blk >= nblk) return;  // whole workgroup
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  i32x4 set[2][MT][4], acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[t][j] = i32x4{0, 0, 0, 0};
  auto step = [&](int c, i32x4 (&v)[MT][4]) {
    // Step c's image and w rows have landed, and this wave has read the buffer that the copy
    // below refills.  Loads complete in order: the w rows of step c + 1 stay in flight.
    load_barrier<4 * MT>();
    if (c + 2 < steps) blk.copy(c + 2, lds + (c + 2) % 3 * B::CHUNK);  // uniform
    const i32x4* b = (const i32x4*)(smem + c % 3 * B::CHUNK) + blk.lane;
#pragma unroll
    for (int t = 0; t < MT; t++) quad_transpose(v[t], blk.lane);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const i32x4 f = b[(i * NT + j) * 64];
#pragma unroll
        for (int t = 0; t < MT; t++) acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[t][i], f, acc[t][j], 0, 0, 0);
      }
    blk.template load<true>(min(c + 2, steps - 1), v);  // always the same number of loads in flight
  };
  blk.copy(0, lds);
  blk.copy(1, lds + B::CHUNK);
  blk.template load<true>(0, set[0]);
  blk.template load<true>(1, set[1]);
  for (int c = 0; c < steps; c += 2) {  // an even number
    step(c, set[0]);
    step(c + 1, set[1]);
  }
  load_barrier<0>();  // the last (repeated) loads
  blk.template store<DT>(p, acc, smem);
}

// ---------------------------------------------------------------------------
// Passes of 256 a rows, bound by the matrix cores: 4 waves x 64 w rows per workgroup.  A wave
// holds 4 x 16 tiles of 16 x 16 in 256 accumulator registers (one wave per SIMD), so a 1 KiB
// fragment of the image read from LDS serves four MFMAs: 64 B a clock per CU of LDS reads at
// the full MFMA rate.  The image passes through two LDS buffers of one step, each refilled
// one step ahead.  The next step's copies and w loads are issued one at a time between the
// MFMAs of this one (32 in a row would hold up the wave, whose MFMAs wait behind them), and its
// w rows are transposed there too.  1,024 x 262,144 x 5,120 to bf16: 1,300-1,350 us, 2.0-2.1 POP/s (the
// copies in a row before the MFMAs: 1,454).  The MFMAs alone run 777 us; the L2 reads of the
// image and the w rows by 256 x 256 tiles, and the stores at the end of a tile, with one
// workgroup per CU and nothing else to run meanwhile, are the rest.  160 rows of it take 402
// us, the kernel above 294 (K = 1,001: 113 / 124; 32,000 w rows x 5,120: 68 / 62).
// ---------------------------------------------------------------------------
static constexpr int kTileWaves = 4, kTileMT = 4, kTileNT = 16;

// acc += a b, in assembly so that the accumulators stay where they are: the compiler rotates
// them through other registers, and copies and spills what no longer fits.  An accumulator is
// used again 64 MFMAs later, and read otherwise only after mfma_settle.
__device__ __forceinline__ void mfma_in_place(i32x4& acc, const i32x4& a, const i32x4& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int DT>
__global__ void __launch_bounds__(64 * kTileWaves, 1) tile_i8_kernel(MatmulI8 p, const unsigned char* __restrict__ img,
                                                                     int steps, int passes, int nblk) {
  constexpr int MT = kTileMT, NT = kTileNT, F = 4 * NT, AHEAD = 2;
  static_assert(F == 64 && MT == 4 && NT * 4 == 16 * kTileWaves, "the schedule of a step below");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // [2][CHUNK]
  using B = I8Block<NT, MT, kTileWaves>;
  const B blk(p, img, steps, passes);
  if (blk.blk >= nblk) return;  // whole workgroup
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem;
  i32x4 set[2][MT][4], acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[t][j] = i32x4{0, 0, 0, 0};
  auto step = [&](int c, i32x4 (&v)[MT][4], i32x4 (&next)[MT][4]) {
    // Step c's image has landed and every wave has read step c - 1's buffer, which the copy
    // below refills.
    load_barrier<0>();
    const int ahead = min(c + 1, steps - 1);  // the last step's own again: not read
    const uint32_t off = blk.load_offset(ahead), to = lds + (c + 1) % 2 * B::CHUNK;
    const i32x4* b = (const i32x4*)(smem + c % 2 * B::CHUNK) + blk.lane;
    i32x4 f[AHEAD + 1];  // fragments read ahead of their MFMAs
#pragma unroll
    for (int x = 0; x < AHEAD; x++) f[x] = b[x * 64];
#pragma unroll
    for (int x = 0; x < F; x++) {
      if (x + AHEAD < F) f[(x + AHEAD) % (AHEAD + 1)] = b[(x + AHEAD) * 64];
#pragma unroll
      for (int t = 0; t < MT; t++) mfma_in_place(acc[t][x % NT], v[t][x / NT], f[x % (AHEAD + 1)]);
      if (x < 32 && x % 2 == 0) blk.copy_part(ahead, to, x / 2);
      if (x < 32 && x % 2 == 1) next[x / 8][x / 2 % 4] = blk.template load_part<false>(off, x / 8, x / 2 % 4);
      if (x >= 44 && x % 4 == 0 && (x - 44) / 4 < MT) quad_transpose(next[(x - 44) / 4], blk.lane);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  blk.copy(0, lds);
  blk.template load<false>(0, set[0]);
#pragma unroll
  for (int t = 0; t < MT; t++) quad_transpose(set[0][t], blk.lane);
  mfma_settle();
  for (int c = 0; c < steps; c += 2) {  // an even number
    step(c, set[0], set[1]);
    step(c + 1, set[1], set[0]);
  }
  load_barrier<0>();  // the last (repeated) loads
  mfma_settle();
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < NT; j++) asm volatile("" : "+a"(acc[t][j]));  // read after the wait
  blk.template store<DT>(p, acc, smem);
}

// ---------------------------------------------------------------------------
// Small products, bound by latency: a workgroup per 16 T x 16 T tile of the output, its
// four waves a quarter of K each (their integer sums add up in LDS in any order to the same
// value).  Both operands come straight from memory, two or four K steps of 64 bytes in flight.
// 256 x 1,024 x 5,120: 13 us (by passes of 256 rows 69: 4 workgroups).  Four waves: sixteen
// took 17.6 us against 13.3 there, as their sums meet in LDS, and won at K = 16,384 (31 / 35).
// ---------------------------------------------------------------------------
static constexpr int kSplitWaves = 4;

template <int DT, int T>
__global__ void __launch_bounds__(64 * kSplitWaves) split_i8_kernel(MatmulI8 p) {
  constexpr int E = 16 * T, U = T == 4 ? 2 : 4;
  __shared__ int sums[E][E + 1];  // [a row][w row]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), K = (int)p.k;
  const int64_t n0 = (int64_t)blockIdx.x * E, m0 = (int64_t)blockIdx.y * E;
  const int steps = (K + 63) / 64;
  const int c0 = steps * wv / kSplitWaves, c1 = steps * (wv + 1) / kSplitWaves;
  const int8_t *wr[T], *ar[T];
#pragma unroll
  for (int t = 0; t < T; t++) {
    wr[t] = p.w + min(n0 + 16 * t + (lane & 15), p.n - 1) * p.w_stride;
    ar[t] = p.a + min(m0 + 16 * t + (lane & 15), p.m - 1) * p.a_stride;
  }
  for (int i = threadIdx.x; i < E * (E + 1); i += 64 * kSplitWaves) ((int*)sums)[i] = 0;
  i32x4 acc[T][T];
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int j = 0; j < T; j++) acc[t][j] = i32x4{0, 0, 0, 0};
  for (int c = c0; c < c1; c += U) {
    i32x4 w[U][T], a[U][T];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int off = min(64 * min(c + u, c1 - 1) + 16 * (lane >> 4), K - 16);
#pragma unroll
      for (int t = 0; t < T; t++) {
        w[u][t] = *(const i32x4u*)(wr[t] + off);
        a[u][t] = *(const i32x4u*)(ar[t] + off);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (c + u >= c1) break;  // uniform
      if (64 * (c + u) + 64 > K) {  // the row's end: bytes of the slot before and past the row count nothing
        const int j = 4 * (c + u) + (lane >> 4);
#pragma unroll
        for (int t = 0; t < T; t++) a[u][t] = image_slot(ar[t], j, K);
      }
#pragma unroll
      for (int t = 0; t < T; t++)
#pragma unroll
        for (int j = 0; j < T; j++)
          acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][t], a[u][j], acc[t][j], 0, 0, 0);
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int j = 0; j < T; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) atomicAdd(&sums[16 * j + (lane & 15)][16 * t + 4 * (lane >> 4) + i], acc[t][j][i]);
  __syncthreads();
  for (int i = threadIdx.x; i < E * E; i += 64 * kSplitWaves) {
    const int64_t m = m0 + i / E, n = n0 + i % E;
    if (m < p.m && n < p.n)
      store_out<DT>(p.out, m * p.out_stride + n,
                    (float)sums[i / E][i % E] * p.a_scale[m * p.a_scale_stride] * p.w_scale[n * p.w_scale_stride]);
  }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
enum { I8_SIMPLE, I8_SPLIT, I8_STREAM, I8_WIDE, I8_TILE };
struct I8Plan {
  int kind, nt, steps;  // steps of 256 (wide, tile: an even number)
  int64_t passes;
  size_t img_bytes;
};

static I8Plan i8_plan(int64_t m, int64_t n, int64_t k) {
  I8Plan p = {};
  p.steps = (int)cdiv(k, 256);
  if (k < 16) {
    p.kind = I8_SIMPLE;
  } else if (cdiv(n, 64) * cdiv(m, 64) <= (m <= 16 ? 128 : 512)) {
    // Few tiles of 64 x 64.  Measured, split against the others (us): 512 tiles m = 128,
    // n = 16,384, k = 5,120 45.9 / 52.4, k = 256 10.9 / 13.5; 1,024 tiles m = 256, k = 5,120
    // 85 / 71.  m = 16: 64 tiles, k = 1,024 4.5 / 6.2, 256 tiles 7.9 / 6.6.  Around the border
    // both are two to four times the bytes' time (128 x 16,384 x 5,120 13 us): split tiles read
    // their operands once per tile, and the others have a workgroup per 256 w rows, too few.
    p.kind = I8_SPLIT;
  } else if (m <= 16 && (size_t)p.steps * 4096 <= kMaxLds) {
    p.kind = I8_STREAM;
  } else {
    p.kind = m <= 192 ? I8_WIDE : I8_TILE;
    p.nt = m <= 32 ? 2 : m <= 64 ? 4 : m <= 96 ? 6 : m <= 128 ? 8 : m <= 192 ? 12 : kTileNT;
    p.steps = (p.steps + 1) / 2 * 2;
    p.passes = cdiv(m, 16 * p.nt);
    p.img_bytes = (size_t)p.passes * p.nt * p.steps * 4096;
  }
  return p;
}

size_t matmul_i8_workspace(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0) return 0;
  return i8_plan(m, n, k).img_bytes;
}

// blocks of rows_per_block w rows, all passes of each on one XCD
template <typename K>
static hipError_t launch_blocks(K kernel, int threads, size_t lds, int rows_per_block, const MatmulI8& p,
                                const I8Plan& pl, const void* img, hipStream_t stream) {
  hipError_t e = set_dynamic_lds((const void*)kernel, lds);
  if (e != hipSuccess) return e;
  const int64_t nblk = cdiv(p.n, rows_per_block);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(align_up((size_t)nblk, 8) * pl.passes)), dim3(threads), lds, stream, p,
                     (const unsigned char*)img, pl.steps, (int)pl.passes, (int)nblk);
  return hipGetLastError();
}

template <int DT, int NT, int MT, int WAVES, int MINW>
static hipError_t launch_wide_i8(const MatmulI8& p, const I8Plan& pl, const void* img, hipStream_t stream) {
  using B = I8Block<NT, MT, WAVES>;
  return launch_blocks(wide_i8_kernel<DT, NT, MT, WAVES, MINW>, 64 * WAVES,
                       std::max((size_t)3 * B::CHUNK, B::template STORE_LDS<DT>), B::ROWS, p, pl, img, stream);
}

template <int DT>
static hipError_t launch_matmul_dt(const MatmulI8& p, void* ws, hipStream_t stream) {
  const I8Plan pl = i8_plan(p.m, p.n, p.k);
  if (pl.kind == I8_SIMPLE) {
    hipLaunchKernelGGL((matmul_i8_kernel<DT>), dim3((unsigned)cdiv(p.n, 64), (unsigned)cdiv(p.m, 16)), dim3(256), 0,
                       stream, p.a, p.a_stride, p.a_scale, p.a_scale_stride, p.w, p.w_stride, p.w_scale,
                       p.w_scale_stride, p.m, p.n, (int)p.k, p.out, p.out_stride);
    return hipGetLastError();
  }
  // the block kernels' row offsets are 32-bit (256 rows and K of at most 2^16 bytes)
  const bool far = (pl.kind == I8_WIDE || pl.kind == I8_TILE) && p.w_stride > (1 << 22);
  if (pl.kind == I8_SPLIT || far) {
    // 32 x 32 where 64 x 64 would leave CUs without a workgroup
    const bool small = cdiv(p.n, 64) * cdiv(p.m, 64) < kTargetBlocks;
    const int e = small ? 32 : 64;
    hipLaunchKernelGGL((small ? split_i8_kernel<DT, 2> : split_i8_kernel<DT, 4>),
                       dim3((unsigned)cdiv(p.n, e), (unsigned)cdiv(p.m, e)), dim3(64 * kSplitWaves), 0, stream, p);
    return hipGetLastError();
  }
  if (pl.kind == I8_STREAM) {
    const size_t lds = (size_t)pl.steps * 4096;
    hipError_t e = set_dynamic_lds((const void*)stream_i8_kernel<DT>, lds);
    if (e != hipSuccess) return e;
    const int64_t ntiles = cdiv(p.n, 16);
    // one 16-wave workgroup per CU, or small ones where there are fewer tiles than waves
    const int nw = ntiles >= 16 * kTargetBlocks ? 16 : 4;
    const int64_t blocks = std::min<int64_t>(cdiv(ntiles, nw), nw == 16 ? kTargetBlocks : 4 * kTargetBlocks);
    hipLaunchKernelGGL((stream_i8_kernel<DT>), dim3((unsigned)blocks), dim3(64 * nw), lds, stream, p, ntiles, pl.steps);
    return hipGetLastError();
  }
  const uint32_t total = (uint32_t)(pl.img_bytes / 16);  // at most 65536 x 66048 bytes
  hipLaunchKernelGGL(i8_image_kernel, dim3((unsigned)cdiv(total, 256)), dim3(256), 0, stream, p, pl.nt, pl.steps,
                     (i32x4*)ws, total);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pl.kind == I8_TILE) {
    using B = I8Block<kTileNT, kTileMT, kTileWaves>;
    static_assert(B::template STORE_LDS<DT> <= 2 * B::CHUNK, "the image's buffers hold the output tile");
    return launch_blocks(tile_i8_kernel<DT>, 64 * kTileWaves, (size_t)2 * B::CHUNK, B::ROWS, p, pl, ws, stream);
  }
  if (pl.nt == 2) return launch_wide_i8<DT, 2, 1, 16, 4>(p, pl, ws, stream);
  if (pl.nt == 4) return launch_wide_i8<DT, 4, 1, 16, 4>(p, pl, ws, stream);
  if (pl.nt == 6) return launch_wide_i8<DT, 6, 1, 16, 4>(p, pl, ws, stream);
  if (pl.nt == 8) return launch_wide_i8<DT, 8, 2, 8, 2>(p, pl, ws, stream);
  return launch_wide_i8<DT, 12, 1, 16, 4>(p, pl, ws, stream);
}

hipError_t launch_matmul_i8(const MatmulI8& p, void* ws, hipStream_t stream) {
  // grids stay below 2^32 threads
  constexpr int64_t kMost = (int64_t)1 << 28;
  for (int64_t n0 = 0; n0 < p.n; n0 += kMost) {
    MatmulI8 q = p;
    q.n = std::min(kMost, p.n - n0);
    q.w += n0 * p.w_stride;
    q.w_scale += n0 * p.w_scale_stride;
    q.out = (uint8_t*)p.out + n0 * (p.out_dtype == DT_F32 ? 4 : 2);
    const hipError_t e = p.out_dtype == DT_F32    ? launch_matmul_dt<DT_F32>(q, ws, stream)
                         : p.out_dtype == DT_BF16 ? launch_matmul_dt<DT_BF16>(q, ws, stream)
                                                  : launch_matmul_dt<DT_F16>(q, ws, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace etg
