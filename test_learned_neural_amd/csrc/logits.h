// The matrix products over a large vocabulary that cross entropy, token log probabilities and distillation
// are made of (gfx950), with their epilogues.  An output tile of a^T b or a b has b's index in its lanes and
// a's, four at a time, in its registers; the operands go straight to LDS, kStages steps deep.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace am {

namespace {

constexpr float kDown = 40.0f;  // KEPT: 2^-kDown on what is kept of bf16 calls, whose 16 bits end at 2
constexpr int kBK = 32;        // contraction elements of a step: two matrix instructions deep
enum { EPI_LSE, EPI_GRAD, EPI_ACC, EPI_OUT, EPI_SUMS, EPI_TOP, EPI_KEPT, EPI_AGAIN, EPI_ROWS, EPI_PART };

// 2^(k2 (a - b)) to a few units in the last place, whatever a - b: what the difference and the factor lost to
// rounding is small, but the same for a whole row.
__device__ __forceinline__ float exp2_of(float a, float b, float k2, float k2_low) {
  const float x = a - b, t = x - a, lost = (a - (x - t)) - (b + t);
  const float low = fabsf(x) < 1.0e30f ? fmaf(x, k2_low, lost * k2) : 0.0f;  // of a masked class there is none
  return __builtin_amdgcn_exp2f(fmaf(x, k2, low));
}

// Sums of squares of floats that lost nothing that counts: far from overflow, and squares below 2^-126 are small beside
// them.
__device__ __forceinline__ bool in_range(float q) { return q > 1.0e-30f && q < 1.0e36f; }
// What a row can have whose squares' sum is zero: 16384 magnitudes below 2^-63.  Rows of zeros, a vocabulary's padding, are
// not worth another look (64 x 2048 x 65536, one class in a hundred zeros: 202 us with one, 74 without).
constexpr float kVanished = 0x1p-56f;
// How far a logit's sum can be off, over c |x|: |w|, or where w has one large entry, a mask's, less.  Of w' without it the
// terms are |x| |w'| at most, and the large one's |z| + |x| |w'|: with c |z|, 2 |w'| will do, which is less where the large
// entry's square is more than 3/4 of all.  `part`: the largest of the parts that the squares' sum q was made of.
__device__ __forceinline__ bool no_large_entry(float q, float part) { return part <= 0.75f * q; }
// |row| of others, in 64 bits, by the lanes `lane` of `lanes` (2: a wave's halves, or 64), 16 bytes each; with ERRS the least
// of that and 2 |w'|, infinite entries left out: a row's logits of those classes are infinite or NaN.  Zero of zeros alone.
template <bool BF16, bool ERRS>
__device__ __forceinline__ float far_norm(const void* row, int dp, int lane, int lanes) {
  double s = 0.0;
  float m = 0.0f;
#pragma unroll 1
  for (int p = lane; p < dp / (BF16 ? 8 : 4); p += lanes) {
    const u32x4 w = ((const u32x4*)row)[p];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < (BF16 ? 2 : 1); ++h) {
        const float v = fabsf(__uint_as_float(!BF16 ? w[k] : h ? w[k] & 0xFFFF0000u : w[k] << 16));
        const float a = ERRS && !(v < INFINITY) ? 0.0f : v;
        const double x = ERRS ? fminf(a, m) : a;  // the largest so far is not in s
        m = fmaxf(a, m);
        s = fma(x, x, s);
      }
  }
#pragma unroll 1
  for (int k = 32; k >= 64 / lanes; k >>= 1) {
    const float om = __shfl_xor(m, k);
    const double x = ERRS ? fminf(m, om) : 0.0;
    s += __shfl_xor(s, k) + x * x;
    m = fmaxf(m, om);
  }
  if (ERRS) s = fmin(4.0 * s, fma((double)m, (double)m, s));
  // planes of the smallest floats lose up to 2^-134 of each: with an error from 2^-17 of the norm on, less than 2^-110 of it
  return m > 0.0f ? (float)(sqrt(s) + 0x1p-110) : 0.0f;
}

struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb;        // elements of a row
  int64_t na, nb;          // rows (or, across the contraction, columns) of a and b
  int64_t K;
  const int* count;        // rows that count (OUT, PART: K, else nb), or null: as given
  int ta, tb;              // tiles of a and b
  int splits;              // pieces of the contraction (ACC, PART; else 1)
  // epilogues
  float2* part;            // LSE: [nb][parts]: (maximum, sum of exponentials)
  int parts;
  const int64_t* labels;   // [rows of X]
  const float* lse;
  const int* index;        // GRAD: [nb], b's rows in X
  int64_t v0;
  void* g;                 // GRAD: [nb][ldg]
  void* gw;                // ... and times weight / *scale, or null; OUT: what b is then
  const int* equal;        // ... where the weights are not all one value
  int both;                // ... beside g, not in its place
  const float* weight;     // GRAD: [rows of X]
  int64_t ldg;
  float* acc;              // ACC: [splits][acc_rows][na]
  int64_t acc_rows;
  int add;
  const float* scale;      // GRAD: see gw; OUT: one factor, or null
  void* out;               // [nb][ldo]
  int64_t ldo;
  float k2, k2_low;        // SUMS, TOP, KEPT, AGAIN: scale log2 e, and what its rounding left
  float4* sums;            // SUMS, TOP: [nb][parts]: (maximum m of z, sum of e = exp(scale (z - m)), sum of e (z - m), -)
  uint4* keys;             // TOP: [nb][4 parts], by group_class's groups: how far below the maximum their four largest
                           // logits are, times k2, with the class's place in the low bits
  float* tops;             // ... [nb][2 parts]: the maxima, of 2 tile + group % 2
  float *a_norm, *b_norm;  // ... [4 parts]: the largest of a group's far_norm; [nb]: |b|
  int apart;               // SUMS, TOP: see tile_rows
  const float* ref;        // KEPT, AGAIN: [rows of X]
  const int* to;           // AGAIN: [nb], rows of g; ROWS: of out
  const int64_t* ids;      // AGAIN: [rows of X][top], the teacher's classes
  const float* prob;       // ... and their probabilities (of no class: zero)
  const float* factor;     // AGAIN: [nb], q / exp(scale (z - ref))
  int top;
  const float* row_weight; // ROWS: [rows of X]
  const int* at;           // ... whether a row counts: a place, or -1
};

// The tiles of SUMS and TOP take every `apart`-th row of a, so that classes that lie together (frequent ones do)
// come to different tiles: of `apart` tiles beside each other, or of the last ones.
struct TileRows {
  int64_t first;  // the tile's first row; the others follow `step` apart
  int step;
};
__device__ __forceinline__ TileRows tile_rows(int tile, int side, int apart, int tiles) {  // apart: a power of two
  const int t = tile & -apart;
  return {(int64_t)t * side + (tile - t), min(apart, tiles - t)};
}
__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t m;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}
// The 16, 32 or 64 of a tile's classes that one lane holds of a row are a group, four a tile: every fourth of the
// tile's rows (spread_row of where they lie in LDS), so that neighbours are in different ones.
__device__ __forceinline__ int64_t group_class(int group, int code, int side, int apart, int tiles) {
  const TileRows t = tile_rows(group >> 2, side, apart, tiles);
  return t.first + (int64_t)t.step * (4 * code + (group & 3));
}
template <int R>
__device__ __forceinline__ int spread_row(int r) {
  const int half = r / (R / 2), in = r % (R / 2);
  return 4 * (in >> 3) * 4 + 4 * (in & 3) + 2 * (in >> 2 & 1) + half;
}

// One operand's step in LDS.  Along the contraction: [R][32], the 16-byte pieces of four rows (256 bytes,
// all banks) exchanged by the four's index; across: [32][R], pairs of 32-byte pieces exchanged by those
// low bits of the contraction index that 256 bytes do not hold.  Either way the lanes that are served
// together lie on distinct banks.
// Loads go straight to LDS, 64 pieces of 16 bytes an instruction, in LDS order: the exchange is in the
// lanes' global offsets.  Those outside the matrix have the top bit, and the range check writes zeros.
//
// The load is written out because the compiler, knowing it, waits for all of them before every
// transposing read.  It has no result register: its address is read when it is issued, and what it
// writes, LDS, is waited for by wait_all alone.  m0, which the compiler takes for its own, is put back.
__device__ __forceinline__ void load_to_lds(rsrc_t rs, uint32_t voff, const void* lds) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)lds;
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
               "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(at), "v"(voff), "s"(rs)
               : "memory");
}
template <int R, bool ACROSS, int WAVES>
struct Tile {
  static constexpr int kElems = R * kBK;
  static constexpr int kLoads = R * kBK / 8 / 64 / WAVES;  // instructions of a wave
  uint32_t off[kLoads];
  int kc;  // along: the lane's first contraction element

  __device__ static constexpr int exchange(int k) { return R == 64 ? k & 2 : (k & 3) << 1; }

  // SPREAD: rows in the order of spread_row
  template <bool SPREAD = false>
  __device__ void init(int64_t ld, int64_t r0, int64_t rows, int wave, int lane) {
    kc = ((lane & 3) ^ ((lane >> 4) & 3)) * 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = (wave * kLoads + i) * 64 + lane;  // piece in LDS order
      if constexpr (ACROSS) {
        const int k = id / (R / 8), at = id % (R / 8);
        const int c = ((((at >> 1) ^ exchange(k)) << 1) | (at & 1)) * 8;
        off[i] = c < rows - r0 ? (uint32_t)((k * ld + c) * 2) : 0x80000000u;
      } else {
        const int r = SPREAD ? spread_row<R>(id >> 2) : id >> 2;
        off[i] = r < rows - r0 ? (uint32_t)((r * ld + kc) * 2) : 0x80000000u;
      }
    }
  }
  // load number i of a step.  p: the matrix at (row or column r0, contraction k); left: contraction
  // elements from k on (none: zeros); room: elements of a row from r0 on (across)
  __device__ void load(int i, uint16_t* s, const uint16_t* p, int left, int64_t ld, int64_t room, int wave) const {
    const uint16_t* d = s + (wave * kLoads + i) * 512;
    if constexpr (ACROSS) {
      const int n = left < kBK ? left : kBK;
      const rsrc_t rs = make_rsrc(p, n > 0 ? (uint32_t)(((n - 1) * ld + room) * 2) : 0u);
      load_to_lds(rs, off[i], d);
    } else {
      const rsrc_t rs = make_rsrc(p, 0x7fffffffu);
      load_to_lds(rs, off[i] | (kc < left ? 0u : 0x80000000u), d);
    }
  }
  // lane's eight contraction elements 16 ks + 8 (lane / 32) + 0..7 of row (column) r0 + lane % 32
  __device__ static u32x4 op(const uint16_t* s, int r0, int ks, int lane) {
    const int hf = lane >> 5;
    if constexpr (ACROSS) {
      const int e = (lane & 15) >> 2;
      const int k = 16 * ks + 8 * hf + e;
      const int c = (((r0 + (lane & 16)) >> 4) ^ exchange(e)) * 16 + 4 * (lane & 3);
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* lds4;
      const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + k * R + c)));
      const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + (k + 4) * R + c)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
      const int r = r0 + (lane & 31);
      return *(const u32x4*)(s + r * kBK + (((2 * ks + hf) ^ ((r >> 2) & 3)) << 3));
    }
  }
};

// The same for fp32, whose operands are read as eight floats.  Along: [R][32], the pieces of a pair of rows
// exchanged by the pair's index; across: [32][R], halves of 64 columns exchanged by the contraction index's
// eights, so that the two halves of a wave read different banks.
template <int R, bool ACROSS, int WAVES>
struct Tile32 {
  static constexpr int kElems = R * kBK;
  static constexpr int kLoads = R * kBK / 4 / 64 / WAVES;
  uint32_t off[kLoads];
  int kc[kLoads];

  template <bool SPREAD = false>
  __device__ void init(int64_t ld, int64_t r0, int64_t rows, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = (wave * kLoads + i) * 64 + lane;
      if constexpr (ACROSS) {
        const int k = id / (R / 4), c = (id % (R / 4) ^ ((k >> 3 & 1) << 3)) * 4;
        kc[i] = 0;
        off[i] = c < rows - r0 ? (uint32_t)((k * ld + c) * 4) : 0x80000000u;
      } else {
        const int at = id >> 3, r = SPREAD ? spread_row<R>(at) : at;
        kc[i] = ((id & 7) ^ ((at >> 1) & 7)) * 4;
        off[i] = r < rows - r0 ? (uint32_t)((r * ld + kc[i]) * 4) : 0x80000000u;
      }
    }
  }
  __device__ void load(int i, float* s, const float* p, int left, int64_t ld, int64_t room, int wave) const {
    const float* d = s + (wave * kLoads + i) * 256;
    if constexpr (ACROSS) {
      const int n = left < kBK ? left : kBK;
      const rsrc_t rs = make_rsrc(p, n > 0 ? (uint32_t)(((n - 1) * ld + room) * 4) : 0u);
      load_to_lds(rs, off[i], d);
    } else {
      const rsrc_t rs = make_rsrc(p, 0x7fffffffu);
      load_to_lds(rs, off[i] | (kc[i] < left ? 0u : 0x80000000u), d);
    }
  }
  __device__ static void op(const float* s, int r0, int ks, int lane, float* v) {
    const int hf = lane >> 5;
    if constexpr (ACROSS) {
      const float* p = s + (16 * ks + 8 * hf) * R + ((r0 ^ (hf << 5)) + (lane & 31));
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = p[n * R];
    } else {
      const int r = r0 + (lane & 31), c = 4 * ks + 2 * hf, x = (r >> 1) & 7;
      const float4 a = *(const float4*)(s + r * kBK + ((c ^ x) << 2));
      const float4 b = *(const float4*)(s + r * kBK + (((c | 1) ^ x) << 2));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  }
};

// Eight floats as three bf16 planes, v = p[0] + p[1] + p[2].
__device__ __forceinline__ void split_planes(float* v, u32x4* p) {
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = cvt_pk_bf16(v[2 * i], v[2 * i + 1]);
      p[n][i] = w;
      if (n < 2) {
        v[2 * i] -= __uint_as_float(w << 16);
        v[2 * i + 1] -= __uint_as_float(w & 0xFFFF0000u);
      }
    }
}

// Waits until at most N of the wave's loads are on their way and its LDS reads are done, then for the
// other waves: what was loaded before is in LDS, and what was read before may be overwritten.
template <int N>
__device__ __forceinline__ void wait_all() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Floats of [0, 2) as 16 bits without a sign, seven of exponent and nine of fraction.
__device__ __forceinline__ uint32_t pack_u16(float a, float b) {
  return (__float_as_uint(a) + 0x2000u) >> 14 | ((__float_as_uint(b) + 0x2000u) << 2 & 0xFFFF0000u);
}
__device__ __forceinline__ float u16_lo(uint32_t w) { return __uint_as_float((w & 0xFFFFu) << 14); }
__device__ __forceinline__ float u16_hi(uint32_t w) { return __uint_as_float((w & 0xFFFF0000u) >> 2); }

// A tile's accumulators, rounded to bf16, to rows r0.. (nr of them) and columns c0.. (nc) of a matrix:
// through LDS, so that a row's columns leave in whole 16-byte pieces side by side.
template <int TA, int TB, int MA, int NB, int NT>
__device__ __forceinline__ void put_rows(uint16_t* sm, f32x16 (&acc)[MA][NB], int wa, int wb, int tid, uint16_t* out,
                         int64_t ld, int64_t c0, int64_t nc, int64_t r0, int64_t nr, const int* to = nullptr) {
  constexpr int CH = TA / 8;  // 16-byte pieces of a row, exchanged by the row's low bits
  const int lane = tid & 63, hf = lane >> 5, col = lane & 31;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int r = wb + 32 * j + col;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& x = acc[i][j];
        const uint2 o = {cvt_pk_bf16(x[4 * q], x[4 * q + 1]), cvt_pk_bf16(x[4 * q + 2], x[4 * q + 3])};
        const int c = (wa + 32 * i + 8 * q) >> 3;
        *(uint2*)(sm + r * TA + ((c ^ (r & (CH - 1))) << 3) + 4 * hf) = o;
      }
  }
  __syncthreads();
  if (ld % 8 == 0 && ((uintptr_t)out & 15) == 0) {
#pragma unroll 4
    for (int id = tid; id < TB * CH; id += NT) {
      const int r = id / CH, c = id % CH;
      const int64_t row = r0 + r, at = c0 + 8 * c;
      if (row >= nr || at >= nc) continue;
      *(u32x4*)(out + (to ? to[row] : row) * ld + at) = *(const u32x4*)(sm + r * TA + ((c ^ (r & (CH - 1))) << 3));
    }
  } else {
    // an element a lane, side by side
#pragma unroll 4
    for (int id = tid; id < TB * TA; id += NT) {
      const int r = id / TA, c = id % TA;
      const int64_t row = r0 + r, at = c0 + c;
      if (row >= nr || at >= nc) continue;
      out[(to ? to[row] : row) * ld + at] = sm[r * TA + (((c >> 3) ^ (r & (CH - 1))) << 3) + (c & 7)];
    }
  }
}

// A wave's accumulators as 16 bits without a sign, to its rows and columns of the same: through its own part of LDS,
// without a wait for other waves.
template <int MA, int NB>
__device__ __forceinline__ void put_wave(uint16_t* sm, f32x16 (&acc)[MA][NB], int lane, uint16_t* out, int64_t ld,
                                         int64_t c0, int64_t r0, int64_t nr) {
  constexpr int CH = 4 * MA;  // 16-byte pieces of a row, exchanged by the row's low bits
  const int hf = lane >> 5, col = lane & 31;
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& x = acc[i][j];
        *(uint2*)(sm + (32 * j + col) * (8 * CH) + (((4 * i + q) ^ (col & (CH - 1))) << 3) + 4 * hf) =
            uint2{pack_u16(x[4 * q], x[4 * q + 1]), pack_u16(x[4 * q + 2], x[4 * q + 3])};
      }
#pragma unroll 4
  for (int id = lane; id < 32 * NB * CH; id += 64) {
    const int r = id / CH, c = id % CH;
    const u32x4 v = *(const u32x4*)(sm + r * (8 * CH) + ((c ^ (r & (CH - 1))) << 3));
    if (r0 + r < nr && c0 + 8 * c < ld) *(u32x4*)(out + (r0 + r) * ld + c0 + 8 * c) = v;
  }
}

// The same in fp32, rows of whole 16-byte pieces, four columns a lane; added to what is there, or not.
template <int MA, int NB>
__device__ __forceinline__ void put_rows32(f32x16 (&acc)[MA][NB], int wa, int wb, int lane, float* out, int64_t ld,
                                           int64_t c0, int64_t r0, int64_t nr, int add, const int* to = nullptr) {
  const int hf = lane >> 5, col = lane & 31;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t r = r0 + wb + 32 * j + col;
    if (r >= nr) continue;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t c = c0 + wa + 32 * i + 8 * q + 4 * hf;
        if (c >= ld) continue;
        float4 x = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        float* p = out + (to ? to[r] : r) * ld + c;
        if (add) {
          const float4 o = *(const float4*)p;
          x.x += o.x, x.y += o.y, x.z += o.z, x.w += o.w;
        }
        *(float4*)p = x;
      }
  }
}

// The same of rows that are not whole 16-byte pieces: through LDS, an element a lane, side by side (a training pass of
// distillation, 6 x 1413 x 29001: 384 -> 330 us; bf16, in put_rows, 2000 x 1001 x 20000: 446 -> 423).
template <int TA, int TB, int MA, int NB, int NT>
__device__ __forceinline__ void put_odd32(float* sm, f32x16 (&acc)[MA][NB], int wa, int wb, int tid, float* out, int64_t ld,
                                          int64_t c0, int64_t r0, int64_t nr, const int* to) {
  constexpr int CH = TA / 4;  // 16-byte pieces of a row, exchanged by the row's low bits
  const int lane = tid & 63, hf = lane >> 5, col = lane & 31;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int r = wb + 32 * j + col;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& x = acc[i][j];
        const int c = (wa + 32 * i + 8 * q + 4 * hf) >> 2;
        *(float4*)(sm + r * TA + ((c ^ (r & (CH - 1))) << 2)) = float4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
      }
  }
  __syncthreads();
#pragma unroll 4
  for (int id = tid; id < TB * TA; id += NT) {
    const int r = id / TA, c = id % TA;
    const int64_t row = r0 + r, at = c0 + c;
    if (row >= nr || at >= ld) continue;
    out[(to ? to[row] : row) * ld + at] = sm[r * TA + (((c >> 2) ^ (r & (CH - 1))) << 2) + (c & 3)];
  }
}

template <int TA, int TB, int WA, int WB, int kStages, bool AX, bool BX, int EPI, bool F32>
__global__ __launch_bounds__(WA* WB * 64, 2) void xe_gemm(GemmArgs g) {
  constexpr int NT = WA * WB * 64;
  constexpr int MA = TA / WA / 32, NB = TB / WB / 32;
  using E = std::conditional_t<F32, float, uint16_t>;
  using A = std::conditional_t<F32, Tile32<TA, AX, WA * WB>, Tile<TA, AX, WA * WB>>;
  using B = std::conditional_t<F32, Tile32<TB, BX, WA * WB>, Tile<TB, BX, WA * WB>>;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  E* sm = (E*)smem;
  constexpr int kStage = A::kElems + B::kElems;
  static_assert(!F32 || TA * TB <= kStages * kStage, "an output tile passes through LDS");
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hf = lane >> 5,
            col = lane & 31;
  const int wa = (wave % WA) * (TA / WA), wb = (wave / WA) * (TB / WB);

  // The workgroups of one XCD are neighbours, and share its L2: the tiles of one piece of the contraction
  // before the next piece's, eight tiles of b beside four of a at a time.
  if (g.count) {
    if constexpr (EPI == EPI_OUT || EPI == EPI_PART) {
      g.K = *g.count;
      if (g.gw && !*g.equal) g.b = g.gw;
    } else {
      g.nb = *g.count;
      g.tb = (int)((g.nb + TB - 1) / TB);
    }
  }
  const int tiles = g.ta * g.tb, total = tiles * g.splits;
  const int per = (total + 7) / 8;
  const int work = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || work >= total) return;
  const int split = work / tiles, t = work % tiles;
  const int group = t / (8 * g.ta), in = t % (8 * g.ta);
  const int width = min(8, g.tb - group * 8);
  const int64_t a0 = (int64_t)(in / width) * TA, b0 = (int64_t)(group * 8 + in % width) * TB;

  int64_t k0 = 0, k1 = g.K;
  if constexpr (EPI == EPI_ACC || EPI == EPI_PART) {
    const int64_t each = ((g.K + kBK - 1) / kBK + g.splits - 1) / g.splits;
    k0 = min(split * each * kBK, g.K);
    k1 = min(k0 + each * kBK, g.K);
  }
  const int iters = (int)((k1 - k0 + kBK - 1) / kBK);

  f32x16 acc[MA][NB];
#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int n = 0; n < 16; ++n) acc[i][j][n] = 0.0f;

  // Step t is computed from one of the LDS buffers while the next steps are on their way to the others;
  // operands are read one matrix-instruction depth (16) ahead.  One barrier a step, between its two
  // depths: behind it step t's buffer is free for its next step's loads, and step t + 1 is there.  Past
  // the end loads are masked off.
  constexpr bool kApart = EPI == EPI_TOP || EPI == EPI_SUMS;
  const int tile_a = (int)(a0 / TA);
  int64_t lda = g.lda, first_a = a0, rows0 = a0, rows = g.na;
  if constexpr (kApart) {
    const TileRows t = tile_rows(tile_a, TA, g.apart, g.ta);
    first_a = t.first, rows0 = 0, rows = (g.na - t.first + t.step - 1) / t.step;
    lda *= t.step;
  }
  A ta;
  B tb;
  ta.template init<kApart>(lda, rows0, rows, wave, lane);
  tb.init(g.ldb, b0, g.nb, wave, lane);
  const int64_t step_a = AX ? kBK * g.lda : kBK, step_b = BX ? kBK * g.ldb : kBK;
  const E* pa = (const E*)g.a + (AX ? k0 * g.lda + a0 : first_a * g.lda + k0);
  const E* pb = (const E*)g.b + (BX ? k0 * g.ldb + b0 : b0 * g.ldb + k0);
  int left = (int)(k1 - k0);
  auto load_a = [&](int n, E* d) { ta.load(n, d, pa, left, g.lda, g.lda - a0, wave); };
  auto load_b = [&](int n, E* d) { tb.load(n, d + A::kElems, pb, left, g.ldb, g.ldb - b0, wave); };
  auto next = [&]() {
    left -= kBK;
    pa += step_a, pb += step_b;
  };
  constexpr int kLoads = A::kLoads + B::kLoads;
  // TOP: squares of the rows that a lane's operands are of, where the products leave time for them (tiles of 256 do
  // not: 8192 x 2048 x 65536 1.85 -> 2.02 ms, even if only some tiles take them)
  constexpr bool kNorms = EPI == EPI_TOP && (F32 || TA < 256);
  float na[MA][2], nb[NB];
#pragma unroll
  for (int i = 0; i < MA; ++i) na[i][0] = na[i][1] = 0.0f;
#pragma unroll
  for (int j = 0; j < NB; ++j) nb[j] = 0.0f;
  auto squares = [](u32x4 v, float& even, float& odd) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x2 x = __builtin_bit_cast(bf16x2, (uint32_t)v[q]);
      float& s = q & 1 ? odd : even;
      s = __builtin_amdgcn_fdot2_f32_bf16(x, x, s, false);
    }
  };
  if constexpr (F32) {
    static_assert(kStages == 2, "a step in use, a step on its way");
    const E *pa0 = pa, *pb0 = pb;
    auto load = [&](E* d) {
#pragma unroll
      for (int n = 0; n < A::kLoads; ++n) load_a(n, d);
#pragma unroll
      for (int n = 0; n < B::kLoads; ++n) load_b(n, d);
      next();
    };
    // logits that are exponents: the five small products are summed apart, which leaves the large one's sum one
    // rounding in place of six for 16 columns (47 x 3616 x 2573: lse 3.7e-7 -> 1.5e-7 off)
    constexpr bool kApartSums = EPI == EPI_SUMS || EPI == EPI_TOP || EPI == EPI_KEPT;
    f32x16 low[kApartSums ? MA : 1][NB];
    if constexpr (kApartSums) {
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int n = 0; n < 16; ++n) low[i][j][n] = 0.0f;
    }
    // PLANES: operands split into three bf16 planes, six products; else fp32 matrix instructions
    auto product = [&](auto planes, f32x16(&acc)[MA][NB]) {
      constexpr bool PLANES = decltype(planes)::value;
      float ra[MA][8], rb[NB][8];
      auto read = [&](const E* s, int ks) {
#pragma unroll
        for (int i = 0; i < MA; ++i) A::op(s, wa + 32 * i, ks, lane, ra[i]);
#pragma unroll
        for (int j = 0; j < NB; ++j) B::op(s + A::kElems, wb + 32 * j, ks, lane, rb[j]);
      };
      if (iters > 0) {
        load(sm);
        load(sm + kStage);
        wait_all<kLoads>();
        read(sm, 0);
      }
      for (int it = 0; it < iters; ++it) {
        E *s = sm + (it & 1) * kStage, *d = sm + (~it & 1) * kStage;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4 ap[MA][3], bp[NB][3];
          if constexpr (PLANES && kNorms) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
#pragma unroll
              for (int i = 0; i < MA; ++i) na[i][n & 1] = fmaf(ra[i][n], ra[i][n], na[i][n & 1]);
#pragma unroll
              for (int j = 0; j < NB; ++j) nb[j] = fmaf(rb[j][n], rb[j][n], nb[j]);
            }
          }
          if constexpr (PLANES) {
#pragma unroll
            for (int i = 0; i < MA; ++i) split_planes(ra[i], ap[i]);
#pragma unroll
            for (int j = 0; j < NB; ++j) split_planes(rb[j], bp[j]);
          } else {
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
              for (int i = 0; i < MA; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                  acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(ra[i][n], rb[j][n], acc[i][j], 0, 0, 0);
          }
          if (ks == 1) {
            wait_all<0>();
            load(s);
          }
          read(ks ? d : s, ks ^ 1);
          if constexpr (PLANES) {
            // the small products first
            constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
            for (int q = 0; q < 6; ++q)
#pragma unroll
              for (int i = 0; i < MA; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                  f32x16& to = kApartSums && q < 5 ? low[i][j] : acc[i][j];
                  to = mfma32(ap[i][kA[q]], bp[j][kB[q]], to);
                }
          }
        }
      }
      // loads past the end may still be on their way to LDS
      wait_all<0>();
    };
    product(std::true_type{}, acc);
    if constexpr (kApartSums) {
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int n = 0; n < 16; ++n) acc[i][j][n] += low[i][j][n];
    }
    // Planes have no infinity (inf - inf, and zero planes times it) and no float beyond bf16's largest: every
    // sum that one enters is NaN.  Such sums (masked classes; or NaN in the inputs) are computed again as
    // the definition has them; the tile's others stay, whatever their neighbours hold.
    bool nan = false;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int n = 0; n < 16; ++n) nan |= acc[i][j][n] != acc[i][j][n];
    int* again = (int*)smem;
    if (tid == 0) *again = 0;
    __syncthreads();
    if (nan) *again = 1;
    __syncthreads();
    const bool redo = __builtin_amdgcn_readfirstlane(*again);
    __syncthreads();
    if (redo) {
      pa = pa0, pb = pb0, left = (int)(k1 - k0);
      f32x16 exact[MA][NB];
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int n = 0; n < 16; ++n) exact[i][j][n] = 0.0f;
      product(std::false_type{}, exact);
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            acc[i][j][n] = acc[i][j][n] == acc[i][j][n] ? acc[i][j][n] : exact[i][j][n];
    }
  } else {
    u32x4 ao[2][MA], bo[2][NB];
    // operands in the order in which the products need them: a 0, b 0.., a 1..
    auto read = [&](int n, int set, const E* s, int ks) {
      if (n == 0) ao[set][0] = A::op(s, wa, ks, lane);
      else if (n <= NB) bo[set][n - 1] = B::op(s + A::kElems, wb + 32 * (n - 1), ks, lane);
      else ao[set][n - NB] = A::op(s, wa + 32 * (n - NB), ks, lane);
    };
    if (iters > 0) {
#pragma unroll
      for (int t = 0; t < kStages; ++t) {
#pragma unroll
        for (int n = 0; n < A::kLoads; ++n) load_a(n, sm + t * kStage);
        if (t + 1 == kStages) break;
#pragma unroll
        for (int n = 0; n < B::kLoads; ++n) load_b(n, sm + t * kStage);
        next();
      }
      wait_all<(kStages - 1) * kLoads - B::kLoads>();
#pragma unroll
      for (int n = 0; n < MA + NB; ++n) read(n, 0, sm, 0);
    }
    // (Left to the compiler, the logits' products are 3 to 4% faster, 8192 x 2048 x 65536 2.02 -> 1.95 ms with what is
    // kept, those that read transposed 4% slower.)
    constexpr bool kFixed = AX || BX || !(EPI == EPI_SUMS || EPI == EPI_TOP || EPI == EPI_KEPT);
    // Behind the barrier a buffer takes a's loads, b's in the next step's first depth.  The source order is
    // the schedule: reads and loads are spread over the matrix instructions, since a burst of them from
    // all waves fills the LDS queue and holds up the matrix instructions behind it.
    E *s = sm, *e = sm + (kStages - 1) * kStage;
    for (int it = 0; it < iters; ++it) {
      E* d = s == sm + (kStages - 1) * kStage ? sm : s + kStage;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks == 1) wait_all<(kStages - 2) * kLoads>();
        constexpr int kM = MA * NB, kR = MA + NB;
#pragma unroll
        for (int n = 0; n < kM; ++n) {
          acc[n / NB][n % NB] = mfma32(ao[ks][n / NB], bo[ks][n % NB], acc[n / NB][n % NB]);
          if constexpr (kNorms) {
            if (n % NB == 0) squares(ao[ks][n / NB], na[n / NB][0], na[n / NB][1]);
            if (n < NB) squares(bo[ks][n], nb[n], nb[n]);
          }
#pragma unroll
          for (int r = n * kR / kM; r < (n + 1) * kR / kM; ++r) read(r, ks ^ 1, ks ? d : s, ks ^ 1);
          if (ks == 0) {
#pragma unroll
            for (int r = n * B::kLoads / kM; r < (n + 1) * B::kLoads / kM; ++r) load_b(r, e);
          } else {
            if (n == 0) next();
#pragma unroll
            for (int r = n * A::kLoads / kM; r < (n + 1) * A::kLoads / kM; ++r) load_a(r, s);
          }
          if constexpr (kFixed) __builtin_amdgcn_sched_barrier(0);
        }
      }
      e = s, s = d;
    }
    // loads past the end may still be on their way to LDS
    wait_all<0>();
  }

  if constexpr (EPI == EPI_LSE) {
    float2* red = (float2*)smem;  // [WA][TB]
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (a0 + TA > g.na) {
        const int end = (int)(g.na - a0) - wa - 4 * hf;
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (32 * i + 8 * (n >> 2) + (n & 3) >= end) acc[i][j][n] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) m = fmaxf(m, acc[i][j][n]);
      m = fmaxf(m, __shfl_xor(m, 32));
      const float from = m > -INFINITY ? m : 0.0f;  // a row of NaN has no maximum, and its sum stays NaN
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) s += __expf(acc[i][j][n] - from);
      s += __shfl_xor(s, 32);
      if (hf == 0) red[(wave % WA) * TB + wb + 32 * j + col] = float2{m, s};
    }
    __syncthreads();
    for (int r = tid; r < TB; r += NT) {
      if (b0 + r >= g.nb) break;
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int w = 0; w < WA; ++w) m = fmaxf(m, red[w * TB + r].x);
#pragma unroll
      for (int w = 0; w < WA; ++w) {
        const float2 q = red[w * TB + r];
        s += q.x == m ? q.y : q.y * __expf(q.x - m);
      }
      g.part[(b0 + r) * g.parts + a0 / TA] = float2{m, s};
    }
  }

  if constexpr (EPI == EPI_SUMS || EPI == EPI_TOP || EPI == EPI_KEPT) {
    // [WA][TB]; behind what put_wave uses
    float4* red = (float4*)(smem + (EPI == EPI_KEPT && !F32 ? TA * TB * 2 : 0));
    if constexpr (kNorms) {
      if (b0 == 0) {
        // the largest of the lane's classes (see far_norm)
        float group_norm = 0.0f;
#pragma unroll
        for (int i = 0; i < MA; ++i) {
          float q = na[i][0] + na[i][1], part = fmaxf(na[i][0], na[i][1]);
          q += __shfl_xor(q, 32), part = fmaxf(part, __shfl_xor(part, 32));
          const int row = spread_row<TA>(wa + 32 * i + col);
          float norm = q > 0.0f || row >= rows ? sqrtf(q) : kVanished;
          if (q > 0.0f && !(in_range(q) && no_large_entry(q, part)))
            norm = far_norm<!F32, true>((const E*)g.a + first_a * g.lda + row * lda, (int)g.K, hf, 2);
          group_norm = fmaxf(group_norm, norm);
        }
        for (int k = 1; k < 32; k <<= 1)
          if (k != 4) group_norm = fmaxf(group_norm, __shfl_xor(group_norm, k));
        if (wave < WA && (lane & ~4) == 0) g.a_norm[tile_a * 4 + (lane >> 1) + wave] = group_norm;
      }
      if (tile_a == 0) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float q = nb[j] + __shfl_xor(nb[j], 32);
          const int64_t row = b0 + wb + 32 * j + col;
          float norm = sqrtf(q);  // zero: see lp_rows
          if (row < g.nb && !in_range(q) && q != 0.0f) norm = far_norm<!F32, false>((const E*)g.b + row * g.ldb, (int)g.K, hf, 2);
          if (wave % WA == 0 && hf == 0 && row < g.nb) g.b_norm[row] = norm;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      if (rows0 + TA > rows) {
        const int left = (int)(rows - rows0);
        const int end = kApart ? (left - 2 * hf - wave % WA + 3) >> 2 : left - wa - 4 * hf;
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if ((kApart ? 16 * i + n : 32 * i + 8 * (n >> 2) + (n & 3)) >= end) acc[i][j][n] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) m = fmaxf(m, acc[i][j][n]);
      m = fmaxf(m, __shfl_xor(m, 32));
      const float from = m > -INFINITY ? m : 0.0f;  // a row of NaN has no maximum, and its sum stays NaN
      float s = 0.0f, t = 0.0f;
      // TOP: how far below the maximum the lane's four largest are (times k2: positive floats in whole numbers' order),
      // each with its place in the low bits
      uint32_t y1 = ~0u, y2 = ~0u, y3 = ~0u, y4 = ~0u;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float x = acc[i][j][n] - from, y = x * g.k2;
          const float e = F32 ? exp2_of(acc[i][j][n], from, g.k2, g.k2_low) : __builtin_amdgcn_exp2f(y);
          s += e;
          if constexpr (EPI == EPI_KEPT) acc[i][j][n] = e;
          else t = fmaf(e, fmaxf(x, -3.4028235e38f), t);
          if constexpr (EPI == EPI_TOP) {
            const uint32_t key = (__float_as_uint(y) & 0x7fffffc0u) | (16 * i + n);
            y4 = med3(y3, y4, key), y3 = med3(y2, y3, key), y2 = med3(y1, y2, key), y1 = min(y1, key);
            if (n % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // or the compiler keeps all differences at once
          }
        }
      if constexpr (EPI == EPI_TOP) {
        if (r < g.nb) {
          const int64_t at = r * (4 * (int64_t)g.parts) + tile_a * 4 + 2 * hf + wave % WA;
          if (hf == 0) g.tops[r * (2 * (int64_t)g.parts) + tile_a * 2 + wave % WA] = from;
          g.keys[at] = uint4{y1, y2, y3, y4};
        }
      }
      s += __shfl_xor(s, 32);
      t += __shfl_xor(t, 32);
      if (hf == 0) red[(wave % WA) * TB + wb + 32 * j + col] = float4{m, s, t, 0.0f};
      if constexpr (EPI == EPI_KEPT) {
        if (g.g) {
          // times exp(scale (m - ref)), and 2^-kDown; where that is no factor to store, the row is written again
          const float ref = r < g.nb ? g.ref[g.index ? g.index[r] : r] : 0.0f;
          const float f = F32 ? fminf(exp2_of(from, ref, g.k2, g.k2_low), 1.0e30f)
                              : fminf(__builtin_amdgcn_exp2f(fmaf(from - ref, g.k2, -kDown)), 1.0f);
#pragma unroll
          for (int i = 0; i < MA; ++i)
#pragma unroll
            for (int n = 0; n < 16; ++n) acc[i][j][n] *= f;
        }
      }
    }
    if constexpr (EPI == EPI_KEPT) {
      if (g.g) {
        if constexpr (F32) put_rows32<MA, NB>(acc, wa, wb, lane, (float*)g.g, g.ldg, a0, b0, g.nb, 0);
        else put_wave<MA, NB>(sm + wave * (32 * MA * 32 * NB), acc, lane, (uint16_t*)g.g, g.ldg, a0 + wa, b0 + wb, g.nb);
      }
    }
    __syncthreads();
    for (int r = tid; r < TB; r += NT) {
      if (b0 + r >= g.nb) break;
      float m = -INFINITY, s = 0.0f, t = 0.0f;
#pragma unroll
      for (int w = 0; w < WA; ++w) m = fmaxf(m, red[w * TB + r].x);
#pragma unroll
      for (int w = 0; w < WA; ++w) {
        const float4 q = red[w * TB + r];
        if (q.x == m) {
          s += q.y, t += q.z;
        } else {
          const float x = q.x - m, e = __builtin_amdgcn_exp2f(x * g.k2);
          s = fmaf(q.y, e, s);
          if (e > 0.0f) t = fmaf(e, fmaf(q.y, x, q.z), t);  // x may be what no factor of it is: a masked class's
        }
      }
      if constexpr (EPI != EPI_KEPT) g.sums[(b0 + r) * g.parts + tile_a] = float4{m, s, t, 0.0f};
      else g.part[(b0 + r) * g.parts + a0 / TA] = float2{m, s};
    }
  }

  if constexpr (EPI == EPI_AGAIN) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      const int64_t row = r < g.nb ? g.index[r] : 0;
      const float ref = r < g.nb ? g.ref[row] : 0.0f, c = r < g.nb ? g.factor[r] : 1.0f;
      const int64_t first = a0 + wa + 4 * hf;
      const int64_t end = g.na - first;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n)
          acc[i][j][n] = 32 * i + 8 * (n >> 2) + (n & 3) < end ? c * exp2_of(acc[i][j][n], ref, g.k2, g.k2_low) : 0.0f;
      for (int k = 0; k < g.top; ++k) {
        const int64_t at = g.ids[row * g.top + k] - first;
        const float p = g.prob[row * g.top + k];
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (32 * i + 8 * (n >> 2) + (n & 3) == at) acc[i][j][n] -= p;
      }
    }
    if constexpr (F32) put_rows32<MA, NB>(acc, wa, wb, lane, (float*)g.g, g.ldg, a0, b0, g.nb, 0, g.to);
    else put_rows<TA, TB, MA, NB, NT>(sm, acc, wa, wb, tid, (uint16_t*)g.g, g.ldg, a0, g.ldg, b0, g.nb, g.to);
  }

  if constexpr (EPI == EPI_GRAD) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      const int64_t row = r < g.nb ? g.index[r] : -1;
      const bool kept = row >= 0;
      const int64_t y = kept ? g.labels[row] : -1;
      const float l = kept ? g.lse[row] : 0.0f;
      // the lane's label and the end of the vocabulary, counted from its first class
      const int64_t first = a0 + wa + 4 * hf;
      const int at = kept && y - g.v0 >= first && y - g.v0 < first + TA ? (int)(y - g.v0 - first) : -1;
      const int end = (int)min(g.na - first, (int64_t)TA);
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) acc[i][j][n] = __expf(acc[i][j][n] - l);
      if (__any(at >= 0)) {
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (32 * i + 8 * (n >> 2) + (n & 3) == at) acc[i][j][n] -= 1.0f;
      }
      if (!__all(kept) || a0 + TA > g.na) {
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (!kept || 32 * i + 8 * (n >> 2) + (n & 3) >= end) acc[i][j][n] = 0.0f;
      }
    }
    const bool weighted = g.gw && !*g.equal;
    auto put = [&](void* out) __attribute__((always_inline)) {
      if constexpr (F32) put_rows32<MA, NB>(acc, wa, wb, lane, (float*)out, g.ldg, a0, b0, g.nb, 0);
      else put_rows<TA, TB, MA, NB, NT>(sm, acc, wa, wb, tid, (uint16_t*)out, g.ldg, a0, g.ldg, b0, g.nb);
    };
    if (g.both || !weighted) put(g.g);
    if (weighted) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int64_t r = b0 + wb + 32 * j + col;
        const float w = r < g.nb ? g.weight[g.index[r]] / *g.scale : 0.0f;
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n) acc[i][j][n] *= w;
      }
      put(g.gw);
    }
  }

  auto put_out32 = [&](const int* to) __attribute__((always_inline)) {
    if (g.ldo % 4 == 0 && ((uintptr_t)g.out & 15) == 0)
      put_rows32<MA, NB>(acc, wa, wb, lane, (float*)g.out, g.ldo, a0, b0, g.nb, 0, to);
    else put_odd32<TA, TB, MA, NB, NT>((float*)smem, acc, wa, wb, tid, (float*)g.out, g.ldo, a0, b0, g.nb, to);
  };
  if constexpr (EPI == EPI_OUT) {
    const float w = g.scale ? *g.scale : 1.0f;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int n = 0; n < 16; ++n) acc[i][j][n] *= w;
    if constexpr (!F32)
      put_rows<TA, TB, MA, NB, NT>(sm, acc, wa, wb, tid, (uint16_t*)g.out, g.ldo, a0, g.ldo, b0, g.nb);
  }

  if constexpr (EPI == EPI_ROWS) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      const int64_t row = r < g.nb ? g.to[r] : 0;
      const bool on = r < g.nb && g.at[row] >= 0;  // else zero, where a masked class's minus infinity made it NaN, too
      const float w = on ? g.row_weight[row] : 0.0f;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) acc[i][j][n] = on ? acc[i][j][n] * w : 0.0f;
    }
    if constexpr (F32) put_out32(g.to);
    else put_rows<TA, TB, MA, NB, NT>(sm, acc, wa, wb, tid, (uint16_t*)g.out, g.ldo, a0, g.ldo, b0, g.nb, g.to);
  }

  if constexpr (EPI == EPI_ACC || EPI == EPI_PART)
    put_rows32<MA, NB>(acc, wa, wb, lane, g.acc + (int64_t)split * g.acc_rows * g.lda, g.lda, a0, b0, g.nb, g.add);
  if constexpr (F32 && EPI == EPI_OUT) put_out32(nullptr);
}

// The rows that count, those whose label is a class, in order (one workgroup): index [rows that count],
// at [n] (a row's place among them, or -1), their number; and of their dloss the value that all have, or the
// largest finite magnitude (1 without), and which.
__global__ __launch_bounds__(1024) void xe_rows(const int64_t* labels, const float* dloss, int64_t n, int64_t vocab,
                                                int* index, int* at, int* count, float* scale, int* equal) {
  __shared__ int s[16];
  __shared__ float sm[16], from[16], to[16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int base = 0;
  float m = 0.0f, lo = INFINITY, hi = -INFINITY;
  bool nan = false;
  for (int64_t i0 = 0; i0 < n; i0 += 1024) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t y = i < n ? labels[i] : -1;
    const bool kept = y >= 0 && y < vocab;
    if (kept && dloss) {
      const float w = dloss[i];
      m = fmaxf(m, fabsf(w) <= 3.0e38f ? fabsf(w) : 0.0f);
      lo = fminf(lo, w), hi = fmaxf(hi, w);
      nan |= w != w;
    }
    const uint64_t mask = __ballot(kept);
    __syncthreads();
    if (lane == 0) s[wave] = __popcll(mask);
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      before += k < wave ? s[k] : 0;
      all += s[k];
    }
    const int place = before + __popcll(mask & ((1ull << lane) - 1));
    if (i < n) at[i] = kept ? place : -1;
    if (kept) index[place] = (int)i;
    base += all;
  }
  if (nan) lo = -INFINITY, hi = INFINITY;
  for (int k = 32; k; k >>= 1) {
    m = fmaxf(m, __shfl_xor(m, k));
    lo = fminf(lo, __shfl_xor(lo, k)), hi = fmaxf(hi, __shfl_xor(hi, k));
  }
  if (lane == 0) sm[wave] = m, from[wave] = lo, to[wave] = hi;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 16; ++k) m = fmaxf(m, sm[k]), lo = fminf(lo, from[k]), hi = fmaxf(hi, to[k]);
    *count = base;
    *equal = lo >= hi;
    *scale = lo == hi ? lo : m > 0.0f ? m : 1.0f;
  }
}

// Rows of an input as the products take them, [rows][dp], zero from column d on: all of them, or with
// `index` those that count.
__global__ void xe_copy(const void* x, int bf16, int64_t rows, int d, int dp, const int* index, const int* count,
                        void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // four columns
  const int64_t per = dp / 4;
  const int64_t r = i / per;
  if (r >= (count ? *count : rows)) return;
  const int c = (int)(i % per) * 4;
  const int64_t row = index ? index[r] : r;
  float v[4];
  if (d % 4 == 0 && ((uintptr_t)x & 15) == 0 && c < d) {
    if (bf16) {
      const uint2 w = *(const uint2*)((const uint16_t*)x + row * d + c);
      v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const float4 w = *(const float4*)((const float*)x + row * d + c);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k < d ? load_in(x, row * d + c + k, bf16) : 0.0f;
  }
  const int64_t at = r * dp + c;
  if (bf16) *(uint2*)((uint16_t*)out + at) = uint2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
  else *(float4*)((float*)out + at) = float4{v[0], v[1], v[2], v[3]};
}

// A wave's products of a row of a with N rows of b, in 64 bits.  Loads of 4 KB of each are on their way together;
// those past the rows' ends are zeros.  The loop over them stays one: few rows wait for their instructions, 400
// cycles for 64 bytes of those.
template <int N, bool BF16>
__device__ __forceinline__ void row_dots(const void* a, const void* b, int64_t ra, const int (&rb)[N], int dp, int lane,
                                         double (&z)[N]) {
  const int bytes = dp * (BF16 ? 2 : 4);
  const rsrc_t ar = make_rsrc((const char*)a + ra * bytes, bytes);
  rsrc_t br[N];
#pragma unroll
  for (int n = 0; n < N; ++n) br[n] = make_rsrc((const char*)b + (int64_t)rb[n] * bytes, bytes), z[n] = 0.0;
#pragma unroll 1
  for (int o = 0; o < bytes; o += 4096) {
    u32x4 x[4], y[N][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = buf_ld16(ar, lane * 16 + o + 1024 * k, 0);
#pragma unroll
      for (int n = 0; n < N; ++n) y[n][k] = buf_ld16(br[n], lane * 16 + o + 1024 * k, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll 1
    for (int k = 0; k < 4 && o + 1024 * k < bytes; ++k) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const uint32_t u = x[0][q], v = y[n][0][q];
          if constexpr (BF16) {
            z[n] = fma((double)__uint_as_float(u << 16), (double)__uint_as_float(v << 16), z[n]);
            z[n] = fma((double)__uint_as_float(u & 0xFFFF0000u), (double)__uint_as_float(v & 0xFFFF0000u), z[n]);
          } else {
            z[n] = fma((double)__uint_as_float(u), (double)__uint_as_float(v), z[n]);
          }
        }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        x[i] = x[i + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) y[n][i] = y[n][i + 1];
      }
    }
  }
#pragma unroll 1
  for (int k = 32; k; k >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) z[n] += __shfl_xor(z[n], k);
}

// The same of rows of at most kShort bytes, 16 a lane: of each `lanes` lanes one product.
constexpr int kShort = 512;
__device__ __forceinline__ int short_lanes(int bytes) {
  return bytes <= 64 ? 4 : bytes <= 128 ? 8 : bytes <= 256 ? 16 : 32;
}
template <bool BF16>
__device__ __forceinline__ double short_dot(const void* a, const void* b, int64_t ra, int64_t rb, int bytes, int lanes,
                                            int lane) {
  const int at = (lane & (lanes - 1)) * 16;
  double v = 0.0;
  if (at < bytes) {
    const u32x4 x = *(const u32x4*)((const char*)a + ra * bytes + at);
    const u32x4 y = *(const u32x4*)((const char*)b + rb * bytes + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (BF16) {
        v = fma((double)__uint_as_float(x[q] << 16), (double)__uint_as_float(y[q] << 16), v);
        v = fma((double)__uint_as_float(x[q] & 0xFFFF0000u), (double)__uint_as_float(y[q] & 0xFFFF0000u), v);
      } else {
        v = fma((double)__uint_as_float(x[q]), (double)__uint_as_float(y[q]), v);
      }
    }
  }
  for (int k = lanes / 2; k; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

__global__ void xe_zero(void* out, int64_t count, int bf16) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    if (bf16) ((uint16_t*)out)[i] = 0;
    else ((float*)out)[i] = 0.0f;
  }
}

// ------------------------------------------------------------------------------------------- host

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
int64_t align256(int64_t b) { return up(b, 256); }

constexpr double kLog2e = 1.4426950408889634;

template <int TA, int TB, int WA, int WB, int ST, bool AX, bool BX, int EPI, bool F32>
atlasmem_status gemm_launch(GemmArgs g, hipStream_t st) {
  constexpr int lds = F32 ? ST * (TA + TB) * kBK * 4
                          : std::max(ST * (TA + TB) * kBK * 2, TA * TB * 2 + (EPI == EPI_KEPT ? WA * TB * 16 : 0));
  auto kern = xe_gemm<TA, TB, WA, WB, ST, AX, BX, EPI, F32>;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return ATLASMEM_E_DEVICE;
  g.ta = (int)((g.na + TA - 1) / TA);
  g.tb = (int)((g.nb + TB - 1) / TB);
  if (EPI != EPI_ACC && EPI != EPI_PART) g.splits = 1;
  const int64_t blocks = up((int64_t)g.ta * g.tb * g.splits, 8);
  kern<<<(unsigned)blocks, WA * WB * 64, lds, st>>>(g);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

// Sides of the tiles.  256 (a workgroup a CU) take 0.7 of the time of 128 (two a CU) for an area (8192 x
// 16384 x 2048: 554 us against 790); the smaller ones fill the chip with less: rounds of workgroups decide,
// or where the contraction is split to fill it (dX), the areas.  Where 128 leave more than half of the chip
// idle, 64: a step of theirs takes a third of the time.  fp32 has no 256: planes and accumulators of two
// workgroups of 128 fill a CU's registers.
int64_t tiles_of(int64_t na, int64_t nb, int side) { return (na + side - 1) / side * ((nb + side - 1) / side); }
int side_of(int64_t na, int64_t nb, bool bf16) {
  const int64_t t = tiles_of(na, nb, 128);
  if (t <= 128) return 64;
  return bf16 && (tiles_of(na, nb, 256) + 255) / 256 * 28 <= (t + 511) / 512 * 20 ? 256 : 128;
}
int side_split(int64_t na, int64_t nb, bool bf16) {
  return bf16 && tiles_of(na, nb, 256) * 28 <= tiles_of(na, nb, 128) * 10 ? 256 : 128;
}

// Of at most 64 rows, tiles of 128 x 64 for bf16 (a workgroup of three on a CU; 1 x 1024 x 50257 26 -> 21 us, 64 x
// 2048 x 65536 51 -> 46; 64 x 64: 23 and 61) and of 64 for fp32 (22 x 504 x 33288 55 -> 30 us; 128 x 64: 34).
constexpr int64_t kFew = 64;
int side_for(int64_t na, int64_t nb, bool bf16) {
  return nb <= kFew ? (bf16 ? 128 : 64) : side_of(na, nb, bf16);
}
template <bool AX, int EPI>
atlasmem_status gemm_few(const GemmArgs& g, bool bf16, hipStream_t st) {
  if (bf16) return gemm_launch<128, 64, 2, 2, 4, AX, false, EPI, false>(g, st);
  return gemm_launch<64, 64, 2, 2, 2, AX, false, EPI, true>(g, st);
}

template <bool AX, bool BX, int EPI>
atlasmem_status gemm(const GemmArgs& g, bool bf16, int side, hipStream_t st) {
  if (bf16) {
    if (side == 256) return gemm_launch<256, 256, 2, 4, 4, AX, BX, EPI, false>(g, st);
    if (side == 128) return gemm_launch<128, 128, 2, 2, 4, AX, BX, EPI, false>(g, st);
    return gemm_launch<64, 64, 2, 2, 4, AX, BX, EPI, false>(g, st);
  }
  if (side == 128) return gemm_launch<128, 128, 2, 2, 2, AX, BX, EPI, true>(g, st);
  return gemm_launch<64, 64, 2, 2, 2, AX, BX, EPI, true>(g, st);
}

// A matrix whose rows the engine can read where they are: whole, aligned 16-byte pieces.
bool direct(const void* p, int d, bool bf16) { return d % (bf16 ? 8 : 4) == 0 && ((uintptr_t)p & 15) == 0; }

// Forward calls of so many operations leave out the rows that do not count: finding and copying the others
// takes 10 us, which the products of a tenth of the rows outweigh from here on (1.1 PFLOP/s).
constexpr double kGatherFrom = 2e11;

atlasmem_status rows_that_count(int64_t n, int64_t vocab, const int64_t* labels, const float* dloss, int* index,
                                int* at, int* count, float* scale, int* equal, hipStream_t st) {
  xe_rows<<<1, 1024, 0, st>>>(labels, dloss, n, vocab, index, at, count, scale, equal);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

atlasmem_status copy_rows(const void* x, bool bf16, int64_t rows, int d, int dp, const int* index, const int* count,
                          void* out, hipStream_t st) {
  const int64_t blocks = (rows * (dp / 4) + 255) / 256;
  xe_copy<<<(unsigned)blocks, 256, 0, st>>>(x, bf16, rows, d, dp, index, count, out);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace

}  // namespace am
