// Softmax cross entropy over a large vocabulary, without keeping the logits (gfx950).
//   z = X W^T, lse_i = log sum_v exp z_iv, loss_i = lse_i - z_i,y_i
//   G_iv = exp(z_iv - lse_i) - [v = y_i],  dX_i = dloss_i (G W)_i,  dW = G^T (dloss X)
// The forward computes tiles of z and leaves of each row and tile its maximum and sum of exponentials;
// the backward computes them again by pieces of the vocabulary, writes the piece's G (bf16), and both
// products read it.  Three matrix products of one engine:
//   z   a = W (lanes v), b = X (lanes i): both rows along the contraction
//   dX  a = W (lanes d, rows across the contraction: read transposed from LDS), b = G
//   dW  a = X, b = G, both across the contraction
// An output tile has b's index in its lanes and a's, four at a time, in its registers.
//
// Types.  bf16 inputs are used as they are.  fp32 ones (and then G) go to LDS as they are and are split in
// registers into three bf16 planes, whose six products down to 2^-16 of the leading one are summed in fp32
// (relative 2^-24, at a sixth of the bf16 rate).  Sums that planes cannot hold (infinities, the lowest float: a
// masked class) come out NaN and are taken from a second pass of the tile by fp32 matrix instructions; the
// check alone costs 3% of a training pass (777 x 384 x 16001: 257 -> 266 us, both timed in turn).
// In bf16 G is rounded, once: kept in fp32 its two products would take twice the matrix instructions.  dX's G is
// rounded without its weight: the label's entry, -1 + p, is the large one and nearly exact while p is small,
// where dloss (-1 + p) has one rounding error for all rows of equal weight (dX 3.7e-3 off instead of
// 1.7e-3); dX takes its rows' weights in the fp32 sums.  dW sums over the rows, and its G is rounded with their
// weights (over the largest one), X as it is.  Where all weights are one value the two are the same,
// and that value is a factor of dW's fp32 sums (8192 x 2048 x 65536, all rows, gradients 5.57 ms; unequal
// weights, with a second G to write, 5.77 ms.  Weights on X instead, a second rounding, took 5.52 ms, and dW of
// 1024 x 256 x 16384 was 2.36e-3 off instead of 2.19e-3, its rows of classes that are no label 2.65e-3
// instead of 2.32e-3).
//
// Rows that are left out are left out of the products: the others' X is copied together, and the kernels
// take their number from the device.
//
// Measured, bf16, 8192 rows (7373 count) x 2048 x 65536: logits 1.69 ms (1.17 PFLOP/s), then for each of
// four pieces G 496 us (1.00; of that 70 us are its stores), dX 431 us (1.15), dW 379 us (1.31): 7.0 ms a
// training pass.  A library's plain product of these sizes reaches 1.2 (logits, written out) to 1.5
// PFLOP/s; both run at 1.65 GHz, the power limit, with the matrix cores 75% (the library 85%) busy.
// One row x 1024 x 50257: 20 us for W's 103 MB (5.2 TB/s).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace am {

namespace {

constexpr int kBK = 32;        // contraction elements of a step: two matrix instructions deep
enum { EPI_LSE, EPI_GRAD, EPI_ACC, EPI_OUT };

struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb;        // elements of a row
  int64_t na, nb;          // rows (or, across the contraction, columns) of a and b
  int64_t K;
  const int* count;        // rows that count (OUT: K, else nb), or null: as given
  int ta, tb;              // tiles of a and b
  int splits;              // pieces of the contraction (ACC; else 1)
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
};

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
        const int r = id >> 2;
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

  __device__ void init(int64_t ld, int64_t r0, int64_t rows, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = (wave * kLoads + i) * 64 + lane;
      if constexpr (ACROSS) {
        const int k = id / (R / 4), c = (id % (R / 4) ^ ((k >> 3 & 1) << 3)) * 4;
        kc[i] = 0;
        off[i] = c < rows - r0 ? (uint32_t)((k * ld + c) * 4) : 0x80000000u;
      } else {
        const int r = id >> 3;
        kc[i] = ((id & 7) ^ ((r >> 1) & 7)) * 4;
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

// A tile's accumulators, rounded to bf16, to rows r0.. (nr of them) and columns c0.. (nc) of a matrix:
// through LDS, so that a row's columns leave in whole 16-byte pieces side by side.
template <int TA, int TB, int MA, int NB, int NT>
__device__ __forceinline__ void put_rows(uint16_t* sm, f32x16 (&acc)[MA][NB], int wa, int wb, int tid, uint16_t* out,
                         int64_t ld, int64_t c0, int64_t nc, int64_t r0, int64_t nr) {
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
  const bool vec = ld % 8 == 0 && ((uintptr_t)out & 15) == 0;
#pragma unroll 4
  for (int id = tid; id < TB * CH; id += NT) {
    const int r = id / CH, c = id % CH;
    const int64_t row = r0 + r, at = c0 + 8 * c;
    if (row >= nr || at >= nc) continue;
    const u32x4 v = *(const u32x4*)(sm + r * TA + ((c ^ (r & (CH - 1))) << 3));
    uint16_t* p = out + row * ld + at;
    if (vec) {
      *(u32x4*)p = v;
    } else {
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (at + n < nc) p[n] = (uint16_t)(v[n >> 1] >> (16 * (n & 1)));
    }
  }
}

// The same in fp32, four columns a lane; added to what is there (rows of whole 16-byte pieces), or not.
template <int MA, int NB>
__device__ __forceinline__ void put_rows32(f32x16 (&acc)[MA][NB], int wa, int wb, int lane, float* out, int64_t ld,
                                           int64_t c0, int64_t r0, int64_t nr, int add) {
  const int hf = lane >> 5, col = lane & 31;
  const bool vec = ld % 4 == 0 && ((uintptr_t)out & 15) == 0;
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
        float* p = out + r * ld + c;
        if (add) {
          const float4 o = *(const float4*)p;
          x.x += o.x, x.y += o.y, x.z += o.z, x.w += o.w;
        }
        if (vec) {
          *(float4*)p = x;
        } else {
          if (c + 0 < ld) p[0] = x.x;
          if (c + 1 < ld) p[1] = x.y;
          if (c + 2 < ld) p[2] = x.z;
          if (c + 3 < ld) p[3] = x.w;
        }
      }
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
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hf = lane >> 5,
            col = lane & 31;
  const int wa = (wave % WA) * (TA / WA), wb = (wave / WA) * (TB / WB);

  // The workgroups of one XCD are neighbours, and share its L2: the tiles of one piece of the contraction
  // before the next piece's, eight tiles of b beside four of a at a time.
  if (g.count) {
    if constexpr (EPI == EPI_OUT) {
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
  if constexpr (EPI == EPI_ACC) {
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
  A ta;
  B tb;
  ta.init(g.lda, a0, g.na, wave, lane);
  tb.init(g.ldb, b0, g.nb, wave, lane);
  const int64_t step_a = AX ? kBK * g.lda : kBK, step_b = BX ? kBK * g.ldb : kBK;
  const E* pa = (const E*)g.a + (AX ? k0 * g.lda + a0 : a0 * g.lda + k0);
  const E* pb = (const E*)g.b + (BX ? k0 * g.ldb + b0 : b0 * g.ldb + k0);
  int left = (int)(k1 - k0);
  auto load_a = [&](int n, E* d) { ta.load(n, d, pa, left, g.lda, g.lda - a0, wave); };
  auto load_b = [&](int n, E* d) { tb.load(n, d + A::kElems, pb, left, g.ldb, g.ldb - b0, wave); };
  auto next = [&]() {
    left -= kBK;
    pa += step_a, pb += step_b;
  };
  constexpr int kLoads = A::kLoads + B::kLoads;
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
                for (int j = 0; j < NB; ++j) acc[i][j] = mfma32(ap[i][kA[q]], bp[j][kB[q]], acc[i][j]);
          }
        }
      }
      // loads past the end may still be on their way to LDS
      wait_all<0>();
    };
    product(std::true_type{}, acc);
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
          __builtin_amdgcn_sched_barrier(0);
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

  if constexpr (EPI == EPI_ACC)
    put_rows32<MA, NB>(acc, wa, wb, lane, g.acc + (int64_t)split * g.acc_rows * g.lda, g.lda, a0, b0, g.nb, g.add);
  if constexpr (F32 && EPI == EPI_OUT)
    put_rows32<MA, NB>(acc, wa, wb, lane, (float*)g.out, g.ldo, a0, b0, g.nb, 0);
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

// loss, lse of a row: a wave joins the tiles' maxima and sums, and takes the row's product with its
// label's class.
__global__ __launch_bounds__(256) void xe_join(const float2* part, int parts, const int* at, const void* X,
                                               const void* W, int in_bf16, int vec, int64_t n, int d, int64_t vocab,
                                               const int64_t* labels, float* loss, float* lse) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= n) return;
  const int64_t y = labels[r];
  if (y < 0 || y >= vocab) {
    if (lane == 0) loss[r] = 0.0f, lse[r] = 0.0f;
    return;
  }
  const float2* p = part + (at ? at[r] : r) * parts;
  float m = -INFINITY, s = 0.0f;
  for (int i = lane; i < parts; i += 64) {
    const float2 q = p[i];
    const float t = fmaxf(m, q.x);
    if (t > -INFINITY) s = s * __expf(m - t) + q.y * __expf(q.x - t);
    else s += q.y;  // NaN stays
    m = t;
  }
  for (int k = 32; k; k >>= 1) {
    const float om = __shfl_xor(m, k), os = __shfl_xor(s, k);
    const float t = fmaxf(m, om);
    if (t > -INFINITY) s = s * __expf(m - t) + os * __expf(om - t);
    else s += os;
    m = t;
  }
  float z = 0.0f;
  for (int c = lane * 8; c < d; c += 512) {  // one order of the sum, whatever the alignment
    if (vec && in_bf16) {
      const u32x4 a = *(const u32x4*)((const uint16_t*)X + r * d + c);
      const u32x4 b = *(const u32x4*)((const uint16_t*)W + y * d + c);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        z = fmaf(__uint_as_float(k & 1 ? a[k >> 1] & 0xFFFF0000u : a[k >> 1] << 16),
                 __uint_as_float(k & 1 ? b[k >> 1] & 0xFFFF0000u : b[k >> 1] << 16), z);
    } else if (vec) {
      const float *a = (const float*)X + r * d + c, *b = (const float*)W + y * d + c;
#pragma unroll
      for (int h = 0; h < 8; h += 4) {
        if (c + h >= d) break;
        const float4 u = *(const float4*)(a + h), v = *(const float4*)(b + h);
        z = fmaf(u.w, v.w, fmaf(u.z, v.z, fmaf(u.y, v.y, fmaf(u.x, v.x, z))));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < d) z = fmaf(load_in(X, r * d + c + k, in_bf16), load_in(W, y * d + c + k, in_bf16), z);
    }
  }
  for (int k = 32; k; k >>= 1) z += __shfl_xor(z, k);
  if (lane == 0) {
    const float l = m + logf(s), q = l - z;
    lse[r] = l;
    loss[r] = q < 0.0f ? 0.0f : q;  // the two sums round apart where the label has all the weight
  }
}

// dX from the partial sums of the contraction's pieces, times the rows' weights: four columns a thread.
__global__ void xe_sum(const float* acc, int splits, int64_t n, int d, int dp, const int* at, const float* dloss,
                       void* out, int out_bf16, int vec) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / (dp / 4);
  const int c = (int)(i % (dp / 4)) * 4;
  if (r >= n || c >= d) return;
  const int64_t place = at[r];
  float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits && place >= 0; ++s) {
    const float4 a = *(const float4*)(acc + (s * n + place) * dp + c);
    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
  }
  const float w = place >= 0 && dloss ? dloss[r] : 1.0f;
  const float x[4] = {v.x * w, v.y * w, v.z * w, v.w * w};
  const int64_t o = r * d + c;
  if (vec && out_bf16) *(uint2*)((uint16_t*)out + o) = uint2{cvt_pk_bf16(x[0], x[1]), cvt_pk_bf16(x[2], x[3])};
  else if (vec) *(float4*)((float*)out + o) = float4{x[0], x[1], x[2], x[3]};
  else
    for (int k = 0; k < 4 && c + k < d; ++k) {
      if (out_bf16) ((uint16_t*)out)[o + k] = (uint16_t)bf16_bits(x[k]);
      else ((float*)out)[o + k] = x[k];
    }
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

template <int TA, int TB, int WA, int WB, int ST, bool AX, bool BX, int EPI, bool F32>
atlasmem_status gemm_launch(GemmArgs g, hipStream_t st) {
  constexpr int lds = F32 ? ST * (TA + TB) * kBK * 4 : std::max(ST * (TA + TB) * kBK * 2, TA * TB * 2);
  auto kern = xe_gemm<TA, TB, WA, WB, ST, AX, BX, EPI, F32>;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return ATLASMEM_E_DEVICE;
  g.ta = (int)((g.na + TA - 1) / TA);
  g.tb = (int)((g.nb + TB - 1) / TB);
  if (EPI != EPI_ACC) g.splits = 1;
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

// The inputs as the engine takes them: bf16 rows of whole, aligned 16-byte pieces.
struct Plan {
  int el, dp;                   // bytes of an element, elements of a copied row
  int64_t piece;                // classes of a piece of G
  int parts, splits;
  int side, side_x;             // of the forward's and of dX's tiles
};

// A piece of G: what the last-level cache holds, and 2048 classes at least (from 65536 bf16 rows on, then, it grows
// with them), since dX's fp32 sums pass through memory once for every piece.
constexpr int64_t kPieceBytes = 256 << 20, kPieceClasses = 2048;

Plan plan_of(const CrossEntropy& s) {
  Plan p = {};
  p.el = s.bf16 ? 2 : 4;
  p.dp = (int)up(s.d, s.bf16 ? 8 : 4);
  int64_t piece = kPieceBytes / std::max<int64_t>(s.n * p.el, 1) / 256 * 256;
  piece = std::max(piece, kPieceClasses);
  const int64_t pieces = (s.vocab + piece - 1) / piece;
  p.piece = up((s.vocab + pieces - 1) / pieces, 256);
  p.side = side_of(s.vocab, s.n, s.bf16);
  p.parts = (int)((s.vocab + p.side - 1) / p.side);
  p.side_x = side_split(p.dp, s.n, s.bf16);
  const int64_t tiles = std::max<int64_t>(tiles_of(p.dp, s.n, p.side_x), 1);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>((p.side_x == 256 ? 256 : 512) / tiles, p.piece / 512));
  if (tiles * p.splits <= 128) p.side_x = 64;
  return p;
}

bool direct(const void* p, const CrossEntropy& s) {
  return s.d % (s.bf16 ? 8 : 4) == 0 && ((uintptr_t)p & 15) == 0;
}

// What a call finds in its workspace, one behind the other.
struct Space {
  int *index, *at, *count, *equal;
  float* scale;
  char *x, *w, *g, *gw;
  float* acc;
  float2* part;
  int64_t bytes;
};
Space space_of(void* p, const CrossEntropy& s, const Plan& l, bool backward) {
  Space w = {};
  char* at = (char*)p;
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += align256(bytes);
    return r;
  };
  const int64_t rows = l.el * s.n * (int64_t)l.dp;
  w.index = (int*)take(4 * s.n), w.at = (int*)take(4 * s.n);
  w.count = (int*)take(12), w.equal = w.count + 1, w.scale = (float*)(w.count + 2);
  w.x = take(rows);
  w.w = take(l.el * s.vocab * (int64_t)l.dp);
  if (backward) {
    w.g = take(l.el * s.n * l.piece);
    w.gw = take(l.el * s.n * l.piece);
    w.acc = (float*)take(4 * (int64_t)l.splits * s.n * l.dp);
  } else {
    w.part = (float2*)take(8 * s.n * (int64_t)l.parts);
  }
  w.bytes = at - (char*)p;
  return w;
}

// Forward calls of so many operations leave out the rows that do not count: finding and copying the others
// takes 10 us, which the products of a tenth of the rows outweigh from here on (1.1 PFLOP/s).
constexpr double kGatherFrom = 2e11;

atlasmem_status rows_that_count(const CrossEntropy& s, const Space& w, const int64_t* labels, const float* dloss,
                                hipStream_t st) {
  xe_rows<<<1, 1024, 0, st>>>(labels, dloss, s.n, s.vocab, w.index, w.at, w.count, w.scale, w.equal);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

atlasmem_status copy_of(const void* x, const CrossEntropy& s, const Plan& p, int64_t rows, const int* index,
                        const int* count, void* out, hipStream_t st) {
  const int64_t blocks = (rows * (p.dp / 4) + 255) / 256;
  xe_copy<<<(unsigned)blocks, 256, 0, st>>>(x, s.bf16, rows, s.d, p.dp, index, count, out);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace

int64_t cross_entropy_workspace_bytes(const CrossEntropy& s, bool backward) {
  return space_of(nullptr, s, plan_of(s), backward).bytes;
}

atlasmem_status cross_entropy(const CrossEntropy& s, const void* X, const void* W, const int64_t* labels, float* loss,
                              float* lse, void* workspace, hipStream_t st) {
  const Plan p = plan_of(s);
  const Space ws = space_of(workspace, s, p, false);
  const bool gather = 2.0 * s.n * s.d * s.vocab * (s.bf16 ? 1 : 6) >= kGatherFrom;
  atlasmem_status e = ATLASMEM_OK;
  if (gather) e = rows_that_count(s, ws, labels, nullptr, st);
  const int *index = gather ? ws.index : nullptr, *count = gather ? ws.count : nullptr;
  if (e == ATLASMEM_OK && (gather || !direct(X, s)))
    e = copy_of(X, s, p, s.n, index, count, ws.x, st);
  if (e == ATLASMEM_OK && !direct(W, s))
    e = copy_of(W, s, p, s.vocab, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  GemmArgs g = {};
  g.part = ws.part;
  g.a = direct(W, s) ? W : ws.w;
  g.b = gather || !direct(X, s) ? ws.x : X;
  g.lda = g.ldb = p.dp;
  g.na = s.vocab, g.nb = s.n, g.K = p.dp;
  g.count = count;
  g.parts = p.parts;
  e = gemm<false, false, EPI_LSE>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  xe_join<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(g.part, g.parts, gather ? ws.at : nullptr, X, W, s.bf16,
                                                     direct(X, s) && direct(W, s), s.n, s.d, s.vocab, labels, loss,
                                                     lse);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

atlasmem_status cross_entropy_backward(const CrossEntropy& s, const void* X, const void* W, const int64_t* labels,
                                       const float* lse, const float* dloss, void* dX, void* dW, void* workspace,
                                       hipStream_t st) {
  if (s.n == 0) {
    if (dW) {
      const int64_t count = s.vocab * (int64_t)s.d;
      xe_zero<<<(unsigned)std::min<int64_t>((count + 255) / 256, 1 << 16), 256, 0, st>>>(dW, count, s.bf16);
      AM_LAUNCH_CHECK();
    }
    return ATLASMEM_OK;
  }
  const Plan p = plan_of(s);
  const Space ws = space_of(workspace, s, p, true);
  const bool weighted = dW && dloss;
  atlasmem_status e = rows_that_count(s, ws, labels, dloss, st);
  if (e == ATLASMEM_OK)
    e = copy_of(X, s, p, s.n, ws.index, ws.count, ws.x, st);
  if (e == ATLASMEM_OK && !direct(W, s))
    e = copy_of(W, s, p, s.vocab, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  const char* wa = direct(W, s) ? (const char*)W : ws.w;
  for (int64_t v0 = 0; v0 < s.vocab; v0 += p.piece) {
    const int64_t nv = std::min(p.piece, s.vocab - v0), ldg = up(nv, 64);
    // G of the piece
    GemmArgs g = {};
    g.count = ws.count;
    g.a = wa + v0 * p.dp * p.el, g.b = ws.x;
    g.lda = g.ldb = p.dp;
    g.na = nv, g.nb = s.n, g.K = p.dp;
    g.labels = labels, g.lse = lse, g.index = ws.index, g.v0 = v0;
    g.g = ws.g, g.ldg = ldg, g.both = dX != nullptr;
    if (weighted) g.gw = dX ? ws.gw : ws.g, g.weight = dloss, g.scale = ws.scale, g.equal = ws.equal;
    e = gemm<false, false, EPI_GRAD>(g, s.bf16, side_of(nv, s.n, s.bf16), st);
    if (e != ATLASMEM_OK) return e;
    if (dX) {
      GemmArgs x = {};
      x.count = ws.count;
      x.a = wa + v0 * p.dp * p.el, x.lda = p.dp, x.na = p.dp;
      x.b = ws.g, x.ldb = ldg, x.nb = s.n;
      x.K = nv;
      x.splits = p.splits, x.acc = ws.acc, x.acc_rows = s.n, x.add = v0 > 0;
      e = gemm<true, false, EPI_ACC>(x, s.bf16, p.side_x, st);
      if (e != ATLASMEM_OK) return e;
    }
    if (dW) {
      GemmArgs x = {};
      x.count = ws.count;
      x.a = ws.x, x.lda = p.dp, x.na = p.dp;
      if (weighted) x.gw = dX ? ws.gw : ws.g, x.scale = ws.scale, x.equal = ws.equal;
      x.b = ws.g, x.ldb = ldg, x.nb = nv;
      x.K = s.n;
      x.out = (char*)dW + v0 * s.d * p.el, x.ldo = s.d;
      e = gemm<true, true, EPI_OUT>(x, s.bf16, side_of(p.dp, nv, s.bf16), st);
      if (e != ATLASMEM_OK) return e;
    }
  }
  if (dX) {
    const int vec = s.d % 4 == 0 && ((uintptr_t)dX & 15) == 0;
    xe_sum<<<(unsigned)((s.n * (p.dp / 4) + 255) / 256), 256, 0, st>>>(ws.acc, p.splits, s.n, s.d, p.dp, ws.at, dloss,
                                                                       dX, s.bf16, vec);
    AM_LAUNCH_CHECK();
  }
  return ATLASMEM_OK;
}

}  // namespace am
