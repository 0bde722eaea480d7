// Softmax cross entropy over a large vocabulary, without keeping the logits (gfx950).
//   z = X W^T, lse_i = log sum_v exp z_iv, loss_i = lse_i - z_i,y_i
//   G_iv = dloss_i (exp(z_iv - lse_i) - [v = y_i]),  dX = G W,  dW = G^T X
// The forward computes tiles of z and leaves of each row and tile its maximum and sum of exponentials;
// the backward computes them again by pieces of the vocabulary, writes the piece's G (bf16), and both
// products read it.  Three matrix products of one engine:
//   z   a = W (lanes v), b = X (lanes i): both rows along the contraction
//   dX  a = W (lanes d, rows across the contraction: read transposed from LDS), b = G
//   dW  a = X, b = G, both across the contraction
// An output tile has b's index in its lanes and a's, four at a time, in its registers.  bf16 inputs are
// used as they are; fp32 ones (and then G) as three bf16 planes, the six products of planes down to
// 2^-16 of the leading one summed in fp32 (relative 2^-24, at the matrix cores' bf16 rate over six).
#include <algorithm>

#include "common.h"
#include "internal.h"

namespace am {

namespace {

constexpr int kBK = 64;        // contraction elements of a step
constexpr int kProducts = 6;   // of planes, fp32
__constant__ const int kPlaneA[kProducts] = {2, 0, 1, 1, 0, 0};
__constant__ const int kPlaneB[kProducts] = {0, 2, 1, 0, 1, 0};

enum { EPI_LSE, EPI_GRAD, EPI_ACC, EPI_OUT };

struct GemmArgs {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb;        // elements of a row
  int64_t pa, pb;          // elements from plane to plane
  int64_t na, nb;          // rows (or, across the contraction, columns) of a and b
  int64_t K;
  int products;            // 1 or kProducts
  int ta, tb;              // tiles of a and b
  int splits;              // pieces of the contraction (EPI_ACC)
  // epilogues
  float2* part;            // LSE: [nb][parts]: (maximum, sum of exponentials)
  int parts;
  int part0;
  const int64_t* labels;   // [nb]
  const float* lse;
  const float* dloss;
  int64_t v0, vocab;
  uint16_t* g;             // GRAD: [nb][ldg], planes of pg elements
  int64_t ldg, pg;
  int planes;
  float* acc;              // ACC: [splits][nb][na]
  int first, add;
  void* out;               // OUT: [nb][ldo]
  int64_t ldo;
  int out_bf16;
};

// One operand's tile in LDS.  Along the contraction: [R][64], 16-byte pieces of a row exchanged by the
// row's low bits; across: [64][R], 32-byte pieces exchanged by the contraction index's low bits.  Either
// way the lanes of a read lie on distinct banks.
template <int R, bool ACROSS>
struct Tile {
  static constexpr int kElems = R * kBK;
  static constexpr int kLoads = R * kBK / 8 / 256;
  __device__ static int place(int i, int tid) {
    const int id = tid + i * 256;
    if constexpr (ACROSS) {
      const int k = id / (R / 8), c = id % (R / 8);
      return k * R + ((((c >> 1) ^ (k & 3)) << 1) | (c & 1)) * 8;
    } else {
      const int r = id >> 3, c = id & 7;
      return r * kBK + ((c ^ (r & 7)) << 3);
    }
  }
  // lane's eight contraction elements 16 ks + 8 (lane / 32) + 0..7 of row (column) r0 + lane % 32
  __device__ static u32x4 op(const uint16_t* s, int r0, int ks, int lane) {
    const int hf = lane >> 5;
    if constexpr (ACROSS) {
      const int e = (lane & 15) >> 2;
      const int k = 16 * ks + 8 * hf + e;
      const int c = (((r0 + (lane & 16)) >> 4) ^ e) * 16 + 4 * (lane & 3);
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* lds4;
      const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + k * R + c)));
      const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + (k + 4) * R + c)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
      const int r = r0 + (lane & 31);
      return *(const u32x4*)(s + r * kBK + (((2 * ks + hf) ^ (r & 7)) << 3));
    }
  }
};

// Global side: one step's pieces of a tile in registers.
template <int R, bool ACROSS>
struct Stage {
  u32x4 v[Tile<R, ACROSS>::kLoads];
  // rows r0.. of a matrix along the contraction, or columns r0.. of one across it; contraction k0..
  __device__ void load(const uint16_t* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t k1, int tid) {
    const int64_t left = rows - r0;
    if constexpr (ACROSS) {
      const int64_t ks = min(k1 - k0, (int64_t)kBK);
      const rsrc_t rs = make_rsrc(p + k0 * ld + r0, (uint32_t)(ks <= 0 ? 0 : (ks * ld - r0) * 2));
#pragma unroll
      for (int i = 0; i < Tile<R, true>::kLoads; ++i) {
        const int id = tid + i * 256, k = id / (R / 8), c = (id % (R / 8)) * 8;
        v[i] = buf_ld16(rs, k < ks && c < left ? (int)((k * ld + c) * 2) : -1, 0);
      }
    } else {
      const rsrc_t rs = make_rsrc(p + r0 * ld + k0, (uint32_t)((min(left, (int64_t)R) * ld - k0) * 2));
#pragma unroll
      for (int i = 0; i < Tile<R, false>::kLoads; ++i) {
        const int id = tid + i * 256, r = id >> 3, c = (id & 7) * 8;
        v[i] = buf_ld16(rs, r < left && k0 + c < k1 ? (int)((r * ld + c) * 2) : -1, 0);
      }
    }
  }
  __device__ void store(uint16_t* s, int tid) const {
#pragma unroll
    for (int i = 0; i < Tile<R, ACROSS>::kLoads; ++i) *(u32x4*)(s + Tile<R, ACROSS>::place(i, tid)) = v[i];
  }
};

template <int TA, int TB, int WA, int WB, bool AX, bool BX, int EPI>
__global__ __launch_bounds__(256, TA* TB >= 65536 ? 1 : 2) void xe_gemm(GemmArgs g) {
  static_assert(WA * WB == 4, "four waves");
  constexpr int MA = TA / WA / 32, NB = TB / WB / 32;
  using A = Tile<TA, AX>;
  using B = Tile<TB, BX>;
  extern __shared__ __attribute__((aligned(16))) uint16_t sm[];
  constexpr int kStage = A::kElems + B::kElems;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hf = lane >> 5, col = lane & 31;
  const int wa = (wave % WA) * (TA / WA), wb = (wave / WA) * (TB / WB);

  // tiles of one XCD are neighbours: eight tiles of b beside four of a at a time share its L2
  const int total = g.ta * g.tb;
  const int bid = blockIdx.x;
  const int per = (total + 7) / 8;
  const int t = (bid & 7) * per + (bid >> 3);
  if ((bid >> 3) >= per || t >= total) return;
  const int group = t / (8 * g.ta), in = t % (8 * g.ta);
  const int width = min(8, g.tb - group * 8);
  const int64_t a0 = (int64_t)(in / width) * TA, b0 = (int64_t)(group * 8 + in % width) * TB;

  int64_t k0 = 0, k1 = g.K;
  if constexpr (EPI == EPI_ACC) {
    const int64_t steps = (g.K + kBK - 1) / kBK, each = (steps + g.splits - 1) / g.splits;
    k0 = min((int64_t)blockIdx.y * each * kBK, g.K);
    k1 = min(k0 + each * kBK, g.K);
  }
  const int steps = (int)((k1 - k0 + kBK - 1) / kBK);
  const int iters = steps * g.products;

  f32x16 acc[MA][NB];
#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int n = 0; n < 16; ++n) acc[i][j][n] = 0.0f;

  Stage<TA, AX> sa;
  Stage<TB, BX> sb;
  auto fetch = [&](int it) {
    const int q = it / steps;
    const int64_t k = k0 + (int64_t)(it - q * steps) * kBK;
    const int p = g.products == 1 ? kProducts - 1 : q;
    sa.load(g.a + kPlaneA[p] * g.pa, g.lda, a0, g.na, k, k1, tid);
    sb.load(g.b + kPlaneB[p] * g.pb, g.ldb, b0, g.nb, k, k1, tid);
  };
  if (iters > 0) {
    fetch(0);
    sa.store(sm, tid);
    sb.store(sm + A::kElems, tid);
  }
  for (int it = 0; it < iters; ++it) {
    __syncthreads();
    const uint16_t* s = sm + (it & 1) * kStage;
    if (it + 1 < iters) fetch(it + 1);
#pragma unroll
    for (int ks = 0; ks < kBK / 16; ++ks) {
      u32x4 ao[MA], bo[NB];
#pragma unroll
      for (int i = 0; i < MA; ++i) ao[i] = A::op(s, wa + 32 * i, ks, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j) bo[j] = B::op(s + A::kElems, wb + 32 * j, ks, lane);
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma32(ao[i], bo[j], acc[i][j]);
    }
    if (it + 1 < iters) {
      uint16_t* d = sm + ((it + 1) & 1) * kStage;
      sa.store(d, tid);
      sb.store(d + A::kElems, tid);
    }
  }

  if constexpr (EPI == EPI_LSE) {
    __syncthreads();
    float2* red = (float2*)sm;  // [WA][TB]
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int64_t v = a0 + wa + 32 * i + 8 * (n >> 2) + 4 * hf + (n & 3);
          if (v >= g.na) acc[i][j][n] = -INFINITY;
          m = fmaxf(m, acc[i][j][n]);
        }
      m = fmaxf(m, __shfl_xor(m, 32));
      float s = 0.0f;
      if (m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n) s += __expf(acc[i][j][n] - m);
      }
      s += __shfl_xor(s, 32);
      if (hf == 0) red[(wave % WA) * TB + wb + 32 * j + col] = float2{m, s};
    }
    __syncthreads();
    for (int r = tid; r < TB; r += 256) {
      if (b0 + r >= g.nb) break;
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int w = 0; w < WA; ++w) m = fmaxf(m, red[w * TB + r].x);
#pragma unroll
      for (int w = 0; w < WA; ++w) {
        const float2 q = red[w * TB + r];
        s += q.x == m ? q.y : q.y * __expf(q.x - m);
      }
      g.part[(b0 + r) * g.parts + g.part0 + a0 / TA] = float2{m, s};
    }
  }

  if constexpr (EPI == EPI_GRAD) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      if (r >= g.nb) continue;
      const int64_t y = g.labels[r];
      const bool kept = y >= 0 && y < g.vocab;
      const float l = kept ? g.lse[r] : 0.0f, w = kept ? (g.dloss ? g.dloss[r] : 1.0f) : 0.0f;
      const int64_t at = kept ? y - g.v0 : -1;
      uint16_t* out = g.g + r * g.ldg;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t v = a0 + wa + 32 * i + 8 * q + 4 * hf;
          if (v >= g.ldg) continue;
          float x[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float p = __expf(acc[i][j][4 * q + n] - l) - (v + n == at ? 1.0f : 0.0f);
            x[n] = kept && v + n < g.na ? p * w : 0.0f;
          }
          for (int n = 0; n < g.planes; ++n) {
            const uint2 o = {cvt_pk_bf16(x[0], x[1]), cvt_pk_bf16(x[2], x[3])};
            *(uint2*)(out + n * g.pg + v) = o;
            x[0] -= __uint_as_float(o.x << 16), x[1] -= __uint_as_float(o.x & 0xFFFF0000u);
            x[2] -= __uint_as_float(o.y << 16), x[3] -= __uint_as_float(o.y & 0xFFFF0000u);
          }
        }
    }
  }

  if constexpr (EPI == EPI_ACC || EPI == EPI_OUT) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = b0 + wb + 32 * j + col;
      if (r >= g.nb) continue;
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t c = a0 + wa + 32 * i + 8 * q + 4 * hf;
          if (c >= g.na) continue;
          float x[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) x[n] = acc[i][j][4 * q + n];
          if constexpr (EPI == EPI_ACC) {
            float4* p = (float4*)(g.acc + ((int64_t)blockIdx.y * g.nb + r) * g.lda + c);
            if (g.add) {
              const float4 o = *p;
              x[0] += o.x, x[1] += o.y, x[2] += o.z, x[3] += o.w;
            }
            *p = float4{x[0], x[1], x[2], x[3]};
          } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
              if (c + n < g.ldo) {
                if (g.out_bf16) ((uint16_t*)g.out)[r * g.ldo + c + n] = (uint16_t)bf16_bits(x[n]);
                else ((float*)g.out)[r * g.ldo + c + n] = x[n];
              }
          }
        }
    }
  }
}

// Rows of an input as bf16 planes [planes][rows][dp], zero from column d on; rows whose label is no
// class become zero (what they hold must not reach the other rows' sums).
__global__ void xe_planes(const void* x, int in_bf16, int64_t rows, int d, int dp, int planes, const int64_t* labels,
                          int64_t vocab, uint16_t* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // a pair of columns
  const int64_t per = dp / 2;
  if (i >= rows * per) return;
  const int64_t r = i / per;
  const int c = (int)(i % per) * 2;
  const bool kept = !labels || (labels[r] >= 0 && labels[r] < vocab);
  float v0 = kept && c < d ? load_in(x, r * d + c, in_bf16) : 0.0f;
  float v1 = kept && c + 1 < d ? load_in(x, r * d + c + 1, in_bf16) : 0.0f;
  for (int n = 0; n < planes; ++n) {
    const uint32_t w = cvt_pk_bf16(v0, v1);
    *(uint32_t*)(out + (n * rows + r) * dp + c) = w;
    v0 -= __uint_as_float(w << 16);
    v1 -= __uint_as_float(w & 0xFFFF0000u);
  }
}

// loss, lse of a row: a wave joins the tiles' maxima and sums, and takes the row's product with its
// label's class.
__global__ __launch_bounds__(256) void xe_join(const float2* part, int parts, const void* X, const void* W, int in_bf16,
                                               int64_t n, int d, int64_t vocab, const int64_t* labels, float* loss,
                                               float* lse) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= n) return;
  const int64_t y = labels[r];
  if (y < 0 || y >= vocab) {
    if (lane == 0) loss[r] = 0.0f, lse[r] = 0.0f;
    return;
  }
  const float2* p = part + r * parts;
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
  for (int c = lane; c < d; c += 64) z += load_in(X, r * d + c, in_bf16) * load_in(W, y * d + c, in_bf16);
  for (int k = 32; k; k >>= 1) z += __shfl_xor(z, k);
  if (lane == 0) {
    const float l = m + logf(s), q = l - z;
    lse[r] = l;
    loss[r] = q < 0.0f ? 0.0f : q;  // the two sums round apart where the label has all the weight
  }
}

// dX from the partial sums of the contraction's pieces.
__global__ void xe_sum(const float* acc, int splits, int64_t n, int d, int dp, void* out, int out_bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n * d) return;
  const int64_t at = i / d * dp + i % d;
  float v = 0.0f;
  for (int s = 0; s < splits; ++s) v += acc[s * n * dp + at];
  if (out_bf16) ((uint16_t*)out)[i] = (uint16_t)bf16_bits(v);
  else ((float*)out)[i] = v;
}

__global__ void xe_zero(void* out, int64_t count, int bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  if (bf16) ((uint16_t*)out)[i] = 0;
  else ((float*)out)[i] = 0.0f;
}

// ------------------------------------------------------------------------------------------- host

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
int64_t align256(int64_t b) { return up(b, 256); }

template <int TA, int TB, int WA, int WB, bool AX, bool BX, int EPI>
atlasmem_status gemm_launch(GemmArgs g, hipStream_t st) {
  constexpr int lds = 2 * (TA + TB) * kBK * 2;
  auto kern = xe_gemm<TA, TB, WA, WB, AX, BX, EPI>;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return ATLASMEM_E_DEVICE;
  g.ta = (int)((g.na + TA - 1) / TA);
  g.tb = (int)((g.nb + TB - 1) / TB);
  const int64_t blocks = up((int64_t)g.ta * g.tb, 8);
  if (blocks > INT32_MAX) return ATLASMEM_E_SHAPE;
  kern<<<dim3((unsigned)blocks, EPI == EPI_ACC ? g.splits : 1), 256, lds, st>>>(g);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

// Tiles of 256 x 256 where they fill the chip, of 128 x 128 otherwise.
bool wide(int64_t na, int64_t nb) { return ((na + 255) / 256) * ((nb + 255) / 256) >= 256; }

template <bool AX, bool BX, int EPI>
atlasmem_status gemm(const GemmArgs& g, bool w, hipStream_t st) {
  if (w) return gemm_launch<256, 256, 2, 2, AX, BX, EPI>(g, st);
  return gemm_launch<128, 128, 2, 2, AX, BX, EPI>(g, st);
}

// The inputs as the engine takes them: bf16 rows of whole, aligned 16-byte pieces.
struct Plan {
  int planes, dp;
  int64_t n, vocab, piece;      // classes of a piece
  int parts, splits;
  bool copy_w;
  int64_t x_bytes, w_bytes, part_bytes, g_bytes, acc_bytes;
};

constexpr int64_t kPieceBytes = 256 << 20;  // of G: what the last-level cache holds

Plan plan_of(const CrossEntropy& s) {
  Plan p = {};
  p.planes = s.bf16 ? 1 : 3;
  p.dp = (int)up(s.d, 8);
  p.n = s.n, p.vocab = s.vocab;
  int64_t piece = kPieceBytes / std::max<int64_t>(s.n * 2 * p.planes, 1) / 256 * 256;
  piece = std::max<int64_t>(piece, 2048);
  const int64_t pieces = (s.vocab + piece - 1) / piece;
  p.piece = up((s.vocab + pieces - 1) / pieces, 256);
  p.parts = (int)((s.vocab + 127) / 128);
  const int64_t tiles = std::max<int64_t>((s.n + 127) / 128, 1) * ((p.dp + 127) / 128);
  p.splits = wide(p.dp, s.n) ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(512 / tiles, p.piece / 512));
  p.x_bytes = align256(2 * p.planes * s.n * (int64_t)p.dp);
  p.w_bytes = align256(2 * p.planes * s.vocab * (int64_t)p.dp);
  p.part_bytes = align256(8 * s.n * (int64_t)p.parts);
  p.g_bytes = align256(2 * p.planes * s.n * p.piece);
  p.acc_bytes = align256(4 * (int64_t)p.splits * s.n * p.dp);
  return p;
}

bool direct(const void* p, const CrossEntropy& s) { return s.bf16 && s.d % 8 == 0 && ((uintptr_t)p & 15) == 0; }

atlasmem_status planes_of(const void* x, const CrossEntropy& s, const Plan& p, int64_t rows, const int64_t* labels,
                          uint16_t* out, hipStream_t st) {
  const int64_t blocks = (rows * (p.dp / 2) + 255) / 256;
  if (blocks > INT32_MAX) return ATLASMEM_E_SHAPE;
  xe_planes<<<(unsigned)blocks, 256, 0, st>>>(x, s.bf16, rows, s.d, p.dp, p.planes, labels, s.vocab, out);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace

int64_t cross_entropy_workspace_bytes(const CrossEntropy& s, bool backward) {
  const Plan p = plan_of(s);
  const int64_t inputs = p.x_bytes + p.w_bytes;
  return backward ? inputs + p.g_bytes + p.acc_bytes : inputs + p.part_bytes;
}

atlasmem_status cross_entropy(const CrossEntropy& s, const void* X, const void* W, const int64_t* labels, float* loss,
                              float* lse, void* workspace, hipStream_t st) {
  const Plan p = plan_of(s);
  char* ws = (char*)workspace;
  uint16_t* xp = (uint16_t*)ws;
  uint16_t* wp = (uint16_t*)(ws + p.x_bytes);
  GemmArgs g = {};
  g.part = (float2*)(ws + p.x_bytes + p.w_bytes);
  atlasmem_status e = ATLASMEM_OK;
  if (!direct(X, s)) e = planes_of(X, s, p, s.n, nullptr, xp, st);
  if (e == ATLASMEM_OK && !direct(W, s)) e = planes_of(W, s, p, s.vocab, nullptr, wp, st);
  if (e != ATLASMEM_OK) return e;
  g.a = direct(W, s) ? (const uint16_t*)W : wp;
  g.b = direct(X, s) ? (const uint16_t*)X : xp;
  g.lda = g.ldb = p.dp;
  g.pa = s.vocab * p.dp, g.pb = s.n * p.dp;
  g.na = s.vocab, g.nb = s.n, g.K = p.dp;
  g.products = s.bf16 ? 1 : kProducts;
  const bool w = wide(s.vocab, s.n);
  g.parts = (int)((s.vocab + (w ? 255 : 127)) / (w ? 256 : 128));
  e = gemm<false, false, EPI_LSE>(g, w, st);
  if (e != ATLASMEM_OK) return e;
  xe_join<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(g.part, g.parts, X, W, s.bf16, s.n, s.d, s.vocab, labels, loss,
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
      xe_zero<<<(unsigned)((count + 255) / 256), 256, 0, st>>>(dW, count, s.bf16);
      AM_LAUNCH_CHECK();
    }
    return ATLASMEM_OK;
  }
  const Plan p = plan_of(s);
  char* ws = (char*)workspace;
  uint16_t* xp = (uint16_t*)ws;
  uint16_t* wp = (uint16_t*)(ws + p.x_bytes);
  uint16_t* gp = (uint16_t*)(ws + p.x_bytes + p.w_bytes);
  float* acc = (float*)(ws + p.x_bytes + p.w_bytes + p.g_bytes);
  // rows that are left out are copied as zeros: their values must not meet G's zeros in dW
  atlasmem_status e = planes_of(X, s, p, s.n, labels, xp, st);
  if (e == ATLASMEM_OK && !direct(W, s)) e = planes_of(W, s, p, s.vocab, nullptr, wp, st);
  if (e != ATLASMEM_OK) return e;
  const uint16_t* wa = direct(W, s) ? (const uint16_t*)W : wp;
  const int products = s.bf16 ? 1 : kProducts;
  for (int64_t v0 = 0; v0 < s.vocab; v0 += p.piece) {
    const int64_t nv = std::min(p.piece, s.vocab - v0), ldg = up(nv, 64);
    GemmArgs g = {};
    g.products = products;
    // G of the piece
    g.a = wa + v0 * p.dp, g.b = xp;
    g.lda = g.ldb = p.dp;
    g.pa = s.vocab * p.dp, g.pb = s.n * p.dp;
    g.na = nv, g.nb = s.n, g.K = p.dp;
    g.labels = labels, g.lse = lse, g.dloss = dloss, g.v0 = v0, g.vocab = s.vocab;
    g.g = gp, g.ldg = ldg, g.pg = s.n * ldg, g.planes = p.planes;
    e = gemm<false, false, EPI_GRAD>(g, wide(nv, s.n), st);
    if (e != ATLASMEM_OK) return e;
    if (dX) {
      GemmArgs x = {};
      x.products = products;
      x.a = wa + v0 * p.dp, x.lda = p.dp, x.pa = s.vocab * p.dp, x.na = p.dp;
      x.b = gp, x.ldb = ldg, x.pb = s.n * ldg, x.nb = s.n;
      x.K = nv;
      x.splits = p.splits, x.acc = acc, x.add = v0 > 0;
      e = gemm<true, false, EPI_ACC>(x, wide(p.dp, s.n), st);
      if (e != ATLASMEM_OK) return e;
    }
    if (dW) {
      GemmArgs x = {};
      x.products = products;
      x.a = xp, x.lda = p.dp, x.pa = s.n * p.dp, x.na = p.dp;
      x.b = gp, x.ldb = ldg, x.pb = s.n * ldg, x.nb = nv;
      x.K = s.n;
      x.out = (char*)dW + v0 * s.d * (s.bf16 ? 2 : 4), x.ldo = s.d, x.out_bf16 = s.bf16;
      e = gemm<true, true, EPI_OUT>(x, wide(p.dp, nv), st);
      if (e != ATLASMEM_OK) return e;
    }
  }
  if (dX) {
    xe_sum<<<(unsigned)((s.n * s.d + 255) / 256), 256, 0, st>>>(acc, p.splits, s.n, s.d, p.dp, dX, s.bf16);
    AM_LAUNCH_CHECK();
  }
  return ATLASMEM_OK;
}

}  // namespace am
