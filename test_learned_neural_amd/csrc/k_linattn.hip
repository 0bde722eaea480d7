// Linear attention with a decay for each head (gfx950).
//
// Per memory m = (b, h), lambda = exp(log_decay[h]):
//   W_t = lambda W_{t-1} + v_t k_t^T,   y_t = scale W_t q_t            (W: d_value x d_key, fp32)
// in the chunked form for many tokens and the recurrence itself for a few; and the gradients of an
// outer loss with respect to q, k, v, W_0 and log_decay.
//
// One chunk kernel serves the forward and the three backward products.  With "queries" x, "keys" y,
// "values" z and a state S [x, z] (chunks of 32 positions i, j; S_0 the state before the chunk):
//   out_i = c_out (lambda^(i+1-e) S_0^T x_i + c_upd sum_{j<=i} lambda^(i-j) (x_i . y_j) z_j)
//   S'    = lambda^r S_0 + c_upd sum_j lambda^(r-1-j+e) y_j z_j^T            (r rows in the chunk)
//   forward   x = q,  y = k,  z = v,  e = 0: y_t, state W^T
//   dq        x = dy, y = v,  z = k,  e = 0: dq_t = scale W_t^T dy_t
//   dk, dv    positions run backwards, e = 1, c_upd = scale, state A_t = lambda A_{t+1} + scale dy_t q_t^T
//             (A_T = dW_T):  dk_t = A_t^T v_t (x = v, y = dy, z = q), dv_t = A_t k_t (x = k, y = q, z = dy)
// and d log_decay is the tangent state's share (dS/dlog lambda, carried beside S) of the outputs:
//   sum_i scale dy_i . (dS_i / dlog lambda)^T q_i + <dW_T, dS_T / dlog lambda>,
// in the dq kernel (t = q, O_i the output's part from before the chunk, P the masked scores, St the tangent):
//   sum_i [(i+1) t_i . O_i + sum_j (i-j) P_ij z_j . t_i] + <St, c_out sum_i lambda^(i+1) x_i t_i^T>,
// every term a product that is there: the shorter identity through sum_t (q.dq - k.dk) cancels.
//
// Layout.  A wave keeps 32 columns of the state in its accumulators, where they are already the operand of
// S_0^T x (the contraction's order inside 16 is the accumulators' own, and x and y are read in it); scores
// are computed as y x^T, whose accumulators are the operand of the product with z.  Only x, y, z pass
// through LDS, y and z once more by transposing reads.  Computed operands are split into two bf16 planes
// where they end in a bf16 output and into three where they end in an fp32 one (state, log_decay).
// Chunks of 32 tokens: the scores of longer ones take more registers than two waves a SIMD have.
// Few memories: the token axis is cut into segments whose own sums (state pass: y and z once more) are
// scanned into start states, so that 512 workgroups fill the chip: two passes over memory, not one.
//
// Measured, bf16, 128 memories x 8192 tokens x 128 x 128, in one run: state pass 130 us, scan 18 us, outputs 291 us
// (1.07 GB at 3.7 TB/s), in a call of 446 us (435 to 459 in others).  Issue-bound: counters show the outputs kernel's
// vector instructions, the splits and masks first, in 42% and its matrix instructions in 32% of a SIMD's cycles.
// Training, 64 memories x 4096 x 64 x 128: 428 to 447 us, of which the tangent's kernel takes 146 (the outputs'
// tangents as rows of their own, St split into planes: 165).
// One token, 1024 memories x 128 x 128: 29 us, 135 MB at 4.7 TB/s (copies reach 4.8 to 5.6).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "mfma_tiles.h"

namespace am {

namespace {

constexpr int kC = 32;          // tokens per chunk: one 32-row matrix-core tile

struct LaRows {                 // a [B, H, T, w] tensor of either layout
  const void* p;
  int64_t sb, sh, st;           // element strides of b, h, t
  int w;
  int vec, vec4;                // rows are whole, aligned pieces of 16 bytes; of four elements
};

struct LaArgs {
  LaRows x, y, z, o;            // o: the output rows (z.w wide)
  LaRows t;                     // the rows that the tangent's outputs are multiplied with
  const float* log_decay;       // [H]
  const int32_t* len;           // [B] or null
  const float* s0;              // start states, or null (zeros)
  float* sT;                    // final states, or null
  const float* t0;              // tangent's start states (nseg > 1), or null (zeros)
  const float* adj;             // tangent: dW_T, or null
  double* dec;                  // tangent: one sum for each (memory, segment, column block, wave)
  float* u;                     // state pass: segment s's own sum goes to slot s + 1
  float* ut;                    // ... and its tangent's
  int64_t T;
  int64_t lseg;                 // tokens of a segment (a multiple of kC)
  int H, nseg;
  int ssx, ssz;                 // element strides of a state's x and z index
  int64_t P;                    // elements of a state
  int svec;                     // states are whole, aligned 16-byte pieces
  float c_out, c_upd;
  int e, rev;
};

// lambda^n
__device__ __forceinline__ float decay_pow(float g, int64_t n) { return n <= 0 ? 1.0f : expf((float)n * g); }

// An operand in N bf16 planes, x = p[0] + p[1] + p[2] (8 significant bits each).
template <int N>
struct Op {
  u32x4 p[N];
};

// WIDE: of fp32 values, whose largest ones would round to an infinity: the first plane stops at bf16's largest,
// and the others take the rest (a NaN stays in them).
template <bool WIDE, int N>
__device__ __forceinline__ void split8(const float* v, Op<N>& o) {
  constexpr float kMost = 0x1.FEp127f;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool stop = WIDE && n == 0;
      const float a = stop ? __builtin_amdgcn_fmed3f(r[2 * i], -kMost, kMost) : r[2 * i];
      const float b = stop ? __builtin_amdgcn_fmed3f(r[2 * i + 1], -kMost, kMost) : r[2 * i + 1];
      const uint32_t w = cvt_pk_bf16(a, b);
      o.p[n][i] = w;
      if (n + 1 < N) {
        r[2 * i] -= __uint_as_float(w << 16);
        r[2 * i + 1] -= __uint_as_float(w & 0xFFFF0000u);
      }
    }
}

template <int N>
__device__ __forceinline__ void join8(const Op<N>& o, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int n = N - 1; n >= 0; --n) {
      const uint32_t w = o.p[n][i >> 1];
      v[i] += __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
  }
}

// Products of planes down to 2^-16 of the leading one: the rest is below fp32's rounding.
template <int NA, int NB>
__device__ __forceinline__ f32x16 mm(const Op<NA>& a, const Op<NB>& b, f32x16 c) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = mfma32(a.p[i], b.p[s - i], c);
  return c;
}

// The rows of a chunk in memory: a buffer from its first token on, rows behind the sequence out of range
// (they read as zeros).  A lane's offset of position i is row_off, less `adj` where positions run
// backwards and the chunk is short.
struct ChunkRows {
  rsrc_t r;
  uint32_t adj;
};
__device__ __forceinline__ ChunkRows chunk_rows(const LaRows& t, int64_t at, int64_t first, int rows, int el, int rev) {
  const uint32_t step = (uint32_t)t.st * el;
  ChunkRows c;
  c.r = make_rsrc((const char*)t.p + (at + first * t.st) * el, rows > 0 ? (rows - 1) * step + (uint32_t)t.w * el : 0u);
  c.adj = rev ? (uint32_t)(kC - rows) * step : 0u;
  return c;
}
constexpr uint32_t kNoRow = 0xC0000000u;  // behind any buffer (rows of a chunk span less than 2^30 bytes)
__device__ __forceinline__ uint32_t row_off(const LaRows& t, int row, int c, int el, int rev) {
  return c < t.w ? (uint32_t)(rev ? kC - 1 - row : row) * (uint32_t)(t.st * el) + (uint32_t)c * el : kNoRow;
}

// Eight consecutive elements of a row as read from memory.
template <bool F32>
struct Raw {
  u32x4 a[F32 ? 2 : 1];
};
// VEC: whole, aligned pieces; else element by element, `left` of them inside the row.
template <bool F32, bool VEC>
__device__ __forceinline__ Raw<F32> load_group(const ChunkRows& c, uint32_t off, int left) {
  Raw<F32> g;
  const uint32_t o = off - c.adj;
  if constexpr (VEC) {
    g.a[0] = buf_ld16(c.r, (int)o, 0);
    if constexpr (F32) g.a[1] = buf_ld16(c.r, left > 4 ? (int)(o + 16) : -1, 0);
  } else {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) g.a[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (F32) g.a[i >> 2][i & 3] = __float_as_uint(buf_ld(c.r, i < left ? (int)(o + 4 * i) : -1, 0));
      else g.a[0][i >> 1] |= buf_ld_u16(c.r, i < left ? (int)(o + 2 * i) : -1, 0) << (16 * (i & 1));
    }
  }
  return g;
}

// Whether a group holds a NaN or an infinity.
template <bool F32>
__device__ __forceinline__ bool any_unbounded(const Raw<F32>& g) {
  if constexpr (F32) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += 0.0f * __uint_as_float(g.a[i >> 2][i & 3]);
    return t != t;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 t = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, g.a[0][i] | 0x80008000u));
    return t[0] >= 0xFF80u || t[1] >= 0xFF80u;
  }
}
// LDS tile of a chunk: 32 rows of W (64 or 128) elements, the 8-byte pieces of a row exchanged by bits of
// its index so that both reads below touch every bank once: 32 rows at one column piece, and 4 rows at
// 8 neighbouring pieces.
template <int W>
__device__ __forceinline__ constexpr int exchange(int row) {
  return W == 128 ? ((row & 3) << 3) | ((row >> 2) & 7) : (((row >> 1) & 1) << 3) | ((row >> 2) & 7);
}
// Eight elements (column c, a multiple of 8) of a row into a tile of planes.
template <int W, bool F32>
__device__ __forceinline__ void store_group(uint16_t* s, int row, int c, const Raw<F32>& g) {
  const int f = exchange<W>(row);
  uint16_t *lo = s + row * W + (((c >> 2) ^ f) << 2), *hi = s + row * W + ((((c >> 2) | 1) ^ f) << 2);
  auto put = [&](int at, u32x4 v) {
    *(uint2*)(lo + at) = uint2{v[0], v[1]};
    *(uint2*)(hi + at) = uint2{v[2], v[3]};
  };
  if constexpr (F32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(g.a[i >> 2][i & 3]);
    Op<3> o;
    split8<F32>(v, o);
#pragma unroll
    for (int n = 0; n < 3; ++n) put(n * kC * W, o.p[n]);
  } else {
    put(0, g.a[0]);
  }
}

// Takes a group's elements that are no finite numbers out of a tile (they show in its last plane), and notes the
// smallest position of each column's, and that there is one.  In pieces of four, as store_group writes them.
template <int W, int NP>
__device__ __forceinline__ void note_unbounded(uint16_t* s, int row, int c, int* from, int* any, int position) {
  *any = 1;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint16_t* piece = s + row * W + ((((c >> 2) | h) ^ exchange<W>(row)) << 2);
    const uint2 w = *(const uint2*)(piece + (NP - 1) * kC * W);
    uint32_t lo = 0xFFFFFFFFu, hi = 0xFFFFFFFFu;  // what stays
    auto look = [&](uint32_t pair, uint32_t exponent, uint32_t& keep, int i) {
      if ((pair & exponent) != exponent) return;
      keep &= exponent > 0xFFFFu ? 0x0000FFFFu : 0xFFFF0000u;
      atomicMin(from + c + 4 * h + i, position);
    };
    look(w.x, 0x7F80u, lo, 0);
    look(w.x, 0x7F800000u, lo, 1);
    look(w.y, 0x7F80u, hi, 2);
    look(w.y, 0x7F800000u, hi, 3);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      uint2* p = (uint2*)(piece + n * kC * W);
      *p = uint2{p->x & lo, p->y & hi};
    }
  }
}

// A row operand: lane l takes row l % 32 and, of every 16 columns, those that an accumulator tile
// has in its registers (4 (l / 32) + {0..3, 8..11}).  at: row_at of the lane.
template <int W>
__device__ __forceinline__ int row_at(int lane) {
  return (lane & 31) * W + (((lane >> 5) ^ exchange<W>(lane & 31)) << 2);
}
template <int W, int NP>
__device__ __forceinline__ Op<NP> row_op(const uint16_t* s, int at, int k) {
  Op<NP> o;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const uint16_t* p = s + n * kC * W;
    o.p[n] = cat2(*(const uint2*)(p + (at ^ (16 * k))), *(const uint2*)(p + (at ^ (16 * k + 8))));
  }
  return o;
}
// A column operand: lane l takes column c0 + l % 32 and the rows 16 k + .. in the same order.  at: col_at.
template <int W>
__device__ __forceinline__ int col_at(int lane) {
  const int row = 4 * (lane >> 5) + ((lane & 15) >> 2);
  return row * W + ((((lane & 16) >> 2) + (lane & 3)) ^ exchange<W>(row)) * 4;
}
template <int W, int NP>
__device__ __forceinline__ Op<NP> col_op(const uint16_t* s, int at, int c0, int k) {
  constexpr int kRow8 = exchange<W>(8), kRow16 = exchange<W>(16);
  const int x = ((c0 >> 2) ^ (k ? kRow16 : 0)) * 4;
  Op<NP> o;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const uint16_t* p = s + n * kC * W + 16 * k * W;
    o.p[n] = cat2(lds_tr16(p + (at ^ x)), lds_tr16(p + 8 * W + (at ^ (x ^ (kRow8 * 4)))));
  }
  return o;
}

// DX: 32-column tiles of x and y; NW: waves side by side, each with 32 columns of z; XS: waves that share
// those columns, each with a part of x.  Everything is linear in the parts of x (scores, state, outputs),
// so a wave carries its own part through and only the outputs are added, a chunk later, through LDS.
// VEC: rows are whole, aligned pieces; OUT: outputs (else the segment's own state alone); DEC: the tangent.
// Two waves a SIMD where their registers suffice (prompt kernel, 128 x 128: 325 us against 383).
template <int DX, int NW, int XS, bool F32, bool VEC, bool OUT, bool DEC>
__global__ __launch_bounds__(NW * XS * 64, DEC || F32 || !VEC ? 1 : 2) void la_chunk(LaArgs a) {
  constexpr int NP = F32 ? 3 : 1;                    // planes of an input
  constexpr int NC = F32 || DEC ? 3 : 2;             // planes of a computed operand of the outputs
  constexpr int WX = DX * 32, WZ = NW * 32;
  constexpr int NT = NW * XS * 64, DW = DX / XS;     // threads; x tiles of a wave
  constexpr int GX = kC * DX * 4 / NT, GZ = kC * NW * 4 / NT;  // 8-element groups per thread
  // 16 bytes between the tiles: at whole multiples of 512 the compiler joins a read of x with one of y,
  // and takes the results apart again with moves
  constexpr int TX = NP * kC * WX + 8, TZ = NP * kC * WZ + 8;
  constexpr bool TAN = OUT && DEC;                   // the tangent's sums: t's rows too
  constexpr int kBuf = (OUT ? 2 : 1) * TX + (TAN ? 2 : 1) * TZ;
  constexpr int kBufs = F32 ? 1 : 2;
  // The next chunk's rows wait in registers where these have room: with the tangent, fp32 or unaligned rows would
  // spill (backward with them waiting and without: bf16 rows of 101 and 66 517 and 513 us, fp32 128 x 128 254,
  // with 180 bytes of scratch a lane, and 260).
  constexpr bool kAhead = !TAN || (VEC && !F32);
  extern __shared__ __attribute__((aligned(16))) uint16_t sm[];
  float* parts = (float*)(sm + kBufs * kBuf);        // outputs of the other parts of x: two chunks
  constexpr int kParts = OUT ? (XS - 1) * NW * 1024 : 0;
  float* pw = parts + 2 * kParts;                    // lambda^0 .. lambda^32
  // Outputs: a NaN or infinity of z would reach the positions before it in its chunk, through zeros of the
  // scores.  It does not enter the tiles: its column is NaN from its position on, the first of which is kept here.
  int* from = (int*)(pw + kC + 4);                   // [WZ], and whether there is one

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hf = lane >> 5, col = lane & 31;
  const int nrun = OUT ? a.nseg : a.nseg - 1;        // the last segment's own sum starts nothing
  const int seg = blockIdx.x % nrun;
  const int m = blockIdx.x / nrun;
  const int b = m / a.H, h = m % a.H;
  const int z0 = blockIdx.y * WZ;
  const int zw = wave % NW, xs = __builtin_amdgcn_readfirstlane(wave / NW);
  const int zc = z0 + zw * 32;
  const int64_t len = a.len ? min((int64_t)max(a.len[b], 0), a.T) : a.T;
  const int64_t p0 = (int64_t)seg * a.lseg, p1 = min(p0 + a.lseg, a.T);
  const float g = a.log_decay[h];
  for (int i = tid; i <= kC; i += NT) pw[i] = decay_pow(g, i);
  if constexpr (OUT) {
    for (int i = tid; i <= WZ; i += NT) from[i] = i < WZ ? INT32_MAX : 0;
  }

  constexpr int EL = F32 ? 4 : 2;
  // of a chunk at position p: rows inside the sequence, and its first token in memory
  auto rows_at = [&](int64_t p) { return (int)max((int64_t)0, min((int64_t)kC, min(len, p1) - p)); };
  auto first_at = [&](int64_t p, int r) { return a.rev ? len - p - r : p; };
  const int64_t atx = b * a.x.sb + h * a.x.sh, atz = b * a.z.sb + h * a.z.sh;  // y lies like x, o and t like z

  // state tiles: column zc + col, rows 32 (xs DW + xt) + 8 q + 4 hf + u
  f32x16 S[DW], St[DEC ? DW : 1];
#pragma unroll
  for (int xt = 0; xt < DW; ++xt) {
    S[xt] = zero16();
    if constexpr (DEC) St[xt] = zero16();
  }
  const int64_t slot = (int64_t)m * a.nseg + seg;
  if constexpr (OUT) {
    auto get = [&](f32x16* D, const float* src) {
      if (!src || zc + col >= a.z.w) return;
      const float* p = src + slot * a.P + (int64_t)(zc + col) * a.ssz;
      if (a.svec && a.ssx == 1) {
#pragma unroll
        for (int xt = 0; xt < DW; ++xt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int x = 32 * (xs * DW + xt) + 8 * q + 4 * hf;
            if (x >= a.x.w) continue;
            const float4 f = *(const float4*)(p + x);
            D[xt][4 * q] = f.x, D[xt][4 * q + 1] = f.y, D[xt][4 * q + 2] = f.z, D[xt][4 * q + 3] = f.w;
          }
        return;
      }
#pragma unroll
      for (int xt = 0; xt < DW; ++xt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 32 * (xs * DW + xt) + 8 * (i >> 2) + 4 * hf + (i & 3);
          if (x < a.x.w) D[xt][i] = p[(int64_t)x * a.ssx];
        }
    };
    get(S, a.s0);
    if constexpr (DEC) get(St, a.t0);
  }

  Raw<F32> rx[OUT ? GX : 1], ry[GX], rz[GZ], rt[TAN ? GZ : 1];
  uint32_t ox[GX], oz[GZ];
#pragma unroll
  for (int i = 0; i < GX; ++i) {
    const int id = tid + i * NT;
    ox[i] = row_off(a.x, id / (DX * 4), (id % (DX * 4)) * 8, EL, a.rev);
  }
#pragma unroll
  for (int i = 0; i < GZ; ++i) {
    const int id = tid + i * NT;
    oz[i] = row_off(a.z, id / (NW * 4), z0 + (id % (NW * 4)) * 8, EL, a.rev);
  }
  auto fetch = [&](int64_t p) {
    const int r = rows_at(p);
    const int64_t t = first_at(p, r);
    const ChunkRows cx = chunk_rows(a.x, atx, t, r, EL, a.rev), cy = chunk_rows(a.y, atx, t, r, EL, a.rev),
                    cz = chunk_rows(a.z, atz, t, r, EL, a.rev);
#pragma unroll
    for (int i = 0; i < GX; ++i) {
      const int left = a.x.w - ((tid + i * NT) % (DX * 4)) * 8;
      if constexpr (OUT) rx[i] = load_group<F32, VEC>(cx, ox[i], left);
      ry[i] = load_group<F32, VEC>(cy, ox[i], left);
    }
#pragma unroll
    for (int i = 0; i < GZ; ++i)
      rz[i] = load_group<F32, VEC>(cz, oz[i], a.z.w - z0 - ((tid + i * NT) % (NW * 4)) * 8);
    if constexpr (TAN) {
      const ChunkRows ct = chunk_rows(a.t, atz, t, r, EL, a.rev);
#pragma unroll
      for (int i = 0; i < GZ; ++i)
        rt[i] = load_group<F32, VEC>(ct, oz[i], a.z.w - z0 - ((tid + i * NT) % (NW * 4)) * 8);
    }
  };
  auto stage = [&](uint16_t* s) {
#pragma unroll
    for (int i = 0; i < GX; ++i) {
      const int id = tid + i * NT, row = id / (DX * 4), c = (id % (DX * 4)) * 8;
      store_group<WX, F32>(s, row, c, ry[i]);
      if constexpr (OUT) store_group<WX, F32>(s + TX + TZ, row, c, rx[i]);
    }
#pragma unroll
    for (int i = 0; i < GZ; ++i) {
      const int id = tid + i * NT, row = id / (NW * 4), c = (id % (NW * 4)) * 8;
      store_group<WZ, F32>(s + TX, row, c, rz[i]);
      if constexpr (TAN) store_group<WZ, F32>(s + 2 * TX + TZ, row, c, rt[i]);
    }
  };
  double dec = 0.0;

  if constexpr (kAhead) fetch(p0);
  __syncthreads();
  // decay from position j (the register's) to i (the lane's), of the carried state, and to the chunk's end
  float D[OUT && !TAN ? 16 : 1], wz[16];
  const float wi = pw[col + 1 - a.e] * a.c_out;
  if constexpr (OUT && !TAN) {
#pragma unroll
    for (int n = 0; n < 16; ++n)
      D[n] = pw[max(col - (8 * (n >> 2) + 4 * hf + (n & 3)), 0)] * a.c_upd * a.c_out;
  }
  auto weights = [&](int r) {
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      const int j = 8 * (n >> 2) + 4 * hf + (n & 3);
      wz[n] = j < r ? pw[r - 1 - j + a.e] * a.c_upd : 0.0f;
    }
  };
  if constexpr (!TAN) weights(kC);
  const int part = 32 * DW * xs;                      // the wave's first x: bits of their own in an offset
  const int rat = row_at<WX>(lane) ^ part, cat = col_at<WX>(lane) ^ part, zat = col_at<WZ>(lane);
  const int tat = row_at<WZ>(lane) ^ (zw * 32);
  const int ci = col - 4 * hf;                        // i >= j: ci >= 8 (n / 4) + n % 4
  uint32_t oo[OUT ? 4 : 1];                           // the lane's output pieces
  if constexpr (OUT) {
#pragma unroll
    for (int q = 0; q < 4; ++q) oo[q] = row_off(a.o, col, zc + 8 * q + 4 * hf, EL, a.rev);
  }

  // The outputs of a chunk at p with r rows in the sequence: the lane's position, four consecutive columns a
  // register group; zeros behind the sequence.
  auto put_piece = [&](const ChunkRows& c, uint32_t off, const float* v, int left) {
    const uint32_t o = off - c.adj;
    if constexpr (F32) {
      if constexpr (VEC) {
        buf_st4(c.r, (int)o, 0, float4{v[0], v[1], v[2], v[3]});
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) buf_st(c.r, n < left ? (int)(o + 4 * n) : -1, 0, v[n]);
      }
    } else {
      const uint2 w = {cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
      if constexpr (VEC) {
        buf_st8(c.r, (int)o, 0, w);
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          buf_st_u16(c.r, n < left ? (int)(o + 2 * n) : -1, 0, (n & 2 ? w.y : w.x) >> (16 * (n & 1)));
      }
    }
  };
  auto put_rows = [&](const f32x16& V, int64_t p, int r) {
    const ChunkRows co = chunk_rows(a.o, atz, first_at(p, r), r, EL, a.rev);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v[4] = {V[4 * q], V[4 * q + 1], V[4 * q + 2], V[4 * q + 3]};
      put_piece(co, oo[q], v, a.z.w - zc - 8 * q - 4 * hf);
    }
    if (r < kC) {
      const int64_t behind = p + r;
      const ChunkRows ce = chunk_rows(a.o, atz, behind, (int)min((int64_t)(kC - r), p1 - behind), EL, 0);
      const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = zc + 8 * q + 4 * hf;
        put_piece(ce, row_off(a.o, col, c, EL, 0), none, a.z.w - c);
      }
    }
  };
  // XS > 1: the first part's outputs of the last chunk, waiting for the others'
  f32x16 Ow = zero16();
  int64_t pwait = -1;
  int rwait = 0;
  bool odd = false;                                   // which half of `parts` this chunk writes
  auto add_parts = [&](int half) {
    if (xs || pwait < 0) return;
#pragma unroll
    for (int t = 0; t < XS - 1; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = *(const float4*)(parts + half * kParts + q * 256 * NW * (XS - 1) +
                                          ((t * NW + zw) * 64 + lane) * 4);
        Ow[4 * q] += v.x, Ow[4 * q + 1] += v.y, Ow[4 * q + 2] += v.z, Ow[4 * q + 3] += v.w;
      }
    put_rows(Ow, pwait, rwait);
  };

  // One chunk; FULL: all its positions are inside the sequence (one block of code without branches, which
  // the scheduler can fill the waits of each part of with the others).
  // With the tangent the scheduler would move so much ahead that registers run out.
  auto hold = [&]() {
    if constexpr (TAN) __builtin_amdgcn_sched_barrier(0);
  };
  auto chunk = [&](auto full, int buf, int64_t p) {
    constexpr bool FULL = decltype(full)::value;
    uint16_t* sy = sm + buf * kBuf;
    const uint16_t *sz = sy + TX, *sx = sz + TZ, *st = sx + TX;
    if constexpr (!kAhead) fetch(p);
    if constexpr (kBufs == 1) __syncthreads();
    stage(sy);
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < GZ; ++i) {
        const int id = tid + i * NT, row = id / (NW * 4);
        if (any_unbounded(rz[i]))
          note_unbounded<WZ, NP>(sy + TX, row, (id % (NW * 4)) * 8, from, from + WZ, (int)(p - p0) + row);
      }
    }
    __syncthreads();
    if constexpr (kAhead) fetch(p + kC);
    if constexpr (OUT && XS > 1) {
      odd = !odd;
      add_parts(odd ? 0 : 1);
    }
    const int r = FULL ? kC : rows_at(p);

    Op<NP> zo[2];
    if constexpr (OUT) {
      f32x16 O = zero16(), P = zero16();
#pragma unroll
      for (int k = 0; k < 2 * DW; ++k) {
        const Op<NP> x = row_op<WX, NP>(sx, rat, k), y = row_op<WX, NP>(sy, rat, k);
        P = mm(y, x, P);
        Op<NC> s;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = S[k >> 1][8 * (k & 1) + i];
        split8<F32>(v, s);
        O = mm(s, x, O);
        hold();
      }
      int cj = ci;
      if constexpr (TAN) asm volatile("" : "+v"(cj));  // else the loop keeps 16 registers of counts
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        O[n] *= wi;
        const int ij = cj - (8 * (n >> 2) + (n & 3));
        P[n] = ij >= 0 ? P[n] * (TAN ? pw[max(ij, 0)] * a.c_upd * a.c_out : D[n]) : 0.0f;
      }
      if constexpr (DEC) {
        // t_i . (dO_i / dlog lambda), summed over i: (i + 1) t_i . O_i of the state before the chunk,
        // sum_j (i - j) P_ij z_j . t_i, and <St, sum_i lambda^(i+1) x_i t_i^T>
        float inter = 0.0f, rest = 0.0f;
        f32x16 R = zero16();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const Op<NP> to = row_op<WZ, NP>(st, tat, k);
          R = mm(row_op<WZ, NP>(sz, tat, k), to, R);
          float v[8];
          join8(to, v);
#pragma unroll
          for (int n = 0; n < 8; ++n) inter += v[n] * O[8 * k + n];
          hold();
        }
#pragma unroll
        for (int n = 0; n < 16; ++n) rest += (float)(cj - (8 * (n >> 2) + (n & 3))) * P[n] * R[n];
        rest += (float)(col + 1) * inter;
        hold();
        Op<3> wt[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[8];
          join8(col_op<WZ, NP>(st, zat, zw * 32, k), v);
#pragma unroll
          for (int n = 0; n < 8; ++n)  // lambda^(i+1) of the register's position
            v[n] *= pw[16 * k + 8 * (n >> 2) + 4 * hf + (n & 3) + 1 - a.e] * a.c_out;
          split8<F32>(v, wt[k]);
        }
        hold();
#pragma unroll
        for (int xt = 0; xt < DW; ++xt) {
          f32x16 X = zero16();
#pragma unroll
          for (int k = 0; k < 2; ++k) X = mm(col_op<WX, NP>(sx, cat, 32 * xt, k), wt[k], X);
#pragma unroll
          for (int n = 0; n < 16; ++n) rest += St[xt][n] * X[n];
          hold();
        }
        dec += rest;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        zo[k] = col_op<WZ, NP>(sz, zat, zw * 32, k);
        float v[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) v[n] = P[8 * k + n];
        Op<NC> s;
        split8<F32>(v, s);
        O = mm(zo[k], s, O);
        hold();
      }
      if (__builtin_amdgcn_readfirstlane(from[WZ])) {
#pragma unroll
        for (int n = 0; n < 16; ++n)
          if ((int)(p - p0) + col >= from[zw * 32 + 8 * (n >> 2) + 4 * hf + (n & 3)]) O[n] = __builtin_nanf("");
      }
      if constexpr (XS == 1) {
        put_rows(O, p, r);
      } else if (xs) {
        float* d = parts + (odd ? kParts : 0) + (((xs - 1) * NW + zw) * 64 + lane) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(float4*)(d + q * 256 * NW * (XS - 1)) = float4{O[4 * q], O[4 * q + 1], O[4 * q + 2], O[4 * q + 3]};
      } else {
        Ow = O, pwait = p, rwait = r;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) zo[k] = col_op<WZ, NP>(sz, zat, zw * 32, k);
    }

    // state: column operands of y times the weighted z (three planes: the state is an fp32 result)
    if constexpr (!FULL || TAN) weights(r);
    int rj = r - 1 - 4 * hf;
    if constexpr (TAN) asm volatile("" : "+v"(rj));
    const float keep = pw[r];
#pragma unroll
    for (int xt = 0; xt < DW; ++xt)
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        if constexpr (DEC) St[xt][n] = keep * (St[xt][n] + (float)r * S[xt][n]);
        S[xt][n] *= keep;
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8];
      join8(zo[k], v);
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] *= wz[8 * k + n];
      Op<3> s, sd;
      split8<F32>(v, s);
      if constexpr (DEC) {
#pragma unroll
        for (int n = 0; n < 8; ++n) v[n] *= (float)max(rj - (16 * k + 8 * (n >> 2) + (n & 3)), 0);
        split8<F32>(v, sd);
      }
#pragma unroll
      for (int xt = 0; xt < DW; ++xt) {
        const Op<NP> yo = col_op<WX, NP>(sy, cat, 32 * xt, k);
        hold();
        S[xt] = mm(yo, s, S[xt]);
        if constexpr (DEC) St[xt] = mm(yo, sd, St[xt]);
      }
    }
  };
  int64_t p = p0;
  int buf = 0;
  if constexpr (DEC || F32 || !VEC) {
    for (; p + kC <= min(len, p1); p += kC, buf ^= kBufs - 1) chunk(std::true_type{}, buf, p);
  } else {
    for (; p + 2 * kC <= min(len, p1); p += 2 * kC) {  // two, so that the buffers' addresses are constants
      chunk(std::true_type{}, 0, p);
      chunk(std::true_type{}, 1, p + kC);
    }
  }
  for (; p < p1; p += kC, buf ^= kBufs - 1) chunk(std::false_type{}, buf, p);
  if constexpr (OUT && XS > 1) {
    __syncthreads();
    add_parts(odd ? 1 : 0);
  }

  if constexpr (OUT) {
    __syncthreads();  // every chunk is staged
    if (from[zw * 32 + col] != INT32_MAX) {
#pragma unroll
      for (int xt = 0; xt < DW; ++xt)
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          S[xt][n] = __builtin_nanf("");
          if constexpr (DEC) St[xt][n] = __builtin_nanf("");
        }
    }
    if (DEC && from[WZ]) dec = __builtin_nan("");
  }

  // the state out: C-layout tiles to the caller's order
  auto put = [&](const f32x16* V, float* dst) {
    if (zc + col >= a.z.w) return;
    float* o = dst + (int64_t)(zc + col) * a.ssz;
    if (a.svec && a.ssx == 1) {
#pragma unroll
      for (int xt = 0; xt < DW; ++xt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int x = 32 * (xs * DW + xt) + 8 * q + 4 * hf;
          if (x < a.x.w)
            *(float4*)(o + x) = float4{V[xt][4 * q], V[xt][4 * q + 1], V[xt][4 * q + 2], V[xt][4 * q + 3]};
        }
      return;
    }
#pragma unroll
    for (int xt = 0; xt < DW; ++xt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int x = 32 * (xs * DW + xt) + 8 * (i >> 2) + 4 * hf + (i & 3);
        if (x < a.x.w) o[(int64_t)x * a.ssx] = V[xt][i];
      }
  };
  if constexpr (OUT) {
    if (seg == a.nseg - 1) {
      if (a.sT) put(S, a.sT + (int64_t)m * a.P);
      if constexpr (DEC) {
        if (a.adj && zc + col < a.z.w) {
          const float* q = a.adj + (int64_t)m * a.P + (int64_t)(zc + col) * a.ssz;
#pragma unroll
          for (int xt = 0; xt < DW; ++xt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int x = 32 * (xs * DW + xt) + 8 * (i >> 2) + 4 * hf + (i & 3);
              if (x < a.x.w) dec += (double)St[xt][i] * q[(int64_t)x * a.ssx];
            }
        }
      }
    }
    if constexpr (DEC) {
#pragma unroll
      for (int s = 32; s; s >>= 1) dec += __shfl_xor(dec, s);
      if (lane == 0) a.dec[(slot * gridDim.y + blockIdx.y) * (NW * XS) + wave] = dec;
    }
  } else {
    put(S, a.u + (slot + 1) * a.P);
    if constexpr (DEC) put(St, a.ut + (slot + 1) * a.P);
  }
}

// Start states of the segments: slot 0 takes the initial state, slot s + 1 (holding segment s's own
// sum) its start state.  Tangent (ut != null): T' = lambda^n (T + n S) + U'.
__global__ void la_scan(const float* w0, float* u, float* ut, const float* log_decay, const int32_t* len, int H,
                        int64_t T, int64_t lseg, int nseg, int64_t P) {
  const int per = (int)((P + 255) / 256);  // workgroups of a memory
  const int64_t i = (int64_t)(blockIdx.x % per) * 256 + threadIdx.x;
  if (i >= P) return;
  const int m = blockIdx.x / per, b = m / H;
  const float g = log_decay[m % H];
  const int64_t n = len ? min((int64_t)max(len[b], 0), T) : T;
  float s = w0 ? w0[(int64_t)m * P + i] : 0.0f, t = 0.0f;
  float* p = u + (int64_t)m * nseg * P + i;
  float* pt = ut ? ut + (int64_t)m * nseg * P + i : nullptr;
  constexpr int kAhead = 8;  // segments whose sums are read before the chain of products uses them
  for (int k0 = 0; k0 < nseg; k0 += kAhead) {
    float v[kAhead], vt[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool in = k0 + k > 0 && k0 + k < nseg;
      v[k] = in ? p[(int64_t)(k0 + k) * P] : 0.0f;
      vt[k] = in && pt ? pt[(int64_t)(k0 + k) * P] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k >= nseg) break;
      if (k0 + k > 0) {
        const int64_t cnt = min(lseg, max((int64_t)0, n - (k0 + k - 1) * lseg));
        const float keep = decay_pow(g, cnt);
        t = keep * (t + (float)cnt * s) + vt[k];
        s = keep * s + v[k];
      }
      p[(int64_t)(k0 + k) * P] = s;
      if (pt) pt[(int64_t)(k0 + k) * P] = t;
    }
  }
}

// d log_decay[h]: the waves' sums of every memory of the head, in one order.
__global__ void la_decay_sum(const double* dec, int B, int H, int per, float* out) {
  __shared__ double s[256];
  const int h = blockIdx.x;
  double v = 0.0;
  for (int i = threadIdx.x; i < B * per; i += 256) v += dec[((int64_t)(i / per) * H + h) * per + i % per];
  s[threadIdx.x] = v;
  __syncthreads();
  for (int k = 128; k; k >>= 1) {
    if ((int)threadIdx.x < k) s[threadIdx.x] += s[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[h] = (float)s[0];
}

// The recurrence for a few tokens: LPR lanes of a row of W hold four columns each, RPT rows a thread.
template <int LPR, bool F32>
__global__ __launch_bounds__(256) void la_step(LaArgs a) {
  constexpr int RPT = 4, RPB = 256 / LPR * RPT;
  const int m = blockIdx.x, b = m / a.H, h = m % a.H;
  const int lr = threadIdx.x % LPR, r0 = blockIdx.y * RPB + threadIdx.x / LPR;
  const int dk = a.x.w, dv = a.z.w, c = 4 * lr;
  const int len = a.len ? min(max(a.len[b], 0), (int)a.T) : (int)a.T;
  const bool vec = a.svec;
  float W[RPT][4];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int row = r0 + i * (256 / LPR);
#pragma unroll
    for (int n = 0; n < 4; ++n) W[i][n] = 0.0f;
    if (a.s0 && row < dv && c < dk) {
      const float* p = a.s0 + (int64_t)m * a.P + (int64_t)row * dk + c;
      if (vec) {
        const float4 f = *(const float4*)p;
        W[i][0] = f.x, W[i][1] = f.y, W[i][2] = f.z, W[i][3] = f.w;
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (c + n < dk) W[i][n] = p[n];
      }
    }
  }
  // a token's elements: the next ones are on their way while these are used
  const bool whole = dk % 4 == 0 && a.x.vec4 && a.y.vec4;
  float nq[4], nk[4], nv[RPT];
  auto fetch = [&](int t) {
#pragma unroll
    for (int n = 0; n < 4; ++n) nq[n] = nk[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) nv[i] = 0.0f;
    if (t >= len) return;
    const int64_t aq = b * a.x.sb + h * a.x.sh + t * a.x.st + c, ak = b * a.y.sb + h * a.y.sh + t * a.y.st + c;
    const int64_t av = b * a.z.sb + h * a.z.sh + t * a.z.st;
    if (c < dk) {
      if (whole && F32) {
        const float4 q = *(const float4*)((const float*)a.x.p + aq), k = *(const float4*)((const float*)a.y.p + ak);
        nq[0] = q.x, nq[1] = q.y, nq[2] = q.z, nq[3] = q.w;
        nk[0] = k.x, nk[1] = k.y, nk[2] = k.z, nk[3] = k.w;
      } else if (whole) {
        const uint2 q = *(const uint2*)((const uint16_t*)a.x.p + aq), k = *(const uint2*)((const uint16_t*)a.y.p + ak);
        nq[0] = bf16_value(q.x & 0xFFFFu), nq[1] = __uint_as_float(q.x & 0xFFFF0000u);
        nq[2] = bf16_value(q.y & 0xFFFFu), nq[3] = __uint_as_float(q.y & 0xFFFF0000u);
        nk[0] = bf16_value(k.x & 0xFFFFu), nk[1] = __uint_as_float(k.x & 0xFFFF0000u);
        nk[2] = bf16_value(k.y & 0xFFFFu), nk[3] = __uint_as_float(k.y & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (c + n < dk) {
            nq[n] = load_in(a.x.p, aq + n, !F32);
            nk[n] = load_in(a.y.p, ak + n, !F32);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = r0 + i * (256 / LPR);
      if (row < dv) nv[i] = load_in(a.z.p, av + row, !F32);
    }
  };
  fetch(0);
  const float lam = decay_pow(a.log_decay[h], 1);
  for (int t = 0; t < (int)a.T; ++t) {
    const bool live = t < len;
    float q[4], k[4], vs[RPT];
#pragma unroll
    for (int n = 0; n < 4; ++n) q[n] = nq[n], k[n] = nk[n];
#pragma unroll
    for (int i = 0; i < RPT; ++i) vs[i] = nv[i];
    if (t + 1 < (int)a.T) fetch(t + 1);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = r0 + i * (256 / LPR);
      float y = 0.0f;
      if (live) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          W[i][n] = lam * W[i][n] + vs[i] * k[n];
          y += W[i][n] * q[n];
        }
      }
#pragma unroll
      for (int s = LPR / 2; s; s >>= 1) y += __shfl_xor(y, s);
      if (lr == 0 && row < dv) {
        const int64_t at = b * a.o.sb + h * a.o.sh + t * a.o.st + row;
        y = live ? y * a.c_out : 0.0f;
        if constexpr (F32) ((float*)a.o.p)[at] = y;
        else ((uint16_t*)a.o.p)[at] = (uint16_t)bf16_bits(y);
      }
    }
  }
  if (!a.sT) return;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int row = r0 + i * (256 / LPR);
    if (row < dv && c < dk) {
      float* p = a.sT + (int64_t)m * a.P + (int64_t)row * dk + c;
      if (vec) {
        *(float4*)p = float4{W[i][0], W[i][1], W[i][2], W[i][3]};
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (c + n < dk) p[n] = W[i][n];
      }
    }
  }
}

LaRows rows_of(const void* p, const LinAttn& s, int w) {
  LaRows r;
  r.p = p;
  r.w = w;
  if (s.tokens_first) {
    r.sb = s.T * s.H * (int64_t)w, r.sh = w, r.st = (int64_t)s.H * w;
  } else {
    r.sb = s.H * s.T * (int64_t)w, r.sh = s.T * (int64_t)w, r.st = w;
  }
  r.vec = ((uintptr_t)p & 15) == 0 && w % (s.bf16 ? 8 : 4) == 0;
  r.vec4 = ((uintptr_t)p & (s.bf16 ? 7 : 15)) == 0 && w % 4 == 0;
  return r;
}

int tiles(int w) { return w <= 64 ? 2 : 4; }
int waves(int w) { return w <= 64 ? 2 : 4; }
// A wide x over a narrow z: two waves share a column tile, so that four fill a CU's SIMDs and keep under
// 256 registers (64 memories, 4096 tokens, 128 over 64: 60 us against 71); with the tangent they need
// more all the same, and one alone is faster (177 us against 226).
constexpr int parts_of_x(int dx, int nw, bool tangent) { return dx == 4 && nw == 2 && !tangent ? 2 : 1; }

template <int DX, int NW, int XS, bool F32, bool VEC, bool OUT, bool DEC>
atlasmem_status chunk_launch(const LaArgs& a, int64_t blocks, hipStream_t st) {
  constexpr int NP = F32 ? 3 : 1;
  constexpr int lds = (F32 ? 1 : 2) * 2 * (kC * NP * ((OUT ? 2 : 1) * DX * 32 + (OUT && DEC ? 2 : 1) * NW * 32) + 32) +
                      4 * (kC + 4) + (OUT ? 4 * (NW * 32 + 4) + 8 * (XS - 1) * NW * 1024 : 0);
  auto kern = la_chunk<DX, NW, XS, F32, VEC, OUT, DEC>;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return ATLASMEM_E_DEVICE;
  const dim3 grid((unsigned)blocks, (unsigned)((a.z.w + NW * 32 - 1) / (NW * 32)));
  kern<<<grid, NW * XS * 64, lds, st>>>(a);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

template <bool F32, bool VEC, bool OUT, bool DEC>
atlasmem_status chunk_pick(const LaArgs& a, int64_t blocks, hipStream_t st) {
  const int dx = tiles(a.x.w), nw = waves(a.z.w);
  if (dx == 2)
    return nw == 2 ? chunk_launch<2, 2, 1, F32, VEC, OUT, DEC>(a, blocks, st)
                   : chunk_launch<2, 4, 1, F32, VEC, OUT, DEC>(a, blocks, st);
  return nw == 2 ? chunk_launch<4, 2, parts_of_x(4, 2, OUT && DEC), F32, VEC, OUT, DEC>(a, blocks, st)
                 : chunk_launch<4, 4, parts_of_x(4, 4, OUT && DEC), F32, VEC, OUT, DEC>(a, blocks, st);
}

template <bool OUT>
atlasmem_status chunk_run(const LaArgs& a, bool bf16, bool dec, int64_t M, hipStream_t st) {
  const int64_t blocks = M * (OUT ? a.nseg : a.nseg - 1);
  const bool vec = a.x.vec && a.y.vec && a.z.vec && (!OUT || (a.o.vec && (!dec || a.t.vec)));
  if (bf16) {
    if (vec)
      return dec ? chunk_pick<false, true, OUT, true>(a, blocks, st)
                 : chunk_pick<false, true, OUT, false>(a, blocks, st);
    return dec ? chunk_pick<false, false, OUT, true>(a, blocks, st)
               : chunk_pick<false, false, OUT, false>(a, blocks, st);
  }
  if (vec)
    return dec ? chunk_pick<true, true, OUT, true>(a, blocks, st) : chunk_pick<true, true, OUT, false>(a, blocks, st);
  return dec ? chunk_pick<true, false, OUT, true>(a, blocks, st) : chunk_pick<true, false, OUT, false>(a, blocks, st);
}

// Segments of the token axis: enough workgroups to fill the chip several times where the memories
// alone do not, none shorter than two chunks (1 x 1 x 1000 x 128 in fp32 forward 43 us, 56 at four chunks, 84
// at eight; 24 memories x 1999 tokens x 64 in fp32 49, 53, 62; 64 x 1024 x 64 x 128 in bf16 49, 49, 42; each
// 5 to 10 us less since states whose rows are consecutive move in 16-byte pieces).
int segments(const LinAttn& s, int64_t& lseg) {
  const int64_t chunks = std::max<int64_t>((s.T + kC - 1) / kC, 1);
  const int64_t M = (int64_t)s.B * s.H;
  int64_t n = std::min<int64_t>((512 + M - 1) / M, (chunks + 1) / 2);
  const int64_t per = (chunks + n - 1) / n;
  lseg = per * kC;
  return (int)((chunks + per - 1) / per);
}

LaArgs base_args(const LinAttn& s) {
  LaArgs a = {};
  a.log_decay = s.log_decay;
  a.len = s.lengths;
  a.T = s.T;
  a.H = s.H;
  a.P = (int64_t)s.dk * s.dv;
  a.nseg = segments(s, a.lseg);
  a.c_out = 1.0f, a.c_upd = 1.0f;
  return a;
}

atlasmem_status run_scan(const LaArgs& a, const float* w0, float* u, float* ut, int64_t M, hipStream_t st) {
  la_scan<<<(unsigned)(M * ((a.P + 255) / 256)), 256, 0, st>>>(w0, u, ut, a.log_decay, a.len, a.H, a.T, a.lseg,
                                                               a.nseg, a.P);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }

}  // namespace

int64_t linear_attention_workspace_bytes(const LinAttn& s, bool backward) {
  int64_t lseg;
  const int64_t M = (int64_t)s.B * s.H, P = (int64_t)s.dk * s.dv, nseg = segments(s, lseg);
  const int64_t states = nseg > 1 ? align256(4 * M * nseg * P) : 0;
  if (!backward) return s.T <= kLinAttnStepTokens ? 0 : states;
  return 2 * states + align256(8 * M * nseg * 4);
}

atlasmem_status linear_attention(const LinAttn& s, const void* Q, const void* K, const void* V, float scale,
                                 const float* W0, float* WT, void* Y, void* workspace, hipStream_t st) {
  LaArgs a = base_args(s);
  const int64_t M = (int64_t)s.B * s.H;
  a.x = rows_of(Q, s, s.dk), a.y = rows_of(K, s, s.dk), a.z = rows_of(V, s, s.dv), a.o = rows_of(Y, s, s.dv);
  a.c_out = scale;
  a.ssx = 1, a.ssz = s.dk;
  a.s0 = W0, a.sT = WT;
  a.svec = s.dk % 4 == 0 && (((uintptr_t)W0 | (uintptr_t)WT) & 15) == 0;
  if (s.T <= kLinAttnStepTokens) {
    const int lpr = s.dk <= 32 ? 8 : s.dk <= 64 ? 16 : 32;
    const dim3 grid((unsigned)M, (unsigned)((s.dv + 1024 / lpr - 1) / (1024 / lpr)));
    if (s.bf16) {
      if (lpr == 8) la_step<8, false><<<grid, 256, 0, st>>>(a);
      else if (lpr == 16) la_step<16, false><<<grid, 256, 0, st>>>(a);
      else la_step<32, false><<<grid, 256, 0, st>>>(a);
    } else {
      if (lpr == 8) la_step<8, true><<<grid, 256, 0, st>>>(a);
      else if (lpr == 16) la_step<16, true><<<grid, 256, 0, st>>>(a);
      else la_step<32, true><<<grid, 256, 0, st>>>(a);
    }
    AM_LAUNCH_CHECK();
    return ATLASMEM_OK;
  }
  if (a.nseg > 1) {
    a.u = (float*)workspace;
    atlasmem_status e = chunk_run<false>(a, s.bf16, false, M, st);
    if (e == ATLASMEM_OK) e = run_scan(a, W0, a.u, nullptr, M, st);
    if (e != ATLASMEM_OK) return e;
    a.s0 = a.u;
  }
  return chunk_run<true>(a, s.bf16, false, M, st);
}

atlasmem_status linear_attention_backward(const LinAttn& s, const void* Q, const void* K, const void* V, float scale,
                                          const float* W0, const void* dY, const float* dWT, void* dQ, void* dK,
                                          void* dV, float* dW0, float* dlog_decay, void* workspace, hipStream_t st) {
  const LaArgs base = base_args(s);
  const int64_t M = (int64_t)s.B * s.H;
  const int64_t states = base.nseg > 1 ? align256(4 * M * base.nseg * base.P) : 0;
  float* u = (float*)workspace;
  float* ut = (float*)((char*)workspace + states);
  double* dec = (double*)((char*)workspace + 2 * states);
  const bool want = dlog_decay != nullptr;
  atlasmem_status e = ATLASMEM_OK;

  // dq (and the tangent's share): forward over (v, k)
  LaArgs a = base;
  a.x = rows_of(dY, s, s.dv), a.y = rows_of(V, s, s.dv), a.z = rows_of(K, s, s.dk), a.o = rows_of(dQ, s, s.dk);
  a.t = rows_of(Q, s, s.dk);
  a.ssx = s.dk, a.ssz = 1;
  a.c_out = scale;
  a.s0 = W0;
  a.adj = dWT;
  a.dec = dec;
  if (a.nseg > 1) {
    a.u = u, a.ut = ut;
    e = chunk_run<false>(a, s.bf16, want, M, st);
    if (e == ATLASMEM_OK) e = run_scan(a, W0, u, want ? ut : nullptr, M, st);
    if (e != ATLASMEM_OK) return e;
    a.s0 = u;
    a.t0 = want ? ut : nullptr;
  }
  e = chunk_run<true>(a, s.bf16, want, M, st);
  if (e != ATLASMEM_OK) return e;
  if (want) {
    const int nw = waves(s.dk);
    const int per = a.nseg * nw * parts_of_x(tiles(s.dv), nw, true) * ((s.dk + nw * 32 - 1) / (nw * 32));
    la_decay_sum<<<s.H, 256, 0, st>>>(dec, s.B, s.H, per, dlog_decay);
    AM_LAUNCH_CHECK();
  }

  // dk, dv: backwards over (q, dy)
  a = base;
  a.rev = 1, a.e = 1, a.c_upd = scale;
  a.x = rows_of(V, s, s.dv), a.y = rows_of(dY, s, s.dv), a.z = rows_of(Q, s, s.dk), a.o = rows_of(dK, s, s.dk);
  a.ssx = s.dk, a.ssz = 1;
  a.s0 = dWT;
  if (a.nseg > 1) {
    a.u = u;
    e = chunk_run<false>(a, s.bf16, false, M, st);
    if (e == ATLASMEM_OK) e = run_scan(a, dWT, u, nullptr, M, st);
    if (e != ATLASMEM_OK) return e;
    a.s0 = u;
  }
  e = chunk_run<true>(a, s.bf16, false, M, st);
  if (e != ATLASMEM_OK) return e;
  a.x = rows_of(K, s, s.dk), a.y = rows_of(Q, s, s.dk), a.z = rows_of(dY, s, s.dv), a.o = rows_of(dV, s, s.dv);
  a.ssx = 1, a.ssz = s.dk;
  a.sT = dW0;
  a.svec = s.dk % 4 == 0 && (((uintptr_t)dWT | (uintptr_t)dW0) & 15) == 0;
  return chunk_run<true>(a, s.bf16, false, M, st);
}

}  // namespace am
