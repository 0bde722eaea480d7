// Distillation from a teacher's top logits (gfx950).  The loss alone keeps no logits; a training step keeps G, [n][V].
//   z = X W^T,  p_i = softmax_j(scale t_ij) over the row's given classes,  q_i = softmax_v(scale z_iv)
//   loss_i = sum_j p_ij (log p_ij - log q_i,id_ij),  G_iv = q_iv - sum_{j: id_ij = v} p_ij
//   dX_i = scale dloss_i (G W)_i,  dW = G^T (scale dloss X)
// The forward computes z once.  For a training step its epilogue leaves exp(scale (z - ref)), with ref a logit of the
// row that is known beforehand, that of the teacher's first class: up to a factor c = exp(scale ref - lse) of the
// row this is q.  A workgroup for each row then joins the sums and writes G: the backward has two products, not
// three.  Rows whose ref is too far from their lse for a factor are computed again with lse for ref.
//
// bf16 calls leave those exponentials with ten significant bits (2^-10) and no sign, in the 16 bits that G (2^-8) then
// takes; the given classes' entries come from their logits in 64 bits, and have G's rounding alone.  c on X instead of
// G, without that pass, was one rounding more of a term of dW (33 x 256 x 1000: 2.8e-3 off instead of 2.3e-3).  fp32
// calls keep G / c, and the rows' weights take c.
//
// What bounds it: the matrix cores (8192 x 2048 x 65536 bf16, a tenth left out: 1.98 TFLOP a product.  z 1.92 ms, 1.03
// PFLOP/s, of which the stores of what is kept take 0.2 to 0.4, not overlapped with the next tile's products; dX 1.56,
// 1.27; dW 1.49, 1.33), beside them the rows' pass over G; few rows launches (33 x 256 x 1000: seven, 32 us a training
// pass).  Where every row's ref is far from its lse that is a product more, 8.4 ms a training pass instead of 5.6.
// Computing z again for the backward instead, a product more, takes 1.7 ms where what is kept costs its
// stores and the rows' pass, 0.7 to 0.9.
#include "logits.h"

namespace am {

namespace {

// how far (times log 2) ref may be from lse: 2^(kFar - kDown) has to stay below 2
constexpr float kFar = 36.0f;
constexpr int kMost = 128;  // entries of a row

// log p of each given class (-inf: none) and p, and of each row a label (0, or -1 for a row that has no class) and the
// logit of its first class.  With `index`, rows are taken as they come, those left out among them.  A wave a row: its
// waits for ids, and for a row of W that they name (8192 x 2048 18 us).
__global__ __launch_bounds__(256) void ds_teacher(const int64_t* ids, const float* teacher, int64_t n, int top,
                                                  int64_t vocab, float scale, const void* X, const void* W, int bf16,
                                                  int vec, int d, float* logp, float* prob, int64_t* label,
                                                  float* ref, int* again_count, int* index, int* at, int* count) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (again_count && r == 0 && lane == 0) *again_count = 0;
  if (count && r == 0 && lane == 0) *count = (int)n;
  if (r >= n) return;
  float t[2];
  int64_t id[2];
  bool on[2];
  float m = -INFINITY;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 64 * h;
    id[h] = j < top ? ids[r * top + j] : -1;
    t[h] = j < top ? teacher[r * top + j] : -INFINITY;
    on[h] = id[h] >= 0 && id[h] < vocab && !(t[h] == -INFINITY);
    if (on[h]) m = fmaxf(m, t[h]);
  }
  for (int k = 32; k; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
  float e[2], down[2], s = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // the difference is scaled: a logit times the scale need not be a float
    down[h] = on[h] ? (t[h] - m) * scale : -INFINITY;
    s += e[h] = expf(down[h]);
  }
  for (int k = 32; k; k >>= 1) s += __shfl_xor(s, k);
  const float ls = logf(s);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 64 * h < top) {
      // p not from log p, whose rounding would be one factor of the row's
      logp[r * top + lane + 64 * h] = on[h] ? down[h] - ls : -INFINITY;
      prob[r * top + lane + 64 * h] = on[h] ? e[h] / s : 0.0f;
    }
  const uint64_t any = __ballot(on[0] || on[1]);
  if (lane == 0) label[r] = any ? 0 : -1;
  if (index && lane == 0) index[r] = (int)r, at[r] = any ? (int)r : -1;
  if (!ref || !any) return;
  const uint64_t f0 = __ballot(on[0] && t[0] == m), f1 = __ballot(on[1] && t[1] == m);
  const int best = f0 ? __builtin_ctzll(f0) : f1 ? __builtin_ctzll(f1) : __builtin_ctzll(any);
  const bool low = f0 || (!f1 && (__ballot(on[0]) >> best & 1));
  const int64_t y = __shfl(low ? id[0] : id[1], best);
  float z = 0.0f;
  for (int c = lane * 8; c < d; c += 512) {
    if (vec && bf16) {
      const u32x4 a = *(const u32x4*)((const uint16_t*)X + r * d + c);
      const u32x4 b = *(const u32x4*)((const uint16_t*)W + y * d + c);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        z = fmaf(__uint_as_float(k & 1 ? a[k >> 1] & 0xFFFF0000u : a[k >> 1] << 16),
                 __uint_as_float(k & 1 ? b[k >> 1] & 0xFFFF0000u : b[k >> 1] << 16), z);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < d) z = fmaf(load_in(X, r * d + c + k, bf16), load_in(W, y * d + c + k, bf16), z);
    }
  }
  for (int k = 32; k; k >>= 1) z += __shfl_xor(z, k);
  if (lane == 0) ref[r] = fabsf(z) < 1.0e30f ? z : 0.0f;
}

struct JoinArgs {
  const float2* part;
  int parts;
  const int* at;           // a row's place among those that count, or null: all are there
  const void *x, *w;       // as the products took them, [..][dp]
  int dp;
  int64_t n;
  const int64_t *label, *ids;
  const float *logp, *prob;
  int top;
  float scale, k2, k2_low;
  float *loss, *lse;
  // a training step
  int all;                 // rows that are left out have a place, too
  float *ref, *coef, *factor;
  void* g;
  int64_t ldg;
  int *again, *to, *again_count;
  void* x_again;
};

// loss, lse of a row, and of a training step its G, in place.  Memory bounds it: it reads and writes what is kept (8192 x
// 2048 x 65536, a tenth left out: 1.9 GB, and 1.0 of the given classes' rows of W, in 455 us, 6.4 TB/s), or reads those
// rows out of L2 (2603 x 3352 x 479 with 128 entries: 2.2 GB, 9 TB/s).  A product's epilogue cannot write G, since a
// row's lse is known behind its last tile.  A workgroup a row, of
//   one wave, whose steps wait for no other, where many rows are short (bytes that it reads and writes; 12224 x 33 x 1135
//     training 153 -> 104 us, 2048 x 256 x 1024 63 -> 60; long rows take longer, 8192 x 2048 x 65536 6.05 -> 6.15 ms, and
//     few, 1024 x 256 x 1024 47 -> 49 us);
//   1024 threads where few rows have more entries than four waves take in two steps (33 x 3744 x 5000 with 128 the loss
//     alone 78 -> 55 us, 33 x 256 x 1000 with 20 training 34.6 -> 34.5; 600 x 512 x 9000 with 128: 112 -> 139);
//   256 else.
constexpr int64_t kManyRows = 2048, kShortRow = 32768;
template <int NT, bool BF16, bool TRAIN>
__global__ __launch_bounds__(NT) void ds_rows(JoinArgs a) {
  constexpr int NW = NT / 64;
  __shared__ float2 part[NW];
  __shared__ int id[kMost], list[kMost];
  __shared__ float p[kMost], lp[kMost];
  __shared__ double z[kMost];
  __shared__ int entries, slot;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    if (a.label[r] < 0) {
      if (tid == 0) a.loss[r] = 0.0f, a.lse[r] = 0.0f;
      if (TRAIN && tid == 0) a.coef[r] = 0.0f;
      if (TRAIN && a.all)
        for (int64_t c = tid; c < a.ldg * (BF16 ? 2 : 4) / 16; c += NT)
          ((u32x4*)((char*)a.g + r * a.ldg * (BF16 ? 2 : 4)))[c] = u32x4{0, 0, 0, 0};
      continue;
    }
    const int place = __builtin_amdgcn_readfirstlane(a.at ? a.at[r] : (int)r);
    __syncthreads();  // the last row's shared values have been read
    if (tid == 0) entries = 0;
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float om, float os) {
      const float t = fmaxf(m, om), from = t > -INFINITY ? t : 0.0f;
      s = s * __builtin_amdgcn_exp2f((m - from) * a.k2) + os * __builtin_amdgcn_exp2f((om - from) * a.k2);
      m = t;
    };
    for (int i = tid; i < a.parts; i += NT) {
      const float2 q = a.part[(int64_t)place * a.parts + i];
      join(q.x, q.y);
    }
    for (int k = 32; k; k >>= 1) {
      const float om = __shfl_xor(m, k), os = __shfl_xor(s, k);
      join(om, os);
    }
    if (lane == 0) part[wave] = float2{m, s};
    __syncthreads();
    for (int j = tid; j < a.top; j += NT) {
      const float l = a.logp[r * a.top + j];
      id[j] = (int)a.ids[r * a.top + j], lp[j] = l, p[j] = a.prob[r * a.top + j];
      if (!(l == -INFINITY)) list[atomicAdd(&entries, 1)] = j;
    }
    m = part[0].x, s = part[0].y;
#pragma unroll
    for (int w = 1; w < NW; ++w) join(part[w].x, part[w].y);
    const float log_s = logf(s), lse = fmaf(a.scale, m, log_s);
    __syncthreads();
    // logits of the given classes: short rows by some lanes each, others by a wave, two at a time
    const int bytes = a.dp * (BF16 ? 2 : 4);
    if (bytes <= kShort) {
      const int lanes = short_lanes(bytes);
      for (int i0 = 0; i0 < entries; i0 += NT / lanes) {
        const int i = i0 + tid / lanes, j = list[min(i, entries - 1)];
        const double v = short_dot<BF16>(a.x, a.w, place, id[j], bytes, lanes, lane);
        if ((lane & (lanes - 1)) == 0 && i < entries) z[j] = v;
      }
    } else {
      for (int i = 2 * wave; i < entries; i += 2 * NW) {
        const int j[2] = {__builtin_amdgcn_readfirstlane(list[i]),
                          __builtin_amdgcn_readfirstlane(list[min(i + 1, entries - 1)])};
        const int c[2] = {__builtin_amdgcn_readfirstlane(id[j[0]]), __builtin_amdgcn_readfirstlane(id[j[1]])};
        double v[2];
        row_dots<2, BF16>(a.x, a.w, place, c, a.dp, lane, v);
        if (lane < 2) z[lane ? j[1] : j[0]] = lane ? v[1] : v[0];
      }
    }
    __syncthreads();
    if (wave == 0) {
      float loss = 0.0f;
      for (int j = lane; j < a.top; j += 64) {
        // log p - log q without lse, whose rounding would be the largest
        if (p[j] != 0.0f) loss += p[j] * (lp[j] - (float)(a.scale * (z[j] - m)) + log_s);
      }
      for (int k = 32; k; k >>= 1) loss += __shfl_xor(loss, k);
      if (lane == 0) a.loss[r] = loss, a.lse[r] = lse;
    }
    if constexpr (TRAIN) {
      float ref = a.ref[r];
      const float l2 = __log2f(s);
      const bool near = fabsf((m - ref) * a.k2 + l2) <= kFar;
      if (!near) ref = m + l2 / a.k2;
      const float c = exp2_of(ref, m, a.k2, a.k2_low) / s;
      if (!near) {
        if (tid == 0) {
          slot = atomicAdd(a.again_count, 1);
          a.again[slot] = (int)r, a.to[slot] = place, a.factor[slot] = c, a.ref[r] = ref;
          a.coef[r] = a.scale;
        }
        __syncthreads();
        const int words = a.dp * (BF16 ? 2 : 4) / 16;
        for (int k = tid; k < words; k += NT)
          ((u32x4*)a.x_again)[(int64_t)slot * words + k] = ((const u32x4*)a.x)[(int64_t)place * words + k];
        continue;
      }
      if (tid == 0) a.coef[r] = BF16 ? a.scale : a.scale * c;
      if constexpr (BF16) {
        u32x4* row = (u32x4*)((uint16_t*)a.g + (int64_t)place * a.ldg);
        const float f = c * exp2f(kDown);
        const int words = (int)(a.ldg / 8);
        for (int k0 = tid; k0 < words; k0 += 4 * NT) {
          u32x4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k0 + NT * k < words) v[k] = row[k0 + NT * k];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[k][q] = cvt_pk_bf16(u16_lo(v[k][q]) * f, u16_hi(v[k][q]) * f);
            if (k0 + NT * k < words) row[k0 + NT * k] = v[k];
          }
        }
        __syncthreads();  // those are there before the given classes' entries
      }
      for (int j = tid; j < a.top; j += NT) {
        if (lp[j] == -INFINITY) continue;
        float sum = 0.0f;
        for (int i = 0; i < a.top; ++i) sum += id[i] == id[j] ? p[i] : 0.0f;
        const float q = exp2_of((float)z[j], ref, a.k2, a.k2_low);
        if (BF16) ((uint16_t*)a.g)[(int64_t)place * a.ldg + id[j]] = (uint16_t)bf16_bits(fmaf(q, c, -sum));
        else ((float*)a.g)[(int64_t)place * a.ldg + id[j]] = q - sum / c;
      }
    }
  }
}

// The weight of each row, coef dloss; of those that count the value that all have, or the largest finite magnitude,
// and which (one workgroup).
__device__ __forceinline__ void ds_weights(const float* coef, const float* dloss, const int* at, int64_t n, float* weight,
                                           float& scale, int& equal) {
  __shared__ float sm[16], from[16], to[16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  float m = 0.0f, lo = INFINITY, hi = -INFINITY;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const bool on = at[i] >= 0;
    const float w = on ? coef[i] * (dloss ? dloss[i] : 1.0f) : 0.0f;
    if (weight) weight[i] = w;
    if (!on) continue;
    m = fmaxf(m, fabsf(w) <= 3.0e38f ? fabsf(w) : 0.0f);
    lo = fminf(lo, w == w ? w : -INFINITY), hi = fmaxf(hi, w == w ? w : INFINITY);
  }
  for (int k = 32; k; k >>= 1) {
    m = fmaxf(m, __shfl_xor(m, k));
    lo = fminf(lo, __shfl_xor(lo, k)), hi = fmaxf(hi, __shfl_xor(hi, k));
  }
  if (lane == 0) sm[wave] = m, from[wave] = lo, to[wave] = hi;
  __syncthreads();
  for (int k = 0; k < waves; ++k) m = fmaxf(m, sm[k]), lo = fminf(lo, from[k]), hi = fmaxf(hi, to[k]);
  equal = lo >= hi;
  scale = lo == hi ? lo : m > 0.0f ? m : 1.0f;
}
__global__ __launch_bounds__(1024) void ds_scale(const float* coef, const float* dloss, const int* at, int64_t n,
                                                 float* weight, float* scale, int* equal) {
  float s;
  int e;
  ds_weights(coef, dloss, at, n, weight, s, e);
  if (threadIdx.x == 0) *scale = s, *equal = e;
}

// Up to so many rows each workgroup finds the weights by itself: a launch less (33 x 256 x 1000 34.7 -> 32.9 us; 1024 x
// 256 x 1024: 43.7 -> 45.2).
constexpr int64_t kFewRows = 512;

// The rows of X that have a place, times their weights over `scale` (where those are one value, as they are), zeros for
// rows that are left out; and zeros for the latter's dX, if it is given.  Four columns a thread.  Memory (8192 x 2048: 63
// MB in 23 us).
__global__ __launch_bounds__(256) void ds_weigh(const void* x, int bf16, int64_t n, int d, int dp, const int* at,
                                                int all, const float* coef, const float* dloss, float* weight,
                                                float* scale, int* equal, void* out, void* dx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = dp / 4, row = i / per;
  float over;
  int same;
  if (n <= kFewRows) {
    ds_weights(coef, dloss, at, n, blockIdx.x == 0 ? weight : nullptr, over, same);
    if (i == 0) *scale = over;
  } else {
    over = *scale, same = *equal;
  }
  if (row >= n) return;
  const int c = (int)(i % per) * 4;
  const int64_t place = all ? row : at[row];
  const bool on = at[row] >= 0;
  if (!on && dx)
    for (int k = 0; k < 4 && c + k < d; ++k) {
      if (bf16) ((uint16_t*)dx)[row * d + c + k] = 0;
      else ((float*)dx)[row * d + c + k] = 0.0f;
    }
  if (!out || place < 0) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (on && d % 4 == 0 && ((uintptr_t)x & 15) == 0 && c < d) {
    if (bf16) {
      const uint2 u = *(const uint2*)((const uint16_t*)x + row * d + c);
      v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
      v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
      const float4 u = *(const float4*)((const float*)x + row * d + c);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
  } else if (on) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k < d ? load_in(x, row * d + c + k, bf16) : 0.0f;
  }
  if (!same) {
    const float w = coef[row] * (dloss ? dloss[row] : 1.0f) / over;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = on ? v[k] * w : 0.0f;
  }
  const int64_t o = place * dp + c;
  if (bf16) *(uint2*)((uint16_t*)out + o) = uint2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
  else *(float4*)((float*)out + o) = float4{v[0], v[1], v[2], v[3]};
}

// The sums of the contraction's pieces: rows of a place (or all) times their weight, or one factor; zeros for the
// others.  Four columns a thread.
__global__ __launch_bounds__(256) void ds_sum(const float* acc, int splits, int64_t rows, int d, int dp, const int* at,
                                              const float* weight, const float* factor, void* out, int out_bf16, int vec) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / (dp / 4);
  const int c = (int)(i % (dp / 4)) * 4;
  if (r >= rows || c >= d) return;
  const int64_t place = at ? at[r] : r;
  float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (place >= 0) {
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const float4 a = *(const float4*)(acc + (s * rows + place) * dp + c);
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
  }
  const float w = place < 0 ? 0.0f : weight ? weight[r] : *factor;
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

struct Plan {
  int el, dp, side, parts, side_x, splits, side_w, splits_w;
  int64_t ldg;
  bool gather;
};
Plan plan_of(const Distillation& s, bool train) {
  Plan p = {};
  p.el = s.bf16 ? 2 : 4;
  p.dp = (int)up(s.d, s.bf16 ? 8 : 4);
  p.side = side_for(s.vocab, s.n, s.bf16);
  p.parts = (int)((s.vocab + p.side - 1) / p.side);
  p.ldg = up(s.vocab, 64);
  // dX is [n][d], of few tiles: V is cut so that they fill the chip, into pieces of 512 classes at least
  p.side_x = s.n <= kFew ? (s.bf16 ? 128 : 64) : side_split(p.dp, s.n, s.bf16);
  int64_t tiles = std::max<int64_t>(tiles_of(p.dp, s.n, p.side_x), 1);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>((p.side_x == 256 ? 256 : 512) / tiles, s.vocab / 512));
  if (tiles * p.splits <= 128) p.side_x = 64;
  p.side_w = side_of(p.dp, s.vocab, s.bf16);
  tiles = tiles_of(p.dp, s.vocab, p.side_w);
  // dW's contraction is cut where its tiles leave more than half of the chip idle (12224 x 33 x 1135 153 -> 104 us, 4096 x
  // 256 x 1024 79 -> 74); more tiles would only add the pieces' sums
  p.splits_w = (int)std::max<int64_t>(1, std::min<int64_t>(tiles <= 128 ? 512 / tiles : 1, s.n / 512));
  // a training step has three products to leave rows out of (2048 x 1024 x 32768: with a tenth of the rows left out
  // 495 -> 486 us, with half 457 -> 320)
  p.gather = 2.0 * s.n * s.d * s.vocab * (s.bf16 ? 1 : 6) * (train ? 4 : 1) >= kGatherFrom;
  return p;
}

// What a training step's forward leaves for its backward.
struct Kept {
  int *index, *at, *count, *equal;
  float *scale, *coef;
  char* g;
  int64_t bytes;
};
Kept kept_of(void* p, const Distillation& s, const Plan& l) {
  Kept k = {};
  char* at = (char*)p;
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += align256(bytes);
    return r;
  };
  k.index = (int*)take(4 * s.n), k.at = (int*)take(4 * s.n);
  k.count = (int*)take(12), k.equal = k.count + 1, k.scale = (float*)(k.count + 2);
  k.coef = (float*)take(4 * s.n);
  k.g = take(l.el * s.n * l.ldg);
  k.bytes = at - (char*)p;
  return k;
}

struct Space {
  char *x, *w, *x_again;
  int64_t* label;
  float *logp, *prob, *ref, *factor, *weight, *acc;
  float2* part;
  int *again, *to, *again_count;
  int *index, *at, *count, *equal;
  float* scale;
  int64_t bytes;
};
Space space_of(void* p, const Distillation& s, const Plan& l, bool backward) {
  Space w = {};
  char* at = (char*)p;
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += align256(bytes);
    return r;
  };
  const int64_t rows = l.el * s.n * (int64_t)l.dp;
  w.x = take(rows);
  w.w = take(l.el * s.vocab * (int64_t)l.dp);
  char* both = at;
  w.label = (int64_t*)take(8 * s.n);
  w.logp = (float*)take(4 * s.n * (int64_t)s.top), w.prob = (float*)take(4 * s.n * (int64_t)s.top);
  w.ref = (float*)take(4 * s.n);
  w.part = (float2*)take(8 * s.n * (int64_t)l.parts);
  if (backward) {
    w.x_again = take(rows);
    w.again = (int*)take(4 * s.n), w.to = (int*)take(4 * s.n), w.again_count = (int*)take(4);
    w.factor = (float*)take(4 * s.n);
  } else {
    w.index = (int*)take(4 * s.n), w.at = (int*)take(4 * s.n);
    w.count = (int*)take(12), w.equal = w.count + 1, w.scale = (float*)(w.count + 2);
  }
  char* end = at;
  if (backward) {
    at = both;
    w.weight = (float*)take(4 * s.n);
    w.equal = (int*)take(8), w.scale = (float*)(w.equal + 1);
    // sums of dX's pieces, and then of dW's
    w.acc = (float*)take(4 * (int64_t)l.dp * std::max(l.splits > 1 ? l.splits * s.n : 0,
                                                      l.splits_w > 1 ? l.splits_w * s.vocab : 0));
  }
  w.bytes = std::max(at, end) - (char*)p;
  return w;
}

atlasmem_status sum_pieces(const float* acc, int splits, int64_t rows, const Distillation& s, const Plan& p, const int* at,
                           const float* weight, const float* factor, void* out, hipStream_t st) {
  const int vec = s.d % 4 == 0 && ((uintptr_t)out & 15) == 0;
  ds_sum<<<(unsigned)((rows * (p.dp / 4) + 255) / 256), 256, 0, st>>>(acc, splits, rows, s.d, p.dp, at, weight, factor,
                                                                      out, s.bf16, vec);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace

int64_t distillation_workspace_bytes(const Distillation& s, bool backward) {
  return space_of(nullptr, s, plan_of(s, backward), backward).bytes;
}
int64_t distillation_kept_bytes(const Distillation& s) { return kept_of(nullptr, s, plan_of(s, true)).bytes; }

atlasmem_status distillation(const Distillation& s, const void* X, const void* W, const int64_t* ids,
                             const float* teacher, float* loss, float* lse, void* kept, void* workspace,
                             hipStream_t st) {
  const bool train = kept != nullptr;
  const Plan p = plan_of(s, train);
  Space ws = space_of(workspace, s, p, train);
  Kept k = {};
  if (train) {
    k = kept_of(kept, s, p);
    ws.index = k.index, ws.at = k.at, ws.count = k.count, ws.equal = k.equal, ws.scale = k.scale;
  }
  const bool vec = direct(X, s.d, s.bf16) && direct(W, s.d, s.bf16), as_they_come = train && !p.gather;
  ds_teacher<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(
      ids, teacher, s.n, s.top, s.vocab, s.scale, X, W, s.bf16, vec, s.d, ws.logp, ws.prob, ws.label,
      train ? ws.ref : nullptr, train ? ws.again_count : nullptr, as_they_come ? ws.index : nullptr, ws.at,
      as_they_come ? ws.count : nullptr);
  AM_LAUNCH_CHECK();
  atlasmem_status e = ATLASMEM_OK;
  if (p.gather) e = rows_that_count(s.n, 1, ws.label, nullptr, ws.index, ws.at, ws.count, ws.scale, ws.equal, st);
  const int *index = p.gather ? ws.index : nullptr, *count = p.gather ? ws.count : nullptr;
  const bool x_direct = !p.gather && direct(X, s.d, s.bf16), w_direct = direct(W, s.d, s.bf16);
  if (e == ATLASMEM_OK && !x_direct) e = copy_rows(X, s.bf16, s.n, s.d, p.dp, index, count, ws.x, st);
  if (e == ATLASMEM_OK && !w_direct) e = copy_rows(W, s.bf16, s.vocab, s.d, p.dp, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  GemmArgs g = {};
  g.a = w_direct ? W : ws.w;
  g.b = x_direct ? X : ws.x;
  g.lda = g.ldb = p.dp;
  g.na = s.vocab, g.nb = s.n, g.K = p.dp;
  g.count = count;
  g.part = ws.part, g.parts = p.parts;
  g.k2 = (float)(s.scale * kLog2e), g.k2_low = (float)(s.scale * kLog2e - g.k2);
  g.g = k.g, g.ldg = p.ldg;
  g.ref = ws.ref, g.index = index;
  e = s.n <= kFew ? gemm_few<false, EPI_KEPT>(g, s.bf16, st) : gemm<false, false, EPI_KEPT>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  JoinArgs a = {};
  a.part = ws.part, a.parts = p.parts, a.at = p.gather ? ws.at : nullptr;
  a.x = g.b, a.w = g.a, a.dp = p.dp, a.n = s.n;
  a.label = ws.label, a.ids = ids, a.logp = ws.logp, a.prob = ws.prob, a.top = s.top;
  a.scale = s.scale, a.k2 = g.k2, a.k2_low = g.k2_low;
  a.loss = loss, a.lse = lse;
  if (train) {
    a.all = !p.gather;
    a.ref = ws.ref, a.coef = k.coef, a.factor = ws.factor, a.g = k.g, a.ldg = p.ldg;
    a.again = ws.again, a.to = ws.to, a.again_count = ws.again_count, a.x_again = ws.x_again;
  }
  const unsigned rows = (unsigned)std::min<int64_t>(s.n, 1 << 20);
  auto launch = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (s.bf16) train ? ds_rows<NT, true, true><<<rows, NT, 0, st>>>(a) : ds_rows<NT, true, false><<<rows, NT, 0, st>>>(a);
    else train ? ds_rows<NT, false, true><<<rows, NT, 0, st>>>(a) : ds_rows<NT, false, false><<<rows, NT, 0, st>>>(a);
  };
  // what a row's workgroup reads and writes
  const int64_t row_bytes = p.el * ((train ? p.ldg : 0) + (int64_t)s.top * p.dp);
  if (s.n <= 256 && s.top > 16) launch(std::integral_constant<int, 1024>{});
  else if (s.n >= kManyRows && row_bytes <= kShortRow) launch(std::integral_constant<int, 64>{});
  else launch(std::integral_constant<int, 256>{});
  AM_LAUNCH_CHECK();
  if (!train) return ATLASMEM_OK;
  g.b = ws.x_again;
  g.count = ws.again_count, g.index = ws.again, g.to = ws.to;
  g.ids = ids, g.prob = ws.prob, g.factor = ws.factor, g.top = s.top;
  return s.n <= kFew ? gemm_few<false, EPI_AGAIN>(g, s.bf16, st)
                     : gemm<false, false, EPI_AGAIN>(g, s.bf16, p.side, st);
}

atlasmem_status distillation_backward(const Distillation& s, const void* X, const void* W, const void* kept,
                                      const float* dloss, void* dX, void* dW, void* workspace, hipStream_t st) {
  if (s.n == 0) {
    if (dW) {
      const int64_t count = s.vocab * (int64_t)s.d;
      xe_zero<<<(unsigned)std::min<int64_t>((count + 255) / 256, 1 << 16), 256, 0, st>>>(dW, count, s.bf16);
      AM_LAUNCH_CHECK();
    }
    return ATLASMEM_OK;
  }
  const Plan p = plan_of(s, true);
  const Kept k = kept_of(const_cast<void*>(kept), s, p);
  const Space ws = space_of(workspace, s, p, true);
  if (s.n > kFewRows) {
    ds_scale<<<1, 1024, 0, st>>>(k.coef, dloss, k.at, s.n, ws.weight, ws.scale, ws.equal);
    AM_LAUNCH_CHECK();
  }
  ds_weigh<<<(unsigned)((s.n * (p.dp / 4) + 255) / 256), 256, 0, st>>>(
      X, s.bf16, s.n, s.d, p.dp, k.at, !p.gather, k.coef, dloss, ws.weight, ws.scale, ws.equal, dW ? ws.x : nullptr,
      p.gather && p.splits == 1 ? dX : nullptr);
  AM_LAUNCH_CHECK();
  atlasmem_status e = ATLASMEM_OK;
  if (dX) {
    const bool w_direct = direct(W, s.d, s.bf16);
    if (!w_direct) e = copy_rows(W, s.bf16, s.vocab, s.d, p.dp, nullptr, nullptr, ws.w, st);
    if (e != ATLASMEM_OK) return e;
    GemmArgs x = {};
    x.count = k.count;
    x.a = w_direct ? W : ws.w, x.lda = p.dp, x.na = p.dp;
    x.b = k.g, x.ldb = p.ldg, x.nb = s.n;
    x.K = s.vocab;
    const bool few = s.n <= kFew && p.side_x != (s.bf16 ? 64 : 128);
    if (p.splits == 1) {
      x.out = dX, x.ldo = s.d, x.to = k.index, x.at = k.at, x.row_weight = ws.weight;
      e = few ? gemm_few<true, EPI_ROWS>(x, s.bf16, st) : gemm<true, false, EPI_ROWS>(x, s.bf16, p.side_x, st);
    } else {
      x.splits = p.splits, x.acc = ws.acc, x.acc_rows = s.n;
      e = few ? gemm_few<true, EPI_ACC>(x, s.bf16, st) : gemm<true, false, EPI_ACC>(x, s.bf16, p.side_x, st);
      if (e == ATLASMEM_OK) e = sum_pieces(ws.acc, p.splits, s.n, s, p, k.at, ws.weight, nullptr, dX, st);
    }
    if (e != ATLASMEM_OK) return e;
  }
  if (dW) {
    GemmArgs x = {};
    x.count = k.count;
    x.a = ws.x, x.lda = p.dp, x.na = p.dp;
    x.b = k.g, x.ldb = p.ldg, x.nb = s.vocab;
    x.K = s.n;
    if (p.splits_w == 1) {
      x.scale = ws.scale;
      x.out = dW, x.ldo = s.d;
      e = gemm<true, true, EPI_OUT>(x, s.bf16, p.side_w, st);
    } else {
      x.splits = p.splits_w, x.acc = ws.acc, x.acc_rows = s.vocab;
      e = gemm<true, true, EPI_PART>(x, s.bf16, p.side_w, st);
      if (e == ATLASMEM_OK) e = sum_pieces(ws.acc, p.splits_w, s.vocab, s, p, nullptr, nullptr, ws.scale, dW, st);
    }
    if (e != ATLASMEM_OK) return e;
  }
  return ATLASMEM_OK;
}

}  // namespace am
