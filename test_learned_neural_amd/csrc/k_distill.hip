// Distillation from a teacher's top logits, without keeping the student's logits (gfx950).
//   z = X W^T,  p_i = softmax_j(scale t_ij) over the row's given classes,  q_i = softmax_v(scale z_iv)
//   loss_i = sum_j p_ij (log p_ij - log q_i,id_ij),  G_iv = q_iv - sum_{j: id_ij = v} p_ij
//   dX_i = scale dloss_i (G W)_i,  dW = G^T (scale dloss X)
// The forward computes z once.  For a training step it leaves of a tile not z but exp(scale (z - ref)) in the type
// of X, with ref a logit of the row that is known beforehand, that of the teacher's first class: up to a factor
// c = exp(scale ref - lse) of the row this is q, rounded once.  Then only the given classes' entries are
// written again, less p / c, and what is kept is G / c: the backward has two products, not three.
// Rows whose ref is too far from their lse for a factor (2^60) are computed again with lse for ref.
#include "logits.h"

namespace am {

namespace {

constexpr float kFar = 60.0f;

// log p of each given class (-inf: none), and of each row a label (0, or -1 for a row that has no class) and the
// logit of its first class.  A wave a row.
__global__ __launch_bounds__(256) void ds_teacher(const int64_t* ids, const float* teacher, int64_t n, int top,
                                                  int64_t vocab, float scale, const void* X, const void* W, int bf16,
                                                  int vec, int d, float* logp, int64_t* label, float* ref,
                                                  int* again_count) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (again_count && r == 0 && lane == 0) *again_count = 0;
  if (r >= n) return;
  float t[2];
  int64_t id[2];
  bool on[2];
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 64 * h;
    id[h] = j < top ? ids[r * top + j] : -1;
    t[h] = j < top ? teacher[r * top + j] * scale : -INFINITY;
    on[h] = id[h] >= 0 && id[h] < vocab && !(t[h] == -INFINITY);
    if (on[h]) m = fmaxf(m, t[h]), nan |= t[h] != t[h];
  }
  for (int k = 32; k; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
  float s = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) s += on[h] ? expf(t[h] - m) : 0.0f;
  for (int k = 32; k; k >>= 1) s += __shfl_xor(s, k);
  const float ls = logf(s);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 64 * h < top) logp[r * top + lane + 64 * h] = on[h] ? t[h] - m - ls : -INFINITY;
  const uint64_t any = __ballot(on[0] || on[1]);
  if (lane == 0) label[r] = any ? 0 : -1;
  if (!ref || !any) return;
  const uint64_t f0 = __ballot(on[0] && t[0] == m), f1 = __ballot(on[1] && t[1] == m);
  const int at = f0 ? __builtin_ctzll(f0) : f1 ? __builtin_ctzll(f1) : __builtin_ctzll(any);
  const bool low = f0 || (!f1 && (__ballot(on[0]) >> at & 1));
  const int64_t y = __shfl(low ? id[0] : id[1], at);
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
  int dp, bf16;
  int64_t n;
  const int64_t *label, *ids;
  const float* logp;
  int top;
  float scale, k2;
  float *loss, *lse;
  // a training step
  float *ref, *coef;
  void* g;
  int64_t ldg;
  int *again, *to, *again_count;
  void* x_again;
};

// loss, lse of a row, and its entries at the given classes.  A wave a row.
__global__ __launch_bounds__(256) void ds_join(JoinArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= a.n) return;
  if (a.label[r] < 0) {
    if (lane == 0) a.loss[r] = 0.0f, a.lse[r] = 0.0f;
    return;
  }
  const int64_t place = __builtin_amdgcn_readfirstlane(a.at ? a.at[r] : (int)r);
  float m = -INFINITY, s = 0.0f;
  auto join = [&](float om, float os) {
    const float t = fmaxf(m, om), from = t > -INFINITY ? t : 0.0f;
    s = s * __builtin_amdgcn_exp2f((m - from) * a.k2) + os * __builtin_amdgcn_exp2f((om - from) * a.k2);
    m = t;
  };
  for (int i = lane; i < a.parts; i += 64) {
    const float2 q = a.part[place * a.parts + i];
    join(q.x, q.y);
  }
  for (int k = 32; k; k >>= 1) {
    const float om = __shfl_xor(m, k), os = __shfl_xor(s, k);
    join(om, os);
  }
  const float lse = fmaf(a.scale, m, logf(s));
  double z[2] = {0.0, 0.0};
  int64_t id[2];
  float lp[2], p[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 64 * h;
    id[h] = j < a.top ? a.ids[r * a.top + j] : -1;
    lp[h] = j < a.top ? a.logp[r * a.top + j] : -INFINITY;
    p[h] = lp[h] == -INFINITY ? 0.0f : expf(lp[h]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (int j = 64 * h; j < min(64 * h + 64, a.top); ++j) {
      if (__shfl(lp[h], j & 63) == -INFINITY) continue;
      const int c[1] = {__builtin_amdgcn_readfirstlane((int)__shfl(id[h], j & 63))};
      double v[1];
      if (a.bf16) row_dots<1, true>(a.x, a.w, place, c, a.dp, lane, v);
      else row_dots<1, false>(a.x, a.w, place, c, a.dp, lane, v);
      if (lane == (j & 63)) z[h] = v[0];
    }
  float loss = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (p[h] != 0.0f) loss += p[h] * (lp[h] - (float)(a.scale * z[h] - lse));
  for (int k = 32; k; k >>= 1) loss += __shfl_xor(loss, k);
  if (lane == 0) a.loss[r] = loss, a.lse[r] = lse;
  if (!a.g) return;

  float ref = a.ref[r];
  const float l2 = __log2f(s);
  const bool near = fabsf((m - ref) * a.k2 + l2) <= kFar;
  if (!near) ref = m + l2 / a.k2;
  const float coef = __builtin_amdgcn_exp2f((ref - m) * a.k2) / s;
  if (lane == 0) a.coef[r] = a.scale * coef;
  if (!near) {
    int slot = 0;
    if (lane == 0) {
      slot = atomicAdd(a.again_count, 1);
      a.again[slot] = (int)r, a.to[slot] = (int)place, a.ref[r] = ref;
    }
    slot = __builtin_amdgcn_readfirstlane(slot);
    const int words = a.dp * (a.bf16 ? 2 : 4) / 16;
    for (int c = lane; c < words; c += 64)
      ((u32x4*)a.x_again)[(int64_t)slot * words + c] = ((const u32x4*)a.x)[place * words + c];
    return;
  }
  float sum[2] = {0.0f, 0.0f};
  for (int j = 0; j < a.top; ++j) {
    const int64_t o = __shfl(j < 64 ? id[0] : id[1], j & 63);
    const float q = __shfl(j < 64 ? p[0] : p[1], j & 63);
    sum[0] += o == id[0] ? q : 0.0f, sum[1] += o == id[1] ? q : 0.0f;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lp[h] != -INFINITY) {
      const float v = __builtin_amdgcn_exp2f((float)(z[h] - ref) * a.k2) - sum[h] / coef;
      if (a.bf16) ((uint16_t*)a.g)[place * a.ldg + id[h]] = (uint16_t)bf16_bits(v);
      else ((float*)a.g)[place * a.ldg + id[h]] = v;
    }
}

// Weights of the rows, dloss coef, and the rows that count times them: four columns a thread.
__global__ void ds_weigh(const void* x, int bf16, int d, int dp, const int* index, const int* count,
                         const float* dloss, const float* coef, float* weight, void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = dp / 4, r = i / per;
  if (r >= *count) return;
  const int c = (int)(i % per) * 4;
  const int64_t row = index[r];
  const float w = coef[row] * (dloss ? dloss[row] : 1.0f);
  if (c == 0) weight[row] = w;
  if (!out) return;
  float v[4];
  if (d % 4 == 0 && ((uintptr_t)x & 15) == 0 && c < d) {
    if (bf16) {
      const uint2 u = *(const uint2*)((const uint16_t*)x + row * d + c);
      v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
      v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
      const float4 u = *(const float4*)((const float*)x + row * d + c);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k < d ? load_in(x, row * d + c + k, bf16) : 0.0f;
  }
  const int64_t at = r * dp + c;
  if (bf16) *(uint2*)((uint16_t*)out + at) = uint2{cvt_pk_bf16(v[0] * w, v[1] * w), cvt_pk_bf16(v[2] * w, v[3] * w)};
  else *(float4*)((float*)out + at) = float4{v[0] * w, v[1] * w, v[2] * w, v[3] * w};
}

struct Plan {
  int el, dp, side, parts, side_x, splits;
  int64_t ldg;
};
Plan plan_of(const Distillation& s) {
  Plan p = {};
  p.el = s.bf16 ? 2 : 4;
  p.dp = (int)up(s.d, s.bf16 ? 8 : 4);
  p.side = side_of(s.vocab, s.n, s.bf16);
  p.parts = (int)((s.vocab + p.side - 1) / p.side);
  p.ldg = up(s.vocab, 64);
  p.side_x = side_split(p.dp, s.n, s.bf16);
  const int64_t tiles = std::max<int64_t>(tiles_of(p.dp, s.n, p.side_x), 1);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>((p.side_x == 256 ? 256 : 512) / tiles, s.vocab / 512));
  if (tiles * p.splits <= 128) p.side_x = 64;
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
  float *logp, *ref, *weight, *acc;
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
  w.logp = (float*)take(4 * s.n * (int64_t)s.top);
  w.ref = (float*)take(4 * s.n);
  w.part = (float2*)take(8 * s.n * (int64_t)l.parts);
  if (backward) {
    w.x_again = take(rows);
    w.again = (int*)take(4 * s.n), w.to = (int*)take(4 * s.n), w.again_count = (int*)take(4);
  } else {
    w.index = (int*)take(4 * s.n), w.at = (int*)take(4 * s.n);
    w.count = (int*)take(12), w.equal = w.count + 1, w.scale = (float*)(w.count + 2);
  }
  char* end = at;
  if (backward) {
    at = both;
    w.weight = (float*)take(4 * s.n);
    w.acc = (float*)take(4 * (int64_t)l.splits * s.n * l.dp);
  }
  w.bytes = std::max(at, end) - (char*)p;
  return w;
}

}  // namespace

int64_t distillation_workspace_bytes(const Distillation& s, bool backward) {
  return space_of(nullptr, s, plan_of(s), backward).bytes;
}
int64_t distillation_kept_bytes(const Distillation& s) { return kept_of(nullptr, s, plan_of(s)).bytes; }

atlasmem_status distillation(const Distillation& s, const void* X, const void* W, const int64_t* ids,
                             const float* teacher, float* loss, float* lse, void* kept, void* workspace,
                             hipStream_t st) {
  const Plan p = plan_of(s);
  const bool train = kept != nullptr;
  Space ws = space_of(workspace, s, p, train);
  Kept k = {};
  if (train) {
    k = kept_of(kept, s, p);
    ws.index = k.index, ws.at = k.at, ws.count = k.count, ws.equal = k.equal, ws.scale = k.scale;
  }
  const bool gather = train || 2.0 * s.n * s.d * s.vocab * (s.bf16 ? 1 : 6) >= kGatherFrom;
  const bool vec = direct(X, s.d, s.bf16) && direct(W, s.d, s.bf16);
  ds_teacher<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(ids, teacher, s.n, s.top, s.vocab, s.scale, X, W, s.bf16, vec,
                                                        s.d, ws.logp, ws.label, train ? ws.ref : nullptr,
                                                        train ? ws.again_count : nullptr);
  AM_LAUNCH_CHECK();
  atlasmem_status e = ATLASMEM_OK;
  if (gather) e = rows_that_count(s.n, 1, ws.label, nullptr, ws.index, ws.at, ws.count, ws.scale, ws.equal, st);
  const int *index = gather ? ws.index : nullptr, *count = gather ? ws.count : nullptr;
  const bool x_direct = !gather && direct(X, s.d, s.bf16), w_direct = direct(W, s.d, s.bf16);
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
  g.k2 = s.scale * 1.4426950408889634f;
  g.g = k.g, g.ldg = p.ldg;
  g.ref = ws.ref, g.index = index;
  e = gemm<false, false, EPI_KEPT>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  JoinArgs a = {};
  a.part = ws.part, a.parts = p.parts, a.at = gather ? ws.at : nullptr;
  a.x = g.b, a.w = g.a, a.dp = p.dp, a.bf16 = s.bf16, a.n = s.n;
  a.label = ws.label, a.ids = ids, a.logp = ws.logp, a.top = s.top;
  a.scale = s.scale, a.k2 = g.k2;
  a.loss = loss, a.lse = lse;
  if (train) {
    a.ref = ws.ref, a.coef = k.coef, a.g = k.g, a.ldg = p.ldg;
    a.again = ws.again, a.to = ws.to, a.again_count = ws.again_count, a.x_again = ws.x_again;
  }
  ds_join<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(a);
  AM_LAUNCH_CHECK();
  if (!train) return ATLASMEM_OK;
  g.b = ws.x_again;
  g.count = ws.again_count, g.index = ws.again, g.to = ws.to;
  g.ids = ids, g.logp = ws.logp, g.coef = k.coef, g.top = s.top, g.q_scale = s.scale;
  return gemm<false, false, EPI_AGAIN>(g, s.bf16, p.side, st);
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
  const Plan p = plan_of(s);
  const Kept k = kept_of(const_cast<void*>(kept), s, p);
  const Space ws = space_of(workspace, s, p, true);
  ds_weigh<<<(unsigned)((s.n * (p.dp / 4) + 255) / 256), 256, 0, st>>>(X, s.bf16, s.d, p.dp, k.index, k.count, dloss,
                                                                       k.coef, ws.weight, dW ? ws.x : nullptr);
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
    x.splits = p.splits, x.acc = ws.acc, x.acc_rows = s.n;
    e = gemm<true, false, EPI_ACC>(x, s.bf16, p.side_x, st);
    if (e != ATLASMEM_OK) return e;
    const int vec = s.d % 4 == 0 && ((uintptr_t)dX & 15) == 0;
    xe_sum<<<(unsigned)((s.n * (p.dp / 4) + 255) / 256), 256, 0, st>>>(ws.acc, p.splits, s.n, s.d, p.dp, k.at,
                                                                       ws.weight, dX, s.bf16, vec);
    AM_LAUNCH_CHECK();
  }
  if (dW) {
    GemmArgs x = {};
    x.count = k.count;
    x.a = ws.x, x.lda = p.dp, x.na = p.dp;
    x.b = k.g, x.ldb = p.ldg, x.nb = s.vocab;
    x.K = s.n;
    x.out = dW, x.ldo = s.d;
    e = gemm<true, true, EPI_OUT>(x, s.bf16, side_of(p.dp, s.vocab, s.bf16), st);
    if (e != ATLASMEM_OK) return e;
  }
  return ATLASMEM_OK;
}

}  // namespace am
