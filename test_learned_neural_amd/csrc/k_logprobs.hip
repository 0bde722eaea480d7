// Log probabilities of given tokens, the entropy of each row and its top alternatives, without keeping the
// logits (gfx950).
//   z = X W^T,  lse_i = log sum_v exp(scale z_iv),  logprob_i = scale z_i,token - lse_i,
//   entropy_i = lse_i - sum_v p_iv scale z_iv,  alternatives: the classes of the largest z
// One pass of the product engine leaves of each row and tile its maximum, its sum of exponentials and their
// product with z; a workgroup for each row joins them.
//
// Alternatives.  Which class is larger is decided in 64 bits, so that an answer does not depend on how a sum
// was cut: equal logits go to the lowest index.  The matrix cores' z is off by at most
// c |x| |w| (c: the roundings on a term's way; Cauchy and Schwarz), so z + c |x| |w| is an upper bound.  A
// lane's 16 to 64 classes of a row are a group; of each the two largest bounds are kept, with the class's
// place in the six bits that this costs.  The row's workgroup takes the best classes of `top` of its threads,
// computes them in 64 bits, and has a lower bound of the last alternative; then every class whose bound
// passes it is computed too: a group whose second bound passes as a whole.
#include "logits.h"

namespace am {

namespace {

constexpr float kLowest = -3.4028235e38f;

// |rows| of a matrix times `factor`, at most the largest float; zeros from `rows` to `end`.  A wave a row.
__global__ __launch_bounds__(256) void lp_norms(const void* x, int bf16, int64_t rows, const int* count, int dp,
                                                float factor, int64_t end, float* out) {
  const int lane = threadIdx.x & 63;
  if (count) rows = *count;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < end; r += (int64_t)gridDim.x * 4) {
    float s = 0.0f;
    if (r < rows) {
      if (bf16) {
        for (int c = lane * 8; c < dp; c += 512) {
          const u32x4 w = *(const u32x4*)((const uint16_t*)x + r * dp + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xFFFF0000u);
            s = fmaf(lo, lo, fmaf(hi, hi, s));
          }
        }
      } else {
        for (int c = lane * 4; c < dp; c += 256) {
          const float4 w = *(const float4*)((const float*)x + r * dp + c);
          s = fmaf(w.x, w.x, fmaf(w.y, w.y, fmaf(w.z, w.z, fmaf(w.w, w.w, s))));
        }
      }
    }
    for (int k = 32; k; k >>= 1) s += __shfl_xor(s, k);
    if (lane == 0) out[r] = fminf(sqrtf(s) * factor, -kLowest);
  }
}

// The largest logit that a key stands for.
__device__ __forceinline__ float bound_of(float key) {
  const uint32_t b = __float_as_uint(key);
  return __uint_as_float(b >> 31 ? b & ~63u : (b & ~63u) ? b | 63u : 0u);
}

struct RowArgs {
  const float4* sums;
  const float2* keys;
  int parts, side;
  const int* at;           // a row's place among those that count, or null: all are there
  const void *x, *w;       // as the products took them, [..][dp]
  int dp, bf16;
  int64_t n, vocab;
  const int64_t* tokens;   // or null
  float scale, k2;
  int top;
  float *logprob, *entropy;
  int64_t* ids;
  float* top_logprobs;
};

constexpr int kTopMost = 64;   // alternatives
constexpr float kMasked = -1.0e38f;  // logits from here down are no alternatives
constexpr int kTake = 16;      // classes a wave computes between two selections
constexpr int kPending = 1024, kFlush = 512;

// (z, class) before (y, other): larger, or equal and of lower index
__device__ __forceinline__ bool ahead(double z, int c, double y, int o) { return z > y || (z == y && c < o); }

__global__ __launch_bounds__(256) void lp_rows(RowArgs g) {
  constexpr int kList = kTopMost + 4 * kTake;
  __shared__ float4 part[4];
  __shared__ float first[256];
  __shared__ double lz[2][kList];
  __shared__ int lc[2][kList];
  __shared__ int items[kPending];
  __shared__ int counts[2];       // entries of the list, pending items
  __shared__ float token_z;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int64_t r = blockIdx.x; r < g.n; r += gridDim.x) {
    const int64_t y = g.tokens ? g.tokens[r] : 0;
    if (y < 0 || y >= g.vocab) {
      if (tid == 0) {
        if (g.logprob) g.logprob[r] = 0.0f;
        if (g.entropy) g.entropy[r] = 0.0f;
      }
      if (tid < g.top) g.ids[r * g.top + tid] = -1, g.top_logprobs[r * g.top + tid] = 0.0f;
      continue;
    }
    const int64_t place = g.at ? g.at[r] : r;

    // the row's maximum, sum and first moment
    float m = -INFINITY, s = 0.0f, t = 0.0f;
    auto join = [&](float om, float os, float ot) {
      const float to = fmaxf(m, om), from = to > -INFINITY ? to : 0.0f;
      const float x = m - from, ox = om - from;  // minus infinity, or a masked class's, where e is zero
      const float e = __builtin_amdgcn_exp2f(x * g.k2), oe = __builtin_amdgcn_exp2f(ox * g.k2);
      t = (e > 0.0f ? e * fmaf(s, x, t) : 0.0f) + (oe > 0.0f ? oe * fmaf(os, ox, ot) : 0.0f);
      s = fmaf(s, e, os * oe);
      m = to;
    };
    for (int i = tid; i < g.parts; i += 256) {
      const float4 q = g.sums[place * g.parts + i];
      join(q.x, q.y, q.z);
    }
    for (int k = 32; k; k >>= 1) {
      const float om = __shfl_xor(m, k), os = __shfl_xor(s, k), ot = __shfl_xor(t, k);
      join(om, os, ot);
    }
    __syncthreads();  // the last row's shared values have been read
    if (lane == 0) part[wave] = float4{m, s, t, 0.0f};
    if (wave == 0 && g.tokens) {
      const double z = row_dot(g.x, g.w, place, y, g.dp, g.bf16, lane);
      if (lane == 0) token_z = (float)z;
    }
    __syncthreads();
    m = -INFINITY, s = t = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) join(part[w].x, part[w].y, part[w].z);
    const float lse = fmaf(g.scale, m, logf(s));
    const bool none = lse == -INFINITY, bad = !none && !(fabsf(lse) < INFINITY);
    if (tid == 0) {
      const float p = fmaf(g.scale, token_z, -lse), h = logf(s) - g.scale * t / s;
      if (g.logprob) g.logprob[r] = bad ? NAN : none ? -INFINITY : p > 0.0f ? 0.0f : p;
      if (g.entropy) g.entropy[r] = bad ? NAN : none || h < 0.0f ? 0.0f : h;
    }
    if (g.top == 0) continue;
    if (none || bad) {
      if (tid < g.top) g.ids[r * g.top + tid] = -1, g.top_logprobs[r * g.top + tid] = bad ? NAN : -INFINITY;
      continue;
    }

    // the first `top` threads by their groups' largest bound
    const int groups = 4 * g.parts;
    const float2* keys = g.keys + place * groups;
    float best = -INFINITY;
    int mine = -1;
    for (int i = tid; i < groups; i += 256) {
      const float k = keys[i].x;
      if (k > best) best = k, mine = i;
    }
    const int64_t own = mine < 0 ? g.vocab : group_class(mine, __float_as_uint(best) & 63, g.side);
    if (own >= g.vocab || bound_of(best) <= kMasked) best = -INFINITY;
    first[tid] = best;
    if (tid < 2) counts[tid] = 0;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < 256; i += 4) {
      const float4 o = *(const float4*)(first + i);
      rank += (o.x > best || (o.x == best && i + 0 < tid)) + (o.y > best || (o.y == best && i + 1 < tid)) +
              (o.z > best || (o.z == best && i + 2 < tid)) + (o.w > best || (o.w == best && i + 3 < tid));
    }
    if (best > -INFINITY && rank < g.top) items[rank] = (int)own, atomicAdd(&counts[1], 1);
    __syncthreads();

    // The list of what is known in 64 bits, in order; `last` of its `top`, if there are so many, is the bar.
    int known = 0, buf = 0;
    double bar = -INFINITY;
    int bar_class = 0x7fffffff;
    // Computes what is pending: a class, or (negative) all classes of a group.
    auto flush = [&]() {
      const int pending = counts[1];
      int at = wave, code = 0;
      bool more = true;
      while (more) {
        for (int k = 0; k < kTake && at < pending; ++k) {
          const int item = items[at];
          int64_t c = item;
          if (item < 0) {
            c = group_class(~item, code, g.side);
            if (++code == g.side / 4) at += 4, code = 0;
          } else {
            at += 4;
          }
          if (c >= g.vocab) continue;
          if (__any(lane < known && lc[buf][lane] == (int)c)) continue;
          const double z = row_dot(g.x, g.w, place, c, g.dp, g.bf16, lane);
          if (lane == 0 && z > kMasked && ahead(z, (int)c, bar, bar_class)) {
            const int e = known + atomicAdd(&counts[0], 1);
            lz[buf][e] = z, lc[buf][e] = (int)c;
          }
        }
        more = __syncthreads_or(at < pending);
        const int total = known + counts[0];
        if (total > known) {
          if (tid < total) {
            const double z = lz[buf][tid];
            const int c = lc[buf][tid];
            int ahead_of = 0;
            for (int i = 0; i < total; ++i) ahead_of += ahead(lz[buf][i], lc[buf][i], z, c);
            if (ahead_of < g.top) lz[buf ^ 1][ahead_of] = z, lc[buf ^ 1][ahead_of] = c;
          }
          buf ^= 1;
          known = min(total, g.top);
        }
        __syncthreads();
        if (known == g.top) bar = lz[buf][known - 1], bar_class = lc[buf][known - 1];
        if (tid == 0) counts[0] = 0;
        __syncthreads();
      }
      if (tid == 0) counts[1] = 0;
      __syncthreads();
    };
    flush();
    // every class that may pass the bar
    for (int i0 = 0; i0 < groups; i0 += 256) {
      const int i = i0 + tid;
      if (i < groups) {
        const float2 k = keys[i];
        const double b1 = bound_of(k.x), b2 = bound_of(k.y);
        const int64_t start = group_class(i, 0, g.side);
        if (start < g.vocab && b1 > kMasked) {
          if (b2 > kMasked && (b2 > bar || (b2 == bar && start < bar_class))) {
            items[atomicAdd(&counts[1], 1)] = ~i;
          } else if (b1 > bar || (b1 == bar && start < bar_class)) {
            items[atomicAdd(&counts[1], 1)] = (int)group_class(i, __float_as_uint(k.x) & 63, g.side);
          }
        }
      }
      __syncthreads();
      const int pending = counts[1];
      __syncthreads();
      if (pending > kFlush || i0 + 256 >= groups) flush();
    }
    if (tid < g.top) {
      const bool there = tid < known;
      g.ids[r * g.top + tid] = there ? lc[buf][tid] : -1;
      g.top_logprobs[r * g.top + tid] =
          there ? fminf((float)(g.scale * lz[buf][tid] - (double)lse), 0.0f) : -INFINITY;
    }
  }
}

struct Plan {
  int el, dp, side, parts;
  bool gather;
};
Plan plan_of(const TokenLogprobs& s, bool tokens) {
  Plan p = {};
  p.el = s.bf16 ? 2 : 4;
  p.dp = (int)up(s.d, s.bf16 ? 8 : 4);
  p.side = side_of(s.vocab, s.n, s.bf16);
  p.parts = (int)((s.vocab + p.side - 1) / p.side);
  p.gather = tokens && 2.0 * s.n * s.d * s.vocab * (s.bf16 ? 1 : 6) >= kGatherFrom;
  return p;
}

struct Space {
  int *index, *at, *count, *equal;
  float* scale;
  char *x, *w;
  float *a_norm, *b_norm;
  float4* sums;
  float2* keys;
  int64_t bytes;
};
Space space_of(void* p, const TokenLogprobs& s, const Plan& l) {
  Space w = {};
  char* at = (char*)p;
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += align256(bytes);
    return r;
  };
  w.index = (int*)take(4 * s.n), w.at = (int*)take(4 * s.n);
  w.count = (int*)take(12), w.equal = w.count + 1, w.scale = (float*)(w.count + 2);
  w.x = take(l.el * s.n * (int64_t)l.dp);
  w.w = take(l.el * s.vocab * (int64_t)l.dp);
  w.sums = (float4*)take(16 * s.n * (int64_t)l.parts);
  if (s.top) {
    w.a_norm = (float*)take(4 * l.parts * (int64_t)l.side), w.b_norm = (float*)take(4 * s.n);
    w.keys = (float2*)take(32 * s.n * (int64_t)l.parts);
  }
  w.bytes = at - (char*)p;
  return w;
}

atlasmem_status norms(const void* x, bool bf16, int64_t rows, const int* count, int dp, float factor, int64_t end,
                      float* out, hipStream_t st) {
  lp_norms<<<(unsigned)std::min<int64_t>((end + 3) / 4, 1 << 16), 256, 0, st>>>(x, bf16, rows, count, dp, factor, end,
                                                                                out);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace

int64_t token_logprobs_workspace_bytes(const TokenLogprobs& s) { return space_of(nullptr, s, plan_of(s, true)).bytes; }

atlasmem_status token_logprobs(const TokenLogprobs& s, const void* X, const void* W, const int64_t* tokens,
                               float* logprob, float* entropy, int64_t* top_ids, float* top_logprobs, void* workspace,
                               hipStream_t st) {
  const Plan p = plan_of(s, tokens != nullptr);
  const Space ws = space_of(workspace, s, p);
  atlasmem_status e = ATLASMEM_OK;
  if (p.gather) e = rows_that_count(s.n, s.vocab, tokens, nullptr, ws.index, ws.at, ws.count, ws.scale, ws.equal, st);
  const int *index = p.gather ? ws.index : nullptr, *count = p.gather ? ws.count : nullptr;
  const bool x_direct = !p.gather && direct(X, s.d, s.bf16);
  const bool w_direct = direct(W, s.d, s.bf16);
  if (e == ATLASMEM_OK && !x_direct) e = copy_rows(X, s.bf16, s.n, s.d, p.dp, index, count, ws.x, st);
  if (e == ATLASMEM_OK && !w_direct) e = copy_rows(W, s.bf16, s.vocab, s.d, p.dp, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  GemmArgs g = {};
  g.a = w_direct ? W : ws.w;
  g.b = x_direct ? X : ws.x;
  g.lda = g.ldb = p.dp;
  g.na = s.vocab, g.nb = s.n, g.K = p.dp;
  g.count = count;
  g.parts = p.parts;
  g.sums = ws.sums;
  g.k2 = s.scale * 1.4426950408889634f;
  if (s.top) {
    // roundings on a term's way: eight for each of dp / 16 matrix instructions; in fp32 six instructions with
    // those for each 16 columns, and the planes that are not multiplied; a hundredth for the norms' own
    const float c = ((s.bf16 ? 0.5f : 3.0f) * p.dp + 128.0f) * 0x1p-24f * 1.01f;
    e = norms(g.a, s.bf16, s.vocab, nullptr, p.dp, 1.0f, (int64_t)p.parts * p.side, ws.a_norm, st);
    if (e == ATLASMEM_OK) e = norms(g.b, s.bf16, s.n, count, p.dp, c, s.n, ws.b_norm, st);
    if (e != ATLASMEM_OK) return e;
    g.keys = ws.keys, g.a_norm = ws.a_norm, g.b_norm = ws.b_norm;
  }
  e = gemm<false, false, EPI_TOP>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  RowArgs a = {};
  a.sums = ws.sums, a.keys = ws.keys, a.parts = p.parts, a.side = p.side;
  a.at = p.gather ? ws.at : nullptr;
  a.x = g.b, a.w = g.a, a.dp = p.dp, a.bf16 = s.bf16;
  a.n = s.n, a.vocab = s.vocab;
  a.tokens = tokens;
  a.scale = s.scale, a.k2 = g.k2, a.top = s.top;
  a.logprob = logprob, a.entropy = entropy, a.ids = top_ids, a.top_logprobs = top_logprobs;
  lp_rows<<<(unsigned)std::min<int64_t>(s.n, 1 << 20), 256, 0, st>>>(a);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace am
