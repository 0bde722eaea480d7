// Group norm with an activation, channels last (gfx950): X [n, L, C], G groups of c = C / G channels,
// statistics of a group over its L positions and c channels.
//   xh = (x - mean) rstd, z = gamma xh + beta, y = act(z)
//   dz = act'(z) dy, dgamma = sum dz xh, dbeta = sum dz   (over n, L)
//   dx = rstd (h - mean(h) - xh mean(h xh)),  h = gamma dz
// Two forms.  Groups that fit a wave's registers (the heads of a token, L = 1): a team of lanes holds a
// group, one pass over memory.  Otherwise: partial sums over spans of positions, a small
// reduction, and a second pass that applies them.  Variances come from differences to a mean, never
// from a difference of sums; fp32 throughout, one rounding at the end; sums run in one order.
//
// Bound by memory.  bf16 16384 rows x 16 groups of 128: forward 25.1 us (134 MB at 5.3 TB/s; 34 us before
// the next row's loads were in flight while one is computed), backward 54.7 us (201 MB and the partial
// sums at 4.0 TB/s) and gamma's and beta's sums 7 us.  fp32 3 x 16385 x 512 with 32 groups: moments 17.4,
// apply 31.8, sums 35.6, gradient 51.1 us (101 MB a tensor, which the last-level cache holds: 5.7 to 6.3 TB/s),
// the small reductions 4 to 8 us each.  One token: 3 us, a launch.
#include <algorithm>

#include "common.h"
#include "internal.h"

namespace am {

namespace {

struct GnArgs {
  const void* x;
  const void* dy;
  void* out;            // y or dx
  const float* gamma;
  const float* beta;
  float* mean;          // [n, G]: written by the forward, read by the backward
  float* rstd;
  float* part;          // workspace
  float* dgamma;
  float* dbeta;
  int64_t n, L;
  int C, G, c;
  float eps;
  int team, across;     // one-pass form: lanes of a group, lanes of one of its positions (powers of two)
  int64_t slots;        // ... and samples in flight
  int splits;           // spans of positions of a sample (two-pass form)
  int64_t span;         // positions of a span
};

// V elements from memory as floats.
template <bool F32, int V>
__device__ __forceinline__ void ld(const void* p, int64_t at, float* v) {
  if constexpr (F32) {
    const float* q = (const float*)p + at;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *(const float4*)(q + i);
        v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = q[i];
    }
  } else {
    const uint16_t* q = (const uint16_t*)p + at;
    if constexpr (V == 8) {
      const u32x4 w = *(const u32x4*)q;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else if constexpr (V == 4) {
      const uint2 w = *(const uint2*)q;
      v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = bf16_value(q[i]);
    }
  }
}
template <bool F32, int V>
__device__ __forceinline__ void st(void* p, int64_t at, const float* v) {
  if constexpr (F32) {
    float* q = (float*)p + at;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V; i += 4) *(float4*)(q + i) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] = v[i];
    }
  } else {
    uint16_t* q = (uint16_t*)p + at;
    if constexpr (V == 8) {
      *(u32x4*)q = u32x4{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[4], v[5]),
                         cvt_pk_bf16(v[6], v[7])};
    } else if constexpr (V == 4) {
      *(uint2*)q = uint2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] = (uint16_t)bf16_bits(v[i]);
    }
  }
}
template <int V>
__device__ __forceinline__ void ldp(const float* p, int c, float none, float* v) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = p ? p[c + i] : none;
}

template <bool SILU>
__device__ __forceinline__ float act_of(float z) {
  return SILU ? siluf_(z) : z;
}
template <bool SILU>
__device__ __forceinline__ float act_slope(float z) {
  return SILU ? silu_primef_(z) : 1.0f;
}

__device__ __forceinline__ float team_sum(float v, int team) {
  for (int s = team >> 1; s; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// -------------------------------------------------------------------------- one pass: a team a group

// BWD: the gradients; a team keeps its group over the rows it walks, so its lanes keep the channels
// whose dgamma, dbeta they sum.
template <bool F32, int V, int NI, bool SILU, bool BWD>
__global__ __launch_bounds__(256) void gn_rows(GnArgs a) {
  const int team = a.team, lane = threadIdx.x & (team - 1);
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / team;
  const int g = (int)(id % a.G);
  const int64_t slot = id / a.G;
  const bool on = slot < a.slots;
  float ga[NI][V], be[NI][V];
  bool in[NI];
  int at[NI];           // offset in the sample
  // one position: the team's lanes side by side, NI times; several: `across` lanes a position
  const int across = a.across;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int l = a.L > 1 ? i * (team / across) + lane / across : 0;
    const int c = (a.L > 1 ? lane % across : i * team + lane) * V;
    in[i] = on && c < a.c && l < a.L;
    at[i] = l * a.C + c;
#pragma unroll
    for (int k = 0; k < V; ++k) ga[i][k] = 1.0f, be[i][k] = 0.0f;
    if (in[i]) {
      ldp<V>(a.gamma, g * a.c + c, 1.0f, ga[i]);
      ldp<V>(a.beta, g * a.c + c, 0.0f, be[i]);
    }
  }
  const float inv = 1.0f / ((float)a.c * (float)a.L);
  float dg[NI][V], db[NI][V];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dg[i][k] = db[i][k] = 0.0f;

  // the next sample is on its way while this one is computed
  float nx[NI][V], nd[BWD ? NI : 1][V], nm = 0.0f, nr = 0.0f;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.n;
    const int64_t base = r * a.L * a.C + (int64_t)g * a.c;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int k = 0; k < V; ++k) nx[i][k] = 0.0f;
      if (live && in[i]) ld<F32, V>(a.x, base + at[i], nx[i]);
      if constexpr (BWD) {
#pragma unroll
        for (int k = 0; k < V; ++k) nd[i][k] = 0.0f;
        if (live && in[i]) ld<F32, V>(a.dy, base + at[i], nd[i]);
      }
    }
    if constexpr (BWD) {
      nm = live ? a.mean[r * a.G + g] : 0.0f;
      nr = live ? a.rstd[r * a.G + g] : 0.0f;
    }
  };
  int64_t r = on ? slot : a.n;
  fetch(r);
  for (; __any(r < a.n); r += a.slots) {
    const bool live = r < a.n;
    const int64_t base = r * a.L * a.C + (int64_t)g * a.c;
    float x[NI][V], d[BWD ? NI : 1][V];
    const float mean_in = nm, rstd_in = nr;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[i][k] = nx[i][k];
        if constexpr (BWD) d[i][k] = nd[i][k];
      }
    fetch(r + a.slots);
    if constexpr (!BWD) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) s += x[i][k];
      const float mean = team_sum(s, team) * inv;
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x[i][k] -= mean;
          if (in[i]) q += x[i][k] * x[i][k];
        }
      const float rstd = 1.0f / sqrtf(team_sum(q, team) * inv + a.eps);
      if (live && lane == 0) {
        if (a.mean) a.mean[r * a.G + g] = mean;
        if (a.rstd) a.rstd[r * a.G + g] = rstd;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) x[i][k] = act_of<SILU>(x[i][k] * rstd * ga[i][k] + be[i][k]);
        if (live && in[i]) st<F32, V>(a.out, base + at[i], x[i]);
      }
    } else {
      const float mean = mean_in, rstd = rstd_in;
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float xh = in[i] ? (x[i][k] - mean) * rstd : 0.0f;
          const float dz = d[i][k] * act_slope<SILU>(xh * ga[i][k] + be[i][k]);
          dg[i][k] += dz * xh;
          db[i][k] += dz;
          x[i][k] = xh;
          d[i][k] = dz * ga[i][k];
          s1 += d[i][k];
          s2 += d[i][k] * xh;
        }
      s1 = team_sum(s1, team) * inv;
      s2 = team_sum(s2, team) * inv;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) x[i][k] = rstd * (d[i][k] - s1 - x[i][k] * s2);
        if (live && in[i]) st<F32, V>(a.out, base + at[i], x[i]);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    if (a.L > 1) {  // positions of a lane, then the lanes of a channel
#pragma unroll
      for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int i = 1; i < NI; ++i) dg[0][k] += dg[i][k], db[0][k] += db[i][k];
        for (int s = team >> 1; s >= across; s >>= 1) {
          dg[0][k] += __shfl_xor(dg[0][k], s);
          db[0][k] += __shfl_xor(db[0][k], s);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (in[i] && (a.L == 1 || (i == 0 && lane < across))) {
        const int64_t p = (slot * 2) * a.C + g * a.c + at[i];  // channels a multiple of V: aligned like X
        st<true, V>(a.part, p, dg[i]);
        st<true, V>(a.part, p + a.C, db[i]);
      }
  }
}

// Sums over rows of partial sums [count][2][C]: dgamma, dbeta [C], or with several pieces of the rows
// (gridDim.z) one such row of sums for each piece.
__global__ __launch_bounds__(1024) void gn_channels(const float* part, int64_t count, int C, float* dgamma,
                                                    float* dbeta, float* pieces) {
  __shared__ float s[16][64];
  const int col = threadIdx.x & 63, rl = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + col, which = blockIdx.y;
  const int64_t per = (count + gridDim.z - 1) / gridDim.z, r0 = blockIdx.z * per, r1 = min(r0 + per, count);
  float v = 0.0f;
  if (c < C) {
#pragma unroll 4
    for (int64_t r = r0 + rl; r < r1; r += 16) v += part[(r * 2 + which) * C + c];
  }
  s[rl][col] = v;
  __syncthreads();
  if (rl == 0 && c < C) {
    for (int k = 1; k < 16; ++k) v += s[k][col];
    float* out = pieces ? pieces + (int64_t)(blockIdx.z * 2 + which) * C : which ? dbeta : dgamma;
    if (out) out[c] = v;
  }
}

// ------------------------------------------------------- two passes: spans of positions of a sample

// A count, a mean and a sum of squared differences to it; and their union (Chan et al.).
struct Mom {
  float n, mean, m2;
};
__device__ __forceinline__ Mom join(Mom a, Mom b) {
  const float n = a.n + b.n;
  if (n == 0.0f) return a;
  const float d = b.mean - a.mean, f = b.n / n;
  return Mom{n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}

// Which vectors of V channels and which rows of a span a thread takes.
template <int V>
struct Lanes {
  int cv, rr, rt;
  bool on;
  __device__ Lanes(const GnArgs& a) {
    const int CV = a.C / V;
    if (CV >= 256) {
      rt = 1, rr = 0, cv = blockIdx.y * 256 + threadIdx.x;
      on = cv < CV;
    } else {
      rt = 256 / CV, rr = threadIdx.x / CV, cv = threadIdx.x % CV;
      on = rr < rt;
    }
  }
};

// part: [n * splits][C / V] pairs (mean, m2)
template <bool F32, int V>
__global__ __launch_bounds__(256) void gn_moments(GnArgs a) {
  constexpr int B = 4;
  __shared__ Mom sm[256];
  const Lanes<V> w(a);
  for (int64_t blk = blockIdx.x; blk < a.n * a.splits; blk += gridDim.x) {
    const int64_t smp = blk / a.splits;
    const int64_t l0 = (blk % a.splits) * a.span, l1 = min(l0 + a.span, a.L);
    Mom m = {0.0f, 0.0f, 0.0f};
    if (w.on) {
      const int64_t base = smp * a.L * a.C + (int64_t)w.cv * V;
      for (int64_t l = l0 + w.rr; l < l1; l += (int64_t)w.rt * B) {
        float v[B][V];
        int cnt = 0;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (l + k * w.rt < l1) {
            ld<F32, V>(a.x, base + (l + k * w.rt) * a.C, v[k]);
            ++cnt;
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
          }
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) s += v[k][i];
        Mom b = {(float)(cnt * V), 0.0f, 0.0f};
        b.mean = s / b.n;
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (k < cnt) {
#pragma unroll
            for (int i = 0; i < V; ++i) b.m2 += (v[k][i] - b.mean) * (v[k][i] - b.mean);
          }
        m = join(m, b);
      }
    }
    if (w.rt > 1) {
      sm[threadIdx.x] = m;
      __syncthreads();
      if (w.on && w.rr == 0)
        for (int k = 1; k < w.rt; ++k) m = join(m, sm[threadIdx.x + k * (a.C / V)]);
    }
    if (w.on && w.rr == 0) {
      float* p = a.part + (blk * (a.C / V) + w.cv) * 2;
      p[0] = m.mean;
      p[1] = m.m2;
    }
    __syncthreads();
  }
}

// mean, rstd of a (sample, group): one workgroup.
template <int V>
__global__ __launch_bounds__(256) void gn_stats(GnArgs a, float* mean, float* rstd) {
  __shared__ Mom sm[4];
  const int per = a.c / V;
  for (int64_t grp = blockIdx.x; grp < a.n * a.G; grp += gridDim.x) {
    const int64_t smp = grp / a.G;
    const int g = (int)(grp % a.G);
    Mom m = {0.0f, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < (int64_t)a.splits * per; i += 256) {
      const int sp = (int)(i / per), cv = g * per + (int)(i % per);
      const float cnt = (float)(min(a.span, a.L - sp * a.span) * V);
      const float* p = a.part + ((smp * a.splits + sp) * (a.C / V) + cv) * 2;
      m = join(m, Mom{cnt, p[0], p[1]});
    }
    for (int s = 32; s; s >>= 1) m = join(m, Mom{__shfl_xor(m.n, s), __shfl_xor(m.mean, s), __shfl_xor(m.m2, s)});
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int k = 1; k < 4; ++k) m = join(m, sm[k]);
      mean[grp] = m.mean;
      rstd[grp] = 1.0f / sqrtf(m.m2 / m.n + a.eps);
    }
    __syncthreads();
  }
}

template <bool F32, int V, bool SILU>
__global__ __launch_bounds__(256) void gn_apply(GnArgs a) {
  const Lanes<V> w(a);
  if (!w.on) return;
  for (int64_t blk = blockIdx.x; blk < a.n * a.splits; blk += gridDim.x) {
    const int64_t smp = blk / a.splits;
    const int64_t l0 = (blk % a.splits) * a.span, l1 = min(l0 + a.span, a.L);
    const int c = w.cv * V, g = c / a.c;
    float ga[V], be[V];
    ldp<V>(a.gamma, c, 1.0f, ga);
    ldp<V>(a.beta, c, 0.0f, be);
    const float mean = a.mean[smp * a.G + g], rstd = a.rstd[smp * a.G + g];
    const int64_t base = smp * a.L * a.C + c;
#pragma unroll 4
    for (int64_t l = l0 + w.rr; l < l1; l += w.rt) {
      float v[V];
      ld<F32, V>(a.x, base + l * a.C, v);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_of<SILU>((v[i] - mean) * rstd * ga[i] + be[i]);
      st<F32, V>(a.out, base + l * a.C, v);
    }
  }
}

// part: [n * splits][2][C], sums of dz xh and of dz over a span
template <bool F32, int V, bool SILU>
__global__ __launch_bounds__(256) void gn_sums(GnArgs a) {
  __shared__ float sm[2][256][V];
  const Lanes<V> w(a);
  const int c = w.cv * V;
  for (int64_t blk = blockIdx.x; blk < a.n * a.splits; blk += gridDim.x) {
    const int64_t smp = blk / a.splits;
    const int64_t l0 = (blk % a.splits) * a.span, l1 = min(l0 + a.span, a.L);
    float dg[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dg[i] = db[i] = 0.0f;
    if (w.on) {
      const int g = c / a.c;
      float ga[V], be[V];
      ldp<V>(a.gamma, c, 1.0f, ga);
      ldp<V>(a.beta, c, 0.0f, be);
      const float mean = a.mean[smp * a.G + g], rstd = a.rstd[smp * a.G + g];
      const int64_t base = smp * a.L * a.C + c;
#pragma unroll 4
      for (int64_t l = l0 + w.rr; l < l1; l += w.rt) {
        float v[V], d[V];
        ld<F32, V>(a.x, base + l * a.C, v);
        ld<F32, V>(a.dy, base + l * a.C, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          const float dz = d[i] * act_slope<SILU>(xh * ga[i] + be[i]);
          dg[i] += dz * xh;
          db[i] += dz;
        }
      }
    }
    if (w.rt > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) sm[0][threadIdx.x][i] = dg[i], sm[1][threadIdx.x][i] = db[i];
      __syncthreads();
      if (w.on && w.rr == 0)
        for (int k = 1; k < w.rt; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dg[i] += sm[0][threadIdx.x + k * (a.C / V)][i];
            db[i] += sm[1][threadIdx.x + k * (a.C / V)][i];
          }
    }
    if (w.on && w.rr == 0) {
      float* p = a.part + blk * 2 * a.C + c;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = dg[i], p[a.C + i] = db[i];
    }
    __syncthreads();
  }
}

// mean(h xh), mean(h) of a (sample, group): [n, G, 2]
__global__ __launch_bounds__(1024) void gn_group_sums(GnArgs a, float* out) {
  __shared__ float sm[2][16];
  for (int64_t grp = blockIdx.x; grp < a.n * a.G; grp += gridDim.x) {
    const int64_t smp = grp / a.G;
    const int g = (int)(grp % a.G);
    float s2 = 0.0f, s1 = 0.0f;
    for (int64_t i = threadIdx.x; i < (int64_t)a.splits * a.c; i += blockDim.x) {
      const int ch = g * a.c + (int)(i % a.c);
      const float* p = a.part + (smp * a.splits + i / a.c) * 2 * a.C + ch;
      const float ga = a.gamma ? a.gamma[ch] : 1.0f;
      s2 += ga * p[0];
      s1 += ga * p[a.C];
    }
    s2 = team_sum(s2, 64), s1 = team_sum(s1, 64);
    if ((threadIdx.x & 63) == 0) sm[0][threadIdx.x >> 6] = s2, sm[1][threadIdx.x >> 6] = s1;
    __syncthreads();
    if (threadIdx.x < 2) {
      float t = 0.0f;
      for (int k = 0; k < (int)blockDim.x / 64; ++k) t += sm[threadIdx.x][k];
      out[grp * 2 + threadIdx.x] = t / ((float)a.L * (float)a.c);
    }
    __syncthreads();
  }
}

template <bool F32, int V, bool SILU>
__global__ __launch_bounds__(256) void gn_apply_grad(GnArgs a, const float* sums) {
  const Lanes<V> w(a);
  if (!w.on) return;
  for (int64_t blk = blockIdx.x; blk < a.n * a.splits; blk += gridDim.x) {
    const int64_t smp = blk / a.splits;
    const int64_t l0 = (blk % a.splits) * a.span, l1 = min(l0 + a.span, a.L);
    const int c = w.cv * V, g = c / a.c;
    float ga[V], be[V];
    ldp<V>(a.gamma, c, 1.0f, ga);
    ldp<V>(a.beta, c, 0.0f, be);
    const float mean = a.mean[smp * a.G + g], rstd = a.rstd[smp * a.G + g];
    const float s2 = sums[(smp * a.G + g) * 2], s1 = sums[(smp * a.G + g) * 2 + 1];
    const int64_t base = smp * a.L * a.C + c;
#pragma unroll 4
    for (int64_t l = l0 + w.rr; l < l1; l += w.rt) {
      float v[V], d[V];
      ld<F32, V>(a.x, base + l * a.C, v);
      ld<F32, V>(a.dy, base + l * a.C, d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (v[i] - mean) * rstd;
        const float h = d[i] * act_slope<SILU>(xh * ga[i] + be[i]) * ga[i];
        v[i] = rstd * (h - s1 - xh * s2);
      }
      st<F32, V>(a.out, base + l * a.C, v);
    }
  }
}

// ------------------------------------------------------------------------------------------- host

constexpr int kLanes = 64, kVecs = 4;             // a group of the one-pass form: at most 64 lanes x 4 vectors
constexpr int64_t kSlotSums = 1 << 21;            // channels of all samples in flight of the backward's
constexpr int64_t kLanesMost = 1 << 19;           // lanes in flight of the forward's: 32 waves a CU
constexpr int64_t kRowsAtOnce = 1024;             // more rows of partial sums are first summed in pieces
constexpr int64_t kPieces = 128;

// Samples in flight, each with lanes that walk every so-manieth sample.  The backward writes two rows of
// channel sums for each: 16 MB fill the chip (2048 channels of bf16, 16384 samples: 1024 in flight 55 us,
// 512 72 us, 2048 70 us).
int64_t row_slots(int64_t n, int C) { return std::min(n, std::max<int64_t>(1, kSlotSums / C)); }
int64_t forward_slots(int64_t n, int64_t lanes) { return std::min(n, std::max<int64_t>(1, kLanesMost / lanes)); }

void set_spans(GnArgs& a) {
  const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(a.n, 1));
  const int64_t s = std::max<int64_t>(1, std::min(want, (a.L + 15) / 16));
  a.span = (a.L + s - 1) / s;
  a.splits = (int)((a.L + a.span - 1) / a.span);
}

// Channels that a lane reads at once: a whole, aligned vector inside one group.
int vec_of(int c, const GnArgs& a, bool f32) {
  const uintptr_t at = (uintptr_t)a.x | (uintptr_t)a.dy | (uintptr_t)a.out;
  if (c % 8 == 0 && at % 16 == 0) return 8;
  if (c % 4 == 0 && at % (f32 ? 16 : 8) == 0) return 4;
  return 1;
}

// Workgroups of a two-pass kernel; beyond, each takes every so-manieth piece of the work.
unsigned blocks_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

int pow2_from(int64_t n) {
  int p = 1;
  while (p < n && p < kLanes) p <<= 1;
  return p;
}
bool one_pass(int64_t L, int c, int V) {
  const int64_t vecs = (c + V - 1) / V;
  return L == 1 ? vecs <= kLanes * kVecs : vecs <= kLanes && L <= (kLanes / pow2_from(vecs)) * kVecs;
}

template <bool F32, int V, bool SILU, bool BWD>
atlasmem_status rows_launch(GnArgs a, hipStream_t st) {
  const int vecs = (a.c + V - 1) / V;
  a.across = pow2_from(vecs);
  a.team = pow2_from(a.across * a.L);
  const int ni = a.L == 1 ? (vecs + a.team - 1) / a.team : (int)((a.L * a.across + a.team - 1) / a.team);
  a.slots = BWD ? row_slots(a.n, a.C) : forward_slots(a.n, (int64_t)a.G * a.team);
  const int64_t blocks = (a.slots * a.G * a.team + 255) / 256;
  if (blocks > INT32_MAX) return ATLASMEM_E_SHAPE;
  if (ni == 1) gn_rows<F32, V, 1, SILU, BWD><<<(unsigned)blocks, 256, 0, st>>>(a);
  else if (ni == 2) gn_rows<F32, V, 2, SILU, BWD><<<(unsigned)blocks, 256, 0, st>>>(a);
  else gn_rows<F32, V, 4, SILU, BWD><<<(unsigned)blocks, 256, 0, st>>>(a);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

template <bool F32, int V, bool SILU>
atlasmem_status forward(GnArgs a, hipStream_t st) {
  if (one_pass(a.L, a.c, V)) return rows_launch<F32, V, SILU, false>(a, st);
  const dim3 grid(blocks_of(a.n * a.splits), (unsigned)((a.C / V + 255) / 256));
  float* stats = a.part + 2 * a.n * a.splits * (int64_t)a.C;
  if (!a.mean) a.mean = stats;
  if (!a.rstd) a.rstd = stats + a.n * a.G;
  gn_moments<F32, V><<<grid, 256, 0, st>>>(a);
  AM_LAUNCH_CHECK();
  gn_stats<V><<<blocks_of(a.n * a.G), 256, 0, st>>>(a, a.mean, a.rstd);
  AM_LAUNCH_CHECK();
  gn_apply<F32, V, SILU><<<grid, 256, 0, st>>>(a);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

atlasmem_status channel_sums(const GnArgs& a, int64_t count, hipStream_t st) {
  const float* part = a.part;
  if (count > kRowsAtOnce) {
    float* pieces = a.part + 2 * count * a.C + 2 * a.n * a.G;
    gn_channels<<<dim3((a.C + 63) / 64, 2, kPieces), 1024, 0, st>>>(part, count, a.C, nullptr, nullptr, pieces);
    AM_LAUNCH_CHECK();
    part = pieces, count = kPieces;
  }
  gn_channels<<<dim3((a.C + 63) / 64, 2), 1024, 0, st>>>(part, count, a.C, a.dgamma, a.dbeta, nullptr);
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

template <bool F32, int V, bool SILU>
atlasmem_status backward(GnArgs a, hipStream_t st) {
  const bool channels = a.dgamma || a.dbeta;
  int64_t count;
  if (one_pass(a.L, a.c, V)) {
    float* part = a.part;
    if (!channels) a.part = nullptr;
    const atlasmem_status e = rows_launch<F32, V, SILU, true>(a, st);
    if (e != ATLASMEM_OK) return e;
    a.part = part;
    count = row_slots(a.n, a.C);
  } else {
    const dim3 grid(blocks_of(a.n * a.splits), (unsigned)((a.C / V + 255) / 256));
    float* sums = a.part + 2 * a.n * a.splits * (int64_t)a.C;
    gn_sums<F32, V, SILU><<<grid, 256, 0, st>>>(a);
    AM_LAUNCH_CHECK();
    gn_group_sums<<<blocks_of(a.n * a.G), (int64_t)a.splits * a.c > 1024 ? 1024 : 128, 0, st>>>(a, sums);
    AM_LAUNCH_CHECK();
    gn_apply_grad<F32, V, SILU><<<grid, 256, 0, st>>>(a, sums);
    AM_LAUNCH_CHECK();
    count = a.n * a.splits;
  }
  return channels ? channel_sums(a, count, st) : ATLASMEM_OK;
}

template <bool BWD, bool F32, int V>
atlasmem_status pick_act(const GnArgs& a, bool silu, hipStream_t st) {
  if constexpr (BWD) return silu ? backward<F32, V, true>(a, st) : backward<F32, V, false>(a, st);
  else return silu ? forward<F32, V, true>(a, st) : forward<F32, V, false>(a, st);
}

template <bool BWD>
atlasmem_status pick(const GnArgs& a, bool bf16, bool silu, hipStream_t st) {
  const int v = vec_of(a.c, a, !bf16);
  if (bf16) {
    if (v == 8) return pick_act<BWD, false, 8>(a, silu, st);
    if (v == 4) return pick_act<BWD, false, 4>(a, silu, st);
    return pick_act<BWD, false, 1>(a, silu, st);
  }
  if (v == 8) return pick_act<BWD, true, 8>(a, silu, st);
  if (v == 4) return pick_act<BWD, true, 4>(a, silu, st);
  return pick_act<BWD, true, 1>(a, silu, st);
}

GnArgs args_of(const GroupNorm& s) {
  GnArgs a = {};
  a.n = s.n, a.L = s.L, a.C = s.C, a.G = s.G, a.c = s.C / s.G;
  a.gamma = s.gamma, a.beta = s.beta;
  a.eps = s.eps;
  set_spans(a);
  return a;
}

}  // namespace

// Partial sums of spans (or of samples in flight), means of the groups, sums of pieces.  The form depends
// on the pointers' alignment: room for either.
int64_t group_norm_workspace_bytes(const GroupNorm& s, bool backward) {
  const GnArgs a = args_of(s);
  const bool rows = one_pass(a.L, a.c, 1);  // whatever the alignment
  if (!backward) return rows ? 0 : 4 * (2 * a.n * a.splits * (int64_t)a.C + 2 * a.n * a.G);
  const int64_t count = std::max(row_slots(a.n, a.C), rows ? (int64_t)0 : a.n * a.splits);
  return 4 * (2 * count * a.C + 2 * a.n * a.G + (count > kRowsAtOnce ? 2 * kPieces * a.C : 0));
}

atlasmem_status group_norm(const GroupNorm& s, const void* X, void* Y, float* mean, float* rstd, void* workspace,
                           hipStream_t st) {
  GnArgs a = args_of(s);
  a.x = X, a.out = Y, a.mean = mean, a.rstd = rstd, a.part = (float*)workspace;
  return pick<false>(a, s.bf16, s.silu, st);
}

atlasmem_status group_norm_backward(const GroupNorm& s, const void* X, const void* dY, const float* mean,
                                    const float* rstd, void* dX, float* dgamma, float* dbeta, void* workspace,
                                    hipStream_t st) {
  GnArgs a = args_of(s);
  a.x = X, a.dy = dY, a.out = dX, a.part = (float*)workspace;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.dgamma = dgamma, a.dbeta = dbeta;
  if (s.n == 0) return dgamma || dbeta ? channel_sums(a, 0, st) : ATLASMEM_OK;
  return pick<true>(a, s.bf16, s.silu, st);
}

}  // namespace am
