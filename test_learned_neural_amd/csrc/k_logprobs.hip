// Log probabilities of given tokens, the entropy of each row and its top alternatives, without keeping the
// logits (gfx950).
//   z = X W^T,  lse_i = log sum_v exp(scale z_iv),  logprob_i = scale z_i,token - lse_i,
//   entropy_i = lse_i - sum_v p_iv scale z_iv,  alternatives: the classes of the largest z
// One pass of the product engine leaves of each row and tile its maximum, its sum of exponentials and their
// product with z; a workgroup for each row joins them.
//
// Alternatives.  Which class is larger is decided in 64 bits, so that an answer does not depend on how a sum
// was cut: equal logits go to the lowest index.  The matrix cores' z is off by at most
// c sum |x w| (c: the roundings on a term's way), and so by c |x| |w| (Cauchy and Schwarz), or where w has one large
// entry, as a finite mask is, by c (|z| + 2 |x| |w'|) with w' the others.  z + c (|z| + |x| far_norm(w)) is an upper
// bound that holds for both, and a mask does not widen its neighbours' (1100 x 1024 x 32003, two fifths of the classes
// masked by -1e9: 0.20 ms; by |w| alone nearly every class was computed, 34 ms).  A
// lane's 16 to 64 classes of a row are a group; of each the four largest z are kept, as how far they are below the
// tile's maximum, with the class's place in the six bits that this costs.  The row's workgroup computes the best
// classes by their bounds in 64 bits, and has a lower bound of the last alternative; then every class whose bound
// passes it is computed too: a group whose fourth bound passes as a whole.
//
// What bounds it: few rows the bytes of W (1 x 1024 x 50257 bf16: products 21.6 us, 4.8 TB/s, rows 15 us; 64 x 2048 x
// 65536: 45 us, 6.0 TB/s with W partly in the last-level cache, and 26), many the matrix cores (8192 x 2048 x 65536, a
// tenth left out: 1.74 ms, 1.14 PFLOP/s, with 20 alternatives; 2047 x 1024 x 32000 without: 121 us, 1.11 PFLOP/s).
// One bound a group of classes side by side, without their places, had whole groups computed: rows 1.81 ms, now 0.26.
#include "logits.h"

namespace am {

namespace {

// far_norm of a row of a bf16 matrix.  A wave's.
template <bool ERRS>
__device__ __forceinline__ float norm_of(const uint16_t* x, int dp, int lane) {
  float s = 0.0f;
#pragma unroll 4
  for (int c = lane * 8; c < dp; c += 512) {
    const u32x4 w = *(const u32x4*)(x + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xFFFF0000u);
      s = fmaf(lo, lo, fmaf(hi, hi, s));
    }
  }
  float part = s;
  for (int k = 32; k; k >>= 1) {
    s += __shfl_xor(s, k);
    if (ERRS) part = fmaxf(part, __shfl_xor(part, k));
  }
  return in_range(s) && (!ERRS || no_large_entry(s, part)) ? sqrtf(s) : far_norm<true, ERRS>(x, dp, lane, 64);
}
// Memory: W and X once more, 268 MB in 44 us and 30 in 7 (6.1 and 4.3 TB/s).  Taken in the products' loop instead where
// those leave time for it (see kNorms).
__global__ __launch_bounds__(256) void lp_row_norms(const uint16_t* x, int64_t rows, const int* count, int dp, float* out) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= (count ? *count : rows)) return;
  const float v = norm_of<false>(x + r * dp, dp, threadIdx.x & 63);
  if ((threadIdx.x & 63) == 0) out[r] = v;
}
// The largest norm of each group's classes: a workgroup's waves take its 64 in turn.
__global__ __launch_bounds__(256) void lp_group_norms(const uint16_t* w, int64_t vocab, int dp, int side, int apart,
                                                      int tiles, float* out) {
  __shared__ float best[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float m = 0.0f;
  for (int code = wave; code < side / 4; code += 4) {
    const int64_t c = group_class(blockIdx.x, code, side, apart, tiles);
    if (c >= vocab) continue;
    m = fmaxf(m, norm_of<true>(w + c * dp, dp, lane));
  }
  if (lane == 0) best[wave] = m;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
}

struct RowArgs {
  const float4* sums;
  const uint4* keys;
  const float *tops, *a_norm, *b_norm;
  float error;             // of z, relative to |a| |b|
  int parts, side, apart;
  const int* at;           // a row's place among those that count, or null: all are there
  const void *x, *w;       // as the products took them, [..][dp]
  int dp;
  int64_t n, vocab;
  const int64_t* tokens;   // or null
  float scale, k2;
  double per_k2;           // the difference and its product were rounded, to 2^-23
  int top;
  float *logprob, *entropy;
  int64_t* ids;
  float* top_logprobs;
};

constexpr int kTopMost = 64;         // alternatives
// z from here down, or so far below the row's largest, are no alternatives.  (2^20 log2 e times that is a float: keys
// hold any distance of less, whatever the scale.)
constexpr float kMasked = -1.0e38f;
constexpr double kBelow = 1.0e32;

// (z, class) before (y, other): larger, or equal and of lower index
__device__ __forceinline__ bool ahead(double z, int c, double y, int o) { return z > y || (z == y && c < o); }

// Two parts of a row's maximum m, sum of e = exp(scale (z - m)) and sum of e (z - m).
__device__ __forceinline__ void join(float& m, float& s, float& t, float om, float os, float ot, float k2) {
  const float to = fmaxf(m, om), from = to > -INFINITY ? to : 0.0f;
  const float x = m - from, ox = om - from;  // minus infinity, or a masked class's, where e is zero
  const float e = __builtin_amdgcn_exp2f(x * k2), oe = __builtin_amdgcn_exp2f(ox * k2);
  t = (e > 0.0f ? e * fmaf(s, x, t) : 0.0f) + (oe > 0.0f ? oe * fmaf(os, ox, ot) : 0.0f);
  s = fmaf(s, e, os * oe);
  m = to;
}

// The row's numbers and alternatives.  What it reads is small (16 bytes a group, 40 MB at 8192 x 2048 x 65536, and some
// rows of W out of L2); its waits are for those reads, one behind the other: bounds, classes, selection, bounds.  So a
// workgroup a row, and the rows that fit on the chip hide each other's waits (8192 x 2048 x 65536: 260 us of 2.1 ms).
// Its threads NT:
//   1024 for up to 256 rows, whose time is one row's and where many classes are computed at once (1 x 1024 x 50257
//     36.8 us, with 256 threads 39.6; 512 rows 129 against 113), unless the rows are short and a wave takes several
//     classes at a time (17 x 80 x 642: 50, with 256 46);
//   64 above 1024 rows and up to 32 alternatives, since joins, bounds and selections cost instructions in every wave
//     (8192 x 2048 x 65536 2.33 -> 2.27 ms, 8192 x 256 x 500 161 -> 43 us); with more, a wave's lanes are few places
//     for a first choice, and many classes pass its bar (8192 x 256 x 2048, 30 of them: 288 -> 190 us; 4096 x 512 x
//     2048, 40: 205 -> 223; 8192 x 256 x 65536, 64: 1.14 -> 4.25 ms);
//   256 else.
// First choices are of all groups' four bounds where those are few, else of the threads' largest (12224 x 33 x 1135, 64
// alternatives: 2.0 ms -> 0.76; in short rows several classes a wave 0.48).  Loops are kept rolled: few rows wait for
// their instructions.
template <int NT, bool BF16>
__global__ __launch_bounds__(NT) void lp_rows(RowArgs g) {
  constexpr int NW = NT / 64;
  constexpr int kTake = 64 / NW;  // classes a wave computes between two selections
  constexpr int kList = kTopMost + 64;
  constexpr int kScan = NT < 1024 ? 4 : 2;  // groups a thread looks at together
  constexpr int kFirst = NT == 64 ? 256 : 1024;  // places for a first choice
  constexpr int kFlush = NT == 64 ? 256 : 1024;  // pending items
  __shared__ float4 part[NW];
  __shared__ uint32_t first[kFirst];
  __shared__ uint32_t bound;
  __shared__ double lz[2][kList];
  __shared__ int lc[2][kList];
  __shared__ int items[kFlush + 4 * kScan * NT];
  __shared__ int counts[2];       // entries of the list, pending items
  __shared__ double token_z;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  // the largest logit that a key stands for (minus infinity: a masked class)
  auto bound_of = [&](float top, uint32_t key) {
    const uint32_t b = key & ~63u;
    if (b >= 0x7f800000u) return -(double)INFINITY;
    const double z = (double)top - (double)__uint_as_float(b) * g.per_k2;
    return fma(fabs(z), (double)g.error, z);
  };
#pragma unroll 1
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
    const int place = __builtin_amdgcn_readfirstlane(g.at ? g.at[r] : (int)r);

    // the best class of each thread's groups, by their largest bound
    const int groups = 4 * g.parts;
    const uint4* keys = g.keys + (int64_t)place * groups;
    const float* tops = g.tops + (int64_t)place * (groups / 2);
    float b_norm = g.top ? g.b_norm[place] : 0.0f;
    if (g.top && b_norm == 0.0f) {  // a row of zeros, all of whose logits are equal, or one whose squares vanish
      const u32x4* x = (const u32x4*)g.x + (int64_t)place * (g.dp / (BF16 ? 8 : 4));
      uint32_t any = 0;
#pragma unroll 1
      for (int i = tid; i < g.dp / (BF16 ? 8 : 4); i += NT) any |= x[i][0] | x[i][1] | x[i][2] | x[i][3];
      if (__syncthreads_or(any & (BF16 ? 0x7fff7fffu : 0x7fffffffu))) b_norm = kVanished;
    }
    const float error = b_norm < 3.0e38f ? g.error * b_norm : 3.0e38f;
    // what the maximum of group i may be in 64 bits, without c |z|.  Zeros have no error; what else was flushed, or
    // rounded among the smallest floats, is less than 2^-100 (2^14 products of 2^-126; a key times 1 / k2)
    auto top_of = [&](int i) {
      const float top = tops[(i >> 2) * 2 + (i & 1)], a_norm = g.a_norm[i];
      const float t = error > 0.0f && a_norm > 0.0f ? fmaf(error, a_norm, top + 0x1p-100f) : top;
      return fmaf(fabsf(t), 0x1p-21f, t);
    };
    // bound i of all groups' four, and its class
    auto bound_at = [&](int i, int& c) {
      const uint32_t key = ((const uint32_t*)keys)[i];
      c = (int)group_class(i >> 2, key & 63, g.side, g.apart, g.parts);
      const float b = (float)bound_of(top_of(i >> 2), key);
      return b > kMasked && c < g.vocab ? b : -INFINITY;
    };
    // floats in the order of whole numbers
    auto order_of = [](float b) { return __float_as_uint(b) ^ (__float_as_int(b) >> 31 | 0x80000000u); };
    const bool few = 4 * groups <= kFirst;  // each bound may be a first choice
    float best = -INFINITY;
    int own = 0x7fffffff;
    if (g.top && !few) {
#pragma unroll 1
      for (int i0 = tid; i0 < groups; i0 += kScan * NT) {
        float top[kScan];
        uint32_t key[kScan];
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
          const int i = i0 + q * NT;
          top[q] = i < groups ? top_of(i) : 0.0f, key[q] = i < groups ? keys[i].x : ~0u;
        }
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
          const float b = (float)bound_of(top[q], key[q]);
          if (b > best) best = b, own = (i0 + q * NT) * 64 + (key[q] & 63);
        }
      }
      if (best > -INFINITY) own = (int)group_class(own >> 6, own & 63, g.side, g.apart, g.parts);
      if (best <= kMasked || own >= g.vocab) best = -INFINITY;
      if (NT == 1024) {  // one of four threads'
#pragma unroll
        for (int k = 1; k < 4; k <<= 1) {
          const float o = __shfl_xor(best, k);
          const int c = __shfl_xor(own, k);
          if (o > best || (o == best && c < own)) best = o, own = c;
        }
      }
    }
    // the row's maximum, sum and first moment
    float m = -INFINITY, s = 0.0f, t = 0.0f;
#pragma unroll 1
    for (int i = tid; i < g.parts; i += NT) {
      const float4 q = g.sums[(int64_t)place * g.parts + i];
      join(m, s, t, q.x, q.y, q.z, g.k2);
    }
#pragma unroll 1
    for (int k = 32; k; k >>= 1) {
      const float om = __shfl_xor(m, k), os = __shfl_xor(s, k), ot = __shfl_xor(t, k);
      join(m, s, t, om, os, ot, g.k2);
    }
    __syncthreads();  // the last row's shared values have been read
    if (lane == 0) part[wave] = float4{m, s, t, 0.0f};
    const uint32_t order = order_of(best);
    constexpr int kChoices = NT == 1024 ? 256 : NT;
    if (!few && (NT < 1024 || tid % 4 == 0)) first[NT < 1024 ? tid : tid / 4] = order;
    if (g.top && few) {
#pragma unroll 1
      for (int i = tid; i < kFirst; i += NT) {
        int c;
        first[i] = i < 4 * groups ? order_of(bound_at(i, c)) : 0;
      }
    }
    if (tid < 2) counts[tid] = 0;
    __syncthreads();
    if (NW > 1) {
      const float4 q = part[lane % NW];
      m = q.x, s = q.y, t = q.z;
#pragma unroll 1
      for (int k = NW / 2; k; k >>= 1) {
        const float om = __shfl_xor(m, k), os = __shfl_xor(s, k), ot = __shfl_xor(t, k);
        join(m, s, t, om, os, ot, g.k2);
      }
    }
    // one lane's for all: joins of two sums round differently from either side, and a row's numbers have one lse
    auto one = [](float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); };
    m = one(m), s = one(s), t = one(t);
    const float log_s = logf(s), lse = fmaf(g.scale, m, log_s);
    const bool none = lse == -INFINITY, bad = !none && !(fabsf(lse) < INFINITY);

    // The list of what is known in 64 bits, in order; the last of its `top`, if there are so many, is the bar.
    int known = 0, buf = 0;
    double bar = -INFINITY;
    int bar_class = 0x7fffffff;
    const double least = fmax((double)kMasked, (double)m - kBelow);
    if (!none && !bad) {
      // first the best `top` of the threads' classes (by 20 bits, which a wave finds one by one), and the token
      if (g.top) {
        if (wave == 0) {
          uint32_t b = 0;
          auto find = [&](auto waves) {
            constexpr int N = decltype(waves)::value;
            uint32_t v[N];
#pragma unroll
            for (int w = 0; w < N; ++w) v[w] = first[w * 64 + lane];
#pragma unroll 1
            for (uint32_t bit = 0x80000000u; bit >= 0x1000u; bit >>= 1) {
              int above = 0;
#pragma unroll
              for (int w = 0; w < N; ++w) above += __popcll(__ballot(v[w] >= (b | bit)));
              if (above >= g.top) b |= bit;
            }
          };
          if (few) find(std::integral_constant<int, kFirst / 64>{});
          else find(std::integral_constant<int, kChoices / 64>{});
          if (lane == 0) bound = b;
        }
        __syncthreads();
        if (few) {
#pragma unroll 1
          for (int i = tid; i < 4 * groups; i += NT) {
            if (first[i] < bound) continue;
            int c;
            if (bound_at(i, c) > -INFINITY && c != (int)y) items[atomicAdd(&counts[1], 1)] = c;
          }
        } else if ((NT < 1024 || tid % 4 == 0) && best > -INFINITY && order >= bound && own != (int)y) {
          items[atomicAdd(&counts[1], 1)] = own;
        }
      }
      if (tid == 0) items[atomicAdd(&counts[1], 1)] = (int)y;
      __syncthreads();
      // what is pending is computed, a class or (negative) a quarter of a group's, two at a time a wave; then
      // every class that may pass the bar is pending
      int scanned = g.top ? 0 : groups;
      auto take = [&](double z, int c) {
        if (c == (int)y) token_z = z;
        if (g.top && z > least && ahead(z, c, bar, bar_class)) {
          const int e = known + atomicAdd(&counts[0], 1);
          lz[buf][e] = z, lc[buf][e] = c;
        }
      };
      const int bytes = g.dp * (BF16 ? 2 : 4), lanes = max(short_lanes(bytes), NW), sub = lane / lanes;
      const bool short_row = NT < 1024 && bytes <= kShort;
#pragma unroll 1
      while (true) {
        const int pending = counts[1];
        int at = wave, code = 0;
        auto next = [&]() {  // a class that is not known, or -1
          while (at < pending) {
            const int item = __builtin_amdgcn_readfirstlane(items[at]);
            int c = item;
            if (item < 0) c = (int)group_class(~item >> 2, (~item & 3) * (g.side / 16) + code++, g.side, g.apart, g.parts);
            if (item >= 0 || code == g.side / 16) at += NW, code = 0;
            if (c < g.vocab && !__any(lane < known && lc[buf][lane] == c)) return c;
          }
          return -1;
        };
        bool more = pending > 0;
#pragma unroll 1
        while (more) {
          if (short_row) {
#pragma unroll 1
            for (int k = 0; k < kTake && at < pending; k += 64 / lanes) {
              const int it = at + NW * sub;
              const int item = it < pending ? items[it] : -1;
              const int lead = __builtin_amdgcn_readfirstlane(item);
              int c = -1;
              if (lead < 0) {  // of a quarter of a group's, as many as there are places
                if (code + sub < g.side / 16)
                  c = (int)group_class(~lead >> 2, (~lead & 3) * (g.side / 16) + code + sub, g.side, g.apart, g.parts);
                code += 64 / lanes;
                if (code >= g.side / 16) at += NW, code = 0;
              } else {  // classes up to the next quarter
                const uint64_t end = __ballot(item < 0);
                const int taken = end ? __builtin_ctzll(end) / lanes : 64 / lanes;
                if (sub < taken) c = item;
                at += NW * taken;
              }
              if (c >= g.vocab) c = -1;
              const int have = lane < known ? lc[buf][lane] : -2;
#pragma unroll 1
              for (int j = 0; j < 64; j += lanes) {
                const bool dup = __any(have == __builtin_amdgcn_readlane(c, j));
                if (dup && sub * lanes == j) c = -1;
              }
              const double zc = short_dot<BF16>(g.x, g.w, place, max(c, 0), bytes, lanes, lane);
              if ((lane & (lanes - 1)) == 0 && c >= 0) take(zc, c);
            }
          } else {
#pragma unroll 1
            for (int k = 0; k < kTake; k += 2) {
              int c[2];
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                const int v = next();
                c[0] = q ? c[0] : v, c[1] = v;
              }
              if (c[0] < 0) break;
              double z[2];
              const int rows[2] = {c[0], max(c[1], 0)};
              row_dots<2, BF16>(g.x, g.w, place, rows, g.dp, lane, z);
              const double zc = lane ? z[1] : z[0];
              const int cc = lane ? c[1] : c[0];
              if (lane < 2 && cc >= 0) take(zc, cc);
            }
          }
          more = __syncthreads_or(at < pending);
          const int total = known + counts[0];
          if (total > known) {
#pragma unroll 1
            for (int e = tid; e < total; e += NT) {
              const double z = lz[buf][e];
              const int c = lc[buf][e];
              int before = 0;
#pragma unroll 4
              for (int i = 0; i < total; ++i) before += ahead(lz[buf][i], lc[buf][i], z, c);
              if (before < g.top) lz[buf ^ 1][before] = z, lc[buf ^ 1][before] = c;
            }
            buf ^= 1;
            known = min(total, g.top);
          }
          __syncthreads();
          if (g.top && known == g.top) bar = lz[buf][known - 1], bar_class = lc[buf][known - 1];
          if (tid == 0) counts[0] = 0;
          __syncthreads();
        }
        if (scanned >= groups) break;
        if (tid == 0) counts[1] = 0;
        __syncthreads();
        int found = 0;
#pragma unroll 1
        for (; scanned < groups && found <= kFlush; scanned += kScan * NT) {
          uint4 k[kScan];
          float top[kScan];
#pragma unroll
          for (int q = 0; q < kScan; ++q) {
            const int i = scanned + q * NT + tid;
            k[q] = i < groups ? keys[i] : uint4{~0u, ~0u, ~0u, ~0u}, top[q] = i < groups ? top_of(i) : 0.0f;
          }
#pragma unroll
          for (int q = 0; q < kScan; ++q) {
            // a bound that passes, or equals the bar where the group has a class of lower index
            const double b1 = bound_of(top[q], k[q].x);
            if (!(b1 > least && b1 >= bar)) continue;
            const int i = scanned + q * NT + tid;
            const int start = (int)group_class(i, 0, g.side, g.apart, g.parts);
            auto passes = [&](uint32_t key) {
              const double b = bound_of(top[q], key);
              return b > least && (b > bar || (b == bar && start < bar_class));
            };
            const bool whole = passes(k[q].w);
            const uint32_t one[3] = {k[q].x, k[q].y, k[q].z};
#pragma unroll 1
            for (int p = 0; p < 4; ++p) {
              const uint32_t key = p == 0 ? one[0] : p == 1 ? one[1] : one[2];
              if (whole) items[atomicAdd(&counts[1], 1)] = ~(4 * i + p);
              else if (p < 3 && passes(key))
                items[atomicAdd(&counts[1], 1)] = (int)group_class(i, key & 63, g.side, g.apart, g.parts);
            }
          }
          __syncthreads();
          found = counts[1];
          __syncthreads();
        }
      }
    }
    if (tid == 0) {
      // without lse, whose rounding would be the largest
      const double p = bad || none ? 0.0 : g.scale * (token_z - (double)m) - (double)log_s;
      const float h = log_s - g.scale * t / s;
      if (g.logprob) g.logprob[r] = bad ? NAN : none ? -INFINITY : p > 0.0 ? 0.0f : (float)p;
      if (g.entropy) g.entropy[r] = bad ? NAN : none || h < 0.0f ? 0.0f : h;
    }
    if (tid < g.top) {
      const bool there = tid < known;
      const double p = there ? g.scale * (lz[buf][tid] - (double)m) - (double)log_s : -INFINITY;
      g.ids[r * g.top + tid] = there ? lc[buf][tid] : -1;
      g.top_logprobs[r * g.top + tid] = bad ? NAN : p > 0.0 ? 0.0f : (float)p;
    }
  }
}

struct Plan {
  int el, dp, side, parts, apart;
  bool gather;
};
Plan plan_of(const TokenLogprobs& s, bool tokens) {
  Plan p = {};
  p.el = s.bf16 ? 2 : 4;
  p.dp = (int)up(s.d, s.bf16 ? 8 : 4);
  p.side = side_for(s.vocab, s.n, s.bf16);
  // Few groups for the alternatives asked for, whose fourth bound then often passes: smaller ones (17 x 80 x 642 with 64:
  // 108 -> 50 us; 12224 x 33 x 1135 with 20: 350 -> 115; 4096 x 512 x 4096 with 20: 163 -> 142).  The products of few rows
  // take longer in them (1 x 184 x 4771 with 64: 35 -> 47 us).
  // Their grids stay below 2^30 lanes.
  if ((s.n <= kFew ? 2 : 1) * s.vocab < (int64_t)s.top * p.side && s.n * s.vocab <= INT64_C(1) << 34) p.side = 64;
  p.parts = (int)((s.vocab + p.side - 1) / p.side);
  // Rows of a tile 64 apart: all tiles' (256 x 256, 2048 columns) takes 10% longer, their pages no longer at hand,
  // and 16 leave frequent classes together (rows 485 us instead of 380).  Byte offsets in a tile stay below 2^31.
  p.apart = 64;
  while (p.apart > p.parts || (int64_t)p.apart * p.side * p.dp * p.el > INT32_MAX) p.apart /= 2;
  p.gather = tokens && 2.0 * s.n * s.d * s.vocab * (s.bf16 ? 1 : 6) >= kGatherFrom;
  return p;
}

struct Space {
  int *index, *at, *count, *equal;
  float* scale;
  char *x, *w;
  float *a_norm, *b_norm;
  float4* sums;
  uint4* keys;
  float* tops;
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
    w.a_norm = (float*)take(16 * (int64_t)l.parts), w.b_norm = (float*)take(4 * s.n);
    w.keys = (uint4*)take(64 * s.n * (int64_t)l.parts), w.tops = (float*)take(8 * s.n * (int64_t)l.parts);
  }
  w.bytes = at - (char*)p;
  return w;
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
  g.parts = p.parts, g.apart = p.apart;
  g.sums = ws.sums;
  g.k2 = (float)(s.scale * kLog2e), g.k2_low = (float)(s.scale * kLog2e - g.k2);
  g.keys = ws.keys, g.tops = ws.tops, g.a_norm = ws.a_norm, g.b_norm = ws.b_norm;
  if (s.top && s.bf16 && p.side == 256) {
    lp_group_norms<<<(unsigned)(4 * p.parts), 256, 0, st>>>((const uint16_t*)g.a, s.vocab, p.dp, p.side, p.apart, p.parts,
                                                            ws.a_norm);
    AM_LAUNCH_CHECK();
    lp_row_norms<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>((const uint16_t*)g.b, s.n, count, p.dp, ws.b_norm);
    AM_LAUNCH_CHECK();
  }
  if (s.n <= kFew && (p.side == 128 || !s.bf16))
    e = s.top ? gemm_few<false, EPI_TOP>(g, s.bf16, st) : gemm_few<false, EPI_SUMS>(g, s.bf16, st);
  else
    e = s.top ? gemm<false, false, EPI_TOP>(g, s.bf16, p.side, st) : gemm<false, false, EPI_SUMS>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  RowArgs a = {};
  a.sums = ws.sums, a.keys = ws.keys, a.tops = ws.tops, a.parts = p.parts, a.side = p.side, a.apart = p.apart;
  a.a_norm = ws.a_norm, a.b_norm = ws.b_norm;
  // roundings on a term's way: eight for each of dp / 16 matrix instructions; in fp32 six instructions with
  // those for each 16 columns, and the planes that are not multiplied; a twentieth for the norms' own, and for |z| as it
  // was computed, off by up to 0.003 (16384 columns) of what it is
  a.error = ((s.bf16 ? 0.5f : 3.0f) * p.dp + 128.0f) * 0x1p-24f * 1.05f;
  a.at = p.gather ? ws.at : nullptr;
  a.x = g.b, a.w = g.a, a.dp = p.dp;
  a.n = s.n, a.vocab = s.vocab;
  a.tokens = tokens;
  a.scale = s.scale, a.k2 = g.k2, a.per_k2 = (1.0 - 0x1p-20) / g.k2, a.top = s.top;
  a.logprob = logprob, a.entropy = entropy, a.ids = top_ids, a.top_logprobs = top_logprobs;
  const unsigned rows = (unsigned)std::min<int64_t>(s.n, 1 << 20);
  auto launch = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (s.bf16) lp_rows<NT, true><<<rows, NT, 0, st>>>(a);
    else lp_rows<NT, false><<<rows, NT, 0, st>>>(a);
  };
  if (s.n <= 256 && p.dp * p.el > kShort) launch(std::integral_constant<int, 1024>{});
  else if (s.n > 1024 && s.top <= 32) launch(std::integral_constant<int, 64>{});
  else launch(std::integral_constant<int, 256>{});
  AM_LAUNCH_CHECK();
  return ATLASMEM_OK;
}

}  // namespace am
