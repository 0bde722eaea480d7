// Softmax cross entropy over a large vocabulary, without keeping the logits (gfx950).
//   z = X W^T, lse_i = log sum_v exp z_iv, loss_i = lse_i - z_i,y_i
//   G_iv = exp(z_iv - lse_i) - [v = y_i],  dX_i = dloss_i (G W)_i,  dW = G^T (dloss X)
// The forward computes tiles of z and leaves of each row and tile its maximum and sum of exponentials;
// the backward computes them again by pieces of the vocabulary, writes the piece's G (bf16), and both
// products read it.  Three matrix products of one engine:
//   z   a = W (lanes v), b = X (lanes i): both rows along the contraction
//   dX  a = W (lanes d, rows across the contraction: read transposed from LDS), b = G
//   dW  a = X, b = G, both across the contraction
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
#include "logits.h"

namespace am {

namespace {

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

// ------------------------------------------------------------------------------------------- host

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
  if (gather) e = rows_that_count(s.n, s.vocab, labels, nullptr, ws.index, ws.at, ws.count, ws.scale, ws.equal, st);
  const int *index = gather ? ws.index : nullptr, *count = gather ? ws.count : nullptr;
  if (e == ATLASMEM_OK && (gather || !direct(X, s.d, s.bf16)))
    e = copy_rows(X, s.bf16, s.n, s.d, p.dp, index, count, ws.x, st);
  if (e == ATLASMEM_OK && !direct(W, s.d, s.bf16))
    e = copy_rows(W, s.bf16, s.vocab, s.d, p.dp, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  GemmArgs g = {};
  g.part = ws.part;
  g.a = direct(W, s.d, s.bf16) ? W : ws.w;
  g.b = gather || !direct(X, s.d, s.bf16) ? ws.x : X;
  g.lda = g.ldb = p.dp;
  g.na = s.vocab, g.nb = s.n, g.K = p.dp;
  g.count = count;
  g.parts = p.parts;
  e = gemm<false, false, EPI_LSE>(g, s.bf16, p.side, st);
  if (e != ATLASMEM_OK) return e;
  xe_join<<<(unsigned)((s.n + 3) / 4), 256, 0, st>>>(g.part, g.parts, gather ? ws.at : nullptr, X, W, s.bf16,
                                                     direct(X, s.d, s.bf16) && direct(W, s.d, s.bf16), s.n, s.d, s.vocab, labels, loss,
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
  atlasmem_status e = rows_that_count(s.n, s.vocab, labels, dloss, ws.index, ws.at, ws.count, ws.scale,
                                      ws.equal, st);
  if (e == ATLASMEM_OK)
    e = copy_rows(X, s.bf16, s.n, s.d, p.dp, ws.index, ws.count, ws.x, st);
  if (e == ATLASMEM_OK && !direct(W, s.d, s.bf16))
    e = copy_rows(W, s.bf16, s.vocab, s.d, p.dp, nullptr, nullptr, ws.w, st);
  if (e != ATLASMEM_OK) return e;
  const char* wa = direct(W, s.d, s.bf16) ? (const char*)W : ws.w;
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
