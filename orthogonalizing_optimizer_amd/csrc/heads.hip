// Norms of queries and keys per head with the rotation by their positions in
// the same pass, and the gradient.
//
//   hat = x rstd,  rstd = 1 / sqrt(mean_j x_j^2 + eps),  u = hat w  (per head)
//   (y_a, y_b) = (u_a cos - u_b sin, u_b cos + u_a sin)   for the pairs (a, b),
//   angle = position freq_i,  i the pair's number;
// backwards
//   du = the rotation of dy by -angle,  a = w du,
//   dx = rstd (a - hat mean_j(a_j hat_j)),  dw = sum over tokens and heads of du hat.
//
// Bound by HBM: everything of a head stays in registers, so q and k are read
// once and written once, and the backward pass needs nothing but x.  A lane
// holds 16 columns, both members of 8 pairs, so the rotation moves nothing
// between lanes; a head takes G lanes (8 for 128 columns), a wave 64 / G heads
// at a time, and every lane of a wave needs the same 8 angles for all of a
// token's heads, which are computed once for them.
#include "checks.h"

namespace dion3 {
namespace {

struct Side {
  const void* x; const void* w; const void* dy;
  void* y;
  long long ldx, hsx, lddy, hsdy, ldy, hsy;
  int heads, batches;             // batches of 64 / G heads
};
struct HeadsP {
  Side s[2];                      // queries, keys
  const double* freqs;
  const void* pos;
  float* part;                    // gradient: one row of 2 D floats a workgroup, or null
  long long T, tasks;
  int D, r, G, parts;             // tasks: parts waves share a token's batches
  int pos64, wtype;
  float eps;
};

// The 16 columns of a lane: two chunks of 8, each with the run of columns that
// it lies in (base, length) and its place there.  Runs: the two halves of the
// rotated columns, or all of them where pairs are neighbours; the columns past
// them.
struct Item {
  int base[2], c[2], lim[2];
  bool on, rot;
};
template <bool IL>
__device__ __forceinline__ Item my_item(int j, int D, int r) {
  Item it;
  const int half = r / 2, nr = IL ? (r + 15) / 16 : (half + 7) / 8;
  it.rot = j < nr;
  if (it.rot) {
    it.on = true;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      it.base[k] = IL ? 0 : k * half;
      it.c[k] = IL ? 16 * j + 8 * k : 8 * j;
      it.lim[k] = IL ? r : half;
    }
  } else {
    const int t = (j - nr) * 16;
    it.on = t < D - r;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      it.base[k] = r;
      it.c[k] = t + 8 * k;
      it.lim[k] = D - r;
    }
  }
  return it;
}

// cos and sin of the lane's 8 angles: the angle in turns, reduced in 64 bits
// (a position of 2^20 times a frequency of 1 leaves no bits of a fraction in 32).
__device__ __forceinline__ void my_freqs(const HeadsP& p, int j, double (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = 8 * j + i < p.r / 2 ? p.freqs[8 * j + i] * 0.15915494309189533577 : 0.0;
}
__device__ __forceinline__ void turn_of(double at, const double (&f)[8], float (&co)[8],
                                        float (&si)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double t = at * f[i];
    sincospif(2.0f * (float)(t - rint(t)), &si[i], &co[i]);
  }
}
__device__ __forceinline__ double position(const HeadsP& p, long long t) {
  return p.pos64 ? (double)((const long long*)p.pos)[t] : (double)((const int*)p.pos)[t];
}

// Pairs (a, b) of the lane's columns: (v[0][i], v[1][i]), or neighbours.
template <bool IL>
__device__ __forceinline__ void rotate(float (&v)[2][8], const float (&co)[8], const float (&si)[8],
                                       bool on) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = IL ? v[i / 4][2 * (i & 3)] : v[0][i];
    float& b = IL ? v[i / 4][2 * (i & 3) + 1] : v[1][i];
    const float x = a, y = b;
    a = on ? __builtin_fmaf(x, co[i], -y * si[i]) : x;
    b = on ? __builtin_fmaf(y, co[i], x * si[i]) : y;
  }
}

template <class E>
__device__ __forceinline__ void load_weight(const HeadsP& p, const Side& s, const Item& it,
                                            float (&w)[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[k][e] = 0.0f;
    if (!it.on || s.heads == 0) continue;
    if (p.wtype == DION3_F32) load8((const float*)s.w + it.base[k], it.c[k], it.lim[k], w[k]);
    else load8((const E*)s.w + it.base[k], it.c[k], it.lim[k], w[k]);
  }
}

__device__ __forceinline__ float head_sum(float v, int G) {
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <class E, bool IL>
__global__ __launch_bounds__(256) void k_heads(HeadsP p) {
  const int lane = threadIdx.x & 63, G = p.G, per = 64 / G;
  const long long task = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= p.tasks) return;
  const long long t = task / p.parts;
  const int part = (int)(task - t * p.parts), nb = p.s[0].batches + p.s[1].batches;
  const Item it = my_item<IL>(lane & (G - 1), p.D, p.r);
  Raw8<E> raw[2];
  bool mine = false;
  auto ask = [&](int b) {
    const bool isk = b >= p.s[0].batches;
    const Side& s = p.s[isk];
    const int h = (isk ? b - p.s[0].batches : b) * per + lane / G;
    mine = it.on && h < s.heads;
    if (!mine) return;
    const E* row = (const E*)s.x + t * s.ldx + h * s.hsx;
#pragma unroll
    for (int k = 0; k < 2; ++k) raw[k] = fetch8(row + it.base[k], it.c[k], it.lim[k]);
  };
  ask(part);
  float w[2][2][8], co[8], si[8];
  load_weight<E>(p, p.s[0], it, w[0]);
  load_weight<E>(p, p.s[1], it, w[1]);
  double f[8];
  my_freqs(p, lane & (G - 1), f);
  turn_of(position(p, t), f, co, si);
  for (int b = part; b < nb; b += p.parts) {
    const bool isk = b >= p.s[0].batches;
    const Side& s = p.s[isk];
    const int h = (isk ? b - p.s[0].batches : b) * per + lane / G;
    float v[2][8];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (mine) chunk8(raw[k], it.c[k], it.lim[k], v[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] = mine ? v[k][e] : 0.0f;
        ss = __builtin_fmaf(v[k][e], v[k][e], ss);
      }
    }
    const bool now = mine;
    if (b + p.parts < nb) ask(b + p.parts);
    const float rs = 1.0f / sqrtf(head_sum(ss, G) / (float)p.D + p.eps);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * rs * (isk ? w[1][k][e] : w[0][k][e]);
    rotate<IL>(v, co, si, it.rot);
    if (!now) continue;
    E* row = (E*)s.y + t * s.ldy + h * s.hsy;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (it.c[k] < it.lim[k]) store8(row + it.base[k], it.c[k], it.lim[k], v[k]);
  }
}

// The weights' gradients: a lane adds up its columns over its tokens and
// heads, the lanes of equal columns and the workgroup's waves are joined at
// the end, and the workgroups' rows by k_join_columns, each in a fixed order.
template <class E, bool IL>
__global__ __launch_bounds__(256) void k_heads_grad(HeadsP p) {
  extern __shared__ float sh[];                        // 3 waves x 2 sides x D
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, G = p.G, per = 64 / G;
  const int nb = p.s[0].batches + p.s[1].batches;
  const Item it = my_item<IL>(lane & (G - 1), p.D, p.r);
  float w[2][2][8], dw[2][2][8];
  load_weight<E>(p, p.s[0], it, w[0]);
  load_weight<E>(p, p.s[1], it, w[1]);
#pragma unroll
  for (int i = 0; i < 32; ++i) dw[i / 16][i / 8 % 2][i % 8] = 0.0f;
  double f[8];
  my_freqs(p, lane & (G - 1), f);
  for (long long task = (long long)blockIdx.x * 4 + wave; task < p.tasks; task += gridDim.x * 4LL) {
    const long long t = task / p.parts;
    const int part = (int)(task - t * p.parts);
    float co[8], si[8];
    turn_of(position(p, t), f, co, si);
#pragma unroll
    for (int i = 0; i < 8; ++i) si[i] = -si[i];
    for (int b = part; b < nb; b += p.parts) {
      const bool isk = b >= p.s[0].batches;
      const Side& s = p.s[isk];
      const int h = (isk ? b - p.s[0].batches : b) * per + lane / G;
      const bool mine = it.on && h < s.heads;
      float x[2][8], u[2][8], ss = 0.0f;
      if (mine) {
        Raw8<E> rx[2], ry[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          rx[k] = fetch8((const E*)s.x + t * s.ldx + h * s.hsx + it.base[k], it.c[k], it.lim[k]);
          ry[k] = fetch8((const E*)s.dy + t * s.lddy + h * s.hsdy + it.base[k], it.c[k], it.lim[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          chunk8(rx[k], it.c[k], it.lim[k], x[k]);
          chunk8(ry[k], it.c[k], it.lim[k], u[k]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i / 8][i % 8] = u[i / 8][i % 8] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = __builtin_fmaf(x[i / 8][i % 8], x[i / 8][i % 8], ss);
      const float rs = 1.0f / sqrtf(head_sum(ss, G) / (float)p.D + p.eps);
      rotate<IL>(u, co, si, it.rot);
      float c = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[k][e] *= rs;
          if (isk) dw[1][k][e] = __builtin_fmaf(u[k][e], x[k][e], dw[1][k][e]);
          else dw[0][k][e] = __builtin_fmaf(u[k][e], x[k][e], dw[0][k][e]);
          u[k][e] *= isk ? w[1][k][e] : w[0][k][e];
          c = __builtin_fmaf(u[k][e], x[k][e], c);
        }
      c = head_sum(c, G) / (float)p.D;
      if (!mine || !s.y) continue;
      E* row = (E*)s.y + t * s.ldy + h * s.hsy;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[k][e] = rs * __builtin_fmaf(-x[k][e], c, u[k][e]);
        if (it.c[k] < it.lim[k]) store8(row + it.base[k], it.c[k], it.lim[k], u[k]);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float& v = dw[i / 16][i / 8 % 2][i % 8];
    for (int o = G; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  }
  const bool mine = it.on && lane < G;                 // one lane for each column
  if (mine && wave > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (it.c[i & 1] < it.lim[i & 1])
        store8(sh + ((wave - 1) * 2 + i / 2) * p.D + it.base[i & 1], it.c[i & 1], it.lim[i & 1],
               dw[i / 2][i & 1]);
  }
  __syncthreads();
  if (wave > 0 || !mine) return;
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      load8(sh + (o * 2 + i / 2) * p.D + it.base[i & 1], it.c[i & 1], it.lim[i & 1], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[i / 2][i & 1][e] += v[e];
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (it.c[i & 1] < it.lim[i & 1])
      store8(p.part + (blockIdx.x * 2LL + i / 2) * p.D + it.base[i & 1], it.c[i & 1], it.lim[i & 1],
             dw[i / 2][i & 1]);
}

// ------------------------------------------------------------------ the calls

constexpr int kMaxHeadDim = 1024, kMaxHeads = 1 << 16;
constexpr long long kMaxStride = 1LL << 38;

struct Split {
  int G, batches[2], parts;
  long long tasks;
};
// 16-column pieces of a head.
int pieces(int D, int r, bool il) {
  return (il ? (r + 15) / 16 : (r / 2 + 7) / 8) + (D - r + 15) / 16;
}
// A head takes the power of two of lanes that holds its columns, 16 a lane.
// About 4096 waves at least (4 a SIMD): a token's heads are shared out between
// waves where there are few tokens.
Split split_heads(long long T, int hq, int hk, int D, int r, bool il) {
  Split q;
  q.G = 1;
  while (q.G < pieces(D, r, il)) q.G *= 2;
  const int per = 64 / q.G;
  q.batches[0] = (hq + per - 1) / per;
  q.batches[1] = (hk + per - 1) / per;
  const int nb = q.batches[0] + q.batches[1];
  const long long want = T > 0 ? (4096 + T - 1) / T : 1;
  q.parts = (int)(want < nb ? want : nb);
  q.tasks = T * q.parts;
  return q;
}
int grad_units(const Split& q) {
  const long long need = (q.tasks + 3) / 4;
  return (int)(need < 1024 ? need : 1024);
}

dion3_status check_heads(const dion3_heads* q, const dion3_heads* k, const double* freqs,
                         const void* pos, int pos_bits, int64_t T, int D, int r, int interleaved,
                         float eps, int wtype, int dtype, bool grad) {
  if (!q || !type16(dtype) || (wtype != DION3_F32 && wtype != dtype)) return DION3_ERR_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps) || (pos_bits != 32 && pos_bits != 64)) return DION3_ERR_ARG;
  if (T < 0 || D < 1 || r < 0 || r > D || (r & 1)) return DION3_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return DION3_ERR_ARG;
  const dion3_heads* both[2] = {q, k};
  for (int i = 0; i < 2; ++i)
    if (both[i] && both[i]->heads < 1) return DION3_ERR_ARG;
  if (T > DION3_MAX_TOKENS || D > kMaxHeadDim || pieces(D, r, interleaved) > 64)
    return DION3_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i) {
    const dion3_heads* s = both[i];
    if (!s) continue;
    if (s->heads > kMaxHeads) return DION3_ERR_UNSUPPORTED;
    if (!s->w || !elem_aligned(s->w, wtype == DION3_F32 ? 4 : 2)) return DION3_ERR_ARG;
    if (T == 0) continue;
    const struct { const void* p; int64_t ld, hs; bool need; } t[3] = {
        {s->X, s->ldx, s->hsx, true}, {s->dY, s->lddy, s->hsdy, grad}, {s->Y, s->ldy, s->hsy, !grad}};
    for (int j = 0; j < 3; ++j) {
      if (j == 1 && !grad) continue;
      if (!t[j].p) {
        if (t[j].need) return DION3_ERR_ARG;
        continue;
      }
      if (!elem_aligned(t[j].p, 2)) return DION3_ERR_ARG;
      if ((T > 1 && t[j].ld < D) || (s->heads > 1 && t[j].hs < D)) return DION3_ERR_ARG;
      if (t[j].ld > kMaxStride || t[j].hs > kMaxStride) return DION3_ERR_UNSUPPORTED;
    }
  }
  if (T > 0 && (!pos || !elem_aligned(pos, pos_bits / 8))) return DION3_ERR_ARG;
  if (r > 0 && (!freqs || !elem_aligned(freqs, 8))) return DION3_ERR_ARG;
  return DION3_OK;
}

HeadsP describe(const dion3_heads* q, const dion3_heads* k, const Split& sp, const double* freqs,
                const void* pos, int pos_bits, int64_t T, int D, int r, float eps, int wtype) {
  HeadsP p = {};
  const dion3_heads* both[2] = {q, k};
  for (int i = 0; i < 2; ++i)
    if (both[i]) {
      const dion3_heads& s = *both[i];
      p.s[i] = {s.X, s.w, s.dY, s.Y, s.ldx, s.hsx, s.lddy, s.hsdy, s.ldy, s.hsy, s.heads,
                sp.batches[i]};
    }
  p.freqs = freqs; p.pos = pos; p.T = T; p.tasks = sp.tasks;
  p.D = D; p.r = r; p.G = sp.G; p.parts = sp.parts;
  p.pos64 = pos_bits == 64; p.wtype = wtype; p.eps = eps;
  return p;
}

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

size_t dion3_heads_size(void) { return sizeof(dion3_heads); }

dion3_status dion3_qk_norm_rope(const dion3_heads* q, const dion3_heads* k, const double* freqs,
                                const void* pos, int32_t pos_bits, int64_t T, int32_t D, int32_t r,
                                int32_t interleaved, float eps, int32_t wtype, int32_t dtype,
                                void* stream) {
  TRY(check_heads(q, k, freqs, pos, pos_bits, T, D, r, interleaved, eps, wtype, dtype, false));
  if (T == 0) return DION3_OK;
  hipStream_t s = (hipStream_t)stream;
  const Split sp = split_heads(T, q->heads, k ? k->heads : 0, D, r, interleaved);
  const HeadsP p = describe(q, k, sp, freqs, pos, pos_bits, T, D, r, eps, wtype);
  TraceScope ts("qk_norm_rope", 0.0, 4.0 * T * D * (q->heads + (k ? k->heads : 0)), s);
  const dim3 grid((unsigned)((sp.tasks + 3) / 4)), block(256);
  if (dtype == DION3_BF16) {
    if (interleaved) hipLaunchKernelGGL((k_heads<bf16, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((k_heads<bf16, false>), grid, block, 0, s, p);
  } else {
    if (interleaved) hipLaunchKernelGGL((k_heads<f16, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((k_heads<f16, false>), grid, block, 0, s, p);
  }
  HIP_TRY(hipGetLastError());
  return DION3_OK;
}

dion3_status dion3_qk_norm_rope_grad_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t D,
                                                    int32_t r, int32_t interleaved, size_t* bytes) {
  if (!bytes || T < 0 || hq < 1 || hk < 0 || D < 1 || r < 0 || r > D || (r & 1)) return DION3_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return DION3_ERR_ARG;
  if (T > DION3_MAX_TOKENS || D > kMaxHeadDim || hq > kMaxHeads || hk > kMaxHeads ||
      pieces(D, r, interleaved) > 64)
    return DION3_ERR_UNSUPPORTED;
  *bytes = (size_t)grad_units(split_heads(T, hq, hk, D, r, interleaved)) * 2 * D * 4;
  return DION3_OK;
}

dion3_status dion3_qk_norm_rope_grad(const dion3_heads* q, const dion3_heads* k,
                                     const double* freqs, const void* pos, int32_t pos_bits,
                                     float* dw, int64_t T, int32_t D, int32_t r,
                                     int32_t interleaved, float eps, int32_t wtype, int32_t dtype,
                                     void* ws, size_t ws_bytes, void* stream) {
  TRY(check_heads(q, k, freqs, pos, pos_bits, T, D, r, interleaved, eps, wtype, dtype, true));
  if (!elem_aligned(dw, 4)) return DION3_ERR_ARG;
  if (T > 0 && !dw && !q->Y && !(k && k->Y)) return DION3_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  const Split sp = split_heads(T, q->heads, k ? k->heads : 0, D, r, interleaved);
  const int units = grad_units(sp);
  if (dw) TRY(check_scratch(ws, ws_bytes, (size_t)units * 2 * D * 4));
  if (T > 0) {
    HeadsP p = describe(q, k, sp, freqs, pos, pos_bits, T, D, r, eps, wtype);
    p.part = dw ? (float*)ws : nullptr;
    TraceScope ts("qk_norm_rope_grad", 0.0, 6.0 * T * D * (q->heads + (k ? k->heads : 0)), s);
    const dim3 grid(units), block(256);
    const size_t lds = dw ? (size_t)6 * D * 4 : 0;
    if (dtype == DION3_BF16) {
      if (interleaved) hipLaunchKernelGGL((k_heads_grad<bf16, true>), grid, block, lds, s, p);
      else hipLaunchKernelGGL((k_heads_grad<bf16, false>), grid, block, lds, s, p);
    } else {
      if (interleaved) hipLaunchKernelGGL((k_heads_grad<f16, true>), grid, block, lds, s, p);
      else hipLaunchKernelGGL((k_heads_grad<f16, false>), grid, block, lds, s, p);
    }
    HIP_TRY(hipGetLastError());
  }
  if (dw) HIP_TRY(launch_join_columns((const float*)ws, units, 2 * D, dw, s));
  return DION3_OK;
}

}  // extern "C"
