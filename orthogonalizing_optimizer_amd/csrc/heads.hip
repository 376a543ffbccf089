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
// (a batch) at a time.  Waves stay and take batch after batch, of queries or of
// keys (one weight and one sum of its gradient in registers), the next one's
// columns on their way.  A wave computes the angles of its batch's token together.
#include "checks.h"
#include "wave.h"

namespace dion3 {
namespace {

struct Side {
  const void* x; const void* w; const void* dy;
  void* y;
  long long ldx, hsx, lddy, hsdy, ldy, hsy;
  int heads, batches, units;       // batches of a token's heads; workgroups
  int tb, hb;                      // tokens and heads of a batch (powers of two, tb hb = 64 / G)
};
struct HeadsP {
  Side s[2];                      // queries, keys
  const double* freqs;
  const void* pos;
  float* part;                    // gradient: one row of D floats a workgroup, or null
  long long T;
  int D, r, G, pitch;             // pitch: angles of a token in LDS (r / 2 rounded up to 8)
  int angles;                     // of a wave
  int pos64, wtype;
  float eps;
};

// The 16 columns of a lane: two chunks of 8, each with the run of columns that
// it lies in (base, length) and its place there.  Runs: the two halves of the
// rotated columns, or all of them where pairs are neighbours; the columns past
// them.
//
// How chunks fit their runs.  WHOLE: no chunk ends early (the checks take 30
// registers).  LAPPED: every run has at least 8 columns, and a chunk that would
// end behind its run lies over the one before instead; what lies over is
// computed and written twice, with the same bits, and left out of sums (8192
// tokens of 16 + 16 heads of 96, 24 turned: 25 us, 34 with ragged chunks;
// backwards 52 and 76).  RAGGED: chunks are cut off at the end of the run.
enum Fit { RAGGED, LAPPED, WHOLE };
struct Item {
  int base[2], c[2], lim[2];
  int dup[2];                      // LAPPED: columns at its start that are not the chunk's own
  bool on, rot;
};
template <bool IL, int FIT>
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
    if (!it.on) it.base[0] = it.base[1] = it.c[0] = it.c[1] = 0;      // (a place inside the head)
  }
  if (FIT == LAPPED && it.on) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = min(it.c[k], it.lim[k] - 8);
      it.dup[k] = min(it.c[k] - c, 8);
      it.c[k] = c;
    }
  } else {
    it.dup[0] = it.dup[1] = 0;
  }
  return it;
}

__device__ __forceinline__ double position(const HeadsP& p, long long t) {
  return p.pos64 ? (double)((const long long*)p.pos)[t] : (double)((const int*)p.pos)[t];
}

// A wave's angles: each lane turns one position and frequency (in turns,
// reduced in 64 bits: a position of 2^20 times a frequency of 1 leaves no bits
// of a fraction in 32) into a cosine and a sine, and takes the 8 of its
// columns from LDS.  Nobody else touches the wave's part of it.
struct Angles {
  float2* at;
  double first;                   // the frequency in turns of the lane's first pair
  __device__ Angles(const HeadsP& p, float2* lds, int wave) {
    at = lds + wave * p.angles;
    first = frequency(p, (int)(threadIdx.x & 63) % p.pitch);
  }
  __device__ static double frequency(const HeadsP& p, int i) {
    return i < p.r / 2 ? p.freqs[i] * 0.15915494309189533577 : 0.0;
  }
  // tb tokens (MULTI; one otherwise), whose positions lanes 0 .. tb - 1 hold; the
  // lane's is dt.
  // pair: of the lane's first four pairs, and of the others.
  template <bool MULTI, int FIT>
  __device__ void set(const HeadsP& p, double pos, int tb, int dt, int pair, int pair4, float sign,
                      float (&co)[8], float (&si)[8]) {
    __builtin_amdgcn_wave_barrier();
    const int n = (MULTI ? tb : 1) * p.pitch, lane = threadIdx.x & 63;
    for (int i0 = 0; i0 < n; i0 += 64) {
      const int i = i0 + lane;
      int k = i;
      double ps = pos;
      if (MULTI) {
        const int tok = min(i / p.pitch, tb - 1);
        k = i - tok * p.pitch;
        ps = __shfl(pos, tok, 64);
      }
      if (i < n) {
        const double t = ps * (i0 == 0 ? first : frequency(p, k));
        float2 v;
        sincospif(2.0f * (float)(t - rint(t)), &v.y, &v.x);
        at[i] = v;
      }
    }
    __builtin_amdgcn_wave_barrier();
    const float2* mine = at + (MULTI ? dt * p.pitch : 0);
    if (FIT == LAPPED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = mine[i < 4 ? pair + i : pair4 + i - 4];
        co[i] = v.x; si[i] = sign * v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 v = *(const float4*)(mine + pair + i);
        co[i] = v.x; si[i] = sign * v.y;
        co[i + 1] = v.z; si[i + 1] = sign * v.w;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
};

// The batches of heads that a wave takes: every W-th of its side's, W its
// waves, so that all waves read and write beside each other.  32 + 8 heads of
// 128 backwards: 56 us at 8192 tokens and 104 at 16384, with a stretch of
// neighbouring batches for each wave, which needs a token's angles less often,
// 61 and 123, with runs of two 58 and 115; forwards at 16384 64, 74 and 72.
// (Smaller heads backwards lose by it: 25 + 25 of 100 at 8192 86 us, 77 and 82.)
struct Walk {
  long long left, t, dt;           // batches left; token, tokens of a step
  int b, db;
  __device__ Walk(const HeadsP& p, const Side& s, long long wave) {
    const long long all = (p.T + s.tb - 1) / s.tb * s.batches;
    const int W = 4 * s.units, q = W / s.batches;
    left = (all - wave + W - 1) / W;
    t = wave / s.batches;
    b = (int)(wave - t * s.batches);
    t *= s.tb;
    db = W - q * s.batches;
    dt = (long long)q * s.tb;
  }
  __device__ bool more() const { return left > 0; }
  __device__ void next(const Side& s) {
    --left;
    t += dt;
    b += db;
    if (b < s.batches) return;
    b -= s.batches;
    t += s.tb;
  }
};

// The lane's token and head within a batch, and whether there are such.  MULTI:
// batches may be of several tokens (a variant of its own, because it costs the
// others 2 to 8 %).
template <bool MULTI>
struct Slot {
  int dt, h;
  __device__ Slot(const Side& s, int slot)
      : dt(MULTI ? slot / s.hb : 0), h(MULTI ? slot % s.hb : slot) {}
  __device__ int head(const Side& s, const Walk& at) const { return at.b * s.hb + h; }
  __device__ bool in(const HeadsP& p, const Side& s, const Walk& at) const {
    return head(s, at) < s.heads && (!MULTI || at.t + dt < p.T);
  }
};
template <bool MULTI>
__device__ __forceinline__ double positions_of(const HeadsP& p, const Side& s, long long t) {
  if (!MULTI) return position(p, t);
  const long long u = t + ((int)(threadIdx.x & 63) & (s.tb - 1));
  return position(p, u < p.T ? u : p.T - 1);
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
    if (!it.on) continue;
    if (p.wtype == DION3_F32) load8((const float*)s.w + it.base[k], it.c[k], it.lim[k], w[k]);
    else load8((const E*)s.w + it.base[k], it.c[k], it.lim[k], w[k]);
  }
}

__device__ __forceinline__ float head_sum(float v, int G) {
  return group_reduce(v, G, [](float a, float b) { return a + b; });
}

// The lane's 16 columns of head h of token t, asked for and as floats (zeros
// where the lane has none).
// ONCE: past the cache (chosen at compile time: of a branch between two loads
// that differ in this alone the compiler makes one load).
template <int FIT, bool ONCE, class E>
__device__ __forceinline__ void ask(const void* x, long long ld, long long hs, long long t, int dt,
                                    int h, const Item& it, bool mine, Raw8<E> (&raw)[2]) {
  if (FIT != RAGGED) {   // no branches between the loads: lanes without a head read the first one's
    const E* row = (const E*)x + t * ld + (mine ? dt * ld + h * hs : 0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const E* at = row + it.base[k] + it.c[k];
      if (ONCE) raw[k].v = load_once<typename Raw8<E>::type>(at);
      else raw[k].v = ((const typename Raw8<E>::Any*)at)->v;
    }
    return;
  }
  if (!mine) return;
  const E* row = (const E*)x + t * ld + (dt * ld + h * hs);
#pragma unroll
  for (int k = 0; k < 2; ++k) raw[k] = fetch8(row + it.base[k], it.c[k], it.lim[k]);
}
template <int FIT, class E>
__device__ __forceinline__ void take(const Raw8<E> (&raw)[2], const Item& it, bool mine,
                                     float (&v)[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (FIT != RAGGED) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = mine ? to_f32((E)raw[k].v[e]) : 0.0f;
    } else if (mine) {
      chunk8(raw[k], it.c[k], it.lim[k], v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
    }
  }
}
template <int FIT, class E>
__device__ __forceinline__ void put(void* y, long long ld, long long hs, long long t, int dt,
                                    int h, const Item& it, const float (&v)[2][8]) {
  E* row = (E*)y + t * ld + (dt * ld + h * hs);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (FIT != RAGGED) {
      Raw8<E> r;
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = (E)v[k][e];
      ((typename Raw8<E>::Any*)(row + it.base[k] + it.c[k]))->v = r.v;
    } else if (it.c[k] < it.lim[k]) {
      store8(row + it.base[k], it.c[k], it.lim[k], v[k]);
    }
}
// v as far as it is the lane's own column.
template <int FIT>
__device__ __forceinline__ float own_column(const Item& it, int k, int e, float v) {
  return FIT != LAPPED || e >= it.dup[k] ? v : 0.0f;
}
template <int FIT>
__device__ __forceinline__ float head_rstd(const Item& it, const float (&v)[2][8], int G, int D,
                                           float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = own_column<FIT>(it, i / 8, i % 8, v[i / 8][i % 8]);
    ss = __builtin_fmaf(x, x, ss);
  }
  return 1.0f / sqrtf(head_sum(ss, G) / (float)D + eps);
}

template <class E, bool IL, int FIT, bool ONCE, bool MULTI>
__global__ __launch_bounds__(256) void k_heads(HeadsP p) {
  extern __shared__ __attribute__((aligned(16))) float2 turns[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = p.G, j = lane & (G - 1);
  const bool isk = (int)blockIdx.x >= p.s[0].units;
  const Side& s = p.s[isk];
  const Slot<MULTI> slot(s, lane / G);
  Walk at(p, s, ((int)blockIdx.x - (isk ? p.s[0].units : 0)) * 4LL + wave);
  if (!at.more()) return;
  const Item it = my_item<IL, FIT>(j, p.D, p.r);
  const int pair = !it.rot ? 0 : FIT != LAPPED ? 8 * j : IL ? it.c[0] / 2 : it.c[0];
  const int pair4 = !it.rot ? 0 : IL ? it.c[1] / 2 : it.c[0] + 4;      // (LAPPED)
  Raw8<E> raw[2];
  bool mine = it.on && slot.in(p, s, at);
  ask<FIT, ONCE>(s.x, s.ldx, s.hsx, at.t, slot.dt, slot.head(s, at), it, mine, raw);
  double pos = positions_of<MULTI>(p, s, at.t);
  float w[2][8], co[8], si[8];
  load_weight<E>(p, s, it, w);
  Angles ang(p, turns, wave);
  for (bool fresh = true;;) {
    if (fresh) ang.template set<MULTI, FIT>(p, pos, s.tb, slot.dt, pair, pair4, 1.0f, co, si);
    float v[2][8];
    take<FIT>(raw, it, mine, v);
    // the next batch's columns, and the next token's position, on their way
    const Walk now = at;
    const bool own = mine;
    at.next(s);
    const bool go = at.more();
    if (go) {
      mine = it.on && slot.in(p, s, at);
      ask<FIT, ONCE>(s.x, s.ldx, s.hsx, at.t, slot.dt, slot.head(s, at), it, mine, raw);
      fresh = at.t != now.t;
      if (fresh) pos = positions_of<MULTI>(p, s, at.t);
    }
    const float rs = head_rstd<FIT>(it, v, G, p.D, p.eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i / 8][i % 8] *= rs * w[i / 8][i % 8];
    rotate<IL>(v, co, si, it.rot);
    if (own) put<FIT, E>(s.y, s.ldy, s.hsy, now.t, slot.dt, slot.head(s, now), it, v);
    if (!go) return;
  }
}

// The weights' gradients: a lane adds up its columns over its tokens and
// heads, the lanes of equal columns and the workgroup's waves are joined at
// the end, and the workgroups' rows by k_heads_join, each in a fixed order.
template <class E, bool IL, int FIT, bool ONCE, bool MULTI>
__global__ __launch_bounds__(256) void k_heads_grad(HeadsP p) {
  extern __shared__ __attribute__((aligned(16))) float2 turns[];
  float* sh = (float*)turns + 8 * p.angles;             // 3 waves x D
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = p.G, j = lane & (G - 1);
  const bool isk = (int)blockIdx.x >= p.s[0].units;
  const Side& s = p.s[isk];
  const Slot<MULTI> slot(s, lane / G);
  Walk at(p, s, ((int)blockIdx.x - (isk ? p.s[0].units : 0)) * 4LL + wave);
  const Item it = my_item<IL, FIT>(j, p.D, p.r);
  const int pair = !it.rot ? 0 : FIT != LAPPED ? 8 * j : IL ? it.c[0] / 2 : it.c[0];
  const int pair4 = !it.rot ? 0 : IL ? it.c[1] / 2 : it.c[0] + 4;      // (LAPPED)
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i / 8][i % 8] = 0.0f;
  if (at.more()) {
    Raw8<E> rx[2], ry[2];
    bool mine = it.on && slot.in(p, s, at);
    ask<FIT, ONCE>(s.x, s.ldx, s.hsx, at.t, slot.dt, slot.head(s, at), it, mine, rx);
    ask<FIT, ONCE>(s.dy, s.lddy, s.hsdy, at.t, slot.dt, slot.head(s, at), it, mine, ry);
    double pos = positions_of<MULTI>(p, s, at.t);
    float w[2][8], co[8], si[8];
    load_weight<E>(p, s, it, w);
    Angles ang(p, turns, wave);
    for (bool fresh = true;;) {
      if (fresh) ang.template set<MULTI, FIT>(p, pos, s.tb, slot.dt, pair, pair4, -1.0f, co, si);
      float x[2][8], u[2][8];
      take<FIT>(rx, it, mine, x);
      take<FIT>(ry, it, mine, u);
      const Walk now = at;
      const bool own = mine;
      at.next(s);
      const bool go = at.more();
      if (go) {
        mine = it.on && slot.in(p, s, at);
        ask<FIT, ONCE>(s.x, s.ldx, s.hsx, at.t, slot.dt, slot.head(s, at), it, mine, rx);
        ask<FIT, ONCE>(s.dy, s.lddy, s.hsdy, at.t, slot.dt, slot.head(s, at), it, mine, ry);
        fresh = at.t != now.t;
        if (fresh) pos = positions_of<MULTI>(p, s, at.t);
      }
      // (no head: nothing in the sums, also where eps is 0 and its statistic infinite)
      const float stat = head_rstd<FIT>(it, x, G, p.D, p.eps), rs = own ? stat : 0.0f;
      rotate<IL>(u, co, si, it.rot);
      float c = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[k][e] *= rs;
          dw[k][e] = __builtin_fmaf(u[k][e], x[k][e], dw[k][e]);
          u[k][e] *= w[k][e];
          c = __builtin_fmaf(u[k][e], own_column<FIT>(it, k, e, x[k][e]), c);
        }
      c = head_sum(c, G) / (float)p.D;
      if (own && s.y) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          u[i / 8][i % 8] = rs * __builtin_fmaf(-x[i / 8][i % 8], c, u[i / 8][i % 8]);
        put<FIT, E>(s.y, s.ldy, s.hsy, now.t, slot.dt, slot.head(s, now), it, u);
      }
      if (!go) break;
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    for (int o = G; o < 64; o <<= 1) dw[i / 8][i % 8] += __shfl_xor(dw[i / 8][i % 8], o, 64);
  const bool mine = it.on && lane < G;                 // one lane for each column
  auto put_sums = [&](float* row) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (FIT == LAPPED) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= it.dup[k]) row[it.base[k] + it.c[k] + e] = dw[k][e];
      } else if (it.c[k] < it.lim[k]) {
        store8(row + it.base[k], it.c[k], it.lim[k], dw[k]);
      }
  };
  if (mine && wave > 0) put_sums(sh + (wave - 1) * p.D);
  __syncthreads();
  if (wave > 0 || !mine) return;
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8];
      load8(sh + o * p.D + it.base[k], it.c[k], it.lim[k], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[k][e] += v[e];
    }
  put_sums(p.part + (long long)blockIdx.x * p.D);
}

// dw[side][c] = the sum over the side's workgroups: 16 columns a workgroup, 64
// slices of the rows.
__global__ __launch_bounds__(1024) void k_heads_join(const float* __restrict__ part, int qunits,
                                                     int kunits, int D, float* __restrict__ dw) {
  __shared__ float sh[64][17];
  const int col = threadIdx.x & 15, slice = threadIdx.x >> 4, c = blockIdx.x * 16 + col;
  const int units = blockIdx.y ? kunits : qunits, per = (units + 63) / 64;
  const float* rows = part + (blockIdx.y ? (long long)qunits * D : 0);
  const int u1 = min(units, (slice + 1) * per);
  float a = 0.0f;
  const int at = min(c, D - 1);                        // (no branch between the loads: 6.1 -> 4.6 us)
#pragma unroll 8
  for (int u = slice * per; u < u1; ++u) a += rows[(long long)u * D + at];
  sh[slice][col] = a;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, mine = blockIdx.x * 16 + wave;
  a = wave_add(sh[lane][wave]);                        // a wave a column
  if (lane == 0 && mine < D) dw[blockIdx.y * D + mine] = a;
}

// ------------------------------------------------------------------ the calls

constexpr int kMaxHeadDim = 1024, kMaxHeads = 1 << 16;
constexpr long long kMaxStride = 1LL << 38;

// 16-column pieces of a head.
int pieces(int D, int r, bool il) {
  return (il ? (r + 15) / 16 : (r / 2 + 7) / 8) + (D - r + 15) / 16;
}
Fit fit_of(int D, int r, bool il) {
  if (r % 16 == 0 && D % 16 == 0) return WHOLE;
  const int turned = il ? r : r / 2, rest = D - r;
  return (turned == 0 || turned >= 8) && (rest == 0 || rest >= 8) ? LAPPED : RAGGED;
}
// A head takes the power of two of lanes that holds its columns, 16 a lane.
// As many waves as stay resident (a few more would run after all others) are
// shared out between queries and keys by their batches: 8192 tokens of 32 + 8
// heads of 128 take 32 us (5.2 TB/s; 36 with 7 workgroups a CU instead of 5) and
// 56 backwards with the join (65 with 2 instead of 3, 72 with 4).  Not kept
// backwards: two batches on their way (3 to 13 % slower at most sizes, spills),
// 4 waves a SIMD that read their weight from LDS (3 % less at that size, when a
// wave's batches were neighbours).
//
// Where a token has at most half as many heads as a batch, a batch takes several
// tokens: 100000 tokens of 4 + 1 heads of 64 take 37 us and 66 backwards, 95 and
// 171 with a token a batch.
constexpr int kAngles = 512;        // a wave's in LDS, at most (one token's may be 512)
struct Split {
  int G, pitch, angles, batches[2], units[2], tb[2], hb[2];
};
Split split_heads(long long T, int hq, int hk, int D, int r, bool il, bool grad) {
  Split q = {};
  q.G = 1;
  while (q.G < pieces(D, r, il)) q.G *= 2;
  const int per = 64 / q.G, heads[2] = {hq, hk};
  const Fit fit = fit_of(D, r, il);
  q.pitch = r ? (r / 2 + 7) / 8 * 8 : 8;
  q.angles = q.pitch;
  long long all[2];
  for (int i = 0; i < 2; ++i) {
    q.tb[i] = 1;
    while (heads[i] * q.tb[i] * 2 <= per && heads[i] > 0 && q.pitch * q.tb[i] * 2 <= kAngles) q.tb[i] *= 2;
    q.hb[i] = per / q.tb[i];
    q.batches[i] = (heads[i] + q.hb[i] - 1) / q.hb[i];
    if (q.pitch * q.tb[i] > q.angles) q.angles = q.pitch * q.tb[i];
    all[i] = (T + q.tb[i] - 1) / q.tb[i] * q.batches[i];
  }
  const bool multi = q.tb[0] > 1 || q.tb[1] > 1;
  const int units = 256 * (grad ? 3 : fit == WHOLE || (fit == LAPPED && !multi) ? 5 : 4);
  for (int i = 0; i < 2; ++i) {
    if (all[i] == 0) continue;
    const long long share = (long long)((double)units * all[i] / (all[0] + all[1]));
    const long long waves = share < 1 ? 4 : share * 4;
    q.units[i] = (int)(((all[i] < waves ? all[i] : waves) + 3) / 4);
  }
  return q;
}
int units_of(const Split& q) { return q.units[0] + q.units[1]; }

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
                sp.batches[i], sp.units[i], sp.tb[i], sp.hb[i]};
    }
  p.freqs = freqs; p.pos = pos; p.T = T;
  p.D = D; p.r = r; p.G = sp.G; p.pitch = sp.pitch; p.angles = sp.angles;
  p.pos64 = pos_bits == 64; p.wtype = wtype; p.eps = eps;
  return p;
}

template <class E, bool GRAD, bool IL, int FIT, bool ONCE, bool MULTI>
void launch_heads_m(const HeadsP& p, int units, size_t lds, hipStream_t s) {
  if (GRAD)
    hipLaunchKernelGGL((k_heads_grad<E, IL, FIT, ONCE, MULTI>), dim3(units), dim3(256), lds, s, p);
  else
    hipLaunchKernelGGL((k_heads<E, IL, FIT, ONCE, MULTI>), dim3(units), dim3(256), lds, s, p);
}
template <class E, bool GRAD, bool IL, int FIT, bool ONCE>
void launch_heads_t(const HeadsP& p, int units, size_t lds, hipStream_t s) {
  if (p.s[0].tb > 1 || p.s[1].tb > 1)
    launch_heads_m<E, GRAD, IL, FIT, ONCE, true>(p, units, lds, s);
  else
    launch_heads_m<E, GRAD, IL, FIT, ONCE, false>(p, units, lds, s);
}
template <class E, bool GRAD, bool IL, int FIT>
void launch_heads_w(const HeadsP& p, int units, size_t lds, hipStream_t s) {
  // What is read, if it is much, passes the cache and leaves it to what is
  // written, which the attention reads next: 32 + 8 heads of 128 with a pass over
  // the outputs take 92 us at 16384 tokens (98 with plain loads, 101 with the
  // outputs past the cache), backwards 139 (150, 156); at 8192 80 backwards (84)
  // and 49 forwards either way; at 4096 (42 MB read) 32 instead of 29 forwards.
  const double read = (GRAD ? 4.0 : 2.0) * p.T * p.D * (p.s[0].heads + p.s[1].heads);
  if (read > 64e6) launch_heads_t<E, GRAD, IL, FIT, true>(p, units, lds, s);
  else launch_heads_t<E, GRAD, IL, FIT, false>(p, units, lds, s);
}
template <class E, bool GRAD, bool IL>
void launch_heads_f(const HeadsP& p, int units, size_t lds, hipStream_t s) {
  const Fit fit = fit_of(p.D, p.r, IL);
  if (fit == WHOLE) launch_heads_w<E, GRAD, IL, WHOLE>(p, units, lds, s);
  else if (fit == LAPPED) launch_heads_w<E, GRAD, IL, LAPPED>(p, units, lds, s);
  else launch_heads_t<E, GRAD, IL, RAGGED, false>(p, units, lds, s);
}
template <class E, bool GRAD>
void launch_heads(const HeadsP& p, int units, size_t lds, int interleaved, hipStream_t s) {
  if (interleaved) launch_heads_f<E, GRAD, true>(p, units, lds, s);
  else launch_heads_f<E, GRAD, false>(p, units, lds, s);
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
  const Split sp = split_heads(T, q->heads, k ? k->heads : 0, D, r, interleaved, false);
  const HeadsP p = describe(q, k, sp, freqs, pos, pos_bits, T, D, r, eps, wtype);
  TraceScope ts("qk_norm_rope", 0.0, 4.0 * T * D * (q->heads + (k ? k->heads : 0)), s);
  const size_t lds = (size_t)p.angles * 4 * 8;
  if (dtype == DION3_BF16) launch_heads<bf16, false>(p, units_of(sp), lds, interleaved, s);
  else launch_heads<f16, false>(p, units_of(sp), lds, interleaved, s);
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
  *bytes = (size_t)units_of(split_heads(T, hq, hk, D, r, interleaved, true)) * D * 4;
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
  const Split sp = split_heads(T, q->heads, k ? k->heads : 0, D, r, interleaved, true);
  if (dw) TRY(check_scratch(ws, ws_bytes, (size_t)units_of(sp) * D * 4));
  if (T > 0) {
    HeadsP p = describe(q, k, sp, freqs, pos, pos_bits, T, D, r, eps, wtype);
    p.part = dw ? (float*)ws : nullptr;
    TraceScope ts("qk_norm_rope_grad", 0.0, 6.0 * T * D * (q->heads + (k ? k->heads : 0)), s);
    const size_t lds = (size_t)p.angles * 4 * 8 + (dw ? (size_t)3 * D * 4 : 0);
    if (dtype == DION3_BF16) launch_heads<bf16, true>(p, units_of(sp), lds, interleaved, s);
    else launch_heads<f16, true>(p, units_of(sp), lds, interleaved, s);
    HIP_TRY(hipGetLastError());
  }
  if (dw) {
    hipLaunchKernelGGL(k_heads_join, dim3((D + 15) / 16, 2), dim3(1024), 0, s, (const float*)ws,
                       sp.units[0], sp.units[1], D, dw);
    HIP_TRY(hipGetLastError());
  }
  return DION3_OK;
}

}  // extern "C"
