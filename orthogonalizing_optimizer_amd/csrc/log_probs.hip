// Log probabilities of given tokens from rows of logits, with the entropy and
// the best alternatives, and the gradient.
//
//   z = scale x,  m = max_j z_j (rounded),  l = ln sum_j exp(z_j - m)   per row of n,
//   logp = (z_target - m) - l,  H = l - sum_j exp(z_j - m) (z_j - m) / exp(l),
//   dx_j = scale (g (1[j = target] - p_j) - gH p_j (ln p_j + H)),
//   p_j = exp((z_j - m) - l).
//
// Bound by HBM, not far from the vector units (an exponential a logit, 4
// issue slots of the about 10 a logit takes; 2 bytes of HBM time are 13).
//
// A workgroup takes one piece of one row, 32 logits a thread, and holds it in
// registers: the maximum first, then the sums, then the best of the piece, all
// from one read.  What the pieces of a row leave (maximum, sums, candidates)
// is joined by a second launch, so that few long rows fill the chip as many
// rows do.  The pair (m, l) is kept apart up to the gradient: where logits are
// large, down to the type's lowest value, m + l would have no bits left for l.
//
// 8192 x 32000 bf16 take 88 us and 5 for the join (5.9 TB/s), the gradient 175
// (6.0 TB/s); 1000 x 50257 fp32 with the entropy and 5 alternatives 42 and 5.
#include <type_traits>

#include "checks.h"
#include "wave.h"

namespace dion3 {
namespace {

constexpr int kChunks = 4;                       // chunks of 8 logits a thread
constexpr int kMaxTop = DION3_MAX_TOP;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLn2 = 0.6931471805599453f;

// Distances count as no farther where they are multiplied: exp is 0 from -104 on,
// and 0 times what a sum or a gradient makes of an infinite or a huge distance
// would be NaN.
constexpr float kFar = -200.0f;
// (d log2 e is rounded and the exponential the hardware's: a term is off by up to
// 3 |d| + 2 units of 2^-24 of itself, for fp32 logits too; below 2^-126 it is 0)
__device__ __forceinline__ float exp_(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// A distance z - m, m the rounded maximum, takes its product with the scale
// unrounded.  At the maximum it is then the product's rounding, at most 32 below
// 2^30, which all distances of the row share and l takes back; m + l and p lose
// nothing by it.  Where m is larger, that would leave exp's range (rows that a
// mask has filled with the type's lowest value, at a temperature): there the
// product is rounded first, the distance is 0 at the maximum, and exp of any
// other one (128 at least) is 0.  A finite logit whose product passes the lowest
// number of fp32 is held there: only rows of -infinity have no probabilities.
constexpr float kLarge = 0x1p30f;
__device__ __forceinline__ bool large(float m) { return fabsf(m) >= kLarge; }
template <bool LARGE>
__device__ __forceinline__ float distance(float x, float scale, float m) {
#pragma clang fp contract(off)
  if (!LARGE) return __builtin_fmaf(x, scale, -m);
  float z = x * scale;
  z = z == -__builtin_inff() && x != z ? kLowest : z;
  return z - m;
}
// (an output's own: in sums and gradients exp of a held product is 0 all the same)
__device__ __forceinline__ float distance(float x, float scale, float m) {
  if (large(m)) return distance<true>(x, scale, m);
  const float d = distance<false>(x, scale, m);
  return d == -__builtin_inff() && x != d ? kLowest : d;
}

// The sums of a set of logits relative to m (kLowest for an empty set or one
// of -infinity): s = sum exp(z - m), e = sum exp(z - m) (z - m).
struct Part {
  float m, s, e, pad;
};
__device__ __forceinline__ Part merge(const Part& a, const Part& b) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, kFar), db = fmaxf(b.m - m, kFar);
  const float fa = exp_(a.m - m), fb = exp_(b.m - m);      // infinities less themselves: NaN
  return {m, __builtin_fmaf(a.s, fa, b.s * fb),
          __builtin_fmaf(__builtin_fmaf(a.s, da, a.e), fa, __builtin_fmaf(b.s, db, b.e) * fb), 0.0f};
}

// The merge of all lanes' parts, in every lane.
__device__ __forceinline__ Part wave_merge(Part a) {
  a = merge(a, {other<1>(a.m), other<1>(a.s), other<1>(a.e), 0.0f});
  a = merge(a, {other<2>(a.m), other<2>(a.s), other<2>(a.e), 0.0f});
  a = merge(a, {other<4>(a.m), other<4>(a.s), other<4>(a.e), 0.0f});
  a = merge(a, {other<8>(a.m), other<8>(a.s), other<8>(a.e), 0.0f});
  auto row = [&](int i) { return Part{lane_of(a.m, i), lane_of(a.s, i), lane_of(a.e, i), 0.0f}; };
  return merge(merge(row(0), row(16)), merge(row(32), row(48)));
}

// Whole numbers in the order of the logits; zeros of both signs alike, NaN
// above all, none is 0.  The lower kLow bits of a type's keys are those of
// their sign: all clear in the upper half of the order, all set in the lower.
template <class E>
constexpr int kLow = __is_same(E, bf16) ? 16 : __is_same(E, f16) ? 13 : 0;
template <class E>
__device__ __forceinline__ unsigned order_key(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x + 0.0f);
  return x != x ? 0xffffffffu << kLow<E> : u ^ (unsigned)((int)u >> 31 | (int)0x80000000);
}
__device__ __forceinline__ float order_value(unsigned k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A candidate as one number: the larger, the earlier (0: none).
typedef unsigned long long u64;
__device__ __forceinline__ u64 candidate(unsigned key, int at) {
  return (u64)key << 32 | (0xffffffffu - (unsigned)at);
}

// How many of c[from .. nc) (LDS, padded with zeros to a multiple of 4), taken 4
// at a time, `step` apart, come before `mine`.
__device__ __forceinline__ int count_before(const u64* c, int from, int nc, int step, u64 mine) {
  int n = 0;
#pragma unroll 4
  for (int j = from; j < nc; j += step) {
    const ulonglong2 a = *(const ulonglong2*)(c + j), b = *(const ulonglong2*)(c + j + 2);
    n += (a.x > mine) + (a.y > mine) + (b.x > mine) + (b.y > mine);
  }
  return n;
}

struct LogpP {
  const void* x; long long ldx;
  const void* target; int target64;
  float* logp; float* stats; float* entropy;
  float* top_logp; long long* top_index;
  Part* part; u64* best;                   // of piece (t, s): part[t S + s], best[(t S + s) top ..]
  long long T;
  int n, top, S, len;                      // pieces a row, logits a piece (a multiple of 8)
  float scale;
};

__device__ __forceinline__ long long flat_block() {
  return (long long)blockIdx.y * gridDim.x + blockIdx.x;
}
dim3 blocks_grid(long long blocks) {
  const long long row = 1LL << 21;
  return blocks <= row ? dim3((unsigned)blocks)
                       : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}

constexpr int kWaveBest = 128;     // candidates a wave leaves at most (at least kMaxTop)

// The wave's candidates for the `top` best of its logits: at least those (where
// it has as many), at most kWaveBest, padded with zeros to a multiple of 4.
// Logits at or above the top-th largest of the lanes' maxima are a superset,
// most often of few more than `top`: one comparison a logit.  Where they are
// too many, a threshold above that one is looked for by halves, until it
// leaves few enough.  Where none does (equal logits), or there are fewer than
// `top` above -infinity, the logits above the threshold and the first of those
// equal to it are taken; where there is NaN (`odd`), that threshold is found by
// the keys' bits.  mx: the wave's maximum.
template <class E>
__device__ __forceinline__ int wave_best(const float (&v)[kChunks][8], const float (&cm)[kChunks],
                                         const int (&col)[kChunks], int to, int top, float mx,
                                         bool odd, u64* out) {
  constexpr int SH = kLow<E>;
  constexpr unsigned kNone = 0x007fffffu;              // the key of -infinity (and of what is no column)
  const int lane = threadIdx.x & 63;
  const u64 below = (1ull << lane) - 1;
  int have = 0;
  unsigned t = 0;
  bool equal = odd;                                    // candidates equal to a threshold
  if (!odd) {
    float lm = cm[0];
#pragma unroll
    for (int i = 1; i < kChunks; ++i) lm = fmaxf(lm, cm[i]);
    const unsigned lk = order_key<E>(lm);
    for (int b = 31; b >= 16; --b) {               // (to within 2^-7: few more than needed)
      const unsigned c = t | 1u << b;
      if (__popcll(__ballot(lk >= c)) >= top) t = c;
    }
    t = max(t, kNone + 1);
    unsigned hi = (unsigned)__builtin_amdgcn_readfirstlane((int)order_key<E>(mx)) + 1;
    for (;;) {
      const float tau = order_value(t);
      have = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (!__ballot(cm[i] >= tau)) continue;
        int from = col[i];
        asm volatile("" : "+v"(from));   // (nothing computed ahead for a second time around)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x = v[i][e];
          const bool in = x >= tau;
          const u64 b = __ballot(in);
          if (!b) continue;
          asm volatile("" : "+v"(x));
          const int at = have + __popcll(b & below);
          if (in && at < kWaveBest) out[at] = candidate(order_key<E>(x), from + e);
          have += __popcll(b);
        }
      }
      if (have <= kWaveBest) break;
      bool found = false;
      while (hi - t > 1 && !found) {
        const unsigned c = t + (hi - t) / 2;
        const float x = order_value(c);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) n += __popcll(__ballot(v[i][e] >= x));
        if (n >= top) t = c;
        else hi = c;
        found = n >= top && n <= kWaveBest;
      }
      if (!found) {
        equal = true;
        break;
      }
    }
    if (have < top) {
      equal = true;
      t = kNone;
    }
  }
  if (equal) {
    auto key = [&](int i, int e) {
      float x = v[i][e];
      asm volatile("" : "+v"(x));      // (computed where it is used: 32 registers fewer)
      return col[i] + e < to ? order_key<E>(x) : 0u;
    };
    if (odd) {
      for (int b = 31; b >= SH; --b) {
        const unsigned c = t | 1u << b;
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) cnt += __popcll(__ballot(key(i, e) >= c));
        if (cnt >= top) t = c;
      }
      if (SH > 0 && t && !(t & 0x80000000u)) t |= (1u << SH) - 1;
    }
    have = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = key(i, e) > t;
        const u64 b = __ballot(in);
        const int at = have + __popcll(b & below);
        if (in && at < kWaveBest) out[at] = candidate(key(i, e), col[i] + e);
        have += __popcll(b);
      }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {        // the columns' order: chunks, lanes, then e
      int mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine += t && key(i, e) == t ? 1 : 0;
      int at = have;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const u64 w = __ballot(mine >> b & 1);
        at += __popcll(w & below) << b;
        have += __popcll(w) << b;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t && key(i, e) == t) {
          if (at < top) out[at] = candidate(t, col[i] + e);
          ++at;
        }
    }
    have = min(have, top);
  }
  if (lane < 4 && have + lane < kWaveBest) out[have + lane] = 0;
  return have;
}

// Up to this many candidates of a workgroup are ranked by comparing all with
// all; of more, one wave takes the `top` largest, in no order (the join ranks
// them): 1000 x 32000 with 64 best takes 67 us, 100 ranked; 424 x 53616 with 20,
// where there are fewer, 35 ranked and 39 not.
constexpr int kRanked = 128;
template <class E>
__device__ __forceinline__ void best_of(const u64* cand, const int* count, int nw, int from,
                                        int top, u64* best) {
  constexpr int SH = kLow<E>, PL = 15;                 // (a piece's columns: 15 bits)
  const int lane = threadIdx.x & 63;
  auto each = [&](auto f) {
#pragma unroll 2
    for (int u = 0; u < nw; ++u) {
      const int n = count[u];
      const u64 a = lane < n ? cand[u * kWaveBest + lane] : 0;
      const u64 b = lane + 64 < n ? cand[u * kWaveBest + 64 + lane] : 0;
      f(a);
      f(b);
    }
  };
  // Thresholds by halves of (key without its constant bits, column from the
  // end): the largest that `top` candidates reach.
  auto at = [&](u64 c) {
    const unsigned k = (unsigned)(c >> PL) << SH;
    return candidate(k & 0x80000000u ? k : k | ((1u << SH) - 1),
                     from + (1 << PL) - 1 - (int)(c & ((1u << PL) - 1)));
  };
  unsigned k0 = ~0u, k1 = 0;
  each([&](u64 c) {
    const unsigned k = (unsigned)(c >> 32);
    k0 = c ? min(k0, k) : k0;
    k1 = max(k1, k);
  });
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    k0 = min(k0, (unsigned)__shfl_xor((int)k0, o, 64));
    k1 = max(k1, (unsigned)__shfl_xor((int)k1, o, 64));
  }
  k0 = (unsigned)__builtin_amdgcn_readfirstlane((int)k0);
  k1 = (unsigned)__builtin_amdgcn_readfirstlane((int)k1);
  u64 lo = (u64)(k0 >> SH) << PL, hi = ((u64)(k1 >> SH) + 1 << PL) - 1;
  for (int n = 0; lo < hi && n != top;) {
    const u64 mid = lo + (hi - lo + 1) / 2, c = at(mid);
    n = 0;
    each([&](u64 a) { n += __popcll(__ballot(a >= c)); });
    if (n >= top) lo = mid;
    else hi = mid - 1;
  }
  const u64 least = at(lo), below = (1ull << lane) - 1;
  int have = 0;
  each([&](u64 c) {
    const bool in = c >= least;
    const u64 b = __ballot(in);
    const int i = have + __popcll(b & below);
    if (in && i < top) best[i] = c;
    have += __popcll(b);
  });
}

// The 8 logits from column c on of a row that ends at `to`: -infinity behind it.
template <class E>
__device__ __forceinline__ void logits8(const Raw8<E>& raw, int c, int to, int n, float (&v)[8]) {
  if (c < to) {
    chunk8(raw, c, n, v);
    if (c + 8 <= to) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= to) v[e] = -__builtin_inff();
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = -__builtin_inff();
  }
}
__device__ __forceinline__ float max8(const float (&v)[8]) {
  return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
}
// The sums of 32 logits relative to w.m; e with ENT only.
template <bool ENT, bool LARGE>
__device__ __forceinline__ void add_logits(const float (&v)[kChunks][8], float scale, Part& w) {
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = distance<LARGE>(v[i][e], scale, w.m);
      const float q = exp_(d);
      w.s += q;
      if (ENT) w.e = __builtin_fmaf(q, fmaxf(d, kFar), w.e);
    }
}

// (TOP at 8 waves a SIMD, which it would miss by a few registers: 1000 x 50257
// fp32 with 5 alternatives 41.5 us, 44 at 6)
template <class E, bool TOP, bool ENT>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(TOP ? 8 : 1)))
void k_logp_piece(LogpP p) {
  extern __shared__ __attribute__((aligned(16))) u64 cand[];     // TOP: kWaveBest a wave
  __shared__ Part sh[16];
  __shared__ int count[16];
  const long long block = flat_block();
  if (block >= p.T * p.S) return;
  const int nt = blockDim.x, wave = threadIdx.x >> 6, nw = nt >> 6;
  const long long t = block / p.S;
  const int from = (int)(block - t * p.S) * p.len, to = min(from + p.len, p.n);
  const E* row = (const E*)p.x + t * p.ldx;
  float v[kChunks][8], cm[kChunks];
  int col[kChunks];
  {
    Raw8<E> raw[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      col[i] = from + (i * nt + (int)threadIdx.x) * 8;
      if (col[i] < to) raw[i] = fetch8(row, col[i], p.n);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) logits8(raw[i], col[i], to, p.n, v[i]);
  }
  float mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    cm[i] = max8(v[i]);
    mx = fmaxf(mx, cm[i]);
  }
  mx = wave_max(mx);
  Part w = {fmaxf(mx * p.scale, kLowest), 0.0f, 0.0f, 0.0f};
  if (__builtin_amdgcn_readfirstlane(large(w.m))) add_logits<ENT, true>(v, p.scale, w);
  else add_logits<ENT, false>(v, p.scale, w);
  w.s = wave_add(w.s);
  if (ENT) w.e = wave_add(w.e);
  if ((threadIdx.x & 63) == 0) sh[wave] = w;
  if constexpr (TOP) {
    const bool odd = __builtin_amdgcn_readfirstlane(w.s != w.s ? 1 : 0);    // the wave's sum is NaN
    const int c = wave_best<E>(v, cm, col, to, p.top, mx, odd, cand + wave * kWaveBest);
    if ((threadIdx.x & 63) == 0) count[wave] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Part a = sh[0];
    for (int i = 1; i < nw; ++i) a = merge(a, sh[i]);
    p.part[block] = a;
  }
  if constexpr (TOP) {
    int all = 0;
    for (int u = 0; u < nw; ++u) all += count[u];
    if (all > kRanked) {
      if (wave == 0) best_of<E>(cand, count, nw, from, p.top, p.best + block * p.top);
      return;
    }
    // every candidate of the wave against all waves' candidates
    for (int i = threadIdx.x & 63; i < count[wave]; i += 64) {
      const u64 mine = cand[wave * kWaveBest + i];
      int rank = 0;
      for (int u = 0; u < nw; ++u) rank += count_before(cand + u * kWaveBest, 0, count[u], 4, mine);
      if (rank < p.top) p.best[block * p.top + rank] = mine;
    }
    for (int i = all + threadIdx.x; i < p.top; i += nt) p.best[block * p.top + i] = 0;
  }
}

__device__ __forceinline__ long long target_of(const void* target, int is64, long long t) {
  return is64 ? ((const long long*)target)[t] : (long long)((const int*)target)[t];
}

// What a row's log probabilities, x scale - m - l, take.
struct RowSums {
  float m, l;
  bool none;                                           // every logit is -infinity
};
// The target's logit, asked for before the pieces are joined.
template <class E>
__device__ __forceinline__ float target_logit(const LogpP& p, long long t, bool& token) {
  token = false;
  if (!p.target) return 0.0f;
  const long long j = target_of(p.target, p.target64, t);
  token = j >= 0 && j < p.n;
  return token ? to_f32(((const E*)p.x)[t * p.ldx + j]) : 0.0f;
}
// A row from its joined pieces, its outputs written by one thread.
__device__ __forceinline__ RowSums row_sums(const LogpP& p, long long t, const Part& a, bool write,
                                            float x, bool token) {
  RowSums r;
  r.none = a.s == 0.0f && a.m < 0.0f;      // (the largest logit's exp is at least exp(-32))
  // (an infinite maximum, of a logit or of its product with scale, has no log)
  r.l = r.none ? 0.0f : a.m > -kLowest ? __builtin_nanf("") : logf(a.s);
  r.m = r.none ? -__builtin_inff() : a.m;
  if (!write) return r;
  p.stats[2 * t] = r.m;
  p.stats[2 * t + 1] = r.l;
  if (p.entropy) p.entropy[t] = r.none ? 0.0f : r.l - a.e / a.s;
  if (p.target)
    p.logp[t] = !token ? 0.0f : r.none ? -__builtin_inff() : distance(x, p.scale, r.m) - r.l;
  return r;
}

// Rows from their pieces: a thread a row, or with TOP a workgroup a row, whose
// threads rank the pieces' candidates, several threads a candidate where there
// are fewer of them (taking the best first, as best_of does, is slower for few
// rows: 12 us instead of 7 for 4 of 16 x 20 candidates).
constexpr int kJoinTop = 512;
template <class E, bool TOP>
__global__ __launch_bounds__(TOP ? kJoinTop : 64) void k_logp_join(LogpP p) {
  extern __shared__ __attribute__((aligned(16))) u64 cand[];
  const long long t = TOP ? flat_block() : flat_block() * 64 + threadIdx.x;
  if (t >= p.T) return;
  const int nc = TOP ? p.S * p.top : 0, nt = blockDim.x;
  Part a = {kLowest, 0.0f, 0.0f, 0.0f};
  const bool write = !TOP || threadIdx.x == 0;
  bool token = false;
  const float x = write ? target_logit<E>(p, t, token) : 0.0f;
  if constexpr (TOP) {
    for (int i = threadIdx.x; i < (nc + 3) / 4 * 4; i += nt) cand[i] = i < nc ? p.best[t * nc + i] : 0;
    const int lane = threadIdx.x & 63;
    if (lane < p.S) a = p.part[t * p.S + lane];        // (S is at most 32)
    a = wave_merge(a);
  } else {
#pragma unroll 4
    for (int s = 0; s < p.S; ++s) a = merge(a, p.part[t * p.S + s]);
  }
  const RowSums r = row_sums(p, t, a, write, x, token);
  if constexpr (TOP) {
    __syncthreads();
    int q = 1;                                         // threads a candidate
    while (q < 16 && nc * q * 2 <= nt) q *= 2;
    const int sub = threadIdx.x & (q - 1);
    for (int i = threadIdx.x / q; i < (nc + 63) / 64 * 64; i += nt / q) {
      const u64 mine = i < nc ? cand[i] : 0;
      int rank = count_before(cand, sub * 4, nc, q * 4, mine);
      for (int o = 1; o < q; o <<= 1) rank += __shfl_xor(rank, o, 64);
      if (mine && sub == 0 && rank < p.top) {
        p.top_logp[t * p.top + rank] =
            r.none ? -__builtin_inff()
                   : distance(order_value((unsigned)(mine >> 32)), p.scale, r.m) - r.l;
        p.top_index[t * p.top + rank] = 0xffffffffu - (unsigned)mine;
      }
    }
  }
}

struct GradP {
  const float* g; const void* x; const void* target; const float* stats;
  const float* entropy; const float* gh;
  void* dx;
  long long ldx, lddx, T;
  int target64, n, S, len;
  float scale;
};

// One read and one write of a logit; in place where dX is X (a thread reads its
// logits before it writes them; at the end of a row it also reads up to 7 of
// its neighbour's, which it drops).  Both pass the cache:
// the logits, which the forward pass may have left there, are not needed again,
// and what they leave of it speeds up what follows at every size (8192 x 32000
// alone 199 -> 178 us; forward, gradient and a pass over it: 402 -> 350, and
// 56 -> 52 at 1000 x 32000; with the forward pass's loads past the cache too,
// 360 and 59).
template <class E, bool ENT>
__global__ __launch_bounds__(256) void k_logp_grad(GradP p) {
  const long long block = flat_block();
  if (block >= p.T * p.S) return;
  const long long t = block / p.S;
  const int from = (int)(block - t * p.S) * p.len, to = min(from + p.len, p.n);
  const E* row = (const E*)p.x + t * p.ldx;
  Raw8<E> raw[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = from + (i * 256 + (int)threadIdx.x) * 8;
    if (c < to) raw[i] = fetch8_once(row, c, p.n);
  }
  const float m = p.stats[2 * t], l = p.stats[2 * t + 1];
  long long j = p.target ? target_of(p.target, p.target64, t) : -1;
  if (j < 0 || j >= p.n) j = -1;
  const bool none = m == -__builtin_inff() || (!ENT && j < 0);    // no gradient
  const float g = j >= 0 ? p.scale * p.g[t] : 0.0f;
  // dx = p (a + b ln p) + g at the target; a statistic that is NaN reaches
  // every logit through a
  float a = -g + (l - l), b = 0.0f;
  if (ENT) {
    b = -p.scale * p.gh[t];
    a = __builtin_fmaf(b, p.entropy[t], a);
  }
  auto write = [&](auto is_large) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = from + (i * 256 + (int)threadIdx.x) * 8;
      if (c >= to) continue;
      float v[8];
      chunk8(raw[i], c, p.n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = distance<decltype(is_large)::value>(v[e], p.scale, m) - l;
        const float pr = exp_(q);
        v[e] = none ? 0.0f : pr * (ENT ? __builtin_fmaf(b, fmaxf(q, kFar), a) : a);
        if (c + e == j && !none) v[e] += g;
      }
      store8_once((E*)p.dx + t * p.lddx, c, min(to, p.n), v);
    }
  };
  if (__builtin_amdgcn_readfirstlane(large(m))) write(std::true_type());
  else write(std::false_type());
}

// --------------------------------------------------------------- the launches

// Pieces of at most 8192 logits (4 waves), of 32768 (16 waves) where a row
// would have more than 16, of equal length; one or two waves for rows that fill
// no more (20000 x 1500 without alternatives 22 us, 52 with four; 20000 x 4000
// 40 and 59).  16 waves keep the longest rows at 32 pieces (the join's wave
// holds 64), at a price, and from earlier on than that needs: with the entropy
// and 20 alternatives of bf16, 4 and 16 waves take 26 and 47 us at 100 x 131072,
// 224 and 283 at 2000 x 131072; past the border 26 and 50 at 100 x 131073, 243 and
// 341 at 2000 x 131073, 450 and 520 at 2000 x 256000 (188 and 202 without).
struct Pieces {
  int S, len, threads;
};
Pieces pieces_of(int n) {
  Pieces q;
  q.threads = n > 16 * 8192 ? 1024 : n > 4096 ? 256 : n > 2048 ? 128 : 64;
  const int most = q.threads * 8 * kChunks;
  q.S = (n + most - 1) / most;
  q.len = ((n + q.S - 1) / q.S + 7) / 8 * 8;
  return q;
}

size_t logp_scratch(long long T, int n, int top) {
  const Pieces q = pieces_of(n);
  return (size_t)T * q.S * (sizeof(Part) + (size_t)top * sizeof(u64));
}

template <class E, bool ENT>
hipError_t launch_logp_t(const LogpP& p, const Pieces& q, hipStream_t s) {
  const dim3 grid = blocks_grid(p.T * q.S), block(q.threads);
  const size_t lds = (size_t)(q.threads / 64) * kWaveBest * sizeof(u64);
  if (p.top) hipLaunchKernelGGL((k_logp_piece<E, true, ENT>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((k_logp_piece<E, false, ENT>), grid, block, 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.top) {
    // (few rows: as many threads as help one; many: one a candidate)
    const int nc = q.S * p.top;
    int nt = kJoinTop;
    while (p.T > 512 && nt > 64 && nt >= 2 * nc) nt /= 2;
    hipLaunchKernelGGL((k_logp_join<E, true>), blocks_grid(p.T), dim3(nt),
                       (size_t)pad_to(nc, 4) * sizeof(u64), s, p);
  } else {
    hipLaunchKernelGGL((k_logp_join<E, false>), blocks_grid((p.T + 63) / 64), dim3(64), 0, s, p);
  }
  return hipGetLastError();
}
template <class E>
hipError_t launch_logp(const LogpP& p, const Pieces& q, hipStream_t s) {
  return p.entropy ? launch_logp_t<E, true>(p, q, s) : launch_logp_t<E, false>(p, q, s);
}

template <class E>
hipError_t launch_logp_grad(const GradP& p, hipStream_t s) {
  const dim3 grid = blocks_grid(p.T * p.S);
  if (p.gh) hipLaunchKernelGGL((k_logp_grad<E, true>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((k_logp_grad<E, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

bool any_type(int t) { return type16(t) || t == DION3_F32; }
int size_of(int t) { return t == DION3_F32 ? 4 : 2; }

dion3_status check_targets(const void* target, int bits) {
  if (!target) return DION3_OK;
  if (bits != 32 && bits != 64) return DION3_ERR_ARG;
  return elem_aligned(target, bits / 8) ? DION3_OK : DION3_ERR_ARG;
}

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

dion3_status dion3_log_probs_workspace_size(int64_t T, int64_t n, int32_t top, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, 1));
  if (top < 0 || top > n) return DION3_ERR_ARG;
  if (top > kMaxTop) return DION3_ERR_UNSUPPORTED;
  *bytes = logp_scratch(T, (int)n, top);
  return DION3_OK;
}

dion3_status dion3_log_probs(const void* X, int64_t ldx, const void* target, int32_t target_bits,
                             float* logp, float* stats, float* entropy, float* top_logp,
                             int64_t* top_index, int64_t T, int64_t n, int32_t top, float scale,
                             int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  if (!any_type(dtype) || !(scale > 0.0f) || !isfinite(scale)) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, 1));
  if (top < 0 || top > n) return DION3_ERR_ARG;
  if (top > kMaxTop) return DION3_ERR_UNSUPPORTED;
  TRY(check_far_ld(ldx, n));
  TRY(check_targets(target, target_bits));
  if (T == 0) return DION3_OK;
  if (!X || !stats || (target != nullptr) != (logp != nullptr)) return DION3_ERR_ARG;
  if (top && (!top_logp || !top_index)) return DION3_ERR_ARG;
  if (!elem_aligned(X, size_of(dtype)) || !elem_aligned(logp, 4) || !elem_aligned(stats, 4) ||
      !elem_aligned(entropy, 4) || !elem_aligned(top_logp, 4) || !elem_aligned(top_index, 8))
    return DION3_ERR_ARG;
  TRY(check_scratch(ws, ws_bytes, logp_scratch(T, (int)n, top)));
  const Pieces q = pieces_of((int)n);
  LogpP p = {};
  p.x = X; p.ldx = ldx; p.target = target; p.target64 = target_bits == 64;
  p.logp = logp; p.stats = stats; p.entropy = entropy;
  p.top_logp = top_logp; p.top_index = (long long*)top_index;
  p.part = (Part*)ws; p.best = (u64*)(p.part + T * q.S);
  p.T = T; p.n = (int)n; p.top = top; p.S = q.S; p.len = q.len; p.scale = scale;
  hipStream_t s = (hipStream_t)stream;
  TraceScope ts("log_probs", 0.0, (double)T * n * size_of(dtype), s);
  if (dtype == DION3_BF16) HIP_TRY(launch_logp<bf16>(p, q, s));
  else if (dtype == DION3_F16) HIP_TRY(launch_logp<f16>(p, q, s));
  else HIP_TRY(launch_logp<float>(p, q, s));
  return DION3_OK;
}

dion3_status dion3_log_probs_grad(const float* dlogp, const void* X, int64_t ldx,
                                  const void* target, int32_t target_bits, const float* stats,
                                  const float* entropy, const float* dentropy, void* dX,
                                  int64_t lddx, int64_t T, int64_t n, float scale, int32_t dtype,
                                  void* stream) {
  if (!any_type(dtype) || !(scale > 0.0f) || !isfinite(scale)) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, 1));
  TRY(check_far_ld(ldx, n));
  TRY(check_far_ld(lddx, n));
  TRY(check_targets(target, target_bits));
  if ((target != nullptr) != (dlogp != nullptr) && T > 0) return DION3_ERR_ARG;
  if (T == 0) return DION3_OK;
  if (!X || !stats || !dX || (dentropy && !entropy) || (!dlogp && !dentropy)) return DION3_ERR_ARG;
  const int e = size_of(dtype);
  if (!elem_aligned(X, e) || !elem_aligned(dX, e) || !elem_aligned(dlogp, 4) ||
      !elem_aligned(stats, 4) || !elem_aligned(entropy, 4) || !elem_aligned(dentropy, 4))
    return DION3_ERR_ARG;
  GradP p = {dlogp, X, target, stats, entropy, dentropy, dX, ldx, lddx, T,
             target_bits == 64, (int)n, 0, 0, scale};
  const int most = 256 * 8 * kChunks;
  p.S = ((int)n + most - 1) / most;
  p.len = (((int)n + p.S - 1) / p.S + 7) / 8 * 8;
  hipStream_t s = (hipStream_t)stream;
  TraceScope ts("log_probs_grad", 0.0, 2.0 * T * n * e, s);
  if (dtype == DION3_BF16) HIP_TRY(launch_logp_grad<bf16>(p, s));
  else if (dtype == DION3_F16) HIP_TRY(launch_logp_grad<f16>(p, s));
  else HIP_TRY(launch_logp_grad<float>(p, s));
  return DION3_OK;
}

}  // extern "C"
