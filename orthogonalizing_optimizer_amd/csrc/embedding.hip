// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   y_t = E(scale W[token_t]),     dW[v] = scale sum over t with token_t = v of dy_t.
//
// The lookup is a copy of rows, bound by HBM.
//
// The gradient is summed without atomics, in an order fixed by the tokens:
// their places are sorted by token, places of one token in order.  The sorted
// list is cut into chunks of up to 32 places, a wave sums the rows of one chunk
// for 512 columns, and writes a token's sum at the end of its run.  A run
// longer than two chunks leaves one partial row a chunk, which a last launch
// adds up in order, and in 64 bits: a token that fills the batch has up to 2^19
// of them (equal rows added in fp32 are off by 6e-5 at 2^20 places, by 1e-3 at
// 2^24).  The rows of dW without one are cleared last, by the flags that the
// others' waves have set: cleared before, all of it, the rows with sums would be
// written twice, and beside the sums the two hold up each other.
//
// Bound by HBM: dW is written once (fp32, most of the bytes), dy read once.
// 8192 tokens of 32000 x 4096 (591 MB) take 100 us (5.9 TB/s): 9 for the places,
// 23 for the sums (rows of 8 KB at random), 67 for the other rows and the joins.
// More than kCountMax tokens take 15 to 20 us a digit.
#include "checks.h"

namespace dion3 {
namespace {

constexpr int kMaxChunk = 32;         // places of one wave at most
// Tokens up to which places are counted, not sorted by digits.  Counting grows
// with their square: 4100 tokens of 50257 x 768 take 37 us counted and 49
// sorted, 8192 41 and 51; 8193 would take 46 and take 51, 10240 50 and 52, 12288
// (48 KB of LDS) the same, added to a buffer 46 and 44.
constexpr int kCountMax = 8192;
constexpr int kTile = 1024;           // tokens of a workgroup of the sort by digits

__device__ __forceinline__ int token_key(const void* tokens, int is64, long long t, int n) {
  const long long v = is64 ? ((const long long*)tokens)[t] : (long long)((const int*)tokens)[t];
  return v >= 0 && v < n ? (int)v : n;             // no token: behind all rows
}

// ------------------------------------------------------------------ the lookup

template <class WT, class E>
__global__ __launch_bounds__(256) void k_embed(const void* __restrict__ tokens, int is64,
                                               const WT* __restrict__ w, long long ldw,
                                               E* __restrict__ y, long long ldy, long long chunks,
                                               int n, int m, unsigned nch, float scale, int once) {
  const long long base = flat_base();
  if (base + threadIdx.x >= chunks) return;
  const long long row0 = base / nch;
  const unsigned c0 = (unsigned)(base - row0 * nch) + threadIdx.x, dr = c0 / nch;
  const int c = (int)(c0 - dr * nch) * 8;
  const int key = token_key(tokens, is64, row0 + dr, n);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (key < n) {
    load8(w + key * ldw, c, m, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= scale;
  }
  if (once) store8_once(y + (row0 + dr) * ldy, c, m, v);
  else store8(y + (row0 + dr) * ldy, c, m, v);
}

// ------------------------------------------------------------ places by token

__device__ __forceinline__ long long grid_block() {
  return (long long)blockIdx.y * gridDim.x + blockIdx.x;
}

// Clears the rows of dW whose flag is not set (all of them without flags), 16
// bytes a thread and 4 KB a workgroup, the workgroups in the order of their
// addresses: 410 MB take 66 us (6.2 TB/s); with 16 stores a thread, whose writes
// lie further apart at any time, a fourth more.  They pass the cache, as the sums do
// (8192 tokens of 32000 x 4096 132 -> 100 us; with a pass over dW 246 -> 186 at
// 32000 rows, 71 either way at 8000, 29 at 1000).
struct Zero {
  float* dw;
  const unsigned char* set;
  long long ldw, blocks, items;         // items: 4 columns of a row
  unsigned nch;                         // items of a row
  int m;
};
template <int THREADS>
__device__ __forceinline__ void zero_block(const Zero& z, long long block) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  const long long base = block * THREADS;
  if (base + threadIdx.x >= z.items) return;
  const long long row0 = base / z.nch;
  const unsigned c0 = (unsigned)(base - row0 * z.nch) + threadIdx.x, dr = c0 / z.nch;
  const int c = (int)(c0 - dr * z.nch) * 4;
  if (z.set && z.set[row0 + dr]) return;
  float* d = z.dw + (row0 + dr) * z.ldw + c;
  if (c + 4 <= z.m) {
    store_once(d, f4{0, 0, 0, 0});
  } else {
    for (int e = 0; c + e < z.m; ++e) d[e] = 0.0f;
  }
}
__global__ __launch_bounds__(256) void k_embed_zero(Zero z) { zero_block<256>(z, grid_block()); }

// Up to kCountMax tokens: the place of t in the order is the number of tokens
// before it, counted by comparing all with all (two instructions a pair).  A
// workgroup places 32 tokens; its groups of 32 lanes share out the keys in
// blocks of 32: a block before the workgroup's own counts keys up to
// the token's, one behind it keys below, its own both by their places.
constexpr int kGroups = 32;           // groups of 32 lanes in a workgroup
__global__ __launch_bounds__(1024) void k_embed_count(const void* __restrict__ tokens, int is64,
                                                      int T, int n, int* __restrict__ skey,
                                                      int* __restrict__ spos,
                                                      uint4* __restrict__ set, int sets, Zero z) {
  extern __shared__ __attribute__((aligned(16))) int keys[];    // padded to whole blocks with n + 1
  __shared__ int part[kGroups][33];
  const int nb = (T + 31) / 32;
  if (grid_block() >= nb) {             // the other workgroups clear the rows' flags, or dW
    const long long rest = grid_block() - nb, i = rest * 1024 + threadIdx.x;
    if (!set) zero_block<1024>(z, rest);
    else if (i < sets) set[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int block = (int)grid_block();
  for (int i0 = 0; i0 < nb * 32; i0 += 1024 * 8) {        // 8 loads on their way at a time
    int k[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * 1024 + (int)threadIdx.x;
      k[u] = token_key(tokens, is64, i < T ? i : T - 1, n);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * 1024 + (int)threadIdx.x;
      if (i < nb * 32) keys[i] = i < T ? k[u] : n + 1;
    }
  }
  __syncthreads();
  const int mine = threadIdx.x & 31, group = threadIdx.x >> 5, own = block;
  const int key = keys[own * 32 + mine];
  int cnt = 0;
  for (int b = group; b < nb; b += kGroups) {
    const int lim = key + (b < own ? 1 : 0);
    const int4* k4 = (const int4*)(keys + b * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int4 k = k4[i];
      cnt += (k.x < lim) + (k.y < lim) + (k.z < lim) + (k.w < lim);
    }
  }
  if (group == (own & (kGroups - 1))) {
    for (int i = 0; i < mine; ++i) cnt += keys[own * 32 + i] == key;
  }
  part[group][mine] = cnt;
  __syncthreads();
  // (a group a token here: its lanes hold the groups' counts)
  cnt = part[mine][group];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) cnt += __shfl_xor(cnt, o, 64);
  const int t = own * 32 + group;
  if (mine == 0 && t < T) {
    skey[cnt] = keys[t];
    spos[cnt] = t;
  }
}

// More tokens: a stable sort by digits of 8 bits, the lowest first.  Per digit:
// a histogram of every tile, an exclusive scan over (digit, tile), and the
// tiles' tokens to their places.  The first digit reads the tokens themselves.
// Up to kOwnScan tiles every workgroup of the last adds the histograms up for
// itself, instead of a launch for the scan (8193 tokens of 50257 x 768 48 us
// instead of 52, 262144 of 50000 x 256 93 instead of 108).
constexpr int kOwnScan = 256;
struct DigitP {
  const void* tokens; int is64;       // first digit, else null
  const int* key; const int* pos;
  int* okey; int* opos;
  int* hist;                          // [256][tiles]
  long long T;
  int n, tiles, shift;
};
__device__ __forceinline__ int digit_key(const DigitP& p, long long i) {
  return p.tokens ? token_key(p.tokens, p.is64, i, p.n) : p.key[i];
}

__global__ __launch_bounds__(256) void k_embed_hist(DigitP p) {
  __shared__ int h[256];
  h[threadIdx.x] = 0;
  __syncthreads();
  const long long from = (long long)blockIdx.x * kTile;
  for (int i = threadIdx.x; i < kTile; i += 256)
    if (from + i < p.T) atomicAdd(&h[digit_key(p, from + i) >> p.shift & 255], 1);
  __syncthreads();
  p.hist[(long long)threadIdx.x * p.tiles + blockIdx.x] = h[threadIdx.x];
}

__global__ __launch_bounds__(1024) void k_embed_scan(int* __restrict__ hist, int count) {
  __shared__ int sums[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int from = 0; from < count; from += 16384) {         // 16 entries a thread
    int4 v[4];
    int s = 0;
    const int at = from + (int)threadIdx.x * 16;            // (count is a multiple of 256)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = at < count ? ((const int4*)(hist + at))[k] : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) s += v[k].x + v[k].y + v[k].z + v[k].w;
    int run = s;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(run, o, 64);
      if (lane >= o) run += u;
    }
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    int before = carry + run - s, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < wave) before += sums[i];
      all += sums[i];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int4 w = v[k];
      v[k].x = before;
      v[k].y = before + w.x;
      v[k].z = v[k].y + w.y;
      v[k].w = v[k].z + w.z;
      before = v[k].w + w.w;
      if (at < count) ((int4*)(hist + at))[k] = v[k];
    }
    carry += all;
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void k_embed_place(DigitP p) {
  __shared__ int count[4][256];
  __shared__ int sums[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 4; ++i) count[i][threadIdx.x] = 0;
  __syncthreads();
  // a wave takes a quarter of the tile in order, 64 tokens at a time
  constexpr int R = kTile / 256;
  const long long from = (long long)blockIdx.x * kTile + wave * (kTile / 4);
  const unsigned long long below = (1ull << lane) - 1;
  int key[R], pos[R], at[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long i = from + r * 64 + lane;
    key[r] = i < p.T ? digit_key(p, i) : 0;
    pos[r] = i < p.T ? (p.tokens ? (int)i : p.pos[i]) : 0;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = from + r * 64 + lane < p.T;
    const int dig = key[r] >> p.shift & 255;
    unsigned long long same = __ballot(in);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const unsigned long long w = __ballot(dig >> b & 1);
      same &= dig >> b & 1 ? w : ~w;
    }
    const int rank = __popcll(same & below);
    volatile int* c = &count[wave][dig];
    const int had = *c;
    __builtin_amdgcn_wave_barrier();
    if (in && rank == 0) *c = had + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    at[r] = had + rank;
  }
  __syncthreads();
  {                                   // the waves' counts to their first places
    const int* row = p.hist + (long long)threadIdx.x * p.tiles;
    int first;
    if (p.tiles > kOwnScan) {
      first = row[blockIdx.x];
    } else {                          // a digit a thread
      int before = 0, all = 0;
#pragma unroll 8
      for (int i = 0; i < p.tiles; ++i) {
        const int h = row[i];
        before += i < (int)blockIdx.x ? h : 0;
        all += h;
      }
      int run = all;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(run, o, 64);
        if (lane >= o) run += u;
      }
      if (lane == 63) sums[wave] = run;
      __syncthreads();
      first = before + run - all;
#pragma unroll
      for (int i = 0; i < 3; ++i) first += i < wave ? sums[i] : 0;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int c = count[w][threadIdx.x];
      count[w][threadIdx.x] = first;
      first += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (from + r * 64 + lane >= p.T) continue;
    const int to = count[wave][key[r] >> p.shift & 255] + at[r];
    p.okey[to] = key[r];
    p.opos[to] = pos[r];
  }
}

// --------------------------------------------------------------- the gradient

struct EmbedGradP {
  const void* dy; long long lddy;
  const int* key; const int* pos;     // sorted
  float* dw; long long ldw;
  unsigned char* set;                 // a flag for each row of dW that gets a sum, or null
  float* part;                        // [chunks][2][m]: a run from before, one that goes on
  long long T;
  int n, m, len;                      // places of a chunk
  int slices, width;                  // slices of the columns, of up to 512
  float scale;
  int accumulate;
};

// W columns of a row of m >= W from c on, or its last W where it ends before:
// neighbouring lanes of a wave then hold some columns both, and write the same
// to them (no slice begins less than W columns before the end, so that no two
// waves do, one of which might read what the other has added to).
template <class E, int W>
struct Cols {
  typedef E type __attribute__((ext_vector_type(W)));
  struct __attribute__((packed, aligned(sizeof(E)))) Any { type v; };
};

// One wave: chunk x slice, W columns a lane in each half of the slice, so that
// every store of a sum is one stretch.  A run of up to two chunks' length that begins in the
// chunk is finished by its wave (the next one leaves its first places out);
// only longer ones leave partial rows.  Rows are asked for U at a time, and with
// ACC the rows of dW that their runs end in too (one by one, each waits for its
// own).
template <class E, bool ACC, int W>
__device__ __forceinline__ void sum_chunk(const EmbedGradP& p, long long chunk, int slice) {
  const int lane = threadIdx.x & 63, len = p.len;
  int c[2];
  bool on[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int o = (h * 64 + lane) * W;
    on[h] = o < p.width && slice * p.width + o < p.m;
    c[h] = min(slice * p.width + o, p.m - W);
  }
  const long long from = chunk * len, rest = p.T - from;
  const int cnt = rest < len ? (int)rest : len, known = rest < 2 * len ? (int)rest : 2 * len;
  const int k = lane < known ? p.key[from + lane] : p.n;
  const int at = lane < known ? p.pos[from + lane] : 0;
  const int before = from > 0 ? p.key[from - 1] : -1;
  const int back = from > 0 ? p.key[from - len] : -1, back1 = from > len ? p.key[from - len - 1] : -1;
  const int beyond = rest > 2 * len ? p.key[from + 2 * len] : -1;
  auto end_of = [&](int key, int i) {               // the first of the known places from i on of another key
    const unsigned long long b = __ballot(k != key || lane >= known) >> i;
    return b ? i + __builtin_ctzll(b) : known;
  };
  const int first = __builtin_amdgcn_readlane(k, 0), last = __builtin_amdgcn_readlane(k, cnt - 1);
  int i0 = 0, stop = cnt;
  bool head = false, tail = false;
  if (first == before) {
    const int e = end_of(first, 0);
    if (e <= len && !(back == first && back1 == first)) i0 = e;     // finished by the wave before
    else head = true;
  }
  if (i0 >= cnt) return;
  if (known > cnt && __builtin_amdgcn_readlane(k, cnt) == last && !(head && last == first)) {
    tail = beyond == last;
    if (!tail) stop = end_of(last, cnt);
  }
  typedef typename Cols<E, W>::Any In;
  typedef typename Cols<float, W>::Any Sum;
  Sum acc[2] = {};
  constexpr int U = ACC ? 4 : 8;
  for (; i0 < stop; i0 += U) {
    In raw[U][2];
    Sum old[ACC ? U : 1][2];
    // (without branches, which would wait for one load before the next; past the
    // end the last place's row, and any row of dW, are asked for and not used)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, stop - 1);
      const E* row = (const E*)p.dy + __builtin_amdgcn_readlane(at, i) * p.lddy;
      const float* sum = p.dw + min(__builtin_amdgcn_readlane(k, i), p.n - 1) * p.ldw;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        raw[u][h] = *(const In*)(row + c[h]);
        if (ACC) old[u][h] = *(const Sum*)(sum + c[h]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= stop) continue;
      const int key = __builtin_amdgcn_readlane(k, i);
      if (key == p.n) return;                       // no tokens from here on
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < W; ++e) acc[h].v[e] += to_f32((E)raw[u][h].v[e]);
      if (i + 1 < stop && __builtin_amdgcn_readlane(k, i + 1) == key) continue;
      const bool part = head || (tail && i + 1 == stop);
      if (p.set && slice == 0 && lane == 0) p.set[key] = 1;
      float* row = part ? p.part + (chunk * 2 + (head ? 0 : 1)) * p.m : p.dw + key * p.ldw;
      const float scale = part ? 1.0f : p.scale;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < W; ++e)
          acc[h].v[e] = ACC && !part ? old[u][h].v[e] + scale * acc[h].v[e] : scale * acc[h].v[e];
        if (on[h]) {
          if constexpr (ACC) *(Sum*)(row + c[h]) = acc[h];
          else store_once(row + c[h], acc[h].v);
        }
        acc[h] = Sum{};
      }
      head = false;
    }
  }
}

template <class E, bool ACC, int W>
__global__ __launch_bounds__(256) void k_embed_grad(EmbedGradP p) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long task = grid_block() * 4 + wave, chunk = task / p.slices;
  if (chunk * p.len < p.T) sum_chunk<E, ACC, W>(p, chunk, (int)(task - chunk * p.slices));
}

// The last launch.  The long runs: a workgroup looks through 16 chunks for those in which one
// begins and adds up its partial rows in 256 columns, its 4 waves a quarter of
// the rows each.  The other workgroups clear the rows of dW without a token.
constexpr int kJoinChunks = 16;
__global__ __launch_bounds__(256) void k_embed_join(EmbedGradP p, long long chunks, long long joins,
                                                    Zero z) {
  __shared__ double sh[3][64][4];
  if (grid_block() >= joins) {
    zero_block<256>(z, grid_block() - joins);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, len = p.len;
  const long long block = grid_block();
  const int cols = (p.m + 255) / 256;
  const long long group = block / cols;
  if (group * kJoinChunks >= chunks) return;
  const int c = (int)(block - group * cols) * 256 + lane * 4;
  int key = p.n;
  {
    const long long from = (group * kJoinChunks + lane) * len;
    if (lane < kJoinChunks && from + 2 * len < p.T) {
      const int first = p.key[from], last = p.key[from + len - 1], beyond = p.key[from + 2 * len];
      const int before = from > 0 ? p.key[from - 1] : -1;
      if (last == beyond && !(first == last && before == last)) key = last;
    }
  }
  for (unsigned long long todo = __ballot(key != p.n); todo; todo &= todo - 1) {
    const int which = __builtin_ctzll(todo), row = __builtin_amdgcn_readlane(key, which);
    const long long c0 = group * kJoinChunks + which;
    long long c1 = c0 + 1;                            // the run's last chunk:
    for (;;) {                                        // those it fills, 64 at a time
      const long long i = (c1 + lane) * len + len - 1;
      const unsigned long long not_full =
          ~__ballot(i + 1 < p.T && p.key[i] == row && p.key[i + 1] == row);
      const int full = not_full ? __builtin_ctzll(not_full) : 64;
      c1 += full;
      if (full < 64) break;
    }
    const long long count = c1 - c0 + 1, per = (count + 3) / 4;
    const long long a = wave * per, b = a + per < count ? a + per : count;
    double v[4] = {0, 0, 0, 0};
    const bool vec = c + 4 <= p.m;
    struct __attribute__((packed, aligned(4))) F4 { float x[4]; };
#pragma unroll 8
    for (long long i = a; i < b; ++i) {
      const float* part = p.part + ((c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.m;
      if (vec) {
        const F4 f = *(const F4*)(part + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += (double)f.x[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.m) v[e] += (double)part[c + e];
      }
    }
    __syncthreads();                                  // (the run before has been read)
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sh[wave - 1][lane][e] = v[e];
    }
    __syncthreads();
    if (wave > 0) continue;
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += sh[w][lane][e];
    float* d = p.dw + row * p.ldw;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < p.m) d[c + e] = (float)((p.accumulate ? (double)d[c + e] : 0.0) + p.scale * v[e]);
  }
}

// --------------------------------------------------------------- the launches

dim3 grid_of(long long blocks) {
  const long long row = 1LL << 21;
  return blocks <= row ? dim3((unsigned)blocks)
                       : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}

// The workspace: sorted keys and places (twice for the sort by digits, which
// swaps them, and its histograms), the rows' flags, then the partial rows.  A chunk is of
// kMaxChunk places, of fewer where there would be less than 4096 waves.  Two chunks
// have no run to join: up to 64 tokens take two, and no launch for it.
struct EmbedPlan {
  int digits, tiles, len;
  long long chunks;
  size_t at_hist, at_set, at_part, bytes;
};
EmbedPlan plan_embed(long long T, int n, int m) {
  EmbedPlan q = {};
  q.len = kMaxChunk;
  while (q.len > 8 && T / q.len * ((m + 511) / 512) < 4096) q.len /= 2;
  if (T <= 2 * kMaxChunk) q.len = (int)(T + 1) / 2;
  if (q.len < 1) q.len = 1;
  q.chunks = (T + q.len - 1) / q.len;
  const size_t list = (size_t)pad_to(T, 64) * 4;
  size_t b = 2 * list;
  if (T > kCountMax) {
    q.tiles = (int)((T + kTile - 1) / kTile);
    for (int k = n; k; k >>= 8) ++q.digits;        // keys 0 .. n
    b += 2 * list;
    q.at_hist = b;
    b += (size_t)q.tiles * 1024;
  }
  q.at_set = b;
  b += (size_t)pad_to(n, 256);
  q.at_part = b;
  q.bytes = T ? b + (size_t)q.chunks * 2 * m * 4 : 0;
  return q;
}

// The widest slice that leaves none of 1 to 3 columns behind (found for every
// m: with q = m / 512, 508 leaves 4 q + m % 512 modulo 508, and where q is a
// multiple of 127, 504 leaves 8 more for each).
int slice_width(int m) {
  for (int w = 512; w > 504; w -= 4)
    if (m % w == 0 || m % w >= 4 || m < 4) return w;
  return 504;
}

Zero zeros(float* dw, const unsigned char* set, long long n, int m, long long ldw) {
  Zero z = {dw, set, ldw, 0, n * ((m + 3) / 4), (unsigned)((m + 3) / 4), m};
  z.blocks = (z.items + 255) / 256;
  return z;
}

hipError_t sort_tokens(const void* tokens, int is64, long long T, int n, const EmbedPlan& q,
                       char* ws, unsigned char* set, const Zero& z, const int*& key,
                       const int*& pos, hipStream_t s) {
  const size_t list = (size_t)pad_to(T, 64) * 4;
  int* buf[2][2] = {{(int*)ws, (int*)(ws + list)}, {(int*)(ws + 2 * list), (int*)(ws + 3 * list)}};
  if (!q.digits) {
    const int sets = set ? (n + 15) / 16 : 0;
    const long long more = set ? (sets + 1023) / 1024 : (z.items + 1023) / 1024;
    hipLaunchKernelGGL(k_embed_count, grid_of((T + 31) / 32 + more), dim3(1024),
                       (size_t)pad_to(T, 32) * 4, s, tokens, is64, (int)T, n, buf[0][0], buf[0][1],
                       (uint4*)set, sets, z);
    key = buf[0][0];
    pos = buf[0][1];
    return hipGetLastError();
  }
  if (set) {
    const int words = (n + 3) / 4;
    hipLaunchKernelGGL(k_embed_zero, dim3((words + 1023) / 1024), dim3(256), 0, s,
                       zeros((float*)set, nullptr, 1, words, words));
  }
  for (int d = 0; d < q.digits; ++d) {
    const int o = d & 1;
    const DigitP p = {d ? nullptr : tokens, is64, buf[1 - o][0], buf[1 - o][1], buf[o][0], buf[o][1],
                      (int*)(ws + q.at_hist), T, n, q.tiles, 8 * d};
    hipLaunchKernelGGL(k_embed_hist, dim3(q.tiles), dim3(256), 0, s, p);
    if (q.tiles > kOwnScan)
      hipLaunchKernelGGL(k_embed_scan, dim3(1), dim3(1024), 0, s, p.hist, 256 * q.tiles);
    hipLaunchKernelGGL(k_embed_place, dim3(q.tiles), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    key = buf[o][0];
    pos = buf[o][1];
  }
  return hipSuccess;
}

template <class WT, class E>
hipError_t launch_embed(const void* tokens, int is64, const void* W, long long ldw, void* Y,
                        long long ldy, long long T, int n, int m, float scale, hipStream_t s) {
  const unsigned nch = (unsigned)((m + 7) / 8);
  const long long chunks = T * nch;
  // Rows longer than the cache keeps are written past it (with a pass over them:
  // 349 -> 316 us at 512 MB, 90 -> 87 at 128, 45.7 -> 46.5 at 64).
  const int once = (double)T * m * sizeof(E) > 96e6;
  hipLaunchKernelGGL((k_embed<WT, E>), flat_grid(chunks), dim3(256), 0, s, tokens, is64,
                     (const WT*)W, ldw, (E*)Y, ldy, chunks, n, m, nch, scale, once);
  return hipGetLastError();
}

template <class E>
void launch_embed_grad(const EmbedGradP& p, dim3 grid, hipStream_t s) {
  if (p.m < 4) {
    if (p.accumulate) hipLaunchKernelGGL((k_embed_grad<E, true, 1>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_embed_grad<E, false, 1>), grid, dim3(256), 0, s, p);
  } else {
    if (p.accumulate) hipLaunchKernelGGL((k_embed_grad<E, true, 4>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_embed_grad<E, false, 4>), grid, dim3(256), 0, s, p);
  }
}

bool any_type(int t) { return type16(t) || t == DION3_F32; }
int size_of(int t) { return t == DION3_F32 ? 4 : 2; }

dion3_status check_tokens(const void* tokens, int bits, int64_t T) {
  if (bits != 32 && bits != 64) return DION3_ERR_ARG;
  if (T > 0 && (!tokens || !elem_aligned(tokens, bits / 8))) return DION3_ERR_ARG;
  return DION3_OK;
}

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

dion3_status dion3_embedding(const void* tokens, int32_t token_bits, const void* W, int64_t ldw,
                             int32_t wtype, void* Y, int64_t ldy, int64_t T, int64_t n, int64_t m,
                             float scale, int32_t dtype, void* stream) {
  if (!any_type(dtype) || (wtype != DION3_F32 && wtype != dtype) || !isfinite(scale))
    return DION3_ERR_ARG;
  TRY(check_sizes(T, n, m));
  TRY(check_far_ld(ldw, m));
  TRY(check_far_ld(ldy, m));
  TRY(check_tokens(tokens, token_bits, T));
  if (T == 0) return DION3_OK;
  if (!W || !Y || !elem_aligned(W, size_of(wtype)) || !elem_aligned(Y, size_of(dtype)))
    return DION3_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  const int is64 = token_bits == 64, N = (int)n, M = (int)m;
  TraceScope ts("embedding", 0.0, (double)T * m * (size_of(wtype) + size_of(dtype)), s);
  if (wtype == DION3_F32) {
    if (dtype == DION3_F32) HIP_TRY((launch_embed<float, float>(tokens, is64, W, ldw, Y, ldy, T, N, M, scale, s)));
    else if (dtype == DION3_BF16) HIP_TRY((launch_embed<float, bf16>(tokens, is64, W, ldw, Y, ldy, T, N, M, scale, s)));
    else HIP_TRY((launch_embed<float, f16>(tokens, is64, W, ldw, Y, ldy, T, N, M, scale, s)));
  } else if (dtype == DION3_BF16) {
    HIP_TRY((launch_embed<bf16, bf16>(tokens, is64, W, ldw, Y, ldy, T, N, M, scale, s)));
  } else {
    HIP_TRY((launch_embed<f16, f16>(tokens, is64, W, ldw, Y, ldy, T, N, M, scale, s)));
  }
  return DION3_OK;
}

dion3_status dion3_embedding_grad_workspace_size(int64_t T, int64_t n, int64_t m, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, m));
  *bytes = plan_embed(T, (int)n, (int)m).bytes;
  return DION3_OK;
}

dion3_status dion3_embedding_grad(const void* tokens, int32_t token_bits, const void* dY,
                                  int64_t lddy, float* dW, int64_t ldw, int32_t accumulate,
                                  int64_t T, int64_t n, int64_t m, float scale, int32_t dtype,
                                  void* ws, size_t ws_bytes, void* stream) {
  if (!any_type(dtype) || !isfinite(scale)) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, m));
  TRY(check_far_ld(lddy, m));
  TRY(check_far_ld(ldw, m));
  TRY(check_tokens(tokens, token_bits, T));
  if (!dW || !elem_aligned(dW, 4)) return DION3_ERR_ARG;
  if (T > 0 && (!dY || !elem_aligned(dY, size_of(dtype)))) return DION3_ERR_ARG;
  const EmbedPlan q = plan_embed(T, (int)n, (int)m);
  TRY(check_scratch(ws, ws_bytes, q.bytes));
  if (T == 0 && accumulate) return DION3_OK;
  hipStream_t s = (hipStream_t)stream;
  EmbedGradP p = {};
  p.dy = dY; p.lddy = lddy; p.dw = dW; p.ldw = ldw;
  p.T = T; p.n = (int)n; p.m = (int)m;
  p.width = slice_width((int)m); p.slices = (int)((m + p.width - 1) / p.width);
  p.scale = scale; p.accumulate = accumulate != 0; p.len = q.len;
  p.part = (float*)((char*)ws + q.at_part);
  // Few tokens (no joins) have dW cleared beside their sort, two launches in
  // all: 14 tokens of 84376 x 424 take 25 us instead of 31.
  const double cleared = accumulate ? 0.0 : 4.0 * n * m;
  const bool early = T <= 2 * kMaxChunk;
  Zero z = {}, none = {};
  if (!accumulate) {
    p.set = early ? nullptr : (unsigned char*)ws + q.at_set;
    z = zeros(dW, p.set, n, (int)m, ldw);
  }
  if (T == 0) {
    TraceScope ts("embedding_zero", 0.0, cleared, s);
    hipLaunchKernelGGL(k_embed_zero, grid_of(z.blocks), dim3(256), 0, s, z);
    HIP_TRY(hipGetLastError());
    return DION3_OK;
  }
  {
    TraceScope ts("embedding_sort", 0.0, 16.0 * T + (early ? cleared : 0.0), s);
    HIP_TRY(sort_tokens(tokens, token_bits == 64, T, (int)n, q, (char*)ws, p.set, early ? z : none,
                        p.key, p.pos, s));
  }
  {
    TraceScope ts("embedding_grad", 0.0, (double)T * m * size_of(dtype), s);
    const dim3 grid = grid_of((q.chunks * p.slices + 3) / 4);
    if (dtype == DION3_BF16) launch_embed_grad<bf16>(p, grid, s);
    else if (dtype == DION3_F16) launch_embed_grad<f16>(p, grid, s);
    else launch_embed_grad<float>(p, grid, s);
    HIP_TRY(hipGetLastError());
  }
  const long long joins =
      T > 2 * q.len ? (q.chunks + kJoinChunks - 1) / kJoinChunks * ((m + 255) / 256) : 0;
  if (early) z = none;
  if (joins + z.blocks > 0) {
    TraceScope ts("embedding_join", 0.0, early ? 0.0 : cleared, s);
    hipLaunchKernelGGL(k_embed_join, grid_of(joins + z.blocks), dim3(256), 0, s, p, q.chunks, joins, z);
    HIP_TRY(hipGetLastError());
  }
  return DION3_OK;
}

}  // extern "C"
