// Row kernels of the layer operators: the root-mean-square norm with the
// residual's addition and its gradient, the 8-bit format of activation
// checkpoints, and the activation's gradient.  All of them are bound by HBM:
// each reads its inputs once and writes its outputs once; statistics and
// column sums are held in fp32 and added in a fixed order (no atomics), so a
// call's result does not depend on how its workgroups are scheduled.
#include "layer_internal.h"

namespace dion3 {
namespace {

// Sum over the threads that share a row, the same bits in every one of them:
// butterfly inside each wave, then (WIDE: a row is the whole workgroup's) one
// over the waves' sums, each 16 lanes reading all of them at once (a loop over
// them waits for LDS once a wave; the 2048-wide norm took 57 us instead of
// 44).  `sh` holds two sets, used in turn by consecutive
// calls (`turn`), so that one barrier a call is enough: a set is written again
// only after every thread has passed the next call's barrier.
constexpr int kMaxWaves = 16;
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, float* sh, int turn) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  if constexpr (WIDE) {
    const int nw = blockDim.x >> 6;
    float* set = sh + (turn & 1) * kMaxWaves;
    if ((threadIdx.x & 63) == 0) set[threadIdx.x >> 6] = v;
    __syncthreads();
    const int w = threadIdx.x & (kMaxWaves - 1);
    v = w < nw ? set[w] : 0.0f;
#pragma unroll
    for (int o = 1; o < kMaxWaves; o <<= 1) v += __shfl_xor(v, o, 64);
  }
  return v;
}

// Threads of a row of m columns with at most `ch` chunks of 8 columns each: a
// whole wave up to 512 columns (four rows a workgroup), else as many waves as
// the chunks need, so that few lanes idle at any width.
struct RowShape {
  bool wide;
  int ch, nt;       // chunks a thread, threads of the workgroup
};
RowShape row_shape(long long cols) {
  const long long chunks = (cols + 7) / 8;
  if (chunks <= 64) return {false, 1, 256};
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  return {true, ch, (int)((chunks + 64 * ch - 1) / (64 * ch)) * 64};
}

// ------------------------------------------------------------------ the norm

//   h = E(x + r),  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y = E(h rstd w),
//   and y in 8 bits.  The statistics and y come from the rounded h, the one
//   that the layers after this one read.
// Bound by HBM: 8192 x 4096 with the residual 44 us (6.1 TB/s), with the 8-bit
// output too 55-57 us (5.4 TB/s); 1 x 4096 3 us.
// The threads of a row (RowShape) hold CH chunks of 8 columns each in
// registers, so x and r are read once and h never read back; a workgroup takes
// every gridDim-th row and keeps w in registers.
struct NormP {
  const void* x; const void* r; const void* w;
  void* h; void* y;
  unsigned char* q; unsigned char* s;
  float* rstd;
  long long ldx, ldr, ldh, ldy, T;
  int m;
  float eps;
};

__device__ __forceinline__ float norm_rstd(float sumsq, int m, float eps) {
  return 1.0f / sqrtf(sumsq / (float)m + eps);
}

template <class E, class WT, bool WIDE, int CH>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void k_add_norm(NormP p) {
  const int NT = WIDE ? blockDim.x : 64, RPW = WIDE ? 1 : 4;   // threads a row, rows a workgroup
  __shared__ float sh[2 * kMaxWaves];
  const int t = WIDE ? threadIdx.x : threadIdx.x & 63;
  const int m = p.m, mp = (m + kF8Block - 1) / kF8Block * kF8Block;
  float w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) load8((const WT*)p.w, (t + i * NT) * 8, m, w[i]);
  int turn = 0;
  const long long step = (long long)gridDim.x * RPW;
  long long row = (long long)blockIdx.x * RPW + (WIDE ? 0 : threadIdx.x >> 6);
  // a row's chunks are on their way while the row before it is summed and
  // written (where the registers hold them)
  constexpr bool AHEAD = CH <= 2;
  Raw8<E> rx[CH], rr[CH];
  auto ask = [&](long long at) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rx[i] = fetch8((const E*)p.x + at * p.ldx, (t + i * NT) * 8, m);
      if (p.r) rr[i] = fetch8((const E*)p.r + at * p.ldr, (t + i * NT) * 8, m);
    }
  };
  if (AHEAD && row < p.T) ask(row);
  for (; row < p.T; row += step) {
    if (!AHEAD) ask(row);
    float v[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      chunk8(rx[i], (t + i * NT) * 8, m, v[i]);
      if (p.r) {
        float u[8];
        chunk8(rr[i], (t + i * NT) * 8, m, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = to_f32((E)(v[i][e] + u[e]));
      }
    }
    if (AHEAD && row + step < p.T) ask(row + step);
    if (p.r) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if ((t + i * NT) * 8 < m) store8((E*)p.h + row * p.ldh, (t + i * NT) * 8, m, v[i]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[i][e], v[i][e], ss);
    ss = row_sum<WIDE>(ss, sh, turn++);
    const float rs = norm_rstd(ss, m, p.eps);
    if (t == 0 && p.rstd) p.rstd[row] = rs;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (t + i * NT) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = to_f32((E)(v[i][e] * rs * w[i][e]));
      if (p.y && c < m) store8((E*)p.y + row * p.ldy, c, m, v[i]);
      if (p.q) {
        // columns past m hold zeros: inf rstd would make them NaN
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= m) v[i][e] = 0.0f;
        int byte;
        const uint2 q8 = f8_encode_block<E>(v[i], byte);
        if (c < mp) {
          *(uint2*)(p.q + row * mp + c) = q8;
          if ((c & (kF8Block - 1)) == 0) p.s[row * (mp / kF8Block) + c / kF8Block] = byte;
        }
      }
    }
  }
}

// Rows too long for registers: one workgroup a row, h read back for the
// second pass (from L2: the row was written by the same workgroup).
template <class E, class WT>
__global__ __launch_bounds__(1024) void k_add_norm_long(NormP p) {
  constexpr int NT = 1024;
  __shared__ float sh[2 * kMaxWaves];
  const int t = threadIdx.x;
  const int m = p.m, mp = (m + kF8Block - 1) / kF8Block * kF8Block;
  int turn = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const E* xr = (const E*)p.x + row * p.ldx;
    const E* rr = p.r ? (const E*)p.r + row * p.ldr : nullptr;
    float ss = 0.0f;
    for (int c = t * 8; c < m; c += NT * 8) {
      float v[8];
      load8(xr, c, m, v);
      if (rr) {
        float u[8];
        load8(rr, c, m, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32((E)(v[e] + u[e]));
        store8((E*)p.h + row * p.ldh, c, m, v);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
    }
    ss = row_sum<true>(ss, sh, turn++);
    const float rs = norm_rstd(ss, m, p.eps);
    if (t == 0 && p.rstd) p.rstd[row] = rs;
    // (each thread reads back only what it wrote itself)
    const E* hr = p.r ? (const E*)p.h + row * p.ldh : xr;
    for (int c0 = 0; c0 < mp; c0 += NT * 8) {      // whole waves stay for the block maxima
      const int c = c0 + t * 8;
      float v[8], w[8];
      load8(hr, c, m, v);
      load8((const WT*)p.w, c, m, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = to_f32((E)(v[e] * rs * w[e]));
      if (p.y && c < m) store8((E*)p.y + row * p.ldy, c, m, v);
      if (p.q) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= m) v[e] = 0.0f;
        int byte;
        const uint2 q8 = f8_encode_block<E>(v, byte);
        if (c < mp) {
          *(uint2*)(p.q + row * mp + c) = q8;
          if ((c & (kF8Block - 1)) == 0) p.s[row * (mp / kF8Block) + c / kF8Block] = byte;
        }
      }
    }
  }
}

template <class E, class WT>
hipError_t launch_norm_t(const NormP& p, hipStream_t s) {
  const long long T = p.T;
  const int mp = (int)f8_cols(p.m);
  if (mp > 32768) {
    hipLaunchKernelGGL((k_add_norm_long<E, WT>), dim3((unsigned)(T < 512 ? T : 512)), dim3(1024), 0, s,
                       p);
    return hipGetLastError();
  }
  const RowShape q = row_shape(mp);
  // workgroups that stay resident (6 waves a SIMD with one chunk a thread; more
  // rows are taken in turns), and half as many again of the wider ones, whose
  // sizes leave gaps (8192 x 4096 44 us, 4096 x 11008 72 us; 46 and 79 with
  // the other's rule)
  const long long rows = q.wide ? 1 : 4, need = (T + rows - 1) / rows, most = 256LL * (q.ch == 1 ? 1536 : 2048) / q.nt;
  const dim3 grid((unsigned)(need < most ? need : most)), block(q.nt);
  if (!q.wide) hipLaunchKernelGGL((k_add_norm<E, WT, false, 1>), grid, block, 0, s, p);
  else if (q.ch == 1) hipLaunchKernelGGL((k_add_norm<E, WT, true, 1>), grid, block, 0, s, p);
  else if (q.ch == 2) hipLaunchKernelGGL((k_add_norm<E, WT, true, 2>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_add_norm<E, WT, true, 4>), grid, block, 0, s, p);
  return hipGetLastError();
}

// ------------------------------------------------------- the norm's gradient

//   a = w dy, hat = h rstd, c = mean_j a_j hat_j,
//   dx = E(rstd (a - hat c) + dh),  dw = sum over rows of dy hat.
// Bound by HBM: 8192 x 4096 50 us (5.4 TB/s) and 7 us for the join.
// The same split as the norm; a workgroup (a unit) takes every gridDim-th row
// (or four rows at a time), keeps w and its part of dw in registers and leaves
// its part as one row of the scratch, which k_join_columns adds up in unit
// order.
struct NormGradP {
  const void* dy; const void* h; const void* dh; const void* w;
  const float* rstd;
  void* dx;
  float* part;             // null: dw not wanted
  float* c;                // the long form's row means
  long long lddy, ldh, lddh, lddx, T;
  int m;
  long long rows_per_unit; // the long form's row blocks
};

template <class E, class WT, bool WIDE, int CH>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void k_norm_grad(NormGradP p) {
  const int NT = WIDE ? blockDim.x : 64, RPW = WIDE ? 1 : 4;
  __shared__ float sh[WIDE ? 2 * kMaxWaves : 3 * 512];
  const int t = WIDE ? threadIdx.x : threadIdx.x & 63;
  const int m = p.m;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    load8((const WT*)p.w, (t + i * NT) * 8, m, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  int turn = 0;
  const long long step = (long long)gridDim.x * RPW;
  long long row = (long long)blockIdx.x * RPW + (WIDE ? 0 : threadIdx.x >> 6);
  const bool more = p.dh && p.dx;
  Raw8<E> rh[CH], ry[CH], rd[CH];
  float rs = 0.0f;
  auto ask = [&](long long at) {
    rs = p.rstd[at];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rh[i] = fetch8((const E*)p.h + at * p.ldh, (t + i * NT) * 8, m);
      ry[i] = fetch8((const E*)p.dy + at * p.lddy, (t + i * NT) * 8, m);
      if (more) rd[i] = fetch8((const E*)p.dh + at * p.lddh, (t + i * NT) * 8, m);
    }
  };
  // (a row ahead costs more in resident workgroups than it hides: 8192 x 4096
  // 66 us instead of 55)
  for (; row < p.T; row += step) {
    ask(row);
    const float r1 = rs;
    float hat[CH][8], dy[CH][8], dh[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      chunk8(rh[i], (t + i * NT) * 8, m, hat[i]);
      chunk8(ry[i], (t + i * NT) * 8, m, dy[i]);
      if (more) chunk8(rd[i], (t + i * NT) * 8, m, dh[i]);
    }
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hat[i][e] *= r1;
        dw[i][e] = __builtin_fmaf(dy[i][e], hat[i][e], dw[i][e]);
        dy[i][e] *= w[i][e];
        c = __builtin_fmaf(dy[i][e], hat[i][e], c);
      }
    if (!p.dx) continue;
    c = row_sum<WIDE>(c, sh, turn++) / (float)m;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * NT) * 8;
      if (col >= m) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = r1 * __builtin_fmaf(-hat[i][e], c, dy[i][e]);
        if (more) o[e] += dh[i][e];
      }
      store8((E*)p.dx + row * p.lddx, col, m, o);
    }
  }
  if (!p.part) return;
  if constexpr (!WIDE) {          // the four waves' parts, in wave order
    const int wave = threadIdx.x >> 6;
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sh[(wave - 1) * 512 + t * 8 + e] = dw[0][e];
    }
    __syncthreads();
    if (wave > 0) return;
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[0][e] += sh[w * 512 + t * 8 + e];
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int col = (t + i * NT) * 8;
    if (col < m) store8(p.part + (long long)blockIdx.x * m, col, m, dw[i]);
  }
}

// Rows too long for registers: the row means first, then a pass by blocks of
// columns, each thread on its own 8 columns of a block of rows.
template <class E, class WT>
__global__ __launch_bounds__(1024) void k_norm_grad_mean(NormGradP p) {
  __shared__ float sh[2 * kMaxWaves];
  const int m = p.m;
  int turn = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const float rs = p.rstd[row];
    float c = 0.0f;
    for (int col = threadIdx.x * 8; col < m; col += 1024 * 8) {
      float hat[8], dy[8], w[8];
      load8((const E*)p.h + row * p.ldh, col, m, hat);
      load8((const E*)p.dy + row * p.lddy, col, m, dy);
      load8((const WT*)p.w, col, m, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) c = __builtin_fmaf(dy[e] * w[e], hat[e] * rs, c);
    }
    c = row_sum<true>(c, sh, turn++) / (float)m;
    if (threadIdx.x == 0) p.c[row] = c;
  }
}

template <class E, class WT>
__global__ __launch_bounds__(256) void k_norm_grad_cols(NormGradP p) {
  const int m = p.m, col = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= m) return;
  float w[8], dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  load8((const WT*)p.w, col, m, w);
  const long long r0 = (long long)blockIdx.y * p.rows_per_unit;
  const long long r1 = r0 + p.rows_per_unit < p.T ? r0 + p.rows_per_unit : p.T;
  for (long long row = r0; row < r1; ++row) {
    const float rs = p.rstd[row];
    float hat[8], dy[8], dh[8], o[8];
    load8((const E*)p.h + row * p.ldh, col, m, hat);
    load8((const E*)p.dy + row * p.lddy, col, m, dy);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hat[e] *= rs;
      dw[e] = __builtin_fmaf(dy[e], hat[e], dw[e]);
    }
    if (!p.dx) continue;
    const float c = p.c[row];
    if (p.dh) load8((const E*)p.dh + row * p.lddh, col, m, dh);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] = rs * __builtin_fmaf(-hat[e], c, dy[e] * w[e]);
      if (p.dh) o[e] += dh[e];
    }
    store8((E*)p.dx + row * p.lddx, col, m, o);
  }
  if (p.part) store8(p.part + (long long)blockIdx.y * m, col, m, dw);
}

constexpr int kLongCols = 16384;      // rows up to this many columns stay in registers

// Units (partial rows of dw) of the gradient: as many as stay resident, so that
// one row's reduction overlaps the others' loads, and no more, since each unit
// writes and reads a row of fp32 (8192 x 4096: 55 us with 6 waves a SIMD, 59
// with 4, 65 with 8).
RowsPlan norm_grad_plan(long long T, long long m) {
  RowsPlan q;
  if (m > kLongCols) {
    const long long blocks = T < 64 ? T : 64;
    q.rows_per_unit = (int)((T + blocks - 1) / blocks);
    q.units = (int)((T + q.rows_per_unit - 1) / q.rows_per_unit);
    return q;
  }
  const RowShape r = row_shape(m);
  const long long most = 256LL * (r.ch == 1 ? 1536 : 1280) / r.nt, rows = r.wide ? 1 : 4;
  const long long need = (T + rows - 1) / rows;
  q.units = (int)(need < most ? need : most);
  q.rows_per_unit = 0;
  return q;
}

template <class E, class WT>
hipError_t launch_norm_grad_t(NormGradP p, const RowsPlan& plan, hipStream_t s) {
  const int m = p.m;
  if (m > kLongCols) {
    p.rows_per_unit = plan.rows_per_unit;
    if (p.dx) {
      hipLaunchKernelGGL((k_norm_grad_mean<E, WT>), dim3((unsigned)(p.T < 512 ? p.T : 512)),
                         dim3(1024), 0, s, p);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_norm_grad_cols<E, WT>), dim3((m + 2047) / 2048, plan.units), dim3(256), 0,
                       s, p);
    return hipGetLastError();
  }
  const RowShape r = row_shape(m);
  const dim3 grid(plan.units), block(r.nt);
  if (!r.wide) hipLaunchKernelGGL((k_norm_grad<E, WT, false, 1>), grid, block, 0, s, p);
  else if (r.ch == 1) hipLaunchKernelGGL((k_norm_grad<E, WT, true, 1>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_norm_grad<E, WT, true, 2>), grid, block, 0, s, p);
  return hipGetLastError();
}

// out[j] = sum over units of part[u][j].  A workgroup takes 16 columns: 4
// threads across (4 columns each), 64 slices of the units down, whose sums
// are added in slice order.  768 x 4096: 7 us; 140 x 11008: 4 us.
__global__ __launch_bounds__(256) void k_join_columns(const float* __restrict__ part, int units,
                                                      int m, float* __restrict__ out) {
  __shared__ float sh[64][16];
  const int cq = threadIdx.x & 3, slice = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + cq * 4;
  const bool vec = (m & 3) == 0;
  float a[4] = {0, 0, 0, 0};
  const int per = (units + 63) / 64;
  const int u1 = min(units, (slice + 1) * per);
#pragma unroll 4
  for (int u = slice * per; u < u1; ++u) {
    const float* row = part + (long long)u * m;
    if (vec && c < m) {
      const float4 v = *(const float4*)(row + c);
      a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < m) a[e] += row[c + e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sh[slice][cq * 4 + e] = a[e];
  __syncthreads();
  if (threadIdx.x < 16) {
    float s = 0.0f;
    for (int i = 0; i < 64; ++i) s += sh[i][threadIdx.x];
    const int j = blockIdx.x * 16 + threadIdx.x;
    if (j < m) out[j] = s;
  }
}

// ------------------------------------------------------------- 8-bit format

// One chunk of 8 columns a thread, those of all rows numbered through (a row
// has mp / 8 of them, a multiple of 4, so the 4 lanes of a scale's block never
// straddle rows).  Bound by HBM: 8192 x 4096 18.5 us (5.5 TB/s).  Two or four
// chunks a thread were slower (20.5 us before the branch of f8_encode_block,
// 24 us with either).
template <class E>
__global__ __launch_bounds__(256) void k_pack(const E* __restrict__ x, long long ldx,
                                              unsigned char* __restrict__ q,
                                              unsigned char* __restrict__ sc, long long chunks,
                                              int m, unsigned nch) {
  const long long base = flat_base(), at = base + threadIdx.x;
  const long long row0 = base / nch;
  const unsigned c0 = (unsigned)(base - row0 * nch) + threadIdx.x, dr = c0 / nch;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (at < chunks) load8(x + (row0 + dr) * ldx, (int)(c0 - dr * nch) * 8, m, v);
  int byte;
  const uint2 w = f8_encode_block<E>(v, byte);
  if (at >= chunks) return;
  *(uint2*)(q + at * 8) = w;
  if ((threadIdx.x & 3) == 0) sc[at >> 2] = (unsigned char)byte;
}

template <class E>
__device__ __forceinline__ void f8_decode8(uint2 w, unsigned byte, float (&v)[8]) {
  const float s = f8_scale_float(byte);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const unsigned u = h ? w.y : w.x;
    const auto a = f8_decode2<false>(E(), u, s), b = f8_decode2<true>(E(), u, s);
    v[4 * h] = to_f32((E)a[0]);
    v[4 * h + 1] = to_f32((E)a[1]);
    v[4 * h + 2] = to_f32((E)b[0]);
    v[4 * h + 3] = to_f32((E)b[1]);
  }
}

// The values back, a chunk a thread: 8192 x 4096 17 us (6.0 TB/s).
template <class E>
__global__ __launch_bounds__(256) void k_unpack(const unsigned char* __restrict__ q,
                                                const unsigned char* __restrict__ sc,
                                                E* __restrict__ y, long long ldy,
                                                long long chunks, int m, unsigned nch) {
  const long long base = flat_base();
  if (base + threadIdx.x >= chunks) return;
  const long long row0 = base / nch;
  const unsigned c0 = (unsigned)(base - row0 * nch) + threadIdx.x;
  const unsigned dr = c0 / nch;
  const int c = (int)(c0 - dr * nch) * 8;
  if (c >= m) return;
  float v[8];
  f8_decode8<E>(*(const uint2*)(q + (base + threadIdx.x) * 8), sc[(base + threadIdx.x) >> 2], v);
  store8(y + (row0 + dr) * ldy, c, m, v);
}

// ------------------------------------------------- the activation's gradient

//   dz = E(dy act'(z)),  db = sum over rows of dy act'(z) (before rounding).
// Bound by HBM: 8192 x 11008 108 us whatever the activation (5.0 TB/s).
// A wave takes 512 columns (8 a lane), a workgroup a block of rows, its 4
// waves every fourth row of it, the next row's loads in flight; the
// waves' column sums join in LDS, the blocks' in k_join_columns.
struct ActGradP {
  const void* dy; const void* z;
  const unsigned char* zq; const unsigned char* zs;
  void* dz;
  float* part;
  long long lddy, ldz, lddz, T;
  int n, act, rows_per_unit;
};

template <class E, int ACT>
__global__ __launch_bounds__(256) void k_act_grad(ActGradP p) {
  __shared__ float sh[3][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = p.n, np = (n + kF8Block - 1) / kF8Block * kF8Block;
  const int c = blockIdx.x * 512 + lane * 8;
  float db[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const long long r0 = (long long)blockIdx.y * p.rows_per_unit;
  const long long r1 = r0 + p.rows_per_unit < p.T ? r0 + p.rows_per_unit : p.T;
  if (c < n) {
    Raw8<E> ry, rz;
    uint2 zq = make_uint2(0, 0);
    unsigned zs = 0;
    auto ask = [&](long long r) {
      ry = fetch8((const E*)p.dy + r * p.lddy, c, n);
      if (ACT == DION3_ACT_NONE) return;
      if (p.zq) {
        zq = *(const uint2*)(p.zq + r * np + c);
        zs = p.zs[r * (np / kF8Block) + c / kF8Block];
      } else {
        rz = fetch8((const E*)p.z + r * p.ldz, c, n);
      }
    };
    long long row = r0 + wave;
    if (row < r1) ask(row);
    for (; row < r1; row += 4) {
      float dy[8], z[8];
      chunk8(ry, c, n, dy);
      if (ACT != DION3_ACT_NONE) {
        if (p.zq) f8_decode8<float>(zq, zs, z);
        else chunk8(rz, c, n, z);
      }
      if (row + 4 < r1) ask(row + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (ACT != DION3_ACT_NONE) dy[e] *= slope(ACT, z[e]);
        db[e] += dy[e];
      }
      if (p.dz) store8((E*)p.dz + row * p.lddz, c, n, dy);
    }
  }
  if (!p.part) return;
  if (wave > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[wave - 1][lane * 8 + e] = db[e];
  }
  __syncthreads();
  if (wave == 0 && c < n) {
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) db[e] += sh[w][lane * 8 + e];
    store8(p.part + (long long)blockIdx.y * n, c, n, db);
  }
}

// Row blocks: about 4096 workgroups over the matrix, blocks of at least 16
// rows and at most 1024 blocks.
RowsPlan act_grad_plan(long long T, long long n) {
  const long long cols = (n + 511) / 512;
  long long blocks = (4096 + cols - 1) / cols;
  if (blocks > 1024) blocks = 1024;
  if (blocks > (T + 15) / 16) blocks = (T + 15) / 16;
  if (blocks < 1) blocks = 1;
  RowsPlan q;
  q.rows_per_unit = (int)((T + blocks - 1) / blocks);
  q.units = (int)((T + q.rows_per_unit - 1) / q.rows_per_unit);
  return q;
}

template <class E>
hipError_t launch_act_grad_t(const ActGradP& p, const RowsPlan& plan, hipStream_t s) {
  const dim3 grid((p.n + 511) / 512, plan.units);
#define DION3_ACT_GRAD(A) \
  case A: hipLaunchKernelGGL((k_act_grad<E, A>), grid, dim3(256), 0, s, p); break
  switch (p.act) {
    DION3_ACT_GRAD(DION3_ACT_NONE);
    DION3_ACT_GRAD(DION3_ACT_RELU);
    DION3_ACT_GRAD(DION3_ACT_GELU);
    DION3_ACT_GRAD(DION3_ACT_GELU_TANH);
    DION3_ACT_GRAD(DION3_ACT_SILU);
    default: return hipErrorInvalidValue;
  }
#undef DION3_ACT_GRAD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s) {
  const NormP p = {a.x, a.r, a.w, a.h, a.y, a.q, a.s, a.rstd,
                   a.ldx, a.ldr, a.ldh, a.ldy, a.T, a.m, a.eps};
  const double el = (double)a.T * a.m;
  TraceScope ts("add_rms_norm", 0.0, el * (2.0 + (a.r ? 4.0 : 0.0) + (a.y ? 2.0 : 0.0) +
                                           (a.q ? 1.0 + 1.0 / kF8Block : 0.0)), s);
  if (a.dtype == DION3_BF16)
    return a.wtype == DION3_F32 ? launch_norm_t<bf16, float>(p, s) : launch_norm_t<bf16, bf16>(p, s);
  return a.wtype == DION3_F32 ? launch_norm_t<f16, float>(p, s) : launch_norm_t<f16, f16>(p, s);
}

// The partial rows of dw, then the long form's row means.
size_t norm_grad_scratch(long long T, long long m) {
  if (T == 0) return 0;
  size_t b = (size_t)norm_grad_plan(T, m).units * m * 4;
  if (m > kLongCols) b += (size_t)T * 4;
  return b;
}

hipError_t launch_add_rms_norm_grad(const NormGradArgs& a, void* ws, hipStream_t s) {
  hipError_t e;
  RowsPlan plan = {0, 0};
  if (a.T > 0) {
    plan = norm_grad_plan(a.T, a.m);
    NormGradP p = {a.dy, a.h, a.dh, a.w, a.rstd, a.dx, a.dw ? (float*)ws : nullptr,
                   (float*)ws + (size_t)plan.units * a.m,
                   a.lddy, a.ldh, a.lddh, a.lddx, a.T, a.m, 0};
    TraceScope ts("rms_norm_grad", 0.0, (double)a.T * a.m * (4.0 + (a.dx ? 2.0 : 0.0) +
                                                             (a.dx && a.dh ? 2.0 : 0.0)), s);
    if (a.dtype == DION3_BF16)
      e = a.wtype == DION3_F32 ? launch_norm_grad_t<bf16, float>(p, plan, s)
                               : launch_norm_grad_t<bf16, bf16>(p, plan, s);
    else
      e = a.wtype == DION3_F32 ? launch_norm_grad_t<f16, float>(p, plan, s)
                               : launch_norm_grad_t<f16, f16>(p, plan, s);
    if (e != hipSuccess) return e;
  }
  return a.dw ? launch_join_columns((const float*)ws, plan.units, a.m, a.dw, s) : hipSuccess;
}

hipError_t launch_join_columns(const float* part, int units, int m, float* out, hipStream_t s) {
  TraceScope ts("join_columns", 0.0, ((double)units + 1.0) * m * 4.0, s);
  hipLaunchKernelGGL(k_join_columns, dim3((m + 15) / 16), dim3(256), 0, s, part, units, m, out);
  return hipGetLastError();
}

hipError_t launch_pack_f8(const void* x, long long ldx, unsigned char* q, unsigned char* sc,
                          long long T, int m, int dtype, hipStream_t s) {
  const unsigned nch = (unsigned)(f8_cols(m) / kChunk);
  const long long chunks = T * nch;
  const dim3 grid = flat_grid(chunks);
  TraceScope ts("pack_f8", 0.0, (double)T * m * ((dtype == DION3_F32 ? 4.0 : 2.0) + 1.0 + 1.0 / kF8Block), s);
  if (dtype == DION3_BF16)
    hipLaunchKernelGGL((k_pack<bf16>), grid, dim3(256), 0, s, (const bf16*)x, ldx, q, sc, chunks, m, nch);
  else if (dtype == DION3_F16)
    hipLaunchKernelGGL((k_pack<f16>), grid, dim3(256), 0, s, (const f16*)x, ldx, q, sc, chunks, m, nch);
  else
    hipLaunchKernelGGL((k_pack<float>), grid, dim3(256), 0, s, (const float*)x, ldx, q, sc, chunks, m, nch);
  return hipGetLastError();
}

hipError_t launch_unpack_f8(const unsigned char* q, const unsigned char* sc, void* y, long long ldy,
                            long long T, int m, int dtype, hipStream_t s) {
  const unsigned nch = (unsigned)(f8_cols(m) / kChunk);
  const long long chunks = T * nch;
  const dim3 grid = flat_grid(chunks);
  TraceScope ts("unpack_f8", 0.0, (double)T * m * ((dtype == DION3_F32 ? 4.0 : 2.0) + 1.0 + 1.0 / kF8Block), s);
  if (dtype == DION3_BF16)
    hipLaunchKernelGGL((k_unpack<bf16>), grid, dim3(256), 0, s, q, sc, (bf16*)y, ldy, chunks, m, nch);
  else if (dtype == DION3_F16)
    hipLaunchKernelGGL((k_unpack<f16>), grid, dim3(256), 0, s, q, sc, (f16*)y, ldy, chunks, m, nch);
  else
    hipLaunchKernelGGL((k_unpack<float>), grid, dim3(256), 0, s, q, sc, (float*)y, ldy, chunks, m, nch);
  return hipGetLastError();
}

size_t act_grad_scratch(long long T, long long n) {
  return T == 0 ? 0 : (size_t)act_grad_plan(T, n).units * n * 4;
}

hipError_t launch_act_grad(const ActGradArgs& a, void* ws, hipStream_t s) {
  RowsPlan plan = {0, 0};
  if (a.T > 0) {
    plan = act_grad_plan(a.T, a.n);
    const ActGradP p = {a.dy, a.z, a.zq, a.zs, a.dz, a.db ? (float*)ws : nullptr,
                        a.lddy, a.ldz, a.lddz, a.T, a.n, a.act, plan.rows_per_unit};
    const double zb = a.act == DION3_ACT_NONE ? 0.0 : a.zq ? 1.0 + 1.0 / kF8Block : 2.0;
    TraceScope ts("act_grad", 0.0, (double)a.T * a.n * (2.0 + zb + (a.dz ? 2.0 : 0.0)), s);
    const hipError_t e = a.dtype == DION3_BF16 ? launch_act_grad_t<bf16>(p, plan, s)
                                               : launch_act_grad_t<f16>(p, plan, s);
    if (e != hipSuccess) return e;
  }
  return a.db ? launch_join_columns((const float*)ws, plan.units, a.n, a.db, s) : hipSuccess;
}

}  // namespace dion3
