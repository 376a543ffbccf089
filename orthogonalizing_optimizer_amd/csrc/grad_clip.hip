// The global norm of many gradients and their clipping, in place or summed
// into fp32 buffers (the optimizer's momenta).
//
//   norm = scale (sum over all tensors of g^2)^(1/2),
//   c = norm <= max_norm ? 1 : max_norm / norm,
//   g <- E(c scale g)   or   M <- fp32(M + c scale g).
//
// Bound by HBM: the norm reads every gradient once (303 M bf16 elements 99.5 us,
// 6.1 TB/s), the second pass reads it again (such sizes pass the 256 MB cache)
// and writes it, or reads and writes the sums (582 us, 5.2 TB/s; the call 689).
// Not so tensors whose rows lie apart, which take an element and a division a
// lane at a time: 4096 x 4096 of fp32 with rows of 4104 31 us for the norm (14
// without gaps), 44 clipped in place (23), 96 into such sums (46).
// Squares are summed in 64 bits: no gradient of a 16- or 32-bit type leaves
// their range, and a conversion and a 64-bit fma an element take less than the
// element's time on HBM.  So do the products with c, whose factor leaves fp32's
// normal range where gradients are huge.
//
// A workgroup takes one chunk of one tensor and leaves one partial sum; the
// second pass adds all partial sums up in every workgroup, in one order, so
// that no launch stands between the two and no atomics are needed.  Where that
// would be more than about 2048 (16 KB for each workgroup to read), one
// workgroup adds them up in between.  The tensors' table travels in the
// kernel's arguments, kBatch tensors a launch: nothing is copied to the device,
// so a call can be captured.
#include "checks.h"

namespace dion3 {
namespace {

constexpr int kBatch = 56;              // 56 bytes each: 3.1 KB of arguments
constexpr long long kChunkMin = 8192;   // elements; a multiple of 256 threads x 8
constexpr long long kChunkMax = 32768;
constexpr int kPartials = 2048;         // partial sums that every workgroup adds up by itself

struct Entry {
  void* g; float* m;
  long long n, cols, ldg, ldm;          // cols == 0: dense
  int chunk0, dtype;
};
struct Table {
  Entry e[kBatch];
  int count, part0;                     // entries; the batch's first partial sum
  long long chunk;                      // elements
};

// The entry that a chunk belongs to, and the chunk's elements [lo, hi).
__device__ __forceinline__ const Entry& my_entry(const Table& t, int chunk, long long& lo,
                                                 long long& hi) {
  const int lane = threadIdx.x & 63;
  const bool mine = lane < t.count && t.e[lane < t.count ? lane : 0].chunk0 <= chunk;
  const int i = __builtin_amdgcn_readfirstlane(__popcll(__ballot(mine)) - 1);
  const Entry& e = t.e[i];
  lo = ((long long)chunk - e.chunk0) * t.chunk;
  hi = lo + t.chunk < e.n ? lo + t.chunk : e.n;
  return e;
}

// 16 bytes of elements, at any element alignment.
template <class E>
struct Vec {
  static constexpr int W = 16 / sizeof(E);
  typedef E type __attribute__((ext_vector_type(W)));
  struct __attribute__((packed, aligned(sizeof(E)))) Any { type v; };
};

__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_down(v, o, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return sh[0] + sh[1] + sh[2] + sh[3];
}

template <class E>
__device__ __forceinline__ double sum_squares(const Entry& e, long long lo, long long hi) {
  constexpr int W = Vec<E>::W, U = 4;
  const E* __restrict__ g = (const E*)e.g;
  double a[W];
#pragma unroll
  for (int k = 0; k < W; ++k) a[k] = 0.0;
  if (e.cols) {                          // rows apart: an element at a time
    for (long long i = lo + threadIdx.x; i < hi; i += 256) {
      const long long r = i / e.cols;
      const double x = (double)to_f32(g[r * e.ldg + (i - r * e.cols)]);
      a[0] = __builtin_fma(x, x, a[0]);
    }
    return a[0];
  }
  constexpr int S = 256 * W;             // elements of one load of the workgroup
  long long i = lo + threadIdx.x * W;
  auto add = [&](const typename Vec<E>::type& v) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const double x = (double)to_f32((E)v[k]);
      a[k] = __builtin_fma(x, x, a[k]);
    }
  };
  for (; i + (U - 1) * S + W <= hi; i += U * S) {
    typename Vec<E>::type v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = ((const typename Vec<E>::Any*)(g + i + u * S))->v;
#pragma unroll
    for (int u = 0; u < U; ++u) add(v[u]);
  }
  for (; i < hi; i += S) {
    if (i + W <= hi) {
      add(((const typename Vec<E>::Any*)(g + i))->v);
    } else {
      for (long long j = i; j < hi; ++j) {
        const double x = (double)to_f32(g[j]);
        a[0] = __builtin_fma(x, x, a[0]);
      }
    }
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < W; ++k) s += a[k];
  return s;
}

__global__ __launch_bounds__(256) void k_grad_squares(Table t, double* __restrict__ part) {
  __shared__ double sh[4];
  long long lo, hi;
  const Entry& e = my_entry(t, blockIdx.x, lo, hi);
  double s;
  if (e.dtype == DION3_F32) s = sum_squares<float>(e, lo, hi);
  else if (e.dtype == DION3_BF16) s = sum_squares<bf16>(e, lo, hi);
  else s = sum_squares<f16>(e, lo, hi);
  s = block_sum(s, sh);
  if (threadIdx.x == 0) part[t.part0 + blockIdx.x] = s;
}

// The sum of part[0 .. n), the same bits in every thread.
__device__ __forceinline__ double total_of(const double* __restrict__ part, int n, double* sh) {
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += 256) s += part[i];
  return block_sum(s, sh);
}
__device__ __forceinline__ double norm_of(double total, float scale) {
  return sqrt(total) * (double)scale;
}

// Many partial sums to one.
__global__ __launch_bounds__(256) void k_grad_total(double* __restrict__ part, int n) {
  __shared__ double sh[4];
  const double v = total_of(part, n, sh);
  if (threadIdx.x == 0) part[n] = v;
}

// Norms of single tensors (blocks: the tensors of the table) or of all of them.
struct Ranges {
  int begin[513];
};
__global__ __launch_bounds__(256) void k_grad_norm(Ranges r, const double* __restrict__ part,
                                                   float scale, float* __restrict__ out) {
  __shared__ double sh[4];
  const int b = r.begin[blockIdx.x], e = r.begin[blockIdx.x + 1];
  const double v = norm_of(total_of(part + b, e - b, sh), scale);
  if (threadIdx.x == 0) out[blockIdx.x] = (float)v;
}

template <class E, bool ONCE>
__device__ __forceinline__ void scale_chunk(const Entry& e, long long lo, long long hi, double c) {
  constexpr int W = Vec<E>::W, U = 4;
  E* __restrict__ g = (E*)e.g;
  float* __restrict__ m = e.m;
  if (e.cols) {
    for (long long i = lo + threadIdx.x; i < hi; i += 256) {
      const long long r = i / e.cols, at = r * e.ldg + (i - r * e.cols);
      if (m) {
        float& d = m[r * e.ldm + (i - r * e.cols)];
        d = (float)__builtin_fma((double)to_f32(g[at]), c, (double)d);
      } else {
        g[at] = (E)(float)((double)to_f32(g[at]) * c);
      }
    }
    return;
  }
  // W sums.  ONCE: they pass the cache (the gradients as well: 279 us become 287
  // at 134 M elements, 689 become 685 at 303 M: not kept).
  typedef float f4 __attribute__((ext_vector_type(4)));
  struct __attribute__((packed, aligned(4))) Any4 { f4 v; };
  struct Sums { f4 q[W / 4]; };
  auto load = [&](long long at) {
    Sums r;
#pragma unroll
    for (int k = 0; k < W / 4; ++k)
      r.q[k] = ONCE ? load_once<f4>(m + at + 4 * k) : ((const Any4*)(m + at + 4 * k))->v;
    return r;
  };
  constexpr int S = 256 * W;
  long long i = lo + threadIdx.x * W;
  auto one = [&](const typename Vec<E>::type& v, long long at, Sums s) {
    if (m) {
#pragma unroll
      for (int k = 0; k < W; ++k) {
        float& x = ((float*)&s)[k];
        x = (float)__builtin_fma((double)to_f32((E)v[k]), c, (double)x);
      }
#pragma unroll
      for (int k = 0; k < W / 4; ++k) {
        if (ONCE) store_once(m + at + 4 * k, s.q[k]);
        else ((Any4*)(m + at + 4 * k))->v = s.q[k];
      }
    } else {
      typename Vec<E>::type o;
#pragma unroll
      for (int k = 0; k < W; ++k) o[k] = (E)(float)((double)to_f32((E)v[k]) * c);
      ((typename Vec<E>::Any*)(g + at))->v = o;
    }
  };
  for (; i + (U - 1) * S + W <= hi; i += U * S) {
    typename Vec<E>::type v[U];
    Sums s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = ((const typename Vec<E>::Any*)(g + i + u * S))->v;
    if (m) {
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = load(i + u * S);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) one(v[u], i + u * S, s[u]);
  }
  for (; i < hi; i += S) {
    if (i + W <= hi) {
      Sums s;
      if (m) s = load(i);
      one(((const typename Vec<E>::Any*)(g + i))->v, i, s);
    } else {
      for (long long j = i; j < hi; ++j) {
        const double x = (double)to_f32(g[j]);
        if (m) m[j] = (float)__builtin_fma(x, c, (double)m[j]);
        else g[j] = (E)(float)(x * c);
      }
    }
  }
}

template <bool ONCE>
__global__ __launch_bounds__(256) void k_grad_clip(Table t, const double* __restrict__ part,
                                                   int parts, float max_norm, float scale,
                                                   float* __restrict__ norm) {
  __shared__ double sh[4];
  const double v = norm_of(total_of(part, parts, sh), scale);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  // (a norm that is NaN makes c NaN, an infinite one 0)
  const double c = (v <= (double)max_norm ? 1.0 : (double)max_norm / v) * (double)scale;
  long long lo, hi;
  // (from the end: what the first pass read last is still in the cache; 2 % of
  // the call at 303 M elements)
  const Entry& e = my_entry(t, gridDim.x - 1 - blockIdx.x, lo, hi);
  if (c == 1.0 && !e.m) return;          // g <- 1 g
  if (e.dtype == DION3_F32) scale_chunk<float, ONCE>(e, lo, hi, c);
  else if (e.dtype == DION3_BF16) scale_chunk<bf16, ONCE>(e, lo, hi, c);
  else scale_chunk<f16, ONCE>(e, lo, hi, c);
}

long long elements(const dion3_grad& d) { return (long long)d.rows * d.cols; }

bool dense(const dion3_grad& d) {
  return d.rows == 1 || (d.ldg == d.cols && (!d.M || d.ldm == d.cols));
}

// Elements of a chunk: about kPartials chunks up to kChunkMax, more beyond, and
// no more than 2^21 (2^38 elements).
long long chunk_size(const dion3_grad* d, int count) {
  long long total = 0;
  for (int i = 0; i < count; ++i) total += elements(d[i]);
  const long long c = (total / kPartials + 2047) / 2048 * 2048;
  if (c < kChunkMin) return kChunkMin;
  if (c < kChunkMax) return c;
  const long long least = (total >> 21) / 2048 * 2048;
  return least > kChunkMax ? least : kChunkMax;
}
int chunks_of(const dion3_grad& d, long long chunk) {
  return (int)((elements(d) + chunk - 1) / chunk);
}

// Whether the sums pass the 256 MB cache: sums of 512 MB from bf16 take 279 us
// past it and 307 through it (381 and 397 with a pass over the sums), of 256 MB
// 142 and 149, but of 128 MB 73 and 63, of 64 MB 39 and 36.
bool sums_once(const dion3_grad* d, int count) {
  double b = 0.0;
  for (int i = 0; i < count; ++i)
    if (d[i].M) b += (double)elements(d[i]) * (d[i].dtype == DION3_F32 ? 8.0 : 6.0);
  return b > 288e6;
}

// Calls launch(table, chunks of the batch, first) for every batch.
template <class F>
hipError_t for_batches(const dion3_grad* d, int count, long long chunk, F launch) {
  Table t;
  t.chunk = chunk;
  int part = 0;
  bool first = true;
  for (int i = 0; i < count;) {
    t.count = 0;
    t.part0 = part;
    int chunks = 0;
    for (; i < count && t.count < kBatch; ++i) {
      const int k = chunks_of(d[i], chunk);
      if (k == 0) continue;
      t.e[t.count++] = {d[i].G, d[i].M, elements(d[i]), dense(d[i]) ? 0 : (long long)d[i].cols,
                        d[i].ldg, d[i].ldm, chunks, d[i].dtype};
      chunks += k;
    }
    if (chunks == 0) continue;
    for (int j = t.count; j < kBatch; ++j) t.e[j] = t.e[0];
    const hipError_t e = launch(t, chunks, first);
    if (e != hipSuccess) return e;
    first = false;
    part += chunks;
  }
  return hipSuccess;
}

double grad_bytes(const dion3_grad* d, int count, double sums) {
  double b = 0.0;
  for (int i = 0; i < count; ++i)
    b += (double)elements(d[i]) * (d[i].M && sums > 0 ? sums : 0.0) +
         (double)elements(d[i]) * (d[i].dtype == DION3_F32 ? 4.0 : 2.0);
  return b;
}

hipError_t launch_squares(const dion3_grad* d, int count, long long chunk, double* part,
                          hipStream_t s) {
  TraceScope ts("grad_squares", 0.0, grad_bytes(d, count, 0.0), s);
  return for_batches(d, count, chunk, [&](const Table& t, int chunks, bool) {
    hipLaunchKernelGGL(k_grad_squares, dim3(chunks), dim3(256), 0, s, t, part);
    return hipGetLastError();
  });
}

int partials(const dion3_grad* d, int count, long long chunk) {
  int p = 0;
  for (int i = 0; i < count; ++i) p += chunks_of(d[i], chunk);
  return p;
}

// The partial sums, and their total where there are many.
size_t scratch_of(int parts) { return ((size_t)parts + (parts > kPartials ? 1 : 0)) * 8; }

constexpr int kMaxGrads = 1 << 20;

dion3_status check_grads(const dion3_grad* d, int count, bool sums) {
  if (count < 0 || (count > 0 && !d)) return DION3_ERR_ARG;
  if (count > kMaxGrads) return DION3_ERR_UNSUPPORTED;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    if (d[i].rows < 0 || d[i].cols < 0) return DION3_ERR_ARG;
    if (!type16(d[i].dtype) && d[i].dtype != DION3_F32) return DION3_ERR_ARG;
    constexpr long long most = 1LL << 38;
    if (d[i].rows > most || d[i].cols > most) return DION3_ERR_UNSUPPORTED;
    if (d[i].rows == 0 || d[i].cols == 0) continue;
    if (d[i].rows > most / d[i].cols) return DION3_ERR_UNSUPPORTED;
    total += elements(d[i]);
    if (total > most) return DION3_ERR_UNSUPPORTED;
    if (d[i].rows > 1) {
      if (d[i].ldg < d[i].cols || d[i].ldg > most) return DION3_ERR_ARG;
      if (sums && d[i].M && (d[i].ldm < d[i].cols || d[i].ldm > most)) return DION3_ERR_ARG;
    }
    if (!d[i].G || !elem_aligned(d[i].G, d[i].dtype == DION3_F32 ? 4 : 2)) return DION3_ERR_ARG;
    if (sums && !elem_aligned(d[i].M, 4)) return DION3_ERR_ARG;
  }
  return DION3_OK;
}

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

size_t dion3_grad_size(void) { return sizeof(dion3_grad); }

dion3_status dion3_grad_norm_workspace_size(const dion3_grad* grads, int32_t count, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  TRY(check_grads(grads, count, true));
  *bytes = scratch_of(partials(grads, count, chunk_size(grads, count)));
  return DION3_OK;
}

dion3_status dion3_grad_norm(const dion3_grad* grads, int32_t count, float scale, float* norm,
                             float* norms, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_grads(grads, count, false));
  if (!(scale > 0.0f) || !isfinite(scale)) return DION3_ERR_ARG;
  if (!norm || !elem_aligned(norm, 4) || !elem_aligned(norms, 4)) return DION3_ERR_ARG;
  const long long chunk = chunk_size(grads, count);
  const int parts = partials(grads, count, chunk);
  TRY(check_scratch(ws, ws_bytes, scratch_of(parts)));
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)ws;
  HIP_TRY(launch_squares(grads, count, chunk, part, s));
  Ranges r;
  r.begin[0] = 0;
  r.begin[1] = parts;
  TraceScope ts("grad_norm", 0.0, 8.0 * parts, s);
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, r, part, scale, norm);
  HIP_TRY(hipGetLastError());
  if (norms) {
    for (int i = 0, at = 0; i < count;) {
      const int first = i;
      r.begin[0] = at;
      for (; i < count && i - first < 512; ++i) {
        at += chunks_of(grads[i], chunk);
        r.begin[i - first + 1] = at;
      }
      hipLaunchKernelGGL(k_grad_norm, dim3(i - first), dim3(256), 0, s, r, part, scale,
                         norms + first);
      HIP_TRY(hipGetLastError());
    }
  }
  return DION3_OK;
}

dion3_status dion3_clip_grad_norm(const dion3_grad* grads, int32_t count, float max_norm,
                                  float scale, float* norm, void* ws, size_t ws_bytes,
                                  void* stream) {
  TRY(check_grads(grads, count, true));
  if (!(scale > 0.0f) || !isfinite(scale) || !(max_norm >= 0.0f)) return DION3_ERR_ARG;
  if (!elem_aligned(norm, 4)) return DION3_ERR_ARG;
  const long long chunk = chunk_size(grads, count);
  const int parts = partials(grads, count, chunk);
  TRY(check_scratch(ws, ws_bytes, scratch_of(parts)));
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)ws;
  if (parts == 0) {                      // no elements at all
    if (!norm) return DION3_OK;
    Ranges r;
    r.begin[0] = r.begin[1] = 0;
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, r, part, scale, norm);
    HIP_TRY(hipGetLastError());
    return DION3_OK;
  }
  HIP_TRY(launch_squares(grads, count, chunk, part, s));
  int terms = parts;
  if (parts > kPartials) {
    hipLaunchKernelGGL(k_grad_total, dim3(1), dim3(256), 0, s, part, parts);
    HIP_TRY(hipGetLastError());
    part += parts;
    terms = 1;
  }
  const bool once = sums_once(grads, count);
  TraceScope ts("grad_clip", 0.0, grad_bytes(grads, count, 8.0), s);
  HIP_TRY(for_batches(grads, count, chunk, [&](const Table& t, int chunks, bool first) {
    float* out = first ? norm : nullptr;
    if (once) hipLaunchKernelGGL(k_grad_clip<true>, dim3(chunks), dim3(256), 0, s, t, part, terms, max_norm, scale, out);
    else hipLaunchKernelGGL(k_grad_clip<false>, dim3(chunks), dim3(256), 0, s, t, part, terms, max_norm, scale, out);
    return hipGetLastError();
  }));
  return DION3_OK;
}

}  // extern "C"
