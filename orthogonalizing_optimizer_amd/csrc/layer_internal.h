// Internal interfaces of the layer operators (norm, linear products, 8-bit
// checkpoints) between the C-ABI layer and their gfx950 kernels.
#pragma once

#include "dion3_internal.h"

namespace dion3 {

typedef __bf16 bf16;

// Columns that share one scale of the 8-bit format, and the chunk of columns
// that one thread moves with a 16-byte access of a 16-bit type.
constexpr int kF8Block = DION3_F8_BLOCK;
constexpr int kChunk = 8;

inline long long f8_cols(long long m) { return pad_to(m, kF8Block); }

// ------------------------------------------------------------ element types

__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(f16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Chunks of 8 columns of a row of m elements.  16-byte accesses need no more
// than the element's own alignment here (gfx950 splits unaligned ones), so any
// row stride and any base take the same path.
//
// fetch8 asks for columns c .. c + 7 without a branch, at the row's end for
// its last 8 columns, and chunk8 turns them into floats (zero past m); kept
// apart, because turning the first tensor's chunk into floats would wait for
// it before the next tensor's is asked for.  (fp32 rows, read once a
// workgroup, take their last columns one by one.)
template <class E>
struct Raw8 {
  typedef E type __attribute__((ext_vector_type(8)));
  struct __attribute__((packed, aligned(sizeof(E)))) Any { type v; };
  type v;
};

template <class E>
__device__ __forceinline__ Raw8<E> fetch8(const E* __restrict__ row, int c, int m) {
  Raw8<E> r;
  if (sizeof(E) == 2 ? m >= 8 : c + 8 <= m) {
    r.v = ((const typename Raw8<E>::Any*)(row + min(c, m - 8)))->v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = c + e < m ? row[c + e] : (E)0.0f;
  }
  return r;
}

template <class E>
__device__ __forceinline__ void chunk8(const Raw8<E>& r, int c, int m, float (&v)[8]) {
  // columns of r before c: 0 inside the row
  const int s = sizeof(E) == 2 && m >= 8 ? c - min(c, m - 8) : 0;
  if (s == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32((E)r.v[e]);
  } else if constexpr (sizeof(E) == 2) {
    typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
    u64x2 w = __builtin_bit_cast(u64x2, r.v);
    const int b = 16 * (s & 3);
    const unsigned long long lo = s & 4 ? w[1] : w[0], hi = s & 4 ? 0 : w[1];
    w[0] = lo >> b | (b ? hi << (64 - b) : 0);
    w[1] = hi >> b;
    const typename Raw8<E>::type t = __builtin_bit_cast(typename Raw8<E>::type, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s < 8 ? to_f32((E)t[e]) : 0.0f;
  }
}

template <class E>
__device__ __forceinline__ void load8(const E* __restrict__ row, int c, int m, float (&v)[8]) {
  chunk8(fetch8(row, c, m), c, m, v);
}

template <class E>
__device__ __forceinline__ void store8(E* __restrict__ row, int c, int m, const float (&v)[8]) {
  if (c + 8 <= m) {
    Raw8<E> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = (E)v[e];
    ((typename Raw8<E>::Any*)(row + c))->v = r.v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < m) row[c + e] = (E)v[e];
  }
}

// 16 bytes, or 8 elements, at any element alignment, past the 256 MB cache: for
// what is not read again before as much has passed, or is too long to stay.
template <class E, int N>
struct Once {
  typedef E type __attribute__((ext_vector_type(N), aligned(sizeof(E))));
};
template <class V, class E, int N = sizeof(V) / sizeof(E)>
__device__ __forceinline__ V load_once(const E* p) {
  return __builtin_nontemporal_load((const typename Once<E, N>::type*)p);
}
template <class E, class V, int N = sizeof(V) / sizeof(E)>
__device__ __forceinline__ void store_once(E* p, V v) {
  __builtin_nontemporal_store(v, (typename Once<E, N>::type*)p);
}
template <class E>
__device__ __forceinline__ Raw8<E> fetch8_once(const E* row, int c, int m) {
  if (c + 8 > m) return fetch8(row, c, m);
  Raw8<E> r;
  r.v = load_once<typename Raw8<E>::type>(row + c);
  return r;
}
template <class E>
__device__ __forceinline__ void store8_once(E* row, int c, int m, const float (&v)[8]) {
  if (c + 8 > m) return store8(row, c, m, v);
  Raw8<E> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r.v[e] = (E)v[e];
  store_once(row + c, r.v);
}

// -------------------------------------------------------------- activations
//
// An element of an activation costs as much VALU time as it does HBM time
// (without packed fp32 the chip does about 39 T operations a second, 7 for
// each byte moved at 5.8 TB/s), so the forms below are counted in
// instructions: the hardware's exponential and reciprocal (each within one
// step of fp32, for 16-bit outputs), constants folded into the exponent.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + 2^-u)
__device__ __forceinline__ float sigmoid2(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u));
}

// gelu_tanh: 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v)), which keeps its relative
// accuracy for large negative v = sqrt(2 / pi) (z + 0.044715 z^3).
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  constexpr float k = 2.0f * kGeluC * kLog2e;
  return sigmoid2(z * __builtin_fmaf(k * kGeluA, z * z, k));
}

// The normal distribution function and e = exp(-z^2 / 2): with x = |z| / sqrt 2
// and t = 1 / (1 + 0.3 x), erfc(x) exp(x^2) = t Q(t), Q of degree 8 fitted to
// the smallest largest relative error over 0 <= x <= 12 (2e-8; 5e-7 as
// evaluated in fp32).  The lower tail keeps its relative accuracy.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(
      __builtin_fmaf(0.3f * 0.7071067811865476f, __builtin_fabsf(z), 1.0f));
  float q = -0.129252436f;
  q = __builtin_fmaf(q, t, 0.484298187f);
  q = __builtin_fmaf(q, t, -0.509765608f);
  q = __builtin_fmaf(q, t, 0.544959805f);
  q = __builtin_fmaf(q, t, -0.0928215102f);
  q = __builtin_fmaf(q, t, 0.214179651f);
  q = __builtin_fmaf(q, t, 0.148521671f);
  q = __builtin_fmaf(q, t, 0.170690875f);
  q = __builtin_fmaf(q, t, 0.169189357f);
  e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
  const float tail = 0.5f * t * q * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

// act(z)
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case DION3_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case DION3_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case DION3_ACT_GELU_TANH: return z * gelu_tanh_gate(z);
    case DION3_ACT_SILU: return z * sigmoid2(z * kLog2e);
  }
  return z;
}

// act(z) of 8 values, the choice made once for all of them.
__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
#define DION3_ACT8(A)                                    \
  case A: {                                              \
    _Pragma("unroll") for (int e = 0; e < 8; ++e) v[e] = activate(A, v[e]); \
    return;                                              \
  }
  switch (act) {
    DION3_ACT8(DION3_ACT_RELU)
    DION3_ACT8(DION3_ACT_GELU)
    DION3_ACT8(DION3_ACT_GELU_TANH)
    DION3_ACT8(DION3_ACT_SILU)
  }
#undef DION3_ACT8
}

// act'(z)
__device__ __forceinline__ float slope(int act, float z) {
  switch (act) {
    case DION3_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case DION3_ACT_GELU: {
      float e;
      const float c = normal_cdf(z, e);
      return __builtin_fmaf(z * kInvSqrt2Pi, e, c);
    }
    case DION3_ACT_GELU_TANH: {
      // s + z s (1 - s) u'(z).  From |z| = 32 on s is 0 or 1, and so is the
      // slope; z^2 ends there, since the cubic's overflow times 0 would be NaN
      const float s = gelu_tanh_gate(z);
      const float q = z * __builtin_fmaf(-s, s, s);
      return __builtin_fmaf(
          q, __builtin_fmaf(6.0f * kGeluC * kGeluA, fminf(z * z, 1024.0f), 2.0f * kGeluC), s);
    }
    case DION3_ACT_SILU: {
      const float s = sigmoid2(z * kLog2e);
      return __builtin_fmaf(z, __builtin_fmaf(-s, s, s), s);
    }
  }
  return 1.0f;
}

// --------------------------------------------------------- the 8-bit format

// e4m3 values q (4 exponent bits, 3 mantissa bits, largest 448, no infinity)
// with one scale 2^e for 32 columns of a row, held as the byte e + 127.
// e = the smallest exponent with amax <= 448 * 2^e, so nothing saturates: from
// the bits of amax = 1.f * 2^x, e = x - 8 when 1.f <= 1.75, else x - 7.
// A block of zeros takes the byte 0.
__device__ __forceinline__ int f8_scale_byte(float amax) {
  const unsigned u = __builtin_bit_cast(unsigned, amax);
  const int x = (int)(u >> 23);                        // biased exponent (0: subnormal or zero)
  const int e = x - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
  return e < 0 ? 0 : e;
}

// 2^(127 - byte), the factor that maps the block into e4m3's range; a normal
// float for every byte a block can take (0 .. 247).
__device__ __forceinline__ float f8_inv_scale(int byte) {
  return __builtin_bit_cast(float, (unsigned)(254 - byte) << 23);
}

// The value of lane ^ 1 (X = 1) or lane ^ 2 (X = 2), inside groups of 4 lanes.
template <int X>
__device__ __forceinline__ unsigned quad_xor(unsigned v) {
  return __builtin_amdgcn_update_dpp(0, v, X == 1 ? 0xB1 : 0x4E, 0xF, 0xF, true);
}
__device__ __forceinline__ unsigned quad_max(unsigned v) {
  v = max(v, quad_xor<1>(v));
  return max(v, quad_xor<2>(v));
}

// A block of 32 columns, 8 in each of 4 neighbouring lanes (all of them take
// part): its scale byte, and this lane's 8 values as e4m3, round to nearest
// even.  Magnitudes are compared as the bits of |v|, whose order is that of
// the floats.  Finite blocks below the type's last scale (nearly all) need one
// multiplication and half a conversion a value; the others take the branch.
constexpr unsigned kInfBits = 0x7f800000u;
template <class E>
__device__ __forceinline__ uint2 f8_encode_block(const float (&v)[8], int& byte) {
  unsigned a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, __builtin_bit_cast(unsigned, v[e]) & 0x7fffffffu);
  a = quad_max(a);
  byte = f8_scale_byte(__builtin_bit_cast(float, a));
  constexpr int last = __is_same(E, f16) ? 127 + 8 : 127 + 120;
  float u[8];
  if (a < kInfBits && byte != last) {
    const float inv = f8_inv_scale(byte);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = v[e] * inv;
  } else {
    // infinities and NaN take no part in the scale and become NaN
    a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned b = __builtin_bit_cast(unsigned, v[e]) & 0x7fffffffu;
      a = max(a, b < kInfBits ? b : 0u);
    }
    a = quad_max(a);
    byte = f8_scale_byte(__builtin_bit_cast(float, a));
    // 448 of the type's last scale would be past its largest finite value
    const float inv = f8_inv_scale(byte), lim = byte == last ? 240.0f : 448.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned b = __builtin_bit_cast(unsigned, v[e]) & 0x7fffffffu;
      const float c = fminf(fmaxf(v[e] * inv, -lim), lim);
      u[e] = b < kInfBits ? c : __builtin_nanf("");
    }
  }
  int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], w0, true);
  int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], 0, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], w1, true);
  return make_uint2((unsigned)w0, (unsigned)w1);
}

// 2 of the 4 e4m3 bytes of `w` times 2^(byte - 127), the scale given as the
// float whose exponent field is the byte (byte 0 stands for 2^-127).
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float f8_scale_float(unsigned byte) {
  return __builtin_bit_cast(float, byte << 23);
}
template <bool HI>
__device__ __forceinline__ bf16x2 f8_decode2(bf16, unsigned w, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI);
}
template <bool HI>
__device__ __forceinline__ f16x2 f8_decode2(f16, unsigned w, float s) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, HI));
}
template <bool HI>
__device__ __forceinline__ f32x2 f8_decode2(float, unsigned w, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, HI);
}

// ------------------------------------------------------------------ launches

// One workgroup of 256 threads for each 256 of n items numbered through.  A
// side of a grid holds fewer than 2^32 threads (HIP's limit), so workgroups
// past 2^23 go to further rows of the grid.
inline dim3 flat_grid(long long n) {
  const long long groups = (n + 255) / 256, row = 1LL << 23;
  return groups <= row ? dim3((unsigned)groups)
                       : dim3((unsigned)row, (unsigned)((groups + row - 1) / row));
}
__device__ __forceinline__ long long flat_base() {       // the workgroup's first item
  return ((long long)blockIdx.y * gridDim.x + blockIdx.x) * 256;
}

// A scratch layout: partial column sums, one row of m floats per unit.
struct RowsPlan {
  int units;            // partial rows
  int rows_per_unit;    // (act_grad) consecutive rows of one unit
};

struct NormArgs {
  const void* x; long long ldx;
  const void* r; long long ldr;        // null: h = x and h is not written
  const void* w; int wtype;            // DION3_F32 or the rows' type
  void* h; long long ldh;
  void* y; long long ldy;              // null: not written
  unsigned char* q; unsigned char* s;  // null: not written
  float* rstd;                         // null: not written
  long long T; int m;
  float eps;
  int dtype;
};
hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void* dy; long long lddy;
  const void* h; long long ldh;
  const float* rstd;
  const void* w; int wtype;
  const void* dh; long long lddh;      // null: none
  void* dx; long long lddx;            // null: not written
  float* dw;                           // null: not written
  long long T; int m;
  int dtype;
};
size_t norm_grad_scratch(long long T, long long m);
hipError_t launch_add_rms_norm_grad(const NormGradArgs& a, void* ws, hipStream_t s);

hipError_t launch_pack_f8(const void* x, long long ldx, unsigned char* q, unsigned char* sc,
                          long long T, int m, int dtype, hipStream_t s);
hipError_t launch_unpack_f8(const unsigned char* q, const unsigned char* sc, void* y, long long ldy,
                            long long T, int m, int dtype, hipStream_t s);

struct ActGradArgs {
  const void* dy; long long lddy;
  const void* z; long long ldz;                           // null: packed z, or act none
  const unsigned char* zq; const unsigned char* zs;
  void* dz; long long lddz;                               // null: not written
  float* db;                                              // null: not written
  long long T; int n;
  int act, dtype;
};
size_t act_grad_scratch(long long T, long long n);
hipError_t launch_act_grad(const ActGradArgs& a, void* ws, hipStream_t s);

// out[j] = sum over units u of part[u][j], in order.
hipError_t launch_join_columns(const float* part, int units, int m, float* out, hipStream_t s);

// One product C = A B^T with A: M x K and B: N x K.
// a_km / b_kn: the operand is given with its K index as rows, [K][M] / [K][N].
struct LinDesc {
  const void* A; long long lda; bool a_km;
  const void* B; long long ldb; bool b_kn;
  const unsigned char* bs;       // b_kn only: B is e4m3 with these scales (pitch ldb / 32)
  long long M, N, K;
  int dtype;
  // outputs: either the 16-bit rows Y = act(C + bias) + R (and Z = C + bias),
  // or the fp32 rows G (+)= C
  void* Y; long long ldy;
  void* Z; long long ldz;
  const void* R; long long ldr;
  const void* bias; int bias_type;
  int act;
  float* G; long long ldg; bool accumulate;
  const char* name;              // of the timing trace
};
size_t lin_scratch(const LinDesc& d);
hipError_t launch_lin(const LinDesc& d, void* ws, hipStream_t s);

}  // namespace dion3
