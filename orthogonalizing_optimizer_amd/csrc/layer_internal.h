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

template <class E>
struct Vec8 {
  typedef E type __attribute__((ext_vector_type(8)));
};

// True when rows of E starting at p with stride ld elements allow 16-byte
// accesses at every chunk.
template <class E>
__host__ __device__ inline bool rows_aligned(const E* p, long long ld) {
  return ((uintptr_t)p & 15) == 0 && (ld * (long long)sizeof(E)) % 16 == 0;
}

// Columns c .. c + 7 of a row of m elements as floats (zero past m).
template <class E>
__device__ __forceinline__ void load8(const E* __restrict__ row, int c, int m, bool vec,
                                      float (&v)[8]) {
  if (vec && c + 8 <= m) {
    if constexpr (sizeof(E) == 4) {
      const float4 a = ((const float4*)(row + c))[0], b = ((const float4*)(row + c))[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const typename Vec8<E>::type x = *(const typename Vec8<E>::type*)(row + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = to_f32((E)x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < m ? to_f32(row[c + e]) : 0.0f;
  }
}

template <class E>
__device__ __forceinline__ void store8(E* __restrict__ row, int c, int m, bool vec,
                                       const float (&v)[8]) {
  if (vec && c + 8 <= m) {
    if constexpr (sizeof(E) == 4) {
      ((float4*)(row + c))[0] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)(row + c))[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      typename Vec8<E>::type x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (E)v[e];
      *(typename Vec8<E>::type*)(row + c) = x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < m) row[c + e] = (E)v[e];
  }
}

// -------------------------------------------------------------- activations

// 1 / (1 + exp(-x)) by the hardware's exponential and reciprocal (each within
// one step of fp32): a divide rounded to the last bit costs ten instructions
// more for every output element, and the outputs are 16-bit.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// act(z).  gelu_tanh: 0.5 (1 + tanh u) = sigmoid(2 u), which keeps its
// relative accuracy for large negative u.  gelu: 0.5 (1 + erf x) = 0.5 erfc(-x)
// for the same reason.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case DION3_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case DION3_ACT_GELU: return 0.5f * z * erfcf(-z * kSqrtHalf);
    case DION3_ACT_GELU_TANH:
      return z * sigmoid(2.0f * kGeluC * __builtin_fmaf(kGeluA * z * z, z, z));
    case DION3_ACT_SILU: return z * sigmoid(z);
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
    case DION3_ACT_GELU:
      return __builtin_fmaf(z * kInvSqrt2Pi, __expf(-0.5f * z * z), 0.5f * erfcf(-z * kSqrtHalf));
    case DION3_ACT_GELU_TANH: {
      const float s = sigmoid(2.0f * kGeluC * __builtin_fmaf(kGeluA * z * z, z, z));
      const float du = kGeluC * __builtin_fmaf(3.0f * kGeluA * z, z, 1.0f);
      return __builtin_fmaf(2.0f * z * du, s * (1.0f - s), s);
    }
    case DION3_ACT_SILU: {
      const float s = sigmoid(z);
      return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
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

// The largest magnitude q may take: 448, except in a block whose scale is the
// type's last, where 448 rounds to past the type's largest finite value and
// the largest q is 240 (bf16, fp32: 240 * 2^120; fp16: 240 * 2^8 = 61440).
template <class E>
__device__ __forceinline__ float f8_limit(int byte) {
  return byte == (sizeof(E) == 2 && __is_same(E, f16) ? 127 + 8 : 127 + 120) ? 240.0f : 448.0f;
}

// |v| where v is finite, else 0 (infinities and NaN do not take part in the
// scale; their q is NaN).
__device__ __forceinline__ float finite_abs(float v) {
  const float a = __builtin_fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// 8 scaled values as 8 bytes of e4m3 (round to nearest even).
__device__ __forceinline__ uint2 f8_encode8(const float (&v)[8], float inv, float lim) {
  unsigned w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = fminf(fmaxf(v[4 * h + e] * inv, -lim), lim);
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], p, true);
    w[h] = (unsigned)p;
  }
  // (fminf / fmaxf drop a NaN, and an infinity would take the limit)
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (!(__builtin_fabsf(v[e]) <= 3.402823466e38f)) w[e >> 2] |= 0x7fu << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

// The largest finite magnitude of the 32-column block that 4 neighbouring
// lanes hold 8 columns each of; every lane of the wave takes part.
__device__ __forceinline__ float f8_block_amax(const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaxf(a, finite_abs(v[e]));
  a = fmaxf(a, __shfl_xor(a, 1, 64));
  return fmaxf(a, __shfl_xor(a, 2, 64));
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
