// The products of a linear layer for gfx950: Y = act(X W^T + b) + R, its
// input gradient dX = dZ W (+ R) and its weight gradient G (+)= dZ^T X with X
// in 16 bits or in the 8-bit checkpoint format.  bf16 or fp16 operands on
// the matrix cores (v_mfma_f32_32x32x16), fp32 accumulation, one rounding at
// the end.
//
// One kernel computes C = A B^T by tiles, K 64 at a time through two LDS
// buffers, for every layout the three products need.  An operand is staged
// in one of three ways:
//   * K-contiguous rows (X and W of the forward product, dZ of the input
//     gradient): rows of 64 + 8 halves in LDS, fragments by 16-byte reads;
//   * K as rows (W of the input gradient, dZ and X of the weight gradient):
//     64 rows of R + 32 halves, fragments by transposing reads
//     (ds_read_b64_tr_b16), so that no transposed copy is ever made;
//   * K as rows in 8 bits: the same, decoded between the global load and the
//     LDS store, two values an instruction (the scale is the instruction's
//     operand), so the checkpoint crosses HBM and the caches at half the size.
// Operands whose rows are not 16-byte aligned, or end inside a chunk, take the
// ragged form of the first two (see Operand).
// Tiles: 256 x 256, 192 x 256 and 128 x 256 (8 waves, one workgroup a CU; the
// first has the best rate, 1.2-1.25 PFLOP/s on 8192 x 4096 x 4096, the others
// fill the last round of workgroups better), 128 x 128 and 64 x 64 (4 waves,
// for few tokens).  Each slice of 16 K issues the next slice's LDS reads ahead
// of its MFMAs; the next tile's LDS stores and the global loads of a later one
// are spread over the step's first slices.  The time of a step is shared by
// MFMA issue (2048 cycles of the large tile) and LDS traffic (192 KB read,
// 64 KB written), at a clock that power limits.
// Few tiles are split over K: each part leaves an fp32 tile in the scratch,
// which k_lin_join adds up in order and finishes.
// The epilogue passes the fp32 accumulators through LDS so that bias,
// residual, outputs and the accumulated G move as 16-byte pieces of rows.
#include <math.h>

#include "layer_internal.h"

namespace dion3 {
namespace {

constexpr int BK = 64;
constexpr int LDSK = BK + 8;      // halves per K-contiguous LDS row
constexpr int kPadN = 32;         // halves of padding of a [K][R] LDS row

typedef short short4v __attribute__((ext_vector_type(4)));
typedef short short8 __attribute__((ext_vector_type(8)));
typedef f16 half8 __attribute__((ext_vector_type(8)));
typedef bf16 bfloat8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;

__device__ __forceinline__ floatx16 mfma32(f16, short8 a, short8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mfma32(bf16, short8 a, short8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bfloat8, a),
                                                 __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma16(f16, short8 a, short8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma16(bf16, short8 a, short8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfloat8, a),
                                                 __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}

// Raw buffer over `bytes` bytes: loads past them return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, bytes, 0x00020000);
}
constexpr int kOut = (int)0x80000000;    // an offset past every buffer

// What becomes of C.
struct Finish {
  void* Y; void* Z; const void* R; const void* bias;
  float* G;
  long long ldy, ldz, ldr, ldg;
  int bias_f32, act, accumulate;
  int N;
};

// The epilogue of columns c .. c + 7: the bias is read once a thread, what a
// row adds (the residual, or the G it is summed into) ahead of the row's turn.
template <class E, bool F32>
struct Chunk {
  float b[8];
  __device__ __forceinline__ void init(const Finish& f, int c) {
    if constexpr (!F32) {
      if (!f.bias) return;
      if (f.bias_f32) load8((const float*)f.bias, c, f.N, b);
      else load8((const E*)f.bias, c, f.N, b);
    }
  }
  static __device__ __forceinline__ void addend(const Finish& f, long long r, int c, float (&o)[8]) {
    if constexpr (F32) load8((const float*)f.G + r * f.ldg, c, f.N, o);
    else load8((const E*)f.R + r * f.ldr, c, f.N, o);
  }
  template <bool ADD>
  __device__ __forceinline__ void put(const Finish& f, long long r, int c, float (&v)[8],
                                      const float (&o)[8]) const {
    if constexpr (F32) {
      if constexpr (ADD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += o[e];
      }
      store8(f.G + r * f.ldg, c, f.N, v);
    } else {
      if (f.bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += b[e];
      }
      if (f.Z) store8((E*)f.Z + r * f.ldz, c, f.N, v);
      if (f.act != DION3_ACT_NONE) activate8(f.act, v);
      if constexpr (ADD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += o[e];
      }
      store8((E*)f.Y + r * f.ldy, c, f.N, v);
    }
  }
};

template <class E, bool F32>
__device__ __forceinline__ void finish8(const Finish& f, long long r, int c, float (&v)[8]) {
  Chunk<E, F32> k;
  float o[8];
  k.init(f, c);
  if (F32 ? f.accumulate != 0 : f.R != nullptr) {
    k.addend(f, r, c, o);
    k.template put<true>(f, r, c, v, o);
  } else {
    k.template put<false>(f, r, c, v, o);
  }
}

struct LinP {
  const void* A; const void* B; const unsigned char* bs;
  long long lda, ldb;
  long long M, K;
  int N;
  int tilesM, tilesN, splits, steps;   // steps: K steps of one split
  long long total;                     // workgroups
  float* part; long long part_stride;  // splits > 1: fp32 [split][M][ldp]
  int ldp;
  Finish f;
};

template <int I>
struct Int { static constexpr int value = I; };

template <int BM_, int BN_, int WAVES_M, int WAVES_N, int SPREAD_, int PF_>
struct Cfg {
  static constexpr int PF = PF_;           // K steps of register prefetch
  static constexpr int SPREAD = SPREAD_;   // slices of a K step that share the staging
  static constexpr int BM = BM_, BN = BN_;
  static constexpr int NT = 64 * WAVES_M * WAVES_N;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int part(int r) { return r * LDSK > BK * (r + kPadN) ? r * LDSK : BK * (r + kPadN); }
  static constexpr int PART = part(BM), STAGE = PART + part(BN);      // halves
  // epilogue staging: rows of BN + 8 floats; the 4 rows between a wave's two
  // halves then lie 32 banks apart
  static constexpr int EP = BN + 8;
  static constexpr int EROWS = BN > 128 ? WTM : BM;          // rows staged at a time
  static constexpr int EBYTES = EROWS * EP * 4;
  static constexpr int BYTES = 2 * STAGE * 2 > EBYTES ? 2 * STAGE * 2 : EBYTES;
  static constexpr int PER_CU = BYTES > 81920 ? 1 : BYTES > 54608 ? 2 : 3;   // workgroups of a CU
};
typedef Cfg<256, 256, 2, 4, 3, 1> CfgL;
typedef Cfg<192, 256, 2, 4, 3, 2> CfgM;
typedef Cfg<128, 256, 2, 4, 3, 1> CfgW;
typedef Cfg<128, 128, 2, 2, 1, 1> CfgS;
typedef Cfg<64, 64, 2, 2, 1, 2> CfgT;

template <bool B, class X, class Y>
struct Pick { typedef X type; };
template <class X, class Y>
struct Pick<false, X, Y> { typedef Y type; };

// 16 bytes at any alignment of 16-bit elements, and the 8 elements moved down
// by s places with zeros behind (s from 8 on: zeros).
struct __attribute__((packed, aligned(2))) Any16 { int4v v; };
__device__ __forceinline__ int4v moved(int4v v, int s) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64x2 w = __builtin_bit_cast(u64x2, v);
  const int b = 16 * (s & 3);
  const unsigned long long hi = s & 4 ? 0 : w[1], lo = s & 4 ? w[1] : w[0];
  w[0] = lo >> b | (hi << 1) << (63 - b);
  w[1] = hi >> b;
  const int4v r = __builtin_bit_cast(int4v, w);
  return s < 8 ? r : int4v{0, 0, 0, 0};
}

enum Kind { kRowsK = 0, kColsK = 1, kColsF8 = 2 };

// One operand of R output rows: its registers, LDS part and fragments.
//
// RAG: rows of any alignment and length (at least 8).  Chunks come by unaligned
// 16-byte loads, whose rows and columns are held inside the operand instead of
// relying on a buffer's bounds: the last chunk of a row is the row's last 8
// elements, moved into place before the LDS store, and what lies past K is
// zeroed there.  Against aligned products of nearly the same sizes it takes a
// fifth to three fifths longer (bf16; forward, input gradient, weight
// gradient): 8192 x 4095 x 4097 270, 273 and 288 us, 8192 x 4096 x 4096 219,
// 225 and 220; 1000 x 2049 x 2047 27.0, 27.7 and 26.4, 1000 x 2048 x 2048
// 19.9, 22.5 and 16.6; 517 x 1000 x 515 7.0, 10.7 and 7.9, 520 x 1000 x 520
// 5.1, 6.8 and 5.5.  Against a copy of the operand and its launch (another
// card, ragged and copied first): forward 517 x 1000 x 515 7.3 us against
// 11.8, 1000 x 2049 x 2047 29.3 against 36.5, 8192 x 4095 x 4097 250 against
// 289; input gradient 10.7 against 10.6, 30 against 37.5, 268 against 311;
// weight gradient 8.0 against 8.4, 27.8 against 37.5, 283 against 378.
template <class E, int R, int NT, int KIND, int PF, bool RAG>
struct Operand {
  static constexpr int RS = R + kPadN;                                 // [K][R] LDS row
  static constexpr int CH = KIND == kColsF8 ? R * BK / 16 / NT : R * BK / 8 / NT;
  static constexpr int CPR = KIND == kRowsK ? BK / 8 : KIND == kColsK ? R / 8 : R / 16;  // chunks a row
  static constexpr int OPS = KIND == kColsF8 ? 2 : 1;                  // loads (and stores) a chunk
  static constexpr int READS = KIND == kRowsK ? 1 : 2;                 // LDS reads a fragment
  const char* base;      // kRowsK: the tile's first row; else column r0 of row 0
  const unsigned char* sbase;
  long long ld;          // bytes
  long long K;
  int bytes;             // kRowsK: of the tile's rows
  int cols;              // else: bytes of a row that may be read
  int scols;
  static constexpr bool FIXED = NT % CPR == 0;    // a thread's chunks share their column
  int voff[FIXED ? 1 : CH];
  static constexpr bool RAGGED = RAG && KIND != kColsF8;
  long long Kt;          // RAGGED: the operand's own K (K: where this part of it ends)
  int roff[RAGGED ? CH : 1];   // kRowsK: the chunks' rows; kColsK: the first chunk's
  int cut;               // kColsK: elements of the chunk before its column
  bool edge;             // kColsK: the columns end inside the tile
  int4v reg[PF][CH];
  unsigned sreg[PF][KIND == kColsF8 ? CH : 1];

  __device__ __forceinline__ void init(const void* p, const unsigned char* sc, long long ldp,
                                       long long rows, long long k, long long kt, long long r0,
                                       int tid) {
    K = k;
    if constexpr (RAGGED) {
      static_assert(NT % CPR == 0, "a thread's chunks share their column");
      Kt = kt;
      ld = ldp * 2;
      if constexpr (KIND == kRowsK) {
        base = (const char*)p + r0 * ld;
        const int last = (int)(rows - r0 < R ? rows - r0 : R) - 1;
#pragma unroll
        for (int i = 0; i < CH; ++i) roff[i] = min((tid + NT * i) / CPR, last) * (int)ld;
      } else {
        // (a part of the output may have fewer than 8 columns left: its last 8
        // then begin before it, in the same row)
        const long long from = r0 < rows - 8 ? r0 : rows - 8;
        const long long c = r0 + tid % CPR * 8, at = c < rows - 8 ? c : rows - 8;
        base = (const char*)p + from * 2;
        cut = (int)(c - at);
        edge = r0 + R > rows;
        voff[0] = (int)(at - from) * 2;
        roff[0] = tid / CPR * (int)ld;
      }
      return;
    }
    if constexpr (KIND == kRowsK) {
      K = (k + 7) & ~7LL;        // rows end in whole chunks (zeros past K: see in_place)
      ld = ldp * 2;
      base = (const char*)p + r0 * ld;
      const int n = (int)(rows - r0 < R ? rows - r0 : R);
      bytes = (int)((n - 1) * ld + K * 2);
    } else if constexpr (KIND == kColsK) {
      ld = ldp * 2;
      base = (const char*)p + r0 * 2;
      cols = (int)(rows - r0 < R ? (rows - r0 + 7) & ~7LL : R) * 2;
    } else {
      ld = ldp;
      base = (const char*)p + r0;
      sbase = sc + r0 / kF8Block;
      cols = (int)(rows - r0 < R ? (rows - r0 + kF8Block - 1) / kF8Block * kF8Block : R);
      scols = cols / kF8Block;
    }
#pragma unroll
    for (int i = 0; i < (FIXED ? 1 : CH); ++i)
      voff[i] = (int)(((tid + NT * i) / CPR) * ld) + (tid + NT * i) % CPR * 16;
  }

  // Buffers over the tile's K rows / columns k0 .. k0 + 63 (loads past K give
  // zero), and the offset of this thread's first chunk in them.
  struct Src {
    __amdgpu_buffer_rsrc_t rs, ss;
    int v;
  };
  struct RagSrc {
    const char* p;       // kColsK: row min(k0, Kt - 1)
    int v;               // kRowsK: the chunk's column; kColsK: the last row that may be read
  };
  typedef typename Pick<RAGGED, RagSrc, Src>::type Source;
  __device__ __forceinline__ Source source(long long k0, int tid) const {
    if constexpr (RAGGED) {
      if constexpr (KIND == kRowsK) {
        const long long k = k0 + (tid & 7) * 8;
        return {base, (int)(k < Kt - 8 ? k : Kt - 8) * 2};
      } else {
        const long long row = k0 < Kt - 1 ? k0 : Kt - 1;
        return {base + row * ld, (int)(Kt - 1 - row < BK ? Kt - 1 - row : BK) * (int)ld};
      }
    } else if constexpr (KIND == kRowsK) {
      const __amdgpu_buffer_rsrc_t rs = rsrc(base, bytes);
      return {rs, rs, k0 + (tid & 7) * 8 < K ? voff[0] + (int)k0 * 2 : kOut};
    } else {
      const long long left = K - k0;
      const int n = left <= 0 ? 0 : left < BK ? (int)left : BK;        // valid rows
      const __amdgpu_buffer_rsrc_t rs = rsrc(base + k0 * ld, n > 0 ? (int)((n - 1) * ld) + cols : 0);
      if constexpr (KIND == kColsF8) {
        const int lds = (int)(ld / kF8Block);
        return {rs, rsrc(sbase + k0 * lds, n > 0 ? (n - 1) * lds + scols : 0), voff[0]};
      }
      return {rs, rs, voff[0]};
    }
  }

  // Chunk i of the tile into this thread's register set P.
  template <int P>
  __device__ __forceinline__ void load(const Source& s, int i, int tid) {
    constexpr int STEP = NT / CPR;
    if constexpr (RAGGED) {
      const unsigned o = KIND == kRowsK ? (unsigned)(roff[i] + s.v)
                                        : (unsigned)(min(roff[0] + i * STEP * (int)ld, s.v) + voff[0]);
      reg[P][i] = ((const Any16*)(s.p + o))->v;
      return;
    } else {
    static_assert(FIXED || KIND == kColsK, "other operands' chunks share their column");
    const int v = FIXED ? s.v + i * STEP * (int)ld : voff[FIXED ? 0 : i];
    reg[P][i] = __builtin_amdgcn_raw_buffer_load_b128(s.rs, v, 0, 0);
    if constexpr (KIND == kColsF8)
      sreg[P][i] = (unsigned char)__builtin_amdgcn_raw_buffer_load_b8(
          s.ss, (tid / CPR + i * STEP) * (int)(ld / kF8Block) + (tid % CPR) / 2, 0, 0);
    }
  }
  template <int P>
  __device__ __forceinline__ void load_all(long long k0, int tid) {
    const Source s = source(k0, tid);
#pragma unroll
    for (int i = 0; i < CH; ++i) load<P>(s, i, tid);
  }

  // RAGGED: chunk i of the tile at k0 moved into place, and zeroed past K.
  template <int P>
  __device__ __forceinline__ int4v placed(int i, long long k0, int tid) const {
    const long long k = k0 + (KIND == kRowsK ? (tid & 7) * 8 : (tid + NT * i) / CPR);
    const int by = KIND == kRowsK ? (int)(k < Kt - 8 ? 0 : k - (Kt - 8)) : cut;
    return moved(reg[P][i], k < K ? by : 8);
  }
  // All of them ahead of a step that reaches past an end (the choice is the
  // workgroup's), so that the other steps pay nothing: 8192 x 4095 x 4097
  // forward 250 us, 261 with every chunk placed as it is stored; input gradient
  // 268 against 293.  The short steps of the small tile (PF 2) would wait for
  // their loads there, and place late: 517 x 1000 x 515 input gradient 10.7 us
  // against 12.8, weight gradient 8.1 against 11.0.
  static constexpr bool LATE = RAGGED && PF > 1;
  template <int P>
  __device__ __forceinline__ void place(long long k0, int tid) {
    if constexpr (RAGGED && !LATE) {
      if (k0 + BK <= K && (KIND == kRowsK || !edge)) return;
#pragma unroll
      for (int i = 0; i < CH; ++i) reg[P][i] = placed<P>(i, k0, tid);
    }
  }

  // Chunk i of the tile at k0 from the registers into the LDS part s.
  template <int P>
  __device__ __forceinline__ void store(short* __restrict__ s, int i, int tid, long long k0) const {
    const int c = tid + NT * i;
    if constexpr (KIND == kRowsK) {
      int4v v = reg[P][i];
      if constexpr (LATE) v = placed<P>(i, k0, tid);
      *(int4v*)(s + (c / CPR) * LDSK + (c % CPR) * 8) = v;
    } else if constexpr (KIND == kColsK) {
      int4v v = reg[P][i];
      if constexpr (LATE) v = placed<P>(i, k0, tid);
      *(int4v*)(s + (c / CPR) * RS + (c % CPR) * 8) = v;
    } else {
      const float sc = f8_scale_float(sreg[P][i]);
      short* d = s + (c / CPR) * RS + (c % CPR) * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int4v o;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const unsigned u = (unsigned)reg[P][i][2 * h + w];
          o[2 * w] = __builtin_bit_cast(int, f8_decode2<false>(E(), u, sc));
          o[2 * w + 1] = __builtin_bit_cast(int, f8_decode2<true>(E(), u, sc));
        }
        *(int4v*)(d + 8 * h) = o;
      }
    }
  }
  template <int P>
  __device__ __forceinline__ void store_all(short* __restrict__ s, int tid, long long k0) const {
#pragma unroll
    for (int i = 0; i < CH; ++i) store<P>(s, i, tid, k0);
  }

  // This lane's offset into the part for the wave's rows w0 .., and the
  // fragment (8 consecutive K of row lane % 32, from K = 8 (lane / 32)) of
  // block i and slice kk.  Transposing reads: in each group of 16 lanes, lane
  // 4 e + u points at row e, columns 4 u .. 4 u + 3 of a 4 x 16 block and
  // receives that block's column lane % 16.
  static __device__ __forceinline__ int frag_off(int w0, int lane) {
    if constexpr (KIND == kRowsK) return (w0 + (lane & 31)) * LDSK + (lane >> 5) * 8;
    return ((lane >> 5) * 8 + ((lane & 15) >> 2)) * RS + w0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
  }
  static __device__ __forceinline__ short8 frag(const short* p, int i, int kk) {
    if constexpr (KIND == kRowsK) return *(const short8*)(p + i * 32 * LDSK + kk * 16);
    const short* q = p + i * 32 + kk * 16 * RS;
    const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)q);
    const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(q + 4 * RS));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// Scheduling-group masks of __builtin_amdgcn_sched_group_barrier.
constexpr int kSgMfma = 0x008, kSgVmemRead = 0x020, kSgDsRead = 0x100, kSgDsWrite = 0x200;

// The order of a slice: its NM MFMAs, each followed by its share of the NR LDS
// reads, NS LDS stores and NL global loads.
template <int NM, int NR, int NS, int NL, int Q>
__device__ __forceinline__ void slice_order() {
  if constexpr (Q < NM) {
    constexpr int r = ((Q + 1) * NR + NM - 1) / NM - (Q * NR + NM - 1) / NM;
    constexpr int w = ((Q + 1) * NS + NM - 1) / NM - (Q * NS + NM - 1) / NM;
    constexpr int l = ((Q + 1) * NL + NM - 1) / NM - (Q * NL + NM - 1) / NM;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(kSgDsRead, r, 0);
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    if constexpr (w > 0) __builtin_amdgcn_sched_group_barrier(kSgDsWrite, w, 0);
    if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(kSgVmemRead, l, 0);
    slice_order<NM, NR, NS, NL, Q + 1>();
  }
}

// One K step on LDS stage `st`: register set P (the next tile) goes into stage
// `nxt`, and the tile PF steps later is requested into it.  Each slice reads
// the next slice's fragments under its own MFMAs; the step's one barrier sits
// before the last slice, and the next stage's first fragments are read under
// that slice's MFMAs.  Every step does all of it, the last ones with tiles
// past the end, which load as zeros and are not used.
template <class E, class C, int KA, int KB, bool RAG, int P>
__device__ __forceinline__ void k_step(const short* __restrict__ st, short* __restrict__ nxt,
                                       Operand<E, C::BM, C::NT, KA, C::PF, RAG>& A,
                                       Operand<E, C::BN, C::NT, KB, C::PF, RAG>& B, long long k_next,
                                       int tid, int aoff, int boff, short8 (&fa0)[C::FM],
                                       short8 (&fb0)[C::FN], floatx16 (&acc)[C::FM][C::FN]) {
  typedef Operand<E, C::BM, C::NT, KA, C::PF, RAG> OA;
  typedef Operand<E, C::BN, C::NT, KB, C::PF, RAG> OB;
  constexpr int NS = BK / 16, NM = C::FM * C::FN;
  constexpr int NR = OA::READS * C::FM + OB::READS * C::FN;
  constexpr int SPREAD = C::SPREAD;                      // slices that share the staging
  constexpr int CHT = OA::CH + OB::CH;
  short8 af[2][C::FM], bf[2][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i) af[0][i] = fa0[i];
#pragma unroll
  for (int j = 0; j < C::FN; ++j) bf[0][j] = fb0[j];
  const typename OA::Source sa = A.source(k_next, tid);
  const typename OB::Source sb = B.source(k_next, tid);
  const long long ks = k_next - C::PF * BK;              // the tile that is stored
  A.template place<P>(ks, tid);
  B.template place<P>(ks, tid);
  auto slice = [&](auto KK) {
    constexpr int kk = KK.value;
    constexpr int cb = kk & 1;
    constexpr int c0 = kk < SPREAD ? kk * CHT / SPREAD : CHT, c1 = kk < SPREAD ? (kk + 1) * CHT / SPREAD : CHT;
    constexpr int na = (c1 < OA::CH ? c1 : OA::CH) - (c0 < OA::CH ? c0 : OA::CH), nb = c1 - c0 - na;
    constexpr int ops = na * OA::OPS + nb * OB::OPS;
    if constexpr (kk + 1 < NS) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) af[cb ^ 1][i] = OA::frag(st + aoff, i, kk + 1);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) bf[cb ^ 1][j] = OB::frag(st + C::PART + boff, j, kk + 1);
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C::FM; ++i) fa0[i] = OA::frag(nxt + aoff, i, 0);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) fb0[j] = OB::frag(nxt + C::PART + boff, j, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = c0; c < c1; ++c) {
      if (c < OA::CH) {
        A.template store<P>(nxt, c, tid, ks);
        A.template load<P>(sa, c, tid);
      } else {
        B.template store<P>(nxt + C::PART, c - OA::CH, tid, ks);
        B.template load<P>(sb, c - OA::CH, tid);
      }
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = mfma32(E(), af[cb][i], bf[cb][j], acc[i][j]);
    if constexpr (kk + 1 == NS) {
      // (the reads are already ahead of the MFMAs)
    } else if constexpr (kk == 0 && SPREAD == 1) {
      __builtin_amdgcn_sched_group_barrier(kSgDsRead, NR, 0);
      slice_order<NM, 0, ops, ops, 0>();
    } else {
      slice_order<NM, NR, ops, ops, 0>();
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  slice(Int<0>());
  slice(Int<1>());
  slice(Int<2>());
  slice(Int<3>());
}

// PF K steps from step kt (a multiple of PF) on, the register sets in turn.
template <class E, class C, int KA, int KB, bool RAG, int U>
__device__ __forceinline__ void k_steps(short* lds, Operand<E, C::BM, C::NT, KA, C::PF, RAG>& A,
                                        Operand<E, C::BN, C::NT, KB, C::PF, RAG>& B, long long k0, int kt,
                                        int tid, int aoff, int boff, short8 (&fa0)[C::FM],
                                        short8 (&fb0)[C::FN], floatx16 (&acc)[C::FM][C::FN]) {
  if constexpr (U < C::PF) {
    const int t = kt + U;
    k_step<E, C, KA, KB, RAG, (U + 1) % C::PF>(lds + (t & 1) * C::STAGE, lds + ((t + 1) & 1) * C::STAGE, A,
                                          B, k0 + (long long)(t + 1 + C::PF) * BK, tid, aoff, boff, fa0,
                                          fb0, acc);
    k_steps<E, C, KA, KB, RAG, U + 1>(lds, A, B, k0, kt, tid, aoff, boff, fa0, fb0, acc);
  }
}

template <class E, class C, class OA, class OB, int P>
__device__ __forceinline__ void load_ahead(OA& A, OB& B, long long k0, int tid) {
  if constexpr (P < C::PF) {
    A.template load_all<P>(k0 + P * BK, tid);
    B.template load_all<P>(k0 + P * BK, tid);
    __builtin_amdgcn_sched_barrier(0);      // (in tile order, as the loop's waits count them)
    load_ahead<E, C, OA, OB, P + 1>(A, B, k0, tid);
  }
}

// One tile of the output.  8192 x 4096 x 4096 (two rounds of 256 x 256 tiles):
// 215-231 us forward, 222-248 input gradient, 217-241 weight gradient (card to
// card), of which about 1.5 us a K step and 10 us a round for first loads and
// epilogue.  F32: C goes to G; PART: to the scratch (splits); else to Y.
template <class E, class C, int KA, int KB, bool F32, bool PART, bool RAG>
__global__ __launch_bounds__(C::NT, C::PER_CU) void k_lin(LinP p) {
  __shared__ __attribute__((aligned(16))) char lds_raw[C::BYTES];
  short* lds = (short*)lds_raw;

  // Workgroups go round-robin over the 8 XCDs; renumbered so that each XCD
  // takes a contiguous run of tiles.  Within a split: groups of 8 tile rows,
  // columns first, so that consecutive tiles share panels in that XCD's L2.
  const int total = (int)p.total;
  const int w = blockIdx.x, q = total >> 3, rem = total & 7, xcd = w & 7;
  const int lid = xcd * q + min(xcd, rem) + (w >> 3);
  const int tiles = p.tilesM * p.tilesN;
  const int split = PART ? lid / tiles : 0;
  const int t = lid - split * tiles;
  constexpr int GR = 8;
  const int g0 = (t / (GR * p.tilesN)) * GR;
  const int gsz = min(p.tilesM - g0, GR);
  const int r = t - g0 * p.tilesN;
  const int bi = g0 + r % gsz, bj = r / gsz;
  const long long m0 = (long long)bi * C::BM;
  const int n0 = bj * C::BN;

  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / (C::BN / C::WTN), wn = wid % (C::BN / C::WTN);

  floatx16 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  {
    const long long k0 = (long long)split * p.steps * BK;
    long long k1 = k0 + (long long)p.steps * BK;
    if (k1 > p.K) k1 = p.K;
    const int nk = (int)((k1 - k0 + BK - 1) / BK);          // >= 1
    typedef Operand<E, C::BM, C::NT, KA, C::PF, RAG> OA;
    typedef Operand<E, C::BN, C::NT, KB, C::PF, RAG> OB;
    OA A;
    OB B;
    A.init(p.A, nullptr, p.lda, p.M, k1, p.K, m0, tid);       // (nothing past this part's K is read)
    B.init(p.B, p.bs, p.ldb, p.N, k1, p.K, n0, tid);
    const int aoff = OA::frag_off(wm * C::WTM, lane), boff = OB::frag_off(wn * C::WTN, lane);
    // tile j passes through register set j % PF
    load_ahead<E, C, OA, OB, 0>(A, B, k0, tid);
    A.template place<0>(k0, tid);
    B.template place<0>(k0, tid);
    A.template store_all<0>(lds, tid, k0);
    B.template store_all<0>(lds + C::PART, tid, k0);
    A.template load_all<0>(k0 + C::PF * BK, tid);
    B.template load_all<0>(k0 + C::PF * BK, tid);
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    short8 fa0[C::FM], fb0[C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i) fa0[i] = OA::frag(lds + aoff, i, 0);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) fb0[j] = OB::frag(lds + C::PART + boff, j, 0);
    // whole rounds of the register sets: steps past the end multiply zeros
    for (int kt = 0; kt < nk; kt += C::PF)
      k_steps<E, C, KA, KB, RAG, 0>(lds, A, B, k0, kt, tid, aoff, boff, fa0, fb0, acc);
    // (the last step's barrier also frees the LDS for the epilogue)
  }

  // Accumulators of a 32 x 32 block: lane l, value v holds row 8 (v / 4) +
  // 4 (l / 32) + v % 4, column l % 32.
  float* S = (float*)lds_raw;
  constexpr int CPR = C::BN / 8, RPP = C::NT / CPR;      // chunks a row, rows a pass
  static_assert(C::EROWS % (RPP * 2) == 0, "whole batches");
  const int c = (tid % CPR) * 8;
  const bool in = n0 + c < p.N;
  Chunk<E, F32> ch;
  if (!PART && in) ch.init(p.f, n0 + c);
#pragma unroll
  for (int h = 0; h < C::BM / C::EROWS; ++h) {
    if (h > 0) __syncthreads();
    if (C::EROWS == C::BM || wm == h) {
      const int rb = C::EROWS == C::BM ? wm * C::WTM : 0;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            S[(rb + i * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) * C::EP + wn * C::WTN + j * 32 +
              (lane & 31)] = acc[i][j][v];
    }
    __syncthreads();
    if (!in) continue;
    const long long r0 = m0 + h * C::EROWS + tid / CPR;
    const float* s0 = S + tid / CPR * C::EP + c;
    // (the choices are the whole launch's, so each is made once a tile)
    auto rows = [&](auto FULL, auto ADD) {
      // rows in flight (4 with an activation's code spill registers)
      constexpr int U = (F32 || PART) && C::EROWS % (RPP * 4) == 0 ? 4 : 2;
      for (int b = 0; b < C::EROWS / RPP; b += U) {
        float v[U][8], o[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (ADD.value && (FULL.value || r0 + (b + u) * RPP < p.M))
            Chunk<E, F32>::addend(p.f, r0 + (b + u) * RPP, n0 + c, o[u]);
          const float* s = s0 + (b + u) * RPP * C::EP;
          const float4 x = *(const float4*)s, y = *(const float4*)(s + 4);
          v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          v[u][4] = y.x; v[u][5] = y.y; v[u][6] = y.z; v[u][7] = y.w;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long row = r0 + (b + u) * RPP;
          if (!FULL.value && row >= p.M) continue;
          if constexpr (PART)
            store8(p.part + split * p.part_stride + row * p.ldp, n0 + c, p.ldp, v[u]);
          else
            ch.template put<ADD.value>(p.f, row, n0 + c, v[u], o[u]);
        }
      }
    };
    const bool add = !PART && (F32 ? p.f.accumulate != 0 : p.f.R != nullptr);
    if (m0 + (h + 1) * C::EROWS <= p.M) {
      if (add) rows(Int<1>(), Int<1>());
      else rows(Int<1>(), Int<0>());
    } else {
      if (add) rows(Int<0>(), Int<1>());
      else rows(Int<0>(), Int<0>());
    }
  }
}

// The splits' tiles added up, then the epilogue.  A workgroup takes 256 / GR
// chunks of 8 columns (the scratch's rows numbered through), GR threads a
// chunk, each the sum of a run of the splits in order; the runs join in order.
// GR = 8 where one thread a chunk would leave most of the chip idle (64 parts of
// 128 x 512: 3.8 us, 6.4 with one thread a chunk); bound by reading the parts,
// mostly from the caches (2 parts of 1000 x 2048: 5.3 us).
template <class E, bool F32, int GR>
__global__ __launch_bounds__(256) void k_lin_join(const float* __restrict__ part, long long stride,
                                                  int splits, long long M, unsigned nch, Finish f) {
  constexpr int CW = 256 / GR;
  __shared__ float sh[GR > 1 ? GR - 1 : 1][CW][8 + 1];
  const int ci = threadIdx.x % CW, g = threadIdx.x / CW;
  const long long base = (long long)blockIdx.x * CW;
  const bool in = base + ci < M * nch;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (in) {
    const float* s = part + (base + ci) * 8;
    const int per = (splits + GR - 1) / GR;
    const int i1 = min(splits, (g + 1) * per);
#pragma unroll 4
    for (int i = g * per; i < i1; ++i) {
      const float4 a = *(const float4*)(s + i * stride), b = *(const float4*)(s + i * stride + 4);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
  }
  if constexpr (GR > 1) {
    if (g > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sh[g - 1][ci][e] = v[e];
    }
    __syncthreads();
    if (g > 0) return;
    for (int q = 0; q < GR - 1; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sh[q][ci][e];
  }
  if (!in) return;
  const long long row0 = base / nch;
  const unsigned c0 = (unsigned)(base - row0 * nch) + ci;
  const unsigned dr = c0 / nch;
  finish8<E, F32>(f, row0 + dr, (int)(c0 - dr * nch) * 8, v);
}

template <class E, bool F32>
hipError_t launch_join(const float* part, long long stride, int splits, long long M, unsigned nch,
                       const Finish& f, hipStream_t s) {
  const long long chunks = M * nch;
  if (splits >= 4 && chunks <= 65536)
    hipLaunchKernelGGL((k_lin_join<E, F32, 8>), dim3((unsigned)((chunks + 31) / 32)), dim3(256), 0, s,
                       part, stride, splits, M, nch, f);
  else
    hipLaunchKernelGGL((k_lin_join<E, F32, 1>), dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s,
                       part, stride, splits, M, nch, f);
  return hipGetLastError();
}

// No K at all (a gradient over no tokens): C = 0.
template <class E, bool F32>
__global__ __launch_bounds__(256) void k_lin_zero(long long M, unsigned nch, Finish f) {
  const long long e = flat_base() + threadIdx.x;
  if (e >= M * nch) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  finish8<E, F32>(f, e / nch, (int)(e % nch) * 8, v);
}

// An operand that the aligned kernels cannot read in place (rows not 16-byte
// aligned, or a contiguous side that is no multiple of 8) copied into rows of
// a whole number of chunks, zeros at their ends, where the ragged form is
// modelled to take longer or has no 8 elements in a row to read.  The copy
// moves the operand twice more (1000 x 515: 3.6 us, most of it the launch).
__global__ __launch_bounds__(256) void k_lin_copy(const unsigned short* __restrict__ src,
                                                  long long ld, long long rows, int cols,
                                                  unsigned nch, unsigned short* __restrict__ dst) {
  const long long base = flat_base();
  if (base + threadIdx.x >= rows * nch) return;
  const long long row0 = base / nch;
  const unsigned c0 = (unsigned)(base - row0 * nch) + threadIdx.x;
  const unsigned dr = c0 / nch;
  const int c = (int)(c0 - dr * nch) * 8;
  const unsigned short* s = src + (row0 + dr) * ld;
  unsigned short v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? s[c + e] : 0;
  int4v o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (int)(v[2 * e] | (unsigned)v[2 * e + 1] << 16);
  *(int4v*)(dst + (base + threadIdx.x) * 8) = o;
}

// ------------------------------------------------------------- few tokens

// Y for 2 to 16 tokens (see few_tokens): bound by reading W once.  A workgroup takes 16
// rows of W, its 8 waves the K axis in turns of 128; a lane reads 64
// contiguous bytes of one W row (four chunks, one per MFMA: the order of K
// inside the product is free as long as both operands agree) and the same
// columns of its token.  The waves' 16 x 16 sums join in LDS in wave order.
// Both operands are readable in 16-byte chunks (in_place).
// 4096 x 4096: 11 us at 2 tokens, 13 at 16.
struct ThinP {
  const void* X; const void* W;
  long long ldx, ldw, N;
  int T, K;
  Finish f;
};

__device__ __forceinline__ short8 thin_chunk(__amdgpu_buffer_rsrc_t rs, int row_off, int k, int K) {
  const int4v v = __builtin_amdgcn_raw_buffer_load_b128(rs, k < K ? row_off + k * 2 : kOut, 0, 0);
  return __builtin_bit_cast(short8, v);
}

template <class E>
__global__ __launch_bounds__(512) void k_lin_thin(ThinP p) {
  constexpr int NW = 8, U = 2;
  __shared__ float sh[NW][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long n0 = (long long)blockIdx.x * 16;
  const int nrows = (int)(p.N - n0 < 16 ? p.N - n0 : 16);
  const __amdgpu_buffer_rsrc_t rw =
      rsrc((const E*)p.W + n0 * p.ldw, (int)((nrows - 1) * p.ldw + p.K) * 2);
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.X, (int)((p.T - 1) * p.ldx + p.K) * 2);
  const int r = lane & 15, g = lane >> 4;
  const int wo = r < nrows ? (int)(r * p.ldw) * 2 : 0, xo = r < p.T ? (int)(r * p.ldx) * 2 : 0;
  const int wK = r < nrows ? p.K : 0, xK = r < p.T ? p.K : 0;
  floatx4 acc = {0, 0, 0, 0};
  for (int k0 = wave * 128; k0 < p.K; k0 += NW * 128 * U) {
    short8 a[U][4], b[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + u * NW * 128 + g * 32 + i * 8;
        a[u][i] = thin_chunk(rw, wo, k, wK);
        b[u][i] = thin_chunk(rx, xo, k, xK);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = mfma16(E(), a[u][i], b[u][i], acc);
  }
  // lane l, value v: W row 4 (l / 16) + v, token l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) sh[wave][r][g * 4 + v] = acc[v];
  __syncthreads();
  // thread: token t, 8 of the 16 rows
  const int t = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
  if (t < p.T && n0 + c < p.N) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sh[w][t][c + e];
    finish8<E, false>(p.f, t, (int)n0 + c, v);
  }
}

// Y for one token, by vector instructions: a wave's load is 1 KB of one W row
// (the matrix form above reads 64 bytes of 16 rows a load: 24 us for 90 MB of
// cold weights at 11008 x 4096, this one 19; 40 and 27 us at 13824 x 5120), the
// token's 512 columns are read once for 4 rows.  A workgroup takes 8 rows, four
// waves to each 4 of them, which take turns along K; many small waves hide the
// loads better than two steps in flight each (27 and 31 us).  (The same for 4
// tokens keeps too many registers to fill the chip: 34 us at 11008 x 4096.)
template <class E>
__global__ __launch_bounds__(512) void k_lin_vec(ThinP p) {
  constexpr int R = 4, KW = 4;
  __shared__ float sh[KW][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rg = wave / KW, kh = wave % KW;
  const long long n0 = (long long)blockIdx.x * 8;
  const E* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {       // rows past the end repeat the last one, unused
    const long long row = n0 + rg * R + r;
    w[r] = (const E*)p.W + (row < p.N ? row : p.N - 1) * p.ldw;
  }
  float acc[R] = {0, 0, 0, 0};
  for (int k0 = kh * 512; k0 < p.K; k0 += KW * 512) {
    const int c = k0 + lane * 8;
    Raw8<E> rw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rw[r] = fetch8(w[r], c, p.K);
    const Raw8<E> rx = fetch8((const E*)p.X, c, p.K);
    float a[8];
    chunk8(rx, c, p.K, a);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float b[8];
      chunk8(rw[r], c, p.K, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[r] = __builtin_fmaf(a[e], b[e], acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) acc[r] += __shfl_xor(acc[r], o, 64);
    if (lane == 0) sh[kh][rg * R + r] = acc[r];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int q = 0; q < KW; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sh[q][e];
    finish8<E, false>(p.f, 0, (int)n0, v);
  }
}

// Rows of an operand as the aligned kernels read it: 16-byte chunks.
bool in_place(const void* p, long long ld, long long contiguous) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && contiguous % 8 == 0;
}

// The forms for few tokens: by vectors for one; the 16 x 16 matrix form while
// W is small (16 tokens: 4096 x 4096 13 us, 16 by the 64 x 64 tiles; 11008 x
// 4096 36 us, 27 by the tiles: there the tokens, read once by every workgroup,
// cost as much as W).
constexpr int kThinTokens = 16;
constexpr long long kThinWeights = 24LL << 20;
bool few_tokens(const LinDesc& d) {
  return !d.a_km && !d.b_kn && !d.G &&
         (d.M == 1 || (d.M <= kThinTokens && d.N * d.K <= kThinWeights &&
                       in_place(d.A, d.lda, d.K) && in_place(d.B, d.ldb, d.K)));
}

// ------------------------------------------------------------- host side

// A rectangle of the output by one tile shape, its K axis in `splits` parts of
// `steps` K steps.
struct LinPart {
  long long m0, n0, M, N;
  int tile, splits, steps;
};
struct LinPlan {
  bool thin;
  bool ragged;             // operands read unaligned
  bool copyA, copyB;       // or copied first
  long long rowsA, colsA, rowsB, colsB;     // as stored
  size_t oA, oB, oP, total;
  int nparts;
  LinPart part[2];
};

long long up8(long long x) { return pad_to(x, 8); }

// Tile shapes with their time model, microseconds: one K step of a workgroup
// on an idle chip (lo) and with a workgroup on every CU (hi), and the fixed
// part of a workgroup (first loads, epilogue).  Fitted to single launches at
// K = 64 .. 16384 from a few tiles to 1400.  The two small tiles run 2 or 3
// workgroups a CU at the same total rate, so a round is 256 of any shape.
struct Tile { int bm, bn; double lo, hi, fixed; };
constexpr int kNTiles = 5;
constexpr Tile kTiles[kNTiles] = {{256, 256, 1.05, 1.53, 11.0},
                                  {192, 256, 0.85, 1.22, 8.5},
                                  {128, 256, 0.65, 0.89, 6.5},
                                  {128, 128, 0.45, 0.53, 4.5},
                                  {64, 64, 0.20, 0.24, 3.0}};
constexpr int kCus = 256;
// A step of the ragged form against an aligned one, as the plan counts it
// (whole products differ by more, see Operand).  Three shapes have it: the
// large tile, 128 x 256 and 64 x 64, between which the model finds a time
// within 10 % of the best of the five on the shapes named at Operand.
constexpr double kRag = 1.15;
constexpr bool has_ragged(int tile) { return tile == 0 || tile == 2 || tile == 4; }

// The cheapest tile shape and split of one rectangle: rounds of workgroups
// over the 256 CUs, and for splits the join's launch and its traffic.
double choose_tile(LinPart& q, long long K, bool f8, bool rag) {
  static const int kSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32, 40, 48, 64};
  const long long nk = (K + BK - 1) / BK;
  double best = 1e30;
  for (int i = 0; i < kNTiles; ++i) {
    if (rag && !has_ragged(i)) continue;
    const Tile& t = kTiles[i];
    const long long tiles = ((q.M + t.bm - 1) / t.bm) * ((q.N + t.bn - 1) / t.bn);
    for (const int sp : kSplits) {
      if (sp > 1 && (sp > nk || tiles * sp > 4 * kCus)) break;
      const int steps = (int)((nk + sp - 1) / sp);
      const double load = (double)(tiles * sp) / kCus, rounds = ceil(load);
      // (on an idle chip the decoding of 8-bit operands is not hidden)
      const double lo = f8 ? t.lo + 0.15 : rag ? t.lo * kRag : t.lo;
      const double hi = rag ? t.hi * kRag : t.hi > lo ? t.hi : lo;
      const double step = lo + (hi - lo) * (load < 1.0 ? load : 1.0);
      double us = rounds * (steps * step + t.fixed);
      if (sp > 1) us += 4.0 + 8.0 * sp * (double)q.M * q.N / 5.0e6;
      if (us < best) {
        best = us;
        q.tile = i;
        q.splits = (int)((nk + steps - 1) / steps);      // (without parts that would be empty)
        q.steps = steps;
      }
    }
  }
  return best;
}

// More tiles than one round: the rows or columns of tiles that fill whole
// rounds, and what is left as a rectangle of its own with its own tile shape
// (8192 x 11008 outputs are 5.4 rounds of the large tile: 5 rounds and 768
// columns in one round of 128 x 256 tiles instead of 6).
double choose_parts(LinPlan& q, long long M, long long N, long long K, bool f8, bool rag) {
  LinPart whole = {0, 0, M, N, 0, 1, 0};
  double best = choose_tile(whole, K, f8, rag);
  q.nparts = 1;
  q.part[0] = whole;
  const int nk = (int)((K + BK - 1) / BK);
  for (int i = 0; i < kNTiles; ++i) {
    if (rag && !has_ragged(i)) continue;
    const Tile& t = kTiles[i];
    const long long tm = (M + t.bm - 1) / t.bm, tn = (N + t.bn - 1) / t.bn;
    const long long full = tm * tn / kCus;
    if (full < 1) continue;
    const double us = (double)full * (nk * t.hi * (rag ? kRag : 1.0) + t.fixed) + 8.0;
    for (int side = 0; side < 2; ++side) {
      const long long cut = full * kCus / (side ? tn : tm);               // tile rows / columns
      if (cut < 1 || cut >= (side ? tm : tn)) continue;
      const LinPart a = {0, 0, side ? cut * t.bm : M, side ? N : cut * t.bn, i, 1, nk};
      LinPart b = {side ? cut * t.bm : 0, side ? 0 : cut * t.bn, side ? M - cut * t.bm : M,
                   side ? N : N - cut * t.bn, 0, 1, 0};
      const double both = us + choose_tile(b, K, f8, rag);
      if (both < best) {
        best = both;
        q.nparts = 2;
        q.part[0] = a;
        q.part[1] = b;
      }
    }
  }
  return best;
}

LinPlan lin_plan(const LinDesc& d) {
  LinPlan q = {};
  if (d.M == 0 || d.K == 0) return q;
  q.rowsA = d.a_km ? d.K : d.M; q.colsA = d.a_km ? d.M : d.K;
  q.rowsB = d.b_kn ? d.K : d.N; q.colsB = d.b_kn ? d.N : d.K;
  q.thin = few_tokens(d);
  if (q.thin) return q;
  q.copyA = !in_place(d.A, d.lda, q.colsA);
  q.copyB = !d.bs && !in_place(d.B, d.ldb, q.colsB);
  double us = choose_parts(q, d.M, d.N, d.K, d.bs != nullptr, false);
  // unaligned operands: copied first (a launch and their bytes twice), or read
  // as they are by the ragged form (measured: see Operand)
  if (q.copyA || q.copyB) {
    if (q.copyA) us += 4.0 + 4.0 * (double)q.rowsA * q.colsA / 4.5e6;
    if (q.copyB) us += 4.0 + 4.0 * (double)q.rowsB * q.colsB / 4.5e6;
    if (q.colsA >= 8 && (d.bs || q.colsB >= 8)) {
      LinPlan r = q;
      if (choose_parts(r, d.M, d.N, d.K, d.bs != nullptr, true) < us) {
        q = r;
        q.ragged = true;
        q.copyA = q.copyB = false;
      }
    }
  }
  size_t off = 0;
  auto take = [&](size_t b) { const size_t o = off; off = (off + b + 255) & ~(size_t)255; return o; };
  if (q.copyA) q.oA = take((size_t)q.rowsA * up8(q.colsA) * 2);
  if (q.copyB) q.oB = take((size_t)q.rowsB * up8(q.colsB) * 2);
  size_t parts = 0;      // one after the other: they share the scratch of the splits
  for (int i = 0; i < q.nparts; ++i) {
    const LinPart& t = q.part[i];
    if (t.splits > 1) {
      const size_t b = (size_t)t.splits * t.M * up8(t.N) * 4;
      parts = b > parts ? b : parts;
    }
  }
  if (parts) q.oP = take(parts);
  q.total = off;
  return q;
}

template <class E, class C, int KA, int KB, bool F32, bool RAG>
hipError_t launch_tiles(const LinP& p, hipStream_t s) {
  const dim3 grid((unsigned)p.total), block(C::NT);
  if (p.splits > 1)
    hipLaunchKernelGGL((k_lin<E, C, KA, KB, F32, true, RAG>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((k_lin<E, C, KA, KB, F32, false, RAG>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <class E, int KA, int KB, bool F32>
hipError_t launch_cfg(LinP p, int tile, bool rag, hipStream_t s) {
  const Tile& t = kTiles[tile];
  p.tilesM = (int)((p.M + t.bm - 1) / t.bm);
  p.tilesN = (p.N + t.bn - 1) / t.bn;
  p.total = (long long)p.tilesM * p.tilesN * p.splits;
  // (fewer than 2^32 threads; no size within the library's limits gets here)
  if (p.total >= 1LL << 23) return hipErrorInvalidValue;
  if (rag) {
    switch (tile) {
      case 0: return launch_tiles<E, CfgL, KA, KB, F32, true>(p, s);
      case 2: return launch_tiles<E, CfgW, KA, KB, F32, true>(p, s);
      case 4: return launch_tiles<E, CfgT, KA, KB, F32, true>(p, s);
    }
    return hipErrorInvalidValue;
  }
  switch (tile) {
    case 0: return launch_tiles<E, CfgL, KA, KB, F32, false>(p, s);
    case 1: return launch_tiles<E, CfgM, KA, KB, F32, false>(p, s);
    case 2: return launch_tiles<E, CfgW, KA, KB, F32, false>(p, s);
    case 3: return launch_tiles<E, CfgS, KA, KB, F32, false>(p, s);
  }
  return launch_tiles<E, CfgT, KA, KB, F32, false>(p, s);
}

template <class E>
hipError_t launch_lin_t(const LinDesc& d, void* ws, hipStream_t s) {
  const LinPlan q = lin_plan(d);
  Finish f = {d.Y, d.Z, d.R, d.bias, d.G, d.ldy, d.ldz, d.ldr, d.ldg,
              d.bias_type == DION3_F32, d.act, d.accumulate, (int)d.N};
  const unsigned nch = (unsigned)(up8(d.N) / 8);
  if (d.M == 0) return hipSuccess;
  if (d.K == 0) {
    if (d.accumulate) return hipSuccess;
    hipLaunchKernelGGL((k_lin_zero<E, true>), flat_grid(d.M * nch), dim3(256), 0, s, d.M, nch, f);
    return hipGetLastError();
  }
  const double flops = 2.0 * (double)d.M * d.N * d.K;
  if (q.thin) {
    const ThinP p = {d.A, d.B, d.lda, d.ldb, d.N, (int)d.M, (int)d.K, f};
    TraceScope ts("linear_thin", flops, 2.0 * (double)d.N * d.K, s);
    const dim3 grid((unsigned)((d.N + 15) / 16));
    if (d.M == 1)
      hipLaunchKernelGGL((k_lin_vec<E>), dim3((unsigned)((d.N + 7) / 8)), dim3(512), 0, s, p);
    else
      hipLaunchKernelGGL((k_lin_thin<E>), grid, dim3(512), 0, s, p);
    return hipGetLastError();
  }
  LinP p = {};
  p.A = d.A; p.B = d.B; p.bs = d.bs; p.lda = d.lda; p.ldb = d.ldb;
  auto copy = [&](const void* src, long long ld, long long rows, long long cols, size_t o) {
    const unsigned n = (unsigned)(up8(cols) / 8);
    unsigned short* dst = (unsigned short*)((char*)ws + o);
    TraceScope ts("linear_copy", 0.0, 4.0 * (double)rows * cols, s);
    hipLaunchKernelGGL(k_lin_copy, flat_grid(rows * n), dim3(256), 0, s,
                       (const unsigned short*)src, ld, rows, (int)cols, n, dst);
    return hipGetLastError();
  };
  // (A and B may be one array read two ways: each takes its own copy)
  if (q.copyA) {
    const hipError_t e = copy(d.A, d.lda, q.rowsA, q.colsA, q.oA);
    if (e != hipSuccess) return e;
    p.A = (char*)ws + q.oA;
    p.lda = up8(q.colsA);
  }
  if (q.copyB) {
    const hipError_t e = copy(d.B, d.ldb, q.rowsB, q.colsB, q.oB);
    if (e != hipSuccess) return e;
    p.B = (char*)ws + q.oB;
    p.ldb = up8(q.colsB);
  }
  // K-contiguous operands end in whole chunks: a copy's are zero past K, and
  // a K of the other operand's rows past the true K reads zeros either way
  const LinP whole = p;
  for (int i = 0; i < q.nparts; ++i) {
    const LinPart& t = q.part[i];
    p = whole;
    p.A = (const char*)p.A + 2 * (d.a_km ? t.m0 : t.m0 * p.lda);
    if (d.bs) {
      p.B = (const char*)p.B + t.n0;
      p.bs = p.bs + t.n0 / kF8Block;
    } else {
      p.B = (const char*)p.B + 2 * (d.b_kn ? t.n0 : t.n0 * p.ldb);
    }
    p.M = t.M; p.N = (int)t.N; p.K = d.K;
    p.splits = t.splits; p.steps = t.steps;
    p.part = (float*)((char*)ws + q.oP);
    p.ldp = (int)up8(t.N);
    p.part_stride = t.M * p.ldp;
    p.f = f;
    p.f.N = (int)t.N;
    if (f.Y) p.f.Y = (char*)f.Y + 2 * (t.m0 * f.ldy + t.n0);
    if (f.Z) p.f.Z = (char*)f.Z + 2 * (t.m0 * f.ldz + t.n0);
    if (f.R) p.f.R = (const char*)f.R + 2 * (t.m0 * f.ldr + t.n0);
    if (f.G) p.f.G = f.G + t.m0 * f.ldg + t.n0;
    if (f.bias) p.f.bias = (const char*)f.bias + (f.bias_f32 ? 4 : 2) * t.n0;
    hipError_t e;
    {
      TraceScope ts(d.name, 2.0 * (double)t.M * t.N * d.K, 0.0, s);
      if (d.bs) e = launch_cfg<E, kColsK, kColsF8, true>(p, t.tile, q.ragged, s);
      else if (d.G) e = launch_cfg<E, kColsK, kColsK, true>(p, t.tile, q.ragged, s);
      else if (d.b_kn) e = launch_cfg<E, kRowsK, kColsK, false>(p, t.tile, q.ragged, s);
      else e = launch_cfg<E, kRowsK, kRowsK, false>(p, t.tile, q.ragged, s);
    }
    if (e != hipSuccess) return e;
    if (t.splits == 1) continue;
    TraceScope ts("linear_join", 0.0, 4.0 * (double)t.splits * t.M * t.N, s);
    const unsigned nch = (unsigned)(p.ldp / 8);
    e = d.G ? launch_join<E, true>(p.part, p.part_stride, t.splits, t.M, nch, p.f, s)
            : launch_join<E, false>(p.part, p.part_stride, t.splits, t.M, nch, p.f, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t lin_scratch(const LinDesc& d) { return lin_plan(d).total; }

hipError_t launch_lin(const LinDesc& d, void* ws, hipStream_t s) {
  return d.dtype == DION3_BF16 ? launch_lin_t<bf16>(d, ws, s) : launch_lin_t<f16>(d, ws, s);
}

}  // namespace dion3
