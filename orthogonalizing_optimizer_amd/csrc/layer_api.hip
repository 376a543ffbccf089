// C ABI of the layer operators: argument checks and dispatch.  The contract
// of every entry point is stated in include/dion3.h.
#include "checks.h"

using namespace dion3;

namespace {

bool act_ok(int a) { return a >= DION3_ACT_NONE && a <= DION3_ACT_SILU; }

// The descriptions of the three products (see LinDesc).  Each call's
// workspace is sized by the same description its launch uses.
dion3_status describe_linear(LinDesc& d, const void* X, int64_t ldx, const void* W, int64_t ldw,
                             int64_t T, int64_t n, int64_t m) {
  TRY(check_sizes(T, n, m));
  TRY(check_ld(ldx, m));
  TRY(check_ld(ldw, m));
  d = LinDesc{};
  d.A = X; d.lda = ldx; d.B = W; d.ldb = ldw;
  d.M = T; d.N = n; d.K = m;
  d.name = "linear";
  return DION3_OK;
}

dion3_status describe_grad_input(LinDesc& d, const void* dZ, int64_t lddz, const void* W, int64_t ldw,
                                 int64_t T, int64_t n, int64_t m) {
  TRY(check_sizes(T, n, m));
  TRY(check_ld(lddz, n));
  TRY(check_ld(ldw, m));
  d = LinDesc{};
  d.A = dZ; d.lda = lddz; d.B = W; d.ldb = ldw; d.b_kn = true;
  d.M = T; d.N = m; d.K = n;
  d.name = "linear_grad_input";
  return DION3_OK;
}

dion3_status describe_grad_weight(LinDesc& d, const void* dZ, int64_t lddz, const void* X,
                                  int64_t ldx, const uint8_t* S, int64_t T, int64_t n, int64_t m) {
  TRY(check_sizes(T, n, m));
  TRY(check_ld(lddz, n));
  if (!S) TRY(check_ld(ldx, m));
  d = LinDesc{};
  d.A = dZ; d.lda = lddz; d.a_km = true;
  d.B = X; d.ldb = S ? f8_cols(m) : ldx; d.b_kn = true; d.bs = S;
  d.M = n; d.N = m; d.K = T;
  d.name = S ? "linear_grad_weight_f8" : "linear_grad_weight";
  return DION3_OK;
}

dion3_status run_product(const LinDesc& d, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_scratch(ws, ws_bytes, lin_scratch(d)));
  HIP_TRY(launch_lin(d, ws, (hipStream_t)stream));
  return DION3_OK;
}

}  // namespace

extern "C" {

dion3_status dion3_add_rms_norm(const void* X, int64_t ldx, const void* R, int64_t ldr,
                                const void* w, int32_t wtype, void* H, int64_t ldh, void* Y,
                                int64_t ldy, uint8_t* Q, uint8_t* S, float* rstd, int64_t T,
                                int64_t m, float eps, int32_t dtype, void* stream) {
  if (!type16(dtype) || (wtype != DION3_F32 && wtype != dtype)) return DION3_ERR_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return DION3_ERR_ARG;
  TRY(check_sizes(T, m, 1));
  if (!w || !elem_aligned(w, wtype == DION3_F32 ? 4 : 2)) return DION3_ERR_ARG;
  if ((R != nullptr) != (H != nullptr) || (Q != nullptr) != (S != nullptr)) return DION3_ERR_ARG;
  TRY(check_ld(ldx, m));
  if (R) {
    TRY(check_ld(ldr, m));
    TRY(check_ld(ldh, m));
  }
  if (Y) TRY(check_ld(ldy, m));
  if (T == 0) return DION3_OK;
  if (!X || (!Y && !Q)) return DION3_ERR_ARG;
  if (!elem_aligned(X, 2) || !elem_aligned(R, 2) || !elem_aligned(H, 2) || !elem_aligned(Y, 2) ||
      !elem_aligned(rstd, 4) || !elem_aligned(Q, 16))
    return DION3_ERR_ARG;
  const NormArgs a = {X, ldx, R, ldr, w, wtype, H, ldh, Y, ldy, Q, S, rstd, T, (int)m, eps, dtype};
  HIP_TRY(launch_add_rms_norm(a, (hipStream_t)stream));
  return DION3_OK;
}

dion3_status dion3_add_rms_norm_grad_workspace_size(int64_t T, int64_t m, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  TRY(check_sizes(T, m, 1));
  *bytes = norm_grad_scratch(T, m);
  return DION3_OK;
}

dion3_status dion3_add_rms_norm_grad(const void* dY, int64_t lddy, const void* H, int64_t ldh,
                                     const float* rstd, const void* w, int32_t wtype,
                                     const void* dH, int64_t lddh, void* dX, int64_t lddx,
                                     float* dw, int64_t T, int64_t m, int32_t dtype, void* ws,
                                     size_t ws_bytes, void* stream) {
  if (!type16(dtype) || (wtype != DION3_F32 && wtype != dtype)) return DION3_ERR_ARG;
  TRY(check_sizes(T, m, 1));
  if (!w || !elem_aligned(w, wtype == DION3_F32 ? 4 : 2)) return DION3_ERR_ARG;
  if (!elem_aligned(dw, 4)) return DION3_ERR_ARG;
  TRY(check_ld(lddy, m));
  TRY(check_ld(ldh, m));
  if (dH) TRY(check_ld(lddh, m));
  if (dX) TRY(check_ld(lddx, m));
  if (T > 0) {
    if (!dY || !H || !rstd || (!dX && !dw)) return DION3_ERR_ARG;
    if (!elem_aligned(dY, 2) || !elem_aligned(H, 2) || !elem_aligned(dH, 2) ||
        !elem_aligned(dX, 2) || !elem_aligned(rstd, 4))
      return DION3_ERR_ARG;
  }
  TRY(check_scratch(ws, ws_bytes, norm_grad_scratch(T, m)));
  const NormGradArgs a = {dY, lddy, H, ldh, rstd, w, wtype, dH, lddh, dX, lddx, dw, T, (int)m, dtype};
  HIP_TRY(launch_add_rms_norm_grad(a, ws, (hipStream_t)stream));
  return DION3_OK;
}

dion3_status dion3_pack_f8(const void* X, int64_t ldx, uint8_t* Q, uint8_t* S, int64_t T, int64_t m,
                           int32_t dtype, void* stream) {
  if (!type16(dtype) && dtype != DION3_F32) return DION3_ERR_ARG;
  TRY(check_sizes(T, m, 1));
  TRY(check_ld(ldx, m));
  if (T == 0) return DION3_OK;
  if (!X || !Q || !S || !elem_aligned(X, dtype == DION3_F32 ? 4 : 2) || !elem_aligned(Q, 16))
    return DION3_ERR_ARG;
  HIP_TRY(launch_pack_f8(X, ldx, Q, S, T, (int)m, dtype, (hipStream_t)stream));
  return DION3_OK;
}

dion3_status dion3_unpack_f8(const uint8_t* Q, const uint8_t* S, void* Y, int64_t ldy, int64_t T,
                             int64_t m, int32_t dtype, void* stream) {
  if (!type16(dtype) && dtype != DION3_F32) return DION3_ERR_ARG;
  TRY(check_sizes(T, m, 1));
  TRY(check_ld(ldy, m));
  if (T == 0) return DION3_OK;
  if (!Y || !Q || !S || !elem_aligned(Y, dtype == DION3_F32 ? 4 : 2) || !elem_aligned(Q, 16))
    return DION3_ERR_ARG;
  HIP_TRY(launch_unpack_f8(Q, S, Y, ldy, T, (int)m, dtype, (hipStream_t)stream));
  return DION3_OK;
}

dion3_status dion3_linear_workspace_size(const void* X, int64_t ldx, const void* W, int64_t ldw,
                                         int64_t T, int64_t n, int64_t m, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_linear(d, X, ldx, W, ldw, T, n, m));
  *bytes = lin_scratch(d);
  return DION3_OK;
}

dion3_status dion3_linear(const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias,
                          int32_t bias_type, const void* R, int64_t ldr, void* Y, int64_t ldy,
                          void* Z, int64_t ldz, int64_t T, int64_t n, int64_t m, int32_t act,
                          int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  if (!type16(dtype) || !act_ok(act)) return DION3_ERR_ARG;
  if (bias && ((bias_type != DION3_F32 && bias_type != dtype) ||
               !elem_aligned(bias, bias_type == DION3_F32 ? 4 : 2)))
    return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_linear(d, X, ldx, W, ldw, T, n, m));
  if (R) TRY(check_ld(ldr, n));
  if (Z) TRY(check_ld(ldz, n));
  TRY(check_ld(ldy, n));
  if (T == 0) return DION3_OK;
  if (!X || !W || !Y) return DION3_ERR_ARG;
  if (!elem_aligned(X, 2) || !elem_aligned(W, 2) || !elem_aligned(R, 2) || !elem_aligned(Y, 2) ||
      !elem_aligned(Z, 2))
    return DION3_ERR_ARG;
  d.Y = Y; d.ldy = ldy; d.Z = Z; d.ldz = ldz; d.R = R; d.ldr = ldr;
  d.bias = bias; d.bias_type = bias_type; d.act = act; d.dtype = dtype;
  return run_product(d, ws, ws_bytes, stream);
}

dion3_status dion3_act_grad_workspace_size(int64_t T, int64_t n, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, 1));
  *bytes = act_grad_scratch(T, n);
  return DION3_OK;
}

dion3_status dion3_act_grad(const void* dY, int64_t lddy, const void* Z, int64_t ldz,
                            const uint8_t* ZQ, const uint8_t* ZS, void* dZ, int64_t lddz, float* db,
                            int64_t T, int64_t n, int32_t act, int32_t dtype, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!type16(dtype) || !act_ok(act)) return DION3_ERR_ARG;
  TRY(check_sizes(T, n, 1));
  TRY(check_ld(lddy, n));
  if (Z) TRY(check_ld(ldz, n));
  if (dZ) TRY(check_ld(lddz, n));
  if ((ZQ != nullptr) != (ZS != nullptr) || (Z && ZQ) || !elem_aligned(db, 4)) return DION3_ERR_ARG;
  if (T > 0) {
    if (!dY || (act != DION3_ACT_NONE && !Z && !ZQ) || (!dZ && !db)) return DION3_ERR_ARG;
    if (!elem_aligned(dY, 2) || !elem_aligned(Z, 2) || !elem_aligned(ZQ, 16) || !elem_aligned(dZ, 2))
      return DION3_ERR_ARG;
  }
  if (db) TRY(check_scratch(ws, ws_bytes, act_grad_scratch(T, n)));
  const ActGradArgs a = {dY, lddy, Z, ldz, ZQ, ZS, dZ, lddz, db, T, (int)n, act, dtype};
  HIP_TRY(launch_act_grad(a, ws, (hipStream_t)stream));
  return DION3_OK;
}

dion3_status dion3_linear_grad_input_workspace_size(const void* dZ, int64_t lddz, const void* W,
                                                    int64_t ldw, int64_t T, int64_t n, int64_t m,
                                                    size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_grad_input(d, dZ, lddz, W, ldw, T, n, m));
  *bytes = lin_scratch(d);
  return DION3_OK;
}

dion3_status dion3_linear_grad_input(const void* dZ, int64_t lddz, const void* W, int64_t ldw,
                                     const void* R, int64_t ldr, void* dX, int64_t lddx, int64_t T,
                                     int64_t n, int64_t m, int32_t dtype, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!type16(dtype)) return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_grad_input(d, dZ, lddz, W, ldw, T, n, m));
  if (R) TRY(check_ld(ldr, m));
  TRY(check_ld(lddx, m));
  if (T == 0) return DION3_OK;
  if (!dZ || !W || !dX) return DION3_ERR_ARG;
  if (!elem_aligned(dZ, 2) || !elem_aligned(W, 2) || !elem_aligned(R, 2) || !elem_aligned(dX, 2))
    return DION3_ERR_ARG;
  d.Y = dX; d.ldy = lddx; d.R = R; d.ldr = ldr; d.act = DION3_ACT_NONE; d.dtype = dtype;
  return run_product(d, ws, ws_bytes, stream);
}

dion3_status dion3_linear_grad_weight_workspace_size(const void* dZ, int64_t lddz, const void* X,
                                                     int64_t ldx, const uint8_t* S, int64_t T,
                                                     int64_t n, int64_t m, size_t* bytes) {
  if (!bytes) return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_grad_weight(d, dZ, lddz, X, ldx, S, T, n, m));
  *bytes = lin_scratch(d);
  return DION3_OK;
}

dion3_status dion3_linear_grad_weight(const void* dZ, int64_t lddz, const void* X, int64_t ldx,
                                      const uint8_t* S, float* G, int64_t ldg, int32_t accumulate,
                                      int64_t T, int64_t n, int64_t m, int32_t dtype, void* ws,
                                      size_t ws_bytes, void* stream) {
  if (!type16(dtype)) return DION3_ERR_ARG;
  LinDesc d;
  TRY(describe_grad_weight(d, dZ, lddz, X, ldx, S, T, n, m));
  TRY(check_ld(ldg, m));
  if (!G || !elem_aligned(G, 4)) return DION3_ERR_ARG;
  if (T > 0 && (!dZ || !X || !elem_aligned(dZ, 2) || !elem_aligned(X, S ? 16 : 2)))
    return DION3_ERR_ARG;
  d.G = G; d.ldg = ldg; d.accumulate = accumulate != 0; d.dtype = dtype;
  return run_product(d, ws, ws_bytes, stream);
}

}  // extern "C"
