// C ABI of the operators around the feed-forward products: layer norm, dropout,
// quantisation, the 8-bit products.  As in abi.cpp: every check on the host before
// anything is launched, no device memory allocated.
#include <cmath>

#include "abi_check.hpp"
#include "block.hpp"

using namespace coalesce;

namespace {

// Rows and columns of a row-wise operator.
coalesce_status check_rows(int64_t M, int64_t N) {
  if (M < 0 || N < 0)
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "negative extent (M=%lld N=%lld)", (long long)M, (long long)N);
  const int64_t lim = kMaxExtent - 256;
  if (M > lim || N > lim) return fail(COALESCE_ERR_UNSUPPORTED, "extents must be below 2^31 - 256");
  if (N && M > (int64_t(1) << 41) / N) return fail(COALESCE_ERR_UNSUPPORTED, "more than 2^41 elements");
  return COALESCE_OK;
}

// `wide` is `narrow` or F32.
coalesce_status check_types(coalesce_dtype narrow, coalesce_dtype wide) {
  if (!valid_dtype(narrow) || !valid_dtype(wide)) return fail(COALESCE_ERR_INVALID_ARGUMENT, "unknown dtype");
  if (wide != narrow && wide != COALESCE_F32)
    return fail(COALESCE_ERR_UNSUPPORTED, "dtype combination %d and %d not supported", (int)narrow, (int)wide);
  return COALESCE_OK;
}

// The mask of probability p: dropped where a word of 32 bits is below round(p
// 2^32).  p below 2^-33 drops nothing, p = 1 everything.
coalesce_status make_drop(double p, uint64_t seed, uint64_t offset, const uint64_t* device_seed, Drop* d) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(COALESCE_ERR_INVALID_ARGUMENT, "p must lie in [0, 1]");
  if (device_seed && (reinterpret_cast<uintptr_t>(device_seed) & 7u))
    return fail(COALESCE_ERR_UNSUPPORTED, "the seed in device memory must be 8-byte aligned");
  const double words = std::nearbyint(p * 4294967296.0);
  d->on = words > 0.0;
  d->last = d->on ? (uint32_t)((uint64_t)words - 1) : 0u;
  d->scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
  d->seed = seed;
  d->offset = offset;
  d->device_seed = d->on ? device_seed : nullptr;
  return COALESCE_OK;
}

coalesce_status check_stat(const float* t, const char* name) {
  if (reinterpret_cast<uintptr_t>(t) & 3u) return fail(COALESCE_ERR_UNSUPPORTED, "%s must be 4-byte aligned", name);
  return COALESCE_OK;
}

void add_seed(Operands& ops, const Drop& d) {
  if (d.device_seed) ops.run(false, {(uintptr_t)d.device_seed, (uintptr_t)d.device_seed + 16}, "the seed");
}

// A matrix of 8-bit operands: K is limited by what its products may sum to.
constexpr int64_t kMaxInt8K = 131071;  // 128 * 128 * 131071 < 2^31

coalesce_status check_int8(int64_t M, int64_t N, int64_t K, coalesce_dtype out, coalesce_act act) {
  if (M < 0 || N < 0 || K < 0)
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "negative extent (M=%lld N=%lld K=%lld)", (long long)M, (long long)N,
                (long long)K);
  if (!valid_dtype(out)) return fail(COALESCE_ERR_INVALID_ARGUMENT, "unknown dtype");
  if (!valid_ffn_act(act)) return fail(COALESCE_ERR_INVALID_ARGUMENT, "unknown activation %d", (int)act);
  const int64_t lim = kMaxExtent - 256;
  if (M > lim || N > lim) return fail(COALESCE_ERR_UNSUPPORTED, "extents must be below 2^31 - 256");
  if (K > kMaxInt8K)
    return fail(COALESCE_ERR_UNSUPPORTED, "K above %lld may overflow the int32 sums", (long long)kMaxInt8K);
  if (N && M > (int64_t(1) << 41) / N) return fail(COALESCE_ERR_UNSUPPORTED, "a product of two extents above 2^41");
  return COALESCE_OK;
}

// Both products; B[1] only for the gated one, R only for the other.
coalesce_status int8_product(bool gated, const int8_t* A, int64_t lda, const int8_t* const (&B)[2], int64_t ldb,
                             const float* scale_a, const float* const (&scale_b)[2], const float* const (&bias)[2],
                             const void* R, int64_t ldr, void* Y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                             coalesce_dtype out, coalesce_act act, void* workspace, size_t workspace_bytes,
                             void* stream) {
  coalesce_status s = check_int8(M, N, K, out, act);
  if (s != COALESCE_OK) return s;
  if (M == 0 || N == 0) return ok();
  const int64_t os = dsize(out);
  static const char* const bn[2] = {"B (or Bg)", "Bu"};
  static const char* const sn[2] = {"scale_b (or scale_g)", "scale_u"};
  static const char* const vn[2] = {"bias (or bias_g)", "bias_u"};
  Operands ops;
  if ((s = check_mat(Y, ldy, N, os, "Y")) != COALESCE_OK) return s;
  ops.mat(true, Y, M, N, ldy, os, "Y");
  if (K > 0) {
    if ((s = check_mat(A, lda, K, 1, "A")) != COALESCE_OK) return s;
    ops.mat(false, A, M, K, lda, 1, "A");
  }
  if (!scale_a) return fail(COALESCE_ERR_INVALID_ARGUMENT, "scale_a is NULL");
  if ((s = check_stat(scale_a, "scale_a")) != COALESCE_OK) return s;
  ops.mat(false, scale_a, 1, M, M, 4, "scale_a");
  for (int i = 0; i < (gated ? 2 : 1); ++i) {
    if (K > 0) {
      if ((s = check_mat(B[i], ldb, K, 1, bn[i])) != COALESCE_OK) return s;
      ops.mat(false, B[i], N, K, ldb, 1, bn[i]);
    }
    if (!scale_b[i]) return fail(COALESCE_ERR_INVALID_ARGUMENT, "%s is NULL", sn[i]);
    if ((s = check_vec(scale_b[i], sn[i])) != COALESCE_OK) return s;
    ops.mat(false, scale_b[i], 1, N, N, 4, sn[i]);
    if ((s = check_vec(bias[i], vn[i])) != COALESCE_OK) return s;
    ops.mat(false, bias[i], 1, N, N, 4, vn[i]);
  }
  if (R) {
    if ((s = check_mat(R, ldr, N, os, "R")) != COALESCE_OK) return s;
    if (R == Y && ldr != ldy) return fail(COALESCE_ERR_INVALID_ARGUMENT, "in-place residual with different pitches");
    if (R != Y) ops.mat(false, R, M, N, ldr, os, "R");
  }
  if ((s = ops.check()) != COALESCE_OK) return s;
  int cus = 0;
  if ((s = current_cus(&cus)) != COALESCE_OK) return s;
  const size_t need = int8_workspace(M, N, K, gated, cus);
  if ((s = check_workspace(workspace, workspace_bytes, need)) != COALESCE_OK) return s;
  if (need) {
    ops.run(true, {(uintptr_t)workspace, (uintptr_t)workspace + need}, "the workspace");
    if ((s = ops.check()) != COALESCE_OK) return s;
  }
  Int8Params q{};
  q.A = A;
  q.scale_a = scale_a;
  for (int i = 0; i < (gated ? 2 : 1); ++i) {
    q.B[i] = B[i];
    q.scale_b[i] = scale_b[i];
    q.bias[i] = bias[i];
  }
  q.R = R;
  q.Y = Y;
  q.lda = K > 0 ? lda : 0;  // (unchecked where the operands have no elements)
  q.ldb = K > 0 ? ldb : 0;
  q.ldr = ldr;
  q.ldy = ldy;
  q.M = (int)M;
  q.N = (int)N;
  q.K = (int)K;
  q.act = ffn_act_code(act);
  hipError_t e = launch_int8(q, gated, dt_code(out), (hipStream_t)stream, cus, workspace);
  if (e != hipSuccess) return device_fail(e, gated ? "gated 8-bit product launch" : "8-bit product launch");
  return ok();
}

size_t int8_workspace_size(bool gated, int64_t M, int64_t N, int64_t K) {
  if (check_int8(M, N, K, COALESCE_F32, COALESCE_ACT_NONE) != COALESCE_OK) return 0;
  int cus = 0;
  if (current_cus(&cus) != COALESCE_OK) return 0;
  ok();
  return M == 0 || N == 0 ? 0 : int8_workspace(M, N, K, gated, cus);
}

// Rows or columns of X to 8 bits; Q has `rows` rows of `cols`.
coalesce_status quantize(bool columns, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t M,
                         int64_t N, coalesce_dtype dtype, void* stream) {
  coalesce_status s = check_rows(M, N);
  if (s != COALESCE_OK) return s;
  if (!valid_dtype(dtype)) return fail(COALESCE_ERR_INVALID_ARGUMENT, "unknown dtype");
  const int64_t rows = columns ? N : M, cols = columns ? M : N;  // of Q
  if (rows == 0) return ok();
  if (!scale) return fail(COALESCE_ERR_INVALID_ARGUMENT, "scale is NULL");
  if ((s = check_stat(scale, "scale")) != COALESCE_OK) return s;
  Operands ops;
  ops.mat(true, scale, 1, rows, rows, 4, "scale");
  if (cols > 0) {
    if ((s = check_mat(X, ldx, N, dsize(dtype), "X")) != COALESCE_OK) return s;
    ops.mat(false, X, M, N, ldx, dsize(dtype), "X");
    if ((s = check_mat(Q, ldq, cols, 1, "Q")) != COALESCE_OK) return s;
    ops.mat(true, Q, rows, cols, ldq, 1, "Q");
  }
  if ((s = ops.check()) != COALESCE_OK) return s;
  int cus = 0;
  if ((s = current_cus(&cus)) != COALESCE_OK) return s;  // a device that answers, as in every other entry point
  QuantParams q{X, Q, scale, ldx, ldq, (int)M, (int)N};
  hipError_t e = columns ? launch_quantize_columns(q, dt_code(dtype), (hipStream_t)stream)
                         : launch_quantize_rows(q, dt_code(dtype), (hipStream_t)stream);
  if (e != hipSuccess) return device_fail(e, "quantisation launch");
  return ok();
}

}  // namespace

extern "C" {

coalesce_status coalesce_quantize_rows(const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t M,
                                       int64_t N, coalesce_dtype dtype, void* stream) {
  return quantize(false, X, ldx, Q, ldq, scale, M, N, dtype, stream);
}

coalesce_status coalesce_quantize_columns(const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t M,
                                          int64_t N, coalesce_dtype dtype, void* stream) {
  return quantize(true, X, ldx, Q, ldq, scale, M, N, dtype, stream);
}

size_t coalesce_gemm_int8_workspace_size(int64_t M, int64_t N, int64_t K) {
  return int8_workspace_size(false, M, N, K);
}
size_t coalesce_gated_gemm_int8_workspace_size(int64_t M, int64_t N, int64_t K) {
  return int8_workspace_size(true, M, N, K);
}

coalesce_status coalesce_gemm_int8(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* scale_a,
                                   const float* scale_b, const float* bias, const void* R, int64_t ldr, void* Y,
                                   int64_t ldy, int64_t M, int64_t N, int64_t K, coalesce_dtype out_dtype,
                                   coalesce_act act, void* workspace, size_t workspace_bytes, void* stream) {
  return int8_product(false, A, lda, {B, nullptr}, ldb, scale_a, {scale_b, nullptr}, {bias, nullptr}, R, ldr, Y, ldy,
                      M, N, K, out_dtype, act, workspace, workspace_bytes, stream);
}

coalesce_status coalesce_gated_gemm_int8(const int8_t* A, int64_t lda, const int8_t* Bg, const int8_t* Bu, int64_t ldb,
                                         const float* scale_a, const float* scale_g, const float* scale_u,
                                         const float* bias_g, const float* bias_u, void* Y, int64_t ldy, int64_t M,
                                         int64_t N, int64_t K, coalesce_dtype out_dtype, coalesce_act act,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  return int8_product(true, A, lda, {Bg, Bu}, ldb, scale_a, {scale_g, scale_u}, {bias_g, bias_u}, nullptr, 0, Y, ldy,
                      M, N, K, out_dtype, act, workspace, workspace_bytes, stream);
}

coalesce_status coalesce_layer_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, void* S, int64_t lds,
                                    const void* weight, const void* bias, void* Y, int64_t ldy, float* mean,
                                    float* rstd, int64_t M, int64_t N, coalesce_dtype dtype,
                                    coalesce_dtype stream_dtype, coalesce_dtype weight_dtype, double eps, double p,
                                    uint64_t seed, uint64_t offset, const uint64_t* device_seed, void* stream) {
  coalesce_status s = check_rows(M, N);
  if (s != COALESCE_OK) return s;
  if ((s = check_types(dtype, stream_dtype)) != COALESCE_OK) return s;
  if ((s = check_types(dtype, weight_dtype)) != COALESCE_OK) return s;
  if (!(eps >= 0.0) || std::isinf((float)eps))
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "eps must be a number of at least 0 and finite in fp32");
  Drop drop{};
  if ((s = make_drop(p, seed, offset, device_seed, &drop)) != COALESCE_OK) return s;
  if (M == 0 || N == 0) return ok();  // (R of no rows may have no address)
  if (!R && (S || p != 0.0))
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "a sum or a dropout without the stream that X is added to");
  const int64_t es = dsize(dtype), ss = dsize(stream_dtype), xs = R ? es : ss, ws = dsize(weight_dtype);
  Operands ops;
  if ((s = check_mat(X, ldx, N, xs, "X")) != COALESCE_OK) return s;
  ops.mat(false, X, M, N, ldx, xs, "X");
  if ((s = check_mat(Y, ldy, N, es, "Y")) != COALESCE_OK) return s;
  ops.mat(true, Y, M, N, ldy, es, "Y");
  if (S) {
    if ((s = check_mat(S, lds, N, ss, "S")) != COALESCE_OK) return s;
    ops.mat(true, S, M, N, lds, ss, "S");
  }
  if (R) {
    if ((s = check_mat(R, ldr, N, ss, "R")) != COALESCE_OK) return s;
    if (R == S && ldr != lds) return fail(COALESCE_ERR_INVALID_ARGUMENT, "in-place sum with different pitches");
    if (R != S) ops.mat(false, R, M, N, ldr, ss, "R");
  }
  if ((s = check_vec(weight, "weight")) != COALESCE_OK) return s;
  if ((s = check_vec(bias, "bias")) != COALESCE_OK) return s;
  ops.mat(false, weight, 1, N, N, ws, "weight");
  ops.mat(false, bias, 1, N, N, ws, "bias");
  if ((s = check_stat(mean, "mean")) != COALESCE_OK) return s;
  if ((s = check_stat(rstd, "rstd")) != COALESCE_OK) return s;
  ops.mat(true, mean, 1, M, M, 4, "mean");
  ops.mat(true, rstd, 1, M, M, 4, "rstd");
  add_seed(ops, drop);
  if ((s = ops.check()) != COALESCE_OK) return s;
  int cus = 0;
  if ((s = current_cus(&cus)) != COALESCE_OK) return s;  // a device that answers, as in every other entry point
  NormParams q{};
  q.X = X;
  q.R = R;
  q.S = S;
  q.Y = Y;
  q.weight = weight;
  q.bias = bias;
  q.mean = mean;
  q.rstd = rstd;
  q.ldx = ldx;
  q.ldr = ldr;
  q.lds = lds;
  q.ldy = ldy;
  q.M = (int)M;
  q.N = (int)N;
  q.eps = (float)eps;
  q.wt = dt_code(weight_dtype);
  q.drop = drop;
  hipError_t e = launch_norm(q, dt_code(dtype), dt_code(stream_dtype), (hipStream_t)stream);
  if (e != hipSuccess) return device_fail(e, "layer norm launch");
  return ok();
}

size_t coalesce_layer_norm_backward_workspace_size(int64_t M, int64_t N) {
  if (check_rows(M, N) != COALESCE_OK) return 0;
  int cus = 0;
  if (current_cus(&cus) != COALESCE_OK) return 0;
  ok();
  return norm_backward_workspace(M, N, cus);
}

coalesce_status coalesce_layer_norm_backward(const void* S, int64_t lds, const void* weight, const float* mean,
                                             const float* rstd, const void* dY, int64_t ldy, const void* dS,
                                             int64_t ldg, void* dX, int64_t ldx, void* dB, int64_t ldb, void* dweight,
                                             void* dbias, int64_t M, int64_t N, coalesce_dtype dtype,
                                             coalesce_dtype stream_dtype, coalesce_dtype weight_dtype,
                                             coalesce_dtype grad_dtype, double p, uint64_t seed, uint64_t offset,
                                             const uint64_t* device_seed, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  coalesce_status s = check_rows(M, N);
  if (s != COALESCE_OK) return s;
  if ((s = check_types(dtype, stream_dtype)) != COALESCE_OK) return s;
  if ((s = check_types(dtype, weight_dtype)) != COALESCE_OK) return s;
  if ((s = check_types(dtype, grad_dtype)) != COALESCE_OK) return s;
  Drop drop{};
  if ((s = make_drop(p, seed, offset, device_seed, &drop)) != COALESCE_OK) return s;
  if (M == 0) dX = dB = nullptr;
  if (N == 0 || (!dX && !dB && !dweight && !dbias)) return ok();
  if (N >= (int64_t(1) << 23)) return fail(COALESCE_ERR_UNSUPPORTED, "rows must be shorter than 2^23");  // as pitches
  const int64_t es = dsize(dtype), ss = dsize(stream_dtype), gs = dsize(grad_dtype);
  Operands ops;
  if (M > 0) {
    if ((s = check_mat(S, lds, N, ss, "S")) != COALESCE_OK) return s;
    ops.mat(false, S, M, N, lds, ss, "S");
    if ((s = check_mat(dY, ldy, N, es, "dY")) != COALESCE_OK) return s;
    ops.mat(false, dY, M, N, ldy, es, "dY");
    if (!mean || !rstd) return fail(COALESCE_ERR_INVALID_ARGUMENT, "mean or rstd is NULL");
    if ((s = check_stat(mean, "mean")) != COALESCE_OK) return s;
    if ((s = check_stat(rstd, "rstd")) != COALESCE_OK) return s;
    ops.mat(false, mean, 1, M, M, 4, "mean");
    ops.mat(false, rstd, 1, M, M, 4, "rstd");
    if (dS) {
      if ((s = check_mat(dS, ldg, N, ss, "dS")) != COALESCE_OK) return s;
      if (dS == dX && ldg != ldx) return fail(COALESCE_ERR_INVALID_ARGUMENT, "dS in place with different pitches");
      if (dS != dX) ops.mat(false, dS, M, N, ldg, ss, "dS");
    }
    if (dX) {
      if ((s = check_mat(dX, ldx, N, ss, "dX")) != COALESCE_OK) return s;
      ops.mat(true, dX, M, N, ldx, ss, "dX");
    }
    if (dB) {
      if ((s = check_mat(dB, ldb, N, es, "dB")) != COALESCE_OK) return s;
      ops.mat(true, dB, M, N, ldb, es, "dB");
    }
    add_seed(ops, drop);
  }
  if ((s = check_vec(weight, "weight")) != COALESCE_OK) return s;
  if ((s = check_vec(dweight, "dweight")) != COALESCE_OK) return s;
  if ((s = check_vec(dbias, "dbias")) != COALESCE_OK) return s;
  ops.mat(false, weight, 1, N, N, dsize(weight_dtype), "weight");
  ops.mat(true, dweight, 1, N, N, gs, "dweight");
  ops.mat(true, dbias, 1, N, N, gs, "dbias");
  if ((s = ops.check()) != COALESCE_OK) return s;
  int cus = 0;
  if ((s = current_cus(&cus)) != COALESCE_OK) return s;
  const size_t need = dweight || dbias ? norm_backward_workspace(M, N, cus) : 0;
  if ((s = check_workspace(workspace, workspace_bytes, need)) != COALESCE_OK) return s;
  if (need) {
    ops.run(true, {(uintptr_t)workspace, (uintptr_t)workspace + need}, "the workspace");
    if ((s = ops.check()) != COALESCE_OK) return s;
  }
  NormBwdParams q{};
  q.S = S;
  q.dY = dY;
  q.dS = dS;
  q.dX = dX;
  q.dB = dB;
  q.weight = weight;
  q.mean = mean;
  q.rstd = rstd;
  q.dweight = dweight;
  q.dbias = dbias;
  q.partial = (float*)workspace;
  q.lds = lds;
  q.ldy = ldy;
  q.ldg = ldg;
  q.ldx = ldx;
  q.ldb = ldb;
  q.M = (int)M;
  q.N = (int)N;
  q.wt = dt_code(weight_dtype);
  q.gt = dt_code(grad_dtype);
  q.drop = drop;
  hipError_t e = launch_norm_backward(q, dt_code(dtype), dt_code(stream_dtype), (hipStream_t)stream, cus);
  if (e != hipSuccess) return device_fail(e, "layer norm backward launch");
  return ok();
}

coalesce_status coalesce_dropout(const void* X, int64_t ldx, const void* R, int64_t ldr, void* Y, int64_t ldy,
                                 int64_t M, int64_t N, coalesce_dtype dtype, coalesce_dtype out_dtype, double p,
                                 uint64_t seed, uint64_t offset, const uint64_t* device_seed, void* stream) {
  coalesce_status s = check_rows(M, N);
  if (s != COALESCE_OK) return s;
  if ((s = check_types(dtype, out_dtype)) != COALESCE_OK) return s;
  Drop drop{};
  if ((s = make_drop(p, seed, offset, device_seed, &drop)) != COALESCE_OK) return s;
  if (M == 0 || N == 0) return ok();
  const int64_t es = dsize(dtype), os = dsize(out_dtype);
  Operands ops;
  if ((s = check_mat(X, ldx, N, es, "X")) != COALESCE_OK) return s;
  if ((s = check_mat(Y, ldy, N, os, "Y")) != COALESCE_OK) return s;
  ops.mat(true, Y, M, N, ldy, os, "Y");
  if (X == Y && (ldx != ldy || es != os))
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "in place with different pitches or types");
  if (X != Y) ops.mat(false, X, M, N, ldx, es, "X");
  if (R) {
    if ((s = check_mat(R, ldr, N, os, "R")) != COALESCE_OK) return s;
    if (R == Y && ldr != ldy) return fail(COALESCE_ERR_INVALID_ARGUMENT, "in-place residual with different pitches");
    if (R != Y) ops.mat(false, R, M, N, ldr, os, "R");
  }
  add_seed(ops, drop);
  if ((s = ops.check()) != COALESCE_OK) return s;
  int cus = 0;
  if ((s = current_cus(&cus)) != COALESCE_OK) return s;  // a device that answers, as in every other entry point
  DropoutParams q{};
  q.X = X;
  q.R = R;
  q.Y = Y;
  q.ldx = ldx;
  q.ldr = ldr;
  q.ldy = ldy;
  q.M = (int)M;
  q.N = (int)N;
  q.drop = drop;
  hipError_t e = launch_dropout(q, dt_code(dtype), dt_code(out_dtype), (hipStream_t)stream);
  if (e != hipSuccess) return device_fail(e, "dropout launch");
  return ok();
}

}  // extern "C"
