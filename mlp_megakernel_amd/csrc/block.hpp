// Internal launch interface of the operators around the feed-forward products:
// layer norm, dropout, quantisation and the 8-bit products.
#pragma once
#include "launch.hpp"

namespace coalesce {

// A dropout mask: an element is dropped where its word is at most `last`.
struct Drop {
  bool on;
  uint32_t last;
  float scale;  // 1 / (1 - p)
  uint64_t seed, offset;
  const uint64_t* device_seed;  // {seed, offset} in device memory, or nullptr
};

// Layer norm of M rows of N.  The stream (the norm's input) is of type TS, the
// operand (what it gives, and the branch added in front of it) of type T.
struct NormParams {
  const void* X;  // without R the stream, with R the branch
  const void* R;  // stream that the branch is added to, or nullptr
  void* S;        // the sum, or nullptr
  void* Y;
  const void *weight, *bias;  // or nullptr
  float *mean, *rstd;         // or nullptr
  int64_t ldx, ldr, lds, ldy;
  int M, N;
  float eps;
  DType wt;  // type of weight and bias
  Drop drop;
};
hipError_t launch_norm(const NormParams& p, DType operand, DType stream_type, hipStream_t stream);

struct NormBwdParams {
  const void* S;   // the stream (TS)
  const void* dY;  // gradient of the norm's result (T)
  const void* dS;  // gradient that arrives along the stream (TS), or nullptr
  void* dX;        // the stream's gradient (TS), or nullptr
  void* dB;        // the branch's (T), or nullptr
  const void* weight;
  const float *mean, *rstd;
  void *dweight, *dbias;  // of type gt, or nullptr
  float* partial;         // the workspace
  int64_t lds, ldy, ldg, ldx, ldb;
  int M, N;
  int groups, ldp;  // partial sums per column and their pitch (set by the launcher)
  bool alone;       // one workgroup, which writes dweight and dbias itself
  DType wt, gt;
  Drop drop;
};
size_t norm_backward_workspace(int64_t M, int64_t N, int num_cus);
hipError_t launch_norm_backward(NormBwdParams p, DType operand, DType stream_type, hipStream_t stream, int num_cus);

struct DropoutParams {
  const void* X;
  const void* R;  // of the result's type, or nullptr
  void* Y;
  int64_t ldx, ldr, ldy;
  int M, N;
  Drop drop;
};
hipError_t launch_dropout(const DropoutParams& p, DType in, DType out, hipStream_t stream);

// Rows to 8-bit integers: scale = largest magnitude / 127, q = x / scale rounded.
struct QuantParams {
  const void* X;
  int8_t* Q;
  float* scale;
  int64_t ldx, ldq;
  int M, N;  // of X
};
hipError_t launch_quantize_rows(const QuantParams& p, DType dt, hipStream_t stream);
// The same by columns, Q transposed: N rows of M.
hipError_t launch_quantize_columns(const QuantParams& p, DType dt, hipStream_t stream);

// The products on 8-bit operands (int8_forward.hpp): A is M x K, B[i] N x K.
struct Int8Params {
  const int8_t* A;
  const int8_t* B[2];
  const float* scale_a;
  const float* scale_b[2];
  const float* bias[2];
  const void* R;
  void* Y;
  int64_t lda, ldb, ldr, ldy;
  int M, N, K;
  int act;
};
// Joins the ranges of a split contraction: int32 sums P[i] of pitch ldp, `splits` of
// them split_stride elements apart.
struct Int8Join {
  Int8Params q;
  const int32_t* P[2];
  int64_t ldp, split_stride;
  int splits, products;
};
hipError_t launch_int8_sums(const TileOp& o, bool gated, int variant, hipStream_t stream, int num_cus);
hipError_t launch_int8_join(const Int8Join& j, DType out, hipStream_t stream, int num_cus);
#define COALESCE_INT8(NAME) \
  hipError_t launch_int8_##NAME(const Int8Params& p, hipStream_t stream, int num_cus, void* workspace);
COALESCE_INT8(gated_bf16)
COALESCE_INT8(gated_f16)
COALESCE_INT8(gated_f32)
COALESCE_INT8(resid_bf16)
COALESCE_INT8(resid_f16)
COALESCE_INT8(resid_f32)
#undef COALESCE_INT8
// Workspace (bytes, 0: none) and launch; `workspace` holds that many bytes.
size_t int8_workspace(int64_t M, int64_t N, int64_t K, bool gated, int num_cus);
hipError_t launch_int8(const Int8Params& p, bool gated, DType out, hipStream_t stream, int num_cus, void* workspace);

}  // namespace coalesce
