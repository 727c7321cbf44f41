// linear.cuh -- matrix products of token rows with a linear layer's weights
// (linear.cu: the operators; gemm.cu: the tensor-core product).
#pragma once
#include "common.cuh"

namespace vae {

// ------------------------------------------------------------------ operators
size_t linear_ws_bytes(int dtype, long long rows, int n, int k);
int linear(const void *x, int dtype, long long rows, int k, const void *w, const float *bias,
           int n, int act, const void *residual, void *y, void *z, void *ws, cudaStream_t s);

size_t linear_dgrad_ws_bytes(int dtype, long long rows, int n, int k);
int linear_dgrad(const void *dy, int dtype, long long rows, int n, const void *w, int k, int act,
                 const void *z, void *dx, void *ws, cudaStream_t s);

size_t linear_wgrad_ws_bytes(int dtype, long long rows, int n, int k);
int linear_wgrad(const void *dy, const void *x, int dtype, long long rows, int n, int k, float *dw,
                 float *dbias, void *ws, cudaStream_t s);

// ------------------------------------------------------------------ the product
// One operand: 16-bit numbers, `parts` matrices of the same size one after another.
// K-major: [rows of the result][reduction], as the reduction's neighbours lie side by
// side; else [reduction][rows of the result].
struct GemmOperand {
  const void *p = nullptr;
  bool k_major = true;
};

// What becomes of a sum: z = sum + bias, kept where asked; out = act(z) + aux, or, for
// `derivative`, out = sum act'(aux).
struct GemmEpilogue {
  const float *bias = nullptr;
  const void *aux = nullptr;
  void *out = nullptr;
  void *keep = nullptr;
  int act = 0;
  bool derivative = false;
};

// How a product is made: on pairs of SMs or in small tiles, and, where `sliced` sums
// are asked for, its long reduction in how many slices, whose sums [slices][m][n] are
// added up in order afterwards. `columns`: partial sums of A's columns (1: the sums).
struct GemmPlan {
  bool pairs = false;
  int slices = 1, columns = 1;
};
GemmPlan gemm_plan(long long m, int n, long long k, int parts, bool sliced);

// Sums over the reduction of A's columns, taken on the way: src [rows][m], the numbers
// A's parts come from, of `dtype`; part [columns][m] (NULL: none). For float results.
struct GemmColumnSums {
  const void *src = nullptr;
  int dtype = 0;
  long long rows = 0;
  float *part = nullptr;
  int step = 1;  // (the launch's: blocks of 64 rows from one to the next)
};

// out[m][n] = sum over k of A[m][k] B[n][k], A and B of bf16 or f16 numbers, or, with
// parts == 3, each the sum of three bf16 matrices (a float's 24 bits), of whose
// products the six largest are added up. out, aux and keep are of `dtype`; a
// float's sum moves from the tensor core's accumulator to FP32 registers after every
// 32 steps of 16.
struct GemmDesc {
  GemmOperand a, b;
  int parts = 1;
  bool f16 = false;  // the operands' type (bf16 otherwise)
  int dtype = 0;
  long long m = 0;
  int n = 0;
  long long k = 0;
  bool wait = false;  // an operand is made by the launch before this one
  GemmEpilogue epi;
  GemmColumnSums cols;
  GemmPlan plan;
};
int gemm(const GemmDesc &d, cudaStream_t s);

// The same as linear() for few rows, on the FP32 cores (gemv.cu).
constexpr int kFewRows = 8;
int linear_few(const void *x, int dtype, int rows, int k, const void *w, int n,
               const GemmEpilogue &e, cudaStream_t s);

}  // namespace vae
