/* Drives the C ABI of routing by a rule and of the microscaled products without a GPU: sizes,
 * strides and workspaces at the extremes of their types (overflow in the size arithmetic would
 * be undefined behaviour). Device pointers are fake addresses that are never dereferenced. */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "qmoe.h"

#define FAKE(i) ((void*)(uintptr_t)(((uint64_t)(i) + 1) << 48))
#define BAD MOE_ERR_INVALID_ARGUMENT
#define OK MOE_OK

extern int launches;
static int failures = 0;

static void expect(const char* what, moe_status got, moe_status want) {
  if (got != want) {
    printf("MISMATCH %s: status %d, expected %d\n", what, (int)got, (int)want);
    ++failures;
  }
}

static moe_mx_matrix mat(int rows, int cols, int at) {
  moe_mx_matrix m = {(const uint8_t*)FAKE(at), (const uint8_t*)FAKE(at + 1), rows, cols};
  return m;
}

int main(void) {
  const int64_t far[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 8, 32, INT64_MAX / 4, INT64_MAX - 7, INT64_MAX};
  const int ints[] = {INT_MIN, -1, 0, 1, 31, 32, 65536, 65537, 1 << 24, INT_MAX - 31, INT_MAX};
  const int nfar = sizeof far / sizeof *far, nints = sizeof ints / sizeof *ints;
  uint8_t *codes = FAKE(2), *scales = FAKE(3);
  for (int i = 0; i < nfar; ++i)
    for (int j = 0; j < nints; ++j)
      for (int k = 0; k < nfar; ++k)
        for (int dtype = -1; dtype < 5; ++dtype) {
          moe_mx_matrix m = mat(ints[j], ints[j], 5);
          moe_mx_quantize(FAKE(1), dtype, far[i], ints[j], far[k], codes, scales, NULL);
          moe_mx_dequantize(&m, far[i], dtype, FAKE(1), NULL);
        }
  /* one row: its stride is not read; two: it is */
  for (int k = 0; k < nfar; ++k) {
    moe_mx_matrix w = mat(64, 64, 5), x1 = mat(1, 64, 8), x2 = mat(2, 64, 8);
    const int fits = far[k] == 32 || far[k] == 0 || far[k] == 8;
    expect("quantize 1", moe_mx_quantize(FAKE(1), MOE_F32, 1, 64, far[k], codes, scales, NULL), OK);
    expect("quantize 2", moe_mx_quantize(FAKE(1), MOE_BF16, 2, 64, far[k], codes, scales, NULL), fits ? OK : BAD);
    expect("linear 1", moe_mx_linear(FAKE(1), MOE_BF16, far[k], 1, &w, FAKE(2), MOE_F32, far[k], NULL, 0, NULL), OK);
    expect("linear 2", moe_mx_linear(FAKE(1), MOE_BF16, far[k], 2, &w, FAKE(2), MOE_F32, 64, NULL, 0, NULL),
           fits ? OK : BAD);
    expect("linear out 2", moe_mx_linear(FAKE(1), MOE_BF16, 64, 2, &w, FAKE(2), MOE_F32, far[k], NULL, 0, NULL), BAD);
    expect("linear quantized 1", moe_mx_linear_quantized(&x1, &w, FAKE(2), MOE_F16, far[k], NULL), OK);
    expect("linear quantized 2", moe_mx_linear_quantized(&x2, &w, FAKE(2), MOE_F16, far[k], NULL), BAD);
  }
  for (int i = 0; i < nints; ++i)
    for (int j = 0; j < nints; ++j) {
      moe_mx_matrix w = mat(ints[j], 64, 5), x = mat(ints[i], 64, 8);
      moe_mx_linear(FAKE(1), MOE_F32, 64, ints[i], &w, FAKE(2), MOE_F32, INT64_MAX, FAKE(4), SIZE_MAX, NULL);
      moe_mx_linear_quantized(&x, &w, FAKE(2), MOE_F32, INT64_MAX / 2, NULL);
      moe_mx_linear_workspace_bytes(ints[i], ints[j]);
      for (int k = 0; k < nints; ++k) {
        moe_mx_layer L = {ints[j], 64, ints[k], ints[i], mat(64, ints[j], 5), mat(64, ints[j], 8), mat(ints[j], 64, 11)};
        moe_routing r = {FAKE(14), FAKE(15), FAKE(16), FAKE(17)};
        moe_route_rule rule = {MOE_SCORE_SIGMOID, NULL, ints[j], ints[k], MOE_GROUP_MAX, 1, 1.0f};
        for (int n = 0; n < nints; ++n) {
          moe_mx_ffn_workspace_bytes(&L, ints[n]);
          moe_mx_ffn(&L, FAKE(1), MOE_F32, INT64_MAX, ints[n], &r, NULL, FAKE(2), FAKE(4), SIZE_MAX, NULL);
          moe_route_scored(FAKE(1), MOE_F32, ints[n], ints[i], ints[k], &rule, &r, FAKE(4), SIZE_MAX, NULL);
        }
      }
    }
  {
    /* the largest layer and chunk: the workspace is what the call takes */
    moe_mx_layer L = {8192, 8192, 1024, 64, mat(8192, 8192, 5), mat(8192, 8192, 8), mat(8192, 8192, 11)};
    moe_routing r = {FAKE(14), FAKE(15), FAKE(16), FAKE(17)};
    const size_t need = moe_mx_ffn_workspace_bytes(&L, 8192);
    if (need < (size_t)8192 * 64 * 8192 * 4) ++failures;
    expect("ffn", moe_mx_ffn(&L, FAKE(1), MOE_F16, 8192, 8192, &r, NULL, FAKE(2), FAKE(4), need, NULL), OK);
    expect("ffn, a byte less", moe_mx_ffn(&L, FAKE(1), MOE_F16, 8192, 8192, &r, NULL, FAKE(2), FAKE(4), need - 1, NULL),
           MOE_ERR_WORKSPACE_TOO_SMALL);
    expect("ffn 1", moe_mx_ffn(&L, FAKE(1), MOE_F16, INT64_MIN, 1, &r, NULL, FAKE(2), FAKE(4), need, NULL), OK);
  }
  printf("mx driver: %d mismatches, %d launches\n", failures, launches);
  return failures != 0 || launches == 0;
}
