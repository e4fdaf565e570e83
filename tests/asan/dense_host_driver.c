/* Host-side exercise of the dense operators' C ABI for an AddressSanitizer build (no GPU work):
 * workspace sizes over a spread of shapes, and calls that fail validation or have no rows to
 * work on, all of which return before any HIP call.  Exit status 0 when every status is the
 * documented one. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe.h"

static int failures = 0;
#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      fprintf(stderr, "%s:%d: expected %s\n", __FILE__, __LINE__, #cond);   \
      ++failures;                                                           \
    }                                                                       \
  } while (0)

static void* at(int i) { return (void*)((uintptr_t)(i + 1) << 44); } /* aligned, never dereferenced */

int main(void) {
  const int64_t sizes[][3] = {{1, 1, 1},          {1, 7168, 2048},      {17, 1001, 1777},  {300, 64, 8192},
                              {8192, 7168, 2048}, {4096, 2048, 8192},   {1, 2097152, 64},  {268435456, 8, 16},
                              {65536, 4096, 4096}, {8192, 2048, 7168},  {1021, 1416, 2120}, {0, 40, 24}};
  for (size_t i = 0; i < sizeof sizes / sizeof sizes[0]; ++i)
    for (int dtype = 0; dtype < 2; ++dtype)
      for (int act = MOE_ACT_NONE; act <= MOE_ACT_GELU_TANH; ++act)
        for (int grad = 0; grad <= dtype; ++grad) {
          moe_dense_shape s = {sizes[i][0], sizes[i][1], sizes[i][2], dtype, act, grad, 0};
          const size_t b = moe_dense_workspace_bytes(&s, MOE_CALL_GATED_BACKWARD);
          EXPECT(b >= 2u * (size_t)s.T * (size_t)s.N * (dtype == MOE_BF16 ? 2u : 4u));
          for (int call = -1; call < 5; ++call) {
            const size_t n = moe_dense_workspace_bytes(&s, call);
            EXPECT(n % 256 == 0 && (call >= 0 && call < 4 ? n < ((size_t)1 << 42) : n == 0));
          }
          EXPECT(moe_gated_forward(at(0), at(1), at(2), s.T ? NULL : at(3), at(4), NULL, &s, at(9), (size_t)1 << 43,
                                   NULL) == MOE_ERR_INVALID_ARG);
          EXPECT(moe_gated_backward(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), &s, NULL, 0, NULL) ==
                 (b ? MOE_ERR_WORKSPACE : MOE_OK) || s.T == 0);
          EXPECT(moe_linear_forward(at(0), at(1), at(2), at(3), at(4), at(4), &s, at(9), (size_t)1 << 43, NULL) ==
                 (s.T ? MOE_ERR_INVALID_ARG : MOE_OK));
          EXPECT(moe_linear_backward(at(0), at(1), at(2), act ? at(3) : NULL, NULL, NULL, NULL, &s, at(9),
                                     (size_t)1 << 43, NULL) == MOE_ERR_INVALID_ARG);
        }
  for (int64_t h = 1; h < 40000; h = h * 3 + 1)
    for (int64_t t = 0; t < 300000; t = t * 7 + 1) {
      moe_norm_shape s = {t, h, 1e-5f, MOE_BF16, MOE_F32, 0};
      const size_t n = moe_norm_workspace_bytes(&s);
      EXPECT(t == 0 ? n == 0 : n >= (size_t)h * 8);
      EXPECT(moe_layer_norm_forward(at(0), at(1), at(2), at(0), NULL, NULL, &s, NULL) ==
             (t ? MOE_ERR_INVALID_ARG : MOE_OK));
      EXPECT(moe_layer_norm_backward(at(0), at(1), at(2), at(3), at(4), NULL, NULL, NULL, &s, at(9), n, NULL) ==
             MOE_ERR_INVALID_ARG);
    }
  moe_dense_shape bad = {-1, 8, 8, MOE_BF16, MOE_ACT_NONE, MOE_BF16, 0};
  EXPECT(moe_dense_workspace_bytes(&bad, MOE_CALL_LINEAR_FORWARD) == 0);
  EXPECT(moe_dense_workspace_bytes(NULL, MOE_CALL_LINEAR_FORWARD) == 0);
  EXPECT(moe_norm_workspace_bytes(NULL) == 0);
  if (!failures) printf("all checks passed\n");
  return failures != 0;
}
