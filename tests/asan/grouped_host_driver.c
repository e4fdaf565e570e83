/* Host-side exercise of the grouped, integer and combine-gradient calls for an AddressSanitizer build (no GPU
 * work): workspace sizes over a spread of shapes, and calls that fail validation or have no rows to work on, all of which
 * return before any HIP call.  Exit status 0 when every status is the documented one. */
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
  const size_t big = (size_t)1 << 43;
  const int64_t sizes[][4] = {{1, 1, 1, 1},          {8, 2048, 768, 128},     {2048, 1024, 4096, 896}, {17, 1001, 1777, 13},
                              {62580, 7168, 2048, 32}, {268435456, 8, 16, 1024}, {40, 2097152, 64, 1},    {1024, 4, 131072, 1024},
                              {32768, 2048, 768, 128}, {333, 131072, 24, 5},     {0, 40, 24, 7}};
  for (size_t i = 0; i < sizeof sizes / sizeof sizes[0]; ++i)
    for (int dtype = 0; dtype < 2; ++dtype)
      for (int act = MOE_ACT_NONE; act <= MOE_ACT_GELU_TANH; ++act)
        for (int grad = 0; grad <= dtype; ++grad) {
          moe_grouped_shape s = {sizes[i][0], sizes[i][1], sizes[i][2], sizes[i][3], dtype, act, grad, 0};
          const int wide = s.K > (1 << 17);
          for (int call = -1; call < 7; ++call) {
            const int gated = call == 2 || call == 3 || call == 5, int8 = call >= 4;
            const size_t n = moe_grouped_workspace_bytes(&s, call);
            if (call < 0 || call > 5 || (!gated && act != MOE_ACT_NONE) || (int8 && wide)) EXPECT(n == 0);
            EXPECT(n % 256 == 0 && n < ((size_t)1 << 42));
            if (call == 3 && s.R > 0) EXPECT(n >= 2u * (size_t)s.R * (size_t)s.N * (dtype == MOE_BF16 ? 2u : 4u));
          }
          const moe_status bad_act = act == MOE_ACT_NONE ? MOE_OK : MOE_ERR_INVALID_ARG;
          EXPECT(moe_grouped_linear_forward(at(0), at(1), at(2), s.R ? NULL : at(3), &s, at(9), big, NULL) ==
                 (s.R ? MOE_ERR_INVALID_ARG : bad_act));
          EXPECT(moe_grouped_linear_backward(at(0), at(1), at(2), at(3), NULL, NULL, &s, at(9), big, NULL) == MOE_ERR_INVALID_ARG);
          EXPECT(moe_grouped_gated_forward(at(0), at(1), at(2), at(3), at(4), at(5), NULL, &s, at(9), big, NULL) ==
                 MOE_ERR_INVALID_ARG);
          if (s.R)
            EXPECT(moe_grouped_gated_backward(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(10), &s, NULL, 0,
                                              NULL) == MOE_ERR_WORKSPACE);
          EXPECT(moe_grouped_gated_backward(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), NULL, &s, at(9), big,
                                            NULL) == MOE_ERR_INVALID_ARG);
          const moe_status too_wide = wide ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
          EXPECT(moe_grouped_gated_int8_forward(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(0), &s, at(9), big, NULL) ==
                 (s.R == 0 && !wide ? MOE_OK : too_wide));
          moe_dense_shape d = {s.R, s.K, s.N, dtype, act, grad, 0};
          EXPECT(moe_linear_int8_forward(at(0), at(1), at(2), NULL, at(4), at(5), at(6), &d, NULL) == too_wide);
          EXPECT(moe_gated_int8_forward(at(0), at(1), at(2), at(3), at(4), NULL, at(6), &d, NULL) == too_wide);
        }
  for (int64_t cols = -3; cols < 5000000; cols = cols < 40 ? cols + 1 : cols * 3) {
    const int64_t n = moe_int8_row_bytes(cols);
    EXPECT(cols < 1 || cols > 2097152 ? n == 0 : n >= cols && n < cols + 16 && n % 16 == 0);
    EXPECT(moe_quantize_int8(at(0), MOE_BF16, 2, cols, NULL, at(2), NULL) ==
           (cols > 2097152 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG));
  }
  EXPECT(moe_quantize_int8(NULL, MOE_F32, 0, 8, NULL, NULL, NULL) == MOE_OK);
  EXPECT(moe_grouped_workspace_bytes(NULL, 0) == 0);
  EXPECT(moe_grouped_linear_forward(at(0), at(1), at(2), at(3), NULL, at(9), big, NULL) == MOE_ERR_INVALID_ARG);
  if (!failures) printf("all checks passed\n");
  return failures != 0;
}
