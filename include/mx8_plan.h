/*
 * mx8_plan.h -- which of libw12.so's kernels an mx8_gemm (mx8.h) takes, for tests
 * that have to reach all of them and for reading profiles.
 */
#ifndef MX8_PLAN_H
#define MX8_PLAN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mx8_gemm_plan -- the kernel of mx8_gemm(M, N, K) by its name and template
 * arguments, a static string, and the slices of K it works in (rows of x 2^24
 * bytes apart and more make it "small_kernel<2, 4>" in one slice where a
 * tile_kernel is named).  NULL, and 0 slices, for a shape that mx8_gemm refuses
 * and for M = 0.  `slices` may be NULL.
 */
const char *mx8_gemm_plan(int64_t M, int64_t N, int64_t K, int *slices);

#ifdef __cplusplus
}
#endif

#endif /* MX8_PLAN_H */
