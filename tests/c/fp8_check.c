/* The 8-bit-float entry points from plain C: the header compiles as C99 and
 * every call rejects bad arguments without a GPU. Prints "ok" on success. */
#include <stdint.h>
#include <stdio.h>

#include "hxq.h"

static int failures = 0;
#define EXPECT(cond)                                                      \
    do {                                                                  \
        if (!(cond)) {                                                    \
            fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                   \
        }                                                                 \
    } while (0)

int main(void) {
    float f[64] = {0};
    uint8_t q[64] = {0};
    int32_t off[2] = {0, 1};
    int e = 0;
    hxq_fp8_t h = (hxq_fp8_t)0;
    EXPECT(hxq_fp8_ld(100) == 112);
    EXPECT(hxq_fp8_ld(-1) == HXQ_EINVAL);
    EXPECT(hxq_fp8_quantize(NULL, HXQ_TYPE_F32, 1, 16, q, f, NULL) == HXQ_EINVAL);
    EXPECT(hxq_fp8_swiglu(f, 5, 1, 16, q, f, NULL) == HXQ_EINVAL);
    EXPECT(hxq_fp8_encode(f, HXQ_TYPE_F32, 0, 1, 16, q, f, NULL) == HXQ_EINVAL);
    EXPECT(hxq_rmsnorm(f, HXQ_TYPE_F32, NULL, NULL, HXQ_TYPE_F32, NULL, 1e-6f, 1, 16, NULL, NULL, NULL, NULL) ==
           HXQ_EINVAL);
    EXPECT(hxq_fp8_create(q, f, HXQ_FP8_MAX_EXPERTS + 1, 1, 1, &h) == HXQ_EINVAL);
    EXPECT(h == NULL);
    EXPECT(hxq_fp8_forward(NULL, q, f, NULL, f, HXQ_TYPE_F32, 1, NULL) == HXQ_EINVAL);
    EXPECT(hxq_fp8_forward_grouped(NULL, q, f, off, NULL, f, HXQ_TYPE_BF16, 1, NULL) == HXQ_EINVAL);
    EXPECT(hxq_fp8_info(NULL, &e, NULL, NULL) == HXQ_EINVAL);
    EXPECT(hxq_fp8_check(NULL) == HXQ_EINVAL);
    hxq_fp8_destroy(NULL);
    if (failures) return 1;
    printf("ok\n");
    return 0;
}
