/*
 * Host paths of the ds_dispatch_*, ds_distill_* and ds_vocab_ce entry points
 * under the host sanitizers.  Every call here is refused, or has nothing to do,
 * before any device work: the addresses are made up.
 */
#include <stdio.h>

#include "dszero.h"

static int failures = 0;

static void expect(const char* what, ds_status got, ds_status want)
{
    if (got != want) {
        printf("%s: got %s, expected %s\n", what, ds_status_string(got), ds_status_string(want));
        ++failures;
    }
}

static void zero(const char* what, size_t got)
{
    if (got != 0) {
        printf("%s: got %zu, expected 0\n", what, got);
        ++failures;
    }
}

static void* at(uint64_t x) { return (void*)(uintptr_t)(x << 32); }

int main(void)
{
    const int64_t huge = INT64_MAX;
    int32_t* i32 = at(1);
    float* f32 = at(2);

    expect("sort tokens", ds_dispatch_sort(at(3), 8, huge, 8, 2, 2, i32, at(4), at(5), at(6), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("sort stride", ds_dispatch_sort(at(3), 8, 1 << 20, 8, 2, huge, i32, at(4), at(5), at(6), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("sort k", ds_dispatch_sort(at(3), 8, 8, 8, INT32_MIN, 2, i32, at(4), at(5), at(6), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("sort alias", ds_dispatch_sort(at(3), 8, 1000, 8, 2, 2, i32, at(3), at(5), at(6), SIZE_MAX, NULL), DS_ERR_ALIAS);
    zero("sort workspace", ds_dispatch_workspace_bytes(huge, 8, 2));
    zero("sort workspace", ds_dispatch_workspace_bytes(8, INT32_MAX, 2));

    expect("gather width", ds_dispatch_gather(at(3), DS_BF16, 8, 2, huge, huge, i32, at(4), huge, 16, NULL), DS_ERR_SIZE);
    expect("gather stride", ds_dispatch_gather(at(3), DS_BF16, 1 << 20, 2, 64, huge, i32, at(4), 64, 16, NULL), DS_ERR_SIZE);
    expect("gather rows", ds_dispatch_gather(at(3), DS_BF16, 8, 2, 64, 64, i32, at(4), 64, huge, NULL), DS_ERR_SIZE);
    expect("gather alias", ds_dispatch_gather(at(3), DS_FP32, 1 << 20, 2, 1024, 1024, i32, at(3), 1024, 1 << 21, NULL),
           DS_ERR_ALIAS);
    expect("gather grad none", ds_dispatch_gather_grad(NULL, DS_BF16, 0, 2, 64, 64, 0, NULL, NULL, 64, NULL), DS_OK);
    expect("combine gates", ds_dispatch_combine(at(3), DS_BF16, 8, 2, 64, 64, 16, i32, at(4), DS_FP32, INT64_MIN, at(5), 64,
                                                NULL), DS_ERR_SIZE);
    expect("combine type", ds_dispatch_combine(at(3), (ds_dtype)77, 8, 2, 64, 64, 16, i32, at(4), DS_FP32, 2, at(5), 64, NULL),
           DS_ERR_DTYPE);
    expect("combine grad alias", ds_dispatch_combine_grad(at(3), DS_FP16, 8, 2, 64, 64, at(4), 64, 16, i32, at(5), DS_FP32, 2,
                                                          at(4), 64, at(7), 2, NULL), DS_ERR_ALIAS);

    expect("distill vocab", ds_distill_loss(NULL, at(3), DS_BF16, 8, huge, huge, at(4), DS_FP32, 4, at(5), 4, 4, 4, NULL, 1.0f,
                                            1.0f, f32, at(6), at(7), NULL, 0, 0, at(8), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("distill stride", ds_distill_loss(NULL, at(3), DS_BF16, 1 << 30, 100, huge, at(4), DS_FP32, 4, at(5), 4, 4, 4, NULL,
                                             1.0f, 1.0f, f32, at(6), at(7), NULL, 0, 0, at(8), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("distill spans", ds_distill_loss(NULL, at(3), DS_FP32, 1 << 20, 1 << 20, 1 << 20, at(4), DS_FP32, 4, at(5), 4, 4, 4,
                                            NULL, 1.0f, 1.0f, f32, at(6), at(7), NULL, 0, 0, at(8), SIZE_MAX, NULL),
           DS_ERR_ALIAS);
    zero("distill workspace", ds_distill_workspace_bytes(INT64_MIN));

    expect("vocab tokens", ds_vocab_ce(NULL, at(3), 64, at(4), 64, DS_BF16, at(5), 8, huge, 100, 64, NULL, 1.0f, f32, at(6),
                                       at(7), NULL, 0, NULL, DS_BF16, 0, 0, at(8), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("vocab stride", ds_vocab_ce(NULL, at(3), huge, at(4), 64, DS_BF16, at(5), 8, 100, 100, 64, NULL, 1.0f, f32, at(6),
                                       at(7), NULL, 0, NULL, DS_BF16, 0, 0, at(8), SIZE_MAX, NULL), DS_ERR_SIZE);
    expect("vocab workspace", ds_vocab_ce(NULL, at(3), 65536, at(4), 65536, DS_BF16, at(5), 8, 1 << 24, 1 << 24, 65536, NULL,
                                          1.0f, f32, at(6), at(7), NULL, 0, NULL, DS_BF16, 0, 0, at(8), 1 << 30, NULL),
           DS_ERR_SIZE);
    expect("vocab alias", ds_vocab_ce(NULL, at(3), 64, at(4), 64, DS_BF16, at(5), 8, 100, 100, 64, NULL, 1.0f, f32, at(6), at(7),
                                      at(3), 64, NULL, DS_BF16, 0, 0, at(8), SIZE_MAX, NULL), DS_ERR_ALIAS);
    zero("vocab workspace", ds_vocab_ce_workspace_bytes(huge, huge, huge));
    if (ds_vocab_ce_workspace_bytes(1 << 24, 1 << 24, 65536) < ((size_t)1 << 41)) {
        printf("vocab workspace of the largest sizes\n");
        ++failures;
    }
    printf(failures ? "%d failures\n" : "ok\n", failures);
    return failures != 0;
}
