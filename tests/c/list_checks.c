/*
 * Host paths of ds_tensor_list_write, ds_check_overflow_list,
 * ds_adam_step_list, ds_balance_loss and ds_balance_loss_grad under the host
 * sanitizers.  Every call here is refused, or has nothing to do, before any
 * device work: the addresses are made up.
 */
#include <inttypes.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dszero.h"

static int failures = 0;

static void expect(const char* what, ds_status got, ds_status want)
{
    if (got != want) {
        printf("%s: got %s, expected %s\n", what, ds_status_string(got), ds_status_string(want));
        ++failures;
    }
}

static void* at(uint64_t x) { return (void*)(uintptr_t)x; }

static ds_tensor tensor(uint64_t base, int64_t n)
{
    const uint64_t step = 1u << 20;
    ds_tensor t;
    memset(&t, 0, sizeof t);
    t.master = at(base);
    t.p16 = at(base + step);
    t.m = at(base + 2 * step);
    t.v = at(base + 3 * step);
    t.m_scale = at(base + 4 * step);
    t.v_scale = at(base + 5 * step);
    t.grad = at(base + 6 * step);
    t.n = n;
    t.lr_scale = 1.0f;
    t.pdt = DS_BF16;
    t.gdt = DS_FP32;
    return t;
}

/* `count` tensors side by side, the last one's first state inside `into`'s array: found by sorting all ranges. */
static void overlap_among(int count, int into)
{
    ds_tensor* t = malloc(sizeof(ds_tensor) * (size_t)count);
    if (t == NULL)
        exit(2);
    for (int i = 0; i < count; ++i)   /* descending addresses, so that the order has to be found */
        t[i] = tensor(0x100000000ull + (uint64_t)(count - i) * 0x1000000ull, 1 + i % 5000);
    t[count - 1].m = (char*)t[into].v + t[into].n - 1;
    ds_tensor_list list;
    char what[64];
    snprintf(what, sizeof what, "overlap of tensor %d with %d", count - 1, into);
    expect(what, ds_tensor_list_write(&list, at(0x10000000), ds_tensor_list_bytes(count), t, count, DS_FP8, NULL),
           DS_ERR_ALIAS);
    free(t);
}

int main(void)
{
    ds_tensor_list list;
    ds_tensor t = tensor(0x100000000ull, 1000);
    void* table = at(0x10000000);
    ds_scaler* st = at(0x20000000);

    for (int count = 2; count < 3000; count = count * 2 + 1)
        for (int into = 0; into < count - 1; into += 1 + count / 3)
            overlap_among(count, into);

    expect("list NULL", ds_tensor_list_write(NULL, table, 1 << 20, &t, 1, DS_FP8, NULL), DS_ERR_NULL);
    expect("count", ds_tensor_list_write(&list, table, 1 << 20, &t, -1, DS_FP8, NULL), DS_ERR_SIZE);
    expect("table bytes", ds_tensor_list_write(&list, table, 10, &t, 1, DS_FP8, NULL), DS_ERR_SIZE);
    expect("states", ds_tensor_list_write(&list, table, 1 << 20, &t, 1, DS_BF16, NULL), DS_ERR_DTYPE);
    t.n = INT64_MAX;
    expect("n", ds_tensor_list_write(&list, table, 1 << 20, &t, 1, DS_FP8, NULL), DS_ERR_SIZE);
    t.n = INT64_MIN;
    expect("n", ds_tensor_list_write(&list, table, 1 << 20, &t, 1, DS_FP8, NULL), DS_ERR_SIZE);

    ds_tensor many[3] = {tensor(0x100000000ull, (int64_t)1 << 39), tensor(0x90000000000ull, (int64_t)1 << 39),
                         tensor(0xF0000000000ull, 1)};
    expect("sum of n", ds_tensor_list_write(&list, table, 1 << 20, many, 3, DS_FP8, NULL), DS_ERR_SIZE);
    many[2].n = 0;   /* 2^40 in all: within the limit, and each tensor's arrays overlap */
    expect("largest sum of n", ds_tensor_list_write(&list, table, 1 << 20, many, 3, DS_FP8, NULL), DS_ERR_ALIAS);
    many[2].n = ((int64_t)1 << 40) - 5;
    expect("sum of n", ds_tensor_list_write(&list, table, 1 << 20, many + 1, 2, DS_FP8, NULL), DS_ERR_SIZE);

    expect("empty list", ds_tensor_list_write(&list, NULL, 0, NULL, 0, DS_FP8, NULL), DS_OK);
    expect("empty check", ds_check_overflow_list(st, &list, NULL, 0, NULL), DS_OK);
    expect("empty step", ds_adam_step_list(st, &list, 1e-3f, NULL, 0.9, 0.999, 1e-8f, 0.0f, 1, DS_ROUND_NEAREST, 0, 0,
                                           NULL), DS_OK);
    list.table = table;
    list.count = 1;
    list.elems = INT64_MAX;
    list.tiles = INT64_MAX;
    expect("bad list", ds_check_overflow_list(st, &list, NULL, 0, NULL), DS_ERR_SIZE);
    if (ds_tensor_list_workspace_bytes(&list) != 0 || ds_tensor_list_workspace_bytes(NULL) != 0)
        ++failures, printf("workspace of a bad list\n");

    void* z = at(0x30000000);
    int32_t* counts = at(0x40000000);
    float* mean = at(0x50000000);
    expect("tokens", ds_balance_loss(z, DS_BF16, INT64_MAX, 8, 8, NULL, 2, 0.1f, counts, mean, mean + 64, counts + 64,
                                     table, 1 << 20, NULL), DS_ERR_SIZE);
    expect("stride", ds_balance_loss(z, DS_BF16, 1 << 30, 8, INT64_MAX, NULL, 2, 0.1f, counts, mean, mean + 64,
                                     counts + 64, table, 1 << 20, NULL), DS_ERR_SIZE);
    expect("alias", ds_balance_loss(z, DS_BF16, 1 << 30, 512, 1024, NULL, 2, 0.1f, counts, mean, mean + 4, counts + 64,
                                    table, SIZE_MAX, NULL), DS_ERR_ALIAS);
    expect("grad stride", ds_balance_loss_grad(st, z, DS_FP32, 1 << 30, 512, 512, NULL, 2, 0.1f, counts, counts + 600,
                                               table, INT64_MAX, 0, NULL), DS_ERR_SIZE);
    expect("grad alias", ds_balance_loss_grad(st, z, DS_FP32, 9, 512, 512, NULL, 2, 0.1f, counts, counts + 600,
                                              (char*)z + 4 * 512 * 9 - 4, 512, 0, NULL), DS_ERR_ALIAS);
    if (ds_balance_workspace_bytes(INT64_MAX, 8) != 0 || ds_balance_workspace_bytes(8, INT32_MAX) != 0)
        ++failures, printf("workspace of bad sizes\n");
    printf(failures ? "%d failures\n" : "ok\n", failures);
    return failures != 0;
}
