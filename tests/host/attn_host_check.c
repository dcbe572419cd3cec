/*
 * Host-side checks of the attention part of the C ABI (include/mnb.h) meant to
 * run under AddressSanitizer and UndefinedBehaviorSanitizer: descriptions,
 * sizes at the ends of their ranges, workspace sizes and refusals. Every call
 * here returns before anything would be enqueued on a GPU. Exit status 0 when
 * every check holds.
 */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "mnb.h"

static int failures = 0;
#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                          \
        }                                                                        \
    } while (0)

/* A fake, 256-byte aligned device address: only its value is ever used. */
static void *dev(uintptr_t k) { return (void *)(uintptr_t)(0x100000000ull + k * 0x100000ull); }

static mnb_kv_cache a_cache(void) {
    mnb_kv_cache c;
    memset(&c, 0, sizeof c);
    c.k = dev(1);
    c.v = dev(2);
    c.num_blocks = 64;
    c.kv_heads = 8;
    c.page_size = 16;
    c.head_dim = 128;
    c.block_stride = 8 * 16 * 128;
    c.head_stride = 16 * 128;
    c.token_stride = 128;
    c.dtype = MNB_F16;
    return c;
}

static const int64_t ENDS[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 64, 128, 1000, 65536, 65537, 1LL << 26, 1LL << 30,
                               (1LL << 30) + 1, INT_MAX, 1LL << 40, INT64_MAX};
enum { NENDS = sizeof ENDS / sizeof ENDS[0] };

static void check_workspaces(void) {
    /* any sizes: a number of bytes, without overflow on the way */
    for (int b = 0; b < NENDS; ++b)
        for (int t = 0; t < NENDS; ++t)
            for (int n = 0; n < NENDS; ++n)
                for (int h = 0; h < NENDS; ++h)
                    for (int dtype = 0; dtype < 3; ++dtype) {
                        const size_t p = mnb_paged_attn_workspace_bytes(ENDS[b], ENDS[h], ENDS[t], 64, ENDS[n], dtype);
                        const size_t c = mnb_cross_attn_workspace_bytes(ENDS[b], ENDS[t], ENDS[n], ENDS[h], ENDS[h], 128,
                                                                        dtype);
                        CHECK(p < (1ull << 40) && c < (1ull << 40));
                    }
    CHECK(mnb_paged_attn_workspace_bytes(4, 16, 8, 96, 4096, MNB_F16) == 0);
    CHECK(mnb_paged_attn_workspace_bytes(4, 16, 8, 128, 100, MNB_F16) == 0);
    CHECK(mnb_paged_attn_workspace_bytes(1, 16, 8, 128, 100000, MNB_F16) > 0);
    CHECK(mnb_cross_attn_workspace_bytes(1, 1, 1500, 12, 12, 64, MNB_F32) > 0);
}

static void check_refusals(void) {
    mnb_kv_cache c = a_cache();
    const float scale = 0.1f;
    CHECK(mnb_kv_append(dev(3), dev(4), 1024, 1024, dev(5), 0, &c, NULL) == MNB_OK);
    CHECK(mnb_kv_append(dev(3), dev(4), 1024, 1024, dev(5), 4, NULL, NULL) == MNB_ERR_NULL);
    CHECK(mnb_kv_append(dev(3), dev(4), 1024, 1001, dev(5), 4, &c, NULL) == MNB_ERR_ALIGN);
    CHECK(mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 0, 16, 8, 100, scale, NULL, 0, dev(6), NULL) == MNB_OK);
    CHECK(mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 4, 15, 8, 100, scale, NULL, 0, dev(6), NULL) == MNB_ERR_SHAPE);
    CHECK(mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 4, 16, 8, 100, NAN, NULL, 0, dev(6), NULL) == MNB_ERR_INVALID);
    CHECK(mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 1, 16, 80000, 100000, scale, NULL, 0, dev(6), NULL) ==
          MNB_ERR_NULL);
    CHECK(mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 1, 16, 80000, 100000, scale, dev(7), 16, dev(6), NULL) ==
          MNB_ERR_INVALID);
    int64_t *fields[] = {&c.num_blocks, &c.kv_heads, &c.page_size, &c.head_dim, &c.block_stride, &c.head_stride,
                         &c.token_stride};
    for (size_t f = 0; f < sizeof fields / sizeof fields[0]; ++f)
        for (int i = 0; i < NENDS; ++i) {
            c = a_cache();
            *fields[f] = ENDS[i];
            /* B = 0: a status, and nothing to enqueue */
            const int st = mnb_paged_attn(dev(3), 2048, &c, dev(4), dev(5), 0, 1 << 20, 8, 1 << 30, scale, NULL, 0,
                                          dev(6), NULL);
            CHECK(st >= MNB_OK && st <= MNB_ERR_INVALID);
        }
    const mnb_attn_view q = {dev(1), 1 << 20, 768, 64}, k = {dev(2), 1500 * 768, 768, 64};
    for (int i = 0; i < NENDS; ++i)
        for (int j = 0; j < NENDS; ++j) {
            mnb_attn_view v = k;
            v.row_stride = ENDS[i];
            const int st = mnb_cross_attn(&q, &k, &v, NULL, 4, 0, ENDS[j], 12, 12, 64, scale, MNB_F16, NULL, 0, &q, NULL);
            CHECK((ENDS[i] >= 0 && ENDS[i] <= 1 << 26 && ENDS[j] >= 0 && ENDS[j] <= MNB_MAX_KEYS && ENDS[i] % 8 == 0) ==
                  (st == MNB_OK));
        }
    CHECK(mnb_cross_attn(&q, &k, NULL, NULL, 4, 1, 10, 12, 12, 64, scale, MNB_F16, NULL, 0, &q, NULL) == MNB_ERR_NULL);
    for (int i = 0; i < NENDS; ++i)
        for (int j = 0; j < NENDS; ++j) {
            /* no output arrays: refused whatever the sizes */
            const int st = mnb_kv_tables(dev(1), dev(2), dev(3), 4, ENDS[i], 16, ENDS[j], ENDS[i], dev(4), dev(5), NULL,
                                         dev(6), NULL, NULL);
            CHECK(st == MNB_ERR_NULL);
        }
    /* an output in the place of an input, or of another output */
    CHECK(mnb_kv_tables(dev(1), dev(2), dev(3), 4, 8, 16, 8, 4, dev(4), dev(1), dev(6), dev(7), dev(8), NULL) ==
          MNB_ERR_INVALID);
    CHECK(mnb_kv_tables(dev(1), dev(2), dev(3), 4, 8, 16, 8, 4, dev(4), (int32_t *)dev(2) + 7, dev(6), dev(7), dev(8),
                        NULL) == MNB_ERR_INVALID);
    CHECK(mnb_kv_tables(dev(1), dev(2), dev(3), 4, 8, 16, 8, 4, dev(4), dev(5), dev(6), dev(7), (int32_t *)dev(6) + 8,
                        NULL) == MNB_ERR_INVALID);
    CHECK(mnb_kv_tables(dev(1), dev(2), dev(3), 4, 65536, 16, INT64_MAX, 4, dev(4), dev(5), dev(6), dev(7), dev(8),
                        NULL) == MNB_ERR_SHAPE);
}

int main(void) {
    check_workspaces();
    check_refusals();
    if (failures) return 1;
    printf("attention host checks passed\n");
    return 0;
}
