/*
 * Host-side checks of the 8-bit cache's part of the C ABI (include/mnb.h) and of
 * the rotary positions, meant to run under AddressSanitizer and
 * UndefinedBehaviorSanitizer: descriptions, sizes at the ends of their ranges,
 * workspace sizes and refusals. Every call here returns before anything would
 * be enqueued on a GPU. Exit status 0 when every check holds.
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

static mnb_kv_cache_i8 a_cache(void) {
    mnb_kv_cache_i8 c;
    memset(&c, 0, sizeof c);
    c.k = dev(1);
    c.v = dev(2);
    c.k_scale = dev(3);
    c.v_scale = dev(4);
    c.num_blocks = 64;
    c.kv_heads = 8;
    c.page_size = 16;
    c.head_dim = 128;
    c.block_stride = 8 * 16 * 128;
    c.head_stride = 16 * 128;
    c.token_stride = 128;
    c.scale_block_stride = 8 * 16;
    c.scale_head_stride = 16;
    c.dtype = MNB_F16;
    return c;
}

static const int64_t ENDS[] = {INT64_MIN, -1, 0, 1, 2, 8, 15, 16, 64, 128, 1000, 65536, 65537, 1LL << 26, 1LL << 30,
                               (1LL << 30) + 1, INT_MAX, 1LL << 40, INT64_MAX};
enum { NENDS = sizeof ENDS / sizeof ENDS[0] };

static void check_workspaces(void) {
    /* any sizes: a number of bytes, without overflow on the way */
    for (int b = 0; b < NENDS; ++b)
        for (int h = 0; h < NENDS; ++h)
            for (int k = 0; k < NENDS; ++k)
                for (int n = 0; n < NENDS; ++n)
                    for (int m = 0; m < NENDS; ++m)
                        for (int dtype = 0; dtype < 3; ++dtype) {
                            const size_t w = mnb_paged_attn_i8_workspace_bytes(ENDS[b], ENDS[h], ENDS[k], 64, ENDS[n],
                                                                               ENDS[m], dtype);
                            CHECK(w < (1ull << 45));
                        }
    CHECK(mnb_paged_attn_i8_workspace_bytes(4, 16, 8, 96, 4096, 1, MNB_F16) == 0);
    CHECK(mnb_paged_attn_i8_workspace_bytes(4, 16, 8, 128, 100, 1, MNB_F16) == 0);
    CHECK(mnb_paged_attn_i8_workspace_bytes(1, 16, 8, 128, 100000, 1, MNB_F16) > 0);
    CHECK(mnb_paged_attn_i8_workspace_bytes(1, 16, 8, 128, 100000, 62, MNB_F16) > 0);
    CHECK(mnb_paged_attn_i8_workspace_bytes(1, 12, 12, 64, 100000, 62, MNB_F32) > 0);
}

static void check_refusals(void) {
    mnb_kv_cache_i8 c = a_cache();
    int64_t *slots = dev(5);
    int32_t *table = dev(6), *lens = dev(7), *starts = dev(8);
    const float scale = 0.1f;
    CHECK(mnb_kv_append_i8(dev(9), dev(10), 1024, 1024, slots, 0, &c, NULL) == MNB_OK);
    CHECK(mnb_kv_append_i8(dev(9), dev(10), 1024, 1024, slots, 4, NULL, NULL) == MNB_ERR_NULL);
    CHECK(mnb_kv_append_i8(dev(9), dev(10), 1024, 1001, slots, 4, &c, NULL) == MNB_ERR_ALIGN);
    CHECK(mnb_kv_read_i8(slots, 0, &c, dev(9), dev(10), 1024, 1024, NULL) == MNB_OK);
    CHECK(mnb_kv_read_i8(slots, 4, &c, dev(9), dev(9), 1024, 1024, NULL) == MNB_ERR_INVALID);
    CHECK(mnb_kv_read_i8(slots, 4, &c, dev(9), dev(10), 0, 1024, NULL) == MNB_ERR_INVALID);
    /* (no tokens: a status, and nothing to enqueue) */
#define ATTN(T, B, heads, width, len, nw, st, ws, bytes)                                                                  \
    mnb_paged_attn_i8(dev(9), 2048, &c, table, lens, st, T, B, heads, width, len, nw, scale, ws, bytes, dev(11), NULL)
    CHECK(ATTN(0, 0, 16, 8, 100, 1, NULL, NULL, 0) == MNB_OK);
    CHECK(ATTN(0, 4, 16, 8, 100, 5, starts, NULL, 0) == MNB_OK);
    CHECK(ATTN(4, 4, 15, 8, 100, 1, NULL, NULL, 0) == MNB_ERR_SHAPE);
    CHECK(ATTN(5, 4, 16, 8, 100, 1, NULL, NULL, 0) == MNB_ERR_SHAPE);
    CHECK(ATTN(4, 4, 16, 8, 100, 2, NULL, NULL, 0) == MNB_ERR_SHAPE);
    CHECK(ATTN(1, 1, 16, 80000, 100000, 1, NULL, NULL, 0) == MNB_ERR_NULL);
    CHECK(ATTN(1, 1, 16, 80000, 100000, 1, NULL, dev(12), 16) == MNB_ERR_INVALID);
    CHECK(ATTN(62, 1, 16, 80000, 100000, 62, starts, dev(12), 16) == MNB_ERR_INVALID);
    int64_t *fields[] = {&c.num_blocks, &c.kv_heads, &c.page_size, &c.head_dim, &c.block_stride, &c.head_stride,
                         &c.token_stride, &c.scale_block_stride, &c.scale_head_stride};
    for (size_t f = 0; f < sizeof fields / sizeof fields[0]; ++f)
        for (int i = 0; i < NENDS; ++i) {
            c = a_cache();
            *fields[f] = ENDS[i];
            int st = ATTN(0, 0, 1 << 20, 8, 1 << 30, 1, starts, NULL, 0);
            CHECK(st >= MNB_OK && st <= MNB_ERR_INVALID);
            st = mnb_kv_append_i8(dev(9), dev(10), 1024, 1024, slots, 0, &c, NULL);
            CHECK(st >= MNB_OK && st <= MNB_ERR_INVALID);
        }
    c = a_cache();
    for (int i = 0; i < NENDS; ++i)
        for (int j = 0; j < NENDS; ++j)
            for (int k = 0; k < NENDS; ++k) {
                /* every size at its ends, with no queries to answer or no memory to answer from */
                CHECK(ATTN(0, ENDS[i], 16, ENDS[j], 100, ENDS[k], starts, NULL, 0) <= MNB_ERR_INVALID);
                CHECK(ATTN(ENDS[i], 0, 16, 8, ENDS[j], ENDS[k], starts, NULL, 0) <= MNB_ERR_INVALID);
                const int st = mnb_paged_attn_i8(NULL, ENDS[i], &c, table, lens, starts, ENDS[j], 4, 16, 8, 100, ENDS[k],
                                                 scale, NULL, 0, NULL, NULL);
                CHECK(st != MNB_OK || ENDS[j] == 0);
                /* outputs in each other's place: refused whatever the sizes (or nothing to do) */
                CHECK((mnb_kv_read_i8(slots, ENDS[i], &c, dev(9), dev(9), ENDS[j], ENDS[k], NULL) == MNB_OK) <=
                      (ENDS[i] == 0));
                CHECK((mnb_kv_append_i8(NULL, NULL, ENDS[j], ENDS[k], slots, ENDS[i], &c, NULL) == MNB_OK) <=
                      (ENDS[i] == 0));
                CHECK((mnb_rope(dev(9), ENDS[j], dev(10), ENDS[k], 16, dev(11), 1024, dev(10), 1024, 8, table, dev(12),
                                ENDS[i], 128, 128, MNB_ROPE_HALF, 1.0f, MNB_F16, NULL) == MNB_OK) <= (ENDS[i] == 0));
                CHECK((mnb_rope(NULL, 1024, NULL, 1024, ENDS[i], NULL, 1024, NULL, 1024, 8, table, dev(12), 4, ENDS[j],
                                ENDS[k], MNB_ROPE_HALF, 1.0f, MNB_F32, NULL)) != MNB_OK);
            }
    CHECK(mnb_rope(dev(9), 2048, dev(10), 2048, 16, NULL, 0, NULL, 0, 0, table, dev(12), 4, 128, 128, 7, 1.0f, MNB_F16,
                   NULL) == MNB_ERR_INVALID);
    CHECK(mnb_rope(dev(9), 2048, dev(10), 2048, 16, NULL, 0, NULL, 0, 0, table, dev(12), 4, 128, 128, MNB_ROPE_HALF, NAN,
                   MNB_F16, NULL) == MNB_ERR_INVALID);
    CHECK(mnb_rope(NULL, 0, NULL, 0, 0, NULL, 0, NULL, 0, 0, NULL, NULL, 4, 128, 128, MNB_ROPE_HALF, 1.0f, MNB_F16,
                   NULL) == MNB_OK);
    /* an output one element behind its input */
    CHECK(mnb_rope(dev(9), 2048, (char *)dev(9) + 16, 2048, 16, NULL, 0, NULL, 0, 0, table, dev(12), 4, 128, 128,
                   MNB_ROPE_HALF, 1.0f, MNB_F16, NULL) == MNB_ERR_INVALID);
}

int main(void) {
    check_workspaces();
    check_refusals();
    if (failures) return 1;
    printf("8-bit cache host checks passed\n");
    return 0;
}
