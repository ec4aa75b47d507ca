/* A C99 caller of the checkpoint and 4-bit calls of the C ABI (include/mhc.h),
 * compiled and run on the host.  Only calls that return before touching a
 * device are made -- empty batches, workspace sizes and argument errors -- so
 * no GPU is needed.  Prints one line per failed check and exits with the
 * number of failures. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "mhc.h"

static int failures = 0;

#define CHECK(cond)                                             \
    do {                                                        \
        if (!(cond)) {                                          \
            printf("FAILED line %d: %s\n", __LINE__, #cond);    \
            ++failures;                                         \
        }                                                       \
    } while (0)

#define INVALID(call, text)                                             \
    do {                                                                \
        CHECK((call) == MHC_ERR_INVALID_ARGUMENT);                      \
        CHECK(strstr(mhc_last_error(), text) != NULL);                  \
    } while (0)

/* aligned addresses far apart that are never dereferenced: every call that
 * gets them fails validation first, or has no rows */
static void* at(int k) { return (void*)(uintptr_t)(0x10000u + ((uint64_t)k << 40)); }
static uint8_t* bytes_at(int k) { return (uint8_t*)at(k); }
static float* floats_at(int k) { return (float*)at(k); }

static void checkpoints(void)
{
    CHECK(mhc_ckpt_pack(NULL, MHC_BF16, NULL, NULL, 0, 8, MHC_CKPT_E4M3, NULL) == MHC_OK);
    CHECK(mhc_ckpt_unpack(NULL, NULL, NULL, MHC_FP32, 0, 40, MHC_CKPT_INT8, NULL) == MHC_OK);
    CHECK(mhc_last_error()[0] == '\0');
    INVALID(mhc_ckpt_pack(at(0), 2, at(1), bytes_at(2), 4, 64, 0, NULL), "dtype");
    INVALID(mhc_ckpt_pack(at(0), 0, at(1), bytes_at(2), 4, 64, 2, NULL), "format");
    INVALID(mhc_ckpt_pack(at(0), 0, at(1), bytes_at(2), 4, 60, 0, NULL), "multiple of 8");
    INVALID(mhc_ckpt_pack(at(0), 0, at(1), bytes_at(2), 4, INT64_MAX, 0, NULL), "multiple of 8");
    INVALID(mhc_ckpt_pack(at(0), 0, at(1), bytes_at(2), INT64_MAX, 64, 0, NULL), "out of range");
    INVALID(mhc_ckpt_pack(at(0), 0, at(1), bytes_at(2), INT64_MIN, 64, 0, NULL), "out of range");
    INVALID(mhc_ckpt_pack(NULL, 0, at(1), bytes_at(2), 4, 64, 0, NULL), "NULL");
    INVALID(mhc_ckpt_pack(at(0), 0, at(0), bytes_at(2), 4, 64, 0, NULL), "overlaps");
    INVALID(mhc_ckpt_unpack(at(1), bytes_at(2), at(1), 0, 4, 64, 0, NULL), "overlaps");
    INVALID(mhc_ckpt_unpack(at(1), bytes_at(2) + 4, at(0), 0, 4, 64, 0, NULL), "aligned");
}

static void mix(void)
{
    mhc_proj_opts o;
    CHECK(mhc_proj_opts_default(&o) == MHC_OK);
    CHECK(mhc_stream_mix_ckpt(NULL, NULL, NULL, NULL, NULL, NULL, 0, 4, 8, 0, &o, NULL) == MHC_OK);
    CHECK(mhc_stream_mix_bwd_ckpt(NULL, NULL, NULL, NULL, NULL, NULL, 0, 4, 8, 1, NULL) == MHC_OK);
    CHECK(mhc_stream_mix_ckpt(at(0), floats_at(1), NULL, at(2), at(3), bytes_at(4), 5, 2, 64, 0, NULL, NULL) ==
          MHC_ERR_UNSUPPORTED);
    INVALID(mhc_stream_mix_ckpt(at(0), floats_at(1), NULL, at(2), at(3), bytes_at(4), MHC_MAX_TOKENS + 1, 4, 64, 0,
                                NULL, NULL), "out of range");
    INVALID(mhc_stream_mix_ckpt(at(0), floats_at(1), NULL, at(2), at(3), bytes_at(4), 5, 4, INT64_MAX, 0, NULL, NULL),
            "multiple of 8");
    INVALID(mhc_stream_mix_ckpt(at(0), floats_at(1), NULL, at(2), at(0), bytes_at(4), 5, 4, 64, 0, NULL, NULL),
            "overlaps");
    /* H may be written over its own logits, but not over part of them */
    INVALID(mhc_stream_mix_ckpt(at(0), floats_at(1), floats_at(1) + 16, at(2), at(3), bytes_at(4), 5, 4, 64, 0, &o,
                                NULL), "overlaps");
    o.max_iters = 0;
    INVALID(mhc_stream_mix_ckpt(at(0), floats_at(1), floats_at(5), at(2), at(3), bytes_at(4), 5, 4, 64, 0, &o, NULL),
            "max_iters");
    INVALID(mhc_stream_mix_bwd_ckpt(at(0), bytes_at(1), floats_at(2), at(3), at(3), floats_at(5), 5, 4, 64, 0, NULL),
            "overlaps");
    INVALID(mhc_stream_mix_bwd_ckpt(at(0), NULL, floats_at(2), at(3), at(4), floats_at(5), 5, 4, 64, 0, NULL), "NULL");
}

static mhc_layer_args layer_args(int64_t T, int64_t C)
{
    mhc_layer_args a;
    memset(&a, 0, sizeof a);
    a.T = T;
    a.n = 4;
    a.C = C;
    a.eps = 1e-6f;
    a.x = at(0);
    a.W = at(1);
    a.f = at(2);
    a.u = at(3);
    a.x_out = at(4);
    a.rms = floats_at(5);
    a.logits = floats_at(6);
    a.H_pre = floats_at(7);
    a.H_post = floats_at(8);
    a.H_res = floats_at(9);
    a.grad_x_out = at(10);
    a.grad_u = at(11);
    a.grad_x = at(12);
    a.grad_f = at(13);
    a.grad_W = floats_at(14);
    a.grad_logits = floats_at(15);
    a.workspace = at(16);
    a.workspace_bytes = (int64_t)1 << 38;
    return a;
}

static void layer(void)
{
    mhc_layer_ckpt k = {MHC_CKPT_E4M3, NULL, NULL, NULL, NULL};
    mhc_layer_args a = layer_args(0, 64);
    CHECK(mhc_layer_fwd_ckpt(&a, &k, NULL) == MHC_OK);
    CHECK(mhc_layer_bwd_ckpt(&a, &k, NULL) == MHC_OK);
    CHECK(mhc_layer_read(&a, NULL, NULL, NULL) == MHC_OK);
    CHECK(mhc_layer_read_workspace_bytes(0, 4, 64) == 0);
    CHECK(mhc_layer_read_workspace_bytes(1, 4, 1 << 24) > 0);
    CHECK(mhc_layer_read_workspace_bytes(8192, 4, 2048) > 0 && mhc_layer_read_workspace_bytes(8193, 4, 2048) == 0);
    CHECK(mhc_layer_read_workspace_bytes(MHC_MAX_TOKENS, 4, 1 << 24) == 0);
    CHECK(mhc_layer_read_workspace_bytes(MHC_MAX_TOKENS + 1, 4, 64) == -1);
    CHECK(mhc_layer_ckpt_workspace_bytes(0, 4, 64) >= 0);
    CHECK(mhc_layer_ckpt_workspace_bytes(MHC_MAX_TOKENS, 4, 1 << 24) > 0);
    CHECK(mhc_layer_ckpt_workspace_bytes(INT64_MAX, 4, 64) == -1);
    CHECK(mhc_layer_ckpt_workspace_bytes(5, 4, INT64_MAX) == -1);

    a = layer_args(5, 64);
    k.x_codes = at(17);
    k.x_scales = bytes_at(18);
    k.f_codes = at(19);
    k.f_scales = bytes_at(20);
    INVALID(mhc_layer_fwd_ckpt(NULL, &k, NULL), "NULL");
    INVALID(mhc_layer_fwd_ckpt(&a, NULL, NULL), "NULL");
    INVALID(mhc_layer_bwd_ckpt(&a, NULL, NULL), "NULL");
    k.format = 9;
    INVALID(mhc_layer_fwd_ckpt(&a, &k, NULL), "format");
    INVALID(mhc_layer_bwd_ckpt(&a, &k, NULL), "format");
    k.format = MHC_CKPT_INT8;
    k.f_codes = k.x_codes;
    INVALID(mhc_layer_fwd_ckpt(&a, &k, NULL), "overlaps");
    INVALID(mhc_layer_bwd_ckpt(&a, &k, NULL), "overlaps");
    k.f_codes = at(19);
    a.workspace_bytes = 0;
    INVALID(mhc_layer_fwd_ckpt(&a, &k, NULL), "workspace_bytes");
    INVALID(mhc_layer_bwd_ckpt(&a, &k, NULL), "workspace_bytes");
    INVALID(mhc_layer_read(&a, NULL, NULL, NULL), "workspace_bytes");
    a = layer_args(5, 64);
    a.workspace = (char*)a.workspace + 16;
    INVALID(mhc_layer_bwd_ckpt(&a, &k, NULL), "256-byte aligned");
    a = layer_args(5, 64);
    INVALID(mhc_layer_read(&a, at(21), NULL, NULL), "together");
    a.u = NULL;
    INVALID(mhc_layer_read(&a, NULL, NULL, NULL), "u or u_codes");
    INVALID(mhc_layer_read(&a, at(21), bytes_at(0), NULL), "overlaps");
    a.eps = 0.f;
    INVALID(mhc_layer_read(&a, at(21), bytes_at(22), NULL), "eps");
    a = layer_args(5, 96);
    INVALID(mhc_layer_read(&a, NULL, NULL, NULL), "multiple of 64");
    a.n = 3;
    CHECK(mhc_layer_read(&a, NULL, NULL, NULL) == MHC_ERR_UNSUPPORTED);
}

static void quantisers(void)
{
    CHECK(mhc_mx4_quantize(NULL, 0, NULL, NULL, 0, 32, 1, NULL) == MHC_OK);
    CHECK(mhc_mx4_quantize_both(NULL, 0, NULL, NULL, NULL, NULL, 0, 32, NULL) == MHC_OK);
    CHECK(mhc_mx4_quantize_ckpt(NULL, 1, NULL, NULL, NULL, NULL, 0, 32, 1, NULL) == MHC_OK);
    CHECK(mhc_mx4_requantize(NULL, NULL, NULL, NULL, 0, 32, 0, NULL) == MHC_OK);
    CHECK(mhc_mx4_dequantize(NULL, NULL, NULL, 0, 0, 32, NULL) == MHC_OK);
    INVALID(mhc_mx4_quantize(at(0), 0, at(1), bytes_at(2), 32, 32, 2, NULL), "transpose");
    INVALID(mhc_mx4_quantize(at(0), 0, at(1), bytes_at(2), 32, 40, 0, NULL), "multiple of 32");
    INVALID(mhc_mx4_quantize(at(0), 0, at(1), bytes_at(2), 33, 40, 1, NULL), "R must");
    INVALID(mhc_mx4_quantize(at(0), 0, at(1), bytes_at(2), INT64_MAX, 64, 0, NULL), "out of range");
    INVALID(mhc_mx4_quantize_both(at(0), 0, at(1), bytes_at(2), at(3), bytes_at(4), 48, 64, NULL), "R must");
    INVALID(mhc_mx4_quantize_both(at(0), 0, at(1), bytes_at(2), at(1), bytes_at(4), 64, 64, NULL), "overlaps");
    INVALID(mhc_mx4_quantize_both(at(0), 0, at(1), bytes_at(2), at(3), NULL, 64, 64, NULL), "NULL");
    INVALID(mhc_mx4_quantize_ckpt(at(0), 0, at(1), bytes_at(2), at(0), bytes_at(4), 4, 64, 0, NULL), "overlaps");
    INVALID(mhc_mx4_quantize_ckpt(at(0), 0, at(1), bytes_at(2), at(3), bytes_at(4), 4, 64, 5, NULL), "format");
    INVALID(mhc_mx4_requantize(at(0), bytes_at(1), at(2), bytes_at(3), 40, 64, 0, NULL), "R must");
    INVALID(mhc_mx4_requantize(at(0), bytes_at(1), at(0), bytes_at(3), 64, 64, 0, NULL), "overlaps");
    INVALID(mhc_mx4_requantize(at(0), bytes_at(1), at(2), bytes_at(3), 32, (int64_t)1 << 24, 0, NULL), "out of range");
    INVALID(mhc_mx4_dequantize(at(0), bytes_at(1), at(2), 3, 4, 64, NULL), "dtype");
    INVALID(mhc_mx4_dequantize(at(0), bytes_at(1), at(1), 0, 4, 64, NULL), "overlaps");
}

static void products(void)
{
    CHECK(mhc_mx4_matmul(NULL, NULL, NULL, NULL, NULL, 0, 0, 8, 32, NULL) == MHC_OK);
    CHECK(mhc_mx4_matmul_values(NULL, 1, NULL, NULL, NULL, 0, 0, 8, 32, NULL, 0, NULL) == MHC_OK);
    CHECK(mhc_mx4_write_back(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, 4, 8, 32, NULL) == MHC_OK);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(1, 8, 32) == 0);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(300, 8, 64) >= 300 * 34);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(MHC_MAX_TOKENS, 8, 1 << 24) > 0);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(INT64_MAX, 8, 64) == -1);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(4, INT64_MAX, 64) == -1);
    CHECK(mhc_mx4_matmul_values_workspace_bytes(4, 8, INT64_MAX) == -1);
    INVALID(mhc_mx4_matmul(at(0), bytes_at(1), at(2), bytes_at(3), at(4), 0, 4, 8, 40, NULL), "K must");
    INVALID(mhc_mx4_matmul(at(0), bytes_at(1), at(2), bytes_at(3), at(4), 0, 4, 9, 64, NULL), "N must");
    INVALID(mhc_mx4_matmul(at(0), bytes_at(1), at(2), bytes_at(3), at(4), 0, -4, 8, 64, NULL), "out of range");
    INVALID(mhc_mx4_matmul(at(0), bytes_at(1), at(2), bytes_at(3), at(2), 0, 4, 8, 64, NULL), "overlaps");
    INVALID(mhc_mx4_matmul(at(0), bytes_at(1) + 1, at(2), bytes_at(3), at(4), 0, 4, 8, 64, NULL), "aligned");
    INVALID(mhc_mx4_matmul_values(at(0), 0, at(2), bytes_at(3), at(4), 0, 300, 8, 64, NULL, 1 << 20, NULL), "NULL");
    INVALID(mhc_mx4_matmul_values(at(0), 0, at(2), bytes_at(3), at(4), 0, 300, 8, 64, at(5), 10, NULL),
            "workspace_bytes");
    INVALID(mhc_mx4_matmul_values(at(0), 7, at(2), bytes_at(3), at(4), 0, 300, 8, 64, at(5), 1 << 20, NULL), "dtype");
    CHECK(mhc_mx4_write_back(at(0), bytes_at(1), at(2), bytes_at(3), at(4), floats_at(5), floats_at(6), at(7), NULL, 4,
                             2, 8, 64, NULL) == MHC_ERR_UNSUPPORTED);
    INVALID(mhc_mx4_write_back(at(0), bytes_at(1), at(2), bytes_at(3), at(4), floats_at(5), floats_at(6), at(4), NULL,
                               4, 4, 8, 64, NULL), "overlaps");
    INVALID(mhc_mx4_write_back(at(0), bytes_at(1), at(2), bytes_at(3), at(4), NULL, floats_at(6), at(7), at(8), 4, 4, 8,
                               64, NULL), "NULL");
}

int main(void)
{
    checkpoints();
    mix();
    layer();
    quantisers();
    products();
    if (failures == 0) printf("c packed ok\n");
    return failures;
}
