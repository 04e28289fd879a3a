/*
 * A C99 user of the operators on uncompressed weights in include/df11.h: the
 * sizes and refusals that need no GPU; built with -DDF11_C_CHECK_GPU it also
 * runs the gradient norm, AdamW steps (one of them skipped) and an int8 product
 * and compares every result with plain loops.
 * Exit status 0 on success; prints the first failed check otherwise.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "df11.h"

#ifdef DF11_C_CHECK_GPU
#include <hip/hip_runtime_api.h>
#endif

#define CHECK(c)                                                         \
    do {                                                                 \
        if (!(c)) {                                                      \
            fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
            return 1;                                                    \
        }                                                                \
    } while (0)

enum { N = 300, ROWS = 21, COLS = 37, TOKENS = 3 };

#ifdef DF11_C_CHECK_GPU
static void *upload(const void *host, size_t bytes) {
    void *p = NULL;
    if (hipMalloc(&p, bytes) != hipSuccess || hipMemcpy(p, host, bytes, hipMemcpyHostToDevice) != hipSuccess)
        exit(2);
    return p;
}

static void download(void *host, const void *p, size_t bytes) {
    if (hipMemcpy(host, p, bytes, hipMemcpyDeviceToHost) != hipSuccess) exit(2);
}

static float value(uint64_t *s) {
    *s = *s * 6364136223846793005ull + 1442695040888963407ull;
    return (float)((*s >> 40) & 0xFFFFFF) / 16777216.0f - 0.5f;
}

static int adamw_on_the_gpu(void) {
    static float w[N], g[N], m[N], v[N], got[N];
    uint64_t seed = 1;
    double squares = 0.0;
    for (int i = 0; i < N; i++) {
        w[i] = value(&seed);
        g[i] = value(&seed);
        squares += (double)g[i] * g[i];
    }
    const float nan_factor = (float)NAN;
    const uint64_t none = 0;
    float norm[2];
    df11_adamw_tensor t;
    memset(&t, 0, sizeof t);
    t.w = upload(w, sizeof w);
    t.g = upload(g, sizeof g);
    t.m = upload(m, sizeof m);
    t.v = upload(v, sizeof v);
    t.numel = N;
    t.lr_scale = 1.0;
    t.weight_decay = 0.1;
    float *d_norm = upload(norm, sizeof norm), *d_nan = upload(&nan_factor, sizeof nan_factor);
    uint64_t *d_count = upload(&none, sizeof none);
    const uint64_t bytes = df11_grad_norm_scratch_bytes(&t, 1);
    void *scratch = NULL;
    CHECK(hipMalloc(&scratch, bytes) == hipSuccess);
    CHECK(df11_grad_norm(DF11_TYPE_F32, &t, 1, 1.0, d_norm, scratch, bytes, NULL) == DF11_OK);
    df11_adamw_config c;
    memset(&c, 0, sizeof c);
    c.lr = 1e-2, c.beta1 = 0.9, c.beta2 = 0.95, c.eps = 1e-8, c.state_bits = 32;
    /* the second of three calls is skipped: its number is the third's */
    for (int call = 1; call <= 3; call++) {
        c.step = (uint64_t)call;
        c.d_grad_factor = call == 2 ? d_nan : d_norm + 1;
        CHECK(df11_adamw_step_counted(&c, &t, 1, d_count, NULL) == DF11_OK);
    }
    uint64_t skipped = 0;
    download(&skipped, d_count, sizeof skipped);
    CHECK(skipped == 1);
    download(norm, d_norm, sizeof norm);
    CHECK(norm[0] == (float)sqrt(squares) && norm[1] == (float)(1.0 / (sqrt(squares) + 1e-6)));
    const float b1 = (float)0.9, c1 = (float)(1.0 - 0.9), b2 = (float)0.95, c2 = (float)(1.0 - 0.95);
    for (int step = 1; step <= 2; step++) {
        const float root = (float)(1.0 / sqrt(1.0 - pow(0.95, step)));
        const float keep = (float)(1.0 - 1e-2 * 0.1), size = (float)(1e-2 / (1.0 - pow(0.9, step)));
        for (int i = 0; i < N; i++) {
            const float x = g[i] * norm[1];
            m[i] = m[i] * b1 + x * c1;
            v[i] = v[i] * b2 + (x * c2) * x;
            w[i] = w[i] * keep - m[i] / (sqrtf(v[i]) * root + (float)1e-8) * size;
        }
    }
    download(got, t.w, sizeof got);
    CHECK(memcmp(got, w, sizeof w) == 0);
    download(got, t.m, sizeof got);
    CHECK(memcmp(got, m, sizeof m) == 0);
    download(got, t.v, sizeof got);
    CHECK(memcmp(got, v, sizeof v) == 0);
    printf("AdamW: %d weights, two steps and a skipped one, bit-exact\n", N);
    return 0;
}

static void quantise(const float *x, int8_t *q, float *scale) {
    float a = 0.0f;
    for (int i = 0; i < COLS; i++) a = fabsf(x[i]) > a ? fabsf(x[i]) : a;
    *scale = a / 127.0f;
    for (int i = 0; i < COLS; i++) q[i] = (int8_t)nearbyint(127.0 * (double)x[i] / (double)a);
}

static int product_on_the_gpu(void) {
    static float w[ROWS][COLS], x[TOKENS][COLS], y[TOKENS][ROWS];
    static int8_t qw[ROWS][COLS], qx[TOKENS][COLS];
    static float sw[ROWS], sx[TOKENS];
    uint64_t seed = 2;
    for (int r = 0; r < ROWS; r++) {
        for (int i = 0; i < COLS; i++) w[r][i] = value(&seed);
        quantise(w[r], qw[r], &sw[r]);
    }
    for (int t = 0; t < TOKENS; t++) {
        for (int i = 0; i < COLS; i++) x[t][i] = value(&seed);
        quantise(x[t], qx[t], &sx[t]);
    }
    enum { STRIDE = 128 };
    df11_int8_rows rows;
    memset(&rows, 0, sizeof rows);
    void *codes = NULL, *scales = NULL, *out = NULL, *scratch = NULL;
    CHECK(hipMalloc(&codes, ROWS * STRIDE) == hipSuccess && hipMalloc(&scales, ROWS * 4) == hipSuccess &&
          hipMalloc(&out, sizeof y) == hipSuccess);
    rows.src = upload(w, sizeof w);
    rows.codes = codes;
    rows.scales = scales;
    rows.src_stride = COLS;
    rows.code_stride = STRIDE;
    rows.rows = ROWS;
    rows.cols = COLS;
    CHECK(df11_quantize_int8(DF11_TYPE_F32, &rows, 1, NULL) == DF11_OK);
    df11_int8_tensor t;
    memset(&t, 0, sizeof t);
    t.w = codes;
    t.w_scale = scales;
    t.x = upload(x, sizeof x);
    t.y = out;
    t.w_stride = STRIDE;
    t.x_stride = COLS;
    t.y_stride = ROWS;
    t.rows = ROWS;
    t.cols = COLS;
    const uint64_t bytes = df11_linear_int8_scratch_bytes(&t, 1, TOKENS);
    CHECK(bytes > 0 && hipMalloc(&scratch, bytes) == hipSuccess);
    CHECK(df11_linear_int8(DF11_TYPE_F32, DF11_TYPE_F32, &t, 1, TOKENS, scratch, bytes, NULL) == DF11_OK);
    download(y, out, sizeof y);
    for (int k = 0; k < TOKENS; k++)
        for (int r = 0; r < ROWS; r++) {
            int sum = 0;
            for (int i = 0; i < COLS; i++) sum += qx[k][i] * qw[r][i];
            const float want = ((float)sum * sx[k]) * sw[r];
            CHECK(y[k][r] == want);
        }
    printf("int8: %d tokens x %d rows, bit-exact\n", TOKENS, ROWS);
    return 0;
}
#endif

int main(void) {
    df11_adamw_tensor a;
    df11_adamw_config c;
    df11_int8_tensor q;
    df11_int8_rows r;
    memset(&a, 0, sizeof a);
    memset(&c, 0, sizeof c);
    memset(&q, 0, sizeof q);
    memset(&r, 0, sizeof r);
    c.lr = 1e-3, c.beta1 = 0.9, c.beta2 = 0.999, c.eps = 1e-8, c.step = 1, c.state_bits = 32;
    a.lr_scale = 1.0;
    uint64_t count = 0;
    /* nothing to do */
    CHECK(df11_adamw_step(&c, &a, 1, NULL) == DF11_OK);
    CHECK(df11_adamw_step_counted(&c, &a, 1, &count, NULL) == DF11_OK && count == 0);
    CHECK(df11_adamw_values(&a, 1, DF11_TYPE_BF16, NULL, NULL, NULL) == DF11_OK);
    CHECK(df11_quantize_int8(DF11_TYPE_BF16, &r, 1, NULL) == DF11_OK);
    CHECK(df11_gemm_int8(DF11_TYPE_F16, &q, 1, 5, NULL) == DF11_OK);
    CHECK(df11_linear_int8(DF11_TYPE_BF16, DF11_TYPE_BF16, NULL, 0, 5, NULL, 0, NULL) == DF11_OK);
    /* refused */
    a.numel = N;
    CHECK(df11_adamw_step(&c, &a, 1, NULL) == DF11_E_INVALID);
    CHECK(df11_adamw_step_counted(&c, &a, 1, NULL, NULL) == DF11_E_INVALID);
    CHECK(df11_grad_norm(DF11_TYPE_F32, &a, 1, 1.0, NULL, NULL, 0, NULL) == DF11_E_INVALID);
    CHECK(df11_adamw_values(&a, 1, DF11_TYPE_F16, NULL, NULL, NULL) == DF11_E_INVALID);
    q.rows = ROWS;
    q.cols = DF11_INT8_MAX_COLS + 1;
    CHECK(df11_gemm_int8(DF11_TYPE_F32, &q, 1, 5, NULL) == DF11_E_INVALID);
    r.rows = ROWS;
    CHECK(df11_quantize_int8(DF11_TYPE_F32, &r, 1, NULL) == DF11_E_INVALID);
    /* sizes */
    q.cols = COLS;
    CHECK(df11_linear_int8_scratch_bytes(&q, 1, 1) == 0);
    CHECK(df11_linear_int8_scratch_bytes(&q, 1, TOKENS) >= TOKENS * (COLS + 4));
    CHECK(df11_grad_norm_scratch_bytes(&a, 1) >= 8);
    printf("operators: sizes and refusals\n");
#ifdef DF11_C_CHECK_GPU
    if (adamw_on_the_gpu() || product_on_the_gpu()) return 1;
#endif
    return 0;
}
