/*
 * A C99 user of the embedding and of the loss under an output head in
 * include/df11.h: the sizes and refusals that need no GPU; built with
 * -DDF11_C_CHECK_GPU it also runs a lookup, its gradient, and the loss of a head
 * in two pieces with its gradients, and compares every result with plain loops in
 * double precision.
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

enum { ROWS = 50, COLS = 24, TOKENS = 7, FIRST = 30 };

#ifdef DF11_C_CHECK_GPU
static void *upload(const void *host, size_t bytes) {
    void *p = NULL;
    if (hipMalloc(&p, bytes) != hipSuccess || hipMemcpy(p, host, bytes, hipMemcpyHostToDevice) != hipSuccess)
        exit(2);
    return p;
}

static void *room(size_t bytes) {
    void *p = NULL;
    if (hipMalloc(&p, bytes) != hipSuccess) exit(2);
    return p;
}

static void download(void *host, const void *p, size_t bytes) {
    if (hipMemcpy(host, p, bytes, hipMemcpyDeviceToHost) != hipSuccess) exit(2);
}

/* A random float that BF16 holds, and its pattern. */
static float value(uint64_t *s, uint16_t *bits) {
    *s = *s * 6364136223846793005ull + 1442695040888963407ull;
    const float x = (float)((*s >> 40) & 0xFFFF) / 65536.0f - 0.5f;
    uint32_t u;
    memcpy(&u, &x, 4);
    u &= 0xFFFF0000u;
    *bits = (uint16_t)(u >> 16);
    float r;
    memcpy(&r, &u, 4);
    return r;
}

static int on_the_gpu(void) {
    static float w[ROWS][COLS], x[TOKENS][COLS];
    static uint16_t wb[ROWS][COLS], xb[TOKENS][COLS];
    const int64_t tokens[TOKENS] = {3, 49, 3, 0, 17, 3, 31}, targets[TOKENS] = {49, 0, -100, 3, 29, 30, 3};
    uint64_t seed = 1;
    for (int r = 0; r < ROWS; r++)
        for (int c = 0; c < COLS; c++) w[r][c] = value(&seed, &wb[r][c]);
    for (int t = 0; t < TOKENS; t++)
        for (int c = 0; c < COLS; c++) x[t][c] = value(&seed, &xb[t][c]);
    void *d_w = upload(wb, sizeof wb), *d_x = upload(xb, sizeof xb);
    void *d_tokens = upload(tokens, sizeof tokens), *d_targets = upload(targets, sizeof targets);

    df11_embedding_lookup e;
    memset(&e, 0, sizeof e);
    static float y[TOKENS][COLS];
    e.table = d_w, e.tokens = d_tokens, e.out = room(sizeof y);
    e.table_stride = e.out_stride = COLS, e.rows = ROWS, e.n = TOKENS, e.cols = COLS;
    e.table_type = DF11_TYPE_BF16, e.out_type = DF11_TYPE_F32, e.token_bits = 64, e.scale = 1.5f;
    CHECK(df11_embedding(&e, NULL) == DF11_OK);
    download(y, e.out, sizeof y);
    for (int t = 0; t < TOKENS; t++)
        for (int c = 0; c < COLS; c++) CHECK(y[t][c] == 1.5f * w[tokens[t]][c]);

    df11_embedding_grad g;
    memset(&g, 0, sizeof g);
    static float dw[ROWS][COLS];
    g.tokens = d_tokens, g.dy = d_x, g.dw = room(sizeof dw);
    g.dy_stride = g.dw_stride = COLS, g.rows = ROWS, g.n = TOKENS, g.padding = 17, g.cols = COLS;
    g.dy_type = DF11_TYPE_BF16, g.dw_type = DF11_TYPE_F32, g.token_bits = 64, g.scale = 1.0f;
    CHECK(df11_embedding_gradient_scratch_bytes(TOKENS, ROWS, COLS) == 0);
    CHECK(df11_embedding_gradient(&g, NULL, 0, NULL) == DF11_OK);
    download(dw, g.dw, sizeof dw);
    for (int r = 0; r < ROWS; r++)
        for (int c = 0; c < COLS; c++) {
            float sum = 0.0f; /* in the order of the positions */
            for (int t = 0; t < TOKENS; t++)
                if (tokens[t] == r && r != 17) sum += x[t][c];
            CHECK(dw[r][c] == sum);
        }
    printf("embedding: %d tokens of %d rows, bit-exact\n", TOKENS, ROWS);

    /* the head in two pieces, the second one first */
    static float losses[TOKENS], lse[TOKENS], dx[TOKENS][COLS];
    df11_vocab_sizes z;
    memset(&z, 0, sizeof z);
    z.n = TOKENS, z.cols = COLS, z.rows = FIRST, z.dx = 1, z.two_terms = 1;
    df11_vocab_piece p;
    memset(&p, 0, sizeof p);
    p.x = d_x, p.targets = d_targets, p.x_stride = p.w_stride = COLS, p.ignored = -100;
    p.n = TOKENS, p.cols = COLS, p.vocab = ROWS, p.target_bits = 64;
    df11_vocab_grad v;
    memset(&v, 0, sizeof v);
    const uint64_t bytes = df11_vocab_loss_scratch_bytes(&z), more = df11_vocab_loss_gradient_scratch_bytes(&z);
    void *scratch = room(bytes > more ? bytes : more);
    float *d_losses = room(sizeof losses), *d_lse = room(sizeof lse), *d_dw = room(sizeof dw);
    v.lse = d_lse, v.dx = room(sizeof dx), v.dx_stride = v.dw_stride = COLS, v.loss_grad_all = 0.25f;
    v.dx_type = v.dw_type = DF11_TYPE_F32;
    for (int pass = 0; pass < 2; pass++)
        for (int k = 1; k >= 0; k--) {
            p.first = k ? FIRST : 0, p.rows = k ? ROWS - FIRST : FIRST, p.begin = k, p.end = !k;
            p.w = (const uint16_t *)d_w + (size_t)p.first * COLS;
            v.dw = d_dw + (size_t)p.first * COLS;
            CHECK((pass ? df11_vocab_loss_gradient(&p, &v, &z, scratch, more, NULL)
                        : df11_vocab_loss(&p, d_losses, d_lse, &z, scratch, bytes, NULL)) == DF11_OK);
        }
    download(losses, d_losses, sizeof losses);
    download(lse, d_lse, sizeof lse);
    download(dx, v.dx, sizeof dx);
    download(dw, d_dw, sizeof dw);
    static double want_dw[ROWS][COLS];
    for (int t = 0; t < TOKENS; t++) {
        double l[ROWS], sum = 0.0, want[COLS] = {0};
        for (int r = 0; r < ROWS; r++) {
            l[r] = 0.0;
            for (int c = 0; c < COLS; c++) l[r] += (double)x[t][c] * w[r][c];
            sum += exp(l[r]);
        }
        CHECK(fabs(lse[t] - log(sum)) < 1e-5);
        CHECK(targets[t] < 0 ? losses[t] == 0.0f : fabs(losses[t] - (log(sum) - l[targets[t]])) < 1e-5);
        for (int r = 0; r < ROWS && targets[t] >= 0; r++) {
            const double q = 0.25 * (exp(l[r]) / sum - (r == targets[t]));
            for (int c = 0; c < COLS; c++) want[c] += q * w[r][c], want_dw[r][c] += q * x[t][c];
        }
        for (int c = 0; c < COLS; c++) CHECK(fabs(dx[t][c] - want[c]) < 1e-5);
    }
    for (int r = 0; r < ROWS; r++)
        for (int c = 0; c < COLS; c++) CHECK(fabs(dw[r][c] - want_dw[r][c]) < 1e-5);
    printf("loss: %d tokens under %d rows in two pieces, with both gradients\n", TOKENS, ROWS);
    return 0;
}
#endif

int main(void) {
    df11_embedding_lookup e;
    df11_embedding_grad g;
    df11_vocab_piece p;
    df11_vocab_grad v;
    df11_vocab_sizes z;
    memset(&e, 0, sizeof e);
    memset(&g, 0, sizeof g);
    memset(&p, 0, sizeof p);
    memset(&v, 0, sizeof v);
    memset(&z, 0, sizeof z);
    e.token_bits = g.token_bits = p.target_bits = 64;
    p.vocab = 1;
    /* nothing to do */
    CHECK(df11_embedding(&e, NULL) == DF11_OK);
    CHECK(df11_embedding_gradient(&g, NULL, 0, NULL) == DF11_OK);
    CHECK(df11_vocab_loss(&p, NULL, NULL, &z, NULL, 0, NULL) == DF11_OK);
    /* refused */
    e.n = e.rows = TOKENS, e.cols = COLS;
    CHECK(df11_embedding(&e, NULL) == DF11_E_INVALID);
    g.rows = ROWS, g.cols = COLS;
    CHECK(df11_embedding_gradient(&g, NULL, 0, NULL) == DF11_E_INVALID);
    p.n = TOKENS;
    CHECK(df11_vocab_loss(&p, NULL, NULL, NULL, NULL, 0, NULL) == DF11_E_INVALID);
    CHECK(df11_vocab_loss_gradient(&p, &v, &z, NULL, 0, NULL) == DF11_E_INVALID);
    z.n = DF11_VOCAB_MAX_TOKENS + 1;
    CHECK(df11_vocab_loss_scratch_bytes(&z) == 0 && df11_vocab_loss_gradient_scratch_bytes(&z) == 0);
    /* sizes */
    CHECK(df11_embedding_gradient_scratch_bytes(2048, ROWS, COLS) == 0);
    CHECK(df11_embedding_gradient_scratch_bytes(5000, ROWS, COLS) >= 5000 * 16);
    z.n = TOKENS, z.cols = COLS, z.rows = ROWS;
    CHECK(df11_vocab_loss_scratch_bytes(&z) >= TOKENS * 12);
    CHECK(df11_vocab_loss_gradient_scratch_bytes(&z) >= TOKENS * 2 * (COLS + ROWS));
    printf("vocabulary: sizes and refusals\n");
#ifdef DF11_C_CHECK_GPU
    if (on_the_gpu()) return 1;
#endif
    return 0;
}
