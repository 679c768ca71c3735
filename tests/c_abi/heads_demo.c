/* The operators on heads and the orthogonalised update from C: a norm of each
 * head with its rotation, its backward pass, a rotation and back, and
 * Newton-Schulz steps, checked on the host in double. */
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "ar.h"

enum { TOKENS = 3, QH = 4, KH = 2, D = 24, ROT = 16, EACH = QH + KH, ALL = TOKENS * EACH * D, M = 5, N = 9 };

static void ok(int status, const char* what)
{
    if (status != 0) {
        printf("%s: %s\n", what, ar_status_string(status));
        exit(1);
    }
}

static void hip(hipError_t e, const char* what)
{
    if (e != hipSuccess) {
        printf("%s: hipError %d\n", what, (int)e);
        exit(1);
    }
}

static void* on_device(const void* host, size_t bytes)
{
    void* p = NULL;
    hip(hipMalloc(&p, bytes), "hipMalloc");
    if (host)
        hip(hipMemcpy(p, host, bytes, hipMemcpyHostToDevice), "hipMemcpy");
    return p;
}

static void near_to(const void* device, const double* want, size_t n, const char* what)
{
    float got[ALL];
    hip(hipMemcpy(got, device, n * sizeof(float), hipMemcpyDeviceToHost), "hipMemcpy");
    for (size_t i = 0; i < n; ++i)
        if (fabs(got[i] - want[i]) > 1e-5 * (fabs(want[i]) + 1.0)) {
            printf("%s[%zu]: %g, not %g\n", what, i, got[i], want[i]);
            exit(1);
        }
}

static float draw(void)
{
    static unsigned s = 1;
    return (float)((s = s * 1664525u + 1013904223u) >> 8) / (1 << 23) - 1.0f;
}

static void turn(double* v, double at, const double* f, double sign)
{
    for (int i = 0; i < ROT / 2; ++i) {
        const double c = cos(at * f[i]), s = sign * sin(at * f[i]), a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = c * a - s * b;
        v[2 * i + 1] = c * b + s * a;
    }
}

/* One token's heads are a row of EACH * D: the queries', then the keys'. */
static ar_heads_t heads(void* p, int first)
{
    ar_heads_t h = {(float*)p + first * D, (size_t)TOKENS * EACH * D, EACH * D, D};
    return h;
}

int main(void)
{
    float x[ALL], dy[ALL], w[2][D], m[M * N];
    double f[ROT / 2], factor, y[ALL], dx[ALL], turned[ALL], dw[2][D] = {{0}}, z[M * N], a[M * M], q[M * M];
    const int positions[TOKENS] = {-3, 70000, 5};
    ar_rotary_scheme_t scheme = {0};
    scheme.rot_dim = ROT;
    scheme.base = 10000.0;
    ok(ar_rotary_frequencies(&scheme, f, &factor), "ar_rotary_frequencies");
    if (factor != 1.0 || f[0] != 1.0 || fabs(f[1] - pow(10000.0, -2.0 / ROT)) > 1e-15)
        return 1;
    for (int i = 0; i < ALL; ++i) {
        x[i] = draw();
        dy[i] = draw();
    }
    for (int i = 0; i < 2 * D; ++i)
        w[i / D][i % D] = 1.0f + 0.5f * draw();
    for (int h = 0; h < TOKENS * EACH; ++h) {
        const int k = h % EACH >= QH;
        const double at = positions[h / EACH];
        double ms = 0.0, mean = 0.0, u[D];
        for (int i = 0; i < D; ++i)
            ms += (double)x[h * D + i] * x[h * D + i] / D;
        const double r = 1.0 / sqrt(ms + 1e-6);
        for (int i = 0; i < D; ++i) {
            y[h * D + i] = x[h * D + i] * r * w[k][i];
            turned[h * D + i] = x[h * D + i];
            u[i] = dy[h * D + i];
        }
        turn(y + h * D, at, f, 1.0);
        turn(turned + h * D, at, f, 1.0);
        turn(u, at, f, -1.0);
        for (int i = 0; i < D; ++i)
            mean += u[i] * w[k][i] * x[h * D + i] * r / D;
        for (int i = 0; i < D; ++i) {
            dx[h * D + i] = r * (u[i] * w[k][i] - x[h * D + i] * r * mean);
            dw[k][i] += u[i] * x[h * D + i] * r;
        }
    }

    ar_rotation_t rotation = {0};
    rotation.rot_dim = ROT;
    rotation.layout = AR_ROTARY_PAIRS;
    rotation.factor = (float)factor;
    rotation.frequencies = on_device(f, sizeof f);
    rotation.positions = on_device(positions, sizeof positions);
    rotation.position_bytes = 4;
    void *d_x = on_device(x, sizeof x), *d_y = on_device(NULL, sizeof x), *d_dy = on_device(dy, sizeof dy);
    float *d_w = on_device(w, sizeof w), *d_dw = on_device(NULL, sizeof w);

    ar_head_rmsnorm_t n = {0};
    n.dtype = n.weight_dtype = AR_FLOAT32;
    n.eps = 1e-6f;
    n.batch = 1;
    n.tokens = TOKENS;
    n.q_heads = QH;
    n.k_heads = KH;
    n.dim = D;
    n.rotation = rotation;
    n.q = heads(d_x, 0);
    n.k = heads(d_x, QH);
    n.q_out = heads(d_y, 0);
    n.k_out = heads(d_y, QH);
    n.q_weight = d_w;
    n.k_weight = d_w + D;
    ok(ar_head_rmsnorm(&n, NULL), "ar_head_rmsnorm");
    near_to(d_y, y, ALL, "y");

    ar_head_rmsnorm_backward_t b = {0};
    b.dtype = b.weight_dtype = AR_FLOAT32;
    b.ranks = 1;
    b.eps = 1e-6f;
    b.batch = 1;
    b.tokens = TOKENS;
    b.q_heads = QH;
    b.k_heads = KH;
    b.dim = D;
    b.rotation = rotation;
    b.q = n.q;
    b.k = n.k;
    b.dq = b.dq_out = heads(d_dy, 0); /* the gradients in place */
    b.dk = b.dk_out = heads(d_dy, QH);
    b.q_weight = d_w;
    b.k_weight = d_w + D;
    b.q_dweight = d_dw;
    b.k_dweight = d_dw + D;
    b.workspace_bytes = ar_head_rmsnorm_backward_workspace(1, D);
    b.workspace = on_device(NULL, b.workspace_bytes);
    ok(ar_head_rmsnorm_backward(&b, NULL), "ar_head_rmsnorm_backward");
    near_to(d_dy, dx, ALL, "dx");
    near_to(d_dw, dw[0], 2 * D, "dweight");

    ar_rotary_t r = {0};
    r.dtype = AR_FLOAT32;
    r.batch = 1;
    r.tokens = TOKENS;
    r.q_heads = QH;
    r.k_heads = KH;
    r.dim = D;
    r.rotation = rotation;
    r.q = r.q_out = heads(d_x, 0);
    r.k = r.k_out = heads(d_x, QH);
    ok(ar_rotary(&r, NULL), "ar_rotary");
    near_to(d_x, turned, ALL, "turned");
    r.inverse = 1;
    ok(ar_rotary(&r, NULL), "ar_rotary, inverse");
    for (int i = 0; i < ALL; ++i)
        turned[i] = x[i];
    near_to(d_x, turned, ALL, "turned back");
    r.rotation.rot_dim = ROT - 1;
    if (ar_rotary(&r, NULL) != AR_ERR_INVALID_ARG)
        return 1;

    const float coefficients[3][3] = {{3.4445f, -4.7750f, 2.0315f}, {1.875f, -1.25f, 0.375f}, {1.5f, -0.5f, 0.0f}};
    double size = 0.0;
    for (int i = 0; i < M * N; ++i) {
        m[i] = draw();
        size += (double)m[i] * m[i];
    }
    for (int i = 0; i < M * N; ++i)
        z[i] = m[i] / (sqrt(size) + 1e-7);
    for (int s = 0; s < 3; ++s) {
        double out[M * N];
        for (int i = 0; i < M * M; ++i) {
            a[i] = 0.0;
            for (int j = 0; j < N; ++j)
                a[i] += z[i / M * N + j] * z[i % M * N + j];
        }
        for (int i = 0; i < M * M; ++i) {
            q[i] = coefficients[s][1] * a[i];
            for (int j = 0; j < M; ++j)
                q[i] += coefficients[s][2] * a[i / M * M + j] * a[j * M + i % M];
        }
        for (int i = 0; i < M * N; ++i) {
            out[i] = coefficients[s][0] * z[i];
            for (int j = 0; j < M; ++j)
                out[i] += q[i / N * M + j] * z[j * N + i % N];
        }
        for (int i = 0; i < M * N; ++i)
            z[i] = out[i];
    }
    void* d_m = on_device(m, sizeof m);
    const void* in[1] = {d_m};
    void* out[1] = {d_m};
    ar_orthogonalize_t o = {0};
    o.dtype = AR_FLOAT32;
    o.steps = 3;
    o.eps = 1e-7f;
    o.scale = 2.0f;
    o.count = 1;
    o.rows = M;
    o.cols = o.x_stride = o.out_stride = N;
    o.x = in;
    o.out = out;
    o.coefficients = coefficients[0];
    o.workspace_bytes = ar_orthogonalize_workspace(1, M, N);
    o.workspace = on_device(NULL, o.workspace_bytes);
    ok(ar_orthogonalize(&o, NULL), "ar_orthogonalize");
    for (int i = 0; i < M * N; ++i)
        z[i] *= 2.0;
    near_to(d_m, z, M * N, "orthogonalised");
    printf("ok\n");
    return 0;
}
