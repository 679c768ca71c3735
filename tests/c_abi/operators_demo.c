/* The operators from C: a norm with the residual's addition, its backward
 * pass, and the gradients' clipping, checked on the host in double. */
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "ar.h"

enum { ROWS = 3, COLS = 37 };

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

static float* on_device(const float* host, size_t n)
{
    float* p = NULL;
    hip(hipMalloc((void**)&p, n * sizeof(float)), "hipMalloc");
    if (host)
        hip(hipMemcpy(p, host, n * sizeof(float), hipMemcpyHostToDevice), "hipMemcpy");
    return p;
}

static void near_to(const float* got, const double* want, size_t n, const char* what)
{
    for (size_t i = 0; i < n; ++i)
        if (fabs(got[i] - want[i]) > 1e-5 * (fabs(want[i]) + 1.0)) {
            printf("%s[%zu]: %g, not %g\n", what, i, got[i], want[i]);
            exit(1);
        }
}

int main(void)
{
    float x[ROWS * COLS], res[ROWS * COLS], dy[ROWS * COLS], w[COLS], got[ROWS * COLS], norm;
    double y[ROWS * COLS], dx[ROWS * COLS], dw[COLS] = {0}, total = 0.0, c;
    unsigned s = 1;
    for (int i = 0; i < ROWS * COLS; ++i) {
        x[i] = (float)((s = s * 1664525u + 1013904223u) >> 8) / (1 << 23) - 1.0f;
        res[i] = (float)((s = s * 1664525u + 1013904223u) >> 8) / (1 << 23) - 1.0f;
        dy[i] = (float)((s = s * 1664525u + 1013904223u) >> 8) / (1 << 23) - 1.0f;
    }
    for (int i = 0; i < COLS; ++i)
        w[i] = 0.5f + i / (float)COLS;
    for (int t = 0; t < ROWS; ++t) {
        double ms = 0.0, m = 0.0;
        for (int i = t * COLS; i < (t + 1) * COLS; ++i)
            ms += ((double)x[i] + res[i]) * ((double)x[i] + res[i]) / COLS;
        const double r = 1.0 / sqrt(ms + 1e-6);
        for (int i = t * COLS; i < (t + 1) * COLS; ++i) {
            y[i] = ((double)x[i] + res[i]) * r * w[i % COLS];
            m += (double)dy[i] * y[i] / COLS;
        }
        for (int i = t * COLS; i < (t + 1) * COLS; ++i) {
            const double n = ((double)x[i] + res[i]) * r;
            dx[i] = r * ((double)dy[i] * w[i % COLS] - n * m);
            dw[i % COLS] += (double)dy[i] * n;
        }
    }
    for (int i = 0; i < ROWS * COLS; ++i)
        total += dx[i] * dx[i];
    for (int i = 0; i < COLS; ++i)
        total += dw[i] * dw[i];
    c = 0.5 / (sqrt(total) + 1e-6);
    for (int i = 0; i < ROWS * COLS; ++i)
        dx[i] *= c;
    for (int i = 0; i < COLS; ++i)
        dw[i] *= c;

    float *d_res = on_device(res, ROWS * COLS), *d_w = on_device(w, COLS),
          *d_y = on_device(NULL, ROWS * COLS), *d_rstd = on_device(NULL, ROWS),
          *d_dx = on_device(dy, ROWS * COLS), *d_dw = on_device(NULL, COLS),
          *d_norm = on_device(NULL, 1);
    ar_rmsnorm_t f = {0};
    f.dtype = f.out_dtype = f.weight_dtype = AR_FLOAT32;
    f.eps = 1e-6f;
    f.rows = ROWS;
    f.cols = COLS;
    f.x = on_device(x, ROWS * COLS);
    f.residual = f.sum = d_res; /* the residual becomes the sum */
    f.weight = d_w;
    f.y = d_y;
    f.rstd = d_rstd;
    f.x_stride = f.residual_stride = f.sum_stride = f.y_stride = COLS;
    ok(ar_rmsnorm(&f, NULL), "ar_rmsnorm");

    ar_rmsnorm_backward_t b = {0};
    b.dtype = b.weight_dtype = AR_FLOAT32;
    b.ranks = 1;
    b.rows = ROWS;
    b.cols = COLS;
    b.dy = b.dx = d_dx; /* dy becomes dx */
    b.x = d_res;
    b.weight = d_w;
    b.rstd = d_rstd;
    b.dy_stride = b.x_stride = b.dx_stride = COLS;
    b.dweight = d_dw;
    b.workspace_bytes = ar_rmsnorm_backward_workspace(1, ROWS, COLS);
    hip(hipMalloc(&b.workspace, b.workspace_bytes), "hipMalloc");
    ok(ar_rmsnorm_backward(&b, NULL), "ar_rmsnorm_backward");

    ar_comm_t comm = NULL;
    void* ws = NULL;
    ok(ar_init(&comm, 2, 1, AR_FLOAT32, AR_RING, AR_SIMPLE), "ar_init");
    hip(hipMalloc(&ws, ar_workspace_bytes(comm)), "hipMalloc");
    ok(ar_set_workspace(comm, ws, ar_workspace_bytes(comm), NULL), "ar_set_workspace");
    ar_span_t grads[2] = {{d_dx, ROWS * COLS, AR_FLOAT32}, {d_dw, COLS, AR_FLOAT32}};
    ok(ar_grad_norm(comm, grads, 2, d_norm, NULL), "ar_grad_norm");
    ok(ar_grad_clip(grads, grads, 2, d_norm, 0.5f, NULL), "ar_grad_clip");
    hip(hipDeviceSynchronize(), "hipDeviceSynchronize");

    hip(hipMemcpy(got, d_y, sizeof got, hipMemcpyDeviceToHost), "hipMemcpy");
    near_to(got, y, ROWS * COLS, "y");
    hip(hipMemcpy(got, d_dx, sizeof got, hipMemcpyDeviceToHost), "hipMemcpy");
    near_to(got, dx, ROWS * COLS, "dx");
    hip(hipMemcpy(got, d_dw, COLS * sizeof(float), hipMemcpyDeviceToHost), "hipMemcpy");
    near_to(got, dw, COLS, "dweight");
    hip(hipMemcpy(&norm, d_norm, sizeof norm, hipMemcpyDeviceToHost), "hipMemcpy");
    if (fabs(norm - sqrt(total)) > 1e-5 * sqrt(total)) {
        printf("norm: %g, not %g\n", norm, sqrt(total));
        return 1;
    }
    ok(ar_destroy(comm), "ar_destroy");
    printf("ok\n");
    return 0;
}
