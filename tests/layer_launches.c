/* Runs libmxfp4_layer's host code without a GPU: the program's own hipGetDevice, device properties and
 * hipLaunchKernel stand in for the runtime's. Each line of stdin is a call, for which it prints the status,
 * the launches, how many of those exceed what a grid may hold (fewer than 2^32 work-items along each axis, as the
 * HIP runtime checks), and the workspace that the call asked for. Pointers are never followed on the host. */
#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../include/mxfp4_layer.h"

static long launches, beyond;

hipError_t hipGetDevice(int *device)
{
    *device = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600 *prop, int device)
{
    (void)device;
    memset(prop, 0, sizeof *prop);
    strcpy(prop->gcnArchName, "gfx950");
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t shared, hipStream_t stream)
{
    const unsigned long long most = 0xFFFFFFFFull;
    (void)f, (void)args, (void)shared, (void)stream;
    ++launches;
    if (!grid.x || !grid.y || !grid.z || (unsigned long long)grid.x * block.x > most ||
        (unsigned long long)grid.y * block.y > most || (unsigned long long)grid.z * block.z > most || grid.y > 65535 ||
        grid.z > 65535 || block.x * block.y * block.z > 1024) {
        ++beyond;
        return hipErrorInvalidConfiguration;
    }
    return hipSuccess;
}

static long long up(long long v, long long to) { return (v + to - 1) / to * to; }

int main(void)
{
    char name[32];
    long long a, b, c;
    char *p = (char *)(1 << 12);
    const size_t big = (size_t)1 << 62;
    while (scanf("%31s %lld %lld %lld", name, &a, &b, &c) == 4) {
        /* a rows of b columns; c: 1 along the rows, 2 along the columns, 3 both. The clipping: a tensors of b values */
        uint8_t *q1 = c & 1 ? (uint8_t *)p : NULL, *q0 = c & 2 ? (uint8_t *)p : NULL;
        const long long ld1 = up(b, 128), ls1 = up(b, 128) / 128, ld0 = up(a, 128), ls0 = up(a, 128) / 128;
        int status = -1;
        size_t need = 0;
        launches = beyond = 0;
        if (!strcmp(name, "norm"))
            status = mxfp4_rmsnorm_forward(p, MXFP4_IN_BF16, b, p, b, MXFP4_IN_F32, p, MXFP4_IN_BF16, a, b, 1e-5f, p + 4096, b,
                                           (float *)p, p, MXFP4_OUT_BF16, b, q1, ld1, (uint8_t *)p, ls1, q0, ld0, (uint8_t *)p, ls0,
                                           NULL);
        else if (!strcmp(name, "normgrad")) {
            need = mxfp4_rmsnorm_backward_workspace_bytes(a, b);
            status = mxfp4_rmsnorm_backward(p, MXFP4_IN_BF16, b, NULL, 0, p, b, MXFP4_IN_BF16, p, MXFP4_IN_BF16, (float *)p, a, b, p, b,
                                            p, MXFP4_OUT_F32, p, need, NULL);
        } else if (!strcmp(name, "gate"))
            status = mxfp4_swiglu_forward(p, b, p, b, MXFP4_IN_BF16, a, b, NULL, MXFP4_OUT_BF16, 0, q1, ld1, (uint8_t *)p, ls1, q0, ld0,
                                          (uint8_t *)p, ls0, NULL);
        else if (!strcmp(name, "gategrad"))
            status = mxfp4_swiglu_backward(p, MXFP4_IN_F32, b, p, b, p, b, MXFP4_IN_BF16, a, b, NULL, 0, NULL, 0, MXFP4_OUT_BF16, q1, q1,
                                           ld1, (uint8_t *)p, (uint8_t *)p, ls1, q0, q0, ld0, (uint8_t *)p, (uint8_t *)p, ls0, NULL);
        else if (!strcmp(name, "clip") || !strcmp(name, "scale") || !strcmp(name, "sum")) {
            mxfp4_grad_t *g = calloc(a > 0 ? a : 1, sizeof *g);
            long long k;
            char *at = p;
            for (k = 0; k < a; ++k, at += 2 * b) g[k] = (mxfp4_grad_t){at, at, b, MXFP4_IN_BF16, MXFP4_OUT_BF16};
            need = mxfp4_grad_norm_workspace_bytes(g, a);
            if (name[1] == 'l')
                status = mxfp4_grad_clip(g, a, 1.0f, 0.0f, p, need, (float *)p, NULL);
            else if (name[1] == 'c')
                status = mxfp4_grad_scale(g, a, (double *)p, 1.0f, 0.0f, (float *)p, NULL);
            else
                status = mxfp4_grad_norm(g, a, p, need, (double *)p, (float *)p, NULL);
            free(g);
        }
        (void)big;
        printf("%d %ld %ld %zu\n", status, launches, beyond, need);
    }
    return 0;
}
