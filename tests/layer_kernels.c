/* Which kernels libmxfp4_layer's host code launches, without a GPU: the program's own hipGetDevice, device properties and
 * hipLaunchKernel stand in for the runtime's. Each line of stdin is a call: a name, rows, columns, what the row strides have more than
 * the columns, by how many elements pointers are off a multiple of 4096 bytes, the types of the call's two inputs (0 bf16, 1 FP32), and
 * whether codes are wanted (1 along the rows, 2 along the columns, 3 both). It prints the status and the kernels' host addresses,
 * which are only good for a comparison. Pointers are never followed on the host. */
#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <string.h>

#include "../include/mxfp4_layer.h"

static const void *launched[16];
static int launches;

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
    (void)grid, (void)block, (void)args, (void)shared, (void)stream;
    if (launches < 16) launched[launches++] = f;
    return hipSuccess;
}

static long long up(long long v, long long to) { return (v + to - 1) / to * to; }

int main(void)
{
    char name[32];
    long long rows, cols, pad, off;
    int ta, tb, codes;
    while (scanf("%31s %lld %lld %lld %lld %d %d %d", name, &rows, &cols, &pad, &off, &ta, &tb, &codes) == 8) {
        char *const base = (char *)(1 << 20);
        char *a = base + off * (ta ? 4 : 2), *b = base + off * (tb ? 4 : 2), *to = base + (1 << 19);
        uint8_t *q1 = codes & 1 ? (uint8_t *)base : NULL, *q0 = codes & 2 ? (uint8_t *)base : NULL, *s = (uint8_t *)base;
        const long long ld = cols + pad, ld1 = up(cols, 128), ld0 = up(rows, 128);
        const int wide = codes ? 0 : 1;
        int status = -1, k;
        launches = 0;
        if (!strcmp(name, "norm"))
            status = mxfp4_rmsnorm_forward(a, ta, ld, b, ld, tb, NULL, 0, rows, cols, 1e-5f, to, cols, (float *)base, wide ? base : NULL,
                                           MXFP4_OUT_BF16, cols, q1, ld1, s, ld1 / 128, q0, ld0, s, ld0 / 128, NULL);
        else if (!strcmp(name, "normgrad"))
            status = mxfp4_rmsnorm_backward(a, ta, ld, b, ld, b, ld, tb, NULL, 0, (float *)base, rows, cols, to, cols, NULL, 0, NULL, 0, NULL);
        else if (!strcmp(name, "gate"))
            status = mxfp4_swiglu_forward(a, ld, a, ld, ta, rows, cols, wide ? to : NULL, MXFP4_OUT_BF16, cols, q1, ld1, s, ld1 / 128, q0, ld0, s,
                                          ld0 / 128, NULL);
        else if (!strcmp(name, "gategrad"))
            status = mxfp4_swiglu_backward(a, ta, ld, b, ld, b, ld, tb, rows, cols, wide ? to : NULL, cols, wide ? to + 4096 : NULL, cols,
                                           MXFP4_OUT_BF16, q1, q1, ld1, s, s, ld1 / 128, q0, q0, ld0, s, s, ld0 / 128, NULL);
        printf("%d", status);
        for (k = 0; k < launches; ++k) printf(" %p", launched[k]);
        printf("\n");
    }
    return 0;
}
