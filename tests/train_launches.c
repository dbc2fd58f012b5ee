/* Runs libmxfp4_train's host code without a GPU: the program's own hipGetDevice, device properties and
 * hipLaunchKernel stand in for the runtime's. Each line of stdin is a call, for which it prints the status,
 * the launches, how many of those exceed what a grid may hold (fewer than 2^32 work-items along each axis, as the
 * HIP runtime checks), and the workspace that the call asked for. Pointers are never followed on the host. */
#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <string.h>

#include "../include/mxfp4_train.h"

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
        grid.z > 65535) {
        ++beyond;
        return hipErrorInvalidConfiguration;
    }
    return hipSuccess;
}

int main(void)
{
    char name[32];
    long long a, b, c;
    void *p = (void *)(1 << 12);
    const size_t big = (size_t)1 << 62;
    while (scanf("%31s %lld %lld %lld", name, &a, &b, &c) == 4) {
        int status = -1;
        size_t need = 0;
        launches = beyond = 0;
        if (!strcmp(name, "quantize1")) {   /* rows, columns: along the rows */
            status = mxfp4_fp8_quantize(p, MXFP4_IN_BF16, a, b, b, MXFP4_FP8_ROW, p, (b + 127) / 128 * 128, p, (b + 127) / 128,
                                        NULL, 0, NULL, 0, NULL);
        } else if (!strcmp(name, "quantize0")) {
            status = mxfp4_fp8_quantize(p, MXFP4_IN_BF16, a, b, b, MXFP4_FP8_TILE, NULL, 0, NULL, 0, p, (a + 127) / 128 * 128, p,
                                        (a + 127) / 128, NULL);
        } else if (!strcmp(name, "gemm")) {   /* M, N, K */
            const long long lds = (c + 2047) / 2048 * 16;
            need = mxfp4_fp8_gemm_workspace_bytes(a, b, c);
            status = mxfp4_fp8_gemm(p, (c + 127) / 128 * 128, p, lds, p, (c + 127) / 128 * 128, p, lds, a, b, c, 1.0f, 0.0f, p,
                                    MXFP4_OUT_BF16, b, need ? p : NULL, need, NULL);
        } else if (!strcmp(name, "fprop")) {   /* M, K, N */
            need = mxfp4_fp8_linear_workspace_bytes(MXFP4_FPROP, a, b, c);
            status = mxfp4_fp8_linear_fprop(p, p, a, b, c, p, big, p, MXFP4_OUT_F32, NULL);
        } else if (!strcmp(name, "wgrad")) {
            need = mxfp4_fp8_linear_workspace_bytes(MXFP4_WGRAD, a, b, c);
            status = mxfp4_fp8_linear_wgrad(p, p, a, b, c, p, big, p, MXFP4_OUT_F32, NULL);
        } else if (!strcmp(name, "forward")) {   /* T, K, V */
            need = mxfp4_linear_xent_forward_workspace_bytes(a, b, c);
            status = mxfp4_linear_xent_forward(p, (b + 7) / 8 * 8, p, (b + 7) / 8 * 8, p, a, b, c, -100, p, big, p, p, NULL);
        } else if (!strcmp(name, "backward")) {
            need = mxfp4_linear_xent_backward_workspace_bytes(a, b, c);
            status = mxfp4_linear_xent_backward(p, NULL, p, (b + 7) / 8 * 8, p, (b + 7) / 8 * 8, p, p, a, b, c, -100, p, big, p,
                                                MXFP4_OUT_BF16, p, MXFP4_OUT_F32, NULL);
        } else if (!strcmp(name, "orthogonalize")) {   /* batch, m, n */
            need = mxfp4_orthogonalize_workspace_bytes(a, b, c);
            status = mxfp4_orthogonalize(p, MXFP4_IN_F32, a, b, c, c, b * c, 5, 3.4445f, -4.775f, 2.0315f, 1e-7f, 1.0f, 0.0f, p,
                                         MXFP4_OUT_BF16, c, b * c, p, big, NULL);
        }
        printf("%d %ld %ld %zu\n", status, launches, beyond, need);
    }
    return 0;
}
