// int8_gemm.cu -- the projection with 8-bit integers on both sides.
//
//     y[b, n] = bf16(x_scale[b] * w_scale[n] * sum_k x[b, k] W[n, k])
//
// One warp for a weight row and eight batch rows: 16 bytes a lane of the row and
// of each batch row, four-way integer dot products, the lanes' 32-bit sums added
// by shuffles (integers: exact in any order).
#include <cuda_bf16.h>

#include <new>

#include "internal.h"
#include "layer.h"

struct dep_int8_plan_s {
    int64_t N = 0, K = 0;
    int32_t max_rows = 0;
    int device = -1;
    int sm_count = 0;
    void *block = nullptr;  // device memory
    size_t bytes = 0;
    int *status = nullptr;
};

namespace dep {
namespace {

constexpr int64_t kMaxK = 131056;  // 131056 * 128 * 128 < 2^31

__global__ void __launch_bounds__(256)
    int8_rows_kernel(const int8_t *__restrict__ x, const float *__restrict__ xs, const int8_t *__restrict__ W,
                     const float *__restrict__ ws, uint16_t *__restrict__ y, int B, int64_t N, int K)
{
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int b0 = blockIdx.y * 8;
    if (n >= N)
        return;
    int acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int k = lane * 16; k < K; k += 512) {
        const int4 w = *reinterpret_cast<const int4 *>(W + n * K + k);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (b0 + j < B) {
                const int4 v = *reinterpret_cast<const int4 *>(x + (int64_t)(b0 + j) * K + k);
                acc[j] = __dp4a(v.x, w.x, acc[j]);
                acc[j] = __dp4a(v.y, w.y, acc[j]);
                acc[j] = __dp4a(v.z, w.z, acc[j]);
                acc[j] = __dp4a(v.w, w.w, acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int s = __reduce_add_sync(~0u, acc[j]);
        if (lane == 0 && b0 + j < B)
            y[(int64_t)(b0 + j) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn((float)s * (xs[b0 + j] * ws[n])));
    }
}

}  // namespace
}  // namespace dep

extern "C" {

dep_status_t dep_int8_plan(int64_t N, int64_t K, int32_t max_rows, dep_int8_plan_t *out)
{
    if (!out)
        return DEP_ERR_INVALID_ARG;
    *out = nullptr;
    if (N < 1 || K < 16 || max_rows < 1)
        return DEP_ERR_INVALID_ARG;
    if (K % 16 != 0)
        return DEP_ERR_MISALIGNED;
    if (K > dep::kMaxK || N > INT32_MAX)
        return DEP_ERR_UNSUPPORTED;
    dep_int8_plan_s *p = new (std::nothrow) dep_int8_plan_s;
    if (!p)
        return DEP_ERR_OOM;
    p->N = N;
    p->K = K;
    p->max_rows = max_rows;
    cudaDeviceProp prop;
    if (cudaGetDevice(&p->device) != cudaSuccess || cudaGetDeviceProperties(&prop, p->device) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return DEP_ERR_CUDA;
    }
    p->sm_count = prop.multiProcessorCount;
    if (prop.major * 10 + prop.minor < 100) {
        delete p;
        return DEP_ERR_UNSUPPORTED;
    }
    p->bytes = 256;
    if (cudaMalloc(&p->block, p->bytes) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return DEP_ERR_OOM;
    }
    if (cudaMemset(p->block, 0, p->bytes) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(p->block);
        delete p;
        return DEP_ERR_CUDA;
    }
    p->status = static_cast<int *>(p->block);
    *out = p;
    return DEP_OK;
}

dep_status_t dep_int8_run(dep_int8_plan_t p, const void *x, const float *x_scale, const void *W, const float *w_scale,
                          void *y, int32_t B, void *stream)
{
    if (!p || B < 0)
        return DEP_ERR_INVALID_ARG;
    if (B == 0)
        return DEP_OK;
    if (!x || !x_scale || !W || !w_scale || !y)
        return DEP_ERR_INVALID_ARG;
    if (!dep::aligned(x, 16) || !dep::aligned(W, 16) || !dep::aligned(y, 16) || !dep::aligned(x_scale, 4) ||
        !dep::aligned(w_scale, 4))
        return DEP_ERR_MISALIGNED;
    const dep::Rows ry{y, 2 * B * p->N, 0, 1}, rx{x, B * p->K, 0, 1}, rw{W, p->N * p->K, 0, 1},
        rxs{x_scale, 4 * (int64_t)B, 0, 1}, rws{w_scale, 4 * p->N, 0, 1};
    if (overlap(ry, rx) || overlap(ry, rw) || overlap(ry, rxs) || overlap(ry, rws))
        return DEP_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != p->device) {
        cudaGetLastError();
        return DEP_ERR_INVALID_ARG;
    }
    const dim3 grid((unsigned)((p->N + 7) / 8), (unsigned)((B + 7) / 8));
    dep::int8_rows_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const int8_t *>(x), x_scale, static_cast<const int8_t *>(W), w_scale, static_cast<uint16_t *>(y),
        B, p->N, (int)p->K);
    if (cudaGetLastError() != cudaSuccess)
        return DEP_ERR_CUDA;
    return DEP_OK;
}

dep_status_t dep_int8_plan_workspace(dep_int8_plan_t p, size_t *bytes)
{
    if (!p || !bytes)
        return DEP_ERR_INVALID_ARG;
    *bytes = p->bytes;
    return DEP_OK;
}

dep_status_t dep_int8_device_status(dep_int8_plan_t p, void *stream, int32_t *code)
{
    if (!p || !code)
        return DEP_ERR_INVALID_ARG;
    *code = 0;
    int h = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpy(&h, p->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    // After a give-up the exchange may be left mid-protocol: clear everything.
    if (h && (cudaDeviceSynchronize() != cudaSuccess || cudaMemset(p->block, 0, p->bytes) != cudaSuccess)) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    *code = h;
    return h ? DEP_ERR_TIMEOUT : DEP_OK;
}

void dep_int8_plan_destroy(dep_int8_plan_t p)
{
    if (!p)
        return;
    int dev = -1;
    cudaGetDevice(&dev);
    if (dev != p->device)
        cudaSetDevice(p->device);
    cudaFree(p->block);  // waits for the device's work
    if (dev >= 0 && dev != p->device)
        cudaSetDevice(dev);
    cudaGetLastError();
    delete p;
}

}  // extern "C"
