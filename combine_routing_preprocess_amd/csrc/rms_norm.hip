// RMS norm of token rows with the residual's addition and an output in 8 bits,
// and its backward pass: the norm in front of the MoE layer.
//
//   forward   t = x + residual,  r = 1 / sqrt(mean(t^2) + eps),  y = t * r * w
//             codes = e4m3(y / scale), scale = max |y| of 128 columns / 448
//   backward  xh = t * r,  q = gy * w,
//             gt = grad_total + r * (q - xh * mean(q * xh)),
//             gw = sum over the rows of gy * xh
#include "wave_ops.h"

namespace moe {
namespace {

using ops::wave_sum_dpp;

__device__ __forceinline__ float load1(const void* p, int dtype, long long i) {
    return dtype == MOE_BF16 ? bf16_lo(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void store1(void* p, int dtype, long long i, float v) {
    if (dtype == MOE_BF16) ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16(v);
    else ((float*)p)[i] = v;
}

// Sum over the workgroup's four wavefronts, in every lane.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = wave_sum_dpp(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// One workgroup per row.
__global__ __launch_bounds__(256) void k_rms_norm(int H, int xd, int rd, int yd, int wd, const void* x, const void* res,
                                                  const void* w, float eps, void* y, uint8_t* codes, float* scales,
                                                  void* total, float* rstd) {
    __shared__ float s[4];
    const long long at = (long long)blockIdx.x * H;
    float sq = 0.f;
    for (int c = threadIdx.x; c < H; c += 256) {
        float t = load1(x, xd, at + c);
        if (res) t += load1(res, rd, at + c);
        sq = fmaf(t, t, sq);
    }
    const float r = 1.f / sqrtf(block_sum(sq, s) / (float)H + eps);
    if (rstd && threadIdx.x == 0) rstd[blockIdx.x] = r;
    // 128 columns per wavefront and step: two per lane
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int c0 = 128 * wave; c0 < H; c0 += 512) {
        float v[2];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = c0 + 2 * lane + i;
            v[i] = 0.f;
            if (c >= H) continue;
            float t = load1(x, xd, at + c);
            if (res) t += load1(res, rd, at + c);
            v[i] = t * r * (w ? load1(w, wd, c) : 1.f);
            if (total) store1(total, rd, at + c, t);
            if (y) store1(y, yd, at + c, v[i]);
            top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);   // NaN above infinity above all numbers
        }
        if (!codes) continue;
        top = ops::wave_max_dpp(top);
        const float sc = top < 0x7f800000u ? e4m3_scale(__uint_as_float(top)) : __uint_as_float(0x7fc00000u);
        const uint32_t q = e4m3_pack4(v[0], v[1], 0.f, 0.f, sc);
        *(uint16_t*)(codes + at + c0 + 2 * lane) = (uint16_t)q;
        if (lane == 0) scales[(long long)blockIdx.x * (H / 128) + c0 / 128] = sc;
    }
}

// One workgroup per stripe of rows; its sums of gy * xh per column into
// part[stripe][H].
__global__ __launch_bounds__(256) void k_rms_norm_backward(int T, int H, int xd, int yd, int wd, const void* gy,
                                                           const void* t, const float* rstd, const void* w,
                                                           const void* gtot, void* gx, float* part) {
    __shared__ float s[4];
    if (part)
        for (int c = threadIdx.x; c < H; c += 256) part[(long long)blockIdx.x * H + c] = 0.f;
    for (int row = blockIdx.x; row < T; row += gridDim.x) {
        const long long at = (long long)row * H;
        const float r = rstd[row];
        float dot = 0.f;
        for (int c = threadIdx.x; c < H; c += 256)
            dot = fmaf(load1(gy, yd, at + c) * (w ? load1(w, wd, c) : 1.f), load1(t, xd, at + c) * r, dot);
        const float m = block_sum(dot, s) / (float)H;
        for (int c = threadIdx.x; c < H; c += 256) {
            const float g = load1(gy, yd, at + c), xh = load1(t, xd, at + c) * r;
            float o = r * (g * (w ? load1(w, wd, c) : 1.f) - xh * m);
            if (gtot) o += load1(gtot, xd, at + c);
            if (gx) store1(gx, xd, at + c, o);
            if (part) part[(long long)blockIdx.x * H + c] = fmaf(g, xh, part[(long long)blockIdx.x * H + c]);
        }
    }
}

__global__ __launch_bounds__(256) void k_rms_param_grad(const float* part, int nb, int H, float* gw) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= H) return;
    float v = 0.f;
    for (int i = 0; i < nb; ++i) v += part[(long long)i * H + c];
    gw[c] = v;
}

constexpr int kStripes = 256;

}  // namespace

size_t rms_norm_backward_scratch_bytes(int T, int H) {
    return (size_t)(T < kStripes ? T : kStripes) * H * sizeof(float);
}

hipError_t launch_rms_norm(int T, int H, int x_dtype, int r_dtype, int y_dtype, int w_dtype, const void* x,
                           const void* residual, const void* weight, float eps, void* y, void* codes, float* scales,
                           void* total, float* rstd, int num_cu, hipStream_t s) {
    if (T == 0) return hipSuccess;
    hipLaunchKernelGGL(k_rms_norm, dim3(T), dim3(256), 0, s, H, x_dtype, r_dtype, y_dtype, w_dtype, x, residual, weight,
                       eps, y, (uint8_t*)codes, scales, total, rstd);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* gy,
                                    const void* total, const float* rstd, const void* weight, const void* grad_total,
                                    void* gx, float* gw, void* scratch, hipStream_t s) {
    const int nb = T < kStripes ? T : kStripes;
    if (nb > 0) {
        hipLaunchKernelGGL(k_rms_norm_backward, dim3(nb), dim3(256), 0, s, T, H, x_dtype, y_dtype, w_dtype, gy, total,
                           rstd, weight, grad_total, gx, gw ? (float*)scratch : nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!gw) return hipSuccess;
    hipLaunchKernelGGL(k_rms_param_grad, dim3((H + 255) / 256), dim3(256), 0, s, (const float*)scratch, nb, H, gw);
    return hipGetLastError();
}

}  // namespace moe
