// rms_out_kernels.cuh -- RMSNorm forward with the residual's addition and /
// or an output in 8 bits with scales, for sm_103a; instantiated once per
// storage dtype in rms_out_f32.cu, rms_out_f16.cu and rms_out_bf16.cu.
//
// Per row of N elements, with T the storage type and Q = 448 (e4m3) or 127
// (int8):
//   h = round_T(x + residual)          (no residual: h = x)
//   rstd = 1 / sqrt(sum(h^2) / N + eps)
//   y = round_T(gamma * h * rstd), or, with v = gamma * h,
//   a = max |v| over the row (or over each group of 128 columns),
//   code = round(v * (Q / a)),  scale = rstd * a / Q.
// The statistics are those of the stored h, which the backward reads.  rstd
// cancels out of the codes, so one pass over the row gives everything that
// they need, and a code depends on its row's v alone: no order of a sum
// changes it.  Sums and maxima are float32; the roundings to fewer bits are
// h's, y's and the codes', once each, to nearest even.
#pragma once

#include "gbn_device.cuh"
#include "rms_out.h"

namespace gbn {

// the larger of two values, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// maximum over the 32 lanes of values >= 0, NaN if any is
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// What turns v into a code: code = round((v * pre) * mul).  A maximum so
// small that Q / a would overflow is first brought up by 2^100, exactly; a
// row (group) of zeros has codes 0 and scale 0.  a = NaN makes every code
// NaN (int8: 0) and the scale NaN.
struct QuantFactors {
    float pre, mul;
};
template <int KIND>
__device__ __forceinline__ float quant_top() {
    return KIND == kOutE4M3 ? 448.f : 127.f;
}
template <int KIND>
__device__ __forceinline__ QuantFactors quant_factors(float a) {
    QuantFactors f;
    f.pre = a < 0x1p-100f ? 0x1p100f : 1.f;
    f.mul = a == 0.f ? 0.f : quant_top<KIND>() / (a * f.pre);
    return f;
}
template <int KIND>
__device__ __forceinline__ float quant_scale(float rstd, float a) {
    return rstd * a / quant_top<KIND>();
}

// four float32 values as four 8-bit codes, the first in the lowest byte
template <int KIND>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    if constexpr (KIND == kOutE4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return lo | (static_cast<uint32_t>(hi) << 16);
    } else {
        const int i0 = __float2int_rn(a), i1 = __float2int_rn(b), i2 = __float2int_rn(c), i3 = __float2int_rn(d);
        return (i0 & 255) | ((i1 & 255) << 8) | ((i2 & 255) << 16) | (static_cast<uint32_t>(i3) << 24);
    }
}
template <int KIND>
__device__ __forceinline__ uint8_t quant1(float a) {
    return static_cast<uint8_t>(quant4<KIND>(a, 0.f, 0.f, 0.f) & 255u);
}

// ---------------------------------------------------------------------------
// any N, stride and alignment: one row at a time per CTA, scalar accesses.
// A warp owns whole blocks of 128 columns (four columns 32 apart a lane), so
// a group's maximum is a warp's; h is read again for the output, by the
// threads that wrote it.
// ---------------------------------------------------------------------------
constexpr int kOutPlainThreads = 256;

template <typename T, int KIND, bool RES, bool GROUP>
__global__ void __launch_bounds__(kOutPlainThreads) rms_out_plain_kernel(const OutParams p) {
    using Tr = Traits<T>;
    constexpr int NW = kOutPlainThreads / 32;
    __shared__ float sm[NW], sx[NW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int N = p.N;
    const float inv_n = 1.0f / static_cast<float>(N);
    const T *g = static_cast<const T *>(p.gamma);
    const int64_t groups = (N + kQuantGroup - 1) / kQuantGroup;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
        const T *r = RES ? static_cast<const T *>(p.res) + row * p.ld_res : nullptr;
        T *h = RES ? static_cast<T *>(p.h) + row * p.ld_h : nullptr;
        float q = 0.f, a = 0.f;
        for (int c0 = warp * 128; c0 < N; c0 += NW * 128) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                if (c < N) {
                    float f = Tr::load1(x + c);
                    if constexpr (RES) {
                        Tr::store1(h + c, f + Tr::load1(r + c));
                        f = Tr::load1(h + c);
                    }
                    q = fmaf(f, f, q);
                    if constexpr (KIND != kOutSame && !GROUP) a = max_nan(a, fabsf(Tr::load1(g + c) * f));
                }
            }
        }
        q = block_sum(q, sm);
        const float rs = 1.0f / sqrtf(q * inv_n + p.eps);
        if constexpr (KIND != kOutSame && !GROUP) {
            a = warp_max_nan(a);
            if (lane == 0) sx[warp] = a;
            __syncthreads();
            a = sx[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) a = max_nan(a, sx[w]);
            __syncthreads();
        }
        const T *hr = RES ? h : x;
        QuantFactors qf = {1.f, 0.f};
        if constexpr (KIND != kOutSame && !GROUP) qf = quant_factors<KIND>(a);
        for (int c0 = warp * 128; c0 < N; c0 += NW * 128) {
            float v[4], ga = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                const float f = c < N ? Tr::load1(hr + c) : 0.f;
                v[i] = (c < N ? Tr::load1(g + c) : 0.f) * (KIND == kOutSame ? f * rs : f);
                if constexpr (GROUP) ga = max_nan(ga, fabsf(v[i]));
            }
            if constexpr (GROUP) {
                ga = warp_max_nan(ga);
                qf = quant_factors<KIND>(ga);
                if (lane == 0) p.scale[row * groups + c0 / kQuantGroup] = quant_scale<KIND>(rs, ga);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                if (c < N) {
                    if constexpr (KIND == kOutSame)
                        Tr::store1(static_cast<T *>(p.out) + row * p.ld_out + c, v[i]);
                    else
                        static_cast<uint8_t *>(p.out)[row * p.ld_out + c] = quant1<KIND>((v[i] * qf.pre) * qf.mul);
                }
            }
        }
        if (threadIdx.x == 0) {
            p.rstd[row] = rs;
            if constexpr (KIND != kOutSame && !GROUP) p.scale[row] = quant_scale<KIND>(rs, a);
        }
    }
}

template <typename T, int KIND, bool RES>
cudaError_t rms_out_plain_group(bool group, const OutParams &p, int grid, cudaStream_t s) {
    if constexpr (KIND != kOutSame) {
        if (group) {
            rms_out_plain_kernel<T, KIND, RES, true><<<grid, kOutPlainThreads, 0, s>>>(p);
            return cudaGetLastError();
        }
    }
    rms_out_plain_kernel<T, KIND, RES, false><<<grid, kOutPlainThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t rms_out_plain_dispatch(int kind, bool group, const OutParams &p, int sms, cudaStream_t s) {
    const int64_t most = static_cast<int64_t>(sms) * 8;
    const int grid = static_cast<int>(p.M < most ? p.M : most);
    const bool res = p.res != nullptr;
    switch (kind) {
        case kOutSame: return res ? rms_out_plain_group<T, kOutSame, true>(false, p, grid, s) : cudaErrorInvalidValue;
        case kOutE4M3:
            return res ? rms_out_plain_group<T, kOutE4M3, true>(group, p, grid, s)
                       : rms_out_plain_group<T, kOutE4M3, false>(group, p, grid, s);
        case kOutInt8:
            return res ? rms_out_plain_group<T, kOutInt8, true>(group, p, grid, s)
                       : rms_out_plain_group<T, kOutInt8, false>(group, p, grid, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbn
