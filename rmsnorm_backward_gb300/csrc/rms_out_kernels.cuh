// rms_out_kernels.cuh -- RMSNorm forward with the residual's addition and /
// or an output in 8 bits with scales, for sm_103a; instantiated once per
// storage dtype in rms_out_f32.cu, rms_out_f16.cu and rms_out_bf16.cu.
//
// Per row of N elements, with T the storage type and Q = 448 (e4m3) or 127
// (int8):
//   h = round_T(x + residual)          (no residual: h = x)
//   rstd = 1 / sqrt(sum(h^2) * (1/N) + eps)
//   y = round_T(gamma * h * rstd), or, with v = gamma * h,
//   a = max |v| over the row (or over each group of 128 columns),
//   code = round(v * (Q / a)),  scale = rstd * a * (1/Q).
// The statistics are those of the stored h, which the backward reads.  rstd
// cancels out of the codes, so one pass over the row gives everything that
// they need, and a code depends on its row's v alone: no order of a sum
// changes it.  Sums and maxima are float32; the roundings to fewer bits are
// h's, y's and the codes', once each, to nearest even.
#pragma once

#include <atomic>
#include <type_traits>

#include "gbn_device.cuh"
#include "gbn_launch.h"
#include "rms_out.h"
#include "row_phase.h"

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

// the maximum over each L neighbouring lanes (16 or 32)
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t b) {
    if constexpr (L == 32) {
        b = __reduce_max_sync(0xffffffffu, b);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    return b;
}

// What turns v into a code: code = round(v * quant_factor(a)).  Where a is so
// small that Q / a would overflow, v is first brought up by 2^100, exactly
// (`tiny`; the factor is then that of the raised a).  A row (group) of zeros
// has codes 0 and scale 0.  a = NaN makes every code NaN (int8: 0) and the
// scale NaN.
template <int KIND>
__device__ __forceinline__ float quant_top() {
    return KIND == kOutE4M3 ? 448.f : 127.f;
}
constexpr float kTiny = 0x1p-100f, kRaise = 0x1p100f;
__device__ __forceinline__ bool quant_tiny(float a) { return a < kTiny; }
template <int KIND>
__device__ __forceinline__ float quant_factor(float a) {
    if (a == 0.f) return 0.f;
    return quant_top<KIND>() / (quant_tiny(a) ? a * kRaise : a);
}
// (eps = 0 leaves a row of zeros an infinite rstd, whose product with 0 were NaN)
template <int KIND>
__device__ __forceinline__ float quant_scale(float rstd, float a) {
    if (a == 0.f && rstd > 3.402823466e38f) return 0.f;
    return rstd * a * (1.f / quant_top<KIND>());
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
// quant4 of finite values up to 127.5 in magnitude.  int8: adding 1.5 * 2^23
// rounds to the nearest integer, ties to even, and leaves it in the sum's low
// bits: an addition at full rate for a conversion at an eighth of it.
template <int KIND>
__device__ __forceinline__ uint32_t quant4_finite(const float *t) {
    if constexpr (KIND == kOutE4M3) {
        return quant4<KIND>(t[0], t[1], t[2], t[3]);
    } else {
        constexpr float kRound = 12582912.f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(t[0], kRound)),
                                        __float_as_uint(__fadd_rn(t[1], kRound)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(t[2], kRound)),
                                        __float_as_uint(__fadd_rn(t[3], kRound)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}
// Whether a maximum has an ordinary factor: not zero, tiny, infinite or NaN.
__device__ __forceinline__ bool quant_plain(float a) { return a >= kTiny && a < __int_as_float(0x7f800000); }
// the codes of four values whose maximum a has none
template <int KIND>
__device__ __noinline__ uint32_t quant4_odd(float v0, float v1, float v2, float v3, float a) {
    const float raise = quant_tiny(a) ? kRaise : 1.f, f = quant_factor<KIND>(a);
    return quant4<KIND>((v0 * raise) * f, (v1 * raise) * f, (v2 * raise) * f, (v3 * raise) * f);
}
// the same, the first `split` of them of a maximum a0
template <int KIND>
__device__ __noinline__ uint32_t quant4_split(float v0, float v1, float v2, float v3, int split, float a0, float a) {
    const float r0 = quant_tiny(a0) ? kRaise : 1.f, f0 = quant_factor<KIND>(a0);
    const float r = quant_tiny(a) ? kRaise : 1.f, f = quant_factor<KIND>(a);
    return quant4<KIND>((v0 * (split > 0 ? r0 : r)) * (split > 0 ? f0 : f), (v1 * (split > 1 ? r0 : r)) * (split > 1 ? f0 : f),
                        (v2 * (split > 2 ? r0 : r)) * (split > 2 ? f0 : f), (v3 * (split > 3 ? r0 : r)) * (split > 3 ? f0 : f));
}
// the codes of a lane's V values (code.x the first four's) by the factor of
// their maximum a
template <int KIND, int V>
__device__ __forceinline__ uint2 quant_vector(float *t, float factor, float a) {
    uint2 code = make_uint2(0, 0);
    if (quant_plain(a)) {
        // int8: the product is rounded before the addition that rounds it to
        // an integer.  With both as pairs they came out as one fused operation,
        // which rounds ties the other way; so the additions are scalar.
        const float2 f2 = make_float2(factor, factor);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 w = pair_mul(pair_at(t, i), f2);
            t[2 * i] = w.x, t[2 * i + 1] = w.y;
        }
        code.x = quant4_finite<KIND>(t);
        if constexpr (V == 8) code.y = quant4_finite<KIND>(t + 4);
    } else {
        code.x = quant4_odd<KIND>(t[0], t[1], t[2], t[3], a);
        if constexpr (V == 8) code.y = quant4_odd<KIND>(t[4], t[5], t[6], t[7], a);
    }
    return code;
}
template <int KIND>
__device__ __forceinline__ uint8_t quant1(float a) {
    return static_cast<uint8_t>(quant4<KIND>(a, 0.f, 0.f, 0.f) & 255u);
}

// ---------------------------------------------------------------------------
// any N, stride and alignment: one row at a time per CTA, scalar accesses.
// A warp owns whole blocks of 128 columns (four columns 32 apart a lane), so
// a group's maximum is a warp's; h is read again for the output, by the
// threads that wrote it.  For rows too wide for the ring (its threads hold 16384
// elements; two stages of a float32 row with its residual fit up to 14500) and
// tensors whose rows lie differently to 16-byte boundaries (4096x20000 bf16 255
// us, 2.6 TB/s, 2048x16384 float32 156 us, 3.4 TB/s: an element to a load keeps
// too little in flight).
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
        const float rs = __frsqrt_rn(fmaf(q, inv_n, p.eps));
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
        float qf = 0.f, raise = 1.f;
        if constexpr (KIND != kOutSame && !GROUP) qf = quant_factor<KIND>(a), raise = quant_tiny(a) ? kRaise : 1.f;
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
                qf = quant_factor<KIND>(ga), raise = quant_tiny(ga) ? kRaise : 1.f;
                if (lane == 0) p.scale[row * groups + c0 / kQuantGroup] = quant_scale<KIND>(rs, ga);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                if (c < N) {
                    if constexpr (KIND == kOutSame)
                        Tr::store1(static_cast<T *>(p.out) + row * p.ld_out + c, v[i]);
                    else
                        static_cast<uint8_t *>(p.out)[row * p.ld_out + c] = quant1<KIND>((v[i] * raise) * qf);
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

// ---------------------------------------------------------------------------
// One persistent CTA per SM; its 16 warps are slots of tpr threads, and each
// slot streams its rows of x (and residual) through a ring of shared-memory
// stages by 1-D bulk copies, which one warp of the slot issues (a lane for
// each tensor).  A thread owns NV column vectors and their gamma.  It takes
// its part of the row from the stage, writes h, and keeps h (8-bit outputs: v
// = gamma*h) in float32 registers; one exchange within the slot gives the
// sum of squares, the maximum of |v|, and shows that the stage may be
// refilled; then the outputs are written from registers: x and residual are
// read once, h is written once and read by nobody.  Bound by HBM: 16384x4096
// bf16 with the residual 81.7 us, 6.57 TB/s (98% of the measured copy rate);
// to e4m3 by 128 columns, 8192x16384, 144 us, 6.5 TB/s.  Without the residual
// there are fewer bytes to hide the work of a code behind: 16384x4096 bf16 to
// e4m3 37 us, 5.4 TB/s, bound by the latencies of the warps' work: half the
// issue slots are used, the 4 warps a scheduler that 128 registers allow are
// too few to fill the others.  Code counts even where it does not run: with and
// without a residual in one kernel 46 us against 43 (by 128 columns).
//
// How the rows lie (RowLie):
//  * kLieFull: they start and end on 16 bytes (their codes on V) and are as
//    many vectors as the slot's threads own;
//  * kLieWhole: a thread may own fewer;
//  * kLieAcross: rows may lie across 16-byte boundaries, all tensors' alike
//    (the host checks that): such a row is copied with the up to 14 bytes
//    before and after it that share its first and last 16 bytes (never beyond
//    the tensor's first and last element: those two ends are copied element by
//    element); only the vectors that lie wholly in the row are the threads',
//    so that h and y are stored as vectors, and the elements before and after
//    them go to the lanes of the slot's last warp, one each.  Borders of
//    groups then run through vectors, and the groups' maxima meet in shared
//    memory: one atomic for a group's lanes, one for the elements of its last
//    vector that another lane owns (10365x6474 f16 to int8 131 us, 3.6 TB/s;
//    16384x2050 bf16 to e4m3 70 us, 3.4 TB/s; an atomic a vector 171 and 72);
//  * kLieShift (8-bit outputs without a residual, where nothing is stored at
//    the rows' own places): copied as kLieAcross, but a thread's vectors are V
//    columns from the row's first on, put together from two staged ones by
//    shifts; groups are lanes again, and no element stands alone (27711x2202
//    to int8 70 us, by 128 columns 82; as kLieAcross 85 and 137).  With a
//    residual h would have to be shifted back: 16384x2050 by 128 columns 97 us
//    against 70 as kLieAcross.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float round_to(float f) {
    if constexpr (sizeof(T) == 4) {
        return f;
    } else {
        T t;
        Traits<T>::store1(&t, f);
        return Traits<T>::load1(&t);
    }
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// The 16 bytes from the O-th 32-bit word and `bits` bits on (0 or 16, for
// 16-bit elements) of two neighbouring vectors.
template <int V, int O>
__device__ __forceinline__ uint4 vector_from(uint4 a, uint4 b, int bits) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (V == 4) {
        return make_uint4(w[O], w[O + 1], w[O + 2], w[O + 3]);
    } else {
        return make_uint4(__funnelshift_r(w[O], w[O + 1], bits), __funnelshift_r(w[O + 1], w[O + 2], bits),
                          __funnelshift_r(w[O + 2], w[O + 3], bits), __funnelshift_r(w[O + 3], w[O + 4], bits));
    }
}
// f(O) for the words O of s elements, 0 <= s < V: one uniform branch instead
// of a choice for each word
template <int V, typename F>
__device__ __forceinline__ void by_words(int s, F f) {
    switch (V == 8 ? s >> 1 : s) {
        case 0: f(std::integral_constant<int, 0>{}); break;
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        default: f(std::integral_constant<int, 3>{}); break;
    }
}
// the first n of a vector's V elements, zeros for the others
template <int V>
__device__ __forceinline__ uint4 vector_head(uint4 a, int n) {
    uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (V == 4) {
            if (i >= n) w[i] = 0;
        } else {
            if (2 * i >= n)
                w[i] = 0;
            else if (2 * i + 1 >= n)
                w[i] &= 0xffffu;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's codes, V a lane, the bytes [lo, n) of them (lo 0 or V), to
// consecutive places that start m bytes after a boundary of V: a lane stores
// the V bytes that end m bytes before its own end, and the bytes at both ends,
// which fill no such place, go one to a lane.  Out of line: for a row's end
// vectors only.
template <int V>
__device__ __noinline__ void store_codes_part(uint8_t *at, uint2 code, int lane, int lo, int n, int m) {
    const int place = lane * V - m, first = lo + ((V - m) & (V - 1));
    const int of = lane < V ? lo + lane : first + ((n - first) & -V) + lane - V;
    const bool end = lane < 2 * V && of < (lane < V ? min(first, n) : n) && (lane < V || n >= first);
    const bool vec = place >= lo && place + V <= n;
    const int from = end ? of / V : 0;
    uint64_t own = code.x;
    if constexpr (V == 8) own |= static_cast<uint64_t>(code.y) << 32;
    const uint64_t prev = __shfl_up_sync(0xffffffffu, own, 1), other = __shfl_sync(0xffffffffu, own, from);
    const uint64_t w = m ? (own << (8 * m)) | (prev >> (8 * (V - m))) : own;
    if (vec) {
        if constexpr (V == 8)
            *reinterpret_cast<uint64_t *>(at + place) = w;
        else
            *reinterpret_cast<uint32_t *>(at + place) = static_cast<uint32_t>(w);
    }
    if (end) at[of] = static_cast<uint8_t>(other >> (8 * (of & (V - 1))));
}

template <int V>
__device__ __forceinline__ void store_code(uint8_t *at, uint2 code) {
    if constexpr (V == 8)
        *reinterpret_cast<uint2 *>(at) = code;
    else
        *reinterpret_cast<uint32_t *>(at) = code.x;
}

// The same of all 32 V bytes; what depends on m alone is formed once a row.
template <int V>
struct CodePlace {
    int m, bits, from, end;  // end: the lane's byte at an end, or -1
    __device__ __forceinline__ CodePlace(int lane, int m_) : m(m_) {
        const int e = lane & (V - 1);
        bits = 8 * (-m & 3);
        from = lane < V ? 0 : 31;
        end = lane < 2 * V && (lane < V) == (e < V - m) ? from * V + e : -1;
    }
    __device__ __forceinline__ void store(uint8_t *at, uint2 code, int lane) const {
        uint8_t *p = at + lane * V;
        if (m == 0) {
            store_code<V>(p, code);
        } else if constexpr (V == 8) {
            const uint32_t p0 = __shfl_up_sync(0xffffffffu, code.x, 1), p1 = __shfl_up_sync(0xffffffffu, code.y, 1);
            const uint32_t e0 = __shfl_sync(0xffffffffu, code.x, from), e1 = __shfl_sync(0xffffffffu, code.y, from);
            const uint32_t w0 = m > 4 ? p0 : p1, w1 = m > 4 ? p1 : code.x, w2 = m > 4 ? code.x : code.y;
            if (lane > 0)
                *reinterpret_cast<uint2 *>(p - m) = make_uint2(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits));
            if (end >= 0) at[end] = static_cast<uint8_t>(__byte_perm(e0, e1, end & 7));
        } else {
            const uint32_t p1 = __shfl_up_sync(0xffffffffu, code.x, 1), e0 = __shfl_sync(0xffffffffu, code.x, from);
            if (lane > 0) *reinterpret_cast<uint32_t *>(p - m) = __funnelshift_r(p1, code.x, bits);
            if (end >= 0) at[end] = static_cast<uint8_t>(e0 >> (8 * (end & 3)));
        }
    }
};

template <typename T, int KIND, bool RES, bool GROUP, int NV, int LIE>
__global__ void __launch_bounds__(kOutThreads, 1) rms_out_ring_kernel(const OutParams p) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int E = NV * V;
    constexpr bool QUANT = KIND != kOutSame;
    constexpr bool FULL = LIE == kLieFull, ACROSS = LIE == kLieAcross, SHIFT = LIE == kLieShift;
    static_assert(!SHIFT || !RES, "h's vectors are the staged row's");
    constexpr bool GRAW = sizeof(T) == 2 && NV > 3;  // gamma kept in the storage type
    using Out = typename std::conditional<QUANT, uint8_t, T>::type;
    extern __shared__ __align__(128) unsigned char smem[];

    const int tid = threadIdx.x, tpr = p.tpr, W = tpr >> 5, slots = p.slots;
    const int slot = tid / tpr, ts = tid - slot * tpr;
    const int warp = ts >> 5, lane = tid & 31;
    constexpr int streams = RES ? 2 : 1;
    const bool issuer = warp == 0;
    const int N = p.N, S = p.stages;
    const uint32_t rowb = static_cast<uint32_t>(p.nvec) * 16;
    const int groups = (N + kQuantGroup - 1) / kQuantGroup;
    constexpr bool meet = GROUP && ACROSS;  // group maxima through shared memory
    const OutLayout L = out_layout(slots, S, streams, p.nvec, meet ? groups : 0);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L.bar);
    float *reds = reinterpret_cast<float *>(smem + L.red);
    int *flags = reinterpret_cast<int *>(smem + L.flag);

    // the slot's rows: row + k*row_step for k < ns; a CTA's have one shift
    const int64_t row_step = (int64_t)p.G * slots, row0 = blockIdx.x * (int64_t)p.cta_step + slot * (int64_t)p.slot_step;
    int64_t row = row0;
    const int ns = slot < slots && row < p.M ? static_cast<int>((p.M - row + row_step - 1) / row_step) : 0;
    // the row starts s elements into its first staged vector; the threads'
    // vectors are [vb, ve): kLieAcross: those that lie wholly in it;
    // kLieShift: of V columns from the row's first on
    const int s = !ACROSS && !SHIFT ? 0 : row_shift(blockIdx.x, p.shift0, p.shift_step, V);
    const int nvec = !ACROSS && !SHIFT ? p.nvec : (s + N + V - 1) / V;
    const int vb = ACROSS && s > 0 ? 1 : 0, ve = SHIFT ? (N + V - 1) / V : (s + N) / V;
    // they start at vb; with group maxima to meet at 0, so that a group's
    // vectors, but for the first s elements of the next group's first, are
    // those of GL neighbouring lanes
    constexpr int GL = kQuantGroup / V;
    const int v_base = meet ? 0 : vb;
    auto owned = [&](int v) { return FULL || (v < ve && (!meet || v >= vb)); };
    // the lane's element beside them, as a place in the staged row: s <= ce < s + N, or -1
    int ce = -1;
    if (ACROSS && warp == W - 1) {
        if (lane < V)
            ce = s > 0 && lane >= s && lane < s + N ? lane : -1;
        else if (lane < 2 * V && ve >= vb)
            ce = ve * V + lane - V < s + N ? ve * V + lane - V : -1;
    }

    if (tid == 0) {
        for (int i = 0; i < slots * S; ++i) mbar_init(&bars[i], 1);
        fence_barrier_init();
    }
    for (int i = tid; i < slots * 4 * kRedStride; i += kOutThreads) reds[i] = 0.f;
    if constexpr (meet)
        for (int i = tid; i < slots * 3 * groups; i += kOutThreads) reinterpret_cast<uint32_t *>(smem + L.gmax)[i] = 0;
    if (tid < slots) flags[tid] = 0;
    __syncthreads();
    griddep_wait();  // whatever is before this kernel on the stream
    griddep_launch_dependents();

    // lane t < streams of the issuing warp copies tensor t's rows
    unsigned char *ring = smem + (size_t)slot * S * streams * rowb;
    uint64_t *bar = bars + slot * S;
    const T *base = static_cast<const T *>(lane == 0 || !RES ? p.x : p.res);
    const int64_t ld = lane == 0 || !RES ? p.ld_x : p.ld_res;
    const T *src = base + row * ld - s;
    const int end0 = row0 == 0 ? 0 : -1, end1 = ns > 0 && row0 + (ns - 1) * row_step == p.M - 1 ? ns - 1 : -1;
    int issued = 0, pst = 0;
    auto issue = [&]() {
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16;
        uint32_t from = 0, to = bytes;
        unsigned char *dst = ring + (pst * streams + lane) * rowb;
        if ((ACROSS || SHIFT) && (issued == end0 || issued == end1)) {
            // the tensors' first and last rows: nothing outside them is read
            if (lane < streams) {
                const uint2 mid = copy_end_row<T>(reinterpret_cast<T *>(dst), src, base, base + (p.M - 1) * ld + N, s, N, bytes);
                from = mid.x, to = mid.y;
                if (to > from) mbar_expect_tx(&bar[pst], to - from);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[pst]);
        } else if (lane == 0) {
            mbar_arrive_expect_tx(&bar[pst], streams * bytes);
        }
        if (lane < streams && to > from) bulk_load_nohint(dst + from, src + from / sizeof(T), to - from, &bar[pst]);
        src += row_step * ld;
        if (++pst == S) pst = 0;
        ++issued;
    };
    if (issuer)
        while (issued < S && issued < ns) issue();

    const T *gamma = static_cast<const T *>(p.gamma) - (ACROSS ? s : 0);
    const bool gvec = (reinterpret_cast<uintptr_t>(gamma) & 15) == 0;
    float gam[GRAW ? 1 : E];
    uint4 graw[GRAW ? NV : 1];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = v_base + ts + j * tpr;
        float g[V];
        if ((SHIFT ? (v + 1) * V <= N : owned(v)) && gvec) {
            Tr::unpack(ld_global_nc_v4(gamma + v * V), g);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = (SHIFT ? v * V + e < N : owned(v)) ? Tr::load1(gamma + v * V + e) : 0.f;
        }
        if constexpr (GRAW) {
            graw[j] = Tr::pack(g);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) gam[j * V + e] = g[e];
        }
    }
    auto gamma_of = [&](int j, float *g) {
        if constexpr (GRAW) {
            Tr::unpack(graw[j], g);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = gam[j * V + e];
        }
    };
    const float ge = ce >= 0 ? Tr::load1(gamma + ce) : 0.f;

    const float inv_n = 1.0f / static_cast<float>(N);
    const int in_slot = slot < slots ? slot : 0;
    float *red = reds + in_slot * 4 * kRedStride;
    // a thread's vectors of a staged row (kLieShift)
    const bool whole_warp = (ts | 31) + 1 + (NV - 1) * tpr <= N / V;  // none of the warp's beyond the row
    auto shifted = [&](const unsigned char *row_at, uint4 *a) {
        by_words<V>(s, [&](auto o) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v = min(ts + j * tpr, ve - 1);
                a[j] = vector_from<V, decltype(o)::value>(ld_shared_v4(row_at + v * 16),
                                                          ld_shared_v4(row_at + min(v + 1, nvec - 1) * 16), (s & 1) * 16);
            }
        });
        if (!whole_warp) {
#pragma unroll
            for (int j = 0; j < NV; ++j) a[j] = vector_head<V>(a[j], N - (ts + j * tpr) * V);
        }
    };
    uint32_t *gmax = reinterpret_cast<uint32_t *>(smem + L.gmax) + in_slot * 3 * groups;  // of rows k mod 3
    int buf = 0;                                                                           // k mod 3
    volatile int *flag = flags + slot;
    RingPos pos;
    int k = 0;
    for (; k < ns; ++k, row += row_step) {
        const bool timed_out = !mbar_wait_bounded(&bar[pos.stage], pos.parity);
        if (timed_out) record_error(p.err, kErrWaitFull);
        if (p.late && issuer && k > 0 && issued < ns) {  // the row before is in registers, this one landed
            fence_proxy_async();
            issue();
        }
        const unsigned char *sx = ring + pos.stage * streams * rowb;
        T *h = static_cast<T *>(p.h) + (RES ? row * p.ld_h - (ACROSS ? s : 0) : 0);
        float sum = 0.f, held[E], he = 0.f;
        float most = 0.f, vmost[GROUP ? NV : 1];  // max |v|, NaN if any is
        uint4 xs[SHIFT ? NV : 1];
        if constexpr (SHIFT) shifted(sx, xs);
        uint32_t *gm = gmax + buf * groups;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = v_base + ts + j * tpr;
            if constexpr (GROUP) vmost[j] = 0.f;
            if (SHIFT || owned(v)) {
                float f[V];
                Tr::unpack(SHIFT ? xs[j] : ld_shared_v4(sx + v * 16), f);
                if constexpr (RES) {
                    float r[V];
                    Tr::unpack(ld_shared_v4(sx + rowb + v * 16), r);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 t = pair_add(pair_at(f, i), pair_at(r, i));
                        f[2 * i] = t.x, f[2 * i + 1] = t.y;
                    }
                    const uint4 h4 = Tr::pack(f);
                    st_global_cs_v4(h + v * V, h4);
                    Tr::unpack(h4, f);
                }
                float2 t = pair_mul(pair_at(f, 0), pair_at(f, 0));
#pragma unroll
                for (int i = 1; i < V / 2; ++i) t = pair_fma(pair_at(f, i), pair_at(f, i), t);
                sum += t.x + t.y;
                if constexpr (QUANT) {
                    float g[V];
                    gamma_of(j, g);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 w = pair_mul(pair_at(g, i), pair_at(f, i));
                        held[j * V + 2 * i] = w.x, held[j * V + 2 * i + 1] = w.y;
                    }
                    float m = fabsf(held[j * V]);
#pragma unroll
                    for (int e = 1; e < V; ++e) m = max_nan(m, fabsf(held[j * V + e]));
                    if constexpr (GROUP) {
                        vmost[j] = m;
                        if (meet && s > 0 && (lane & (GL - 1)) == 0) {  // in two groups
                            float m1 = m = 0.f;
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                if (e < s)
                                    m1 = max_nan(m1, fabsf(held[j * V + e]));
                                else
                                    m = max_nan(m, fabsf(held[j * V + e]));
                            }
                            vmost[j] = m;
                            atomicMax(gm + v / GL - 1, __float_as_uint(m1));
                        }
                    } else {
                        most = max_nan(most, m);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) held[j * V + e] = f[e];
                }
            }
        }
        if (ACROSS && ce >= 0) {
            he = Tr::load1(reinterpret_cast<const T *>(sx) + ce);
            if constexpr (RES) {
                he = round_to<T>(he + Tr::load1(reinterpret_cast<const T *>(sx + rowb) + ce));
                Tr::store1(h + ce, he);
            }
            sum = fmaf(he, he, sum);
            if constexpr (QUANT) {
                he *= ge;
                most = max_nan(most, fabsf(he));
                if (meet) atomicMax(gm + (ce - s) / kQuantGroup, abs_bits(he));
            }
        }
        if constexpr (meet) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint32_t b = lanes_max<GL>(__float_as_uint(vmost[j]));
                if ((lane & (GL - 1)) == 0 && b != 0) atomicMax(gm + (ts + j * tpr) / GL, b);
            }
        }
        // the exchange: warp sums (and maxima, as bits: the order of the
        // values, NaN above all), added in warp order
        sum = warp_sum(sum);
        uint32_t bits = 0;
        if constexpr (QUANT && !GROUP) bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        if (W > 1) {
            float *b = red + (k & 1) * 2 * kRedStride;
            if (lane == 0) {
                b[warp] = sum;
                if constexpr (QUANT && !GROUP) b[kRedStride + warp] = __uint_as_float(bits);
            }
            slot_meet(flag, k + 1, timed_out, 1 + slot, tpr);
            sum = 0.f;
            for (int w = 0; w < W; w += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(b + w);
                sum += (t.x + t.y) + (t.z + t.w);
                if constexpr (QUANT && !GROUP) {
                    const uint4 m = *reinterpret_cast<const uint4 *>(b + kRedStride + w);
                    bits = max(max(max(bits, m.x), max(m.y, m.z)), m.w);
                }
            }
            if (slot_stops(flag, k + 1)) break;
        } else {
            __syncwarp();
            if (__any_sync(0xffffffffu, timed_out)) break;
        }
        // the slot has the row in registers: refill its stage
        if (!p.late && issuer && issued < ns) {
            fence_proxy_async();
            issue();
        }
        float rs = 0.f;
        if (!QUANT || GROUP || ts == 0) rs = __frsqrt_rn(fmaf(sum, inv_n, p.eps));
        if (ts == 0) p.rstd[row] = rs;
        Out *out = static_cast<Out *>(p.out) + row * p.ld_out - (ACROSS ? s : 0);
        if constexpr (!QUANT) {
            const float2 rs2 = make_float2(rs, rs);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v = v_base + ts + j * tpr;
                if (FULL || v < ve) {
                    float o[V], g[V];
                    gamma_of(j, g);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 t = pair_mul(pair_at(g, i), pair_mul(pair_at(held + j * V, i), rs2));
                        o[2 * i] = t.x, o[2 * i + 1] = t.y;
                    }
                    st_global_cs_v4(out + v * V, Tr::pack(o));
                }
            }
            if (ACROSS && ce >= 0) Tr::store1(out + ce, ge * (he * rs));
        } else {
            float qf = 0.f;
            if constexpr (!GROUP) {
                most = __uint_as_float(bits);
                qf = quant_factor<KIND>(most);
                if (ts == 0) p.scale[row] = quant_scale<KIND>(rs, most);
            }
            float *scale = p.scale + (GROUP ? row * groups : 0);
            if constexpr (meet) {
                // the maxima of row k-1, read by nobody any more, for row k+2
                uint32_t *clear = gmax + (buf == 0 ? 2 : buf - 1) * groups;
                for (int i = ts; i < groups; i += tpr) {
                    clear[i] = 0;
                    scale[i] = quant_scale<KIND>(rs, __uint_as_float(gm[i]));
                }
                // Lane j of a group's lanes divides for their vector j, lane
                // GL/2 + j for the group before it; -1: no ordinary factor.
                const int j = lane & (GL / 2 - 1), at = (ts - lane) + j * tpr + (lane & ~(GL - 1));
                const int g = at / GL - ((lane & (GL / 2)) != 0);
                qf = 1.f;
                if (j < NV && g >= 0 && g < groups) {
                    const float m = __uint_as_float(gm[g]);
                    qf = quant_plain(m) ? quant_factor<KIND>(m) : -1.f;
                }
            }
            if constexpr (GROUP && !meet) {
                // The maximum of a group from its lanes (16 of a 16-bit type,
                // 32 of float32); lane j of them divides for their vector j
                // and writes its scale: one division a row, not one a vector.
                float mine = 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    vmost[j] = __uint_as_float(lanes_max<GL>(__float_as_uint(vmost[j])));
                    if ((lane & (GL - 1)) == j) mine = vmost[j];
                }
                qf = quant_factor<KIND>(mine);
                const int at = (ts - lane) + (lane & (GL - 1)) * tpr + (lane & ~(GL - 1));  // its vector
                if ((lane & (GL - 1)) < NV && at < ve) scale[at / GL] = quant_scale<KIND>(rs, mine);
            }
            const CodePlace<V> place(lane, (!ACROSS && !SHIFT) || p.codes_aligned ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(out) & (V - 1)));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v0 = v_base + (ts - lane) + j * tpr;
                if (!FULL && v0 >= ve) break;  // the whole warp
                float *t = held + j * V;
                uint2 code = make_uint2(0, 0);
                if constexpr (meet) {
                    // of the first of a group's vectors, s elements are the
                    // group's before it
                    const int split = (lane & (GL - 1)) == 0 ? s : 0, of = lane & ~(GL - 1);
                    const float f = __shfl_sync(0xffffffffu, qf, of + j);
                    const float f1 = __shfl_sync(0xffffffffu, qf, of + GL / 2 + j), f0 = split ? f1 : f;
                    if (f > 0.f && f0 > 0.f) {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const float2 w = pair_mul(pair_at(t, i), make_float2(2 * i < split ? f0 : f,
                                                                                 2 * i + 1 < split ? f0 : f));
                            t[2 * i] = w.x, t[2 * i + 1] = w.y;
                        }
                        code.x = quant4_finite<KIND>(t);
                        if constexpr (V == 8) code.y = quant4_finite<KIND>(t + 4);
                    } else {
                        const int v = v0 + lane, g = v / GL;
                        const float a = v < ve ? __uint_as_float(gm[g]) : 1.f;
                        const float a0 = split && v < ve && g > 0 ? __uint_as_float(gm[g - 1]) : a;
                        code.x = quant4_split<KIND>(t[0], t[1], t[2], t[3], split, a0, a);
                        if constexpr (V == 8) code.y = quant4_split<KIND>(t[4], t[5], t[6], t[7], split - 4, a0, a);
                    }
                } else if constexpr (GROUP) {
                    const float f = __shfl_sync(0xffffffffu, qf, (lane & ~(GL - 1)) + j);
                    code = quant_vector<KIND, V>(t, f, vmost[j]);
                } else {
                    code = quant_vector<KIND, V>(t, qf, most);
                }
                if constexpr (!ACROSS && !SHIFT) {
                    if (FULL || v0 + lane < ve) store_code<V>(out + (v0 + lane) * V, code);
                } else {
                    const int lo = meet && v0 < vb ? V : 0, n = SHIFT ? N - v0 * V : (ve - v0) * V;
                    if (n >= 32 * V && lo == 0)
                        place.store(out + v0 * V, code, lane);
                    else
                        store_codes_part<V>(out + v0 * V, code, lane, lo, min(n, 32 * V), place.m);
                }
            }
            if (ACROSS && ce >= 0) {
                const float a = meet ? __uint_as_float(gm[(ce - s) / kQuantGroup]) : most;
                const float f = meet ? quant_factor<KIND>(a) : qf;
                out[ce] = quant1<KIND>((he * (quant_tiny(a) ? kRaise : 1.f)) * f);
            }
        }
        buf = buf == 2 ? 0 : buf + 1;
        pos.next(S);
    }
    // after a wait ran out: let the copies this slot still has in flight land
    // (bounded) before the CTA exits
    if (issuer && lane == 0) {
        for (int kk = k; kk < issued; ++kk) {
            if (!mbar_wait_bounded(&bar[kk % S], (kk / S) & 1, kDrainNs)) {
                record_error(p.err, kErrDrain);
                break;
            }
        }
    }
}

template <typename T, int KIND, bool RES, bool GROUP, int NV, int LIE>
cudaError_t rms_out_ring_start(const OutParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_smem_optin(rms_out_ring_kernel<T, KIND, RES, GROUP, NV, LIE>, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(rms_out_ring_kernel<T, KIND, RES, GROUP, NV, LIE>, p.G, kOutThreads, smem, s, p);
}

template <typename T, int KIND, bool RES, bool GROUP, int NV>
cudaError_t rms_out_ring_lie(int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    if constexpr ((NV & (NV - 1)) == 0) {
        if (lie == kLieFull) return rms_out_ring_start<T, KIND, RES, GROUP, NV, kLieFull>(p, smem, s);
    }
    if (lie == kLieWhole) return rms_out_ring_start<T, KIND, RES, GROUP, NV, kLieWhole>(p, smem, s);
    // rows across 16-byte boundaries
    return rms_out_ring_start<T, KIND, RES, GROUP, NV, RES ? kLieAcross : kLieShift>(p, smem, s);
}

template <typename T, int KIND, bool RES, bool GROUP>
cudaError_t rms_out_ring_nv(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (nv) {
        case 1: return rms_out_ring_lie<T, KIND, RES, GROUP, 1>(lie, p, smem, s);
        case 2: return rms_out_ring_lie<T, KIND, RES, GROUP, 2>(lie, p, smem, s);
        case 3: return rms_out_ring_lie<T, KIND, RES, GROUP, 3>(lie, p, smem, s);
        case 4: return rms_out_ring_lie<T, KIND, RES, GROUP, 4>(lie, p, smem, s);
    }
    if constexpr (sizeof(T) == 4) {
        if (nv == 6) return rms_out_ring_lie<T, KIND, RES, GROUP, 6>(lie, p, smem, s);
        if (nv == 8) return rms_out_ring_lie<T, KIND, RES, GROUP, 8>(lie, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, int KIND, bool RES>
cudaError_t rms_out_ring_group(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    if constexpr (KIND != kOutSame) {
        if (p.group) return rms_out_ring_nv<T, KIND, RES, true>(nv, lie, p, smem, s);
    }
    return rms_out_ring_nv<T, KIND, RES, false>(nv, lie, p, smem, s);
}

template <typename T>
cudaError_t rms_out_ring_dispatch(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    const bool res = p.res != nullptr;
    switch (p.kind) {
        case kOutSame: return res ? rms_out_ring_group<T, kOutSame, true>(nv, lie, p, smem, s) : cudaErrorInvalidValue;
        case kOutE4M3:
            return res ? rms_out_ring_group<T, kOutE4M3, true>(nv, lie, p, smem, s)
                       : rms_out_ring_group<T, kOutE4M3, false>(nv, lie, p, smem, s);
        case kOutInt8:
            return res ? rms_out_ring_group<T, kOutInt8, true>(nv, lie, p, smem, s)
                       : rms_out_ring_group<T, kOutInt8, false>(nv, lie, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// Short rows: L lanes of a warp to a row, so a warp has 32 / L rows at once and
// a row costs no exchange beyond the warp; loads go straight to registers, many
// warps on an SM hide them (65536x256 float32 37 us, 7.2 TB/s with the outputs
// partly in L2; 29631x88 bf16 to e4m3 7.1 us, with the ring 18.7; 100x255 2.2
// us, 3.8).  Bound by the launch on few rows, by latency on many very short.  C: elements to an access, a 16-byte vector's or
// one (rows that do not lie on 16 bytes); a lane owns NV accesses, L apart.
// ---------------------------------------------------------------------------
constexpr int kShortThreads = 256;

template <typename T, int KIND, bool GROUP, int L, int NV, bool VEC>
__global__ void __launch_bounds__(kShortThreads) rms_out_short_kernel(const OutParams p) {
    using Tr = Traits<T>;
    constexpr int C = VEC ? Tr::kVec : 1;
    constexpr int E = NV * C;
    constexpr bool QUANT = KIND != kOutSame;
    static_assert(!GROUP || L == 32, "groups of a row that the whole warp holds");
    // groups of 128 columns: of GL lanes each in every access (vectors), or
    // of 128 / L accesses of all lanes (elements)
    constexpr int GL = VEC ? kQuantGroup / C : 32, NG = !GROUP ? 1 : VEC ? NV : NV * L / kQuantGroup;
    const int N = p.N, lane = threadIdx.x & (L - 1);
    const bool res = QUANT ? p.res != nullptr : true;
    const float inv_n = 1.0f / static_cast<float>(N);
    griddep_wait();  // whatever is before this kernel on the stream
    griddep_launch_dependents();
    float gam[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (lane + (e / C) * L) * C + e % C;
        gam[e] = c < N ? Tr::load1(static_cast<const T *>(p.gamma) + c) : 0.f;
    }
    const int64_t rows = (int64_t)gridDim.x * (kShortThreads / L);
    // rounds are the whole warp's: its lanes meet in shuffles
    for (int64_t r0 = (blockIdx.x * (int64_t)kShortThreads + threadIdx.x) / 32 * (32 / L); r0 < p.M; r0 += rows) {
        const int64_t row = r0 + (threadIdx.x & 31) / L;
        const bool live = row < p.M;
        const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
        const T *r = res ? static_cast<const T *>(p.res) + row * p.ld_res : nullptr;
        T *h = res ? static_cast<T *>(p.h) + row * p.ld_h : nullptr;
        float f[E];
        if constexpr (VEC) {
            uint4 x4[NV], r4[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * L) * C;
                const bool in = live && c < N;
                x4[j] = in ? *reinterpret_cast<const uint4 *>(x + c) : make_uint4(0, 0, 0, 0);
                if (res) r4[j] = in ? *reinterpret_cast<const uint4 *>(r + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * L) * C;
                float a[C];
                Tr::unpack(x4[j], a);
                if (res) {
                    float b[C];
                    Tr::unpack(r4[j], b);
#pragma unroll
                    for (int e = 0; e < C; ++e) a[e] += b[e];
                    const uint4 h4 = Tr::pack(a);
                    if (live && c < N) *reinterpret_cast<uint4 *>(h + c) = h4;
                    Tr::unpack(h4, a);
                }
#pragma unroll
                for (int e = 0; e < C; ++e) f[j * C + e] = a[e];
            }
        } else {
            float b[E];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * L;
                f[j] = live && c < N ? Tr::load1(x + c) : 0.f;
                if (res) b[j] = live && c < N ? Tr::load1(r + c) : 0.f;
            }
            if (res) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = lane + j * L;
                    f[j] = round_to<T>(f[j] + b[j]);
                    if (live && c < N) Tr::store1(h + c, f[j]);
                }
            }
        }
        float sum = 0.f, most[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) most[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sum = fmaf(f[e], f[e], sum);
            if constexpr (QUANT) {
                f[e] *= gam[e];
                most[e / (E / NG)] = max_nan(most[e / (E / NG)], fabsf(f[e]));
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (QUANT && (!GROUP || o < GL)) {
#pragma unroll
                for (int g = 0; g < NG; ++g) most[g] = max_nan(most[g], __shfl_xor_sync(0xffffffffu, most[g], o));
            }
        }
        const float rs = __frsqrt_rn(fmaf(sum, inv_n, p.eps));
        if (!live) continue;
        if (lane == 0) {
            p.rstd[row] = rs;
            if constexpr (QUANT && !GROUP) p.scale[row] = quant_scale<KIND>(rs, most[0]);
        }
        if constexpr (GROUP) {
            const int groups = (N + kQuantGroup - 1) / kQuantGroup;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int at = VEC ? lane / GL + g * (32 / GL) : g;
                if (lane % GL == 0 && at < groups) p.scale[row * groups + at] = quant_scale<KIND>(rs, most[g]);
            }
        }
        if constexpr (!QUANT) {
            T *y = static_cast<T *>(p.out) + row * p.ld_out;
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = gam[e] * (f[e] * rs);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * L) * C;
                if (c < N) {
                    if constexpr (VEC)
                        *reinterpret_cast<uint4 *>(y + c) = Tr::pack(f + j * C);
                    else
                        Tr::store1(y + c, f[j]);
                }
            }
        } else {
            uint8_t *q = static_cast<uint8_t *>(p.out) + row * p.ld_out;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float qf = quant_factor<KIND>(most[g]), raise = quant_tiny(most[g]) ? kRaise : 1.f;
#pragma unroll
                for (int e = 0; e < E / NG; ++e) f[g * (E / NG) + e] = (f[g * (E / NG) + e] * raise) * qf;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * L) * C;
                if (c < N) {
                    if constexpr (VEC) {
                        const float *t = f + j * C;
                        uint2 code;
                        code.x = quant4<KIND>(t[0], t[1], t[2], t[3]);
                        if constexpr (C == 8) {
                            code.y = quant4<KIND>(t[4], t[5], t[6], t[7]);
                            *reinterpret_cast<uint2 *>(q + c) = code;
                        } else {
                            *reinterpret_cast<uint32_t *>(q + c) = code.x;
                        }
                    } else {
                        q[c] = quant1<KIND>(f[j]);
                    }
                }
            }
        }
    }
}

template <typename T, int KIND, bool GROUP, int L, int NV, bool VEC>
cudaError_t rms_out_short_launch(const OutParams &p, int sms, cudaStream_t s) {
    const int64_t want = (p.M + kShortThreads / L - 1) / (kShortThreads / L), most = (int64_t)sms * 8;
    return launch_dependent(rms_out_short_kernel<T, KIND, GROUP, L, NV, VEC>,
                            static_cast<int>(want < most ? want : most), kShortThreads, 0, s, p);
}

// vec: rows of whole 16-byte vectors, codes that can be stored V at a time.
// Groups of columns: rows longer than one (a shorter row is one group).
template <typename T, int KIND>
cudaError_t rms_out_short_kind(bool vec, const OutParams &p, int sms, cudaStream_t s) {
    const int nvec = p.N / Traits<T>::kVec;
    if constexpr (KIND != kOutSame) {
        if (p.group) {
            if (vec && nvec <= 32) return rms_out_short_launch<T, KIND, true, 32, 1, true>(p, sms, s);
            if (vec) return rms_out_short_launch<T, KIND, true, 32, 2, true>(p, sms, s);
            if (p.N <= 256) return rms_out_short_launch<T, KIND, true, 32, 8, false>(p, sms, s);
            return rms_out_short_launch<T, KIND, true, 32, 16, false>(p, sms, s);
        }
    }
    if (vec) {
        if (nvec <= 8) return rms_out_short_launch<T, KIND, false, 8, 1, true>(p, sms, s);
        if (nvec <= 16) return rms_out_short_launch<T, KIND, false, 16, 1, true>(p, sms, s);
        if (nvec <= 32) return rms_out_short_launch<T, KIND, false, 32, 1, true>(p, sms, s);
        return rms_out_short_launch<T, KIND, false, 32, 2, true>(p, sms, s);
    }
    if (p.N <= 64) return rms_out_short_launch<T, KIND, false, 32, 2, false>(p, sms, s);
    if (p.N <= 128) return rms_out_short_launch<T, KIND, false, 32, 4, false>(p, sms, s);
    if (p.N <= 256) return rms_out_short_launch<T, KIND, false, 32, 8, false>(p, sms, s);
    return rms_out_short_launch<T, KIND, false, 32, 16, false>(p, sms, s);
}

template <typename T>
cudaError_t rms_out_short_dispatch(bool vec, const OutParams &p, int sms, cudaStream_t s) {
    switch (p.kind) {
        case kOutSame: return rms_out_short_kind<T, kOutSame>(vec, p, sms, s);
        case kOutE4M3: return rms_out_short_kind<T, kOutE4M3>(vec, p, sms, s);
        case kOutInt8: return rms_out_short_kind<T, kOutInt8>(vec, p, sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbn
