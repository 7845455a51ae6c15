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
template <int KIND>
__device__ __forceinline__ float quant_scale(float rstd, float a) {
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
// threads that wrote it.  For rows too wide for the ring and tensors whose rows
// lie differently to 16-byte boundaries (4096x20000 bf16 259 us, 2.5 TB/s: two
// bytes to a load keep too little in flight).
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
// to e4m3 by 128 columns, 8192x16384, 145 us, 6.5 TB/s.  Without the residual
// there are fewer bytes to hide the work of a code behind: 16384x4096 bf16 to
// e4m3 40 us, 5.0 TB/s, where the warps' instructions bound it.
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
//    and the elements before and after them go to the lanes of the slot's last
//    warp, one each.  The maxima of groups then meet in shared memory, as
//    their borders run through vectors.
// The first two leave out what the third needs: 16384x4096 bf16 to e4m3, without
// the residual, 67 us as kLieAcross alone, 52 as kLieFull.
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

// Stores a warp's codes, V a lane at consecutive places from `at` of lane 0,
// of which the first `live` lanes' exist (live > 0).  Where the places do not
// start on a multiple of V bytes, a lane joins the end of the lane's before
// it to its own; the warp's first and last bytes, which have no such
// neighbour, go one to a lane.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t *at, uint2 code, int lane, int live, bool aligned) {
    uint8_t *p = at + lane * V;
    if (aligned) {
        if (lane < live) {
            if constexpr (V == 8)
                *reinterpret_cast<uint2 *>(p) = code;
            else
                *reinterpret_cast<uint32_t *>(p) = code.x;
        }
        return;
    }
    const int m = static_cast<int>(reinterpret_cast<uintptr_t>(at) & (V - 1));
    uint64_t own = code.x;
    if constexpr (V == 8) own |= static_cast<uint64_t>(code.y) << 32;
    const uint64_t prev = __shfl_up_sync(0xffffffffu, own, 1);
    if (lane > 0 && lane < live) {
        const uint64_t w = m ? (own << (8 * m)) | (prev >> (8 * (V - m))) : own;
        if constexpr (V == 8)
            *reinterpret_cast<uint64_t *>(p - m) = w;
        else
            *reinterpret_cast<uint32_t *>(p - m) = static_cast<uint32_t>(w);
    }
    // lanes 0 .. V-1: the first lane's bytes below V - m; lanes V .. 2V-1: the
    // last one's from there
    const uint64_t end = __shfl_sync(0xffffffffu, own, lane < V ? 0 : live - 1);
    const int e = lane & (V - 1);
    if (lane < 2 * V && (lane < V) == (e < V - m)) at[(lane < V ? 0 : (live - 1) * V) + e] = static_cast<uint8_t>(end >> (8 * e));
}

template <typename T, int KIND, bool GROUP, int NV, int LIE>
__global__ void __launch_bounds__(kOutThreads, 1) rms_out_ring_kernel(const OutParams p) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int E = NV * V;
    constexpr bool QUANT = KIND != kOutSame;
    constexpr bool FULL = LIE == kLieFull, ACROSS = LIE == kLieAcross;
    constexpr bool GRAW = sizeof(T) == 2 && NV > 3;  // gamma kept in the storage type
    using Out = typename std::conditional<QUANT, uint8_t, T>::type;
    extern __shared__ __align__(128) unsigned char smem[];

    const int tid = threadIdx.x, tpr = p.tpr, W = tpr >> 5, slots = p.slots;
    const int slot = tid / tpr, ts = tid - slot * tpr;
    const int warp = ts >> 5, lane = tid & 31;
    const bool res = QUANT ? p.res != nullptr : true;
    const int streams = res ? 2 : 1;
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
    // the row starts s elements into its first vector; vectors [vb, ve) lie
    // wholly in it
    const int s = !ACROSS ? 0 : row_shift(blockIdx.x, p.shift0, p.shift_step, V);
    const int nvec = !ACROSS ? p.nvec : (s + N + V - 1) / V;
    const int vb = s > 0 ? 1 : 0, ve = (s + N) / V;
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
    if (meet)
        for (int i = tid; i < slots * 3 * groups; i += kOutThreads) reinterpret_cast<uint32_t *>(smem + L.gmax)[i] = 0;
    if (tid < slots) flags[tid] = 0;
    __syncthreads();
    griddep_wait();  // whatever is before this kernel on the stream
    griddep_launch_dependents();

    // lane t < streams of the issuing warp copies tensor t's rows
    unsigned char *ring = smem + (size_t)slot * S * streams * rowb;
    uint64_t *bar = bars + slot * S;
    const T *base = static_cast<const T *>(lane == 0 || !res ? p.x : p.res);
    const int64_t ld = lane == 0 || !res ? p.ld_x : p.ld_res;
    const T *src = base + row * ld - s;
    int issued = 0, pst = 0;
    auto issue = [&]() {
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16;
        uint32_t from = 0, to = bytes;
        unsigned char *dst = ring + (pst * streams + lane) * rowb;
        const int64_t r = !ACROSS ? 1 : row0 + issued * row_step;
        if (ACROSS && (r == 0 || r == p.M - 1)) {
            // the tensors' first and last rows: nothing outside them is read
            if (lane < streams) {
                if (src < base) from = 16;
                if (src + (size_t)nvec * V > base + (p.M - 1) * ld + N) to = bytes - 16;
                T *d = reinterpret_cast<T *>(dst);
                for (int c = s; c < s + N && c < static_cast<int>(from / sizeof(T)); ++c) d[c] = src[c];
                for (int c = max(static_cast<int>(to / sizeof(T)), s); c < s + N; ++c) d[c] = src[c];
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

    const T *gamma = static_cast<const T *>(p.gamma) - s;  // by place in the staged row
    const bool gvec = (reinterpret_cast<uintptr_t>(gamma) & 15) == 0;
    float gam[GRAW ? 1 : E];
    uint4 graw[GRAW ? NV : 1];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = vb + ts + j * tpr;
        float g[V];
        if ((FULL || v < ve) && gvec) {
            Tr::unpack(ld_global_nc_v4(gamma + v * V), g);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = FULL || v < ve ? Tr::load1(gamma + v * V + e) : 0.f;
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
    uint32_t *gmax = reinterpret_cast<uint32_t *>(smem + L.gmax) + in_slot * 3 * groups;  // of rows k mod 3
    volatile int *flag = flags + slot;
    RingPos pos;
    int buf = 0;  // k mod 3
    int k = 0;
    for (; k < ns; ++k, row += row_step) {
        const bool timed_out = !mbar_wait_bounded(&bar[pos.stage], pos.parity);
        if (timed_out) record_error(p.err, kErrWaitFull);
        if (p.late && issuer && k > 0 && issued < ns) {  // the row before is in registers, this one landed
            fence_proxy_async();
            issue();
        }
        const unsigned char *sx = ring + pos.stage * streams * rowb;
        uint32_t *gm = gmax + buf * groups;
        T *h = static_cast<T *>(p.h) + (res ? row * p.ld_h - s : 0);
        float sum = 0.f, held[E], he = 0.f;
        float most = 0.f, vmost[GROUP ? NV : 1];  // max |v|, NaN if any is
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + ts + j * tpr;
            if constexpr (GROUP) vmost[j] = 0.f;
            if (FULL || v < ve) {
                float f[V];
                Tr::unpack(ld_shared_v4(sx + v * 16), f);
                if (res) {
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
                        if (meet) {
                            const int c0 = v * V - s, g = c0 / kQuantGroup, split = (g + 1) * kQuantGroup - c0;
                            if (split < V) {  // in two groups
                                float m1 = m = 0.f;
#pragma unroll
                                for (int e = 0; e < V; ++e) {
                                    if (e < split)
                                        m = max_nan(m, fabsf(held[j * V + e]));
                                    else
                                        m1 = max_nan(m1, fabsf(held[j * V + e]));
                                }
                                atomicMax(gm + g + 1, __float_as_uint(m1));
                            }
                            atomicMax(gm + g, __float_as_uint(m));
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
            if (res) {
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
        // the exchange: warp sums (and maxima, as bits: the order of the
        // values, NaN above all), added in warp order
        sum = warp_sum(sum);
        uint32_t bits = 0;
        if constexpr (QUANT && !GROUP) bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        if (W > 1) {
            float *b = red + (k & 1) * 2 * kRedStride;
            if (timed_out) *flag = 1;
            if (lane == 0) {
                b[warp] = sum;
                if constexpr (QUANT && !GROUP) b[kRedStride + warp] = __uint_as_float(bits);
            }
            named_barrier(1 + slot, tpr);
            sum = 0.f;
            for (int w = 0; w < W; w += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(b + w);
                sum += (t.x + t.y) + (t.z + t.w);
                if constexpr (QUANT && !GROUP) {
                    const uint4 m = *reinterpret_cast<const uint4 *>(b + kRedStride + w);
                    bits = max(max(max(bits, m.x), max(m.y, m.z)), m.w);
                }
            }
            if (*flag) break;
        } else {
            __syncwarp();  // the group maxima of the warp's lanes
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
        Out *out = static_cast<Out *>(p.out) + row * p.ld_out - s;
        if constexpr (!QUANT) {
            const float2 rs2 = make_float2(rs, rs);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v = vb + ts + j * tpr;
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
            if (meet) {
                // the maxima of row k-1, read by nobody any more, for row k+2
                uint32_t *clear = gmax + (buf == 0 ? 2 : buf - 1) * groups;
                for (int i = ts; i < groups; i += tpr) {
                    clear[i] = 0;
                    scale[i] = quant_scale<KIND>(rs, __uint_as_float(gm[i]));
                }
            }
            if constexpr (GROUP && !ACROSS) {
                // The maximum of a group from its lanes (16 of a 16-bit type,
                // 32 of float32); lane j of them divides for their vector j
                // and writes its scale: one division a row, not one a vector.
                constexpr int GL = kQuantGroup / V;
                float mine = 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    uint32_t b = __float_as_uint(vmost[j]);
                    if constexpr (GL == 32) {
                        b = __reduce_max_sync(0xffffffffu, b);
                    } else {
#pragma unroll
                        for (int o = GL / 2; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
                    }
                    vmost[j] = __uint_as_float(b);
                    if ((lane & (GL - 1)) == j) mine = vmost[j];
                }
                qf = quant_factor<KIND>(mine);
                const int at = (ts - lane) + (lane & (GL - 1)) * tpr + (lane & ~(GL - 1));  // its vector
                if ((lane & (GL - 1)) < NV && at < ve) scale[at / GL] = quant_scale<KIND>(rs, mine);
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v0 = vb + (ts - lane) + j * tpr, v = v0 + lane;
                if (!FULL && v0 >= ve) break;  // the whole warp
                float *t = held + j * V;
                uint2 code = make_uint2(0, 0);
                if constexpr (meet) {
                    // the vector's columns in one group or two
                    const int c0 = v < ve ? v * V - s : 0, g = c0 / kQuantGroup, split = (g + 1) * kQuantGroup - c0;
                    const float m = __uint_as_float(gm[g]), f0 = quant_factor<KIND>(m);
                    const float r0 = quant_tiny(m) ? kRaise : 1.f;
                    float f1 = f0, r1 = r0;
                    if (split < V) {
                        const float m1 = __uint_as_float(gm[g + 1]);
                        f1 = quant_factor<KIND>(m1), r1 = quant_tiny(m1) ? kRaise : 1.f;
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) t[e] = (t[e] * (e < split ? r0 : r1)) * (e < split ? f0 : f1);
                    code.x = quant4<KIND>(t[0], t[1], t[2], t[3]);
                    if constexpr (V == 8) code.y = quant4<KIND>(t[4], t[5], t[6], t[7]);
                } else if constexpr (GROUP) {
                    constexpr int GL = kQuantGroup / V;
                    const float f = __shfl_sync(0xffffffffu, qf, (lane & ~(GL - 1)) + j);
                    code = quant_vector<KIND, V>(t, f, vmost[j]);
                } else {
                    code = quant_vector<KIND, V>(t, qf, most);
                }
                store_codes<V>(out + v0 * V, code, lane, FULL || ve - v0 > 32 ? 32 : ve - v0, !ACROSS || p.codes_aligned);
            }
            if (ACROSS && ce >= 0) {
                if constexpr (GROUP) {
                    const float a = __uint_as_float(gm[(ce - s) / kQuantGroup]);
                    out[ce] = quant1<KIND>((he * (quant_tiny(a) ? kRaise : 1.f)) * quant_factor<KIND>(a));
                } else {
                    out[ce] = quant1<KIND>((he * (quant_tiny(most) ? kRaise : 1.f)) * qf);
                }
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

template <typename T, int KIND, bool GROUP, int NV, int LIE>
cudaError_t rms_out_ring_launch(const OutParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_smem_optin(rms_out_ring_kernel<T, KIND, GROUP, NV, LIE>, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(rms_out_ring_kernel<T, KIND, GROUP, NV, LIE>, p.G, kOutThreads, smem, s, p);
}

template <typename T, int KIND, bool GROUP, int NV>
cudaError_t rms_out_ring_lie(int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    if constexpr ((NV & (NV - 1)) == 0) {
        if (lie == kLieFull) return rms_out_ring_launch<T, KIND, GROUP, NV, kLieFull>(p, smem, s);
    }
    return lie == kLieAcross ? rms_out_ring_launch<T, KIND, GROUP, NV, kLieAcross>(p, smem, s)
                             : rms_out_ring_launch<T, KIND, GROUP, NV, kLieWhole>(p, smem, s);
}

template <typename T, int KIND, bool GROUP>
cudaError_t rms_out_ring_nv(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (nv) {
        case 1: return rms_out_ring_lie<T, KIND, GROUP, 1>(lie, p, smem, s);
        case 2: return rms_out_ring_lie<T, KIND, GROUP, 2>(lie, p, smem, s);
        case 3: return rms_out_ring_lie<T, KIND, GROUP, 3>(lie, p, smem, s);
        case 4: return rms_out_ring_lie<T, KIND, GROUP, 4>(lie, p, smem, s);
    }
    if constexpr (sizeof(T) == 4) {
        if (nv == 6) return rms_out_ring_lie<T, KIND, GROUP, 6>(lie, p, smem, s);
        if (nv == 8) return rms_out_ring_lie<T, KIND, GROUP, 8>(lie, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t rms_out_ring_dispatch(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (p.kind) {
        case kOutSame: return rms_out_ring_nv<T, kOutSame, false>(nv, lie, p, smem, s);
        case kOutE4M3:
            return p.group ? rms_out_ring_nv<T, kOutE4M3, true>(nv, lie, p, smem, s)
                           : rms_out_ring_nv<T, kOutE4M3, false>(nv, lie, p, smem, s);
        case kOutInt8:
            return p.group ? rms_out_ring_nv<T, kOutInt8, true>(nv, lie, p, smem, s)
                           : rms_out_ring_nv<T, kOutInt8, false>(nv, lie, p, smem, s);
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
