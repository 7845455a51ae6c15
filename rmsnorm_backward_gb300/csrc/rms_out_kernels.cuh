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
        const float2 k2 = make_float2(kRound, kRound);
        const float2 a = pair_add(make_float2(t[0], t[1]), k2), b = pair_add(make_float2(t[2], t[3]), k2);
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
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
// read once, h is written once and read by nobody.
//
// SHIFT: rows that do not start or end on 16 bytes, all tensors' alike (the
// host checks that): a row is copied with the up to 14 bytes before and after
// it that share its first and last 16 bytes (never beyond the tensor's first
// and last element: those two ends are copied element by element).  Only the
// vectors that lie wholly in the row are the threads'; the elements before
// and after them go to the lanes of the slot's last warp, one each.
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
// of which the first `live` lanes' exist.  Where the places do not start on
// a multiple of V bytes, a lane joins the end of the lane's before it to its
// own, and the warp's first and last bytes go one by one.
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
    const unsigned m = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & (V - 1));
    uint64_t own = code.x;
    if constexpr (V == 8) own |= static_cast<uint64_t>(code.y) << 32;
    const uint64_t prev = __shfl_up_sync(0xffffffffu, own, 1);
    if (lane < live) {
        if (lane > 0) {
            const uint64_t w = m ? (own << (8 * m)) | (prev >> (8 * (V - m))) : own;
            if constexpr (V == 8)
                *reinterpret_cast<uint64_t *>(p - m) = w;
            else
                *reinterpret_cast<uint32_t *>(p - m) = static_cast<uint32_t>(w);
        } else {
            for (unsigned e = 0; e < V - m; ++e) p[e] = static_cast<uint8_t>(own >> (8 * e));
        }
        if (lane == live - 1)
            for (unsigned e = V - m; e < V; ++e) p[e] = static_cast<uint8_t>(own >> (8 * e));
    }
}

template <typename T, int KIND, int NV, bool SHIFT>
__global__ void __launch_bounds__(kOutThreads, 1) rms_out_ring_kernel(const OutParams p) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int E = NV * V;
    constexpr bool QUANT = KIND != kOutSame;
    extern __shared__ __align__(128) unsigned char smem[];

    const int tid = threadIdx.x, tpr = p.tpr, W = tpr >> 5, slots = p.slots;
    const int slot = tid / tpr, ts = tid - slot * tpr;
    const int warp = ts >> 5, lane = tid & 31;
    const bool res = QUANT ? p.res != nullptr : true;
    const bool group = QUANT && p.group;
    const int streams = res ? 2 : 1;
    const bool issuer = warp == 0;
    const int N = p.N, S = p.stages;
    const uint32_t rowb = static_cast<uint32_t>(p.nvec) * 16;
    const int groups = (N + kQuantGroup - 1) / kQuantGroup;
    const OutLayout L = out_layout(slots, S, streams, p.nvec, SHIFT && group ? groups : 0);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L.bar);
    float *reds = reinterpret_cast<float *>(smem + L.red);
    int *flags = reinterpret_cast<int *>(smem + L.flag);

    // this CTA's rows: first + step*i for i < nrows, all of one shift; the
    // slot's: i = slot + k*slots
    const int64_t first = blockIdx.x;
    const int step = p.G;
    const int nrows = static_cast<int>((p.M - first + step - 1) / step);
    const int ns = slot < slots && slot < nrows ? (nrows - slot + slots - 1) / slots : 0;
    // the row starts s elements into its first vector; vectors [vb, ve) lie
    // wholly in it
    const int s = SHIFT ? row_shift(first, p.shift0, p.shift_step, V) : 0;
    const int nvec = SHIFT ? (s + N + V - 1) / V : p.nvec;
    const int vb = s > 0 ? 1 : 0, ve = (s + N) / V;
    // the lane's element beside them, as a place in the staged row: s <= ce < s + N, or -1
    int ce = -1;
    if (SHIFT && warp == W - 1) {
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
    if (SHIFT && group)
        for (int i = tid; i < slots * 3 * groups; i += kOutThreads) reinterpret_cast<uint32_t *>(smem + L.gmax)[i] = 0;
    if (tid < slots) flags[tid] = 0;
    __syncthreads();

    // lane t < streams of the issuing warp copies tensor t's rows
    unsigned char *ring = smem + (size_t)slot * S * streams * rowb;
    uint64_t *bar = bars + slot * S;
    const T *base = static_cast<const T *>(lane == 0 || !res ? p.x : p.res);
    const int64_t ld = lane == 0 || !res ? p.ld_x : p.ld_res;
    const T *src = base + (first + (int64_t)slot * step) * ld - s;
    int issued = 0, pst = 0;
    const int64_t row_step = (int64_t)slots * step;
    const int64_t src_step = row_step * ld;
    auto issue = [&]() {
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16;
        uint32_t from = 0, to = bytes;
        unsigned char *dst = ring + ((size_t)pst * streams + lane) * rowb;
        const int64_t row = SHIFT ? first + slot * (int64_t)step + issued * row_step : 0;
        if (SHIFT && (row == 0 || row == p.M - 1)) {
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
        src += src_step;
        if (++pst == S) pst = 0;
        ++issued;
    };
    if (issuer)
        while (issued < S && issued < ns) issue();

    const T *gamma = static_cast<const T *>(p.gamma) - s;  // by place in the staged row
    const bool gvec = (reinterpret_cast<uintptr_t>(gamma) & 15) == 0;
    float gam[E];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = vb + ts + j * tpr;
        if (v < ve && gvec) {
            Tr::unpack(ld_global_nc_v4(gamma + v * V), gam + j * V);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) gam[j * V + e] = v < ve ? Tr::load1(gamma + v * V + e) : 0.f;
        }
    }
    const float ge = ce >= 0 ? Tr::load1(gamma + ce) : 0.f;

    const float inv_n = 1.0f / static_cast<float>(N);
    float *red = reds + (slot < slots ? slot : 0) * 4 * kRedStride;
    uint32_t *gmax = reinterpret_cast<uint32_t *>(smem + L.gmax) + (slot < slots ? slot : 0) * 3 * groups;
    volatile int *flag = flags + slot;
    RingPos pos;
    int buf = 0;  // k mod 3
    int k = 0;
    int64_t row = first + slot * (int64_t)step;
    T *h = static_cast<T *>(p.h) + (res ? row * p.ld_h - s : 0);
    using Out = typename std::conditional<QUANT, uint8_t, T>::type;
    Out *out = static_cast<Out *>(p.out) + row * p.ld_out - s;
    const int64_t h_step = row_step * p.ld_h, out_step = row_step * p.ld_out;
    for (; k < ns; ++k, row += row_step, h += h_step, out += out_step) {
        const bool timed_out = !mbar_wait_bounded(&bar[pos.stage], pos.parity);
        if (timed_out) record_error(p.err, kErrWaitFull);
        const unsigned char *sx = ring + (size_t)pos.stage * streams * rowb;
        uint32_t *gm = gmax + buf * groups;
        float sum = 0.f, held[E], he = 0.f;
        uint32_t most = 0, vmost[QUANT ? NV : 1];  // |v| as bits: the order of the values, NaN above all
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + ts + j * tpr;
            if constexpr (QUANT) vmost[j] = 0;
            if (v < ve) {
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
                    st_global_cs_v4(h + (size_t)v * V, h4);
                    Tr::unpack(h4, f);
                }
                float2 t = pair_mul(pair_at(f, 0), pair_at(f, 0));
#pragma unroll
                for (int i = 1; i < V / 2; ++i) t = pair_fma(pair_at(f, i), pair_at(f, i), t);
                sum += t.x + t.y;
                if constexpr (QUANT) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 w = pair_mul(pair_at(gam + j * V, i), pair_at(f, i));
                        held[j * V + 2 * i] = w.x, held[j * V + 2 * i + 1] = w.y;
                    }
                    float m = fabsf(held[j * V]);
#pragma unroll
                    for (int e = 1; e < V; ++e) m = max_nan(m, fabsf(held[j * V + e]));
                    vmost[j] = __float_as_uint(m);
                    if (SHIFT && group) {
                        const int c0 = v * V - s, split = kQuantGroup - (c0 & (kQuantGroup - 1));
                        if (split >= V) {
                            atomicMax(gm + c0 / kQuantGroup, vmost[j]);
                        } else {
                            uint32_t m0 = 0, m1 = 0;
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                const uint32_t b = abs_bits(held[j * V + e]);
                                if (e < split)
                                    m0 = max(m0, b);
                                else
                                    m1 = max(m1, b);
                            }
                            atomicMax(gm + c0 / kQuantGroup, m0);
                            atomicMax(gm + c0 / kQuantGroup + 1, m1);
                        }
                    }
                    most = max(most, vmost[j]);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) held[j * V + e] = f[e];
                }
            }
        }
        if (SHIFT && ce >= 0) {
            he = Tr::load1(reinterpret_cast<const T *>(sx) + ce);
            if (res) {
                he = round_to<T>(he + Tr::load1(reinterpret_cast<const T *>(sx + rowb) + ce));
                Tr::store1(h + ce, he);
            }
            sum = fmaf(he, he, sum);
            if constexpr (QUANT) {
                he *= ge;
                most = max(most, abs_bits(he));
                if (group) atomicMax(gm + (ce - s) / kQuantGroup, abs_bits(he));
            }
        }
        // the exchange: warp sums (and maxima), added in warp order
        sum = warp_sum(sum);
        if constexpr (QUANT) most = __reduce_max_sync(0xffffffffu, most);
        if (W > 1) {
            float *b = red + (k & 1) * 2 * kRedStride;
            if (timed_out) *flag = 1;
            if (lane == 0) {
                b[warp] = sum;
                if constexpr (QUANT) b[kRedStride + warp] = __uint_as_float(most);
            }
            named_barrier(1 + slot, tpr);
            sum = 0.f;
            for (int w = 0; w < W; w += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(b + w);
                sum += t.x;
                sum += t.y;
                sum += t.z;
                sum += t.w;
                if constexpr (QUANT) {
                    const uint4 m = *reinterpret_cast<const uint4 *>(b + kRedStride + w);
                    most = max(max(max(most, m.x), max(m.y, m.z)), m.w);
                }
            }
            if (*flag) break;
        } else {
            __syncwarp();  // the group maxima of the warp's lanes
            if (__any_sync(0xffffffffu, timed_out)) break;
        }
        // the slot has the row in registers: refill its stage
        if (issuer && issued < ns) {
            fence_proxy_async();
            issue();
        }
        float rs = 0.f;
        if (!QUANT || group || ts == 0) rs = __frsqrt_rn(fmaf(sum, inv_n, p.eps));
        if constexpr (!QUANT) {
            T *y = out;
            const float2 rs2 = make_float2(rs, rs);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v = vb + ts + j * tpr;
                if (v < ve) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 t = pair_mul(pair_at(gam + j * V, i), pair_mul(pair_at(held + j * V, i), rs2));
                        o[2 * i] = t.x, o[2 * i + 1] = t.y;
                    }
                    st_global_cs_v4(y + (size_t)v * V, Tr::pack(o));
                }
            }
            if (SHIFT && ce >= 0) Tr::store1(y + ce, ge * (he * rs));
            if (ts == 0) p.rstd[row] = rs;
        } else {
            uint8_t *q = out;
            float *scale = p.scale + (group ? row * groups : row);
            float qf = quant_factor<KIND>(__uint_as_float(most));
            if (SHIFT && group) {
                // the maxima of row k-1, read by nobody any more, for row k+2
                uint32_t *clear = gmax + (buf == 0 ? 2 : buf - 1) * groups;
                for (int i = ts; i < groups; i += tpr) {
                    clear[i] = 0;
                    scale[i] = quant_scale<KIND>(rs, __uint_as_float(gm[i]));
                }
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v0 = vb + (ts - lane) + j * tpr, v = v0 + lane;
                if (v0 >= ve) break;  // the whole warp
                float *t = held + j * V;
                uint2 code = make_uint2(0, 0);
                uint32_t m = most;
                if (SHIFT && group) {
                    // the vector's columns in one group or two
                    const int c0 = v < ve ? v * V - s : 0, split = kQuantGroup - (c0 & (kQuantGroup - 1));
                    const uint32_t m0 = gm[c0 / kQuantGroup], m1 = split < V ? gm[c0 / kQuantGroup + 1] : m0;
                    const float f0 = quant_factor<KIND>(__uint_as_float(m0));
                    const float f1 = split < V ? quant_factor<KIND>(__uint_as_float(m1)) : f0;
                    const float r0 = quant_tiny(__uint_as_float(m0)) ? kRaise : 1.f;
                    const float r1 = quant_tiny(__uint_as_float(m1)) ? kRaise : 1.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) t[e] = (t[e] * (e < split ? r0 : r1)) * (e < split ? f0 : f1);
                    m = max(m0, m1);
                } else {
                    if (group) {
                        // 128 columns: 16 lanes of a 16-bit type, 32 of float32
                        m = vmost[j];
#pragma unroll
                        for (int o = kQuantGroup / V / 2; o > 0; o >>= 1)
                            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        qf = quant_factor<KIND>(__uint_as_float(m));
                        if ((lane & (kQuantGroup / V - 1)) == 0 && v < ve)
                            scale[v * V / kQuantGroup] = quant_scale<KIND>(rs, __uint_as_float(m));
                    }
                    if (quant_tiny(__uint_as_float(m))) {
#pragma unroll
                        for (int e = 0; e < V; ++e) t[e] *= kRaise;
                    }
                    const float2 f2 = make_float2(qf, qf);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 w = pair_mul(pair_at(t, i), f2);
                        t[2 * i] = w.x, t[2 * i + 1] = w.y;
                    }
                }
                if (KIND == kOutInt8 && m >= 0x7f800000u) {
                    code.x = quant4<KIND>(t[0], t[1], t[2], t[3]);
                    if constexpr (V == 8) code.y = quant4<KIND>(t[4], t[5], t[6], t[7]);
                } else {
                    code.x = quant4_finite<KIND>(t);
                    if constexpr (V == 8) code.y = quant4_finite<KIND>(t + 4);
                }
                store_codes<V>(q + (size_t)v0 * V, code, lane, ve - v0 < 32 ? ve - v0 : 32, p.codes_aligned);
            }
            if (SHIFT && ce >= 0) {
                const float a = __uint_as_float(group ? gm[(ce - s) / kQuantGroup] : most);
                q[ce] = quant1<KIND>((he * (quant_tiny(a) ? kRaise : 1.f)) * quant_factor<KIND>(a));
            }
            if (ts == 0) {
                p.rstd[row] = rs;
                if (!group) *scale = quant_scale<KIND>(rs, __uint_as_float(most));
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

template <typename T, int KIND, int NV, bool SHIFT>
cudaError_t rms_out_ring_launch(const OutParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_smem_optin(rms_out_ring_kernel<T, KIND, NV, SHIFT>, done);
    if (e != cudaSuccess) return e;
    rms_out_ring_kernel<T, KIND, NV, SHIFT><<<p.G, kOutThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int KIND>
cudaError_t rms_out_ring_nv(int nv, bool shift, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (nv) {
#define GBN_CASE(n) \
    case n: return shift ? rms_out_ring_launch<T, KIND, n, true>(p, smem, s) : rms_out_ring_launch<T, KIND, n, false>(p, smem, s)
        GBN_CASE(1);
        GBN_CASE(2);
        GBN_CASE(3);
        GBN_CASE(4);
#undef GBN_CASE
        case 6:
        case 8:
            if constexpr (sizeof(T) == 4) {
                if (nv == 6)
                    return shift ? rms_out_ring_launch<T, KIND, 6, true>(p, smem, s)
                                 : rms_out_ring_launch<T, KIND, 6, false>(p, smem, s);
                return shift ? rms_out_ring_launch<T, KIND, 8, true>(p, smem, s)
                             : rms_out_ring_launch<T, KIND, 8, false>(p, smem, s);
            }
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t rms_out_ring_dispatch(int nv, bool shift, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (p.kind) {
        case kOutSame: return rms_out_ring_nv<T, kOutSame>(nv, shift, p, smem, s);
        case kOutE4M3: return rms_out_ring_nv<T, kOutE4M3>(nv, shift, p, smem, s);
        case kOutInt8: return rms_out_ring_nv<T, kOutInt8>(nv, shift, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbn
