// rms_add_bwd_kernels.cuh -- backward of the RMSNorm with a residual's
// addition, for sm_103a; instantiated once per storage dtype in
// rms_add_bwd_f32.cu, rms_add_bwd_f16.cu and rms_add_bwd_bf16.cu.
//
// Per row, with xhat = h*rstd (recomputed from the saved rstd) and dyhat =
// dy*gamma:
//   dx = rstd*(dyhat - xhat*mean(dyhat*xhat)) + dh,
//   dgamma[j] = sum over rows of dy*xhat.
// The sum with dh is float32, before the one rounding to the storage type.
// dgamma takes the partial rows and the fixed-order column reduce of the
// other backward kernels: no atomics, the same bits from run to run.
#pragma once

#include <atomic>

#include "gbn_device.cuh"
#include "gbn_launch.h"
#include "rms_add_bwd.h"

namespace gbn {

// ---------------------------------------------------------------------------
// any N, stride and alignment, with scalar accesses: CTA b takes a contiguous
// block of rows.  First a warp to a row forms mean(dyhat*xhat); then the CTA
// goes over the rows once for each slab of 8192 columns, a thread owning eight
// of them and their dgamma sums in registers, so h and dy are read twice.
// For rows too wide for the ring (16384 elements of 16 bits, about 9650 of
// float32, less where a CTA has many rows, whose rstd it keeps) and tensors whose
// rows lie differently to 16-byte boundaries: 4096x20000 bf16 228 us, 2.9 TB/s,
// 4096x12288 float32 191 us, 4.2 TB/s.  (Accumulating in global memory in one go, 256
// threads a CTA, took 1808 us at 16384x4096 bf16.)
// ---------------------------------------------------------------------------
constexpr int kAddBwdPlainThreads = 1024, kAddBwdPlainCols = 8;

template <typename T>
__global__ void __launch_bounds__(kAddBwdPlainThreads) rms_add_bwd_plain_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    __shared__ float rs_s[kMaxRowsPerCta], a_s[kMaxRowsPerCta];
    const int N = p.N, lane = threadIdx.x & 31;
    const float inv_n = 1.0f / static_cast<float>(N);
    int64_t row0;
    int nrows;
    block_rows(p.M, p.G, blockIdx.x, row0, nrows);
    griddep_launch_dependents();
    const T *g = static_cast<const T *>(p.gamma);
    for (int i = threadIdx.x >> 5; i < nrows; i += kAddBwdPlainThreads / 32) {
        const T *h = static_cast<const T *>(p.h) + (row0 + i) * p.ld_h;
        const T *dy = static_cast<const T *>(p.dy) + (row0 + i) * p.ld_dy;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        int c = lane;
        for (; c + 96 < N; c += 128) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                s[u] = fmaf(Tr::load1(dy + c + 32 * u) * Tr::load1(g + c + 32 * u), Tr::load1(h + c + 32 * u), s[u]);
        }
        for (; c < N; c += 32) s[0] = fmaf(Tr::load1(dy + c) * Tr::load1(g + c), Tr::load1(h + c), s[0]);
        const float sum = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
        if (lane == 0) {
            const float rs = p.rstd[row0 + i];
            rs_s[i] = rs;
            a_s[i] = -rs * rs * (sum * rs * inv_n);
        }
    }
    __syncthreads();
    float *part = p.part + (size_t)blockIdx.x * p.ldp;
    for (int c0 = 0; c0 < N; c0 += kAddBwdPlainThreads * kAddBwdPlainCols) {
        float acc[kAddBwdPlainCols], gam[kAddBwdPlainCols];
#pragma unroll
        for (int j = 0; j < kAddBwdPlainCols; ++j) {
            const int c = c0 + threadIdx.x + j * kAddBwdPlainThreads;
            acc[j] = 0.f;
            gam[j] = c < N ? Tr::load1(g + c) : 0.f;
        }
        for (int i = 0; i < nrows; ++i) {
            const int64_t row = row0 + i;
            const T *h = static_cast<const T *>(p.h) + row * p.ld_h;
            const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
            const T *dh = static_cast<const T *>(p.dh) + row * p.ld_dh;
            T *dx = static_cast<T *>(p.dx) + row * p.ld_dx;
            const float rs = rs_s[i], a = a_s[i];
            float hf[kAddBwdPlainCols], df[kAddBwdPlainCols], ef[kAddBwdPlainCols];
#pragma unroll
            for (int j = 0; j < kAddBwdPlainCols; ++j) {
                const int c = c0 + threadIdx.x + j * kAddBwdPlainThreads;
                hf[j] = c < N ? Tr::load1(h + c) : 0.f;
                df[j] = c < N ? Tr::load1(dy + c) : 0.f;
                ef[j] = c < N ? Tr::load1(dh + c) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kAddBwdPlainCols; ++j) {
                const int c = c0 + threadIdx.x + j * kAddBwdPlainThreads;
                const float D = df[j] * rs;
                acc[j] = fmaf(D, hf[j], acc[j]);
                if (c < N) Tr::store1(dx + c, fmaf(D, gam[j], fmaf(hf[j], a, ef[j])));
            }
        }
#pragma unroll
        for (int j = 0; j < kAddBwdPlainCols; ++j) {
            const int c = c0 + threadIdx.x + j * kAddBwdPlainThreads;
            if (c < N) part[c] = acc[j];
        }
    }
}

// ---------------------------------------------------------------------------
// One persistent CTA per SM; its 16 warps are slots of tpr threads, and each
// slot streams its rows of h, dy and dh through a ring of shared-memory
// stages by 1-D bulk copies, which one warp of the slot issues (a lane for
// each tensor).  A thread owns NV column vectors, their gamma and their
// dgamma sums in registers.  Pass 1 takes the row from its stage into
// registers, as raw vectors, and forms sum(dyhat*h); the exchange of that sum
// within the slot shows that all of the slot is done with the stage, which is
// refilled at once; pass 2 writes dx with 16-byte streaming stores.  Where
// the raw row does not fit in registers (float32, more than 16 elements a
// thread) pass 2 reads the stage again, which is refilled a row later.  Bound by
// HBM: 16384x4096 bf16 84.7 us with the column reduce (6.33 TB/s, 95% of the
// measured copy rate; the rows alone 80.0 us), 65536x1024 82 us, 8192x16384
// 166 us; rows across 16-byte boundaries 85% (8192x4099 47 us).  (A producer warp for all slots, with mbarriers for
// the release, measured slower on aligned rows: 97 against 85 us at
// 16384x4096 bf16, 80 against 21 us at 32768x256.)
//
// SHIFT: rows that do not start or end on 16 bytes.  All four tensors' rows
// have the same shift (the host checks that), so a row is copied with the up
// to 14 bytes before and after it that share its first and last 16 bytes
// (never beyond the tensor's first and last element: those two ends are
// copied element by element).  Only the vectors that lie wholly in the row
// are the threads'; the elements before and after them go to the lanes of the
// slot's last warp, one each.
// ---------------------------------------------------------------------------
template <typename T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kAddBwdThreads, 1) rms_add_bwd_ring_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int E = NV * V;
    constexpr bool HOLD = NV <= 4;  // the row kept in registers between the passes,
    constexpr bool HOLDF = sizeof(T) == 2 && NV <= 2;  // h and dy unpacked
    // gamma: float32 in registers, or vectors of the storage type in
    // registers, or those in shared memory, as room in registers allows
    constexpr bool GFLT = sizeof(T) == 4 || NV <= 2;
    constexpr bool GSMEM = add_bwd_gamma_smem(sizeof(T), NV);
    extern __shared__ __align__(128) unsigned char smem[];

    const int tid = threadIdx.x, tpr = p.tpr, W = tpr >> 5, slots = p.slots;
    const int slot = tid / tpr, ts = tid - slot * tpr;
    const int warp = ts >> 5, lane = tid & 31;
    const bool issuer = warp == 0;
    const int N = p.N, S = p.stages;
    const uint32_t rowb = static_cast<uint32_t>(p.nvec) * 16;
    const AddBwdLayout L = add_bwd_layout(slots, S, p.nvec, p.stat_rows, GSMEM);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L.bar);
    float *st_rstd = reinterpret_cast<float *>(smem + L.stat);
    float *reds = reinterpret_cast<float *>(smem + L.red);
    int *flags = reinterpret_cast<int *>(smem + L.flag);

    // this CTA's rows: first + step*i for i < nrows, all of one phase; the
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
    for (int i = tid; i < slots * 2 * kRedStride; i += kAddBwdThreads) reds[i] = 0.f;
    if (tid < slots) flags[tid] = 0;
    __syncthreads();
    griddep_wait();  // whatever is before this kernel on the stream

    // lane t < 3 of the issuing warp copies tensor t's rows
    unsigned char *ring = smem + (size_t)slot * S * 3 * rowb;
    uint64_t *bar = bars + slot * S;
    const T *base = static_cast<const T *>(lane == 0 ? p.h : lane == 1 ? p.dy : p.dh);
    const int64_t ld = lane == 0 ? p.ld_h : lane == 1 ? p.ld_dy : p.ld_dh;
    const T *src = base + (first + (int64_t)slot * step) * ld - s;
    const int end0 = first == 0 && slot == 0 ? 0 : -1;
    const int end1 = ns > 0 && slot + (ns - 1) * slots == nrows - 1 && first + (int64_t)(nrows - 1) * step == p.M - 1 ? ns - 1 : -1;
    int issued = 0, pst = 0;
    auto issue = [&]() {
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16;
        uint32_t from = 0, to = bytes;
        unsigned char *dst = ring + ((size_t)pst * 3 + lane) * rowb;
        if (SHIFT && (issued == end0 || issued == end1)) {
            // the tensors' first and last rows: nothing outside them is read
            if (lane < 3) {
                const uint2 mid = copy_end_row<T>(reinterpret_cast<T *>(dst), src, base, base + (p.M - 1) * ld + N, s, N, bytes);
                from = mid.x, to = mid.y;
                if (to > from) mbar_expect_tx(&bar[pst], to - from);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[pst]);
        } else if (lane == 0) {
            mbar_arrive_expect_tx(&bar[pst], 3 * bytes);
        }
        if (lane < 3 && to > from) bulk_load_nohint(dst + from, src + from / sizeof(T), to - from, &bar[pst]);
        src += (int64_t)slots * step * ld;
        if (++pst == S) pst = 0;
        ++issued;
    };
    if (issuer)
        while (issued < S && issued < ns) issue();

    for (int i = tid; i < nrows; i += kAddBwdThreads) st_rstd[i] = p.rstd[first + (int64_t)i * step];
    const T *gamma = static_cast<const T *>(p.gamma) - s;  // by place in the staged row
    float gam[GFLT ? E : 1], acc[E];
    uint4 graw[GFLT || GSMEM ? 1 : NV];
    unsigned char *gs = smem + L.gam;
    if constexpr (GSMEM) {
        for (int c = vb * V + tid; c < ve * V; c += kAddBwdThreads) reinterpret_cast<T *>(gs)[c] = gamma[c];
    }
    const bool gvec = (reinterpret_cast<uintptr_t>(gamma) & 15) == 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = vb + ts + j * tpr;
        float g[V];
        if (!GSMEM && gvec && v < ve) Tr::unpack(ld_global_nc_v4(gamma + v * V), g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (!GSMEM && !(gvec && v < ve)) g[e] = v < ve ? Tr::load1(gamma + v * V + e) : 0.f;
            acc[j * V + e] = 0.f;
            if constexpr (GFLT) gam[j * V + e] = g[e];
        }
        if constexpr (!GFLT && !GSMEM) graw[j] = Tr::pack(g);
    }
    const float ge = ce >= 0 ? Tr::load1(gamma + ce) : 0.f;
    float ae = 0.f;
    __syncthreads();
    griddep_launch_dependents();

    const float inv_n = 1.0f / static_cast<float>(N);
    float *red = reds + (slot < slots ? slot : 0) * 2 * kRedStride;
    volatile int *flag = flags + slot;
    // vector v of gamma, as pairs' source
    auto gamma_of = [&](int j, int v, float *g) {
        if constexpr (GFLT) {
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = gam[j * V + e];
        } else if constexpr (GSMEM) {
            Tr::unpack(ld_shared_v4(gs + v * 16), g);
        } else {
            Tr::unpack(graw[j], g);
        }
    };
    RingPos pos;
    int k = 0;
    for (; k < ns; ++k) {
        const bool timed_out = !mbar_wait_bounded(&bar[pos.stage], pos.parity, p.wait_ns);
        if (timed_out) record_error(p.err, kErrWaitFull);
        const unsigned char *sh = ring + (size_t)pos.stage * 3 * rowb;
        const float rs = st_rstd[slot + k * slots];
        // pass 1: sum(dyhat * h), one sum per vector
        float sum[1] = {0.f};
        uint4 hr[HOLD && !HOLDF ? NV : 1], dr[HOLD && !HOLDF ? NV : 1], er[HOLD ? NV : 1];
        float hx[HOLDF ? E : 1], dyx[HOLDF ? E : 1];
        float he = 0.f, de = 0.f, ee = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + ts + j * tpr;
            if (v < ve) {
                float hf[V], df[V], g[V];
                const uint4 h4 = ld_shared_v4(sh + v * 16), d4 = ld_shared_v4(sh + rowb + v * 16);
                if constexpr (HOLD) er[j] = ld_shared_v4(sh + 2 * rowb + v * 16);
                if constexpr (HOLD && !HOLDF) {
                    hr[j] = h4;
                    dr[j] = d4;
                }
                Tr::unpack(h4, hf);
                Tr::unpack(d4, df);
                if constexpr (HOLDF) {
#pragma unroll
                    for (int e = 0; e < V; ++e) hx[j * V + e] = hf[e], dyx[j * V + e] = df[e];
                }
                gamma_of(j, v, g);
                float2 t = pair_mul(pair_mul(pair_at(df, 0), pair_at(g, 0)), pair_at(hf, 0));
#pragma unroll
                for (int i = 1; i < V / 2; ++i)
                    t = pair_fma(pair_mul(pair_at(df, i), pair_at(g, i)), pair_at(hf, i), t);
                sum[0] += t.x + t.y;
            }
        }
        if (SHIFT && ce >= 0) {
            he = Tr::load1(reinterpret_cast<const T *>(sh) + ce);
            de = Tr::load1(reinterpret_cast<const T *>(sh + rowb) + ce);
            ee = Tr::load1(reinterpret_cast<const T *>(sh + 2 * rowb) + ce);
            sum[0] = fmaf(de * ge, he, sum[0]);
        }
        if (slot_reduce<1>(sum, red + (k & 1) * kRedStride, flag, k + 1, timed_out, W, warp, lane, 1 + slot, tpr)) break;
        // the slot is done with this row's stage (the row before's): refill it
        if (issuer && issued < ns && (HOLD || k > 0)) {
            fence_proxy_async();
            issue();
        }
        // pass 2, with D = dy*rstd and a = -rstd^2 * mean(dyhat*xhat):
        // dgamma += D*h, dx = D*gamma + (h*a + dh)
        const float a = -rs * rs * (sum[0] * rs * inv_n);
        const float2 rs2 = make_float2(rs, rs), a2 = make_float2(a, a);
        T *dx = static_cast<T *>(p.dx) + (first + (int64_t)(slot + k * slots) * step) * p.ld_dx - s;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + ts + j * tpr;
            if (v < ve) {
                float hf[V], df[V], g[V], o[V];
                if constexpr (HOLDF) {
#pragma unroll
                    for (int e = 0; e < V; ++e) hf[e] = hx[j * V + e], df[e] = dyx[j * V + e];
                } else {
                    Tr::unpack(HOLD ? hr[HOLD && !HOLDF ? j : 0] : ld_shared_v4(sh + v * 16), hf);
                    Tr::unpack(HOLD ? dr[HOLD && !HOLDF ? j : 0] : ld_shared_v4(sh + rowb + v * 16), df);
                }
                Tr::unpack(HOLD ? er[HOLD ? j : 0] : ld_shared_v4(sh + 2 * rowb + v * 16), o);
                gamma_of(j, v, g);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const int e = j * V + 2 * i;
                    const float2 D = pair_mul(pair_at(df, i), rs2), h2 = pair_at(hf, i);
                    const float2 ag = pair_fma(D, h2, make_float2(acc[e], acc[e + 1]));
                    acc[e] = ag.x, acc[e + 1] = ag.y;
                    const float2 o2 = pair_fma(D, pair_at(g, i), pair_fma(h2, a2, pair_at(o, i)));
                    o[2 * i] = o2.x, o[2 * i + 1] = o2.y;
                }
                st_global_cs_v4(dx + (size_t)v * V, Tr::pack(o));
            }
        }
        if (SHIFT && ce >= 0) {
            const float D = de * rs;
            ae = fmaf(D, he, ae);
            Tr::store1(dx + ce, fmaf(D, ge, fmaf(he, a, ee)));
        }
        pos.next(S);
    }
    // after a wait ran out: let the copies this slot still has in flight land
    // (bounded) before the CTA goes on
    if (issuer && lane == 0) {
        for (int kk = k; kk < issued; ++kk) {
            if (!mbar_wait_bounded(&bar[kk % S], (kk / S) & 1, kDrainNs)) {
                record_error(p.err, kErrDrain);
                break;
            }
        }
    }

    // the CTA's partial row: the slots' sums added in slot order in shared memory
    float *part = p.part + (size_t)blockIdx.x * p.ldp;
    __syncthreads();
    const int width = nvec * V;
    float *comb = reinterpret_cast<float *>(smem) + (size_t)slot * width;
    if (slot < slots) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + ts + j * tpr;
            if (v < ve) {
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    *reinterpret_cast<float4 *>(comb + v * V + e) =
                        make_float4(acc[j * V + e], acc[j * V + e + 1], acc[j * V + e + 2], acc[j * V + e + 3]);
            }
        }
        if (SHIFT && ce >= 0) comb[ce] = ae;
    }
    __syncthreads();
    comb = reinterpret_cast<float *>(smem) + s;
    for (int c = tid; c < N; c += kAddBwdThreads) {
        float t = comb[c];
        for (int q = 1; q < slots; ++q) t += comb[(size_t)q * width + c];
        part[c] = t;
    }
}

template <typename T, int NV, bool SHIFT>
cudaError_t rms_add_bwd_ring_launch(const AddBwdParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_smem_optin(rms_add_bwd_ring_kernel<T, NV, SHIFT>, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(rms_add_bwd_ring_kernel<T, NV, SHIFT>, p.G, kAddBwdThreads, smem, s, p);
}

template <typename T>
cudaError_t rms_add_bwd_ring_dispatch(int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s) {
    switch (nv) {
#define GBN_CASE(n) \
    case n: return shift ? rms_add_bwd_ring_launch<T, n, true>(p, smem, s) : rms_add_bwd_ring_launch<T, n, false>(p, smem, s)
        GBN_CASE(1);
        GBN_CASE(2);
        GBN_CASE(3);
        GBN_CASE(4);
#undef GBN_CASE
        case 6:
        case 8:
            if constexpr (sizeof(T) == 4) {
                if (nv == 6)
                    return shift ? rms_add_bwd_ring_launch<T, 6, true>(p, smem, s)
                                 : rms_add_bwd_ring_launch<T, 6, false>(p, smem, s);
                return shift ? rms_add_bwd_ring_launch<T, 8, true>(p, smem, s)
                             : rms_add_bwd_ring_launch<T, 8, false>(p, smem, s);
            }
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t rms_add_bwd_plain_dispatch(const AddBwdParams &p, cudaStream_t s) {
    rms_add_bwd_plain_kernel<T><<<p.G, kAddBwdPlainThreads, 0, s>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Short rows: L lanes of a warp to a row, 32 / L rows at once in a warp; loads
// go straight to registers, the CTA's warps hide them.  C: elements to an
// access, a 16-byte vector's or one (rows that do not lie on 16 bytes); a lane
// owns NV accesses, L apart, and their dgamma sums.  At the end a warp's rows
// meet in shuffles and the warps in shared memory, in warp order.  64x256
// float32 2.9 us with the column reduce (the ring 4.9), 32768x256 bf16 15.6;
// bound by the two launches on few rows, by latency on many very short.
// ---------------------------------------------------------------------------
template <typename T, int L, int NV, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) rms_add_bwd_short_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    constexpr int C = VEC ? Tr::kVec : 1;
    constexpr int E = NV * C;
    constexpr int WIDTH = L * E;  // columns
    __shared__ float sums[THREADS / 32][WIDTH];
    const int N = p.N, lane = threadIdx.x & (L - 1), warp = threadIdx.x >> 5;
    const float inv_n = 1.0f / static_cast<float>(N);
    griddep_wait();  // whatever is before this kernel on the stream
    griddep_launch_dependents();
    float gam[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (lane + (e / C) * L) * C + e % C;
        gam[e] = c < N ? Tr::load1(static_cast<const T *>(p.gamma) + c) : 0.f;
        acc[e] = 0.f;
    }
    const int64_t rows = (int64_t)gridDim.x * (THREADS / L);
    // rounds are the whole warp's: its lanes meet in shuffles
    for (int64_t r0 = (blockIdx.x * (int64_t)THREADS + threadIdx.x) / 32 * (32 / L); r0 < p.M; r0 += rows) {
        const int64_t row = r0 + (threadIdx.x & 31) / L;
        const bool live = row < p.M;
        const T *hp = static_cast<const T *>(p.h) + row * p.ld_h;
        const T *dp = static_cast<const T *>(p.dy) + row * p.ld_dy;
        const T *ep = static_cast<const T *>(p.dh) + row * p.ld_dh;
        const float rs = live ? p.rstd[row] : 0.f;
        float h[E], d[E], o[E];
        if constexpr (VEC) {
            uint4 h4[NV], d4[NV], e4[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * L) * C;
                const bool in = live && c < N;
                h4[j] = in ? *reinterpret_cast<const uint4 *>(hp + c) : make_uint4(0, 0, 0, 0);
                d4[j] = in ? *reinterpret_cast<const uint4 *>(dp + c) : make_uint4(0, 0, 0, 0);
                e4[j] = in ? *reinterpret_cast<const uint4 *>(ep + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                Tr::unpack(h4[j], h + j * C);
                Tr::unpack(d4[j], d + j * C);
                Tr::unpack(e4[j], o + j * C);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * L;
                const bool in = live && c < N;
                h[j] = in ? Tr::load1(hp + c) : 0.f;
                d[j] = in ? Tr::load1(dp + c) : 0.f;
                o[j] = in ? Tr::load1(ep + c) : 0.f;
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(d[e] * gam[e], h[e], sum);
#pragma unroll
        for (int s = L / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        // D = dy*rstd, a = -rstd^2 * mean(dyhat*xhat): dgamma += D*h, dx = D*gamma + (h*a + dh)
        const float a = -rs * rs * (sum * rs * inv_n);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float D = d[e] * rs;
            acc[e] = fmaf(D, h[e], acc[e]);
            o[e] = fmaf(D, gam[e], fmaf(h[e], a, o[e]));
        }
        T *dx = static_cast<T *>(p.dx) + row * p.ld_dx;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * L) * C;
            if (live && c < N) {
                if constexpr (VEC)
                    *reinterpret_cast<uint4 *>(dx + c) = Tr::pack(o + j * C);
                else
                    Tr::store1(dx + c, o[j]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int s = 16; s >= L; s >>= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], s);
        if ((threadIdx.x & 31) < L) sums[warp][(lane + (e / C) * L) * C + e % C] = acc[e];
    }
    __syncthreads();
    float *part = p.part + (size_t)blockIdx.x * p.ldp;
    for (int c = threadIdx.x; c < N; c += THREADS) {
        float t = sums[0][c];
        for (int w = 1; w < THREADS / 32; ++w) t += sums[w][c];
        part[c] = t;
    }
}

template <typename T, int L, int NV, bool VEC, int THREADS>
cudaError_t rms_add_bwd_short_launch(const AddBwdParams &p, cudaStream_t s) {
    return launch_dependent(rms_add_bwd_short_kernel<T, L, NV, VEC, THREADS>, p.G, THREADS, 0, s, p);
}

// the rows at once are add_bwd_short_rows()'s
template <typename T>
cudaError_t rms_add_bwd_short_dispatch(bool vec, const AddBwdParams &p, cudaStream_t s) {
    if (vec) {
        const int nvec = p.N / Traits<T>::kVec;
        if (nvec <= 8) return rms_add_bwd_short_launch<T, 8, 1, true, 1024>(p, s);
        if (nvec <= 16) return rms_add_bwd_short_launch<T, 16, 1, true, 1024>(p, s);
        if (nvec <= 32) return rms_add_bwd_short_launch<T, 32, 1, true, 1024>(p, s);
        return rms_add_bwd_short_launch<T, 32, 2, true, 512>(p, s);
    }
    if (p.N <= 64) return rms_add_bwd_short_launch<T, 32, 2, false, 1024>(p, s);
    if (p.N <= 128) return rms_add_bwd_short_launch<T, 32, 4, false, 1024>(p, s);
    return rms_add_bwd_short_launch<T, 32, 8, false, 512>(p, s);
}

}  // namespace gbn
