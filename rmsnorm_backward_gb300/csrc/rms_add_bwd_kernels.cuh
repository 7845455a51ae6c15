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
// any N, stride and alignment: CTA b takes a contiguous block of rows, with
// scalar accesses; its partial row in global memory is the accumulator
// (column j always by thread j mod 256: a fixed order per column)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kGenericThreads) rms_add_bwd_plain_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    __shared__ float sm[kGenericThreads / 32];
    const int N = p.N;
    const float inv_n = 1.0f / static_cast<float>(N);
    int64_t row0;
    int nrows;
    block_rows(p.M, p.G, blockIdx.x, row0, nrows);
    float *pg = p.part + (size_t)blockIdx.x * p.ldp;
    for (int j = threadIdx.x; j < N; j += blockDim.x) pg[j] = 0.f;
    const T *g = static_cast<const T *>(p.gamma);
    for (int i = 0; i < nrows; ++i) {
        const int64_t row = row0 + i;
        const T *h = static_cast<const T *>(p.h) + row * p.ld_h;
        const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
        const T *dh = static_cast<const T *>(p.dh) + row * p.ld_dh;
        T *dx = static_cast<T *>(p.dx) + row * p.ld_dx;
        const float rs = p.rstd[row];
        float s = 0.f;
        for (int j = threadIdx.x; j < N; j += blockDim.x)
            s = fmaf(Tr::load1(dy + j) * Tr::load1(g + j), Tr::load1(h + j) * rs, s);
        const float a = -rs * (block_sum(s, sm) * inv_n);
        for (int j = threadIdx.x; j < N; j += blockDim.x) {
            const float xhat = Tr::load1(h + j) * rs, d = Tr::load1(dy + j);
            const float o = fmaf(d * Tr::load1(g + j), rs, xhat * a) + Tr::load1(dh + j);
            pg[j] = fmaf(d, xhat, pg[j]);
            Tr::store1(dx + j, o);
        }
    }
}

// ---------------------------------------------------------------------------
// One persistent CTA per SM; its 512 threads are slots of tpr threads, and
// each slot streams its rows of h, dy and dh through a ring of shared-memory
// stages filled by 1-D bulk copies.  A thread owns NV column vectors, their
// gamma and their dgamma sums in registers.  Pass 1 forms sum(dyhat*h) from
// the stage (one exchange within the slot), pass 2 reads the stage again and
// writes dx with 16-byte streaming stores: shared memory has the bandwidth for
// the second read, and registers stay free for rows of up to 32 elements a
// thread.  The exchange of row k shows that the whole slot is done with row
// k-1, whose stage is then refilled.
//
// SHIFT: rows that do not start or end on 16 bytes.  All four tensors' rows
// have the same shift (the host checks that), so a row is copied with the up
// to 14 bytes before and after it that share its first and last 16 bytes
// (never beyond the tensor's first and last element: those two edges are
// copied element by element), and the elements beside the row count as zero
// and are never written.
// ---------------------------------------------------------------------------
template <typename T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kAddBwdThreads, 1) rms_add_bwd_ring_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int E = NV * V;
    extern __shared__ __align__(128) unsigned char smem[];

    const int tid = threadIdx.x, tpr = p.tpr, slots = kAddBwdThreads / tpr;
    const int slot = tid / tpr, ts = tid - slot * tpr;
    const int W = tpr >> 5, warp = ts >> 5, lane = tid & 31;
    const int N = p.N, S = p.stages;
    const uint32_t rowb = static_cast<uint32_t>(p.nvec) * 16;
    const AddBwdLayout L = add_bwd_layout(slots, S, p.nvec, p.stat_rows);
    unsigned char *ring = smem + (size_t)slot * S * 3 * rowb;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L.bar) + slot * S;
    float *st_rstd = reinterpret_cast<float *>(smem + L.stat);
    float *red = reinterpret_cast<float *>(smem + L.red) + slot * 2 * kRedStride;
    volatile int *flag = reinterpret_cast<int *>(smem + L.flag) + slot;

    // this CTA's rows: first + step*i for i < nrows
    const int phase = blockIdx.x % p.phases, step = p.phases;
    int64_t i0;
    int nrows;
    block_rows((p.M - phase + step - 1) / step, (p.G - phase + step - 1) / step, blockIdx.x / step, i0, nrows);
    const int64_t first = phase + i0 * step;
    const int s = SHIFT ? row_shift(phase, p.shift0, p.shift_step, V) : 0;
    const int nvec = SHIFT ? (s + N + V - 1) / V : p.nvec;
    const int ns = slot < nrows ? (nrows - slot + slots - 1) / slots : 0;

    if (tid == 0) {
        uint64_t *all = reinterpret_cast<uint64_t *>(smem + L.bar);
        for (int i = 0; i < slots * S; ++i) mbar_init(&all[i], 1);
        fence_barrier_init();
    }
    if (ts == 0) *flag = 0;
    __syncthreads();

    // producer (thread 0 of the slot)
    int issued = 0, pst = 0;
    auto row_of = [&](int k) { return first + (int64_t)(slot + k * slots) * step; };
    auto edge = [&](unsigned char *dst, const T *row, int v) {  // one vector of a row, element by element
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = v * V + e - s;
            if (c >= 0 && c < N) reinterpret_cast<T *>(dst)[v * V + e] = row[c];
        }
    };
    auto issue = [&]() {
        const int64_t row = row_of(issued);
        unsigned char *dst = ring + (size_t)pst * 3 * rowb;
        const T *src[3] = {static_cast<const T *>(p.h) + row * p.ld_h, static_cast<const T *>(p.dy) + row * p.ld_dy,
                           static_cast<const T *>(p.dh) + row * p.ld_dh};
        if constexpr (SHIFT) {
            const T *base[3] = {static_cast<const T *>(p.h), static_cast<const T *>(p.dy), static_cast<const T *>(p.dh)};
            const int64_t ld[3] = {p.ld_h, p.ld_dy, p.ld_dh};
            int v0[3], v1[3];
            uint32_t bytes = 0;
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                const T *end = base[t] + (p.M - 1) * ld[t] + N;
                v0[t] = src[t] - s < base[t] ? 1 : 0;
                v1[t] = src[t] - s + (int64_t)nvec * V > end ? nvec - 1 : nvec;
                if (v0[t]) edge(dst + t * rowb, src[t], 0);
                if (v1[t] < nvec && (nvec > 1 || !v0[t])) edge(dst + t * rowb, src[t], nvec - 1);
                if (v1[t] > v0[t]) bytes += (v1[t] - v0[t]) * 16;
            }
            mbar_arrive_expect_tx(&bar[pst], bytes);
#pragma unroll
            for (int t = 0; t < 3; ++t)
                if (v1[t] > v0[t])
                    bulk_load_nohint(dst + t * rowb + v0[t] * 16, src[t] - s + v0[t] * V, (v1[t] - v0[t]) * 16,
                                     &bar[pst]);
        } else {
            mbar_arrive_expect_tx(&bar[pst], 3 * rowb);
#pragma unroll
            for (int t = 0; t < 3; ++t) bulk_load_nohint(dst + t * rowb, src[t], rowb, &bar[pst]);
        }
        if (++pst == S) pst = 0;
        ++issued;
    };
    if (ts == 0) {
        while (issued < S && issued < ns) issue();
    }

    for (int i = tid; i < nrows; i += kAddBwdThreads) st_rstd[i] = p.rstd[first + (int64_t)i * step];
    float gam[E], acc[E];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = ts + j * tpr;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = v * V + e - s;
            gam[j * V + e] = c >= 0 && c < N ? Tr::load1(static_cast<const T *>(p.gamma) + c) : 0.f;
            acc[j * V + e] = 0.f;
        }
    }
    __syncthreads();
    griddep_launch_dependents();

    const float inv_n = 1.0f / static_cast<float>(N);
    // elements of vector v beside the row count as zero
    auto mask = [&](float *f, int v) {
        if constexpr (SHIFT) {
            if (v == 0 || v == nvec - 1) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = v * V + e - s;
                    if (c < 0 || c >= N) f[e] = 0.f;
                }
            }
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
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = ts + j * tpr;
            if (v < nvec) {
                float hf[V], df[V];
                Tr::unpack(ld_shared_v4(sh + v * 16), hf);
                Tr::unpack(ld_shared_v4(sh + rowb + v * 16), df);
                mask(hf, v);
                mask(df, v);
                float2 t = pair_mul(pair_mul(pair_at(df, 0), pair_at(gam + j * V, 0)), pair_at(hf, 0));
#pragma unroll
                for (int i = 1; i < V / 2; ++i)
                    t = pair_fma(pair_mul(pair_at(df, i), pair_at(gam + j * V, i)), pair_at(hf, i), t);
                sum[0] += t.x + t.y;
            }
        }
        if (slot_reduce<1>(sum, red + (k & 1) * kRedStride, flag, timed_out, W, warp, lane, 1 + slot, tpr)) break;
        // the slot is done with the row before this one: refill its stage
        if (ts == 0 && issued < ns && k > 0) {
            fence_proxy_async();
            issue();
        }
        // pass 2: dx = dyhat*rstd + xhat*a + dh, a = -rstd * mean(dyhat*xhat)
        const float a = -rs * (sum[0] * rs * inv_n);
        const float2 rs2 = make_float2(rs, rs), a2 = make_float2(a, a);
        T *dx = static_cast<T *>(p.dx) + row_of(k) * p.ld_dx - s;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = ts + j * tpr;
            if (v < nvec) {
                float hf[V], df[V], o[V];
                Tr::unpack(ld_shared_v4(sh + v * 16), hf);
                Tr::unpack(ld_shared_v4(sh + rowb + v * 16), df);
                Tr::unpack(ld_shared_v4(sh + 2 * rowb + v * 16), o);
                mask(hf, v);
                mask(df, v);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const int e = j * V + 2 * i;
                    const float2 d2 = pair_at(df, i), xh = pair_mul(pair_at(hf, i), rs2);
                    const float2 ag = pair_fma(d2, xh, make_float2(acc[e], acc[e + 1]));
                    acc[e] = ag.x, acc[e + 1] = ag.y;
                    const float2 o2 = pair_add(pair_fma(pair_mul(d2, make_float2(gam[e], gam[e + 1])), rs2,
                                                        pair_mul(xh, a2)), pair_at(o, i));
                    o[2 * i] = o2.x, o[2 * i + 1] = o2.y;
                }
                if (SHIFT && (v == 0 || v == nvec - 1)) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int c = v * V + e - s;
                        if (c >= 0 && c < N) Tr::store1(dx + v * V + e, o[e]);
                    }
                } else {
                    st_global_cs_v4(dx + (size_t)v * V, Tr::pack(o));
                }
            }
        }
        pos.next(S);
    }
    // after a wait ran out: let the copies this slot still has in flight land
    // (bounded) before the CTA exits
    if (ts == 0) {
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
    float *comb = reinterpret_cast<float *>(smem);
    const int width = nvec * V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = ts + j * tpr;
        if (v < nvec) {
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(comb + (size_t)slot * width + v * V + e) =
                    make_float4(acc[j * V + e], acc[j * V + e + 1], acc[j * V + e + 2], acc[j * V + e + 3]);
        }
    }
    __syncthreads();
    for (int c = tid; c < N; c += kAddBwdThreads) {
        float t = comb[c + s];
        for (int q = 1; q < slots; ++q) t += comb[(size_t)q * width + c + s];
        part[c] = t;
    }
}

template <typename T, int NV, bool SHIFT>
cudaError_t rms_add_bwd_ring_launch(const AddBwdParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_smem_optin(rms_add_bwd_ring_kernel<T, NV, SHIFT>, done);
    if (e != cudaSuccess) return e;
    rms_add_bwd_ring_kernel<T, NV, SHIFT><<<p.G, kAddBwdThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t rms_add_bwd_ring_dispatch(int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s) {
    switch (nv) {
        case 1: return shift ? rms_add_bwd_ring_launch<T, 1, true>(p, smem, s) : rms_add_bwd_ring_launch<T, 1, false>(p, smem, s);
        case 2: return shift ? rms_add_bwd_ring_launch<T, 2, true>(p, smem, s) : rms_add_bwd_ring_launch<T, 2, false>(p, smem, s);
        case 4: return shift ? rms_add_bwd_ring_launch<T, 4, true>(p, smem, s) : rms_add_bwd_ring_launch<T, 4, false>(p, smem, s);
        case 8:
            if constexpr (sizeof(T) == 4)
                return shift ? rms_add_bwd_ring_launch<T, 8, true>(p, smem, s) : rms_add_bwd_ring_launch<T, 8, false>(p, smem, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t rms_add_bwd_plain_dispatch(const AddBwdParams &p, cudaStream_t s) {
    rms_add_bwd_plain_kernel<T><<<p.G, kGenericThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gbn
