// grad_clip.cu -- the global 2-norm of many gradient tensors, and their clip,
// for sm_103a.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + eps)),  out = round(g * coef)
//
// Both kernels walk the same list of 32 KiB chunks; CTA b owns a contiguous
// range of them, so it looks its first tensor up once and then steps.  The
// table of tensors travels in the launch's parameters: nothing is copied to
// the device, nothing outlives the call, and a captured launch keeps its
// own.  Lists longer than a table take several launches.
//  * norm: a thread squares and adds batches of four 16-byte vectors in
//    float32 and gathers the batches' sums as a float32 pair (a sum and what
//    its roundings lost), which holds some 48 bits: sm_103a adds doubles at a
//    64th of that rate, and the doubles of one CTA's last reduction took as
//    long as a megabyte.  Batches whose squares would leave float32's range
//    are scaled by a power of two first and gathered apart, so gradients as
//    small as 1e-38 or as large as 3e38 have their norm.  The CTA's sums go to
//    its own place in the workspace, and whoever needs the norm adds those in
//    one fixed order: no atomics, the same bits from run to run.
//  * clip: every CTA forms coef from the partial sums itself (no kernel in
//    between), then walks its chunks backwards: what the first pass read
//    last is still in L2.  In place with coef = 1 there is nothing to do.
// Both are bound by HBM: 480 MB of float32 in 76.8 us (norm only, 6.25 TB/s,
// 93% of the measured copy rate), 671 MB of bf16 clipped into other tensors in
// 316 us (two reads and a write, 6.4 TB/s), 126 MB in 61 us (the second read
// mostly from L2).  Four CTAs of 256 threads an SM with 32 KiB chunks: six, or
// 16 KiB, took 3 to 8% longer; evict-first hints on all but the last chunks of
// the first pass won 2% of a large clip and lost 4% of a norm.
#include "gbn_device.cuh"
#include "grad_clip.h"

namespace gbn {
namespace {

struct GradEntry {
    const void *src;
    void *dst;
    int64_t n;
    uint32_t first;  // the tensor's first chunk in this launch's list
    int dtype;
};

// kernel parameters hold up to 32764 bytes; short lists take a small table,
// which launches faster
template <int CAP>
struct GradTable {
    GradEntry e[CAP];
    GradSums *partial;
    float *norm;
    uint32_t chunks;  // in this launch
    int count;
    int total;        // CTAs of the norm kernel (partial sums)
    int add;          // a later launch of the same list: add to the partial sums
    float max_norm, eps;
};
constexpr int kSmallTable = 96, kLargeTable = 1016;
static_assert(sizeof(GradTable<kLargeTable>) <= 32764, "kernel parameters");

template <typename T>
__host__ __device__ inline int64_t head_of(const void *p, int64_t n) {
    const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
    return h < n ? h : n;
}

inline int64_t chunks_of(const gbn_tensor &t) {
    const int64_t h = t.dtype == GBN_F32 ? head_of<float>(t.data, t.n) : head_of<uint16_t>(t.data, t.n);
    const int64_t v = (t.n - h) / (t.dtype == GBN_F32 ? 4 : 8);
    const int64_t c = (v + kGradChunkVecs - 1) / kGradChunkVecs;
    return c > 0 ? c : 1;
}

// A float32 sum and what its roundings lost (Knuth's two-sum).
struct Pair {
    float hi = 0.f, lo = 0.f;
};
__device__ __forceinline__ void add(Pair &p, float b) {
    const float s = __fadd_rn(p.hi, b), bb = __fsub_rn(s, p.hi);
    p.lo += __fadd_rn(__fsub_rn(p.hi, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    p.hi = s;
}
__device__ __forceinline__ void add(Pair &p, const Pair &q) {
    add(p, q.hi);
    p.lo += q.lo;
}
__device__ __forceinline__ Pair pair_of(float hi, float lo) {
    Pair p;
    p.hi = hi, p.lo = lo;
    return p;
}
// its value; of an infinite or NaN sum what was lost means nothing
__device__ __forceinline__ double value(const Pair &p) {
    return static_cast<double>(p.hi) + (fabsf(p.hi) <= 3.402823466e38f ? static_cast<double>(p.lo) : 0.0);
}

// A thread's sums of squares, pairs each: of x, of x * 2^-80 where a batch's sum
// is above 2^60 (or not finite), of x * 2^80 where it is below 2^-80.  Squares
// from there on are normal float32 values, exact multiples of 2^-138 or
// negligible in their batch, and the sums stay in range for 2^34 batches.
constexpr float kBatchMost = 0x1p60f, kBatchLeast = 0x1p-80f;
struct Sums {
    Pair mid, big, small;
    __device__ __forceinline__ bool scaled() const { return big.hi != 0.f || small.hi != 0.f; }
};

__device__ __forceinline__ GradSums sums_out(const Sums &s) {
    return GradSums{s.mid.hi, s.mid.lo, s.big.hi, s.small.hi, s.big.lo, s.small.lo};
}
// Adds the GradSums at from, from + step, ... below to: the ordinary sums first,
// four loads at a time, then the scaled ones where there are any (a
// branch at each made 1 us of a clip).
template <bool GLOBAL>
__device__ __forceinline__ void sums_in(Sums &s, const GradSums *from, const GradSums *to, int step) {
    auto half = [](const GradSums *p, int i) {
        const float4 *at = reinterpret_cast<const float4 *>(p) + i;
        return GLOBAL ? __ldcg(at) : *at;
    };
    bool scaled = false;
    for (const GradSums *p = from; p < to; p += 4 * step) {
        float4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = p + i * step < to ? half(p + i * step, 0) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            add(s.mid, pair_of(q[i].x, q[i].y));
            scaled |= q[i].z != 0.f || q[i].w != 0.f;
        }
    }
    if (!scaled) return;
    for (const GradSums *p = from; p < to; p += step) {
        const float4 q = half(p, 0), r = half(p, 1);
        add(s.big, pair_of(q.z, r.x));
        add(s.small, pair_of(q.w, r.y));
    }
}

template <typename T>
__device__ __forceinline__ float sum_squares(const uint4 (&raw)[4], float scale) {
    constexpr int V = Traits<T>::kVec;
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[V];
        Traits<T>::unpack(raw[j], f);
        if (scale != 1.f) {
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] *= scale;
        }
        s[j] = f[0] * f[0];
#pragma unroll
        for (int e = 1; e < V; ++e) s[j] = fmaf(f[e], f[e], s[j]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// p and a batch's squares, scaled
template <typename T>
__device__ __noinline__ Pair scaled_squares(Pair p, uint4 v0, uint4 v1, uint4 v2, uint4 v3, float scale) {
    const uint4 raw[4] = {v0, v1, v2, v3};
    add(p, sum_squares<T>(raw, scale));
    return p;
}

template <typename T>
__device__ __forceinline__ void add_batch(Sums &sums, const uint4 (&raw)[4]) {
    const float b = sum_squares<T>(raw, 1.f);
    if (b >= kBatchLeast && b <= kBatchMost) {
        add(sums.mid, b);
    } else if (b < kBatchLeast) {
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) any |= raw[j].x | raw[j].y | raw[j].z | raw[j].w;
        if (any) sums.small = scaled_squares<T>(sums.small, raw[0], raw[1], raw[2], raw[3], 0x1p80f);
    } else {
        sums.big = scaled_squares<T>(sums.big, raw[0], raw[1], raw[2], raw[3], 0x1p-80f);
    }
}

__device__ __forceinline__ void add_one(Sums &sums, float f) {
    const float b = f * f;
    if (b >= kBatchLeast && b <= kBatchMost)
        add(sums.mid, b);
    else if (b < kBatchLeast)
        add(sums.small, (f * 0x1p80f) * (f * 0x1p80f));
    else
        add(sums.big, (f * 0x1p-80f) * (f * 0x1p-80f));
}

template <typename T>
__device__ __forceinline__ void add_chunk(Sums &sums, const GradEntry &t, uint32_t chunk) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    const T *src = static_cast<const T *>(t.src);
    const int64_t head = head_of<T>(src, t.n);
    const int64_t nvec = (t.n - head) / V;
    const T *body = src + head;
    const int64_t v0 = static_cast<int64_t>(chunk) * kGradChunkVecs + threadIdx.x;
    uint4 raw[kGradVecs / 4][4];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int64_t v = v0 + j * kGradThreads;
        raw[j / 4][j % 4] = v < nvec ? ld_global_nc_v4(body + v * V) : make_uint4(0, 0, 0, 0);
    }
    if (chunk == 0) {  // the elements before and after the 16-byte vectors
        const int64_t tail = t.n - head - nvec * V;
        if (threadIdx.x < head) add_one(sums, Tr::load1(src + threadIdx.x));
        if (threadIdx.x < tail) add_one(sums, Tr::load1(body + nvec * V + threadIdx.x));
    }
#pragma unroll
    for (int j = 0; j < kGradVecs / 4; ++j) add_batch<T>(sums, raw[j]);
}

__device__ __forceinline__ Pair shuffled(const Pair &p, int o) {
    Pair q;
    q.hi = __shfl_xor_sync(0xffffffffu, p.hi, o);
    q.lo = __shfl_xor_sync(0xffffffffu, p.lo, o);
    return q;
}

// The CTA's sums in a fixed order, on every thread; sm holds a GradSums a warp.
// The scaled sums are looked at where there are any.
__device__ __forceinline__ Sums cta_sum(Sums v, GradSums *sm) {
    const bool scaled = __any_sync(0xffffffffu, v.scaled());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        add(v.mid, shuffled(v.mid, o));
        if (scaled) {
            add(v.big, shuffled(v.big, o));
            add(v.small, shuffled(v.small, o));
        }
    }
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = sums_out(v);
    __syncthreads();
    Sums s;
    sums_in<false>(s, sm, sm + kGradThreads / 32, 1);
    __syncthreads();
    return s;
}

// this CTA's chunks [c0, c1)
__device__ __forceinline__ void cta_range(uint32_t chunks, uint32_t &c0, uint32_t &c1) {
    const uint32_t G = gridDim.x, b = blockIdx.x;
    const uint32_t base = chunks / G, rem = chunks % G;
    c0 = b * base + (b < rem ? b : rem);
    c1 = c0 + base + (b < rem ? 1u : 0u);
}

// the last entry whose first chunk is <= c
template <int CAP>
__device__ __forceinline__ int find_entry(const GradTable<CAP> &t, uint32_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kGradCtasPerSm) grad_norm_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ GradSums sm[kGradThreads / 32];
    // the gradients, and whoever still reads the partial sums, come before
    // this kernel on the stream; the clip may launch meanwhile and waits
    griddep_wait();
    griddep_launch_dependents();
    Sums sums;
    if (t.add && threadIdx.x == 0) {  // a later launch of the same list
        sums_in<true>(sums, t.partial + blockIdx.x, t.partial + blockIdx.x + 1, 1);
    }
    uint32_t c, c1;
    cta_range(t.chunks, c, c1);
    if (c < c1) {
        int i = find_entry(t, c);
        for (; c < c1; ++c) {
            while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
            const GradEntry &e = t.e[i];
            const uint32_t k = c - e.first;
            if (e.dtype == GBN_F32)
                add_chunk<float>(sums, e, k);
            else if (e.dtype == GBN_F16)
                add_chunk<__half>(sums, e, k);
            else
                add_chunk<__nv_bfloat16>(sums, e, k);
        }
    }
    sums = cta_sum(sums, sm);
    if (threadIdx.x == 0) t.partial[blockIdx.x] = sums_out(sums);
}

// The norm from the CTAs' sums, in a fixed order: the float32 root of the
// pair, improved by one step of Newton's method from the pair's residual, or
// a float64 root where some batches were scaled or the sum is zero, infinite
// or NaN (a norm above the largest float32 is infinite).
__device__ __forceinline__ float norm_of(const GradSums *partial, int total, GradSums *sm) {
    Sums v;
    sums_in<true>(v, partial + threadIdx.x, partial + total, kGradThreads);
    v = cta_sum(v, sm);
    if (!v.scaled() && v.mid.hi >= 0x1p-100f && v.mid.hi <= 0x1p120f) {
        const float r = sqrtf(v.mid.hi);
        return r + (fmaf(-r, r, v.mid.hi) + v.mid.lo) / (2.f * r);
    }
    const double d = value(v.mid) + value(v.big) * 0x1p160 + value(v.small) * 0x1p-160;
    return static_cast<float>(sqrt(d));
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_finish_kernel(const GradSums *partial, int total,
                                                                       float *norm) {
    __shared__ GradSums sm[kGradThreads / 32];
    griddep_wait();
    const float n = norm_of(partial, total, sm);
    if (threadIdx.x == 0) *norm = n;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const GradEntry &t, uint32_t chunk, float coef) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    const T *src = static_cast<const T *>(t.src);
    T *dst = static_cast<T *>(t.dst);
    const int64_t head = head_of<T>(src, t.n);
    const int64_t nvec = (t.n - head) / V;
    const bool same = (reinterpret_cast<uintptr_t>(dst + head) & 15) == 0;
    // four vectors at a time: registers for four CTAs on an SM
#pragma unroll 1
    for (int64_t v0 = (int64_t)chunk * kGradChunkVecs + threadIdx.x, end = v0 + kGradChunkVecs; v0 < end;
         v0 += 4 * kGradThreads) {
        uint4 raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t v = v0 + j * kGradThreads;
            if (v < nvec) raw[j] = __ldcg(reinterpret_cast<const uint4 *>(src + head + v * V));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t v = v0 + j * kGradThreads;
            if (v < nvec) {
                float f[V];
                Tr::unpack(raw[j], f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] *= coef;
                T *d = dst + head + v * V;
                if (same) {
                    st_global_cs_v4(d, Tr::pack(f));
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) Tr::store1(d + e, f[e]);
                }
            }
        }
    }
    if (chunk == 0) {
        const int64_t at = head + nvec * V, tail = t.n - at;
        if (threadIdx.x < head) Tr::store1(dst + threadIdx.x, Tr::load1(src + threadIdx.x) * coef);
        if (threadIdx.x < tail) Tr::store1(dst + at + threadIdx.x, Tr::load1(src + at + threadIdx.x) * coef);
    }
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kGradCtasPerSm) grad_clip_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ GradSums sm[kGradThreads / 32];
    griddep_wait();
    const float norm = norm_of(t.partial, t.total, sm);
    if (blockIdx.x == 0 && threadIdx.x == 0 && !t.add) *t.norm = norm;
    const float c = t.max_norm / (norm + t.eps);
    const float coef = c >= 1.f || norm == 0.f ? 1.f : c;  // a norm that is NaN stays NaN
    uint32_t c0, k;
    cta_range(t.chunks, c0, k);
    if (c0 >= k) return;
    int i = find_entry(t, k - 1);
    while (k-- > c0) {
        while (t.e[i].first > k) --i;
        const GradEntry &e = t.e[i];
        if (coef == 1.f && e.src == e.dst) continue;
        const uint32_t at = k - e.first;
        if (e.dtype == GBN_F32)
            scale_chunk<float>(e, at, coef);
        else if (e.dtype == GBN_F16)
            scale_chunk<__half>(e, at, coef);
        else
            scale_chunk<__nv_bfloat16>(e, at, coef);
    }
}

// One pass over the list: tables of up to CAP tensors, a launch for each.
template <int CAP>
cudaError_t run_list(const gbn_tensor *g, const gbn_tensor *out, int64_t count, bool clip, int grid, float max_norm,
                     float eps, float *norm, GradSums *partial, cudaStream_t s) {
    GradTable<CAP> t;
    t.partial = partial;
    t.norm = norm;
    t.total = grid;
    t.max_norm = max_norm;
    t.eps = eps;
    int64_t i = 0;
    bool first = true;
    do {
        t.count = 0;
        uint64_t chunks = 0;
        for (; i < count && t.count < CAP; ++i) {
            if (g[i].n == 0) continue;
            GradEntry &e = t.e[t.count++];
            e.src = g[i].data;
            e.dst = out ? out[i].data : g[i].data;
            e.n = g[i].n;
            e.dtype = g[i].dtype;
            e.first = static_cast<uint32_t>(chunks);
            chunks += chunks_of(g[i]);
        }
        t.chunks = static_cast<uint32_t>(chunks);
        t.add = first ? 0 : 1;
        const cudaError_t r = clip ? launch_dependent(grad_clip_kernel<CAP>, grid, kGradThreads, 0, s, t)
                                   : launch_dependent(grad_norm_kernel<CAP>, grid, kGradThreads, 0, s, t);
        if (r != cudaSuccess) return r;
        first = false;
    } while (i < count);
    return cudaSuccess;
}

cudaError_t run_any(const gbn_tensor *g, const gbn_tensor *out, int64_t count, bool clip, int grid, float max_norm,
                    float eps, float *norm, GradSums *partial, cudaStream_t s) {
    return count <= kSmallTable
               ? run_list<kSmallTable>(g, out, count, clip, grid, max_norm, eps, norm, partial, s)
               : run_list<kLargeTable>(g, out, count, clip, grid, max_norm, eps, norm, partial, s);
}

int grid_of(const gbn_tensor *g, int64_t count, int sms) {
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) chunks += g[i].n > 0 ? chunks_of(g[i]) : 0;
    return grad_grid(chunks, sms);
}

}  // namespace

cudaError_t launch_grad_norm(const gbn_tensor *g, int64_t count, float *norm, GradSums *partial, int sms,
                             cudaStream_t s) {
    const int grid = grid_of(g, count, sms);
    cudaError_t e = run_any(g, nullptr, count, false, grid, 0.f, 0.f, norm, partial, s);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kGradThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const GradSums *>(partial), grid, norm);
}

cudaError_t launch_grad_clip(const gbn_tensor *g, const gbn_tensor *out, int64_t count, float max_norm, float eps,
                             float *norm, GradSums *partial, int sms, cudaStream_t s) {
    const int grid = grid_of(g, count, sms);
    const cudaError_t e = run_any(g, nullptr, count, false, grid, 0.f, 0.f, norm, partial, s);
    if (e != cudaSuccess) return e;
    return run_any(g, out, count, true, grid, max_norm, eps, norm, partial, s);
}

}  // namespace gbn
