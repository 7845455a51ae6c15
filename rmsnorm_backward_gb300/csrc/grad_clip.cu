// grad_clip.cu -- the global 2-norm of many gradient tensors, and their clip,
// for sm_103a.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + eps)),  out = round(g * coef)
//
// Both kernels walk the same list of 16 KiB chunks; CTA b owns a contiguous
// range of them, so it looks its first tensor up once and then steps.  The
// table of tensors travels in the launch's parameters: nothing is copied to
// the device, nothing outlives the call, and a captured launch keeps its
// own.  Lists longer than a table take several launches.
//  * norm: a thread squares the 16 bytes x 4 it loads of a chunk in float32
//    and adds the batch's sum to a double; the CTA's sum goes to its own
//    double of the workspace, and whoever needs the norm adds those in one
//    fixed order: no atomics, the same bits from run to run.  A batch whose
//    float32 sum left the range in which squares keep their precision is
//    squared again in double from registers, so gradients as small as 1e-38
//    or as large as 3e38 have their norm.
//  * clip: every CTA forms coef from the partial sums itself (no kernel in
//    between), then walks its chunks backwards: what the first pass read
//    last is still in L2.  In place with coef = 1 there is nothing to do.
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
    double *partial;
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

// sum of a batch's squares in double, from its raw vectors
template <typename T>
__device__ __noinline__ double slow_squares(uint4 v0, uint4 v1, uint4 v2, uint4 v3) {
    const uint4 v[kGradVecs] = {v0, v1, v2, v3};
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        float f[Traits<T>::kVec];
        Traits<T>::unpack(v[j], f);
#pragma unroll
        for (int e = 0; e < Traits<T>::kVec; ++e) d += static_cast<double>(f[e]) * static_cast<double>(f[e]);
    }
    return d;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const GradEntry &t, uint32_t chunk) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    const T *src = static_cast<const T *>(t.src);
    const int64_t head = head_of<T>(src, t.n);
    const int64_t nvec = (t.n - head) / V;
    const T *body = src + head;
    const int64_t v0 = static_cast<int64_t>(chunk) * kGradChunkVecs + threadIdx.x;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int64_t v = v0 + j * kGradThreads;
        raw[j] = v < nvec ? ld_global_nc_v4(body + v * V) : make_uint4(0, 0, 0, 0);
    }
    double extra = 0.0;
    if (chunk == 0) {  // the elements before and after the 16-byte vectors
        const int64_t tail = t.n - head - nvec * V;
        if (threadIdx.x < head) {
            const double f = Tr::load1(src + threadIdx.x);
            extra += f * f;
        }
        if (threadIdx.x < tail) {
            const double f = Tr::load1(body + nvec * V + threadIdx.x);
            extra += f * f;
        }
    }
    float s[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        float f[V];
        Tr::unpack(raw[j], f);
        s[j] = f[0] * f[0];
#pragma unroll
        for (int e = 1; e < V; ++e) s[j] = fmaf(f[e], f[e], s[j]);
    }
    static_assert(kGradVecs == 4, "the sum below");
    const float b = (s[0] + s[1]) + (s[2] + s[3]);
    // squares below 2^-126 lose bits, above 2^128 they overflow
    if (!(b >= 0x1p-80f && b <= 0x1p100f)) {
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < kGradVecs; ++j) any |= raw[j].x | raw[j].y | raw[j].z | raw[j].w;
        if (any) return extra + slow_squares<T>(raw[0], raw[1], raw[2], raw[3]);
    }
    return extra + static_cast<double>(b);
}

// sum over the CTA in a fixed order; every thread gets it
__device__ __forceinline__ double cta_sum(double v, double *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
#pragma unroll
    for (int w = 1; w < kGradThreads / 32; ++w) v += sm[w];
    __syncthreads();
    return v;
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
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ double sm[kGradThreads / 32];
    // the gradients, and whoever still reads the partial sums, come before
    // this kernel on the stream; the clip may launch meanwhile and waits
    griddep_wait();
    griddep_launch_dependents();
    double sum = 0.0;
    uint32_t c, c1;
    cta_range(t.chunks, c, c1);
    if (c < c1) {
        int i = find_entry(t, c);
        for (; c < c1; ++c) {
            while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
            const GradEntry &e = t.e[i];
            const uint32_t k = c - e.first;
            sum += e.dtype == GBN_F32   ? chunk_squares<float>(e, k)
                   : e.dtype == GBN_F16 ? chunk_squares<__half>(e, k)
                                        : chunk_squares<__nv_bfloat16>(e, k);
        }
    }
    sum = cta_sum(sum, sm);
    if (threadIdx.x == 0) t.partial[blockIdx.x] = t.add ? t.partial[blockIdx.x] + sum : sum;
}

// the norm from the CTAs' sums, in a fixed order
__device__ __forceinline__ double norm_of(const double *partial, int total, double *sm) {
    double v = 0.0;
    for (int i = threadIdx.x; i < total; i += kGradThreads) v += __ldcg(partial + i);
    return sqrt(cta_sum(v, sm));
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_finish_kernel(const double *partial, int total,
                                                                       float *norm) {
    __shared__ double sm[kGradThreads / 32];
    griddep_wait();
    const double n = norm_of(partial, total, sm);
    if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const GradEntry &t, uint32_t chunk, float coef) {
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    const T *src = static_cast<const T *>(t.src);
    T *dst = static_cast<T *>(t.dst);
    const int64_t head = head_of<T>(src, t.n);
    const int64_t nvec = (t.n - head) / V;
    const int64_t v0 = static_cast<int64_t>(chunk) * kGradChunkVecs + threadIdx.x;
    const bool same = (reinterpret_cast<uintptr_t>(dst + head) & 15) == 0;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int64_t v = v0 + j * kGradThreads;
        if (v < nvec) raw[j] = *reinterpret_cast<const uint4 *>(src + head + v * V);
    }
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int64_t v = v0 + j * kGradThreads;
        if (v < nvec) {
            float f[V];
            Tr::unpack(raw[j], f);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] *= coef;
            T *d = dst + head + v * V;
            if (same) {
                *reinterpret_cast<uint4 *>(d) = Tr::pack(f);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) Tr::store1(d + e, f[e]);
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
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ double sm[kGradThreads / 32];
    griddep_wait();
    const double norm = norm_of(t.partial, t.total, sm);
    if (blockIdx.x == 0 && threadIdx.x == 0 && !t.add) *t.norm = static_cast<float>(norm);
    const double c = static_cast<double>(t.max_norm) / (norm + static_cast<double>(t.eps));
    const float coef = c >= 1.0 ? 1.f : static_cast<float>(c);  // NaN stays NaN
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
            chunk_scale<float>(e, at, coef);
        else if (e.dtype == GBN_F16)
            chunk_scale<__half>(e, at, coef);
        else
            chunk_scale<__nv_bfloat16>(e, at, coef);
    }
}

template <typename K, typename P>
cudaError_t launch_pdl(K kernel, int grid, cudaStream_t s, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kGradThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// One pass over the list: tables of up to CAP tensors, a launch for each.
template <int CAP>
cudaError_t run_list(const gbn_tensor *g, const gbn_tensor *out, int64_t count, bool clip, int grid, float max_norm,
                     float eps, float *norm, double *partial, cudaStream_t s) {
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
        const cudaError_t r = clip ? launch_pdl(grad_clip_kernel<CAP>, grid, s, t)
                                   : launch_pdl(grad_norm_kernel<CAP>, grid, s, t);
        if (r != cudaSuccess) return r;
        first = false;
    } while (i < count);
    return cudaSuccess;
}

cudaError_t run_any(const gbn_tensor *g, const gbn_tensor *out, int64_t count, bool clip, int grid, float max_norm,
                    float eps, float *norm, double *partial, cudaStream_t s) {
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

cudaError_t launch_grad_norm(const gbn_tensor *g, int64_t count, float *norm, double *partial, int sms,
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
    return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const double *>(partial), grid, norm);
}

cudaError_t launch_grad_clip(const gbn_tensor *g, const gbn_tensor *out, int64_t count, float max_norm, float eps,
                             float *norm, double *partial, int sms, cudaStream_t s) {
    const int grid = grid_of(g, count, sms);
    const cudaError_t e = run_any(g, nullptr, count, false, grid, 0.f, 0.f, norm, partial, s);
    if (e != cudaSuccess) return e;
    return run_any(g, out, count, true, grid, max_norm, eps, norm, partial, s);
}

}  // namespace gbn
