// clip.cu -- the norm of many gradients together, and clipping by it.
//
//   norm = sqrt( sum over tensors and elements of g^2 )
//   out  = round(g * c),  c = max_norm / norm where max_norm < norm < inf, else 1
//
// Both are bound by HBM: 1.08 G BF16 values take 323 us (6.69 TB/s, 0.99 of a copy's rate) and,
// to BF16, 680 us (6.37 TB/s, 0.94); the second reading comes from L2 only as far as that
// reaches.  A launch takes up to kManyVectors tensors, described in its arguments, and cuts
// them into chunks of kChunk elements that its CTAs take in turn.
//
// Squares are summed in 32 bits over a thread's 32 elements of a chunk, and those sums
// with the rounding error of each addition beside them (Knuth's two-sum), so that a sum
// over any number of elements has the error of one over 32; CTAs' sums are joined in 64
// bits.  32 elements whose squares could leave 32 bits' range (largest magnitude above
// 2^48 or below 2^-50) are squared and summed in 64 bits instead.  Sums' order is
// fixed: equal calls give equal bits.
#include <cstdint>

#include "block_mma.cuh"

namespace fp8k {

namespace {

constexpr int kClipThreads = 512;
constexpr int kEach = 32;                       // elements of a chunk per thread
constexpr int kChunk = kClipThreads * kEach;
constexpr int kManyVectors = 1000, kFewVectors = 64;
constexpr int kClipCtas = 2;                    // per SM
constexpr int kClipSms = 152;

// Positions count from the 16-byte boundary at or before a tensor's first element, `off`
// elements before it, so that 16-byte blocks are whole vectors whatever its alignment.
template <int MOST>
struct NormTable {
    const void *base[MOST];   // the boundary
    int64_t end[MOST];        // position past the last element
    uint32_t chunk[MOST];     // the tensor's first chunk
    uint8_t type[MOST], off[MOST];
    uint32_t chunks;
    int count;
};
template <int MOST>
struct ClipTable {
    NormTable<MOST> in;
    void *out[MOST];   // of the element at position 0
    uint8_t out_type[MOST];
};

// The last tensor whose first chunk is not behind c (one without elements has no chunks,
// and is never the last of those that start at c).
template <int MOST>
__device__ __forceinline__ int tensor_of(const NormTable<MOST> &t, uint32_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // elements of a 16-byte block

// This thread's part of a chunk: 32 elements in 16-byte blocks, a chunk's blocks in order of
// the threads.  Positions outside the tensor give 0.
template <typename T>
__device__ __forceinline__ int64_t block_at(int64_t chunk, int i) {
    return chunk * kChunk + (static_cast<int64_t>(i) * kClipThreads + threadIdx.x) * kVec<T>;
}
template <typename T>
__device__ __forceinline__ void load_part(const T *base, int64_t chunk, int off, int64_t end, float (&v)[kEach]) {
    uint4 u[kEach / kVec<T>];
#pragma unroll
    for (int i = 0; i < kEach / kVec<T>; ++i) {
        const int64_t p = block_at<T>(chunk, i);
        if (p >= off && p + kVec<T> <= end) {
            u[i] = *reinterpret_cast<const uint4 *>(base + p);
        } else {
            __align__(16) T e[kVec<T>];
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k)
                e[k] = p + k >= off && p + k < end ? base[p + k] : from_f32<T>(0.0f);
            u[i] = *reinterpret_cast<const uint4 *>(e);
        }
    }
#pragma unroll
    for (int i = 0; i < kEach / kVec<T>; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) {
                v[4 * i + k] = __uint_as_float(w[k]);
            } else {
                const float2 f = unpack2<T>(w[k]);
                v[8 * i + 2 * k] = f.x, v[8 * i + 2 * k + 1] = f.y;
            }
        }
    }
}

struct SquareSum {
    float sum = 0.0f, error = 0.0f;
    double wide = 0.0;

    __device__ __forceinline__ void add(const float (&v)[kEach]) {
        float m = 0.0f;
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < kEach; i += 4) {
            m = absmax3(absmax3(m, v[i], v[i + 1]), v[i + 2], v[i + 3]);
            const uint64_t a = f32x2_pack(v[i], v[i + 1]), b = f32x2_pack(v[i + 2], v[i + 3]);
            s0 = f32x2_fma(a, a, s0);
            s1 = f32x2_fma(b, b, s1);
        }
        if (m == 0.0f || (m >= 0x1p-50f && m <= 0x1p48f)) {   // m is never NaN
            float lo, hi;
            f32x2_unpack(f32x2_add(s0, s1), lo, hi);
            const float x = __fadd_rn(lo, hi);
            const float t = __fadd_rn(sum, x), back = __fsub_rn(t, sum);
            error = __fadd_rn(error, __fadd_rn(__fsub_rn(sum, __fsub_rn(t, back)), __fsub_rn(x, back)));
            sum = t;
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) wide = __fma_rn(static_cast<double>(v[i]), static_cast<double>(v[i]), wide);
        }
    }
    __device__ __forceinline__ double total() const {
        return __dadd_rn(__dadd_rn(static_cast<double>(sum), static_cast<double>(error)), wide);
    }
};

// The sum over the CTA, in a fixed order, in thread 0.
__device__ __forceinline__ double cta_sum(double v) {
    __shared__ double red[32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    }
    return v;
}

// A CTA's sum of squares over its chunks, in thread 0.
template <int MOST>
__device__ __forceinline__ double sum_of_squares(const NormTable<MOST> &t) {
    SquareSum s;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int64_t at = c - t.chunk[k];
        float v[kEach];
        if (t.type[k] == kTypeF32)
            load_part(static_cast<const float *>(t.base[k]), at, t.off[k], t.end[k], v);
        else if (t.type[k] == kTypeBF16)
            load_part(static_cast<const __nv_bfloat16 *>(t.base[k]), at, t.off[k], t.end[k], v);
        else
            load_part(static_cast<const __half *>(t.base[k]), at, t.off[k], t.end[k], v);
        s.add(v);
    }
    return cta_sum(s.total());
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    grad_norm_kernel(const __grid_constant__ NormTable<MOST> t, double *__restrict__ part) {
    pdl_wait();
    pdl_trigger();
    const double sum = sum_of_squares(t);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// Few chunks: one cluster, whose first CTA joins the others' sums.  (148,737 values in three
// tensors: norm and clipping 8.5 us in two launches, 10.3 in three.)
constexpr int kSmallCtas = 8;
constexpr int64_t kSmallChunks = 4 * kSmallCtas;
__global__ void __launch_bounds__(kClipThreads, 1)
    grad_norm_small_kernel(const __grid_constant__ NormTable<kFewVectors> t, float *__restrict__ norm) {
    __shared__ double mine;
    pdl_wait();
    pdl_trigger();
    const double sum = sum_of_squares(t);
    if (threadIdx.x == 0) mine = sum;
    __syncwarp();
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < kSmallCtas; ++k) {
            double v;
            asm volatile("ld.shared::cluster.f64 %0, [%1];"
                         : "=d"(v)
                         : "r"(mapa_shared(smem_u32(&mine), k))
                         : "memory");
            s = __dadd_rn(s, v);
        }
        *norm = __double2float_rn(__dsqrt_rn(s));
    }
    __syncwarp();
    cluster_sync();   // the others' sums have been read
}

__global__ void __launch_bounds__(1024) grad_norm_join_kernel(const double *__restrict__ part, int64_t parts,
                                                              float *__restrict__ norm) {
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += 1024) s = __dadd_rn(s, part[i]);
    s = cta_sum(s);
    if (threadIdx.x == 0) *norm = __double2float_rn(__dsqrt_rn(s));
}

// N elements to `p`, which is aligned to its elements at least.
template <typename T, int N>
__device__ __forceinline__ void store_any(T *p, const float (&v)[N]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if constexpr (sizeof(T) == 4) {
        if (at % 16 == 0) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = v[i];
        }
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        if (at % (N == 8 ? 16 : 8) == 0) {
            if constexpr (N == 8)
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if (at % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

template <typename TI, typename TO>
__device__ __forceinline__ void clip_part(const TI *base, TO *out, int64_t chunk, int off, int64_t end, float c) {
    constexpr int V = kVec<TI>;
    float v[kEach];
    load_part(base, chunk, off, end, v);
#pragma unroll
    for (int i = 0; i < kEach / V; ++i) {
        const int64_t p = block_at<TI>(chunk, i);
        float o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = __fmul_rn(v[V * i + k], c);
        if (p >= off && p + V <= end) {
            store_any<TO, V>(out + p, o);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (p + k >= off && p + k < end) out[p + k] = from_f32<TO>(o[k]);
        }
    }
}

template <typename TI>
__device__ __forceinline__ void clip_to(const TI *base, void *out, int type, int64_t chunk, int off, int64_t end,
                                        float c) {
    if (type == kTypeF32)
        clip_part(base, static_cast<float *>(out), chunk, off, end, c);
    else if (type == kTypeBF16)
        clip_part(base, static_cast<__nv_bfloat16 *>(out), chunk, off, end, c);
    else
        clip_part(base, static_cast<__half *>(out), chunk, off, end, c);
}

// Chunks from the last one back: what the norm's pass read last is still in L2.  A tensor
// that is clipped in place by a factor of 1 is left alone.
template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    grad_clip_kernel(const __grid_constant__ ClipTable<MOST> t, const float *__restrict__ norm, float max_norm) {
    pdl_wait();
    pdl_trigger();
    const float n = *norm;
    const float c = n > max_norm && !is_inf(n) ? __fdiv_rn(max_norm, n) : 1.0f;
    for (uint32_t i = blockIdx.x; i < t.in.chunks; i += gridDim.x) {
        const uint32_t chunk = t.in.chunks - 1 - i;
        const int k = tensor_of(t.in, chunk);
        const int64_t at = chunk - t.in.chunk[k];
        if (c == 1.0f && t.out[k] == t.in.base[k] && t.out_type[k] == t.in.type[k]) continue;
        if (t.in.type[k] == kTypeF32)
            clip_to(static_cast<const float *>(t.in.base[k]), t.out[k], t.out_type[k], at, t.in.off[k], t.in.end[k], c);
        else if (t.in.type[k] == kTypeBF16)
            clip_to(static_cast<const __nv_bfloat16 *>(t.in.base[k]), t.out[k], t.out_type[k], at, t.in.off[k],
                    t.in.end[k], c);
        else
            clip_to(static_cast<const __half *>(t.in.base[k]), t.out[k], t.out_type[k], at, t.in.off[k], t.in.end[k], c);
    }
}

// --------------------------------------------------------------------- host --

int size_of(int type) { return type == kTypeF32 ? 4 : 2; }

template <int MOST>
void fill(NormTable<MOST> &t, const VectorView *v, int count) {
    uint32_t chunks = 0;
    for (int k = 0; k < count; ++k) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(v[k].data);
        const int off = static_cast<int>((p & 15) / size_of(v[k].type));
        t.base[k] = reinterpret_cast<const void *>(p & ~uintptr_t(15));
        t.off[k] = static_cast<uint8_t>(off);
        t.end[k] = off + v[k].n;
        t.type[k] = static_cast<uint8_t>(v[k].type);
        t.chunk[k] = chunks;
        if (v[k].n > 0) chunks += static_cast<uint32_t>((t.end[k] + kChunk - 1) / kChunk);
    }
    t.count = count;
    t.chunks = chunks;
}

template <int MOST>
cudaError_t norm_some(const VectorView *v, int count, double *part, int grid, cudaStream_t st) {
    NormTable<MOST> t;
    fill(t, v, count);
    return launch_pdl(grad_norm_kernel<MOST>, dim3(grid), dim3(kClipThreads), 0, st, t, part);
}

template <int MOST>
cudaError_t clip_some(const VectorView *v, const VectorView *out, int count, const float *norm, float max_norm,
                      int grid, cudaStream_t st) {
    ClipTable<MOST> t;
    fill(t.in, v, count);
    for (int k = 0; k < count; ++k) {
        t.out_type[k] = static_cast<uint8_t>(out[k].type);
        t.out[k] = static_cast<uint8_t *>(out[k].data) - static_cast<int64_t>(t.in.off[k]) * size_of(out[k].type);
    }
    return launch_pdl(grad_clip_kernel<MOST>, dim3(grid), dim3(kClipThreads), 0, st, t, norm, max_norm);
}

int64_t chunks_of(const VectorView *v, int count) {
    int64_t n = 0;
    for (int k = 0; k < count; ++k)
        if (v[k].n > 0) n += (v[k].n + 7 + kChunk - 1) / kChunk;
    return n;
}

int grid_of(const VectorView *v, int count, int sms) {
    const int64_t chunks = chunks_of(v, count), most = static_cast<int64_t>(sms < kClipSms ? sms : kClipSms) * kClipCtas;
    return static_cast<int>(chunks < 1 ? 1 : chunks < most ? chunks : most);
}

}  // namespace

int64_t grad_norm_workspace(int64_t count) {
    const int64_t launches = count <= 0 ? 1 : (count + kManyVectors - 1) / kManyVectors;
    return launches * kClipSms * kClipCtas * static_cast<int64_t>(sizeof(double));
}

cudaError_t launch_grad_norm(const VectorView *v, int count, float *norm, void *ws, int sm_count, cudaStream_t st) {
    if (count <= kFewVectors && chunks_of(v, count) <= kSmallChunks) {
        NormTable<kFewVectors> t;
        fill(t, v, count);
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = cluster_config(dim3(kSmallCtas), kClipThreads, 0, kSmallCtas, attr, st);
        return cudaLaunchKernelEx(&cfg, grad_norm_small_kernel, t, norm);
    }
    double *part = static_cast<double *>(ws);
    int64_t parts = 0;
    for (int k = 0; k < count; k += kManyVectors) {
        const int some = count - k < kManyVectors ? count - k : kManyVectors;
        const int grid = grid_of(v + k, some, sm_count);
        const cudaError_t e = some <= kFewVectors ? norm_some<kFewVectors>(v + k, some, part + parts, grid, st)
                                                  : norm_some<kManyVectors>(v + k, some, part + parts, grid, st);
        if (e != cudaSuccess) return e;
        parts += grid;
    }
    return launch_pdl(grad_norm_join_kernel, dim3(1), dim3(1024), 0, st, static_cast<const double *>(part), parts, norm);
}

cudaError_t launch_grad_clip(const VectorView *v, const VectorView *out, int count, const float *norm,
                             float max_norm, int sm_count, cudaStream_t st) {
    // the last tensors first, as within a launch
    for (int k = (count - 1) / kManyVectors * kManyVectors; k >= 0 && count > 0; k -= kManyVectors) {
        const int some = count - k < kManyVectors ? count - k : kManyVectors;
        const int grid = grid_of(v + k, some, sm_count);
        const cudaError_t e = some <= kFewVectors
                                  ? clip_some<kFewVectors>(v + k, out + k, some, norm, max_norm, grid, st)
                                  : clip_some<kManyVectors>(v + k, out + k, some, norm, max_norm, grid, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace fp8k
