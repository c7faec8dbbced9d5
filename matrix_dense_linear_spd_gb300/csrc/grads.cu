// Global gradient norm over many tensors, and clipping to a norm.
//
//   norm = sqrt(sum_i sum_j x_ij^2),   y_ij = c * x_ij,   c = norm > max_norm ? max_norm / norm : 1
//
// (c = 1 too where the norm is not finite, or not in f32.) The norm reads every element once and does one
// multiply-add each, so HBM bandwidth bounds it; clipping reads every element twice and writes it
// once. Two launches whatever the number of tensors (up to kMany per launch): the sum kernel
// leaves one f64 partial sum per CTA, and every CTA of the second kernel adds those partials in
// the same order, so no atomics are needed and the result does not depend on the schedule. One
// launch of a single cluster took longer than the two at every size above 10,000 values.
//
// Measured on a GB300: the norm of 1e9 bf16 values 282 us (7.1 TB/s), clipping them 928 us (6.5 TB/s
// for the 6 GB that move), of 1.2e8 f32 values 233 us, 400 odd pieces of a 60 MB buffer 36 us (34 on
// the GPU), 24 small tensors 6.0 us (two short kernels). f64, which its own unit bounds: 1.25e8 values
// 262 us (3.8 TB/s), clipping them 564. Of 2, 4 and 8 loads a thread at 8, 5 and 3 CTAs an SM the middle
// was fastest or within 2% of it at every size.
//
// The tensors' pointers and sizes travel in the kernel's parameters (no host-to-device copy, and
// the call can be captured in a graph). Each tensor is cut into 16 KB chunks that start on a
// 16-byte boundary of memory, wherever the tensor itself starts; a CTA takes a contiguous run of
// chunks, is told the tensor that it starts in and walks.
//
// Squares are summed in f32 over the 16 or 32 values that a thread holds of one chunk and in f64
// from there on. Where that f32 sum leaves [1e-20, 1e30] (squares that overflow, or underflow to
// nothing) the thread adds the same values again in f64: the range of f32 and bf16 is safe. Values of
// 1e-9 and more do not pay for it; where all are below about 2e-11 the f64 unit bounds the norm (values
// of 1e-12: 1e9 of bf16 3,670 us, 2.5e8 of f32 944 us in place of 144).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "host.h"
#include "pdl.cuh"

namespace bl {
namespace grads {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                                     // 16-byte loads a thread has in flight
constexpr int kChunk = kThreads * kVecs * 16;               // 16 KB
constexpr int kCtasPerSm = 5;
constexpr int kMaxCtas = 768;                               // of one launch
constexpr int kFew = 64, kMany = 896;                       // tensors per launch: two sizes of the parameter block

// One cache line's half per tensor: a CTA that walks on to the next tensor waits for one load.
struct Entry {
    const void *x;
    void *y;
    int64_t n;
    int first;                // first chunk; entry[count].first = all chunks
    int dtype;
};
template <int MAXT>
struct Tensors {
    Entry entry[MAXT + 1];
    int count;
    uint16_t start[kMaxCtas];         // the tensor that each CTA's run of chunks starts in (scaling: ends in)
};

static_assert(sizeof(Tensors<kMany>) + 64 <= 32764, "more than a kernel's parameters may hold");

// One 16-byte vector's values as floats (f64: as doubles).
template <typename T> struct Elem;
template <> struct Elem<float> {
    using Wide = float;
    __device__ static float up(float v) { return v; }
    __device__ static float down(float v) { return v; }
};
template <> struct Elem<double> {
    using Wide = double;
    __device__ static double up(double v) { return v; }
    __device__ static double down(double v) { return v; }
};
template <> struct Elem<__nv_bfloat16> {
    using Wide = float;
    __device__ static float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
    using Wide = float;
    __device__ static float up(__half v) { return __half2float(v); }
    __device__ static __half down(float v) { return __float2half_rn(v); }
};

template <typename T>
union Vec {
    static constexpr int N = 16 / sizeof(T);
    uint4 q;
    T e[N];
    __device__ Vec() {}
};

// The part of a tensor that one chunk covers: bytes [lo, hi) of memory, `base` 16-byte aligned.
struct Span {
    uintptr_t base, lo, hi;
};
__device__ __forceinline__ Span span_of(const void *x, int64_t bytes, int64_t k) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(x), a = p & ~uintptr_t(15);
    Span s;
    s.base = a + static_cast<uintptr_t>(k) * kChunk;
    s.lo = s.base > p ? s.base : p;
    const uintptr_t end = p + static_cast<uintptr_t>(bytes), stop = s.base + kChunk;
    s.hi = stop < end ? stop : end;
    return s;
}

// Load the vector at byte address a; elements outside [lo, hi) read as zero and touch no memory.
// LAST: nothing reads it again, L2 need not keep it (with streamed stores: 43.7 us against 51.9 for
// clipping 400 pieces of 60 MB, 935 against 961 us for 2 GB of bf16, f32 the same).
template <bool LAST, typename T>
__device__ __forceinline__ void load(Vec<T> &v, uintptr_t a, const Span &s) {
    if (a >= s.lo && a + 16 <= s.hi) {
        v.q = LAST ? __ldcs(reinterpret_cast<const uint4 *>(a)) : *reinterpret_cast<const uint4 *>(a);
    } else {
        v.q = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) {
            const uintptr_t b = a + i * sizeof(T);
            if (b >= s.lo && b < s.hi) v.e[i] = *reinterpret_cast<const T *>(b);
        }
    }
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const Span &s, int tid) {
      Vec<T> v[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) load<false>(v[u], s.base + (u * kThreads + tid) * 16, s);
    typename Elem<T>::Wide acc = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) {
            const typename Elem<T>::Wide w = Elem<T>::up(v[u].e[i]);
            acc += w * w;
        }
    if constexpr (sizeof(typename Elem<T>::Wide) == 4) {
        if (!(acc >= 1e-20f && acc <= 1e30f)) {       // also taken by all-zero and NaN values
            uint32_t any = 0;
#pragma unroll
            for (int u = 0; u < kVecs; ++u) any |= v[u].q.x | v[u].q.y | v[u].q.z | v[u].q.w;
            if (any == 0) return 0.0;
            double d = 0.0;
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
#pragma unroll
                for (int i = 0; i < Vec<T>::N; ++i) {
                    const double w = static_cast<double>(Elem<T>::up(v[u].e[i]));
                    d = fma(w, w, d);
                }
            return d;
        }
    }
    return static_cast<double>(acc);
}

// The factor, for f64 values and for the others. One near the end of f32's range (norms of 1e30 and more) has
// few bits there or none: it is `single` times `rest`, and the product with `rest` is exact.
struct Factor {
    double whole;
    float single, rest;
    __device__ static Factor of(double c) {
        const bool tiny = c < 0x1p-100;
        return {c, static_cast<float>(tiny ? c * 0x1p64 : c), tiny ? 0x1p-64f : 1.f};
    }
};
__device__ __forceinline__ float scaled(float v, const Factor &c) { return v * c.single * c.rest; }
__device__ __forceinline__ double scaled(double v, const Factor &c) { return v * c.whole; }

template <typename T>
__device__ __forceinline__ void chunk_scale(const Span &s, const void *x, void *y, const Factor &c, int tid) {
    const intptr_t shift = reinterpret_cast<intptr_t>(y) - reinterpret_cast<intptr_t>(x);
    const bool together = (shift & 15) == 0;
    Vec<T> v[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) load<true>(v[u], s.base + (u * kThreads + tid) * 16, s);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const uintptr_t a = s.base + (u * kThreads + tid) * 16;
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) v[u].e[i] = Elem<T>::down(scaled(Elem<T>::up(v[u].e[i]), c));
        if (together && a >= s.lo && a + 16 <= s.hi) {
            __stcs(reinterpret_cast<uint4 *>(a + shift), v[u].q);
        } else {
#pragma unroll
            for (int i = 0; i < Vec<T>::N; ++i) {
                const uintptr_t b = a + i * sizeof(T);
                if (b >= s.lo && b < s.hi) *reinterpret_cast<T *>(b + shift) = v[u].e[i];
            }
        }
    }
}

// Sum of the block's values, for thread 0 only. f64 runs at 1/64 of the f32 rate here, 16 cycles
// of the SM's f64 unit for a warp's instruction, so one warp adds and one thread takes the root: with
// every thread doing it clipping 500,000 values took 17 us instead of 9.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double *slots) {
    slots[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    double t = 0.0, u = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS; w += 64) {
        t += slots[w + threadIdx.x];
        u += slots[w + 32 + threadIdx.x];
    }
    t += u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_down_sync(0xffffffffu, t, o);
    return t;
}

__device__ __forceinline__ int64_t elem_bytes(int dtype) {
    return dtype == BL_F64 ? 8 : dtype == BL_F32 ? 4 : 2;
}

__device__ __forceinline__ double sum_of(const Entry &e, int64_t k, int tid) {
    const Span s = span_of(e.x, e.n * elem_bytes(e.dtype), k);
    if (e.dtype == BL_F32) return chunk_sum<float>(s, tid);
    if (e.dtype == BL_BF16) return chunk_sum<__nv_bfloat16>(s, tid);
    if (e.dtype == BL_F16) return chunk_sum<__half>(s, tid);
    return chunk_sum<double>(s, tid);
}
__device__ __forceinline__ void scale_by(const Entry &e, int64_t k, const Factor &c, int tid) {
    const Span s = span_of(e.x, e.n * elem_bytes(e.dtype), k);
    if (e.dtype == BL_F32) chunk_scale<float>(s, e.x, e.y, c, tid);
    else if (e.dtype == BL_BF16) chunk_scale<__nv_bfloat16>(s, e.x, e.y, c, tid);
    else if (e.dtype == BL_F16) chunk_scale<__half>(s, e.x, e.y, c, tid);
    else chunk_scale<double>(s, e.x, e.y, c, tid);
}
// A norm that the caller sees as not finite, in the f32 that it gets, changes nothing.
__device__ __forceinline__ double factor(double norm, double max_norm) {
    return norm > max_norm && isfinite(static_cast<float>(norm)) ? max_norm / norm : 1.0;
}

template <int MAXT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grads_sum_kernel(const __grid_constant__ Tensors<MAXT> t, double *partials) {
    __shared__ double slots[kThreads];
    pdl_release();
    const int64_t chunks = t.entry[t.count].first;
    const int k0 = static_cast<int>(chunks * blockIdx.x / gridDim.x);
    const int k1 = static_cast<int>(chunks * (blockIdx.x + 1) / gridDim.x);
    int i = t.start[blockIdx.x];
    pdl_wait();
    double acc = 0.0;
    for (int k = k0; k < k1; ++i) {
        const Entry e = t.entry[i];
        const int end = min(t.entry[i + 1].first, k1);
        for (; k < end; ++k) acc += sum_of(e, k - e.first, threadIdx.x);
    }
    acc = block_sum<kThreads>(acc, slots);
    if (threadIdx.x == 0) partials[blockIdx.x] = acc;
}

// Sum of the partials, for thread 0 only (one warp adds them).
__device__ __forceinline__ double total_of(const double *partials, int count) {
    if (threadIdx.x >= 32) return 0.0;
    double t[4] = {0.0, 0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < count; i += 128) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 32 * j < count) t[j] += partials[i + 32 * j];
    }
    double v = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(32) grads_norm_kernel(const double *partials, int count, float *norm) {
    pdl_release();
    pdl_wait();
    const double sum = total_of(partials, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

template <int MAXT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    grads_scale_kernel(const __grid_constant__ Tensors<MAXT> t, const double *partials, int count, double max_norm,
                       float *norm) {
    __shared__ Factor shared_factor;
    pdl_release();
    const int64_t chunks = t.entry[t.count].first;
    const int k0 = static_cast<int>(chunks * blockIdx.x / gridDim.x);
    const int k1 = static_cast<int>(chunks * (blockIdx.x + 1) / gridDim.x);
    int i = t.start[blockIdx.x];
    pdl_wait();
    const double sum = total_of(partials, count);
    if (threadIdx.x == 0) {
        const double all = sqrt(sum);
        if (norm && blockIdx.x == 0) *norm = static_cast<float>(all);
        shared_factor = Factor::of(factor(all, max_norm));
    }
    __syncthreads();
    const Factor c = shared_factor;
    // backwards: what the sum kernel read last is what L2 still holds
    for (int k = k1 - 1; k >= k0; --i) {
        const Entry e = t.entry[i];
        const int stop = max(e.first, k0);
        if (c.whole == 1.0 && e.x == e.y) k = stop - 1;           // in place and nothing to change
        for (; k >= stop; --k) scale_by(e, k - e.first, c, threadIdx.x);
    }
}

// ------------------------------------------------------------------ host

int64_t host_bytes(int dtype) { return dtype == BL_F64 ? 8 : dtype == BL_F32 ? 4 : 2; }

int64_t chunks_of(const void *x, int64_t n, int dtype) {
    const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) & 15);
    return n == 0 ? 0 : (off + n * host_bytes(dtype) + kChunk - 1) / kChunk;
}

bl_status check(const char *op, int64_t count, const int32_t *dtypes, const void *const *x, void *const *y, bool clip,
                const int64_t *sizes, double max_norm, const float *norm, const void *ws, int64_t ws_bytes) {
    if (count < 0 || count > (int64_t(1) << 24))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: count=%lld outside [0, 2^24]", op, (long long)count);
    if (count > 0 && (!dtypes || !x || !sizes || (clip && !y)))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: a list is NULL", op);
    if (!norm || reinterpret_cast<uintptr_t>(norm) % 4 != 0)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: norm is NULL or not 4-byte aligned", op);
    const int64_t need = bl_gnorm_workspace(count);
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 8 != 0 || ws_bytes < need)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: workspace is NULL, not 8-byte aligned or smaller than %lld bytes", op,
                    (long long)need);
    if (clip && !(max_norm >= 0.0)) return fail(BL_ERR_INVALID_ARGUMENT, "%s: max_norm=%g is not >= 0", op, max_norm);
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int d = dtypes[i];
        if (d != BL_F32 && d != BL_F64 && d != BL_BF16 && d != BL_F16)
            return fail(BL_ERR_INVALID_ARGUMENT, "%s: tensor %lld has dtype %d, not f32, f64, bf16 or f16", op, (long long)i, d);
        if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 40))
            return fail(BL_ERR_INVALID_ARGUMENT, "%s: tensor %lld has %lld elements", op, (long long)i, (long long)sizes[i]);
        if (sizes[i] == 0) continue;
        if ((all += sizes[i] * host_bytes(d)) > (int64_t(1) << 44))
            return fail(BL_ERR_INVALID_ARGUMENT, "%s: the tensors hold more than 2^44 bytes", op);
        const uintptr_t es = static_cast<uintptr_t>(host_bytes(d));
        if (!x[i] || reinterpret_cast<uintptr_t>(x[i]) % es != 0)
            return fail(BL_ERR_INVALID_ARGUMENT, "%s: tensor %lld is NULL or not aligned to its element", op, (long long)i);
        if (clip && (!y[i] || reinterpret_cast<uintptr_t>(y[i]) % es != 0))
            return fail(BL_ERR_INVALID_ARGUMENT, "%s: output %lld is NULL or not aligned to its element", op, (long long)i);
    }
    return BL_SUCCESS;
}

// Every result lies in memory of its own: it may be its input, but meets no other tensor of the call
// (the same tensor listed twice in place would be scaled by two CTAs at once). Inputs that are only read
// may meet one another. One walk over both lists in the order of addresses, in which most lists already are (the
// refusal of 400 tensors whose last two meet, with all other checks: 3.7 us in place, 4.8 with outputs, 7.8 of
// the host's time if they are in no order; 60 tensors 1.5 to 2).
bl_status check_overlap(const char *op, int64_t count, const int32_t *dtypes, const void *const *x, void *const *y,
                        const int64_t *sizes) {
    const auto below = [](const Range &a, const Range &b) { return a.lo < b.lo; };
    std::vector<Range> written, read;
    written.reserve(count);
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const int64_t bytes = sizes[i] * host_bytes(dtypes[i]);
        written.push_back(range_of(y[i], bytes));
        if (x[i] != y[i]) read.push_back(range_of(x[i], bytes));
    }
    if (!std::is_sorted(written.begin(), written.end(), below)) std::sort(written.begin(), written.end(), below);
    if (!std::is_sorted(read.begin(), read.end(), below)) std::sort(read.begin(), read.end(), below);
    uintptr_t written_to = 0, read_to = 0;               // what has been passed ends there
    size_t r = 0;
    for (const Range &w : written) {
        for (; r < read.size() && read[r].lo <= w.lo; ++r) {
            if (read[r].lo < written_to) return fail(BL_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input that it is not the result of", op);
            read_to = std::max(read_to, read[r].hi);
        }
        if (w.lo < read_to) return fail(BL_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input that it is not the result of", op);
        if (w.lo < written_to) return fail(BL_ERR_INVALID_ARGUMENT, "%s: two outputs overlap", op);
        written_to = w.hi;
    }
    if (r < read.size() && read[r].lo < written_to)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input that it is not the result of", op);
    return BL_SUCCESS;
}

// Fill the parameter block with tensors [from, ...): as many as fit, none that is empty. Returns
// the first tensor that was not taken. (2^44 bytes are 2^30 chunks: an int holds them.)
template <int MAXT>
int64_t fill(Tensors<MAXT> &t, int64_t from, int64_t count, const int32_t *dtypes, const void *const *x,
             void *const *y, const int64_t *sizes) {
    t.count = 0;
    t.entry[0].first = 0;
    int64_t i = from;
    for (; i < count && t.count < MAXT; ++i) {
        if (sizes[i] == 0) continue;
        Entry &e = t.entry[t.count++];
        e.x = x[i];
        e.y = y ? y[i] : nullptr;
        e.n = sizes[i];
        e.dtype = dtypes[i];
        t.entry[t.count].first = e.first + static_cast<int>(chunks_of(x[i], sizes[i], dtypes[i]));
    }
    return i;
}

// The tensors that hold the first (last) chunk of each of `grid` equal runs of chunks.
template <int MAXT>
void set_starts(Tensors<MAXT> &t, int grid, bool last) {
    const int64_t chunks = t.entry[t.count].first;
    int i = 0;
    for (int b = 0; b < grid; ++b) {
        const int64_t k = last ? chunks * (b + 1) / grid - 1 : chunks * b / grid;
        while (t.entry[i + 1].first <= k) ++i;
        t.start[b] = static_cast<uint16_t>(i);
    }
}

template <int MAXT>
cudaError_t run(int64_t count, const int32_t *dtypes, const void *const *x, void *const *y, const int64_t *sizes,
                double max_norm, float *norm, double *partials, int sms, cudaStream_t s) {
    Tensors<MAXT> t;
    t.count = 0;
    cudaError_t e = cudaSuccess;
    int done = 0;
    bool one = false;
    for (int64_t i = 0; i < count && e == cudaSuccess;) {
        const int64_t from = i;
        i = fill(t, i, count, dtypes, x, y, sizes);
        one = from == 0 && i == count;
        if (t.count == 0) continue;
        const int grid = std::min(std::min(sms * kCtasPerSm, kMaxCtas), t.entry[t.count].first);
        set_starts(t, grid, false);
        e = launch_pdl(grads_sum_kernel<MAXT>, grid, kThreads, 0, s, t, partials + done);
        done += grid;
    }
    if (e != cudaSuccess) return e;
    if (!y || done == 0) return launch_pdl(grads_norm_kernel, 1, 32, 0, s, partials, done, norm);
    bool first = true;
    for (int64_t i = 0; i < count && e == cudaSuccess;) {
        if (!one) i = fill(t, i, count, dtypes, x, y, sizes);
        else i = count;                                  // the block is filled already
        if (t.count == 0) continue;
        const int grid = std::min(std::min(sms * kCtasPerSm, kMaxCtas), t.entry[t.count].first);
        set_starts(t, grid, true);
        e = launch_pdl(grads_scale_kernel<MAXT>, grid, kThreads, 0, s, t, partials, done, max_norm, first ? norm : nullptr);
        first = false;
    }
    return e;
}

bl_status entry(const char *op, int64_t count, const int32_t *dtypes, const void *const *x, void *const *y, bool clip,
                const int64_t *sizes, double max_norm, float *norm, void *ws, int64_t ws_bytes, bl_stream_t stream) {
    clear_error();
    bl_status st = check(op, count, dtypes, x, y, clip, sizes, max_norm, norm, ws, ws_bytes);
    if (st == BL_SUCCESS && clip) {
        try {
            st = check_overlap(op, count, dtypes, x, y, sizes);
        } catch (const std::bad_alloc &) {
            st = fail(BL_ERR_INTERNAL, "%s: out of host memory", op);
        }
    }
    if (st != BL_SUCCESS) return st;
    const int sms = sm_count();
    if (sms <= 0) return fail(BL_ERR_CUDA, "%s: cannot query the current CUDA device", op);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *partials = static_cast<double *>(ws);
    const cudaError_t e = count <= kFew ? run<kFew>(count, dtypes, x, clip ? y : nullptr, sizes, max_norm, norm, partials, sms, s)
                                        : run<kMany>(count, dtypes, x, clip ? y : nullptr, sizes, max_norm, norm, partials, sms, s);
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "%s launch failed: %s", op, cudaGetErrorString(e));
    return BL_SUCCESS;
}

}  // namespace grads
}  // namespace bl

extern "C" {

int64_t bl_gnorm_workspace(int64_t count) {
    using namespace bl::grads;
    if (count < 0 || count > (int64_t(1) << 24)) return -1;
    // one launch's partial sums, for each launch that the list takes
    return 8 * static_cast<int64_t>(kMaxCtas) * (1 + count / kMany);
}

bl_status bl_gnorm(int64_t count, const int32_t *dtypes, const void *const *x, const int64_t *sizes, float *norm,
                   void *workspace, int64_t workspace_bytes, bl_stream_t stream) {
    return bl::grads::entry("gnorm", count, dtypes, x, nullptr, false, sizes, 0.0, norm, workspace, workspace_bytes, stream);
}

bl_status bl_gclip(int64_t count, const int32_t *dtypes, const void *const *x, void *const *y, const int64_t *sizes,
                   double max_norm, float *norm, void *workspace, int64_t workspace_bytes, bl_stream_t stream) {
    return bl::grads::entry("gclip", count, dtypes, x, y, true, sizes, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
