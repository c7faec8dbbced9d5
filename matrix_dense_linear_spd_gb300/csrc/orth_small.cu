// The orthogonalisation of small matrices: one CTA takes a matrix, or several that fill its 128 rows, through all
// steps without going back to memory.
//
// The shorter side, up to 128, lies along the rows of tensor memory and the longer, up to 256, along its columns,
// whichever of them is contiguous in memory. X stays in registers in f32, a thread holding a quarter of a row; its f16
// planes (the one that is multiplied, or both) are in shared memory in 64-column panels, which the Gram matrix reads
// K-major and the product with B MN-major. A and then B take one further buffer. Three products follow each other
// in every step, each waiting for the previous one's epilogue: latency bounds it. One 128 x 128 bf16 matrix takes
// five steps in 20 us (730 in elementary operations; 82 with a launch for each product), 200 f32 matrices of 96 x 64 in
// 30 us (1,050 and 157). Of the 20, 3 go to loading and the norm, 2 to the end; a product of 128 x 128 x 128 takes
// 0.4 and its epilogue 0.2 to 0.6.
//
// Sides of up to 64, 32 and 16 leave room for 2, 4 and 8 matrices in the 128 rows: blocks of A off the diagonal are
// set to 0, and what no f16 holds (a matrix that diverges) is cut, so that it meets its neighbours' zeros as a
// finite number. Matrices share a CTA only where there are more of them than SMs.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "host.h"
#include "orth.h"
#include "orth_gemm.cuh"

namespace bl {
namespace orth {

namespace {

constexpr int kRows = 128, kSides = 4, kSmallThreads = kSides * kRows;

struct Small {
    const void *g;
    void *x;
    int64_t ldg, stride_g, ldx, stride_x;
    int m, n;                       // shorter and longer side
    bool turned;                    // the shorter side is the contiguous one
    bool vec_g, vec_x;              // 16-byte pieces
    int batch, share, rows_each;    // matrices of a CTA, and their rows
    int steps;
    float a, b, c;
    int spoil;
};

// Row `row` of what lies in 64-column panels of 128 lines, 128-byte swizzle: 8 values starting at column c.
__device__ __forceinline__ unsigned char *at128(unsigned char *base, int row, int c) {
    return base + (c >> 6) * (kRows * 128) + row * 128 + ((((c & 63) >> 3) ^ (row & 7)) << 4);
}

// CUT: what f16 does not hold is cut to what it does.
template <int PLANES, bool CUT = false>
__device__ __forceinline__ void put8(unsigned char *base, int plane_bytes, int row, int c, const float *v) {
    const __half2 limit = __float2half2_rn(65504.f);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        if (CUT) h = __hmax2(__hmin2(h, limit), __hneg2(limit));
        hi[i] = *reinterpret_cast<const uint32_t *>(&h);
        if (PLANES == 2) {
            const float2 back = __half22float2(h);
            __half2 l = __floats2half2_rn(v[2 * i] - back.x, v[2 * i + 1] - back.y);
            if (CUT) l = __hmax2(__hmin2(l, limit), __hneg2(limit));
            lo[i] = *reinterpret_cast<const uint32_t *>(&l);
        }
    }
    *reinterpret_cast<uint4 *>(at128(base, row, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (PLANES == 2) *reinterpret_cast<uint4 *>(at128(base + plane_bytes, row, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
__device__ __forceinline__ float2 sum2(uint32_t hi, uint32_t lo) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&hi)), y = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    return make_float2(x.x + y.x, x.y + y.y);
}
template <int PLANES>
__device__ __forceinline__ void get8(unsigned char *base, int plane_bytes, int row, int c, float *v) {
    const uint4 h = *reinterpret_cast<const uint4 *>(at128(base, row, c));
    uint4 l = make_uint4(0, 0, 0, 0);
    if (PLANES == 2) l = *reinterpret_cast<const uint4 *>(at128(base + plane_bytes, row, c));
    const uint32_t hi[4] = {h.x, h.y, h.z, h.w}, lo[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = sum2(hi[i], lo[i]);
        v[2 * i] = x.x, v[2 * i + 1] = x.y;
    }
}

// The values that a thread holds: which matrix, its row, and from which column on how many.
struct Held {
    int64_t item;
    int r, c, count;
    __device__ __forceinline__ Held(const Small &q, int block, int row, int c0, int most) {
        const int slot = row / q.rows_each;
        item = static_cast<int64_t>(block) * q.share + slot;
        r = row - slot * q.rows_each;
        c = c0;
        count = slot < q.share && item < q.batch && r < q.m ? max(0, min(most, q.n - c0)) : 0;
    }
    __device__ __forceinline__ int64_t at(int64_t ld, int64_t stride, bool turned) const {
        return count > 0 ? item * stride + (turned ? c * ld + r : r * ld + c) : 0;
    }
};

// NC: columns that a thread holds (the longer side is 4 NC at most).
template <typename T, int NC>
__global__ void __launch_bounds__(kSmallThreads, NC == 16 && sizeof(T) == 2 ? 2 : 1) small_kernel(const __grid_constant__ Small q) {
    constexpr int PLANES = sizeof(T) == 4 ? 2 : 1, PAIRS = PLANES == 1 ? 1 : 3;
    constexpr int N = kSides * NC, kPlaneX = N / 64 * kRows * 128, kPlaneP = 2 * kRows * 128;
    constexpr uint32_t kColumns = N > kRows ? N : kRows;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *const xs = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *const ps = xs + PLANES * kPlaneX;
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sums[8][kSides];
    __shared__ double wide_sums[8][kSides];
    __shared__ int lost[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = (warp & 3) * 32 + lane, side = warp >> 2;
    if (warp == 0) {
        tc::tmem_alloc(&tmem_slot, kColumns);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        tc::mbar_init(&bar, 1);
        tc::mbar_fence_init();
    }
    if (threadIdx.x < 8) lost[threadIdx.x] = 0;
    __syncthreads();
    pdl_release();
    pdl_wait();

    // this thread's quarter of a row
    const int slot = row / q.rows_each, c0 = side * NC;
    const Held here(q, blockIdx.x, row, c0, NC);
    const int held = here.count;
    const T *const g = static_cast<const T *>(q.g) + here.at(q.ldg, q.stride_g, q.turned);
    float x[NC];
    constexpr int PER = 16 / sizeof(T);
    if (q.vec_g) {
#pragma unroll
        for (int i = 0; i < NC; i += PER) {
            __align__(16) T v[PER];
            if (i + PER <= held) {
                *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(g + i);
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) v[e] = i + e < held ? g[i + e] : T(0.f);
            }
#pragma unroll
            for (int e = 0; e < PER; ++e) x[i + e] = static_cast<float>(v[e]);
        }
    } else {
        const int64_t step = q.turned ? q.ldg : 1;
        const T *p = g;
#pragma unroll
        for (int i = 0; i < NC; ++i, p += step) x[i] = i < held ? static_cast<float>(*p) : 0.f;
    }
    // The norm: in f32, pairs of lanes and warps, and once more in f64, which an SM has little of, for a matrix whose
    // squares leave f32's comfortable range.
    constexpr int GROUP = NC < 32 ? NC : 32;
    float sum = 0.f, most = 0.f;
#pragma unroll
    for (int i = 0; i < NC; i += GROUP) {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < GROUP; ++e) s[e & 1] = fmaf(x[i + e], x[i + e], s[e & 1]), most = fmaxf(most, fabsf(x[i + e]));
        sum += s[0] + s[1];
    }
    if (slot < q.share && !(sum <= 1e30f && (sum >= 1e-25f || most == 0.f))) lost[slot] = 1;
    const int together = min(32, q.rows_each);
    for (int o = 1; o < together; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // by 32-row groups (or 16-row ones), the four quarters of a row together
    if ((lane & 15) == 0) sums[(warp & 3) * 2 + (lane >> 4)][side] = sum;
    __syncthreads();
    const bool wide = slot < q.share && lost[slot];
    // this matrix's entries: one of 16 rows, or every other one, of 32
    const int step_w = together == 16 ? 1 : 2, from = slot * q.rows_each / 16, until = min(8, from + max(1, q.rows_each / 16));
    float2 factor = make_float2(0.f, 0.f);
    if (__syncthreads_or(wide)) {
        double all = 0.0;
#pragma unroll 1
        for (int i = 0; i < held && wide; ++i) {
            const double y = static_cast<double>(static_cast<float>(g[i * (q.turned ? q.ldg : 1)]));
            all = fma(y, y, all);
        }
        for (int o = 1; o < together; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if ((lane & 15) == 0) wide_sums[(warp & 3) * 2 + (lane >> 4)][side] = all;
        __syncthreads();
        all = 0.0;
        for (int w = from; w < until; w += step_w) all += (wide_sums[w][0] + wide_sums[w][1]) + (wide_sums[w][2] + wide_sums[w][3]);
        factor = scale_of(all);
        if (threadIdx.x < 8) lost[threadIdx.x] = 0;
        __syncthreads();
    }
    if (!wide) {
        sum = 0.f;
        for (int w = from; w < until; w += step_w) {
            const float4 t = *reinterpret_cast<const float4 *>(sums[w]);
            sum += (t.x + t.y) + (t.z + t.w);
        }
        factor = sum > 0.f ? make_float2(1.f, kScaleX / sqrtf(sum)) : make_float2(0.f, 0.f);
    }
    bool bad = factor.y != factor.y;
#pragma unroll
    for (int i = 0; i < NC; ++i) x[i] = bad ? 0.f : x[i] * factor.x * factor.y;

    const auto x_out = [&] {
#pragma unroll
        for (int i = 0; i < NC; i += 8) {
            put8<PLANES, true>(xs, kPlaneX, row, c0 + i, x + i);
        }
    };
    x_out();
    const int rows = q.share == 1 ? (q.m + 15) & ~15 : kRows;            // of A and B
    const int cols = (q.n + 31) & ~31;                                   // X is zero from n on
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    // One thread issues a product, all wait for it: A = X X^T (of_x), A A, or B X (apply)
    const auto product = [&](int parity, bool of_x, bool apply, int k, int n) {
        tc::fence_before_sync();
        tc::fence_proxy_async_smem();
        ok = !__syncthreads_or(!ok);
        tc::fence_after_sync();
        if (!ok) return;
        if (warp == 0) {
            // by the warp as a whole, one lane issuing: 40 cycles a product, 115 in a branch of one thread's
            const uint32_t tmem = tmem_slot, idesc = tc::idesc_f16(kRows, n, false, apply);
            const uint64_t da0 = tc::sdesc_sw128(tc::smem_u32(of_x ? xs : ps));
            const uint64_t db0 = apply ? tc::sdesc_mn_sw128(tc::smem_u32(xs), kRows * 128) : da0;
            const int plane_a = (of_x ? kPlaneX : kPlaneP) >> 4, plane_b = (apply || of_x ? kPlaneX : kPlaneP) >> 4;
            const int panel_b = apply ? 4 * 2048 / 16 : kRows * 128 / 16, step_b = apply ? 2048 / 16 : 2;
            if (tc::elect()) {
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) {
                    uint64_t da = da0 + (PLANES == 2 && p == 1 ? plane_a : 0), db = db0 + (PLANES == 2 && p == 0 ? plane_b : 0);
#pragma unroll 1
                    for (int j0 = 0; j0 < k; j0 += 64) {
                        // 16 k: 32 bytes along a line, lines of 64 k in panels; or 16 lines
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j0 + 16 * j < k) tc::mma_f16<1>(tmem, da + j * 2, db + j * step_b, idesc, p > 0 || j0 > 0 || j > 0);
                        da += kRows * 128 / 16;
                        db += panel_b;
                    }
                }
                tc::mma_commit(&bar);
            }
            __syncwarp();
        }
        ok = tc::mbar_wait(&bar, parity, kPolls);
        tc::fence_after_sync();
    };
    constexpr int READ = NC == 32 ? 32 : 16;     // 64 values of X leave no room for more
    constexpr int PC = kRows / kSides;           // columns of A that a thread holds
    const int p0 = side * PC, shift = 31 - __clz(q.rows_each), own = row >> shift;     // its matrix
    const auto read = [&](int c, float (&t)[READ]) {
        __syncwarp();
        if constexpr (READ == 32) tc::tmem_ld32(tmem_slot + lanes + c, t);
        else tc::tmem_ld16(tmem_slot + lanes + c, t);
    };
    const bool mine[2] = {p0 >> shift == own, (p0 + 16) >> shift == own};
#pragma unroll 1
    for (int step = 0; step < q.steps; ++step) {
        // A, times 2^12
        product(step & 1, true, false, cols, rows);
        float t[READ];
#pragma unroll
        for (int h = 0; h < PC; h += READ) {
            read(p0 + h, t);
#pragma unroll
            for (int i = 0; i < READ; ++i) t[i] = mine[(h + i) >> 4] ? t[i] * (4096.f / (8192.f * 8192.f)) : 0.f;
#pragma unroll
            for (int i = 0; i < READ; i += 8) put8<PLANES>(ps, kPlaneP, row, p0 + h + i, t + i);
        }
        // B = b A + c A A, times 2^12, in A's place
        product(~step & 1, false, false, rows, rows);
#pragma unroll
        for (int h = 0; h < PC; h += READ) {
            read(p0 + h, t);
#pragma unroll
            for (int i = 0; i < READ; i += 8) {
                float v[8];
                get8<PLANES>(ps, kPlaneP, row, p0 + h + i, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = mine[(h + i) >> 4] ? fmaf(q.c / 4096.f, t[i + e], q.b * v[e]) : 0.f;
                put8<PLANES>(ps, kPlaneP, row, p0 + h + i, v);
            }
        }
        // X
        product(step & 1, false, true, rows, cols);
        uint32_t largest = 0;
#pragma unroll
        for (int h = 0; h < NC; h += READ) {
            if (c0 + h >= cols) break;
            read(c0 + h, t);
#pragma unroll
            for (int i = 0; i < READ; ++i) {
                x[h + i] = fmaf(q.a, x[h + i], t[i] * (1.f / 4096.f));
                largest = max(largest, __float_as_uint(x[h + i]) & 0x7fffffffu);        // NaN is larger than infinity
            }
        }
        // between steps X is f16, the last one is not
        const bool last = step + 1 == q.steps;
        bad |= largest > __float_as_uint(last ? 3.4028235e38f : 65504.f);
        if (!last) x_out();
    }
    // what a matrix or a product lost is seen in all of it
    if (!ok) tc::mbar_wait(&bar, 0, kPolls), tc::mbar_wait(&bar, 1, kPolls);         // what gave up may still come to its end
    bad |= !ok || q.spoil;
    if (bad && slot < 8) lost[slot] = 1;
    __syncthreads();
    bad = slot < 8 && lost[slot];
    int again = row;                             // worked out again: kept, it crowds X out of its registers
    asm volatile("" : "+r"(again));
    const Held there(q, blockIdx.x, again, c0, NC);
    T *const to = static_cast<T *>(q.x) + there.at(q.ldx, q.stride_x, q.turned);
    const auto value = [&](float f) {
        const float y = bad ? NAN : f * (1.f / 8192.f);
        if constexpr (PLANES == 1) return __float2bfloat16_rn(y);
        else return y;
    };
    if (q.vec_x) {
#pragma unroll
        for (int i = 0; i < NC; i += PER) {
            __align__(16) T v[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) v[e] = value(x[i + e]);
            if (i + PER <= there.count) {
                *reinterpret_cast<uint4 *>(to + i) = *reinterpret_cast<const uint4 *>(v);
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (i + e < there.count) to[i + e] = v[e];
            }
        }
    } else {
        const int64_t step = q.turned ? q.ldx : 1;
        T *p = to;
#pragma unroll
        for (int i = 0; i < NC; ++i, p += step)
            if (i < there.count) *p = value(x[i]);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem_slot, kColumns);
}

template <typename T, int NC>
cudaError_t launch(const Small &q, cudaStream_t s) {
    constexpr int PLANES = sizeof(T) == 4 ? 2 : 1;
    constexpr int kSmem = PLANES * (kSides * NC / 64 + 2) * kRows * 128 + 1024;
    static std::atomic<unsigned long long> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(bit & done.load(std::memory_order_acquire))) {
        e = cudaFuncSetAttribute(small_kernel<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_pdl(small_kernel<T, NC>, static_cast<unsigned>((q.batch + q.share - 1) / q.share), kSmallThreads, kSmem, s, q);
}
template <typename T>
cudaError_t launch(const Small &q, cudaStream_t s) {
    return q.n <= 64 ? launch<T, 16>(q, s) : q.n <= 128 ? launch<T, 32>(q, s) : launch<T, 64>(q, s);
}

}  // namespace

bool fits_small(int64_t lines, int64_t width) { return std::min(lines, width) <= kRows && std::max(lines, width) <= 256; }

cudaError_t launch_small(int dtype, int64_t lines, int64_t width, int64_t batch, const void *g, int64_t ldg, int64_t stride_g, void *x,
                         int64_t ldx, int64_t stride_x, int steps, const double *coefficients, int sms, cudaStream_t s) {
    Small q{};
    const int64_t es = dtype == BL_F32 ? 4 : 2;
    q.g = g, q.x = x, q.ldg = ldg, q.stride_g = stride_g, q.ldx = ldx, q.stride_x = stride_x;
    q.turned = lines > width;
    q.m = static_cast<int>(std::min(lines, width));
    q.n = static_cast<int>(std::max(lines, width));
    const auto vec = [&](const void *p, int64_t ld, int64_t stride) {
        return !q.turned && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && (batch == 1 || stride * es % 16 == 0);
    };
    q.vec_g = vec(g, ldg, stride_g);
    q.vec_x = vec(x, ldx, stride_x);
    q.batch = static_cast<int>(batch);
    q.rows_each = q.m <= 16 ? 16 : q.m <= 32 ? 32 : q.m <= 64 ? 64 : kRows;
    q.share = 1;
    while (q.share * 2 * q.rows_each <= kRows && (batch + q.share - 1) / q.share > sms) q.share *= 2;
    if (q.share == 1) q.rows_each = kRows;
    q.steps = steps;
    q.a = static_cast<float>(coefficients[0]), q.b = static_cast<float>(coefficients[1]), q.c = static_cast<float>(coefficients[2]);
    q.spoil = gave_up_wanted();
    return dtype == BL_F32 ? launch<float>(q, s) : launch<__nv_bfloat16>(q, s);
}

}  // namespace orth
}  // namespace bl
