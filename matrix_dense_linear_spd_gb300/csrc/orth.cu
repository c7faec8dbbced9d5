// Orthogonalised steps: Newton-Schulz products on a matrix, or a batch of them.
//
//   X_0 = G / |G|_F,   A = X X^T (on the shorter side),   X <- a X + (b A + c A A) X
//
// The singular vectors stay and every singular value s goes to a s + b s^3 + c s^5, step by step towards 1. A value
// that starts near 0 is multiplied by a in each step, 485 times in all for a = 3.4445 and five steps, and so is
// what a rounding of X leaves in those directions; directions that have grown take the products' roundings as they
// are. So the term a X carries 22 bits (two planes of f16) whatever the type, and for bf16 the three products take
// one plane (11 bits): against 64 bits, bf16 matrices of 256 x 512 with eight strong directions come out 4e-4 off
// (relative 2-norm, before the result's rounding of 1.7e-3), with X in one plane of f16 4e-2, with all in bf16
// 0.3. f32 operands multiply both planes.
//
// Three launches a step: the Gram matrix, its polynomial and the product with X each leave in the form that the next
// one reads. A matrix is stored as lines of contiguous values; whether
// those are its rows or its columns changes only which of the operands are read K-major (orth_gemm.cuh), so
// nothing is ever transposed in memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "orth.h"
#include "orth_gemm.cuh"
#include "pdl.cuh"
#include "tensor_map.h"

namespace bl {
namespace orth {

// ------------------------------------------------------------------ elementwise kernels

struct Source {
    const void *g;
    int64_t ld, stride;
    uint32_t lines, width, per_line;      // per_line: groups of 8 values
    int chunks;                           // CTAs of an item
    int vec;                              // groups may be read whole
    double *sums;                         // [item][chunks]
};

template <typename T>
__device__ __forceinline__ void load8(const Source &q, const T *item, uint32_t at, float (&x)[8]) {
    const uint32_t line = at / q.per_line, c = (at - line * q.per_line) * 8;
    const T *const p = item + line * q.ld + c;
    if (q.vec && c + 8 <= q.width) {
        __align__(16) T v[8];
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(v) / 16); ++e)
            reinterpret_cast<uint4 *>(v)[e] = reinterpret_cast<const uint4 *>(p)[e];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = c + e < q.width ? static_cast<float>(p[e]) : 0.f;
    }
}

// A block's sum, in thread 0 and the same every time.
__device__ __forceinline__ double block_sum(double s) {
    __shared__ double warps[8];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int w = 0; w < 8; ++w) s += warps[w];
    }
    return s;
}

// (An SM adds f64 values at a sixtieth of its f32 rate: with all threads of the first X's CTAs adding up the norm and one CTA for 1024
// groups of values, 12 x 1024 x 4096 took 994 us in place of 960.)
// Sums of squares: eight in f32, from there on f64. Where eight leave f32's comfortable range they are formed
// again in f64.
template <typename T>
__global__ void __launch_bounds__(256) sums_kernel(const __grid_constant__ Source q, int32_t *gave_up) {
    pdl_release();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *gave_up = 0;
    const int64_t item = blockIdx.x / q.chunks;
    const uint32_t chunk = blockIdx.x - item * q.chunks, all = q.lines * q.per_line;
    const T *const g = static_cast<const T *>(q.g) + item * q.stride;
    double sum = 0.0;
    for (uint32_t i = chunk * 256 + threadIdx.x; i < all; i += q.chunks * 256) {
        float x[8], s = 0.f;
        load8(q, g, i, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
        if (s >= 1e-25f && s <= 1e30f) {
            sum += s;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(x[e]), static_cast<double>(x[e]), sum);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) q.sums[blockIdx.x] = sum;
}

// X_0 in two planes. A matrix of zeros stays one; a norm that is not finite makes all of X NaN.
template <typename T>
__global__ void __launch_bounds__(256) begin_kernel(const __grid_constant__ Source q, __half *x, int64_t ldx, int64_t plane) {
    pdl_release();
    pdl_wait();
    const int64_t item = blockIdx.x / q.chunks;
    const uint32_t chunk = blockIdx.x - item * q.chunks, all = q.lines * q.per_line;
    __shared__ float2 shared_factor;
    if (threadIdx.x < 32) {               // of the small f64 unit as little as will do: a warp, then a thread
        double sum = 0.0;
        for (int i = threadIdx.x; i < q.chunks; i += 32) sum += q.sums[item * q.chunks + i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x == 0) shared_factor = scale_of(sum);
    }
    __syncthreads();
    const float2 factor = shared_factor;
    const T *const g = static_cast<const T *>(q.g) + item * q.stride;
    __half *const to = x + item * q.lines * ldx;
    for (uint32_t i = chunk * 256 + threadIdx.x; i < all; i += q.chunks * 256) {
        float v[8];
        load8(q, g, i, v);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float a = v[e] * factor.x * factor.y, b = v[e + 1] * factor.x * factor.y;
            const __half ha = __float2half_rn(a), hb = __float2half_rn(b);
            hi[e / 2] = pack(ha, hb);
            lo[e / 2] = pack(__float2half_rn(a - __half2float(ha)), __float2half_rn(b - __half2float(hb)));
        }
        const uint32_t line = i / q.per_line;
        const int64_t at = line * ldx + static_cast<int64_t>(i - line * q.per_line) * 8;
        *reinterpret_cast<uint4 *>(to + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(to + plane + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// A product that gave up makes all results NaN.
template <typename T>
__global__ void __launch_bounds__(256) spoil_kernel(const int32_t *gave_up, T *out, int64_t ld, int64_t stride, int64_t lines,
                                                    int64_t all_lines, int64_t width) {
    pdl_release();
    pdl_wait();
    if (*gave_up == 0) return;
    for (int64_t l = blockIdx.x; l < all_lines; l += gridDim.x)
        for (int64_t c = threadIdx.x; c < width; c += 256) put(out + l / lines * stride + l % lines * ld + c, NAN);
}

// ------------------------------------------------------------------ plan

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t cdiv(int64_t v, int64_t by) { return (v + by - 1) / by; }

struct Shape {
    int ctas, tile_n, tiles_m, tiles_n, per_item;
};
int tiles_of(const Shape &s, bool symmetric) {
    if (!symmetric) return s.tiles_m * s.tiles_n;
    int n = 0;
    for (int tm = 0; tm < s.tiles_m; ++tm)
        n += std::min<int64_t>(s.tiles_n, cdiv(static_cast<int64_t>(tm + 1) * s.ctas * kTileM, s.tile_n));
    return n;
}
// Cycles of a 64-deep step: the products' own, 8192 multiply-adds a cycle on two SMs, or the operands' way into shared
// memory, 64 bytes a cycle and SM, whichever takes longer.
int64_t step_cycles(int ctas, int tile_n, int planes) {
    const int64_t products = (planes == 1 ? 1 : 3) * 2 * tile_n, bytes = planes * (kTileM * 128 + tile_n / ctas * 128);
    return std::max(products, bytes / 64);
}
// The tile that takes the least time, in rounds of all SMs. What comes before and after a round's steps takes some
// 2000 cycles, and as many the start and end of a launch in pairs: 512 x 512 bf16 on pairs 127 us, on single CTAs 107; 1024 x 1024
// 157 and 147; 2048 x 2048 274 and 302.
Shape shape_for(int64_t rows, int64_t cols, bool symmetric, bool b_mn, int64_t batch, int64_t kblocks, int planes, int sms) {
    Shape best{};
    int64_t least = 0;
    for (int ctas = 2; ctas >= 1; --ctas) {
        if (ctas == 2 && rows <= kTileM) continue;
        for (int t = ctas * 128; t >= (ctas == 2 && b_mn ? 128 : 64); t /= 2) {        // a pair's halves: whole groups of 64
            Shape s{ctas, t, static_cast<int>(cdiv(rows, ctas * kTileM)), static_cast<int>(cdiv(cols, t)), 0};
            s.per_item = tiles_of(s, symmetric);
            const int64_t rounds = cdiv(batch * s.per_item, std::max(1, sms / ctas));
            const int64_t cost = rounds * (kblocks * step_cycles(ctas, t, planes) + 2000) + (ctas == 2 ? 2000 : 0);
            if (best.ctas == 0 || cost < least) best = s, least = cost;
        }
    }
    return best;
}
template <int PLANES>
int stages_of(const Shape &s) {
    return std::min(kMostStages, Ring<PLANES, 1>::kBytes / (s.ctas == 1 ? Ring<PLANES, 1>::stage(s.tile_n) : Ring<PLANES, 2>::stage(s.tile_n)));
}

struct Plan {
    int planes;
    int64_t lines, width, small, batch;
    bool wide;                                     // lines are the shorter side
    int64_t ldx, lda;
    int chunks;
    Shape gram, square, apply;
    int64_t gave_up, sums, x[2], a, b, bytes;      // offsets into the workspace
};

Plan plan_for(int dtype, int64_t lines, int64_t width, int64_t batch, int sms) {
    Plan q{};
    if (fits_small(lines, width)) return q;
    q.planes = dtype == BL_F32 ? 2 : 1;
    q.lines = lines, q.width = width, q.batch = batch;
    q.wide = lines <= width;
    q.small = std::min(lines, width);
    q.ldx = up(width, 64);
    q.lda = up(q.small, 64);
    const int64_t groups = lines * cdiv(width, 8);
    // by the matrix alone, so that its norm is the same to the last bit in any batch
    q.chunks = static_cast<int>(std::max(std::min<int64_t>(cdiv(groups, 1024), 128), std::min<int64_t>(cdiv(groups, 4096), 1216)));
    const int64_t kb_small = cdiv(q.small, kTileK), kb_long = cdiv(std::max(lines, width), kTileK);
    q.gram = shape_for(q.small, q.small, true, !q.wide, batch, kb_long, q.planes, sms);
    q.square = shape_for(q.small, q.small, true, false, batch, kb_small, q.planes, sms);
    q.apply = shape_for(lines, width, false, q.wide, batch, kb_small, q.planes, sms);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t r = at;
        at += up(bytes, 256);
        return r;
    };
    q.gave_up = take(4);
    q.sums = take(batch * q.chunks * 8);
    for (int64_t &x : q.x) x = take(2 * batch * lines * q.ldx * 2);
    q.a = take(q.planes * batch * q.small * q.lda * 2);
    q.b = take(q.planes * batch * q.small * q.lda * 2);
    q.bytes = at;
    return q;
}

// ------------------------------------------------------------------ launches

// Bytes of B whose tiles are worked on together. 4096 x 8192 and 8192 x 4096 bf16 at 8, 16 and 32 MB: 1868 and 1853,
// 1812 and 1820, 1810 and 1838 us (1735 to 1795 at 16 since whole warps issue products and copies).
constexpr int64_t kGroupBytes = int64_t(16) << 20;
// K is added in tensor memory over so many 64-deep steps at a time: two planes as in the cross entropy's f32
// products, one plane (whose results are rounded to 11 bits, or added to a X) without end.
constexpr int kChunkTwo = 2, kChunkOne = 1 << 20;

struct Call {
    const void *G;
    int64_t ldg, stride_g;
    void *X;
    int64_t ldx, stride_x;
    int steps;
    const double *coefficients;
    char *ws;
    int sms;
    cudaStream_t s;
};

#define BL_TRY(call)                                                                                  \
    do {                                                                                              \
        const cudaError_t e_ = (call);                                                                \
        if (e_ != cudaSuccess) return fail(BL_ERR_CUDA, "orth: %s", cudaGetErrorString(e_));          \
    } while (0)
#define BL_MAP(call)                                                                                  \
    do {                                                                                              \
        if (!(call)) return fail(BL_ERR_CUDA, "orth: cannot encode a tensor map");                    \
    } while (0)

template <typename T>
bl_status run(const Plan &q, const Call &c) {
    constexpr int PLANES = sizeof(T) == 4 ? 2 : 1;
    const auto product = PLANES == 1 ? launch_one : launch_two;
    int32_t *const gave_up = reinterpret_cast<int32_t *>(c.ws + q.gave_up);
    Source src{c.G, c.ldg, c.stride_g, static_cast<uint32_t>(q.lines), static_cast<uint32_t>(q.width),
               static_cast<uint32_t>(cdiv(q.width, 8)), q.chunks, 0, reinterpret_cast<double *>(c.ws + q.sums)};
    src.vec = for_tma(c.G, c.ldg, sizeof(T)) && (q.batch == 1 || c.stride_g * static_cast<int64_t>(sizeof(T)) % 16 == 0);
    const unsigned blocks = static_cast<unsigned>(q.batch * q.chunks);
    const int64_t plane_x = q.batch * q.lines * q.ldx;
    // tiles of B's side whose operands are kGroupBytes at most
    const int64_t tile_bytes = (q.wide ? q.apply.ctas * kTileM : q.apply.tile_n) * q.small * 2 * PLANES;
    const int group = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kGroupBytes / tile_bytes, 1 << 16)));
    BL_TRY(launch_pdl(sums_kernel<T>, blocks, 256, 0, c.s, src, gave_up));
    BL_TRY(launch_pdl(begin_kernel<T>, blocks, 256, 0, c.s, src, reinterpret_cast<__half *>(c.ws + q.x[0]), q.ldx, plane_x));
    const float a = static_cast<float>(c.coefficients[0]), b = static_cast<float>(c.coefficients[1]), cc = static_cast<float>(c.coefficients[2]);

    // maps: operands in lines of 128 bytes; results, and what products are added to, in lines of UNIT columns
    const auto map_f16 = [&](CUtensorMap *m, int64_t at, int64_t inner, int64_t rows, int64_t planes, int64_t ld, int box_rows, int line) {
        return make_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, c.ws + at, inner, rows, planes * q.batch, ld, rows * ld, box_rows, line);
    };
    const auto operand = [&](CUtensorMap *m, const Plan &p, bool is_x, int which, bool mn, int box_rows) {
        return is_x ? map_f16(m, p.x[which], p.width, p.lines, 2, p.ldx, mn ? kTileK : box_rows, 128)
                    : map_f16(m, which == 0 ? p.a : p.b, p.small, p.small, PLANES, p.lda, mn ? kTileK : box_rows, 128);
    };
    CUtensorMap a_out, b_out, x_out[2], user_out{};
    constexpr int LINE = Ring<PLANES, 1>::kUnit * 2;
    BL_MAP(map_f16(&a_out, q.a, q.small, q.small, PLANES, q.lda, 32, LINE));
    BL_MAP(map_f16(&b_out, q.b, q.small, q.small, PLANES, q.lda, 32, LINE));
    for (int i = 0; i < 2; ++i) BL_MAP(map_f16(&x_out[i], q.x[i], q.width, q.lines, 2, q.ldx, 32, LINE));
    // A tensor map's items are whole lines apart, as many as an item has or more: items in each other's gaps, or at other
    // distances, are stored without TMA (12 x 1024 x 4096 bf16 945 us, by TMA 911, with a line between items 928).
    const int64_t line_x = q.lines == 1 && q.batch > 1 ? c.stride_x : c.ldx, item_x = q.batch == 1 ? line_x * q.lines : c.stride_x;
    const bool by_tma = for_tma(c.X, line_x, sizeof(T)) && item_x % line_x == 0 && item_x / line_x >= q.lines;
    if (by_tma)
        BL_MAP(make_map(&user_out, PLANES == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, sizeof(T), c.X, q.width,
                        q.lines, q.batch, line_x, item_x, 32));

    const auto args = [&](const Shape &s, int64_t rows, int64_t cols, int64_t k) {
        Args r{};
        r.batch = static_cast<int>(q.batch);
        r.rows = static_cast<int>(rows), r.cols = static_cast<int>(cols);
        r.kblocks = static_cast<int>(cdiv(k, kTileK));
        r.chunk = PLANES == 1 ? kChunkOne : kChunkTwo;
        r.tile_n = s.tile_n, r.tiles_m = s.tiles_m, r.tiles_n = s.tiles_n;
        r.per_item = s.per_item, r.total = static_cast<int>(q.batch * s.per_item);
        r.stages = stages_of<PLANES>(s);
        r.gave_up = gave_up;
        return r;
    };
    CUtensorMap sq_a, sq_b, ap_s;
    BL_MAP(operand(&sq_a, q, false, 0, false, kTileM));
    BL_MAP(operand(&sq_b, q, false, 0, false, q.square.tile_n / q.square.ctas));
    BL_MAP(operand(&ap_s, q, false, 1, false, q.wide ? kTileM : q.apply.tile_n / q.apply.ctas));
    Args gram = args(q.gram, q.small, q.small, std::max(q.lines, q.width));
    gram.alpha = kScaleA / (kScaleX * kScaleX);
    Args square = args(q.square, q.small, q.small, q.small);
    square.alpha = cc / kScaleA, square.beta = b;
    gram.result = reinterpret_cast<__half *>(c.ws + q.a), square.result = reinterpret_cast<__half *>(c.ws + q.b);
    gram.result_ld = square.result_ld = q.lda;
    for (int step = 0; step < c.steps; ++step) {
        const int from = step & 1;
        CUtensorMap x_gram_a, x_gram_b, x_apply;
        BL_MAP(operand(&x_gram_a, q, true, from, !q.wide, kTileM));
        BL_MAP(operand(&x_gram_b, q, true, from, !q.wide, q.gram.tile_n / q.gram.ctas));
        BL_MAP(operand(&x_apply, q, true, from, q.wide, kTileM));
        BL_TRY(product(q.wide ? GRAM_LINES : GRAM_WIDTH, q.gram.ctas, x_gram_a, x_gram_b, a_out, a_out, gram, c.sms, c.s));
        BL_TRY(product(SQUARE_A, q.square.ctas, sq_a, sq_b, a_out, b_out, square, c.sms, c.s));
        Args apply = args(q.apply, q.lines, q.width, q.small);
        apply.alpha = 1 / kScaleA, apply.beta = a;
        apply.rows_first = q.wide;
        apply.group = group;
        apply.last = step + 1 == c.steps;
        if (apply.last) {
            apply.alpha /= kScaleX, apply.beta /= kScaleX;
            if (!by_tma) apply.out = c.X;
            apply.ldo = c.ldx, apply.stride_o = c.stride_x;
        }
        const CUtensorMap &to = !apply.last ? x_out[from ^ 1] : by_tma ? user_out : x_out[0];
        if (q.wide) BL_TRY(product(APPLY_LEFT, q.apply.ctas, ap_s, x_apply, x_out[from], to, apply, c.sms, c.s));
        else BL_TRY(product(APPLY_RIGHT, q.apply.ctas, x_apply, ap_s, x_out[from], to, apply, c.sms, c.s));
    }
    if (gave_up_wanted()) BL_TRY(cudaMemsetAsync(gave_up, 1, 4, c.s));
    BL_TRY(launch_pdl(spoil_kernel<T>, static_cast<unsigned>(std::min<int64_t>(c.sms, q.batch * q.lines)), 256, 0, c.s, gave_up,
                      static_cast<T *>(c.X), c.ldx, c.stride_x, q.lines, q.batch * q.lines, q.width));
    return BL_SUCCESS;
}

// ------------------------------------------------------------------ arguments

bl_status check_shape(const char *op, int dtype, int64_t rows, int64_t cols, int64_t batch) {
    if (dtype != BL_F32 && dtype != BL_BF16) return fail(BL_ERR_INVALID_ARGUMENT, "%s: dtype %d is not f32 or bf16", op, dtype);
    if (rows < 1 || rows > (int64_t(1) << 16)) return fail(BL_ERR_INVALID_ARGUMENT, "%s: rows=%lld outside [1, 2^16]", op, (long long)rows);
    if (cols < 1 || cols > (int64_t(1) << 16)) return fail(BL_ERR_INVALID_ARGUMENT, "%s: cols=%lld outside [1, 2^16]", op, (long long)cols);
    if (batch < 1 || batch > (int64_t(1) << 20))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: batch=%lld outside [1, 2^20]", op, (long long)batch);
    if (rows * cols > (int64_t(1) << 40) / batch) return fail(BL_ERR_INVALID_ARGUMENT, "%s: more than 2^40 elements", op);
    return BL_SUCCESS;
}

bl_status check_matrix(const char *name, const void *p, int64_t ld, int64_t stride, int64_t rows, int64_t cols, int64_t batch, int64_t es) {
    if (!p || reinterpret_cast<uintptr_t>(p) % es != 0)
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: %s is NULL or not aligned to its %lld-byte element", name, (long long)es);
    if (cols > 1 && ld < rows)
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: ld of %s is %lld < rows=%lld", name, (long long)ld, (long long)rows);
    if (cols > 1 && ld > (int64_t(1) << 32)) return fail(BL_ERR_INVALID_ARGUMENT, "orth: ld of %s is %lld, too large", name, (long long)ld);
    if (batch > 1 && (stride < 0 || stride > (int64_t(1) << 36)))
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: stride of %s is %lld, negative or too large", name, (long long)stride);
    return BL_SUCCESS;
}

// Whether no two items share an element: one after the other, side by side in the gaps of each other's columns, or wherever
// else no column of the d-th item after one meets any of its own.
bool items_apart(int64_t rows, int64_t cols, int64_t batch, int64_t ld, int64_t stride) {
    const int64_t extent = (cols - 1) * ld + rows;
    if (stride >= extent || (stride >= rows && (batch - 1) * stride + rows <= ld)) return true;
    for (int64_t d = 1; d < batch && d * stride < extent; ++d) {
        const int64_t column = d * stride / ld, past = d * stride - column * ld;      // where that item's first column starts
        if ((column < cols && past < rows) || (column + 1 < cols && ld - past < rows)) return false;
    }
    return true;
}

}  // namespace orth
}  // namespace bl

extern "C" {

int64_t bl_orth_workspace(bl_dtype dtype, int64_t rows, int64_t cols, int64_t batch) {
    using namespace bl::orth;
    bl::clear_error();
    if (check_shape("orth_workspace", dtype, rows, cols, batch) != BL_SUCCESS) return -1;
    const int sms = bl::sm_count();
    if (sms <= 0) {
        bl::fail(BL_ERR_CUDA, "orth_workspace: cannot query the current CUDA device");
        return -1;
    }
    return plan_for(dtype, cols, rows, batch, sms).bytes;
}

bl_status bl_orth(bl_dtype dtype, int64_t rows, int64_t cols, int64_t batch, const void *G, int64_t ldg, int64_t stride_g, void *X,
                  int64_t ldx, int64_t stride_x, int steps, const double *coefficients, void *workspace, int64_t workspace_bytes,
                  bl_stream_t stream) {
    using namespace bl::orth;
    using bl::fail;
    bl::clear_error();
    bl_status st = check_shape("orth", dtype, rows, cols, batch);
    const int64_t es = dtype == BL_F32 ? 4 : 2;
    if (st == BL_SUCCESS) st = check_matrix("G", G, ldg, stride_g, rows, cols, batch, es);
    if (st == BL_SUCCESS) st = check_matrix("X", X, ldx, stride_x, rows, cols, batch, es);
    if (st != BL_SUCCESS) return st;
    if (cols == 1) ldg = ldx = rows;
    if (batch > 1 && !items_apart(rows, cols, batch, ldx, stride_x)) return fail(BL_ERR_INVALID_ARGUMENT, "orth: items of X overlap");
    if (steps < 1 || steps > 64) return fail(BL_ERR_INVALID_ARGUMENT, "orth: steps=%d outside [1, 64]", steps);
    if (!coefficients || !std::isfinite(coefficients[0]) || !std::isfinite(coefficients[1]) || !std::isfinite(coefficients[2]))
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: coefficients are NULL or not finite");
    if (fits_small(cols, rows)) workspace = nullptr, workspace_bytes = 0;          // not looked at
    else if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: workspace is NULL or not 256-byte aligned");
    Call c{G, ldg, stride_g, X, ldx, stride_x, steps, coefficients, static_cast<char *>(workspace), bl::sm_count(),
           reinterpret_cast<cudaStream_t>(stream)};
    if (c.sms <= 0) return fail(BL_ERR_CUDA, "orth: cannot query the current CUDA device");
    const Plan q = plan_for(dtype, cols, rows, batch, c.sms);
    if (workspace_bytes < q.bytes)
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: workspace of %lld bytes is smaller than %lld", (long long)workspace_bytes, (long long)q.bytes);
    const bl::Range ws = bl::range_of(workspace, q.bytes);
    const auto span = [&](const void *p, int64_t ld, int64_t stride) {
        return bl::range_of(p, ((batch > 1 ? (batch - 1) * stride : 0) + (cols - 1) * ld + rows) * es);
    };
    if (bl::meet(ws, span(G, ldg, stride_g)) || bl::meet(ws, span(X, ldx, stride_x)))
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: the workspace overlaps G or X");
    const bool in_place = G == X && (cols == 1 || ldg == ldx) && (batch == 1 || stride_g == stride_x);
    if (!in_place && bl::meet(span(G, ldg, stride_g), span(X, ldx, stride_x)))
        return fail(BL_ERR_INVALID_ARGUMENT, "orth: X overlaps G and is not G");
    if (fits_small(cols, rows)) {
        const cudaError_t e = launch_small(dtype, cols, rows, batch, G, ldg, stride_g, X, ldx, stride_x, steps, coefficients, c.sms, c.s);
        return e == cudaSuccess ? BL_SUCCESS : fail(BL_ERR_CUDA, "orth: %s", cudaGetErrorString(e));
    }
    return dtype == BL_F32 ? run<float>(q, c) : run<__nv_bfloat16>(q, c);
}

}  // extern "C"
