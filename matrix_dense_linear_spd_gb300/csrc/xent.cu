// Softmax cross entropy over a large vocabulary and its gradients, without keeping the logits.
//
//   s_rv = sum_k H_rk W_vk,  lse_r = log sum_v exp s_rv,  loss_r = lse_r - s_r,t(r)
//   P_rv = g_r (exp(s_rv - lse_r) - [v = t(r)]),  dH = P W,  dW = P^T H
//
// The loss is one product over the vocabulary whose tiles leave a maximum and a sum of exponentials
// each. The gradient computes the logits again, piece of the vocabulary by piece: a piece's P (in
// bf16, or as the three bf16 planes of f32) is all that is ever stored of them, and its two
// products follow. The products run in xent_gemm.cuh.
//
// Rows without a target are left out: the rows that count are copied together (their order kept),
// so that the products do not spend time on a prompt's rows, and what stands in the others (NaN
// included) reaches no result. How many they are is known on the device only; the products read it
// there. Up to one tile of rows there is nothing to gain: rows keep their places, and the loss reads
// H itself if TMA can. W is read in place if it is bf16 and its rows start on 16-byte boundaries;
// otherwise each piece is copied (f32: as planes) before its products. The loss of a few rows has a
// kernel of its own (few_kernel), which reads H and W as they are.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "host.h"
#include "pdl.cuh"
#include "xent_gemm.cuh"

namespace bl {
namespace xent {

// ------------------------------------------------------------------ elementwise kernels

__device__ __forceinline__ bool has_target(const int64_t *target, int64_t row, int64_t vocab) {
    return !target || (target[row] >= 0 && target[row] < vocab);
}

// One block: the rows that count, in order; each row's place among them (-1: does not count); how
// many they are, the parts of dH's K axis, and the unit of P (g: or null). The rows that do not count
// get the results they have (loss, lse: or null).
__global__ void __launch_bounds__(1024)
    index_kernel(const int64_t *target, int64_t vocab, int rows, int *order, int *place, int *kept, Cut cut,
                 const float *g, float *unit, float *loss, float *lse) {
    __shared__ int sums[2][32];
    __shared__ float most[32];
    pdl_release();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int before = 0;
    float m = 0.f;
    for (int r0 = 0, turn = 0; r0 < rows; r0 += 1024, turn ^= 1) {
        const int row = r0 + threadIdx.x;
        const bool in = row < rows, counts = in && has_target(target, row, vocab);
        const uint32_t votes = __ballot_sync(0xffffffffu, counts);
        if (lane == 0) sums[turn][warp] = __popc(votes);
        __syncthreads();                    // sums[turn] is written again two rounds, and a barrier, from here
        const int mine = sums[turn][lane];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const int at = before + __shfl_sync(0xffffffffu, upto - mine, warp) + __popc(votes & ((1u << lane) - 1));
        before += __shfl_sync(0xffffffffu, upto, 31);
        if (in) {
            place[row] = counts ? at : -1;
            if (counts && g) m = fmaxf(m, fabsf(g[row]));
            if (counts) order[at] = row;
            else if (loss) loss[row] = lse[row] = 0.f;
        }
    }
    m = warp_max(m);
    if (lane == 0) most[warp] = m;
    __syncthreads();
    if (warp == 0) {
        m = warp_max(most[lane]);
        if (lane == 0) {
            kept[0] = before;
            kept[1] = parts_for(cut, before);
            if (g) *unit = unit_from(m);
        }
    }
}

// Copy rows into bf16 planes of 64-column panels ([plane][panel][height][64]); columns past dim are
// zero. With `order` row j of the copy is row order[j]; whole row tiles are filled, with zeros after
// the last row. Rows without a target (`target` given) become zero too.
struct Copy {
    const void *src;
    int64_t ld, rows;
    int dim;
    const int64_t *target;
    int64_t vocab;
    const int *order, *kept;
    int tile;
    __nv_bfloat16 *dst;
    int panels;
    int64_t height;
    int vec, blocks;
    const float *g;           // of the gradient's rows in their places: the unit of P is found on the way
    float *unit;
};
// Two copies in one launch, H's and the first piece's of W (either may be without blocks).
template <typename T, int PLANES>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ Copy one, const __grid_constant__ Copy two) {
    pdl_release();
    pdl_wait();
    const bool second = static_cast<int>(blockIdx.x) >= one.blocks;
    const int block = second ? blockIdx.x - one.blocks : blockIdx.x;
    const Copy &w = second ? two : one;
    if (w.g && block == 0 && threadIdx.x < 32) {
        const float u = unit_of_rows(w.g, w.target, w.vocab, static_cast<int>(w.rows));
        if (threadIdx.x == 0) *w.unit = u;
    }
    const int64_t count = w.kept ? *w.kept : w.rows, filled = max((count + w.tile - 1) / w.tile, int64_t(1)) * w.tile;
    const int64_t per_row = w.panels * 8, all = filled * per_row, plane = w.panels * w.height * 64;
    for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < all;
         i += static_cast<int64_t>(w.blocks) * 256) {
        const int64_t j = i / per_row;
        const int c = static_cast<int>(i - j * per_row) * 8;
        const int64_t row = j >= count ? -1 : w.order ? w.order[j] : j;
        const T *const s = static_cast<const T *>(w.src) + row * w.ld + c;
        __align__(16) T x[8];
        if (row < 0 || (w.target && !has_target(w.target, row, w.vocab))) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = T(0.f);
        } else if (w.vec && c + 8 <= w.dim) {
#pragma unroll
            for (int e = 0; e < static_cast<int>(sizeof(x) / 16); ++e)
                reinterpret_cast<uint4 *>(x)[e] = reinterpret_cast<const uint4 *>(s)[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = c + e < w.dim ? s[e] : T(0.f);
        }
        __nv_bfloat16 *const d = w.dst + ((c >> 6) * w.height + j) * 64 + (c & 63);
        if constexpr (PLANES == 1) {
            *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(x);
        } else {
            float p[3][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split3(x[e], p[0][e], p[1][e], p[2][e]);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                *reinterpret_cast<uint4 *>(d + q * plane) = make_uint4(bf16x2(p[q][0], p[q][1]), bf16x2(p[q][2], p[q][3]),
                                                                       bf16x2(p[q][4], p[q][5]), bf16x2(p[q][6], p[q][7]));
        }
    }
}

// Whether any CTA of the call's products gave up: this thread's share of the flags.
__device__ __forceinline__ int flags_seen(const int32_t *flags, int count) {
    int bad = 0;
    for (int i = threadIdx.x; i < count; i += blockDim.x) bad |= flags[i];
    return bad;
}

// One warp a row: join the tiles' maxima and sums. A product that gave up makes every loss NaN.
// Latency is all there is to it for few rows, so every load that can be is issued at once.
__global__ void __launch_bounds__(256)
    loss_kernel(const float2 *part, int64_t part_ld, const float *picked, const int64_t *target, int64_t vocab, int rows,
                const int *order, const int *kept, const int32_t *flags, int flag_count, float *loss, float *lse) {
    constexpr int HELD = 8;
    pdl_release();
    pdl_wait();
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const bool in = j < rows;                       // rows past the last that counts hold anything and are dropped below
    const float2 *const p = part + (in ? j : 0) * part_ld;
    float2 v[HELD];
#pragma unroll
    for (int h = 0; h < HELD; ++h) v[h] = lane + 32 * h < part_ld ? p[lane + 32 * h] : make_float2(-INFINITY, 0.f);
    const float chosen = in ? picked[j] : 0.f;
    const int count = kept ? *kept : rows, row = in ? (order ? order[j] : j) : 0;
    const bool bad = __syncthreads_or(flags_seen(flags, flag_count)) != 0;
    if (j >= count) return;
    float l = 0.f, s = 0.f;
    if (has_target(target, row, vocab)) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int h = 0; h < HELD; ++h) top = fmaxf(top, v[h].x);
        for (int64_t i = lane + 32 * HELD; i < part_ld; i += 32) top = fmaxf(top, p[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int h = 0; h < HELD; ++h) sum += v[h].y * expf(v[h].x - ref);
        for (int64_t i = lane + 32 * HELD; i < part_ld; i += 32) sum += p[i].y * expf(p[i].x - ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        // not s - chosen: s has been rounded, by up to |s| 2^-24, and a sure row's loss is less than that. Both
        // terms are exact or small, and neither is negative.
        s = ref + logf(sum);
        l = (ref - chosen) + logf(sum);
    }
    if (bad) l = s = NAN;
    if (lane == 0) {
        loss[row] = l;
        lse[row] = s;
    }
}

// The loss of a few rows (a token or a handful): too few for a tile, so each W row meets all of them
// while it is in registers, in f32 multiply-adds. HBM bandwidth bounds it up to four rows (one row,
// dim 4096, vocabulary 131072: bf16 153 us, 7.0 TB/s; f32 296 us, 7.2 TB/s), the multiply-adds and
// shared-memory reads of H above. A warp takes four vocabulary entries
// at a time, its lanes share K; H waits in shared memory as f32. Each CTA leaves one maximum and sum
// a row. W is read in place whatever its type: no planes, no copies.
template <typename T, bool VEC>
struct FewVec {                                    // rows that start anywhere: value by value
    static constexpr int N = 1;
    __device__ static void load(const T *p, float (&v)[1]) { v[0] = static_cast<float>(__ldcs(p)); }
};
template <>
struct FewVec<float, true> {
    static constexpr int N = 4;
    __device__ static void load(const float *p, float (&v)[4]) {
        const float4 q = __ldcs(reinterpret_cast<const float4 *>(p));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    }
};
template <>
struct FewVec<__nv_bfloat16, true> {
    static constexpr int N = 8;
    __device__ static void load(const __nv_bfloat16 *p, float (&v)[8]) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {              // bf16 is the upper half of an f32
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
// Entries a warp takes at a time, steps of K in flight for each, and CTAs per SM
constexpr int few_entries(int R) { return R == 1 ? 2 : 4; }
constexpr int few_ahead(int R, bool vec) { return (R == 1 ? 4 : 2) * (vec ? 1 : 2); }
constexpr int few_ctas(int R) { return R == 1 ? 4 : R == 4 ? 2 : 1; }
constexpr int few_smem(int R) { return 200 * 1024 / few_ctas(R); }      // H's share of the SM's shared memory

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(256, few_ctas(R))
    few_kernel(const T *H, int64_t ldh, int rows, int dim, const T *W, int64_t ldw, int vocab, const int64_t *target,
               float2 *part, int64_t part_ld, float *picked) {
    constexpr int N = FewVec<T, VEC>::N, E = few_entries(R), AHEAD = few_ahead(R, VEC);
    extern __shared__ __align__(16) float few_h[];           // [R][dim]
    __shared__ float2 joined[8][R];
    pdl_release();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < R * dim; i += 256) {
        const int r = i / dim, k = i - r * dim;
        few_h[i] = r < rows ? static_cast<float>(H[r * ldh + k]) : 0.f;
    }
    int64_t at[R];
    float top[R], sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        at[r] = r < rows ? target[r] : -1;
        top[r] = -INFINITY;
        sum[r] = 0.f;
    }
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * E;
    for (int64_t v0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * E; v0 < vocab; v0 += step) {
        float acc[E][R];
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[e][r] = 0.f;
        const T *w[E];                                       // past the last entry: the last one again, dropped below
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = W + min(v0 + e, static_cast<int64_t>(vocab) - 1) * ldw;
#pragma unroll AHEAD
        for (int k = lane * N; k < dim; k += 32 * N) {
            float x[E][N];
#pragma unroll
            for (int e = 0; e < E; ++e) FewVec<T, VEC>::load(w[e] + k, x[e]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float *const h = few_h + r * dim + k;
                float y[N];
                if constexpr (VEC) {
#pragma unroll
                    for (int q = 0; q < N; q += 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(h + q);
                        y[q] = t.x, y[q + 1] = t.y, y[q + 2] = t.z, y[q + 3] = t.w;
                    }
                } else {
                    y[0] = h[0];
                }
#pragma unroll
                for (int q = 0; q < N; ++q)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e][r] = fmaf(x[e][q], y[q], acc[e][r]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float s = acc[e][r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                acc[e][r] = v0 + e < vocab ? s : -INFINITY;
                if (lane == 0 && v0 + e == at[r] && at[r] < vocab) picked[r] = s;
            }
            float m = top[r];
#pragma unroll
            for (int e = 0; e < E; ++e) m = fmaxf(m, acc[e][r]);
            const float ref = m == -INFINITY ? 0.f : m;
            float t = sum[r] * expf(top[r] - ref);
#pragma unroll
            for (int e = 0; e < E; ++e) t += expf(acc[e][r] - ref);
            sum[r] = t;
            top[r] = m;
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) joined[warp][r] = make_float2(top[r], sum[r]);
    }
    __syncthreads();
    if (threadIdx.x < rows) {
        float m = -INFINITY, t = 0.f;
        for (int q = 0; q < 8; ++q) m = fmaxf(m, joined[q][threadIdx.x].x);
        const float ref = m == -INFINITY ? 0.f : m;
        for (int q = 0; q < 8; ++q) t += joined[q][threadIdx.x].y * expf(joined[q][threadIdx.x].x - ref);
        part[threadIdx.x * part_ld + blockIdx.x] = make_float2(m, t);
    }
}

__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
}

// What the gradient writes where a product gave up: NaN over all of dW (dw null: none is wanted).
template <typename T>
struct Spoiled {
    T *dw;
    int64_t ld, rows;
    int dim;
    __device__ void fill() const {
        if (!dw) return;
        for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
            for (int c = threadIdx.x; c < dim; c += blockDim.x) put(dw + r * ld + c, NAN);
    }
};
// The last kernel of a gradient without dH: all that is left to do is to look at the flags.
template <typename T>
__global__ void __launch_bounds__(256) spoil_kernel(const int32_t *flags, int flag_count, const Spoiled<T> dw) {
    pdl_release();
    pdl_wait();
    if (__syncthreads_or(flags_seen(flags, flag_count))) dw.fill();
}

// dH from the parts' sums, four columns a thread, times the unit of P; rows without a target are zero. A product that
// gave up makes it NaN, and dW. With SHARE = 8 eight lanes of a warp add every eighth part each (many parts
// mean few results: 64 rows x 1024 in 38 parts took 14 us with one thread a result).
template <typename T, int SHARE>
__global__ void __launch_bounds__(256)
    dh_kernel(const float *part, int all_parts, int64_t rows, int64_t ldo, int dim, const int64_t *target, int64_t vocab,
              const int *place, const int *kept_rows, const float *unit_of_p, const int32_t *flags, int flag_count,
              T *dh, int64_t ld, int vec, const Spoiled<T> dw) {
    constexpr int SIDE = 32 / SHARE;                // results that a warp works on at once
    pdl_release();
    pdl_wait();
    const bool bad = __syncthreads_or(flags_seen(flags, flag_count)) != 0;
    if (bad) dw.fill();
    const int kept = kept_rows ? kept_rows[0] : static_cast<int>(rows), splits = kept_rows ? kept_rows[1] : all_parts;
    const float unit = *unit_of_p;
    const int64_t height = part_rows(kept), part_step = SHARE * height * (ldo / 4);
    const int lane = threadIdx.x & 31, mine = SHARE == 1 ? 0 : lane / SIDE;
    const int64_t per_row = (dim + 3) / 4, all = rows * per_row, step = static_cast<int64_t>(gridDim.x) * 256 / SHARE;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * 256 + (threadIdx.x & ~31)) / SHARE;
    for (int64_t i0 = first; i0 < all; i0 += step) {        // the warp's first result: all lanes stay together
        const int64_t i = i0 + lane % SIDE;
        const int64_t row = i < all ? i / per_row : 0;
        const int c = i < all ? static_cast<int>(i - row * per_row) * 4 : 0;
        const int64_t j = i >= all ? -1 : place ? place[row] : has_target(target, row, vocab) ? row : -1;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j >= 0) {
            const float4 *p = reinterpret_cast<const float4 *>(part + (mine * height + j) * ldo + c);
#pragma unroll 4
            for (int s = mine; s < splits; s += SHARE, p += part_step) {
                const float4 x = *p;
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
        }
#pragma unroll
        for (int o = SIDE; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
        }
        v.x *= unit, v.y *= unit, v.z *= unit, v.w *= unit;
        if (bad) v = make_float4(NAN, NAN, NAN, NAN);
        if (i >= all || mine != 0) continue;
        T *const d = dh + row * ld + c;
        if (vec && c + 4 <= dim) {
            put4(d, v);
        } else {
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < dim) put(d + e, x[e]);
        }
    }
}

// ------------------------------------------------------------------ plan

// K is added in tensor memory over so many 64-deep steps at a time where the result is f32: f32 operands, the
// logits of bf16 operands, and those of P where the loss of few rows has added them in f32 (W's way from memory
// hides it: step of 1 row x 4096 x 32000 216 us, 212 with the chain uncut). bf16 results, dH and dW, have long chunks.
constexpr int kChunkF32 = 2, kChunkLoss = 16, kChunkFew = 1, kChunkBf16 = 256;
// Bytes of P, and of a piece's copy of W, that a piece of the vocabulary may take (4096 entries may take more: 8 KB of P
// a row in bf16, 24 KB in f32). Steps of 4096 x 4096 x
// 131072 in bf16 and 1024 x 1024 x 32000 in f32 at 64, 128, 512 and 2048 MB: 11.04, 10.84, 10.66, 10.65 ms
// and 1.22, 1.13, 1.04, 1.04 ms
constexpr int64_t kPieceBytes = int64_t(512) << 20;

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t cdiv(int64_t v, int64_t by) { return (v + by - 1) / by; }

// P of bf16 operands takes two planes up to so many rows, so that a sum over few of them does not show its
// rounding: errors of dH and dW against 64 bits, in units of those with P in f32, over sizes and seeds, at worst: 1
// row 1.6 and 2.0, 2 rows 1.4 and 1.7, 5 and 8 rows 1.5, 16 rows 1.25, 64 rows and more 1.3 (1.2 on average). The
// second plane costs what the doubled products do not hide behind W's way from memory: step of 8 rows x 1024 x 32000
// 80 us instead of 71, of 32 rows x 4096 x 32000 223 instead of 207.
constexpr int kTwoPlaneRows = 16;

struct Plan {
    int planes, pairs;
    int p_planes;             // of P
    int ctas;                 // that share a tile
    int groups;               // CTAs or pairs that the device's SMs hold
    bool copy_h, copy_w, compact, grad;
    int few;                  // rows of the kernel for few rows (0: the tiled products)
    bool few_loss;            // the gradient's lse comes from that kernel
    int64_t rows, dim, vocab;
    int64_t tiled;            // rows of the copy of H and of P: whole tiles
    int64_t seen;             // of them, those that tensor maps see: the rest reads as zero without being read
    int64_t panels;           // of 64 columns in the copies of H and W
    int64_t piece, pieces;    // vocabulary entries per piece
    int wide, tile_n;         // columns of a tile, at most; of a tile of logits
    int64_t part_ld;          // partial maxima and sums of a row: two per tile
    int parts;                // of dH's K axis if every row counts
    int first_kb;             // 64-deep steps of the first piece
    int64_t slab_rows;        // of dH's partial sums, all parts together
    int64_t ldo;              // row length of dH's partial sums
    int64_t flags, kept, unit, order, place, h, w, part, picked, p, dh, bytes;   // offsets into the workspace
};

bool for_tma(const void *p, int64_t ld, int64_t elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0;
}

// The rows that the kernel for few rows takes (1, 4 or 8), or 0 where the tiled products are used:
// where there are too many rows, or H does not fit shared memory. Measured, loss over a vocabulary of
// 32000, this kernel against the tiles: dim 1024, bf16 1 row 15.7 us against 19.5, 2 rows 22 against 19.6;
// f32 1, 4, 8 rows 25.5, 29.5, 45 us against 106 (the tiles' copies of W); dim 1021, whose rows start off the
// vectors and which the tiles copy, bf16 1, 4, 8 rows 29, 37, 64 us against 43, f32 35, 42, 69 against 116. (Of a W
// far larger than L2 only one row was measured: dim 4096, vocabulary 131072, bf16 153 us against 216.)
bool few_vec(const void *W, int64_t ldw, int64_t dim, int64_t elem) { return for_tma(W, ldw, elem) && dim * elem % 16 == 0; }
int few_rows(int dtype, int64_t rows, int64_t dim, const void *W, int64_t ldw) {
    const bool vec = few_vec(W, ldw, dim, dtype == BL_F32 ? 4 : 2);
    if (rows > (dtype == BL_F32 ? 8 : vec ? 1 : 4)) return 0;
    const int r = rows <= 1 ? 1 : rows <= 4 ? 4 : 8;
    return r * dim * 4 <= few_smem(r) ? r : 0;
}

Plan plan_for(int dtype, const void *H, int64_t ldh, int64_t rows, int64_t dim, int64_t vocab, const void *W, int64_t ldw,
              bool grad, int sms) {
    Plan q{};
    q.planes = dtype == BL_F32 ? 3 : 1;
    q.pairs = dtype == BL_F32 ? 6 : 1;
    q.p_planes = dtype == BL_F32 ? 3 : rows <= kTwoPlaneRows ? 2 : 1;
    q.compact = rows > kTileM;
    // pairs of CTAs above one row tile: steps at dim 1024, vocabulary 32000 on single CTAs against pairs: bf16
    // 64 rows 75 us, 93; 128 rows 78, 93; 200 rows 111, 108; f32 64 rows 319, 358; 200 rows 467, 398
    q.ctas = rows > kTileM ? 2 : 1;
    q.groups = std::max(1, sms / q.ctas);
    q.wide = q.ctas == 1 && q.planes == 3 ? Ring<1, 3, 3>::kTile : kTileN;
    // a row without a target may hold anything: only the loss of uncopied rows ignores it
    q.copy_h = dtype == BL_F32 || grad || q.compact || !for_tma(H, ldh, 2);
    q.copy_w = dtype == BL_F32 || !for_tma(W, ldw, 2);
    q.grad = grad;
    q.rows = rows;
    q.dim = dim;
    q.vocab = vocab;
    q.tiled = up(rows, q.ctas * kTileM);
    q.seen = q.compact ? q.tiled : rows;
    q.panels = cdiv(dim, 64);
    // a piece: what keeps P and the copy of W within their size, but 4096 entries at least, so
    // that a piece's products fill the GPU; pieces of one size
    int64_t most = up(vocab, kTileN);
    if (grad) most = std::min(most, kPieceBytes / (q.tiled * 2 * q.p_planes));
    if (q.copy_w) most = std::min(most, kPieceBytes / (q.panels * 128 * q.planes));
    most = std::max<int64_t>(most / kTileN * kTileN, 4096);
    q.pieces = cdiv(vocab, most);
    q.piece = up(cdiv(vocab, q.pieces), kTileN);
    q.pieces = cdiv(vocab, q.piece);
    // tiles of logits: the width that takes the least time in rounds of all SMs, when a tile takes as
    // long as its width plus 64 columns (f32 loss, 77 rows, vocabulary 5003: 20 tiles of 256, 79 of 64)
    q.tile_n = q.wide;
    const int64_t groups = q.groups, tall = cdiv(rows, q.ctas * kTileM);
    int64_t least = 0;
    for (int t = q.wide; t >= 64; t /= 2) {
        const int64_t cost = cdiv(tall * cdiv(std::min(q.piece, vocab), t), groups) * (t + 64);
        if (t == q.wide || cost < least) q.tile_n = t, least = cost;
    }
    q.part_ld = 2 * cdiv(vocab, q.tile_n);
    const int few = few_rows(dtype, rows, dim, W, ldw);
    q.few_loss = grad && few;
    if (!grad) {
        q.few = few;
        if (q.few) {
            q.part_ld = std::min<int64_t>(cdiv(vocab, 8 * few_entries(q.few)), static_cast<int64_t>(sms) * few_ctas(q.few));
            q.copy_h = q.copy_w = false;
            q.pieces = 1;
            q.piece = up(vocab, kTileN);
        }
    }
    q.ldo = up(dim, 32);
    // dH's partial sums: room for as many parts as are wanted if every row counts, and up to six (256 MB)
    // for the case that few do
    q.first_kb = static_cast<int>(cdiv(std::min(q.piece, vocab), kTileK));
    const int64_t high = part_rows(static_cast<int>(rows));
    const Cut roomy{q.ctas, static_cast<int>(dim), q.wide, q.first_kb, q.pairs, static_cast<int>(std::min<int64_t>(1 << 28, high * 1024)), q.groups};
    q.parts = parts_for(roomy, static_cast<int>(rows));
    const int64_t spare = q.compact ? std::min<int64_t>(6, (int64_t(256) << 20) / (high * q.ldo * 4)) : 1;
    q.slab_rows = high * std::max<int64_t>(q.parts, spare);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t r = at;
        at += up(bytes, 256);
        return r;
    };
    q.flags = take(q.pieces * 3 * sms * 4);
    q.kept = take(8);
    q.unit = take(4);
    if (q.compact) {
        q.order = take(rows * 4);
        q.place = take(rows * 4);
    }
    if (q.copy_h) q.h = take(q.planes * q.tiled * q.panels * 128);
    if (q.copy_w) q.w = take(q.planes * std::min(q.piece, vocab) * q.panels * 128);
    if (!grad) {
        q.part = take(rows * q.part_ld * 8);
        q.picked = take(rows * 4);
    } else {
        q.p = take(q.p_planes * q.tiled * q.piece * 2);
        q.dh = take(q.slab_rows * q.ldo * 4);
    }
    q.bytes = at;
    return q;
}

// ------------------------------------------------------------------ launches

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess)
            return EncodeFn(nullptr);
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Planes of rows x inner values, copied in boxes of box_rows lines of line_bytes (128 or 64, the
// swizzle's width too); what lies outside reads as zero and is not written. Planes are `plane`
// values apart; with one plane any multiple of 16 bytes will do.
bool make_map(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *base, int64_t inner, int64_t rows, int64_t planes,
              int64_t ld, int64_t plane, int box_rows, int line_bytes = 128) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * elem), static_cast<cuuint64_t>(plane * elem)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(line_bytes / elem), static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
    return fn(map, type, 3, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              line_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_bf16(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t planes, int64_t ld, int64_t plane,
              int box_rows, int line_bytes = 128) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, inner, rows, planes, ld, plane, box_rows, line_bytes);
}
// The first `rows` rows of 64-column panels of `height` rows.
bool map_panels(CUtensorMap *map, const void *base, int64_t rows, int64_t height, int64_t panels, int box_rows,
                int line_bytes = 128) {
    return map_bf16(map, base, 64, rows, panels, 64, height * 64, box_rows, line_bytes);
}
bool map_f32(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t planes, int64_t ld, int64_t plane) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, inner, rows, planes, ld, plane, 32);
}

// Launch a product; its CTAs' flags follow those of the call's earlier products.
template <int MODE, int PLANES, int CTAS>
cudaError_t launch_tiles(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, GemmArgs &a, int &flags, int sms,
                         cudaStream_t s) {
    constexpr int kSmem = RingOf<MODE, PLANES, CTAS>::kSmem;
    const auto kernel = gemm_kernel<MODE, PLANES, CTAS>;
    static std::atomic<int> groups[64];         // CTAs, or pairs of CTAs, that the device runs at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int most = dev < 64 ? groups[dev].load(std::memory_order_acquire) : 0;
    if (most == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        most = sms;
        if constexpr (CTAS > 1) {
            cudaLaunchConfig_t c{};
            c.gridDim = dim3(sms / CTAS * CTAS);
            c.blockDim = dim3(kThreads);
            c.dynamicSmemBytes = kSmem;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = CTAS;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            c.attrs = &at;
            c.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&most, kernel, &c);
            if (e != cudaSuccess) return e;
            most = std::max(1, std::min(most, sms / CTAS));
        }
        if (dev < 64) groups[dev].store(most, std::memory_order_release);
    }
    const int64_t total = cdiv(a.m, CTAS * kTileM) * a.tiles_n;
    const int grid = static_cast<int>(MODE == DH ? most : std::min<int64_t>(total, most)) * CTAS;    // DH is cut to fill the device
    a.flags += flags;
    flags += grid;
    return launch_pdl_cluster(kernel, grid, kThreads, kSmem, CTAS, s, ma, mb, mo, a);
}
template <int MODE, int PLANES>
cudaError_t launch_gemm(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, GemmArgs &a, int ctas, int &flags,
                        int sms, cudaStream_t s) {
    return ctas == 1 ? launch_tiles<MODE, PLANES, 1>(ma, mb, mo, a, flags, sms, s)
                     : launch_tiles<MODE, PLANES, 2>(ma, mb, mo, a, flags, sms, s);
}
// One of the products that make P or take it. Two planes of it only ever meet single CTAs.
template <int MODE, int PLANES>
cudaError_t launch_with_p(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, GemmArgs &a, const Plan &q, int &flags,
                          int sms, cudaStream_t s) {
    if constexpr (PLANES == 1)
        if (q.p_planes == 2) return launch_tiles<MODE, 2, 1>(ma, mb, mo, a, flags, sms, s);
    return launch_gemm<MODE, PLANES>(ma, mb, mo, a, q.ctas, flags, sms, s);
}

// Raise a kernel's dynamic shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (bit & done.load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <typename T>
Copy copy_of(const void *src, int64_t ld, int64_t rows, int64_t dim, const int64_t *target, int64_t vocab, const int *order,
             const int *kept, int tile, void *dst, int64_t height, int sms) {
    Copy w{};
    w.src = src, w.ld = ld, w.rows = rows, w.dim = static_cast<int>(dim);
    w.target = target, w.vocab = vocab, w.order = order, w.kept = kept, w.tile = tile;
    w.dst = static_cast<__nv_bfloat16 *>(dst);
    w.panels = static_cast<int>(cdiv(dim, 64));
    w.height = height;
    w.vec = for_tma(src, ld, sizeof(T));
    w.blocks = static_cast<int>(std::min<int64_t>(cdiv(up(rows, tile) * w.panels * 8, 256), static_cast<int64_t>(sms) * 8));
    return w;
}

thread_local bool t_gave_up = false;       // bl_debug_xent_gave_up

struct Call {
    int64_t rows, dim, vocab;
    const void *H;
    int64_t ldh;
    const void *W;
    int64_t ldw;
    const int64_t *target;
    float *loss, *lse;               // bl_xent
    const float *lse_in, *g;         // bl_xent_grad
    void *dH;
    int64_t lddh;
    void *dW;
    int64_t lddw;
    char *ws;
    int sms;
    cudaStream_t s;
};

#define BL_TRY(call)                                                                                  \
    do {                                                                                              \
        const cudaError_t e_ = (call);                                                                \
        if (e_ != cudaSuccess) return fail(BL_ERR_CUDA, "%s: %s", op, cudaGetErrorString(e_));        \
    } while (0)
#define BL_MAP(call)                                                                                  \
    do {                                                                                              \
        if (!(call)) return fail(BL_ERR_CUDA, "%s: cannot encode a tensor map", op);                  \
    } while (0)

template <typename T, int PLANES>
bl_status run(const char *op, const Plan &q, const Call &c) {
    const int64_t piece_w = std::min(q.piece, c.vocab);
    const int rows = static_cast<int>(c.rows), dim = static_cast<int>(c.dim);
    int *const kept = q.compact ? reinterpret_cast<int *>(c.ws + q.kept) : nullptr;
    int *const order = q.compact ? reinterpret_cast<int *>(c.ws + q.order) : nullptr;
    int *const place = q.compact ? reinterpret_cast<int *>(c.ws + q.place) : nullptr;
    float *const unit = reinterpret_cast<float *>(c.ws + q.unit);
    int32_t *const flags = reinterpret_cast<int32_t *>(c.ws + q.flags);
    int flag_count = 0;
    if (q.compact)
        BL_TRY(launch_pdl(index_kernel, 1, 1024, 0, c.s, c.target, c.vocab, rows, order, place, kept,
                          Cut{q.ctas, dim, q.wide, q.first_kb, q.pairs, static_cast<int>(q.slab_rows), q.groups}, c.g, unit, c.loss, c.lse));
    if (q.few) {
        const bool vec = few_vec(c.W, c.ldw, c.dim, sizeof(T));
        auto kernel = q.few == 1 ? (vec ? few_kernel<T, 1, true> : few_kernel<T, 1, false>) : few_kernel<T, 4, false>;
        if constexpr (PLANES == 3) {
            if (q.few == 4 && vec) kernel = few_kernel<T, 4, true>;
            if (q.few == 8) kernel = vec ? few_kernel<T, 8, true> : few_kernel<T, 8, false>;
        }
        float2 *const part = reinterpret_cast<float2 *>(c.ws + q.part);
        float *const picked = reinterpret_cast<float *>(c.ws + q.picked);
        static std::atomic<unsigned long long> allowed[6];
        BL_TRY(allow_smem(kernel, few_smem(q.few), allowed[q.few / 4 + 3 * vec]));
        BL_TRY(launch_pdl(kernel, static_cast<unsigned>(q.part_ld), 256, static_cast<size_t>(q.few) * c.dim * 4, c.s,
                          static_cast<const T *>(c.H), c.ldh, rows, dim, static_cast<const T *>(c.W), c.ldw,
                          static_cast<int>(c.vocab), c.target, part, q.part_ld, picked));
        BL_TRY(launch_pdl(loss_kernel, 1, 256, 0, c.s, part, q.part_ld, picked, c.target, c.vocab, rows, nullptr, nullptr, flags, 0,
                          c.loss, c.lse));
        return BL_SUCCESS;
    }
    const Columns in_place{64, 0, 1}, in_panels{0, 1, static_cast<int>(q.panels)};
    CUtensorMap h_k;
    Copy copy_h{};
    if (q.copy_h) {
        copy_h = copy_of<T>(c.H, c.ldh, c.rows, c.dim, c.target, c.vocab, order, kept, q.ctas * kTileM, c.ws + q.h, q.tiled, c.sms);
        if (!q.compact) copy_h.g = c.g, copy_h.unit = unit;
        BL_MAP(map_panels(&h_k, c.ws + q.h, q.seen, q.tiled, PLANES * q.panels, kTileM));
    } else {
        BL_MAP(map_bf16(&h_k, c.H, c.dim, c.rows, 1, c.ldh, c.ldh, kTileM));
    }
    GemmArgs base{};
    base.rows = rows;
    base.kept = kept;
    base.order = order;
    base.flags = flags;
    base.chunk = PLANES == 3 ? kChunkF32 : kChunkBf16;
    base.target = c.target;
    base.vocab = c.vocab;
    base.g = c.g;
    base.unit = unit;
    for (int64_t i = 0; i < q.pieces; ++i) {
        const int64_t v0 = i * q.piece, n = std::min(q.piece, c.vocab - v0);
        const char *const w_at = static_cast<const char *>(c.W) + v0 * c.ldw * static_cast<int64_t>(sizeof(T));
        CUtensorMap w_k, w_mn;
        Copy copy_w{};
        if (q.copy_w)
            copy_w = copy_of<T>(w_at, c.ldw, n, c.dim, nullptr, 0, nullptr, nullptr, 1, c.ws + q.w, piece_w, c.sms);
        if (i > 0) copy_h.blocks = 0;
        if (copy_h.blocks + copy_w.blocks > 0)
            BL_TRY(launch_pdl(pack_kernel<T, PLANES>, copy_h.blocks + copy_w.blocks, 256, 0, c.s, copy_h, copy_w));
        if (q.copy_w) {
            BL_MAP(map_panels(&w_k, c.ws + q.w, n, piece_w, PLANES * q.panels, q.tile_n / q.ctas));
            BL_MAP(map_panels(&w_mn, c.ws + q.w, n, piece_w, PLANES * q.panels, kTileK));
        } else {
            BL_MAP(map_bf16(&w_k, w_at, c.dim, n, 1, c.ldw, c.ldw, q.tile_n / q.ctas));
            BL_MAP(map_bf16(&w_mn, w_at, c.dim, n, 1, c.ldw, c.ldw, kTileK));
        }
        const Columns cols_h = q.copy_h ? in_panels : in_place, cols_w = q.copy_w ? in_panels : in_place;
        GemmArgs a = base;
        a.m = rows;
        a.n = static_cast<int>(n);
        a.kblocks = static_cast<int>(cdiv(c.dim, kTileK));
        a.tile_n = q.tile_n;
        a.tiles_n = static_cast<int>(cdiv(n, q.tile_n));
        a.v0 = static_cast<int>(v0);
        a.ca = cols_h;
        a.cb = cols_w;
        if (PLANES == 1) a.chunk = q.few_loss ? kChunkFew : kChunkLoss;
        if (!q.grad) {
            a.part = reinterpret_cast<float2 *>(c.ws + q.part) + 2 * (v0 / q.tile_n);
            a.part_ld = q.part_ld;
            a.picked = reinterpret_cast<float *>(c.ws + q.picked);
            BL_TRY((launch_gemm<LOGITS, PLANES>(h_k, w_k, w_k, a, q.ctas, flag_count, c.sms, c.s)));
            continue;
        }
        char *const pp = c.ws + q.p;
        const int64_t p_panels = cdiv(n, 64);
        const Columns cols_p{0, 1, static_cast<int>(p_panels)};
        CUtensorMap p_out;
        BL_MAP(map_panels(&p_out, pp, q.seen, q.tiled, q.p_planes * p_panels, 32, q.p_planes == 1 ? 128 : 64));
        a.p_panels = static_cast<int>(p_panels);
        a.lse = c.lse_in;
        BL_TRY((launch_with_p<PROBS, PLANES>(h_k, w_k, p_out, a, q, flag_count, c.sms, c.s)));
        if (c.dH) {
            CUtensorMap p_k, sums;
            BL_MAP(map_panels(&p_k, pp, q.seen, q.tiled, q.p_planes * p_panels, kTileM));
            BL_MAP(map_f32(&sums, c.ws + q.dh, c.dim, q.slab_rows, 1, q.ldo, q.ldo));
            GemmArgs d = base;
            d.m = rows;
            d.n = dim;
            d.kblocks = static_cast<int>(cdiv(n, kTileK));
            d.parts = q.parts;
            d.tile_n = q.wide;
            d.tiles_n = static_cast<int>(cdiv(c.dim, q.wide));
            d.accumulate = i > 0;
            d.ca = cols_p;
            d.cb = cols_w;
            BL_TRY((launch_with_p<DH, PLANES>(p_k, w_mn, sums, d, q, flag_count, c.sms, c.s)));
        }
        if (c.dW) {
            CUtensorMap p_mn, h_mn, to;
            BL_MAP(map_panels(&p_mn, pp, q.seen, q.tiled, q.p_planes * p_panels, kTileK));
            BL_MAP(map_panels(&h_mn, c.ws + q.h, q.seen, q.tiled, PLANES * q.panels, kTileK));      // the gradient always copies H
            GemmArgs d = base;
            d.m = static_cast<int>(n);
            d.n = dim;
            d.tile_n = q.wide;
            d.tiles_n = static_cast<int>(cdiv(c.dim, q.wide));
            d.ca = cols_p;
            d.cb = in_panels;
            char *const out = static_cast<char *>(c.dW) + v0 * c.lddw * static_cast<int64_t>(sizeof(T));
            if (!for_tma(c.dW, c.lddw, sizeof(T))) {
                d.out = out;
                d.ldo = c.lddw;
                to = p_mn;
            } else if (PLANES == 1) {
                BL_MAP(map_bf16(&to, out, c.dim, n, 1, c.lddw, c.lddw, 32));
            } else {
                BL_MAP(map_f32(&to, out, c.dim, n, 1, c.lddw, c.lddw));
            }
            BL_TRY((launch_with_p<DW, PLANES>(p_mn, h_mn, to, d, q, flag_count, c.sms, c.s)));
        }
    }
    if (t_gave_up) BL_TRY(cudaMemsetAsync(flags, 1, 4, c.s));
    const Spoiled<T> spoiled{static_cast<T *>(c.dW), c.lddw, c.vocab, dim};
    if (!q.grad) {
        BL_TRY(launch_pdl(loss_kernel, static_cast<unsigned>(cdiv(c.rows, 8)), 256, 0, c.s,
                          reinterpret_cast<const float2 *>(c.ws + q.part), q.part_ld, reinterpret_cast<const float *>(c.ws + q.picked),
                          c.target, c.vocab, rows, order, kept, flags, flag_count, c.loss, c.lse));
    } else if (c.dH) {
        const int share = q.parts >= 8 ? 8 : 1;
        const int64_t blocks = std::min<int64_t>(cdiv(c.rows * cdiv(c.dim, 4) * share, 256), static_cast<int64_t>(c.sms) * 8);
        const int64_t es = sizeof(T);
        const int vec = reinterpret_cast<uintptr_t>(c.dH) % (4 * es) == 0 && c.lddh % 4 == 0;
        BL_TRY(launch_pdl(share == 8 ? dh_kernel<T, 8> : dh_kernel<T, 1>, static_cast<unsigned>(blocks), 256, 0, c.s,
                          reinterpret_cast<const float *>(c.ws + q.dh), q.parts, c.rows, q.ldo, dim, c.target, c.vocab, place, kept, unit,
                          flags, flag_count, static_cast<T *>(c.dH), c.lddh, vec, spoiled));
    } else {
        BL_TRY(launch_pdl(spoil_kernel<T>, static_cast<unsigned>(c.sms), 256, 0, c.s, flags, flag_count, spoiled));
    }
    return BL_SUCCESS;
}

// ------------------------------------------------------------------ arguments

bl_status check_shape(const char *op, int dtype, int64_t rows, int64_t dim, int64_t vocab) {
    if (dtype != BL_F32 && dtype != BL_BF16) return fail(BL_ERR_INVALID_ARGUMENT, "%s: dtype %d is not f32 or bf16", op, dtype);
    if (rows < 1 || rows > (int64_t(1) << 22))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: rows=%lld outside [1, 2^22]", op, (long long)rows);
    if (dim < 1 || dim > (int64_t(1) << 16))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: dim=%lld outside [1, 2^16]", op, (long long)dim);
    if (vocab < 1 || vocab > (int64_t(1) << 24))
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: vocab=%lld outside [1, 2^24]", op, (long long)vocab);
    return BL_SUCCESS;
}

bl_status check_matrix(const char *op, const char *name, const void *p, int64_t ld, int64_t dim, int dtype) {
    const int64_t es = dtype == BL_F32 ? 4 : 2;
    if (!p) return fail(BL_ERR_INVALID_ARGUMENT, "%s: %s is NULL", op, name);
    if (reinterpret_cast<uintptr_t>(p) % es != 0)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its %lld-byte element", op, name, (long long)es);
    if (ld < dim) return fail(BL_ERR_INVALID_ARGUMENT, "%s: ld of %s is %lld < dim=%lld", op, name, (long long)ld, (long long)dim);
    if (ld > (int64_t(1) << 32)) return fail(BL_ERR_INVALID_ARGUMENT, "%s: ld of %s is %lld, too large", op, name, (long long)ld);
    return BL_SUCCESS;
}

// The bytes of rows of `dim` values, ld apart, that a matrix consists of.
struct Rows {
    uintptr_t at;
    uintptr_t step, length;
    int64_t rows;
    Range all() const { return {at, at + static_cast<uintptr_t>(rows - 1) * step + length}; }
};
Rows rows_at(const void *p, int64_t rows, int64_t dim, int64_t ld, int64_t es) {
    return {reinterpret_cast<uintptr_t>(p), static_cast<uintptr_t>(ld * es), static_cast<uintptr_t>(dim * es), rows};
}
// Whether two matrices share a byte. One may lie in the gaps of the other: as another column range of one
// buffer, or in some other way, for which every row of the shorter one is looked up.
bool meet(const Rows &a, const Rows &b) {
    if (!bl::meet(a.all(), b.all())) return false;
    if (a.rows > b.rows) return meet(b, a);
    if (a.step == b.step && a.rows > 1) {
        const uintptr_t d = (b.at - a.at + (a.at > b.at ? (a.at - b.at + a.step - 1) / a.step * a.step : 0)) % a.step;
        if (d >= a.length && d + b.length <= a.step) return false;
    }
    for (int64_t r = 0; r < a.rows; ++r) {
        const uintptr_t lo = a.at + static_cast<uintptr_t>(r) * a.step, hi = lo + a.length;
        // the first row of b that ends past lo
        const uintptr_t j = b.at + b.length > lo ? 0 : (lo - b.at - b.length) / b.step + 1;
        if (j < static_cast<uintptr_t>(b.rows) && b.at + j * b.step < hi) return true;
    }
    return false;
}
struct Named {
    const char *name;
    Rows rows;
};
// No result overlaps another tensor of the call. The first `written` of the list are results or scratch.
bl_status check_apart(const char *op, const Named *t, int written, int count) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < count; ++j)
            if (t[i].rows.at && t[j].rows.at && meet(t[i].rows, t[j].rows))
                return fail(BL_ERR_INVALID_ARGUMENT, "%s: %s overlaps %s", op, t[i].name, t[j].name);
    return BL_SUCCESS;
}

bl_status check_vector(const char *op, const char *name, const void *p, int align) {
    if (!p || reinterpret_cast<uintptr_t>(p) % align != 0)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: %s is NULL or not %d-byte aligned", op, name, align);
    return BL_SUCCESS;
}

bl_status entry(const char *op, int dtype, Call &c, bool grad, void *ws, int64_t ws_bytes, bl_stream_t stream) {
    clear_error();
    bl_status st = check_shape(op, dtype, c.rows, c.dim, c.vocab);
    if (st == BL_SUCCESS) st = check_matrix(op, "H", c.H, c.ldh, c.dim, dtype);
    if (st == BL_SUCCESS) st = check_matrix(op, "W", c.W, c.ldw, c.dim, dtype);
    if (st == BL_SUCCESS) st = check_vector(op, "target", c.target, 8);
    if (!grad) {
        if (st == BL_SUCCESS) st = check_vector(op, "loss", c.loss, 4);
        if (st == BL_SUCCESS) st = check_vector(op, "lse", c.lse, 4);
    } else {
        if (st == BL_SUCCESS) st = check_vector(op, "lse", c.lse_in, 4);
        if (st == BL_SUCCESS) st = check_vector(op, "g", c.g, 4);
        if (st == BL_SUCCESS && !c.dH && !c.dW) st = fail(BL_ERR_INVALID_ARGUMENT, "%s: dH and dW are both NULL", op);
        if (st == BL_SUCCESS && c.dH) st = check_matrix(op, "dH", c.dH, c.lddh, c.dim, dtype);
        if (st == BL_SUCCESS && c.dW) st = check_matrix(op, "dW", c.dW, c.lddw, c.dim, dtype);
    }
    if (st == BL_SUCCESS) st = check_vector(op, "workspace", ws, 256);
    if (st != BL_SUCCESS) return st;
    c.sms = sm_count();
    if (c.sms <= 0) return fail(BL_ERR_CUDA, "%s: cannot query the current CUDA device", op);
    const Plan q = plan_for(dtype, c.H, c.ldh, c.rows, c.dim, c.vocab, c.W, c.ldw, grad, c.sms);
    if (ws_bytes < q.bytes)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: workspace of %lld bytes is smaller than %lld", op, (long long)ws_bytes,
                    (long long)q.bytes);
    const auto vector = [&](const void *p, int64_t bytes) { return rows_at(p, 1, bytes, bytes, 1); };
    const int64_t es = dtype == BL_F32 ? 4 : 2;
    Named all[8] = {{"dH", rows_at(c.dH, c.rows, c.dim, c.lddh, es)}, {"dW", rows_at(c.dW, c.vocab, c.dim, c.lddw, es)},
                    {"the workspace", vector(ws, q.bytes)},           {"H", rows_at(c.H, c.rows, c.dim, c.ldh, es)},
                    {"W", rows_at(c.W, c.vocab, c.dim, c.ldw, es)},   {"target", vector(c.target, c.rows * 8)},
                    {"lse", vector(c.lse_in, c.rows * 4)},            {"g", vector(c.g, c.rows * 4)}};
    if (!grad) {
        all[0] = {"loss", vector(c.loss, c.rows * 4)};
        all[1] = {"lse", vector(c.lse, c.rows * 4)};
    }
    st = check_apart(op, all, 3, grad ? 8 : 6);
    if (st != BL_SUCCESS) return st;
    c.ws = static_cast<char *>(ws);
    c.s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == BL_F32 ? run<float, 3>(op, q, c) : run<__nv_bfloat16, 1>(op, q, c);
}

}  // namespace xent
}  // namespace bl

extern "C" {

int64_t bl_xent_workspace(bl_dtype dtype, int64_t rows, int64_t dim, int64_t vocab, const void *H, int64_t ldh,
                          const void *W, int64_t ldw, int grad) {
    using namespace bl::xent;
    bl::clear_error();
    if (check_shape("xent_workspace", dtype, rows, dim, vocab) != BL_SUCCESS) return -1;
    const int sms = bl::sm_count();
    if (sms <= 0) {
        bl::fail(BL_ERR_CUDA, "xent_workspace: cannot query the current CUDA device");
        return -1;
    }
    return plan_for(dtype, H, ldh, rows, dim, vocab, W, ldw, grad != 0, sms).bytes;
}

bl_status bl_xent(bl_dtype dtype, int64_t rows, int64_t dim, int64_t vocab, const void *H, int64_t ldh, const void *W,
                  int64_t ldw, const int64_t *target, float *loss, float *lse, void *workspace, int64_t workspace_bytes,
                  bl_stream_t stream) {
    bl::xent::Call c{};
    c.rows = rows, c.dim = dim, c.vocab = vocab;
    c.H = H, c.ldh = ldh, c.W = W, c.ldw = ldw, c.target = target;
    c.loss = loss, c.lse = lse;
    return bl::xent::entry("xent", dtype, c, false, workspace, workspace_bytes, stream);
}

bl_status bl_xent_grad(bl_dtype dtype, int64_t rows, int64_t dim, int64_t vocab, const void *H, int64_t ldh,
                       const void *W, int64_t ldw, const int64_t *target, const float *lse, const float *g, void *dH,
                       int64_t lddh, void *dW, int64_t lddw, void *workspace, int64_t workspace_bytes,
                       bl_stream_t stream) {
    bl::xent::Call c{};
    c.rows = rows, c.dim = dim, c.vocab = vocab;
    c.H = H, c.ldh = ldh, c.W = W, c.ldw = ldw, c.target = target;
    c.lse_in = lse, c.g = g;
    c.dH = dH, c.lddh = lddh, c.dW = dW, c.lddw = lddw;
    return bl::xent::entry("xent_grad", dtype, c, true, workspace, workspace_bytes, stream);
}

bl_status bl_debug_xent_gave_up(int on) {
    bl::clear_error();
    bl::xent::t_gave_up = on != 0;
    return BL_SUCCESS;
}

}  // extern "C"
