// The tensor-core products of the orthogonalisation (orth.cu), one persistent kernel for all. With X stored as
// `lines` rows of `width` contiguous values, A its Gram matrix on the shorter side and B = b A + c A A:
//
//   GRAM    A = X X^T or X^T X (K-major operands, or both MN-major)
//   SQUARE  B from A A (K-major)
//   APPLY   a X + B X (K-major, MN-major) or a X + X B (both K-major)
//
// Everything between the products is f16 in two planes, x = hi + lo (22 bits), scaled by a power of two so that no
// value leaves f16's range. PLANES = 1 multiplies the hi planes only; PLANES = 2 adds hi lo + lo hi + hi hi, which
// leaves out 2^-22 of a product. The term a X is added from both planes in f32 in the epilogue in either case:
// what the iteration multiplies by a in every step, the directions of small singular values, keeps 22 bits, and the
// products' own rounding meets only directions that have grown (see orth.cu).
//
// A and B are symmetric: tiles above the diagonal are left out, and what lies below it is stored twice, the second
// time from the lanes side by side, block by block transposed.
//
// A CTA computes 128 x tile_n tiles, or a pair of CTAs 256 x tile_n tiles (each holds its 128 rows and half of B).
// Roles, waits and registers as in xent_gemm.cuh: a producer warp for each operand, an issuing warp, eight
// epilogue warps that work on one accumulator of tensor memory while the next tile is added up in another. With
// PLANES = 2 the chain of K is cut into chunks that are added in registers: tensor memory's f32 sums cut where f32
// would round, up to 2^-23.4 of the sum a step for the diagonal of A.
//
// What bounds it: for large matrices the operands' way into shared memory, 64 bytes a cycle and SM at full rate, and the
// power cap (8192 x 4096 bf16: tensor pipe 84% busy in A, 76 to 82% in B X, whose addend and result take their share of L2;
// 1,340 to 1,390 TFLOP/s over the call); for small ones latency, some 5 us a product: 1.4 from the end of one kernel to the start
// of the next, 1.3 to the first operands, 2.5 from the last product to the end.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "pdl.cuh"
#include "tma_sm100.cuh"

namespace bl {
namespace orth {

enum Kind : int { GRAM = 0, SQUARE = 1, APPLY = 2 };

constexpr int kTileM = 128, kTileN = 256, kTileK = 64;          // columns of a tile, at most
constexpr int kEpilogueWarps = 8;                               // two share 32 rows
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kRegsLaunch = 168, kRegsFew = 56, kRegsMany = 224;
static_assert(128 * kRegsFew + 32 * kEpilogueWarps * kRegsMany <= kThreads * kRegsLaunch, "more registers than the block has");
constexpr uint32_t kPolls = 1u << 22;

// X is kept times 2^13, A and B times 2^12: for (3.4445, -4.7750, 2.0315) elements of X are at most 1.3, of A 1.7, of B 3, and
// f16 reaches 65504; typical ones, 1 / sqrt(long side), stay in f16's normal range for 22 bits up to sides of 2^16.
constexpr float kScaleX = 8192.f, kScaleA = 4096.f;

// What X_0's values are multiplied by, one after the other, for a given sum of squares: a power of two where the norm
// lies outside of what f32 multiplies by without loss, then the rest. A matrix of zeros stays one; NaN if the norm is not finite.
__device__ __forceinline__ float2 scale_of(double sum) {
    if (!(sum < INFINITY)) return make_float2(1.f, NAN);
    if (sum == 0.0) return make_float2(0.f, 0.f);
    const float f = static_cast<float>(sum);
    if (f >= 1e-30f && f <= 1e30f) return make_float2(1.f, kScaleX / sqrtf(f));      // the f64 unit is slow
    const double norm = sqrt(sum);
    const float power = norm < 1.0 ? 0x1p126f : 0x1p-126f;
    return make_float2(power, static_cast<float>(kScaleX / (norm * power)));
}

// Shared memory of a CTA: the operands' ring, and lines for each epilogue warp, by which results leave and what a
// product is added to comes in, both by TMA: UNIT columns of the warp's 32 rows at a time, a plane after the other. The
// same lines serve both ways, a lane writing where it has read; only A and B in one plane are small enough to take
// turns between two halves. TMA takes as long for a line of 64 bytes as for one of 128, some two cycles, and the
// operands alone keep it busy (a 256 x 256 tile's stage 512 cycles, as long as its products), so lines are 128 bytes where
// there is room: 8192 x 4096 bf16, five steps 1898 us with lines of 64 bytes, 1855 of 128. (These two, and those
// at the order of tiles below, were taken with one thread issuing products and copies; 1735 to 1795 with whole warps. Lines
// read and written with 16 bytes a lane instead took 1705, but 12 x 1024 x 4096 971 in place of 910 and 512 x 512 no less.)
// A stage is as small as the tile's columns allow: narrow tiles, of small matrices, wait for memory, and the more
// of their stages are on their way the better.
constexpr int kMostStages = 8;
// Accumulators: tensor memory's 512 columns hold as many as the tile's width allows. Two would do for wide tiles; the
// chunks of narrow ones, of two planes, take less time than an epilogue takes to answer (517 x 1031 f32 208 us
// with two, 192 so).
constexpr int kMostAccs = 8;
template <int PLANES, int CTAS>
struct Ring {
    static constexpr int kTile = CTAS == 1 ? 128 : 256;             // columns of a tile, at most
    static constexpr int kBytesA = kTileM * kTileK * 2, kStageA = PLANES * kBytesA;
    static constexpr int kUnit = PLANES == 1 ? 64 : 32;
    static constexpr int kPlane = 32 * kUnit * 2, kLines = 2 * kPlane;            // bytes of a warp
    static constexpr int kBytes = (PLANES == 1 ? 160 : 192) * 1024;
    static constexpr int kSmem = kBytes + kEpilogueWarps * kLines + 1024;
    static constexpr int stage(int tile_n) { return kStageA + PLANES * (tile_n / CTAS * 128); }
};

struct Args {
    int batch;
    int rows, cols;            // of the product, of each item
    int kblocks, chunk;        // 64-deep steps; how many are added in tensor memory before registers take over
    int tile_n, tiles_m, tiles_n;
    int per_item, total;       // tiles
    float alpha, beta;         // result = alpha * product + beta * what is added
    int stages;                // of the ring
    __half *result;            // GRAM, SQUARE: [plane][item][rows][result_ld], for what lies above the diagonal
    int64_t result_ld;
    bool last;                 // APPLY: the result is the caller's, f32 or bf16
    void *out;                 // where its lines or items are not where a tensor map has them: stored without TMA
    int64_t ldo, stride_o;
    bool rows_first;           // APPLY: the order of tiles
    int group;
    int32_t *gave_up;
};

struct Work {
    int item, tm, tn;
};
template <int KIND, int CTAS>
__device__ __forceinline__ Work work_of(int w, const Args &a) {
    Work r;
    r.item = w / a.per_item;
    w -= r.item * a.per_item;
    if constexpr (KIND != APPLY) {
        // row tile after row tile, as many columns as reach its last row's diagonal
        r.tm = 0;
        while (true) {
            const int n = min(a.tiles_n, ((r.tm + 1) * (CTAS * kTileM) + a.tile_n - 1) / a.tile_n);
            if (w < n) break;
            w -= n;
            ++r.tm;
        }
        r.tn = w;
    } else {
        // B's side of the tiles varies first, `group` of them at a time, so that this much of B stays in L2 while X
        // goes by: with all of its 32 MB at a time one product of 8192 x 4096 reads 540 MB of memory, and the five steps take
        // 1855 us; in groups of 16 MB 1820.
        const int inner = a.rows_first ? a.tiles_m : a.tiles_n, outer = a.rows_first ? a.tiles_n : a.tiles_m;
        const int g = w / (a.group * outer), size = min(a.group, inner - g * a.group);
        w -= g * a.group * outer;
        const int o = w / size, i = g * a.group + w - o * size;
        r.tm = a.rows_first ? i : o;
        r.tn = a.rows_first ? o : i;
    }
    return r;
}
// Columns of the tile that the product has, rounded up to what the instruction (a pair: each CTA's half; an
// MN-major operand: whole groups of 64) can take.
template <bool B_MN, int CTAS>
__device__ __forceinline__ int cols_of(int tn, const Args &a) {
    constexpr int UNIT = CTAS == 1 ? 16 : B_MN ? 128 : 32;
    const int left = min(a.cols - tn * a.tile_n, a.tile_n);
    return (left + UNIT - 1) & ~(UNIT - 1);
}

__device__ __forceinline__ uint32_t pack(__half lo, __half hi) {
    const __half2 t = __halves2half2(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}

// ---- epilogue

template <int KIND, int PLANES>
struct Form {
    using R = Ring<PLANES, 1>;
    static constexpr int kUnit = R::kUnit, kPlane = R::kPlane;
    static constexpr int kAdd = KIND == GRAM ? 0 : KIND == SQUARE ? PLANES : 2;        // planes of what is added
    static constexpr int kOut = KIND == APPLY ? 2 : PLANES;                            // of the result
    static constexpr bool kTurns = KIND != APPLY && PLANES == 1;                       // two units have lines of their own
};
// 16 bytes of a line, in the swizzle of its length.
template <int UNIT>
__device__ __forceinline__ uint32_t at_line(int line, int chunk) {
    return UNIT == 64 ? line * 128 + ((chunk ^ (line & 7)) << 4) : line * 64 + ((chunk ^ ((line >> 1) & 3)) << 4);
}
__device__ __forceinline__ void lines_free() {          // the stores of earlier units have read their lines
    if ((threadIdx.x & 31) == 0) tc::bulk_wait_read_all();
    __syncwarp();
}
__device__ __forceinline__ void lines_free_but_last() {
    if ((threadIdx.x & 31) == 0) tc::bulk_wait_read_but_one();
    __syncwarp();
}
template <int KIND, int PLANES>
__device__ __forceinline__ void addend_ask(const CUtensorMap *map, const Args &a, int item, unsigned char *lines, uint64_t *bar, int row0,
                                           int col0) {
    using F = Form<KIND, PLANES>;
    if ((threadIdx.x & 31) != 0) return;
    tc::mbar_expect_tx(bar, F::kPlane * F::kAdd);
#pragma unroll
    for (int p = 0; p < F::kAdd; ++p) tc::tma_load_3d<1>(lines + p * F::kPlane, map, tc::smem_u32(bar), col0, row0, p * a.batch + item);
}

// 32 columns of a warp's 32 rows, the b-th of a unit: from the product to the result's lines.
template <int KIND, int PLANES>
__device__ __forceinline__ void block_out(const Args &a, int item, int row0, int col0, int b, float (&v)[32], unsigned char *lines) {
    using F = Form<KIND, PLANES>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[4] = {}, l[4] = {};
        if constexpr (F::kAdd >= 1) *reinterpret_cast<uint4 *>(h) = *reinterpret_cast<const uint4 *>(lines + at_line<F::kUnit>(lane, 4 * b + j));
        if constexpr (F::kAdd == 2)
            *reinterpret_cast<uint4 *>(l) = *reinterpret_cast<const uint4 *>(lines + F::kPlane + at_line<F::kUnit>(lane, 4 * b + j));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float &x = v[8 * j + 2 * q], &y = v[8 * j + 2 * q + 1];
            x *= a.alpha, y *= a.alpha;
            if constexpr (F::kAdd == 2) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&l[q]));
                x = fmaf(a.beta, t.x, x), y = fmaf(a.beta, t.y, y);
            }
            if constexpr (F::kAdd >= 1) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[q]));
                x = fmaf(a.beta, t.x, x), y = fmaf(a.beta, t.y, y);
            }
        }
    }
    if (KIND == APPLY && a.last) {
        if constexpr (PLANES == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(lines + at_line<64>(lane, 4 * b + j)) = make_uint4(
                    bf16x2(v[8 * j], v[8 * j + 1]), bf16x2(v[8 * j + 2], v[8 * j + 3]), bf16x2(v[8 * j + 4], v[8 * j + 5]),
                    bf16x2(v[8 * j + 6], v[8 * j + 7]));
        } else {
            __syncwarp();                   // lines of f32 lie across what other lanes have read
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(lines + at_line<64>(lane, j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
        return;
    }
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        hi[i] = *reinterpret_cast<const uint32_t *>(&h);
        if constexpr (F::kOut == 2) {
            const float2 back = __half22float2(h);
            const __half2 l = __floats2half2_rn(v[2 * i] - back.x, v[2 * i + 1] - back.y);
            lo[i] = *reinterpret_cast<const uint32_t *>(&l);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<uint4 *>(lines + at_line<F::kUnit>(lane, 4 * b + j)) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
        if constexpr (F::kOut == 2)
            *reinterpret_cast<uint4 *>(lines + F::kPlane + at_line<F::kUnit>(lane, 4 * b + j)) =
                make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
    if (KIND != APPLY && (row0 & ~(F::kUnit - 1)) > col0 && row0 + lane < a.rows) {
        // the same block in its place above the diagonal: column i is a line there, on which the lanes lie side by side
        // (col0 + 31 lies before this unit's rows: such lines are there)
        uint16_t *p = reinterpret_cast<uint16_t *>(a.result) + (static_cast<int64_t>(item) * a.rows + col0) * a.result_ld + row0 + lane;
        const int64_t plane = static_cast<int64_t>(a.batch) * a.rows * a.result_ld;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += a.result_ld) {
            *p = static_cast<uint16_t>(hi[i / 2] >> (i % 2 * 16));
            if constexpr (F::kOut == 2) p[plane] = static_cast<uint16_t>(lo[i / 2] >> (i % 2 * 16));
        }
    }
}
// A unit's lines leave.
template <int KIND, int PLANES>
__device__ __forceinline__ void unit_out(const CUtensorMap *map, const Args &a, int item, int row0, int col0, unsigned char *lines) {
    using F = Form<KIND, PLANES>;
    using T = std::conditional_t<PLANES == 1, __nv_bfloat16, float>;
    const int lane = threadIdx.x & 31;
    if (KIND == APPLY && a.last && a.out) {             // lines that TMA cannot store
        __syncwarp();
        const int rows = min(32, a.rows - row0);
        for (int c = lane; c < F::kUnit; c += 32) {
            T *p = static_cast<T *>(a.out) + item * a.stride_o + row0 * a.ldo + col0 + c;
            constexpr int PER = 16 / sizeof(T);
            for (int q = 0; q < rows; ++q, p += a.ldo) {
                const T x = *reinterpret_cast<const T *>(lines + at_line<64>(q, c / PER) + c % PER * sizeof(T));
                if (col0 + c < a.cols) *p = x;
            }
        }
        __syncwarp();
        return;
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tc::tma_store_3d(map, lines, col0, row0, item, false);
        if (F::kOut == 2 && !(KIND == APPLY && a.last)) tc::tma_store_3d(map, lines + F::kPlane, col0, row0, a.batch + item, false);
        tc::bulk_commit();
    }
}

template <int KIND, bool A_MN, bool B_MN, int PLANES, int CTAS>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_add, const __grid_constant__ CUtensorMap map_out,
                   const __grid_constant__ Args a) {
    using R = Ring<PLANES, CTAS>;
    constexpr int kBytesA = R::kBytesA, kStageA = R::kStageA;
    constexpr int PAIRS = PLANES == 1 ? 1 : 3, BLOCKS = R::kTile / 64;
    const uint32_t accs = 512 / a.tile_n, acc_bits = 31 - __clz(accs);       // a power of two
    const uint32_t stages = a.stages, bytes_b = a.tile_n / CTAS * 128, stage_b = PLANES * bytes_b;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *const base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *const tiles_a = base, *const tiles_b = base + stages * kStageA;
    unsigned char *const all_lines = base + R::kBytes;
    __shared__ uint64_t full[kMostStages], empty[kMostStages], acc_full[kMostAccs], acc_empty[kMostAccs], add_full[kEpilogueWarps], drained;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t rank = CTAS == 1 ? 0 : tc::cluster_rank();
    if (warp == 1) tc::tmem_take<CTAS>(&tmem_slot, 512);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMostStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kMostAccs; ++s) {
            tc::mbar_init(&acc_full[s], 1);
            tc::mbar_init(&acc_empty[s], CTAS * kEpilogueWarps);
        }
        for (int s = 0; s < kEpilogueWarps; ++s) tc::mbar_init(&add_full[s], 1);
        tc::mbar_init(&drained, 1);
        tc::mbar_fence_init();
        gave_up = 0;
        tc::tma_prefetch_map(&map_a);
        tc::tma_prefetch_map(&map_b);
        tc::tma_prefetch_map(&map_add);
        tc::tma_prefetch_map(&map_out);
    }
    __syncwarp();
    pdl_release();
    tc::fence_before_sync();
    if constexpr (CTAS == 1) __syncthreads();
    else tc::cluster_sync();                 // the peer's barriers are ready too
    tc::fence_after_sync();
    pdl_wait();
    const uint32_t tmem = tmem_slot;

    if (warp < 4) {
      tc::regs_dec<kRegsFew>();
      if (warp == 0 || warp == 2) {
        {
            const bool for_a = warp == 0, announce = for_a && rank == 0;
            const uint32_t bar0 = CTAS == 1 ? tc::smem_u32(full) : tc::at_leader(full);
            uint32_t s = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int w = blockIdx.x / CTAS; ok && w < a.total; w += gridDim.x / CTAS) {
                const Work k = work_of<KIND, CTAS>(w, a);
                const int part = cols_of<B_MN, CTAS>(k.tn, a) / CTAS;       // this CTA's columns of B
                const int m0 = (k.tm * CTAS + rank) * kTileM, n0 = k.tn * a.tile_n + rank * part;
                const int groups_b = (part + 63) >> 6;
                const uint32_t bytes = CTAS * PLANES * (kBytesA + (B_MN ? groups_b * (kTileK * 128) : a.tile_n / CTAS * 128));
                for (int kb = 0; kb < a.kblocks; ++kb) {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], phase ^ 1, kPolls));
                    if (!ok) break;
                    const uint32_t bar = bar0 + 8 * s;
                    if (tc::elect()) {
                        if (announce) tc::mbar_expect_tx(&full[s], bytes);
#pragma unroll 1
                        for (int p = 0; p < PLANES; ++p) {
                            const int z = p * a.batch + k.item;
                            if (for_a) {
                                unsigned char *const d = tiles_a + s * kStageA + p * kBytesA;
                                if constexpr (A_MN) {
#pragma unroll
                                    for (int j = 0; j < kTileM / 64; ++j)
                                        tc::tma_load_3d<CTAS>(d + j * kTileK * 128, &map_a, bar, m0 + 64 * j, kb * kTileK, z);
                                } else {
                                    tc::tma_load_3d<CTAS>(d, &map_a, bar, kb * kTileK, m0, z);
                                }
                            } else {
                                unsigned char *const d = tiles_b + s * stage_b + p * bytes_b;
                                if constexpr (B_MN) {
#pragma unroll 1
                                    for (int j = 0; j < groups_b; ++j)
                                        tc::tma_load_3d<CTAS>(d + j * kTileK * 128, &map_b, bar, n0 + 64 * j, kb * kTileK, z);
                                } else {
                                    tc::tma_load_3d<CTAS>(d, &map_b, bar, kb * kTileK, n0, z);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    issued = min(issued + 1, stages);
                    if (++s == stages) s = 0, phase ^= 1;
                }
            }
            if (!ok && lane == 0) {
                gave_up = 1;
                // the copies in flight: the last `issued` stages before s, oldest first
                for (uint32_t i = 0; rank == 0 && i < issued; ++i) {
                    const uint32_t t = s + stages - issued + i;
                    tc::mbar_wait(&full[t % stages], t >= stages ? phase : phase ^ 1, kPolls);
                }
            }
        }
      } else if (warp == 1) {
        // The whole warp goes through the steps, so that what the products are issued with is known to be the same in
        // all lanes; one lane issues. A lane looks at one stage's barrier, so that all that is there is found at once:
        // a barrier takes 150 cycles to look at, the four products of a stage 160 to issue.
        if (rank == 0) {
            const uint64_t da0 = A_MN ? tc::sdesc_mn_sw128(tc::smem_u32(tiles_a), kTileK * 128) : tc::sdesc_sw128(tc::smem_u32(tiles_a));
            const uint64_t db0 = B_MN ? tc::sdesc_mn_sw128(tc::smem_u32(tiles_b), kTileK * 128) : tc::sdesc_sw128(tc::smem_u32(tiles_b));
            uint32_t s = 0, phase = 0, done = 0, there = 0;
            bool ok = true;
            const auto look = [&] {                    // how many stages from s on are there
                const uint32_t t = s + lane, wrapped = t >= stages;
                for (uint32_t i = 0; there == 0 && i < kPolls; ++i) {
                    const bool full_now = lane < static_cast<int>(stages) && tc::mbar_wait(&full[wrapped ? t - stages : t], phase ^ wrapped, 1);
                    there = __ffs(~__ballot_sync(0xffffffffu, full_now)) - 1;
                }
                __syncwarp();
                return there > 0;
            };
            for (int w = blockIdx.x / CTAS; ok && w < a.total; w += gridDim.x / CTAS) {
                const Work k = work_of<KIND, CTAS>(w, a);
                const uint32_t idesc = tc::idesc_f16(CTAS * kTileM, cols_of<B_MN, CTAS>(k.tn, a), A_MN, B_MN);
                for (int c = 0; ok && c < a.kblocks; c += a.chunk, ++done) {
                    const uint32_t at = done & (accs - 1), acc = tmem + at * a.tile_n;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_empty[at], (done >> acc_bits & 1) ^ 1, kPolls));
                    if (!ok) break;
                    const int steps = min(c + a.chunk, a.kblocks) - c;
                    for (int i = 0; i < steps; ++i) {
                        if (there == 0) ok = look();
                        if (!ok) break;
                        --there;
                        tc::fence_after_sync();
                        const uint64_t da = da0 + s * (kStageA >> 4), db = db0 + s * (stage_b >> 4);
                        if (tc::elect()) {
#pragma unroll
                            for (int q = 0; q < PAIRS; ++q) {
                                const int pa = PLANES == 2 && q == 1, pb = PLANES == 2 && q == 0;       // hi lo, lo hi, hi hi
#pragma unroll
                                for (int j = 0; j < kTileK / 16; ++j)   // 16 k: 32 bytes along a line, or 16 lines
                                    tc::mma_f16<CTAS>(acc, da + pa * (kBytesA >> 4) + j * (A_MN ? 2048 / 16 : 2),
                                                      db + pb * (bytes_b >> 4) + j * (B_MN ? 2048 / 16 : 2), idesc,
                                                      i > 0 || q > 0 || j > 0);
                            }
                            tc::mma_commit_all<CTAS>(&empty[s]);
                            if (i + 1 == steps) tc::mma_commit_all<CTAS>(&acc_full[at]);
                        }
                        __syncwarp();
                        if (++s == stages) s = 0, phase ^= 1;
                    }
                }
            }
            if (!ok) {
                // by the lane that issued: a commit covers its own thread's products
                if (tc::elect()) {
                    gave_up = 1;
                    tc::mma_commit_all<CTAS>(&drained);
                    tc::mbar_wait(&drained, 0, kPolls);
                }
            }
        }
      }
    } else {
        tc::regs_inc<kRegsMany>();
        const int quad = warp & 3, half = (warp - 4) >> 2;  // a warp may read its quarter of the lanes
        using F = Form<KIND, PLANES>;
        constexpr int UNIT = F::kUnit;
        unsigned char *const lines0 = all_lines + (warp - 4) * R::kLines;
        uint64_t *const bar = &add_full[warp - 4];
        uint32_t done = 0, units = 0;
        bool ok = true;
        // columns of a tile that this warp has: a half, or all where a half is less than a unit
        const int mine = max(a.tile_n / 2, UNIT), first = half * mine;
        for (int w = blockIdx.x / CTAS; ok && w < a.total; w += gridDim.x / CTAS) {
            const Work k = work_of<KIND, CTAS>(w, a);
            const int n0 = k.tn * a.tile_n, row0 = (k.tm * CTAS + rank) * kTileM + quad * 32;
            int cols = min(a.cols - n0, min(first + mine, a.tile_n));                      // they end there
            if (KIND != APPLY) cols = min(cols, (row0 & ~(UNIT - 1)) + UNIT - n0);         // or with the diagonal's unit
            if (row0 >= a.rows) cols = 0;
            const auto lines_of = [&](uint32_t u) { return lines0 + (F::kTurns ? (u & 1) * F::kPlane : 0); };
            const auto ask = [&](int c0) {             // for the next unit, whose lines are free before
                if constexpr (F::kTurns) lines_free_but_last();
                else lines_free();
                if constexpr (F::kAdd > 0) addend_ask<KIND, PLANES>(&map_add, a, k.item, lines_of(units), bar, row0, n0 + c0);
            };
            const auto take = [&] {
                if constexpr (F::kAdd > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, units & 1, kPolls)) && ok;
            };
            if (first < cols) ask(first);              // on its way while the products run
            if constexpr (PLANES == 1) {
                // blocks go out as they leave tensor memory
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_full[done & (accs - 1)], done >> acc_bits & 1, kPolls));
                if (!ok) {
                    if (first < cols) take();
                } else {
                    tc::fence_after_sync();
                    const uint32_t acc = tmem + (done & (accs - 1)) * a.tile_n + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
                    for (int c0 = first; c0 < cols; c0 += UNIT) {
                        take();
#pragma unroll 1
                        for (int b = 0; b < 2 && n0 + c0 + 32 * b < a.cols; ++b) {
                            float v[32];
                            __syncwarp();
                            tc::tmem_ld32(acc + c0 + 32 * b, v);
                            block_out<KIND, PLANES>(a, k.item, row0, n0 + c0 + 32 * b, b, v, lines_of(units));
                        }
                        unit_out<KIND, PLANES>(&map_out, a, k.item, row0, n0 + c0, lines_of(units));
                        ++units;
                        if (c0 + UNIT < cols) ask(c0 + UNIT);
                    }
                    __syncwarp();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CTAS == 1) tc::mbar_arrive(&acc_empty[done & (accs - 1)]);
                        else tc::mbar_arrive_at(tc::at_leader(&acc_empty[done & (accs - 1)]));
                    }
                    ++done;
                }
            } else {
                float v[BLOCKS][32];
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[b][i] = 0.f;
#pragma unroll 1
                for (int c = 0; c < a.kblocks; c += a.chunk, ++done) {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_full[done & (accs - 1)], done >> acc_bits & 1, kPolls));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t acc = tmem + (done & (accs - 1)) * a.tile_n + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        const int c0 = first + 32 * b;
                        if (c0 < cols) {
                            float x[32];
                            __syncwarp();
                            tc::tmem_ld32(acc + c0, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[b][i] += x[i];
                        }
                    }
                    __syncwarp();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CTAS == 1) tc::mbar_arrive(&acc_empty[done & (accs - 1)]);
                        else tc::mbar_arrive_at(tc::at_leader(&acc_empty[done & (accs - 1)]));
                    }
                }
                if (ok) {
                    // one copy of the code for the blocks, whose sums move up
#pragma unroll 1
                    for (int c0 = first; c0 < cols; c0 += UNIT) {
                        if (c0 > first) ask(c0);
                        take();
                        block_out<KIND, PLANES>(a, k.item, row0, n0 + c0, 0, v[0], lines0);
                        unit_out<KIND, PLANES>(&map_out, a, k.item, row0, n0 + c0, lines0);
                        ++units;
#pragma unroll
                        for (int b = 0; b + 1 < BLOCKS; ++b)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[b][i] = v[b + 1][i];
                    }
                    __syncwarp();
                } else if (first < cols) {
                    take();
                }
            }
            if (!ok && lane == 0) gave_up = 1;
        }
        if (lane == 0) tc::bulk_wait_read_all();         // the grid's end, which the next kernel waits for, is the stores' too
    }
    __syncwarp();
    tc::fence_before_sync();
    if constexpr (CTAS == 1) __syncthreads();
    else tc::cluster_sync();                 // nothing of the pair's is in flight towards either CTA
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_give<CTAS>(tmem, 512);
    if (threadIdx.x == 0 && gave_up) atomicExch(a.gave_up, 1);
}

}  // namespace orth
}  // namespace bl
