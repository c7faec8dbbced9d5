// The tensor-core products of the softmax cross entropy, one persistent kernel for all four:
//
//   LOGITS  s = H W^T           A = H (K-major), B = W (K-major); keeps max and sum of exp per tile
//   PROBS   s again, then       P = g (exp(s - lse) - onehot) as bf16 planes
//   DH      dH = P W            A = P (K-major), B = W (MN-major); f32 partial sums
//   DW      dW = P^T H          A = P (MN-major), B = H (MN-major); stored in W's type
//
// A CTA computes 128 x 256 tiles. One thread streams 64-deep operand tiles into a ring of shared
// memory by TMA, one thread issues tcgen05.mma (bf16 operands, f32 accumulators in tensor
// memory), and eight warps turn finished accumulators into the mode's output while the next tile's
// products already run: tensor memory holds two accumulators of 256 columns.
//
// f32 operands are three bf16 planes each, x = x0 + x1 + x2 (8 bits of the 24-bit mantissa in
// each), and six of the nine plane products are added, the ones above 2^-25 of the result,
// smallest first. That costs as much tensor time as three tf32 products and is closer to f32.
//
// The tensor cores' f32 accumulation cuts where f32 would round, so a long chain of products is
// biased towards zero, by about 2^-25 of the sum a step. Where the result is f32 (the loss; every
// product of f32 operands) the chain is cut into chunks of K, whose sums are added in registers.
// Measured at rows 1024, dim 1024, vocabulary 32000, f32: dH 9.6e-6 off without chunks.
//
// Every wait is bounded: a role that gives up marks *status, waits (bounded) for its own copies
// and products in flight, and leaves; the others then run out of time too.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "tma_sm100.cuh"

namespace bl {
namespace xent {

enum Mode : int { LOGITS = 0, PROBS = 1, DH = 2, DW = 3 };

constexpr int kTileM = 128, kTileN = 256, kTileK = 64;
constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTileN * kTileK * 2;
constexpr int kStages = 4;
constexpr int kEpilogueWarps = 8, kHalf = kTileN / 2;           // two warps share 32 rows: 128 columns each
constexpr int kStageRow = 17;                                   // f32 words per row of the store staging
constexpr int kStagingBytes = kEpilogueWarps * 32 * kStageRow * 4;
constexpr int kSmem = kStages * (kBytesA + kBytesB) + kStagingBytes + 1024;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;             // producer, issuer (and two idle warps), epilogue
// 384 threads start with 168 registers each; the first four warps give most of theirs to the
// epilogue, whose rows hold 128 sums: 128 * 40 + 256 * 232 = 384 * 168.
constexpr int kRegsLaunch = 168, kRegsFew = 40, kRegsMany = 232;
static_assert(128 * kRegsFew + 32 * kEpilogueWarps * kRegsMany <= kThreads * kRegsLaunch, "more registers than the block has");
constexpr uint32_t kPolls = 1u << 22;
constexpr int kGroupM = 16;                                     // row tiles that share a column of B tiles
constexpr float kLog2e = 1.4426950408889634f;

struct GemmArgs {
    int m, n;                  // rows and columns of the product
    int kblocks;               // 64-deep steps of one pair of planes
    int chunk;                 // of them, how many are added in tensor memory before registers take over
    int tiles_m, tiles_n;
    int splits, kb_per_split;  // DH: the K axis is cut and every part has its own partial sums
    int pairs;                 // pairs of planes multiplied, 1 or 6
    int accumulate;            // DH: add to the partial sums of earlier pieces
    int32_t *status;
    // LOGITS, PROBS
    const int64_t *target;
    int64_t vocab;
    int v0;                    // first vocabulary entry of this piece
    float2 *part;              // LOGITS: [row][part_ld] max and sum
    int64_t part_ld;
    float *picked;             // LOGITS: the target's logit of each row
    const float *lse, *g;      // PROBS
    __nv_bfloat16 *p;          // PROBS: planes of [row][ldp]
    int64_t ldp, p_plane;
    // DH: f32 partial sums [split][m][ldo]; DW: the result's rows
    void *out;
    int64_t ldo;
    int out_vec;               // DW: rows start on 16-byte boundaries
};

__device__ __forceinline__ void pair_of(int i, int pairs, int &a, int &b) {
    // (1,1) (2,0) (0,2) (1,0) (0,1) (0,0), from the end
    const uint32_t as = 0x0u | (0u << 4) | (1u << 8) | (0u << 12) | (2u << 16) | (1u << 20);
    const uint32_t bs = 0x0u | (1u << 4) | (0u << 8) | (2u << 12) | (0u << 16) | (1u << 20);
    const int j = pairs - 1 - i;
    a = (as >> (4 * j)) & 15;
    b = (bs >> (4 * j)) & 15;
}

struct Work {
    int tm, tn, split;
};
__device__ __forceinline__ Work work_of(int w, const GemmArgs &a) {
    Work r;
    const int tiles = a.tiles_m * a.tiles_n;
    r.split = w / tiles;
    w -= r.split * tiles;
    const int per = kGroupM * a.tiles_n, g = w / per;
    w -= g * per;
    const int rest = a.tiles_m - g * kGroupM, gm = rest < kGroupM ? rest : kGroupM;
    r.tn = w / gm;
    r.tm = g * kGroupM + (w - r.tn * gm);
    return r;
}
// Columns of the tile that the product has, rounded up to the instruction's granularity.
__device__ __forceinline__ int cols_of(int tn, const GemmArgs &a) {
    const int left = a.n - tn * kTileN;
    return left >= kTileN ? kTileN : (left + 15) & ~15;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&t);
}

// x = x0 + x1 + x2 in bf16. A value that rounds past the largest bf16 is cut instead; what is
// not finite stays in x0 alone.
__device__ __forceinline__ void split3(float x, float &x0, float &x1, float &x2) {
    x0 = __bfloat162float(__float2bfloat16_rn(x));
    if (isinf(x0) && !isinf(x)) x0 = __bfloat162float(__float2bfloat16_rz(x));
    const float r = x - x0;
    const bool fine = fabsf(x) <= 3.4028235e38f;
    x1 = fine ? __bfloat162float(__float2bfloat16_rn(r)) : 0.f;
    x2 = fine ? __bfloat162float(__float2bfloat16_rn(r - x1)) : 0.f;
}

// ---- epilogues. A warp owns 32 rows (a lane each) and 128 columns, in blocks of 32 columns.

struct Row {              // what an epilogue keeps of its row
    int row, at;          // row of the product; the target's column within this tile or -1
    bool counted;
    float top, sum, picked;    // LOGITS
    float lse, ref, g;         // PROBS
};

template <int MODE>
__device__ __forceinline__ void begin(Row &r, const GemmArgs &a, const Work &w, int row) {
    r.row = row;
    if constexpr (MODE == LOGITS || MODE == PROBS) {
        const int n0 = w.tn * kTileN;
        const int64_t t = row < a.m ? a.target[row] : -1, at = t - a.v0 - n0;
        r.counted = t >= 0 && t < a.vocab;
        r.at = r.counted && at >= 0 && at < min(a.n - n0, kTileN) ? static_cast<int>(at) : -1;
        r.top = -INFINITY;
        r.sum = r.picked = 0.f;
        if constexpr (MODE == PROBS) {
            r.lse = r.counted ? a.lse[row] : 0.f;
            r.g = r.counted ? a.g[row] : 0.f;
            r.ref = r.lse * kLog2e;
        }
    }
}

// Columns c0 .. c0 + 31 of the tile; those past the product's edge hold anything.
__device__ __forceinline__ void block_logits(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
    const int left = a.n - w.tn * kTileN - c0;
    if (left < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < left ? v[i] : -INFINITY;
    }
    const uint32_t hit = r.at >= c0 && r.at < c0 + 32 ? 1u << (r.at - c0) : 0u;
    float m = r.top;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (hit >> i & 1) r.picked = v[i];
        m = fmaxf(m, v[i]);
    }
    const float ref = m == -INFINITY ? 0.f : m * kLog2e;      // a row of -inf: every term is 0
    r.sum *= exp2f(fmaf(r.top, kLog2e, -ref));
#pragma unroll
    for (int i = 0; i < 32; ++i) r.sum += exp2f(fmaf(v[i], kLog2e, -ref));
    r.top = m;
}

template <int PLANES>
__device__ __forceinline__ void block_probs(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        // the f32 form keeps s - lse exact where it can; the bf16 form rounds the result to 8
        // bits anyway
        float e = PLANES == 1 ? exp2f(fmaf(v[i], kLog2e, -r.ref)) : expf(v[i] - r.lse);
        if (i == r.at - c0) e -= 1.f;
        v[i] = r.counted ? r.g * e : 0.f;
    }
    if (r.row >= a.m) return;
    __nv_bfloat16 *const dst = a.p + static_cast<int64_t>(r.row) * a.ldp + w.tn * kTileN + c0;
    if constexpr (PLANES == 1) {
        uint4 *const q = reinterpret_cast<uint4 *>(dst);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q[j] = make_uint4(bf16x2(v[8 * j], v[8 * j + 1]), bf16x2(v[8 * j + 2], v[8 * j + 3]),
                              bf16x2(v[8 * j + 4], v[8 * j + 5]), bf16x2(v[8 * j + 6], v[8 * j + 7]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[3][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split3(v[8 * j + i], x[0][i], x[1][i], x[2][i]);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl)
                *reinterpret_cast<uint4 *>(dst + pl * a.p_plane + 8 * j) =
                    make_uint4(bf16x2(x[pl][0], x[pl][1]), bf16x2(x[pl][2], x[pl][3]),
                               bf16x2(x[pl][4], x[pl][5]), bf16x2(x[pl][6], x[pl][7]));
        }
    }
}

__device__ __forceinline__ void block_dh(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
    if (r.row >= a.m) return;
    float4 *const q = reinterpret_cast<float4 *>(static_cast<float *>(a.out) +
                                                 (static_cast<int64_t>(w.split) * a.m + r.row) * a.ldo + w.tn * kTileN + c0);
    if (a.accumulate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 o = q[j];
            v[4 * j] += o.x, v[4 * j + 1] += o.y, v[4 * j + 2] += o.z, v[4 * j + 3] += o.w;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// A row that starts on a 16-byte boundary and has all 32 columns.
template <typename T>
__device__ __forceinline__ void block_dw(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
    if (r.row >= a.m) return;
    T *const dst = static_cast<T *>(a.out) + r.row * a.ldo + w.tn * kTileN + c0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            reinterpret_cast<float4 *>(dst)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4 *>(dst)[j] =
                make_uint4(bf16x2(v[8 * j], v[8 * j + 1]), bf16x2(v[8 * j + 2], v[8 * j + 3]),
                           bf16x2(v[8 * j + 4], v[8 * j + 5]), bf16x2(v[8 * j + 6], v[8 * j + 7]));
    }
}

// Rows that start anywhere, or end within the block: through shared memory, 16 columns at a time,
// so that a warp stores along its rows.
template <typename T>
__device__ __forceinline__ void block_dw_any(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32],
                                             float *staging) {
    const int left = a.n - w.tn * kTileN - c0, lane = threadIdx.x & 31, rows = a.m - (r.row - lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) staging[lane * kStageRow + i] = v[16 * h + i];
        __syncwarp();
        const int col = 16 * h + (lane & 15);
        T *p = static_cast<T *>(a.out) + (r.row - lane + (lane >> 4)) * a.ldo + w.tn * kTileN + c0 + col;
#pragma unroll 1
        for (int q = lane >> 4; q < 32 && q < rows && col < left; q += 2, p += 2 * a.ldo)
            put(p, staging[q * kStageRow + (lane & 15)]);
    }
}

template <int MODE, int PLANES, bool ANY>
__device__ __forceinline__ void block(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32], float *staging) {
    using T = std::conditional_t<PLANES == 1, __nv_bfloat16, float>;
    if constexpr (MODE == LOGITS) block_logits(r, a, w, c0, v);
    else if constexpr (MODE == PROBS) block_probs<PLANES>(r, a, w, c0, v);
    else if constexpr (MODE == DH) block_dh(r, a, w, c0, v);
    else if constexpr (ANY) block_dw_any<T>(r, a, w, c0, v, staging);
    else block_dw<T>(r, a, w, c0, v);
}

template <int MODE>
__device__ __forceinline__ void end(const Row &r, const GemmArgs &a, const Work &w, int half) {
    if constexpr (MODE == LOGITS) {
        if (r.row < a.m) {
            a.part[r.row * a.part_ld + 2 * w.tn + half] = make_float2(r.top, r.sum);
            if (r.at >= half * kHalf && r.at < (half + 1) * kHalf) a.picked[r.row] = r.picked;
        }
    }
}

template <int MODE, int PLANES>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ GemmArgs a) {
    constexpr bool A_MN = MODE == DW, B_MN = MODE == DH || MODE == DW;
    constexpr bool SUMS = MODE == LOGITS || PLANES == 3;      // chunks are added in registers
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *const base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *const tiles_a = base, *const tiles_b = base + kStages * kBytesA;
    float *const staging = reinterpret_cast<float *>(base + kStages * (kBytesA + kBytesB));
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 1) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&acc_full[s], 1);
            tc::mbar_init(&acc_empty[s], 32 * kEpilogueWarps);
        }
        tc::mbar_init(&drained, 1);
        tc::mbar_fence_init();
        tc::tma_prefetch_map(&map_a);
        tc::tma_prefetch_map(&map_b);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const int total = a.tiles_m * a.tiles_n * a.splits;

    if (warp < 4) {
      tc::regs_dec<kRegsFew>();
      if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
                const Work k = work_of(w, a);
                const int m0 = k.tm * kTileM, n0 = k.tn * kTileN;
                const int kb0 = k.split * a.kb_per_split, kb1 = min(a.kblocks, kb0 + a.kb_per_split);
                const int groups_b = (cols_of(k.tn, a) + 63) >> 6;
                const uint32_t bytes = kBytesA + (B_MN ? groups_b * (kTileK * 128) : kBytesB);
                for (int c = kb0; ok && c < kb1; c += a.chunk)
                for (int pr = 0; ok && pr < a.pairs; ++pr) {
                    int pa, pb;
                    pair_of(pr, a.pairs, pa, pb);
                    for (int kb = c; kb < min(c + a.chunk, kb1); ++kb, ++it) {
                        const uint32_t s = it % kStages;
                        if (!tc::mbar_wait(&empty[s], (it / kStages & 1) ^ 1, kPolls)) {
                            ok = false;
                            break;
                        }
                        tc::mbar_expect_tx(&full[s], bytes);
                        unsigned char *const da = tiles_a + s * kBytesA, *const db = tiles_b + s * kBytesB;
                        if constexpr (A_MN) {
                            for (int j = 0; j < kTileM / 64; ++j)
                                tc::tma_load_3d(da + j * kTileK * 128, &map_a, &full[s], m0 + 64 * j, kb * kTileK, pa);
                        } else {
                            tc::tma_load_3d(da, &map_a, &full[s], kb * kTileK, m0, pa);
                        }
                        if constexpr (B_MN) {
                            for (int j = 0; j < groups_b; ++j)
                                tc::tma_load_3d(db + j * kTileK * 128, &map_b, &full[s], n0 + 64 * j, kb * kTileK, pb);
                        } else {
                            tc::tma_load_3d(db, &map_b, &full[s], kb * kTileK, n0, pb);
                        }
                    }
                }
            }
            if (!ok) {
                atomicExch(a.status, 2);
                for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                    tc::mbar_wait(&full[i % kStages], i / kStages & 1, kPolls);
            }
        }
      } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0, done = 0;
            bool ok = true;
            for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
                const Work k = work_of(w, a);
                const int kb0 = k.split * a.kb_per_split, kb1 = min(a.kblocks, kb0 + a.kb_per_split);
                const uint32_t idesc = tc::idesc_bf16(kTileM, cols_of(k.tn, a), A_MN, B_MN);
                for (int c = kb0; ok && c < kb1; c += a.chunk, ++done) {
                    const uint32_t acc = tmem + (done & 1) * kTileN;
                    if (!tc::mbar_wait(&acc_empty[done & 1], (done >> 1 & 1) ^ 1, kPolls)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const int steps = (min(c + a.chunk, kb1) - c) * a.pairs;
                    for (int i = 0; i < steps; ++i, ++it) {
                        const uint32_t s = it % kStages;
                        if (!tc::mbar_wait(&full[s], it / kStages & 1, kPolls)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t sa = tc::smem_u32(tiles_a + s * kBytesA), sb = tc::smem_u32(tiles_b + s * kBytesB);
                        const uint64_t da = A_MN ? tc::sdesc_mn_sw128(sa, kTileK * 128) : tc::sdesc_sw128(sa);
                        const uint64_t db = B_MN ? tc::sdesc_mn_sw128(sb, kTileK * 128) : tc::sdesc_sw128(sb);
#pragma unroll
                        for (int j = 0; j < kTileK / 16; ++j)   // 16 k: 32 bytes along a line, or 16 lines
                            tc::mma_f16(acc, da + j * (A_MN ? 2048 / 16 : 2), db + j * (B_MN ? 2048 / 16 : 2), idesc,
                                        i > 0 || j > 0);
                        tc::mma_commit(&empty[s]);
                    }
                    if (ok) tc::mma_commit(&acc_full[done & 1]);
                }
            }
            if (!ok) {
                atomicExch(a.status, 2);
                tc::mma_commit(&drained);
                tc::mbar_wait(&drained, 0, kPolls);
            }
        }
      }
    } else {
        tc::regs_inc<kRegsMany>();
        const int quad = warp & 3, half = (warp - 4) >> 2;  // a warp may read its quarter of the lanes
        float *const stage = staging + (warp - 4) * 32 * kStageRow;
        uint32_t done = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
            const Work k = work_of(w, a);
            const int cols = min(a.n - k.tn * kTileN, (half + 1) * kHalf);     // this warp's columns end there
            const int kb0 = k.split * a.kb_per_split, kb1 = min(a.kblocks, kb0 + a.kb_per_split);
            const bool any = MODE == DW && !(a.out_vec && cols == (half + 1) * kHalf);
            Row r;
            begin<MODE>(r, a, k, k.tm * kTileM + quad * 32 + lane);
            float v[SUMS ? kHalf / 32 : 1][32];
            if constexpr (SUMS) {
#pragma unroll
                for (int b = 0; b < kHalf / 32; ++b)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[b][i] = 0.f;
            }
#pragma unroll 1
            for (int c = kb0; c < kb1; c += a.chunk, ++done) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_full[done & 1], done >> 1 & 1, kPolls));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (done & 1) * kTileN + (static_cast<uint32_t>(quad * 32) << 16);
                if constexpr (SUMS) {
#pragma unroll
                    for (int b = 0; b < kHalf / 32; ++b) {
                        const int c0 = half * kHalf + 32 * b;
                        if (c0 < cols) {
                            float x[32];
                            tc::tmem_ld32(acc + c0, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[b][i] += x[i];
                        }
                    }
                } else {
#pragma unroll 1
                    for (int c0 = half * kHalf; c0 < cols; c0 += 32) {
                        __syncwarp();
                        tc::tmem_ld32(acc + c0, v[0]);
                        if (any) block<MODE, PLANES, true>(r, a, k, c0, v[0], stage);
                        else block<MODE, PLANES, false>(r, a, k, c0, v[0], stage);
                    }
                }
                __syncwarp();
                tc::fence_before_sync();
                tc::mbar_arrive(&acc_empty[done & 1]);
            }
            if (!ok) {
                if (lane == 0) atomicExch(a.status, 2);
                break;
            }
            if constexpr (SUMS) {
                if (any) {
#pragma unroll
                    for (int b = 0; b < kHalf / 32; ++b)
                        if (half * kHalf + 32 * b < cols) block<MODE, PLANES, true>(r, a, k, half * kHalf + 32 * b, v[b], stage);
                } else {
#pragma unroll
                    for (int b = 0; b < kHalf / 32; ++b)
                        if (half * kHalf + 32 * b < cols) block<MODE, PLANES, false>(r, a, k, half * kHalf + 32 * b, v[b], stage);
                }
                __syncwarp();
            }
            end<MODE>(r, a, k, half);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

}  // namespace xent
}  // namespace bl
