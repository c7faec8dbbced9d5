// Token scores: what follows the products of logits in bl_score.
//
//   logp_r = s_r,t(r) - lse_r,   entropy_r = -sum_v p_rv log p_rv,   the `top` largest of s_r, lowest index first
//
// Every part of a row (a tile's 128 columns, or a CTA's entries for few rows) leaves its maximum m, the sum S of
// exp(s - m) and the sum T of exp(s - m) (s - m). Joined, entropy = log S - T / S: neither term is negative, so
// that nothing cancels for a row that is sure of its token. (S is 1 and more and rounded to 24 bits: the entropies of such
// rows, as their losses, are exact to a few 2^-24, and -T / S, their larger part, to a relative 2^-18.)
//
// The alternatives come from the largest logits of 32-wide blocks: one of the `top` largest logits of a row lies
// in one of its `top` first blocks, in the order of (largest logit, lower index). Only those blocks' logits are
// read; the products keep a block's logits only where they may be among them (block_scores).
#pragma once

#include "xent_gemm.cuh"

namespace bl {
namespace xent {

constexpr int kMostTop = 32;                      // a warp holds a row's list, a lane each

// (value, index) as one whole number: the larger is the likelier, of equal values the one with the lower index.
// 0 stands for none.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
    const uint32_t order = static_cast<uint32_t>(in_order(__float_as_int(v + 0.f))) ^ 0x80000000u;     // -0 is +0
    return v != v ? 0ull : (static_cast<uint64_t>(order) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    return __int_as_float(in_order(static_cast<int32_t>(static_cast<uint32_t>(key >> 32) ^ 0x80000000u)));
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

// A warp's list, sorted: lane i holds the i-th. Every lane offers a key (0: none); `top` of the list count.
struct List {
    uint64_t mine, least;                         // least: the last that counts
    __device__ __forceinline__ void start(uint64_t key, int top) {
        mine = key;
        least = __shfl_sync(0xffffffffu, mine, top - 1);
    }
    __device__ __forceinline__ void offer(uint64_t key, int top) {
        const int lane = threadIdx.x & 31;
        uint32_t votes = __ballot_sync(0xffffffffu, key > least);
        while (votes) {
            const uint64_t k = __shfl_sync(0xffffffffu, key, __ffs(votes) - 1);
            votes &= votes - 1;
            if (k <= least) continue;
            const int at = __ffs(__ballot_sync(0xffffffffu, k > mine)) - 1;
            const uint64_t above = __shfl_up_sync(0xffffffffu, mine, 1);
            mine = lane > at ? above : lane == at ? k : mine;
            least = __shfl_sync(0xffffffffu, mine, top - 1);
        }
    }
};

// Sorted by all lanes of a warp, the largest in lane 0.
__device__ __forceinline__ uint64_t sorted(uint64_t key) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size / 2; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0);      // this lane keeps the larger one
            key = (key > other) == larger ? key : other;
        }
    return key;
}

// The `top` largest of many keys, by the WARPS warps that share a row.
//
// A floor first: of 32 interleaved sets of keys the `top`-th largest maximum, which `top` keys reach. Some 130 keys
// at most reach it where their order is anything but contrived (of n in random order 32 ln(32 / (32 - top)), for top =
// 20 that is 31); those are gathered in shared memory, and each finds its place by counting the larger ones. Where
// more than kGathered reach the floor, a warp keeps a sorted list instead. Inserting all keys one by one into such a list
// costs some 150 cycles for each that enters (one row of 1000 blocks, 20 alternatives: 48 us a call in place of 25).
constexpr int kGathered = 256;
struct Gather {
    uint64_t keys[kGathered], chosen[kMostTop], blocks[kMostTop], lanes[32];
    int count;
};
template <int WARPS>
__device__ __forceinline__ void row_sync() {
    if constexpr (WARPS == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;\n" ::"r"(1 + static_cast<int>(threadIdx.x) / (WARPS * 32)), "n"(WARPS * 32) : "memory");
}
// key(i) for i < n; `given`: a further key of this lane (0: none; first warp only). The result is g.chosen, 0 where there
// are fewer. floor: what `top` keys are known to reach, or 0.
template <int WARPS, typename F>
__device__ __forceinline__ void select(Gather &g, int64_t n, uint64_t given, int top, uint64_t floor, const F &key) {
    constexpr int HELD = 16, STEP = WARPS * 32;
    const int lane = threadIdx.x & 31, thread = threadIdx.x % STEP;
    // Keys are looked at twice; where a thread can hold its own they are read once.
    uint64_t k[HELD];
    const auto read = [&](int64_t i0) {
#pragma unroll
        for (int h = 0; h < HELD; ++h) k[h] = i0 + h * STEP < n ? key(i0 + h * STEP) : 0;
    };
    bool held = false;
    const auto each = [&](const auto &f) {
        for (int64_t i0 = thread; i0 - thread < n; i0 += STEP * HELD) {
            if (!held) read(i0);
#pragma unroll
            for (int h = 0; h < HELD; ++h) f(k[h]);
        }
        held = n <= STEP * HELD;
    };
    if (thread < 32) {
        g.chosen[lane] = 0;
        if (lane == 0) g.count = 0;
    }
    if (floor == 0) {
        uint64_t most = 0;
        each([&](uint64_t k) { most = k > most ? k : most; });
        if constexpr (WARPS > 1) {
            if (thread < 32) g.lanes[lane] = 0;
            row_sync<WARPS>();
            atomicMax(reinterpret_cast<unsigned long long *>(&g.lanes[lane]), static_cast<unsigned long long>(most));
            row_sync<WARPS>();
            most = g.lanes[lane];
        }
        floor = __shfl_sync(0xffffffffu, sorted(most), top - 1);
    }
    row_sync<WARPS>();
    const auto gather = [&](uint64_t k) {
        if (k != 0 && k >= floor) {
            const int at = atomicAdd(&g.count, 1);
            if (at < kGathered) g.keys[at] = k;
        }
    };
    each(gather);
    gather(given);
    row_sync<WARPS>();
    const int count = g.count;
    if (count <= kGathered) {
        for (int i = thread; i < count; i += STEP) {
            const uint64_t k = g.keys[i];
            int place = 0;
            for (int j = 0; j < count; ++j) place += g.keys[j] > k;
            if (place < top) g.chosen[place] = k;
        }
    } else if (thread < 32) {
        List list;
        list.start(0, top);
        list.offer(given, top);
        for (int64_t i0 = 0; i0 < n; i0 += 32) list.offer(i0 + lane < n ? key(i0 + lane) : 0, top);
        if (lane < top) g.chosen[lane] = list.mine;
    }
    row_sync<WARPS>();
}

// The largest logit of every 32, where the logits come from the kernel for few rows. A warp takes 32 blocks.
__global__ void __launch_bounds__(256) block_max_kernel(const float *logits, int64_t block_ld, int64_t vocab, int64_t groups,
                                                        int64_t all, float *block_max) {
    pdl_release();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (w >= all) return;
    const int64_t row = w / groups, first = (w - row * groups) * 32;             // the warp's first block
    const float *const p = logits + row * block_ld * 32;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t c = first * 32 + i * 128 + lane * 4;
        v[i] = c < block_ld * 32 ? *reinterpret_cast<const float4 *>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (c >= vocab) v[i].x = -INFINITY;
        if (c + 1 >= vocab) v[i].y = -INFINITY;
        if (c + 2 >= vocab) v[i].z = -INFINITY;
        if (c + 3 >= vocab) v[i].w = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float m = fmaxf(fmaxf(v[i].x, v[i].y), fmaxf(v[i].z, v[i].w));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int64_t block = first + i * 4 + lane / 8;
        if (lane % 8 == 0 && block < block_ld) block_max[row * block_ld + block] = m;
    }
}

// The floors of the rows start at minus infinity. (Words that fill a line up to slot_ld stay out of the way.)
__global__ void __launch_bounds__(256) slots_kernel(int32_t *slots, int64_t count, int top, int slot_ld) {
    pdl_release();
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < count) slots[i] = i % slot_ld < top ? kLowest : 0x7fffffff;
}

struct Scores {
    const int64_t *target;
    int64_t vocab;
    int rows;
    const int *place;             // each row's place among those that count; null: its own
    // alternatives, of the piece of the vocabulary that starts at v0
    int top;
    const float *block_max, *logits;
    int64_t block_ld, v0, n;
    uint64_t *best;               // [row][top]: the list so far, where there are several pieces
    bool first, last;
    // the last piece: what is left of the rows
    const float2 *part;
    const float *part_t, *picked;
    int64_t part_ld;
    const int32_t *flags;
    int flag_count;
    float *logp, *entropy, *lse, *top_logp;
    int64_t *top_id;
};

// WARPS warps share a row. With 1, 2, 4 and 8 calls of dim 256 take: 4096 rows of 250 blocks 66, 72, 85, 115 us; of 1000 blocks
// 216, 212, 224, 252; 1000 rows of 500 blocks 50, 47, 46, 53; (dim 2048) 4096 rows of 3126 blocks 1129, 1124, 1118, 1138.
template <int WARPS>
__global__ void __launch_bounds__(256) scores_kernel(const __grid_constant__ Scores a) {
    constexpr int ROWS = 8 / WARPS, HELD = 8;
    __shared__ Gather gathers[ROWS];
    pdl_release();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % WARPS;
    const int row = blockIdx.x * ROWS + warp / WARPS, top = a.top;
    const bool bad = a.last && __syncthreads_or(flags_seen(a.flags, a.flag_count)) != 0;
    int64_t j = -1;
    if (row < a.rows) j = a.place ? a.place[row] : has_target(a.target, row, a.vocab) ? row : -1;
    const bool counts = j >= 0;
    uint64_t likeliest = 0;                              // the lane's
    if (top > 0 && counts) {
        Gather &g = gathers[warp / WARPS];
        const uint64_t before = !a.first && share == 0 && lane < top ? a.best[j * top + lane] : 0;
        // Blocks, by their largest logits. What the list holds already comes first among equals and is no block: its
        // indices are below 32.
        const float *const most = a.block_max + j * a.block_ld, *const s = a.logits + j * a.block_ld * 32;
        select<WARPS>(g, (a.n + 31) / 32, before ? (before | 0xffffffffull) - lane : 0, top, 0,
                      [&](int64_t b) { return key_of(most[b], static_cast<uint32_t>(b) + 32); });
        if (share == 0) g.blocks[lane] = g.chosen[lane];
        row_sync<WARPS>();
        // their logits: as many as are wanted reach the last block's
        select<WARPS>(g, top * 32, before, top, g.blocks[top - 1] >> 32 << 32, [&](int64_t i) -> uint64_t {
            const uint64_t k = g.blocks[i >> 5];
            const int64_t at = (static_cast<int64_t>(index_of(k)) - 32) * 32 + (i & 31);
            return k && at >= 0 && at < a.n ? key_of(s[at], static_cast<uint32_t>(a.v0 + at)) : 0;
        });
        likeliest = g.chosen[lane];
        if (!a.last && share == 0 && lane < top) a.best[j * top + lane] = likeliest;
    }
    if (!a.last) return;
    // what is left of the row, by all of its warps
    __shared__ float tops[8], sums[8], sums_t[8];
    float logp = 0.f, entropy = 0.f, lse = 0.f, ref = 0.f, log_sum = 0.f;
    bool sound = false;
    if (counts) {
        constexpr int STEP = WARPS * 32;
        const int thread = threadIdx.x % STEP;
        const float2 *const p = a.part + j * a.part_ld;
        const float *const pt = a.part_t + j * a.part_ld;
        float2 v[HELD];
        float t[HELD];
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const bool in = thread + STEP * h < a.part_ld;
            v[h] = in ? p[thread + STEP * h] : make_float2(-INFINITY, 0.f);
            t[h] = in ? pt[thread + STEP * h] : 0.f;
        }
        const float picked = a.picked[j];
        float most = -INFINITY, sum = 0.f, sum_t = 0.f;
#pragma unroll
        for (int h = 0; h < HELD; ++h) most = fmaxf(most, v[h].x);
#pragma unroll 8
        for (int64_t i = thread + STEP * HELD; i < a.part_ld; i += STEP) most = fmaxf(most, p[i].x);
        most = warp_max(most);
        if constexpr (WARPS > 1) {
            if (lane == 0) tops[warp] = most;
            row_sync<WARPS>();
            for (int w = 0; w < WARPS; ++w) most = fmaxf(most, tops[warp - share + w]);
        }
        ref = most == -INFINITY ? 0.f : most;
        const auto add = [&](float2 x, float xt) {
            const float d = fmaxf(x.x - ref, -1e30f);
            sum += x.y * expf(x.x - ref);                    // an infinite logit makes NaN here
            sum_t += expf(d) * fmaf(d, x.y, xt);
        };
#pragma unroll
        for (int h = 0; h < HELD; ++h) add(v[h], t[h]);
#pragma unroll 8
        for (int64_t i = thread + STEP * HELD; i < a.part_ld; i += STEP) add(p[i], pt[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum_t += __shfl_xor_sync(0xffffffffu, sum_t, o);
        }
        if constexpr (WARPS > 1) {
            if (lane == 0) sums[warp] = sum, sums_t[warp] = sum_t;
            row_sync<WARPS>();
            sum = sum_t = 0.f;
            for (int w = 0; w < WARPS; ++w) sum += sums[warp - share + w], sum_t += sums_t[warp - share + w];
        }
        log_sum = logf(sum);
        sound = sum > 0.f && !bad;
        lse = sound ? ref + log_sum : NAN;
        // the difference of two logits first, as in the loss: lse has been rounded
        logp = sound ? (picked - ref) - log_sum : NAN;
        entropy = sound ? log_sum - sum_t / sum : NAN;
    }
    if (row >= a.rows || share != 0) return;
    if (lane == 0) {
        a.logp[row] = logp;
        a.entropy[row] = entropy;
        a.lse[row] = lse;
    }
    if (lane < top) {
        const bool there = sound && likeliest != 0;
        a.top_logp[static_cast<int64_t>(row) * top + lane] = there ? (value_of(likeliest) - ref) - log_sum : counts ? NAN : 0.f;
        a.top_id[static_cast<int64_t>(row) * top + lane] = there ? static_cast<int64_t>(index_of(likeliest)) : -1;
    }
}

}  // namespace xent
}  // namespace bl
