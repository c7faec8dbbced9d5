// The tensor-core products of the softmax cross entropy and of token scores, one persistent kernel for all:
//
//   LOGITS  s = H W^T           A = H (K-major), B = W (K-major); keeps max and sum of exp per tile
//   PROBS   s again, then       P = g (exp(s - lse) - onehot) as bf16 planes
//   DH      dH = P W            A = P (K-major), B = W (MN-major); f32 partial sums
//   DW      dW = P^T H          A = P (MN-major), B = H (MN-major); stored in W's type
//   SCORES  s as in LOGITS      keeps the entropy's sum per tile too, the largest logit of every 32, and the
//                               logits themselves where they may be among a row's likeliest (see score.cuh)
//   SPROBS  s as in PROBS       P = g (onehot - exp(x)) - e exp(x) (x + entropy), x = s - lse
//
// A CTA computes 128 x 256 tiles, or a pair of CTAs 256 x 256 tiles (CTAS = 2: each holds its 128
// rows of A and of the result and half of B, so B crosses shared memory once for 256 rows). One
// warp per operand streams 64-deep tiles into a ring of shared memory by TMA, one warp (of the
// pair's leader) issues tcgen05.mma (bf16 operands, f32 accumulators in tensor
// memory), and eight warps turn finished accumulators into the mode's output while the next tile's
// products already run: tensor memory holds two accumulators of 256 columns.
//
// f32 operands are three bf16 planes each, x = x0 + x1 + x2 (8 bits of the 24-bit mantissa in
// each), and six of the nine plane products are added, the ones above 2^-25 of the result,
// smallest first. That costs as much tensor time as three tf32 products and is closer to f32.
//
// The tensor cores' f32 accumulation cuts where f32 would round, so a long chain of products is
// biased towards zero: by about 2^-25 of the sum a step in these products, by up to 2^-23.4 where all terms have one
// sign (dW over 2^21 equal rows in one chain: 1.2e-2 low). Where the result is f32 (the logits; every
// product of f32 operands) the chain is cut into chunks of K, whose sums are added in registers. The loss and P
// cut theirs alike, so that both form the same logits: exp(s - lse) - 1 at the target of a row that is sure of it
// shows every difference (dim 4096, logits of 57, p = 0.9999: with P's chain uncut several times P's size).
// bf16 results are cut every 16384 of K, 1e-4 of the sum at most, where their own rounding is 4e-3.
// Measured at rows 1024, dim 1024, vocabulary 32000, f32: dH 9.6e-6 off without chunks, 4.2e-7 with
// chunks of 128 (9.2e-7 with 256, 2.5% faster); the bf16 loss of 4096 x 4096 x 16384 with chunks of 512,
// 1024, 2048 and none: 317, 301, 294, 291 us (of 1024, as here, 280 since the issuing warp works as a whole).
//
// What bounds it: the operands' way into shared memory. A bf16 stage brings 32 KB for the 512 cycles of
// its products, 64 bytes a cycle, and the tensor pipe is 87 to 94% busy (280 to 301 us for each of the
// products at 4096 x 4096 x 16384, 1,820 to 1,960 TFLOP/s); an f32 stage brings half of that a cycle, and
// the pipe is 93 to 96% busy. Then the power cap: back to back the clock falls from 1.9 to 1.65 GHz.
//
// P and the copies of H and W are stored in panels of 64 columns ([plane][panel][row][64]), so that
// every operand tile is one contiguous piece of memory in either direction of use.
//
// bf16 operands have P in one bf16 plane, or in two where few rows add up to little averaging of its roundings
// (PLANES = 2: LOGITS and PROBS take one plane of H and W, DH and DW two of P and one of the other operand).
//
// Every wait is bounded: a role that gives up marks its CTA's flag, waits (bounded) for its own
// copies and products in flight, and leaves; the others then run out of time too.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "pdl.cuh"
#include "tma_sm100.cuh"

namespace bl {
namespace xent {

enum Mode : int { LOGITS = 0, PROBS = 1, DH = 2, DW = 3, SCORES = 4, SPROBS = 5 };
__host__ __device__ constexpr bool forms_logits(int mode) { return mode == LOGITS || mode == SCORES; }
__host__ __device__ constexpr bool forms_p(int mode) { return mode == PROBS || mode == SPROBS; }

constexpr int kTileM = 128, kTileN = 256, kTileK = 64;          // rows are each CTA's
constexpr int kEpilogueWarps = 8, kHalf = kTileN / 2;           // two warps share 32 rows: 128 columns each
constexpr int kStageBytes = 32 * 128;                           // an epilogue warp's lines on their way out
// Operand ring of a CTA that is one of CTAS that share a tile: A whole, its part of B. A stage holds
// every plane of both, so that f32 operands cross the chip once for their six products (copied again
// for each product: 1024 x 1024 x 32000 1.12 ms a step instead of 1.03, 20 rows x 3918 x 3275 137 us
// instead of 86). A single CTA has room for the planes of 128 columns of B only.
template <int CTAS, int PLANES_A, int PLANES_B>
struct Ring {
    static constexpr int kTile = CTAS == 1 && PLANES_B == 3 ? kTileN / 2 : kTileN;     // columns of a tile, at most
    static constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTile / CTAS * kTileK * 2;     // of a plane
    static constexpr int kStageA = PLANES_A * kBytesA, kStageB = PLANES_B * kBytesB;
    static constexpr int kStages = PLANES_A == 3 ? 2 : PLANES_A == 2 ? 3 : CTAS == 1 ? 4 : 6;                // 192 KB
    static constexpr int kSmem = kStages * (kStageA + kStageB) + kEpilogueWarps * kStageBytes + 1024;
};
// Planes of a product's operands
__host__ __device__ constexpr int planes_a(int mode, int planes) { return planes == 3 || mode == DH || mode == DW ? planes : 1; }
__host__ __device__ constexpr int planes_b(int planes) { return planes == 3 ? 3 : 1; }
template <int MODE, int PLANES, int CTAS>
using RingOf = Ring<CTAS, planes_a(MODE, PLANES), planes_b(PLANES)>;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;             // producers, issuer (and an idle warp), epilogue
// 384 threads start with 168 registers each; the first four warps give most of theirs to the
// epilogue, whose rows hold 128 sums: 128 * 56 + 256 * 224 = 384 * 168.
constexpr int kRegsLaunch = 168, kRegsFew = 56, kRegsMany = 224;
static_assert(128 * kRegsFew + 32 * kEpilogueWarps * kRegsMany <= kThreads * kRegsLaunch, "more registers than the block has");
constexpr uint32_t kPolls = 1u << 22;
constexpr int kGroupM = 16;                                     // row tiles that share a column of B tiles
constexpr float kLog2e = 1.4426950408889634f;

// Where an operand's tile of 64 columns starts in its tensor map: x = column group * x, z = column
// group * z + plane * plane. Rows as they are stored: (64, 0, 1); panels: (0, 1, panels).
struct Columns {
    int x, z, plane;
};

struct GemmArgs {
    Columns ca, cb;
    int m, n;                  // rows and columns of the product (m: at most, see `kept`)
    int rows;                  // rows of H
    const int *kept;           // how many of them count (LOGITS, PROBS, DH: m; DW: K), parts; null: all
    const int *order;          // the rows that count, in order; null: every row in its place
    int kblocks;               // 64-deep steps of one pair of planes (DW: follows from `kept`)
    int chunk;                 // of them, how many are added in tensor memory before registers take over
    int tile_n, tiles_n;       // columns of a tile: 256, or 128 or 64 where tiles are few (LOGITS, PROBS)
    int parts;                 // DH: of the K axis, if every row counts (else kept[1])
    int accumulate;            // DH: add to the partial sums of earlier pieces
    int32_t *flags;            // one word per CTA: not 0 if it gave up
    // LOGITS, PROBS
    const int64_t *target;
    int64_t vocab;
    int v0;                    // first vocabulary entry of this piece
    float2 *part;              // LOGITS: [row][part_ld] max and sum
    int64_t part_ld;
    float *picked;             // LOGITS: the target's logit of each row
    const float *lse, *g;      // PROBS, SPROBS
    const float *entropy, *e;  // SPROBS
    // SCORES
    float *part_t;             // beside `part`: sum of exp(s - max) (s - max)
    int top;                   // alternatives wanted; 0: none of the following is looked at
    float *block_max, *logits; // [row][block_ld] largest logit of 32, [row][32 block_ld]
    int64_t block_ld;
    int32_t *slots;            // [row][slot_ld] the largest logit of each of `top` groups of tiles so far; or null
    int slot_ld;
    const float *unit;         // PROBS, DW: the scale of P, below
    int p_panels;              // of a plane of P
    void *out;                 // DW: the result, where its rows do not start on 16-byte boundaries
    int64_t ldo;
};

// The products of planes, smallest first: all where only A has several, six of nine for f32 operands.
__host__ __device__ constexpr int pairs_of(int pa, int pb) { return pb == 3 ? 6 : pa; }
__host__ __device__ constexpr int pair_a(int q, int pairs) {
    return pairs < 6 ? pairs - 1 - q : q == 1 ? 2 : q == 0 || q == 3 ? 1 : 0;
}
__host__ __device__ constexpr int pair_b(int q, int pairs) { return pairs < 6 ? 0 : q == 2 ? 2 : q == 0 || q == 4 ? 1 : 0; }

// DH has few tiles and a long K axis, so K is cut into parts that have partial sums of their own:
// as many as make the least of the rounds that the device needs, times a part's steps (and 4 to
// start), plus what writing and reading a part's sums costs; all in steps, the 0.27 us of a
// 128 x 256 x 64 product on one SM. Only the numbers that fill whole rounds are looked at.
// In 1024ths of a step.
__host__ __device__ inline int parts_of(int tiles, int kblocks, int pairs, int64_t result_bytes, int groups, int most) {
    int best = 1;
    int64_t least = 0;
    for (int rounds = 1; rounds <= 8; ++rounds) {
        int s = rounds * groups / tiles;
        s = s < 1 ? 1 : s > most ? most : s;
        const int64_t need = (tiles * s + groups - 1) / groups, steps = (kblocks + s - 1) / s * pairs + 4;
        const int64_t cost = need * steps * 1024 + s * (result_bytes >> 10);
        if (rounds == 1 || cost < least) best = s, least = cost;
    }
    const int per = (kblocks + best - 1) / best;
    return (kblocks + per - 1) / per;
}

// What depends on how many rows count. One row tile and one step of K remain where none does, so
// that P and dW become zero.
struct Shape {
    int m, tiles_m, kblocks, splits, kb_per_split, total;
};
// Rows of a part's partial sums: what the epilogue's warps, 32 rows each, store.
__host__ __device__ inline int part_rows(int kept) { return kept < 32 ? 32 : (kept + 31) & ~31; }
// How the first piece's K axis is cut into parts whose sums fit slab_rows; the others' likewise.
struct Cut {
    int ctas, dim, tile_n, first_kb, pairs, slab_rows, groups;
};
__host__ __device__ inline int parts_for(const Cut &q, int kept) {
    const int tile = q.ctas * kTileM, tall = kept < tile ? 1 : (kept + tile - 1) / tile;
    int most = q.slab_rows / part_rows(kept);
    const int longest = q.pairs > 1 ? q.first_kb : q.first_kb / 4;
    if (most > longest) most = longest;
    if (most < 1) most = 1;
    return parts_of(tall * ((q.dim + q.tile_n - 1) / q.tile_n), q.first_kb, q.pairs, static_cast<int64_t>(part_rows(kept)) * q.dim * 4,
                    q.groups, most);
}
template <int MODE, int CTAS>
__device__ __forceinline__ Shape shape_of(const GemmArgs &a) {
    const int kept = a.kept ? *a.kept : a.rows;
    Shape s;
    s.m = MODE == DW ? a.m : kept;
    s.tiles_m = max(1, (s.m + CTAS * kTileM - 1) / (CTAS * kTileM));
    s.kblocks = MODE == DW ? max(1, (kept + kTileK - 1) / kTileK) : a.kblocks;
    s.splits = 1;
    s.kb_per_split = s.kblocks;
    if constexpr (MODE == DH) {
        const int parts = a.kept ? a.kept[1] : a.parts;     // the first piece's; a shorter one has no more
        s.kb_per_split = (s.kblocks + parts - 1) / parts;
        s.splits = (s.kblocks + s.kb_per_split - 1) / s.kb_per_split;
    }
    s.total = s.tiles_m * a.tiles_n * s.splits;
    return s;
}

struct Work {
    int tm, tn, kb0, kb1, split;
};
__device__ __forceinline__ Work work_of(int w, const GemmArgs &a, const Shape &s) {
    Work r;
    const int tiles = s.tiles_m * a.tiles_n;
    r.split = w / tiles;
    w -= r.split * tiles;
    const int per = kGroupM * a.tiles_n, g = w / per;
    w -= g * per;
    const int rest = s.tiles_m - g * kGroupM, gm = rest < kGroupM ? rest : kGroupM;
    r.tn = w / gm;
    r.tm = g * kGroupM + (w - r.tn * gm);
    r.kb0 = r.split * s.kb_per_split;
    r.kb1 = min(s.kblocks, r.kb0 + s.kb_per_split);
    return r;
}
// Columns of the tile that the product has, rounded up to what one CTA can hold of them: 16, the
// instruction's granularity (a pair: 32), or for a pair's halves of an MN-major B whole groups of 64.
template <bool B_MN, int CTAS>
__device__ __forceinline__ int cols_of(int tn, const GemmArgs &a) {
    constexpr int UNIT = CTAS == 1 ? 16 : B_MN ? 128 : 32;
    const int left = min(a.n - tn * a.tile_n, a.tile_n);
    return (left + UNIT - 1) & ~(UNIT - 1);
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&t);
}

// x = x0 + x1 + x2 in bf16. A value that rounds past the largest bf16 is cut instead. NaN stays in x0
// alone. An infinity is its sign in x0 and itself in x2, the plane that meets the other operand's x0 only: in
// x0 it would meet that operand's x1 and x2 as well, which are mostly zero, and 0 * inf is NaN.
__device__ __forceinline__ void split3(float x, float &x0, float &x1, float &x2) {
    const bool fine = fabsf(x) <= 3.4028235e38f, infinite = isinf(x);
    x0 = __bfloat162float(__float2bfloat16_rn(x));
    if (isinf(x0)) x0 = infinite ? copysignf(1.f, x) : __bfloat162float(__float2bfloat16_rz(x));
    const float r = x - x0;
    x1 = fine ? __bfloat162float(__float2bfloat16_rn(r)) : 0.f;
    x2 = fine ? __bfloat162float(__float2bfloat16_rn(r - x1)) : infinite ? x : 0.f;
}

// P is kept in units of the largest |g| (SPROBS: or |e|) of a row that counts, and dH and dW are multiplied by it in f32
// at the end: where all rows weigh the same, as in a mean, g then rounds nothing. (P_rv is close to
// -g at the targets of unsure rows, so g's own rounding to bf16, up to 2^-8, would be the same for all of
// them: gradients of 1279 rows of equal weight were up to 3.1e-3 off, rounded to bf16 themselves 1.7e-3.)
__device__ __forceinline__ float unit_from(float most) { return most > 0.f && most < INFINITY ? most : 1.f; }
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// By all lanes of a warp, for rows in their places (at most a row tile).
__device__ __forceinline__ float unit_of_rows(const float *g, const float *e, const int64_t *target, int64_t vocab, int rows) {
    float m = 0.f;
    for (int r = threadIdx.x & 31; r < rows; r += 32)
        if (target[r] >= 0 && target[r] < vocab) m = fmaxf(m, e ? fmaxf(fabsf(g[r]), fabsf(e[r])) : fabsf(g[r]));
    return unit_from(warp_max(m));
}

// Floats in the order of whole numbers.
__host__ __device__ __forceinline__ int32_t in_order(int32_t bits) { return bits < 0 ? bits ^ 0x7fffffff : bits; }
constexpr int32_t kLowest = static_cast<int32_t>(0x807fffff);     // minus infinity's place

__device__ __forceinline__ bool has_target(const int64_t *target, int64_t row, int64_t vocab) {
    return !target || (target[row] >= 0 && target[row] < vocab);
}
// Whether any CTA of the call's products gave up: this thread's share of the flags.
__device__ __forceinline__ int flags_seen(const int32_t *flags, int count) {
    int bad = 0;
    for (int i = threadIdx.x; i < count; i += blockDim.x) bad |= flags[i];
    return bad;
}

// ---- epilogues. A warp owns 32 rows (a lane each) and 128 columns, in blocks of 32 columns.

struct Row {              // what an epilogue keeps of its row
    int row, m, at;       // row of the product, its rows; the target's column within this tile or -1
    int part_rows;        // DH
    bool counted;
    float top, sum, picked;    // LOGITS
    float t, floor;            // SCORES
    float4 blocks;             // largest logits of its blocks, the last one last
    float lse, g;              // PROBS
    float entropy, e;          // SPROBS
    float unit;                // PROBS, DW
};

template <int MODE>
__device__ __forceinline__ void begin(Row &r, const GemmArgs &a, const Shape &s, const Work &w, int row, unsigned char *stage) {
    r.row = row;
    r.m = s.m;
    if constexpr (MODE == DH) r.part_rows = part_rows(s.m);
    if constexpr (forms_logits(MODE) || forms_p(MODE)) {
        const int n0 = w.tn * a.tile_n;
        const int64_t src = row < s.m ? (a.order ? a.order[row] : row) : -1;
        const int64_t t = src >= 0 ? a.target[src] : -1, at = t - a.v0 - n0;
        r.counted = t >= 0 && t < a.vocab;
        r.at = r.counted && at >= 0 && at < min(a.n - n0, a.tile_n) ? static_cast<int>(at) : -1;
        r.top = -INFINITY;
        r.sum = r.picked = 0.f;
        if constexpr (MODE == SCORES) {
            r.t = 0.f;
            r.floor = -INFINITY;
            // the row's slots, on their way to shared memory while the products run
            if (a.top > 0 && a.slots && row < s.m) {
                const int32_t *const p = a.slots + static_cast<int64_t>(row) * a.slot_ld;
                for (int j = 0; j < a.slot_ld; j += 4) tc::copy16_async(stage + (threadIdx.x & 31) * 128 + 4 * j, p + j);
            }
        }
        if constexpr (forms_p(MODE)) {
            r.lse = r.counted ? a.lse[src] : 0.f;
            r.g = r.counted ? a.g[src] / r.unit : 0.f;
        }
        if constexpr (MODE == SPROBS) {
            r.entropy = r.counted ? a.entropy[src] : 0.f;
            r.e = r.counted ? a.e[src] / r.unit : 0.f;
        }
    }
}

// Columns c0 .. c0 + 31 of the tile; those past the product's edge hold anything.
__device__ __forceinline__ void block_logits(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
    const int left = a.n - w.tn * a.tile_n - c0;
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
    // The difference comes before the product: m * log2(e) overflows for logits near the type's lowest value
    // (a mask), and its rounding would move the sum by |m| 2^-24 against the exp(m) that it stands beside.
    const float ref = m == -INFINITY ? 0.f : m;               // a row of -inf: every term is 0
    r.sum *= exp2f((r.top - ref) * kLog2e);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = exp2f((v[i] - ref) * kLog2e);
    // pairwise: beside a sure row's 1 each addition may round 2^-24 of its loss away
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) v[i] += v[i + o];
    r.sum += v[0];
    r.top = m;
}

// As block_logits, with the entropy's sum. Where alternatives are wanted the block's largest logit is always
// kept, the logits only where one of them reaches the row's floor: the least of the largest logits of `top`
// groups of tiles, so that `top` logits at least are as large. What lies below is among no row's likeliest.
// The instructions count: with K of 256 the products are done long before the epilogue.
__device__ __forceinline__ void block_scores(Row &r, const GemmArgs &a, const Work &w, int c0, float (&v)[32]) {
    const int left = a.n - w.tn * a.tile_n - c0;
    if (left < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < left ? v[i] : -INFINITY;
    }
    const uint32_t hit = r.at >= c0 && r.at < c0 + 32 ? 1u << (r.at - c0) : 0u;
    if (hit) {                                       // seldom for any of a warp's rows
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (hit >> i & 1) r.picked = v[i];
    }
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(fmaxf(v[i], v[i + 8]), fmaxf(v[i + 16], v[i + 24]));
    const float most = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), fmaxf(fmaxf(m[4], m[5]), fmaxf(m[6], m[7])));
    if (a.top > 0 && r.row < r.m) {
        if (most >= r.floor) {
            float *const p = a.logits + (r.row * a.block_ld + (w.tn * a.tile_n + c0) / 32) * 32;
#pragma unroll
            for (int j = 0; j < 32; j += 8) tc::store8(p + j, v + j);
        }
    }
    r.blocks = make_float4(r.blocks.y, r.blocks.z, r.blocks.w, most);
    const float top = fmaxf(r.top, most), ref = top == -INFINITY ? 0.f : top;
    // Moving the reference by d: sum of e (x + d) = t + d sum, all times exp(d). Nothing is left of tiles whose
    // exponentials are 0, and an infinite d (no tile before) must not meet that 0.
    const float d = fmaxf(r.top - ref, -1e30f), scale = exp2f(d * kLog2e);
    float t[4] = {scale * fmaf(d, r.sum, r.t), 0.f, 0.f, 0.f};         // of one sign: the order matters little
    r.sum *= scale;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float at = v[i] - ref;
        v[i] = tc::ex2(at * kLog2e);
        t[i & 3] = fmaf(v[i], fmaxf(at, -1e30f), t[i & 3]);            // a logit of minus infinity: 0 times a finite number
    }
    // pairwise, as in block_logits
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) v[i] += v[i + o];
    r.sum += v[0];
    r.t = (t[0] + t[1]) + (t[2] + t[3]);
    r.top = top;
}
// The row's floor, from the slots that begin() asked for.
__device__ __forceinline__ void floor_of(Row &r, const GemmArgs &a, const unsigned char *stage) {
    if (a.top == 0 || !a.slots) return;
    tc::copies_wait();
    int32_t least = 0x7fffffff;
    for (int j = 0; j < a.slot_ld; j += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(stage + (threadIdx.x & 31) * 128 + 4 * j);
        least = min(min(least, min(q.x, q.y)), min(q.z, q.w));
    }
    if (r.row < r.m) r.floor = __int_as_float(in_order(least));
}

template <int MODE>
__device__ __forceinline__ void end(const Row &r, const GemmArgs &a, const Work &w, int half) {
    if constexpr (forms_logits(MODE)) {
        if (r.row < r.m) {
            a.part[r.row * a.part_ld + 2 * w.tn + half] = make_float2(r.top, r.sum);
            if (r.at >= half * kHalf && r.at < (half + 1) * kHalf) a.picked[r.row] = r.picked;
            if constexpr (MODE == SCORES) {
                a.part_t[r.row * a.part_ld + 2 * w.tn + half] = r.t;
                // the blocks of this part; its first one's place is a multiple of four in a row of whole fours
                const int first = w.tn * a.tile_n + half * kHalf;
                const int blocks = a.top > 0 ? (min(min(a.n - w.tn * a.tile_n, a.tile_n) - half * kHalf, kHalf) + 31) / 32 : 0;
                float *const most = a.block_max + r.row * a.block_ld + first / 32;
                if (blocks == 4) *reinterpret_cast<float4 *>(most) = r.blocks;
                if (blocks == 3) most[0] = r.blocks.y, most[1] = r.blocks.z, most[2] = r.blocks.w;
                if (blocks == 2) most[0] = r.blocks.z, most[1] = r.blocks.w;
                if (blocks == 1) most[0] = r.blocks.w;
                // parts in turn, those that have columns: a tile of 128 or 64 is one part (as two it left every other of an even
                // number of slots at minus infinity, and the floor with them: 128 f32 rows x 64 x 200000, 20 alternatives 166 us, 139 so)
                if (a.top > 0 && a.slots && r.top > r.floor)
                    atomicMax(a.slots + static_cast<int64_t>(r.row) * a.slot_ld + (a.tile_n > kHalf ? 2 * w.tn + half : w.tn) % a.top,
                              in_order(__float_as_int(r.top)));
            }
        }
    }
}

// Results leave through a warp's 4 KB of shared memory: 32 lines (a lane's row each) of 128 bytes,
// in the 128-byte swizzle, that one thread hands to TMA. Lines are stored whole whatever the
// lanes hold, and TMA drops what lies past the result's edges.
__device__ __forceinline__ void line_put(unsigned char *stage, int chunk, uint4 q) {
    const int lane = threadIdx.x & 31;
    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = q;
}
__device__ __forceinline__ void lines_free() {          // the last store has read its lines
    if ((threadIdx.x & 31) == 0) tc::bulk_wait_read_all();
    __syncwarp();
}
__device__ __forceinline__ void lines_store(const CUtensorMap *map, unsigned char *stage, int x, int y, int z, bool add) {
    tc::fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        tc::tma_store_3d(map, stage, x, y, z, add);
        tc::bulk_commit();
    }
}
__device__ __forceinline__ void put_bf16(unsigned char *stage, int c0, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        line_put(stage, (c0 & 32) / 8 + j, make_uint4(bf16x2(v[8 * j], v[8 * j + 1]), bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                                      bf16x2(v[8 * j + 4], v[8 * j + 5]), bf16x2(v[8 * j + 6], v[8 * j + 7])));
}

// DW, where the result's rows start off the 16-byte boundaries that TMA wants: the warp stores the
// lines itself, one row after the other.
template <typename T>
__device__ __forceinline__ void lines_copy(const GemmArgs &a, const unsigned char *stage, int row0, int col0) {
    constexpr int PER = 4 / sizeof(T);                  // values in a lane's word
    const int lane = threadIdx.x & 31, rows = min(32, a.m - row0), col = col0 + lane * PER;
    T *p = static_cast<T *>(a.out) + row0 * a.ldo + col;
    __syncwarp();
#pragma unroll 4
    for (int q = 0; q < rows; ++q, p += a.ldo) {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(stage + q * 128 + (((lane >> 2) ^ (q & 7)) << 4) + (lane & 3) * 4);
        if constexpr (PER == 1) {
            if (col < a.n) *p = __uint_as_float(x);
        } else {
            const __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162 *>(&x);
            if (col < a.n) p[0] = t.x;
            if (col + 1 < a.n) p[1] = t.y;
        }
    }
    __syncwarp();
}

// PROBS, DH and DW. `cols`: where this warp's columns of the tile end. A line holds two blocks of
// bf16 values or one of f32 values.
template <int MODE, int PLANES>
__device__ __forceinline__ void block_out(const Row &r, const GemmArgs &a, const Work &w, int c0, int cols, float (&v)[32],
                                          const CUtensorMap *map, unsigned char *stage) {
    const int n0 = w.tn * a.tile_n, row0 = r.row - (threadIdx.x & 31);
    if constexpr (MODE == SPROBS) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = v[i] - r.lse, e = PLANES == 3 ? expf(x) : exp2f(x * kLog2e);
            const float g = i == r.at - c0 ? e - 1.f : e;           // where p is near 1 the difference is what counts
            const float p = fmaf(r.e * e, fmaxf(x, -1e30f) + r.entropy, r.g * g);    // the floor as in block_scores
            v[i] = r.counted && n0 + c0 + i < a.n ? -p : 0.f;
        }
    }
    if constexpr (MODE == PROBS) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            // the difference first, as in block_logits; the bf16 form rounds the result to 8 or 16 bits anyway. What the
            // exponential is off by where it is near 1 (2^-22) is no more than what lse's own rounding leaves.
            float e = PLANES == 3 ? expf(v[i] - r.lse) : exp2f((v[i] - r.lse) * kLog2e);
            if (i == r.at - c0) e -= 1.f;
            v[i] = r.counted && n0 + c0 + i < a.n ? r.g * e : 0.f;      // panels are whole: zero to their end
        }
    }
    if constexpr (MODE == DW) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= r.unit;
    }
    // where the rows that count are copied together P has whole row tiles: dW multiplies their zeros
    const bool there = row0 < r.m || (forms_p(MODE) && a.kept != nullptr);
    if constexpr (MODE == DH || PLANES == 3 || (forms_p(MODE) && PLANES == 2)) {
        if constexpr (forms_p(MODE)) {
            // planes of 32 values: 64 bytes a line each
#pragma unroll
            for (int pl = 0; pl < PLANES; ++pl) {
                lines_free();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = __bfloat162float(__float2bfloat16_rn(v[8 * j + i]));
                        v[8 * j + i] -= x[i];
                    }
                    *reinterpret_cast<uint4 *>(stage + (threadIdx.x & 31) * 64 + ((j ^ ((threadIdx.x >> 1) & 3)) << 4)) =
                        make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
                }
                if (there) lines_store(map, stage, c0 & 32, row0, pl * a.p_panels + (n0 + c0) / 64, false);
            }
        } else {
            lines_free();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                line_put(stage, j, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                              __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
            if (MODE == DW && a.out) lines_copy<float>(a, stage, row0, n0 + c0);
            else if (there) lines_store(map, stage, n0 + c0, row0 + (MODE == DH ? w.split * r.part_rows : 0), 0, MODE == DH && a.accumulate);
        }
    } else {
        if ((c0 & 32) == 0) lines_free();
        put_bf16(stage, c0, v);
        if ((c0 & 32) || c0 + 32 >= cols) {
            if (MODE == DW && a.out) lines_copy<__nv_bfloat16>(a, stage, row0, n0 + (c0 & ~63));
            else if (there && forms_p(MODE)) lines_store(map, stage, 0, row0, (n0 + c0) / 64, false);
            else if (there) lines_store(map, stage, n0 + (c0 & ~63), row0, 0, false);
        }
    }
}

template <int MODE, int PLANES>
__device__ __forceinline__ void block(Row &r, const GemmArgs &a, const Work &w, int c0, int cols, float (&v)[32],
                                      const CUtensorMap *map, unsigned char *stage) {
    if constexpr (MODE == LOGITS) block_logits(r, a, w, c0, v);
    else if constexpr (MODE == SCORES) block_scores(r, a, w, c0, v);
    else block_out<MODE, PLANES>(r, a, w, c0, cols, v, map, stage);
}

template <int MODE, int PLANES, int CTAS>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_out, const __grid_constant__ GemmArgs a) {
    using R = RingOf<MODE, PLANES, CTAS>;
    constexpr int PA = planes_a(MODE, PLANES), PB = planes_b(PLANES), PAIRS = pairs_of(PA, PB);
    constexpr int kBytesA = R::kBytesA, kBytesB = R::kBytesB, kStageA = R::kStageA, kStageB = R::kStageB, kStages = R::kStages;
    constexpr bool A_MN = MODE == DW, B_MN = MODE == DH || MODE == DW;
    constexpr int BLOCKS = kHalf / 32;                        // a warp's columns
    // Chunks of K are added in registers. Where one chunk is all there is, the results of bf16 operands go out block
    // by block as they leave tensor memory instead.
    constexpr bool MAY_BE_DIRECT = !forms_logits(MODE) && PLANES != 3;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *const base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *const tiles_a = base, *const tiles_b = base + kStages * kStageA;
    unsigned char *const staging = base + kStages * (kStageA + kStageB);
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t rank = CTAS == 1 ? 0 : tc::cluster_rank();
    if (warp == 1) tc::tmem_take<CTAS>(&tmem_slot, 512);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&acc_full[s], 1);
            tc::mbar_init(&acc_empty[s], CTAS * kEpilogueWarps);
        }
        tc::mbar_init(&drained, 1);
        tc::mbar_fence_init();
        gave_up = 0;
        tc::tma_prefetch_map(&map_a);
        tc::tma_prefetch_map(&map_b);
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
        // Two producers, one for each operand, each a warp of which an elected lane issues (in a branch of one thread a copy takes
        // 100 to 200 cycles, and a stage's products 512: dH and dW of 4096 x 4096 x 16384 had the tensor pipe 85% busy,
        // and 92 so). The leader's first announces the bytes of both CTAs.
        {
            const Shape sh = shape_of<MODE, CTAS>(a);
            const bool for_a = warp == 0, announce = for_a && rank == 0;
            const uint32_t bar0 = CTAS == 1 ? tc::smem_u32(full) : tc::at_leader(full);
            uint32_t s = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int w = blockIdx.x / CTAS; ok && w < sh.total; w += gridDim.x / CTAS) {
                const Work k = work_of(w, a, sh);
                const int part = cols_of<B_MN, CTAS>(k.tn, a) / CTAS;       // this CTA's columns of B
                const int m0 = (k.tm * CTAS + rank) * kTileM, n0 = k.tn * a.tile_n + rank * part;
                const int groups_b = (part + 63) >> 6;
                const uint32_t bytes = CTAS * (PA * kBytesA + PB * (B_MN ? groups_b * (kTileK * 128) : a.tile_n / CTAS * 128));
                for (int kb = k.kb0; kb < k.kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], phase ^ 1, kPolls));
                    if (!ok) break;
                    const uint32_t bar = bar0 + 8 * s;
                    if (tc::elect()) {
                        if (announce) tc::mbar_expect_tx(&full[s], bytes);
#pragma unroll 1
                        for (int p = 0; p < (for_a ? PA : PB); ++p) {
                            if (for_a) {
                                unsigned char *const d = tiles_a + s * kStageA + p * kBytesA;
                                const int z = p * a.ca.plane;
                                if constexpr (A_MN) {
#pragma unroll
                                    for (int j = 0; j < kTileM / 64; ++j) {
                                        const int g = m0 / 64 + j;
                                        tc::tma_load_3d<CTAS>(d + j * kTileK * 128, &map_a, bar, g * a.ca.x, kb * kTileK, z + g * a.ca.z);
                                    }
                                } else {
                                    tc::tma_load_3d<CTAS>(d, &map_a, bar, kb * a.ca.x, m0, z + kb * a.ca.z);
                                }
                            } else {
                                unsigned char *const d = tiles_b + s * kStageB + p * kBytesB;
                                const int z = p * a.cb.plane;
                                if constexpr (B_MN) {
#pragma unroll 1
                                    for (int j = 0; j < groups_b; ++j) {
                                        const int g = n0 / 64 + j;
                                        tc::tma_load_3d<CTAS>(d + j * kTileK * 128, &map_b, bar, g * a.cb.x, kb * kTileK, z + g * a.cb.z);
                                    }
                                } else {
                                    tc::tma_load_3d<CTAS>(d, &map_b, bar, kb * a.cb.x, n0, z + kb * a.cb.z);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    issued = min(issued + 1, static_cast<uint32_t>(kStages));
                    if (++s == kStages) s = 0, phase ^= 1;
                }
            }
            if (!ok && lane == 0) {
                gave_up = 1;
                // the copies in flight: the last `issued` stages before s, oldest first
                for (uint32_t i = 0; rank == 0 && i < issued; ++i) {
                    const uint32_t t = s + kStages - issued + i;
                    tc::mbar_wait(&full[t % kStages], t >= kStages ? phase : phase ^ 1, kPolls);
                }
            }
        }
      } else if (warp == 1) {
        // The whole warp goes through the steps, so that what the products are issued with is known to be the same in all
        // lanes; an elected lane issues, in 40 cycles a product. (In a branch of one lane it took 115, and a stage's
        // four products with the look at its barrier longer than the 512 cycles that the products take.) A lane looks
        // at one stage's barrier, 150 cycles, so that all that is there is found at once.
        if (rank == 0) {
            const Shape sh = shape_of<MODE, CTAS>(a);
            const uint64_t da0 = A_MN ? tc::sdesc_mn_sw128(tc::smem_u32(tiles_a), kTileK * 128) : tc::sdesc_sw128(tc::smem_u32(tiles_a));
            const uint64_t db0 = B_MN ? tc::sdesc_mn_sw128(tc::smem_u32(tiles_b), kTileK * 128) : tc::sdesc_sw128(tc::smem_u32(tiles_b));
            uint32_t s = 0, phase = 0, done = 0, there = 0;
            bool ok = true;
            const auto look = [&] {                    // how many stages from s on are there
                const uint32_t t = s + lane, wrapped = t >= kStages;
                for (uint32_t i = 0; there == 0 && i < kPolls; ++i) {
                    const bool now = lane < kStages && tc::mbar_wait(&full[wrapped ? t - kStages : t], phase ^ wrapped, 1);
                    there = __ffs(~__ballot_sync(0xffffffffu, now)) - 1;
                }
                __syncwarp();
                return there > 0;
            };
            for (int w = blockIdx.x / CTAS; ok && w < sh.total; w += gridDim.x / CTAS) {
                const Work k = work_of(w, a, sh);
                const uint32_t idesc = tc::idesc_bf16(CTAS * kTileM, cols_of<B_MN, CTAS>(k.tn, a), A_MN, B_MN);
                for (int c = k.kb0; ok && c < k.kb1; c += a.chunk, ++done) {
                    const uint32_t acc = tmem + (done & 1) * kTileN;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_empty[done & 1], (done >> 1 & 1) ^ 1, kPolls));
                    if (!ok) break;
                    const int steps = min(c + a.chunk, k.kb1) - c;
                    for (int i = 0; i < steps; ++i) {
                        if (there == 0) ok = look();
                        if (!ok) break;
                        --there;
                        tc::fence_after_sync();
                        const uint64_t da = da0 + s * (kStageA >> 4), db = db0 + s * (kStageB >> 4);
                        if (tc::elect()) {
#pragma unroll
                            for (int q = 0; q < PAIRS; ++q) {
                                const int pa = pair_a(q, PAIRS), pb = pair_b(q, PAIRS);
#pragma unroll
                                for (int j = 0; j < kTileK / 16; ++j)   // 16 k: 32 bytes along a line, or 16 lines
                                    tc::mma_f16<CTAS>(acc, da + pa * (kBytesA >> 4) + j * (A_MN ? 2048 / 16 : 2),
                                                      db + pb * (kBytesB >> 4) + j * (B_MN ? 2048 / 16 : 2), idesc,
                                                      i > 0 || q > 0 || j > 0);
                            }
                            tc::mma_commit_all<CTAS>(&empty[s]);
                            if (i + 1 == steps) tc::mma_commit_all<CTAS>(&acc_full[done & 1]);
                        }
                        __syncwarp();
                        if (++s == kStages) s = 0, phase ^= 1;
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
        unsigned char *const stage = staging + (warp - 4) * kStageBytes;
        const Shape sh = shape_of<MODE, CTAS>(a);
        float unit = 1.f;
        if constexpr (forms_p(MODE) || MODE == DW) unit = *a.unit;
        // A warp's columns: half a tile's. (Parts of logits are a half of the widest tile each, whatever the tile.) With the
        // first half alone at work on tiles of 128 columns dW of 20 rows x 1130 x 67549 in f32 took 280 us.
        const int mine = MODE == DH || MODE == DW ? a.tile_n / 2 : kHalf, first = half * mine;
        uint32_t done = 0;
        bool ok = true;
        for (int w = blockIdx.x / CTAS; ok && w < sh.total; w += gridDim.x / CTAS) {
            const Work k = work_of(w, a, sh);
            int cols = min(a.n - k.tn * a.tile_n, a.tile_n);                   // this warp's columns end there
            if (forms_p(MODE)) cols = (cols + 63) & ~63;
            cols = min(cols, first + mine);
            Row r;
            r.unit = unit;
            begin<MODE>(r, a, sh, k, (k.tm * CTAS + rank) * kTileM + quad * 32 + lane, stage);
            const bool direct = MAY_BE_DIRECT && k.kb1 - k.kb0 <= a.chunk;
            float v[BLOCKS][32];
            if (!direct) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[b][i] = 0.f;
            }
#pragma unroll 1
            for (int c = k.kb0; c < k.kb1; c += a.chunk, ++done) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_full[done & 1], done >> 1 & 1, kPolls));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (done & 1) * kTileN + (static_cast<uint32_t>(quad * 32) << 16);
                if (direct) {
                    if constexpr (MAY_BE_DIRECT) {
#pragma unroll 1
                        for (int c0 = first; c0 < cols; c0 += 32) {
                            __syncwarp();
                            tc::tmem_ld32(acc + c0, v[0]);
                            block<MODE, PLANES>(r, a, k, c0, cols, v[0], &map_out, stage);
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        const int c0 = first + 32 * b;
                        if (c0 < cols) {
                            float x[32];
                            tc::tmem_ld32(acc + c0, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[b][i] += x[i];
                        }
                    }
                }
                __syncwarp();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 1) tc::mbar_arrive(&acc_empty[done & 1]);
                    else tc::mbar_arrive_at(tc::at_leader(&acc_empty[done & 1]));
                }
            }
            if (!ok) {
                if (lane == 0) gave_up = 1;
                break;
            }
            if (!direct) {
                if constexpr (MODE == SCORES) floor_of(r, a, stage);
                // One copy of the code for the four blocks, whose sums move up: a CTA with one tile fetches it
                // once, and fetching is what four copies cost (P of 64 rows x 2048 x 32000 32 us instead of
                // 28, the loss of 64 rows x 1024 x 32000 17.7 us instead of 17.0)
#pragma unroll 1
                for (int c0 = first; c0 < cols; c0 += 32) {
                    block<MODE, PLANES>(r, a, k, c0, cols, v[0], &map_out, stage);
#pragma unroll
                    for (int b = 0; b + 1 < BLOCKS; ++b)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[b][i] = v[b + 1][i];
                }
                __syncwarp();
            }
            end<MODE>(r, a, k, half);
        }
        if (!forms_logits(MODE) && lane == 0) tc::bulk_wait_all();
    }
    __syncwarp();
    tc::fence_before_sync();
    if constexpr (CTAS == 1) __syncthreads();
    else tc::cluster_sync();                 // nothing of the pair's is in flight towards either CTA
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_give<CTAS>(tmem, 512);
    if (threadIdx.x == 0) a.flags[blockIdx.x] = gave_up;
}

}  // namespace xent
}  // namespace bl
