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
// H is copied once per call, with the rows that have no target zeroed: what stands in such a row
// (NaN included) reaches no result, and the copy's rows start where TMA wants them. W is read in
// place if it is bf16 and its rows start on 16-byte boundaries; otherwise each piece is copied
// (f32: as planes) before its products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "host.h"
#include "xent_gemm.cuh"

namespace bl {
namespace xent {

// ------------------------------------------------------------------ elementwise kernels

__device__ __forceinline__ bool has_target(const int64_t *target, int64_t row, int64_t vocab) {
    return !target || (target[row] >= 0 && target[row] < vocab);
}

// Copy rows into bf16 planes of row length ldp (a multiple of 8; the tail is zero). Rows without
// a target become zero. Thread 0 also clears the call's status word.
template <typename T, int PLANES>
__global__ void __launch_bounds__(256)
    pack_kernel(const T *src, int64_t ld, int64_t rows, int dim, const int64_t *target, int64_t vocab,
                __nv_bfloat16 *dst, int64_t ldp, int64_t plane, int vec, int32_t *status) {
    if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const int64_t per_row = ldp / 8, all = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / per_row;
        const int c = static_cast<int>(i - row * per_row) * 8;
        const T *const s = src + row * ld + c;
        __align__(16) T x[8];
        if (!has_target(target, row, vocab)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = T(0.f);
        } else if (vec && c + 8 <= dim) {
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(x) / 16); ++j)
                reinterpret_cast<uint4 *>(x)[j] = reinterpret_cast<const uint4 *>(s)[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = c + j < dim ? s[j] : T(0.f);
        }
        __nv_bfloat16 *const d = dst + row * ldp + c;
        if constexpr (PLANES == 1) {
            *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(x);
        } else {
            float p[3][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(x[j], p[0][j], p[1][j], p[2][j]);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                *reinterpret_cast<uint4 *>(d + q * plane) = make_uint4(bf16x2(p[q][0], p[q][1]), bf16x2(p[q][2], p[q][3]),
                                                                       bf16x2(p[q][4], p[q][5]), bf16x2(p[q][6], p[q][7]));
        }
    }
}

// One warp a row: join the tiles' maxima and sums. A product that gave up makes every loss NaN.
__global__ void __launch_bounds__(256)
    loss_kernel(const float2 *part, int64_t part_ld, const float *picked, const int64_t *target, int64_t vocab,
                int rows, const int32_t *status, float *loss, float *lse) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= rows) return;
    float l = 0.f, v = 0.f;
    if (has_target(target, row, vocab)) {
        const float2 *const p = part + row * part_ld;
        float top = -INFINITY, sum = 0.f;
        for (int64_t i = lane; i < part_ld; i += 32) top = fmaxf(top, p[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -INFINITY ? 0.f : top;
        for (int64_t i = lane; i < part_ld; i += 32) sum += p[i].y * expf(p[i].x - ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        v = ref + logf(sum);
        l = v - picked[row];
    }
    if (*status != 0) l = v = NAN;
    if (lane == 0) {
        loss[row] = l;
        lse[row] = v;
    }
}

// dH from the parts' sums; rows without a target are zero. A product that gave up makes it NaN.
template <typename T>
__global__ void __launch_bounds__(256)
    dh_kernel(const float *part, int splits, int64_t ldo, const int64_t *target, int64_t vocab, int64_t rows, int dim,
              const int32_t *status, T *dh, int64_t ld) {
    const bool bad = *status != 0;
    const int64_t all = rows * dim;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / dim;
        const int c = static_cast<int>(i - row * dim);
        float v = 0.f;
        if (has_target(target, row, vocab))
            for (int s = 0; s < splits; ++s) v += part[(s * rows + row) * ldo + c];
        put(dh + row * ld + c, bad ? NAN : v);
    }
}

// ------------------------------------------------------------------ plan

// K is added in tensor memory over so many 64-deep steps at a time where the result is f32
constexpr int kChunkF32 = 4, kChunkLoss = 8, kWhole = 1 << 30;
constexpr int64_t kPieceBytes = int64_t(512) << 20;     // of P, and of a piece's copy of W

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t cdiv(int64_t v, int64_t by) { return (v + by - 1) / by; }

struct Plan {
    int planes, pairs;
    bool copy_w, grad;
    int64_t rows, dim, vocab;
    int64_t ldp;              // row length of the copies of H and W
    int64_t piece, pieces;    // vocabulary entries per piece
    int64_t part_ld;          // partial maxima and sums of a row: two per tile
    int splits;
    int64_t kb_per_split;     // 64-deep steps of one part of dH
    int64_t ldo;              // row length of dH's partial sums
    int64_t status, h, w, part, picked, p, dh, bytes;   // offsets into the workspace
};

Plan plan_for(int dtype, int64_t rows, int64_t dim, int64_t vocab, const void *W, int64_t ldw, bool grad, int sms) {
    Plan q{};
    q.planes = dtype == BL_F32 ? 3 : 1;
    q.pairs = dtype == BL_F32 ? 6 : 1;
    q.copy_w = dtype == BL_F32 || reinterpret_cast<uintptr_t>(W) % 16 != 0 || ldw % 8 != 0;
    q.grad = grad;
    q.rows = rows;
    q.dim = dim;
    q.vocab = vocab;
    q.ldp = up(dim, 8);
    // a piece: what keeps P and the copy of W within their size, but 4096 entries at least, so
    // that a piece's products fill the GPU; pieces of one size
    int64_t most = up(vocab, kTileN);
    if (grad) most = std::min(most, kPieceBytes / (rows * 2 * q.planes));
    if (q.copy_w) most = std::min(most, kPieceBytes / (q.ldp * 2 * q.planes));
    most = std::max<int64_t>(most / kTileN * kTileN, 4096);
    q.pieces = cdiv(vocab, most);
    q.piece = up(cdiv(vocab, q.pieces), kTileN);
    q.pieces = cdiv(vocab, q.piece);
    q.part_ld = 2 * cdiv(vocab, kTileN);
    // dH has few tiles and a long K axis (the piece): cut K until there is work for every SM
    const int64_t tiles = cdiv(rows, kTileM) * cdiv(dim, kTileN), kb = cdiv(std::min(q.piece, vocab), kTileK);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(sms / tiles, kb / 4));
    q.kb_per_split = cdiv(kb, splits);
    q.splits = static_cast<int>(cdiv(kb, q.kb_per_split));
    q.ldo = up(dim, 32);
    int64_t at = 256;
    auto take = [&](int64_t bytes) {
        const int64_t r = at;
        at += up(bytes, 256);
        return r;
    };
    q.status = 0;
    q.h = take(q.planes * rows * q.ldp * 2);
    if (q.copy_w) q.w = take(q.planes * std::min(q.piece, vocab) * q.ldp * 2);
    if (!grad) {
        q.part = take(rows * q.part_ld * 8);
        q.picked = take(rows * 4);
    } else {
        q.p = take(q.planes * rows * q.piece * 2);
        q.dh = take(q.splits * rows * q.ldo * 4);
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

// Planes of rows x inner bf16 values, copied in boxes of box_rows x 64 with the 128-byte swizzle;
// what lies outside reads as zero.
bool make_map(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t planes, int64_t ld, int64_t plane,
              int box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(plane * 2)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int PLANES>
cudaError_t launch_gemm(const CUtensorMap &ma, const CUtensorMap &mb, const GemmArgs &a, int sms, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(gemm_kernel<MODE, PLANES>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int64_t total = static_cast<int64_t>(a.tiles_m) * a.tiles_n * a.splits;
    gemm_kernel<MODE, PLANES><<<static_cast<unsigned>(std::min<int64_t>(total, sms)), kThreads, kSmem, s>>>(ma, mb, a);
    return cudaGetLastError();
}

template <typename T, int PLANES>
cudaError_t launch_pack(const void *src, int64_t ld, int64_t rows, int64_t dim, const int64_t *target, int64_t vocab,
                        void *dst, int64_t ldp, int64_t plane, int32_t *status, int sms, cudaStream_t s) {
    const int vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && ld * sizeof(T) % 16 == 0;
    const int64_t blocks = std::min<int64_t>(cdiv(rows * (ldp / 8), 256), static_cast<int64_t>(sms) * 8);
    pack_kernel<T, PLANES><<<static_cast<unsigned>(blocks), 256, 0, s>>>(
        static_cast<const T *>(src), ld, rows, static_cast<int>(dim), target, vocab, static_cast<__nv_bfloat16 *>(dst), ldp,
        plane, vec, status);
    return cudaGetLastError();
}

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
    int32_t *const status = reinterpret_cast<int32_t *>(c.ws + q.status);
    char *const hp = c.ws + q.h;
    const int64_t h_plane = c.rows * q.ldp, piece_w = std::min(q.piece, c.vocab), w_plane = piece_w * q.ldp;
    BL_TRY((launch_pack<T, PLANES>(c.H, c.ldh, c.rows, c.dim, c.target, c.vocab, hp, q.ldp, h_plane, status, c.sms, c.s)));
    CUtensorMap h_k, h_mn;
    BL_MAP(make_map(&h_k, hp, c.dim, c.rows, PLANES, q.ldp, h_plane, kTileM));
    BL_MAP(make_map(&h_mn, hp, c.dim, c.rows, PLANES, q.ldp, h_plane, kTileK));
    GemmArgs base{};
    base.status = status;
    base.pairs = q.pairs;
    base.target = c.target;
    base.vocab = c.vocab;
    base.splits = 1;
    base.chunk = PLANES == 3 ? kChunkF32 : kWhole;
    for (int64_t i = 0; i < q.pieces; ++i) {
        const int64_t v0 = i * q.piece, n = std::min(q.piece, c.vocab - v0);
        const char *const w_at = static_cast<const char *>(c.W) + v0 * c.ldw * static_cast<int64_t>(sizeof(T));
        const void *wp = w_at;
        int64_t ldw = c.ldw, wpl = ldw;                     // one plane in place: its stride is not used
        if (q.copy_w) {
            BL_TRY((launch_pack<T, PLANES>(w_at, c.ldw, n, c.dim, nullptr, 0, c.ws + q.w, q.ldp, w_plane, nullptr, c.sms, c.s)));
            wp = c.ws + q.w;
            ldw = q.ldp;
            wpl = w_plane;
        }
        CUtensorMap w_k;
        BL_MAP(make_map(&w_k, wp, c.dim, n, PLANES, ldw, wpl, kTileN));
        GemmArgs a = base;
        a.m = static_cast<int>(c.rows);
        a.n = static_cast<int>(n);
        a.kblocks = static_cast<int>(cdiv(c.dim, kTileK));
        a.kb_per_split = a.kblocks;
        a.tiles_m = static_cast<int>(cdiv(c.rows, kTileM));
        a.tiles_n = static_cast<int>(cdiv(n, kTileN));
        a.v0 = static_cast<int>(v0);
        if (!q.grad) {
            if (PLANES == 1) a.chunk = kChunkLoss;
            a.part = reinterpret_cast<float2 *>(c.ws + q.part) + 2 * (v0 / kTileN);
            a.part_ld = q.part_ld;
            a.picked = reinterpret_cast<float *>(c.ws + q.picked);
            BL_TRY((launch_gemm<LOGITS, PLANES>(h_k, w_k, a, c.sms, c.s)));
            continue;
        }
        char *const pp = c.ws + q.p;
        const int64_t p_plane = c.rows * q.piece;
        a.lse = c.lse_in;
        a.g = c.g;
        a.p = reinterpret_cast<__nv_bfloat16 *>(pp);
        a.ldp = q.piece;
        a.p_plane = p_plane;
        BL_TRY((launch_gemm<PROBS, PLANES>(h_k, w_k, a, c.sms, c.s)));
        if (c.dH) {
            CUtensorMap p_k, w_mn;
            BL_MAP(make_map(&p_k, pp, n, c.rows, PLANES, q.piece, p_plane, kTileM));
            BL_MAP(make_map(&w_mn, wp, c.dim, n, PLANES, ldw, wpl, kTileK));
            GemmArgs d = base;
            d.m = static_cast<int>(c.rows);
            d.n = static_cast<int>(c.dim);
            d.kblocks = static_cast<int>(cdiv(n, kTileK));
            // the last piece may be shorter: its parts shrink, and every part still has a step
            d.kb_per_split = static_cast<int>(i == 0 ? q.kb_per_split : cdiv(d.kblocks, q.splits));
            d.splits = static_cast<int>(cdiv(d.kblocks, d.kb_per_split));
            d.tiles_m = static_cast<int>(cdiv(c.rows, kTileM));
            d.tiles_n = static_cast<int>(cdiv(c.dim, kTileN));
            d.accumulate = i > 0;
            d.out = c.ws + q.dh;
            d.ldo = q.ldo;
            BL_TRY((launch_gemm<DH, PLANES>(p_k, w_mn, d, c.sms, c.s)));
        }
        if (c.dW) {
            CUtensorMap p_mn;
            BL_MAP(make_map(&p_mn, pp, n, c.rows, PLANES, q.piece, p_plane, kTileK));
            GemmArgs d = base;
            d.m = static_cast<int>(n);
            d.n = static_cast<int>(c.dim);
            d.kblocks = static_cast<int>(cdiv(c.rows, kTileK));
            d.kb_per_split = d.kblocks;
            d.tiles_m = static_cast<int>(cdiv(n, kTileM));
            d.tiles_n = static_cast<int>(cdiv(c.dim, kTileN));
            d.out = static_cast<char *>(c.dW) + v0 * c.lddw * static_cast<int64_t>(sizeof(T));
            d.ldo = c.lddw;
            d.out_vec = reinterpret_cast<uintptr_t>(c.dW) % 16 == 0 && c.lddw * static_cast<int64_t>(sizeof(T)) % 16 == 0;
            BL_TRY((launch_gemm<DW, PLANES>(p_mn, h_mn, d, c.sms, c.s)));
        }
    }
    if (!q.grad) {
        loss_kernel<<<static_cast<unsigned>(cdiv(c.rows, 8)), 256, 0, c.s>>>(
            reinterpret_cast<const float2 *>(c.ws + q.part), q.part_ld, reinterpret_cast<const float *>(c.ws + q.picked),
            c.target, c.vocab, static_cast<int>(c.rows), status, c.loss, c.lse);
        BL_TRY(cudaGetLastError());
    } else if (c.dH) {
        const int64_t blocks = std::min<int64_t>(cdiv(c.rows * c.dim, 256), static_cast<int64_t>(c.sms) * 8);
        dh_kernel<T><<<static_cast<unsigned>(blocks), 256, 0, c.s>>>(reinterpret_cast<const float *>(c.ws + q.dh), q.splits,
                                                                    q.ldo, c.target, c.vocab, c.rows, static_cast<int>(c.dim),
                                                                    status, static_cast<T *>(c.dH), c.lddh);
        BL_TRY(cudaGetLastError());
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
    const Plan q = plan_for(dtype, c.rows, c.dim, c.vocab, c.W, c.ldw, grad, c.sms);
    if (ws_bytes < q.bytes)
        return fail(BL_ERR_INVALID_ARGUMENT, "%s: workspace of %lld bytes is smaller than %lld", op, (long long)ws_bytes,
                    (long long)q.bytes);
    c.ws = static_cast<char *>(ws);
    c.s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == BL_F32 ? run<float, 3>(op, q, c) : run<__nv_bfloat16, 1>(op, q, c);
}

}  // namespace xent
}  // namespace bl

extern "C" {

int64_t bl_xent_workspace(bl_dtype dtype, int64_t rows, int64_t dim, int64_t vocab, const void *W, int64_t ldw, int grad) {
    using namespace bl::xent;
    bl::clear_error();
    if (check_shape("xent_workspace", dtype, rows, dim, vocab) != BL_SUCCESS) return -1;
    const int sms = bl::sm_count();
    if (sms <= 0) {
        bl::fail(BL_ERR_CUDA, "xent_workspace: cannot query the current CUDA device");
        return -1;
    }
    return plan_for(dtype, rows, dim, vocab, W, ldw, grad != 0, sms).bytes;
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

}  // extern "C"
