// pa_rope_write_kv: rotary positions applied to the queries and keys of new
// tokens, and the scatter write of the rotated K rows and the V rows into the
// block pool, in one pass over the projections' output.
//
// A pair (x, y) of a head becomes m (x cos a - y sin a, x sin a + y cos a) with
// a = position * frequency (rope.cuh).  The kernel is bound by HBM: every
// q, k and v element is read once and written once.  A CTA takes kTokens
// tokens; it first computes their cosines and sines into shared memory, one
// pair a thread, because all heads of a token share them (32 + 8 heads: one
// sincos for 40 uses), then its threads walk the tokens' head rows, two 16-byte
// vectors a thread: the two that hold the pairs of the half layout, or two
// neighbours of the interleaved one, so no lane needs another's values and a
// query may be rotated in place.  8192 tokens of 32 + 8 heads (201 MB): 35 us, 5.7
// TB/s, 84 % of the copy bandwidth; 1999 tokens of 64 + 8 heads into FP8 pages (78
// MB): 18 us, 4.3 TB/s.  ncu: DRAM 55 % of its peak, issue slots 57 % used, 39
// registers; two rows a thread in flight were slower (fewer warps), the first rows
// asked for before the angles are computed saved 2 us.
#include <cmath>

#include "host_common.h"
#include "rope.cuh"

namespace pa {

struct RopeWriteParams {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    int32_t q_heads, kv_heads, head_dim, block_size;
    int32_t log2_bp;                       // -1: not a power of two
    const uint64_t* turns;
    int32_t rot_dim, interleaved;
    float magnitude;
    const int64_t *positions, *slots;
    int32_t tokens;
    int64_t num_slots;
    void* q_out;
    void *k_pool, *v_pool;
    float *k_scale, *v_scale;
    int32_t* d_err;
};

constexpr int kRopeThreads = 256;

PA_DEVICE uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// One thread's share of a row: two vectors.
template <typename T>
struct Row {
    bool live, is_q, is_v;
    int t, head;          // token of the CTA, head of q or of the pool
    int64_t tok, slot;
    uint4 a, b;
};

// Turns the two vectors and stores them.  FP8 pools: the 8 units of a row are 8
// neighbouring lanes, which agree on the row's largest magnitude by shuffles.
template <typename T, bool FP8>
PA_DEVICE void finish_row(const RopeWriteParams& p, Row<T>& y, const float2* cs, int u, bool has_pairs, int va,
                          int vb) {
    constexpr int N = Vec16<T>::N;
    float fa[N], fb[N];
    const bool turn = y.live && !y.is_v && has_pairs;
    if (turn || FP8) {
        Vec16<T>::open(y.a, fa);
        Vec16<T>::open(y.b, fb);
    }
    if (turn) {
        rope_turn_vectors<T>(p.interleaved, cs, fa, fb);
        y.a = Vec16<T>::close(fa);
        y.b = Vec16<T>::close(fb);
    }
    float inv = 0.f, scale = 0.f;
    if (FP8) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) top = fmaxf(top, fmaxf(fabsf(fa[j]), fabsf(fb[j])));
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        scale = __fdiv_rn(top, 448.f);
        inv = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
    }
    if (!y.live) return;
    if (y.is_q) {
        uint4* dst = (uint4*)((T*)p.q_out + (y.tok * p.q_heads + y.head) * (int64_t)p.head_dim);
        dst[va] = y.a;
        dst[vb] = y.b;
        return;
    }
    if (y.slot < 0 || y.slot >= p.num_slots) {
        if (y.head == 0 && u == 0) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const int64_t blk = p.log2_bp >= 0 ? y.slot >> p.log2_bp : y.slot / p.block_size;
    const int64_t off = y.slot - blk * p.block_size;
    const int64_t row = (blk * p.kv_heads + y.head) * p.block_size + off;
    void* pool = y.is_v ? p.v_pool : p.k_pool;
    if (FP8) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[j] = e4m3_pair(__fmul_rn(fa[4 * j], inv), __fmul_rn(fa[4 * j + 1], inv)) |
                   e4m3_pair(__fmul_rn(fa[4 * j + 2], inv), __fmul_rn(fa[4 * j + 3], inv)) << 16;
            w[2 + j] = e4m3_pair(__fmul_rn(fb[4 * j], inv), __fmul_rn(fb[4 * j + 1], inv)) |
                       e4m3_pair(__fmul_rn(fb[4 * j + 2], inv), __fmul_rn(fb[4 * j + 3], inv)) << 16;
        }
        uint2* dst = (uint2*)((uint8_t*)pool + row * p.head_dim);
        dst[va] = make_uint2(w[0], w[1]);
        dst[vb] = make_uint2(w[2], w[3]);
        if (u == 0) (y.is_v ? p.v_scale : p.k_scale)[row] = scale;
    } else {
        uint4* dst = (uint4*)((T*)pool + row * p.head_dim);
        dst[va] = y.a;
        dst[vb] = y.b;
    }
}

// blockDim = (units of a row, rows at a time); a unit is two 16-byte vectors.
// kTokens tokens a CTA, one or two.  The kernel issues in over half of its cycles, so
// its loops have no division (block sizes that are no power of two apart).
template <typename T, bool FP8>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeWriteParams p,
                                                                  const int kTokens) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ float2 cs[];  // [kTokens][rot_dim / 2]
    griddep_wait();
    griddep_launch();
    const int pairs = p.rot_dim >> 1;
    const int t0 = blockIdx.x * kTokens;
    const int tokens = min(kTokens, p.tokens - t0);
    const int u = threadIdx.x;
    const int turning = p.rot_dim / (2 * N);  // units with pairs; the others are copied
    // vectors of this unit within a row, and its first pair
    const bool apart = u < turning && !p.interleaved;
    const int va = apart ? u : 2 * u, vb = apart ? u + turning : 2 * u + 1, pair = u * N;
    const int rows = p.q_heads + 2 * p.kv_heads;
    const int all = tokens * rows;
    auto load = [&](int r) {
        Row<T> y;
        y.live = r < all;
        y.t = y.live && r >= rows ? 1 : 0;
        const int h = y.live ? r - y.t * rows : 0;
        y.tok = t0 + y.t;
        y.is_q = h < p.q_heads;
        y.is_v = h >= p.q_heads + p.kv_heads;
        y.head = y.is_q ? h : h - p.q_heads - (y.is_v ? p.kv_heads : 0);
        const T* base = (const T*)(y.is_q ? p.q : y.is_v ? p.v : p.k);
        const int64_t stride = y.is_q ? p.q_stride : y.is_v ? p.v_stride : p.k_stride;
        const uint4* src = (const uint4*)(base + y.tok * stride + (int64_t)y.head * p.head_dim);
        y.a = y.b = make_uint4(0, 0, 0, 0);
        y.slot = 0;
        if (y.live) {
            y.a = src[va];
            y.b = src[vb];
            if (!y.is_q) y.slot = __ldg(p.slots + y.tok);
        }
        return y;
    };
    // the first rows are on their way while the angles are computed
    Row<T> y = load(threadIdx.y);
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    for (int i = tid; i < tokens * pairs; i += blockDim.x * blockDim.y) {
        const int t = i >= pairs ? 1 : 0, j = i - t * pairs;
        cs[i] = rope_angle(__ldg(p.turns + j), __ldg(p.positions + t0 + t), p.magnitude);
    }
    __syncthreads();
    // every lane of a warp makes the same number of rounds (the FP8 shuffles)
    for (int n = 0; n < all; n += blockDim.y) {
        if (n > 0) y = load(n + threadIdx.y);
        finish_row<T, FP8>(p, y, cs + y.t * pairs + pair, u, u < turning, va, vb);
    }
}

pa_status check_rope(const pa_rope* r) {
    if (r == nullptr || r->turns == nullptr) return PA_ERR_INVALID_ARG;
    if (r->rot_dim <= 0 || (r->rot_dim & 1)) return PA_ERR_INVALID_ARG;
    if (r->layout != PA_ROPE_HALF && r->layout != PA_ROPE_INTERLEAVED) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(r->magnitude)) return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_turns(const double* frequencies, int32_t n, uint64_t* turns) {
    if (n < 0 || (n > 0 && (!frequencies || !turns))) return PA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i)
        if (!std::isfinite(frequencies[i])) return PA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const double t = frequencies[i] / 6.283185307179586476925;
        double left = t - std::floor(t);
        if (left >= 1.0) left = 0.0;  // a tiny negative t rounds up to a whole turn
        turns[i] = (uint64_t)std::ldexp(left, 64);
    }
    return PA_OK;
}

extern "C" pa_status pa_rope_write_kv(const pa_kv_pool* pool, const pa_rope* rope, const void* q,
                                      int64_t q_stride, int32_t num_q_heads, const void* k_new,
                                      int64_t k_stride, const void* v_new, int64_t v_stride,
                                      const int64_t* positions, const int64_t* slot_mapping,
                                      int32_t num_tokens, void* q_out, int32_t* d_err,
                                      pa_stream_t stream) {
    pa_status st = check_pool(pool);
    if (st != PA_OK) return st;
    st = check_rope(rope);
    if (st != PA_OK) return st;
    if (num_tokens < 0 || num_q_heads < 0) return PA_ERR_INVALID_ARG;
    if (rope->rot_dim > pool->head_dim) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!k_new || !v_new || !positions || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out)) return PA_ERR_INVALID_ARG;
    const bool fp8 = pool->dtype == PA_DTYPE_FP8_E4M3, f32 = pool->dtype == PA_DTYPE_F32;
    const int N = f32 ? 4 : 8;  // elements of a 16-byte vector of the input type
    const int units = pool->head_dim / (2 * N);
    if (pool->head_dim % (2 * N) != 0 || rope->rot_dim % (2 * N) != 0 || units > 64)
        return PA_ERR_UNSUPPORTED;
    if (fp8 && pool->head_dim != 128) return PA_ERR_UNSUPPORTED;
    const int64_t kv_row = (int64_t)pool->num_kv_heads * pool->head_dim;
    const int64_t q_row = (int64_t)num_q_heads * pool->head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (num_q_heads > 0 && q_stride < q_row))
        return PA_ERR_INVALID_ARG;
    if (k_stride % N || v_stride % N || (num_q_heads > 0 && q_stride % N)) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(pool->k_pool) ||
        !aligned16(pool->v_pool))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) return PA_ERR_INVALID_ARG;
    if (q_row + 2 * kv_row > (int64_t)1 << 24) return PA_ERR_UNSUPPORTED;

    RopeWriteParams p;
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.head_dim = pool->head_dim;
    p.block_size = pool->block_size;
    p.log2_bp = is_pow2(pool->block_size) ? ilog2(pool->block_size) : -1;
    p.turns = rope->turns;
    p.rot_dim = rope->rot_dim;
    p.interleaved = rope->layout == PA_ROPE_INTERLEAVED;
    p.magnitude = rope->magnitude;
    p.positions = positions;
    p.slots = slot_mapping;
    p.tokens = num_tokens;
    p.num_slots = (int64_t)pool->num_blocks * pool->block_size;
    p.q_out = q_out;
    p.k_pool = pool->k_pool;
    p.v_pool = pool->v_pool;
    p.k_scale = (float*)pool->k_scale;
    p.v_scale = (float*)pool->v_scale;
    p.d_err = d_err;
    // tokens a CTA (8192 tokens of 32 + 8 heads: 41.0, 37.3, 39.3 us with 1, 2, 4); small
    // batches need the CTAs
    const int per = num_tokens >= 4 * device_sm_count() ? 2 : 1;
    const dim3 block((unsigned)units, (unsigned)(kRopeThreads / units));
    const size_t smem = (size_t)per * (rope->rot_dim / 2) * sizeof(float2);
    const dim3 grid((unsigned)((num_tokens + per - 1) / per));
    cudaError_t e;
    if (fp8)
        e = launch_pdl(rope_write_kernel<uint16_t, true>, grid, block, smem, (cudaStream_t)stream, p, per);
    else if (f32)
        e = launch_pdl(rope_write_kernel<float, false>, grid, block, smem, (cudaStream_t)stream, p, per);
    else
        e = launch_pdl(rope_write_kernel<uint16_t, false>, grid, block, smem, (cudaStream_t)stream, p, per);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PA_ERR_CUDA;
    }
    return launch_status();
}
