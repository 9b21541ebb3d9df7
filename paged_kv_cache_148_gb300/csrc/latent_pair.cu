// Latent attention for units of 65 to 128 query rows: a CTA pair a unit, on
// tcgen05's cta_group::2.
//
// Both CTAs hold 64 of the unit's rows.  Of a tile of 64 tokens each loads what the
// paired products take from it:
//   S [128 x 64]    = Q (A: own rows)  x K (B: own 32 tokens, the whole row),
//   O [128 x dims] += P (A: own rows)  x V (B: all tokens, a half of every 256 dims),
// 36 + 32 KB instead of the 72 KB of the one-CTA kernel, for twice the rows.  Rows
// stay lanes in both products: with M = 128 a CTA's 64 rows sit in lanes 0-63 with the
// first half of N, and again in lanes 64-127 with the second, so S takes 32 columns
// and O 128 for every 256 dims, and a row's maximum, sum and scale are its lanes' own.
//
// Roles (256 threads, one CTA per SM): warp 0 loads Q and K, warp 7 V; warps 1 and 6
// of the leader issue S and O; warps 2-5 are softmax and epilogue: a thread has one
// row and half of a tile's tokens.  K's barrier lies in the leader and counts both
// CTAs' bytes; V's is each CTA's own, and a CTA's P is only announced when its V is
// there too.  Products are released to both CTAs by multicast commits.
//
// What bounds it.  The MMAs of a tile take 36 x 25.5 + 8 x 64.5 = 1434 cycles for 128
// rows (S reads 3 KB of shared memory an MMA and SM; O runs at the tensor core's
// rate), 717 a CTA, where the one-CTA kernel takes 1920.  A tile takes about 1500
// with its operands in L2, and 6500 more stand between two units (the epilogue takes
// the softmax warps, Q has one buffer).  16 x 512 queries of 32 heads behind 2048
// tokens: 0.94 ms, 1.40 PFLOP/s, 75 % of the measured bf16 rate.  Decoding on 128 heads
// HBM's latency shows, with two slots a ring: eight contexts of 100K tokens 184 us, 74 %
// of the copy bandwidth.  K in two separately released parts was no faster (1060 us
// against 1035).
#include "latent.cuh"

namespace pa {
namespace lat {

namespace {

constexpr int kPairThreads = 256;
constexpr int kPairBars = 2048;
constexpr int kPairAhead = 3;        // tiles

template <int NJ>  // 256 dims each
struct PairLayout {
    static constexpr int kBlocks = 4 * NJ + 1;               // of 64 dims, the rotary one last
    static constexpr int kQBlock = 64 * 128;
    static constexpr int kP = kBlocks * kQBlock;
    static constexpr int kPBytes = 64 * 128;
    static constexpr int kK = kP + 2 * kPBytes;
    static constexpr int kKBytes = 32 * kBlocks * 128;       // [4 groups of 8 tokens][blocks][1024]
    static constexpr int kVBytes = 64 * NJ * 256;            // [8 groups][NJ][2][1024]
    static constexpr int kFit = (kSmemLimit - 1024 - kPairBars - kK) / (kKBytes + kVBytes);
    static constexpr int kSlots = kFit < 4 ? kFit : 4;
    static constexpr int kV = kK + kSlots * kKBytes;
    static constexpr int kBars = kV + kSlots * kVBytes;
    static constexpr int kBytes = kBars + kPairBars + 1024;
    static_assert(kSlots >= 2 && kBytes <= kSmemLimit, "two tiles fit");
};

struct PairBars {
    uint64_t q_full, q_empty, o_free;          // q_full, o_free, k_full, p_full: the leader's
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t info[kInfo], unit_info[kUnits];
    int32_t unit_tiles[kUnits];
    uint32_t valid[kInfo];                     // slices of a tile that were loaded, by tile
    uint32_t tmem_base;
    int32_t abort;
    float top[2][64], sum[2][64];              // a row's halves, exchanged
    Scan scan;
};
static_assert(sizeof(PairBars) <= kPairBars, "barrier area");

// One lane's slice of a tile: its page's row in the pool.
struct Slices {
    const Params& p;
    int log2_size, lane;                       // tokens of a slice: a page, at most 32

    PA_DEVICE int32_t fetch(const Part& w, const int32_t* table, int t) const {
        const int64_t pos = (int64_t)t * kTok + (lane << log2_size);
        if (lane >= (kTok >> log2_size) || t >= w.t1 || pos >= w.context) return INT32_MIN;
        const int64_t e = pos >> p.log2_bp;
        return e < p.max_blocks ? max(__ldg(table + e), -1) : p.num_blocks;
    }
    PA_DEVICE bool row(int32_t id, int t, int32_t* d_err, int& row) const {
        row = 0;
        if (id == INT32_MIN) return false;
        if (id < 0 || id >= p.num_blocks) {
            set_error(d_err, id < 0 ? PA_ERR_NEGATIVE_BLOCK : PA_ERR_OUT_OF_RANGE);
            return false;
        }
        row = (id << p.log2_bp) + ((t * kTok + (lane << log2_size)) & ((1 << p.log2_bp) - 1));
        return true;
    }
};

template <int NJ>
__global__ void __launch_bounds__(kPairThreads, 1)
latent_pair_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const Params p) {
    using L = PairLayout<NJ>;
    constexpr int kDim = NJ * 256;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PairBars* bars = reinterpret_cast<PairBars*>(smem + L::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const int group = blockIdx.x >> 1;

    if (warp == 0) {
        if (lane < 4) {
            mbar_init(&bars->k_full[lane], 1);
            mbar_init(&bars->k_empty[lane], 1);
            mbar_init(&bars->v_full[lane], 1);
            mbar_init(&bars->v_empty[lane], 1);
        }
        if (lane < kInfo) mbar_init(&bars->info[lane], 1);
        if (lane < kUnits) mbar_init(&bars->unit_info[lane], 1);
        if (lane < 2) {
            mbar_init(&bars->s_full[lane], 1);
            mbar_init(&bars->p_full[lane], 8);
            mbar_init(&bars->pv_done[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&bars->q_full, 1);
            mbar_init(&bars->q_empty, 1);
            mbar_init(&bars->o_free, 8);       // softmax warps of both CTAs
            bars->abort = 0;
            tc::prefetch_tmap(&tmap_q);
            tc::prefetch_tmap(&tmap_k);
            tc::prefetch_tmap(&tmap_v);
        }
        fence_mbar_init();
        __syncwarp();
    }
    if (warp == 1) {
        tc::tmem_alloc2(&bars->tmem_base, 512);
        tc::tmem_relinquish2();
    }
    griddep_wait();
    griddep_launch();

    find_stretch<kPairThreads>(p, group, blockIdx.x == 0, bars->scan);
    tc::fence_before_sync();
    tc::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = bars->tmem_base;     // S of tile i: columns 32 (i mod 2) ..; O: 128 + 128 j ..

    if (warp == 0) {
        // ------------------------------------------------------------ Q and K
        const Slices sl{p, min(p.log2_bp, 5), lane};
        const int size = 1 << sl.log2_size;
        bool ok = true;
        uint32_t it = 0, q_n = 0;
        auto tell = [&](int unit, int tiles) {
            if (lane == 0) {
                bars->unit_tiles[unit % kUnits] = tiles;
                mbar_arrive(&bars->unit_info[unit % kUnits]);
            }
            __syncwarp();
        };
        Line line = bars->scan.line;
        Part w = bars->scan.part;
        const bool some = bars->scan.some;
        int unit = 0;
        for (; ok && (unit == 0 ? some : next_part(p, line, w)); ++unit) {
            const int32_t* table = p.tables + (int64_t)w.seq * p.max_blocks;
            auto load_q = [&] {
                if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&bars->q_full, 2 * L::kBlocks * L::kQBlock);
                __syncwarp();
                if (lane < L::kBlocks)
                    tc::tma2_load_2d(smem + lane * L::kQBlock, &tmap_q, lane * 64, w.row + 64 * (int)rank,
                                     tc::cluster_addr(&bars->q_full, 0));
                __syncwarp();
                ++q_n;
            };
            int32_t next = sl.fetch(w, table, w.t0);
            tell(unit, w.t1 - w.t0);
            if (unit == 0) load_q();
            if (lane == 0 && rank == 0) ask_next_q(p, line, w, 128, L::kBlocks * 128);
            __syncwarp();
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int32_t id = next;
                next = sl.fetch(w, table, t + 1);
                int row;
                const bool live = sl.row(id, t, p.d_err, row);
                const uint32_t mask = __ballot_sync(0xffffffffu, live);
                const int slot = it % L::kSlots;
                if (it >= (uint32_t)L::kSlots &&
                    !(ok = wait_warp(&bars->k_empty[slot], (it / L::kSlots - 1) & 1, bars, p.d_err)))
                    break;
                if (lane == 0) {
                    if (rank == 0) mbar_arrive_expect_tx(&bars->k_full[slot], __popc(mask) * size * L::kBlocks * 128);
                    bars->valid[it % kInfo] = mask;
                    mbar_arrive(&bars->info[it % kInfo]);
                }
                __syncwarp();
                const int tok = lane << sl.log2_size;
                if (live && (uint32_t)(tok >> 5) == rank)
                    tc::tma2_load_4d(smem + L::kK + slot * L::kKBytes + ((tok & 31) >> 3) * (L::kBlocks * 1024),
                                     &tmap_k, 0, 0, 0, row >> 3, tc::cluster_addr(&bars->k_full[slot], 0));
                if (t == w.t0 && unit > 0) {  // Q behind the unit's first tile: it waits for the unit before
                    if (!(ok = wait_warp(&bars->q_empty, (unit - 1) & 1, bars, p.d_err))) break;
                    load_q();
                }
            }
        }
        if (ok) tell(unit, 0);
        __syncwarp();
        if (!ok && rank == 0) {  // a wait ran out: no copy may still be on its way when the CTAs end
            for (uint32_t n = it - min(it, (uint32_t)L::kSlots); n < it; ++n)
                mbar_wait(&bars->k_full[n % L::kSlots], (n / L::kSlots) & 1, p.d_err);
            if (q_n > 0) mbar_wait(&bars->q_full, (q_n - 1) & 1, p.d_err);
        }
    } else if (warp == 7) {
        // ------------------------------------------------------------ V
        const Slices sl{p, min(p.log2_bp, 5), lane};
        const int size = 1 << sl.log2_size;
        bool ok = true;
        uint32_t it = 0;
        Line line = bars->scan.line;
        Part w = bars->scan.part;
        const bool some = bars->scan.some;
        for (int unit = 0; ok && (unit == 0 ? some : next_part(p, line, w)); ++unit) {
            const int32_t* table = p.tables + (int64_t)w.seq * p.max_blocks;
            int32_t next = sl.fetch(w, table, w.t0), ahead = sl.fetch(w, table, w.t0 + kPairAhead);
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int32_t id = next, far = ahead;
                next = sl.fetch(w, table, t + 1);
                ahead = sl.fetch(w, table, t + kPairAhead + 1);
                int row;
                const bool live = sl.row(id, t, nullptr, row);
                const uint32_t mask = __ballot_sync(0xffffffffu, live);
                const int slot = it % L::kSlots;
                if (it >= (uint32_t)L::kSlots &&
                    !(ok = wait_warp(&bars->v_empty[slot], (it / L::kSlots - 1) & 1, bars, p.d_err)))
                    break;
                if (lane == 0) mbar_arrive_expect_tx(&bars->v_full[slot], __popc(mask) * size * NJ * 256);
                __syncwarp();
                if (live)
                    tc::tma2_load_5d(smem + L::kV + slot * L::kVBytes + ((lane << sl.log2_size) >> 3) * (NJ * 2048),
                                     &tmap_v, 0, 0, 2 * (int)rank, 0, row >> 3,
                                     tc::cluster_addr(&bars->v_full[slot], rank));
                if (sl.row(far, t + kPairAhead, nullptr, row) && (uint32_t)((lane << sl.log2_size) >> 5) == rank)
                    ask_rows(p, row, size, L::kBlocks * 128);
                __syncwarp();
            }
        }
        __syncwarp();
        if (!ok)
            for (uint32_t n = it - min(it, (uint32_t)L::kSlots); n < it; ++n)
                mbar_wait(&bars->v_full[n % L::kSlots], (n / L::kSlots) & 1, p.d_err);
    } else if (warp == 1) {
        // ------------------------------------------------------------ S (leader)
        constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kTok, 0, 0);
        const uint64_t dq = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk = tc::smem_desc_sw128(smem_u32(smem + L::kK), 16, L::kBlocks * 1024);
        uint32_t slot = 0, phase = 0, it = 0;
        bool ok = rank == 0;
        for (int unit = 0; ok && (ok = wait_warp(&bars->unit_info[unit % kUnits], (unit / kUnits) & 1, bars, p.d_err)); ++unit) {
            const int n = __reduce_max_sync(0xffffffffu, *(volatile int32_t*)&bars->unit_tiles[unit % kUnits]);
            if (n == 0 || !(ok = wait_warp(&bars->q_full, unit & 1, bars, p.d_err))) break;
            for (int t = 0; t < n; ++t, ++it) {
                // the softmax of both CTAs has read this buffer's last tile
                if (it >= 2 && !(ok = wait_warp(&bars->p_full[it & 1], ((it >> 1) - 1) & 1, bars, p.d_err))) break;
                if (!(ok = wait_warp(&bars->k_full[slot], phase, bars, p.d_err))) break;
                tc::fence_after_sync();
                const uint32_t d = tmem + 32u * (it & 1);
                if (tc::elected()) {
                    const uint32_t a = (uint32_t)dq, b = (uint32_t)dk + slot * (L::kKBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4 * L::kBlocks; ++k)
                        tc::mma2_ss(d, a + (((k >> 2) * L::kQBlock + (k & 3) * 32) >> 4), dq >> 32,
                                    b + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), dk >> 32, idesc, k > 0 ? 1u : 0u);
                }
                __syncwarp();
                tc::commit2_warp(&bars->s_full[it & 1]);
                tc::commit2_warp(&bars->k_empty[slot]);
                if (t + 1 == n) tc::commit2_warp(&bars->q_empty);
                if (++slot == L::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------ O (leader)
        constexpr uint32_t idesc = tc::idesc_bf16_f32(128, 256, 0, 1);
        const uint64_t dp = tc::smem_desc_sw128(smem_u32(smem + L::kP), 16, 1024);
        const uint64_t dv = tc::smem_desc_sw128(smem_u32(smem + L::kV), 1024, NJ * 2048);
        uint32_t slot = 0, it = 0;
        bool ok = rank == 0;
        for (int unit = 0; ok && (ok = wait_warp(&bars->unit_info[unit % kUnits], (unit / kUnits) & 1, bars, p.d_err)); ++unit) {
            const int n = __reduce_max_sync(0xffffffffu, *(volatile int32_t*)&bars->unit_tiles[unit % kUnits]);
            if (n == 0) break;
            if (unit > 0 && !(ok = wait_warp(&bars->o_free, (unit - 1) & 1, bars, p.d_err))) break;
            for (int t = 0; t < n; ++t, ++it) {
                if (!(ok = wait_warp(&bars->p_full[it & 1], (it >> 1) & 1, bars, p.d_err))) break;
                tc::fence_after_sync();
                const uint32_t a = (uint32_t)dp + (it & 1) * (L::kPBytes >> 4);
                const uint32_t b = (uint32_t)dv + slot * (L::kVBytes >> 4);
                const uint32_t first = t > 0 ? 1u : 0u;
                if (tc::elected()) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma2_ss(tmem + 128 + 128 * j, a + (k * 32 >> 4), dp >> 32,
                                        b + ((j * 2048 + k * NJ * 4096) >> 4), dv >> 32, idesc, k > 0 ? 1u : first);
                }
                __syncwarp();
                tc::commit2_warp(&bars->pv_done[it & 1]);
                tc::commit2_warp(&bars->v_empty[slot]);
                if (++slot == L::kSlots) slot = 0;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3;                  // TMEM lanes 32 quarter ..
        const int half = quarter >> 1;                 // tokens 32 half .. of a tile, dims 128 half .. of 256
        const int tid = quarter * 32 + lane;
        const int r = (quarter & 1) * 32 + lane;       // row of this CTA
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const int log2_size = min(p.log2_bp, 5);
        const uint32_t all = 0xffffffffu >> (32 - (kTok >> log2_size));
        const uint32_t p_row = smem_u32(smem + L::kP) + r * 128;
        const uint32_t leader_p = tc::cluster_addr(&bars->p_full[0], 0);
        const uint32_t leader_o = tc::cluster_addr(&bars->o_free, 0);
        uint32_t it = 0;
        // every warp walks all tiles even after a wait ran out (named barriers have no
        // limit, so none may stay away)
        bool ok = true;
        int32_t chain_rows = 0, chain_row = 0, chain = 0;
        Line line = bars->scan.line;
        Part w = bars->scan.part;
        const bool some = bars->scan.some;
        const int64_t per = bars->scan.per;
        for (int unit = 0; unit == 0 ? some : next_part(p, line, w); ++unit) {
            const int ur = r + 64 * (int)rank;         // row of the unit
            const int lim = w.seen(p, ur), ctx = w.seen(p, w.rows - 1);  // tokens that this row sees, and the last
            float m = -INFINITY, l = 0.f;
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const uint32_t b = it & 1;
                ok &= wait_warp(&bars->info[it % kInfo], (it / kInfo) & 1, bars, p.d_err);
                ok &= wait_warp(&bars->s_full[b], (it >> 1) & 1, bars, p.d_err);
                tc::fence_after_sync();
                const int pos = t * kTok;
                const uint32_t valid = *(volatile uint32_t*)&bars->valid[it % kInfo];
                const bool whole = valid == all && pos + kTok <= ctx;
                uint32_t s[32];
                tc::tmem_ld32(tmem + 32 * b + lanes, s);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    s[e] = __float_as_uint(__uint_as_float(s[e]) * p.scale_log2);
                if (!whole || pos + kTok > lim) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = half * 32 + e;
                        if (pos + c >= lim || !((valid >> (c >> log2_size)) & 1)) s[e] = 0xff800000u;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool first = t == w.t0;
                const bool grow = m == -INFINITY ? top > -INFINITY : top > m + kRescale;
                if (first || named_any(1, grow)) {
                    // the row's two threads agree on its reference
                    bars->top[half][r] = top;
                    named_sync(2);
                    const float both = fmaxf(bars->top[0][r], bars->top[1][r]);
                    const float up = m == -INFINITY || both > m + kRescale ? both : m;
                    const float f = m == -INFINITY || m == up ? 1.f : ex2(m - up);
                    m = up;
                    l *= f;
                    if (__any_sync(0xffffffffu, f != 1.f)) {
                        ok &= wait_warp(&bars->pv_done[b ^ 1], ((it - 1) >> 1) & 1, bars, p.d_err);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < NJ * 128; c += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32(tmem + 128 + c + lanes, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::tmem_st32(tmem + 128 + c + lanes, o);
                        }
                        tc::tmem_wait_st();
                    }
                }
                const float u = m == -INFINITY ? 0.f : m;
                uint32_t pk[16];
                float ls[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    // P as bf16 (the operand type of the rows that it multiplies); the sums
                    // are of the rounded values, so the weights still add up to one
                    const uint32_t a = pack_bf16(ex2(__uint_as_float(s[e]) - u), ex2(__uint_as_float(s[e + 1]) - u));
                    ls[0] += bf16_lo(a);
                    ls[1] += bf16_hi(a);
                    pk[e >> 1] = a;
                }
                l += ls[0] + ls[1];
                // P's buffer was last read by the product two tiles ago
                if (it >= 2) ok &= wait_warp(&bars->pv_done[b], ((it >> 1) - 1) & 1, bars, p.d_err);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(p_row + b * L::kPBytes + (((half * 4 + i) ^ (r & 7)) << 4)), "r"(pk[4 * i]),
                                 "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3]) : "memory");
                ok &= wait_warp(&bars->v_full[it % L::kSlots], (it / L::kSlots) & 1, bars, p.d_err);
                if (!whole) {
                    // tokens behind the unit's last row, which nobody may have written, and those
                    // that were not loaded: their probability is zero, and so must their value
                    // be (zero times NaN is NaN)
                    const int tok = tid & 63;
                    if (pos + tok >= ctx || !((valid >> (tok >> log2_size)) & 1)) {
                        const uint32_t at = smem_u32(smem + L::kV) + (it % L::kSlots) * L::kVBytes +
                                            (tok >> 3) * (NJ * 2048) + (tok & 7) * 128;
                        for (int i = tid >> 6; i < 2 * NJ; i += 2)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                                             ::"r"(at + i * 1024 + (((c + tok) & 7) << 4)), "r"(0) : "memory");
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(leader_p + 8 * b);
            }
            // ---- the unit's end: O over l, or the part as it is
            const bool cut = w.t0 > 0 || w.t1 < w.tiles;
            const int64_t slot = (int64_t)group * 2 + (w.t0 > 0 ? 0 : 1);  // a stretch's first cut part, its last
            bars->sum[half][r] = l;
            named_sync(2);
            l = bars->sum[0][r] + bars->sum[1][r];
            const float inv = l > 0.f ? 1.f / l : 0.f;
            if (cut && half == 0) p.stats[slot * p.R + ur] = make_float2(m, l);
            if (cut && w.t0 == 0) {  // this stretch holds the unit's beginning: it names the parts
                chain = (int)((w.unit_at + w.tiles - 1) / per - group) + 1;
                chain_row = w.row;
                chain_rows = w.rows;
            }
            ok &= wait_warp(&bars->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, bars, p.d_err);
            tc::fence_after_sync();
            // a warp's 32 rows x 128 bytes at a time through its quarter of the P buffers
            // (their products are done), so that stores fill whole lines: a lane's own row
            // would be 32 pieces of 16 bytes a store
            const uint32_t stage = smem_u32(smem + L::kP) + quarter * 4096;
            const int base = 64 * (int)rank + (quarter & 1) * 32;  // unit row of the warp's first lane
            auto spill = [&](int e, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             ::"r"(stage + lane * 128 + ((e ^ (lane & 7)) << 4)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
            };
            auto drain = [&](char* dst, int64_t pitch) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + (lane >> 3);
                    uint4 x;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                 : "r"(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4)));
                    if (base + row < w.rows)
                        *reinterpret_cast<uint4*>(dst + row * pitch + (lane & 7) * 16) = x;
                }
                __syncwarp();
            };
            if (cut) {
#pragma unroll 1
                for (int c = 0; c < NJ * 128; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(tmem + 128 + c + lanes, o);
                    tc::tmem_wait_ld();
                    const int dim = (c >> 7) * 256 + half * 128 + (c & 127);
#pragma unroll
                    for (int e = 0; e < 8; ++e) spill(e, o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    drain((char*)(p.parts + (slot * p.R + base) * kDim + dim), kDim * 4);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < NJ * 128; c += 64) {
                    const int dim = (c >> 7) * 256 + half * 128 + (c & 127);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint32_t o[32];
                        tc::tmem_ld32(tmem + 128 + c + 32 * g + lanes, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[i] = pack_bf16(__uint_as_float(o[8 * e + 2 * i]) * inv,
                                                 __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                            spill(4 * g + e, x[0], x[1], x[2], x[3]);
                        }
                    }
                    drain((char*)(p.out + (int64_t)(w.row + base) * kDim + dim), kDim * 2);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster(leader_o);
        }
        if (tid == 0 && rank == 0) p.meta[group] = make_int4(ok ? chain : 0, chain_row, chain_rows, 0);
    }
    // neither CTA ends, or gives up its TMEM, before the other's products, arrivals and
    // loads that reach into it are done
    __syncwarp();
    tc::fence_before_sync();
    tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc2(tmem, 512);
    }
}

template <int NJ>
cudaError_t launch(const Params& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                   cudaStream_t stream) {
    constexpr int smem = PairLayout<NJ>::kBytes;
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= 64 || !attr_done[dev])) {
        e = cudaFuncSetAttribute(latent_pair_kernel<NJ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(latent_pair_kernel<NJ>, 2, dim3((unsigned)(2 * p.groups)), dim3(kPairThreads),
                              (size_t)smem, stream, mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_pair(const Params& p, const void* q, const pa_latent_pool* pool, int64_t q_rows,
                        cudaStream_t stream) {
    const uint64_t width = pool->latent_dim + pool->rope_dim, row = width * 2;
    const uint64_t rows = (uint64_t)pool->num_blocks * pool->block_size;
    const uint32_t size = pool->block_size < 32 ? pool->block_size : 32;
    CUtensorMap mq, mk, mv;
    const uint64_t qdims[2] = {width, (uint64_t)q_rows}, qstr[1] = {row};
    const uint32_t qbox[2] = {64, 64};
    // the pool as [rows / 8][blocks of 64][8][64], and its latent part with the blocks as
    // [256 dims][4 blocks], of which a CTA takes two of every four
    const uint64_t kdims[4] = {64, 8, width / 64, rows / 8}, kstr[3] = {row, 128, row * 8};
    const uint32_t kbox[4] = {64, 8, (uint32_t)(width / 64), size / 8};
    const uint64_t vdims[5] = {64, 8, 4, (uint64_t)pool->latent_dim / 256, rows / 8};
    const uint64_t vstr[4] = {row, 128, 512, row * 8};
    const uint32_t vbox[5] = {64, 8, 2, (uint32_t)pool->latent_dim / 256, size / 8};
    if (!encode_bf16_map_sw128(&mq, q, 2, qdims, qstr, qbox) ||
        !encode_bf16_map_sw128(&mk, pool->rows, 4, kdims, kstr, kbox) ||
        !encode_bf16_map_sw128(&mv, pool->rows, 5, vdims, vstr, vbox))
        return cudaErrorInvalidValue;
    return pool->latent_dim == 256 ? launch<1>(p, mq, mk, mv, stream) : launch<2>(p, mq, mk, mv, stream);
}

}  // namespace lat
}  // namespace pa
