// pa_decode_latent and pa_prefill_latent: attention over a latent pool in the
// absorbed form, on the 5th-generation tensor cores.
//
// A token's row is [latent | rotary key] and serves every head, as key whole and
// as value by its latent part:  s_j = scale * q . row_j,
// out = sum_j softmax(s)_j latent_j.
//
// One unit of work is up to 64 query rows (token, head) of one sequence against
// a stretch of its context in tiles of 64 tokens.  A staged tile is used twice
// from the same shared memory:
//   S   [64 rows x 64 tokens] = Q (A, K-major)  x tile (B, K-major),
//   O^T [dims x rows]        += tile^T (A, MN-major, 128 dims an MMA) x P^T (B, K-major).
// The second product is transposed because its accumulator then has one TMEM
// column a query row and 128 dims a lane block: 512 dims x 64 rows take 256
// columns and leave room for two S buffers, where O with rows as lanes would
// fill all 512.
//
// Roles (224 threads, one CTA per SM):
//   warp 0     TMA producer: Q of a unit; the tiles as boxes of one page (at most 64
//              tokens) through the block table, into a ring of parts and a ring
//              of rotary blocks (128-byte swizzle); asks for the tile ahead in L2.
//   warp 1     issues the MMAs of S, a part as it lands.
//   warp 6     issues the MMAs of O^T, a tile when its P is there.  Two issuers,
//              each waiting for its own operands: with one, either product waits
//              behind the other's (a tile's slots come free only behind its O^T,
//              so the loads of S then take turns with the tensor core).
//   warps 2-5  softmax of S (each warp 16 rows, a row over 4 lanes), base 2;
//              P as bf16 into shared memory; the epilogue.
//
// All units' tiles of a call form one line, cut into equal stretches, one a CTA.
// A unit whose tiles lie in one stretch is written at once; the parts of a cut
// one go to the workspace as (max, sum, unnormalised O) in float32, and a second
// kernel joins them.
//
// The running reference of a row's scores moves only when its maximum grew by
// more than 2^16 (bf16 has float32's range, so P loses nothing by it): the
// rescaling of O^T, which takes all four warps, is then rare.
//
// What bounds it.  The MMAs of a tile take 36 x 32 + 16 x 48 = 1920 cycles at 64 rows
// (M = 64 runs at half rate, N = 64 of M = 128 is bound by shared memory), HBM at its
// copy rate 3140: long contexts run near HBM's rate.  Eight contexts of 32K to 131K
// tokens on 64 heads (755 MB): 136 us, 5.5 TB/s, 82 % of the copy bandwidth (ncu: DRAM
// 1.01 x the algorithmic bytes, tensor pipe 48 % active); of 100K on 16 heads 149 us,
// 91 %.  Short calls are bound by the way to the first product, about 8000 cycles
// (lengths, table and rows are three loads that wait for one another, and all code is
// cold): one context of 700 tokens takes 14.6 us.
// On the way (us, the eight contexts above): one issuer 234, then 203 with offsets that
// are compile-time constants, 173 with O^T and S in the order of their operands, 157
// with two issuers, 149 without a search from unit to unit, 139 with the next tile in L2.
#include "latent.cuh"

namespace pa {
namespace lat {

constexpr int kThreads = 224;
constexpr int kBarBytes = 1536;
constexpr int kMaxParts = 12;        // ring slots
constexpr int kMaxRope = 2;

// Shared memory of a unit of up to R rows (a multiple of 16) and PAIRS x 128
// latent dims: Q | P (two) | rotary ring | ring of parts | barriers.  A part is C
// blocks of 64 dims of a tile, laid out [8 tokens][C][8 x 128 bytes]: one TMA box
// of a page brings all C (a box costs the TMA unit about 50 cycles whatever its
// size: a tile of 16-token pages took 2330 cycles with boxes of one block, 1000
// with four), and both products find a stride for the 8-token groups in it.
// The S product reads 64 rows of Q whatever R is: for R < 64 it reads on into what
// follows, whose values reach only rows of S that nobody uses.  The ring holds two
// tiles at least (S of the next tile goes before O^T of this one).
template <int PAIRS, int R>
struct Layout {
    static constexpr int C = PAIRS % 2 == 0 ? 4 : 2;
    static constexpr int kParts = 2 * PAIRS / C;             // of a tile
    static constexpr int kPart = C * kBlock;
    static constexpr int kP = (2 * PAIRS + 1) * R * 128;
    static constexpr int kPBytes = R * 128;
    static constexpr int kRope = kP + 2 * kPBytes;
    static constexpr int kRoom = kSmemLimit - 1024 - kBarBytes - kRope;
    static constexpr int kRopeSlots = (kRoom - 2 * kBlock) / kPart >= 2 * kParts ? 2 : 1;
    static constexpr int kRing = kRope + kRopeSlots * kBlock;
    static constexpr int kFit = (kRoom - kRopeSlots * kBlock) / kPart;
    static constexpr int kSlots = kFit < kMaxParts ? kFit : kMaxParts;
    static constexpr int kBars = kRing + kSlots * kPart;
    static constexpr int kBytes = kBars + kBarBytes + 1024;
    static_assert(kSlots >= 2 * kParts && kBytes <= kSmemLimit, "two tiles fit");
};

struct Bars {
    uint64_t q_full, q_empty, o_free;
    uint64_t part_full[kMaxParts], part_empty[kMaxParts];
    uint64_t rope_full[kMaxRope], rope_empty[kMaxRope];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint32_t tmem_base;
    int32_t abort;
    uint64_t info[kInfo], unit_info[kUnits];
    int32_t unit_tiles[kUnits];
    uint32_t valid[kInfo];           // pages of a tile that were loaded, by tile
    float factor[64];                // rescaling factors of the rows
    float inv[2][64];                // one over the rows' sums, by unit mod 2
    Scan scan;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier area");

// 16 lanes x 64 columns: thread t gets, for column group i of 8, rows t / 4 (regs
// 4i, 4i + 1) and t / 4 + 8 (4i + 2, 4i + 3), columns 8i + 2 (t % 4) and the next.
PA_DEVICE void tmem_ld_16x256_x8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
PA_DEVICE void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
PA_DEVICE void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
          "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
          "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int PAIRS, int R>
__global__ void __launch_bounds__(kThreads, 1)
latent_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_rows,
              const __grid_constant__ CUtensorMap tmap_rope, const Params p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using L = Layout<PAIRS, R>;
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kDim = PAIRS * 128;
    const int group = blockIdx.x;

    if (warp == 0) {
        if (lane < kMaxParts) {
            mbar_init(&bars->part_full[lane], 1);
            mbar_init(&bars->part_empty[lane], 1);
        }
        if (lane < kInfo) mbar_init(&bars->info[lane], 1);
        if (lane < kUnits) mbar_init(&bars->unit_info[lane], 1);
        if (lane < 2) {
            mbar_init(&bars->rope_full[lane], 1);
            mbar_init(&bars->rope_empty[lane], 1);
            mbar_init(&bars->s_full[lane], 1);
            mbar_init(&bars->p_full[lane], 128);
            mbar_init(&bars->pv_done[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&bars->q_full, 1);
            mbar_init(&bars->q_empty, 1);
            mbar_init(&bars->o_free, 128);
            bars->abort = 0;
            tc::prefetch_tmap(&tmap_q);
            tc::prefetch_tmap(&tmap_rows);
            tc::prefetch_tmap(&tmap_rope);
        }
        fence_mbar_init();
        __syncwarp();
    }
    if (warp == 1) {
        tc::tmem_alloc(&bars->tmem_base, 512);
        tc::tmem_relinquish();
    }
    griddep_wait();
    griddep_launch();

    find_stretch<kThreads>(p, group, blockIdx.x == 0, bars->scan);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = bars->tmem_base;

    const uint32_t tP = smem_u32(smem + L::kP);
    const uint32_t tRing = smem_u32(smem + L::kRing);
    // S of tile i in columns [64 (i mod 2), + 64); O^T of pair m in [128 + m R, + R)
    auto tS = [&](int64_t i) { return tmem + 64u * (uint32_t)(i & 1); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const int bp = 1 << p.log2_bp;
        const int box = min(bp, kTok);               // rows of one box
        const int pages = kTok / box;                // boxes of one tile
        bool ok = true;
        uint32_t part_n = 0, rope_n = 0, q_n = 0;    // loads issued so far
        uint32_t it = 0;
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
            auto fetch = [&](int t) -> int32_t {     // this lane's page of tile t; -1 past the end
                const int64_t pos = (int64_t)t * kTok + lane * box;
                if (lane >= pages || t >= w.t1 || pos >= w.context) return INT32_MIN;
                const int64_t e = pos >> p.log2_bp;
                return e < p.max_blocks ? max(__ldg(table + e), -1) : p.num_blocks;
            };
            auto load_q = [&] {
                if (lane == 0) mbar_arrive_expect_tx(&bars->q_full, (2 * PAIRS + 1) * R * 128);
                __syncwarp();
                if (lane <= 2 * PAIRS)
                    tc::tma_load_2d(smem + lane * R * 128, &tmap_q, lane * 64, w.row, &bars->q_full);
                __syncwarp();
                ++q_n;
            };
            int32_t next = fetch(w.t0);
            tell(unit, w.t1 - w.t0);
            if (unit == 0) load_q();
            if (lane == 0) ask_next_q(p, line, w, R, (kDim + p.rope_dim) * 2);
            __syncwarp();
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int32_t id = next;
                next = fetch(t + 1);
                bool live = id != INT32_MIN;
                if (live && (id < 0 || id >= p.num_blocks)) {
                    set_error(p.d_err, id < 0 ? PA_ERR_NEGATIVE_BLOCK : PA_ERR_OUT_OF_RANGE);
                    live = false;
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, live);
                const int row = live ? (id << p.log2_bp) + ((t * kTok + lane * box) & (bp - 1)) : 0;
                const uint32_t bytes = __popc(mask) * box * 128;
                for (int m = 0; m < L::kParts; ++m, ++part_n) {
                    const int slot = part_n % L::kSlots;
                    if (part_n >= (uint32_t)L::kSlots &&
                        !(ok = wait_warp(&bars->part_empty[slot], (part_n / L::kSlots - 1) & 1, bars, p.d_err)))
                        break;
                    uint64_t* bar = &bars->part_full[slot];
                    if (lane == 0) mbar_arrive_expect_tx(bar, L::C * bytes);
                    __syncwarp();
                    if (live)
                        tc::tma_load_4d(smem + L::kRing + slot * L::kPart + lane * box * (L::C * 128), &tmap_rows,
                                        0, 0, m * L::C, row >> 3, bar);
                }
                if (!ok) break;
                const int slot = rope_n % L::kRopeSlots;
                if (rope_n >= (uint32_t)L::kRopeSlots &&
                    !(ok = wait_warp(&bars->rope_empty[slot], (rope_n / L::kRopeSlots - 1) & 1, bars, p.d_err)))
                    break;
                uint64_t* bar = &bars->rope_full[slot];
                if (lane == 0) {
                    bars->valid[it % kInfo] = mask;
                    mbar_arrive(&bars->info[it % kInfo]);
                    mbar_arrive_expect_tx(bar, bytes);
                }
                __syncwarp();
                if (live)
                    tc::tma_load_2d(smem + L::kRope + slot * kBlock + lane * box * 128, &tmap_rope,
                                    kDim, row, bar);
                ++rope_n;
                if (next >= 0 && next < p.num_blocks)  // the next tile, which waits for its slots
                    ask_rows(p, (next << p.log2_bp) + (((t + 1) * kTok + lane * box) & (bp - 1)), box, (kDim + p.rope_dim) * 2);
                __syncwarp();
                if (t == w.t0 && unit > 0) {  // Q behind the unit's first tile: it waits for the unit before
                    if (!(ok = wait_warp(&bars->q_empty, (unit - 1) & 1, bars, p.d_err))) break;
                    load_q();
                }
            }
        }
        if (ok) tell(unit, 0);
        __syncwarp();
        if (!ok) {  // a wait ran out: no copy may still be on its way when the CTA ends
            for (uint32_t n = part_n - min(part_n, (uint32_t)L::kSlots); n < part_n; ++n)
                mbar_wait(&bars->part_full[n % L::kSlots], (n / L::kSlots) & 1, p.d_err);
            for (uint32_t n = rope_n - min(rope_n, (uint32_t)L::kRopeSlots); n < rope_n; ++n)
                mbar_wait(&bars->rope_full[n % L::kRopeSlots], (n / L::kRopeSlots) & 1, p.d_err);
            if (q_n > 0) mbar_wait(&bars->q_full, (q_n - 1) & 1, p.d_err);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ S
        constexpr uint32_t idesc = tc::idesc_bf16_f32(64, kTok, 0, 0);
        constexpr uint64_t q_block = (uint64_t)(R * 128) >> 4;
        const uint64_t dq = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk = tc::smem_desc_sw128(tRing, 16, L::C * 1024);
        const uint64_t dr = tc::smem_desc_sw128(smem_u32(smem + L::kRope), 16, 1024);
        const int rope_steps = p.rope_dim >> 4;
        uint32_t slot = 0, phase = 0, slot_r = 0, phase_r = 0, it = 0;
        bool ok = true;
        for (int unit = 0; ok && (ok = wait_warp(&bars->unit_info[unit % kUnits], (unit / kUnits) & 1, bars, p.d_err)); ++unit) {
            const int n = __reduce_max_sync(0xffffffffu, *(volatile int32_t*)&bars->unit_tiles[unit % kUnits]);
            if (n == 0 || !(ok = wait_warp(&bars->q_full, unit & 1, bars, p.d_err))) break;
            for (int t = 0; t < n; ++t, ++it) {
                // the softmax has read this buffer's last tile
                if (it >= 2 && !(ok = wait_warp(&bars->p_full[it & 1], ((it >> 1) - 1) & 1, bars, p.d_err))) break;
                const uint32_t d = tmem + 64u * (it & 1);
#pragma unroll
                for (int m = 0; m < L::kParts; ++m) {
                    if (!(ok = wait_warp(&bars->part_full[slot], phase, bars, p.d_err))) break;
                    tc::fence_after_sync();
                    const uint64_t b = dk + (uint64_t)(slot * (L::kPart >> 4));
                    const uint64_t a = dq + m * L::C * q_block;
#pragma unroll
                    for (int k = 0; k < 4 * L::C; ++k)
                        tc::mma_ss_warp(d, a + (k >> 2) * q_block + ((k & 3) * 32 >> 4),
                                        b + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc, m + k > 0 ? 1u : 0u);
                    if (++slot == L::kSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (!ok || !(ok = wait_warp(&bars->rope_full[slot_r], phase_r, bars, p.d_err))) break;
                tc::fence_after_sync();
                const uint64_t b = dr + (uint64_t)(slot_r * (kBlock >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < rope_steps)
                        tc::mma_ss_warp(d, dq + 2 * PAIRS * q_block + k * 2, b + k * 2, idesc, 1u);
                tc::commit_warp(&bars->s_full[it & 1]);
                tc::commit_warp(&bars->rope_empty[slot_r]);
                if (t + 1 == n) tc::commit_warp(&bars->q_empty);
                if (++slot_r == L::kRopeSlots) {
                    slot_r = 0;
                    phase_r ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------ O^T
        constexpr uint32_t idesc = tc::idesc_bf16_f32(128, R, 1, 0);
        const uint64_t dv = tc::smem_desc_sw128(tRing, 1024, L::C * 1024);
        const uint64_t dp = tc::smem_desc_sw128(tP, 16, 1024);
        uint32_t slot = 0, it = 0;
        bool ok = true;
        for (int unit = 0; ok && (ok = wait_warp(&bars->unit_info[unit % kUnits], (unit / kUnits) & 1, bars, p.d_err)); ++unit) {
            const int n = __reduce_max_sync(0xffffffffu, *(volatile int32_t*)&bars->unit_tiles[unit % kUnits]);
            if (n == 0) break;
            if (unit > 0 && !(ok = wait_warp(&bars->o_free, (unit - 1) & 1, bars, p.d_err))) break;
            for (int t = 0; t < n; ++t, ++it) {
                if (!(ok = wait_warp(&bars->p_full[it & 1], (it >> 1) & 1, bars, p.d_err))) break;
                tc::fence_after_sync();
                const uint64_t b = dp + (uint64_t)((it & 1) * (L::kPBytes >> 4));
                const uint32_t more = t > 0 ? 1u : 0u;
#pragma unroll
                for (int m = 0; m < PAIRS; ++m) {
                    constexpr int per = L::C / 2;                // pairs of a part
                    const uint64_t a = dv + (uint64_t)(slot * (L::kPart >> 4) + m % per * (2048 >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_ss_warp(tmem + 128 + m * R, a + (k * 2 * L::C * 1024 >> 4), b + (k * 32 >> 4), idesc,
                                        k > 0 ? 1u : more);
                    if (m % per == per - 1) {
                        tc::commit_warp(&bars->part_empty[slot]);
                        if (++slot == L::kSlots) slot = 0;
                    }
                }
                tc::commit_warp(&bars->pv_done[it & 1]);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3;                  // TMEM lanes 32 quarter ..
        const int tid = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const bool active = quarter * 16 < R;
        const int r0 = quarter * 16 + (lane >> 2), r1 = r0 + 8;
        const int log2_box = min(p.log2_bp, 6);
        int64_t it = 0;
        // every warp walks all tiles even after a wait ran out (named barriers have no
        // limit, so none may stay away)
        bool ok = true;
        int32_t chain_rows = 0, chain_row = 0, chain = 0;
        Line line = bars->scan.line;
        Part w = bars->scan.part;
        const bool some = bars->scan.some;
        const int64_t per = bars->scan.per;
        for (int unit = 0; unit == 0 ? some : next_part(p, line, w); ++unit) {
            const int lim0 = w.seen(p, r0), lim1 = w.seen(p, r1);  // tokens that the two rows see
            const int ctx = w.seen(p, w.rows - 1);                 // and the unit's last row
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int b = (int)(it & 1);
                ok &= wait_warp(&bars->info[it % kInfo], (it / kInfo) & 1, bars, p.d_err);
                ok &= wait_warp(&bars->s_full[b], (it >> 1) & 1, bars, p.d_err);
                tc::fence_after_sync();
                const int pos = t * kTok;
                const int boxes = kTok >> log2_box;
                const uint32_t valid = *(volatile uint32_t*)&bars->valid[it % kInfo];
                const bool whole = valid == (0xffffffffu >> (32 - boxes)) && pos + kTok <= ctx;
                uint32_t s[32];
                float t0 = -INFINITY, t1 = -INFINITY;
                bool grow = false;
                if (active) {
                    tmem_ld_16x256_x8(tS(it) + lanes, s);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        s[e] = __float_as_uint(__uint_as_float(s[e]) * p.scale_log2);
                    if (!whole || pos + kTok > min(lim0, lim1)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int c = (e >> 2) * 8 + (lane & 3) * 2 + (e & 1);
                            const int lim = (e & 2) ? lim1 : lim0;
                            if (pos + c >= lim || !((valid >> (c >> log2_box)) & 1)) s[e] = 0xff800000u;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        t0 = fmaxf(t0, fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
                        t1 = fmaxf(t1, fmaxf(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])));
                    }
#pragma unroll
                    for (int off = 1; off < 4; off <<= 1) {
                        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, off));
                        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, off));
                    }
                    if (m0 == -INFINITY) m0 = t0;
                    if (m1 == -INFINITY) m1 = t1;
                    grow = t0 > m0 + kRescale || t1 > m1 + kRescale;
                }
                if (t > w.t0 && named_any(1, grow)) {
                    // O^T columns and l of the rows whose reference moves
                    const float n0 = t0 > m0 + kRescale ? t0 : m0, n1 = t1 > m1 + kRescale ? t1 : m1;
                    const float f0 = m0 == n0 ? 1.f : ex2(m0 - n0), f1 = m1 == n1 ? 1.f : ex2(m1 - n1);
                    if (active && (lane & 3) == 0) {
                        bars->factor[r0] = f0;
                        bars->factor[r1] = f1;
                    }
                    if (active) {
                        l0 *= f0;
                        l1 *= f1;
                        m0 = n0;
                        m1 = n1;
                    }
                    ok &= wait_warp(&bars->pv_done[b ^ 1], ((it - 1) >> 1) & 1, bars, p.d_err);
                    tc::fence_after_sync();
                    named_sync(2);
#pragma unroll 1
                    for (int c = 0; c < PAIRS * R; c += 16) {
                        uint32_t o[16];
                        tmem_ld_x16(tmem + 128 + c + lanes, o);
                        tc::tmem_wait_ld();
                        const int h = c % R;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * bars->factor[h + e]);
                        tmem_st_x16(tmem + 128 + c + lanes, o);
                    }
                    tc::tmem_wait_st();
                }
                // P's buffer was last read by the product two tiles ago
                if (it >= 2) ok &= wait_warp(&bars->pv_done[b], ((it >> 1) - 1) & 1, bars, p.d_err);
                if (active) {
                    const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
                    const uint32_t dst = tP + b * L::kPBytes;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a0 = ex2(__uint_as_float(s[4 * i]) - u0);
                        const float a1 = ex2(__uint_as_float(s[4 * i + 1]) - u0);
                        const float c0 = ex2(__uint_as_float(s[4 * i + 2]) - u1);
                        const float c1 = ex2(__uint_as_float(s[4 * i + 3]) - u1);
                        // P as bf16 (the operand type of the tile that it multiplies); the
                        // sums are of the rounded values, so the weights still add up to one
                        const uint32_t a = pack_bf16(a0, a1), c = pack_bf16(c0, c1);
                        l0 += bf16_lo(a) + bf16_hi(a);
                        l1 += bf16_lo(c) + bf16_hi(c);
                        const uint32_t col = (uint32_t)((i ^ (r0 & 7)) * 16 + (lane & 3) * 4);
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + r0 * 128 + col), "r"(a) : "memory");
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + r1 * 128 + col), "r"(c) : "memory");
                    }
                }
                if (!whole) {
                    // tokens behind the unit's last row, which nobody may have written, and those
                    // that were not loaded: their probability is zero, and so must their value
                    // be (zero times NaN is NaN)
                    const int tok = tid & 63;
                    if (pos + tok >= ctx || !((valid >> (tok >> log2_box)) & 1)) {
                        for (int m = tid >> 6; m < 2 * PAIRS; m += 2) {
                            const uint32_t n = (uint32_t)(it * L::kParts + m / L::C);
                            const uint32_t at = tRing + (n % L::kSlots) * L::kPart + (tok >> 3) * (L::C * 1024) +
                                                m % L::C * 1024 + (tok & 7) * 128;
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                                             ::"r"(at + (((c + tok) & 7) << 4)), "r"(0) : "memory");
                        }
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                mbar_arrive(&bars->p_full[b]);
            }
            // ---- the unit's end: O^T over l, or the part as it is
            const bool cut = w.t0 > 0 || w.t1 < w.tiles;
            // a stretch's first cut part in slot 0, its last in slot 1
            const int which = w.t0 > 0 ? 0 : 1;
            const int64_t slot = (int64_t)group * 2 + which;
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, off);
                l1 += __shfl_xor_sync(0xffffffffu, l1, off);
            }
            float* inv = bars->inv[unit & 1];
            if (active && (lane & 3) == 0) {
                inv[r0] = cut ? 1.f : l0 > 0.f ? 1.f / l0 : 0.f;
                inv[r1] = cut ? 1.f : l1 > 0.f ? 1.f / l1 : 0.f;
                if (cut) {
                    p.stats[slot * R + r0] = make_float2(m0, l0);
                    p.stats[slot * R + r1] = make_float2(m1, l1);
                }
            }
            if (cut && w.t0 == 0) {  // this stretch holds the unit's beginning: it names the parts
                chain = (int)((w.unit_at + w.tiles - 1) / per - group) + 1;
                chain_row = w.row;
                chain_rows = w.rows;
            }
            ok &= wait_warp(&bars->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, bars, p.d_err);
            tc::fence_after_sync();
            named_sync(2);
            for (int m = 0; m < PAIRS; ++m) {
                for (int c = 0; c < R; c += 16) {
                    uint32_t o[16];
                    tmem_ld_x16(tmem + 128 + m * R + c + lanes, o);
                    tc::tmem_wait_ld();
                    if (cut) {
                        float* dst = p.parts + (slot * R + c) * kDim + m * 128 + tid;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c + e < w.rows) dst[(int64_t)e * kDim] = __uint_as_float(o[e]);
                    } else {
                        // neighbouring lanes swap rows, so that each stores two dims of one row
                        const int odd = lane & 1;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float a = __uint_as_float(o[e]) * inv[c + e];
                            const float d = __uint_as_float(o[e + 1]) * inv[c + e + 1];
                            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : d, 1);
                            const int row = c + e + odd;
                            if (row < w.rows) {
                                uint16_t* dst = p.out + (int64_t)(w.row + row) * kDim + m * 128 + (tid & ~1);
                                *reinterpret_cast<uint32_t*>(dst) = odd ? pack_bf16(got, d) : pack_bf16(a, got);
                            }
                        }
                    }
                }
            }
            tc::fence_before_sync();
            mbar_arrive(&bars->o_free);
        }
        if (tid == 0) p.meta[blockIdx.x] = make_int4(ok ? chain : 0, chain_row, chain_rows, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of a cut unit: out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// meta[g] names the unit that begins in stretch g and goes on behind it: its part
// 0 is that stretch's last, part i the first of the i-th stretch behind it.  Both
// kernels are bound by the latency of their loads (meta, then statistics and
// parts), so the parts' are issued before the statistics are looked at.
PA_DEVICE int64_t part_slot(int g, int i) { return ((int64_t)g + i) * 2 + (i == 0 ? 1 : 0); }

// The j-th cut unit of the call (blockDim.x >= groups): its meta and stretch.
PA_DEVICE int4 find_cut(const Params& p, int j, int& g) {
    __shared__ int counts[16];
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 meta = (int)threadIdx.x < p.groups ? p.meta[threadIdx.x] : make_int4(0, 0, 0, 0);
    const uint32_t cut = __ballot_sync(0xffffffffu, meta.x >= 2);
    if (threadIdx.x == 0) found = -1;
    if (lane == 0) counts[warp] = __popc(cut);
    __syncthreads();
    int before = __popc(cut & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) before += counts[w];
    if (meta.x >= 2 && before == j) found = threadIdx.x;
    __syncthreads();
    g = found;
    return g >= 0 ? p.meta[g] : make_int4(0, 0, 0, 0);
}

PA_DEVICE void add_scaled(float4& a, float f, const float4& x) {
    a.x += f * x.x;
    a.y += f * x.y;
    a.z += f * x.z;
    a.w += f * x.w;
}

PA_DEVICE void store_row(const Params& p, int row, int col, const float4& a, float l) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint2*>(p.out + (int64_t)row * p.latent_dim)[col] =
        make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
}

// Few parts a unit: a warp a row, K float4 columns a lane, all rows of all units at
// once (64 contexts on 128 heads: 5 us; a block a row went through the machine in
// four waves of three latencies, 14 us).
template <int K>
__global__ void __launch_bounds__(256) latent_merge_few_kernel(const Params p) {
    griddep_wait();
    griddep_launch();
    const int g = blockIdx.y, r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int4 meta = p.meta[g];
    if (meta.x < 2 || r >= meta.z) return;
    auto part = [&](int i) { return reinterpret_cast<const float4*>(p.parts + (part_slot(g, i) * p.R + r) * p.latent_dim) + lane; };
    auto stat = [&](int i) { return p.stats[part_slot(g, i) * p.R + r]; };
    float4 o[2][K];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < K; ++k) o[e][k] = part(e)[32 * k];
    float top = -INFINITY;
    for (int i = 0; i < meta.x; ++i) top = fmaxf(top, stat(i).x);
    float4 acc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int i = 0; i < meta.x; i += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (i + e >= meta.x) break;
            const float2 st = stat(i + e);
            const float f = st.x == -INFINITY ? 0.f : ex2(st.x - top);
            l += f * st.y;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                add_scaled(acc[k], f, o[e][k]);
                if (i + 2 + e < meta.x) o[e][k] = part(i + 2 + e)[32 * k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) store_row(p, meta.y + r, lane + 32 * k, acc[k], l);
}

// Many parts a unit: a block a row; a thread has one float4 column of every
// shares-th part, eight in flight, and the shares meet in shared memory.
constexpr int kMergeParts = 256;     // at most one a stretch

__global__ void __launch_bounds__(512) latent_merge_many_kernel(const Params p) {
    griddep_wait();
    griddep_launch();
    const int r = blockIdx.x;
    int g;
    const int4 meta = find_cut(p, blockIdx.y, g);
    if (meta.x < 2 || r >= meta.z) return;
    const int n = min(meta.x, kMergeParts);
    const int columns = p.latent_dim >> 2;
    const int col = threadIdx.x % columns, share = threadIdx.x / columns, shares = blockDim.x / columns;
    __shared__ float2 st[kMergeParts];
    __shared__ float4 sums[512];
    float4 o[8];
    auto load = [&](int i0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = i0 + e * shares;
            if (i < n) o[e] = reinterpret_cast<const float4*>(p.parts + (part_slot(g, i) * p.R + r) * p.latent_dim)[col];
        }
    };
    load(share);
    for (int i = threadIdx.x; i < n; i += blockDim.x) st[i] = p.stats[part_slot(g, i) * p.R + r];
    __syncthreads();
    float top = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) top = fmaxf(top, st[i].x);
    for (int i = 0; i < n; ++i) l += st[i].x == -INFINITY ? 0.f : ex2(st[i].x - top) * st[i].y;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = share; i0 < n; i0 += 8 * shares) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = i0 + e * shares;
            if (i < n) add_scaled(acc, st[i].x == -INFINITY ? 0.f : ex2(st[i].x - top), o[e]);
        }
        load(i0 + 8 * shares);
    }
    sums[threadIdx.x] = acc;
    __syncthreads();
    if (share > 0) return;
    for (int i = 1; i < shares; ++i) add_scaled(acc, 1.f, sums[i * columns + col]);
    store_row(p, meta.y + r, col, acc, l);
}

static cudaError_t launch_merge(const Params& p, int64_t units, cudaStream_t stream) {
    // a unit is cut into groups / units parts or so: 20 of them at this border, which the
    // first kernel reads in 23 us (eight contexts on 152 stretches) and the second in 13;
    // for two or three parts a unit it is 14 us by the second and 9 by the first
    if (p.groups >= 6 * units) {
        // a block for every unit, not for every stretch: empty ones would cost a launch each
        const unsigned cuts = (unsigned)units;
        const int columns = p.latent_dim / 4;
        return launch_pdl(latent_merge_many_kernel, dim3((unsigned)p.R, cuts),
                          dim3((unsigned)(512 / columns * columns)), 0, stream, p);
    }
    const dim3 grid((unsigned)(p.R / 8), (unsigned)p.groups);
    switch (p.latent_dim / 128) {
        case 1: return launch_pdl(latent_merge_few_kernel<1>, grid, dim3(256), 0, stream, p);
        case 2: return launch_pdl(latent_merge_few_kernel<2>, grid, dim3(256), 0, stream, p);
        case 3: return launch_pdl(latent_merge_few_kernel<3>, grid, dim3(256), 0, stream, p);
        default: return launch_pdl(latent_merge_few_kernel<4>, grid, dim3(256), 0, stream, p);
    }
}

// ---------------------------------------------------------------- host side
// Least tiles of a stretch (one context of 700 tokens on 16 heads: 14.5 us with 1 or 2,
// 16.6 with 4, 18.6 with 6; of 2000 on 64 heads 16.6, 16.5, 19.3, 22.6).
constexpr int kMinTiles = 2;

// Shapes of a call: which kernel, rows of a unit, stretches, workspace.
struct Shape {
    bool pair;
    int unit_rows, R, groups;
    int64_t units;                     // at most
    size_t meta_bytes, stats_bytes, bytes;
};

static size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

static Shape shape_of(const pa_latent_pool* pool, int heads, int seqs, bool prefill, int max_q,
                      int total_q, int max_context) {
    Shape s;
    if (max_q > total_q) max_q = total_q;
    const int64_t rows = (int64_t)max_q * heads;   // most of a sequence
    // units of two times 64 rows where there are more than 64 (64 contexts of 128 to 4096
    // tokens on 65, 96, 128 heads: 54, 56, 59 us, by units of 64 rows 81, 80, 84; 5 drafted
    // tokens on 16 heads 50 and 68; at 64 rows the one-CTA kernel takes 161 us for eight
    // contexts of 100K, pairs with half their rows empty as long as for 128, 184)
    s.pair = rows > 64 && pool->rope_dim == 64 && pool->latent_dim % 256 == 0;
    if (s.pair) {
        s.unit_rows = s.R = 128;
    } else {
        const int64_t units = (rows + 63) / 64;    // as even as two rows of units can be
        s.unit_rows = units == 2 && max_q == 1 ? (int)((rows + 1) / 2) : (int)(rows < 64 ? rows : 64);
        s.R = (s.unit_rows + 15) / 16 * 16;
    }
    // a sequence's last unit may not be full, and the line holds up to two tiles more a unit
    s.units = (int64_t)total_q * heads / s.unit_rows + seqs;
    if (max_q == 1 && rows <= s.unit_rows) s.units = seqs;
    const int64_t tiles = s.units * ((max_context + kTok - 1) / kTok + (prefill ? 2 : 0));
    const int64_t most = device_sm_count() / (s.pair ? 2 : 1), need = (tiles + kMinTiles - 1) / kMinTiles;
    s.groups = (int)(need < most ? need : most);
    if (s.groups < 1) s.groups = 1;
    if (s.groups > kMergeParts) s.groups = kMergeParts;
    const size_t slots = (size_t)2 * s.groups;
    s.meta_bytes = round256((size_t)s.groups * sizeof(int4));
    s.stats_bytes = round256(slots * s.R * sizeof(float2));
    s.bytes = s.meta_bytes + s.stats_bytes + slots * s.R * pool->latent_dim * sizeof(float);
    return s;
}

template <int PAIRS, int R>
static cudaError_t launch(const Params& p, const CUtensorMap& mq, const CUtensorMap& mr, const CUtensorMap& mp,
                          cudaStream_t stream) {
    constexpr int smem = Layout<PAIRS, R>::kBytes;
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= 64 || !attr_done[dev])) {
        e = cudaFuncSetAttribute(latent_kernel<PAIRS, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_kernel<PAIRS, R>, dim3((unsigned)p.groups), dim3(kThreads),
                      (size_t)smem, stream, mq, mr, mp, p);
}

template <int R>
static cudaError_t launch_rows(const Params& p, const CUtensorMap& mq, const CUtensorMap& mr,
                               const CUtensorMap& mp, cudaStream_t stream) {
    switch (p.latent_dim / 128) {
        case 1: return launch<1, R>(p, mq, mr, mp, stream);
        case 2: return launch<2, R>(p, mq, mr, mp, stream);
        case 3: return launch<3, R>(p, mq, mr, mp, stream);
        default: return launch<4, R>(p, mq, mr, mp, stream);
    }
}

static cudaError_t launch_one(const Params& p, const void* q, const pa_latent_pool* pool, int64_t q_rows,
                              cudaStream_t stream) {
    const uint64_t width = pool->latent_dim + pool->rope_dim;
    CUtensorMap mq, mr, mp;
    const uint64_t qdims[2] = {width, (uint64_t)q_rows};
    const uint64_t strides[1] = {width * 2};
    const uint32_t qbox[2] = {64, (uint32_t)p.R};
    // the pool as [rows / 8][blocks of 64 dims][8][64], and as rows for the rotary part
    const uint64_t rows = (uint64_t)pool->num_blocks * pool->block_size;
    const uint32_t box = pool->block_size < kTok ? pool->block_size : kTok;
    const uint64_t rdims[4] = {64, 8, (uint64_t)pool->latent_dim / 64, rows / 8};
    const uint64_t rstrides[3] = {width * 2, 128, width * 16};
    const uint32_t rbox[4] = {64, 8, pool->latent_dim % 256 == 0 ? 4u : 2u, box / 8};
    const uint64_t pdims[2] = {width, rows};
    const uint32_t pbox[2] = {64, box};
    if (!encode_bf16_map_sw128(&mq, q, 2, qdims, strides, qbox) ||
        !encode_bf16_map_sw128(&mr, pool->rows, 4, rdims, rstrides, rbox) ||
        !encode_bf16_map_sw128(&mp, pool->rows, 2, pdims, strides, pbox))
        return cudaErrorInvalidValue;
    switch (p.R / 16) {
        case 1: return launch_rows<16>(p, mq, mr, mp, stream);
        case 2: return launch_rows<32>(p, mq, mr, mp, stream);
        case 3: return launch_rows<48>(p, mq, mr, mp, stream);
        default: return launch_rows<64>(p, mq, mr, mp, stream);
    }
}

static pa_status attention(const pa_latent_pool* pool, const void* q, int32_t heads,
                           const int32_t* starts, const int32_t* tables, int32_t max_blocks,
                           const int32_t* lens, int32_t seqs, int32_t max_q, int32_t total_q,
                           int32_t max_context, float scale, int causal, void* out, void* workspace,
                           size_t workspace_bytes, int32_t* d_err, cudaStream_t stream) {
    const Shape sh = shape_of(pool, heads, seqs, starts != nullptr, max_q, total_q, max_context);
    if (workspace == nullptr || workspace_bytes < sh.bytes || !aligned16(workspace))
        return PA_ERR_INVALID_ARG;
    Params p;
    p.q = (const char*)q;
    p.rows = (const char*)pool->rows;
    p.num_blocks = pool->num_blocks;
    p.log2_bp = ilog2(pool->block_size);
    p.latent_dim = pool->latent_dim;
    p.rope_dim = pool->rope_dim;
    p.heads = heads;
    p.starts = starts;
    p.lens = lens;
    p.tables = tables;
    p.max_blocks = max_blocks;
    p.seqs = seqs;
    p.max_q = max_q;
    p.total_q = total_q;
    p.max_context = max_context;
    p.causal = causal;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.unit_rows = sh.unit_rows;
    p.R = sh.R;
    // unit_rows / heads tokens more a unit, 64 tokens a tile: a tile more every `step` units
    p.step = sh.unit_rows > 64 && heads > 1 ? heads / 2 : heads;
    p.more = sh.unit_rows > 64 && heads == 1 ? 2 : 1;
    p.unit_shift = is_pow2(sh.unit_rows) && sh.unit_rows >= 64 ? ilog2(sh.unit_rows) : 0;
    p.slack = (sh.unit_rows - 1) / heads;
    p.unit_tokens = sh.unit_rows / heads;
    p.unit_rest = sh.unit_rows % heads;
    p.per_head = (65536u + heads - 1) / heads;
    p.groups = sh.groups;
    p.min_tiles = kMinTiles;
    p.out = (uint16_t*)out;
    p.meta = (int4*)workspace;
    p.stats = (float2*)((char*)workspace + sh.meta_bytes);
    p.parts = (float*)((char*)workspace + sh.meta_bytes + sh.stats_bytes);
    p.d_err = d_err;

    const int64_t q_rows = (int64_t)total_q * heads;
    cudaError_t e = sh.pair ? launch_pair(p, q, pool, q_rows, stream) : launch_one(p, q, pool, q_rows, stream);
    if (e == cudaSuccess && sh.groups > 1) e = launch_merge(p, sh.units, stream);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PA_ERR_CUDA;
    }
    return launch_status();
}

static pa_status check(const pa_latent_pool* pool, int32_t heads, int32_t seqs, int32_t max_context) {
    pa_status st = check_latent_pool(pool);
    if (st != PA_OK) return st;
    if (heads <= 0 || seqs < 0 || max_context < 0) return PA_ERR_INVALID_ARG;
    if (pool->latent_dim % 128 != 0 || pool->latent_dim > 512 || pool->rope_dim > 64 ||
        !is_pow2(pool->block_size) || pool->block_size < 8 || pool->block_size > 128 ||
        heads > 128 || seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)pool->num_blocks * pool->block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace lat
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_decode_latent_workspace_bytes(const pa_latent_pool* pool, int32_t num_seqs,
                                                      int32_t num_q_heads, int32_t max_context,
                                                      size_t* bytes) {
    if (bytes == nullptr) return PA_ERR_INVALID_ARG;
    pa_status st = lat::check(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    *bytes = num_seqs == 0 || max_context == 0
                 ? 0
                 : lat::shape_of(pool, num_q_heads, num_seqs, false, 1, num_seqs, max_context).bytes;
    return PA_OK;
}

extern "C" pa_status pa_decode_latent(const pa_latent_pool* pool, const void* q, int32_t num_q_heads,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs,
                                      int32_t max_context, float scale, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* d_err, pa_stream_t stream) {
    pa_status st = lat::check(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    if (max_blocks_per_seq < 0 || !(scale == scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_context == 0) return PA_OK;
    if (!q || !block_tables || !context_lens || !out) return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(pool->rows)) return PA_ERR_INVALID_ARG;
    return lat::attention(pool, q, num_q_heads, nullptr, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, 1, num_seqs, max_context, scale, 0, out, workspace,
                          workspace_bytes, d_err, (cudaStream_t)stream);
}

extern "C" pa_status pa_prefill_latent_workspace_bytes(const pa_latent_pool* pool, int32_t num_seqs,
                                                       int32_t num_q_heads, int32_t total_q,
                                                       int32_t max_q_len, int32_t max_context,
                                                       size_t* bytes) {
    if (bytes == nullptr || total_q < 0 || max_q_len < 0) return PA_ERR_INVALID_ARG;
    pa_status st = lat::check(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    if ((int64_t)total_q * num_q_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
    *bytes = num_seqs == 0 || total_q == 0 || max_q_len == 0 || max_context == 0
                 ? 0
                 : lat::shape_of(pool, num_q_heads, num_seqs, true, max_q_len, total_q, max_context).bytes;
    return PA_OK;
}

extern "C" pa_status pa_prefill_latent(const pa_latent_pool* pool, const void* q, int32_t total_q,
                                       int32_t num_q_heads, const int32_t* cu_seqlens_q,
                                       const int32_t* context_lens, const int32_t* block_tables,
                                       int32_t max_blocks_per_seq, int32_t num_seqs,
                                       int32_t max_q_len, int32_t max_context, float scale,
                                       int32_t causal, void* out, void* workspace,
                                       size_t workspace_bytes, int32_t* d_err, pa_stream_t stream) {
    pa_status st = lat::check(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    if (total_q < 0 || max_q_len < 0 || max_blocks_per_seq < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    if ((int64_t)total_q * num_q_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0 || max_context == 0) return PA_OK;
    if (!q || !cu_seqlens_q || !context_lens || !block_tables || !out) return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(pool->rows)) return PA_ERR_INVALID_ARG;
    return lat::attention(pool, q, num_q_heads, cu_seqlens_q, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, max_q_len < total_q ? max_q_len : total_q, total_q,
                          max_context, scale, causal ? 1 : 0, out, workspace, workspace_bytes, d_err,
                          (cudaStream_t)stream);
}
