// shared.cu -- MLA decode attention for a batch whose sequences begin with the same cached prefix.
//
// The result is that of mla_decode: per query row r of sequence b, over the V visible keys of b,
//   s_j = scale <q_r, k_j>,  lse = log sum_j e^{s_j},  out = sum_j e^{s_j - lse} k_j[0:512].
// The sum over keys splits at the end of the prefix, and each part's normalised result and lse merge
// exactly (up to rounding): lse = log(e^{lse_1} + e^{lse_2}), out = sum_i e^{lse_i - lse} out_i. The
// prefix keys are the same for every row of the batch, so its part is ONE attention of all batch * s_q *
// h_q rows over one key list: the rows fill 128-row tensor tiles whatever the head count (16 heads alone
// fill an eighth of one) and a key block is read once per tile of rows, not once per sequence.
//
// Work units (partitioned into parts by metadata.cu, in 128-token tiles):
//  * rows per sequence not a multiple of 128: first ceil(rows of the batch / 128) prefix units (128
//    rows of the flat [batch * s_q * h_q] row space, the shared blocks), then one unit per (sequence,
//    128-row group) over the sequence's own blocks;
//  * a multiple of 128 (every row tile belongs to one sequence) or no shared block: one unit per
//    (sequence, group) over shared and own blocks alike, so that an unsplit unit needs no merge.
// A unit cut into pieces, or one of the first kind, leaves fp32 partials for the combine kernel.
//
// The kernel: one persistent 2-CTA pair per part, MMAs with cta_group::2.
//  * 128 rows x 512 value dims of fp32 output are a whole SM's tensor memory, so a pair shares a tile:
//    64 rows in each CTA. M = 128 over the pair puts a CTA's 64 rows into all of its 128 TMEM lanes
//    (lane l: row l % 64; lanes 64-127 hold the upper half of the columns): O takes 256 columns and the
//    scores of 128 tokens 64, so two score buffers fit beside it and no partial score or probability
//    ever crosses between the SMs.
//  * A tile is two cache blocks. S = Q K^T: 36 MMAs of 128 x 128 x 16 (K-major boxes of 64 tokens x 64 dims);
//    CTA h provides the tokens of block h, all 576 dims of it. O += P V: 16 MMAs of 128 x 256 x 16 (MN-major
//    boxes); CTA h provides value dims [256h, 256h + 256) of both blocks. K's boxes cannot serve as V as well: an
//    MMA takes its operand at the same offset in both CTAs, and there each holds its own block's tokens. So V is
//    loaded on its own (from L2, where K has just put it) and K's boxes are free once Gemm1 has read them: K (9
//    boxes), V (8) and Q (9) have one buffer each, refilled in groups behind the MMAs (139 KB a tile and CTA).
//  * One thread of the leader issues QK(g + 1) before PV(g), so the tensor cores work through the softmax of a
//    tile (two tiles ahead instead of one, with four score buffers: the same time).
//  * What bounds it: a tile takes 2,480 cycles at 1.8 GHz against the 2,176 of its MMAs, and no role's waits
//    are on the way any more; on calls of a few 100 us the power limit takes the clock to about 1.35 GHz. Beside that a
//    call has about 5 us until its first tile (set-up, then 147 KB of Q and K a CTA at once), 5 us for its last
//    piece's output, and as much again at each piece in between. Back to back, on 74 pairs: 64 sequences of 16 heads
//    over 16,384 shared tokens 48 us (37 GFLOP); 128 of 128 heads over 4,096, 158 us with the merge (165 GFLOP,
//    1,040 TFLOP/s); 33 of 64 heads over 65,536, 275 us (303 GFLOP, 1,100 TFLOP/s, where cuBLAS sustains 1,374).
//  * Eight softmax warps, one thread per (row, 32 tokens); the four threads of a row agree on the running
//    maximum through shared memory, O is rescaled only when it grows by more than 2^8 (P <= 2^8, exact
//    in the fp32 sums). P is rounded to bf16 once (to nearest): an error of at most 2^-8 of each term, the
//    size of the output's own rounding, where a second term would add half to the MMA time.
//  * Roles: warp 0 = loads; warp 1 of the leader = MMAs; warp 2 = zeroing of value rows past the unit's end
//    (undefined contents must not meet a zero probability); warp 3 = table look-ups ahead; warps 4-11 softmax
//    and epilogue.
// Every wait is bounded; a timeout sets the device error word and the pair exits cleanly.
#include "pair_ptx.cuh"
#include "shared.cuh"

namespace mla {
using namespace sm100;

namespace shr {
constexpr int kTileTok = kSharedTileTok;       // 128 tokens: one cache block per CTA
constexpr int kSoftWarps = 8, kThreads = 32 * (4 + kSoftWarps);
constexpr int kGroups = 3;                     // of K's and Q's boxes
constexpr int kBox = kBlk * 128;               // 64 rows x 64 bf16, 128-byte swizzle
constexpr int kBoxes = kDqk / 64;              // 9
constexpr int kGroupBoxes = kBoxes / kGroups;  // 3
constexpr int kGroupBytes = kGroupBoxes * kBox;
constexpr int kValueBytes = 4 * kBox;          // 256 value dims of one block
constexpr int kAhead = 4;                      // tiles whose cache rows are looked up before they are loaded
constexpr float kRescaleThreshold = 8.0f;      // log2 units
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemSCols = 64, kTmemCols = 512;

struct __align__(1024) Smem {
    uint8_t q[kBoxes * kBox];                  // this CTA's 64 query rows
    uint8_t k[kBoxes * kBox];                  // its cache block of the tile
    uint8_t v[2][kValueBytes];                 // its value dims of the tile's two blocks
    uint8_t p[2][kBox];                        // P of its 64 rows, per block
    float xmax[2][4][64];                      // block maxima of a row's four threads; their sums at the end
    // leader's, completed by both CTAs' loads: a group of K (and, on a piece's first tile, of Q); a block of V
    uint64_t k_full[kGroups], v_full[2];
    // a unit's last, partial tile instead: this CTA's V; both CTAs' after zeroing (leader's)
    uint64_t tail_full, tail_ready;
    uint64_t p_full;                           // leader's: both CTAs' softmax warps
    // commits to both CTAs: Gemm1 has read a group; S is complete; Gemm2 has read a block of V (and P)
    uint64_t k_free[kGroups], s_full[2], v_free[2];
    uint64_t mma_done;
    uint64_t r_full[kAhead], r_free[kAhead];   // tiles whose cache rows are known; whose loads are issued
    int row[kAhead][2];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Smem) <= 232448, "shared memory must fit 227 KB");

// One piece: tiles [lo, hi) of a unit. Tile t holds blocks first_blk + 2t and the next, up to end_blk.
struct Piece {
    int seq, group;  // seq < 0: a prefix unit
    int lo, hi, first_blk, end_blk, end_tok, nsplit;
    int64_t part_row;  // first row of its partial slot
};

struct Walker {
    int unit, begin_unit, begin_tile, end_unit, end_tile, first_piece, prefix_tok;
    Piece pc;
    int tile, piece_k;
    bool live;

    __device__ bool next_piece(const SharedParams &p) {
        while (unit <= end_unit) {
            const int u = unit++;
            if (u < p.prefix_units) {
                pc.seq = -1;
                pc.group = u;
                pc.first_blk = 0;
                pc.end_tok = prefix_tok;
            } else {
                const int o = u - p.prefix_units;
                pc.seq = o / p.groups;
                pc.group = o % p.groups;
                pc.first_blk = p.prefix_units > 0 ? p.shared_blocks : 0;
                pc.end_tok = clamp_len(p.seqlens[pc.seq]);
            }
            pc.end_blk = num_blocks_of(pc.end_tok);
            const int w = (max(pc.end_blk - pc.first_blk, 0) + 1) / 2;
            pc.lo = u == begin_unit ? max(begin_tile, 0) : 0;
            pc.hi = u == end_unit ? min(end_tile, w) : w;
            if (pc.hi <= pc.lo) continue;
            // partial slots: the prefix units' of 128 rows, then the own units' of own_rows
            const int s0 = p.num_splits[u], own0 = p.num_splits[p.prefix_units];
            pc.nsplit = p.num_splits[u + 1] - s0;
            const int slot = s0 + (u == begin_unit ? first_piece : 0) - (pc.seq < 0 ? 0 : own0);
            const int slots = (pc.seq < 0 ? p.prefix_units : p.units - p.prefix_units) + p.num_parts;
            if (pc.nsplit < 1 || slot < 0 || slot >= slots) continue;  // malformed
            pc.part_row = pc.seq < 0 ? (int64_t)slot * 128 : p.own_base + (int64_t)slot * p.own_rows;
            return true;
        }
        return false;
    }
    __device__ void init(const int32_t *meta, const SharedParams &p) {
        begin_unit = meta[0];
        begin_tile = meta[1];
        end_unit = meta[2];
        end_tile = meta[3];
        first_piece = meta[4];
        prefix_tok = min(max(meta[5], 0), p.shared_blocks * kBlk);
        if (end_unit >= begin_unit && (begin_unit < 0 || end_unit >= p.units)) end_unit = begin_unit - 1;  // malformed
        unit = begin_unit;
        piece_k = -1;
        step(p);
    }
    __device__ void step(const SharedParams &p) {
        live = next_piece(p);
        tile = live ? pc.lo : 0;
        ++piece_k;
    }
    __device__ bool first() const { return tile == pc.lo; }
    __device__ bool last() const { return tile == pc.hi - 1; }
    // the unit ends inside the tile: rows past its end hold undefined contents
    __device__ bool tail() const { return pc.end_tok - blk() * kBlk < kTileTok; }
    __device__ int blk() const { return pc.first_blk + 2 * tile; }
    __device__ void advance(const SharedParams &p) {
        if (++tile >= pc.hi) step(p);
    }
    // flat row of q that starts this CTA's 64 rows
    __device__ int q_row(const SharedParams &p, int rank) const {
        return (pc.seq < 0 ? 0 : pc.seq * p.rows) + pc.group * 128 + rank * 64;
    }
};

// Cache row of block `blk` of the piece, or one past the cache (TMA then fills zeros) when the piece has
// no such block or its table entry is out of range.
__device__ __forceinline__ int block_row(const SharedParams &p, const Piece &pc, int blk, bool &bad) {
    const int none = (int)(p.num_blocks * kBlk);
    if (blk >= pc.end_blk) return none;
    int phys;
    if (blk < p.shared_blocks)
        phys = p.shared_table[blk];
    else
        phys = blk < p.bt_stride ? p.block_table[(size_t)pc.seq * p.bt_stride + blk] : -1;
    if (phys < 0 || (int64_t)phys >= p.num_blocks) {
        bad = true;
        return none;
    }
    return phys * kBlk;
}

// ---------------------------------------------------------------- warp 0, one thread: loads
// In the order of use: K(g) (and Q), then V(g - 1).
struct Loader {
    Smem &sm;
    const SharedParams &p;
    const CUtensorMap *map_k, *map_v, *map_q;
    uint32_t rank;
    // K of own blocks and Q leave L2 first; V is hinted like shared keys, since its two halves are read by both
    // CTAs and right after K (evicting it first cost 1-2%: 306 against 302 us of a 65,536-token prefix)
    uint64_t pol_shared, pol_own;
    int k_fills, v_fills, tails;  // groups and blocks issued; partial tiles among them

    __device__ bool load_k(const Walker &w, int g) {
        const int blk = w.blk() + (int)rank;
        if (!mbar_poll(&sm.r_full[g % kAhead], (g / kAhead) & 1, &sm.abort)) return false;
        const int y = *(volatile int *)&sm.row[g % kAhead][rank];
        const uint64_t pol = blk < p.shared_blocks ? pol_shared : pol_own;
        const bool first = w.first();
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if (g > 0 && !mbar_poll(&sm.k_free[i], (g - 1) & 1, &sm.abort)) return false;
            const uint32_t bar = map_to_rank(&sm.k_full[i], 0);
            if (rank == 0) mbar_arrive_expect_tx(&sm.k_full[i], (first ? 4 : 2) * kGroupBytes);
            tma_load_3d_pair(sm.k + i * kGroupBytes, map_k, 0, y, kGroupBoxes * i, bar, pol);
            if (first)
                tma_load_3d_pair(sm.q + i * kGroupBytes, map_q, 0, w.q_row(p, (int)rank), kGroupBoxes * i, bar, pol_own);
            ++k_fills;
        }
        return true;
    }
    __device__ bool load_v(const Walker &w, int g) {
        const bool tail = w.tail();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (g > 0 && !mbar_poll(&sm.v_free[t], (g - 1) & 1, &sm.abort)) return false;
            const int y = *(volatile int *)&sm.row[g % kAhead][t];
            if (!tail) {
                if (rank == 0) mbar_arrive_expect_tx(&sm.v_full[t], 2 * kValueBytes);
                tma_load_3d_pair(sm.v[t], map_v, 0, y, 4 * (int)rank, map_to_rank(&sm.v_full[t], 0), pol_shared);
            } else {
                if (rank == 0) mbar_arrive(&sm.v_full[t]);  // keeps the phases in step
                if (t == 0) mbar_arrive_expect_tx(&sm.tail_full, 2 * kValueBytes);
                tma_load_3d(sm.v[t], map_v, 0, y, 4 * (int)rank, &sm.tail_full, pol_own);
            }
            ++v_fills;
        }
        tails += tail;
        mbar_arrive(&sm.r_free[g % kAhead]);
        return true;
    }
};

// Before the pair exits: fill number `fills` of a barrier's buffer has landed (bounded; independent of
// the abort flag).
__device__ void landed(uint64_t *bar, int fills) {
    const long long t0 = clock64();
    while (fills > 0 && !mbar_sleep_test(bar, (fills - 1) & 1) && clock64() - t0 < kSpinCycles) {
    }
}

__device__ void load_role(Smem &sm, const SharedParams &p, const CUtensorMap *map_k, const CUtensorMap *map_v,
                          const CUtensorMap *map_q, Walker w, uint32_t rank) {
    Loader ld{sm, p, map_k, map_v, map_q, rank, l2_evict_normal_policy(), l2_evict_first_policy(), 0, 0, 0};
    Walker wv = w;  // of V, one tile behind
    bool ok = true;
    int g = 0;
    for (; ok && w.live; w.advance(p), ++g) {
        ok = ld.load_k(w, g);
        if (ok && g > 0) {
            ok = ld.load_v(wv, g - 1);
            wv.advance(p);
        }
    }
    if (ok && g > 0) ld.load_v(wv, g - 1);
    if (rank == 0) {  // the leader's barriers see both CTAs' loads
        for (int i = 0; i < kGroups; ++i) landed(&sm.k_full[i], (ld.k_fills + kGroups - 1 - i) / kGroups);
        for (int t = 0; t < 2; ++t) landed(&sm.v_full[t], (ld.v_fills + 1 - t) / 2);
    }
    landed(&sm.tail_full, ld.tails);
}

// ---------------------------------------------------------------- warp 3, one thread: cache rows ahead of the loads
// A tile's blocks are found by dependent loads (unit, length, table), and contents that only one
// sequence owns come from HBM: the rows are looked up kAhead tiles early and such blocks brought into L2.
__device__ void resolve_role(Smem &sm, const SharedParams &p, const CUtensorMap *map_k, const CUtensorMap *map_q, Walker w,
                             uint32_t rank) {
    bool bad = false;
    for (int g = 0; w.live; w.advance(p), ++g) {
        const int s = g % kAhead;
        const int y0 = block_row(p, w.pc, w.blk(), bad), y1 = block_row(p, w.pc, w.blk() + 1, bad);
        if (g >= kAhead && !mbar_wait(&sm.r_free[s], (g / kAhead - 1) & 1, &sm.abort)) break;
        *(volatile int *)&sm.row[s][0] = y0;
        *(volatile int *)&sm.row[s][1] = y1;
        mbar_arrive(&sm.r_full[s]);
        if (g > 0 && w.first())
#pragma unroll
            for (int i = 0; i < kGroups; ++i) tma_prefetch_3d(map_q, 0, w.q_row(p, (int)rank), kGroupBoxes * i);
        const int blk = w.blk() + (int)rank;
        if (g > 0 && blk >= p.shared_blocks && blk < w.pc.end_blk)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) tma_prefetch_3d(map_k, 0, rank == 0 ? y0 : y1, kGroupBoxes * i);
    }
    if (bad) raise_error(kErrBounds);
}

// Zero this CTA's value rows past the unit's end in one block of the tile (4 boxes).
__device__ void zero_rows(uint8_t *boxes, int valid, int lane) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int e = lane; e < (kBlk - valid) * 8; e += 32) {
        const int off = (valid + (e >> 3)) * 128 + ((e & 7) << 4);
#pragma unroll
        for (int b = 0; b < 4; ++b) *reinterpret_cast<uint4 *>(boxes + b * kBox + off) = z;
    }
}

// ---------------------------------------------------------------- warp 2: partial tiles
__device__ void tail_role(Smem &sm, const SharedParams &p, Walker w) {
    const int lane = threadIdx.x & 31;
    int tails = 0;
    for (; w.live; w.advance(p)) {
        if (!w.tail()) continue;
        if (!warp_poll(&sm.tail_full, tails & 1, &sm.abort)) break;
        ++tails;
        const int left = w.pc.end_tok - w.blk() * kBlk;  // tokens of the tile (a missing block is zeros)
        if (left < kBlk) zero_rows(sm.v[0], max(left, 0), lane);
        if (left > kBlk) zero_rows(sm.v[1], left - kBlk, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(map_to_rank(&sm.tail_ready, 0));
        __syncwarp();
    }
}

// ---------------------------------------------------------------- warp 1 of the leader, one thread: MMAs
// Its own instruction stream bounds the tensor cores: with the whole warp in the role and one lane elected for each
// group, a wait whose phase was there cost about 280 cycles (a branch, a shuffle), an election 75, a reconvergence
// 90, some 2,500 in all per tile beside 2,176 of MMAs. One elected thread throughout: 306 -> 285 us of a
// 65,536-token prefix, 179 -> 165 with 128 x 128 heads.
struct Issuer {
    Smem &sm;
    uint32_t tmem;
    int tails;

    // S(g) = Q K^T. The score buffer is free: P of tile g - 2 was awaited before this.
    __device__ bool scores(int g) {
        constexpr uint32_t id = idesc_bf16_f32(128, 128, 0);
        const uint64_t qd = smem_desc(smem_addr(sm.q), 16, 1024, 2), kd = smem_desc(smem_addr(sm.k), 16, 1024, 2);
        const uint32_t d = tmem + kTmemS + kTmemSCols * (g & 1);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if (!mbar_poll(&sm.k_full[i], g & 1, &sm.abort)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4 * kGroupBoxes; ++k) {
                const uint64_t off = (uint64_t)(((i * kGroupBoxes + (k >> 2)) * kBox + (k & 3) * 32) >> 4);
                mma_ss_pair(d, qd + off, kd + off, id, i + k > 0 ? 1u : 0u);
            }
            mma_commit_pair(&sm.k_free[i]);
            if (i == kGroups - 1) mma_commit_pair(&sm.s_full[g & 1]);
        }
        return true;
    }
    // O (+)= P V of tile g
    __device__ bool values(int g, bool first, bool tail) {
        constexpr uint32_t id = idesc_bf16_f32(128, 256, 1);  // MN-major B
        const uint64_t pd = smem_desc(smem_addr(sm.p), 16, 1024, 2), vd = smem_desc(smem_addr(sm.v), kBox, 1024, 2);
        if (!mbar_poll(&sm.p_full, g & 1, &sm.abort)) return false;
        if (tail && !mbar_poll(&sm.tail_ready, tails & 1, &sm.abort)) return false;
        tails += tail;
        const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (!tail && !mbar_poll(&sm.v_full[t], g & 1, &sm.abort)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 tokens each
#pragma unroll
                for (int n = 0; n < 2; ++n)  // 128 value dims of each CTA
                    mma_ss_pair(tmem + kTmemO + 128 * n, pd + (uint64_t)((t * kBox + k * 32) >> 4),
                                vd + (uint64_t)((t * kValueBytes + 2 * n * kBox + k * 2048) >> 4), id,
                                t + k > 0 ? 1u : acc0);
            mma_commit_pair(&sm.v_free[t]);
        }
        return true;
    }
};

__device__ void mma_role(Smem &sm, const SharedParams &p, Walker w, uint32_t tmem) {
    Issuer is{sm, tmem, 0};
    bool first = false, tail = false;  // of the tile before
    for (int g = 0;; ++g) {
        if (w.live && !is.scores(g)) break;
        if (g > 0 && !is.values(g - 1, first, tail)) break;
        if (!w.live) break;
        first = w.first();
        tail = w.tail();
        w.advance(p);
    }
}

// Every MMA this thread issued completes before teardown (bounded; independent of the abort flag).
__device__ void drain_mmas(Smem &sm) {
    mma_commit_pair_local(&sm.mma_done);
    const long long t0 = clock64();
    while (!mbar_sleep_test(&sm.mma_done, 0) && clock64() - t0 < kSpinCycles) {
    }
}

// ---------------------------------------------------------------- warps 4-11: softmax and epilogue
// Warp w: TMEM lane quarter w & 3 (rows 32 (w & 1) .. + 32 of the CTA's 64; block (w >> 1) & 1 of the tile),
// 32 of that block's tokens (th). Of O, its lanes hold dims [256 blk + 128 th, + 128) of its rows.
__device__ void softmax_role(Smem &sm, const SharedParams &p, Walker w, uint32_t tmem, uint32_t rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wq = warp & 3, blk = wq >> 1, th = (warp - 4) >> 2;
    const int i = (wq & 1) * 32 + lane;  // row of this CTA's 64
    const int bar_id = 1 + (wq & 1);     // the four warps of these 32 rows
    const int x = 2 * blk + th;          // this thread's place among the row's four
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const float sl2 = p.scale_log2;
    const uint32_t p_full = map_to_rank(&sm.p_full, 0);
    // After a failed wait the warp walks on without waiting, so that no named barrier misses it.
    bool dead = false;
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !warp_poll(bar, parity, &sm.abort)) dead = true;
    };
    float m_ref = -INFINITY, l = 0.f;
    int vis = 0, flat = 0;
    bool row_ok = false;
    for (int g = 0; w.live; ++g) {
        const bool first = w.first();
        if (first) {  // this row's visible keys within the piece
            flat = w.q_row(p, (int)rank) + i;
            const int seq = w.pc.seq < 0 ? min(flat, p.total_rows - 1) / p.rows : w.pc.seq;
            const int r = flat - seq * p.rows;
            row_ok = w.pc.seq < 0 ? flat < p.total_rows : r < p.rows;
            vis = row_ok ? visible_keys(p.seqlens[seq], p.s_q, r / p.h_q, p.causal) : 0;
            vis = min(vis, min(w.pc.first_blk + 2 * w.pc.hi, w.pc.end_blk) * kBlk);
            __syncwarp();
        }
        const int key0 = w.blk() * kBlk + blk * kBlk + 32 * th;
        wait(&sm.s_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        uint32_t raw[32];
        tmem_ld32(tmem + kTmemS + kTmemSCols * (g & 1) + lane_off + 32 * th, raw);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
        if (__any_sync(0xffffffffu, key0 + 32 > vis)) {  // the same way for all lanes: a barrier of whole warps follows
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = key0 + j < vis ? v[j] : -INFINITY;
        }
        sm.xmax[g & 1][x][i] = max32(v);
        named_bar_sync(bar_id, 128);
        const float mx = fmaxf(fmaxf(sm.xmax[g & 1][0][i], sm.xmax[g & 1][1][i]),
                               fmaxf(sm.xmax[g & 1][2][i], sm.xmax[g & 1][3][i]));
        const float mb = mx == -INFINITY ? -INFINITY : mx * sl2;  // sl2 > 0: the maximum commutes with it
        bool need = false;
        float alpha = 1.f;
        if (first) {
            m_ref = mb;
            l = 0.f;
        } else if (mb > m_ref + kRescaleThreshold) {
            if (m_ref != -INFINITY) {  // else nothing is accumulated yet: O and l are zero
                alpha = ex2_approx(m_ref - mb);
                l *= alpha;
                need = true;
            }
            m_ref = mb;
        }
        const float off = m_ref == -INFINITY ? 0.f : -m_ref;
        const f32x2 sc = pack2(sl2, sl2), of = pack2(off, off);
        f32x2 su[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float a, b;
            unpack2(fma2(pack2(v[j], v[j + 1]), sc, of), a, b);
            a = ex2_approx(a);
            b = ex2_approx(b);
            su[(j >> 1) & 3] = add2(su[(j >> 1) & 3], pack2(a, b));
            __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
            pk[j >> 1] = *reinterpret_cast<uint32_t *>(&two);
        }
        {
            float a, b;
            unpack2(add2(add2(su[0], su[1]), add2(su[2], su[3])), a, b);
            l += a + b;
        }
        // Gemm2 of the previous tile is done with P and O
        if (g > 0) wait(&sm.v_free[1], (g - 1) & 1);
        if (__any_sync(0xffffffffu, need)) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16(tmem + kTmemO + lane_off + 128 * th + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st16(tmem + kTmemO + lane_off + 128 * th + 16 * c, o);
            }
            tmem_wait_st();
        }
        uint8_t *prow = sm.p[blk] + i * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4 *>(prow + (((4 * th + c) ^ (i & 7)) << 4)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(p_full);
        __syncwarp();

        if (w.last()) {
            // the row's four sums, through the maxima's slots of the other parity (read before the barrier above)
            sm.xmax[(g + 1) & 1][x][i] = l;
            named_bar_sync(bar_id, 128);
            const float lr = (sm.xmax[(g + 1) & 1][0][i] + sm.xmax[(g + 1) & 1][1][i]) +
                             (sm.xmax[(g + 1) & 1][2][i] + sm.xmax[(g + 1) & 1][3][i]);
            named_bar_sync(bar_id, 128);  // read before the next tile's maxima take the slots
            const bool empty = lr == 0.f;
            const float inv = empty ? 0.f : 1.f / lr;
            const float lse2 = empty ? -INFINITY : m_ref + log2f(lr);
            const bool whole = p.prefix_units == 0 && w.pc.nsplit == 1;
            const int64_t part_row = w.pc.part_row + (int)rank * 64 + i;
            wait(&sm.v_free[1], g & 1);
            tc_fence_after();
            const int col = 256 * blk + 128 * th;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16(tmem + kTmemO + lane_off + 128 * th + 16 * c, o);
                tmem_wait_ld();
                if (row_ok && whole) {
                    uint32_t wv[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv,
                                                                   __uint_as_float(o[2 * j + 1]) * inv);
                        wv[j] = *reinterpret_cast<uint32_t *>(&two);
                    }
                    __nv_bfloat16 *dst = p.out + (size_t)flat * kDv + col + 16 * c;
                    if (p.out_v8) {
                        st_global_v8(dst, wv);
                    } else {
                        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
                        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(wv[4], wv[5], wv[6], wv[7]);
                    }
                } else if (row_ok) {
                    float *dst = p.o_part + (size_t)part_row * kDv + col + 16 * c;
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
                    st_global_v8(dst, o);
                    st_global_v8(dst + 8, o + 8);
                }
                __syncwarp();  // a slice may be partly filled, and the next load is the whole warp's
            }
            if (row_ok && x == 0) {
                if (whole) {
                    const int r = flat % p.rows;
                    p.lse[((size_t)(flat / p.rows) * p.h_q + r % p.h_q) * p.s_q + r / p.h_q] =
                        lse2 * 0.69314718055994530942f;
                } else {
                    p.lse_part[part_row] = lse2;
                }
            }
            __syncwarp();
            tc_fence_before();  // ordered before the next tile's P, which lets Gemm2 overwrite O
        }
        w.advance(p);
    }
}

// (bounds of 512 threads for 128 registers at most: 1% faster than the 149 that 384 would give)
__global__ void __launch_bounds__(512, 1)
shared_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const __grid_constant__ CUtensorMap map_q, const SharedParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // all of it is used: no room to align by hand
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5;
    const int32_t *meta = p.tile_meta + (size_t)(blockIdx.x >> 1) * kMetaInts;
    if (smem_addr(smem_raw) & 1023) {  // the swizzled boxes need it; both CTAs of the pair see the same
        if (threadIdx.x == 0) raise_error(kErrBounds);
        return;
    }

    if (warp == 1) tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_free[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.v_full[t], 1);
            mbar_init(&sm.v_free[t], 1);
            mbar_init(&sm.s_full[t], 1);
        }
        for (int k = 0; k < kAhead; ++k) {
            mbar_init(&sm.r_full[k], 1);
            mbar_init(&sm.r_free[k], 1);
        }
        mbar_init(&sm.tail_full, 1);
        mbar_init(&sm.tail_ready, 2);
        mbar_init(&sm.p_full, 2 * kSoftWarps);
        mbar_init(&sm.mma_done, 1);
        sm.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        prefetch_tensormap(&map_q);
    }
    wait_for_previous_kernel();  // the set-up above needs nothing of it
    Walker w;
    const bool early = warp == 0 || warp == 3;  // the loads are waited for: their first piece during the set-up
    if (early) w.init(meta, p);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist
    tc_fence_after();
    if (!early) w.init(meta, p);
    const uint32_t tmem = sm.tmem_base;

    if (warp == 0) {
        if (elect_one()) load_role(sm, p, &map_k, &map_v, &map_q, w, rank);
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            mma_role(sm, p, w, tmem);
            drain_mmas(sm);
        }
    } else if (warp == 2) {
        tail_role(sm, p, w);
    } else if (warp == 3) {
        if (elect_one()) resolve_role(sm, p, &map_k, &map_q, w, rank);
    } else {
        softmax_role(sm, p, w, tmem, rank);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) raise_error(kErrTimeout);
    cluster_sync();  // nothing of the pair is in flight any more
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- merging the pieces of a row
// Two warps per row, 8 dims per lane: the pieces of its prefix unit, then those of its own unit. Bound by
// latency (a few dependent rounds of loads) and, for many rows, by the partials' bytes (2 KB a piece and
// row, from L2): lane k reads the lse of piece k, two pieces' outputs are in flight per warp beside it. Most
// rows have two or three pieces: four in flight load some twice, and cost 1.5 of 180 us at 16,384 rows.
constexpr int kMergeWarps = 8, kMergeFly = 2;
__global__ void __launch_bounds__(32 * kMergeWarps, 4) merge_kernel(const SharedParams p) {
    const int64_t w = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    const int flat = (int)(w >> 1), lane = threadIdx.x & 31;
    if (flat >= p.total_rows) return;
    const int d0 = (int)(w & 1) * (kDv / 2) + 8 * lane;
    const int seq = flat / p.rows, r = flat % p.rows;
    const int ou = p.prefix_units + seq * p.groups + r / 128;
    wait_for_previous_kernel();
    const int o0 = p.num_splits[ou], no = p.num_splits[ou + 1] - o0;
    int p0 = 0, np = 0, ob = 0;
    if (p.prefix_units > 0) {
        p0 = p.num_splits[flat / 128];
        np = p.num_splits[flat / 128 + 1] - p0;
        ob = p.num_splits[p.prefix_units];
    } else if (no == 1) {
        return;  // written by the attention kernel
    }
    if (no < 0 || np < 0 || p0 < 0 || o0 < ob || p0 + np > p.prefix_units + p.num_parts ||
        o0 - ob + no > p.units - p.prefix_units + p.num_parts) {  // malformed metadata
        if (lane == 0) raise_error(kErrBounds);
        return;
    }
    const int64_t prow = (int64_t)p0 * 128 + flat % 128;
    const int64_t orow = p.own_base + (int64_t)(o0 - ob) * p.own_rows + r % 128;
    const int ns = np + no;
    const auto row_of = [&](int k) { return k < np ? prow + (int64_t)k * 128 : orow + (int64_t)(k - np) * p.own_rows; };
    float acc[8], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int base = 0; base < ns; base += 32) {
        const int n = min(32, ns - base);
        const float ls = lane < n ? p.lse_part[row_of(base + lane)] : -INFINITY;
        float mx = m, wgt = 0.f, a = 1.f;
        for (int k0 = 0; k0 < n; k0 += kMergeFly) {
            float4 v[kMergeFly][2];
#pragma unroll
            for (int d = 0; d < kMergeFly; ++d) {
                const float4 *src =
                    reinterpret_cast<const float4 *>(p.o_part + (size_t)row_of(base + min(k0 + d, n - 1)) * kDv + d0);
                v[d][0] = src[0];
                v[d][1] = src[1];
            }
            if (k0 == 0) {  // the weights of these pieces, while the outputs arrive
                mx = fmaxf(m, isnan(ls) ? 0.f : ls);  // a NaN piece weighs NaN; fmaxf would take it for one without keys
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (mx == -INFINITY) break;  // no key so far
                wgt = exp2f(ls - mx);
                a = exp2f(m - mx);
                float s = wgt;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                sum = fmaf(sum, a, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] *= a;
                m = mx;
            }
#pragma unroll
            for (int d = 0; d < kMergeFly; ++d) {  // a piece without keys has zeros; past the last, weight 0
                const float wd = __shfl_sync(0xffffffffu, wgt, min(k0 + d, 31));
                const float u = k0 + d < n ? wd : 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    acc[4 * j + 0] = fmaf(u, v[d][j].x, acc[4 * j + 0]);
                    acc[4 * j + 1] = fmaf(u, v[d][j].y, acc[4 * j + 1]);
                    acc[4 * j + 2] = fmaf(u, v[d][j].z, acc[4 * j + 2]);
                    acc[4 * j + 3] = fmaf(u, v[d][j].w, acc[4 * j + 3]);
                }
            }
        }
    }
    const float inv = m == -INFINITY ? 0.f : 1.f / sum;
    uint4 packed;
    uint32_t *pw = reinterpret_cast<uint32_t *>(&packed);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        __nv_bfloat162 two = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
        pw[k] = *reinterpret_cast<uint32_t *>(&two);
    }
    *reinterpret_cast<uint4 *>(p.out + (size_t)flat * kDv + d0) = packed;
    if (lane == 0 && d0 == 0)
        p.lse[((size_t)seq * p.h_q + r % p.h_q) * p.s_q + r / p.h_q] =
            m == -INFINITY ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
}
}  // namespace shr

size_t shared_smem_bytes() { return sizeof(shr::Smem); }

// Both kernels take programmatic launches, without an early trigger: their launch overlaps the end of the
// kernel before them (a small call back to back 17.3 -> 13.7 us; triggering early was slower).
cudaError_t launch_shared(const SharedParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                          const CUtensorMap &map_q, cudaStream_t stream) {
    const size_t smem = shared_smem_bytes();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> ready[kMaxDevices];  // the kernel's shared-memory limit, raised once per device
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(shr::shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.num_parts, 1, 1);
    cfg.blockDim = dim3(shr::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, shr::shared_kernel, map_k, map_v, map_q, p);
}

cudaError_t launch_shared_merge(const SharedParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * (int64_t)p.total_rows + shr::kMergeWarps - 1) / shr::kMergeWarps), 1, 1);
    cfg.blockDim = dim3(32 * shr::kMergeWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shr::merge_kernel, p);
}

}  // namespace mla
