// chunk_attn.cu: attention of a chunk of new tokens of each sequence over its paged cache
// (pa_chunk_attn) on the 5th-generation tensor cores.
//
// Source: "nano-vLLM Part 4", section 3 (attention over the cached history through a block table);
// smzdm nano-vLLM deep dive, "GPU执行优化" (cu_seqlens mark sequence boundaries).
//
// The mathematics: new token t of a sequence with n keys and c new tokens sits at position
// p = n - c + t and sees keys max(0, p - window + 1) .. p. Its row of every query head is a softmax
// over scale * q.K in base 2 with a running maximum and sum (fp32); a key range can be cut anywhere
// and the pieces (m, l, O) joined by 2^(m - max m).
//
// Work: the query rows that share a kv head's keys are packed into one tile, row = token * G + head
// of the group, so a chunk of 16 tokens with groups of 8 fills the 128 rows of one matrix
// instruction. An item is two such row tiles (A, B; B empty for short chunks) of one sequence and
// kv head against all their keys, 128 at a time. The (item, key tile) pairs of the whole call lie
// on one line that is cut into equal shares, one per CTA, whatever the lengths are: one long
// sequence fills the machine as a large batch does. A CTA's range touches at most two items that it
// shares with others, one at each end: their pieces go to the workspace and a second kernel joins
// them. The shares follow from the device's own lengths, so that the call needs no host copy of them
// and can be captured.
//
//   warp 3      scheduler: walks the CTA's share and queues its segments (item, key tile range).
//   warp 0      producer: TMA loads of each segment's Q tiles and of 128-key K and V tiles through
//               the block table, 128-byte swizzled, into a ring in the order the MMAs take them (K0,
//               K1, V0, K2, V1, ...). Blocks of fewer than 8 aligned rows are gathered row by row
//               with cp.async into the same layout.
//   warps 1, 2  one MMA issuer per row tile: S = Q K^T and O += P V, accumulators in tensor memory.
//   warps 4-11  softmax, thread = one row = one TMEM lane (4-7 tile A, 8-11 tile B): as S is read it
//               is released for the next key tile's QK; O is rescaled only when the row's maximum
//               grew by more than 2^8. Warps without rows only keep the barriers going.
// Every wait is bounded (PA_DEVERR_TIMEOUT); on a timeout every role drains what it started.
//
// Bound by the softmax warps' latency: two chunks of 2k tokens at contexts of 12-16k (16/8 heads x 128, bf16)
// 333-347 us = 1.28-1.23 PFLOP/s, the tensor pipe 58 % active, a key tile of both row tiles every 3300 clocks against
// 1024 of MMAs and as many of exponentials. Two threads a row, which exchange maxima: 8 % slower; P
// stored while the exponentials run: 4 % slower.
#include <type_traits>

#include "chunk_wide.cuh"
#include "tensor_map.h"

namespace pa {

namespace {

using namespace chunk;

constexpr int kPTile = BM * BN * 2;  // P, and the output stage
constexpr int kRing = 3;
enum {
    B_QFULL = 0,               // the segment's Q tiles landed
    B_QEMPTY,                  // both issuers are past the segment's last QK
    B_FULL,                    // + slot: a K/V tile landed
    B_EMPTY = B_FULL + kRing,  // + slot: both issuers' MMAs are done with it
    B_S = B_EMPTY + kRing,     // + h: S is in TMEM
    B_F = B_S + 2,             // + h: the softmax has read S (4 arrivals)
    B_P = B_F + 2,             // + h: P is written (4 arrivals)
    B_O = B_P + 2,             // + h: O += P V is done, P's buffer is free
    B_OFREE = B_O + 2,         // + h: the segment's O has been read out (4 arrivals)
    B_END = B_OFREE + 2,       // + h: every MMA of that issuer has completed
    B_VZ = B_END + 2,          // a V tile's rows outside the keys are zero
    B_VZACK,                   // issuer B has waited for that (A never runs two zeroings ahead)
    B_IFULL = B_VZACK + 1,     // + k: segment k of the queue is published
    B_IEMPTY = B_IFULL + 2,    // + k: every role has read it
    NBAR = B_IEMPTY + 2
};
template <int HD>
struct Layout {
    static constexpr int kHalves = HD / 64;
    static constexpr int kQ = BM * HD * 2;
    static constexpr int kKV = BN * HD * 2;
    static constexpr uint32_t kKVDesc = kKV >> 4;
    static constexpr int OFF_QA = 0, OFF_QB = kQ, OFF_PA = 2 * kQ, OFF_PB = OFF_PA + kPTile,
                         OFF_RING = OFF_PB + kPTile, OFF_BAR = OFF_RING + kRing * kKV;
    static constexpr int OFF_ITEMS = OFF_BAR + NBAR * 8;
    static constexpr int OFF_BAD = OFF_ITEMS + 2 * static_cast<int>(sizeof(SegInfo));
    static constexpr int OFF_PLAN = (OFF_BAD + kBadRing * 4 + 15) / 16 * 16;  // 12 warp sums, then the share
    static constexpr int OFF_MISC = OFF_PLAN + 12 * 8 + static_cast<int>(sizeof(Share));
    static constexpr int kSmem = OFF_MISC + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr size_t kPieceFloats = wide_piece_floats(HD);
};

template <class E, int HD, bool kGather>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkParams p) {
    using T = typename E::T;
    using Lay = Layout<HD>;
    constexpr int OFF_QA = Lay::OFF_QA, OFF_QB = Lay::OFF_QB, OFF_PA = Lay::OFF_PA, OFF_PB = Lay::OFF_PB,
                  OFF_RING = Lay::OFF_RING, OFF_BAR = Lay::OFF_BAR;
    constexpr int kHalves = Lay::kHalves;
    constexpr bool kPTmem = HD == 64;  // P in TMEM columns of its own at head dim 64
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    SegInfo *items = reinterpret_cast<SegInfo *>(smem + Lay::OFF_ITEMS);
    volatile int *bad_seg = reinterpret_cast<volatile int *>(smem + Lay::OFF_BAD);
    long long *plan = reinterpret_cast<long long *>(smem + Lay::OFF_PLAN);
    Share *share = reinterpret_cast<Share *>(plan + 12);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + OFF_BAR + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    T *out = static_cast<T *>(p.out);

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            uint32_t count = 1;
            if (i == B_QEMPTY || (i >= B_EMPTY && i < B_EMPTY + kRing)) count = 2;
            if ((i >= B_F && i < B_O) || (i >= B_OFREE && i < B_END)) count = 4;
            if (i >= B_IEMPTY) count = kItemReaders;
            mbar_init(bar(i), count);
        }
        *abort_flag = 0;
        for (int i = 0; i < kBadRing; ++i) bad_seg[i] = 0;
        fence_mbar_init();
    }

    // Launched beside what precedes it in the stream: nothing that it wrote is read, and nothing that it reads is
    // written, before it has finished (the set-up above takes place meanwhile).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Tensor memory is taken only now, and the joining kernel (and with it what follows) let in only when it is
    // there: no block holds tensor memory while it waits for another grid, whose blocks on this SM may want some.
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), 512);
    plan_share(p, plan, share);
    zero_bad_sequences<T, HD>(p);
    if (tid == 0) p.recs[blockIdx.x].valid = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel waits for this grid itself
    const uint32_t tmem = *tmem_slot;

    // every role reads the segments in the same order: segment n sits in queue entry n % 2
    auto read_seg = [&](int n, SegInfo &it) -> bool {
        if (!warp_wait(bar(B_IFULL + (n & 1)), (n >> 1) & 1, abort_flag)) return false;
        it = items[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IEMPTY + (n & 1)));
        return true;
    };
    auto has_b = [&](const SegInfo &it) { return it.tok > p.tt; };

    if (warp == 3) {
        // ================================== scheduler ==================================
        int published = 0;
        auto publish = [&](const SegInfo &it) {
            if (!warp_wait(bar(B_IEMPTY + (published & 1)), ((published >> 1) & 1) ^ 1, abort_flag)) return false;
            if (lane == 0) {
                items[published & 1] = it;
                mbar_arrive(bar(B_IFULL + (published & 1)));
            }
            __syncwarp();
            ++published;
            return true;
        };
        const bool ok = walk_share(p, *share, publish);
        if (!ok && lane == 0) give_up(p.err, abort_flag);
    } else if (warp == 0) {
        // =================================== producer ===================================
        prefetch_tmap(&p.tm_q);
        if constexpr (!kGather) {
            prefetch_tmap(&p.tm_k);
            prefetch_tmap(&p.tm_v);
        }
        const int R = p.box_rows, nbox = BN / R;
        const uint32_t box_bytes = static_cast<uint32_t>(R) * 128;
        long long L = 0;  // tiles loaded
        int n = 0;        // segments taken
        bool ok = true;
        constexpr int kRowsLane = kGather ? BN / 32 : 1;
        struct Rows {
            long long r[kRowsLane];
        };
        // the rows this lane loads of key tile j: its box's first row, or rows lane, lane + 32, ...
        auto rows_of = [&](const SegInfo &it, int j, int seg_no) {
            Rows w;
#pragma unroll
            for (int i = 0; i < kRowsLane; ++i) {
                const int pos = j * BN + (kGather ? lane + 32 * i : lane * R);
                w.r[i] = kGather || lane < nbox ? pool_row(p, it, pos, kGather ? pos : pos + R - 1, bad_seg, seg_no) : -1;
            }
            return w;
        };
        // gathered tiles are announced one load late, when their copies have landed
        auto announce = [&](long long i) {
            if (!kGather || i < 0) return;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_FULL + static_cast<int>(i % kRing)));
        };
        auto load_tile = [&](const SegInfo &it, const Rows &w, bool is_v) -> bool {
            const int slot = static_cast<int>(L % kRing);
            const uint32_t base = sbase + OFF_RING + slot * Lay::kKV;
            if (!warp_wait(bar(B_EMPTY + slot), static_cast<uint32_t>((L / kRing) & 1) ^ 1, abort_flag)) return false;
            if constexpr (kGather) {
                gather_tile<T, HD>(base, static_cast<const T *>(is_v ? p.v_cache : p.k_cache), w.r, p.Hkv, it.g);
                cp_async_wait<1>();
                announce(L - 1);
            } else {
                const uint32_t bytes = __popc(__ballot_sync(kFull, w.r[0] >= 0)) * box_bytes * kHalves;
                if (lane == 0) mbar_arrive_expect_tx(bar(B_FULL + slot), bytes);
                __syncwarp();
                if (w.r[0] >= 0) {
                    const uint32_t dst = base + lane * R * 128;
                    for (int half = 0; half < kHalves; ++half)
                        tma_load_3d(dst + half * kHalf, is_v ? &p.tm_v : &p.tm_k, half * 64, it.g,
                                    static_cast<int>(w.r[0]), bar(B_FULL + slot));
                }
            }
            ++L;
            return true;
        };
        SegInfo cur{};
        Rows wc{}, wn{};
        while (ok) {
            if (!(ok = read_seg(n, cur)) || cur.j0 == cur.j1) break;
            wc = rows_of(cur, cur.j0, n);
            // this segment's Q once both issuers are past the previous segment's last QK, its first K before
            if (!(ok = load_tile(cur, wc, false))) break;
            if (n > 0 && !(ok = warp_wait(bar(B_QEMPTY), (n - 1) & 1, abort_flag))) break;
            if (lane == 0) {
                const int tiles = has_b(cur) ? 2 : 1;
                const uint32_t half_bytes = static_cast<uint32_t>(p.tt) * p.G * 128;
                mbar_arrive_expect_tx(bar(B_QFULL), tiles * kHalves * half_bytes);
                for (int h = 0; h < tiles; ++h)
                    for (int half = 0; half < kHalves; ++half)
                        tma_load_3d(sbase + (h ? OFF_QB : OFF_QA) + half * kHalf, &p.tm_q, half * 64, cur.g * p.G,
                                    cur.tok0 + h * p.tt, bar(B_QFULL));
            }
            __syncwarp();
            if (cur.j0 + 1 < cur.j1) wn = rows_of(cur, cur.j0 + 1, n);
            for (int j = cur.j0 + 1; ok && j < cur.j1; ++j) {
                const Rows w = wn;
                if (j + 1 < cur.j1) wn = rows_of(cur, j + 1, n);  // in flight while this tile is loaded
                ok = load_tile(cur, w, false) && load_tile(cur, wc, true);
                wc = w;
            }
            ok = ok && load_tile(cur, wc, true);
            ++n;
        }
        if constexpr (kGather) {
            cp_async_wait<0>();
            if (ok) announce(L - 1);
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        // no copy may still be in flight at exit: the last load of every slot, the last Q
        if (lane == 0) {
            if (!kGather)
                for (long long i = L > kRing ? L - kRing : 0; i < L; ++i)
                    if (!mbar_wait(bar(B_FULL + static_cast<int>(i % kRing)), static_cast<uint32_t>((i / kRing) & 1)))
                        give_up(p.err, abort_flag);
            if (n > 0 && !mbar_wait(bar(B_QFULL), (n - 1) & 1)) give_up(p.err, abort_flag);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ============================ MMA issuer of one row tile =============================
        const int h = warp - 1;
        constexpr uint32_t IQK = idesc_f16(BM, BN, E::kIsBf16, false);
        constexpr uint32_t IPV = idesc_f16(BM, HD, E::kIsBf16, true);
        const uint64_t dq = smem_desc_sw128(sbase + (h ? OFF_QB : OFF_QA), 16, 1024);
        const uint64_t dp = smem_desc_sw128(sbase + (h ? OFF_PB : OFF_PA), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(sbase + OFF_RING, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(sbase + OFF_RING, kHalf, 1024);
        const uint32_t s_tm = tmem + (h ? 128 : 0), o_tm = tmem + 256 + (h ? 128 : 0);
        const uint32_t p_tm = tmem + 256 + HD + (h ? 128 : 0);
        auto qk = [&](int slot) {  // S = Q K^T
            const uint64_t kb = dk0 + slot * Lay::kKVDesc;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                tc_mma_ss(s_tm, dq + off, kb + off, IQK, kk > 0);
            }
        };
        auto pv = [&](int slot, bool acc) {  // O += P V
            const uint64_t vb = dv0 + slot * Lay::kKVDesc;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                if constexpr (kPTmem)
                    tc_mma_ts(o_tm, p_tm + kk * 8, vb + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
                else
                    tc_mma_ss(o_tm, dp + off, vb + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
            }
        };
        long long ci = 0;  // tiles consumed
        auto next_load = [&](int &slot) -> bool {
            slot = static_cast<int>(ci % kRing);
            const bool r = warp_wait(bar(B_FULL + slot), static_cast<uint32_t>((ci / kRing) & 1), abort_flag);
            ++ci;
            return r;
        };
        // QK of the next key tile; `last`: the segment's last. Without rows in this row tile (B of a
        // short chunk) the tile is only handed back.
        auto issue_qk = [&](bool rows, bool last) -> bool {
            int slot;
            if (!next_load(slot)) return false;
            tc_fence_after();
            if (lane == 0) {
                if (rows) {
                    qk(slot);
                    tc_commit(bar(B_S + h));
                    tc_commit(bar(B_EMPTY + slot));
                    if (last) tc_commit(bar(B_QEMPTY));
                } else {
                    mbar_arrive(bar(B_EMPTY + slot));
                    if (last) mbar_arrive(bar(B_QEMPTY));
                }
            }
            __syncwarp();
            return true;
        };
        int zt = 0;       // zeroed tiles that both row tiles take
        long long t = 0;  // key tiles of this row tile so far
        int done = 0;     // segments of this row tile so far
        SegInfo cur{};
        bool ok = true;
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, cur)) || cur.j0 == cur.j1) break;
            const bool rows = h == 0 || has_b(cur);
            if (!(ok = warp_wait(bar(B_QFULL), n & 1, abort_flag))) break;
            // S(t) as soon as the softmax holds S(t - 1) in registers
            if (rows && t > 0 && !(ok = warp_wait(bar(B_F + h), static_cast<uint32_t>((t - 1) & 1), abort_flag))) break;
            if (!(ok = issue_qk(rows, cur.j0 + 1 == cur.j1))) break;
            for (int j = cur.j0; j < cur.j1; ++j, t += rows) {
                if (j + 1 < cur.j1) {
                    if (rows && !(ok = warp_wait(bar(B_F + h), static_cast<uint32_t>(t & 1), abort_flag))) break;
                    if (!(ok = issue_qk(rows, j + 2 == cur.j1))) break;
                }
                // PV of key tile j
                int slot;
                if (!(ok = next_load(slot))) break;
                const int z0 = max(cur.n_lo - j * BN, 0), z1 = min(cur.n_end - j * BN, BN);  // rows that hold keys
                if (rows && (z0 > 0 || z1 < BN)) {
                    const bool both = has_b(cur);
                    if (h == 0) {
                        if (both && zt > 0 &&
                            !(ok = warp_wait(bar(B_VZACK), static_cast<uint32_t>((zt - 1) & 1), abort_flag)))
                            break;
                        zero_rows<HD>(smem + OFF_RING + slot * Lay::kKV, z0, z1);
                        if (both && lane == 0) mbar_arrive(bar(B_VZ));
                    } else {
                        if (!(ok = warp_wait(bar(B_VZ), zt & 1, abort_flag))) break;
                        if (lane == 0) mbar_arrive(bar(B_VZACK));
                    }
                    zt += both;
                }
                if (rows && !(ok = warp_wait(bar(B_P + h), static_cast<uint32_t>(t & 1), abort_flag))) break;
                // the previous segment's output must be out of TMEM before its O is overwritten
                if (rows && j == cur.j0 && done > 0 &&
                    !(ok = warp_wait(bar(B_OFREE + h), (done - 1) & 1, abort_flag)))
                    break;
                tc_fence_after();
                if (lane == 0) {
                    if (rows) {
                        pv(slot, j > cur.j0);
                        tc_commit(bar(B_O + h));
                        tc_commit(bar(B_EMPTY + slot));
                    } else {
                        mbar_arrive(bar(B_EMPTY + slot));
                    }
                }
                __syncwarp();
            }
            done += rows;
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        if (lane == 0) {  // every MMA this thread issued has finished before the TMEM is freed
            tc_commit(bar(B_END + h));
            if (!mbar_wait(bar(B_END + h), 0)) give_up(p.err, abort_flag);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // =================================== softmax ===================================
        const int h = warp >= 8 ? 1 : 0;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t srow = tmem + lane_off + (h ? 128 : 0);
        const uint32_t orow = tmem + lane_off + 256 + (h ? 128 : 0);
        unsigned char *ptile = smem + (h ? OFF_PB : OFF_PA);
        unsigned char *prow = ptile + r * 128;  // half 0
        const uint32_t s_full = bar(B_S + h), s_free = bar(B_F + h), p_full = bar(B_P + h);
        const uint32_t o_done = bar(B_O + h), o_free = bar(B_OFREE + h);
        const int row_tok = p.div_g(r);  // this row's token within its tile
        long long t = 0;
        bool ok = true;
        SegInfo it{};
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, it)) || it.j0 == it.j1) break;
            const int tok = it.tok - h * p.tt;  // tokens of this row tile
            if (tok <= 0) continue;
            const int rows = min(tok, p.tt) * p.G;
            const bool live = quarter * 32 < rows;  // this warp holds rows
            const int pos = it.p0 + h * p.tt + row_tok;
            const int lim = r < rows ? pos + 1 : 0;  // the keys this row sees: [lo, lim)
            const int lo = p.window > 0 ? pos - p.window + 1 : 0;
            float m_use = -INFINITY, l = 0.f;
            for (int j = it.j0; j < it.j1; ++j, ++t) {
                if (!(ok = warp_wait(s_full, static_cast<uint32_t>(t & 1), abort_flag))) break;
                if (!live) {
                    if (lane == 0) mbar_arrive(s_free);
                    // P's barrier counts tiles: not before the previous tile's PV has been issued
                    if (t > 0 && !(ok = warp_wait(o_done, static_cast<uint32_t>((t - 1) & 1), abort_flag))) break;
                    if (lane == 0) mbar_arrive(p_full);
                    continue;
                }
                tc_fence_after();
                uint32_t sv[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t(&chunk)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * c);
                    tmem_ld32(srow + c * 32, chunk);
                }
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
                const int n0 = j * BN;
                if (n0 + BN > lim) {
                    const int from = lim - n0;
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e >= from) sv[e] = 0xff800000u;  // -inf
                }
                if (n0 < lo) {
                    const int to = lo - n0;
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e < to) sv[e] = 0xff800000u;
                }
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 2)
                    mq[(e >> 1) & 3] = max3(mq[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                const float mraw = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                const float mx = mraw == -INFINITY ? -INFINITY : mraw * p.scale_log2;
                // the reference moves only when the maximum grew by more than 2^8 (or was unset): the
                // sum uses the same reference, so the result is exact, and P stays below 2^8
                const bool need = mx > m_use + 8.f;
                const float f = need ? fast_exp2(m_use - mx) : 1.f;
                if (need) m_use = mx;
                const float mu = m_use == -INFINITY ? 0.f : m_use;
                const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(-mu, -mu);
                uint64_t l2 = f2_pack(0.f, 0.f);
                uint32_t pk[64];
#pragma unroll
                for (int e = 0; e < 128; e += 2) {
                    const uint64_t x2 = f2_fma(u2_pack(sv[e], sv[e + 1]), sc2, nm2);
                    const float p0 = fast_exp2(f2_lo(x2)), p1 = fast_exp2(f2_hi(x2));
                    l2 = f2_add(l2, f2_pack(p0, p1));
                    // P is rounded to the storage type (the tensor cores' operand), the sum is not
                    pk[e >> 1] = E::pack2(p0, p1);
                }
                l = l * f + (f2_lo(l2) + f2_hi(l2));
                if (t > 0) {  // the previous tile's PV has consumed P and completed O
                    if (!(ok = warp_wait(o_done, static_cast<uint32_t>((t - 1) & 1), abort_flag))) break;
                    tc_fence_after();
                }
                if (!kPTmem && j == it.j0) {  // the warp's rows may still leave for the previous segment
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                }
                if constexpr (kPTmem) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        tmem_st4(orow + HD + 4 * c, pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                    tmem_wait_st();
                } else {
                    // 128-byte swizzle: 16-byte chunk q of a half sits at q ^ (r % 8)
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        *reinterpret_cast<uint4 *>(prow + (q >> 3) * kHalf + (((q & 7) ^ (r & 7)) << 4)) =
                            make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                }
                if (j > it.j0 && __any_sync(kFull, need)) {
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(orow + c * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                        tmem_st32(orow + c * 32, ov);
                    }
                    tmem_wait_st();
                }
                if constexpr (!kPTmem) fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (ok) ok = warp_wait(o_done, static_cast<uint32_t>((t - 1) & 1), abort_flag);
            if (!ok) break;
            if (!live) {
                if (lane == 0) mbar_arrive(o_free);
                continue;
            }
            tc_fence_after();
            const bool bad = bad_seg[n & (kBadRing - 1)] == n + 1;  // a table entry of the segment was bad
            if (it.part >= 0) {
                // a piece: O unnormalised, with its maximum and sum (sum -1: bad)
                float *w = p.pieces + (static_cast<size_t>(blockIdx.x) * 2 + it.part) * Lay::kPieceFloats + h * 128 + r;
                if (r < rows) {
                    w[0] = m_use;
                    w[256] = bad ? -1.f : l;
                }
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(orow + c * 32, v);
                    tmem_wait_ld();
                    if (r < rows) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[512 + (c * 32 + e) * 256] = __uint_as_float(v[e]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
                continue;
            }
            const float inv = l > 0.f && !bad ? 1.f / l : 0.f;
            uint32_t acc[HD];
#pragma unroll
            for (int c = 0; c < HD / 32; ++c)
                tmem_ld32(orow + c * 32, *reinterpret_cast<uint32_t(*)[32]>(acc + 32 * c));
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            // The warp's rows leave through its rows of the P buffer, swizzled like P: by TMA when they are whole
            // tokens, all of the item, else 16 bytes a lane, whole rows.
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < HD / 8; ++c)
            {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)  // bad: zero, whatever the accumulator holds
                    o[e] = bad ? 0u : E::pack2(__uint_as_float(acc[c * 8 + e * 2]) * inv, __uint_as_float(acc[c * 8 + e * 2 + 1]) * inv);
                *reinterpret_cast<uint4 *>(prow + (c >> 3) * kHalf + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (quarter * 32 + 32 <= rows && p.store_tok > 0) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (int half = 0; half < kHalves; ++half)
                        tma_store_3d(&p.tm_o, half * 64, it.g * p.G, it.tok0 + h * p.tt + quarter * p.store_tok,
                                     smem_addr(ptile + half * kHalf + quarter * 32 * 128));
                    bulk_commit();
                }
                __syncwarp();
                continue;
            }
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < HD / 8; ++i) {
                const int k = i * 32 + lane, rr = quarter * 32 + k / (HD / 8), c = k % (HD / 8);
                const uint4 u = *reinterpret_cast<const uint4 *>(ptile + (c >> 3) * kHalf + rr * 128 +
                                                                 (((c & 7) ^ (rr & 7)) << 4));
                if (rr < rows) {
                    const int in_tile = p.div_g(rr);
                    const int tk = it.tok0 + h * p.tt + in_tile, head = it.g * p.G + rr - in_tile * p.G;
                    *reinterpret_cast<uint4 *>(out + (static_cast<size_t>(tk) * p.Hq + head) * HD + c * 8) = u;
                }
            }
            __syncwarp();  // the rows are read before the next tile's P overwrites them
        }
        if (lane == 0) bulk_wait_all();  // the output stores are complete before the CTA exits
        __syncwarp();
        if (!ok && lane == 0) give_up(p.err, abort_flag);
    }
    // ------------------------------------------------------------------------------------------
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------------
// launch
// ------------------------------------------------------------------------------------------

// [rows, heads, hd] tensor, box of box_rows x box_heads x 64 columns, 128-byte swizzle
bool encode(CUtensorMap *m, const void *base, pa_dtype dt, int heads, int hd, long long rows, int box_heads,
            int box_rows) {
    return encode_rows_3d(m, base, dt, heads, hd, rows, box_heads, box_rows, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <class E, int HD, bool kGather>
cudaError_t launch_typed(const ChunkParams &prm, cudaStream_t stream) {
    auto kern = chunk_attn_kernel<E, HD, kGather>;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD>::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev] = 1;
    }
    const unsigned P = device_sm_count();
    // Both kernels are launched beside what precedes them (programmatic dependent launch): the set-up of the first
    // overlaps the end of the call before, and the second is on the SMs when the last share ends.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(P);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<HD>::kSmem;
    if ((e = cudaLaunchKernelEx(&cfg, kern, prm)) != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    const int rows = prm.max_seqlen_q > prm.tt ? 256 : (prm.max_seqlen_q * prm.G + kJoinRows - 1) / kJoinRows * kJoinRows;
    cfg.gridDim = dim3(P, rows / kJoinRows, HD / kJoinCols);
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<E, HD>, prm);
}

size_t piece_bytes(int D) { return wide_piece_floats(D) * 4; }

}  // namespace

size_t chunk_attn_workspace(int D) {
    const size_t P = device_sm_count();
    return P * 2 * piece_bytes(D) + P * sizeof(PieceRec);
}

cudaError_t launch_chunk_attn(const ChunkArgs &a, cudaStream_t stream) {
    ChunkParams prm{};
    int R = 1;  // rows per K/V box: the largest power of two dividing the block size, at most 128
    while (R < 128 && a.block_size % (2 * R) == 0) R *= 2;
    const bool gather = R < 8;  // less than a swizzle atom of 8 rows
    prm.G = a.Hq / a.Hkv;
    prm.inv_g = (65536 + prm.G - 1) / prm.G;
    prm.tt = BM / prm.G;
    // Chunks of at most 64 query rows a kv head take the form with keys as the rows: an item is a
    // whole chunk, its Q box as many tokens as the columns hold.
    const long long rows = static_cast<long long>(a.max_seqlen_q) * prm.G;
    const bool narrow = rows <= 64;
    if (narrow) {
        prm.tt = prm.item_tok = (gather || rows > 32 ? 64 : rows > 16 ? 32 : 16) / prm.G;
    } else {
        prm.item_tok = 2 * prm.tt;
    }
    const long long krows = static_cast<long long>(a.num_blocks) * a.block_size;
    if (!encode(&prm.tm_q, a.q, a.dtype, a.Hq, a.D, a.total_q, prm.G, prm.tt)) return cudaErrorInvalidValue;
    if (!gather && (!encode(&prm.tm_k, a.k_cache, a.dtype, a.Hkv, a.D, krows, 1, R) ||
                    !encode(&prm.tm_v, a.v_cache, a.dtype, a.Hkv, a.D, krows, 1, R)))
        return cudaErrorInvalidValue;
    // a warp's 32 output rows as one box, where they are whole tokens
    prm.store_tok = 32 % prm.G == 0 && BM % prm.G == 0 ? 32 / prm.G : 0;
    if (!narrow && prm.store_tok > 0 &&
        !encode(&prm.tm_o, a.out, a.dtype, a.Hq, a.D, a.total_q, prm.G, prm.store_tok))
        return cudaErrorInvalidValue;
    prm.cu_q = a.cu_q;
    prm.ctx = a.ctx;
    prm.block_tables = a.block_tables;
    prm.k_cache = a.k_cache;
    prm.v_cache = a.v_cache;
    prm.out = a.out;
    prm.err = a.err;
    const size_t P = device_sm_count();
    prm.pieces = static_cast<float *>(a.workspace);
    prm.recs = reinterpret_cast<PieceRec *>(static_cast<char *>(a.workspace) + P * 2 * piece_bytes(a.D));
    prm.S = a.S, prm.Hq = a.Hq, prm.Hkv = a.Hkv;
    prm.max_blocks = a.max_blocks, prm.num_blocks = a.num_blocks;
    prm.total_q = a.total_q, prm.max_seqlen_q = a.max_seqlen_q, prm.window = a.window;
    prm.box_rows = gather ? 1 : R;
    prm.geom.block_size = a.block_size;
    prm.geom.shift = log2_if_pow2(a.block_size);
    prm.scale_log2 = a.scale * kLog2e;
    if (narrow) return launch_chunk_narrow(prm, a.dtype, a.D, gather, stream);
    auto go = [&](auto e, auto hd) {
        using E = decltype(e);
        constexpr int HD = decltype(hd)::value;
        return gather ? launch_typed<E, HD, true>(prm, stream) : launch_typed<E, HD, false>(prm, stream);
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (a.dtype == PA_BF16) return a.D == 64 ? go(BF16{}, I64{}) : go(BF16{}, I128{});
    return a.D == 64 ? go(F16{}, I64{}) : go(F16{}, I128{});
}

}  // namespace pa
