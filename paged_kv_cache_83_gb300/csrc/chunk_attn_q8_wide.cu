// chunk_attn_q8_wide.cu: pa_chunk_attn_q8 for chunks of more than 64 query rows a kv head (tokens x group), such as pieces of
// long prompts.
//
// The mathematics is chunk_attn.cu's, with the scales of an 8-bit cache: scores ks_j (scale q.K8_j), weights p_j,
// O = sum (vs_j p_j) V8_j. In bf16 the weights are multiplied by vs_j before they are rounded; fp16 has not the range for that
// and takes vs_j into the exponent, w_j = 2^(x_j - m) with x_j = s_j + log2 vs_j, and the sum is of w_j / vs_j.
//
// The cache's e4m3 rows are widened to the storage type, exactly, on their way to shared memory, once for the 256 query rows of
// an item, and queries and weights stay whole operands. (As sums of e4m3 pieces beside rows that are used as they lie, the
// weights cost the softmax three conversions each: that form, of 64 rows an item, took 955 us where this one takes 533: two
// chunks of 2k tokens at contexts of 12-16k, 16/8 heads x 128, bf16.) A producer brings halves of tiles by TMA and four warps
// widen them into the swizzled tile that the matrix instructions read (loaders that copied for themselves: 675 us). There is
// room for one buffer of K and one of V; a tile's K is wanted a whole softmax before its V.
//
// Bound by shared memory and by the softmax and loader warps together: at that shape 0.80 PFLOP/s, 0.42 of the burst peak, a key
// tile of both row tiles every 5250 clocks, of which the operands, P, the rows' way through the stage and the numbers of the keys
// keep shared memory busy for some 4000. Without the widening it would be 468 us, without the numbers of the keys 516, without
// both 382. Measured and not kept: P in the columns of its S, the next QK behind this PV, and two buffers of K and V
// in P's place (584); sixteen softmax warps, half of a row's keys each (568, registers spill); V widened with its scales
// (550); 184 registers for the softmax (537); for bf16, too, log2 vs in the exponent and 1 / vs in the sum (587).
//
// The softmax spills a little at its 176 registers (head dim 128: bf16 20 bytes stored and 28 loaded, fp16 94 and 120; 64: bf16 4 and 20).
//
//   warp 3        scheduler, as in chunk_attn.cu; brings the queries of a segment by TMA
//   warp 0        producer: halves of K and V tiles as they lie in the cache, and the scales of their keys
//   warps 1, 2    one MMA issuer per row tile
//   warps 4-11    softmax, a thread a query row
//   warps 12-15   loaders: K and V tiles, and the numbers of a key: scale * ks, and vs, or log2 vs and 1 / vs
#include <type_traits>

#include "chunk_wide.cuh"
#include "tensor_map.h"

namespace pa {

namespace {

using namespace chunk;

constexpr int kWideThreads = 512;
constexpr int kWideReaders = 15;  // roles that read the queue of segments, by warp: all but the scheduler
constexpr int kKeyRing = 4;       // key tiles whose numbers are held
constexpr int kQueue = 4;         // segments
constexpr int kStages = 3;        // halves of tiles (64 keys) that are under way as they lie in the cache
constexpr int kHalfKeys = BN / 2;
// registers of a thread by warpgroup: 72 + 2 * 176 + 88 = 4 * 128
constexpr int kRegsSmall = 72, kRegsSoftmax = 176, kRegsLoad = 88;

struct WideParams : ChunkParams {
    const float *k_scale, *v_scale;  // [num_blocks, Hkv, block_size]
};

enum {
    W_QFULL = 0,            // the segment's Q tiles landed
    W_QEMPTY,               // both issuers are past the segment's last QK
    W_KFULL,                // a K tile is written (the loaders' 4 warps), with its keys' numbers
    W_KEMPTY,               // both issuers' QKs are done with it
    W_VFULL,                // a V tile is written
    W_VEMPTY,               // both issuers' PVs are done with it
    W_SFULL,                // + half tile % kStages: it landed, with its keys' scales if it is of K (the tile, and 32 lanes' copies)
    W_SEMPTY = W_SFULL + kStages,  // the loaders have read it (4 arrivals)
    W_KEYS = W_SEMPTY + kStages,   // + tile % kKeyRing: the keys' numbers are written (4 arrivals)
    W_S = W_KEYS + kKeyRing,  // + h: S is in TMEM
    W_F = W_S + 2,          // + h: the softmax has read S (4 arrivals)
    W_P = W_F + 2,          // + h: P is written (4 arrivals)
    W_O = W_P + 2,          // + h: O += P V is done, P's buffer is free
    W_OFREE = W_O + 2,      // + h: the segment's O has been read out (4 arrivals)
    W_END = W_OFREE + 2,    // + h: every MMA of that issuer has completed
    W_IFULL = W_END + 2,    // + k: segment k of the queue is published
    W_IEMPTY = W_IFULL + kQueue,  // + k: every role has read it
    W_BARS = W_IEMPTY + kQueue
};
template <int HD>
struct LayWide {
    static constexpr int kHalves = HD / 64;
    static constexpr int kQ = BM * HD * 2, kKV = BN * HD * 2, kP = BM * BN * 2;
    static constexpr int OFF_QA = 0, OFF_QB = kQ, OFF_PA = 2 * kQ, OFF_PB = OFF_PA + kP, OFF_K = OFF_PB + kP, OFF_V = OFF_K + kKV,
                         OFF_STAGE = OFF_V + kKV, OFF_SCALE = OFF_STAGE + kStages * kHalfKeys * HD,  // of K, then of V
                         OFF_KEYS = OFF_SCALE + kStages * 2 * kHalfKeys * 4;  // per tile of the ring: scale * ks [BN], vs or log2 vs [BN], 1 / vs [BN]
    static constexpr int OFF_BAR = OFF_KEYS + kKeyRing * 3 * BN * 4;
    static constexpr int OFF_ITEMS = OFF_BAR + W_BARS * 8;
    static constexpr int OFF_BAD = OFF_ITEMS + kQueue * static_cast<int>(sizeof(SegInfo));
    static constexpr int OFF_PLAN = (OFF_BAD + kBadRing * 4 + 15) / 16 * 16;  // 16 warp sums, then the share
    static constexpr int OFF_MISC = OFF_PLAN + 16 * 8 + static_cast<int>(sizeof(Share));
    static constexpr int kSmem = OFF_MISC + 16 + 1024;
    static_assert(kSmem <= 232448 && OFF_BAR % 8 == 0, "shared memory per CTA");
};

template <int kRegs>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// Two e4m3 numbers in the upper bytes of x's halves, in 16 bits, exactly. The fields move as they are, which leaves the value
// times 2^(bias - 7): fp16 keeps its 2^-8 (the keys' numbers make up for it), bf16's 2^-120 is multiplied away. (With the
// conversion instructions e4m3 -> fp16 (-> fp32 -> bf16) the loaders took 1130 clocks for what takes them 500 so.) The pattern
// of a NaN becomes +-480: a row that held a NaN or an infinity has a scale that is not finite, which makes NaN of it.
template <class E>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t x) {
    if constexpr (!E::kIsBf16) return ((x >> 1) & 0x3f803f80u) | (x & 0x80008000u);
    uint32_t y = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
    asm("mul.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x7b807b80u));  // 2^120 twice
    return y;
}
template <class E>
__device__ __forceinline__ uint4 widen_e4m3x8(uint32_t a, uint32_t b) {
    return make_uint4(widen_e4m3x2<E>(__byte_perm(a, 0, 0x1404)), widen_e4m3x2<E>(__byte_perm(a, 0, 0x3424)),
                      widen_e4m3x2<E>(__byte_perm(b, 0, 0x1404)), widen_e4m3x2<E>(__byte_perm(b, 0, 0x3424)));
}

template <class E, int HD, bool kGather>
__global__ void __launch_bounds__(kWideThreads, 1) chunk_q8_wide_kernel(const __grid_constant__ WideParams p) {
    using T = typename E::T;
    using Lay = LayWide<HD>;
    constexpr int kHalves = Lay::kHalves;
    constexpr bool kPTmem = HD == 64;  // P in TMEM columns of its own at head dim 64
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    SegInfo *items = reinterpret_cast<SegInfo *>(smem + Lay::OFF_ITEMS);
    volatile int *bad_seg = reinterpret_cast<volatile int *>(smem + Lay::OFF_BAD);
    long long *plan = reinterpret_cast<long long *>(smem + Lay::OFF_PLAN);
    Share *share = reinterpret_cast<Share *>(plan + 16);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + Lay::OFF_BAR + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    T *out = static_cast<T *>(p.out);

    if (tid < W_BARS) {
        uint32_t count = 1;
        if (tid == W_QEMPTY || tid == W_KEMPTY || tid == W_VEMPTY) count = 2;
        if (tid == W_KFULL || tid == W_VFULL || (tid >= W_SEMPTY && tid < W_S)) count = 4;  // W_SEMPTY, W_KEYS
        if (tid >= W_SFULL && tid < W_SEMPTY) count = 1 + 32;
        if ((tid >= W_F && tid < W_O) || (tid >= W_OFREE && tid < W_END)) count = 4;
        if (tid >= W_IEMPTY) count = kWideReaders;
        mbar_init(bar(tid), count);
        fence_mbar_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kBadRing; ++i) bad_seg[i] = 0;
    }
    // as in chunk_attn.cu
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), 512);
    plan_share<kWideThreads>(p, plan, share);
    zero_bad_sequences<T, HD, kWideThreads>(p);
    if (tid == 0) p.recs[blockIdx.x].valid = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel waits for this grid itself
    const uint32_t tmem = *tmem_slot;

    // every role reads the segments in the same order: segment n sits in queue entry n % kQueue
    auto read_seg = [&](int n, SegInfo &it) -> bool {
        if (!short_wait(bar(W_IFULL + n % kQueue), (n / kQueue) & 1, abort_flag)) return false;
        it = items[n % kQueue];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_IEMPTY + n % kQueue));
        return true;
    };
    auto has_b = [&](const SegInfo &it) { return it.tok > p.tt; };

    if (warp < 4) {
        regs_down<kRegsSmall>();
        if (warp == 3) {
            // =========================== scheduler, and the queries ===========================
            prefetch_tmap(&p.tm_q);
            int n = 0;  // segments published
            bool ok = walk_share(p, *share, [&](const SegInfo &it) {
                if (!short_wait(bar(W_IEMPTY + n % kQueue), ((n / kQueue) & 1) ^ 1, abort_flag)) return false;
                if (lane == 0) {
                    items[n % kQueue] = it;
                    mbar_arrive(bar(W_IFULL + n % kQueue));
                }
                __syncwarp();
                if (it.j0 == it.j1) return true;
                // its queries, once both issuers are past the previous segment's last QK
                if (n > 0 && !short_wait(bar(W_QEMPTY), (n - 1) & 1, abort_flag)) return false;
                if (lane == 0) {
                    const int tiles = has_b(it) ? 2 : 1;
                    const uint32_t half_bytes = static_cast<uint32_t>(p.tt) * p.G * 128;
                    mbar_arrive_expect_tx(bar(W_QFULL), tiles * kHalves * half_bytes);
                    for (int h = 0; h < tiles; ++h)
                        for (int half = 0; half < kHalves; ++half)
                            tma_load_3d(sbase + (h ? Lay::OFF_QB : Lay::OFF_QA) + half * kHalf, &p.tm_q, half * 64, it.g * p.G,
                                        it.tok0 + h * p.tt, bar(W_QFULL));
                }
                __syncwarp();
                ++n;
                return true;
            });
            if (!ok && lane == 0) give_up(p.err, abort_flag);
            // no copy may still be in flight at exit
            if (lane == 0 && n > 0 && !mbar_wait(bar(W_QFULL), (n - 1) & 1)) give_up(p.err, abort_flag);
            __syncwarp();
        } else if (warp == 0) {
            // =================================== producer ===================================
            // Halves of K and V tiles as they lie in the cache, in the order K 0, K 1, V 0, K 2, V 1, ..., with the scales of their keys
            // with K; boxes of R rows by TMA, or (blocks of fewer than 8 aligned rows) row by row.
            if constexpr (!kGather) {
                prefetch_tmap(&p.tm_k);
                prefetch_tmap(&p.tm_v);
            }
            constexpr int kRowsLane = kGather ? BN / 32 : 1;
            const int R = p.box_rows, nbox = BN / R;
            struct Tile {
                int r[kRowsLane], id[kRowsLane];  // pool rows of the lane's boxes (keys), -1: not read; their blocks
                int g;
            };
            int next_id[kRowsLane];  // the table entries of the next tile, fetched ahead
            bool next_needed[kRowsLane];
            auto pos_of = [&](int j, int i) { return j * BN + (kGather ? lane + 32 * i : lane * R); };
            auto fetch = [&](const SegInfo &it, int j) {
                const int32_t *row = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks;
#pragma unroll
                for (int i = 0; i < kRowsLane; ++i) {
                    const int pos = pos_of(j, i);
                    next_needed[i] = (kGather || lane < nbox) && pos < it.n_end && pos + (kGather ? 0 : R - 1) >= it.n_lo;
                    next_id[i] = next_needed[i] ? ld_index(row + p.geom.block_of(pos)) : 0;
                }
            };
            auto scale_at = [&](int r, int id, int g) {
                return r + (static_cast<long long>(id) * (p.Hkv - 1) + g) * p.geom.block_size;
            };
            // of the four keys whose scales this lane copies (lanes 0-15 those of K, 16-31 of V), in a tile's first half
            const int key4 = (lane & 15) * 4, box4 = key4 / R, in_box4 = key4 - box4 * R, boxes_half = kGather ? 0 : kHalfKeys / R;
            uint32_t u = 0;  // halves loaded
            auto load = [&](const Tile &t, bool is_v) -> bool {
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf, ++u) {
                    const uint32_t slot = u % kStages, full = bar(W_SFULL) + 8 * slot;
                    if (!short_wait(bar(W_SEMPTY) + 8 * slot, ((u / kStages) & 1) ^ 1, abort_flag)) return false;
                    const uint32_t dst = sbase + Lay::OFF_STAGE + slot * kHalfKeys * HD, sc = sbase + Lay::OFF_SCALE + slot * 2 * kHalfKeys * 4;
                    if constexpr (kGather) {
                        if (lane == 0) mbar_arrive(full);
                        const unsigned char *pool = static_cast<const unsigned char *>(is_v ? p.v_cache : p.k_cache);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = hf ? t.r[2 + e] : t.r[e], id = hf ? t.id[2 + e] : t.id[e], k = lane + 32 * e;
                            if (r < 0) continue;
                            const unsigned char *src = pool + (static_cast<size_t>(r) * p.Hkv + t.g) * HD;
#pragma unroll
                            for (int c = 0; c < HD / 16; ++c) cp_async16(dst + k * HD + c * 16, src + c * 16, 16);
                            if (!is_v) {
                                const long long from = scale_at(r, id, t.g);
                                cp_async4(sc + k * 4, p.k_scale + from);
                                cp_async4(sc + (kHalfKeys + k) * 4, p.v_scale + from);
                            }
                        }
                    } else {
                        const int b = lane - hf * boxes_half;
                        const bool mine = b >= 0 && b < boxes_half && t.r[0] >= 0;
                        const uint32_t boxes = __popc(__ballot_sync(kFull, mine));
                        if (lane == 0) mbar_arrive_expect_tx(full, boxes * static_cast<uint32_t>(R) * HD);
                        __syncwarp();
                        if (mine) tma_load_3d(dst + b * R * HD, is_v ? &p.tm_v : &p.tm_k, 0, t.g, t.r[0], full);
                        if (!is_v) {
                            const int r = __shfl_sync(kFull, t.r[0], box4 + hf * boxes_half), id = __shfl_sync(kFull, t.id[0], box4 + hf * boxes_half);
                            if (r >= 0)
                                cp_async16(sc + lane * 16, (lane < 16 ? p.k_scale : p.v_scale) + scale_at(r, id, t.g) + in_box4, 16);
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
                }
                return true;
            };
            SegInfo cur{};
            Tile last{};        // whose V is still to come
            bool owed = false;
            bool ok = read_seg(0, cur);
            if (ok && cur.j0 < cur.j1) fetch(cur, cur.j0);
            int n = 0, j = cur.j0;
#pragma unroll 1
            while (ok && (cur.j0 < cur.j1 || owed)) {
                Tile t{};
                const bool there = cur.j0 < cur.j1;
                if (there) {
                    t.g = cur.g;
#pragma unroll
                    for (int i = 0; i < kRowsLane; ++i) {
                        t.id[i] = next_id[i];
                        t.r[i] = next_needed[i] ? next_id[i] * p.geom.block_size + p.geom.offset_of(pos_of(j, i)) : -1;
                        if (next_needed[i] && static_cast<unsigned>(next_id[i]) >= static_cast<unsigned>(p.num_blocks)) {
                            t.r[i] = -1;
                            bad_seg[n & (kBadRing - 1)] = n + 1;
                            raise_err(p.err, PA_DEVERR_TABLE);
                        }
                    }
                    if (j + 1 < cur.j1) fetch(cur, j + 1);  // in flight while this tile is loaded
                    ok = load(t, false);
                }
                if (ok && owed) ok = load(last, true);
                last = t;
                owed = there;
                if (ok && there && ++j == cur.j1) {
                    ok = read_seg(++n, cur);
                    if (!ok) break;
                    j = cur.j0;
                    if (cur.j0 < cur.j1) fetch(cur, j);
                }
            }
            if (!ok && lane == 0) give_up(p.err, abort_flag);
            // no copy may still be in flight at exit
            if (lane == 0)
                for (uint32_t i = u > kStages ? u - kStages : 0; i < u; ++i)
                    if (!mbar_wait(bar(W_SFULL) + 8 * (i % kStages), (i / kStages) & 1)) give_up(p.err, abort_flag);
            __syncwarp();
        } else {
            // ============================ MMA issuer of one row tile =============================
            const int h = warp - 1;
            constexpr uint32_t IQK = idesc_f16(BM, BN, E::kIsBf16, false);
            constexpr uint32_t IPV = idesc_f16(BM, HD, E::kIsBf16, true);
            const uint64_t dq = smem_desc_sw128(sbase + (h ? Lay::OFF_QB : Lay::OFF_QA), 16, 1024);
            const uint64_t dp = smem_desc_sw128(sbase + (h ? Lay::OFF_PB : Lay::OFF_PA), 16, 1024);
            const uint64_t dk = smem_desc_sw128(sbase + Lay::OFF_K, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sbase + Lay::OFF_V, kHalf, 1024);
            const uint32_t s_tm = tmem + (h ? 128 : 0), o_tm = tmem + 256 + (h ? 128 : 0);
            const uint32_t p_tm = tmem + 256 + HD + (h ? 128 : 0);
            auto qk = [&]() {  // S = Q K^T
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                    tc_mma_ss(s_tm, dq + off, dk + off, IQK, kk > 0);
                }
            };
            auto pv = [&](bool acc) {  // O += P V
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                    if constexpr (kPTmem)
                        tc_mma_ts(o_tm, p_tm + kk * 8, dv + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
                    else
                        tc_mma_ss(o_tm, dp + off, dv + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
                }
            };
            uint32_t k_tiles = 0, v_tiles = 0;  // of all segments
            uint32_t t = 0;    // key tiles of this row tile so far
            int done = 0;      // segments of this row tile so far
            SegInfo cur{};
            bool ok = true;
            for (int n = 0; ok; ++n) {
                if (!(ok = read_seg(n, cur)) || cur.j0 == cur.j1) break;
                const bool rows = h == 0 || has_b(cur);
                if (!(ok = short_wait(bar(W_QFULL), n & 1, abort_flag))) break;
#pragma unroll 1
                for (int j = cur.j0 - 1; j < cur.j1; ++j) {  // the next tile's QK, then this one's PV
                    if (j + 1 < cur.j1) {
                        // S as soon as the softmax holds the one before in registers. Without rows in this row tile (B of a
                        // short chunk) a tile is only handed back.
                        const uint32_t before = t + (j >= cur.j0);  // S tiles issued
                        if (rows && before > 0 && !(ok = short_wait(bar(W_F + h), (before - 1) & 1, abort_flag))) break;
                        if (!(ok = short_wait(bar(W_KFULL), k_tiles & 1, abort_flag))) break;
                        ++k_tiles;
                        tc_fence_after();
                        if (lane == 0) {
                            const bool last = j + 2 == cur.j1;
                            if (rows) {
                                qk();
                                tc_commit(bar(W_S + h));
                                tc_commit(bar(W_KEMPTY));
                                if (last) tc_commit(bar(W_QEMPTY));
                            } else {
                                mbar_arrive(bar(W_KEMPTY));
                                if (last) mbar_arrive(bar(W_QEMPTY));
                            }
                        }
                        __syncwarp();
                    }
                    if (j < cur.j0) continue;
                    if (!(ok = short_wait(bar(W_VFULL), v_tiles & 1, abort_flag))) break;
                    ++v_tiles;
                    if (rows && !(ok = short_wait(bar(W_P + h), t & 1, abort_flag))) break;
                    // the previous segment's output must be out of TMEM before its O is overwritten
                    if (rows && j == cur.j0 && done > 0 && !(ok = short_wait(bar(W_OFREE + h), (done - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    if (lane == 0) {
                        if (rows) {
                            pv(j > cur.j0);
                            tc_commit(bar(W_O + h));
                            tc_commit(bar(W_VEMPTY));
                        } else {
                            mbar_arrive(bar(W_VEMPTY));
                        }
                    }
                    __syncwarp();
                    t += rows;
                }
                done += rows;
            }
            if (!ok && lane == 0) give_up(p.err, abort_flag);
            if (lane == 0) {  // every MMA this thread issued has finished before the TMEM is freed
                tc_commit(bar(W_END + h));
                if (!mbar_wait(bar(W_END + h), 0)) give_up(p.err, abort_flag);
            }
            __syncwarp();
        }
    } else if (warp >= 12) {
        // =================================== loaders ===================================
        regs_down<kRegsLoad>();
        // They widen the halves that landed into the tile that the matrix instructions read, in the order in which they come: K
        // while it is less than two tiles ahead of V. A warp has 16 keys of a half, a lane 16 elements (one 16-byte piece) of every
        // kStepKeys-th of them.
        constexpr int kPieces = HD / 16, kStepKeys = 32 / kPieces, kSteps = 16 / kStepKeys;
        const int w = warp - 12, piece = lane % kPieces, row0 = w * 16 + lane / kPieces;
        // chunks 2 * piece and 2 * piece + 1 of a row; lanes of the second 64 columns write theirs in the other
        // order, so that eight lanes meet eight different groups of banks
        const bool other = piece >= 4;
        const int chunk = (2 * piece + other) & 7;
        SegInfo it{};
        bool ok = read_seg(0, it), end = !ok || it.j0 == it.j1;
        int n = 0, j = it.j0;
        uint32_t wk = 0, wv = 0, u = 0;      // tiles of K and V widened, halves used
        int lo[2] = {0, 0}, hi[2] = {0, 0};  // the keys that some row sees, in the tiles whose K was widened last, and before it
#pragma unroll 1
        while (ok) {
            if (!end && wk - wv < 2 && j == it.j1) {
                ok = read_seg(++n, it);
                if (!ok) break;
                j = it.j0;
                end = it.j0 == it.j1;
            }
            const bool is_v = end || wk - wv == 2;
            if (is_v && wv == wk) break;
            if (!is_v) {
                lo[1] = lo[0], hi[1] = hi[0];
                lo[0] = it.n_lo - j * BN, hi[0] = it.n_end - j * BN;
                ++j;
            }
            const bool before = is_v && wk - wv == 2;
            const int z0 = before ? lo[1] : lo[0], z1 = before ? hi[1] : hi[0];
            const uint32_t i = is_v ? wv : wk;
            if (!(ok = short_wait(bar(is_v ? W_VEMPTY : W_KEMPTY), (i & 1) ^ 1, abort_flag))) break;
            unsigned char *tile = smem + (is_v ? Lay::OFF_V : Lay::OFF_K) + (piece >> 2) * kHalf;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf, ++u) {
                const uint32_t slot = u % kStages;
                if (!(ok = short_wait(bar(W_SFULL) + 8 * slot, (u / kStages) & 1, abort_flag))) break;
                const uint32_t src = sbase + Lay::OFF_STAGE + slot * kHalfKeys * HD + row0 * HD + piece * 16;
                uint4 x[kSteps];  // all read before any is written: the order of reads and writes stays as it is here
#pragma unroll
                for (int e = 0; e < kSteps; ++e) x[e] = lds128(src + e * kStepKeys * HD);
                if (!is_v && lane < 16) {
                    const int k = hf * kHalfKeys + w * 16 + lane;
                    const float *sc = reinterpret_cast<const float *>(smem + Lay::OFF_SCALE) + slot * 2 * kHalfKeys + w * 16 + lane;
                    float ks = finite_or_nan(sc[0]), vs = finite_or_nan(sc[kHalfKeys]);
                    if (k < z0 || k >= z1) ks = vs = 1.f;  // no row sees it: numbers that do no harm, whatever lies there
                    float *keys = reinterpret_cast<float *>(smem + Lay::OFF_KEYS) + (i % kKeyRing) * 3 * BN + k;
                    if constexpr (E::kIsBf16) {
                        keys[0] = ks * p.scale_log2;
                        keys[BN] = vs;
                    } else {  // (the widened rows are 2^-8 of what they stand for)
                        keys[0] = ks * p.scale_log2 * 256.f;
                        keys[BN] = __log2f(vs);
                        keys[2 * BN] = __frcp_rn(vs) * 0x1p-8f;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(W_SEMPTY) + 8 * slot);
                if (z0 > hf * kHalfKeys || z1 < (hf + 1) * kHalfKeys) {  // keys that no row sees are zeros, whatever lies there
#pragma unroll
                    for (int e = 0; e < kSteps; ++e) {
                        const int k = hf * kHalfKeys + row0 + e * kStepKeys;
                        if (k < z0 || k >= z1) x[e] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int k = hf * kHalfKeys + row0 + e * kStepKeys;
                    unsigned char *at = tile + k * 128;
                    *reinterpret_cast<uint4 *>(at + ((chunk ^ (k & 7)) << 4)) =
                        widen_e4m3x8<E>(other ? x[e].z : x[e].x, other ? x[e].w : x[e].y);
                    *reinterpret_cast<uint4 *>(at + ((chunk ^ 1 ^ (k & 7)) << 4)) =
                        widen_e4m3x8<E>(other ? x[e].x : x[e].z, other ? x[e].y : x[e].w);
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (!is_v) mbar_arrive(bar(W_KEYS + wk % kKeyRing));
                mbar_arrive(bar(is_v ? W_VFULL : W_KFULL));
            }
            wk += !is_v, wv += is_v;
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        __syncwarp();
    } else {
        // =================================== softmax ===================================
        regs_up<kRegsSoftmax>();
        const int h = warp >= 8 ? 1 : 0;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t srow = tmem + lane_off + (h ? 128 : 0);
        const uint32_t orow = tmem + lane_off + 256 + (h ? 128 : 0);
        unsigned char *ptile = smem + (h ? Lay::OFF_PB : Lay::OFF_PA);
        unsigned char *prow = ptile + r * 128;  // half 0
        const uint32_t s_full = bar(W_S + h), s_free = bar(W_F + h), p_full = bar(W_P + h);
        const uint32_t o_done = bar(W_O + h), o_free = bar(W_OFREE + h);
        const int row_tok = p.div_g(r);  // this row's token within its tile
        uint32_t t = 0;     // key tiles of this row tile
        uint32_t tile = 0;  // key tiles of all segments
        bool ok = true;
        SegInfo it{};
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, it)) || it.j0 == it.j1) break;
            const int tok = it.tok - h * p.tt;  // tokens of this row tile
            if (tok <= 0) {
                tile += it.j1 - it.j0;
                continue;
            }
            const int rows = min(tok, p.tt) * p.G;
            const bool live = quarter * 32 < rows;  // this warp holds rows
            // The keys this row sees: [lo, lim). Rows without a token take the last one's, and nobody reads what comes of them:
            // with bounds of their own their warp would mask every tile (66 rows of 128: 92 us where 128 rows take 68).
            const int pos = it.p0 + h * p.tt + min(row_tok, tok - 1), lim = pos + 1;
            const int lo = p.window > 0 ? pos - p.window + 1 : 0;
            float m_use = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = it.j0; j < it.j1; ++j, ++t, ++tile) {
                if (!(ok = short_wait(s_full, t & 1, abort_flag))) break;
                if (!live) {
                    if (lane == 0) mbar_arrive(s_free);
                    // P's barrier counts tiles: not before the previous tile's PV has been issued
                    if (t > 0 && !(ok = short_wait(o_done, (t - 1) & 1, abort_flag))) break;
                    if (lane == 0) mbar_arrive(p_full);
                    continue;
                }
                if (!(ok = short_wait(bar(W_KEYS + tile % kKeyRing), (tile / kKeyRing) & 1, abort_flag))) break;
                const float4 *ks4 = reinterpret_cast<const float4 *>(smem + Lay::OFF_KEYS) + (tile % kKeyRing) * 3 * (BN / 4),
                             *v4 = ks4 + BN / 4, *iv4 = v4 + BN / 4;
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
                // x = log2 of the weight (fp16: times its value's scale) before the reference
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    const float4 k4 = ks4[e >> 2];
                    uint64_t a = f2_mul(u2_pack(sv[e], sv[e + 1]), f2_pack(k4.x, k4.y)), b = f2_mul(u2_pack(sv[e + 2], sv[e + 3]), f2_pack(k4.z, k4.w));
                    if constexpr (!E::kIsBf16) {
                        const float4 l4 = v4[e >> 2];
                        a = f2_add(a, f2_pack(l4.x, l4.y)), b = f2_add(b, f2_pack(l4.z, l4.w));
                    }
                    sv[e] = __float_as_uint(f2_lo(a)), sv[e + 1] = __float_as_uint(f2_hi(a));
                    sv[e + 2] = __float_as_uint(f2_lo(b)), sv[e + 3] = __float_as_uint(f2_hi(b));
                }
                if (n0 + BN > lim || n0 < lo) {
                    const unsigned from = static_cast<unsigned>(max(lo - n0, 0)), count = static_cast<unsigned>(max(lim - n0, 0)) - from;
                    const unsigned seen = lim - n0 <= static_cast<int>(from) ? 0u : count;
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (static_cast<unsigned>(e) - from >= seen) sv[e] = 0xff800000u;  // -inf
                }
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 2)
                    mq[(e >> 1) & 3] = max3(mq[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                // the reference moves only when the maximum grew by more than 2^8 (or was unset): the
                // sum uses the same reference, so the result is exact, and P stays below 2^8
                const bool need = mx > m_use + 8.f;
                const float f = need ? fast_exp2(m_use - mx) : 1.f;
                if (need) m_use = mx;
                const float mu = m_use == -INFINITY ? 0.f : m_use;
                const uint64_t nm2 = f2_pack(-mu, -mu);
                uint64_t l2 = f2_pack(0.f, 0.f);
                uint32_t pk[64];
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    const float4 i4 = E::kIsBf16 ? v4[e >> 2] : iv4[e >> 2];
                    const uint64_t xa = f2_add(u2_pack(sv[e], sv[e + 1]), nm2), xb = f2_add(u2_pack(sv[e + 2], sv[e + 3]), nm2);
                    const float p0 = fast_exp2(f2_lo(xa)), p1 = fast_exp2(f2_hi(xa)), p2 = fast_exp2(f2_lo(xb)), p3 = fast_exp2(f2_hi(xb));
                    uint64_t wa = f2_pack(p0, p1), wb = f2_pack(p2, p3);
                    if constexpr (E::kIsBf16) {
                        l2 = f2_add(f2_add(l2, wa), wb);
                        wa = f2_mul(wa, f2_pack(i4.x, i4.y)), wb = f2_mul(wb, f2_pack(i4.z, i4.w));
                    } else {
                        l2 = f2_fma(wa, f2_pack(i4.x, i4.y), l2);
                        l2 = f2_fma(wb, f2_pack(i4.z, i4.w), l2);
                    }
                    // P is rounded to the storage type (the tensor cores' operand), the sum is not
                    pk[e >> 1] = E::pack2(f2_lo(wa), f2_hi(wa));
                    pk[(e >> 1) + 1] = E::pack2(f2_lo(wb), f2_hi(wb));
                }
                l = l * f + (f2_lo(l2) + f2_hi(l2));
                if (t > 0) {  // the previous tile's PV has consumed P and completed O
                    if (!(ok = short_wait(o_done, (t - 1) & 1, abort_flag))) break;
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
            if (ok) ok = short_wait(o_done, (t - 1) & 1, abort_flag);
            if (!ok) break;
            if (!live) {
                if (lane == 0) mbar_arrive(o_free);
                continue;
            }
            tc_fence_after();
            const bool bad = bad_seg[n & (kBadRing - 1)] == n + 1;  // a table entry of the segment was bad
            if (it.part >= 0) {
                // a piece: O unnormalised, with its reference and sum (sum -1: bad)
                float *x = p.pieces + (static_cast<size_t>(blockIdx.x) * 2 + it.part) * wide_piece_floats(HD) + h * 128 + r;
                if (r < rows) {
                    x[0] = m_use;
                    x[256] = bad ? -1.f : l;
                }
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(orow + c * 32, v);
                    tmem_wait_ld();
                    if (r < rows) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[512 + (c * 32 + e) * 256] = __uint_as_float(v[e]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
                continue;
            }
            const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;  // NaN stays
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
            for (int c = 0; c < HD / 8; ++c) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)  // bad: zero, whatever the accumulator holds
                    o[e] = bad ? 0u : E::pack2(__uint_as_float(acc[c * 8 + e * 2]) * inv, __uint_as_float(acc[c * 8 + e * 2 + 1]) * inv);
                *reinterpret_cast<uint4 *>(prow + (c >> 3) * kHalf + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
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
                const uint4 u = *reinterpret_cast<const uint4 *>(ptile + (c >> 3) * kHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
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

template <class E, int HD, bool kGather>
cudaError_t launch_wide(const WideParams &prm, cudaStream_t stream) {
    auto kern = chunk_q8_wide_kernel<E, HD, kGather>;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LayWide<HD>::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev] = 1;
    }
    const unsigned P = device_sm_count();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(P);
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = LayWide<HD>::kSmem;
    if ((e = cudaLaunchKernelEx(&cfg, kern, prm)) != cudaSuccess) return e;  // as in chunk_attn.cu
    cfg.dynamicSmemBytes = 0;
    const int rows = prm.max_seqlen_q > prm.tt ? 256 : (prm.max_seqlen_q * prm.G + kJoinRows - 1) / kJoinRows * kJoinRows;
    cfg.gridDim = dim3(P, rows / kJoinRows, HD / kJoinCols);
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<E, HD>, static_cast<const ChunkParams &>(prm));
}

}  // namespace

cudaError_t launch_chunk_q8_wide(const chunk::ChunkParams &common, const ChunkQ8Args &x, cudaStream_t stream) {
    const ChunkArgs &a = x.chunk;
    WideParams prm{};
    static_cast<ChunkParams &>(prm) = common;
    prm.k_scale = x.k_scale;
    prm.v_scale = x.v_scale;
    prm.tt = BM / prm.G;
    prm.item_tok = 2 * prm.tt;
    const auto encode = [&](CUtensorMap *m, const void *base, int tokens) {
        return encode_rows_3d(m, base, a.dtype, a.Hq, a.D, a.total_q, prm.G, tokens, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    };
    if (!encode(&prm.tm_q, a.q, prm.tt)) return cudaErrorInvalidValue;
    // a warp's 32 output rows as one box, where they are whole tokens
    prm.store_tok = 32 % prm.G == 0 && BM % prm.G == 0 ? 32 / prm.G : 0;
    if (prm.store_tok > 0 && !encode(&prm.tm_o, a.out, prm.store_tok)) return cudaErrorInvalidValue;
    const bool gather = prm.box_rows < 8;
    if (prm.box_rows > kHalfKeys) prm.box_rows = kHalfKeys;
    const long long rows = static_cast<long long>(a.num_blocks) * a.block_size;
    if (!gather && (!encode_rows_e4m3(&prm.tm_k, a.k_cache, a.Hkv, a.D, rows, prm.box_rows, false) ||
                    !encode_rows_e4m3(&prm.tm_v, a.v_cache, a.Hkv, a.D, rows, prm.box_rows, false)))
        return cudaErrorInvalidValue;
    auto go = [&](auto e, auto hd) {
        using E = decltype(e);
        constexpr int HD = decltype(hd)::value;
        return gather ? launch_wide<E, HD, true>(prm, stream) : launch_wide<E, HD, false>(prm, stream);
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (a.dtype == PA_BF16) return a.D == 64 ? go(BF16{}, I64{}) : go(BF16{}, I128{});
    return a.D == 64 ? go(F16{}, I64{}) : go(F16{}, I128{});
}

}  // namespace pa
