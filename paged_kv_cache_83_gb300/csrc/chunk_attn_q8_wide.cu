// chunk_attn_q8_wide.cu: pa_chunk_attn_q8 for chunks of more than 64 query rows a kv head (tokens x group), such as pieces of
// long prompts.
//
// The mathematics is chunk_attn.cu's, with the scales of an 8-bit cache: x_j = ks_j (scale q.K8_j) + log2 vs_j, weights
// 2^(x_j - m), O = sum 2^(x_j - m) V8_j, and the sum takes 2^(x_j - m) / vs_j.
//
// Bound by the softmax warps, as there. So the cache's e4m3 rows are widened to the storage type, exactly, on their way to
// shared memory, once for the 256 query rows of an item, and queries and weights stay whole operands (as sums of e4m3 pieces they
// cost the softmax three conversions a weight; that form of 64 rows an item took 955 us for two chunks of 2k tokens at 12-16k, 16/8
// heads x 128). Four warps copy the rows ahead, any page size alike, widen them and write the swizzled
// tile that the matrix instructions read; one buffer for K and one for V suffice, since a tile's K is wanted a
// whole softmax before its V.
//
//   warp 3        scheduler, as in chunk_attn.cu
//   warp 0        brings the queries of a segment by TMA
//   warps 1, 2    one MMA issuer per row tile
//   warps 4-11    softmax, a thread a query row
//   warps 12-15   loaders: K and V tiles, and the three numbers of a key: scale * ks, log2 vs, 1 / vs
#include <type_traits>

#include "chunk_wide.cuh"
#include "tensor_map.h"

namespace pa {

namespace {

using namespace chunk;

constexpr int kWideThreads = 512;
constexpr int kWideReaders = 15;  // roles that read the queue of segments, by warp
constexpr int kKeyRing = 4;       // key tiles whose numbers are held
// Segments in the queue. The loaders look two tiles ahead of the products, which may be two segments: they wait for segment
// n + 2 to be published, before they bring the V of n - 1, and so for all roles to have read n + 2 - kQueue.
constexpr int kQueue = 4;
constexpr int kUnit = 4, kUnits = 3;  // pieces of a loader's unit, units in flight
// registers of a thread by warpgroup: 88 + 2 * 168 + 88 = 4 * 128
constexpr int kRegsSmall = 88, kRegsSoftmax = 168, kRegsLoad = 88;

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
    W_KEYS,                 // + tile % kKeyRing: the keys' numbers are written (4 arrivals)
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
                         OFF_STAGE = OFF_V + kKV,  // the loaders' units: 16 bytes a thread and piece
                         OFF_KEYS = OFF_STAGE + kUnits * kUnit * 2048;  // per tile of the ring: scale * ks [BN], log2 vs [BN], 1 / vs [BN]
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
// of a NaN becomes +-480: a row that held a NaN has a NaN scale.
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

template <class E, int HD>
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
        if (tid == W_KFULL || tid == W_VFULL || (tid >= W_KEYS && tid < W_S)) count = 4;
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
            // ================================== scheduler ==================================
            int published = 0;
            const bool ok = walk_share(p, *share, [&](const SegInfo &it) {
                if (!short_wait(bar(W_IEMPTY + published % kQueue), ((published / kQueue) & 1) ^ 1, abort_flag)) return false;
                if (lane == 0) {
                    items[published % kQueue] = it;
                    mbar_arrive(bar(W_IFULL + published % kQueue));
                }
                __syncwarp();
                ++published;
                return true;
            });
            if (!ok && lane == 0) give_up(p.err, abort_flag);
        } else if (warp == 0) {
            // =================================== queries ===================================
            prefetch_tmap(&p.tm_q);
            int n = 0;
            bool ok = true;
            for (SegInfo cur{};; ++n) {
                if (!(ok = read_seg(n, cur)) || cur.j0 == cur.j1) break;
                // once both issuers are past the previous segment's last QK
                if (n > 0 && !(ok = short_wait(bar(W_QEMPTY), (n - 1) & 1, abort_flag))) break;
                if (lane == 0) {
                    const int tiles = has_b(cur) ? 2 : 1;
                    const uint32_t half_bytes = static_cast<uint32_t>(p.tt) * p.G * 128;
                    mbar_arrive_expect_tx(bar(W_QFULL), tiles * kHalves * half_bytes);
                    for (int h = 0; h < tiles; ++h)
                        for (int half = 0; half < kHalves; ++half)
                            tma_load_3d(sbase + (h ? Lay::OFF_QB : Lay::OFF_QA) + half * kHalf, &p.tm_q, half * 64, cur.g * p.G,
                                        cur.tok0 + h * p.tt, bar(W_QFULL));
                }
                __syncwarp();
            }
            if (!ok && lane == 0) give_up(p.err, abort_flag);
            // no copy may still be in flight at exit
            if (lane == 0 && n > 0 && !mbar_wait(bar(W_QFULL), (n - 1) & 1)) give_up(p.err, abort_flag);
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
        // A warp has 32 keys of a tile, a lane 16 elements (one 16-byte piece) of every kStepKeys-th of them: kSteps pieces a tile,
        // which it copies to room of its own in shared memory, kUnit pieces (a unit) at a time and kUnits units ahead, and
        // widens from there itself: nobody else waits for its copies. Lane l looks up key l's place in the pool and loads its
        // scales. One loop, one copy of the code: with the loads in registers, and with the loop's ends unrolled, it did not stay in
        // the instruction cache beside the softmax's (1001 and 715 us for the two chunks).
        constexpr int kPieces = HD / 16, kStepKeys = 32 / kPieces, kSteps = 32 / kStepKeys;
        static_assert(kSteps % kUnit == 0);
        const int w = warp - 12, piece = lane % kPieces, key_of_lane = lane / kPieces;
        const uint32_t mine = sbase + Lay::OFF_STAGE + (tid - 384) * 16;  // pieces 2 KB apart
        // chunks 2 * piece and 2 * piece + 1 of a row; lanes of the second 64 columns write theirs in the other
        // order, so that eight lanes meet eight different groups of banks
        const int chunk = (2 * piece + (piece >= 4)) & 7;
        const uint32_t stride = static_cast<uint32_t>(p.Hkv) * HD;
        SegInfo it{};
        int n = 0, j = 0, id = 0;  // the tile whose K is copied next; the table entry of this lane's key in it
        auto fetch = [&]() {
            const int pos = j * BN + w * 32 + lane;
            id = 0;
            if (it.j0 < it.j1 && pos >= it.n_lo && pos < it.n_end)
                id = ld_index(p.block_tables + static_cast<size_t>(it.s) * p.max_blocks + p.geom.block_of(pos));
        };
        bool ok = read_seg(0, it);
        if (!ok) it.j1 = it.j0;
        j = it.j0;
        fetch();
        // Tiles are copied, and widened, in the order K 0, K 1, V 0, K 2, V 1, ...: K while it is less than two ahead of V.
        uint32_t ck = 0, cv = 0;                         // copied
        int row[2] = {-1, -1}, head[2] = {0, 0};         // of this lane's key, in the tiles whose K was copied last, and before it
        float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
        int from = -1, from_head = 0, step = kSteps;     // of the tile that is being copied
        const unsigned char *pool = nullptr;             // (nullptr: none is left)
        uint32_t wk = 0, wv = 0;                         // widened
        bool is_v = false;                               // the tile that is being widened
        int done = kSteps;                               // of it
#pragma unroll 1
        for (uint32_t u = 0; ok; ++u) {
            if (u >= kUnits) {  // the unit that was copied kUnits steps ago
                if (done == kSteps) {
                    done = 0;
                    is_v = !(wk < ck && wk - wv < 2);
                    if (is_v && wv == wk) break;
                    const uint32_t i = is_v ? wv : wk;
                    if (!(ok = short_wait(bar(is_v ? W_VEMPTY : W_KEMPTY), (i & 1) ^ 1, abort_flag))) break;
                    if (!is_v) {
                        const bool before = ck == i + 2;  // the next tile's copies have begun
                        const float key_vs = before ? vs[1] : vs[0];
                        float *keys = reinterpret_cast<float *>(smem + Lay::OFF_KEYS) + (i % kKeyRing) * 3 * BN + w * 32 + lane;
                        keys[0] = (before ? ks[1] : ks[0]) * p.scale_log2 * (E::kIsBf16 ? 1.f : 256.f);
                        keys[BN] = __log2f(key_vs);
                        keys[2 * BN] = __frcp_rn(key_vs) * (E::kIsBf16 ? 1.f : 0x1p-8f);
                    }
                }
                cp_async_wait<kUnits - 1>();
                const uint32_t src = mine + (u % kUnits) * (kUnit * 2048);
                unsigned char *tile = smem + (is_v ? Lay::OFF_V : Lay::OFF_K) + (piece >> 2) * kHalf;
                uint4 x[kUnit];  // all read before any is written: the order of reads and writes stays as it is here
#pragma unroll
                for (int i = 0; i < kUnit; ++i) x[i] = lds128(src + i * 2048);
#pragma unroll
                for (int i = 0; i < kUnit; ++i) {
                    const int k = w * 32 + (done + i) * kStepKeys + key_of_lane;
                    const bool other = piece >= 4;
                    unsigned char *at = tile + k * 128;
                    *reinterpret_cast<uint4 *>(at + ((chunk ^ (k & 7)) << 4)) =
                        widen_e4m3x8<E>(other ? x[i].z : x[i].x, other ? x[i].w : x[i].y);
                    *reinterpret_cast<uint4 *>(at + ((chunk ^ 1 ^ (k & 7)) << 4)) =
                        widen_e4m3x8<E>(other ? x[i].x : x[i].z, other ? x[i].y : x[i].w);
                }
                done += kUnit;
                if (done == kSteps) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (!is_v) mbar_arrive(bar(W_KEYS + wk % kKeyRing));
                        mbar_arrive(bar(is_v ? W_VFULL : W_KFULL));
                    }
                    wk += !is_v, wv += is_v;
                }
            }
            if (step == kSteps) {  // what is copied next
                step = 0;
                pool = nullptr;
                if (it.j0 < it.j1 && ck - cv < 2) {
                    row[1] = row[0], head[1] = head[0], ks[1] = ks[0], vs[1] = vs[0];
                    const int pos = j * BN + w * 32 + lane;
                    row[0] = -1, head[0] = it.g;
                    ks[0] = vs[0] = 1.f;  // where no row sees the key: numbers that do no harm
                    if (pos >= it.n_lo && pos < it.n_end) {
                        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) {
                            const int off = p.geom.offset_of(pos);
                            row[0] = id * p.geom.block_size + off;
                            const size_t at = (static_cast<size_t>(id) * p.Hkv + it.g) * p.geom.block_size + off;
                            ks[0] = __ldcg(p.k_scale + at);
                            vs[0] = __ldcg(p.v_scale + at);
                        } else {
                            bad_seg[n & (kBadRing - 1)] = n + 1;
                            raise_err(p.err, PA_DEVERR_TABLE);
                        }
                    }
                    __syncwarp();
                    from = row[0], from_head = head[0];
                    pool = static_cast<const unsigned char *>(p.k_cache);
                    ++ck;
                    if (++j >= it.j1) {
                        ok = read_seg(++n, it);
                        j = it.j0;
                        if (!ok) it.j1 = it.j0;
                    }
                    fetch();
                } else if (cv < ck) {
                    const bool before = ck == cv + 2;
                    from = before ? row[1] : row[0], from_head = before ? head[1] : head[0];
                    pool = static_cast<const unsigned char *>(p.v_cache);
                    ++cv;
                }
            }
            if (pool) {
                const unsigned char *base = pool + from_head * HD + piece * 16;
                const uint32_t dst = mine + (u % kUnits) * (kUnit * 2048);
#pragma unroll
                for (int i = 0; i < kUnit; ++i) {
                    const int r = __shfl_sync(kFull, from, (step + i) * kStepKeys + key_of_lane);
                    cp_async16(dst + i * 2048, base + static_cast<uint64_t>(static_cast<uint32_t>(max(r, 0))) * stride, r < 0 ? 0 : 16);
                }
            }
            step += kUnit;
            cp_async_commit();
        }
        cp_async_wait<0>();
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
            const int pos = it.p0 + h * p.tt + row_tok;
            const int lim = r < rows ? pos + 1 : 0;  // the keys this row sees: [lo, lim)
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
                             *lv4 = ks4 + BN / 4, *iv4 = lv4 + BN / 4;
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
                // x = log2 of the weight before the reference
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    const float4 k4 = ks4[e >> 2], l4 = lv4[e >> 2];
                    const uint64_t a = f2_fma(u2_pack(sv[e], sv[e + 1]), f2_pack(k4.x, k4.y), f2_pack(l4.x, l4.y)),
                                   b = f2_fma(u2_pack(sv[e + 2], sv[e + 3]), f2_pack(k4.z, k4.w), f2_pack(l4.z, l4.w));
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
                    const float4 i4 = iv4[e >> 2];
                    const uint64_t xa = f2_add(u2_pack(sv[e], sv[e + 1]), nm2), xb = f2_add(u2_pack(sv[e + 2], sv[e + 3]), nm2);
                    const float p0 = fast_exp2(f2_lo(xa)), p1 = fast_exp2(f2_hi(xa)), p2 = fast_exp2(f2_lo(xb)), p3 = fast_exp2(f2_hi(xb));
                    l2 = f2_fma(f2_pack(p0, p1), f2_pack(i4.x, i4.y), l2);
                    l2 = f2_fma(f2_pack(p2, p3), f2_pack(i4.z, i4.w), l2);
                    // P is rounded to the storage type (the tensor cores' operand), the sum is not
                    pk[e >> 1] = E::pack2(p0, p1);
                    pk[(e >> 1) + 1] = E::pack2(p2, p3);
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

template <class E, int HD>
cudaError_t launch_wide(const WideParams &prm, cudaStream_t stream) {
    auto kern = chunk_q8_wide_kernel<E, HD>;
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
    if (a.dtype == PA_BF16) return a.D == 64 ? launch_wide<BF16, 64>(prm, stream) : launch_wide<BF16, 128>(prm, stream);
    return a.D == 64 ? launch_wide<F16, 64>(prm, stream) : launch_wide<F16, 128>(prm, stream);
}

}  // namespace pa
