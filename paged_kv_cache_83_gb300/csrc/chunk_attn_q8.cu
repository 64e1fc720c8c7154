// chunk_attn_q8.cu: causal attention of one or more new tokens of each sequence over a paged cache of 8 bits
// (pa_chunk_attn_q8) on the 5th-generation tensor cores.
//
// Source: as chunk_attn.cu ("nano-vLLM Part 4", section 3; smzdm nano-vLLM deep dive, "GPU执行优化").
//
// The mathematics: K_j = ks_j K8_j and V_j = vs_j V8_j with e4m3 rows and a scale for each row and kv head. The e4m3 rows go
// to the tensor cores as they lie in the cache, without a conversion: keys are the 128 rows, query rows the
// columns, as in chunk_attn_narrow.cu,
//   S^T = K8 Q^T,   O^T += V8^T W^T,
// and what meets them is split into pieces of 8 bits, side by side as further columns of the same instruction:
//   q = 2^e (q0 + q1 / 32 [+ q2 / 1024]) in e4m3: two pieces hold a bf16 number (8 bits) exactly, three an fp16 number (11 bits),
//     where its magnitude is above 2^-14 of its row's largest; below that the error is at most 2^-22 (2^-27) of the largest;
//   w, a weight of the softmax. In fp16 w0 + w1 / 32 + w2 / 1024 in e4m3: off by at most 2^-11 of itself, as an fp16 number is, or
//     2^-20. In bf16 w0 + (w1 + w2) / 8 in e5m2, whose 3 bits each reach down to 2^-16: off by at most 2^-8 of itself, as a
//     bf16 number is, or 2^-19, which is 2^-30 of a largest w of 2^11. (As two e4m3 pieces what lay below 2^-19 of the largest
//     counted in the sum but not in the output: behind one heavy key a tail of 20,000 such keys was lost. The third piece costs
//     0.2 to 9 % more time, most at 17 to 32 query rows; an e5m2 number is the upper byte of an fp16 one, so that it takes no
//     conversions.)
// A softmax thread owns one key, so that both scales are one number a thread. The values' scale goes into the
// exponent: x_j = s_j + log2 vs_j, w_j = 2^(x_j - m), O = sum w_j V8_j, and the sum takes w_j / vs_j = 2^(s_j - m). The reference m is
// 4 (bf16: 11) below the largest x of the first tile and moves when some x exceeds it by more than 8 (15): a w is at most
// 2^8 (2^15), below e4m3's (e5m2's) largest number.
//
// Bound by HBM for few query rows: (2 D + 8) bytes a key and kv head. 256 single tokens over 100-4096 keys, 16/8 heads x 128,
// block 256: 190-195 us by box, 6.1-6.2 TB/s, 0.90-0.93 of a copy (fp16, in sixteen columns, 202-206). The loads run ahead in rings of tiles; two streams of softmax
// warps take the key tiles in turn, each with its own reference, sum and accumulator, and join at the end of a segment. On
// the way to that: 305 us before the code of all roles stayed in the instruction cache, the scales came by cp.async and table
// entries a tile ahead (229), 224 with packed arithmetic on the scores and three K tiles a stream, 209 without a meeting of
// the streams at a segment's start; on a box where that took 222, 201 with the line of work by head (see Share), 190 (another
// box: 197 before) with a form of eight columns. A segment's end costs about 1 us that the rings cover in part: one segment a CTA
// (19 sequences of 28k) reads 6.1 TB/s from cold caches, 16 segments of 1760 keys 5.8.
// With more than 32 query rows a kv head the streams take half of the columns each, of every key tile; chunks of more than 64
// go to chunk_attn_q8_wide.cu.
//
//   warp 3      scheduler, as in chunk_attn.cu; splits each segment's queries into pieces
//   warp 0      producer: K and V tiles of the streams in turn, the scales with the K tile
//   warps 1, 2  one MMA issuer per stream
//   warps 4-7   softmax of stream A (tiles 0, 2, ... of a segment), warps 8-11 of stream B (1, 3, ...)
//   TMEM columns: S_A, S_B (NT for each piece of a query), O_A, O_B (NT for each piece of a weight); lanes are keys in S and
//   head elements in O.
#include <type_traits>

#include "chunk_narrow.cuh"
#include "chunk_wide.cuh"
#include "tensor_map.h"

namespace pa {

namespace {

using namespace chunk;

struct Q8Params : ChunkParams {
    const void *q;
    const float *k_scale, *v_scale;  // [num_blocks, Hkv, block_size]
};

// NT columns a stream. kCols: the streams halve the query rows (2 NT of them) and both take every key tile, from
// rings that they share; else they halve the key tiles, each with rings of its own. QP: pieces of a number.
template <int HD, int NT, int QP, bool kCols>
struct LayQ8 {
    static constexpr int kNC = kCols ? 2 * NT : NT;         // query rows
    static constexpr int PP = 3;                            // pieces of a weight
    static constexpr int kKV = BN * HD;                     // bytes of a tile
    static constexpr int kQ = kNC * QP * HD;
    static constexpr int kP = BN * 128;                     // W^T: a 128-byte row a key, PP * NT of it used
    static constexpr int kTiles = HD == 128 ? 4 : 8;        // V tiles held; of K half as many more where there is room
    static constexpr bool kMoreK = !kCols && (NT <= 16 || QP == 2);
    static constexpr int kVSlots = kTiles, kKSlots = kMoreK ? kTiles * 3 / 2 : kTiles;
    static constexpr int kVD = kCols ? kVSlots : kVSlots / 2, kKD = kCols ? kKSlots : kKSlots / 2;  // of a ring
    static constexpr int kQf = 4;                           // segments whose queries' scales are held
    // barriers; rings, S, F, P, O, WG: + stream
    static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_KEMPTY = B_KFULL + kKSlots,
                         B_VFULL = B_KEMPTY + kKSlots, B_VEMPTY = B_VFULL + kVSlots, B_S = B_VEMPTY + kVSlots, B_F = B_S + 2,
                         B_P = B_F + 2, B_WG = B_P + 2, B_O = B_WG + 2, B_OFREE = B_O + 2, B_BOTH = B_OFREE + 2,
                         B_END = B_BOTH + 1, B_QS = B_END + 2, B_IFULL = B_QS + kQf, B_IEMPTY = B_IFULL + 4, NBAR = B_IEMPTY + 4;
    // shared memory: V's rings before K's (at head dim 64 the V operand's unused upper half of rows reads
    // one tile further)
    static constexpr int OFF_V = 0, OFF_K = kVSlots * kKV, OFF_Q = OFF_K + kKSlots * kKV, OFF_P = OFF_Q + 2 * kQ,
                         OFF_SCALE = OFF_P + 2 * kP;        // per K slot: the tile's scales of K, then of V
    static constexpr int OFF_F = OFF_SCALE + kKSlots * 2 * BN * 4;  // floats below
    // per segment parity and stream: references [NT], sums by warp [4][NT], weights [NT]; scratch; the queries' scales
    static constexpr int kMax = 0, kSum = 2 * 2 * NT, kWgt = kSum + 2 * 2 * 4 * NT, kRed = kWgt + 2 * 2 * NT,
                         kFac = kRed + 2 * 4 * NT, kQs = kFac + 2 * NT, kZero = kQs + kQf * kNC, kFloats = kZero + NT;
    static constexpr int OFF_BAR = OFF_F + kFloats * 4 + 16;  // after the votes
    static constexpr int OFF_ITEMS = OFF_BAR + NBAR * 8;
    static constexpr int OFF_BAD = OFF_ITEMS + 4 * static_cast<int>(sizeof(SegInfo));
    static constexpr int OFF_PLAN = (OFF_BAD + kBadRing * 4 + 15) / 16 * 16;
    static constexpr int OFF_MISC = OFF_PLAN + 12 * 8 + static_cast<int>(sizeof(Share));
    static constexpr int kSmem = OFF_MISC + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static_assert(kQ % 1024 == 0 && kKV % 1024 == 0 && OFF_BAR % 8 == 0);
    static constexpr int kS = QP * NT, kO = (PP * NT + 15) / 16 * 16;  // columns of a stream's S and O (a multiple of 16 for an instruction of 128 rows)
    static constexpr int kNeed = 2 * (kS + kO);
    static constexpr int kTmem = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static constexpr size_t kPieceFloats = piece_floats(kNC, HD);
};

// Shared-memory matrix descriptor of rows of HD bytes in groups of eight (128-byte swizzle at HD = 128, 64-byte at 64); lbo:
// from one HD-element column block of an MN-major operand to the next.
template <int HD>
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t lbo) {
    uint64_t d = smem_desc_sw128(saddr, lbo, 8 * HD);
    if constexpr (HD == 64) d = (d & ~(7ull << 61)) | 4ull << 61;
    return d;
}
// where the swizzle puts 16-byte chunk c of row r of a tile with rows of HD bytes
template <int HD>
__device__ __forceinline__ int swizzled(int r, int c) {
    return r * HD + ((HD == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}
// warp_wait with one copy of its loop for the whole kernel: the roles' code has to stay in the instruction cache (inlined
// everywhere, fetching instructions bounded the kernel: 305 us for 256 single tokens over 100-4096 keys)
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return warp_wait(bar, parity, abort_flag);
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(kFull, mbar_try_wait(bar, parity)) || wait_on(bar, parity, abort_flag);
}
// D (+)= A B of e4m3 operands with fp32 accumulation
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// the types e4m3 x e4m3 -> fp32 of kind::f8f6f4 are those of fp16 x fp16 -> fp32 of kind::f16 in number: 0, 0 and 1
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool b_mn_major) { return idesc_f16(M, N, false, b_mn_major); }

// two fp16 numbers -> two e4m3 (nearest even; beyond 448: 448), and back
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<uint32_t *>(&v)));
    return r;
}
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return *reinterpret_cast<__half2 *>(&r);
}
// what a piece leaves of v, times 32 (exact: v has 11 bits)
__device__ __forceinline__ __half2 left_of(__half2 v, uint32_t piece) {
    const __half2 k = __float2half2_rn(32.f);
    return __hfma2(from_e4m3x2(piece), __hneg2(k), __hmul2(v, k));
}

// Two fp16 numbers of at most 2^15 in e5m2, the upper bytes of the halves: the nearest (half-way cases away from zero), or the next towards
// zero; and what that leaves of them, exact, times 8 if asked for. (Of a NaN comes any number: the sum of the weights keeps it.)
__device__ __forceinline__ uint32_t to_e5m2x2(__half2 v, bool nearest) { return *reinterpret_cast<uint32_t *>(&v) + (nearest ? 0x00800080u : 0u); }
__device__ __forceinline__ __half2 left_of_e5m2(__half2 v, uint32_t piece, bool times8) {
    piece &= 0xff00ff00u;
    const __half2 r = __hsub2(v, *reinterpret_cast<__half2 *>(&piece));
    return times8 ? __hmul2(r, __float2half2_rn(8.f)) : r;
}
// where the reference lies below the largest x that sets it, and how far above it an x may be before it moves
template <bool kBf16>
constexpr float kBelow = kBf16 ? 11.f : 4.f;
template <bool kBf16>
constexpr float kAbove = kBf16 ? 15.f : 8.f;

__device__ __forceinline__ float max_of(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float warp_most(float v) {  // the largest over the warp, in every lane
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

template <class E, int HD, int NT, bool kCols, bool kGather>
__global__ void __launch_bounds__(kThreads, 1) chunk_q8_kernel(const __grid_constant__ Q8Params p) {
    using T = typename E::T;
    constexpr int QP = E::kIsBf16 ? 2 : 3;
    using Lay = LayQ8<HD, NT, QP, kCols>;
    constexpr int kStep = kCols ? 1 : 2;  // key tiles from one to the next of a stream
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    SegInfo *items = reinterpret_cast<SegInfo *>(smem + Lay::OFF_ITEMS);
    volatile int *bad_seg = reinterpret_cast<volatile int *>(smem + Lay::OFF_BAD);
    long long *plan = reinterpret_cast<long long *>(smem + Lay::OFF_PLAN);
    Share *share = reinterpret_cast<Share *>(plan + 12);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    float *fl = reinterpret_cast<float *>(smem + Lay::OFF_F);
    auto bar = [&](int i) { return sbase + Lay::OFF_BAR + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    static_assert(Lay::NBAR <= kThreads);
    if (tid < Lay::NBAR) {
        uint32_t count = 1;
        if (tid >= Lay::B_QEMPTY && tid < Lay::B_KFULL) count = 2;                    // both issuers
        if (!kGather && tid >= Lay::B_KFULL && tid < Lay::B_KEMPTY) count = 1 + 32;  // the tile, and each lane's scales
        if (tid >= Lay::B_KEMPTY && tid < Lay::B_VFULL) count = kCols ? 2 + 8 : 1 + 4;  // issuers and softmax warps
        if (kCols && tid >= Lay::B_VEMPTY && tid < Lay::B_S) count = 2;
        if (tid >= Lay::B_F && tid < Lay::B_O) count = 4;                // F, P, WG: four warps
        if (tid >= Lay::B_OFREE && tid < Lay::B_END) count = 8;
        if (kCols && tid >= Lay::B_OFREE && tid < Lay::B_BOTH) count = 4;
        if (tid >= Lay::B_IEMPTY) count = kItemReaders;
        mbar_init(bar(tid), count);
        fence_mbar_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kBadRing; ++i) bad_seg[i] = 0;
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(fl + Lay::kFloats)[i] = 0;  // votes
    }
    if (tid < NT) fl[Lay::kZero + tid] = 0.f;
    // Launched beside what precedes it in the stream: nothing that it wrote is read, and nothing that it reads is
    // written, before it has finished (the set-up above takes place meanwhile).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Tensor memory is taken only now, and the joining kernel (and with it what follows) let in only when it is
    // there: no block holds tensor memory while it waits for another grid, whose blocks on this SM may want some.
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), Lay::kTmem);
    if (tid == 0) p.recs[blockIdx.x].valid = 0;
    plan_share<kThreads, true>(p, plan, share);
    zero_bad_sequences<T, HD>(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel waits for this grid itself
    const uint32_t tmem = *tmem_slot;

    // every role reads the segments in the same order: segment n sits in queue entry n % 4
    auto read_seg = [&](int n, SegInfo &it) -> bool {
        if (!wait_for(bar(Lay::B_IFULL + (n & 3)), (n >> 2) & 1, abort_flag)) return false;
        it = items[n & 3];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_IEMPTY + (n & 3)));
        return true;
    };

    if (warp == 3) {
        // ================================== scheduler ==================================
        int published = 0;
        // The rows of segment n's queries as pieces: row r, times the power of two that brings its largest magnitude into
        // [128, 256). The factor that takes scores back, with the softmax's scale, goes to the segment's entry of four:
        // the softmax of segment n - 4 is over when the issuers have let go of segment n - 2's queries.
        auto split_q = [&](const SegInfo &it, int n) -> bool {
            if (!wait_for(bar(Lay::B_QEMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag)) return false;
            // 16 elements a lane, one 16-byte chunk of each piece; kStepRows rows at a time, two such steps in flight
            constexpr int kLanes = HD / 16, kStepRows = 32 / kLanes;
            const int rows = it.tok * p.G, c16 = lane % kLanes;
            unsigned char *dst = smem + Lay::OFF_Q + (n & 1) * Lay::kQ;
            float *qs = fl + Lay::kQs + (n & 3) * Lay::kNC;
            auto load = [&](int r, uint4 (&w)[2]) {
                r = min(r, rows - 1);
                const int tok = p.div_g(r);
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(p.q) + (static_cast<size_t>(it.tok0 + tok) * p.Hq + it.g * p.G + (r - tok * p.G)) * HD + c16 * 16);
                w[0] = __ldcg(src), w[1] = __ldcg(src + 1);
            };
            uint4 ahead[2];
            load(lane / kLanes, ahead);
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += kStepRows) {
                const int r = r0 + lane / kLanes;
                const uint4 w0 = ahead[0], w1 = ahead[1];
                load(r + kStepRows, ahead);
                const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                uint32_t most = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = E::unpack2(w[e]);
                    most = max(most, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
                }
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
                const uint32_t e8 = max(most >> 23, 8u);  // exponent, kept where both factors are normal
                const float up = __uint_as_float((261u - e8) << 23);
                // a row that is not finite gives scores that are not
                const float down = e8 == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((e8 - 7u) << 23) * p.scale_log2;
                uint32_t piece[QP][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = E::unpack2(w[e]);
                    __half2 v = __floats2half2_rn(f.x * up, f.y * up);  // exact down to 2^-17 of the largest
#pragma unroll
                    for (int i = 0; i < QP; ++i) {
                        const uint32_t a = to_e4m3x2(v);
                        if (i + 1 < QP) v = left_of(v, a);
                        piece[i][e >> 1] = e & 1 ? piece[i][e >> 1] | a << 16 : a;
                    }
                }
                if (r < rows) {
                    const int row0 = r / NT * QP * NT + r % NT;
#pragma unroll
                    for (int i = 0; i < QP; ++i)
                        *reinterpret_cast<uint4 *>(dst + swizzled<HD>(row0 + i * NT, c16)) =
                            make_uint4(piece[i][0], piece[i][1], piece[i][2], piece[i][3]);
                    if (c16 == 0) qs[r] = down;
                }
            }
            // columns without a query row: their scores count for nothing, whatever the pieces there hold
            for (int r = rows + lane; r < Lay::kNC; r += 32) qs[r] = 0.f;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(Lay::B_QFULL + (n & 1)));
                mbar_arrive(bar(Lay::B_QS + (n & 3)));
            }
            return true;
        };
        const bool ok = walk_share<true>(p, *share, [&](const SegInfo &it) {
            if (!wait_for(bar(Lay::B_IEMPTY + (published & 3)), ((published >> 2) & 1) ^ 1, abort_flag)) return false;
            if (lane == 0) {
                items[published & 3] = it;
                mbar_arrive(bar(Lay::B_IFULL + (published & 3)));
            }
            __syncwarp();
            const bool r = it.j0 == it.j1 || split_q(it, published);
            ++published;
            return r;
        });
        if (!ok && lane == 0) give_up(p.err, abort_flag);
    } else if (warp == 0) {
        // =================================== producer ===================================
        if constexpr (!kGather) {
            prefetch_tmap(&p.tm_k);
            prefetch_tmap(&p.tm_v);
        }
        const int R = p.box_rows, nbox = BN / R;
        constexpr int kRowsLane = kGather ? BN / 32 : 1;
        // The table entries of the boxes (rows) that this lane loads of a key tile: fetched a tile ahead, looked at when
        // the tile is loaded.
        struct Entries {
            int id[kRowsLane];
            bool needed[kRowsLane];
        };
        struct Rows {
            int r[kRowsLane], id[kRowsLane];  // pool rows, -1: not read; their blocks
            int g;
        };
        const int box = 4 * lane / R, in_box = 4 * lane - box * R;  // of the four keys whose scales this lane copies
        auto pos_of = [&](int j, int i) { return j * BN + (kGather ? lane + 32 * i : lane * R); };
        auto fetch = [&](const SegInfo &it, int j) {
            Entries e;
            const int32_t *table = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks;
#pragma unroll
            for (int i = 0; i < kRowsLane; ++i) {
                const int pos = pos_of(j, i);
                e.needed[i] = (kGather || lane < nbox) && pos < it.n_end && pos + (kGather ? 0 : R - 1) >= it.n_lo;
                e.id[i] = e.needed[i] ? ld_index(table + p.geom.block_of(pos)) : 0;
            }
            return e;
        };
        auto rows_of = [&](const SegInfo &it, int j, const Entries &e, int seg_no) {
            Rows w;
            w.g = it.g;
#pragma unroll
            for (int i = 0; i < kRowsLane; ++i) {
                w.id[i] = e.id[i];
                w.r[i] = e.needed[i] ? e.id[i] * p.geom.block_size + p.geom.offset_of(pos_of(j, i)) : -1;
                if (e.needed[i] && static_cast<unsigned>(e.id[i]) >= static_cast<unsigned>(p.num_blocks)) {
                    w.r[i] = -1;
                    bad_seg[seg_no & (kBadRing - 1)] = seg_no + 1;
                    raise_err(p.err, PA_DEVERR_TABLE);
                }
            }
            return w;
        };
        // where the scale of pool row r of a block lies
        auto scale_at = [&](int r, int id, int g) {
            return r + (static_cast<long long>(id) * (p.Hkv - 1) + g) * p.geom.block_size;
        };
        // where the next tile goes in a stream's ring: slot, and times round before
        struct At {
            uint32_t slot, lap;
        };
        At ak[2] = {}, av[2] = {};
        auto advance = [&](At &x, int slots) {
            if (++x.slot == static_cast<uint32_t>(slots)) x.slot = 0, ++x.lap;
        };
        // gathered tiles are announced one load late, when their copies have landed
        uint32_t owed = 0;  // the barrier of the tile whose copies are in flight
        auto announce = [&](uint32_t b) {
            if constexpr (kGather) {
                if (owed) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(owed);
                }
                owed = b;
            }
        };
        auto flush = [&]() {
            if constexpr (kGather) {
                cp_async_wait<0>();
                announce(0);
            }
        };
        // One tile of K with its scales, or of V, into its slot once that is free.
        auto load = [&](const Rows &w, auto v, int h, At &at) -> bool {
            constexpr bool is_v = decltype(v)::value;
            constexpr int kD = is_v ? Lay::kVD : Lay::kKD;
            const uint32_t slot = h * kD + at.slot, par = (at.lap & 1) ^ 1;
            const uint32_t full = bar((is_v ? Lay::B_VFULL : Lay::B_KFULL)) + 8 * slot, empty = bar(is_v ? Lay::B_VEMPTY : Lay::B_KEMPTY) + 8 * slot;
            const uint32_t dst = sbase + (is_v ? Lay::OFF_V : Lay::OFF_K) + slot * Lay::kKV;
            const uint32_t sc = sbase + Lay::OFF_SCALE + slot * 2 * BN * 4;
            // a gathered tile is not held back while this one waits for its slot
            if (kGather && !__all_sync(kFull, mbar_try_wait(empty, par))) flush();
            if (!wait_for(empty, par, abort_flag)) return false;
            if constexpr (kGather) {
                const unsigned char *pool = static_cast<const unsigned char *>(is_v ? p.v_cache : p.k_cache);
#pragma unroll
                for (int e = 0; e < kRowsLane; ++e) {
                    const int k = lane + 32 * e;
                    const bool there = w.r[e] >= 0;
                    const unsigned char *src = pool + (static_cast<size_t>(there ? w.r[e] : 0) * p.Hkv + w.g) * HD;
#pragma unroll
                    for (int c = 0; c < HD / 16; ++c) cp_async16(dst + swizzled<HD>(k, c), src + c * 16, there ? 16 : 0);
                    if (!is_v && there) {
                        const long long from = scale_at(w.r[e], w.id[e], w.g);
                        cp_async4(sc + k * 4, p.k_scale + from);
                        cp_async4(sc + (BN + k) * 4, p.v_scale + from);
                    }
                }
                cp_async_commit();
                cp_async_wait<1>();
                announce(full);
            } else {
                const uint32_t boxes = __popc(__ballot_sync(kFull, w.r[0] >= 0));
                if (lane == 0) mbar_arrive_expect_tx(full, boxes * static_cast<uint32_t>(R) * HD);
                __syncwarp();
                if (w.r[0] >= 0) tma_load_3d(dst + lane * R * HD, is_v ? &p.tm_v : &p.tm_k, 0, w.g, w.r[0], full);
                if constexpr (!is_v) {
                    // the scales of four keys a lane, of the box that holds them; the barrier counts every lane's copies
                    const int row = __shfl_sync(kFull, w.r[0], box), id = __shfl_sync(kFull, w.id[0], box);
                    if (row >= 0) {
                        const long long from = scale_at(row, id, w.g) + in_box;
                        cp_async16(sc + lane * 16, p.k_scale + from, 16);
                        cp_async16(sc + BN * 4 + lane * 16, p.v_scale + from, 16);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
                }
            }
            advance(at, kD);
            return true;
        };
        SegInfo cur{};
        Rows pend[2]{};                // the last tile of each stream whose V is still to come
        bool has[2] = {false, false};
        // The V of a stream's tile is loaded after the stream's next K, and
        // those of the segment before as soon as a segment's first K is under way. An issuer takes the first
        // K of a segment only when the V of the segment before has been used, and a K slot is free when the softmax has read
        // the scales in it, at the start of the tile: no load waits for a tile whose predecessors' Vs are outstanding.
        bool ok = read_seg(0, cur);
        Entries next{};
        if (ok && cur.j0 < cur.j1) next = fetch(cur, cur.j0);
        for (int n = 0; ok && cur.j0 < cur.j1; ++n) {
            flush();
            SegInfo after{};
            const auto late = [&](auto stream) {  // the V that a stream owes
                constexpr int h = decltype(stream)::value;
                if (!has[h]) return true;
                has[h] = false;
                return load(pend[h], std::true_type{}, h, av[h]);
            };
            const auto tile = [&](int j, auto stream) {
                constexpr int h = decltype(stream)::value;
                const Rows mine = rows_of(cur, j, next, n);
                if (j + 1 < cur.j1) {  // in flight while this tile is loaded
                    next = fetch(cur, j + 1);
                } else {
                    if (!read_seg(n + 1, after)) return false;
                    if (after.j0 < after.j1) next = fetch(after, after.j0);
                }
                if (!load(mine, std::false_type{}, h, ak[h]) || !late(stream)) return false;
                pend[h] = mine;
                has[h] = true;
                return true;
            };
            using A = std::integral_constant<int, 0>;
            using B = std::integral_constant<int, kCols ? 0 : 1>;
            for (int j = cur.j0; ok && j < cur.j1; j += kStep) {
                ok = tile(j, A{});
                if (!kCols && ok && j == cur.j0) ok = late(B{});
                if (!kCols && ok && j + 1 < cur.j1) ok = tile(j + 1, B{});
            }
            cur = after;
        }
#pragma unroll
        for (int h = 0; h < (kCols ? 1 : 2); ++h)
            if (ok && has[h]) ok = load(pend[h], std::true_type{}, h, av[h]);
        flush();
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        // no copy may still be in flight at exit: the last load of every slot, of this lap or the one before
        if (lane == 0 && !kGather) {
#pragma unroll
            for (int h = 0; h < (kCols ? 1 : 2); ++h)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const At x = v ? av[h] : ak[h];
                    const int slots = v ? Lay::kVD : Lay::kKD;
#pragma unroll 1
                    for (int i = 0; i < slots; ++i) {
                        const uint32_t loads = x.lap + (i < static_cast<int>(x.slot));
                        if (loads > 0 && !mbar_wait(bar((v ? Lay::B_VFULL : Lay::B_KFULL) + h * slots + i), (loads - 1) & 1))
                            give_up(p.err, abort_flag);
                    }
                }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ============================ MMA issuer of one stream =============================
        const int h = warp - 1;
        constexpr uint32_t IQK = idesc_e4m3(BM, Lay::kS, false);             // A = K rows, B = Q pieces, both K-major
        // A = V^T, B = W^T pieces, both MN-major; B's type 0 is e4m3, 1 e5m2
        constexpr uint32_t IPV = idesc_a_mn(idesc_e4m3(BM, Lay::kO, true)) | (E::kIsBf16 ? 1u << 10 : 0u);
        const int k_ring = kCols ? 0 : h * Lay::kKD, v_ring = kCols ? 0 : h * Lay::kVD;  // the stream's first slots
        const int first = kCols ? 0 : h;                                      // and key tile
        const uint64_t dq0 = desc_rows<HD>(sbase + Lay::OFF_Q + (kCols ? h * Lay::kS * HD : 0), 16);
        const uint64_t dk0 = desc_rows<HD>(sbase + Lay::OFF_K + k_ring * Lay::kKV, 16);
        const uint64_t dv0 = desc_rows<HD>(sbase + Lay::OFF_V + v_ring * Lay::kKV, Lay::kKV);
        const uint64_t dp = smem_desc_sw128(sbase + Lay::OFF_P + h * Lay::kP, 16, 1024);
        const uint32_t s_tm = tmem + h * Lay::kS, o_tm = tmem + 2 * Lay::kS + h * Lay::kO;
        auto qk = [&](int slot, int q) {  // S^T = K Q^T, 32 elements an instruction
            const uint64_t a = dk0 + slot * (Lay::kKV >> 4), b = dq0 + q * (Lay::kQ >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) tc_mma_e4m3(s_tm, a + kk * 2, b + kk * 2, IQK, kk > 0);
        };
        auto pv = [&](int slot, bool acc) {  // O^T += V^T W^T, 32 keys an instruction
            const uint64_t a = dv0 + slot * (Lay::kKV >> 4);
#pragma unroll
            for (int kk = 0; kk < BN / 32; ++kk)
                tc_mma_e4m3(o_tm, a + ((kk * 32 * HD) >> 4), dp + ((kk * 32 * 128) >> 4), IPV, (acc || kk > 0));
        };
        uint32_t t = 0;  // key tiles of this stream: QKs issued
        bool ok = true;
        SegInfo it{};
        // QK of the stream's next tile once S has been read; `last`: of the segment
        auto issue_qk = [&](int n, bool last) -> bool {
            const int slot = static_cast<int>(t % Lay::kKD);
            if (t > 0 && !wait_for(bar(Lay::B_F + h), (t - 1) & 1, abort_flag)) return false;
            if (!wait_for(bar(Lay::B_KFULL + k_ring + slot), (t / Lay::kKD) & 1, abort_flag)) return false;
            tc_fence_after();
            if (lane == 0) {
                qk(slot, n & 1);
                tc_commit(bar(Lay::B_S + h));
                tc_commit(bar(Lay::B_KEMPTY + k_ring + slot));
                if (last) tc_commit(bar(Lay::B_QEMPTY + (n & 1)));
            }
            __syncwarp();
            ++t;
            return true;
        };
        uint32_t done = 0;  // PVs issued
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, it)) || it.j0 == it.j1) break;
            const int cnt = it.j1 - it.j0;
            if (!(ok = wait_for(bar(Lay::B_QFULL + (n & 1)), (n >> 1) & 1, abort_flag))) break;
            if (first >= cnt) {  // a segment of one tile has none for stream B
                if (lane == 0) mbar_arrive(bar(Lay::B_QEMPTY + (n & 1)));
                __syncwarp();
                continue;
            }
#pragma unroll 1
            for (int i = first - kStep; i < cnt; i += kStep) {  // the next tile's QK, then this one's PV
                if (i + kStep < cnt && !(ok = issue_qk(n, i + 2 * kStep >= cnt))) break;
                if (i < first) continue;
                const int slot = static_cast<int>(done % Lay::kVD);
                if (!(ok = wait_for(bar(Lay::B_VFULL + v_ring + slot), (done / Lay::kVD) & 1, abort_flag))) break;
                const int n0 = (it.j0 + i) * BN, z0 = max(it.n_lo - n0, 0), z1 = min(it.n_end - n0, BN);
                // rows outside [z0, z1) are zeroed: their weights are zero, but 0 * NaN is not
                // (streams that share the tile both write the zeros)
                if (z0 > 0 || z1 < BN) {
                    uint4 *tile = reinterpret_cast<uint4 *>(smem + Lay::OFF_V + (v_ring + slot) * Lay::kKV);
                    for (int x = lane; x < z0 * (HD / 16); x += 32) tile[x] = make_uint4(0, 0, 0, 0);
                    for (int x = z1 * (HD / 16) + lane; x < BN * (HD / 16); x += 32) tile[x] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!(ok = wait_for(bar(Lay::B_P + h), done & 1, abort_flag))) break;
                // the previous segment's output must be out of TMEM before its O is overwritten. (B may have
                // had no tile in it; its softmax warps have then passed the end of that segment with A's.)
                if (i == first && n > 0 && !(ok = wait_for(bar(Lay::B_OFREE + (kCols ? h : 0)), (n - 1) & 1, abort_flag)))
                    break;
                tc_fence_after();
                if (lane == 0) {
                    pv(slot, i > first);
                    tc_commit(bar(Lay::B_O + h));
                    tc_commit(bar(Lay::B_VEMPTY + v_ring + slot));
                }
                __syncwarp();
                ++done;
            }
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        if (lane == 0) {  // every MMA this thread issued has finished before the TMEM is freed
            tc_commit(bar(Lay::B_END + h));
            if (!mbar_wait(bar(Lay::B_END + h), 0)) give_up(p.err, abort_flag);
        }
        __syncwarp();
    } else {
        // =================================== softmax ===================================
        const int h = warp >= 8 ? 1 : 0;
        const int quarter = warp & 3, wt = tid & 127;  // thread of the stream = key of the tile
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t s_row = tmem + lane_off + h * Lay::kS, o_row = tmem + lane_off + 2 * Lay::kS + h * Lay::kO;
        unsigned char *prow = smem + Lay::OFF_P + h * Lay::kP + wt * 128;
        const int ring = kCols ? 0 : h * Lay::kKD;
        constexpr int kC = NT < 16 ? NT : 16;    // columns that are taken at a time
        const int first = kCols ? 0 : h;         // the stream's first key tile of a segment
        const int col0 = kCols ? h * NT : 0;     // the query row of its first column
        float *red = fl + Lay::kRed + h * 4 * NT, *fac = fl + Lay::kFac + h * NT;
        volatile uint32_t *votes = reinterpret_cast<volatile uint32_t *>(fl + Lay::kFloats) + h * 2;
        uint32_t t = 0;                  // key tiles of this stream before this one
        uint32_t syncs = 0;              // of the stream's warps so far
        bool ok = true;
        SegInfo it{};
        // All warps of the stream meet (shared memory written before is visible after); true in `any` if one
        // of them voted. A bounded wait like every other: false ends the role. A warp can be one meeting
        // ahead of another at most, so the votes of two suffice.
        auto meet = [&](bool vote, bool &any) -> bool {
            if (__any_sync(kFull, vote) && lane == 0) votes[syncs & 1] = syncs + 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Lay::B_WG + h));
            const bool r = wait_for(bar(Lay::B_WG + h), syncs & 1, abort_flag);
            any = votes[syncs & 1] == syncs + 1;
            ++syncs;
            return r;
        };
        bool any = false;
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, it)) || it.j0 == it.j1) break;
            const int cnt = it.j1 - it.j0, rows = it.tok * p.G, par = n & 1;
            float *mx = fl + Lay::kMax + (par * 2 + h) * NT;
            const float *qs = fl + Lay::kQs + (n & 3) * Lay::kNC + col0;
            if (!(ok = wait_for(bar(Lay::B_QS + (n & 3)), (n >> 2) & 1, abort_flag))) break;  // the queries' scales
            float l[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) l[c] = 0.f;
            const int last_pos = it.p0 + it.tok - 1;
            for (int i = first; i < cnt; i += kStep, ++t) {
                const int key = (it.j0 + i) * BN + wt, n0 = (it.j0 + i) * BN;
                const int slot = ring + static_cast<int>(t % Lay::kKD);
                if (!(ok = wait_for(bar(Lay::B_KFULL + slot), (t / Lay::kKD) & 1, abort_flag))) break;
                const float *sc = reinterpret_cast<const float *>(smem + Lay::OFF_SCALE + slot * 2 * BN * 4);
                float ks = finite_or_nan(sc[wt]), vs = finite_or_nan(sc[BN + wt]);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_KEMPTY + slot));  // the scales have been read
                if (key < it.n_lo || key >= it.n_end) ks = vs = 1.f;    // no row sees it: whatever lies there
                const float lv = __log2f(vs), inv_vs = __frcp_rn(vs);
                if (!(ok = wait_for(bar(Lay::B_S + h), t & 1, abort_flag))) break;
                tc_fence_after();
                // every row sees every key of the tile?
                const bool masked = n0 + BN > it.p0 + 1 || (p.window > 0 && n0 < last_pos - p.window + 1);
                // the columns that see the key are [see0, see1): tokens from the key's own on, up to the window's
                const int since = key - it.p0;  // the first token that sees it
                const int see0 = min(max(since, 0), Lay::kNC) * p.G - col0;
                const int until = p.window > 0 && since < Lay::kNC - p.window ? max(since + p.window, 0) : Lay::kNC;
                const int see1 = max(until * p.G - col0, see0);
                float x[NT];
                const uint64_t ks2 = f2_pack(ks, ks), lv2 = f2_pack(lv, lv);
                // x = log2 of the weights, less `less` (the references, or 0); the largest
                auto read_s = [&](const float *less) {
#pragma unroll
                    for (int c = 0; c < NT; c += kC) {
                        uint32_t s0[kC], s1[kC];
                        tmem_ld<kC>(s_row + c, s0);
                        tmem_ld<kC>(s_row + NT + c, s1);
                        tmem_wait_ld();
                        uint64_t y[kC / 2];
#pragma unroll
                        for (int e = 0; e < kC / 2; ++e)
                            y[e] = f2_fma(u2_pack(s1[2 * e], s1[2 * e + 1]), f2_pack(0x1p-5f, 0x1p-5f), u2_pack(s0[2 * e], s0[2 * e + 1]));
                        if constexpr (QP == 3) {
                            tmem_ld<kC>(s_row + 2 * NT + c, s0);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < kC / 2; ++e)
                                y[e] = f2_fma(u2_pack(s0[2 * e], s0[2 * e + 1]), f2_pack(0x1p-10f, 0x1p-10f), y[e]);
                        }
#pragma unroll
                        for (int e = 0; e < kC; e += 4) {
                            const float4 f4 = *reinterpret_cast<const float4 *>(qs + c + e), m4 = *reinterpret_cast<const float4 *>(less + c + e);
                            const uint64_t a = f2_fma(f2_mul(y[e >> 1], f2_pack(f4.x, f4.y)), ks2, lv2),
                                           b = f2_fma(f2_mul(y[(e >> 1) + 1], f2_pack(f4.z, f4.w)), ks2, lv2);
                            if constexpr (E::kIsBf16) {  // (packed, which gains 2 % there; in fp16 it costs as much at 63 rows)
                                const uint64_t neg = f2_pack(-1.f, -1.f);
                                const uint64_t xa = f2_fma(f2_pack(m4.x, m4.y), neg, a), xb = f2_fma(f2_pack(m4.z, m4.w), neg, b);
                                x[c + e] = f2_lo(xa), x[c + e + 1] = f2_hi(xa), x[c + e + 2] = f2_lo(xb), x[c + e + 3] = f2_hi(xb);
                            } else {
                                x[c + e] = f2_lo(a) - m4.x, x[c + e + 1] = f2_hi(a) - m4.y;
                                x[c + e + 2] = f2_lo(b) - m4.z, x[c + e + 3] = f2_hi(b) - m4.w;
                            }
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < NT; ++c)
                            if (static_cast<unsigned>(c - see0) >= static_cast<unsigned>(see1 - see0)) x[c] = -INFINITY;
                    }
                    float most = -INFINITY;
#pragma unroll
                    for (int c = 0; c < NT; c += 2) most = max_of(most, x[c], x[c + 1]);
                    return most;
                };
                // A reference moves when some x exceeds it by more than kAbove: the sum uses the same
                // reference, so the result is exact, and the weights stay at most 2^kAbove. The segment's first tile sets the
                // references. (Where they move the scores are read once more, by the same code.)
                any = i == first;
#pragma unroll 1
                for (bool set = false;;) {
                    const float most = read_s(any ? fl + Lay::kZero : mx);
                    if (!any) {
                        if (set || !(ok = meet(most > kAbove<E::kIsBf16>, any)) || !any) break;
                        continue;
                    }
#pragma unroll
                    for (int c = 0; c < NT; c += 4) {
                        const float4 top = make_float4(warp_most(x[c]), warp_most(x[c + 1]), warp_most(x[c + 2]), warp_most(x[c + 3]));
                        if (lane == 0) *reinterpret_cast<float4 *>(red + quarter * NT + c) = top;
                    }
                    if (!(ok = meet(false, any))) break;
                    if (wt < NT) {
                        const float most = fmaxf(fmaxf(red[wt], red[NT + wt]), fmaxf(red[2 * NT + wt], red[3 * NT + wt]));
                        // columns without a query row have a reference that leaves them no weight
                        const float old = i > first ? mx[wt] : col0 + wt < rows ? kUnset : INFINITY;
                        const bool move = most > old + kAbove<E::kIsBf16>;  // never where old is +inf, or the largest -inf
                        fac[wt] = move ? fast_exp2(old - (most - kBelow<E::kIsBf16>)) : 1.f;
                        mx[wt] = move ? most - kBelow<E::kIsBf16> : old;
                    }
                    if (!(ok = meet(false, any))) break;
#pragma unroll
                    for (int c = 0; c < NT; c += 4) {
                        const float4 f4 = *reinterpret_cast<const float4 *>(fac + c);
                        l[c] *= f4.x, l[c + 1] *= f4.y, l[c + 2] *= f4.z, l[c + 3] *= f4.w;
                    }
                    if (i > first) {
                        if (!(ok = wait_for(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < Lay::kO; c += 16) {
                            uint32_t ov[16];
                            tmem_ld<16>(o_row + c, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * fac[(c + e) % NT]);
                            tmem_st16(o_row + c, ov);
                        }
                        tmem_wait_st();
                    }
                    any = false;
                    set = true;
                }
                if (!ok) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_F + h));  // S has been read
                // the stream's previous PV has read W
                if (t > 0 && !(ok = wait_for(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
                // the weights as the tensor cores take them, three pieces each; the sum is of the weights themselves
                const uint64_t inv2 = f2_pack(inv_vs, inv_vs);
#pragma unroll
                for (int q = 0; q < NT / kC; ++q) {
                    uint32_t piece[Lay::PP][kC / 4];
#pragma unroll
                    for (int e = 0; e < kC / 4; ++e) {
                        const int c = q * kC + e * 4;
                        __half2 w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float w0 = fast_exp2(x[c + 2 * i]), w1 = fast_exp2(x[c + 2 * i + 1]);
                            if constexpr (E::kIsBf16) {
                                const uint64_t sum = f2_fma(f2_pack(w0, w1), inv2, f2_pack(l[c + 2 * i], l[c + 2 * i + 1]));
                                l[c + 2 * i] = f2_lo(sum), l[c + 2 * i + 1] = f2_hi(sum);
                            } else {
                                l[c + 2 * i] = fmaf(w0, inv_vs, l[c + 2 * i]);
                                l[c + 2 * i + 1] = fmaf(w1, inv_vs, l[c + 2 * i + 1]);
                            }
                            w[i] = __floats2half2_rn(w0, w1);
                        }
#pragma unroll
                        for (int i = 0; i < Lay::PP; ++i) {
                            if constexpr (E::kIsBf16) {
                                const bool last = i + 1 == Lay::PP;
                                const uint32_t a = to_e5m2x2(w[0], !last), b = to_e5m2x2(w[1], !last);
                                piece[i][e] = __byte_perm(a, b, 0x7531);
                                if (!last) w[0] = left_of_e5m2(w[0], a, i == 0), w[1] = left_of_e5m2(w[1], b, i == 0);
                            } else {
                                const uint32_t a = to_e4m3x2(w[0]), b = to_e4m3x2(w[1]);
                                piece[i][e] = a | b << 16;
                                if (i + 1 < Lay::PP) w[0] = left_of(w[0], a), w[1] = left_of(w[1], b);
                            }
                        }
                    }
                    // 16-byte chunk c of a key's row sits at c ^ (key % 8)
                    if constexpr (kC == 8) {  // two pieces in a chunk
                        *reinterpret_cast<uint4 *>(prow + ((wt & 7) << 4)) = make_uint4(piece[0][0], piece[0][1], piece[1][0], piece[1][1]);
                        *reinterpret_cast<uint4 *>(prow + ((1 ^ (wt & 7)) << 4)) = make_uint4(piece[2][0], piece[2][1], 0u, 0u);
                    } else {
#pragma unroll
                        for (int i = 0; i < Lay::PP; ++i)
                            *reinterpret_cast<uint4 *>(prow + (((i * (NT / 16) + q) ^ (wt & 7)) << 4)) =
                                make_uint4(piece[i][0], piece[i][1], piece[i][2], piece[i][3]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_P + h));
            }
            if (!ok) break;
            // ---- the segment's end: sums over the warp's keys
            float *sums = fl + Lay::kSum + ((par * 2 + h) * 4 + quarter) * NT;
            const float sum_c = fold(l, [](float a, float b) { return a + b; });
            if (lane < NT) sums[lane] = sum_c;
            const int cnt_b = kCols ? 0 : cnt / 2;  // tiles of the other stream's accumulator to be joined with A's
            // this stream's products are complete; then, where the streams halve the keys, both streams', with
            // their references and sums
            if (cnt > first && !(ok = wait_for(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
            if constexpr (kCols) {
                if (!(ok = meet(false, any))) break;
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_BOTH));
                if (!(ok = wait_for(bar(Lay::B_BOTH), n & 1, abort_flag))) break;
            }
            tc_fence_after();
            // this stream writes the query rows [c_lo, c_lo + kMine): its own, or half of the streams' common ones (A all of eight)
            constexpr int kMine = kCols || NT == 8 ? NT : NT / 2;
            const int c_lo = h * kMine, acc = kCols ? h : 0;  // the stream whose state counts as A's
            const bool bad = bad_seg[n & (kBadRing - 1)] == n + 1;  // a table entry of the segment was bad
            float *piece = it.part < 0 ? nullptr
                                       : p.pieces + (static_cast<size_t>(blockIdx.x) * 2 + it.part) * Lay::kPieceFloats;
            float *wa = fl + Lay::kWgt + par * 2 * NT, *wb = wa + NT;
            if (wt < kMine && c_lo < Lay::kNC) {
                const int c = c_lo + wt, ca = c - (kCols ? col0 : 0);  // its column in the stream
                const float *sa = fl + Lay::kSum + (par * 2 + acc) * 4 * NT + ca, *sb = fl + Lay::kSum + (par * 2 + 1) * 4 * NT + ca;
                const float ma = fl[Lay::kMax + (par * 2 + acc) * NT + ca], mb = cnt_b > 0 ? fl[Lay::kMax + (par * 2 + 1) * NT + ca] : kUnset;
                const float la = (sa[0] + sa[NT]) + (sa[2 * NT] + sa[3 * NT]);
                const float lb = cnt_b > 0 ? (sb[0] + sb[NT]) + (sb[2 * NT] + sb[3 * NT]) : 0.f;
                const float m = fmaxf(ma, mb), fa = fast_exp2(ma - m), fb = cnt_b > 0 ? fast_exp2(mb - m) : 0.f;
                const float sum = fa * la + fb * lb;
                float scale = 1.f;  // a piece: O unnormalised, with its reference and sum (sum -1: bad)
                if (!piece) scale = sum > 0.f ? 1.f / sum : sum == sum ? 0.f : sum;
                wa[c] = fa * scale;
                if (!kCols) wb[c] = fb * scale;
                if (piece) {
                    piece[c] = m;
                    piece[Lay::kNC + c] = bad ? -1.f : sum;
                }
            }
            if (!(ok = meet(false, any))) break;
            const uint32_t oa = tmem + lane_off + 2 * Lay::kS + acc * Lay::kO - (kCols ? col0 : 0), ob = oa + Lay::kO;  // at column c: + c
            const int d = wt;  // element of the head
            T *out = static_cast<T *>(p.out);
            constexpr int W = 8;
#pragma unroll 1
            for (int c0 = c_lo; c0 < c_lo + kMine && c0 < rows; c0 += W) {
                float o[W];
                // the pieces of column c0 + e of an accumulator, joined
                auto read_o = [&](uint32_t at, float (&v)[W]) {
                    uint32_t part[Lay::PP][W];
#pragma unroll
                    for (int i = 0; i < Lay::PP; ++i) tmem_ld<W>(at + i * NT + c0, part[i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        v[e] = __uint_as_float(part[Lay::PP - 1][e]);
#pragma unroll
                        for (int i = Lay::PP - 2; i >= 0; --i)
                            v[e] = fmaf(v[e], !E::kIsBf16 ? 0x1p-5f : i == 0 ? 0x1p-3f : 1.f, __uint_as_float(part[i][e]));
                    }
                };
                read_o(oa, o);
#pragma unroll
                for (int e = 0; e < W; ++e) o[e] *= wa[c0 + e];
                if (cnt_b > 0) {
                    float v[W];
                    read_o(ob, v);
#pragma unroll
                    for (int e = 0; e < W; ++e) o[e] = fmaf(v[e], wb[c0 + e], o[e]);
                }
                if (d >= HD) continue;
                if (piece) {
                    float *pc = piece + 2 * Lay::kNC + c0 * HD + d;  // columns behind the rows: room, never read
#pragma unroll
                    for (int e = 0; e < W; ++e) pc[e * HD] = o[e];
                } else {
                    const int tk = p.div_g(c0);
                    int in_tok = c0 - tk * p.G;
                    T *oc = out + (static_cast<size_t>(it.tok0 + tk) * p.Hq + it.g * p.G + in_tok) * HD + d;
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        if (c0 + e < rows) *oc = T(bad ? 0.f : o[e]);
                        oc += HD;
                        if (++in_tok == p.G) in_tok = 0, oc += (p.Hq - p.G) * HD;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Lay::B_OFREE + acc));
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
    }
    // ------------------------------------------------------------------------------------------
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, Lay::kTmem);
    }
}

template <class E, int HD, int NT, bool kCols, bool kGather>
cudaError_t launch_typed(const Q8Params &prm, cudaStream_t stream) {
    using Lay = LayQ8<HD, NT, E::kIsBf16 ? 2 : 3, kCols>;
    auto kern = chunk_q8_kernel<E, HD, NT, kCols, kGather>;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmem);
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay::kSmem;
    if ((e = cudaLaunchKernelEx(&cfg, kern, prm)) != cudaSuccess) return e;  // as in chunk_attn.cu
    cfg.dynamicSmemBytes = 0;
    const int rows = (prm.max_seqlen_q < prm.item_tok ? prm.max_seqlen_q : prm.item_tok) * prm.G;
    cfg.gridDim = dim3(P, (rows * (HD / 4) + kJoinWork - 1) / kJoinWork);
    cfg.blockDim = dim3(kJoinWork * kJoinGroups);
    return cudaLaunchKernelEx(&cfg, chunk_narrow_join_kernel<E, HD, Lay::kNC>, static_cast<const ChunkParams &>(prm));
}

// room for the pieces of every form: two row tiles of chunk_attn_q8_wide.cu are the largest
size_t piece_bytes(int D) { return wide_piece_floats(D) * 4; }

}  // namespace

size_t chunk_q8_workspace(int D) {
    const size_t P = device_sm_count();
    return P * 2 * piece_bytes(D) + P * sizeof(PieceRec);
}

cudaError_t launch_chunk_q8(const ChunkQ8Args &x, cudaStream_t stream) {
    const ChunkArgs &a = x.chunk;
    Q8Params prm{};
    int R = 1;  // rows per K/V box: the largest power of two dividing the block size, at most 128
    while (R < 128 && a.block_size % (2 * R) == 0) R *= 2;
    const bool gather = R < 8;  // less than a swizzle atom of 8 rows
    prm.G = a.Hq / a.Hkv;
    prm.inv_g = (65536 + prm.G - 1) / prm.G;
    const long long rows = static_cast<long long>(a.max_seqlen_q) * prm.G;
    // Up to eight rows (bf16, whose two pieces of eight columns are the least N of the instruction) a form of their own halves the
    // softmax: 256 single tokens 197 -> 190 us.
    // gathered keys are bound by the one warp that copies them, whatever the columns: one form for all
    const int form = gather || rows > 32 ? 64 : rows > 16 ? 32 : rows > 8 || a.dtype != PA_BF16 ? 16 : 8;
    prm.tt = prm.item_tok = form / prm.G;
    prm.cu_q = a.cu_q;
    prm.ctx = a.ctx;
    prm.block_tables = a.block_tables;
    prm.q = a.q;
    prm.k_cache = a.k_cache;
    prm.v_cache = a.v_cache;
    prm.k_scale = x.k_scale;
    prm.v_scale = x.v_scale;
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
    // Items of 256 rows from 65 rows a kv head on. 8 sequences of 6000 keys, 16/8 heads x 128, bf16: 34 rows 51 us here, 64 rows
    // 63.5 (there 65.5), 66 rows 65.5 there; at 64 rows and head dim 64 (32 sequences of 4000) 65.5 here, 71.6 there.
    if (rows > 64) return launch_chunk_q8_wide(prm, x, stream);
    const long long krows = static_cast<long long>(a.num_blocks) * a.block_size;
    if (!gather && (!encode_rows_e4m3(&prm.tm_k, a.k_cache, a.Hkv, a.D, krows, R, true) ||
                    !encode_rows_e4m3(&prm.tm_v, a.v_cache, a.Hkv, a.D, krows, R, true)))
        return cudaErrorInvalidValue;
    auto go = [&](auto e, auto hd) {
        using E = decltype(e);
        constexpr int HD = decltype(hd)::value;
        if (gather) return launch_typed<E, HD, 32, true, true>(prm, stream);
        if constexpr (E::kIsBf16) {
            if (form == 8) return launch_typed<E, HD, 8, false, false>(prm, stream);
        }
        if (form == 16) return launch_typed<E, HD, 16, false, false>(prm, stream);
        if (form == 32) return launch_typed<E, HD, 32, false, false>(prm, stream);
        return launch_typed<E, HD, 32, true, false>(prm, stream);
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (a.dtype == PA_BF16) return a.D == 64 ? go(BF16{}, I64{}) : go(BF16{}, I128{});
    return a.D == 64 ? go(F16{}, I64{}) : go(F16{}, I128{});
}

}  // namespace pa
