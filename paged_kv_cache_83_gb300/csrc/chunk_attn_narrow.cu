// chunk_attn_narrow.cu: pa_chunk_attn for chunks of at most 64 query rows a kv head (tokens x group),
// such as drafts to verify.
//
// With few query rows a tile of 128 rows would leave most of the matrix instructions' rows and, worse,
// of the softmax's threads empty while the others walk over 128 keys each. So the operands change
// places: keys are the 128 rows, query rows the NT = 16, 32 or 64 columns,
//   S^T = K Q^T,   O^T += V^T P^T,
// and a softmax thread owns one key and all query rows, NT elements a tile. The running maximum of a
// column then lies across threads; it moves only when some score exceeds it by more than 2^8, which a
// block-wide vote finds, so that the reduction over threads runs about once a segment. Sums stay
// in each thread until the segment ends.
//
// Bound by HBM: every key and value is read once per kv head (2.2 GB for 256 drafts of up to 5 tokens
// over contexts to 4096 take 345-353 us, 0.93 of the copy bandwidth; with 128-row tiles 684 us). The
// loads run ahead in rings of tiles; two streams of softmax warps take the key tiles in
// turn, each with its own maximum, sum and accumulator, so that one computes while the other waits
// for its matrix products. They join at the end of a segment.
//
//   warp 3      scheduler, as in chunk_attn.cu (an item is a whole chunk here)
//   warp 0      producer: Q of up to two segments, and the streams' K and V tiles in turn
//   warps 1, 2  one MMA issuer per stream
//   warps 4-7   softmax of stream A (tiles 0, 2, ... of a segment), warps 8-11 of stream B (1, 3, ...)
// With 33 to 64 query rows the streams take half of the columns each instead, of every key tile: 64 scores
// and 64 sums a thread do not fit the registers (3 drafts of 3-8 tokens, groups of 7, at 9-16k
// contexts: 28 us against 22).
//   TMEM columns: S_A, S_B, O_A, O_B of NT columns each; lanes are keys in S and head elements in O.
#include <type_traits>

#include "chunk_common.cuh"

namespace pa {

namespace {

using namespace chunk;

// NT columns a stream. kCols: the streams halve the query rows (2 NT of them) and both take every key tile, from
// rings that they share; else they halve the key tiles, each with rings of its own.
template <int HD, int NT, bool kCols>
struct Narrow {
    static constexpr int kNC = kCols ? 2 * NT : NT;     // query rows
    static constexpr int kKV = BN * HD * 2;
    static constexpr int kHalves = HD / 64;
    static constexpr int kQHalf = kNC * 128;            // 64 columns of the query rows
    static constexpr int kQ = kQHalf * kHalves;
    static constexpr int kQStep = (kQ + 1023) / 1024 * 1024;
    static constexpr int kP = BN * 128;                 // P^T: a 128-byte row a key
    static constexpr int kSlots = HD == 128 ? 2 : 4;    // K tiles held, and V tiles
    static constexpr int kD = kCols ? kSlots : kSlots / 2;  // of a ring
    // barriers; rings, S, F, P, O, WG: + stream
    static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_KEMPTY = B_KFULL + kSlots,
                         B_VFULL = B_KEMPTY + kSlots, B_VEMPTY = B_VFULL + kSlots, B_S = B_VEMPTY + kSlots, B_F = B_S + 2,
                         B_P = B_F + 2, B_WG = B_P + 2, B_O = B_WG + 2, B_OFREE = B_O + 2, B_BOTH = B_OFREE + 2,
                         B_END = B_BOTH + 1, B_IFULL = B_END + 2, B_IEMPTY = B_IFULL + 4, NBAR = B_IEMPTY + 4;
    // shared memory: V's rings before K's (at head dim 64 the V operand's unused upper half of rows reads
    // one tile further)
    static constexpr int OFF_V = 0, OFF_K = kSlots * kKV, OFF_Q = OFF_K + kSlots * kKV, OFF_P = OFF_Q + 2 * kQStep;
    static constexpr int OFF_F = OFF_P + 2 * kP;        // floats below
    // per segment parity and stream: maxima [NT], sums by warp [4][NT], weights [NT]; and scratch
    static constexpr int kMax = 0, kSum = 2 * 2 * NT, kWgt = kSum + 2 * 2 * 4 * NT, kRed = kWgt + 2 * 2 * NT,
                         kFac = kRed + 2 * 4 * NT, kFloats = kFac + 2 * NT;
    static constexpr int OFF_BAR = OFF_F + kFloats * 4 + 16;  // after the votes
    static constexpr int OFF_ITEMS = OFF_BAR + NBAR * 8;
    static constexpr int OFF_BAD = OFF_ITEMS + 4 * static_cast<int>(sizeof(SegInfo));
    static constexpr int OFF_PLAN = (OFF_BAD + kBadRing * 4 + 15) / 16 * 16;
    static constexpr int OFF_MISC = OFF_PLAN + 12 * 8 + static_cast<int>(sizeof(Share));
    static constexpr int kSmem = OFF_MISC + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr int kTmem = 4 * NT < 32 ? 32 : 4 * NT;
    static constexpr size_t kPieceFloats = static_cast<size_t>(kNC) * (HD + 2);  // m[kNC], l[kNC], O[kNC][HD]
};

// instruction descriptor with A stored with its rows (M) contiguous
__host__ __device__ constexpr uint32_t idesc_a_mn(uint32_t idesc) { return idesc | (1u << 15); }

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t *r) {
    static_assert(N == 8 || N == 16);
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
}
// Reduces W columns over the warp's lanes: lane c (of 32; c % W) gets column c's result. Halves of the columns
// change places with the lane W / 2, W / 4, ... away.
template <int W, class F>
__device__ __forceinline__ float fold(float (&v)[W], F op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = W / 2; w > 0; w >>= 1) {
        const bool upper = lane & w;
#pragma unroll
        for (int c = 0; c < w; ++c) {
            const float give = upper ? v[c] : v[c + w], keep = upper ? v[c + w] : v[c];
            v[c] = op(keep, __shfl_xor_sync(kFull, give, w));
        }
    }
#pragma unroll
    for (int w = W; w < 32; w <<= 1) v[0] = op(v[0], __shfl_xor_sync(kFull, v[0], w));
    return v[0];
}
constexpr float kUnset = -3e38f;  // the maximum of a column that has seen no key: finite, below every score

template <class E, int HD, int NT, bool kCols, bool kGather>
__global__ void __launch_bounds__(kThreads, 1) chunk_narrow_kernel(const __grid_constant__ ChunkParams p) {
    using T = typename E::T;
    using Lay = Narrow<HD, NT, kCols>;
    constexpr int kStep = kCols ? 1 : 2;  // key tiles from one to the next of a stream
    constexpr int kHalves = Lay::kHalves;
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
        if (tid >= Lay::B_QEMPTY && tid < Lay::B_KFULL) count = 2;       // both issuers
        if (kCols && ((tid >= Lay::B_KEMPTY && tid < Lay::B_VFULL) || (tid >= Lay::B_VEMPTY && tid < Lay::B_S))) count = 2;
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
    // Launched beside what precedes it in the stream: nothing that it wrote is read, and nothing that it reads is
    // written, before it has finished (the set-up above takes place meanwhile).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Tensor memory is taken only now, and the joining kernel (and with it what follows) let in only when it is
    // there: no block holds tensor memory while it waits for another grid, whose blocks on this SM may want some.
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), Lay::kTmem);
    if (tid == 0) p.recs[blockIdx.x].valid = 0;
    plan_share(p, plan, share);
    zero_bad_sequences<T, HD>(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel waits for this grid itself
    const uint32_t tmem = *tmem_slot;

    // every role reads the segments in the same order: segment n sits in queue entry n % 4
    auto read_seg = [&](int n, SegInfo &it) -> bool {
        if (!warp_wait(bar(Lay::B_IFULL + (n & 3)), (n >> 2) & 1, abort_flag)) return false;
        it = items[n & 3];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_IEMPTY + (n & 3)));
        return true;
    };

    if (warp == 3) {
        // ================================== scheduler ==================================
        int published = 0;
        const bool ok = walk_share(p, *share, [&](const SegInfo &it) {
            if (!warp_wait(bar(Lay::B_IEMPTY + (published & 3)), ((published >> 2) & 1) ^ 1, abort_flag)) return false;
            if (lane == 0) {
                items[published & 3] = it;
                mbar_arrive(bar(Lay::B_IFULL + (published & 3)));
            }
            __syncwarp();
            ++published;
            return true;
        });
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
        constexpr int kRowsLane = kGather ? BN / 32 : 1;
        struct Rows {
            long long r[kRowsLane];
            int g;
        };
        auto rows_of = [&](const SegInfo &it, int j, int seg_no) {
            Rows w;
            w.g = it.g;
#pragma unroll
            for (int i = 0; i < kRowsLane; ++i) {
                const int pos = j * BN + (kGather ? lane + 32 * i : lane * R);
                w.r[i] = kGather || lane < nbox ? pool_row(p, it, pos, kGather ? pos : pos + R - 1, bad_seg, seg_no) : -1;
            }
            return w;
        };
        uint32_t nk[2] = {0, 0}, nv[2] = {0, 0};  // tiles loaded, by stream
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
        auto load = [&](const Rows &w, bool is_v, auto stream) -> bool {
            constexpr int h = decltype(stream)::value;
            const uint32_t i = is_v ? nv[h]++ : nk[h]++;
            const int slot = h * Lay::kD + static_cast<int>(i % Lay::kD);
            const uint32_t full = bar((is_v ? Lay::B_VFULL : Lay::B_KFULL) + slot);
            const uint32_t dst = sbase + (is_v ? Lay::OFF_V : Lay::OFF_K) + slot * Lay::kKV;
            const uint32_t empty = bar((is_v ? Lay::B_VEMPTY : Lay::B_KEMPTY) + slot), par = ((i / Lay::kD) & 1) ^ 1;
            // a gathered tile is not held back while this one waits for its slot
            if (kGather && !__all_sync(kFull, mbar_try_wait(empty, par))) flush();
            if (!warp_wait(empty, par, abort_flag)) return false;
            if constexpr (kGather) {
                gather_tile<T, HD>(dst, static_cast<const T *>(is_v ? p.v_cache : p.k_cache), w.r, p.Hkv, w.g);
                cp_async_wait<1>();
                announce(full);
            } else {
                const uint32_t bytes = __popc(__ballot_sync(kFull, w.r[0] >= 0)) * box_bytes * kHalves;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (w.r[0] >= 0)
                    for (int half = 0; half < kHalves; ++half)
                        tma_load_3d(dst + lane * R * 128 + half * kHalf, is_v ? &p.tm_v : &p.tm_k, half * 64, w.g,
                                    static_cast<int>(w.r[0]), full);
            }
            return true;
        };
        int n = 0;  // segments taken
        bool ok = true;
        SegInfo cur{};
        Rows pend[2]{}, next{};
        bool has[2] = {false, false};
        // The last tile of each stream whose V is still to come: loaded after the stream's next K, and
        // those of the segment before as soon as a segment's first K is under way. An issuer takes the first
        // K of a segment only when the V of the segment before has been used, so that no load may
        // wait for that K to be taken with such a V outstanding.
        using A = std::integral_constant<int, 0>;
        using B = std::integral_constant<int, 1>;
        auto pending = [&](auto stream) -> bool {
            constexpr int h = decltype(stream)::value;
            const bool r = !has[h] || load(pend[h], true, stream);
            has[h] = false;
            return r;
        };
        while (ok) {
            if (!(ok = read_seg(n, cur)) || cur.j0 == cur.j1) break;
            // the segment's Q, ahead of the issuers
            flush();
            if (!(ok = warp_wait(bar(Lay::B_QEMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag))) break;
            next = rows_of(cur, cur.j0, n);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Lay::B_QFULL + (n & 1)), kHalves * static_cast<uint32_t>(p.item_tok) * p.G * 128);
                for (int half = 0; half < kHalves; ++half)
                    tma_load_3d(sbase + Lay::OFF_Q + (n & 1) * Lay::kQStep + half * Lay::kQHalf, &p.tm_q, half * 64,
                                cur.g * p.G, cur.tok0, bar(Lay::B_QFULL + (n & 1)));
            }
            __syncwarp();
            auto tile = [&](int j, auto stream) -> bool {
                constexpr int h = decltype(stream)::value;
                const Rows w = next;
                if (j + 1 < cur.j1) next = rows_of(cur, j + 1, n);  // in flight while this tile is loaded
                if (!load(w, false, stream) || !pending(stream) || (j == cur.j0 && !pending(B{}))) return false;
                pend[h] = w;
                has[h] = true;
                return true;
            };
            for (int j = cur.j0; ok && j < cur.j1; j += kStep)
                ok = tile(j, A{}) && (kCols || j + 1 == cur.j1 || tile(j + 1, B{}));
            ++n;
        }
        ok = ok && pending(A{}) && pending(B{});
        flush();
        if (!ok && lane == 0) give_up(p.err, abort_flag);
        // no copy may still be in flight at exit: the last load of every slot, the last two Q
        if (lane == 0) {
            if (!kGather)
#pragma unroll
                for (int h = 0; h < (kCols ? 1 : 2); ++h)
#pragma unroll
                    for (uint32_t back = 1; back <= Lay::kD; ++back) {
                        if (nk[h] >= back) {
                            const uint32_t i = nk[h] - back;
                            if (!mbar_wait(bar(Lay::B_KFULL + h * Lay::kD + i % Lay::kD), (i / Lay::kD) & 1))
                                give_up(p.err, abort_flag);
                        }
                        if (nv[h] >= back) {
                            const uint32_t i = nv[h] - back;
                            if (!mbar_wait(bar(Lay::B_VFULL + h * Lay::kD + i % Lay::kD), (i / Lay::kD) & 1))
                                give_up(p.err, abort_flag);
                        }
                    }
            for (int i = n > 2 ? n - 2 : 0; i < n; ++i)
                if (!mbar_wait(bar(Lay::B_QFULL + (i & 1)), (i >> 1) & 1)) give_up(p.err, abort_flag);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ============================ MMA issuer of one stream =============================
        const int h = warp - 1;
        constexpr uint32_t IQK = idesc_f16(BM, NT, E::kIsBf16, false);              // A = K rows, B = Q rows, both K-major
        constexpr uint32_t IPV = idesc_a_mn(idesc_f16(BM, NT, E::kIsBf16, true));   // A = V^T, B = P^T, both MN-major
        const int ring = kCols ? 0 : h * Lay::kD, first = kCols ? 0 : h;  // the stream's first slot, and key tile
        const uint64_t dq0 = smem_desc_sw128(sbase + Lay::OFF_Q + (kCols ? h * NT * 128 : 0), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(sbase + Lay::OFF_K + ring * Lay::kKV, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(sbase + Lay::OFF_V + ring * Lay::kKV, kHalf, 1024);
        const uint64_t dp = smem_desc_sw128(sbase + Lay::OFF_P + h * Lay::kP, kHalf, 1024);
        const uint32_t s_tm = tmem + h * NT, o_tm = tmem + (2 + h) * NT;
        auto qk = [&](int slot, int q) {  // S^T = K Q^T
            const uint64_t a = dk0 + slot * (Lay::kKV >> 4), b = dq0 + q * (Lay::kQStep >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
                tc_mma_ss(s_tm, a + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                          b + (((kk >> 2) * Lay::kQHalf + (kk & 3) * 32) >> 4), IQK, kk > 0);
        };
        auto pv = [&](int slot, bool acc) {  // O^T += V^T P^T, 16 keys an instruction
            const uint64_t a = dv0 + slot * (Lay::kKV >> 4);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                tc_mma_ss(o_tm, a + ((kk * 2048) >> 4), dp + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
        };
        uint32_t t = 0;  // key tiles of this stream: QKs issued
        bool ok = true;
        SegInfo it{};
        // QK of the stream's next tile once S has been read; `last`: of the segment
        auto issue_qk = [&](int n, bool last) -> bool {
            const int slot = static_cast<int>(t % Lay::kD);
            if (t > 0 && !warp_wait(bar(Lay::B_F + h), (t - 1) & 1, abort_flag)) return false;
            if (!warp_wait(bar(Lay::B_KFULL + ring + slot), (t / Lay::kD) & 1, abort_flag)) return false;
            tc_fence_after();
            if (lane == 0) {
                qk(slot, n & 1);
                tc_commit(bar(Lay::B_S + h));
                tc_commit(bar(Lay::B_KEMPTY + ring + slot));
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
            if (!(ok = warp_wait(bar(Lay::B_QFULL + (n & 1)), (n >> 1) & 1, abort_flag))) break;
            if (first >= cnt) {  // a segment of one tile has none for stream B
                if (lane == 0) mbar_arrive(bar(Lay::B_QEMPTY + (n & 1)));
                __syncwarp();
                continue;
            }
            if (!(ok = issue_qk(n, first + kStep >= cnt))) break;
            for (int i = first; i < cnt; i += kStep, ++done) {
                if (i + kStep < cnt && !(ok = issue_qk(n, i + 2 * kStep >= cnt))) break;
                const int slot = static_cast<int>(done % Lay::kD);
                if (!(ok = warp_wait(bar(Lay::B_VFULL + ring + slot), (done / Lay::kD) & 1, abort_flag))) break;
                const int n0 = (it.j0 + i) * BN, z0 = max(it.n_lo - n0, 0), z1 = min(it.n_end - n0, BN);
                // (streams that share the tile both write the zeros)
                if (z0 > 0 || z1 < BN) zero_rows<HD>(smem + Lay::OFF_V + (ring + slot) * Lay::kKV, z0, z1);
                if (!(ok = warp_wait(bar(Lay::B_P + h), done & 1, abort_flag))) break;
                // the previous segment's output must be out of TMEM before its O is overwritten. (B may have
                // had no tile in it; its softmax warps have then passed the end of that segment with A's.)
                if (i == first && n > 0 && !(ok = warp_wait(bar(Lay::B_OFREE + (kCols ? h : 0)), (n - 1) & 1, abort_flag)))
                    break;
                tc_fence_after();
                if (lane == 0) {
                    pv(slot, i > first);
                    tc_commit(bar(Lay::B_O + h));
                    tc_commit(bar(Lay::B_VEMPTY + ring + slot));
                }
                __syncwarp();
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
        const uint32_t s_row = tmem + lane_off + h * NT, o_row = tmem + lane_off + (2 + h) * NT;
        unsigned char *prow = smem + Lay::OFF_P + h * Lay::kP + wt * 128;
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
            const bool r = warp_wait(bar(Lay::B_WG + h), syncs & 1, abort_flag);
            any = votes[syncs & 1] == syncs + 1;
            ++syncs;
            return r;
        };
        bool any = false;
        for (int n = 0; ok; ++n) {
            if (!(ok = read_seg(n, it)) || it.j0 == it.j1) break;
            const int cnt = it.j1 - it.j0, rows = it.tok * p.G, par = n & 1;
            float *mx = fl + Lay::kMax + (par * 2 + h) * NT;
            // columns without a query row have a maximum that leaves them no weight
            if (wt < NT) mx[wt] = col0 + wt < rows ? kUnset : INFINITY;
            if (!(ok = meet(false, any))) break;
            float l[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) l[c] = 0.f;
            const int last_pos = it.p0 + it.tok - 1;
            for (int i = first; i < cnt; i += kStep, ++t) {
                if (!(ok = warp_wait(bar(Lay::B_S + h), t & 1, abort_flag))) break;
                tc_fence_after();
                const int key = (it.j0 + i) * BN + wt, n0 = (it.j0 + i) * BN;
                // every row sees every key of the tile?
                const bool masked = n0 + BN > it.p0 + 1 || (p.window > 0 && n0 < last_pos - p.window + 1);
                uint32_t sv[NT];
                auto read_s = [&]() {
#pragma unroll
                    for (int c = 0; c < NT; c += 16) tmem_ld<16>(s_row + c, sv + c);
                    tmem_wait_ld();
                    if (masked) {
                        const int tok_c = p.div_g(col0);
                        int pos = it.p0 + tok_c, in_tok = col0 - tok_c * p.G;
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            if (key > pos || (p.window > 0 && key <= pos - p.window)) sv[c] = 0xff800000u;  // -inf
                            if (++in_tok == p.G) in_tok = 0, ++pos;
                        }
                    }
                };
                auto shift = [&]() {  // s -> s * scale - reference, in place; the largest
                    float most = -INFINITY;
#pragma unroll
                    for (int c = 0; c < NT; c += 4) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(mx + c);
                        const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = fmaf(__uint_as_float(sv[c + e]), p.scale_log2, -mm[e]);
                            most = fmaxf(most, x);
                            sv[c + e] = __float_as_uint(x);
                        }
                    }
                    return most;
                };
                read_s();
                any = true;  // the segment's first tile sets the references
                if (i > first) {
                    // A reference moves when some score exceeds it by more than 2^8: the sum uses the same
                    // reference, so the result is exact, and P stays below 2^8.
                    if (!(ok = meet(shift() > 8.f, any))) break;
                }
                if (any) {
                    if (i > first) read_s();
                    float v[NT];
#pragma unroll
                    for (int c = 0; c < NT; ++c) v[c] = __uint_as_float(sv[c]);
                    const float top = fold(v, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < NT) red[quarter * NT + lane] = top;
                    if (!(ok = meet(false, any))) break;
                    if (wt < NT) {
                        const float x = fmaxf(fmaxf(red[wt], red[NT + wt]), fmaxf(red[2 * NT + wt], red[3 * NT + wt]));
                        const float old = mx[wt], top = x * p.scale_log2;
                        const bool move = top > old + 8.f;  // never where old is +inf, or x -inf
                        fac[wt] = move ? fast_exp2(old - top) : 1.f;
                        if (move) mx[wt] = top;
                    }
                    if (!(ok = meet(false, any))) break;
#pragma unroll
                    for (int c = 0; c < NT; c += 4) {
                        const float4 f4 = *reinterpret_cast<const float4 *>(fac + c);
                        l[c] *= f4.x, l[c + 1] *= f4.y, l[c + 2] *= f4.z, l[c + 3] *= f4.w;
                    }
                    if (i > first) {
                        if (!(ok = warp_wait(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < NT; c += 16) {
                            uint32_t ov[16];
                            tmem_ld<16>(o_row + c, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * fac[c + e]);
                            tmem_st16(o_row + c, ov);
                        }
                        tmem_wait_st();
                    }
                    shift();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_F + h));  // S has been read
                // the stream's previous PV has read P
                if (t > 0 && !(ok = warp_wait(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
#pragma unroll
                for (int q = 0; q < NT / 8; ++q) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = q * 8 + e * 2;
                        const float p0 = fast_exp2(__uint_as_float(sv[c])), p1 = fast_exp2(__uint_as_float(sv[c + 1]));
                        l[c] += p0;
                        l[c + 1] += p1;
                        // P is rounded to the storage type (the tensor cores' operand), the sum is not
                        pk[e] = E::pack2(p0, p1);
                    }
                    // 16-byte chunk q of a key's row sits at q ^ (key % 8)
                    *reinterpret_cast<uint4 *>(prow + ((q ^ (wt & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
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
            // their maxima and sums
            if (cnt > first && !(ok = warp_wait(bar(Lay::B_O + h), (t - 1) & 1, abort_flag))) break;
            if constexpr (kCols) {
                if (!(ok = meet(false, any))) break;
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Lay::B_BOTH));
                if (!(ok = warp_wait(bar(Lay::B_BOTH), n & 1, abort_flag))) break;
            }
            tc_fence_after();
            // this stream writes the query rows [c_lo, c_lo + kMine): its own, or half of the streams' common ones
            constexpr int kMine = kCols ? NT : NT / 2;
            const int c_lo = h * kMine, acc = kCols ? h : 0;  // the stream whose state counts as A's
            const bool bad = bad_seg[n & (kBadRing - 1)] == n + 1;  // a table entry of the segment was bad
            float *piece = it.part < 0 ? nullptr
                                       : p.pieces + (static_cast<size_t>(blockIdx.x) * 2 + it.part) * Lay::kPieceFloats;
            float *wa = fl + Lay::kWgt + par * 2 * NT, *wb = wa + NT;
            if (wt < kMine) {
                const int c = c_lo + wt, ca = c - (kCols ? col0 : 0);  // its column in the stream
                const float *sa = fl + Lay::kSum + (par * 2 + acc) * 4 * NT + ca, *sb = fl + Lay::kSum + (par * 2 + 1) * 4 * NT + ca;
                const float ma = fl[Lay::kMax + (par * 2 + acc) * NT + ca], mb = cnt_b > 0 ? fl[Lay::kMax + (par * 2 + 1) * NT + ca] : kUnset;
                const float la = (sa[0] + sa[NT]) + (sa[2 * NT] + sa[3 * NT]);
                const float lb = cnt_b > 0 ? (sb[0] + sb[NT]) + (sb[2 * NT] + sb[3 * NT]) : 0.f;
                const float m = fmaxf(ma, mb), fa = fast_exp2(ma - m), fb = cnt_b > 0 ? fast_exp2(mb - m) : 0.f;
                const float sum = fa * la + fb * lb;
                float scale = 1.f;  // a piece: O unnormalised, with its maximum and sum (sum -1: bad)
                if (!piece) scale = sum > 0.f ? 1.f / sum : sum == sum ? 0.f : sum;
                wa[c] = fa * scale;
                if (!kCols) wb[c] = fb * scale;
                if (piece) {
                    piece[c] = m;
                    piece[Lay::kNC + c] = bad ? -1.f : sum;
                }
            }
            if (!(ok = meet(false, any))) break;
            const uint32_t oa = tmem + lane_off + (2 + acc) * NT - (kCols ? col0 : 0), ob = oa + NT;  // at column c: + c
            const int d = wt;  // element of the head
            T *out = static_cast<T *>(p.out);
            constexpr int W = kMine < 16 ? 8 : 16;
#pragma unroll 1
            for (int c0 = c_lo; c0 < c_lo + kMine && c0 < rows; c0 += W) {
                uint32_t a[W], b[W];
                tmem_ld<W>(oa + c0, a);
                if (cnt_b > 0) tmem_ld<W>(ob + c0, b);
                tmem_wait_ld();
                float o[W];
#pragma unroll
                for (int e = 0; e < W; e += 4) {
                    const float4 fa = *reinterpret_cast<const float4 *>(wa + c0 + e);
                    o[e] = __uint_as_float(a[e]) * fa.x, o[e + 1] = __uint_as_float(a[e + 1]) * fa.y;
                    o[e + 2] = __uint_as_float(a[e + 2]) * fa.z, o[e + 3] = __uint_as_float(a[e + 3]) * fa.w;
                }
                if (cnt_b > 0)
#pragma unroll
                    for (int e = 0; e < W; ++e) o[e] = fmaf(__uint_as_float(b[e]), wb[c0 + e], o[e]);
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

// ------------------------------------------------------------------------------------------
// joining the pieces
// ------------------------------------------------------------------------------------------

constexpr int kJoinWork = 64, kJoinGroups = 4;  // outputs of four columns of a block; the pieces are dealt out to groups

// Block (c, y): outputs [64 y, 64 y + 64) of four columns each of the item whose first piece CTA c holds (its slot
// 1); the pieces after it are slot 0 of the CTAs up to last_cta. An item of a long sequence has tens of
// pieces: four groups of threads read four pieces each at a time (a thread for all 25 pieces of
// one, one after the other, took 41 us; so 4 us).
template <class E, int HD, int NT, bool kCols>
__global__ void __launch_bounds__(kJoinWork * kJoinGroups) chunk_narrow_join_kernel(const __grid_constant__ ChunkParams p) {
    using Lay = Narrow<HD, NT, kCols>;
    __shared__ float part[kJoinGroups][6][kJoinWork];
    // the next call's kernel may set itself up beside this one: it waits for this grid itself
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PieceRec rec = p.recs[blockIdx.x];
    if (!rec.valid) return;
    const int w = threadIdx.x % kJoinWork, grp = threadIdx.x / kJoinWork;
    const int at = blockIdx.y * kJoinWork + w, row = at / (HD / 4), col = at % (HD / 4) * 4;
    const bool live = row < rec.tok * p.G;
    const int first = blockIdx.x;
    float m = -INFINITY, l = 0.f, o[4] = {};
    bool bad = false;
    if (live) {
        for (int c0 = first + grp; c0 <= rec.last_cta; c0 += 4 * kJoinGroups) {
            float pm[4], pl[4];
            float4 po[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = c0 + k * kJoinGroups;
                pm[k] = -INFINITY, pl[k] = 0.f, po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c <= rec.last_cta) {
                    const float *src = p.pieces + (static_cast<size_t>(c) * 2 + (c == first)) * Lay::kPieceFloats;
                    pm[k] = __ldcg(src + row);  // written by the kernel this one was launched beside: not the read-only path
                    pl[k] = __ldcg(src + Lay::kNC + row);
                    po[k] = __ldcg(reinterpret_cast<const float4 *>(src + 2 * Lay::kNC + row * HD + col));
                }
            }
            const float mn = fmaxf(m, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
            const float mu = mn == -INFINITY ? 0.f : mn, f0 = fast_exp2(m - mu);
            l *= f0, o[0] *= f0, o[1] *= f0, o[2] *= f0, o[3] *= f0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = fast_exp2(pm[k] - mu);
                bad |= pl[k] == -1.f;
                l += f * pl[k];
                o[0] += f * po[k].x, o[1] += f * po[k].y, o[2] += f * po[k].z, o[3] += f * po[k].w;
            }
            m = mn;
        }
    }
    part[grp][0][w] = m;
    part[grp][1][w] = bad ? -1.f : l;
#pragma unroll
    for (int e = 0; e < 4; ++e) part[grp][2 + e][w] = o[e];
    __syncthreads();
    if (grp != 0 || !live) return;
    for (int g = 1; g < kJoinGroups; ++g) m = fmaxf(m, part[g][0][w]);
    const float mu = m == -INFINITY ? 0.f : m;
    l = o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll
    for (int g = 0; g < kJoinGroups; ++g) {
        const float f = fast_exp2(part[g][0][w] - mu), pl = part[g][1][w];
        bad |= pl == -1.f;
        l += f * pl;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += f * part[g][2 + e][w];
    }
    const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
    uint2 u = make_uint2(E::pack2(o[0] * inv, o[1] * inv), E::pack2(o[2] * inv, o[3] * inv));
    if (bad) u = make_uint2(0, 0);
    using T = typename E::T;
    const int tk = rec.tok0 + row / p.G, head = rec.g * p.G + row % p.G;
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (static_cast<size_t>(tk) * p.Hq + head) * HD + col) = u;
}

template <class E, int HD, int NT, bool kCols, bool kGather>
cudaError_t launch_typed(const ChunkParams &prm, cudaStream_t stream) {
    using Lay = Narrow<HD, NT, kCols>;
    auto kern = chunk_narrow_kernel<E, HD, NT, kCols, kGather>;
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
    cfg.gridDim = dim3(P, (prm.max_seqlen_q * prm.G * (HD / 4) + kJoinWork - 1) / kJoinWork);
    cfg.blockDim = dim3(kJoinWork * kJoinGroups);
    return cudaLaunchKernelEx(&cfg, chunk_narrow_join_kernel<E, HD, NT, kCols>, prm);
}

template <class E, int HD>
cudaError_t launch_rows(const ChunkParams &prm, bool gather, cudaStream_t stream) {
    const int rows = prm.max_seqlen_q * prm.G;
    // gathered keys are bound by the one warp that copies them, whatever the columns: one form for all (128 sequences at
    // contexts to 4096, 16/8 heads x 128, pages of 4: 470 us with 2 query rows a head, 482 with 32, 514 with 64, by
    // boxes 190-236; pages of one row 1365-1373)
    if (gather) return launch_typed<E, HD, 32, true, true>(prm, stream);
    if (rows <= 16) return launch_typed<E, HD, 16, false, false>(prm, stream);
    if (rows <= 32) return launch_typed<E, HD, 32, false, false>(prm, stream);
    return launch_typed<E, HD, 32, true, false>(prm, stream);
}

}  // namespace

cudaError_t launch_chunk_narrow(const chunk::ChunkParams &prm, pa_dtype dtype, int D, bool gather, cudaStream_t stream) {
    if (dtype == PA_BF16)
        return D == 64 ? launch_rows<BF16, 64>(prm, gather, stream) : launch_rows<BF16, 128>(prm, gather, stream);
    return D == 64 ? launch_rows<F16, 64>(prm, gather, stream) : launch_rows<F16, 128>(prm, gather, stream);
}

}  // namespace pa
