// chunk_common.cuh: what the kernels of pa_chunk_attn share: the items, the equal shares of the work, the
// scheduler's walk over a share, and the launch's tensor maps.
#pragma once

#include <cuda.h>
#include <math.h>

#include "pa_internal.h"

namespace pa {
namespace chunk {

constexpr int BM = 128, BN = 128;    // query rows of a tile, keys of a tile
constexpr int kThreads = 384;
constexpr int kHalf = BM * 64 * 2;   // one 128-row x 64-column half tile: 16 KB
constexpr unsigned kFull = 0xffffffffu;
constexpr int kItemReaders = 11;     // roles that read the queue of segments, by warp
constexpr int kBadRing = 8;          // segments whose table entries were bad, by segment number

// A segment: key tiles [j0, j1) of an item. tok0: its first token's row of q; tok: its tokens;
// p0: position of its first token; [n_lo, n_end): the keys that any of its rows sees.
// part: -1 the whole item, else the CTA's workspace slot. j1 == j0 marks the end of the work.
struct SegInfo {
    int s, g, tok0, tok, p0, n_lo, n_end, j0, j1, part;
};
// What the joining kernel needs about the item whose first piece a CTA holds (in slot 1).
struct PieceRec {
    int valid, tok0, tok, g, last_cta, pad[3];
};

struct ChunkParams {
    CUtensorMap tm_q, tm_k, tm_v;  // q: [total_q, Hq, D], boxes of `tt` tokens x G heads x 64
    CUtensorMap tm_o;              // out, boxes of `store_tok` tokens (0: no boxes)
    const int32_t *cu_q, *ctx, *block_tables;
    const void *k_cache, *v_cache;
    void *out;
    int32_t *err;
    float *pieces;
    PieceRec *recs;
    int S, Hq, Hkv, G;
    int tt;        // tokens of a row tile
    int item_tok;  // tokens of an item
    int store_tok;
    int max_blocks, num_blocks, total_q, max_seqlen_q, window, box_rows;
    uint32_t inv_g;  // 2^16 / G, rounded up: x inv_g >> 16 is x / G for x < 256
    BlockGeom geom;
    float scale_log2;
    __device__ __forceinline__ int div_g(int x) const { return static_cast<int>(x * inv_g >> 16); }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    const bool ok = mbar_wait(bar, parity) && !*abort_flag;
    const bool all = __all_sync(kFull, ok);
    __syncwarp();
    return all;
}
__device__ __forceinline__ void give_up(int32_t *err, volatile int *abort_flag) {
    raise_err(err, PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
}

// ------------------------------------------------------------------------------------------
// the shares
// ------------------------------------------------------------------------------------------

// A length or a table entry. The kernels are launched beside what precedes them, which may still write these: they are
// read after the wait, by plain loads (the read-only path asks for data that is constant from the kernel's start
// on, and its loads may be moved before the wait). Past L1, with __ldcg, they cost 0.4 us of a small draft's 8.2.
__device__ __forceinline__ int ld_index(const int32_t *p) { return *p; }

struct SeqShape {
    int q0, ql, kl;
    bool bad;  // lengths outside the contract: the rows are zero, no work
};
__device__ __forceinline__ SeqShape seq_shape(const ChunkParams &p, int s) {
    SeqShape r;
    r.q0 = ld_index(p.cu_q + s);
    const int q1 = ld_index(p.cu_q + s + 1);
    r.kl = ld_index(p.ctx + s);
    r.bad = r.q0 < 0 || q1 < r.q0 || q1 > p.total_q;
    r.ql = r.bad ? 0 : q1 - r.q0;
    if (r.ql > 0 && (r.ql > p.max_seqlen_q || r.kl < r.ql ||
                     static_cast<long long>(r.kl) > static_cast<long long>(p.max_blocks) * p.geom.block_size))
        r.bad = true;
    return r;
}
// key tiles of item i of a sequence
__device__ __forceinline__ int item_tiles(const ChunkParams &p, const SeqShape &q, int i) {
    const int t0 = i * p.item_tok, t1 = min(t0 + p.item_tok, q.ql), p0 = q.kl - q.ql;
    const int lo = p.window > 0 ? max(0, p0 + t0 - p.window + 1) : 0;
    return (p0 + t1 + BN - 1) / BN - lo / BN;
}
// key tiles of all the sequence's items of one kv head
__device__ __forceinline__ long long head_tiles(const ChunkParams &p, const SeqShape &q) {
    if (q.bad || q.ql <= 0) return 0;
    long long n = 0;
    for (int i = 0; i * p.item_tok < q.ql; ++i) n += item_tiles(p, q, i);
    return n;
}
__device__ __forceinline__ long long warp_sum(long long v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// A CTA's share [b0, b1) of the line of (item, key tile) pairs; N of them on P CTAs. Sequence s0, which
// starts at place base0 of the line, holds b0.
struct Share {
    long long N, P, b0, b1, base0;
    int s0;
};

// Every thread of the block calls this; sm: 12 words of shared memory, the result is in *out after the
// next __syncthreads (in shared memory too: only the scheduler reads it).
__device__ __forceinline__ void plan_share(const ChunkParams &p, long long *sm, Share *out) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kW = kThreads / 32;
    // the sum over the block so far, and the sum before this thread, of one value a thread
    auto scan = [&](long long v, long long &before) {
        long long incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) sm[warp] = incl;
        __syncthreads();
        long long total = 0;
        before = incl - v;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w < warp) before += sm[w];
            total += sm[w];
        }
        return total;
    };
    auto tiles_of = [&](int s) { return s < p.S ? head_tiles(p, seq_shape(p, s)) * p.Hkv : 0; };
    Share r;
    long long v = tiles_of(tid), before;
    r.N = scan(v, before);
    const long long first = r.N;  // of the first kThreads sequences
    if (p.S > kThreads) {
        long long more = 0, unused;
        for (int s = tid + kThreads; s < p.S; s += kThreads) more += tiles_of(s);
        r.N += scan(more, unused);
    }
    // CTAs 0 .. P - 1 take a share, at least one tile each (no piece of an item is then empty)
    r.P = min(static_cast<long long>(gridDim.x), r.N);
    const long long me = blockIdx.x;
    r.b0 = r.b1 = r.N;
    if (me < r.P) {
        if (r.N <= 0xffffffffll / gridDim.x) {  // 64-bit divisions cost some hundred cycles
            const uint32_t n = static_cast<uint32_t>(r.N), c = static_cast<uint32_t>(r.P), i = blockIdx.x;
            r.b0 = i * n / c;
            r.b1 = (i + 1) * n / c;
        } else {
            r.b0 = me * r.N / r.P;
            r.b1 = (me + 1) * r.N / r.P;
        }
    }
    if (r.b0 < r.b1) {
        long long base = 0, total = first;
        for (int sb = 0;; sb += kThreads) {
            if (sb > 0) {
                v = tiles_of(sb + tid);
                total = scan(v, before);
            }
            if (base + before <= r.b0 && r.b0 < base + before + v) {  // one thread of the block, once
                out->s0 = sb + tid;
                out->base0 = base + before;
            }
            base += total;
            if (r.b0 < base) break;  // the same for every thread
        }
    }
    if (tid == 0) out->N = r.N, out->P = r.P, out->b0 = r.b0, out->b1 = r.b1;
}

// Sequences whose lengths are outside the contract: an error bit and zero rows.
template <class T, int HD>
__device__ __forceinline__ void zero_bad_sequences(const ChunkParams &p) {
    T *out = static_cast<T *>(p.out);
    for (int s = blockIdx.x; s < p.S; s += gridDim.x) {
        const SeqShape q = seq_shape(p, s);
        if (!q.bad) continue;
        if (threadIdx.x == 0) raise_err(p.err, PA_DEVERR_LENGTH);
        const int a = max(q.q0, 0), b = min(ld_index(p.cu_q + s + 1), p.total_q);
        for (long long i = static_cast<long long>(a) * p.Hq * HD + threadIdx.x; i < static_cast<long long>(b) * p.Hq * HD;
             i += kThreads)
            out[i] = T(0.f);
    }
}

// One warp walks the CTA's share and hands each of its segments to publish (false: stop); the record
// of an item that starts in this share and ends in another's goes to the joining kernel.
template <class F>
__device__ __forceinline__ bool walk_share(const ChunkParams &p, const Share sh, F publish) {
    const int lane = threadIdx.x & 31;
    int s = sh.s0;
    long long at = sh.b0, off = sh.b0 - sh.base0;  // places on the line, and in the sequence
    while (at < sh.b1) {
        const SeqShape q = seq_shape(p, s);
        const long long per_head = head_tiles(p, q);
        // order within a sequence: kv head, then item: a CTA's next item reads the same keys
        int g = per_head > 0 ? 0 : p.Hkv;
        while (off > 0 && off >= per_head) off -= per_head, ++g;
        long long in_head = off;
        int i = 0;
        if (g < p.Hkv)
            for (int n; in_head >= (n = item_tiles(p, q, i)); ++i) in_head -= n;
        for (; g < p.Hkv && at < sh.b1; ++g, i = 0)
            for (; i * p.item_tok < q.ql && at < sh.b1; ++i) {
                const int n = item_tiles(p, q, i), t0 = i * p.item_tok;
                const int first = static_cast<int>(in_head);
                const int last = static_cast<int>(min(static_cast<long long>(n), first + (sh.b1 - at)));
                in_head = 0;
                SegInfo it;
                it.s = s, it.g = g, it.tok0 = q.q0 + t0, it.tok = min(p.item_tok, q.ql - t0);
                it.p0 = q.kl - q.ql + t0;
                it.n_end = it.p0 + it.tok;
                it.n_lo = p.window > 0 ? max(0, it.p0 - p.window + 1) : 0;
                it.j0 = it.n_lo / BN + first, it.j1 = it.n_lo / BN + last;
                it.part = first > 0 ? 0 : last < n ? 1 : -1;
                if (!publish(it)) return false;
                if (it.part == 1 && lane == 0) {
                    // the CTA that holds the item's last tile: share c is [c N / P, (c + 1) N / P)
                    PieceRec r{};
                    const long long x = at + n - 1;
                    r.valid = 1, r.tok0 = it.tok0, r.tok = it.tok, r.g = g;
                    r.last_cta = static_cast<int>(((x + 1) * sh.P - 1) / sh.N);
                    p.recs[blockIdx.x] = r;
                }
                at += last - first;
            }
        ++s;
        off = 0;
    }
    return publish(SegInfo{});  // the end marker
}

// The pool row of key `pos` of the segment's sequence, the first of a box that ends at `last`; -1 where
// the box is not to be read (behind the keys, or before the first). A bad table entry marks the segment.
__device__ __forceinline__ long long pool_row(const ChunkParams &p, const SegInfo &it, int pos, int last,
                                              volatile int *bad_seg, int seg_no) {
    if (pos >= it.n_end || last < it.n_lo) return -1;
    const int id = ld_index(p.block_tables + static_cast<size_t>(it.s) * p.max_blocks + p.geom.block_of(pos));
    if (id < 0 || id >= p.num_blocks) {
        bad_seg[seg_no & (kBadRing - 1)] = seg_no + 1;
        raise_err(p.err, PA_DEVERR_TABLE);
        return -1;
    }
    return static_cast<long long>(id) * p.geom.block_size + p.geom.offset_of(pos);
}

// the 128 rows of a K or V tile of kv head g, one by one, into the swizzled layout that TMA writes; rows
// r[i] = pool row of lane + 32 i, or -1 (zeros)
template <class T, int HD>
__device__ __forceinline__ void gather_tile(uint32_t dst, const T *pool, const long long (&r)[BN / 32], int Hkv, int g) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) {
        const int k = lane + 32 * i;
        const T *src = pool + (static_cast<size_t>(r[i] < 0 ? 0 : r[i]) * Hkv + g) * HD;
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
            cp_async16(dst + (c >> 3) * kHalf + k * 128 + (((c & 7) ^ (k & 7)) << 4), src + c * 8, r[i] < 0 ? 0 : 16);
    }
    cp_async_commit();
}

// Rows of a V tile outside [z0, z1) (unwritten slots, blocks given back, an earlier tile's) are zeroed by
// one warp before the PV product reads them: P is zero there, but 0 * NaN is not.
template <int HD>
__device__ __forceinline__ void zero_rows(unsigned char *tile, int z0, int z1) {
    constexpr int kRows = 32 / (HD / 8);  // rows that the warp writes at a time, 16 bytes a lane
    const int lane = threadIdx.x & 31, c16 = lane % (HD / 8), r0 = lane / (HD / 8);
    unsigned char *at = tile + (c16 >> 3) * kHalf + (c16 & 7) * 16;
#pragma unroll 4
    for (int r = r0; r < z0; r += kRows) *reinterpret_cast<uint4 *>(at + r * 128) = make_uint4(0, 0, 0, 0);
#pragma unroll 4
    for (int r = z1 + r0; r < BN; r += kRows) *reinterpret_cast<uint4 *>(at + r * 128) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace chunk

// chunk_attn_narrow.cu: items of at most 64 query rows
cudaError_t launch_chunk_narrow(const chunk::ChunkParams &prm, pa_dtype dtype, int D, bool gather, cudaStream_t stream);

}  // namespace pa
