// chunk_narrow.cuh: what the kernels of few query rows share (chunk_attn_narrow.cu, chunk_attn_q8.cu): reads of tensor memory,
// reductions of columns over a warp's lanes, and the kernel that joins the pieces of an item.
#pragma once

#include "chunk_common.cuh"

namespace pa {
namespace chunk {

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

// A piece of an item of `columns` query rows in the workspace: m[columns], l[columns], O[columns][hd]
__host__ __device__ constexpr size_t piece_floats(int columns, int hd) { return static_cast<size_t>(columns) * (hd + 2); }

// ------------------------------------------------------------------------------------------
// joining the pieces
// ------------------------------------------------------------------------------------------

constexpr int kJoinWork = 64, kJoinGroups = 4;  // outputs of four columns of a block; the pieces are dealt out to groups

// Block (c, y): outputs [64 y, 64 y + 64) of four columns each of the item whose first piece CTA c holds (its slot
// 1); the pieces after it are slot 0 of the CTAs up to last_cta. An item of a long sequence has tens of
// pieces: four groups of threads read four pieces each at a time (a thread for all 25 pieces of
// one, one after the other, took 41 us; so 4 us).
template <class E, int HD, int kNC>
__global__ void __launch_bounds__(kJoinWork * kJoinGroups) chunk_narrow_join_kernel(const __grid_constant__ ChunkParams p) {
    constexpr size_t kPieceFloats = piece_floats(kNC, HD);
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
                    const float *src = p.pieces + (static_cast<size_t>(c) * 2 + (c == first)) * kPieceFloats;
                    pm[k] = __ldcg(src + row);  // written by the kernel this one was launched beside: not the read-only path
                    pl[k] = __ldcg(src + kNC + row);
                    po[k] = __ldcg(reinterpret_cast<const float4 *>(src + 2 * kNC + row * HD + col));
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

}  // namespace chunk
}  // namespace pa
