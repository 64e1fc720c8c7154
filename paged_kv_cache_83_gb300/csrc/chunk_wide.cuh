// chunk_wide.cuh: what the kernels of 128-row query tiles share (chunk_attn.cu, chunk_attn_q8_wide.cu): the layout of an item's
// pieces, and the kernel that joins them.
#pragma once

#include "chunk_common.cuh"

namespace pa {
namespace chunk {

// A piece of an item of two row tiles in the workspace: m[256], l[256], O[hd][256], fp32 (rows fastest: lanes = rows)
__host__ __device__ constexpr size_t wide_piece_floats(int hd) { return static_cast<size_t>(256) * (hd + 2); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// ------------------------------------------------------------------------------------------
// joining the pieces
// ------------------------------------------------------------------------------------------

constexpr int kJoinRows = 32, kJoinCols = 32;  // of a block: threads = rows x 4 chunks of 8 columns
constexpr int kJoinThreads = kJoinRows * (kJoinCols / 8);

// Block (c, y, z): rows [32 y, 32 y + 32) and columns [32 z, 32 z + 32) of the item whose first piece CTA c
// holds (its slot 1); the pieces after it are slot 0 of the CTAs up to last_cta. The reads run along
// the rows, with four pieces' in flight: what bounds it is their latency.
template <class E, int HD>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    // the next call's kernel may set itself up beside this one: it waits for this grid itself
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PieceRec rec = p.recs[blockIdx.x];
    if (!rec.valid) return;
    const int rt = p.tt * p.G;  // rows of a full row tile
    // row r of the item: tile r / 128, row r % 128 of it
    const int r = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, col = blockIdx.z * kJoinCols + threadIdx.x / kJoinRows * 8;
    const int h = r >> 7, rr = r & 127;
    if (rr >= rt || h * p.tt + rr / p.G >= rec.tok) return;
    const int first = blockIdx.x;
    float m = -INFINITY, l = 0.f, o[8] = {};
    bool bad = false;
    for (int c0 = first; c0 <= rec.last_cta; c0 += 4) {
        float pm[4], pl[4], po[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = c0 + k;
            pm[k] = -INFINITY, pl[k] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) po[k][e] = 0.f;
            if (c <= rec.last_cta) {
                const float *w = p.pieces + (static_cast<size_t>(c) * 2 + (c == first)) * wide_piece_floats(HD) + r;
                pm[k] = __ldcg(w);  // written by the kernel this one was launched beside: not the read-only path
                pl[k] = __ldcg(w + 256);
#pragma unroll
                for (int e = 0; e < 8; ++e) po[k][e] = __ldcg(w + 512 + (col + e) * 256);
            }
        }
        const float mn = fmaxf(m, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
        const float mu = mn == -INFINITY ? 0.f : mn, f0 = fast_exp2(m - mu);
        l *= f0;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = fast_exp2(pm[k] - mu);
            bad |= pl[k] == -1.f;
            l += f * pl[k];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += f * po[k][e];
        }
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint4 u;
    u.x = E::pack2(o[0] * inv, o[1] * inv);
    u.y = E::pack2(o[2] * inv, o[3] * inv);
    u.z = E::pack2(o[4] * inv, o[5] * inv);
    u.w = E::pack2(o[6] * inv, o[7] * inv);
    if (bad) u = make_uint4(0, 0, 0, 0);
    using T = typename E::T;
    const int tk = rec.tok0 + h * p.tt + rr / p.G, head = rec.g * p.G + rr % p.G;
    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (static_cast<size_t>(tk) * p.Hq + head) * HD + col) = u;
}

}  // namespace chunk
}  // namespace pa
