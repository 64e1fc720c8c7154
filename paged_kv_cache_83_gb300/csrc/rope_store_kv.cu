// rope_store_kv.cu: position rotation of a step's queries and keys, with the keys and values
// appended to the paged cache on the way (pa_rope_store_kv).
//
// Source: "nano-vLLM Part 4", section 3 (K/V written for every new token through the slot mapping);
// smzdm nano-vLLM deep dive, "模型实现细节" (the attention layer's store before attention). The
// rotation is the one of the engines' Qwen models, generalised to positions with several axes.
//
// The mathematics: pair i of a head row (x0, x1) becomes (x0 cos - x1 sin, x1 cos + x0 sin) with the
// cosine and sine that the caller's table holds for the position of the pair's axis; products and
// sums in fp32, one rounding to the storage type. Values and unrotated elements are bit copies.
//
// Bound by HBM: q, k, v are read once, q_out and the pools written once
// (T * D * 2 * (2 Hq + 4 Hkv) bytes); the table rows of a step come from L2. So a thread owns one
// unit of 16 elements (8 pairs) of a token and walks over the token's head rows with the unit's
// eight cosines and sines in registers: the table is read once per thread, not once per head, and
// every access to the big tensors is 16 bytes wide. 33,673 tokens of 16/8 heads x 128 (556 MB): 90 us, 0.91
// of the copy bandwidth (a plain copy of as many bytes, alternating buffers like this: 85 us).
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 4;     // on an SM: 64 registers a thread (33,673 tokens: 90 us, at 94 registers 116, at 80 94)
constexpr int kRopeMaxUnits = 16;  // rot_dim <= 256

struct RopeParams {
    const unsigned char *q, *k, *v;  // token strides below, in bytes
    unsigned char *q_out, *k_cache, *v_cache;
    long long q_stride, k_stride, v_stride, qo_stride;
    const int32_t *slot_mapping, *positions;
    const float *cos_sin;
    int32_t *err;
    long long num_slots;
    int T, Hq, Hkv, D, rot, n_axes, max_pos, units, row_par;
    uint32_t axis[kRopeMaxUnits];  // four bits per pair: the axis of each of a unit's eight pairs
};

// 16-byte load that may alias q_out (the in-place form), so not through the read-only path
__device__ __forceinline__ uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// two packed words of elements (x0 in a, x1 in b), two pairs, rotated in place
template <class E>
__device__ __forceinline__ void rotate_word(uint32_t &a, uint32_t &b, float c0, float s0, float c1, float s1) {
    const float2 x = E::unpack2(a), y = E::unpack2(b);
    a = E::pack2(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
    b = E::pack2(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
}
// one packed word holding a pair (x0, x1)
template <class E>
__device__ __forceinline__ void rotate_pair(uint32_t &w, float c, float s) {
    const float2 x = E::unpack2(w);
    w = E::pack2(x.x * c - x.y * s, x.y * c + x.x * s);
}

// kRows head rows per thread, loaded together before any is stored.
template <class E, int kRows, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_store_kv_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;");  // the attention's set-up may run beside this grid
    const int per_token = p.units * p.row_par;
    const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
    const int t = static_cast<int>(idx / per_token);
    if (t >= p.T) return;
    const int in_token = static_cast<int>(idx - static_cast<long long>(t) * per_token);
    const int row0 = in_token / p.units, u = in_token - row0 * p.units;
    const long long slot = __ldg(p.slot_mapping + t);
    if (slot < 0) return;  // padding: nothing of this token is read or written
    bool bad_pos = false;
    // The positions of the token's axes stay in registers for the table rows (9001 tokens on three axes: 13.2 -> 11.9
    // us), where registers are left: with four rows a thread they spill (33,673 tokens: 90 -> 93 us).
    constexpr bool kHold = kRows < 4;
    const auto load_pos = [&](uint32_t a) { return __ldg(p.positions + static_cast<size_t>(a) * p.T + t); };
    int pos[4];  // of each axis; those that are not there hold the first's
    if constexpr (kHold) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            pos[a] = a == 0 || a < p.n_axes ? load_pos(a) : pos[0];
            bad_pos |= static_cast<unsigned>(pos[a]) >= static_cast<unsigned>(p.max_pos);
        }
    } else {
        for (int a = 0; a < p.n_axes; ++a)
            bad_pos |= static_cast<unsigned>(load_pos(a)) >= static_cast<unsigned>(p.max_pos);
    }
    const auto pos_of = [&](uint32_t a) {  // a < 4
        if constexpr (kHold)
            return a & 2u ? a & 1u ? pos[3] : pos[2] : a & 1u ? pos[1] : pos[0];
        else
            return load_pos(a);
    };
    if (slot >= p.num_slots || bad_pos) {
        if (in_token == 0)
            raise_err(p.err, (slot >= p.num_slots ? PA_DEVERR_SLOT : 0) | (bad_pos ? PA_DEVERR_POSITION : 0));
        return;
    }
    const int n8 = p.rot / 16;  // units that hold rotated pairs
    const int rows = p.Hq + 2 * p.Hkv;
    const size_t row_bytes = static_cast<size_t>(p.D) * 2;
    // byte offsets of the unit's two 16-byte chunks in a head row of q or k, and of v (a bit copy).
    // The last unit of a row may have one chunk only.
    int o0, o1;
    if (u < n8) {
        o0 = kPairs ? u * 32 : u * 16;
        o1 = kPairs ? u * 32 + 16 : p.rot + u * 16;  // the second half starts rot / 2 elements in
    } else {
        o0 = p.rot * 2 + (u - n8) * 32;
        o1 = o0 + 16;
    }
    const int vo0 = u * 32, vo1 = vo0 + 16;

    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = row0 + i * p.row_par;
        if (r >= rows) continue;
        const bool is_v = r >= p.Hq + p.Hkv;
        const unsigned char *src = r < p.Hq ? p.q + t * p.q_stride + r * row_bytes
                                   : is_v   ? p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * row_bytes
                                            : p.k + t * p.k_stride + (r - p.Hq) * row_bytes;
        const int a = is_v ? vo0 : o0, b = is_v ? vo1 : o1;
        if (a < static_cast<int>(row_bytes)) x0[i] = ld_stream(src + a);
        if (b < static_cast<int>(row_bytes)) x1[i] = ld_stream(src + b);
    }
    float c[8], s[8];
    if (u < n8 && row0 < p.Hq + p.Hkv) {
        const uint32_t axes = p.axis[u];
        const int half = p.rot / 2;
        if (axes == (axes & 15u) * 0x11111111u) {
            // one position for the unit: four 16-byte loads
            const float4 *row =
                reinterpret_cast<const float4 *>(p.cos_sin + static_cast<size_t>(pos_of(axes & 3u)) * p.rot + u * 8);
            const float4 *srow = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row) + half);
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(srow), s1 = __ldg(srow + 1);
            c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
            s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float *row = p.cos_sin + static_cast<size_t>(pos_of((axes >> (4 * e)) & 3u)) * p.rot + u * 8 + e;
                c[e] = __ldg(row);
                s[e] = __ldg(row + half);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = row0 + i * p.row_par;
        if (r >= rows) continue;
        const bool is_v = r >= p.Hq + p.Hkv;
        if (!is_v && u < n8) {
            if constexpr (kPairs) {
                rotate_pair<E>(x0[i].x, c[0], s[0]);
                rotate_pair<E>(x0[i].y, c[1], s[1]);
                rotate_pair<E>(x0[i].z, c[2], s[2]);
                rotate_pair<E>(x0[i].w, c[3], s[3]);
                rotate_pair<E>(x1[i].x, c[4], s[4]);
                rotate_pair<E>(x1[i].y, c[5], s[5]);
                rotate_pair<E>(x1[i].z, c[6], s[6]);
                rotate_pair<E>(x1[i].w, c[7], s[7]);
            } else {
                rotate_word<E>(x0[i].x, x1[i].x, c[0], s[0], c[1], s[1]);
                rotate_word<E>(x0[i].y, x1[i].y, c[2], s[2], c[3], s[3]);
                rotate_word<E>(x0[i].z, x1[i].z, c[4], s[4], c[5], s[5]);
                rotate_word<E>(x0[i].w, x1[i].w, c[6], s[6], c[7], s[7]);
            }
        }
        unsigned char *dst =
            r < p.Hq ? p.q_out + t * p.qo_stride + r * row_bytes
            : is_v   ? p.v_cache + (static_cast<size_t>(slot) * p.Hkv + (r - p.Hq - p.Hkv)) * row_bytes
                     : p.k_cache + (static_cast<size_t>(slot) * p.Hkv + (r - p.Hq)) * row_bytes;
        const int a = is_v ? vo0 : o0, b = is_v ? vo1 : o1;
        if (a < static_cast<int>(row_bytes)) stg128(dst + a, x0[i]);
        if (b < static_cast<int>(row_bytes)) stg128(dst + b, x1[i]);
    }
}

template <class E, int kRows>
cudaError_t launch_rope_typed(const RopeParams &prm, bool pairs, unsigned grid, cudaStream_t stream) {
    if (pairs)
        rope_store_kv_kernel<E, kRows, true><<<grid, kRopeThreads, 0, stream>>>(prm);
    else
        rope_store_kv_kernel<E, kRows, false><<<grid, kRopeThreads, 0, stream>>>(prm);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_store_kv(const RopeStoreArgs &a, cudaStream_t stream) {
    RopeParams prm{};
    prm.q = static_cast<const unsigned char *>(a.q);
    prm.k = static_cast<const unsigned char *>(a.k);
    prm.v = static_cast<const unsigned char *>(a.v);
    prm.q_out = static_cast<unsigned char *>(a.q_out);
    prm.k_cache = static_cast<unsigned char *>(a.k_cache);
    prm.v_cache = static_cast<unsigned char *>(a.v_cache);
    prm.q_stride = a.q_stride * 2;
    prm.k_stride = a.k_stride * 2;
    prm.v_stride = a.v_stride * 2;
    prm.qo_stride = a.q_out_stride * 2;
    prm.slot_mapping = a.slot_mapping;
    prm.positions = a.positions;
    prm.cos_sin = a.cos_sin;
    prm.err = a.err;
    prm.num_slots = static_cast<long long>(a.num_blocks) * a.block_size;
    prm.T = a.T, prm.Hq = a.Hq, prm.Hkv = a.Hkv, prm.D = a.D, prm.rot = a.rot_dim;
    prm.n_axes = a.n_axes, prm.max_pos = a.max_pos;
    // a row's rotated units, then its other chunks in pairs; v rows, all chunks in pairs, never need more
    prm.units = a.rot_dim / 16 + (a.D - a.rot_dim + 15) / 16;
    for (int i = 0; a.pair_axis && i < a.rot_dim / 2; ++i)
        prm.axis[i / 8] |= static_cast<uint32_t>(a.pair_axis[i]) << (4 * (i % 8));
    const int rows = a.Hq + 2 * a.Hkv;
    // One row a thread while the SMs hold all threads at once: the time is one chain of dependent loads, and more
    // threads shorten it (256 tokens of 16/8 heads x 128: 2.6 us, four rows 3.4; 600 tokens: 3.6 and 4.3). Beyond
    // that three or four rows, as leaves fewer of the last thread's without work (inputs and pools not in L2:
    // 800 tokens 5.2 us, one row 5.7; 1000: 6.0 and 6.9; 33,673: four rows 90, three 95, two 105. 9001 tokens of
    // 14/2 heads x 64, so 18 rows: three rows 13.2, four 14.9, two 14.4, one 19.1, before positions were held).
    const long long all = static_cast<long long>(a.T) * prm.units * rows;
    int each = 1;
    if (all > static_cast<long long>(device_sm_count()) * kRopeThreads * kRopeBlocks)
        each = (rows + 3) / 4 * 4 <= (rows + 2) / 3 * 3 ? 4 : 3;
    prm.row_par = (rows + each - 1) / each;
    const long long threads = static_cast<long long>(a.T) * prm.units * prm.row_par;
    const unsigned grid = static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads);
    auto go = [&](auto e) {
        using E = decltype(e);
        return each == 4   ? launch_rope_typed<E, 4>(prm, a.interleaved, grid, stream)
               : each == 3 ? launch_rope_typed<E, 3>(prm, a.interleaved, grid, stream)
                           : launch_rope_typed<E, 1>(prm, a.interleaved, grid, stream);
    };
    return a.dtype == PA_BF16 ? go(BF16{}) : go(F16{});
}

}  // namespace pa
