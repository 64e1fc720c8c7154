// norm_rope_store_kv.cu: norms of a step's queries and keys for each head, their rotation, and the append of keys and
// values to the paged cache, in the storage type or in 8 bits (pa_norm_rope_store_kv).
//
// Source: as rope_store_kv.cu; the norms are those of the engines' Qwen3 models (smzdm nano-vLLM deep dive,
// "模型实现细节").
//
// The mathematics: a head row x of D elements becomes y = x / sqrt(mean x^2 + eps) * w (queries and keys, where a weight
// is given), then the rotation of rope_store_kv.cu; everything in fp32, rounded once to the storage type. An 8-bit
// cache row is y / s rounded once to e4m3, s = max(max |y| / 448, 2^-90), held in fp32 for each slot and kv head.
//
// Bound by HBM: q, k, v are read once, q_out and the pools written once. A row's sum of squares (and its largest
// magnitude, for the 8-bit cache) lies across threads: a row belongs to L lanes of a warp, a power of two, 16 elements a
// lane, so that two or three shuffles reduce it and the row itself never leaves the registers. As in the
// rotation without norms, a thread takes the same elements of several rows of its token, whose cosines and sines
// it loads once. The weights come from L1.
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormRotUnits = 16;  // rot_dim <= 256

struct NormRopeParams {
    const unsigned char *q, *k, *v;  // token strides below, in bytes
    unsigned char *q_out, *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const unsigned char *q_weight, *k_weight;
    long long q_stride, k_stride, v_stride, qo_stride;
    const int32_t *slot_mapping, *positions;
    const float *cos_sin;
    int32_t *err;
    long long num_slots;
    BlockGeom geom;
    int T, Hq, Hkv, D, rot, n_axes, max_pos, units, lanes, row_par;
    float inv_d, eps;
    uint32_t axis[kNormRotUnits];  // four bits per pair: the axis of each of a unit's eight pairs
};

// 16-byte load that may alias q_out (the in-place form), so not through the read-only path
__device__ __forceinline__ uint4 ld_row(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <class E>
__device__ __forceinline__ float squares(const uint4 &x, float sum) {
    float f[8];
    unpack8<E>(x, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
    return sum;
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float *f) {
    return make_uint4(E::pack2(f[0], f[1]), E::pack2(f[2], f[3]), E::pack2(f[4], f[5]), E::pack2(f[6], f[7]));
}
// eight quotients f / s, each correctly rounded, then rounded to e4m3 (nearest even, beyond 448: 448, NaN stays NaN)
__device__ __forceinline__ uint2 quantise8(const float *f, float s) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(__fdiv_rn(f[2 * e + 1], s)), "f"(__fdiv_rn(f[2 * e], s)));
        w[e] = two;
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// kRows head rows per thread, loaded together before any is stored.
template <class E, int kRows, bool kPairs, bool kQ8>
__global__ void __launch_bounds__(kNormThreads) norm_rope_store_kv_kernel(const __grid_constant__ NormRopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;");  // the attention's set-up may run beside this grid
    const int per_token = p.lanes * p.row_par;
    const long long idx = static_cast<long long>(blockIdx.x) * kNormThreads + threadIdx.x;
    const int t = static_cast<int>(idx / per_token);
    const int in_token = static_cast<int>(idx - static_cast<long long>(t) * per_token);
    const int row0 = in_token / p.lanes, u = in_token & (p.lanes - 1);
    // Every lane stays for the shuffles; those of a token that is not there, padding or refused load and store nothing.
    bool live = t < p.T;
    const long long slot = live ? __ldg(p.slot_mapping + t) : -1;
    live = slot >= 0;
    int pos[4] = {0, 0, 0, 0};  // of each axis; those that are not there hold the first's
    bool bad_pos = false;
    if (p.rot > 0 && live) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            pos[a] = a == 0 || a < p.n_axes ? __ldg(p.positions + static_cast<size_t>(a) * p.T + t) : pos[0];
            bad_pos |= static_cast<unsigned>(pos[a]) >= static_cast<unsigned>(p.max_pos);
        }
    }
    if (live && (slot >= p.num_slots || bad_pos)) {
        if (in_token == 0)
            raise_err(p.err, (slot >= p.num_slots ? PA_DEVERR_SLOT : 0) | (bad_pos ? PA_DEVERR_POSITION : 0));
        live = false;
    }
    live = live && u < p.units;
    const int n8 = p.rot / 16;  // units that hold rotated pairs
    const int rows = p.Hq + 2 * p.Hkv;
    // The unit's two chunks of 8 elements in a head row of q or k, and of v. The last unit of a row may have one only.
    int e0, e1;
    if (u < n8) {
        e0 = kPairs ? u * 16 : u * 8;
        e1 = kPairs ? u * 16 + 8 : p.rot / 2 + u * 8;
    } else {
        e0 = p.rot + (u - n8) * 16;
        e1 = e0 + 8;
    }
    const int v0 = u * 16, v1 = v0 + 8;

    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = row0 + i * p.row_par;
        x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
        if (!live || r >= rows) continue;
        const bool is_v = r >= p.Hq + p.Hkv;
        const unsigned char *src = r < p.Hq ? p.q + t * p.q_stride + static_cast<size_t>(r) * p.D * 2
                                   : is_v   ? p.v + t * p.v_stride + static_cast<size_t>(r - p.Hq - p.Hkv) * p.D * 2
                                            : p.k + t * p.k_stride + static_cast<size_t>(r - p.Hq) * p.D * 2;
        const int a = is_v ? v0 : e0, b = is_v ? v1 : e1;
        if (a < p.D) x0[i] = ld_row(src + a * 2);
        if (b < p.D) x1[i] = ld_row(src + b * 2);
    }
    float c[8], s[8];
    if (live && u < n8 && row0 < p.Hq + p.Hkv) {
        const uint32_t axes = p.axis[u];
        const int half = p.rot / 2;
        const auto pos_of = [&](uint32_t a) { return a & 2u ? a & 1u ? pos[3] : pos[2] : a & 1u ? pos[1] : pos[0]; };
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
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
    }
    // the rows' sums of squares, all rows side by side
    float rstd[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) rstd[i] = squares<E>(x1[i], squares<E>(x0[i], 0.f));
    for (int o = 1; o < p.lanes; o <<= 1)
#pragma unroll
        for (int i = 0; i < kRows; ++i) rstd[i] += __shfl_xor_sync(0xffffffffu, rstd[i], o);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = row0 + i * p.row_par;
        const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv, there = live && r < rows;
        const int a = is_v ? v0 : e0, b = is_v ? v1 : e1;
        float f[16];
        unpack8<E>(x0[i], *reinterpret_cast<float(*)[8]>(f));
        unpack8<E>(x1[i], *reinterpret_cast<float(*)[8]>(f + 8));
        const unsigned char *w = is_q ? p.q_weight : is_v ? nullptr : p.k_weight;
        if (w && there) {
            const float m = rsqrtf(fmaf(rstd[i], p.inv_d, p.eps));
            float g[8];
            unpack8<E>(a < p.D ? __ldg(reinterpret_cast<const uint4 *>(w + a * 2)) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * m * g[e];
            unpack8<E>(b < p.D ? __ldg(reinterpret_cast<const uint4 *>(w + b * 2)) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[8 + e] = f[8 + e] * m * g[e];
        }
        if (!is_v && u < n8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &y0 = kPairs ? f[2 * e] : f[e], &y1 = kPairs ? f[2 * e + 1] : f[8 + e];
                const float z0 = y0 * c[e] - y1 * s[e], z1 = y1 * c[e] + y0 * s[e];
                y0 = z0, y1 = z1;
            }
        }
        if (!kQ8 || is_q) {
            if (there) {
                unsigned char *dst = is_q   ? p.q_out + t * p.qo_stride + static_cast<size_t>(r) * p.D * 2
                                     : is_v ? p.v_cache + (static_cast<size_t>(slot) * p.Hkv + (r - p.Hq - p.Hkv)) * p.D * 2
                                            : p.k_cache + (static_cast<size_t>(slot) * p.Hkv + (r - p.Hq)) * p.D * 2;
                if (a < p.D) stg128(dst + a * 2, is_v ? x0[i] : pack8<E>(f));  // values are bit copies
                if (b < p.D) stg128(dst + b * 2, is_v ? x1[i] : pack8<E>(f + 8));
            }
        }
        if constexpr (kQ8) {
            // magnitudes as whole numbers, so that a NaN is the largest
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) most = max(most, __float_as_uint(f[e]) & 0x7fffffffu);
            for (int o = 1; o < p.lanes; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            float scale = __fdiv_rn(__uint_as_float(most), 448.f);
            if (scale < 0x1p-90f) scale = 0x1p-90f;
            if (there && !is_q) {
                const int g = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
                unsigned char *dst = (is_v ? p.v_cache : p.k_cache) + (static_cast<size_t>(slot) * p.Hkv + g) * p.D;
                if (a < p.D) *reinterpret_cast<uint2 *>(dst + a) = quantise8(f, scale);
                if (b < p.D) *reinterpret_cast<uint2 *>(dst + b) = quantise8(f + 8, scale);
                const int s32 = static_cast<int>(slot), block = p.geom.block_of(s32);
                if (u == 0)
                    (is_v ? p.v_scale : p.k_scale)[(static_cast<size_t>(block) * p.Hkv + g) * p.geom.block_size +
                                                   p.geom.offset_of(s32)] = scale;
            }
        }
    }
}

template <class E, int kRows, bool kQ8>
cudaError_t launch_norm_typed(const NormRopeParams &prm, bool pairs, unsigned grid, cudaStream_t stream) {
    if (pairs)
        norm_rope_store_kv_kernel<E, kRows, true, kQ8><<<grid, kNormThreads, 0, stream>>>(prm);
    else
        norm_rope_store_kv_kernel<E, kRows, false, kQ8><<<grid, kNormThreads, 0, stream>>>(prm);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope_store_kv(const NormRopeStoreArgs &n, cudaStream_t stream) {
    const RopeStoreArgs &a = n.rows;
    NormRopeParams prm{};
    prm.q = static_cast<const unsigned char *>(a.q);
    prm.k = static_cast<const unsigned char *>(a.k);
    prm.v = static_cast<const unsigned char *>(a.v);
    prm.q_out = static_cast<unsigned char *>(a.q_out);
    prm.k_cache = static_cast<unsigned char *>(a.k_cache);
    prm.v_cache = static_cast<unsigned char *>(a.v_cache);
    prm.k_scale = n.k_scale, prm.v_scale = n.v_scale;
    prm.q_weight = static_cast<const unsigned char *>(n.q_weight);
    prm.k_weight = static_cast<const unsigned char *>(n.k_weight);
    prm.q_stride = a.q_stride * 2;
    prm.k_stride = a.k_stride * 2;
    prm.v_stride = a.v_stride * 2;
    prm.qo_stride = a.q_out_stride * 2;
    prm.slot_mapping = a.slot_mapping;
    prm.positions = a.positions;
    prm.cos_sin = a.cos_sin;
    prm.err = a.err;
    prm.num_slots = static_cast<long long>(a.num_blocks) * a.block_size;
    prm.geom.block_size = a.block_size;
    prm.geom.shift = log2_if_pow2(a.block_size);
    prm.T = a.T, prm.Hq = a.Hq, prm.Hkv = a.Hkv, prm.D = a.D, prm.rot = a.rot_dim;
    prm.n_axes = a.n_axes, prm.max_pos = a.max_pos;
    prm.inv_d = 1.f / a.D, prm.eps = n.eps;
    // a row's rotated units, then its other chunks in pairs; v rows, all chunks in pairs, never need more
    prm.units = a.rot_dim / 16 + (a.D - a.rot_dim + 15) / 16;
    for (prm.lanes = 1; prm.lanes < prm.units;) prm.lanes *= 2;
    for (int i = 0; a.pair_axis && i < a.rot_dim / 2; ++i)
        prm.axis[i / 8] |= static_cast<uint32_t>(a.pair_axis[i]) << (4 * (i % 8));
    const int rows = a.Hq + 2 * a.Hkv;
    const long long all = static_cast<long long>(a.T) * prm.lanes * rows;
    const int each = all > static_cast<long long>(device_sm_count()) * 2048 ? 4 : 1;
    prm.row_par = (rows + each - 1) / each;
    const long long threads = static_cast<long long>(a.T) * prm.lanes * prm.row_par;
    const unsigned grid = static_cast<unsigned>((threads + kNormThreads - 1) / kNormThreads);
    auto go = [&](auto e) {
        using E = decltype(e);
        if (n.q8)
            return each == 4 ? launch_norm_typed<E, 4, true>(prm, a.interleaved, grid, stream)
                             : launch_norm_typed<E, 1, true>(prm, a.interleaved, grid, stream);
        return each == 4 ? launch_norm_typed<E, 4, false>(prm, a.interleaved, grid, stream)
                         : launch_norm_typed<E, 1, false>(prm, a.interleaved, grid, stream);
    };
    return a.dtype == PA_BF16 ? go(BF16{}) : go(F16{});
}

}  // namespace pa
