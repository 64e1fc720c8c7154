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
// it loads once. The weights come from L1. 33,673 tokens of 16/8 heads x 128 in bf16, into the 8-bit cache: 89 us, 0.84 of a copy
// (101 without a form for whole rows of 64 or 128 elements, 182 before a warp took a token, 16 elements a lane); 9001 tokens of
// 14/2 x 64 with three axes into the cache of the storage type: 12.3 us, 0.51, in 1.85 waves of blocks (64 registers a thread hold eight of
// them on an SM; the general forms spill 40 to 90 bytes there, those of whole rows none or 8 to 16); a step of 256 tokens 3.6 us, of 4
// tokens 3.2: the call's host side.
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kNormThreads = 128;
constexpr int kNormRotUnits = 16;  // rot_dim <= 256
constexpr int kAhead = 2;       // steps in flight
constexpr int kNormBlocks = 8;  // of an SM
constexpr int kFullWarps = 16;  // of an SM: tokens from which on a warp takes a whole one

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
    int T, Hq, Hkv, D, rot, n_axes, max_pos, units, lanes, lanes_log2;
    int qk_steps, steps, parts, part_steps;
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
__device__ __forceinline__ float max_nan3(float a, float b, float c) {  // NaN where one is NaN
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// eight numbers of a row in fp32, as four pairs
struct Eight {
    uint64_t p[4];
};
template <class E>
__device__ __forceinline__ Eight widen8(const uint4 &x) {
    return {{unpack_pair<E>(x.x), unpack_pair<E>(x.y), unpack_pair<E>(x.z), unpack_pair<E>(x.w)}};
}
template <class E>
__device__ __forceinline__ uint4 pack8(const Eight &f) {
    return make_uint4(E::pack2(f2_lo(f.p[0]), f2_hi(f.p[0])), E::pack2(f2_lo(f.p[1]), f2_hi(f.p[1])),
                      E::pack2(f2_lo(f.p[2]), f2_hi(f.p[2])), E::pack2(f2_lo(f.p[3]), f2_hi(f.p[3])));
}
__device__ __forceinline__ float largest(const Eight &f, float most) {
#pragma unroll
    for (int e = 0; e < 4; ++e) most = max_nan3(most, fabsf(f2_lo(f.p[e])), fabsf(f2_hi(f.p[e])));
    return most;
}
// f * inv, rounded to e4m3 (nearest even, beyond 448: 448, NaN stays NaN)
__device__ __forceinline__ uint2 quantise8(const Eight &f, float inv) {
    const uint64_t by = f2_pack(inv, inv);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t x = f2_mul(f.p[e], by);
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(f2_hi(x)), "f"(f2_lo(x)));
        w[e] = two;
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A warp takes a token, or a part of it. It goes over the token's rows 32 / lanes at a time (a step): first queries and keys
// side by side, then values. kAhead steps are loaded together before any is stored. kD: the head dim where whole rows of
// that many elements are rotated in halves, 0: any (33,673 tokens of 16/8 heads x 128 into 8 bits: 89 us, with the general form 101).
template <class E, bool kPairs, bool kQ8, int kD>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks) norm_rope_store_kv_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr bool kWhole = kD > 0;
    const int D = kWhole ? kD : p.D, rot = kWhole ? kD : p.rot, lanes = kWhole ? kD / 16 : p.lanes;
    const int lanes_log2 = kD == 64 ? 2 : kD == 128 ? 3 : p.lanes_log2;
    const int lane = threadIdx.x & 31;
    const unsigned warp = blockIdx.x * (kNormThreads / 32) + threadIdx.x / 32;
    const int t = static_cast<int>(warp / static_cast<unsigned>(p.parts)), part = static_cast<int>(warp) - t * p.parts;
    const int u = lane & (lanes - 1), row_of_lane = lane >> lanes_log2;
    const int n8 = rot / 16;  // units that hold rotated pairs
    const bool turns = kWhole || u < n8;
    const int n_qk = p.Hq + p.Hkv;
    // The unit's two chunks of 8 elements in a head row of q or k, and of v. The last unit of a row may have one only.
    const int e0 = turns ? kPairs ? u * 16 : u * 8 : rot + (u - n8) * 16;
    const int e1 = turns && !kPairs ? rot / 2 + u * 8 : e0 + 8;
    const bool there0 = kWhole || (u < p.units && e0 < D), there1 = kWhole || (u < p.units && e1 < D);
    const bool v_there0 = kWhole || u * 16 < D, v_there1 = kWhole || u * 16 + 8 < D;
    // launched beside what precedes it in the stream, whose results are read and written from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");  // the attention's set-up may run beside this grid
    if (t >= p.T) return;
    // slot and positions side by side; the axes that are not there hold the first's position
    const int slot = *(p.slot_mapping + t);
    int pos[4] = {0, 0, 0, 0};
    if (rot > 0) {
#pragma unroll
        for (int a = 0; a < 4; ++a) pos[a] = a == 0 || a < p.n_axes ? *(p.positions + static_cast<size_t>(a) * p.T + t) : pos[0];
    }
    if (slot < 0) return;  // padding: none of this token's rows is read or written
    const unsigned top = max(max(static_cast<unsigned>(pos[0]), static_cast<unsigned>(pos[1])),
                             max(static_cast<unsigned>(pos[2]), static_cast<unsigned>(pos[3])));
    const bool bad_pos = rot > 0 && top >= static_cast<unsigned>(p.max_pos);
    if (slot >= p.num_slots || bad_pos) {
        if (part == 0 && lane == 0)
            raise_err(p.err, (slot >= p.num_slots ? PA_DEVERR_SLOT : 0) | (bad_pos ? PA_DEVERR_POSITION : 0));
        return;
    }
    // cosines and sines of the unit's pairs: pair e is element e of both chunks, or elements 2e and 2e + 1
    uint64_t c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = f2_pack(1.f, 1.f), s[e] = f2_pack(0.f, 0.f);
    if (turns) {
        const uint32_t axes = p.axis[u];
        const int half = rot / 2;
        const auto pos_of = [&](uint32_t a) { return a & 2u ? a & 1u ? pos[3] : pos[2] : a & 1u ? pos[1] : pos[0]; };
        if (axes == (axes & 15u) * 0x11111111u) {
            // one position for the unit: four 16-byte loads
            const float *row = p.cos_sin + static_cast<size_t>(pos_of(axes & 3u)) * rot + u * 8;
            const float4 c0 = *reinterpret_cast<const float4 *>(row), c1 = *reinterpret_cast<const float4 *>(row + 4),
                         s0 = *reinterpret_cast<const float4 *>(row + half), s1 = *reinterpret_cast<const float4 *>(row + half + 4);
            c[0] = f2_pack(c0.x, c0.y), c[1] = f2_pack(c0.z, c0.w), c[2] = f2_pack(c1.x, c1.y), c[3] = f2_pack(c1.z, c1.w);
            s[0] = f2_pack(s0.x, s0.y), s[1] = f2_pack(s0.z, s0.w), s[2] = f2_pack(s1.x, s1.y), s[3] = f2_pack(s1.z, s1.w);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float *x = p.cos_sin + static_cast<size_t>(pos_of((axes >> (8 * e)) & 3u)) * rot + u * 8 + 2 * e;
                const float *y = p.cos_sin + static_cast<size_t>(pos_of((axes >> (8 * e + 4)) & 3u)) * rot + u * 8 + 2 * e + 1;
                c[e] = f2_pack(*x, *y);
                s[e] = f2_pack(x[half], y[half]);
            }
        }
    }
    const unsigned char *const q_row = p.q + t * p.q_stride + e0 * 2, *const k_row = p.k + t * p.k_stride + e0 * 2,
                        *const v_row = p.v + t * p.v_stride + u * 32;
    const int row_bytes = D * 2, next = (e1 - e0) * 2, per_step = 32 >> lanes_log2;
    const size_t cache_row = static_cast<size_t>(slot) * p.Hkv;
    size_t scale_row = 0;  // index of the slot's scale of kv head 0
    if constexpr (kQ8) scale_row = static_cast<size_t>(p.geom.block_of(slot)) * p.Hkv * p.geom.block_size + p.geom.offset_of(slot);
    // a row of keys or values in 8 bits; the warp's lanes all come here
    const auto store8 = [&](const Eight &f, const Eight &g, unsigned char *dst, float *scales, int h, bool on0, bool on1, int apart) {
        float most = largest(g, largest(f, 0.f));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            if (o < lanes) most = max_nan3(most, most, __shfl_xor_sync(0xffffffffu, most, o));
        float scale = __fdiv_rn(most, 448.f);
        if (scale < 0x1p-90f) scale = 0x1p-90f;
        const float inv = __frcp_rn(scale);
        if (on0) *reinterpret_cast<uint2 *>(dst) = quantise8(f, inv);
        if (on1) *reinterpret_cast<uint2 *>(dst + apart) = quantise8(g, inv);
        if (on0 && u == 0) scales[scale_row + static_cast<size_t>(h) * p.geom.block_size] = scale;
    };
    const int end = min((part + 1) * p.part_steps, p.steps);
    for (int step = part * p.part_steps; step < end; step += kAhead) {
        uint4 x0[kAhead], x1[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
            if (step + i < p.qk_steps) {
                const int r = (step + i) * per_step + row_of_lane;
                const unsigned char *src = r < p.Hq ? q_row + r * row_bytes : k_row + (r - p.Hq) * row_bytes;
                const bool mine = step + i < end && r < n_qk;  // a step behind the part's last is another warp's, which may store it in place
                if (mine && there0) x0[i] = ld_row(src);
                if (mine && there1) x1[i] = ld_row(src + next);
            } else {
                const int r = (step + i - p.qk_steps) * per_step + row_of_lane;
                const unsigned char *src = v_row + r * row_bytes;
                const bool mine = step + i < end && r < p.Hkv;
                if (mine && v_there0) x0[i] = ld_row(src);
                if (mine && v_there1) x1[i] = ld_row(src + 16);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (step + i >= end) break;
            if (step + i >= p.qk_steps) {
                const int r = (step + i - p.qk_steps) * per_step + row_of_lane;
                const bool on0 = r < p.Hkv && v_there0, on1 = r < p.Hkv && v_there1;
                if constexpr (kQ8) {
                    store8(widen8<E>(x0[i]), widen8<E>(x1[i]), p.v_cache + (cache_row + r) * D + u * 16, p.v_scale, r, on0, on1, 8);
                } else {
                    unsigned char *dst = p.v_cache + (cache_row + r) * row_bytes + u * 32;  // values are bit copies
                    if (on0) stg128(dst, x0[i]);
                    if (on1) stg128(dst + 16, x1[i]);
                }
                continue;
            }
            const int r = (step + i) * per_step + row_of_lane;
            const bool is_q = r < p.Hq, on0 = there0 && r < n_qk, on1 = there1 && r < n_qk;
            Eight f = widen8<E>(x0[i]), g = widen8<E>(x1[i]);
            if (p.q_weight || p.k_weight) {
                uint64_t sum = f2_mul(f.p[0], f.p[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) sum = f2_fma(f.p[e], f.p[e], sum);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = f2_fma(g.p[e], g.p[e], sum);
                float squares = f2_lo(sum) + f2_hi(sum);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    if (o < lanes) squares += __shfl_xor_sync(0xffffffffu, squares, o);
                const unsigned char *w = is_q ? p.q_weight : p.k_weight;
                if (w) {
                    const float m1 = rsqrtf(fmaf(squares, p.inv_d, p.eps));
                    const uint64_t m = f2_pack(m1, m1);
                    const uint4 w0 = on0 ? *reinterpret_cast<const uint4 *>(w + e0 * 2) : make_uint4(0, 0, 0, 0),
                                w1 = on1 ? *reinterpret_cast<const uint4 *>(w + e1 * 2) : make_uint4(0, 0, 0, 0);
                    const Eight wf = widen8<E>(w0), wg = widen8<E>(w1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f.p[e] = f2_mul(f2_mul(f.p[e], m), wf.p[e]);
                        g.p[e] = f2_mul(f2_mul(g.p[e], m), wg.p[e]);
                    }
                }
            }
            if (turns) {
                if constexpr (kPairs) {
                    // pairs lie side by side: (x0, x1) c + (-x1, x0) s, the latter product rounded (as in the rotation without norms)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto turn = [](uint64_t x, float cc, float ss) {
                            return f2_fma(x, f2_pack(cc, cc), f2_mul(f2_pack(-f2_hi(x), f2_lo(x)), f2_pack(ss, ss)));
                        };
                        uint64_t &lo = f.p[e], &hi = g.p[e];
                        lo = turn(lo, e & 1 ? f2_hi(c[e >> 1]) : f2_lo(c[e >> 1]), e & 1 ? f2_hi(s[e >> 1]) : f2_lo(s[e >> 1]));
                        hi = turn(hi, e & 1 ? f2_hi(c[2 + (e >> 1)]) : f2_lo(c[2 + (e >> 1)]),
                                  e & 1 ? f2_hi(s[2 + (e >> 1)]) : f2_lo(s[2 + (e >> 1)]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t minus = f2_pack(-f2_lo(g.p[e]), -f2_hi(g.p[e]));
                        const uint64_t y0 = f2_fma(f.p[e], c[e], f2_mul(minus, s[e])), y1 = f2_fma(g.p[e], c[e], f2_mul(f.p[e], s[e]));
                        f.p[e] = y0, g.p[e] = y1;
                    }
                }
            }
            if (!kQ8 || is_q) {
                unsigned char *dst = is_q ? p.q_out + t * p.qo_stride + r * row_bytes : p.k_cache + (cache_row + (r - p.Hq)) * row_bytes;
                if (on0) stg128(dst + e0 * 2, pack8<E>(f));
                if (on1) stg128(dst + e1 * 2, pack8<E>(g));
            }
            if constexpr (kQ8) {
                // (steps of queries alone have nothing for the cache)
                if ((step + i + 1) * per_step > p.Hq)
                    store8(f, g, p.k_cache + (cache_row + (r - p.Hq)) * D + e0, p.k_scale, r - p.Hq, on0 && !is_q, on1 && !is_q, e1 - e0);
            }
        }
    }
}

template <class E, bool kQ8>
cudaError_t launch_norm_typed(const NormRopeParams &prm, bool pairs, unsigned grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kNormThreads);
    if (pairs) return cudaLaunchKernelEx(&cfg, norm_rope_store_kv_kernel<E, true, kQ8, 0>, prm);
    if (prm.rot == 64 && prm.D == 64) return cudaLaunchKernelEx(&cfg, norm_rope_store_kv_kernel<E, false, kQ8, 64>, prm);
    if (prm.rot == 128 && prm.D == 128) return cudaLaunchKernelEx(&cfg, norm_rope_store_kv_kernel<E, false, kQ8, 128>, prm);
    return cudaLaunchKernelEx(&cfg, norm_rope_store_kv_kernel<E, false, kQ8, 0>, prm);
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
    for (prm.lanes = 1; prm.lanes < prm.units; prm.lanes *= 2) ++prm.lanes_log2;
    for (int i = 0; a.pair_axis && i < a.rot_dim / 2; ++i)
        prm.axis[i / 8] |= static_cast<uint32_t>(a.pair_axis[i]) << (4 * (i % 8));
    const int per_step = 32 >> prm.lanes_log2;
    prm.qk_steps = (a.Hq + a.Hkv + per_step - 1) / per_step;
    prm.steps = prm.qk_steps + (a.Hkv + per_step - 1) / per_step;
    // A warp a token where that leaves the SMs full, else a step each: the time is then one chain of dependent loads (a step
    // each, and a warp a token, us: 14/2 heads x 64 with three axes, cache of the storage type: 1500 tokens 4.2, 4.9; 2400: 6.3, 5.6;
    // 9001: 17.3, 12.2; 16/8 heads x 128 into 8 bits: 256: 3.7, 7.6; 1500: 9.0, 9.2; 2400: 12.6, 10.2; 5000: 27.4, 20.3).
    prm.part_steps = a.T > device_sm_count() * kFullWarps ? prm.steps : 1;
    prm.parts = (prm.steps + prm.part_steps - 1) / prm.part_steps;
    const long long warps = static_cast<long long>(a.T) * prm.parts;
    const unsigned grid = static_cast<unsigned>((warps + kNormThreads / 32 - 1) / (kNormThreads / 32));
    auto go = [&](auto e) {
        using E = decltype(e);
        return n.q8 ? launch_norm_typed<E, true>(prm, a.interleaved, grid, stream)
                    : launch_norm_typed<E, false>(prm, a.interleaved, grid, stream);
    };
    return a.dtype == PA_BF16 ? go(BF16{}) : go(F16{});
}

}  // namespace pa
