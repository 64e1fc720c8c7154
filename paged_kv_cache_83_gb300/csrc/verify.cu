// verify.cu: drafted tokens against the target's probabilities, from given random numbers (pa_verify).
//
// Source: smzdm nano-vLLM deep dive (sampling from each request's distribution); "nano-vLLM Part 4" section 3 (step 3: the
// next tokens). The acceptance rule is that of speculative sampling: a draft x is taken with probability
// min(1, p(x) / q(x)), the token after the last one taken comes from max(p - q, 0), so that the tokens have
// the target's distribution p whatever the drafter's q.
//
// The mathematics: the tests u q(x) < p(x) are exact, being products of two fp32 numbers in 64 bits (and this file is compiled without
// the fast mathematics that takes subnormal numbers for 0). A weight is the whole
// number rint(r 2^44), r in [0, 1]; whole numbers add up to the same sum in any order, so that the token does not depend
// on how the row is divided.
//
// Bound by HBM where there are many sequences (one row of p and one of q each), by the chain of dependent loads where there are
// few. So a sequence belongs to a cluster of CTAs: each finds the number of accepted drafts by itself (a few
// gathered numbers), sums the weights of its slice of the one row that matters, and all learn each other's sums through
// distributed shared memory; the CTA whose slice holds the token reads one warp's part of it again, from L2. One launch, no
// workspace. 256 sequences, 151,936 fp32 numbers in p and in q: 51 us, 0.71 of a copy (one CTA a sequence: 78 us); one
// sequence with a draft of four tokens and a drafter without probabilities, bf16: 7.0 us (8.9 in smaller clusters).
#include <atomic>

#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kVerifySm = 1536;  // threads of an SM, in CTAs of 384 or 512
constexpr int kMostCtas = 8;     // of a sequence: the portable cluster
constexpr unsigned kAll = 0xffffffffu;

struct F32 {
    using T = float;
};

struct VerifyParams {
    int32_t *next_tokens, *accepted, *err;
    const int32_t *tokens, *cu_q;
    const float *u;
    const void *probs, *draft_probs;
    long long p_stride, q_stride;  // elements
    int S, V, total_q, slice;      // slice: weights of a warp, a multiple of 32 loads
};

// 16-byte load of what the grid before may have written (not the read-only path: this grid is launched beside that one)
__device__ __forceinline__ uint4 ld_probs(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <class E>
__device__ __forceinline__ void widen(const uint4 &w, float *f) {
    unpack8<E>(w, *reinterpret_cast<float(*)[8]>(f));
}
template <>
__device__ __forceinline__ void widen<F32>(const uint4 &w, float *f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }

// kN numbers of a row from index i on; 0 outside [0, V). `wide`: the address of index i is 16-byte aligned.
template <class E, int kN>
__device__ __forceinline__ void load_row(const typename E::T *row, int i, int V, bool wide, float (&f)[kN]) {
    if (wide && i >= 0 && i + kN <= V) {
        widen<E>(ld_probs(row + i), f);
    } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) f[e] = i + e >= 0 && i + e < V ? widen1(row[i + e]) : 0.f;
    }
}

// What the token is drawn from: `diff`: max(p - q, 0), else p, but for the token `bare` (-1: none), which has no weight
template <class T>
struct Drawn {
    const T *p, *q;
    bool diff;
    int bare;
    int shift;      // index 0 of the row lies `shift` numbers behind a 16-byte boundary
    bool same;      // q's row as well
};

// rint(r 2^44) = hi 2^22 + lo, r in [0, 1]. The sum r + 2 holds r in steps of 2^-22, what is missing of r is exact, and its sum with
// 1.5 * 2^-21 holds it in steps of 2^-44 (each rounded to nearest even).
__device__ __forceinline__ void weight(float r, int &hi, int &lo) {
    r = fminf(fmaxf(r, 0.f), 1.f);  // NaN: 0
    const float h = __fadd_rn(r, 2.f);
    const float rest = __fsub_rn(r, __fsub_rn(h, 2.f));
    hi = __float_as_int(h) - __float_as_int(2.f);
    lo = __float_as_int(__fadd_rn(rest, 0x1.8p-21f)) - __float_as_int(0x1.8p-21f);
}
// Sums of hi and lo of up to kLaneMost weights, each at most 2^22 and 2^21 in magnitude, whatever the row holds
constexpr int kLaneMost = 1023;
__device__ __forceinline__ long long whole(uint32_t hi, int lo) { return (static_cast<long long>(hi) << 22) + lo; }

template <class E, int kN>
__device__ __forceinline__ void weights_at(const Drawn<typename E::T> &d, int i, int V, float (&r)[kN]) {
    load_row<E>(d.p, i, V, true, r);
    if (d.diff) {
        float q[kN];
        load_row<E>(d.q, i, V, d.same, q);
#pragma unroll
        for (int e = 0; e < kN; ++e) r[e] = __fsub_rn(r[e], q[e]);
    }
#pragma unroll
    for (int e = 0; e < kN; ++e)
        if (i + e == d.bare) r[e] = 0.f;
}

template <class E, int kThreads>
__global__ void __launch_bounds__(kThreads, kVerifySm / kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
    using T = typename E::T;
    constexpr int kN = 16 / sizeof(T), kWarps = kThreads / 32;
    __shared__ long long warp_sum[2][kWarps], cta_sum[2];
    __shared__ int taken, ended;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
    const int s = blockIdx.x / ctas;
    // launched beside what precedes it in the stream, whose results are read and written from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int a0 = p.cu_q[s], a1 = p.cu_q[s + 1];
    if (a0 < 0 || a1 < a0 || a1 > p.total_q || a1 == a0) {  // the same for every CTA of the cluster
        if (rank == 0 && tid == 0) {
            p.accepted[s] = 0;
            if (a1 != a0 || a0 < 0 || a0 > p.total_q) raise_err(p.err, PA_DEVERR_LENGTH);
        }
        return;
    }
    const int n = a1 - a0 - 1;  // drafts
    const T *probs = static_cast<const T *>(p.probs), *draft_probs = static_cast<const T *>(p.draft_probs);
    if (warp == 0) {
        int got = n;
        bool end = false;
        for (int r0 = 0; r0 < n; r0 += 32) {
            const int r = r0 + lane;
            bool stop = false, none = false;
            if (r < n) {
                const int x = p.tokens[a0 + r + 1];
                none = static_cast<unsigned>(x) >= static_cast<unsigned>(p.V);
                stop = true;
                if (!none) {
                    const double px = widen1(probs[(a0 + r) * p.p_stride + x]);
                    const double qx = draft_probs ? static_cast<double>(widen1(draft_probs[(a0 + r) * p.q_stride + x])) : 1.0;
                    stop = !(static_cast<double>(p.u[a0 + r]) * qx < px);
                }
            }
            const unsigned stops = __ballot_sync(kAll, stop), nones = __ballot_sync(kAll, none);
            if (stops) {
                const int first = __ffs(stops) - 1;
                got = r0 + first;
                end = nones >> first & 1u;
                break;
            }
        }
        if (lane == 0) taken = got, ended = end;
    }
    __syncthreads();
    const int a = taken;
    Drawn<T> d;
    d.p = probs + (a0 + a) * p.p_stride;
    d.q = draft_probs ? draft_probs + (a0 + a) * p.q_stride : nullptr;
    const bool rejected = a < n && !ended;
    d.diff = rejected && draft_probs;
    d.bare = rejected && !draft_probs ? p.tokens[a0 + a + 1] : -1;
    d.shift = static_cast<int>(reinterpret_cast<uintptr_t>(d.p) % 16 / sizeof(T));
    d.same = d.diff && reinterpret_cast<uintptr_t>(d.q) % 16 == reinterpret_cast<uintptr_t>(d.p) % 16;
    if (rank == 0) {
        for (int r = tid; r <= n; r += kThreads)
            if (r != a) p.next_tokens[a0 + r] = r < a ? p.tokens[a0 + r + 1] : -1;
        if (tid == 0) p.accepted[s] = a;
    }
    const float uf = p.u[a1 - 1];
    const uint32_t u31 = uf > 0.f ? uf < 1.f ? static_cast<uint32_t>(uf * 0x1p31f) : 0x7fffffffu : 0u;
    const int first = (static_cast<int>(rank) * kWarps + warp) * p.slice - d.shift;  // of this warp's slice
    for (int attempt = 0;; ++attempt) {
        // ---- the sums of the slices
        uint32_t hi = 0;
        int lo = 0;
#pragma unroll 2
        for (int i = first + lane * kN; i < first + p.slice && i < p.V; i += 32 * kN) {
            float r[kN];
            weights_at<E>(d, i, p.V, r);
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                int h, l;
                weight(r[e], h, l);
                hi += static_cast<uint32_t>(h), lo += l;
            }
        }
        long long sum = whole(hi, lo);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) warp_sum[attempt][warp] = sum;
        __syncthreads();
        if (warp == 0) {
            long long v = lane < kWarps ? warp_sum[attempt][lane] : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
            if (lane == 0) cta_sum[attempt] = v;
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        long long all = 0, before = 0, mine = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
            uint32_t at;
            long long v;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&cta_sum[attempt])), "r"(c));
            asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(at));
            if (c < rank) before += v;
            if (c == rank) mine = v;
            all += v;
        }
        if (all == 0 && attempt == 0 && rejected) {
            // nothing is left where the drafter is nowhere below the target: the target's own row
            d.diff = false;
            d.bare = -1;
            continue;
        }
        // the first token whose running sum exceeds u times the whole
        const long long border = (all >> 31) * u31 + (((all & 0x7fffffffll) * u31) >> 31);
        if (all == 0) {
            if (rank == 0 && tid == 0) {
                p.next_tokens[a0 + a] = -1;
                raise_err(p.err, PA_DEVERR_ROW);
            }
        } else if (before <= border && border < before + mine) {
            long long left = border - before;  // in this CTA's slice
            int w = 0;
            while (left >= warp_sum[attempt][w]) left -= warp_sum[attempt][w++];
            const int begin = (static_cast<int>(rank) * kWarps + w) * p.slice - d.shift;
            // the block takes the warp's slice, a few numbers a thread
            __shared__ long long step_sum[kWarps];
            for (int at = begin; at < begin + p.slice; at += kThreads * kN) {
                const int i = at + tid * kN;
                float r[kN];
                long long v = 0;
                if (i < begin + p.slice) {
                    weights_at<E>(d, i, p.V, r);
                    int h, l, hs = 0, ls = 0;
#pragma unroll
                    for (int e = 0; e < kN; ++e) weight(r[e], h, l), hs += h, ls += l;
                    v = whole(hs, ls);
                }
                long long upto = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long x = __shfl_up_sync(kAll, upto, o);
                    if (lane >= o) upto += x;
                }
                __syncthreads();
                if (lane == 31) step_sum[warp] = upto;
                __syncthreads();
                long long ahead = upto - v, step = 0;
                for (int k = 0; k < kWarps; ++k) {
                    if (k < warp) ahead += step_sum[k];
                    step += step_sum[k];
                }
                if (ahead <= left && left < ahead + v) {  // one thread
                    long long rest = left - ahead;
                    int token = -1;
#pragma unroll
                    for (int e = 0; e < kN; ++e) {
                        int h, l;
                        weight(r[e], h, l);
                        const long long x = whole(h, l);
                        if (token < 0 && rest < x) token = i + e;
                        rest -= x;
                    }
                    p.next_tokens[a0 + a] = token;
                }
                if (left < step) break;  // the same for every thread
                left -= step;
            }
        }
        break;
    }
    // no CTA leaves while another may read its sums
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Clusters of 1 .. kMostCtas CTAs that are on the SMs at once (asked for once for each kernel and device; threads that ask at the
// same time write the same numbers, and whoever sees the mark of a full table sees them)
template <class E, int kThreads>
cudaError_t active_clusters(int dev, int (&most)[kMostCtas + 1]) {
    static std::atomic<int> table[64][kMostCtas + 1];  // [0]: filled
    if (!table[dev][0].load(std::memory_order_acquire)) {
        for (int ctas = 1; ctas <= kMostCtas; ++ctas) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = ctas;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg{};
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(ctas);
            cfg.blockDim = dim3(kThreads);
            int clusters = 0;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, verify_kernel<E, kThreads>, &cfg);
            if (e != cudaSuccess) return e;
            table[dev][ctas].store(clusters, std::memory_order_relaxed);
        }
        table[dev][0].store(1, std::memory_order_release);
    }
    for (int ctas = 1; ctas <= kMostCtas; ++ctas) most[ctas] = table[dev][ctas].load(std::memory_order_relaxed);
    return cudaSuccess;
}

template <class E, int kThreads>
cudaError_t launch_verify_as(VerifyParams &prm, int ctas, cudaStream_t stream) {
    constexpr int kN = 16 / sizeof(typename E::T);
    constexpr int per = 32 * kN;
    const auto slice_of = [](int V, int parts) constexpr { return ((V + kN + parts - 1) / parts + per - 1) / per * per; };
    static_assert(slice_of(kSampleMaxVocab, kThreads / 32) / 32 <= kLaneMost, "a lane's sums");
    prm.slice = slice_of(prm.V, ctas * (kThreads / 32));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(prm.S) * ctas);
    cfg.blockDim = dim3(kThreads);
    return cudaLaunchKernelEx(&cfg, verify_kernel<E, kThreads>, prm);
}

template <class E>
cudaError_t launch_verify_typed(const VerifyParams &in, cudaStream_t stream) {
    VerifyParams prm = in;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int most_384[kMostCtas + 1], most_512[kMostCtas + 1];
    if ((e = active_clusters<E, 384>(dev, most_384)) != cudaSuccess || (e = active_clusters<E, 512>(dev, most_512)) != cudaSuccess) return e;
    // CTAs of a sequence: slices of at least 4096 numbers, and no more CTAs than are on the SMs at once: each begins and ends
    // with a chain of dependent loads and barriers. Of the two sizes of CTA the one that leaves more threads (p and q in fp32, us,
    // powers of two of 384 threads before, this rule after: 4 sequences 18.4, 16.6; 76: 36.0, 26.7; 152: 51.0, 38.8; 256: 54.9,
    // 54.8; 400: 89.1, 78.0).
    const auto ctas_of = [&](const int *most) {
        int ctas = 1;
        for (int c = 2; c <= kMostCtas; ++c)
            if (prm.V > 4096 * (c - 1) && prm.S <= most[c]) ctas = c;
        return ctas;
    };
    const int c384 = ctas_of(most_384), c512 = ctas_of(most_512);
    return prm.S <= most_512[c512] && 512 * c512 > 384 * c384 ? launch_verify_as<E, 512>(prm, c512, stream)
                                                              : launch_verify_as<E, 384>(prm, c384, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t stream) {
    VerifyParams prm{};
    prm.next_tokens = a.next_tokens, prm.accepted = a.accepted, prm.err = a.err;
    prm.tokens = a.tokens, prm.cu_q = a.cu_q, prm.u = a.u;
    prm.probs = a.probs, prm.draft_probs = a.draft_probs;
    prm.p_stride = a.p_stride, prm.q_stride = a.q_stride;
    prm.S = a.S, prm.V = a.V, prm.total_q = a.total_q;
    if (a.dtype == PA_F32) return launch_verify_typed<F32>(prm, stream);
    return a.dtype == PA_BF16 ? launch_verify_typed<BF16>(prm, stream) : launch_verify_typed<F16>(prm, stream);
}

}  // namespace pa
