// sample.cu: one token per row of logits from a given random number, with temperature, top-k, top-p
// and min-p (pa_sample).
//
// Source: smzdm nano-vLLM deep dive (the sampler with its per-request temperature); "nano-vLLM Part 4",
// section 3 (rank 0 samples the step's tokens from the logits).
//
// The mathematics: weights w_j = exp((x_j - max x) / T); the kept set is a prefix of the tokens
// ordered by descending logit, lowest index first among equals (top-k by count, then top-p by the
// sum of weights), less those below min-p; the token is the first in the order of the vocabulary at
// which the running sum of kept weights exceeds u times their whole sum.
//
// A token is decided at borders of long sums, so the sums are exact integers: a weight is computed
// to about 2^-31 of itself in pairs of fp32 numbers (no 64-bit floating point: this GPU has little)
// and held as a multiple of 2^-44; 64-bit integer sums do not depend on their order, so the result
// is the same for any number of threads and CTAs.
//
// A cluster of CTAs holds one row in shared memory: logits are read from HBM once, every later pass
// runs on chip, and the CTAs exchange their partial counts and sums through distributed shared
// memory.
#include <cooperative_groups.h>
#include <float.h>

#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kFrac = 44;     // weights are multiples of 2^-44; the largest is 2^44
constexpr int kTable = 33;    // 2^(k / 32), k = -16 .. 16

struct SampleParams {
    const void *logits;
    long long row_stride;
    int V, per_warp;  // elements of a row that each warp holds (a multiple of 32)
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    int32_t *err;
};

using u64 = unsigned long long;

struct alignas(16) Pow {  // 2^(k / 32): a multiple of 2^-44, and rounded
    u64 fixed;
    float f;
    float pad;
};

struct Shared {
    Pow pow[kTable];
    u64 mass[2][kMaxCluster];       // one CTA's partial sums each, written by that CTA
    uint32_t count[2][kMaxCluster];
    u64 warp_mass[kWarps];
    uint32_t warp_count[kWarps];
    u64 bcast[2];
};

// order-preserving map of a float that is not NaN (and no negative zero)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// A row's temperature as a pair of floats: log2(e) / T = ch + cl
struct Heat {
    float max, ch, cl;
};

// The weight 2^(44 + (x - max) log2(e) / T), by Dekker's pair arithmetic: the difference and its
// rounding error (Knuth's two-sum), times the pair ch + cl; then 2^t = 2^n 2^(k/32) e^z with
// |z| < 0.011 and four terms of the exponential series (the fifth is below 2^-39).
__device__ __forceinline__ u64 weight(const Pow *pow, const Heat &h, float x) {
    if (x == h.max) return 1ull << kFrac;
    const float d = __fadd_rn(x, -h.max);
    const float bb = __fadd_rn(d, -x);
    const float e = __fadd_rn(__fadd_rn(x, -__fadd_rn(d, -bb)), __fadd_rn(-h.max, -bb));
    const float th = __fmul_rn(d, h.ch);
    if (!(th > -46.f)) return 0;  // below 2^-45; x = -inf; a temperature near zero
    const float tl = __fmaf_rn(d, h.ch, -th) + __fmaf_rn(d, h.cl, e * h.ch);
    const float n = rintf(th), f = th - n;
    const float k = rintf(f * 32.f);
    const float z = (__fmaf_rn(k, -1.f / 32.f, f) + tl) * 0.693147180559945f;
    const float q = z * __fmaf_rn(z, __fmaf_rn(z, __fmaf_rn(z, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
    const Pow w = pow[static_cast<int>(k) + 16];
    // |w.f q| < 2^-5.9: as a multiple of 2^-36 it fits 32 bits, to the accuracy it has
    const long long lo = static_cast<long long>(__float2int_rn(w.f * q * 68719476736.f)) << (kFrac - 36);
    return (w.fixed + lo) >> static_cast<int>(-n);
}

template <class L>
__device__ __forceinline__ void load16(const unsigned char *src, float (&f)[16 / sizeof(L)]);
template <>
__device__ __forceinline__ void load16<float>(const unsigned char *src, float (&f)[4]) {
    const uint4 v = ldg_stream(src);
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void load16<__half>(const unsigned char *src, float (&f)[8]) {
    unpack8<F16>(ldg_stream(src), f);
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const unsigned char *src, float (&f)[8]) {
    unpack8<BF16>(ldg_stream(src), f);
}

template <class L>
__global__ void __launch_bounds__(kSampleThreads, 1) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    float *vals = reinterpret_cast<float *>(smem_raw + sizeof(Shared));  // [kWarps * per_warp]
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / CS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int PW = p.per_warp;
    float *mine = vals + warp * PW;  // this warp's part of the row, in the row's order
    const int base = (rank * kWarps + warp) * PW;

    if (tid < kTable) {
        const double v = exp2((tid - 16) / 32.0);
        sh.pow[tid] = Pow{static_cast<u64>(v * static_cast<double>(1ull << kFrac) + 0.5), static_cast<float>(v), 0.f};
    }

    // ---- the row into shared memory: whole 16-byte words, those that hold elements of the row.
    // Element i of the held row is element i - skew of the row: rows may start off the 16-byte grid.
    constexpr int EV = 16 / static_cast<int>(sizeof(L));
    const unsigned char *src = static_cast<const unsigned char *>(p.logits) + row * p.row_stride * static_cast<long long>(sizeof(L));
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(L));
    src -= skew * sizeof(L);
    const int end = p.V + skew;
    float mx = -INFINITY;
#pragma unroll 4
    for (int i = lane * EV; i < PW; i += 32 * EV) {
        float f[EV];
        if (base + i < end) {
            load16<L>(src + static_cast<size_t>(base + i) * sizeof(L), f);
        }
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            const int at = base + i + e;
            float x = at >= skew && at < end ? f[e] : -INFINITY;
            if (!(x > -INFINITY)) x = -INFINITY;  // NaN is never chosen
            if (x == 0.f) x = 0.f;                // -0 equals 0
            mine[i + e] = x;
            mx = fmaxf(mx, x);
        }
    }
    cluster.sync();  // the table is set, and every CTA of the cluster runs before another writes to it

    int turn = 0;
    // every CTA's (mass, count) into every CTA of the cluster: call with the warps' values in lane 0's
    // registers reduced already
    auto exchange = [&](u64 m, uint32_t c) {
#pragma unroll
        for (int o = 16; o; o >>= 1) m += __shfl_xor_sync(kAll, m, o);
        c = __reduce_add_sync(kAll, c);
        if (lane == 0) sh.warp_mass[warp] = m, sh.warp_count[warp] = c;
        __syncthreads();
        if (warp == 0) {
            m = lane < kWarps ? sh.warp_mass[lane] : 0;
            c = lane < kWarps ? sh.warp_count[lane] : 0;
#pragma unroll
            for (int o = kWarps / 2; o; o >>= 1) m += __shfl_xor_sync(kAll, m, o);
            c = __reduce_add_sync(kAll, c);
            m = __shfl_sync(kAll, m, 0);
            if (lane < CS) {
                Shared *to = cluster.map_shared_rank(&sh, lane);
                to->mass[turn][rank] = m;
                to->count[turn][rank] = c;
            }
        }
        cluster.sync();
        turn ^= 1;
    };
    auto total_mass = [&]() {
        u64 t = 0;
        for (int i = 0; i < CS; ++i) t += sh.mass[turn ^ 1][i];
        return t;
    };
    auto total_count = [&]() {
        uint32_t t = 0;
        for (int i = 0; i < CS; ++i) t += sh.count[turn ^ 1][i];
        return t;
    };
    // after an exchange of the sums of f over the row: the held index at which the running sum of f
    // first exceeds `target` (below the total). Found by one warp of the cluster, -1 elsewhere.
    auto locate = [&](u64 target, auto f) {
        int r = 0;
        for (; r < CS - 1 && target >= sh.mass[turn ^ 1][r]; ++r) target -= sh.mass[turn ^ 1][r];
        if (r != rank) return -1;
        int w = 0;
        for (; w < kWarps - 1 && target >= sh.warp_mass[w]; ++w) target -= sh.warp_mass[w];
        if (w != warp) return -1;
        for (int i = 0; i < PW; i += 32) {
            const u64 v = f(mine[i + lane], base + i + lane);
            u64 s = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(kAll, s, o);
                if (lane >= o) s += t;
            }
            const unsigned over = __ballot_sync(kAll, s > target);
            if (over) return base + i + __ffs(over) - 1;
            target -= __shfl_sync(kAll, s, 31);
        }
        return -1;
    };

    // ---- the largest logit
    {
        uint32_t k = __reduce_max_sync(kAll, key_of(mx));
        if (lane == 0) sh.warp_count[warp] = k;
        __syncthreads();
        if (warp == 0) {
            k = __reduce_max_sync(kAll, lane < kWarps ? sh.warp_count[lane] : 0);
            if (lane < CS) cluster.map_shared_rank(&sh, lane)->count[turn][rank] = k;
        }
        cluster.sync();
        turn ^= 1;
    }
    uint32_t kmax = 0;
    for (int i = 0; i < CS; ++i) kmax = max(kmax, sh.count[turn ^ 1][i]);
    const float T = p.temperature ? __ldg(p.temperature + row) : 1.f;
    const bool greedy = !(T > 0.f);
    Heat heat;
    heat.max = __uint_as_float(kmax & 0x80000000u ? kmax ^ 0x80000000u : ~kmax);
    {
        const double c = 1.4426950408889634 / static_cast<double>(greedy ? 1.f : T);
        heat.ch = static_cast<float>(fmin(c, static_cast<double>(FLT_MAX)));
        heat.cl = heat.ch < FLT_MAX ? static_cast<float>(c - static_cast<double>(heat.ch)) : 0.f;
    }
    const uint32_t kfloor = key_of(-INFINITY);
    if (kmax == kfloor) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            raise_err(p.err, PA_DEVERR_ROW);
        }
        cluster.sync();
        return;
    }

    // kept: keys above `tau`, and those equal to it up to held index `cut`
    uint32_t tau = kfloor;
    int cut = 0x7fffffff;
    // count of keys >= t over the row
    auto count_from = [&](uint32_t t) {
        uint32_t c = 0;
        for (int i = lane; i < PW; i += 32) c += key_of(mine[i]) >= t;
        exchange(0, c);
        return total_count();
    };
    auto kept = [&](float x, int at) {
        const uint32_t k = key_of(x);
        return k > tau || (k == tau && at <= cut);
    };
    auto kept_mass_from = [&](uint32_t t) {
        u64 m = 0;
        for (int i = lane; i < PW; i += 32) {
            const float x = mine[i];
            if (key_of(x) >= t && kept(x, base + i)) m += weight(sh.pow, heat, x);
        }
        exchange(m, 0);
        return total_mass();
    };
    // the held index of the r-th (r >= 1) element equal to key t
    auto nth_equal = [&](uint32_t t, uint32_t r) {
        u64 c = 0;
        for (int i = lane; i < PW; i += 32) c += key_of(mine[i]) == t;
        exchange(c, 0);
        const int at = locate(r - 1, [&](float x, int) { return static_cast<u64>(key_of(x) == t); });
        if (at >= 0 && lane < CS) cluster.map_shared_rank(&sh, lane)->bcast[0] = at;
        cluster.sync();
        const int found = static_cast<int>(sh.bcast[0]);
        cluster.sync();
        return found;
    };

    if (greedy) {
        tau = kmax;
    } else {
        const int k = p.top_k ? __ldg(p.top_k + row) : 0;
        if (k > 0 && k < p.V) {
            uint32_t lo = kfloor, hi = kmax;  // the largest key t with count(>= t) >= k
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                if (count_from(mid) >= static_cast<uint32_t>(k))
                    lo = mid;
                else
                    hi = mid - 1;
            }
            tau = lo;
            const uint32_t above = tau == 0xffffffffu ? 0 : count_from(tau + 1);
            cut = nth_equal(tau, static_cast<uint32_t>(k) - above);
        }
        const float pp = p.top_p ? __ldg(p.top_p + row) : 1.f;
        if (pp < 1.f) {
            const u64 whole = kept_mass_from(0);
            // kept while the sum before a token is below pp of the whole
            const double want = fmax(static_cast<double>(pp), 0.0) * static_cast<double>(whole);
            uint32_t lo = tau, hi = kmax;  // the largest key t with mass(>= t) >= want
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                if (static_cast<double>(kept_mass_from(mid)) >= want)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const u64 above = kept_mass_from(lo + 1);
            const uint32_t key = lo;
            const float x = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
            const double w = static_cast<double>(weight(sh.pow, heat, x));
            const double more = ceil((want - static_cast<double>(above)) / fmax(w, 1.0));
            const uint32_t r = more < 1.0 ? 1u : more > 1e9 ? 1000000000u : static_cast<uint32_t>(more);
            // at most as many equals as top-k left
            u64 c = 0;
            for (int i = lane; i < PW; i += 32) c += key_of(mine[i]) == key && kept(mine[i], base + i);
            exchange(c, 0);
            const u64 equals = total_mass();
            if (r < equals)
                cut = nth_equal(key, r);
            else if (key != tau)
                cut = 0x7fffffff;  // all of them
            tau = key;
        }
    }

    // ---- the kept sum, and the token
    const float mp = !greedy && p.min_p ? __ldg(p.min_p + row) : 0.f;
    const u64 least =
        mp > 0.f ? static_cast<u64>(ceil(static_cast<double>(fminf(mp, 1.f)) * static_cast<double>(1ull << kFrac))) : 0;
    auto share = [&](float x, int at) {
        if (!kept(x, at)) return static_cast<u64>(0);
        const u64 w = weight(sh.pow, heat, x);
        return w >= least ? w : static_cast<u64>(0);
    };
    u64 m = 0;
    for (int i = lane; i < PW; i += 32) m += share(mine[i], base + i);
    exchange(m, 0);
    const u64 whole = total_mass();
    const float u = greedy || !p.u ? 0.f : __ldg(p.u + row);
    u64 target = u > 0.f ? static_cast<u64>(static_cast<double>(fminf(u, 1.f)) * static_cast<double>(whole)) : 0;
    if (target >= whole) target = whole - 1;
    const int at = locate(target, share);
    if (at >= 0 && lane == 0) p.tokens[row] = at - skew;
    cluster.sync();  // no CTA leaves while another may still write to it
}

template <class L>
cudaError_t launch_typed(const SampleArgs &a, cudaStream_t stream) {
    SampleParams prm{};
    prm.logits = a.logits;
    prm.row_stride = a.row_stride;
    prm.V = a.V;
    prm.u = a.u, prm.temperature = a.temperature, prm.top_p = a.top_p, prm.min_p = a.min_p, prm.top_k = a.top_k;
    prm.tokens = a.tokens;
    prm.err = a.err;
    // a CTA for every 4096 elements of a row, up to eight
    int CS = 1;
    while (CS < kMaxCluster && a.V > 4096 * CS) CS *= 2;
    const int held = a.V + 16 / static_cast<int>(sizeof(L)) - 1;  // the row and the skew of its start
    prm.per_warp = (held + CS * kWarps * 32 - 1) / (CS * kWarps * 32) * 32;
    const size_t smem = sizeof(Shared) + static_cast<size_t>(kWarps) * prm.per_warp * 4;
    auto kern = sample_kernel<L>;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448)) != cudaSuccess)
            return e;
        configured[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * CS);
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    if (a.dtype == PA_F32) return launch_typed<float>(a, stream);
    return a.dtype == PA_BF16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<__half>(a, stream);
}

}  // namespace pa
