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
// A cluster of CTAs holds one row in shared memory: logits are read from HBM once, by one bulk copy a warp, every
// later pass runs on chip, and the CTAs exchange their partial counts and sums through distributed
// shared memory. Top-k of up to as many tokens as the cluster has warps: the k-th largest of the
// warps' maxima bounds it, close to k tokens lie above, and one CTA decides among them. Else tokens
// fall into 1024 bins by their distance from the maximum, the bin that holds the border into 1024 again if it is
// full, and the last candidates are ordered by counting; equal logits are told apart by index.
//
// Compiled without flush-to-zero: subnormal logits are ordered, and weighed, like any others.
//
// Measured: 256 rows of 151,936 fp32 with settings of every kind 147 us (the reads alone: 23); by kind,
// greedy 50, top-k 85, temperature alone 131, top-p 317 (bf16: 46, 81, 126, 329): what bounds the last two is the
// instructions of the weights and the bins, 40 and 100 a token, at two CTAs an SM. One row: greedy 5 us, top-k 11,
// temperature alone 11, top-p 19-31 by the row, chains of cluster-wide barriers of about a microsecond.
#include <cooperative_groups.h>

#include <cmath>
#include <type_traits>

#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 16;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kFrac = 44;     // weights are multiples of 2^-44; the largest is 2^44
constexpr int kTable = 64;    // 2^(k / 32), k = -16 .. 16, at index k mod 64
// Below this temperature log2(e) / T may leave fp32, and logits whose weights differ may lie a subnormal number
// apart: the row is then scaled by kWarm, and log2(e) / T by its inverse.
constexpr float kCold = 0x1p-62f, kWarm = 0x1p64f;

using u64 = unsigned long long;

struct Pow {  // 2^(k / 32) 2^31: rounded to an integer, and as a float
    uint32_t fixed;
    float f;
};

struct SampleParams {
    const void *logits;
    long long row_stride;
    int V, per_warp;  // elements of a row that each warp holds (a multiple of 32)
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    int32_t *err;
    Pow pow[kTable];
};

constexpr int kBins = 1024;
constexpr float kBinsPerOctave = 22.f;  // the last bin, from 46.5 octaves below the maximum on, has no weight
constexpr int kCandidates = 256;
// A weight is added to a bin as three pieces of 15 bits with 32-bit atomics (the 64-bit form is a
// retry loop): a CTA holds under 2^16 elements, so no piece's sum passes 2^31.
constexpr int kPieces = 3, kPieceBits = 15;

struct alignas(16) Candidate {
    u64 order;  // the logit's key, then the complement of the held index: descending in the order of tokens
    u64 f;
};

struct Shared {
    Pow pow[kTable];
    u64 mass[2][kMaxCluster];  // one CTA's partial sums each, written by that CTA
    u64 warp_mass[kWarps];
    u64 bcast[2][2];
    u64 landed[kWarps];  // mbarriers: each warp's part of the row
    Candidate cand[kCandidates];  // this CTA's own; rank 0 then joins them in `joined`
    Candidate joined[kCandidates];
    u64 warp_max[kMaxCluster * kWarps];  // of every warp of the cluster: key of its maximum, and ...
    uint32_t n_cand;
    float ch, cl;
    uint32_t kth;
    uint32_t hist[kPieces][kBins];  // sums of the weights' 15-bit pieces (counts: the first)
};
static_assert(sizeof(Shared) % 16 == 0, "the row follows on a 16-byte boundary");

// Order-preserving maps between floats that are not NaN (without negative zero) and integers.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// log2(e) / T of a row as a pair of floats, ch + cl, and its largest logit
struct Heat {
    float max, ch, cl;
};

// (x - max) log2(e) / T in one float, for ordering: monotone in x, 0 for the maximum (which is finite)
__device__ __forceinline__ float octaves(const Heat &h, float x) {
    return __fmul_rn(__fadd_rn(x, -h.max), h.ch);
}

// The weights 2^(44 + (x - max) log2(e) / T) of two logits, by Dekker's pair arithmetic: the difference and
// its rounding error (Knuth's two-sum), times the pair ch + cl; then 2^t = 2^n 2^(k/32) 2^y with |y| < 1/64
// and four terms of the exponential series in y ln 2 (the fifth is below 2^-39). Rounding to an
// integer is the addition of 1.5 * 2^23, whose low bits then hold it. From 45 octaves below the
// maximum on (x = -inf, a temperature near zero) the shift leaves nothing. The arithmetic before the table runs
// on both numbers at a time (the packed fp32 instructions).
__device__ __forceinline__ void weight2(const Pow *pow, const Heat &h, float x0, float x1, u64 &w0, u64 &w1) {
    constexpr float kRound = 12582912.f;
    const uint64_t x = f2_pack(x0, x1), neg_max = f2_pack(-h.max, -h.max), ch = f2_pack(h.ch, h.ch),
                   cl = f2_pack(h.cl, h.cl), minus = f2_pack(-1.f, -1.f),
                   up = f2_pack(kRound, kRound), down = f2_pack(-kRound, -kRound);
    auto sub = [&](uint64_t a, uint64_t b) { return f2_fma(b, minus, a); };  // exact product: rounds once
    const uint64_t d = f2_add(x, neg_max);
    const uint64_t t = f2_mul(d, ch);
    const uint64_t th = f2_pack(fmaxf(f2_lo(t), -60.f), fmaxf(f2_hi(t), -60.f));
    const uint64_t bb = sub(d, x);
    const uint64_t e = f2_add(sub(x, sub(d, bb)), sub(neg_max, bb));
    const uint64_t lo = f2_add(f2_fma(d, ch, f2_mul(th, minus)), f2_fma(d, cl, f2_mul(e, ch)));
    const uint64_t nr = f2_add(th, up), f = sub(th, f2_add(nr, down));
    const uint64_t kr = f2_fma(f, f2_pack(32.f, 32.f), up), k = f2_add(kr, down);
    const uint64_t y = f2_add(f2_fma(k, f2_pack(-1.f / 32.f, -1.f / 32.f), f), lo);
    uint64_t q = f2_fma(y, f2_pack(9.618129e-3f, 9.618129e-3f), f2_pack(5.550411e-2f, 5.550411e-2f));
    q = f2_fma(y, q, f2_pack(2.4022651e-1f, 2.4022651e-1f));
    q = f2_fma(y, q, f2_pack(6.9314718e-1f, 6.9314718e-1f));
    q = f2_mul(y, q);
    auto finish = [&](float kr1, float nr1, float q1) {
        const Pow w = pow[__float_as_uint(kr1) & (kTable - 1)];
        const uint32_t m = w.fixed + __float2int_rn(w.f * q1);
        return (static_cast<u64>(m) << (kFrac - 31)) >> ((__float_as_int(kRound) - __float_as_int(nr1)) & 63);
    };
    w0 = finish(f2_lo(kr), f2_lo(nr), f2_lo(q));
    w1 = finish(f2_hi(kr), f2_hi(nr), f2_hi(q));
}
__device__ __forceinline__ u64 weight(const Pow *pow, const Heat &h, float x) {
    u64 w, unused;
    weight2(pow, h, x, x, w, unused);
    return w;
}

// the elements of a 16-byte word
__device__ __forceinline__ void split(const uint4 &v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <class L>
__device__ __forceinline__ void split(const uint4 &v, float (&f)[8]) {
    unpack8<std::conditional_t<std::is_same_v<L, __half>, F16, BF16>>(v, f);
}

template <class L>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
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

    // ---- The row into shared memory: one bulk copy a warp, of the whole 16-byte words that hold elements of the
    // row. Element i of the held row is element i - skew of the row: rows may start off the 16-byte grid.
    // 16-bit logits land in the upper half of the warp's part and spread over it from below.
    constexpr int EV = 16 / static_cast<int>(sizeof(L));
    const unsigned char *src = static_cast<const unsigned char *>(p.logits) + row * p.row_stride * static_cast<long long>(sizeof(L));
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(L));
    src -= skew * sizeof(L);
    const int end = p.V + skew, words = max(0, (min(PW, end - base) + EV - 1) / EV);
    const unsigned char *raw = reinterpret_cast<unsigned char *>(mine) + (4 - sizeof(L)) * PW;
    const uint32_t landed = smem_addr(&sh.landed[warp]);
    if (lane == 0) {
        mbar_init(landed, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(landed, words * 16);
        if (words > 0) bulk_load(smem_addr(raw), src + static_cast<size_t>(base) * sizeof(L), words * 16, landed);
    }
    if (tid < kTable) sh.pow[tid] = p.pow[tid];
    const float T = p.temperature ? __ldg(p.temperature + row) : 1.f;
    const bool greedy = !(T > 0.f);
    const int top_k = !greedy && p.top_k ? __ldg(p.top_k + row) : 0;
    const float pp = p.top_p ? __ldg(p.top_p + row) : 1.f, mp = p.min_p ? __ldg(p.min_p + row) : 0.f;
    const u64 least = mp > 0.f ? __float2ull_ru(fminf(mp, 1.f) * static_cast<float>(1ull << kFrac)) : 0;
    const float u = p.u ? __ldg(p.u + row) : 0.f;
    if (tid == kTable) {  // one thread: there are few 64-bit units
        const double c = 1.4426950408889634 / static_cast<double>(greedy ? 1.f : T < kCold ? T * kWarm : T);
        sh.ch = static_cast<float>(c);
        sh.cl = static_cast<float>(c - static_cast<double>(sh.ch));
    }

    __syncwarp();
    if (!mbar_wait(landed, 0)) {
        raise_err(p.err, PA_DEVERR_TIMEOUT);
        mbar_wait(landed, 0);  // the copy may still land: once more as long before the CTA can end
    }
    float mx = -INFINITY;
    int mx_at = lane * EV;  // where in `mine` this lane's first word with its maximum lies
#pragma unroll 2
    for (int i0 = 0; i0 < PW; i0 += 32 * EV) {
        const int i = i0 + lane * EV, at = base + i;
        const bool in = i < PW;
        float f[EV];
        if constexpr (EV == 4)
            split(*reinterpret_cast<const uint4 *>(raw + (in ? i : 0) * sizeof(L)), f);
        else
            split<L>(*reinterpret_cast<const uint4 *>(raw + (in ? i : 0) * sizeof(L)), f);
        if (at < skew || at + EV > end) {  // the row's first and last word, and what lies behind
#pragma unroll
            for (int e = 0; e < EV; ++e)
                if (at + e < skew || at + e >= end) f[e] = -INFINITY;
        }
        float m = -INFINITY;
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            f[e] = fmaxf(f[e], -INFINITY) + 0.f;  // NaN is never chosen; -0 equals 0
            m = fmaxf(m, f[e]);
        }
        if (in && m > mx) mx = m, mx_at = i;
        __syncwarp();  // the words have been read before they are written over
        if (in)
#pragma unroll
            for (int e = 0; e < EV; e += 4)
                *reinterpret_cast<float4 *>(mine + i + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        if constexpr (EV > 4) __syncwarp();
    }
    cluster.sync();  // the table is set, and every CTA of the cluster runs before another writes to it

    int turn = 0;
    // every CTA's reduction of v into every CTA of the cluster (mass[turn ^ 1] afterwards)
    auto exchange = [&](u64 v, auto reduce) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v = reduce(v, __shfl_xor_sync(kAll, v, o));
        if (lane == 0) sh.warp_mass[warp] = v;
        __syncthreads();
        if (warp == 0) {
            v = sh.warp_mass[lane % kWarps];
#pragma unroll
            for (int o = kWarps / 2; o; o >>= 1) v = reduce(v, __shfl_xor_sync(kAll, v, o));
            if (lane < CS) cluster.map_shared_rank(&sh, lane)->mass[turn][rank] = v;
        }
        cluster.sync();
        turn ^= 1;
        v = sh.mass[turn ^ 1][0];
        for (int i = 1; i < CS; ++i) v = reduce(v, sh.mass[turn ^ 1][i]);
        return v;
    };
    auto plus = [](u64 a, u64 b) { return a + b; };
    auto sum = [&](u64 v) { return exchange(v, plus); };
    // Two values from the one thread of the cluster with `from` to all (bcast[told ^ 1] afterwards); the lanes of
    // its warp write to a CTA each.
    int told = 0;
    auto tell = [&](bool from, u64 a, u64 b) {
        const unsigned who = __ballot_sync(kAll, from);
        if (who) {
            a = __shfl_sync(kAll, a, __ffs(who) - 1);
            b = __shfl_sync(kAll, b, __ffs(who) - 1);
            if (lane < CS) {
                Shared *to = cluster.map_shared_rank(&sh, lane);
                to->bcast[told][0] = a;
                to->bcast[told][1] = b;
            }
        }
        cluster.sync();
        told ^= 1;
    };
    // after a sum of f over the row: the held index at which the running sum of f first exceeds
    // `target` (below the whole). Found by one warp of the cluster, -1 elsewhere.
    auto locate = [&](u64 target, auto f) {
        int r = 0;
        for (; r < CS - 1 && target >= sh.mass[turn ^ 1][r]; ++r) target -= sh.mass[turn ^ 1][r];
        if (r != rank) return -1;
        int w = 0;
        for (; w < kWarps - 1 && target >= sh.warp_mass[w]; ++w) target -= sh.warp_mass[w];
        if (w != warp) return -1;
        // a stretch of the warp's elements per lane, then one stretch 32 elements at a time
        const int n = PW / 32;
        u64 s = 0;
#pragma unroll 4
        for (int i = lane * n; i < lane * n + n; ++i) s += f(mine[i], base + i);
        auto scan = [&](u64 v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(kAll, v, o);
                if (lane >= o) v += t;
            }
            return v;
        };
        const u64 upto = scan(s);
        const int l = __ffs(__ballot_sync(kAll, upto > target)) - 1;
        target -= __shfl_sync(kAll, upto - s, l);
        for (int i = l * n; i < l * n + n; i += 32) {
            const u64 v = scan(i + lane < l * n + n ? f(mine[i + lane], base + i + lane) : 0);
            const unsigned over = __ballot_sync(kAll, v > target);
            if (over) return base + i + __ffs(over) - 1;
            target -= __shfl_sync(kAll, v, 31);
        }
        return -1;
    };

    // ---- The largest logit, and a bound that no token of the top k lies below: with at least k groups
    // of elements, the k-th largest of the groups' maxima (what a warp holds) or the smallest (a lane).
    // Close to k elements lie above the former.
    const int full = end / PW, part = end % PW, lanes = min(32, PW / EV);
    const int warps_used = full + (part > 0), lanes_used = full * lanes + min(lanes, (part + EV - 1) / EV);
    {
        const bool in_use = lane < lanes && base + lane * EV < end;
        const uint32_t wmax = __reduce_max_sync(kAll, key_of(mx));
        const uint32_t lmin = __reduce_min_sync(kAll, in_use ? key_of(mx) : 0xffffffffu);
        if (lane < CS)
            cluster.map_shared_rank(&sh, lane)->warp_max[rank * kWarps + warp] = static_cast<u64>(wmax) << 32 | lmin;
        cluster.sync();
    }
    uint32_t kmax = 0, kmin = 0xffffffffu;
    for (int i = lane; i < CS * kWarps; i += 32) {
        kmax = max(kmax, static_cast<uint32_t>(sh.warp_max[i] >> 32));
        kmin = min(kmin, static_cast<uint32_t>(sh.warp_max[i]));
    }
    kmax = __reduce_max_sync(kAll, kmax);
    kmin = __reduce_min_sync(kAll, kmin);
    const bool short_list = top_k > 0 && top_k <= warps_used && top_k < p.V;
    if (short_list) {
        if (tid < CS * kWarps) {
            const u64 me = sh.warp_max[tid] >> 32;
            int above = 0;
#pragma unroll 8
            for (int i = 0; i < CS * kWarps; ++i) {
                const u64 o = sh.warp_max[i] >> 32;
                above += o > me || (o == me && i < tid);
            }
            if (above == top_k - 1) sh.kth = static_cast<uint32_t>(me);
        }
        if (tid == 0) sh.n_cand = 0;
        __syncthreads();
        kmin = sh.kth;
    }
    float k_bound = top_k <= lanes_used ? value_of(kmin) : -INFINITY;
    auto max_both = [](u64 a, u64 b) {  // of the halves, each by itself
        return max(a & 0xffffffff00000000ull, b & 0xffffffff00000000ull) | max(static_cast<uint32_t>(a), static_cast<uint32_t>(b));
    };
    Heat heat;
    heat.max = value_of(kmax);
    heat.ch = sh.ch, heat.cl = sh.cl;
    if (heat.max == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            raise_err(p.err, PA_DEVERR_ROW);
        }
        return;  // nothing of this CTA's memory is read or written by another after an exchange
    }

    if (greedy) {
        int at = 0;
        if (mx == heat.max)
            for (; mine[mx_at + at] != mx; ++at) {
            }
        const u64 first = exchange(mx == heat.max ? static_cast<uint32_t>(~(base + mx_at + at)) : 0u, max_both);
        if (rank == 0 && tid == 0) p.tokens[row] = static_cast<int>(~static_cast<uint32_t>(first)) - skew;
        return;
    }

    if (heat.max == INFINITY) {  // it takes all of the weight: the same as 0 among -infinity
        heat.max = 0.f;
        k_bound = -INFINITY;
        for (int i = lane; i < PW; i += 32) mine[i] = mine[i] == INFINITY ? 0.f : -INFINITY;
        __syncwarp();
    }

    if (T < kCold) {
        // A largest logit of at least 2^-20 is 2^-44 from every other, 2^18 octaves at this temperature: its equals
        // alone have weight. Below, scaling is exact but for logits that it takes to -infinity, without weight.
        const bool alone = fabsf(heat.max) >= 0x1p-20f;
        for (int i = lane; i < PW; i += 32)
            mine[i] = alone ? (mine[i] == heat.max ? 0.f : -INFINITY) : mine[i] * kWarm;
        heat.max = alone ? 0.f : heat.max * kWarm;
        k_bound = -INFINITY;
        __syncwarp();
    }

    // no logit below this has a weight (with room for rounding)
    const float floor_x = heat.max - 46.01f / heat.ch;
    // kept: logits above `tau`, and those equal to it up to held index `cut`
    float tau = -INFINITY;
    int cut = 0x7fffffff;
    auto kept = [&](float x, int at) { return x > tau || (x == tau && at <= cut); };
    // fn(logit, held index) of the kept elements in [lo, hi] that this lane takes of the warp's
    auto each = [&](float lo, float hi, auto fn) {
        lo = fmaxf(lo, tau);
#pragma unroll 2
        for (int i = lane * 4; i < PW; i += 128) {
            const float4 v = *reinterpret_cast<const float4 *>(mine + i);
            const float x[4] = {v.x, v.y, v.z, v.w};
            bool in[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) in[e] = x[e] >= lo && x[e] <= hi;
            if (!(in[0] | in[1] | in[2] | in[3])) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (in[e] && (x[e] > tau || base + i + e <= cut)) fn(x[e], base + i + e);
        }
    };
    // fn(four weights, four logits) of the kept elements from `lo` on, four together so that their
    // chains of dependent operations overlap; the others' weights are zero
    auto each_weight = [&](float lo, auto fn) {
        lo = fmaxf(lo, tau);
        for (int i = lane * 4; i < PW; i += 128) {
            const float4 v = *reinterpret_cast<const float4 *>(mine + i);
            float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = x[e] >= lo ? x[e] : -INFINITY;
            if (cut != 0x7fffffff)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (x[e] == tau && base + i + e > cut) x[e] = -INFINITY;
            if (fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) == -INFINITY) continue;
            u64 w[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) weight2(sh.pow, heat, x[e], x[e + 1], w[e], w[e + 1]);
            fn(w, x);
        }
    };
    auto one = [](float) { return 1ull; };
    auto weigh = [&](float x) { return weight(sh.pow, heat, x); };

    // Candidates: each CTA's own in sh.cand (n_cand of them, more than fit included) are joined in rank
    // 0's sh.joined if they all fit. Returns how many there are; the candidates of other CTAs have been
    // read only after another cluster-wide barrier.
    auto offer = [&](float x, int at, u64 f) {
        const uint32_t c = atomicAdd(&sh.n_cand, 1u);
        if (c < kCandidates) sh.cand[c] = Candidate{static_cast<u64>(key_of(x)) << 32 | static_cast<uint32_t>(~at), f};
    };
    auto join = [&]() {
        cluster.sync();
        // lane i: the candidates of CTA i, and of those before it
        const uint32_t c = lane < CS ? cluster.map_shared_rank(&sh, lane)->n_cand : 0;
        uint32_t upto = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += t;
        }
        const uint32_t n = __shfl_sync(kAll, upto, 31);
        const int from = tid % CS;  // the CTA whose candidates this thread fetches
        const uint32_t before_me = __shfl_sync(kAll, upto - c, from), theirs = __shfl_sync(kAll, c, from);
        if (rank == 0 && n <= kCandidates) {
            const Shared *other = cluster.map_shared_rank(&sh, from);
            for (uint32_t j = tid / CS; j < theirs; j += kSampleThreads / CS)
                sh.joined[before_me + j] = other->cand[j];
            __syncthreads();
        }
        return n;
    };
    // the sum of f over the n joined candidates that precede (two threads to each of them, both get it)
    auto before_in = [&](uint32_t n, auto precedes, auto f) {
        u64 s = 0;
        if (static_cast<uint32_t>(tid / 2) < n) {
            const u64 me = sh.joined[tid / 2].order;
#pragma unroll 4
            for (uint32_t j = tid % 2; j < n; j += 2) {
                const Candidate o = sh.joined[j];
                s += precedes(o.order, me) ? f(o) : 0;
            }
        }
        return s + __shfl_xor_sync(kAll, s, 1);
    };
    auto higher = [](u64 a, u64 b) { return a > b; };
    auto mass_of = [](const Candidate &c) { return c.f; };

    // Cuts the kept set to its shortest prefix, in descending order and lowest index first among
    // equals, whose sum of f is at least want(whole sum); f is 1 (kPiecesUsed 1) or the weight. No
    // element below `bound` is in that prefix (their part of the whole is then left out).
    auto cut_to = [&](auto pieces, auto f, auto want_of, float bound) {
        constexpr int kUsed = decltype(pieces)::value;
        // the bin of an element at this level: its distance from the maximum in 1 / 22 octaves, then the
        // 1024 parts of one of those; both are monotone in the logit
        int in_bin = -1;
        auto bin_of = [&](float x) {
            const float t = -octaves(heat, x) * kBinsPerOctave;
            const int b = static_cast<int>(fminf(t, static_cast<float>(kBins - 1)));
            if (in_bin < 0) return b;
            return b == in_bin ? static_cast<int>((t - static_cast<float>(b)) * kBins) : -1;
        };
        // bin b of CTA i
        auto bin_sum = [&](int i, int b) {
            const Shared *from = cluster.map_shared_rank(&sh, i);
            u64 v = from->hist[0][b];
            if constexpr (kUsed > 1)
                v += (static_cast<u64>(from->hist[1][b]) << kPieceBits) +
                     (static_cast<u64>(from->hist[2][b]) << (2 * kPieceBits));
            return v;
        };
        // the logits of a bin: between its borders (with room for rounding); bin_of decides
        float lo = fmaxf(bound, kUsed > 1 ? floor_x : -INFINITY), hi = INFINITY;
        auto narrow = [&](float t0, float t1) {
            const float per_bin = 1.f / (kBinsPerOctave * heat.ch);
            lo = fmaxf(lo, heat.max - (t1 + t1 * 1e-5f) * per_bin);
            hi = fminf(hi, heat.max - (t0 - t0 * 1e-5f) * per_bin + fabsf(heat.max) * 1e-6f);
            lo -= fabsf(heat.max) * 1e-6f;
        };
        u64 above = 0, want = 0;
        int bin = 0;
        for (int level = 0; level < 2; ++level) {
            for (int i = tid; i < kBins; i += kSampleThreads)
                for (int j = 0; j < kUsed; ++j) sh.hist[j][i] = 0;
            if (tid == 0) sh.n_cand = 0;
            __syncthreads();
            auto add = [&](int b, u64 w) {
                constexpr uint32_t kMask = (1u << kPieceBits) - 1;
                atomicAdd(&sh.hist[0][b], static_cast<uint32_t>(w) & kMask);
                atomicAdd(&sh.hist[1][b], static_cast<uint32_t>(w >> kPieceBits) & kMask);
                const uint32_t top = static_cast<uint32_t>(w >> (2 * kPieceBits));
                if (top) atomicAdd(&sh.hist[2][b], top);
            };
            if (kUsed == 1 || level > 0) {
                each(lo, hi, [&](float x, int) {
                    const int b = bin_of(x);
                    if (b < 0 || (level == 0 && b == kBins - 1)) return;
                    if constexpr (kUsed == 1)
                        atomicAdd(&sh.hist[0][b], 1u);
                    else
                        add(b, f(x));
                });
            } else {
                each_weight(lo, [&](const u64(&w)[4], const float(&x)[4]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (w[e]) add(bin_of(x[e]), w[e]);
                });
            }
            cluster.sync();
            // Each CTA joins a slice of the bins: its threads read along the bins, each group of
            // threads two CTAs' parts (a CTA by itself: two bins a thread)
            const int per = kBins / CS;
            u64 v = 0;
            if (CS == 1) {
                v = bin_sum(0, 2 * tid) + bin_sum(0, 2 * tid + 1);
            } else {
                u64 *parts = reinterpret_cast<u64 *>(sh.joined);
                const int b = rank * per + tid % per, c = 2 * (tid / per);
                parts[tid] = bin_sum(c, b) + bin_sum(c + 1, b);
                __syncthreads();
                if (tid < per)
                    for (int j = tid; j < kSampleThreads; j += per) v += parts[j];
            }
            const u64 whole = sum(v);
            if (level == 0) want = want_of(whole);
            if (whole < want && level == 0) return;  // it ends in the last bin: every token with weight stays
            // the bin in which the running sum reaches want
            u64 before = above;
            for (int i = 0; i < rank; ++i) before += sh.mass[turn ^ 1][i];
            u64 incl = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += t;
            }
            for (int w = 0; w < warp; ++w) before += sh.warp_mass[w];
            before += incl - v;
            const bool here = v > 0 && before < want && want <= before + v;
            int b = CS == 1 ? 2 * tid : rank * per + tid;
            u64 held = v;
            if (here && CS == 1) {
                held = bin_sum(0, b);
                if (want > before + held) before += held, held = v - held, ++b;
            }
            // how many elements it holds: its sum over the weight in its middle
            float count = static_cast<float>(held);
            auto border = [&](int b) {  // in bins of the first level
                return level == 0 ? static_cast<float>(b) : static_cast<float>(in_bin) + static_cast<float>(b) * (1.f / kBins);
            };
            if (kUsed > 1) count *= fast_exp2((border(b) + border(b + 1)) * (0.5f / kBinsPerOctave) - kFrac);
            tell(here, static_cast<u64>(__float2uint_rn(count)) << 32 | static_cast<uint32_t>(b), before);
            bin = static_cast<int>(sh.bcast[told ^ 1][0] & 0xffffffffu);
            const bool few = sh.bcast[told ^ 1][0] >> 32 <= kCandidates;
            above = sh.bcast[told ^ 1][1];
            narrow(border(bin), border(bin + 1));
            if (few) {
                // its elements to rank 0
                each(lo, hi, [&](float x, int at) {
                    if (bin_of(x) == bin) offer(x, at, f(x));
                });
                const uint32_t n = join();
                if (n <= kCandidates) {
                    bool last = false;
                    Candidate c{};
                    if (rank == 0) {
                        const u64 s = above + before_in(n, higher, mass_of);
                        if (static_cast<uint32_t>(tid / 2) < n) c = sh.joined[tid / 2];
                        last = static_cast<uint32_t>(tid / 2) < n && tid % 2 == 0 && s < want && want <= s + c.f;
                    }
                    tell(last, c.order, 0);
                    tau = value_of(static_cast<uint32_t>(sh.bcast[told ^ 1][0] >> 32));
                    cut = static_cast<int>(~static_cast<uint32_t>(sh.bcast[told ^ 1][0]));
                    return;
                }
                cluster.sync();  // the counts have been read
            }
            if (level == 0) in_bin = bin;
        }
        // Many elements within 2^-10 of a bin, most often equals (16-bit logits): a binary search over
        // the keys in it
        uint32_t part_min = 0xffffffffu, part_max = 0;
        each(lo, hi, [&](float x, int) {
            if (bin_of(x) != bin) return;
            part_min = min(part_min, key_of(x));
            part_max = max(part_max, key_of(x));
        });
        const u64 ends = exchange(static_cast<u64>(part_max) << 32 | static_cast<uint32_t>(~part_min), max_both);
        uint32_t klo = ~static_cast<uint32_t>(ends), khi = static_cast<uint32_t>(ends >> 32);
        u64 more = above;    // the sum above klo
        while (klo < khi) {  // the largest key t with sum(>= t) >= want
            const uint32_t mid = klo + (khi - klo) / 2 + 1;
            u64 m = 0;
            each(value_of(mid), hi, [&](float x, int) {
                if (bin_of(x) == bin) m += f(x);
            });
            m = above + sum(m);
            if (m >= want)
                klo = mid;
            else
                khi = mid - 1, more = m;
        }
        const float last = value_of(klo);
        auto equal = [&](float x, int at) { return static_cast<u64>(x == last && kept(x, at)); };
        u64 c = 0;
        each(last, last, [&](float, int) { ++c; });
        const u64 equals = sum(c), weight_each = f(last);
        const u64 r = weight_each ? (want - more + weight_each - 1) / weight_each : equals;  // of the equals, the first r
        if (r < equals) {
            const int at = locate(r - 1, equal);
            tell(at >= 0 && lane == 0, static_cast<u64>(at), 0);
            cut = static_cast<int>(sh.bcast[told ^ 1][0]);
        } else if (last != tau) {
            cut = 0x7fffffff;  // all of them
        }
        tau = last;
    };

    // floor and ceiling of x * m for x in [0, 1), exact to 2^-64 of m
    auto down = [](float x, u64 m) { return __umul64hi(__float2ull_rz(x * 18446744073709551616.f), m); };
    auto up = [](float x, u64 m) {
        const u64 f = __float2ull_rz(x * 18446744073709551616.f);
        return __umul64hi(f, m) + (f * m != 0);
    };
    auto target_of = [&](u64 whole) { return u >= 1.f ? whole - 1 : u > 0.f ? down(u, whole) : 0; };
    // kept by top-p while the sum before a token is below pp of the whole
    auto want_of = [&](u64 whole) { return max(up(fmaxf(pp, 0.f), whole), 1ull); };

    if (short_list) {
        // the top k and a few more, all at rank 0: the rest is decided among them
        each(k_bound, INFINITY, [&](float x, int at) { offer(x, at, weigh(x)); });
        const uint32_t n = join();
        if (n <= kCandidates) {
            cluster.sync();  // the other CTAs' candidates have been read
            if (rank != 0) return;
            const uint32_t i = tid / 2;
            const bool first = i < n && tid % 2 == 0;  // one thread a candidate writes
            auto set = [&](bool stays) {  // the others weigh nothing from here on
                __syncthreads();
                if (first && !stays) sh.joined[i].f = 0;
                __syncthreads();
            };
            auto whole_of = [&]() {
                u64 s = 0;
                for (uint32_t j = lane; j < n; j += 32) s += sh.joined[j].f;
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
                return s;
            };
            set(before_in(n, higher, [](const Candidate &) { return 1ull; }) < static_cast<u64>(top_k));
            if (pp < 1.f) {
                const u64 want = want_of(whole_of());
                set(before_in(n, higher, mass_of) < want);
            }
            if (least) set(i < n && sh.joined[i].f >= least);
            const u64 target = target_of(whole_of());
            const u64 s = before_in(n, [](u64 a, u64 b) { return static_cast<uint32_t>(a) > static_cast<uint32_t>(b); }, mass_of);
            if (first && s <= target && target < s + sh.joined[i].f)
                p.tokens[row] = static_cast<int>(~static_cast<uint32_t>(sh.joined[i].order)) - skew;
            return;
        }
        cluster.sync();  // the counts have been read
    }
    if (top_k > 0 && top_k < p.V)
        cut_to(std::integral_constant<int, 1>{}, one, [&](u64) { return static_cast<u64>(top_k); }, k_bound);
    if (pp < 1.f) cut_to(std::integral_constant<int, kPieces>{}, weigh, want_of, -INFINITY);

    // ---- the kept sum, and the token
    // no logit below this is kept: min-p's border with room for rounding
    const float from = fmaxf(tau, mp > 0.f ? heat.max + fminf((__log2f(fminf(mp, 1.f)) - 0.01f) / heat.ch, 0.f) : floor_x);
    auto share = [&](float x, int at) {  // without branches, so that several run at a time
        const u64 w = weight(sh.pow, heat, x >= from && kept(x, at) ? x : -INFINITY);
        return w >= least ? w : static_cast<u64>(0);
    };
    u64 m = 0;
    if (least)
        each_weight(from, [&](const u64(&w)[4], const float(&)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) m += w[e] >= least ? w[e] : 0;
        });
    else
        each_weight(from, [&](const u64(&w)[4], const float(&)[4]) { m += (w[0] + w[1]) + (w[2] + w[3]); });
    const u64 whole = sum(m);
    const u64 target = target_of(whole);
    const int at = locate(target, share);
    if (at >= 0 && lane == 0) p.tokens[row] = at - skew;
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
    // A CTA for every 4096 elements of a row, up to eight (256 rows of 151,936 fp32 with settings of every kind: 148 us,
    // with clusters of four 174, of sixteen 245; greedy rows 50, 46 and 106); sixteen where that still leaves half
    // of the SMs idle (top-p, one row: 22 us against 29 with eight, four rows 28 against 37). Five to nine rows
    // would gain from sixteen too (28-34 us against 37), 16 rows not (51 against 43).
    int CS = 1;
    while (CS < 8 && a.V > 4096 * CS) CS *= 2;
    const bool few = a.V > 4096 * 8 && a.B * 16 <= device_sm_count() / 2;
    for (int k = -16; k <= 16; ++k) {
        const double v = std::exp2(k / 32.0);
        prm.pow[k & (kTable - 1)] = Pow{static_cast<uint32_t>(v * 2147483648.0 + 0.5), static_cast<float>(v * 2147483648.0)};
    }
    auto kern = sample_kernel<L>;
    static int configured[64] = {0}, sixteen[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448)) != cudaSuccess)
            return e;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        configured[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kSampleThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto divide = [&](int V, int ctas) {
        const int held = V + 16 / static_cast<int>(sizeof(L)) - 1;  // the row and the skew of its start
        prm.per_warp = (held + ctas * kWarps * 32 - 1) / (ctas * kWarps * 32) * 32;
        attr[0].val.clusterDim.x = ctas;
        cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
        cfg.dynamicSmemBytes = sizeof(Shared) + static_cast<size_t>(kWarps) * prm.per_warp * 4;
    };
    if (few) {  // clusters of sixteen, where the device has room for one with the longest rows (asked once)
        if (sixteen[dev] == 0) {
            int n = 0;
            divide(kSampleMaxVocab, 16);
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) cudaGetLastError();  // that answer is not the launch's
            sixteen[dev] = e == cudaSuccess && n > 0 ? 1 : -1;
        }
        if (sixteen[dev] > 0) CS = 16;
    }
    divide(a.V, CS);
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    if (a.dtype == PA_F32) return launch_typed<float>(a, stream);
    return a.dtype == PA_BF16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<__half>(a, stream);
}

}  // namespace pa
