// logprobs.cu -- log probabilities of given tokens, entropy and the likeliest
// tokens of every row of logits in one pass over them, and their gradient.
//
// With z the row, m = max z, S = sum exp(z - m):
//   log p(t) = (z_t - m) - log S        entropy H = log S - sum (z - m) exp(z - m) / S
//   d logits = g (onehot(t) - p) - h p (log p + H)   for d log p(t) = g, d H = h
//
// Forward (k_logprobs): a cluster of 1 to 8 CTAs per row, each reading a
// contiguous share of the row's 16-byte vectors once.  A thread keeps a running
// maximum, S and the weighted sum in fp32 in base 2: with L = log2(e) and
// r = rn(m L), e = 2^(z L - r) is one fused multiply-add and one exponential;
// that r is a rounded m L scales every e by the same 2^(m L - r), which the
// row's end takes back out.  The likeliest tokens cost nothing during the pass: the
// k-th largest of the threads' maxima is a lower bound of the k-th largest element,
// and only the (about k of 256) threads whose maximum reaches it hold elements that
// do.  Their elements alone are read again (out of L2) and those at or above the
// bound are listed as keys (value, ~index).  A key's place in the answer is the
// number of larger keys, so ties go to the lowest index and the order of the list
// does not matter.  Rows of many equal values overflow the list and are gone through
// once more with a rising threshold.
//
// m L is rounded by up to 2^-24 of itself, so rows whose maximum is beyond +-1e8 (masks of
// a huge value everywhere) would leave fp32's range by 2^(m L - r) and take a
// second pass with z - m first.  All -inf: log p = -inf, H = 0.  NaN or +inf in a row: NaN, and no tokens (-1).
//
// Backward (k_logprobs_bwd): elementwise, one read and one write; the rows of
// the output may be aligned differently from those of the input, in which case a
// thread joins two aligned vectors of the input into one of the output.  Both go past
// the caches as streams.
//
// What bounds them, 2048 x 128256 bf16: the gradient HBM (159 to 164 us, as long as a copy of the same bytes takes).
// The forward 98 us without alternatives (a read at the copy's rate: 81) and 116 with 8: the pass loads an
// iteration's vectors only when it has used the last (37% of the warps' time is waiting for loads; DRAM 59%, the
// exponentials' pipe 57%), and a row's listing and ranking follow behind barriers.  One row: 5 us, and
// 5 more for ranking 20 tokens.
#include "common.cuh"
#include "lut.cuh"
#include "tc.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sherry {

constexpr int kLpThreads = 256;
constexpr int kLpVecs = 4;       // 16-byte vectors per thread and iteration
constexpr int kLpCap = 1024;     // candidate keys held
constexpr int kLpRefine = 96;    // keys beyond the wanted ones that make a cut worth its pass
constexpr int kLpMaxTop = SHERRY_MAX_TOP;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kEdge = 1e8f;    // row maxima beyond this: 2^(m L - r), up to 2^9 here, would leave fp32's range
static_assert(8 * kLpMaxTop <= kLpCap, "the cluster's best fit the list");
static_assert(kLpMaxTop <= 32, "the first threshold is a bound of the 32nd largest");

struct LpParams {
    const void* z;
    int64_t ld;
    const int32_t* targets;
    float* logp;
    float* entropy;
    float* stats;
    float* top_logp;
    int32_t* top_ids;
    int V, top;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// r = rn(m L): the product must be rounded by itself everywhere, never inside a fused multiply-add
__device__ __forceinline__ float ref_of(float m) { return __fmul_rn(fmaxf(m, -kEdge), kLog2e); }

// two floats side by side: one instruction for both
__device__ __forceinline__ uint64_t pair(float x, float y) {
    return ((uint64_t)__float_as_uint(y) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ float lo_of(uint64_t p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float hi_of(uint64_t p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Elements below kFloor count as kFloor: 0 * -inf would be NaN in the weighted sum, while 2^(kFloor L - r)
// is 0 for every r of a row that is not at the edge (its maximum is above -kEdge), and kFloor L - r finite.
constexpr float kFloor = -2e8f;

template <typename T>
struct LpVec;
template <>
struct LpVec<__nv_bfloat16> {
    static constexpr int N = 8;
    // the largest element (NaN only where all are)
    static __device__ __forceinline__ float max(uint4 v) {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(bf16lo(m), bf16hi(m));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // the elements as pairs, raised to kFloor (NaN stays)
    static __device__ __forceinline__ void pairs(uint4 v, uint64_t* p) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(w[i]), "r"(0xcd3fcd3fu));  // bf16(kFloor)
            p[i] = pair(bf16lo(c), bf16hi(c));
        }
    }
    static __device__ __forceinline__ void unpack(uint4 v, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo(w[i]);
            f[2 * i + 1] = bf16hi(w[i]);
        }
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ __nv_bfloat16 round(float f) { return __float2bfloat16_rn(f); }
    static __device__ __forceinline__ uint32_t pad() { return 0xff80ff80u; }  // two -inf
};
template <>
struct LpVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float max(uint4 v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ void pairs(uint4 v, uint64_t* p) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %1, %2;" : "=f"(c[i]) : "f"(__uint_as_float(w[i])), "f"(kFloor));
        p[0] = pair(c[0], c[1]);
        p[1] = pair(c[2], c[3]);
    }
    static __device__ __forceinline__ void unpack(uint4 v, float* f) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float round(float f) { return f; }
    static __device__ __forceinline__ uint32_t pad() { return 0xff800000u; }
};

// order-preserving bits of a float; -0 and +0 are one value
__device__ __forceinline__ uint32_t lp_order(float z) {
    const uint32_t u = __float_as_uint(z + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float lp_unorder(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}
__device__ __forceinline__ uint64_t lp_key(float z, int i) { return ((uint64_t)lp_order(z) << 32) | (uint32_t)~i; }

// One vector of the row whose first element is `e0` (may be negative, or reach past
// the row: those elements read as -inf).
template <typename T>
__device__ __forceinline__ uint4 lp_load(const T* row, int e0, int V) {
    constexpr int N = LpVec<T>::N;
    if (e0 >= 0 && e0 + N <= V) return *reinterpret_cast<const uint4*>(row + e0);
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = (e0 + j >= 0 && e0 + j < V) ? LpVec<T>::one(row + e0 + j) : -INFINITY;
    return LpVec<T>::pack(f);
}

template <int TH>
struct LpTop {  // shared state of the likeliest tokens
    float tmax[TH];    // the threads' maxima
    static constexpr int kCap = kLpCap / kLpThreads * TH;  // candidate keys held
    uint64_t buf[kCap];
    uint64_t best[kLpMaxTop];
    uint64_t thr;
    uint8_t list[TH];  // threads that hold candidates
    int cnt, listed;
};

// The `k` largest of buf[0..n), in order, into best (0 where there are fewer).
template <int TH>
__device__ __forceinline__ void lp_rank(LpTop<TH>& s, int n, int k) {
    if ((int)threadIdx.x < k) s.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += TH) {
        const uint64_t me = s.buf[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += s.buf[j] > me;
        if (r < k) s.best[r] = me;
    }
    __syncthreads();
}

// Append a vector's keys at or above the threshold; elements [0, hi) of the row count.
template <typename T, int TH>
__device__ __forceinline__ void lp_push(LpTop<TH>& s, uint4 x, int e0, int hi, uint64_t thr, float tv) {
    float f[LpVec<T>::N];
    LpVec<T>::unpack(x, f);
#pragma unroll
    for (int j = 0; j < LpVec<T>::N; ++j) {
        const int e = e0 + j;
        if (f[j] >= tv && e >= 0 && e < hi) {
            const uint64_t key = lp_key(f[j], e);
            if (key >= thr) {
                const int at = atomicAdd(&s.cnt, 1);
                if (at < LpTop<TH>::kCap) s.buf[at] = key;
            }
        }
    }
}

// Append one iteration's keys, after which the list is whole: where more keys pass than it holds,
// the threshold rises to the k-th best of those held (each is in the row, so that is a bound) and
// the iteration's are appended again.  A long list is cut back to its best.  Called by all threads.
template <typename T, int TH>
__device__ __noinline__ void lp_collect(LpTop<TH>& s, const uint4 (&xs)[kLpVecs], int v, int v1, int off, int V, int k) {
    constexpr int N = LpVec<T>::N;
    const int held = s.cnt;
    __syncthreads();
    while (true) {
        const uint64_t thr = s.thr;
        const float tv = lp_unorder((uint32_t)(thr >> 32));
        for (int u = 0; u < kLpVecs; ++u)
            if (v + u * TH < v1 && LpVec<T>::max(xs[u]) >= tv)
                lp_push<T, TH>(s, xs[u], off + N * (v + u * TH), V, thr, tv);
        __syncthreads();
        const int n = s.cnt;
        const bool over = n > LpTop<TH>::kCap;
        if (over || n > k + kLpRefine) {
            lp_rank(s, min(n, LpTop<TH>::kCap), k);
            if (threadIdx.x == 0) {
                s.thr = max(s.thr, s.best[k - 1]);
                s.cnt = over ? held : k;
            }
            if (!over && (int)threadIdx.x < k) s.buf[threadIdx.x] = s.best[threadIdx.x];
        }
        __syncthreads();
        if (!over) return;
    }
}

// TH threads per CTA
template <typename T, bool TOP, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) k_logprobs(const LpParams P) {
    constexpr int N = LpVec<T>::N;
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t rowi = blockIdx.x / C;
    const T* row = reinterpret_cast<const T*>(P.z) + rowi * P.ld;
    const int V = P.V, top = TOP ? P.top : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    __shared__ typename std::conditional<TOP, LpTop<TH>, int>::type top_s;
    __shared__ float4 red[TH / 32];  // the warps' maxima, S, weighted sums
    __shared__ float4 part;                  // this CTA's

    // the row's 16-byte vectors: vector v holds elements off + N v ..; this CTA's share is [v0, v1)
    const int off = -(int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int nv = (V - off + N - 1) / N;
    const int share = (nv + C - 1) / C;
    const int v0 = min(rank * share, nv), v1 = min(v0 + share, nv);
    const int iters = (v1 - v0 + TH * kLpVecs - 1) / (TH * kLpVecs);

    auto fetch = [&](int it, uint4* x) {
#pragma unroll
        for (int u = 0; u < kLpVecs; ++u) {
            const int v = v0 + (it * kLpVecs + u) * TH + tid;
            x[u] = v < v1 ? lp_load(row, off + N * v, V)
                          : make_uint4(LpVec<T>::pad(), LpVec<T>::pad(), LpVec<T>::pad(), LpVec<T>::pad());
        }
    };

    // the target's logit is fetched beside the pass
    int target = -1;
    float zt = 0.0f;
    if (tid == 0 && rank == 0 && P.logp) {
        target = P.targets[rowi];
        if (target >= 0 && target < V) zt = LpVec<T>::one(row + target);
    }
    float m = -INFINITY, r = ref_of(-INFINITY);
    uint64_t a1 = 0, a2 = 0;  // S and the weighted sum, of even and odd elements
    const uint64_t L2 = pair(kLog2e, kLog2e);
    uint4 x[kLpVecs];
    for (int it = 0; it < iters; ++it) {
        fetch(it, x);
        float bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kLpVecs; ++u) bm = fmaxf(bm, LpVec<T>::max(x[u]));
        if (bm > m) {
            const float nr = ref_of(bm);
            const float d = fmaxf(r - nr, -1e4f), f = ex2(d);
            const uint64_t f2 = pair(f, f);
            a2 = fma2(f2, fma2(pair(d, d), a1, a2), 0);
            a1 = fma2(f2, a1, 0);
            m = bm;
            r = nr;
        }
        const uint64_t mr = pair(-r, -r);
#pragma unroll
        for (int u = 0; u < kLpVecs; ++u) {
            uint64_t p[N / 2];
            LpVec<T>::pairs(x[u], p);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const uint64_t y = fma2(p[j], L2, mr);
                const uint64_t e = pair(ex2(lo_of(y)), ex2(hi_of(y)));
                a1 = add2(a1, e);
                a2 = fma2(e, y, a2);
            }
        }
    }
    float s1 = lo_of(a1) + hi_of(a1), s2 = lo_of(a2) + hi_of(a2);
    if constexpr (TOP) {
        // a value that k of the threads' maxima reach bounds the k-th largest element from below, and
        // only threads whose maximum reaches it hold an element that does
        top_s.tmax[tid] = m;
        if (tid == 0) top_s.cnt = top_s.listed = 0;
        __syncthreads();
        if (warp == 0) {
            // the largest value of 16 leading bits that at least k of the maxima reach, bit by bit
            uint32_t o[TH / 32], t = 0;
#pragma unroll
            for (int j = 0; j < TH / 32; ++j) o[j] = lp_order(top_s.tmax[lane + 32 * j]);
#pragma unroll
            for (int bit = 31; bit >= 16; --bit) {
                const uint32_t want = t | (1u << bit);
                int n = 0;
#pragma unroll
                for (int j = 0; j < TH / 32; ++j) n += o[j] >= want;
                if (__reduce_add_sync(kFull, n) >= top) t = want;
            }
            if (lane == 0) top_s.thr = (uint64_t)max(t, lp_order(-INFINITY)) << 32;  // (below -inf: NaNs)
        }
        __syncthreads();
        const uint64_t thr = top_s.thr;
        const float tv = lp_unorder((uint32_t)(thr >> 32));
        if (m >= tv) top_s.list[atomicAdd(&top_s.listed, 1)] = (uint8_t)tid;
        __syncthreads();
        const int per = iters * kLpVecs, total = top_s.listed * per;
        for (int i = tid; i < total; i += TH) {
            const int v = v0 + (i % per) * TH + top_s.list[i / per];
            if (v < v1) {
                const uint4 y = lp_load(row, off + N * v, V);
                if (LpVec<T>::max(y) >= tv) lp_push<T, TH>(top_s, y, off + N * v, V, thr, tv);
            }
        }
        __syncthreads();
        if (top_s.cnt > LpTop<TH>::kCap) {  // (uniform) many equal values: again, with the threshold rising
            __syncthreads();
            if (tid == 0) top_s.cnt = 0;
            __syncthreads();
            for (int it = 0; it < iters; ++it) {
                uint4 cx[kLpVecs];  // (not x: what a call takes by address leaves the registers)
                fetch(it, cx);
                lp_collect<T, TH>(top_s, cx, v0 + it * kLpVecs * TH + tid, v1, off, V, top);
            }
        }
        lp_rank(top_s, top_s.cnt, top);
    }

    // the row's sums: threads of a warp, warps of the CTA, CTAs of the cluster, in order
    auto rebase = [](float& a, float& b, float from, float to) {  // sums relative to `from`, now to `to`
        const float d = fmaxf(from - to, -1e4f), f = ex2(d);
        b = f * fmaf(d, a, b);
        a *= f;
    };
    float bmax = m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) bmax = fmaxf(bmax, __shfl_xor_sync(kFull, bmax, o));
    rebase(s1, s2, r, ref_of(bmax));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        s1 += __shfl_xor_sync(kFull, s1, o);
        s2 += __shfl_xor_sync(kFull, s2, o);
    }
    if (lane == 0) red[warp] = make_float4(bmax, s1, s2, 0.0f);
    __syncthreads();
    auto join = [&](auto get, int n) {  // (maximum, sums) of n parts
        float4 q = get(0);
        bmax = q.x;
        for (int i = 1; i < n; ++i) bmax = fmaxf(bmax, get(i).x);
        s1 = s2 = 0.0f;
        for (int i = 0; i < n; ++i) {
            q = get(i);
            rebase(q.y, q.z, ref_of(q.x), ref_of(bmax));
            s1 += q.y;
            s2 += q.z;
        }
    };
    join([&](int i) { return red[i]; }, TH / 32);
    if (C > 1) {
        if (tid == 0) part = make_float4(bmax, s1, s2, 0.0f);
        cluster.sync();
        join([&](int i) { return *cluster.map_shared_rank(&part, i); }, C);
    }
    float ref = ref_of(bmax);
    const bool edge = bmax > kEdge || (bmax < -kEdge && bmax != -INFINITY);
    if (edge) {
        // m log2(e) overflows: this row again, with z - m first
        s1 = s2 = 0.0f;
        for (int v = v0 + tid; v < v1; v += TH) {
            float f[N];
            LpVec<T>::unpack(lp_load(row, off + N * v, V), f);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float y = (f[j] - bmax) * kLog2e;
                const float e = ex2(y);
                s1 += e;
                s2 = fmaf(e, fmaxf(y, -1e4f), s2);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            s1 += __shfl_xor_sync(kFull, s1, o);
            s2 += __shfl_xor_sync(kFull, s2, o);
        }
        __syncthreads();
        if (lane == 0) red[warp] = make_float4(0.0f, s1, s2, 0.0f);
        __syncthreads();
        s1 = s2 = 0.0f;
        for (int w = 0; w < TH / 32; ++w) {
            s1 += red[w].y;
            s2 += red[w].z;
        }
        if (C > 1) {
            cluster.sync();
            if (tid == 0) part = make_float4(0.0f, s1, s2, 0.0f);
            cluster.sync();
            s1 = s2 = 0.0f;
            for (int c = 0; c < C; ++c) {
                const float4 q = *cluster.map_shared_rank(&part, c);
                s1 += q.y;
                s2 += q.z;
            }
        }
    }
    if (rank == 0) {
        // log S relative to the true maximum: S was summed relative to ref = rn(m L)
        const bool dead = bmax == -INFINITY, bad = !(s1 < INFINITY);
        // (S holds a 1, so its logarithm is not below 0: rounding must not make a probability above 1)
        float lsum = fmaxf(logf(s1) + (edge ? 0.0f : fmaf(-bmax, kLog2e, ref) * kLn2), 0.0f);
        if (dead) lsum = 0.0f;
        if (bad) lsum = NAN;
        if (tid == 0) {
            if (P.logp) {
                float lp = 0.0f;
                if (target >= 0 && target < V)
                    lp = bad ? NAN : (dead || zt == -INFINITY) ? -INFINITY : (zt - bmax) - lsum;
                P.logp[rowi] = lp;
            }
            if (P.entropy)
                P.entropy[rowi] = bad ? NAN : dead ? 0.0f : fmaxf(logf(s1) - s2 / s1 * kLn2, 0.0f);
            P.stats[2 * rowi] = bad ? NAN : bmax;
            P.stats[2 * rowi + 1] = lsum;
        }
        if constexpr (TOP) {
            // every CTA's best, brought here; a key's place is the number of larger ones
            const int all = C * top;
            __syncthreads();
            for (int i = tid; i < all; i += TH)
                top_s.buf[i] = cluster.map_shared_rank(&top_s.best[0], i / top)[i % top];
            __syncthreads();
            for (int i = tid; i < all; i += TH) {
                const uint64_t me = top_s.buf[i];
                int place = 0;
#pragma unroll 4
                for (int j = 0; j < all; ++j) place += top_s.buf[j] > me;
                if (me != 0 && place < top && !bad) {
                    const float zt = lp_unorder((uint32_t)(me >> 32));
                    P.top_ids[rowi * top + place] = (int32_t)~(uint32_t)me;
                    P.top_logp[rowi * top + place] = (dead || zt == -INFINITY) ? -INFINITY : (zt - bmax) - lsum;
                }
            }
            if (bad) {
                for (int i = tid; i < top; i += TH) {
                    P.top_ids[rowi * top + i] = -1;
                    P.top_logp[rowi * top + i] = NAN;
                }
            }
        }
    }
    if (C > 1) cluster.sync();  // the others' shared memory is read until here
}

// ---- backward --------------------------------------------------------------------

struct LpBwdParams {
    const void* z;
    int64_t ld;
    const int32_t* targets;
    const float* stats;
    const float* entropy;
    const float* dlogp;
    const float* dentropy;
    void* out;
    int64_t ldo;
    int V, segs;
};

constexpr int kLpBwdVecs = 4;

// the 16 bytes that start `shift` bytes into the 32 bytes (a, b); shift is the same for the whole row
__device__ __forceinline__ uint4 lp_join(uint4 a, uint4 b, int shift) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int bits = (shift & 3) * 8;
    uint32_t o[5];
    switch (shift >> 2) {
        case 0:
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = w[i];
            break;
        case 1:
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = w[i + 1];
            break;
        case 2:
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = w[i + 2];
            break;
        default:
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = w[i + 3];
            break;
    }
    return make_uint4(__funnelshift_r(o[0], o[1], bits), __funnelshift_r(o[1], o[2], bits),
                      __funnelshift_r(o[2], o[3], bits), __funnelshift_r(o[3], o[4], bits));
}

template <typename T, int TH>
__global__ void __launch_bounds__(TH) k_logprobs_bwd(const LpBwdParams P) {
    constexpr int N = LpVec<T>::N;
    pdl_wait();
    const int64_t rowi = blockIdx.x / P.segs;
    const int seg = (int)(blockIdx.x % P.segs);
    const T* row = reinterpret_cast<const T*>(P.z) + rowi * P.ld;
    T* out = reinterpret_cast<T*>(P.out) + rowi * P.ldo;
    const int V = P.V;
    // vectors of the output: vector v holds elements off + N v ..; in the input they
    // start `shift` bytes past an aligned vector
    const int off = -(int)((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T));
    const int shift = (int)(((reinterpret_cast<uintptr_t>(row) & 15u) + 16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u);
    const int nv = (V - off + N - 1) / N;
    const int vb = seg * (TH * kLpBwdVecs) + threadIdx.x;

    uint4 x[kLpBwdVecs];
#pragma unroll
    for (int u = 0; u < kLpBwdVecs; ++u) {
        const int v = vb + u * TH;
        const int e0 = off + N * v;
        const int lead = shift / (int)sizeof(T);
        if (v < nv) {
            if (shift == 0) {
                x[u] = (e0 >= 0 && e0 + N <= V) ? __ldcs(reinterpret_cast<const uint4*>(row + e0)) : lp_load(row, e0, V);
            } else if (e0 - lead >= 0 && e0 - lead + 2 * N <= V) {
                const uint4* p = reinterpret_cast<const uint4*>(row + e0 - lead);
                x[u] = lp_join(p[0], p[1], shift);
            } else {
                float f[N];
#pragma unroll
                for (int j = 0; j < N; ++j)
                    f[j] = (e0 + j >= 0 && e0 + j < V) ? LpVec<T>::one(row + e0 + j) : -INFINITY;
                x[u] = LpVec<T>::pack(f);
            }
        }
    }
    float m = P.stats[2 * rowi], lsum = P.stats[2 * rowi + 1];
    const int t0 = P.targets ? P.targets[rowi] : -1;
    const int t = (t0 >= 0 && t0 < V) ? t0 : -1;
    const bool dead = m == -INFINITY;
    if (dead) m = 0.0f, lsum = INFINITY;  // every p is 0
    const float g = (t < 0 || dead) ? 0.0f : P.dlogp[rowi];
    const float h = P.dentropy ? P.dentropy[rowi] : 0.0f;
    const float H = P.dentropy ? P.entropy[rowi] : 0.0f;
    if (t < 0 && h == 0.0f) {  // left out: zeros, whatever the row holds (padding may hold NaN)
#pragma unroll
        for (int u = 0; u < kLpBwdVecs; ++u) {
            const int v = vb + u * TH, e0 = off + N * v;
            if (v >= nv) break;
            if (e0 >= 0 && e0 + N <= V) {
                __stcs(reinterpret_cast<uint4*>(out + e0), make_uint4(0u, 0u, 0u, 0u));
            } else {
                for (int j = 0; j < N; ++j)
                    if (e0 + j >= 0 && e0 + j < V) out[e0 + j] = LpVec<T>::round(0.0f);
            }
        }
        return;
    }
    // -p (g + h (log p + H)), two elements an instruction
    const float k = -fmaf(h, H, g);
    const uint64_t m2 = pair(-m, -m), l2 = pair(-lsum, -lsum), h2 = pair(-h, -h), k2 = pair(k, k), L2 = pair(kLog2e, kLog2e);
#pragma unroll
    for (int u = 0; u < kLpBwdVecs; ++u) {
        const int v = vb + u * TH;
        if (v >= nv) break;
        const int e0 = off + N * v;
        float f[N];
        LpVec<T>::unpack(x[u], f);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const uint64_t d = add2(add2(pair(f[j], f[j + 1]), m2), l2);
            // below -200 p is 0: held there (NaN stays), 0 * -inf would be NaN
            float a, b;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(lo_of(d)), "f"(-200.0f));
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(hi_of(d)), "f"(-200.0f));
            const uint64_t lp = pair(a, b), y = fma2(lp, L2, 0);
            const uint64_t o = fma2(pair(ex2(lo_of(y)), ex2(hi_of(y))), fma2(h2, lp, k2), 0);
            f[j] = lo_of(o);
            f[j + 1] = hi_of(o);
        }
        if ((uint32_t)(t - e0) < (uint32_t)N && t >= 0) {
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] += e0 + j == t ? g : 0.0f;
        }
        if (e0 >= 0 && e0 + N <= V) {
            __stcs(reinterpret_cast<uint4*>(out + e0), LpVec<T>::pack(f));
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (e0 + j >= 0 && e0 + j < V) out[e0 + j] = LpVec<T>::round(f[j]);
        }
    }
}

// ---- host ---------------------------------------------------------------------------

template <typename T, int TH>
static int lp_launch_th(const LpParams& P, int64_t M, int sms, cudaStream_t stream) {
    // CTAs per row: several while there are fewer rows than SMs to share them, as long as each CTA
    // has a full iteration of vectors.  A cluster's launch and joins cost more than an idle slot:
    // 128256 bf16, top 8: 64 rows 18.5 / 11.5 / 13.0 us with 1 / 4 / 8 CTAs, 600 rows 52 / 55 with 1 / 2
    const int64_t iters = (P.V / LpVec<T>::N + TH * kLpVecs - 1) / (TH * kLpVecs);
    int c = 1;
    while (TH == kLpThreads && c < 8 && 2 * M * c < 3 * (int64_t)sms && c < iters) c *= 2;
    if (M * c > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    auto kernel = P.top > 0 ? k_logprobs<T, true, TH> : k_logprobs<T, false, TH>;
    return launch_after(kernel, (unsigned)(M * c), TH, 0, stream, c, true, P);
}

template <typename T>
static int lp_launch(const LpParams& P, int64_t M, int sms, cudaStream_t stream) {
    // Threads per CTA: a row's joins cost the more the more threads take part, and short rows leave most of
    // them idle.  top 8, 64 / 128 / 256 threads in us: bf16 4096 x 2000 15 / 22 / 41, 4096 x 16000 41 / 44 / 58,
    // 4096 x 32000 76 / 69 / 80, 1000 x 4000 7.9 / 7.1 / 12.6, 1000 x 32000 25 / 19 / 21, 300 x 32000 19 / 12.2 / 10.5
    const int64_t bytes = P.V * (int64_t)sizeof(T);
    if (M >= 2048 && bytes <= 32 * 1024) return lp_launch_th<T, 64>(P, M, sms, stream);
    if (bytes <= (M >= 512 ? 64 : 16) * 1024) return lp_launch_th<T, 128>(P, M, sms, stream);
    return lp_launch_th<T, kLpThreads>(P, M, sms, stream);
}

int token_logprobs_launch(const void* z, int dtype, int64_t M, int64_t V, int64_t ld, const int32_t* targets, int top,
                          float* logp, float* entropy, float* stats, float* top_logp, int32_t* top_ids, int sms,
                          cudaStream_t stream) {
    const LpParams P{z, ld, targets, logp, entropy, stats, top_logp, top_ids, (int)V, top};
    return dtype == SHERRY_BF16 ? lp_launch<__nv_bfloat16>(P, M, sms, stream) : lp_launch<float>(P, M, sms, stream);
}

template <typename T, int TH>
static int bwd_launch_th(LpBwdParams P, int64_t M, cudaStream_t stream) {
    // a row that starts inside a vector has one more of them
    const int64_t segs = (P.V / LpVec<T>::N + 2 + TH * kLpBwdVecs - 1) / (TH * kLpBwdVecs);
    if (M * segs > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    P.segs = (int)segs;
    return launch_after(k_logprobs_bwd<T, TH>, (unsigned)(M * segs), TH, 0, stream, 1, true, P);
}

template <typename T>
static int bwd_launch(const LpBwdParams& P, int64_t M, cudaStream_t stream) {
    // small CTAs waste the fewest threads at a row's end (bf16 20000 x 2000: 31 / 35 / 47 us with 64 / 128 / 256
    // threads, 2048 x 128256: 172 / 173 / 176); few rows want wide ones (fp32 300 x 1000: 3.0 / 2.5 / 2.3)
    return M >= 1024 ? bwd_launch_th<T, 64>(P, M, stream) : bwd_launch_th<T, 128>(P, M, stream);
}

int token_logprobs_bwd_launch(const void* z, int dtype, int64_t M, int64_t V, int64_t ld, const int32_t* targets,
                              const float* stats, const float* entropy, const float* dlogp, const float* dentropy,
                              void* out, int64_t ldo, cudaStream_t stream) {
    const LpBwdParams P{z, ld, targets, stats, entropy, dlogp, dentropy, out, ldo, (int)V, 0};
    return dtype == SHERRY_BF16 ? bwd_launch<__nv_bfloat16>(P, M, stream) : bwd_launch<float>(P, M, stream);
}

}  // namespace sherry
