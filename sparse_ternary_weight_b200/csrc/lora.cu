// lora.cu -- low-rank adapters of many requests beside a packed linear:
//
//   Y[m] = X[m] (T alpha)^T + U[m] B_a^T,   U[m] = s_a X[m] A_a^T,   a = ids[m]
//
// and their gradients, P[m] = s_a dY[m] B_a, dA_a = sum P[m]^T X[m], dB_a = sum
// dY[m]^T U[m] over the tokens of adapter a ("Sherry, Tequila and Fairies in
// Python", section 1.1, has the layer: F.linear on t * alpha; the adapters are the
// usual rank-R residual beside it, kept in bf16, with every sum and U, P in fp32).
//
// Where many tokens run on the tensor cores the products with B (forward) and with
// A (dX) are extra steps of the base kernels (prefill.cu, dgrad.cu).  Here are the
// rest: the plan of tokens by adapter, the products into rank space, the product
// out of it for few tokens, and the adapters' gradients.  U and P are fp32; where
// one is a tensor-core operand it is split into bf16 terms (LoraImage) whose sum is
// the value to 16 (bf16 results) or 24 bits (fp32 results).
#include "lora.cuh"
#include "lut.cuh"
#include "tc.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sherry {

static inline int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }
static inline int64_t lora_tiles(int64_t M) { return (M + kLoraTile - 1) / kLoraTile; }
// Slots that a call has room for.  One adapter after the other they are at most tiles + n_adapters;
// tokens stay in place while they make no more than this: a slot too many costs each product a
// masked pass over its tile, taking tokens in another order a copy of X or dY.
// A slot holds a token, so in either order there are no more than M, however many adapters there are.
static inline int64_t lora_slots_in_place(int64_t M, int n_adapters) {
    return std::min(lora_tiles(M) * n_adapters, M);
}
static inline int64_t lora_max_slots(int64_t M, int n_adapters) {
    return std::min(2 * lora_tiles(M) + n_adapters, lora_slots_in_place(M, n_adapters));
}

bool lora_may_permute(int64_t M, int n_adapters) {
    return lora_slots_in_place(M, n_adapters) > lora_max_slots(M, n_adapters);
}

size_t lora_image_bytes(int64_t M, int n_adapters, int R, int terms) {
    return (size_t)up256(lora_max_slots(M, n_adapters) * kLoraTile * terms * lora_rp(R) * 2);
}

size_t lora_plan_bytes(int64_t M, int n_adapters) {
    const int64_t s = lora_max_slots(M, n_adapters);
    return (size_t)(256 + up256(4 * M) + up256(4 * (lora_tiles(M) + 1)) + 3 * up256(4 * s) + 2 * up256(4 * (n_adapters + 1)) +
                    up256(16 * s));
}

LoraPlan lora_plan_in(void* mem, int64_t M, int n_adapters) {
    const int64_t s = lora_max_slots(M, n_adapters);
    char* p = static_cast<char*>(mem);
    auto take = [&](int64_t bytes) {
        int32_t* at = reinterpret_cast<int32_t*>(p);
        p += up256(bytes);
        return at;
    };
    LoraPlan plan;
    plan.head = take(8);
    plan.perm = take(4 * M);
    plan.tiles = lora_tiles(M);
    plan.tile_b = take(4 * (plan.tiles + 1));
    plan.slot_a = take(4 * s);
    plan.slot_t = take(4 * s);
    plan.adap_s = take(4 * s);
    plan.adap_b = take(4 * (n_adapters + 1));
    plan.bad = take(4 * n_adapters);
    plan.mask = reinterpret_cast<uint32_t*>(take(16 * s));
    plan.max_slots = (int)s;
    plan.may_permute = lora_may_permute(M, n_adapters);
    return plan;
}

// ---- plan ----------------------------------------------------------------------------
// CTA 0 lists the slots, 32 tiles at a time: a warp marks its tile's adapters in a bitmap, whose
// columns place each slot among its adapter's (work linear in the slots).
// Where the plan may permute, one further CTA per bucket (an adapter, or none) reads all
// ids: the tokens of smaller buckets are its offset, its own are compacted in order
// (ballots), so the order depends on the ids alone.  ids stay in L2; one launch.
constexpr int kPlanThreads = 1024;
constexpr int kPlanHeld = 2048;
constexpr int kPlanAhead = 8;  // ids a thread holds while it places them

__device__ __forceinline__ int lora_id(const int32_t* ids, int64_t m, int n_adapters) {
    const int a = ids[m];
    return (a < 0 || a >= n_adapters) ? n_adapters : a;
}

// inclusive sum over the block; `ws` holds 32 ints
__device__ __forceinline__ int block_scan(int x, int* ws) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += v;
    }
    __syncthreads();
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    const int w = lane < warp ? ws[lane] : 0;
    return x + __reduce_add_sync(kFull, w);
}

__device__ __forceinline__ void plan_slots(const int32_t* ids, int M, int n, const LoraPlan& plan) {
    __shared__ uint32_t bits[32][32];
    __shared__ int ws[32], cnt[SHERRY_MAX_ADAPTERS], found;
    __shared__ uint32_t col[SHERRY_MAX_ADAPTERS];  // which of the 32 tiles hold the adapter
    __shared__ uint32_t held[kPlanHeld];  // the first slots' adapters, and their places << 10 among the adapter's slots
    static_assert(SHERRY_MAX_ADAPTERS <= 1024 && kPlanHeld <= 1 << 22, "an adapter and a place in a word");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tiles = (int)plan.tiles;
    cnt[tid] = 0;
    if (tid < n) plan.bad[tid] = 0;
    int total = 0;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
        const int t = t0 + warp;
        bits[warp][lane] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kLoraTile / 32; ++j) {
            const int64_t m = (int64_t)t * kLoraTile + 32 * j + lane;
            const int a = t < tiles && m < M ? lora_id(ids, m, n) : n;
            const unsigned same = __match_any_sync(kFull, a);  // (neighbours are mostly of one adapter)
            if (a < n && lane == __ffs(same) - 1) atomicOr(&bits[warp][a >> 5], 1u << (a & 31));
        }
        __syncthreads();
        uint32_t tiles_of = 0;  // adapter tid's
        if (32 * warp < n) {
#pragma unroll
            for (int j = 0; j < 32; ++j) tiles_of |= (bits[j][warp] >> lane & 1u) << j;
        }
        col[tid] = tiles_of;
        const uint32_t word = bits[warp][lane];
        const int mine = __popc(word), at = total + block_scan(mine, ws) - mine;
        if (lane == 0 && t < tiles) plan.tile_b[t] = at;
        for (unsigned some = __ballot_sync(kFull, word != 0u); some; some &= some - 1) {
            const int w = __ffs(some) - 1;  // a lane per adapter of each 32
            const uint32_t ws32 = __shfl_sync(kFull, word, w);
            const int s = __shfl_sync(kFull, at, w) + __popc(ws32 & ((1u << lane) - 1u)), a = 32 * w + lane;
            if (ws32 >> lane & 1u) {
                const uint32_t place = (uint32_t)cnt[a] + __popc(col[a] & ((1u << warp) - 1u));
                if (s < plan.max_slots) {
                    plan.slot_a[s] = a;
                    plan.slot_t[s] = t;
                    if (s >= kPlanHeld) plan.mask[4 * (int64_t)s] = place;  // (the masks come later)
                }
                if (s < kPlanHeld) held[s] = (uint32_t)a | place << 10;
            }
        }
        const int all = __reduce_add_sync(kFull, ws[lane]);
        total += all;
        __syncthreads();
        cnt[tid] += __popc(tiles_of);
    }
    __syncthreads();
    if (total <= plan.max_slots) {
        const int c = cnt[tid], end = block_scan(c, ws);
        cnt[tid] = end - c;
        if (tid < n) plan.adap_b[tid] = end - c;
        if (tid == n - 1) plan.adap_b[n] = end;
        __syncthreads();
        for (int s = tid; s < total; s += kPlanThreads) {
            const uint32_t h = s < kPlanHeld ? held[s] : 0u;
            const int a = s < kPlanHeld ? (int)(h & 1023u) : plan.slot_a[s];
            plan.adap_s[cnt[a] + (s < kPlanHeld ? h >> 10 : plan.mask[4 * (int64_t)s])] = s;
        }
        if (tid == 0) {
            plan.head[0] = 0;
            plan.head[1] = total;
            plan.tile_b[tiles] = total;
        }
        return;
    }
    // adapter by adapter: a tile's slots are the adapters whose tokens reach into it
    cnt[tid] = 0;
    __syncthreads();
    for (int m0 = 0; m0 < M; m0 += kPlanThreads) {
        const int m = m0 + tid;
        const int a = m < M ? lora_id(ids, m, n) : n;
        const unsigned same = __match_any_sync(kFull, a);
        if (a < n && lane == __ffs(same) - 1) atomicAdd(&cnt[a], __popc(same));
    }
    __syncthreads();
    const int c = cnt[tid], end = block_scan(c, ws), first = end - c;
    const int tb = first / kLoraTile, slots = c > 0 ? (end - 1) / kLoraTile - tb + 1 : 0;
    const int send = block_scan(slots, ws);
    for (int i = 0; i < slots; ++i) {
        plan.slot_a[send - slots + i] = tid;
        plan.slot_t[send - slots + i] = tb + i;
        plan.adap_s[send - slots + i] = send - slots + i;
    }
    if (tid < n) plan.adap_b[tid] = send - slots;
    if (tid == n - 1) {
        plan.adap_b[n] = send;
        plan.head[0] = 1;
        plan.head[1] = send;
        found = send;
    }
    __syncthreads();
    total = found;
    for (int t = tid; t <= tiles; t += kPlanThreads) {  // slots of smaller tiles
        int lo = 0, hi = total;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (plan.slot_t[mid] < t)
                lo = mid + 1;
            else
                hi = mid;
        }
        plan.tile_b[t] = lo;
    }
}

__global__ void __launch_bounds__(kPlanThreads) k_lora_plan(const int32_t* ids, int M, int n_adapters,
                                                            const LoraPlan plan) {
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0) {
        plan_slots(ids, M, n_adapters, plan);
        return;
    }
    __shared__ int red[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int me = blockIdx.x - 1;
    int below = 0;
#pragma unroll 8
    for (int64_t m = tid; m < M; m += kPlanThreads) below += lora_id(ids, m, n_adapters) < me;
    below = __reduce_add_sync(kFull, below);
    if (lane == 0) red[warp] = below;
    __syncthreads();
    int at = __reduce_add_sync(kFull, red[lane]);
    for (int64_t m0 = 0; m0 < M; m0 += kPlanAhead * kPlanThreads) {
        bool mine[kPlanAhead];
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            const int64_t m = m0 + u * kPlanThreads + tid;
            mine[u] = m < M && lora_id(ids, m, n_adapters) == me;
        }
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            if (m0 + u * kPlanThreads >= M) break;
            const unsigned mask = __ballot_sync(kFull, mine[u]);
            __syncthreads();
            if (lane == 0) red[warp] = __popc(mask);
            __syncthreads();
            const int c = red[lane];
            const int before = __reduce_add_sync(kFull, lane < warp ? c : 0);
            if (mine[u])
                plan.perm[at + before + __popc(mask & ((1u << lane) - 1u))] = (int)(m0 + u * kPlanThreads + tid);
            at += __reduce_add_sync(kFull, c);
        }
    }
}

int lora_plan_launch(const int32_t* ids, int64_t M, int n_adapters, const LoraPlan& plan, cudaStream_t stream) {
    const unsigned grid = plan.may_permute ? (unsigned)n_adapters + 2u : 1u;
    return launch_after(k_lora_plan, grid, kPlanThreads, 0, stream, 1, true, ids, (int)M, n_adapters, plan);
}

// ---- rows in the plan's order, or with an aligned length ------------------------------
// TMA wants rows whose bytes are a multiple of 16, and tiles whose rows stand together.
struct RowsParams {
    LoraRows job[2];
    int64_t M;
    const int32_t* head;  // null: no plan
    const int32_t* perm;
    int count;
};

constexpr int kRowsThreads = 256, kRowsVecs = 4;  // 16-byte pieces of the copy per thread

// elements e0 .. e0 + 8 of rows that are not a multiple of 16 bytes, `n` of them in the row, `all` in the matrix
__device__ __forceinline__ uint4 rows_piece(const uint16_t* src, int64_t e0, int n, int64_t all) {
    if (n >= 8 && e0 + 9 <= all) {
        // whole words: from e0, or shifted by half a word from e0 - 1
        const uint32_t* q = reinterpret_cast<const uint32_t*>(src + (e0 & ~(int64_t)1));
        const uint32_t sh = (uint32_t)(e0 & 1) * 16;
        const uint32_t a = __ldg(q), b = __ldg(q + 1), c = __ldg(q + 2), d = __ldg(q + 3), e = sh ? __ldg(q + 4) : 0u;
        return make_uint4(__funnelshift_r(a, b, sh), __funnelshift_r(b, c, sh), __funnelshift_r(c, d, sh),
                          __funnelshift_r(d, e, sh));
    }
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = k < n ? __ldg(src + e0 + k) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

template <typename I>  // of the pieces' numbers
__global__ void __launch_bounds__(kRowsThreads) k_lora_rows(const RowsParams P) {
    pdl_trigger();
    pdl_wait();
    const bool permuted = P.head && P.head[0] != 0;
    const I stride = (I)gridDim.x * kRowsThreads;
    for (int j = 0; j < P.count; ++j) {
        const LoraRows& J = P.job[j];
        if (!permuted && !J.always) continue;
        const I vecs = (I)(J.ld / 8), total = (I)P.M * vecs;
        for (I i0 = (I)blockIdx.x * kRowsThreads + threadIdx.x; i0 < total; i0 += kRowsVecs * stride) {
            uint4 v[kRowsVecs];
#pragma unroll
            for (int u = 0; u < kRowsVecs; ++u) {
                const I i = i0 + u * stride, p = i / vecs, c = i - p * vecs;
                if (i < total) {
                    const int64_t row = (permuted ? (int64_t)P.perm[p] : (int64_t)p) * J.N;
                    v[u] = J.N == J.ld ? __ldg(reinterpret_cast<const uint4*>(J.src + row) + c)
                                       : rows_piece(J.src, row + 8 * c, (int)(J.N - 8 * c), P.M * J.N);
                }
            }
#pragma unroll
            for (int u = 0; u < kRowsVecs; ++u) {
                const I i = i0 + u * stride;
                if (i < total) reinterpret_cast<uint4*>(J.dst)[i] = v[u];  // (rows of dst stand close)
            }
        }
    }
}

int lora_rows_launch(const LoraRows* jobs, int count, int64_t M, const LoraPlan& plan, int sms, cudaStream_t stream) {
    RowsParams P{};
    P.M = M;
    P.count = count;
    for (int j = 0; j < count; ++j) P.job[j] = jobs[j];
    const bool planned = plan.head && plan.may_permute;
    P.head = planned ? plan.head : nullptr;
    P.perm = plan.perm;
    int64_t pieces = 1;
    bool always = false;
    for (int j = 0; j < count; ++j) {
        pieces = std::max(pieces, M * (jobs[j].ld / 8));
        always = always || jobs[j].always;
    }
    // copies that are seldom made have few CTAs to start and end for nothing (331 x 2050 x 8192: 46 -> 42 us)
    const unsigned grid = (unsigned)std::min<int64_t>((pieces + kRowsThreads - 1) / kRowsThreads, (always ? 8 : 2) * (int64_t)sms);
    auto kernel = pieces < (int64_t)1 << 29 ? k_lora_rows<uint32_t> : k_lora_rows<uint64_t>;
    return launch_after(kernel, grid, kRowsThreads, 0, stream, 1, plan.head != nullptr, P);
}

// ---- into rank space -----------------------------------------------------------------
// A cluster per slot: the tile's 128 rows of G by the adapter's W on the tensor cores,
// D [128 tokens][rp ranks], the sum over C split over the cluster's CTAs and joined in order
// through distributed shared memory.  Rows of other tokens are computed along (a row of D
// depends on its own row of G alone) and dropped at the end, where the slot's mask is made.
// W comes by rank rows (A_a: K-major operand) or by rows of C (B_a: MN-major).  The warps
// that end a slot are idle until then: first they make V2's image and V's zeros.
//   warps 0..3 end a slot, warp 4 TMA, warp 5 MMA issue
constexpr int kDnThreads = 192;
constexpr int kDnMaxStages = 6;
constexpr int kDnG = 128 * 64 * 2;   // 16 KB of G a stage, then up to 16 KB of W
constexpr int kDnHalf = 110 * 1024;  // two CTAs per SM: more clusters run at once than with one

struct DownParams {
    LoraPlan plan;
    const int32_t* ids;
    const float* scaling;
    const float* unit;
    int64_t unit_n;
    float* V;
    uint16_t* img;
    const float* V2;
    uint16_t* img2;
    int M, C, R, rp, terms, terms2, n_adapters;
    const uint16_t* A;
    int64_t rk;  // R x K, elements of an adapter's A
    int by_row, product;  // product: there is a W
    int stages, stage_bytes;
};

// the token at position p if it is adapter a's, else -1
__device__ __forceinline__ int slot_token(const DownParams& P, bool permuted, int64_t p, int a) {
    if (p >= P.M) return -1;
    const int m = permuted ? P.plan.perm[p] : (int)p;
    return P.ids[m] == a ? m : -1;
}

// eight ranks of an image row in every term
__device__ __forceinline__ void put_terms(uint16_t* at, int rp, int terms, const float* f) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f[i];
    for (int t = 0; t < terms; ++t) {
        uint4 v;
        v.x = split_next(x[0], x[1]);
        v.y = split_next(x[2], x[3]);
        v.z = split_next(x[4], x[5]);
        v.w = split_next(x[6], x[7]);
        *reinterpret_cast<uint4*>(at + t * rp) = v;
    }
}

// f[i] = the cluster's sums of column i of eight, in order; the columns are `stride` floats apart
__device__ __forceinline__ void cluster_sum8(cg::cluster_group& cluster, int CL, float* at, int stride, float* f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
#pragma unroll 4
    for (int q = 0; q < CL; ++q) {
        const float* p = cluster.map_shared_rank(at, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += p[i * stride];
    }
}

// Look through the A of every adapter with a token, 4096 elements a warp at a time.
__device__ __forceinline__ void down_scan(const DownParams& P, int w0, int ws) {
    constexpr int kPart = 4096;
    const int lane = threadIdx.x & 31, parts = (int)((P.rk + kPart - 1) / kPart);
    for (int64_t u = w0; u < (int64_t)parts * P.n_adapters; u += ws) {
        const int a = (int)(u / parts);
        if (P.plan.adap_b[a] == P.plan.adap_b[a + 1]) continue;
        const int64_t e0 = (u % parts) * kPart, e1 = min(e0 + kPart, P.rk);  // (multiples of 8)
        const uint4* p = reinterpret_cast<const uint4*>(P.A + a * P.rk);
        uint32_t found = 0;
#pragma unroll 8
        for (int64_t e = e0 / 8 + lane; e < e1 / 8; e += 32) {
            const uint4 v = __ldg(p + e);
            found |= __vcmpgeu2(v.x & 0x7fff7fffu, 0x7f807f80u) | __vcmpgeu2(v.y & 0x7fff7fffu, 0x7f807f80u) |
                     __vcmpgeu2(v.z & 0x7fff7fffu, 0x7f807f80u) | __vcmpgeu2(v.w & 0x7fff7fffu, 0x7f807f80u);
        }
        if (__any_sync(kFull, found != 0) && lane == 0) P.plan.bad[a] = 1;  // (all writers write 1)
    }
}

// 32 tokens at a time, a warp each: V's zeros for tokens of no adapter, and a quarter of a slot of V2's image
__device__ __forceinline__ void down_side(const DownParams& P, bool permuted, int slots, int w0, int ws) {
    const int lane = threadIdx.x & 31;
    if (P.A) down_scan(P, w0, ws);
    if (P.V)
        for (int64_t u = w0; u * 32 < P.M; u += ws) {
            const int64_t m = u * 32 + lane;
            const bool none = m < P.M && lora_id(P.ids, m, P.n_adapters) == P.n_adapters;
            for (unsigned left = __ballot_sync(kFull, none); left; left &= left - 1) {
                float* row = P.V + (u * 32 + __ffs(left) - 1) * P.R;
                for (int r = lane; r < P.R; r += 32) row[r] = 0.0f;
            }
        }
    if (P.V2)
        for (int u = w0; u < 4 * slots; u += ws) {
            const int s = u >> 2, q = u & 3;
            const int m = slot_token(P, permuted, (int64_t)P.plan.slot_t[s] * kLoraTile + 32 * q + lane, P.plan.slot_a[s]);
            const unsigned in = __ballot_sync(kFull, m >= 0);
            if (lane == 0) P.plan.mask[u] = in;
#pragma unroll 2
            for (int r = 0; r < P.rp; r += 8) {
                float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                if (m >= 0 && r < P.R) {
                    const float4* src = reinterpret_cast<const float4*>(P.V2 + (int64_t)m * P.R + r);
                    const float4 x = src[0], y = src[1];
                    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
                }
                put_terms(P.img2 + ((int64_t)u * 32 + lane) * (P.terms2 * P.rp) + r, P.rp, P.terms2, f);
            }
        }
}

__global__ void __launch_bounds__(kDnThreads, 2)
k_lora_down(const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap gpmap,
            const __grid_constant__ CUtensorMap wmap, const __grid_constant__ DownParams P) {
    extern __shared__ __align__(1024) unsigned char dsm[];
    __shared__ uint64_t bars[2 * kDnMaxStages + 1];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(&bars[0]);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (kDnMaxStages + i); };
    const uint32_t done = bar0 + 8u * (2 * kDnMaxStages);
    const int ST = P.stages;
    uint32_t cols = 32;
    while ((int)cols < P.rp) cols *= 2;
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                     "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();  // only now: the next kernel reads the plan and the rows in its order at once, and waits for the rest
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int slot0 = blockIdx.x / CL, held = min(slot0, P.plan.max_slots - 1);
    int a = P.plan.slot_a[held], tile = P.plan.slot_t[held];  // loaded beside the head, in vain past the last slot
    const bool permuted = P.plan.may_permute && P.plan.head[0] != 0;
    const int slots = P.plan.head[1];
    const int steps = (P.C + 63) / 64;
    const int s0 = (int)((int64_t)steps * cr / CL), s1 = (int)((int64_t)steps * (cr + 1) / CL);
    const int wboxes = P.by_row ? (P.rp + 63) / 64 : 1;
    const uint32_t wbytes = P.by_row ? (uint32_t)wboxes * 64 * 128 : (uint32_t)P.rp * 128;
    float* sum = reinterpret_cast<float*>(dsm + (base - smem_u32(dsm)));
    const float inv = P.unit ? 1.0f / dgrad_unit(P.unit, P.unit_n) : 1.0f;
    if (warp < 4 && !P.product) down_side(P, permuted, slots, 4 * blockIdx.x + warp, 4 * gridDim.x);

    int c = 0;  // stage and its phase, of the TMA and the MMA thread
    uint32_t ph = 0, dph = 0;
    int used = 0;  // loads of the TMA thread
    for (int s = P.product ? slot0 : slots; s < slots; s += gridDim.x / CL) {  // (whole clusters)
        if (s != slot0) {
            a = P.plan.slot_a[s];
            tile = P.plan.slot_t[s];
        }
        const int64_t p0 = (int64_t)tile * kLoraTile;
        int m = -1;  // warps 0..3: the thread's token
        if (warp == 4) {
            if (lane == 0) {
                for (int st = s0; st < s1; ++st) {
                    if (!mbar_wait(empty(c), ph ^ 1u, &abort_s)) break;
                    const uint32_t dst = base + (uint32_t)(c * P.stage_bytes);
                    mbar_expect_tx(full(c), kDnG + wbytes);
                    tma_load_2d(dst, permuted ? &gpmap : &gmap, st * 64, (int)p0, full(c));
                    if (P.by_row) {
                        for (int j = 0; j < wboxes; ++j)
                            tma_load_3d(dst + kDnG + (uint32_t)j * 64 * 128, &wmap, 64 * j, st * 64, a, full(c));
                    } else {
                        tma_load_3d(dst + kDnG, &wmap, st * 64, 0, a, full(c));
                    }
                    ++used;
                    if (++c == ST) { c = 0; ph ^= 1u; }
                }
                for (int i = 0; i < ST && i < used; ++i)  // every load lands before shared memory is reused
                    mbar_drain(full(i), (uint32_t)(((used - 1 - i) / ST) & 1));
            }
            __syncwarp();
        } else if (warp == 5) {
            if (lane == 0) {
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)P.by_row << 16) |
                                       ((uint32_t)(P.rp >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
                for (int st = s0; st < s1; ++st) {
                    if (!mbar_wait(full(c), ph, &abort_s)) break;
                    tc_fence_after();
                    const uint32_t at = base + (uint32_t)(c * P.stage_bytes);
                    const uint64_t da = smem_desc(at);
                    const uint64_t db = P.by_row ? smem_desc_mn(at + kDnG, 64 * 128) : smem_desc(at + kDnG);
                    const uint64_t bstep = P.by_row ? 2 * (1024 >> 4) : 2;  // 16 rows of C: two atoms, or 32 bytes
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss(tmem, da + (uint64_t)(2 * kk), db + kk * bstep, idesc, (st == s0 && kk == 0) ? 0u : 1u);
                    mma_commit(empty(c));
                    if (++c == ST) { c = 0; ph ^= 1u; }
                }
                mma_commit(done);
                mbar_drain(done, dph);
                dph ^= 1u;
            }
            __syncwarp();
        } else {
            m = slot_token(P, permuted, p0 + tid, a);
            const unsigned in = __ballot_sync(kFull, m >= 0);
            if (cr == 0 && lane == 0) P.plan.mask[4 * s + warp] = in;
            if (s == slot0) down_side(P, permuted, slots, 4 * blockIdx.x + warp, 4 * gridDim.x);
        }
        tc_fence_before();
        __syncthreads();  // all products done, no load in flight
        tc_fence_after();
        // lane = token: eight ranks at a time, straight from TMEM or as [rank][token] for the cluster
        const float scale = P.scaling ? P.scaling[a] : 1.0f;
        auto put = [&](int r, float* f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = m >= 0 ? f[i] * scale : 0.0f;
            if (P.V && m >= 0 && r < P.R) {
                float4* dst = reinterpret_cast<float4*>(P.V + (int64_t)m * P.R + r);
                dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
            if (P.img) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= inv;
                put_terms(P.img + ((int64_t)s * kLoraTile + tid) * (P.terms * P.rp) + r, P.rp, P.terms, f);
            }
        };
        if (warp < 4) {
            const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
            for (int r = 0; r < P.rp; r += 16) {
                uint32_t v[16];
                SHERRY_TMEM_LD16(t_row + (uint32_t)r, v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = s0 < s1 ? __uint_as_float(v[i]) : 0.0f;
                if (CL == 1) {
                    put(r, f);
                    put(r + 8, f + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[(r + i) * kLoraTile + tid] = f[i];
                }
            }
        }
        tc_fence_before();
        cluster.sync();
        tc_fence_after();
        if (CL > 1) {
            if (warp < 4)
                for (int r = 8 * cr; r < P.rp; r += 8 * CL) {
                    float f[8];
                    cluster_sum8(cluster, CL, sum + r * kLoraTile + tid, kLoraTile, f);
                    put(r, f);
                }
            fence_proxy_async();  // the sums were read and written here; the next slot's loads come through TMA
            cluster.sync();       // the others' partial sums are read until here
        }
    }
    // clusters without a slot still have a share of the side work
    if (P.product && warp < 4 && slot0 >= slots)
        down_side(P, permuted, slots, 4 * blockIdx.x + warp, 4 * gridDim.x);
    __syncthreads();
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

int lora_down_launch(const LoraDown& d, int64_t M, int R, int n_adapters, const LoraPlan& plan, int sms,
                     cudaStream_t stream) {
    DownParams P{};
    P.plan = plan;
    P.ids = d.ids;
    P.scaling = d.scaling;
    P.unit = d.unit;
    P.unit_n = d.unit_n;
    P.V = d.V;
    P.img = d.img.data;
    P.V2 = d.V2;
    P.img2 = d.img2.data;
    P.M = (int)M;
    P.C = (int)d.C;
    P.R = R;
    P.rp = lora_rp(R);
    P.terms = d.img.terms;
    P.terms2 = d.img2.terms;
    P.n_adapters = n_adapters;
    P.A = d.A;
    P.rk = (int64_t)R * d.K;
    P.by_row = d.by_row;
    P.product = d.W != nullptr;
    CUtensorMap gmap{}, gpmap{}, wmap{};
    // slots where tokens are well placed; with more of them a cluster takes several
    const int64_t est = std::min<int64_t>(plan.max_slots, plan.tiles + n_adapters), steps = (d.C + 63) / 64;
    int cl = 1;
    if (d.W) {
        int st = encode_2d(&gmap, d.G, d.ldg, M, kLoraTile);
        if (st) return st;
        gpmap = gmap;
        if (d.Gp && (st = encode_2d(&gpmap, d.Gp, d.ldg, M, kLoraTile))) return st;
        st = d.by_row ? encode_3d(&wmap, d.W, R, d.C, n_adapters, 64) : encode_3d(&wmap, d.W, d.C, R, n_adapters, P.rp);
        if (st) return st;
        // the sum is split until the slots fill the SMs once; or, where that still gives each slot four
        // CTAs, the SMs that the next kernel, which starts beside this one, leaves (331 x 2050 x 8192, rank
        // 8: 51 -> 43 us; with one CTA per slot 1000 x 2048 x 8192, rank 16, backward: 72 -> 78)
        const int64_t room = d.beside_ctas + 4 * est <= sms ? sms - d.beside_ctas : sms;
        while (cl < 8 && est * cl * 2 <= room && steps >= 8 * cl) cl *= 2;
    }
    P.stage_bytes = kDnG + (d.by_row ? (P.rp + 63) / 64 * 64 * 128 : (P.rp * 128 + 1023) / 1024 * 1024);
    P.stages = std::min(kDnMaxStages, (kDnHalf - 2048) / P.stage_bytes);
    const int smem = std::max(P.stages * P.stage_bytes, P.rp * kLoraTile * 4) + 1024;
    // clusters beyond the slots share the side work: units of a warp
    const int64_t units = (d.V ? (M + 31) / 32 : 0) + (d.V2 ? 4 * est : 0) + (d.A ? (P.rk + 4095) / 4096 * n_adapters : 0);
    const int64_t clusters = std::max(est, std::min<int64_t>(units / (4 * cl), sms / cl));
    const int64_t grid = std::min<int64_t>(clusters, 4 * sms / cl) * cl;
    if ((int64_t)plan.max_slots * 4 > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    static PerDevice once;
    int v = 0;
    const int st = per_device(once, &v, [](int& x) {
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_lora_down, cudaFuncAttributeMaxDynamicSharedMemorySize, kDnHalf));
        x = 1;
        return SHERRY_OK;
    });
    if (st) return st;
    return launch_after(k_lora_down, (unsigned)grid, kDnThreads, (size_t)smem, stream, cl, true, gmap, gpmap, wmap, P);
}

// ---- out of rank space, where the linear is not the prefill kernel's --------------------
__global__ void __launch_bounds__(128) k_lora_up(const float* Yin, int N, int nblocks, const float* __restrict__ U,
                                                 const uint16_t* __restrict__ B, int R, const int32_t* __restrict__ ids,
                                                 int n_adapters, void* Y, int y_bf16) {
    const int64_t m = blockIdx.x / nblocks;
    const int n = (int)(blockIdx.x % nblocks) * 128 + threadIdx.x;
    if (n >= N) return;
    const int a = ids[m];
    float y = Yin[m * N + n];
    if (a >= 0 && a < n_adapters) {
        const uint16_t* b = B + ((int64_t)a * N + n) * R;
        const float* u = U + m * R;
        float s = 0.0f;
        for (int r = 0; r < R; r += 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(b + r));
            const float4 p = __ldg(reinterpret_cast<const float4*>(u + r)), q = __ldg(reinterpret_cast<const float4*>(u + r) + 1);
            s = fmaf(bf16lo(v.x), p.x, s);
            s = fmaf(bf16hi(v.x), p.y, s);
            s = fmaf(bf16lo(v.y), p.z, s);
            s = fmaf(bf16hi(v.y), p.w, s);
            s = fmaf(bf16lo(v.z), q.x, s);
            s = fmaf(bf16hi(v.z), q.y, s);
            s = fmaf(bf16lo(v.w), q.z, s);
            s = fmaf(bf16hi(v.w), q.w, s);
        }
        y += s;
    }
    if (y_bf16)
        reinterpret_cast<__nv_bfloat16*>(Y)[m * N + n] = __float2bfloat16_rn(y);
    else
        reinterpret_cast<float*>(Y)[m * N + n] = y;
}

int lora_up_launch(const float* Yin, int64_t M, int64_t N, const float* U, const uint16_t* B, int R,
                   const int32_t* ids, int n_adapters, void* Y, int y_bf16, cudaStream_t stream) {
    const int64_t nb = (N + 127) / 128;
    if (nb * M > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    k_lora_up<<<(unsigned)(nb * M), 128, 0, stream>>>(Yin, (int)N, (int)nb, U, B, R, ids, n_adapters, Y, y_bf16);
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

// ---- gradients of the adapters ---------------------------------------------------------
// out_a[r][c] = sum over adapter a's tokens of V[m][r] G[m][c] on the tensor cores: D [128 columns
// of G][terms x rp], the tokens of the adapter's slots summed in stages of 64.  Both operands come
// by TMA as they are stored and are MN-major (tokens are the rows); V is the image, so other
// tokens' rows are zero, and in tiles that the adapter shares G's rows of other tokens are
// zeroed too, in shared memory: an infinity there would make NaN of 0 * inf.  The terms of V
// are columns of D side by side, added at the end.  Stages are split over the CTAs of a
// cluster, whose sums are joined in order.
//   warps 0..3 make the rows ready and end the tile, warp 4 TMA, warp 5 MMA issue
constexpr int kGrThreads = 192;
constexpr int kGrCols = 128, kGrTok = 64;
constexpr int kGrG = kGrTok * kGrCols * 2;  // two boxes of 64 columns: 16 KB
constexpr int kGrV = kGrTok * 64 * 2;       // each 64 columns of the image: 8 KB
constexpr int kGrMaxStages = 6;
constexpr int kGrHeld = 32;                 // slots whose table a CTA holds in shared memory
constexpr int kGrExtra = 3328;              // a CTA's shared memory beside its stages: alignment, statics, the system's

struct GradParams {
    LoraPlan plan;
    void* out[2];
    const float* unit[2];
    int64_t unit_n[2];
    int64_t C[2];
    int by_column[2], cblocks[2];
    int R, rp, terms, n_adapters, out_bf16;
    int vboxes, stages;
    int beside;  // runs beside the kernel before it
};
struct GradMaps {
    CUtensorMap g[2], gp[2], v[2];
};

__global__ void __launch_bounds__(kGrThreads)
k_lora_grad(const __grid_constant__ GradMaps maps, const __grid_constant__ GradParams P) {
    extern __shared__ __align__(1024) unsigned char gsm[];
    __shared__ uint64_t bars[3 * kGrMaxStages + 1];
    __shared__ int2 held[kGrHeld];
    __shared__ uint4 held_mask[kGrHeld];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int b = blockIdx.x / CL;
    const int j = b >= P.cblocks[0] * P.n_adapters ? 1 : 0;
    if (j) b -= P.cblocks[0] * P.n_adapters;
    const int a = b / P.cblocks[j], c0 = (b % P.cblocks[j]) * kGrCols;
    const uint32_t base = (smem_u32(gsm) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(&bars[0]);
    const int ST = P.stages, ncols = P.terms * P.rp;
    const uint32_t SB = (uint32_t)(kGrG + P.vboxes * kGrV);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto ready = [&](int i) { return bar0 + 8u * (kGrMaxStages + i); };
    auto empty = [&](int i) { return bar0 + 8u * (2 * kGrMaxStages + i); };
    const uint32_t done = bar0 + 8u * (3 * kGrMaxStages);
    uint32_t tcols = 32;
    while ((int)tcols < ncols) tcols *= 2;
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(ready(i), 128);
            mbar_init(empty(i), 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                     "r"(tcols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // After the input gradient, which itself waited for what this kernel reads before it let this one
    // start, there is nothing to wait for; only the first cluster sees to it, at its end, that this
    // kernel does not end before that one.
    if (!P.beside) {
        pdl_trigger();
        pdl_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const bool permuted = P.plan.may_permute && P.plan.head[0] != 0;
    const int first = P.plan.adap_b[a], stages = 2 * (P.plan.adap_b[a + 1] - first);
    const int32_t* list = P.plan.adap_s + first;
    const int s0 = (int)((int64_t)stages * cr / CL), s1 = (int)((int64_t)stages * (cr + 1) / CL);
    // the first slots of this CTA's stages, their tiles and masks: loaded at once, not stage by stage
    const int held0 = s0 >> 1, held1 = min(held0 + kGrHeld, (s1 + 1) >> 1);
    if (tid < held1 - held0) {
        const int s = list[held0 + tid];
        held[tid] = make_int2(s, P.plan.slot_t[s]);
        held_mask[tid] = *reinterpret_cast<const uint4*>(P.plan.mask + 4 * s);
    }
    __syncthreads();
    auto slot_of = [&](int i) {
        if (i < held1) return held[i - held0];
        const int s = list[i];
        return make_int2(s, P.plan.slot_t[s]);
    };

    if (warp < 4) {
        int c = 0;
        uint32_t ph = 0;
        for (int st = s0; st < s1; ++st) {
            const int i = st >> 1;
            const uint4 mk = i < held1 ? held_mask[i - held0]
                                       : *reinterpret_cast<const uint4*>(P.plan.mask + 4 * list[i]);
            const uint32_t lo = (st & 1) ? mk.z : mk.x, hi = (st & 1) ? mk.w : mk.y;
            if (!mbar_wait(full(c), ph, &abort_s)) break;
            if ((lo & hi) != 0xffffffffu) {
                const int row = tid & 63;
                if (!(((row & 32) ? hi : lo) >> (row & 31) & 1u)) {
                    const uint32_t at = base + (uint32_t)c * SB + (uint32_t)((tid >> 6) * (kGrTok * 128) + row * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16u * i), "r"(0) : "memory");
                }
                fence_proxy_async();
            }
            mbar_arrive(ready(c));
            if (++c == ST) { c = 0; ph ^= 1u; }
        }
    } else if (warp == 4) {
        if (lane == 0) {
            int c = 0, n = 0;
            uint32_t ph = 0;
            for (int st = s0; st < s1; ++st, ++n) {
                const int2 sl = slot_of(st >> 1);
                const int s = sl.x, row = sl.y * kLoraTile + kGrTok * (st & 1);
                if (!mbar_wait(empty(c), ph ^ 1u, &abort_s)) break;
                const uint32_t dst = base + (uint32_t)c * SB;
                mbar_expect_tx(full(c), SB);
                const CUtensorMap* gm = permuted ? &maps.gp[j] : &maps.g[j];
                for (int q = 0; q < 2; ++q) tma_load_2d(dst + q * (kGrG / 2), gm, c0 + 64 * q, row, full(c));
                for (int q = 0; q < P.vboxes; ++q)
                    tma_load_2d(dst + kGrG + q * kGrV, &maps.v[j], 64 * q, s * kLoraTile + kGrTok * (st & 1), full(c));
                if (++c == ST) { c = 0; ph ^= 1u; }
            }
            for (int i = 0; i < ST && i < n; ++i) mbar_drain(full(i), (uint32_t)(((n - 1 - i) / ST) & 1));
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            const int n0 = min(ncols, 256), n1 = ncols - n0;
            const uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(128 >> 4) << 24);
            int c = 0;
            uint32_t ph = 0;
            for (int st = s0; st < s1; ++st) {
                if (!mbar_wait(ready(c), ph, &abort_s)) break;
                tc_fence_after();
                const uint32_t at = base + (uint32_t)c * SB;
                const uint64_t da = smem_desc_mn(at, kGrG / 2), db = smem_desc_mn(at + kGrG, kGrV);
#pragma unroll
                for (int kk = 0; kk < kGrTok / 16; ++kk) {  // 16 tokens: two atoms of eight rows
                    const uint64_t step = (uint64_t)(2 * kk * (1024 >> 4));
                    const uint32_t acc = (st == s0 && kk == 0) ? 0u : 1u;
                    mma_bf16_ss(tmem, da + step, db + step, id | ((uint32_t)(n0 >> 3) << 17), acc);
                    if (n1 > 0)
                        mma_bf16_ss(tmem + 256, da + step, db + step + (uint64_t)((4 * kGrV) >> 4),
                                    id | ((uint32_t)(n1 >> 3) << 17), acc);
                }
                mma_commit(empty(c));
                if (++c == ST) { c = 0; ph ^= 1u; }
            }
            mma_commit(done);
            mbar_drain(done, 0u);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();  // all products done, no load in flight
    tc_fence_after();
    // lane = column: eight ranks at a time, straight from TMEM or as [rank][column] for the cluster
    const int R = P.R;
    const int64_t C = P.C[j], cc = c0 + tid;
    const float unit = P.unit[j] ? dgrad_unit(P.unit[j], P.unit_n[j]) : 1.0f;
    float* sum = reinterpret_cast<float*>(gsm + (base - smem_u32(gsm)));
    auto put = [&](int r, float* f) {
        if (cc >= C || r >= R) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= unit;
        if (P.by_column[j]) {
            const int64_t at = ((int64_t)a * C + cc) * R + r;
            if (P.out_bf16) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    h[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(P.out[j]) + at) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(P.out[j]) + at);
                dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
        } else {
            const int64_t at = ((int64_t)a * R + r) * C + cc;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (P.out_bf16)
                    reinterpret_cast<__nv_bfloat16*>(P.out[j])[at + i * C] = __float2bfloat16_rn(f[i]);
                else
                    reinterpret_cast<float*>(P.out[j])[at + i * C] = f[i];
            }
        }
    };
    if (warp < 4) {
        const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
        for (int r = 0; r < P.rp; r += 16) {
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = 0.0f;
            if (s0 < s1) {
                for (int t = P.terms - 1; t >= 0; --t) {  // the small terms first
                    uint32_t v[16];
                    SHERRY_TMEM_LD16(t_row + (uint32_t)(t * P.rp + r), v);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] += __uint_as_float(v[i]);
                }
            }
            if (CL == 1) {
                put(r, f);
                put(r + 8, f + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[(r + i) * kGrCols + tid] = f[i];
            }
        }
    }
    tc_fence_before();
    cluster.sync();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tcols));
    }
    if (CL > 1) {
        if (warp < 4)
            for (int r = 8 * cr; r < R; r += 8 * CL) {
                float f[8];
                cluster_sum8(cluster, CL, sum + r * kGrCols + tid, kGrCols, f);
                put(r, f);
            }
        cluster.sync();  // the others' partial sums are read until here
    }
    if (P.beside && blockIdx.x == 0) pdl_wait();
}

int lora_grad_launch(const LoraGradJob* jobs, int count, int R, int n_adapters, int64_t M, const LoraPlan& plan,
                     int out_bf16, bool beside, int sms, cudaStream_t stream) {
    GradParams P{};
    P.beside = beside;
    GradMaps maps{};
    int64_t blocks = 0;
    P.terms = jobs[0].V.terms;
    P.rp = jobs[0].V.rp;
    for (int j = 0; j < count; ++j) {
        const LoraGradJob& J = jobs[j];
        P.out[j] = J.out;
        P.unit[j] = J.unit;
        P.unit_n[j] = J.unit_n;
        P.C[j] = J.C;
        P.by_column[j] = J.by_column;
        P.cblocks[j] = (int)((J.C + kGrCols - 1) / kGrCols);
        blocks += (int64_t)P.cblocks[j] * n_adapters;
        int st = encode_2d(&maps.g[j], J.G, J.ldg, M, kGrTok);
        maps.gp[j] = maps.g[j];
        if (!st && J.Gp) st = encode_2d(&maps.gp[j], J.Gp, J.ldg, M, kGrTok);
        if (!st) st = encode_2d(&maps.v[j], J.V.data, P.terms * P.rp, (int64_t)plan.max_slots * kLoraTile, kGrTok);
        if (st) return st;
    }
    P.plan = plan;
    P.R = R;
    P.n_adapters = n_adapters;
    P.out_bf16 = out_bf16;
    P.vboxes = (P.terms * P.rp + 63) / 64;
    // tokens split while three CTAs per SM hold them all, each with a few stages on average
    const int64_t avg = 2 * ((plan.tiles + n_adapters - 1) / n_adapters);
    int cl = 1;
    while (cl < 8 && blocks * cl * 2 <= 3 * (int64_t)sms && avg >= 4 * cl) cl *= 2;
    if (blocks * cl > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    // as many CTAs per SM as make one wave, or as have two stages each and TMEM; the stages that fit then
    const int SB = kGrG + P.vboxes * kGrV, smem_sm = 228 * 1024, sum = kGrCols * P.rp * 4;
    int tcols = 32;
    while (tcols < P.terms * P.rp) tcols *= 2;
    int64_t per = std::min<int64_t>((blocks * cl + sms - 1) / sms, std::min(512 / tcols, smem_sm / (2 * SB + kGrExtra)));
    if (per < 1) per = 1;
    P.stages = (int)std::min<int64_t>(kGrMaxStages, (smem_sm / per - kGrExtra) / SB);
    const int smem = std::max(P.stages * SB, sum) + 1024;
    static PerDevice once;
    int v = 0;
    const int st = per_device(once, &v, [](int& x) {
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_lora_grad, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024));
        x = 1;
        return SHERRY_OK;
    });
    if (st) return st;
    return launch_after(k_lora_grad, (unsigned)(blocks * cl), kGrThreads, (size_t)smem, stream, cl, true, maps, P);
}

int lora_status_take() { return tc_status_take(); }

}  // namespace sherry
