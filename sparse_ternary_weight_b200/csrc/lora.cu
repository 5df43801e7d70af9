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
// one is a tensor-core operand it is split into bf16 terms whose sum is the value to
// 16 (bf16 results) or 24 bits (fp32 results).
#include "lora.cuh"
#include "lut.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sherry {

static inline int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

size_t lora_plan_bytes(int64_t M, int n_adapters) {
    const int64_t tiles = (M + kLoraTile - 1) / kLoraTile;
    return (size_t)(up256(4 * M) + up256(4 * (n_adapters + 2)) + up256(4 * tiles) + up256(4 * tiles * kLoraTile));
}

LoraPlan lora_plan_in(void* mem, int64_t M, int n_adapters) {
    const int64_t tiles = (M + kLoraTile - 1) / kLoraTile;
    char* p = static_cast<char*>(mem);
    LoraPlan plan;
    plan.perm = reinterpret_cast<int32_t*>(p);
    p += up256(4 * M);
    plan.offs = reinterpret_cast<int32_t*>(p);
    p += up256(4 * (n_adapters + 2));
    plan.tile_n = reinterpret_cast<int32_t*>(p);
    p += up256(4 * tiles);
    plan.tile_a = reinterpret_cast<int32_t*>(p);
    return plan;
}

// ---- plan ----------------------------------------------------------------------------
// One CTA per bucket reads all ids: the tokens of smaller buckets are its offset, its
// own are compacted in order (ballots), so the plan depends on the ids alone.  Further
// CTAs list the different adapters of each 128-token tile.  ids stay in L2; one launch.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) k_lora_plan(const int32_t* __restrict__ ids, int M, int n_adapters,
                                                            const LoraPlan plan) {
    __shared__ int red[32];
    __shared__ int tile_ids[kLoraTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if ((int)blockIdx.x > n_adapters) {
        const int t = blockIdx.x - n_adapters - 1;
        int a = -1;
        if (tid < kLoraTile) {
            const int m = t * kLoraTile + tid;
            a = m < M ? ids[m] : -1;
            if (a < 0 || a >= n_adapters) a = -1;
            tile_ids[tid] = a;
        }
        __syncthreads();
        bool first = a >= 0;
        if (first)
            for (int j = 0; j < tid; ++j)
                if (tile_ids[j] == a) {
                    first = false;
                    break;
                }
        const unsigned mask = __ballot_sync(kFull, first);
        if (lane == 0) red[warp] = __popc(mask);
        __syncthreads();
        int at = 0;
        for (int w = 0; w < warp; ++w) at += red[w];
        if (first) plan.tile_a[(int64_t)t * kLoraTile + at + __popc(mask & ((1u << lane) - 1u))] = a;
        if (tid == 0) plan.tile_n[t] = red[0] + red[1] + red[2] + red[3];
        return;
    }
    const int me = blockIdx.x;
    int below = 0;
    for (int m = tid; m < M; m += kPlanThreads) {
        const int a = ids[m];
        below += ((a < 0 || a >= n_adapters) ? n_adapters : a) < me;
    }
    below = __reduce_add_sync(kFull, below);
    if (lane == 0) red[warp] = below;
    __syncthreads();
    int at = __reduce_add_sync(kFull, red[lane]);
    if (tid == 0) plan.offs[me] = at;
    for (int m0 = 0; m0 < M; m0 += kPlanThreads) {
        const int m = m0 + tid;
        bool mine = false;
        if (m < M) {
            const int a = ids[m];
            mine = ((a < 0 || a >= n_adapters) ? n_adapters : a) == me;
        }
        const unsigned mask = __ballot_sync(kFull, mine);
        __syncthreads();
        if (lane == 0) red[warp] = __popc(mask);
        __syncthreads();
        const int c = red[lane];
        const int before = __reduce_add_sync(kFull, lane < warp ? c : 0);
        if (mine) plan.perm[at + before + __popc(mask & ((1u << lane) - 1u))] = m;
        at += __reduce_add_sync(kFull, c);
    }
    if (tid == 0 && me == n_adapters) plan.offs[n_adapters + 1] = at;
}

int lora_plan_launch(const int32_t* ids, int64_t M, int n_adapters, const LoraPlan& plan, cudaStream_t stream) {
    const int64_t tiles = (M + kLoraTile - 1) / kLoraTile;
    k_lora_plan<<<(unsigned)(n_adapters + 1 + tiles), kPlanThreads, 0, stream>>>(ids, (int)M, n_adapters, plan);
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

// ---- into rank space -----------------------------------------------------------------
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct DownParams {
    const uint16_t* G;
    const uint16_t* W;
    const float* scaling;
    const int32_t* ids;
    float* V;
    int64_t ldg, ldw;
    LoraPlan plan;
    int M, C, R, n_adapters;
};

// Bucket and token range [t0, t1) (places in perm) of tile `tile` when each bucket is cut
// into tiles of T tokens; false past the last.  Called by whole warps.
__device__ __forceinline__ bool bucket_tile(const LoraPlan& plan, int buckets, int T, int tile, int& bucket, int& t0,
                                            int& t1) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < buckets; b0 += 32) {
        const int b = b0 + lane;
        const int lo = b < buckets ? plan.offs[b] : 0, hi = b < buckets ? plan.offs[b + 1] : 0;
        const int n = (hi - lo + T - 1) / T;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(kFull, before + sum > tile);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int j = tile - before - __shfl_sync(kFull, sum - n, src);
            bucket = b0 + src;
            t0 = __shfl_sync(kFull, lo, src) + j * T;
            t1 = min(t0 + T, __shfl_sync(kFull, hi, src));
            return true;
        }
        before += __shfl_sync(kFull, sum, 31);
    }
    return false;
}

// 64 tokens of one adapter x R ranks; the sum over C is split over the CTAs of a cluster and
// two halves of each CTA's warps (4 groups of 16 tokens x 2), and joined in a fixed order
// through distributed shared memory.  mma.sync fragments are loaded from global memory as
// they are: 16 bytes per lane are four k pairs of a row, and both operands use the same
// order of k.
constexpr int kDownTok = 64;

template <int NT>  // 8-rank tiles
__global__ void __launch_bounds__(256) k_lora_down(const DownParams P) {
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp & 3, half = warp >> 2;
    __shared__ float part[kDownTok][8 * NT];
    int bucket, t0, t1;
    if (!bucket_tile(P.plan, P.n_adapters + 1, kDownTok, blockIdx.x / CL, bucket, t0, t1)) return;
    const int R = P.R;
    if (bucket == P.n_adapters) {  // tokens of no adapter
        if (cr == 0)
            for (int i = threadIdx.x; i < (t1 - t0) * R; i += 256)
                P.V[(int64_t)P.plan.perm[t0 + i / R] * R + i % R] = 0.0f;
        return;
    }
    const int g = lane >> 2, c = lane & 3;
    const int ta = t0 + group * 16 + g, tb = ta + 8;
    const uint16_t* ga = P.G + (int64_t)(ta < t1 ? P.plan.perm[ta] : 0) * P.ldg + 8 * c;
    const uint16_t* gb = P.G + (int64_t)(tb < t1 ? P.plan.perm[tb] : 0) * P.ldg + 8 * c;
    const bool oka = ta < t1, okb = tb < t1;
    const uint16_t* wr = P.W + ((int64_t)bucket * R + g) * P.ldw + 8 * c;
    const int steps = (P.C + 31) / 32;
    const int parts = 2 * CL, mine = 2 * cr + half;
    const int s0 = (int)((int64_t)steps * mine / parts), s1 = (int)((int64_t)steps * (mine + 1) / parts);
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    constexpr int UB = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if (t0 + group * 16 < t1) {
        for (int s = s0; s < s1; s += UB) {
            uint4 xa[UB], xb[UB], w[UB][NT];
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                const int k = 32 * (s + u);
                const bool in = s + u < s1 && k + 8 * c < P.C;
                xa[u] = in && oka ? __ldg(reinterpret_cast<const uint4*>(ga + k)) : zero;
                xb[u] = in && okb ? __ldg(reinterpret_cast<const uint4*>(gb + k)) : zero;
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    w[u][i] = in && 8 * i + g < R ? __ldg(reinterpret_cast<const uint4*>(wr + 8 * i * P.ldw + k)) : zero;
            }
#pragma unroll
            for (int u = 0; u < UB; ++u)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma16816(acc[i], xa[u].x, xb[u].x, xa[u].y, xb[u].y, w[u][i].x, w[u][i].y);
                    mma16816(acc[i], xa[u].z, xb[u].z, xa[u].w, xb[u].w, w[u][i].z, w[u][i].w);
                }
        }
    }
    // accumulator (row g or g + 8, rank 2c or 2c + 1 of each tile): the first half's, plus the second's
    const int r0 = group * 16 + g;
    if (half == 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            *reinterpret_cast<float2*>(&part[r0][8 * i + 2 * c]) = make_float2(acc[i][0], acc[i][1]);
            *reinterpret_cast<float2*>(&part[r0 + 8][8 * i + 2 * c]) = make_float2(acc[i][2], acc[i][3]);
        }
    }
    __syncthreads();
    if (half == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            part[r0][8 * i + 2 * c] += acc[i][0];
            part[r0][8 * i + 2 * c + 1] += acc[i][1];
            part[r0 + 8][8 * i + 2 * c] += acc[i][2];
            part[r0 + 8][8 * i + 2 * c + 1] += acc[i][3];
        }
    }
    cluster.sync();
    const float scale = P.scaling ? P.scaling[bucket] : 1.0f;
    for (int i = cr * 256 + threadIdx.x; i < (t1 - t0) * R; i += 256 * CL) {
        const int row = i / R, r = i % R;
        float sum = 0.0f;
        for (int q = 0; q < CL; ++q) sum += cluster.map_shared_rank(&part[0][0], q)[row * (8 * NT) + r];
        P.V[(int64_t)P.plan.perm[t0 + row] * R + r] = scale * sum;
    }
    cluster.sync();  // the others' partial sums are read until here
}

template <int NT>
static int down_launch_nt(const DownParams& P, int cl, int64_t tiles, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * cl));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cl;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    SHERRY_CUDA_CHECK(cudaLaunchKernelEx(&cfg, k_lora_down<NT>, P));
    return SHERRY_OK;
}

int lora_down_launch(const uint16_t* G, int64_t ldg, int64_t M, int64_t C, const uint16_t* W, int64_t ldw, int R,
                     const int32_t* ids, const float* scaling, int n_adapters, const LoraPlan& plan, float* V, int sms,
                     cudaStream_t stream) {
    const DownParams P{G, W, scaling, ids, V, ldg, ldw, plan, (int)M, (int)C, R, n_adapters};
    const int64_t full = (M + kDownTok - 1) / kDownTok;
    const int64_t tiles = full + n_adapters + 1;  // every bucket may end inside a tile
    const int64_t steps = (C + 31) / 32;
    int cl = 1;
    while (cl < 8 && full * cl < 2 * (int64_t)sms && steps >= 8 * cl) cl *= 2;
    const int nt = R / 8;
    if (nt <= 1) return down_launch_nt<1>(P, cl, tiles, stream);
    if (nt <= 2) return down_launch_nt<2>(P, cl, tiles, stream);
    if (nt <= 4) return down_launch_nt<4>(P, cl, tiles, stream);
    if (nt <= 8) return down_launch_nt<8>(P, cl, tiles, stream);
    return down_launch_nt<16>(P, cl, tiles, stream);
}

// Few tokens: a CTA per token and four ranks, 16-byte loads, fp32 on the CUDA cores.
__global__ void __launch_bounds__(128) k_lora_down_few(const DownParams P) {
    __shared__ float red[4][4];
    const int m = blockIdx.y, r0 = 4 * blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int a = P.ids[m];
    float* out = P.V + (int64_t)m * P.R + r0;
    if (a < 0 || a >= P.n_adapters) {
        if (threadIdx.x < 4) out[threadIdx.x] = 0.0f;
        return;
    }
    const uint16_t* g = P.G + (int64_t)m * P.ldg;
    const uint16_t* w = P.W + ((int64_t)a * P.R + r0) * P.ldw;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int k = 8 * threadIdx.x; k < P.C; k += 8 * 128) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(g + k));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(w + r * P.ldw + k));
            const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[r] = fmaf(bf16lo(xs[j]), bf16lo(vs[j]), acc[r]);
                acc[r] = fmaf(bf16hi(xs[j]), bf16hi(vs[j]), acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) acc[r] += __shfl_xor_sync(kFull, acc[r], o);
        if (lane == 0) red[warp][r] = acc[r];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        const float s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
        out[threadIdx.x] = (P.scaling ? P.scaling[a] : 1.0f) * s;
    }
}

int lora_down_few_launch(const uint16_t* G, int64_t ldg, int64_t M, int64_t C, const uint16_t* W, int64_t ldw, int R,
                         const int32_t* ids, const float* scaling, int n_adapters, float* V, cudaStream_t stream) {
    const DownParams P{G, W, scaling, ids, V, ldg, ldw, LoraPlan{}, (int)M, (int)C, R, n_adapters};
    k_lora_down_few<<<dim3((unsigned)(R / 4), (unsigned)M), 128, 0, stream>>>(P);
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

// ---- out of rank space, few tokens ---------------------------------------------------
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

// ---- layouts ---------------------------------------------------------------------------
// B_a [N][R] -> [R][ld]: the product dY B sums over n, which the fragments want contiguous.
__global__ void __launch_bounds__(256) k_lora_transpose(const uint16_t* __restrict__ src, int N, int R,
                                                        uint16_t* __restrict__ dst, int64_t ld, int nblocks) {
    __shared__ uint16_t t[64][SHERRY_MAX_RANK + 2];
    const int a = blockIdx.x / nblocks, n0 = (blockIdx.x % nblocks) * 64;
    for (int i = threadIdx.x; i < 64 * R; i += 256) {
        const int n = n0 + i / R;
        t[i / R][i % R] = n < N ? src[((int64_t)a * N + n) * R + i % R] : (uint16_t)0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * R; i += 256) {
        const int r = i >> 6, n = i & 63;
        if (n0 + n < ld) dst[((int64_t)a * R + r) * ld + n0 + n] = t[n][r];
    }
}

int lora_transpose_launch(const uint16_t* src, int n_adapters, int64_t N, int R, uint16_t* dst, int64_t ld,
                          cudaStream_t stream) {
    const int64_t nb = (ld + 63) / 64;
    if (nb * n_adapters > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    k_lora_transpose<<<(unsigned)(nb * n_adapters), 256, 0, stream>>>(src, (int)N, R, dst, ld, (int)nb);
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

// Rows of an odd width, copied 16-byte aligned (TMA and the vector loads need it).
__global__ void __launch_bounds__(256) k_lora_pad(const uint16_t* __restrict__ src, int64_t M, int64_t N,
                                                  uint16_t* __restrict__ dst, int64_t ld) {
    const int64_t total = M * ld;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / ld, n = i % ld;
        dst[i] = n < N ? src[m * N + n] : (uint16_t)0;
    }
}

int lora_pad_launch(const uint16_t* src, int64_t M, int64_t N, uint16_t* dst, int64_t ld, cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>((M * ld + 255) / 256, 148 * 16);
    k_lora_pad<<<(unsigned)blocks, 256, 0, stream>>>(src, M, N, dst, ld);
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

// ---- gradients of the adapters ---------------------------------------------------------
// out_a[r][c] = sum over adapter a's tokens of V[m][r] G[m][c]: 128 columns per CTA, tokens in
// chunks of 32.  G's rows are gathered by cp.async into shared memory and enter mma.sync as
// operand B through ldmatrix.trans; V's split terms are stored transposed ([r][m]) as operand
// A.  The tokens are split over the CTAs of a cluster, whose sums are joined in order.
constexpr int kGradCols = 128, kGradTok = 32;
constexpr int kGradGRow = kGradCols * 2 + 16;  // bytes per token row of G, padded for ldmatrix
constexpr int kGradVRow = kGradTok * 2 + 16;   // bytes per rank row of V^T

struct GradParams {
    LoraGradJob job[2];
    int cblocks[2];  // column blocks of each job
    LoraPlan plan;
    int R, n_adapters, out_bf16;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    const int n = in ? 16 : 0;  // 0: zero fill, nothing read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// RT: 16-rank tiles; SPL: split terms of V
template <int RT, int SPL>
__global__ void __launch_bounds__(256) k_lora_grad(const GradParams P) {
    constexpr int kV = SPL * 16 * RT * kGradVRow, kG = kGradTok * kGradGRow;
    constexpr int kSum = 16 * RT * kGradCols * 4;
    constexpr int kBytes = (2 * kG + kV) > kSum ? (2 * kG + kV) : kSum;
    extern __shared__ __align__(16) unsigned char gs[];
    static_assert(kBytes <= 100 * 1024, "shared memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int b = blockIdx.x / CL;
    const int j = b >= P.cblocks[0] * P.n_adapters ? 1 : 0;
    if (j) b -= P.cblocks[0] * P.n_adapters;
    const LoraGradJob& J = P.job[j];
    const int a = b / P.cblocks[j], c0 = (b % P.cblocks[j]) * kGradCols;
    const int R = P.R;
    const int lo = P.plan.offs[a], hi = P.plan.offs[a + 1];
    const int chunks = (hi - lo + kGradTok - 1) / kGradTok;
    const int ch0 = (int)((int64_t)chunks * cr / CL), ch1 = (int)((int64_t)chunks * (cr + 1) / CL);
    const uint32_t sG = smem_u32(gs), sV = sG + 2 * kG;
    float acc[RT][2][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.0f;

    auto load_g = [&](int ch, int buf) {
        // 32 rows x 16 pieces of 16 bytes
#pragma unroll
        for (int i = 0; i < kGradTok * 16 / 256; ++i) {
            const int p = tid + 256 * i, row = p >> 4, piece = p & 15;
            const int t = lo + ch * kGradTok + row;
            const bool in = t < hi && c0 + 8 * piece < J.ldg;
            const uint16_t* src = in ? J.G + (int64_t)P.plan.perm[t] * J.ldg + c0 + 8 * piece : J.G;
            cp_async16(sG + buf * kG + row * kGradGRow + piece * 16, src, in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (ch0 < ch1) load_g(ch0, 0);
    for (int ch = ch0; ch < ch1; ++ch) {
        const int buf = (ch - ch0) & 1;
        if (ch + 1 < ch1)
            load_g(ch + 1, buf ^ 1);
        else
            asm volatile("cp.async.commit_group;" ::: "memory");
        // V^T: thread = token pair x ranks; two tokens make one 4-byte store
        for (int i = tid; i < (kGradTok / 2) * 16 * RT; i += 256) {
            const int r = i % (16 * RT), t = lo + ch * kGradTok + 2 * (i / (16 * RT));
            const float v0 = (r < R && t < hi) ? J.V[(int64_t)P.plan.perm[t] * R + r] : 0.0f;
            const float v1 = (r < R && t + 1 < hi) ? J.V[(int64_t)P.plan.perm[t + 1] * R + r] : 0.0f;
#pragma unroll
            for (int s = 0; s < SPL; ++s)
                *reinterpret_cast<uint32_t*>(gs + 2 * kG + (s * 16 * RT + r) * kGradVRow + (i / (16 * RT)) * 4) =
                    split_pair(v0, v1, s);
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kGradTok / 16; ++kk) {
            // operand B: tokens 16 kk .. +16 x this warp's 16 columns; matrices (k 0-7, n 0-7), (k 8-15, n 0-7), (.., n 8-15)
            uint32_t bf[4];
            ldsm4t(bf, sG + buf * kG + (16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8) * kGradGRow +
                           (16 * warp + (lane >> 4) * 8) * 2);
#pragma unroll
            for (int s = 0; s < SPL; ++s)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    uint32_t af[4];
                    ldsm4(af, sV + (s * 16 * RT + 16 * i + (lane & 15)) * kGradVRow + (16 * kk + (lane >> 4) * 8) * 2);
                    mma16816(acc[i][0], af[0], af[1], af[2], af[3], bf[0], bf[1]);
                    mma16816(acc[i][1], af[0], af[1], af[2], af[3], bf[2], bf[3]);
                }
        }
        __syncthreads();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // this CTA's sums [16 RT][128] in shared memory, then the cluster's in order
    float* sum = reinterpret_cast<float*>(gs);
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float* p = sum + (16 * i + g) * kGradCols + 16 * warp + 8 * t + 2 * c;
            *reinterpret_cast<float2*>(p) = make_float2(acc[i][t][0], acc[i][t][1]);
            *reinterpret_cast<float2*>(p + 8 * kGradCols) = make_float2(acc[i][t][2], acc[i][t][3]);
        }
    cluster.sync();
    for (int i = cr * 256 + tid; i < R * kGradCols; i += 256 * CL) {
        const int r = J.by_column ? i % R : i / kGradCols, cc = J.by_column ? i / R : i % kGradCols;
        if (c0 + cc >= J.C) continue;
        float v = 0.0f;
        for (int q = 0; q < CL; ++q) v += cluster.map_shared_rank(sum, q)[r * kGradCols + cc];
        const int64_t at = J.by_column ? ((int64_t)a * J.C + c0 + cc) * R + r : ((int64_t)a * R + r) * J.C + c0 + cc;
        if (P.out_bf16)
            reinterpret_cast<__nv_bfloat16*>(J.out)[at] = __float2bfloat16_rn(v);
        else
            reinterpret_cast<float*>(J.out)[at] = v;
    }
    cluster.sync();
}

template <int RT, int SPL>
static int grad_launch(const GradParams& P, int64_t blocks, int cl, cudaStream_t stream) {
    constexpr int kV = SPL * 16 * RT * kGradVRow, kG = kGradTok * kGradGRow;
    constexpr int kSum = 16 * RT * kGradCols * 4;
    constexpr int kBytes = (2 * kG + kV) > kSum ? (2 * kG + kV) : kSum;
    static PerDevice once;
    int v = 0;
    int st = per_device(once, &v, [](int& x) {
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_lora_grad<RT, SPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes));
        x = 1;
        return SHERRY_OK;
    });
    if (st) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(blocks * cl));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cl;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    SHERRY_CUDA_CHECK(cudaLaunchKernelEx(&cfg, k_lora_grad<RT, SPL>, P));
    return SHERRY_OK;
}

int lora_grad_launch(const LoraGradJob* jobs, int count, int R, int n_adapters, int64_t M, const LoraPlan& plan,
                     int out_bf16, int sms, cudaStream_t stream) {
    GradParams P{};
    int64_t blocks = 0;
    for (int j = 0; j < 2; ++j) {
        P.job[j] = jobs[j < count ? j : 0];
        P.cblocks[j] = (int)((P.job[j].C + kGradCols - 1) / kGradCols);
        if (j < count) blocks += (int64_t)P.cblocks[j] * n_adapters;
    }
    P.plan = plan;
    P.R = R;
    P.n_adapters = n_adapters;
    P.out_bf16 = out_bf16;
    // tokens split until there are CTAs enough, each with a few chunks on average
    const int64_t chunks = M / kGradTok / n_adapters;
    int cl = 1;
    while (cl < 8 && blocks * cl < 2 * (int64_t)sms && chunks >= 4 * cl) cl *= 2;
    if (blocks * cl > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    const int rt = (R + 15) / 16;
    // bf16 gradients: two terms of V (16 bits) are 2^-8 of their rounding; fp32: all 24 bits
    if (out_bf16) {
        if (rt <= 1) return grad_launch<1, 2>(P, blocks, cl, stream);
        if (rt <= 2) return grad_launch<2, 2>(P, blocks, cl, stream);
        if (rt <= 4) return grad_launch<4, 2>(P, blocks, cl, stream);
        return grad_launch<8, 2>(P, blocks, cl, stream);
    }
    if (rt <= 1) return grad_launch<1, 3>(P, blocks, cl, stream);
    if (rt <= 2) return grad_launch<2, 3>(P, blocks, cl, stream);
    if (rt <= 4) return grad_launch<4, 3>(P, blocks, cl, stream);
    return grad_launch<8, 3>(P, blocks, cl, stream);
}

}  // namespace sherry
