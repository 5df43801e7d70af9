// dgrad.cu -- input gradient of the packed linear, with the adapters' share:
//
//   dX[m][k] = sum_n dY[m][n] t[n][k] alpha(n,k)  +  sum_r P[m][r] A_a[r][k]
//
// (the layer is Y = X (T alpha)^T, "Sherry, Tequila and Fairies in Python" section
// 1.1: F.linear; a = ids[m] is the token's adapter and P = s_a dY B_a, lora.cu).
//
// The sum runs over weight rows n, whose scale changes with every n: unlike in the
// forward pass alpha cannot be taken out of a group's sum, so it enters the bf16
// operand, as T = 2 terms, t hi and t lo with hi = bf16(alpha / unit) and lo = bf16 of
// what is left.  They keep alpha to 2^-18 of itself, below the fp32 sums' own error, so
// that dX is rounded once, to its bf16 (one term instead would halve the tensor work, but
// an error of 0.0013 in the mean square beside the rounding's 0.0017).  A per-tensor
// scale needs one term: unit makes it 1.71875 exactly, and is undone in fp32 at the end.
//
// CTA tile: 128 TM tokens x 256 k (TM = 1 or 2 MMAs of 128 x 256 that share the
// decoded operand); n runs in stages of 64 / T rows, 64 operand rows with the second
// terms after the first.  dY is operand A, K-major, by TMA, and multiplied by both.
// The weights are operand B in the layout they unpack to, k contiguous (MN-major,
// 128-byte swizzle): a decode thread owns 64 / T consecutive k of a row, looks each
// block of 4 up in the 32 patterns, scales it with one packed multiply per pair and term and
// stores 16 bytes at a time, conflict-free (eight lanes take the eight rows of a swizzle
// atom).  After the last rows come the adapters' stages, one or two per slot and 64
// ranks, all by TMA: operand B is A_a as it is stored, operand A is P of the tile's
// tokens, zero for tokens of other adapters, in 2 bf16 terms (16 significant bits).
// An adapter whose A is not finite would make NaN of those zeros: it gets no stage, and
// the epilogue adds its product to its own tokens' rows, element by element.
//   warps 0..7   epilogue: TMEM -> registers -> dX (bf16) or, where n is split over
//                CTAs, fp32 partial sums that k_dgrad_join adds in order
//   warps 8..23  decode, two groups that take the stages in turn: a stage's waits, lookups and
//                fences are a chain of some 1500 cycles (one term, 4096 x 8192 x 2048: 116 -> 107 us)
//   warp 24      TMA, warp 25 MMA issue
// n is split where there are fewer tiles than SMs.
//
// Bound by the tensor cores: at 4096 x 8192 x 2048 with adapters of rank 32 the tensor pipe is
// 89% busy on the 128 SMs that have a tile.  Without adapters 174 us for two terms (the
// operations of both at the measured rate: 165), 111 for a per-tensor scale (83).
#include "common.cuh"
#include "lora.cuh"
#include "lut.cuh"
#include "tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace sherry {

constexpr int kGDecGroups = 2;               // groups of eight decode warps, a stage each in turn
constexpr int kGTmaWarp = 8 + 8 * kGDecGroups, kGMmaWarp = kGTmaWarp + 1;
constexpr int kGThreads = 32 * (kGMmaWarp + 1);
constexpr int kGK = 256;                     // k columns per tile
constexpr int kGN = 64;                      // operand rows per stage: weight rows x terms of alpha
constexpr int kGBBytes = kGN * kGK * 2;      // 32 KB of decoded weights per stage
constexpr int kGABytes = 128 * kGN * 2;      // 16 KB: 64 columns of dY, or of P, for 128 tokens
constexpr int kGStageSum = 192 * 1024;       // 3 stages of 64 KB (TM = 2, one term) or 4 of 48 KB
constexpr int kGSmem = kGStageSum + 256 + 1024;
constexpr int kGMaxStages = 4;
static_assert(128 * (kGK * 4 + 16) <= kGStageSum && 256 * (kGK * 2 + 16) <= kGStageSum, "results fit the stages");

// bf16 x bf16 -> fp32, M = 128, N = 256, A K-major, B MN-major (bit 16)
constexpr uint32_t kGIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(kGK >> 3) << 17) |
                             ((uint32_t)(128 >> 4) << 24);

struct GParams {
    const uint32_t* idx;
    const uint8_t* sgn;
    const float* scales;
    int64_t nscales;
    void* out;             // dX bf16 [M][K], or fp32 partial sums [splits][M][K]
    int M, N, K, words;
    int gran, group, spr;
    int mtiles, ktiles, splits, nstages;
    // adapters (LORA)
    LoraPlan plan;
    const uint16_t* A;   // bf16 [n_adapters][R][K]
    const uint16_t* Pi;  // the image of P
    int R, terms;
    int rp;
    int terms_box;  // terms of P in one tile of 64 columns: 2, or 1
    int rows_box;   // rows of A_a per load
};

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <int TM, bool LORA, int T>
__global__ void __launch_bounds__(kGThreads, 1)
k_dgrad(const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap ypmap,
        const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap amap,
        const __grid_constant__ GParams P) {
    constexpr int ROWS = kGN / T;                      // weight rows per stage
    constexpr int YB = 128 * ROWS * 2;                 // bytes of dY per 128 tokens and stage
    constexpr int AB = TM * YB > kGABytes ? TM * YB : kGABytes;  // bytes of operand A: dY, or P's tiles
    constexpr int SB = AB + kGBBytes;                  // bytes per stage
    constexpr int ST = kGStageSum / SB;                // stages
    constexpr int AC = 2 / TM;                         // accumulators of TM x 256 columns in TMEM
    static_assert(ST <= kGMaxStages && SB % 1024 == 0, "stage plan");
    extern __shared__ __align__(1024) unsigned char gsmem[];
    __shared__ uint64_t bars[3 * kGMaxStages + 5];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    __shared__ volatile int skip_s[kGMaxStages];  // LORA: the stage holds nothing

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(gsmem) + 1023u) & ~1023u;
    const uint32_t table = base + kGStageSum;  // 256-aligned
    const uint32_t bar0 = smem_u32(&bars[0]);
    auto full_a = [&](int s) { return bar0 + 8u * s; };
    auto full_b = [&](int s) { return bar0 + 8u * (ST + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * ST + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (3 * ST + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (3 * ST + 2 + b); };
    const uint32_t drain = bar0 + 8u * (3 * ST + 4);

    const int items = P.mtiles * P.ktiles * P.splits;
    // item -> token tile, k tile, stages [st0, st1) of the rows and slots [sl0, sl1) of its one or two
    // token tiles (from slh on those of the second)
    struct Item {
        int mt, kt, sp, st0, st1, sl0, slh, sl1;
    };
    const int rblocks = LORA ? (P.rp + 63) / 64 : 0;
    // stages per slot and 64 ranks: P's terms in one stage (as one tile or, with room, two), or one after the other
    const int tstages = LORA && AB < 2 * kGABytes && P.terms_box == 1 ? 2 : 1;
    auto item = [&](int w) {
        Item it;
        it.kt = w % P.ktiles;
        const int q = w / P.ktiles;
        it.mt = q % P.mtiles;
        it.sp = q / P.mtiles;
        it.st0 = (int)((int64_t)P.nstages * it.sp / P.splits);
        it.st1 = (int)((int64_t)P.nstages * (it.sp + 1) / P.splits);
        it.sl0 = it.slh = it.sl1 = 0;
        if constexpr (LORA) {  // this split's share of the slots
            const int t0 = P.plan.tile_b[it.mt * TM], t1 = P.plan.tile_b[it.mt * TM + 1];
            const int t2 = TM == 2 && it.mt * TM + 2 <= P.plan.tiles ? P.plan.tile_b[it.mt * TM + 2] : t1;
            it.sl0 = t0 + (t2 - t0) * it.sp / P.splits;
            it.sl1 = t0 + (t2 - t0) * (it.sp + 1) / P.splits;
            it.slh = min(max(t1, it.sl0), it.sl1);
        }
        return it;
    };

    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int s = 0; s < ST; ++s) {
            mbar_init(full_a(s), 1);
            mbar_init(full_b(s), 256);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 256);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (threadIdx.x < 32) {
        // the 32 patterns: low halves (weights 0, 1), then high halves, conflict-free
        const uint2 e = decode_block_bf16((uint32_t)threadIdx.x & 15u, (uint32_t)threadIdx.x >> 4);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + 4u * threadIdx.x), "r"(e.x) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + 128u + 4u * threadIdx.x), "r"(e.y) : "memory");
    }
    if (warp == kGMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    // LORA: the plan, and dY in its order, are ready when this kernel is launched (k_lora_down lets it
    // start only then); P's image is waited for where it is loaded.  The adapters' gradients, launched
    // next, may start as soon as the image is there.
    if (LORA && warp == kGTmaWarp && lane == 1) {
        pdl_wait();
        pdl_trigger();
    }
    const bool permuted = LORA && P.plan.may_permute && P.plan.head[0] != 0;

    if (warp < 8) {
        // ---------------- epilogue: lane = token; the two groups of four warps take the two
        // token halves (TM = 2) or the two halves of the columns (TM = 1) ----------------
        const int q = warp & 3, half = warp >> 2;
        constexpr int COLS = TM == 2 ? kGK : kGK / 2;
        const float unit = P.splits == 1 ? dgrad_unit(P.scales, P.nscales) : 1.0f;
        auto round8 = [&](const uint32_t* x) {  // eight columns of dX
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 p =
                    __floats2bfloat162_rn(__uint_as_float(x[2 * i]) * unit, __uint_as_float(x[2 * i + 1]) * unit);
                h[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            return make_uint4(h[0], h[1], h[2], h[3]);
        };
        // A CTA with one item has its stages to itself once the last product is done: results go through them, so
        // that a store covers whole lines of a row and not 16 bytes of 32 rows
        // (one term, 256 x 2048 x 2048: 15.4 -> 13.5 us)
        const bool staged = items <= (int)gridDim.x;
        const int pitch = kGK * (P.splits == 1 ? 2 : 4) + 16;  // bytes
        const int c0 = TM == 2 ? 0 : half * COLS;
        unsigned char* out_s = gsmem + (base - smem_u32(gsmem)) + ((TM == 2 ? half * 128 : 0) + q * 32 + lane) * pitch;
        int b = 0;
        uint32_t bph = 0;
        for (int w = blockIdx.x; w < items; w += gridDim.x) {
            const Item it = item(w);
            int bad_slot = -1;  // the row's slot where its adapter's A is not finite
            if (LORA && it.sl0 < it.sl1) {
                pdl_wait();
                const int first = TM == 2 && half ? it.slh : it.sl0, last = TM == 2 && !half ? it.slh : it.sl1;
                for (int s0 = first; s0 < last; s0 += 32) {  // a lane per slot
                    unsigned bad = __ballot_sync(kFull, s0 + lane < last && P.plan.bad[P.plan.slot_a[min(s0 + lane, last - 1)]]);
                    for (; bad; bad &= bad - 1) {
                        const int sl = s0 + __ffs(bad) - 1;
                        if (P.plan.mask[4 * sl + q] >> lane & 1u) bad_slot = sl;
                    }
                }
            }
            if (!mbar_wait(acc_full(b), bph, &abort_s)) break;
            tc_fence_after();
            const int64_t pos0 = (int64_t)it.mt * (TM * 128) + (TM == 2 ? half * 128 : 0) + q * 32;
            int64_t m = pos0 + lane;
            if (LORA && permuted && m < P.M) m = P.plan.perm[m];
            const int kc = it.kt * kGK + (TM == 2 ? 0 : half * COLS);
            const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kGK + half * COLS);
#pragma unroll 1
            for (int c = 0; c < COLS / 32; ++c) {
                uint32_t v[32];
                SHERRY_TMEM_LD32(t_row + 32 * c, v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                const int k = kc + 32 * c;
                if (LORA && bad_slot >= 0 && k < P.K) {
                    const uint16_t* pr = P.Pi + ((int64_t)bad_slot * kLoraTile + q * 32 + lane) * (P.terms * P.rp);
                    const uint16_t* ar = P.A + (int64_t)P.plan.slot_a[bad_slot] * P.R * P.K + k;
#pragma unroll 1
                    for (int r = 0; r < P.R; ++r) {
                        float p = 0.0f;
                        for (int t = P.terms - 1; t >= 0; --t) p += bf16lo(pr[t * P.rp + r]);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(fmaf(p, bf16lo(ar[(int64_t)r * P.K + j]), __uint_as_float(v[j])));
                    }
                }
                if (staged) {
                    unsigned char* dst = out_s + (c0 + 32 * c) * (P.splits == 1 ? 2 : 4);
                    if (P.splits == 1) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(dst)[j] = round8(v + 8 * j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            reinterpret_cast<uint4*>(dst)[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                } else if (m < P.M && k < P.K) {
                    if (P.splits == 1) {
                        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(P.out) + m * P.K + k);
#pragma unroll
                        for (int j = 0; j < 4; ++j) dst[j] = round8(v + 8 * j);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<float*>(P.out) +
                                                              ((int64_t)it.sp * P.M + m) * P.K + k);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
            }
            if (staged) {
                // this warp's rows, whole lines at a time
                __syncwarp();
                const int esz = P.splits == 1 ? 2 : 4, per = 32 * 16 / (COLS * esz);  // rows a store takes: one, or two
                const int lanes = 32 / per, col = (lane % lanes) * (16 / esz);        // the lane's first column of a row
                const int rows = (int)max((int64_t)0, min((int64_t)32, P.M - pos0));
#pragma unroll 4
                for (int i = 0; i < rows; i += per) {
                    const int row = i + lane / lanes;
                    const int mr = __shfl_sync(kFull, (int)m, row);
                    if (row < rows && kc + col < P.K)
                        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(P.out) +
                                                  (((int64_t)it.sp * P.M + mr) * P.K + kc + col) * esz) =
                            *reinterpret_cast<const uint4*>(out_s + (row - lane) * pitch + (c0 + col) * esz);
                }
            }
            tc_fence_before();
            mbar_arrive(acc_empty(b));
            if (++b == AC) { b = 0; bph ^= 1u; }
        }
    } else if (warp < kGTmaWarp) {
        // ---------------- decode: eight lanes = the eight rows of one swizzle atom, so their 16-byte
        // stores cover all banks; a thread has two words of a row, or (T = 2) both terms of one ----------------
        const int dt = threadIdx.x & 255, group = (warp - 8) >> 3;
        constexpr int W = 2 / T;  // words of a thread
        const int r = (T == 1 ? dt >> 5 : (dt >> 5) & 3) * 8 + (lane & 7);
        const int word = T == 1 ? 2 * (lane >> 3) : 4 * (dt >> 7) + (lane >> 3);  // (of the tile's eight)
        const uint32_t brow = (uint32_t)(AB + (word >> 1) * (kGN * 128) + (r >> 3) * 1024 + (r & 7) * 128);
        const float inv = 1.0f / dgrad_unit(P.scales, P.nscales);
        int s = 0;
        uint32_t ph = 0;
        int turn = 0;  // stages so far: a group waits for one of two, and so for every one before it
        bool ok = true;
        for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
            const Item it = item(w);
            const int kw = it.kt * (kGK / 32) + word;  // first of this thread's words
            int sc[W];                                 // their scales' places within a row
#pragma unroll
            for (int h = 0; h < W; ++h) sc[h] = P.gran == SHERRY_PER_GROUP ? 32 * (kw + h) / P.group : 0;
            auto fetch = [&](int st, uint32_t* wd, uint32_t* sg, float* al) {
                const int64_t n = (int64_t)st * ROWS + r;
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    wd[h] = 0u;
                    sg[h] = 0u;
                    al[h] = 0.0f;
                    if (st < it.st1 && n < P.N && kw + h < P.words) {
                        wd[h] = __ldg(P.idx + n * P.words + kw + h);
                        sg[h] = __ldg(P.sgn + n * P.words + kw + h);
                        al[h] = __ldg(P.scales + (P.gran == SHERRY_PER_TENSOR ? 0 : n * P.spr + sc[h]));
                    }
                }
            };
            uint32_t wd[W], sg[W];
            float al[W];
            fetch(it.st0 + ((turn ^ group) & 1), wd, sg, al);
            for (int st = it.st0; st < it.st1; ++st, ++turn) {
                if (kGDecGroups > 1 && ((turn ^ group) & 1)) {  // the other group's
                    if (++s == ST) { s = 0; ph ^= 1u; }
                    continue;
                }
                uint32_t nwd[W], nsg[W];
                float nal[W];
                fetch(st + kGDecGroups, nwd, nsg, nal);
                if (!mbar_wait(empty(s), ph ^ 1u, &abort_s)) { ok = false; break; }
                const uint32_t dst = base + (uint32_t)(s * SB) + brow;
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    uint32_t ev, od;
                    spread_word(wd[h], sg[h], ev, od);
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t at = __byte_perm((j & 1) ? od : ev, table, (uint32_t)(j >> 1) | 0x7650u);
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[2 * j]) : "r"(at));
                        asm volatile("ld.shared.u32 %0, [%1+128];" : "=r"(v[2 * j + 1]) : "r"(at));
                    }
                    float x = al[h] * inv, same = x;
                    const int half = T == 1 ? h : word & 1;  // of the 64 k that stand together
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        const uint32_t a = split_next(x, same);  // the term twice; x keeps what is left
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            sts128(dst + (uint32_t)(t * (ROWS * 128) + ((4 * half + c) ^ (r & 7)) * 16),
                                   make_uint4(mul_bf16x2(v[4 * c], a), mul_bf16x2(v[4 * c + 1], a),
                                              mul_bf16x2(v[4 * c + 2], a), mul_bf16x2(v[4 * c + 3], a)));
                    }
                }
                fence_proxy_async();
                mbar_arrive(full_b(s));
                if (++s == ST) { s = 0; ph ^= 1u; }
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    wd[h] = nwd[h];
                    sg[h] = nsg[h];
                    al[h] = nal[h];
                }
            }
            if constexpr (LORA) {
                // the adapters' stages take their turns without this warp, which waits for them all
                // the same: no barrier gets two phases ahead of it
                for (int i = (it.sl1 - it.sl0) * rblocks * tstages; i > 0 && ok; --i, ++turn) {
                    ok = mbar_wait(empty(s), ph ^ 1u, &abort_s);
                    if (++s == ST) { s = 0; ph ^= 1u; }
                }
            }
        }
    } else if (warp == kGTmaWarp) {
        // ---------------- TMA: dY tiles; in an adapters' stage both operands, P and A_a ----------------
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int issued[ST] = {};  // phases of full_a started per stage
            bool ok = true;
            for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const Item it = item(w);
                for (int st = it.st0; st < it.st1; ++st) {
                    if (!mbar_wait(empty(s), ph ^ 1u, &abort_s)) { ok = false; break; }
                    mbar_expect_tx(full_a(s), TM * YB);
#pragma unroll
                    for (int h = 0; h < TM; ++h)
                        tma_load_2d(base + (uint32_t)(s * SB + h * YB), LORA && permuted ? &ypmap : &ymap, st * ROWS,
                                    (it.mt * TM + h) * 128, full_a(s));
                    ++issued[s];
                    if (++s == ST) { s = 0; ph ^= 1u; }
                }
                if constexpr (LORA) {
                    // the next slot's adapter and state are loaded while this one's stages are waited for
                    int a1 = 0, bad1 = 0, a2 = 0;
                    if (it.sl0 < it.sl1) {
                        a1 = P.plan.slot_a[it.sl0];
                        a2 = P.plan.slot_a[min(it.sl0 + 1, it.sl1 - 1)];
                        pdl_wait();
                        bad1 = P.plan.bad[a1];
                    }
                    for (int sl = it.sl0; sl < it.sl1 && ok; ++sl) {
                        const int a = a1, bad = bad1;
                        a1 = a2;
                        bad1 = P.plan.bad[a1];
                        a2 = P.plan.slot_a[min(sl + 2, it.sl1 - 1)];
                        for (int u = 0; u < rblocks * tstages; ++u) {
                            if (!mbar_wait(empty(s), ph ^ 1u, &abort_s)) { ok = false; break; }
                            skip_s[s] = bad;
                            if (bad) {
                                mbar_arrive(full_a(s));
                                ++issued[s];
                                if (++s == ST) { s = 0; ph ^= 1u; }
                                continue;
                            }
                            const int r0 = 64 * (u / tstages), t0 = u % tstages;
                            const int boxes = 2 / (P.terms_box * tstages);
                            const uint32_t dst = base + (uint32_t)(s * SB);
                            mbar_expect_tx(full_a(s), (uint32_t)(boxes * kGABytes + 4 * P.rows_box * 128));
                            for (int i = 0; i < boxes; ++i)
                                tma_load_2d(dst + (uint32_t)(i * kGABytes), &pmap, (t0 + i) * P.rp + r0, sl * kLoraTile,
                                            full_a(s));
                            for (int c = 0; c < kGK / 64; ++c)
                                tma_load_3d(dst + (uint32_t)(AB + c * kGN * 128), &amap, it.kt * kGK + 64 * c,
                                            r0, a, full_a(s));
                            ++issued[s];
                            if (++s == ST) { s = 0; ph ^= 1u; }
                        }
                    }
                }
            }
            // every load lands before the CTA's shared memory goes away
            for (int i = 0; i < ST; ++i)
                if (issued[i] > 0) mbar_drain(full_a(i), (uint32_t)((issued[i] - 1) & 1));
        }
    } else {
        // ---------------- MMA issue ----------------
        if (lane == 0) {
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 0;
            uint32_t bmask = 0;  // phase parities of full_b per stage (the adapters' stages do not use it)
            bool ok = true;
            for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const Item it = item(w);
                if (!mbar_wait(acc_empty(b), bph ^ 1u, &abort_s)) break;
                tc_fence_after();
                for (int st = it.st0; st < it.st1; ++st) {
                    if (!mbar_wait(full_a(s), ph, &abort_s) || !mbar_wait(full_b(s), (bmask >> s) & 1u, &abort_s)) {
                        ok = false;
                        break;
                    }
                    bmask ^= 1u << s;
                    tc_fence_after();
                    const uint64_t da = T == 1 ? smem_desc(base + (uint32_t)(s * SB)) : smem_desc_64(base + (uint32_t)(s * SB));
                    const uint64_t db = smem_desc_mn(base + (uint32_t)(s * SB + AB), kGN * 128);
#pragma unroll
                    for (int kk = 0; kk < kGN / 16; ++kk)  // 16 rows: +32 bytes in A's row, two 8-row atoms of B
#pragma unroll
                        for (int h = 0; h < TM; ++h)
                            mma_bf16_ss(tmem + (uint32_t)((TM == 2 ? h : b) * kGK),
                                        da + (uint64_t)((h * YB) >> 4) + (uint64_t)(2 * (kk % (ROWS / 16))),
                                        db + (uint64_t)(2 * kk * (1024 >> 4)), kGIdesc,
                                        (st == it.st0 && kk == 0) ? 0u : 1u);
                    mma_commit(empty(s));
                    if (++s == ST) { s = 0; ph ^= 1u; }
                }
                if constexpr (LORA) {
                    for (int sl = it.sl0; sl < it.sl1 && ok; ++sl) {
                        const uint32_t td = tmem + (uint32_t)((TM == 2 ? (sl >= it.slh) : b) * kGK);
                        for (int u = 0; u < rblocks * tstages; ++u) {
                            if (!mbar_wait(full_a(s), ph, &abort_s)) { ok = false; break; }
                            tc_fence_after();
                            if (skip_s[s]) {
                                mma_commit(empty(s));
                                if (++s == ST) { s = 0; ph ^= 1u; }
                                continue;
                            }
                            const uint64_t dp = smem_desc(base + (uint32_t)(s * SB));
                            const uint64_t da = smem_desc_mn(base + (uint32_t)(s * SB + AB), kGN * 128);
                            const int n16 = min(4, (P.rp - 64 * (u / tstages)) / 16);
                            for (int i = 0; i < 2 / tstages; ++i) {  // the stage's terms: in one tile, or one tile each
                                const uint64_t term = (uint64_t)(P.terms_box == 2 ? i * P.rp / 8 : (i * kGABytes) >> 4);
                                for (int kk = 0; kk < n16; ++kk)
                                    mma_bf16_ss(td, dp + term + (uint64_t)(2 * kk), da + (uint64_t)(2 * kk * (1024 >> 4)),
                                                kGIdesc, 1u);
                            }
                            mma_commit(empty(s));
                            if (++s == ST) { s = 0; ph ^= 1u; }
                        }
                    }
                }
                if (!ok) break;
                mma_commit(acc_full(b));
                if (++b == AC) { b = 0; bph ^= 1u; }
            }
            mma_commit(drain);
            mbar_drain(drain, 0u);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kGMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// dX = (the splits' partial sums, in order) * unit, bf16
__global__ void __launch_bounds__(256) k_dgrad_join(const float* part, int splits, int64_t total, const float* scales, int64_t nscales,
                                                    uint16_t* out) {
    pdl_trigger();
    pdl_wait();
    const float unit = dgrad_unit(scales, nscales);
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= total) return;  // total = M * K, a multiple of 32
    float4 a = *reinterpret_cast<const float4*>(part + i);
#pragma unroll 8
    for (int s = 1; s < splits; ++s) {
        const float4 b = *reinterpret_cast<const float4*>(part + (int64_t)s * total + i);
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * unit, a.y * unit), hi = __floats2bfloat162_rn(a.z * unit, a.w * unit);
    *reinterpret_cast<uint2*>(out + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// ---- host -------------------------------------------------------------------------

// Stages of the adapters that a 128-token tile is likely to have
static int lora_stages(int64_t M, int n_adapters, int R) {
    if (n_adapters == 0) return 0;
    const int64_t tiles = (M + 127) / 128, slots = std::min<int64_t>({(tiles + n_adapters) / tiles, n_adapters, 128, M});
    const int rp = lora_rp(R);
    return (int)slots * (2 * rp <= 64 ? 1 : 2 * ((rp + 63) / 64));
}

struct GPlan {
    int tm, mtiles, ktiles, splits, nstages;
};
// bf16 terms of alpha
static int alpha_terms(const ProbShape& s) { return s.granularity == SHERRY_PER_TENSOR ? 1 : 2; }

// Two 128-token MMAs per CTA once that still gives every SM a tile (the decoded operand is then used
// twice); rows split over CTAs where there are fewer tiles than SMs, at least 4 stages each, or beside adapters
// 256 rows, since their gradients take the SMs that are left (group scales, 128 / 256 rows at least, in us: 280 x 616 x
// 2048 plain 14.4 / 16.5, with adapters 33 / 30; 64 x 2048 x 2048 16.4 / 16.5 and 31 / 27.5).  (With one term, 256-token
// tiles with split rows instead: 256 x 2048 x 2048 15 -> 20 us, 2171 x 2444 x 1920 43 -> 41 + 8 for the partial sums.)
// lstages: 64-row stages that a token tile's adapters are worth (at a time when its slots are not known)
static GPlan dgrad_plan(int64_t M, int64_t N, int64_t K, int terms, int lstages, int sms) {
    GPlan g;
    g.ktiles = (int)((K + kGK - 1) / kGK);
    g.tm = ((M + 255) / 256) * g.ktiles * 10 >= (int64_t)sms * 7 ? 2 : 1;
    g.mtiles = (int)((M + 128 * g.tm - 1) / (128 * g.tm));
    const int64_t tiles = (int64_t)g.mtiles * g.ktiles;
    g.nstages = (int)((N * terms + kGN - 1) / kGN);
    g.splits = 1;
    if (g.tm == 1 && tiles * 2 <= sms)
        g.splits = (int)std::max<int64_t>(1, std::min<int64_t>({sms / tiles, (g.nstages + lstages * terms) / (lstages ? 4 * terms : 4), g.nstages}));
    return g;
}

size_t dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int n_adapters, int R, int sms) {
    int splits = 1;  // the more of either form's
    for (int terms : {1, 2}) splits = std::max(splits, dgrad_plan(M, N, K, terms, lora_stages(M, n_adapters, R), sms).splits);
    return splits > 1 ? (size_t)splits * (size_t)(M * K) * sizeof(float) : 0;
}

int64_t dgrad_ctas(const ProbShape& s, int64_t M, int n_adapters, int R, int sms) {
    const GPlan g = dgrad_plan(M, s.N, s.K, alpha_terms(s), lora_stages(M, n_adapters, R), sms);
    return std::min<int64_t>((int64_t)g.mtiles * g.ktiles * g.splits, sms);
}

int dgrad_launch(const ProbShape& s, const uint32_t* idx, const uint8_t* sgn, const float* scales, const uint16_t* dY,
                 int64_t ldy, int64_t M, uint16_t* dX, const LoraGradArgs* lora, void* workspace, int sms,
                 cudaStream_t stream) {
    const int terms = alpha_terms(s);
    const GPlan g = dgrad_plan(M, s.N, s.K, terms, lora ? lora_stages(M, lora->n_adapters, lora->R) : 0, sms);
    CUtensorMap map;
    int st = encode_2d(&map, dY, ldy, M, 128, kGN / terms);
    if (st) return st;
    GParams P{};
    P.idx = idx;
    P.sgn = sgn;
    P.scales = scales;
    P.nscales = scale_count(s);
    P.out = g.splits > 1 ? workspace : dX;
    P.M = (int)M;
    P.N = (int)s.N;
    P.K = (int)s.K;
    P.words = (int)(s.K / 32);
    P.gran = s.granularity;
    P.group = s.granularity == SHERRY_PER_GROUP ? s.group : 32;
    P.spr = s.granularity == SHERRY_PER_GROUP ? (int)(s.K / s.group) : 1;
    P.mtiles = g.mtiles;
    P.ktiles = g.ktiles;
    P.splits = g.splits;
    P.nstages = g.nstages;
    CUtensorMap ypmap = map, pmap = map, amap = map;
    if (lora) {
        P.plan = lora->plan;
        P.A = lora->A;
        P.Pi = lora->P.data;
        P.R = lora->R;
        P.terms = lora->P.terms;
        P.rp = lora->P.rp;
        P.terms_box = 2 * P.rp <= 64 ? 2 : 1;
        P.rows_box = std::min(P.rp, 64);
        if (lora->Gp && (st = encode_2d(&ypmap, lora->Gp, ldy, M, 128, kGN / terms))) return st;
        st = encode_2d(&pmap, lora->P.data, lora->P.terms * P.rp, (int64_t)lora->plan.max_slots * kLoraTile, 128);
        if (!st) st = encode_3d(&amap, lora->A, s.K, lora->R, lora->n_adapters, P.rows_box);
        if (st) return st;
    }
    static PerDevice once;
    int v = 0;
    st = per_device(once, &v, [](int& x) {
        for (auto kernel : {k_dgrad<1, false, 1>, k_dgrad<1, false, 2>, k_dgrad<1, true, 1>, k_dgrad<1, true, 2>,
                            k_dgrad<2, false, 1>, k_dgrad<2, false, 2>, k_dgrad<2, true, 1>, k_dgrad<2, true, 2>})
            SHERRY_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem));
        x = 1;
        return SHERRY_OK;
    });
    if (st) return st;
    const int64_t items = (int64_t)g.mtiles * g.ktiles * g.splits;
    if (items > 0x7fffffff) return SHERRY_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)std::min<int64_t>(items, sms);
    auto of = [&](auto one, auto two) { return terms == 1 ? one : two; };
    auto kernel = g.tm == 2 ? (lora ? of(k_dgrad<2, true, 1>, k_dgrad<2, true, 2>) : of(k_dgrad<2, false, 1>, k_dgrad<2, false, 2>))
                            : (lora ? of(k_dgrad<1, true, 1>, k_dgrad<1, true, 2>) : of(k_dgrad<1, false, 1>, k_dgrad<1, false, 2>));
    return launch_after(kernel, grid, kGThreads, kGSmem, stream, 1, lora != nullptr, map, ypmap, pmap, amap, P);
}

int dgrad_join_launch(const ProbShape& s, const float* scales, int64_t M, uint16_t* dX, const void* workspace,
                      int n_adapters, int R, int sms, cudaStream_t stream) {
    const GPlan g = dgrad_plan(M, s.N, s.K, alpha_terms(s), lora_stages(M, n_adapters, R), sms);
    if (g.splits == 1) return SHERRY_OK;
    const int64_t total = M * s.K;
    return launch_after(k_dgrad_join, (unsigned)((total / 4 + 255) / 256), 256, 0, stream, 1, true,
                        static_cast<const float*>(workspace), g.splits, total, scales, scale_count(s), dX);
}

int dgrad_status_take() { return tc_status_take(); }

}  // namespace sherry
