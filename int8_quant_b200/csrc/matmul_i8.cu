// matmul_i8.cu — the projections of a W8A8 layer: the product of INT8 codes with a scale per
// token and a scale per output channel,
//   out[t,n] = s_t[t] * s_w[n] * sum_k q[t,k] * Wq[n,k] + bias[n]      (bf16),
// the sum exact in INT32 on the tensor cores (tcgen05.mma kind::i8, operands by TMA with the
// 128-byte swizzle in K slices of 128; what lies outside the matrices arrives as zeros).
//
// In both kernels the MMA's rows (TMEM lanes) are output channels and its columns tokens, so
// a thread of the epilogue owns a channel: its scale and bias stay in registers, and a warp
// stores 32 consecutive channels of a token at a time, 64 contiguous bytes whatever n's
// alignment.
//
//   matmul_pair_kernel  many tokens: a CTA pair (cta_group::2) per 256 x 256 output tile,
//                       persistent, a 6-stage ring, two accumulators.
//   matmul_few_kernel   few tokens or few tiles: one 128-channel tile of up to 128 tokens
//                       per cluster, the K axis split over the cluster's CTAs and the
//                       INT32 partial sums joined through distributed shared memory.
//
// Every wait is bounded; an expired wait raises the CTA's abort flag and records
// SSD_ERR_TIMEOUT in the status word.
#include "kernels.h"
#include "tc.cuh"

namespace ssd {

namespace {

constexpr int kBK = 128;                              // K slice: one 128-byte swizzled row
constexpr int kWarps = 6;                             // 0 TMA, 1 MMA, 2-5 epilogue
constexpr long long kDrainLimit = 400000000LL;        // cycles an aborting CTA waits for its copies and MMAs

struct MatmulArgs {
    int T, K, N;
    int tiles_t, tiles_n;
    const float* s_t;
    const float* s_w;
    const float* bias;
    uint16_t* out;
    int* status;
};

// 32 columns (tokens t0 ..) of this thread's channel: scale and store.  `dst` points at token
// t0's element; `live` tokens of the 32 exist.
__device__ __forceinline__ void store_tokens(const uint32_t (&v)[32], const float* __restrict__ s_t, float sw,
                                             float bias, uint16_t* dst, long long N, int live) {
    if (live >= 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float f = fmaf((float)(int)v[j] * sw, __ldg(s_t + j), bias);
            *dst = float_to_bf16_bits(f);
            dst += N;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < live) {
                const float f = fmaf((float)(int)v[j] * sw, __ldg(s_t + j), bias);
                *dst = float_to_bf16_bits(f);
                dst += N;
            }
        }
    }
}

// ---------------------------------------------------------------- many tokens: CTA pairs

namespace pair {

constexpr int kRows = 128;                            // rows of each operand per CTA; the pair's tile is 256 x 256
constexpr int kTile = 2 * kRows;
constexpr int kStages = 6, kAcc = 2;
constexpr int kOpBytes = kRows * kBK;
constexpr int OFF_A = 0, OFF_B = kStages * kOpBytes, OFF_BAR = 2 * kStages * kOpBytes;
constexpr int B_FULL = 0, B_EMPTY = kStages, B_AFULL = 2 * kStages, B_AEMPTY = B_AFULL + kAcc,
              B_DRAIN = B_AEMPTY + kAcc, NBAR = B_DRAIN + 1;
constexpr int OFF_FLAG = OFF_BAR + NBAR * 8, OFF_TMEM = OFF_FLAG + 8, SMEM = OFF_TMEM + 8;
constexpr int kGroup = 8;                             // token tiles that share the weights while they are in L2

// Tile `t` of the persistent order: groups of kGroup token tiles, in a group all channel
// tiles, the group's token tiles fastest.
__device__ __forceinline__ void tile_at(const MatmulArgs& p, long long t, int* n0, int* t0) {
    const long long per = (long long)kGroup * p.tiles_n;
    const int g = (int)(t / per);
    const int r = (int)(t % per);
    const int left = p.tiles_t - g * kGroup;
    const int in = left < kGroup ? left : kGroup;
    *t0 = (g * kGroup + r % in) * kTile;
    *n0 = (r / in) * kTile;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWarps * 32, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ MatmulArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_FLAG);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const bool leader = rank == 0;
    const int nk = (p.K + kBK - 1) / kBK;
    const long long tiles = (long long)p.tiles_t * p.tiles_n;
    const int pairs = gridDim.x >> 1, me = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        // an accumulator is free once the four epilogue warps of both CTAs have read it
        for (int i = 0; i < NBAR; ++i) tc::mbar_init(bar + i, i >= B_AEMPTY && i < B_DRAIN ? 8 : 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tmem_slot, kAcc * kTile);
        tc::tmem_relinquish_pair();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            tc::prefetch_tmap(&tm_w);
            tc::prefetch_tmap(&tm_q);
            long long kc = 0;                                     // K slices issued so far (ring position)
            bool ok = true;
            for (long long t = me; ok && t < tiles; t += pairs) {
                int n0, t0;
                tile_at(p, t, &n0, &t0);
                n0 += (int)rank * kRows;
                t0 += (int)rank * kRows;
                for (int k = 0; k < nk; ++k, ++kc) {
                    const int s = (int)(kc % kStages);
                    if (!(ok = tc::wait_or_abort(bar + B_EMPTY + s, (((uint32_t)(kc / kStages)) & 1) ^ 1, abort_flag,
                                                 p.status, kStatusTimeout)))
                        break;
                    // both CTAs' loads of a stage count on the even CTA's barrier
                    if (leader) tc::mbar_arrive_expect_tx(bar + B_FULL + s, 4 * kOpBytes);
                    const uint32_t full = tc::map_rank(tc::smem_u32(bar + B_FULL + s), 0);
                    tc::tma_load_2d_pair(sm + OFF_A + s * kOpBytes, &tm_w, full, k * kBK, n0);
                    tc::tma_load_2d_pair(sm + OFF_B + s * kOpBytes, &tm_q, full, k * kBK, t0);
                }
            }
            if (!ok && leader)                                    // the copies in flight land before the CTA ends
                for (long long j = kc > kStages ? kc - kStages : 0; j < kc; ++j)
                    tc::mbar_wait(bar + B_FULL + j % kStages, ((uint32_t)(j / kStages)) & 1, kDrainLimit);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint32_t idesc = tc::idesc_s8_s32(kTile, kTile, tc::kMajorK, tc::kMajorK);
            long long kc = 0;
            int it = 0;                                           // tiles of this pair so far
            bool ok = true;
            for (long long t = me; ok && t < tiles; t += pairs, ++it) {
                const int a = it & 1;
                // the epilogues have drained this accumulator (its use two tiles ago)
                ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_AEMPTY + a, (((uint32_t)(it >> 1)) & 1) ^ 1,
                                                              abort_flag, p.status, kStatusTimeout));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dacc = tmem + (uint32_t)(a * kTile);
                for (int k = 0; k < nk; ++k, ++kc) {
                    const int s = (int)(kc % kStages);
                    ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_FULL + s, ((uint32_t)(kc / kStages)) & 1,
                                                                  abort_flag, p.status, kStatusTimeout));
                    if (!ok) break;
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
                        const uint64_t da = tc::smem_desc(tc::smem_u32(sm + OFF_A + s * kOpBytes), 16, 1024, tc::kLayoutSw128);
                        const uint64_t db = tc::smem_desc(tc::smem_u32(sm + OFF_B + s * kOpBytes), 16, 1024, tc::kLayoutSw128);
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)        // K = 32 codes = 32 bytes per MMA
                            tc::mma_i8_ss_pair(dacc, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc,
                                               (k | kk) != 0);
                        tc::mma_commit_pair(bar + B_EMPTY + s);
                        if (k == nk - 1) tc::mma_commit_pair(bar + B_AFULL + a);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {                                            // the MMAs in flight end before TMEM is freed
                if (tc::elect_one()) tc::mma_commit_pair(bar + B_DRAIN);
                __syncwarp();
                tc::mbar_wait(bar + B_DRAIN, 0, kDrainLimit);
            }
        }
    } else {
        // epilogue: warp w reads TMEM lanes 32 (w % 4) .. +31, channels n0 + 128 rank + 32 (w % 4) + lane
        const int quarter = warp & 3;
        int it = 0;
        for (long long t = me; t < tiles; t += pairs, ++it) {
            const int a = it & 1;
            int n0, t0;
            tile_at(p, t, &n0, &t0);
            const int ch = n0 + (int)rank * kRows + quarter * 32 + lane;
            const bool in = ch < p.N;
            const float sw = in ? __ldg(p.s_w + ch) : 0.f;
            const float bias = in && p.bias ? __ldg(p.bias + ch) : 0.f;
            const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * kTile);
            const bool ok = tc::wait_or_abort(bar + B_AFULL + a, ((uint32_t)(it >> 1)) & 1, abort_flag, p.status,
                                              kStatusTimeout);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::tc_fence_after();
            uint16_t* dst = p.out + (long long)t0 * p.N + ch;
            for (int c = 0; c < kTile / 32; ++c, dst += 32LL * p.N) {
                uint32_t v[32];
                tc::tmem_ld32(trow + c * 32, v);
                tc::tmem_wait_ld();
                if (c == kTile / 32 - 1) {
                    // the whole accumulator is in registers: hand it back to the MMA warp
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(tc::smem_u32(bar + B_AEMPTY + a), 0));
                }
                const int live = p.T - t0 - c * 32;
                if (in) store_tokens(v, p.s_t + t0 + c * 32, sw, bias, dst, p.N, live);
            }
        }
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();                                           // no CTA leaves while the other may reach it
    if (warp == 1) tc::tmem_dealloc_pair(tmem, kAcc * kTile);
}

}  // namespace pair

// ---------------------------------------------------------------- few tokens: K split over a cluster

namespace few {

constexpr int kRows = 128;                            // channels of a tile
constexpr int kMaxStages = 6;
constexpr int B_FULL = 0, B_EMPTY = kMaxStages, B_DONE = 2 * kMaxStages, NBAR = B_DONE + 1;

template <int BN>
struct Layout {
    static constexpr int A_BYTES = kRows * kBK, B_BYTES = BN * kBK, STAGE = A_BYTES + B_BYTES;
    static constexpr int RED = BN * kRows * 4;                    // partial sums, over the stages
    static constexpr int STAGES = 98304 / STAGE < kMaxStages ? 98304 / STAGE : kMaxStages;
    static constexpr int BUF = STAGES * STAGE > RED ? STAGES * STAGE : RED;
    static constexpr int OFF_BAR = BUF, OFF_FLAG = OFF_BAR + NBAR * 8, OFF_TMEM = OFF_FLAG + 8, SMEM = OFF_TMEM + 8;
    static constexpr int COLS = BN < 32 ? 32 : BN;                // TMEM columns
};

// Cluster rank r takes the K slices [r nk / S, (r + 1) nk / S) of the tile (channels n0 ..,
// tokens t0 ..), keeps its partial sums in shared memory, and then finishes the tokens
// r, r + S, ... of the tile with every rank's partial sums.
template <int BN>
__global__ void __launch_bounds__(kWarps * 32)
matmul_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ MatmulArgs p, int S) {
    using Ly = Layout<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Ly::OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::OFF_FLAG);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Ly::OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank();
    const int tile = blockIdx.x / S;
    const int n0 = (tile % p.tiles_n) * kRows, t0 = (tile / p.tiles_n) * BN;
    const int nk = (p.K + kBK - 1) / kBK;
    const int k0 = (int)((long long)rank * nk / S), k1 = (int)((long long)(rank + 1) * nk / S);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBAR; ++i) tc::mbar_init(bar + i, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, Ly::COLS);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int k = k0;
            for (; k < k1; ++k) {
                const int j = k - k0, s = j % Ly::STAGES;
                if (!(ok = tc::wait_or_abort(bar + B_EMPTY + s, (((uint32_t)(j / Ly::STAGES)) & 1) ^ 1, abort_flag,
                                             p.status, kStatusTimeout)))
                    break;
                uint8_t* st = sm + s * Ly::STAGE;
                tc::mbar_arrive_expect_tx(bar + B_FULL + s, Ly::STAGE);
                tc::tma_load_2d(st, &tm_w, bar + B_FULL + s, k * kBK, n0);
                tc::tma_load_2d(st + Ly::A_BYTES, &tm_q, bar + B_FULL + s, k * kBK, t0);
            }
            if (!ok)
                for (int j = max(0, k - k0 - Ly::STAGES); j < k - k0; ++j)
                    tc::mbar_wait(bar + B_FULL + j % Ly::STAGES, ((uint32_t)(j / Ly::STAGES)) & 1, kDrainLimit);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = tc::idesc_s8_s32(kRows, BN, tc::kMajorK, tc::kMajorK);
        for (int k = k0; ok && k < k1; ++k) {
            const int j = k - k0, s = j % Ly::STAGES;
            ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_FULL + s, ((uint32_t)(j / Ly::STAGES)) & 1,
                                                          abort_flag, p.status, kStatusTimeout));
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
                const uint8_t* st = sm + s * Ly::STAGE;
                const uint64_t da = tc::smem_desc(tc::smem_u32(st), 16, 1024, tc::kLayoutSw128);
                const uint64_t db = tc::smem_desc(tc::smem_u32(st + Ly::A_BYTES), 16, 1024, tc::kLayoutSw128);
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    tc::mma_i8_ss(tmem, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc, (j | kk) != 0);
                tc::mma_commit(bar + B_EMPTY + s);
            }
            __syncwarp();
        }
        if (tc::elect_one()) tc::mma_commit(bar + B_DONE);          // every MMA issued, also when the loop gave up
        __syncwarp();
        if (!ok) tc::mbar_wait(bar + B_DONE, 0, kDrainLimit);
    }
    const int quarter = warp & 3, row = quarter * 32 + lane, ch = n0 + row;
    const bool in = ch < p.N;
    const float sw = in ? __ldg(p.s_w + ch) : 0.f;
    const float bias = in && p.bias ? __ldg(p.bias + ch) : 0.f;
    const int live = min(BN, p.T - t0);
    int* red = reinterpret_cast<int*>(sm);
    if (warp >= 2) {
        // thread = channel: partial sums to shared memory, a token's 128 channels in a row
        ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_DONE, 0, abort_flag, p.status, kStatusTimeout));
        tc::tc_fence_after();
        if (ok) {
            const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                uint32_t v[16];
                tc::tmem_ld16(trow + c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) red[(c + j) * kRows + row] = (int)v[j];
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    if (warp >= 2 && ok && in) {
        const uint32_t mine = tc::smem_u32(red + row);
        uint16_t* dst = p.out + (long long)t0 * p.N + ch;
        for (int j = rank; j < live; j += S) {
            int sum = 0;
            for (int r = 0; r < S; ++r) sum += tc::ld_cluster_s32(tc::map_rank(mine + j * kRows * 4, r));
            dst[(long long)j * p.N] = float_to_bf16_bits(fmaf((float)sum * sw, __ldg(p.s_t + t0 + j), bias));
        }
    }
    tc::cluster_sync();                                           // the others have read this CTA's sums
    if (warp == 1) tc::tmem_dealloc(tmem, Ly::COLS);
}

template <int BN>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mq, MatmulArgs p, int S, cudaStream_t st) {
    const int smem = Layout<BN>::SMEM + 1024;
    cudaError_t e = cudaFuncSetAttribute(matmul_few_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)((long long)p.tiles_n * p.tiles_t * S));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, matmul_few_kernel<BN>, mw, mq, p, S);
}

}  // namespace few

int tiles_of(int n, int tile) { return (n - 1) / tile + 1; }

bool operand_map(CUtensorMap* m, const int8_t* base, int rows, int K, int box_rows) {
    return make_tmap_2d(m, true, base, (unsigned long long)K, (unsigned long long)rows, (unsigned long long)K, kBK,
                        (unsigned)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_matmul_i8(int T, int K, int N, const int8_t* q, const float* s_t, const int8_t* Wq,
                             const float* s_w, const float* bias, uint16_t* out, int* status, cudaStream_t st) {
    CUtensorMap mw, mq;
    MatmulArgs p{T, K, N, 0, 0, s_t, s_w, bias, out, status};
    const int sms = device_sm_count(), nk = (K + kBK - 1) / kBK;
    const long long pair_tiles = (long long)tiles_of(T, pair::kTile) * tiles_of(N, pair::kTile);
    if (T <= 128 || pair_tiles < sms / 4) {
        const int bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
        p.tiles_n = tiles_of(N, few::kRows);
        p.tiles_t = tiles_of(T, bn);
        const long long tiles = (long long)p.tiles_n * p.tiles_t;
        // split K until every SM has a CTA, over at most 8 (the portable cluster) non-empty parts
        int S = 1;
        while (S < 8 && tiles * S < sms && 2 * S <= nk) S *= 2;
        if (!operand_map(&mw, Wq, N, K, few::kRows) || !operand_map(&mq, q, T, K, bn)) return cudaErrorInvalidValue;
        if (bn == 16) return few::launch<16>(mw, mq, p, S, st);
        if (bn == 32) return few::launch<32>(mw, mq, p, S, st);
        if (bn == 64) return few::launch<64>(mw, mq, p, S, st);
        return few::launch<128>(mw, mq, p, S, st);
    }
    if (!operand_map(&mw, Wq, N, K, pair::kRows) || !operand_map(&mq, q, T, K, pair::kRows)) return cudaErrorInvalidValue;
    const int smem = pair::SMEM + 1024;
    const cudaError_t e = cudaFuncSetAttribute(pair::matmul_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    p.tiles_n = tiles_of(N, pair::kTile);
    p.tiles_t = tiles_of(T, pair::kTile);
    const int pairs = (int)(pair_tiles < sms / 2 ? pair_tiles : sms / 2);
    pair::matmul_pair_kernel<<<2 * pairs, kWarps * 32, smem, st>>>(mw, mq, p);
    return cudaGetLastError();
}

}  // namespace ssd
