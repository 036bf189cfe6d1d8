// matmul_i8.cu — the projections of a W8A8 layer: the product of INT8 codes with a scale per
// token and a scale per output channel,
//   out[t,n] = s_t[t] * s_w[n] * sum_k q[t,k] * Wq[n,k] + bias[n]      (bf16),
// the sum exact in INT32 on the tensor cores (tcgen05.mma kind::i8, operands by TMA with the
// 128-byte swizzle in K slices of 128; what lies outside the matrices arrives as zeros).
//
//   matmul_pair_kernel  many tokens: a CTA pair (cta_group::2) per 256 x 256 output tile,
//                       persistent, a ring of K slices, two accumulators.  Its rows (TMEM
//                       lanes) are tokens and its columns channels.  Tiles leave through
//                       shared memory, by TMA where n % 8 == 0; otherwise no row of the output
//                       is aligned, and each is stored from a copy that is shifted in shared
//                       memory until their 16-byte vectors match.
//   matmul_few_kernel   few tokens or few tiles: one tile of up to 128 channels (rows) and up to
//                       128 tokens per cluster, the K axis split over the cluster's CTAs and
//                       the INT32 partial sums joined through distributed shared memory.  Bound
//                       by the weights' way in: a barrier's answer takes some 60 cycles and a
//                       slice's MMAs 130, so that one warp that loads and one that issues spent
//                       450 cycles a slice, whatever its bytes.  Two of each spend under 200
//                       (unsplit 8 x 5120 -> 2560, from L2, when they were added: 11.5 us with
//                       one, 9.2 with two that issue, 6.9 with two that load as well; 6.8 now).
// Times in this file: one call among many in a graph, the weights in HBM unless said.
//
// Every wait is bounded; an expired wait raises the CTA's abort flag and records
// SSD_ERR_TIMEOUT in the status word.  Whichever role gave up, the CTA then waits, again with a
// limit, for every copy and MMA that was issued: they use its shared memory and TMEM.
#include "kernels.h"
#include "ring.h"
#include "tc.cuh"

namespace ssd {

namespace {

constexpr int kBK = 128;                              // K slice: one 128-byte swizzled row
constexpr int kWarps = 10;                            // 0 TMA, 1 MMA, 2-9 epilogue
constexpr int kEpi = 8;                               // epilogue warps: two per TMEM lane quarter, half the columns each
constexpr long long kDrainLimit = 400000000LL;        // cycles an aborting CTA waits for its copies and MMAs

struct MatmulArgs {
    int T, K, N;
    int tiles_t, tiles_n;
    const float* s_t;
    const float* s_w;
    const float* bias;
    uint16_t* out;
    int* status;
    int rows;                   // channels of a tile of matmul_few_kernel
    const int8_t* Wq;           // for it to prefetch
};

// After an abort: waits until the last copy into each stage has landed, `loaded(stage)` slices
// having been asked for in the stage's turn, or until `deadline`.
template <typename F>
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, long long deadline, F loaded) {
    for (int s = 0; s < stages; ++s) {
        const long long u = ring_last_use(loaded(s), s, stages);
        if (u >= 0) tc::mbar_wait(full + s, (uint32_t)(u & 1), deadline - clock64());
    }
}

// ---------------------------------------------------------------- many tokens: CTA pairs

namespace pair {

constexpr int kRows = 128;                            // rows of each operand per CTA; the pair's tile is 256 x 256
constexpr int kTile = 2 * kRows;
constexpr int kAcc = 2;
constexpr int kOpBytes = kRows * kBK;

// ALIGNED: n % 8 == 0, stores by TMA.
template <bool ALIGNED>
struct Layout {
    static constexpr int STAGES = ALIGNED ? 6 : 5;
    // a warp's 32 rows on their way out: 32 bf16 columns, or 64 and room to shift them by up to 7
    static constexpr int OUT_ROW = ALIGNED ? 64 : 144, OUT = 32 * OUT_ROW;
    static constexpr int OFF_A = 0, OFF_B = STAGES * kOpBytes, OFF_OUT = 2 * STAGES * kOpBytes;
    static constexpr int OFF_COL = OFF_OUT + kEpi * OUT;  // [kAcc][2][kTile] fp32: the columns' scales and biases
    static constexpr int OFF_BAR = OFF_COL + kAcc * 2 * kTile * 4;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_AFULL = 2 * STAGES, B_AEMPTY = B_AFULL + kAcc,
                         B_DRAIN = B_AEMPTY + kAcc, NBAR = B_DRAIN + 1;
    static constexpr int OFF_FLAG = OFF_BAR + NBAR * 8, OFF_TMEM = OFF_FLAG + 8, OFF_LOADED = OFF_TMEM + 8,
                         SMEM = OFF_LOADED + 8;
    static_assert(SMEM + 1024 <= 227 * 1024, "shared memory of a CTA");
};
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

// 32 columns of this thread's row (token), scaled and rounded, into its 64 bytes of `buf`
// (32 such rows, 64-byte swizzle).
__device__ __forceinline__ void fill_box(const uint32_t (&v)[32], float st, const float* sw, const float* bias,
                                         uint8_t* buf, int lane) {
    const f32x2 st2 = both2(st);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 8 * j + 4 * e;
            const float4 w = *reinterpret_cast<const float4*>(sw + c), b = *reinterpret_cast<const float4*>(bias + c);
            const f32x2 x = mul2(pair2((float)(int)v[c], (float)(int)v[c + 1]), pair2(w.x, w.y));
            const f32x2 y = mul2(pair2((float)(int)v[c + 2], (float)(int)v[c + 3]), pair2(w.z, w.w));
            o[2 * e] = pack2(fma2(x, st2, pair2(b.x, b.y)));
            o[2 * e + 1] = pack2(fma2(y, st2, pair2(b.z, b.w)));
        }
        *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// 64 columns of a warp's 32 rows to rows of `n` elements of no alignment: `dst` points at this
// lane's row, column 0 of the 64; `rows` and `cols` of them exist.  Each row is written to
// shared memory shifted by the elements that its first lacks to a 16-byte boundary, so that
// the row's aligned vectors are vectors there; then 8 lanes store a row's, and its up to 7
// elements in front of and behind them one by one.  4096 x 1024 -> 8193 takes 51 us (8208,
// aligned, 33; weights from L2); 32 two-byte stores a row, from a tile with the channels in its rows, took 66.
__device__ __forceinline__ void store_shifted(const uint32_t (&lo)[32], const uint32_t (&hi)[32], float st,
                                              const float* sw, const float* bias, uint8_t* buf, int lane,
                                              uint16_t* dst, int rows, int cols) {
    constexpr int kPitch = Layout<false>::OUT_ROW;
    const int sh = (int)(((uintptr_t)dst >> 1) & 7);              // elements past the boundary
    const bool odd = sh & 1;
    uint32_t* mine = reinterpret_cast<uint32_t*>(buf + lane * kPitch) + (sh >> 1);
    __syncwarp();                                                 // the rows before have been read
    float before = 0.f;                                           // column 4 j - 1
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float4 w = *reinterpret_cast<const float4*>(sw + 4 * j), b = *reinterpret_cast<const float4*>(bias + 4 * j);
        const auto acc = [&](int e) { return (float)(int)(j < 8 ? lo[(4 * j + e) & 31] : hi[(4 * j + e) & 31]); };
        const f32x2 st2 = both2(st);
        const float2 x = split2(fma2(mul2(pair2(acc(0), acc(1)), pair2(w.x, w.y)), st2, pair2(b.x, b.y)));
        const float2 y = split2(fma2(mul2(pair2(acc(2), acc(3)), pair2(w.z, w.w)), st2, pair2(b.z, b.w)));
        mine[2 * j] = odd ? pack2(before, x.x) : pack2(x.x, x.y);
        mine[2 * j + 1] = odd ? pack2(x.y, y.x) : pack2(y.x, y.y);
        before = y.y;
    }
    if (odd) mine[32] = pack2(before, 0.f);
    __syncwarp();
    const int l8 = lane & 7;
#pragma unroll 4
    for (int r0 = 0; r0 < 32; r0 += 4) {
        const int r = r0 + (lane >> 3);                           // 32 rows have addresses, whether they exist or not
        uint16_t* d = reinterpret_cast<uint16_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
        const int s = (int)(((uintptr_t)d >> 1) & 7), head = min((8 - s) & 7, cols);
        const int nv = (cols - head) >> 3, tail = cols - head - 8 * nv;
        const uint16_t* row = reinterpret_cast<const uint16_t*>(buf + r * kPitch) + s;
        if (r < rows && l8 < nv) {
            const int e = head + 8 * l8;
            *reinterpret_cast<uint4*>(d + e) = *reinterpret_cast<const uint4*>(row + e);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = l8 + 8 * h;
            if (r < rows && i < head + tail) {
                const int e = i < head ? i : cols - tail + (i - head);
                d[e] = row[e];
            }
        }
    }
}

// Clusters of 2.
template <bool ALIGNED>
__global__ void __launch_bounds__(kWarps * 32, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ MatmulArgs p) {
    using Ly = Layout<ALIGNED>;
    constexpr int kStages = Ly::STAGES, B_FULL = Ly::B_FULL, B_EMPTY = Ly::B_EMPTY, B_AFULL = Ly::B_AFULL,
                  B_AEMPTY = Ly::B_AEMPTY, B_DRAIN = Ly::B_DRAIN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Ly::OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::OFF_FLAG);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Ly::OFF_TMEM);
    long long* loaded = reinterpret_cast<long long*>(sm + Ly::OFF_LOADED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const bool leader = rank == 0;
    const int nk = (p.K + kBK - 1) / kBK;
    const long long tiles = (long long)p.tiles_t * p.tiles_n;
    const int pairs = gridDim.x >> 1, me = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        // an accumulator is free once the epilogue warps of both CTAs have read it
        for (int i = 0; i < Ly::NBAR; ++i) tc::mbar_init(bar + i, i >= B_AEMPTY && i < B_DRAIN ? 2 * kEpi : 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tmem_slot, kAcc * kTile);
        tc::tmem_relinquish_pair();
    }
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&tm_q);
        tc::prefetch_tmap(&tm_w);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_release();
    grid_wait();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 1;                                   // a fresh stage counts as free
            long long issued = 0;                                 // slices asked for
            bool ok = true;
            for (long long t = me; ok && t < tiles; t += pairs) {
                int n0, t0;
                tile_at(p, t, &n0, &t0);
                n0 += (int)rank * kRows;
                t0 += (int)rank * kRows;
                for (int k = 0; k < nk; ++k) {
                    if (!(ok = tc::wait_or_abort(bar + B_EMPTY + s, phase, abort_flag, p.status, kStatusTimeout))) break;
                    // both CTAs' loads of a stage count on the even CTA's barrier
                    if (leader) tc::mbar_arrive_expect_tx(bar + B_FULL + s, 4 * kOpBytes);
                    const uint32_t full = tc::map_rank(tc::smem_u32(bar + B_FULL + s), 0);
                    tc::tma_load_2d_pair(sm + Ly::OFF_A + s * kOpBytes, &tm_q, full, k * kBK, t0);
                    tc::tma_load_2d_pair(sm + Ly::OFF_B + s * kOpBytes, &tm_w, full, k * kBK, n0);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            *loaded = issued;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint32_t idesc = tc::idesc_s8_s32(kTile, kTile, tc::kMajorK, tc::kMajorK);
            int s = 0, it = 0;                                    // ring position; tiles of this pair so far
            uint32_t phase = 0;
            bool ok = true;
            for (long long t = me; ok && t < tiles; t += pairs, ++it) {
                const int a = it & 1;
                // the epilogues have drained this accumulator (its use two tiles ago)
                ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_AEMPTY + a, (((uint32_t)(it >> 1)) & 1) ^ 1,
                                                              abort_flag, p.status, kStatusTimeout));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dacc = tmem + (uint32_t)(a * kTile);
                for (int k = 0; k < nk; ++k) {
                    ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_FULL + s, phase, abort_flag, p.status,
                                                                  kStatusTimeout));
                    if (!ok) break;
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
                        const uint64_t da = tc::smem_desc(tc::smem_u32(sm + Ly::OFF_A + s * kOpBytes), 16, 1024, tc::kLayoutSw128);
                        const uint64_t db = tc::smem_desc(tc::smem_u32(sm + Ly::OFF_B + s * kOpBytes), 16, 1024, tc::kLayoutSw128);
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)        // K = 32 codes = 32 bytes per MMA
                            tc::mma_i8_ss_pair(dacc, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc,
                                               (k | kk) != 0);
                        tc::mma_commit_pair(bar + B_EMPTY + s);
                        if (k == nk - 1) tc::mma_commit_pair(bar + B_AFULL + a);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else {
        // epilogue: warp w reads TMEM lanes 32 (w % 4) .. +31, the tile's rows 128 rank + 32 (w % 4) + lane,
        // and columns half .. half + 127
        const int quarter = warp & 3, half = (warp - 2) / 4 * kRows;
        uint8_t* out_buf = sm + Ly::OFF_OUT + (warp - 2) * Ly::OUT;
        int it = 0;
        // scales (and biases) of a tile are loaded while the one before it is worked on
        float srow = 0.f, ccol = 0.f, bcol = 0.f;
        const auto load_scales = [&](long long t) {
            int n0, t0;
            if (t >= tiles) return;
            tile_at(p, t, &n0, &t0);
            const int row = t0 + (int)rank * kRows + quarter * 32 + lane, c = n0 + half + quarter * 32 + lane;
            srow = row < p.T ? p.s_t[row] : 0.f;
            ccol = c < p.N ? p.s_w[c] : 0.f;
            bcol = c < p.N && p.bias ? p.bias[c] : 0.f;
        };
        load_scales(me);
        for (long long t = me; t < tiles; t += pairs, ++it) {
            const int a = it & 1;
            int n0, t0;
            tile_at(p, t, &n0, &t0);
            const int row0 = t0 + (int)rank * kRows + quarter * 32;
            const float st = srow;
            float* col = reinterpret_cast<float*>(sm + Ly::OFF_COL) + a * 2 * kTile;
            // the channels' scales and biases, for every warp; the other half of the buffer may
            // still be read by a warp that is one tile behind
            col[half + quarter * 32 + lane] = ccol;
            col[kTile + half + quarter * 32 + lane] = bcol;
            tc::named_sync(1, kEpi * 32);
            load_scales(t + pairs);
            const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * kTile + half);
            const bool ok = tc::wait_or_abort(bar + B_AFULL + a, ((uint32_t)(it >> 1)) & 1, abort_flag, p.status,
                                              kStatusTimeout);
            // the warps stay together: the named barrier above counts all of them
            if (!tc::named_and(2, kEpi * 32, ok)) break;
            tc::tc_fence_after();
            // this warp's part of the accumulator to registers, and the accumulator back to the MMA warp
            uint32_t v[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::tmem_ld32(trow + i * 32, v[i]);
            tc::tmem_wait_ld();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(tc::smem_u32(bar + B_AEMPTY + a), 0));
            if (row0 >= p.T || n0 + half >= p.N) continue;
            if (!ALIGNED) {
                uint16_t* dst = p.out + (long long)(row0 + lane) * p.N + n0 + half;
                const int rows = min(32, p.T - row0), cols = p.N - n0 - half;
                store_shifted(v[0], v[1], st, col + half, col + kTile + half, out_buf, lane, dst, rows, min(64, cols));
                if (cols > 64)
                    store_shifted(v[2], v[3], st, col + half + 64, col + kTile + half + 64, out_buf, lane, dst + 64, rows,
                                  min(64, cols - 64));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = half + i * 32;
                    if (n0 + c >= p.N) break;
                    if (lane == 0) tc::tma_store_wait_read0();    // the box before has left the buffer
                    __syncwarp();
                    fill_box(v[i], st, col + c, col + kTile + c, out_buf, lane);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_2d(&tm_out, out_buf, n0 + c, row0);
                        tc::tma_store_commit();
                    }
                }
            }
        }
        if (ALIGNED && lane == 0) tc::tma_store_wait0();            // the stores have read shared memory and are done
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag)                          // one CTA's abort is the pair's
        tc::st_cluster_u32(tc::map_rank(tc::smem_u32(sm + Ly::OFF_FLAG), rank ^ 1), 1);
    tc::cluster_sync();                                           // no CTA leaves while the other may reach it
    if (*abort_flag) {
        // The roles of both CTAs are over.  The MMAs read both CTAs' shared memory and their commit
        // arrives at both; both CTAs' copies count on the even CTA's barriers (a slice that only one
        // of them asked for leaves its phase open: the deadline ends that wait, long after the copy).
        if (warp == 1 && leader && tc::elect_one()) tc::mma_commit_pair(bar + B_DRAIN);
        if (threadIdx.x == 0) {
            const long long deadline = clock64() + kDrainLimit;
            tc::mbar_wait(bar + B_DRAIN, 0, kDrainLimit);
            if (leader) {
                const long long other = tc::ld_cluster_s64(tc::map_rank(tc::smem_u32(loaded), 1));
                const long long n = other > *loaded ? other : *loaded;
                drain_ring(bar + B_FULL, kStages, deadline, [&](int) { return n; });
            }
        }
        __syncthreads();
        tc::cluster_sync();
    }
    if (warp == 1) tc::tmem_dealloc_pair(tmem, kAcc * kTile);
}

template <bool ALIGNED>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mw, const CUtensorMap& mo, const MatmulArgs& p,
                   cudaStream_t st) {
    const int smem = Layout<ALIGNED>::SMEM + 1024;
    const cudaError_t e =
        cudaFuncSetAttribute(matmul_pair_kernel<ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)p.tiles_t * p.tiles_n;
    const int most = device_sm_count() / 2, pairs = tiles < most ? (int)tiles : most;
    return launch_programmatic(matmul_pair_kernel<ALIGNED>, 2 * pairs, kWarps * 32, smem, st, 2, mq, mw, mo, p);
}

}  // namespace pair

// ---------------------------------------------------------------- few tokens: K split over a cluster

namespace few {

constexpr int kRows = 128;                            // rows of the MMA; a tile has up to as many channels
constexpr int kMaxStages = 16, kLeastRows = 64;
// Lines that a CTA prefetches at most (8 x 4096 -> 18560 14.5 us with all 4096, 13.0 so; 64 tokens
// 15.8, 14.3; 64 x 5120 -> 2560 6.7 with 768, 6.2 with all its 1280).
constexpr int kAhead = 1280;
constexpr int kLoader2 = 3;                           // the second loading warp, until its epilogue
// Shared memory for stages where two CTAs share an SM, and where none has to: the bytes on their
// way bound an SM's rate (8 x 5120 -> 2560 6.8 us with 96 KB, 5.2 with 148 or 208; 256 x 8192 -> 4096
// 18.6, 15.6 and 14.4).  For few tokens 148 KB leave room for the next kernels' CTAs (a 2560-feature
// layer's decode step, bf16 scan: batch 1 20.7 us, 20.8 with 208; batch 8 26.9, 27.1).
constexpr int kBudget = 98304;
constexpr int alone_budget(int bn) { return bn < 64 ? 151552 : 212992; }
constexpr int B_FULL = 0, B_EMPTY = kMaxStages, B_DONE = 2 * kMaxStages, NBAR = B_DONE + 1;
constexpr int OFF_FLAG = NBAR * 8, OFF_TMEM = OFF_FLAG + 8, OFF_LOADED = OFF_TMEM + 8, OFF_BUF = 1024;
static_assert(OFF_LOADED + 8 <= OFF_BUF, "barriers in front of the stages");

template <int BN>
struct Layout {
    static constexpr int RED = BN * kRows * 4;                    // partial sums, over the stages
    // Warps that issue MMAs, and that load.  With 128 tokens a slice's MMAs take as long as the
    // barriers, and three stages of 32 KB are no two pairs.
    static constexpr int ISSUE = BN <= 64 ? 2 : 1;
    static constexpr int COLS = ISSUE * BN;                       // TMEM columns, a power of two from 32
    // A stage has `rows` rows of weights and BN of tokens.  The MMA reads 128 rows: what lies behind
    // the weights' own makes sums that nobody reads.
    static __host__ __device__ constexpr int stage(int rows) { return (rows + BN) * kBK; }
    static constexpr int behind(int rows) { return kRows > rows + BN ? (kRows - rows - BN) * kBK : 0; }
    static int stages(int rows, int slices, int budget) {
        int n = (budget - behind(rows)) / stage(rows);
        if (n > kMaxStages) n = kMaxStages;
        return n >= slices ? slices : n / ISSUE * ISSUE;          // a stage keeps to one issuing warp
    }
    // with room to align the first
    static int smem(int rows, int n) {
        const int bytes = n * stage(rows) + behind(rows);
        return 1024 + OFF_BUF + (bytes > RED ? bytes : RED);
    }
};

// Cluster rank r takes the K slices [r nk / S, (r + 1) nk / S) of the tile (channels n0 ..,
// tokens t0 ..), keeps its partial sums in shared memory, and then finishes the tokens
// r, r + S, ... of the tile with every rank's partial sums.
template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32)
matmul_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ MatmulArgs p, int split, int stages) {
    using Ly = Layout<BN>;
    const int S = SPLIT ? split : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_FLAG);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
    int* loaded = reinterpret_cast<int*>(sm + OFF_LOADED);          // by each loading warp: its next slice
    uint8_t* buf = sm + OFF_BUF;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = SPLIT ? (int)tc::cluster_rank() : 0;
    const int tile = blockIdx.x / S;
    const int n0 = (tile % p.tiles_n) * p.rows, t0 = (tile / p.tiles_n) * BN;
    const int stage = Ly::stage(p.rows);
    const int nk = (p.K + kBK - 1) / kBK;
    const int k0 = (int)((long long)rank * nk / S), k1 = (int)((long long)(rank + 1) * nk / S);
    const int first = min(stages, k1 - k0);                       // slices loaded before anything waits
    const auto load = [&](int j, int s) {
        tc::mbar_arrive_expect_tx(bar + B_FULL + s, stage);
        tc::tma_load_2d(buf + s * stage, &tm_w, bar + B_FULL + s, (k0 + j) * kBK, n0);
        tc::tma_load_2d(buf + s * stage + p.rows * kBK, &tm_q, bar + B_FULL + s, (k0 + j) * kBK, t0);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBAR; ++i) tc::mbar_init(bar + i, i == B_DONE ? Ly::ISSUE : 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::fence_proxy_async_smem();
        tc::prefetch_tmap(&tm_w);
        tc::prefetch_tmap(&tm_q);
        grid_wait();
        for (int j = 0; j < first; ++j) load(j, j);
    }
    // The weights on their way to L2 while the kernel ahead in the stream ends, a line a thread (no
    // value is read: what is written in between is seen).  TMA's prefetches would stand in front of
    // its loads (8 x 4096 -> 18560 20.5 us).
    if (warp >= 2) {
        for (int k = k0; k < min(k1, k0 + kAhead / p.rows); ++k)
            for (int r = (int)threadIdx.x - 64; r < min(p.rows, p.N - n0); r += kEpi * 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.Wq + (long long)(n0 + r) * p.K + k * kBK));
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, Ly::COLS);
        tc::tmem_relinquish();
        // not before: a CTA of the next kernel that took the columns this one still needs would
        // wait for this kernel's end with them
        grid_release();
    }
    grid_wait();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // The epilogue's factors, asked for ahead of everything that it waits for (8 x 5120 -> 2560
    // 5.7 us without, 5.4 so, and 64 x 2560 -> 10576 7.9 us with the split at run time, 7.1 so, when
    // these were added; 5.2 and 7.2 now).  Unsplit, a thread has a channel, and lane i the scale of
    // the token 16 part + i % 16; split, a lane has four channels, and lane i the scale of its warp's i-th token
    // (at most BN / kEpi).
    const int quarter = warp & 3, row = quarter * 32 + lane, ch = n0 + row, part = (warp - 2) / 4;
    const int c4 = SPLIT ? n0 + 4 * lane : ch, end = min(p.N, n0 + p.rows), live = min(BN, p.T - t0);
    const int j0 = rank + (warp - 2) * S, token = SPLIT ? j0 + lane * kEpi * S : 16 * part + (lane & 15);
    float sw[4], bias[4], scale = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool in = warp >= 2 && c4 + e < end && (e == 0 || SPLIT);
        sw[e] = in ? p.s_w[c4 + e] : 0.f;
        bias[e] = in && p.bias ? p.bias[c4 + e] : 0.f;
    }
    if ((SPLIT || BN <= 32) && warp >= 2 && token < live) scale = p.s_t[t0 + token];

    bool ok = true;
    if (warp == 0 || warp == kLoader2) {
        if (lane == 0 && (warp == 0 || Ly::ISSUE > 1)) {
            // each loading warp refills the stages of one issuing warp
            int j = first + (warp == 0 ? 0 : 1), s = j - first;
            uint32_t phase = 0;                                   // of the stage's previous use
            bool ready = false;                                   // asked a slice ahead: an answer takes a while
            for (; j < k1 - k0; j += Ly::ISSUE) {
                if (!ready && !(ok = tc::wait_or_abort(bar + B_EMPTY + s, phase, abort_flag, p.status, kStatusTimeout)))
                    break;
                const int at = s;
                if ((s += Ly::ISSUE) >= stages) {
                    s -= stages;
                    phase ^= 1;
                }
                ready = j + Ly::ISSUE < k1 - k0 && tc::mbar_test(bar + B_EMPTY + s, phase);
                load(j, at);
            }
            loaded[warp == 0 ? 0 : 1] = j;
        }
        __syncwarp();
    } else if (warp <= Ly::ISSUE) {
        // each of the issuing warps takes every Ly::ISSUE-th slice, into sums of its own
        const uint32_t idesc = tc::idesc_s8_s32(kRows, BN, tc::kMajorK, tc::kMajorK);
        const uint32_t acc = tmem + (uint32_t)((warp - 1) * BN);
        const uint64_t da0 = tc::smem_desc(tc::smem_u32(buf), 16, 1024, tc::kLayoutSw128);
        const uint32_t da = (uint32_t)da0, hi = (uint32_t)(da0 >> 32), db = da + (uint32_t)(p.rows * kBK >> 4);
        const bool lead = tc::elect_one();
        int s = warp - 1;
        uint32_t phase = 0;
        bool ready = false;                                       // asked a slice ahead: an answer takes a while
        for (int j = warp - 1; j < k1 - k0; j += Ly::ISSUE) {
            if (!ready && !(ok = tc::wait_or_abort(bar + B_FULL + s, phase, abort_flag, p.status, kStatusTimeout))) break;
            const int at = s;
            if ((s += Ly::ISSUE) >= stages) {
                s -= stages;
                phase ^= 1;
            }
            ready = j + Ly::ISSUE < k1 - k0 && tc::mbar_test(bar + B_FULL + s, phase);
            tc::tc_fence_after();
            if (lead) {
                const uint32_t off = (uint32_t)(at * (stage >> 4));
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    tc::mma_i8_ss(acc, (uint64_t)hi << 32 | (da + off + kk * 2), (uint64_t)hi << 32 | (db + off + kk * 2),
                                  idesc, j >= Ly::ISSUE || kk);
                tc::mma_commit(bar + B_EMPTY + at);
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (lead) tc::mma_commit(bar + B_DONE);                     // every MMA issued, also when the loop gave up
        __syncwarp();
        if (ok) tc::wait_or_abort(bar + B_DONE, 0, abort_flag, p.status, kStatusTimeout);
        __syncwarp();
    }
    const bool in = warp >= 2 && ch < end;
    int* red = reinterpret_cast<int*>(buf);
    // the other warps wait here, not at the MMA's barrier: eight of them asking it slow every
    // barrier of the CTA down
    __syncthreads();
    ok = !*abort_flag;
    if (warp >= 2) {
        tc::tc_fence_after();
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        uint16_t* dst = p.out + (long long)t0 * p.N + ch;
        if (ok) {
            // thread = channel: partial sums to shared memory, a token's 128 channels in a row;
            // a CTA on its own stores what it has
#pragma unroll 1
            for (int c = 16 * part; c < live; c += 32) {
                uint32_t v[16], v1[16];
                tc::tmem_ld16(trow + c, v);
                if (Ly::ISSUE > 1 && k1 - k0 > 1) tc::tmem_ld16(trow + BN + c, v1);
                tc::tmem_wait_ld();
                if (Ly::ISSUE > 1 && k1 - k0 > 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += v1[j];
                }
                if (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) red[(c + j) * kRows + row] = (int)v[j];
                } else {
                    const int mine = c + (lane & 15);
                    const float now = BN <= 32 ? scale : mine < live ? p.s_t[t0 + mine] : 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float st = __shfl_sync(0xffffffffu, now, j);
                        if (in && c + j < live)
                            dst[(long long)(c + j) * p.N] =
                                float_to_bf16_bits(fmaf((float)(int)v[j] * sw[0], st, bias[0]));
                    }
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (SPLIT) {
        tc::cluster_sync();
        if (warp >= 2 && ok) {
            // a warp takes a token of this rank's share, a lane four channels
            const uint32_t mine = tc::smem_u32(red) + 16u * lane;
#pragma unroll 4
            for (int j = j0, i = 0; j < live; j += kEpi * S, ++i) {
                const float st = __shfl_sync(0xffffffffu, scale, i);
                int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 4
                for (int r = 0; r < S; ++r) {
                    const int4 v = tc::ld_cluster_s32x4(tc::map_rank(mine + j * kRows * 4, r));
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                const int s4[4] = {sum.x, sum.y, sum.z, sum.w};
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = fmaf((float)s4[e] * sw[e], st, bias[e]);
                uint16_t* dst = p.out + (long long)(t0 + j) * p.N + c4;
                if ((p.N & 3) == 0) {                             // 8-byte aligned, and no lane half inside
                    if (c4 < end) *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c4 + e < end) dst[e] = float_to_bf16_bits(f[e]);
                }
            }
        }
        // The others have read this CTA's sums: each sum that a warp loaded goes into f[0] of its lane 0,
        // whose channel n0 exists, and is stored.  Its stores need not be through (4 to 6% of a split call).
        tc::cluster_done();
    }
    // here, behind the code that every call fetches (ahead of the epilogue it took 0.25 us of a split call)
    if (!ok) {
        if (threadIdx.x == 0) {
            const long long deadline = clock64() + kDrainLimit;
            tc::mbar_wait(bar + B_DONE, 0, kDrainLimit);
            drain_ring(bar + B_FULL, stages, deadline,
                       [&](int s) { return (long long)min(loaded[s % Ly::ISSUE], k1 - k0); });
        }
        __syncthreads();
    }
    if (warp == 1) tc::tmem_dealloc(tmem, Ly::COLS);
}

// CTAs of a call that are resident together with `per` on each SM.  Clusters of more than two
// leave some SMs of their part of the GPU unused (35 of four with an SM a CTA run in two turns:
// 5 x 4464 -> 4480 10.9 us, 7.2 with two CTAs an SM).
long long resident(int S, int per, int sms) { return (long long)per * sms * (S > 2 ? 7 : 8) / 8; }

// Channels of a tile.  Unsplit, as few (from 64 on) as let all CTAs still be resident, on an SM
// each if those of 128 are, else on two, so that every SM loads its share (8 x 2560 -> 10576 6.5 us
// with 133 tiles of 80, 7.3 with 83 of 128 or 166 of 64).  Small weights would rather have fewer
// (8 x 1024 -> 4376 3.26 us with 128 channels, 3.44 with 64, 4.36 with 32).
// Split, more CTAs cost more in clusters and joins than they load sooner (8 x 5120 -> 2560, S = 4:
// 5.6 with 80 channels, 5.2 with 128; a layer's decode step of batch 8 25.1, 24.6).
int tile_rows(int N, int tiles_t, int S, int sms) {
    if (S > 1) return kRows;
    const auto ctas = [&](int rows) { return (long long)((N - 1) / rows + 1) * tiles_t; };
    const long long room = (ctas(kRows) <= sms ? 1LL : 2LL) * sms * 15 / 16;
    int rows = kRows;
    while (rows > kLeastRows && ctas(rows - 8) <= room) rows -= 8;
    return rows;
}

// Stages of a CTA's ring, `nk` slices of K split S ways.
template <int BN>
int ring_stages(long long ctas, int rows, int nk, int S, int sms) {
    return Layout<BN>::stages(rows, (nk - 1) / S + 1, ctas <= resident(S, 1, sms) ? alone_budget(BN) : kBudget);
}

template <int BN>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mq, const MatmulArgs& p, int S, cudaStream_t st) {
    using Ly = Layout<BN>;
    const long long ctas = (long long)p.tiles_n * p.tiles_t * S;
    const int stages = ring_stages<BN>(ctas, p.rows, (p.K - 1) / kBK + 1, S, device_sm_count());
    const auto kernel = S > 1 ? matmul_few_kernel<BN, true> : matmul_few_kernel<BN, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               1024 + OFF_BUF + alone_budget(BN));
    if (e != cudaSuccess) return e;
    return launch_programmatic(kernel, (unsigned)ctas, kWarps * 32, Ly::smem(p.rows, stages), st, S, mw, mq,
                               p, S, stages);
}

}  // namespace few

int tiles_of(int n, int tile) { return (n - 1) / tile + 1; }

bool operand_map(CUtensorMap* m, const int8_t* base, int rows, int K, int box_rows) {
    return make_tmap_2d(m, true, base, (unsigned long long)K, (unsigned long long)rows, (unsigned long long)K, kBK,
                        (unsigned)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Microseconds that a call on matmul_few_kernel is expected to take, its weights in HBM, with its
// K axis split S ways: start, end and a tile's rows out; the join (each rank reads (S - 1) / S of
// a tile's sums from the others, at about 2.4 TB/s over all SMs); and a rank's slices, each
// (rows + bn) x 128 bytes at 111 bytes a nanosecond into an SM that holds one CTA, 38 for each of
// two, 1.25 times that with rows that are not whole 32-byte sectors.
double few_estimate(long long tiles, int rows, int nk, int bn, int S, bool sectors, int sms) {
    const long long ctas = tiles * S;
    const double slices = (double)nk / S * (rows + bn) * (sectors ? 1.0 : 1.25);
    const double fixed = 2.4 + 1.2 * bn / 128 +
                         (S > 1 ? 0.2 + 0.1 * S + (double)ctas * bn * 512e-6 * (S - 1) / S / 2.4 : 0.0);
    if (ctas <= few::resident(S, 1, sms)) return fixed + slices / 870.0;
    double turns = (double)ctas / (2 * sms);
    turns = turns <= 1.0 ? 1.0 : 0.5 * (turns + (double)((ctas - 1) / (2 * sms) + 1));
    return fixed + turns * slices / 300.0 + (turns - 1.0) * 4.0;
}

// The same for matmul_pair_kernel: start and end, then for each turn of the pairs over the
// tiles the slices and a tile's rows out, which cost more where they are not aligned.
double pair_estimate(long long tiles, int nk, bool sectors, bool aligned, int sms) {
    const double turns = (double)((tiles + sms / 2 - 1) / (sms / 2));
    return 3.3 + turns * (nk * (sectors ? 0.30 : 0.36) + (aligned ? 1.9 : 3.9));
}

struct Choice {
    bool pair;                  // matmul_pair_kernel
    int bn, rows, S;            // else matmul_few_kernel: its tile's tokens and channels, its split of K
};

// Which kernel, and how many ranks: matmul_few_kernel up to 64 tokens, else the one that is
// expected to take less; the split S that is (all CTAs resident at a time).  Over 48 sizes of usual
// widths the choice takes 1.2% longer than the best of all in the geometric mean, over 120 sizes that
// the estimates were not fitted to (1 to 1024 tokens, K to 8192, N to 18560) 1.4%; 23% at most, at
// 512 x 2048 -> 1024.  Measured in a graph, each call's weights in HBM, microseconds with S = 1, 2, 4,
// 8 and on pairs:
//    8 x 5120 -> 2560   6.9  6.7  5.2  5.4 15.8      64 x 4096 -> 2048   6.9  7.0  5.3  6.6  13.8
//    8 x 8192 -> 4096  10.0  9.7  8.3  9.0 23.6     512 x 8192 -> 4096  19.7 20.3 29.4 47.8  24.7
Choice choose(int T, int K, int N, int sms) {
    const int nk = tiles_of(K, kBK);
    const int bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
    const int few_t = tiles_of(T, bn);
    const long long pair_tiles = (long long)tiles_of(T, pair::kTile) * tiles_of(N, pair::kTile);
    const bool sectors = K % 32 == 0;
    Choice best{false, bn, 0, 1};
    double few_us = 0.0;
    for (int c : {1, 2, 4, 8}) {
        if (c > 1 && (c > nk || (long long)tiles_of(N, few::kRows) * few_t * c * 4 > 7LL * sms)) break;
        const int rows = few::tile_rows(N, few_t, c, sms);
        const double us = few_estimate((long long)tiles_of(N, rows) * few_t, rows, nk, bn, c, sectors, sms);
        if (c == 1 || us < few_us) {
            few_us = us;
            best.S = c;
            best.rows = rows;
        }
    }
    best.pair = T > 64 && few_us > pair_estimate(pair_tiles, nk, sectors, N % 8 == 0, sms);
    return best;
}

template <int BN>
MatmulPlan few_plan(const Choice& c, int T, int K, int N, int sms) {
    const long long ctas = (long long)tiles_of(N, c.rows) * tiles_of(T, BN) * c.S;
    const int stages = few::ring_stages<BN>(ctas, c.rows, tiles_of(K, kBK), c.S, sms);
    return MatmulPlan{false, BN, c.rows, c.S, stages, few::Layout<BN>::smem(c.rows, stages), few::Layout<BN>::COLS, ctas};
}

template <bool ALIGNED>
MatmulPlan pair_plan(int T, int N, int sms) {
    const long long tiles = (long long)tiles_of(T, pair::kTile) * tiles_of(N, pair::kTile), most = sms / 2;
    using Ly = pair::Layout<ALIGNED>;
    return MatmulPlan{true, pair::kTile, pair::kTile, 1, Ly::STAGES, Ly::SMEM + 1024, pair::kAcc * pair::kTile,
                      2 * (tiles < most ? tiles : most)};
}

}  // namespace

MatmulPlan plan_matmul_i8(int T, int K, int N, int sms) {
    const Choice c = choose(T, K, N, sms);
    if (c.pair) return N % 8 == 0 ? pair_plan<true>(T, N, sms) : pair_plan<false>(T, N, sms);
    if (c.bn == 16) return few_plan<16>(c, T, K, N, sms);
    if (c.bn == 32) return few_plan<32>(c, T, K, N, sms);
    if (c.bn == 64) return few_plan<64>(c, T, K, N, sms);
    return few_plan<128>(c, T, K, N, sms);
}

cudaError_t launch_matmul_i8(int T, int K, int N, const int8_t* q, const float* s_t, const int8_t* Wq,
                             const float* s_w, const float* bias, uint16_t* out, int* status, cudaStream_t st) {
    CUtensorMap mw, mq;
    MatmulArgs p{T, K, N, 0, 0, s_t, s_w, bias, out, status, 0, Wq};
    const Choice c = choose(T, K, N, device_sm_count());
    if (!c.pair) {
        p.rows = c.rows;
        p.tiles_n = tiles_of(N, c.rows);
        p.tiles_t = tiles_of(T, c.bn);
        if (!operand_map(&mw, Wq, N, K, c.rows) || !operand_map(&mq, q, T, K, c.bn)) return cudaErrorInvalidValue;
        if (c.bn == 16) return few::launch<16>(mw, mq, p, c.S, st);
        if (c.bn == 32) return few::launch<32>(mw, mq, p, c.S, st);
        if (c.bn == 64) return few::launch<64>(mw, mq, p, c.S, st);
        return few::launch<128>(mw, mq, p, c.S, st);
    }
    if (!operand_map(&mw, Wq, N, K, pair::kRows) || !operand_map(&mq, q, T, K, pair::kRows)) return cudaErrorInvalidValue;
    p.tiles_n = tiles_of(N, pair::kTile);
    p.tiles_t = tiles_of(T, pair::kTile);
    if (N % 8 != 0) return pair::launch<false>(mq, mw, mq, p, st);     // the third map is not read
    CUtensorMap mo;
    if (!make_tmap_2d(&mo, false, out, (unsigned long long)N, (unsigned long long)T, (unsigned long long)N * 2, 32, 32,
                      CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    return pair::launch<true>(mq, mw, mo, p, st);
}

}  // namespace ssd
