// matmul_i8.cu — the projections of a W8A8 layer: the product of INT8 codes with a scale per
// token and a scale per output channel,
//   out[t,n] = s_t[t] * s_w[n] * sum_k q[t,k] * Wq[n,k] + bias[n]      (bf16),
// the sum exact in INT32 on the tensor cores.
//
// Persistent, one CTA per SM over 128 x 256 output tiles (tokens x channels): a 4-stage TMA
// ring of 128-byte K slices (128-byte swizzle; what lies outside the matrices arrives as
// zeros), tcgen05.mma kind::i8 issued by one elected lane into one of two 256-column INT32
// TMEM accumulators, and four epilogue warps (one per TMEM lane quarter) that scale and
// store a tile while the next one accumulates.  Every wait is bounded; an expired wait
// raises the CTA's abort flag and records SSD_ERR_TIMEOUT in the status word.
#include "kernels.h"
#include "tc.cuh"

namespace ssd {

namespace {

constexpr int kBM = 128, kBN = 256, kBK = 128, kStages = 4, kAcc = 2;
constexpr int kWarps = 6;                            // 0 TMA, 1 MMA, 2-5 epilogue
constexpr int A_BYTES = kBM * kBK, B_BYTES = kBN * kBK;
constexpr int OFF_A = 0, OFF_B = kStages * A_BYTES, OFF_BAR = OFF_B + kStages * B_BYTES;
constexpr int B_FULL = 0, B_EMPTY = kStages, B_AFULL = 2 * kStages, B_AEMPTY = 2 * kStages + kAcc,
              NBAR = 2 * kStages + 2 * kAcc;
constexpr int OFF_FLAG = OFF_BAR + NBAR * 8, OFF_TMEM = OFF_FLAG + 8, SMEM = OFF_TMEM + 8;

struct MatmulArgs {
    int T, K, N;
    int tiles_n;
    long long tiles;
    const float* s_t;
    const float* s_w;
    const float* bias;
    uint16_t* out;
    int* status;
};

__global__ void __launch_bounds__(kWarps * 32, 1)
matmul_i8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ MatmulArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_FLAG);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (p.K + kBK - 1) / kBK;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBAR; ++i) tc::mbar_init(bar + i, i >= B_AEMPTY ? 4 : 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, kAcc * kBN);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            long long kc = 0;                                     // K slices issued so far (ring position)
            bool ok = true;
            for (long long t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
                const int m0 = (int)(t / p.tiles_n) * kBM, n0 = (int)(t % p.tiles_n) * kBN;
                for (int k = 0; k < nk; ++k, ++kc) {
                    const int s = (int)(kc % kStages);
                    if (!(ok = tc::wait_or_abort(bar + B_EMPTY + s, (((uint32_t)(kc / kStages)) & 1) ^ 1, abort_flag,
                                                 p.status, kStatusTimeout)))
                        break;
                    tc::mbar_arrive_expect_tx(bar + B_FULL + s, A_BYTES + B_BYTES);
                    tc::tma_load_2d(sm + OFF_A + s * A_BYTES, &tm_a, bar + B_FULL + s, k * kBK, m0);
                    tc::tma_load_2d(sm + OFF_B + s * B_BYTES, &tm_b, bar + B_FULL + s, k * kBK, n0);
                }
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = tc::idesc_s8_s32(kBM, kBN, tc::kMajorK, tc::kMajorK);
        long long kc = 0;
        int it = 0;                                               // tiles of this CTA so far
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < p.tiles; t += gridDim.x, ++it) {
            const int a = it & 1;
            // the epilogue has drained this accumulator (its use two tiles ago)
            ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_AEMPTY + a, (((uint32_t)(it >> 1)) & 1) ^ 1,
                                                          abort_flag, p.status, kStatusTimeout));
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t dacc = tmem + (uint32_t)(a * kBN);
            for (int k = 0; k < nk; ++k, ++kc) {
                const int s = (int)(kc % kStages);
                ok = __all_sync(0xffffffffu, tc::wait_or_abort(bar + B_FULL + s, ((uint32_t)(kc / kStages)) & 1,
                                                              abort_flag, p.status, kStatusTimeout));
                if (!ok) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    const uint64_t da = tc::smem_desc(tc::smem_u32(sm + OFF_A + s * A_BYTES), 16, 1024, tc::kLayoutSw128);
                    const uint64_t db = tc::smem_desc(tc::smem_u32(sm + OFF_B + s * B_BYTES), 16, 1024, tc::kLayoutSw128);
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)            // K = 32 codes = 32 bytes per MMA
                        tc::mma_i8_ss(dacc, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc, (k | kk) != 0);
                    tc::mma_commit(bar + B_EMPTY + s);
                    if (k == nk - 1) tc::mma_commit(bar + B_AFULL + a);
                }
                __syncwarp();
            }
        }
    } else {
        // epilogue: warp w reads TMEM lanes 32 (w % 4) .. +31, i.e. output rows m0 + 32 (w % 4) + lane
        const int quarter = warp & 3;
        const bool vec = (p.N & 7) == 0;                          // every output row 16-byte aligned
        int it = 0;
        for (long long t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
            const int a = it & 1;
            const int m0 = (int)(t / p.tiles_n) * kBM, n0 = (int)(t % p.tiles_n) * kBN;
            const int row = m0 + quarter * 32 + lane;
            const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * kBN);
            const bool ok = tc::wait_or_abort(bar + B_AFULL + a, ((uint32_t)(it >> 1)) & 1, abort_flag, p.status,
                                              kStatusTimeout);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::tc_fence_after();
            const float st = row < p.T ? __ldg(p.s_t + row) : 0.f;
            for (int c = 0; c < kBN / 32; ++c) {
                uint32_t v[32];
                tc::tmem_ld32(trow + c * 32, v);
                tc::tmem_wait_ld();
                if (c == kBN / 32 - 1) {
                    // the whole accumulator is in registers: hand it back to the MMA warp
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar + B_AEMPTY + a);
                }
                uint16_t* dst = p.out + (long long)row * p.N + n0 + c * 32;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = n0 + c * 32 + 8 * i;
                    uint16_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool in = c0 + e < p.N;
                        float f = (float)(int)v[8 * i + e] * (st * (in ? __ldg(p.s_w + c0 + e) : 0.f));
                        if (p.bias && in) f += __ldg(p.bias + c0 + e);
                        h[e] = float_to_bf16_bits(f);
                    }
                    if (row < p.T && vec && c0 < p.N) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = (uint32_t)h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
                        reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[0], o[1], o[2], o[3]);
                    } else if (row < p.T) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c0 + e < p.N) dst[8 * i + e] = h[e];
                    }
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, kAcc * kBN);
}

}  // namespace

cudaError_t launch_matmul_i8(int T, int K, int N, const int8_t* q, const float* s_t, const int8_t* Wq,
                             const float* s_w, const float* bias, uint16_t* out, int* status, cudaStream_t st) {
    CUtensorMap ma, mb;
    if (!make_tmap_2d(&ma, true, q, (unsigned long long)K, (unsigned long long)T, (unsigned long long)K, kBK, kBM,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&mb, true, Wq, (unsigned long long)K, (unsigned long long)N, (unsigned long long)K, kBK, kBN,
                      CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const int smem = SMEM + 1024;
    const cudaError_t e = cudaFuncSetAttribute(matmul_i8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    MatmulArgs p{T, K, N, (N + kBN - 1) / kBN, 0, s_t, s_w, bias, out, status};
    p.tiles = (long long)p.tiles_n * ((T + kBM - 1) / kBM);
    const int grid = (int)(p.tiles < device_sm_count() ? p.tiles : device_sm_count());
    matmul_i8_kernel<<<grid, kWarps * 32, smem, st>>>(ma, mb, p);
    return cudaGetLastError();
}

}  // namespace ssd
