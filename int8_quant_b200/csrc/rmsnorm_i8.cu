// rmsnorm_i8.cu — RMSNorm of a token's features to INT8 codes with one scale per token, the
// two norms of a W8A8 Mamba-2 layer:
//   ssd_add_rmsnorm_i8    v = x + residual (kept as the next residual), ahead of in_proj
//   ssd_gated_rmsnorm_i8  v = y * silu(z), silu(z) = z / (1 + exp(-z)), ahead of out_proj
// and then, with r = 1 / sqrt(mean(v^2) + eps) and u = v * w * r,
//   scale = max|u| / 127,  q = rint(u / scale).
// r is common to the row, so it cancels in the codes: with p = v * w and a = max|p|,
//   q = rint(p * (127 / a)),   scale = a * r / 127,
// and the row is read once, kept in registers, and needs one reduction (of v^2 and |p|
// together) before its codes are written.
//
// Bound by HBM: 11 bytes a feature with an fp32 residual (2 + 4 read, 4 + 1 written), 5 with
// the gate, 2 more where the codes' values are asked for.  One CTA per token and VPT vectors
// of 8 features a thread, all loads issued before anything else; many small CTAs resident on
// an SM cover each other's barrier.  Measured, in a graph (6.53 TB/s is the copy bandwidth):
//   65536 x 2560, fp32 residual   265 us = 7.0 TB/s, with values 318 us = 6.9 TB/s
//   65536 x 2560, bf16 residual   176 us = 6.7 TB/s, with values 221 us = 6.8 TB/s
//   65536 x 2560, no residual     111 us = 4.5 TB/s, with values 140 us = 6.0 TB/s
//   16384 x 5120, gate             67 us = 6.3 TB/s, with values  89 us = 6.6 TB/s
// The gate spends two special-function instructions a feature (exponential, reciprocal); with
// packed fp32 arithmetic it takes half the instructions of the plain form (95 us).  A
// persistent grid that loads the next token ahead needs twice the registers and was slower:
// 291 and 94 us.
#include "kernels.h"

namespace ssd {

namespace {

enum : int { kResNone = 0, kResF32 = 1, kResBf16 = 2, kGate = 3 };

constexpr int kMaxThreads = 512;
constexpr float kMagic = 12582912.0f;       // 1.5 * 2^23: adding it rounds a small number to a whole one

struct NormArgs {
    int d;
    long long ld2;              // row stride of the second input (z; d for a residual)
    const uint16_t* x;          // x or y
    const void* in2;            // residual or z (null: none)
    const float* w;             // null: ones
    float eps;
    void* res_out;              // may be null, may be in2 or x itself
    bool res_f32;               // its type
    int8_t* q;
    float* scale;
    uint16_t* values;           // q * scale as bf16, or null
};

template <int KIND, int VPT>
struct RowIn {
    uint4 x[VPT];
    uint4 r[VPT][KIND == kResF32 ? 2 : 1];
};

template <int KIND, int VPT>
__device__ __forceinline__ void load_row(const NormArgs& a, long long row, int nv, RowIn<KIND, VPT>& in) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nv) continue;
        in.x[k] = reinterpret_cast<const uint4*>(a.x + row * a.d)[i];
        if (KIND == kResF32) {
            const uint4* rp = reinterpret_cast<const uint4*>(static_cast<const float*>(a.in2) + row * a.d) + 2 * i;
            in.r[k][0] = rp[0];
            in.r[k][KIND == kResF32 ? 1 : 0] = rp[1];
        } else if (KIND != kResNone) {
            in.r[k][0] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.in2) + row * a.ld2)[i];
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// The largest of a warp's values, none of them negative (their bits are in their order).
__device__ __forceinline__ float warp_max(float v) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// RES: CTAs of 512 threads that the registers leave room for on an SM.
template <int KIND, int VPT, int RES>
__global__ void __launch_bounds__(kMaxThreads, RES)
rmsnorm_i8_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float2 part[kMaxThreads / 32], row_scale;
    const int nv = a.d >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const float inf = __int_as_float(0x7f800000);
    const long long row = blockIdx.x;
    grid_release();
    grid_wait();
    RowIn<KIND, VPT> in;
    load_row<KIND, VPT>(a, row, nv, in);
    // With a residual, each vector's weights are loaded ahead of the residual stores in front of
    // it, which the compiler cannot tell apart from them (2047 x 2048 11.0 -> 9.8 us); four
    // vectors a thread have no registers for that (16384 x 8192 218 -> 259 us).
    constexpr bool kEarly = KIND != kGate && VPT == 2;
    f32x2 w[4] = {both2(1.f), both2(1.f), both2(1.f), both2(1.f)};
    if (kEarly && a.w && (int)threadIdx.x < nv) load8(a.w + 8 * threadIdx.x, w);
    f32x2 p[VPT][4];
    f32x2 ss2 = both2(0.f);
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nv) continue;
        f32x2 v[4], wk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) wk[e] = w[e];
        if (kEarly && k + 1 < VPT && a.w && i + (int)blockDim.x < nv) load8(a.w + 8 * (i + blockDim.x), w);
        unpack8(in.x[k], v);
        if (KIND == kGate) {
            f32x2 z[4];
            unpack8(in.r[k][0], z);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], fast_silu2(z[e]));
        } else if (KIND == kResF32) {
            const uint4 r0 = in.r[k][0], r1 = in.r[k][KIND == kResF32 ? 1 : 0];
            const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = add2(v[e], pair2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])));
        } else if (KIND == kResBf16) {
            f32x2 r[4];
            unpack8(in.r[k][0], r);
            // the norm is of the residual as it is stored: rounded to bf16
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = add2(v[e], r[e]);
            unpack8(pack8(v), v);
        }
        if (KIND != kGate && a.res_out) {
            if (KIND == kResF32 || (KIND == kResNone && a.res_f32)) {
                ulonglong2* op = reinterpret_cast<ulonglong2*>(static_cast<float*>(a.res_out) + row * a.d) + 2 * i;
                op[0] = make_ulonglong2(v[0], v[1]);
                op[1] = make_ulonglong2(v[2], v[3]);
            } else {
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + row * a.d)[i] = pack8(v);
            }
        }
        if (!kEarly && a.w) load8(a.w + 8 * i, wk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ss2 = fma2(v[e], v[e], ss2);
            p[k][e] = mul2(v[e], wk[e]);
            const float2 m = split2(p[k][e]);
            top = fmaxf(fmaxf(top, fabsf(m.x)), fabsf(m.y));     // a NaN is dropped here, but not by ss2
        }
    }
    float ss = split2(ss2).x + split2(ss2).y;
    ss = warp_sum(ss);
    top = warp_max(top);
    if (lane == 0) part[warp] = make_float2(ss, top);
    __syncthreads();
    // One warp finishes the reduction.  A row that is not finite gets the scale NaN and codes
    // 0; a row of zeros (below 2^-100, where 127 / top would overflow) the scale 1 and codes 0.
    if (warp == 0) {
        const float2 mine = lane < nw ? part[lane] : make_float2(0.f, 0.f);
        ss = warp_sum(mine.x);
        top = warp_max(mine.y);
        const bool finite = ss < inf && top < inf;
        const bool some = finite && top >= 0x1p-100f;
        const float s = some ? top * rsqrtf(ss / (float)a.d + a.eps) / 127.0f
                             : finite ? 1.0f : __int_as_float(0x7fffffff);
        if (lane == 0) {
            a.scale[row] = s;
            row_scale = make_float2(some ? 127.0f / top : 0.f, s);
        }
    }
    __syncthreads();
    const float inv = row_scale.x, scale = row_scale.y;
    const bool some = inv != 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nv) continue;
        uint2 o = make_uint2(0u, 0u);
        f32x2 c[4];
        if (some) {
            // 1.5 * 2^23 + c has the code's two's complement in its low byte, rounded to nearest
            // even; |p * inv| <= 127 (1 + 2^-22), so no code passes 127
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = fma2(p[k][e], both2(inv), both2(kMagic));
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = __byte_perm(__float_as_uint(split2(c[e]).x), __float_as_uint(split2(c[e]).y), 0x0040);
            o = make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
        }
        reinterpret_cast<uint2*>(a.q + row * a.d)[i] = o;
        if (a.values) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = mul2(some ? add2(c[e], both2(-kMagic)) : both2(0.f), both2(scale));
            reinterpret_cast<uint4*>(a.values + row * a.d)[i] = pack8(c);
        }
    }
}

template <int KIND, int VPT, int RES>
cudaError_t launch_vpt(const NormArgs& a, int T, cudaStream_t st) {
    const int nv = a.d >> 3;
    const int threads = ((nv + VPT - 1) / VPT + 31) / 32 * 32;
    return launch_programmatic(rmsnorm_i8_kernel<KIND, VPT, RES>, (unsigned)T, threads, 0, st, 1, a);
}

// Two vectors a thread as long as a few CTAs fit an SM's registers, then four: with a residual
// up to 320 threads (16384 x 5120 135 us, 139 with four; 8192 216 with four), with the gate up
// to 512 (16384 x 8192 109 us, 127 with four).  The residual's loads want registers (135 us
// with 48, 158 with 32).  The gate's arithmetic wants warps to hide behind where there are many
// tokens (16384 x 5120 68 us with 2048 threads of 32 registers an SM, 81 with 1536 of 40); few
// tokens want their loads at once (128 x 5120 back to back 6.0 and 4.5 us).
template <int KIND>
cudaError_t launch_kind(const NormArgs& a, int T, cudaStream_t st) {
    if constexpr (KIND == kGate) {
        if (a.d <= 16 * kMaxThreads)
            return T <= 2 * device_sm_count() ? launch_vpt<KIND, 2, 3>(a, T, st) : launch_vpt<KIND, 2, 4>(a, T, st);
    } else {
        if (a.d <= 5120) return launch_vpt<KIND, 2, 2>(a, T, st);
    }
    if (a.d <= 32 * kMaxThreads) return launch_vpt<KIND, 4, 2>(a, T, st);
    return launch_vpt<KIND, 8, 1>(a, T, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm_i8(int T, int d, const uint16_t* x, const void* residual, bool fp32, const float* w,
                                  float eps, void* res_out, int8_t* q, float* scale, uint16_t* values,
                                  cudaStream_t st) {
    const NormArgs a{d, d, x, residual, w, eps, res_out, fp32, q, scale, values};
    if (!residual) return launch_kind<kResNone>(a, T, st);
    return fp32 ? launch_kind<kResF32>(a, T, st) : launch_kind<kResBf16>(a, T, st);
}

cudaError_t launch_gated_rmsnorm_i8(int T, int d, const uint16_t* y, const uint16_t* z, long long ld_z,
                                    const float* w, float eps, int8_t* q, float* scale, uint16_t* values,
                                    cudaStream_t st) {
    return launch_kind<kGate>(NormArgs{d, ld_z, y, z, w, eps, nullptr, false, q, scale, values}, T, st);
}

}  // namespace ssd
