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
// One CTA per token; each thread holds VPT vectors of 8 features.  Bound by HBM: 11 bytes a
// feature with an fp32 residual (2 + 4 read, 4 + 1 written), 5 with the gate.
#include "kernels.h"

namespace ssd {

namespace {

enum : int { kResNone = 0, kResF32 = 1, kResBf16 = 2, kGate = 3 };

struct NormArgs {
    int d;
    long long ld2;              // row stride of the second input (z; d for a residual)
    const uint16_t* x;          // x or y
    const void* in2;            // residual or z (null: none)
    const float* w;             // null: ones
    float eps;
    void* res_out;              // may be null, may be in2 itself
    int8_t* q;
    float* scale;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
}
// max that keeps a NaN (fmaxf drops it), so that a row with one is seen
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int KIND, int VPT>
__global__ void __launch_bounds__(1024)
rmsnorm_i8_kernel(const __grid_constant__ NormArgs a) {
    const long long row = blockIdx.x;
    const int nv = a.d >> 3;
    float p[VPT][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nv) break;
        float v[8];
        unpack8(*(reinterpret_cast<const uint4*>(a.x + row * a.d) + i), v);
        if (KIND == kGate) {
            float z[8];
            unpack8(*(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.in2) + row * a.ld2) + i), z);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= __fdividef(z[e], 1.0f + __expf(-z[e]));
        } else if (KIND == kResF32) {
            const float4* rp = reinterpret_cast<const float4*>(static_cast<const float*>(a.in2) + row * a.d) + 2 * i;
            const float4 r0 = rp[0], r1 = rp[1];
            v[0] += r0.x; v[1] += r0.y; v[2] += r0.z; v[3] += r0.w;
            v[4] += r1.x; v[5] += r1.y; v[6] += r1.z; v[7] += r1.w;
        } else if (KIND == kResBf16) {
            float r[8];
            unpack8(*(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.in2) + row * a.d) + i), r);
            // the norm is of the residual as it is stored: rounded to bf16
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = bf16_bits_to_float(float_to_bf16_bits(v[e] + r[e]));
        }
        if (KIND != kGate && a.res_out) {
            if (KIND == kResF32) {
                float4* op = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + row * a.d) + 2 * i;
                op[0] = make_float4(v[0], v[1], v[2], v[3]);
                op[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + row * a.d)[i] =
                    make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            }
        }
        float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.w) {
            const float4* wp = reinterpret_cast<const float4*>(a.w) + 2 * i;
            const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
            w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
            w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(v[e], v[e], ss);
            p[k][e] = v[e] * w[e];
            top = max_nan(top, fabsf(p[k][e]));
        }
    }
    __shared__ float part_s[32], part_m[32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, off);
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        part_s[warp] = ss;
        part_m[warp] = top;
    }
    __syncthreads();
    const int nw = blockDim.x >> 5;
    ss = lane < nw ? part_s[lane] : 0.f;
    top = lane < nw ? part_m[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, off);
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    }
    // A row that is not finite gets the scale NaN and codes 0; a row of zeros (below 2^-100,
    // where 127 / top would overflow) the scale 1 and codes 0.
    const bool finite = ss < __int_as_float(0x7f800000) && top < __int_as_float(0x7f800000);
    const bool some = finite && top >= 0x1p-100f;
    const float inv = some ? 127.0f / top : 0.f;
    if (threadIdx.x == 0) {
        const float r = rsqrtf(ss / (float)a.d + a.eps);
        a.scale[row] = some ? top * r / 127.0f : finite ? 1.0f : __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nv) break;
        uint32_t o[2] = {0u, 0u};
        if (some) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e >> 2] |= ((uint32_t)quant_i8(p[k][e], inv) & 0xffu) << (8 * (e & 3));
        }
        reinterpret_cast<uint2*>(a.q + row * a.d)[i] = make_uint2(o[0], o[1]);
    }
}

template <int KIND>
cudaError_t launch_kind(int T, const NormArgs& a, cudaStream_t st) {
    const int nv = a.d >> 3;
    const int vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : 4;
    const int per = (nv + vpt - 1) / vpt;
    const int threads = (per + 31) / 32 * 32;
    if (vpt == 1) rmsnorm_i8_kernel<KIND, 1><<<T, threads, 0, st>>>(a);
    else if (vpt == 2) rmsnorm_i8_kernel<KIND, 2><<<T, threads, 0, st>>>(a);
    else rmsnorm_i8_kernel<KIND, 4><<<T, threads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm_i8(int T, int d, const uint16_t* x, const void* residual, bool fp32, const float* w,
                                  float eps, void* res_out, int8_t* q, float* scale, cudaStream_t st) {
    const NormArgs a{d, d, x, residual, w, eps, res_out, q, scale};
    if (!residual) return launch_kind<kResNone>(T, a, st);
    return fp32 ? launch_kind<kResF32>(T, a, st) : launch_kind<kResBf16>(T, a, st);
}

cudaError_t launch_gated_rmsnorm_i8(int T, int d, const uint16_t* y, const uint16_t* z, long long ld_z,
                                    const float* w, float eps, int8_t* q, float* scale, cudaStream_t st) {
    return launch_kind<kGate>(T, NormArgs{d, ld_z, y, z, w, eps, nullptr, q, scale}, st);
}

}  // namespace ssd
