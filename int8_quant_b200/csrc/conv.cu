// conv.cu — the short causal convolution ahead of the scan: of the W last inputs of each of
// the C = H*P + 2*G*N channels (x | B | C, a slice of in_proj's rows), with SiLU, split into
// the dense x, B and C that the scan reads, and dt = softplus(dt_raw + dt_bias):
//   u[t,c] = bias[c] + sum_{i<W} weight[i,c] * s[t - (W-1) + i, c],   out = u / (1 + exp(-u))
// s is the row's inputs, with the W-1 inputs of its state (or zeros) in front.
//
// conv_fwd_kernel: a thread owns 8 channels (16 bytes) of a run of tokens and slides the
// window along it in registers, so each input is read once but for the W-1 in front of a
// run.  Bound by HBM (2 bytes read, 2 written per channel and token).  Blocks behind those
// of the convolution form dt and the final state.
// conv_step_kernel: one token; a thread owns 8 channels of a batch row and shifts their
// state in place.
#include "kernels.h"

namespace ssd {

namespace {

constexpr int kConvThreads = 256;

struct ConvArgs {
    int B, L, HP, GN, H, C;
    int nvec;                   // C / 8
    int run, runs;              // tokens per run, runs per batch row
    long long ld;
    const uint16_t* xbc;
    const uint16_t* dt_raw;
    const float* w;
    const float* bias;
    const float* dt_bias;
    const int* lengths;
    const uint16_t* init;
    uint16_t* x;
    float* dt;
    uint16_t* Bo;
    uint16_t* Co;
    uint16_t* fin;
    long long conv_blocks, dt_blocks;
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
__device__ __forceinline__ float silu(float u) { return __fdividef(u, 1.0f + __expf(-u)); }
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

__device__ __forceinline__ int row_length(const ConvArgs& a, int b) {
    if (!a.lengths) return a.L;
    const int n = __ldg(a.lengths + b);
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// 8 consecutive fp32 parameters, or zeros.
__device__ __forceinline__ void load_params(const float* p, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Where channels [c, c + 8) of a row go, and the distance between two rows there.
__device__ __forceinline__ uint16_t* out_of(const ConvArgs& a, int c, int* stride) {
    if (c < a.HP) {
        *stride = a.HP;
        return a.x + c;
    }
    *stride = a.GN;
    return c < a.HP + a.GN ? a.Bo + (c - a.HP) : a.Co + (c - a.HP - a.GN);
}

template <int W>
__global__ void __launch_bounds__(kConvThreads)
conv_fwd_kernel(const __grid_constant__ ConvArgs a) {
    if (blockIdx.x < a.conv_blocks) {
        const long long idx = (long long)blockIdx.x * kConvThreads + threadIdx.x;
        const int vec = (int)(idx % a.nvec);
        const long long r = idx / a.nvec;
        const int b = (int)(r / a.runs);
        if (b >= a.B) return;
        const int t0 = (int)(r % a.runs) * a.run;
        const int t1 = min(t0 + a.run, a.L);
        const int len = row_length(a, b);
        const int c = vec * 8;
        float w[W][8], bias[8], h[W][8];
#pragma unroll
        for (int i = 0; i < W; ++i) load_params(a.w + (long long)i * a.C + c, w[i]);
        load_params(a.bias ? a.bias + c : nullptr, bias);
        const uint16_t* in = a.xbc + (long long)b * a.L * a.ld + c;
        // the W-1 inputs in front of the run
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const int t = t0 - W + i;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (t >= 0)
                v = *reinterpret_cast<const uint4*>(in + t * a.ld);
            else if (a.init)
                v = *reinterpret_cast<const uint4*>(a.init + ((long long)b * (W - 1) + (t + W - 1)) * a.C + c);
            unpack8(v, h[i]);
        }
        int stride;
        uint16_t* out = out_of(a, c, &stride);
        out += ((long long)b * a.L + t0) * stride;
        for (int t = t0; t < t1; ++t, out += stride) {
            uint4 o = make_uint4(0u, 0u, 0u, 0u);
            if (t < len) {
#pragma unroll
                for (int i = 0; i + 1 < W; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[i][e] = h[i + 1][e];
                unpack8(*reinterpret_cast<const uint4*>(in + t * a.ld), h[W - 1]);
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u[e] = bias[e];
#pragma unroll
                    for (int i = 0; i < W; ++i) u[e] = fmaf(w[i][e], h[i][e], u[e]);
                    u[e] = silu(u[e]);
                }
                o = make_uint4(pack2(u[0], u[1]), pack2(u[2], u[3]), pack2(u[4], u[5]), pack2(u[6], u[7]));
            }
            *reinterpret_cast<uint4*>(out) = o;
        }
    } else if (blockIdx.x < a.conv_blocks + a.dt_blocks) {
        const long long i = ((long long)blockIdx.x - a.conv_blocks) * kConvThreads + threadIdx.x;
        const long long row = i / a.H;
        const int h = (int)(i % a.H);
        if (row >= (long long)a.B * a.L) return;
        const int b = (int)(row / a.L), t = (int)(row % a.L);
        a.dt[i] = t < row_length(a, b) ? softplus(bf16_bits_to_float(a.dt_raw[row * a.ld + h]) + __ldg(a.dt_bias + h))
                                       : 0.f;
    } else {
        const long long i = ((long long)blockIdx.x - a.conv_blocks - a.dt_blocks) * kConvThreads + threadIdx.x;
        const int vec = (int)(i % a.nvec);
        const long long r = i / a.nvec;
        const int b = (int)(r / (W - 1)), j = (int)(r % (W - 1));
        if (b >= a.B) return;
        const int t = row_length(a, b) - (W - 1) + j;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0)
            v = *reinterpret_cast<const uint4*>(a.xbc + ((long long)b * a.L + t) * a.ld + vec * 8);
        else if (a.init)
            v = *reinterpret_cast<const uint4*>(a.init + ((long long)b * (W - 1) + (t + W - 1)) * a.C + vec * 8);
        *reinterpret_cast<uint4*>(a.fin + r * a.C + vec * 8) = v;
    }
}

template <int W>
__global__ void __launch_bounds__(kConvThreads)
conv_step_kernel(const __grid_constant__ ConvArgs a, uint16_t* state) {
    const long long idx = (long long)blockIdx.x * kConvThreads + threadIdx.x;
    if (blockIdx.x < a.conv_blocks) {
        const int vec = (int)(idx % a.nvec), c = vec * 8;
        const int b = (int)(idx / a.nvec);
        if (b >= a.B) return;
        uint4 s[W];
        uint4* sp = reinterpret_cast<uint4*>(state + (long long)b * (W - 1) * a.C + c);
        const int sv = a.C / 8;
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) s[i] = sp[(long long)i * sv];
        s[W - 1] = *reinterpret_cast<const uint4*>(a.xbc + b * a.ld + c);
        float u[8];
        load_params(a.bias ? a.bias + c : nullptr, u);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float w[8], h[8];
            load_params(a.w + (long long)i * a.C + c, w);
            unpack8(s[i], h);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = fmaf(w[e], h[e], u[e]);
            if (i > 0) sp[(long long)(i - 1) * sv] = s[i];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = silu(u[e]);
        int stride;
        uint16_t* out = out_of(a, c, &stride);
        out += (long long)b * stride;
        *reinterpret_cast<uint4*>(out) =
            make_uint4(pack2(u[0], u[1]), pack2(u[2], u[3]), pack2(u[4], u[5]), pack2(u[6], u[7]));
    } else {
        const long long i = idx - a.conv_blocks * kConvThreads;
        if (i >= (long long)a.B * a.H) return;
        const int b = (int)(i / a.H), h = (int)(i % a.H);
        a.dt[i] = softplus(bf16_bits_to_float(a.dt_raw[b * a.ld + h]) + __ldg(a.dt_bias + h));
    }
}

long long blocks_for(long long threads) { return (threads + kConvThreads - 1) / kConvThreads; }

ConvArgs conv_args(const ConvDims& d, const ConvIn& in, const ConvOut& out) {
    ConvArgs a{};
    a.B = d.B; a.L = d.L; a.H = d.H; a.HP = d.HP; a.GN = d.GN; a.C = d.HP + 2 * d.GN;
    a.nvec = a.C / 8;
    a.ld = in.ld;
    a.xbc = in.xbc; a.dt_raw = in.dt_raw; a.w = in.weight; a.bias = in.bias; a.dt_bias = in.dt_bias;
    a.lengths = in.lengths; a.init = in.init;
    a.x = out.x; a.dt = out.dt; a.Bo = out.B; a.Co = out.C; a.fin = out.final_state;
    return a;
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvDims& d, const ConvIn& in, const ConvOut& out, cudaStream_t st) {
    ConvArgs a = conv_args(d, in, out);
    a.run = 32;
    a.runs = (a.L + a.run - 1) / a.run;
    a.conv_blocks = blocks_for((long long)a.nvec * a.runs * a.B);
    a.dt_blocks = a.dt ? blocks_for((long long)a.B * a.L * a.H) : 0;
    const long long fin = a.fin ? blocks_for((long long)a.B * (d.W - 1) * a.nvec) : 0;
    const unsigned grid = (unsigned)(a.conv_blocks + a.dt_blocks + fin);
    if (d.W == 2) conv_fwd_kernel<2><<<grid, kConvThreads, 0, st>>>(a);
    else if (d.W == 3) conv_fwd_kernel<3><<<grid, kConvThreads, 0, st>>>(a);
    else conv_fwd_kernel<4><<<grid, kConvThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_conv_step(const ConvDims& d, const ConvIn& in, uint16_t* state, const ConvOut& out,
                             cudaStream_t st) {
    ConvArgs a = conv_args(d, in, out);
    a.conv_blocks = blocks_for((long long)a.nvec * a.B);
    const unsigned grid = (unsigned)(a.conv_blocks + (a.dt ? blocks_for((long long)a.B * a.H) : 0));
    if (d.W == 2) conv_step_kernel<2><<<grid, kConvThreads, 0, st>>>(a, state);
    else if (d.W == 3) conv_step_kernel<3><<<grid, kConvThreads, 0, st>>>(a, state);
    else conv_step_kernel<4><<<grid, kConvThreads, 0, st>>>(a, state);
    return cudaGetLastError();
}

}  // namespace ssd
