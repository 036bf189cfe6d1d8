// conv.cu — the short causal convolution ahead of the scan: of the W last inputs of each of
// the C = H*P + 2*G*N channels (x | B | C, a slice of in_proj's rows), with SiLU, split into
// the dense x, B and C that the scan reads, and dt = softplus(dt_raw + dt_bias):
//   u[t,c] = bias[c] + sum_{i<W} weight[i,c] * s[t - (W-1) + i, c],   out = u / (1 + exp(-u))
// s is the row's inputs, with the W-1 inputs of its state (or zeros) in front.
//
// conv_fwd_kernel: a CTA stages a tile of kTile tokens (and the W-1 in front of them) of 256
// channels in shared memory with cp.async, then each thread slides the window along half the
// tile's tokens for 4 channels.  Bound by HBM (2 bytes read, 2 written per channel and token);
// loads wait in shared memory, not in registers, so 6 CTAs of 128 threads an SM keep 200 KB
// of them in flight.  8 rows of 8192 tokens of 5376 channels, and 80 dt: 1.44 GB in 227 us
// (6.3 TB/s; 6.5 is the copy bandwidth), 257 us once the power limit has lowered the clock to
// 1.6 GHz.  Tiles of 32 tokens (more halo, more parameter loads) take 239 and 280 us, of 128
// (3 CTAs an SM) 251 and 274; plain instead of packed fp32 arithmetic 258 and 283; a window
// slid along registers, without the staging, 344.  Blocks behind those of the convolution form
// dt and the final state.
// conv_step_kernel: one token; a thread owns 8 channels of one or two batch rows and shifts
// their state in place (8 x 5376 channels in a graph 1.8 us, the launch; 128 x 10240, 21 MB,
// 3.8 us = 5.5 TB/s from L2).
#include "kernels.h"

namespace ssd {

namespace {

constexpr int kStepThreads = 128;
constexpr int kThreads = 128;               // of conv_fwd_kernel
constexpr int kTile = 64;                   // its tokens
constexpr int kBlock = 256;                 // its channels
constexpr int kCh = 4;                      // channels of a thread
constexpr int kGroups = kBlock / kCh, kSubs = kThreads / kGroups, kSub = kTile / kSubs;
constexpr int kDtRows = 8;                  // tokens whose dt (of one head) a thread forms

struct ConvArgs {
    int B, L, HP, GN, H, C;
    int tiles, blocks;          // tiles of a batch row, channel blocks
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

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

__device__ __forceinline__ int row_length(const ConvArgs& a, int b) {
    if (!a.lengths) return a.L;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// Where channel c of a row goes, and the distance between two rows there.
__device__ __forceinline__ uint16_t* out_of(const ConvArgs& a, int c, int* stride) {
    if (c < a.HP) {
        *stride = a.HP;
        return a.x + c;
    }
    *stride = a.GN;
    return c < a.HP + a.GN ? a.Bo + (c - a.HP) : a.Co + (c - a.HP - a.GN);
}

__device__ __forceinline__ void load_params(const float* p, f32x2 (&f)[2]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    f[0] = pair2(a.x, a.y);
    f[1] = pair2(a.z, a.w);
}
__device__ __forceinline__ void unpack4(const uint2& v, f32x2 (&f)[2]) {
    f[0] = pair2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = pair2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
// 16 bytes to shared memory, asynchronously; zeros if !`some` (`src` is then not read).
__device__ __forceinline__ void stage16(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(some ? 16 : 0)
                 : "memory");
}

// Four channels of one token: the window h of the W-1 inputs in front of it moves on.
template <int W>
__device__ __forceinline__ uint2 conv_token(const uint2& raw, const f32x2 (&w)[W][2], const f32x2 (&bias)[2],
                                            f32x2 (&h)[W - 1][2]) {
    f32x2 s[2], u[2];
    unpack4(raw, s);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        u[e] = bias[e];
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) u[e] = fma2(w[i][e], h[i][e], u[e]);
        u[e] = fast_silu2(fma2(w[W - 1][e], s[e], u[e]));
#pragma unroll
        for (int i = 0; i + 2 < W; ++i) h[i][e] = h[i + 1][e];
        h[W - 2][e] = s[e];
    }
    return make_uint2(pack2(u[0]), pack2(u[1]));
}

template <int W>
__device__ __forceinline__ void conv_tile(const ConvArgs& a) {
    __shared__ __align__(16) uint16_t tile[kTile + W - 1][kBlock];
    const int block = (int)(blockIdx.x % a.blocks), r = (int)(blockIdx.x / a.blocks);
    const int b = r / a.tiles, t0 = (r % a.tiles) * kTile, c0 = block * kBlock;
    const int t1 = min(t0 + kTile, a.L), live = min(t1, row_length(a, b));
    const uint16_t* in = a.xbc + (long long)b * a.L * a.ld + c0;
    // row i of the tile is token t0 + i - (W-1), behind the row's start an input of its state
    if (t0 < live) {
        constexpr int kChunks = kBlock / 8;
        const int cols = min(kBlock, a.C - c0) / 8, rows = live - t0 + W - 1;
        for (int i = threadIdx.x; i < rows * kChunks; i += kThreads) {
            const int t = t0 + i / kChunks - (W - 1), j = i % kChunks;
            if (j >= cols) continue;
            const uint16_t* src = in;
            if (t >= 0) src = in + t * a.ld + j * 8;
            else if (a.init) src = a.init + ((long long)b * (W - 1) + (t + W - 1)) * a.C + c0 + j * 8;
            stage16(&tile[i / kChunks][j * 8], src, t >= 0 || a.init);
        }
    }
    const int c = c0 + (threadIdx.x % kGroups) * kCh, s0 = (threadIdx.x / kGroups) * kSub;
    const bool mine = c < a.C;
    f32x2 w[W][2], bias[2] = {0, 0}, h[W - 1][2];
    if (mine) {
#pragma unroll
        for (int i = 0; i < W; ++i) load_params(a.w + (long long)i * a.C + c, w[i]);
        if (a.bias) load_params(a.bias + c, bias);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!mine || t0 + s0 >= t1) return;
    const uint2* col = reinterpret_cast<const uint2*>(&tile[s0][c - c0]);
    constexpr int kRow = kBlock / 4;                              // uint2s of a tile row
    int stride;
    uint16_t* out = out_of(a, c, &stride);
    out += ((long long)b * a.L + t0 + s0) * stride;
    const int n = live - t0 - s0, end = min(kSub, t1 - t0 - s0);    // tokens to compute, to write
    if (n > 0) {
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) unpack4(col[i * kRow], h[i]);
        col += (W - 1) * kRow;
    }
    if (n >= kSub) {
#pragma unroll 8
        for (int j = 0; j < kSub; ++j, out += stride)
            *reinterpret_cast<uint2*>(out) = conv_token<W>(col[j * kRow], w, bias, h);
    } else {
        for (int j = 0; j < end; ++j, out += stride)
            *reinterpret_cast<uint2*>(out) = j < n ? conv_token<W>(col[j * kRow], w, bias, h) : make_uint2(0u, 0u);
    }
}

template <int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const __grid_constant__ ConvArgs a) {
    grid_release();
    grid_wait();
    if (blockIdx.x < a.conv_blocks) {
        conv_tile<W>(a);
    } else if (blockIdx.x < a.conv_blocks + a.dt_blocks) {
        const long long i = ((long long)blockIdx.x - a.conv_blocks) * kThreads + threadIdx.x;
        const int h = (int)(i % a.H);
        const long long row0 = i / a.H * kDtRows, rows = (long long)a.B * a.L;
        uint16_t raw[kDtRows];
#pragma unroll
        for (int j = 0; j < kDtRows; ++j)
            if (row0 + j < rows) raw[j] = a.dt_raw[(row0 + j) * a.ld + h];
        const float bias = a.dt_bias[h];
#pragma unroll
        for (int j = 0; j < kDtRows; ++j) {
            const long long row = row0 + j;
            if (row >= rows) break;
            const bool real = !a.lengths || (int)(row % a.L) < row_length(a, (int)(row / a.L));
            a.dt[row * a.H + h] = real ? softplus(bf16_bits_to_float(raw[j]) + bias) : 0.f;
        }
    } else {
        const long long i = ((long long)blockIdx.x - a.conv_blocks - a.dt_blocks) * kThreads + threadIdx.x;
        const int nvec = a.C / 8, c = (int)(i % nvec) * 8;
        const long long r = i / nvec;
        const int b = (int)(r / (W - 1)), j = (int)(r % (W - 1));
        if (b >= a.B) return;
        const int t = row_length(a, b) - (W - 1) + j;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0)
            v = *reinterpret_cast<const uint4*>(a.xbc + ((long long)b * a.L + t) * a.ld + c);
        else if (a.init)
            v = *reinterpret_cast<const uint4*>(a.init + ((long long)b * (W - 1) + (t + W - 1)) * a.C + c);
        *reinterpret_cast<uint4*>(a.fin + r * a.C + c) = v;
    }
}

// R batch rows a thread: their parameters are read once.
template <int W, int R>
__global__ void __launch_bounds__(kStepThreads)
conv_step_kernel(const __grid_constant__ ConvArgs a, uint16_t* state) {
    grid_release();
    grid_wait();
    const long long idx = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    if (blockIdx.x < a.conv_blocks) {
        const int nvec = a.C / 8, sv = nvec;
        const int c = (int)(idx % nvec) * 8;
        const long long b = idx / nvec * R;
        if (b >= a.B) return;
        const int rows = min(R, (int)(a.B - b));
        // every load is ahead of the first store, which the compiler cannot tell apart from them
        uint4 s[R][W];
        uint4* sp = reinterpret_cast<uint4*>(state + b * (W - 1) * a.C + c);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) break;
#pragma unroll
            for (int i = 0; i + 1 < W; ++i) s[r][i] = sp[(long long)(r * (W - 1) + i) * sv];
            s[r][W - 1] = *reinterpret_cast<const uint4*>(a.xbc + (b + r) * a.ld + c);
        }
        f32x2 w[W][4], bias[4] = {0, 0, 0, 0};
        if (a.bias) load8(a.bias + c, bias);
#pragma unroll
        for (int i = 0; i < W; ++i) load8(a.w + (long long)i * a.C + c, w[i]);
        int stride;
        uint16_t* out = out_of(a, c, &stride);
        out += b * stride;
#pragma unroll
        for (int r = 0; r < R; ++r, out += stride) {
            if (r >= rows) break;
            f32x2 u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = bias[e];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                f32x2 h[4];
                unpack8(s[r][i], h);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = fma2(w[i][e], h[e], u[e]);
                if (i > 0) sp[(long long)(r * (W - 1) + i - 1) * sv] = s[r][i];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = fast_silu2(u[e]);
            *reinterpret_cast<uint4*>(out) = pack8(u);
        }
    } else {
        const long long i = idx - a.conv_blocks * kStepThreads;
        if (i >= (long long)a.B * a.H) return;
        const int b = (int)(i / a.H), h = (int)(i % a.H);
        a.dt[i] = softplus(bf16_bits_to_float(a.dt_raw[b * a.ld + h]) + a.dt_bias[h]);
    }
}

long long blocks_for(long long threads, int block) { return (threads + block - 1) / block; }

ConvArgs conv_args(const ConvDims& d, const ConvIn& in, const ConvOut& out) {
    ConvArgs a{};
    a.B = d.B; a.L = d.L; a.H = d.H; a.HP = d.HP; a.GN = d.GN; a.C = d.HP + 2 * d.GN;
    a.ld = in.ld;
    a.xbc = in.xbc; a.dt_raw = in.dt_raw; a.w = in.weight; a.bias = in.bias; a.dt_bias = in.dt_bias;
    a.lengths = in.lengths; a.init = in.init;
    a.x = out.x; a.dt = out.dt; a.Bo = out.B; a.Co = out.C; a.fin = out.final_state;
    return a;
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvDims& d, const ConvIn& in, const ConvOut& out, cudaStream_t st) {
    ConvArgs a = conv_args(d, in, out);
    a.tiles = (a.L - 1) / kTile + 1;
    a.blocks = (a.C - 1) / kBlock + 1;
    const long long rows = (long long)a.B * a.L;
    a.conv_blocks = (long long)a.blocks * a.tiles * a.B;
    a.dt_blocks = a.dt ? blocks_for(blocks_for(rows, kDtRows) * a.H, kThreads) : 0;
    const long long fin = a.fin ? blocks_for((long long)a.B * (d.W - 1) * (a.C / 8), kThreads) : 0;
    const unsigned grid = (unsigned)(a.conv_blocks + a.dt_blocks + fin);
    if (d.W == 2) return launch_programmatic(conv_fwd_kernel<2>, grid, kThreads, 0, st, 1, a);
    if (d.W == 3) return launch_programmatic(conv_fwd_kernel<3>, grid, kThreads, 0, st, 1, a);
    return launch_programmatic(conv_fwd_kernel<4>, grid, kThreads, 0, st, 1, a);
}

template <int R>
static cudaError_t launch_step(const ConvDims& d, ConvArgs a, uint16_t* state, cudaStream_t st) {
    a.conv_blocks = blocks_for((long long)(a.C / 8) * (((long long)a.B + R - 1) / R), kStepThreads);
    const unsigned grid = (unsigned)(a.conv_blocks + (a.dt ? blocks_for((long long)a.B * a.H, kStepThreads) : 0));
    if (d.W == 2) return launch_programmatic(conv_step_kernel<2, R>, grid, kStepThreads, 0, st, 1, a, state);
    if (d.W == 3) return launch_programmatic(conv_step_kernel<3, R>, grid, kStepThreads, 0, st, 1, a, state);
    return launch_programmatic(conv_step_kernel<4, R>, grid, kStepThreads, 0, st, 1, a, state);
}

// Two rows a thread where one each would be more threads than the GPU holds at a time (128 x
// 5376 channels 3.4 us with one, 3.6 with two; 128 x 10240 4.3, 3.8; 256 x 10240 7.0, 5.9).
cudaError_t launch_conv_step(const ConvDims& d, const ConvIn& in, uint16_t* state, const ConvOut& out,
                             cudaStream_t st) {
    const ConvArgs a = conv_args(d, in, out);
    return (long long)(a.C / 8) * a.B > 768LL * device_sm_count() ? launch_step<2>(d, a, state, st)
                                                                   : launch_step<1>(d, a, state, st);
}

}  // namespace ssd
