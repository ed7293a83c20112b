// mhc_mx4.cu -- the 4-bit serving path around the residual streams on
// sm_100a: the read map that writes the layer's input as microscaled e2m1
// codes, the product of two such matrices, and the same product with the
// residual mix as its epilogue.
//
//   read map       a[t] = codes of x_in[t,c] = sum_j sigmoid(h_pre[t,j]) X[t,j,c]
//   product        out[t,n] = sum_b sa[t,b] sw[n,b] sum_{k in b} a[t,k] w[n,k]
//   product + mix  Y[t,i,c] = sum_j H[t,i,j] X[t,j,c] + h_post[t,i] out[t,c]
#include "birkhoff_math.cuh"
#include "launch.h"
#include "mix_common.cuh"
#include "mx_common.cuh"

namespace mhc {

namespace {

// ------------------------------------------------------------------ read map

// A CTA takes chunks of 128 vectors (1024 channels) of a token, so that a
// single token's streams are spread over several CTAs.
constexpr int kReadThreads = 128;

__global__ void __launch_bounds__(kReadThreads)
premap_fwd_mx4_kernel(const uint4* X, const float* hpre, uint8_t* codes, uint8_t* scales, int64_t items, int chunks,
                      int CV)
{
    const int64_t sp = mx_scale_pitch((int64_t)CV * 8);
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t t = it / chunks;
        const int v = (int)(it - t * chunks) * kReadThreads + threadIdx.x;
        const bool in = v < CV;
        const float4 q = __ldg(reinterpret_cast<const float4*>(hpre) + t);
        const float s[4] = {sigmoidf(q.x), sigmoidf(q.y), sigmoidf(q.z), sigmoidf(q.w)};
        float xf[4][8], o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            unpack8(in ? __ldcs(X + (t * 4 + j) * CV + v) : make_uint4(0u, 0u, 0u, 0u), xf[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = s[0] * xf[0][e];
#pragma unroll
            for (int j = 1; j < 4; ++j) a = fmaf(s[j], xf[j][e], a);
            o[e] = in ? a : 0.0f;
        }
        const int S = mx_scale_byte<MHC_MX_E2M1>(mx_block_max(mx_amax8(o)));
        if (in) {
            reinterpret_cast<uint32_t*>(codes)[t * CV + v] = mx_encode8<MHC_MX_E2M1>(o, S).x;
            mx_store_scale(scales + t * sp, v, CV, S);
        }
    }
}

// ------------------------------------------------------------------- product

constexpr int kDotThreads = 256;  // one warp for each of 8 channels
constexpr int kDotTokens = 8;

struct MixArgs {
    const uint4* X;  // nullptr: the plain product
    const float *H, *hpost;
};

// Eight tokens by eight channels a CTA: a warp holds one channel, its lanes
// walk the blocks of 32 along K.
template <bool kMix>
__global__ void __launch_bounds__(kDotThreads)
mx4_dot_kernel(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws, MixArgs m, uint4* out,
               int64_t T, int N, int K)
{
    __shared__ float f[kDotTokens][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, KB = K / kMxBlock;
    const int64_t t0 = (int64_t)blockIdx.y * kDotTokens, sp = mx_scale_pitch(K);
    const int n = blockIdx.x * 8 + warp;
    float acc[kDotTokens] = {};
    for (int b = lane; b < KB; b += 32) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(W + ((int64_t)n * K + b * kMxBlock) / 2);
        const float sw = mx_scale_value(Ws[n * sp + b]);
        float wf[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx_decode8<MHC_MX_E2M1>(make_uint2(w[q], 0u), 1.0f, wf[q]);
        for (int k = 0; k < kDotTokens && t0 + k < T; ++k) {
            const uint32_t* a = reinterpret_cast<const uint32_t*>(A + ((t0 + k) * K + b * kMxBlock) / 2);
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float af[8];
                mx_decode8<MHC_MX_E2M1>(make_uint2(a[q], 0u), 1.0f, af);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(af[e], wf[q][e], s);
            }
            acc[k] = fmaf(s * sw, mx_scale_value(As[(t0 + k) * sp + b]), acc[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kDotTokens; ++k) {
        const float s = warp_sum(acc[k]);
        if (lane == 0) f[k][warp] = s;
    }
    __syncthreads();
    const int k = threadIdx.x;
    if (k >= kDotTokens || t0 + k >= T) return;
    const int64_t t = t0 + k;
    const int NV = N / 8;
    if (kMix) {
        float h[16], hp[4];
        load_maps(m.H, m.hpost, t, h, hp);
        float xf[4][8];
        for (int j = 0; j < 4; ++j) unpack8(m.X[(t * 4 + j) * NV + blockIdx.x], xf[j]);
        for (int i = 0; i < 4; ++i) {
            float o[8];
            for (int e = 0; e < 8; ++e) {
                float s = hp[i] * f[k][e];
                for (int j = 0; j < 4; ++j) s = fmaf(h[4 * i + j], xf[j][e], s);
                o[e] = s;
            }
            out[(t * 4 + i) * NV + blockIdx.x] = pack8(o);
        }
    } else {
        float o[8];
        for (int e = 0; e < 8; ++e) o[e] = f[k][e];
        out[t * NV + blockIdx.x] = pack8(o);
    }
}

}  // namespace

cudaError_t launch_premap_fwd_mx4(const uint16_t* X, const float* hpre, uint8_t* codes, uint8_t* scales, int64_t T,
                                  int64_t C, cudaStream_t s)
{
    const int CV = (int)(C / 8), chunks = (CV + kReadThreads - 1) / kReadThreads;
    const int64_t items = T * chunks;
    const int grid = persistent_grid((const void*)premap_fwd_mx4_kernel, kReadThreads, 0, items);
    premap_fwd_mx4_kernel<<<grid, kReadThreads, 0, s>>>((const uint4*)X, hpre, codes, scales, items, chunks, CV);
    return cudaGetLastError();
}

cudaError_t launch_mx4_linear(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws, uint16_t* out,
                              int64_t T, int64_t N, int64_t K, cudaStream_t s)
{
    const dim3 grid((unsigned)(N / 8), (unsigned)((T + kDotTokens - 1) / kDotTokens));
    mx4_dot_kernel<false><<<grid, kDotThreads, 0, s>>>(A, As, W, Ws, MixArgs{}, (uint4*)out, T, (int)N, (int)K);
    return cudaGetLastError();
}

cudaError_t launch_mx4_linear_mix(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws,
                                  const uint16_t* X, const float* H, const float* hpost, uint16_t* Y, int64_t T,
                                  int64_t C, int64_t K, cudaStream_t s)
{
    const dim3 grid((unsigned)(C / 8), (unsigned)((T + kDotTokens - 1) / kDotTokens));
    mx4_dot_kernel<true><<<grid, kDotThreads, 0, s>>>(A, As, W, Ws, MixArgs{(const uint4*)X, H, hpost}, (uint4*)Y, T,
                                                      (int)C, (int)K);
    return cudaGetLastError();
}

}  // namespace mhc
