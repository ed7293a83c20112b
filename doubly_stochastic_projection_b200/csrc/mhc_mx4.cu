// mhc_mx4.cu -- the 4-bit serving path around the residual streams on
// sm_100a: the read map that writes the layer's input as microscaled e2m1
// codes, the product of two such matrices, and the same product with the
// residual mix as its epilogue.
//
//   read map       a[t] = codes of x_in[t,c] = sum_j sigmoid(h_pre[t,j]) X[t,j,c]
//   product        out[t,n] = sum_b sa[t,b] sw[n,b] sum_{k in b} a[t,k] w[n,k]
//   product + mix  Y[t,i,c] = sum_j H[t,i,j] X[t,j,c] + h_post[t,i] out[t,c]
#include <cuda.h>

#include <atomic>
#include <climits>

#include "birkhoff_math.cuh"
#include "launch.h"
#include "mix_common.cuh"
#include "mx_common.cuh"
#include "pdl.cuh"
#include "tc5.cuh"

namespace mhc {

namespace {

// ------------------------------------------------------------------ read map

// A CTA takes chunks of 128 vectors (1024 channels) of a token, so that a
// single token's streams are spread over several CTAs.  It finds its token by
// one division at the start and additions after it, and each lane computes one of
// the token's four sigmoids: with a division a chunk and all four in every lane
// the kernel issued in 72% of its cycles and took 49 us for 8192 tokens of
// 4 x 4096, now 42.5 to 45.5 by the GPU (286 MB, a copy's 44 us).
constexpr int kReadThreads = 128;

__global__ void __launch_bounds__(kReadThreads)
premap_fwd_mx4_kernel(const uint4* X, const float* hpre, uint8_t* codes, uint8_t* scales, int64_t T, int chunks, int CV)
{
    const int64_t sp = mx_scale_pitch((int64_t)CV * 8);
    pdl_release();  // the product waits for this kernel's end by itself
    const unsigned dt = gridDim.x / chunks, dk = gridDim.x % chunks;
    unsigned k = blockIdx.x % chunks;
    int64_t t = blockIdx.x / chunks;
    while (t < T) {
        const int v = (int)k * kReadThreads + threadIdx.x;
        const bool in = v < CV;
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = in ? __ldcs(X + (t * 4 + j) * CV + v) : make_uint4(0u, 0u, 0u, 0u);
        const float mine = sigmoidf(__ldg(hpre + 4 * t + (threadIdx.x & 3)));
        float s[4], xf[4][8], o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = __shfl_sync(0xffffffffu, mine, j);
            unpack8(x[j], xf[j]);
        }
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
            if ((v & 3) == 0) mx_store_scale(scales + t * sp + (v >> 2), v >> 2, (CV + 3) >> 2, S);
        }
        t += dt;
        k += dk;
        if (k >= (unsigned)chunks) {
            k -= chunks;
            ++t;
        }
    }
}

// ------------------------------------------------------------------- product
//
// D[n, t] = W A^T on the tensor cores' block-scaled 4-bit kind: a CTA takes a
// tile of 128 channels (the rows of tensor memory) by kTok tokens (its
// columns) and walks K in tiles of 256 elements, 128 bytes a row.  Its warps:
//   0     loads the code tiles by TMA (128-byte swizzle) into a ring of stages
//   1     issues the products, four steps of 64 a tile
//   2     issues the copies of the scales into tensor memory
//   3, 12, ...  bring the scales, one warp for each chunk of 128 rows of W or
//         A.  They are rows of bytes in memory and have to be, for the tensor
//         cores, chunks of 512 bytes with the four bytes of rows r, r + 32,
//         r + 64, r + 96 side by side: a lane reads 32 bytes (four tiles' worth)
//         of four rows, a round ahead, and stores 16-byte vectors
//   4-11  the epilogue: tensor memory -> shared memory, turned so that a
//         thread holds eight consecutive channels of a token -> the output
// Two forms.  Whole: one persistent CTA an SM walks output tiles, the sums of
// one tile in one half of tensor memory while the epilogue drains the other.
// Split: a cluster shares one output tile, each CTA a part of K; the partial
// sums meet in shared memory and are added in the order of the ranks.
// No form has operands in two CTAs.  Pairs of CTAs on one tile (256 channels,
// 28 KB a K tile and CTA instead of 40) need word, for each K tile, that the
// other's operands are there.  Given by an arrival that releases at cluster scope
// a K tile took 1400 cycles, of which the products need 384 (8192 tokens, N =
// 8192, K = 4096 229 us); given by TMA loads that count their bytes at the other
// CTA's barrier, 600 (175 us).  A commit without tensor work before it is quick,
// but nothing says that it orders what its thread has waited for.
//
// Measured (device, back to back, operands not in L2 for few tokens): 8192
// tokens, N = 8192, K = 4096 115 us, 4.8 PFLOP/s (the instruction's own rate
// would be 65 us; operands, scales and outputs share the path between L2 and the
// SMs); 200 tokens, N = 4104, K = 4096 9.3 us; one token, N = 8192, K = 7168
// 9.8 us (3.2 TB/s, latency: the launch, the first bytes of memory and the
// cluster's sum).  With the mix: 16384 tokens, C = 4096, K = 8192 322 to 333 us by
// the GPU; 280 without the loads of the streams, 291 without the stores of Y, 256
// without both.  An SM has the loads of 32 tokens in flight, between two barriers
// of the epilogue, so their latency shows.
//
// Every wait at an mbarrier is bounded, by the device's clock (tc5.cuh).  One that
// runs out, as it does when a role of the CTA fails or the process is switched out
// for the whole limit, sets mx4_wait_expired, makes the other roles give up too,
// and leaves NaN in the outputs that are not done.  Not bounded are what all
// CTAs of a launch come to: the end of the grid before this one, tensor memory
// (held by no other CTA of this kernel on the SM) and the barriers of a cluster.

constexpr int kChan = 128;      // channels of a tile
constexpr int kRowBytes = 128;  // of K of a tile: 256 elements
constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;

constexpr uint64_t kDrainNs = 100000000;  // for all that is in flight, once a wait has run out

__device__ int mx4_wait_expired;

struct ProductArgs {
    const uint8_t *As, *Ws;
    uint4* out;      // [T][N] bf16, or Y [T][4][N]
    const uint4* X;  // the mix's: [T][4][N] bf16, [T][4][4], [T][4]
    const float *H, *hpost;
    int64_t T;
    int N, K;
    int chan_tiles, tok_tiles;
    uint64_t wait_ns;  // kDiag: limit of a wait
    int idle;          // kDiag: enum mhc_mx4_role
};

template <int kTok_, int kStages_, bool kSplit_>
struct ProductShape {
    static constexpr int kTok = kTok_, kStages = kStages_;
    static constexpr bool kSplit = kSplit_;
    static constexpr int kTokChunks = (kTok + 127) / 128;  // 128-row chunks of A's scales
    static constexpr int kThreads = 32 * (12 + kTokChunks);  // four warps a scheduler: 128 registers at most
    static constexpr int kWBytes = kChan * kRowBytes, kABytes = kTok * kRowBytes;
    static constexpr int kStageBytes = kWBytes + kABytes;
    // scales: two buffers of kBufTiles K tiles, each tile two steps of 128
    // elements, a step's being one chunk of W's and kTokChunks of A's
    static constexpr int kBufTiles = 4, kBufSteps = 2 * kBufTiles;
    static constexpr int kScaleStep = 512 * (1 + kTokChunks), kScaleBytes = 2 * kBufSteps * kScaleStep;
    static constexpr int kSums = kSplit ? 1 : 2;  // accumulator tiles
    // the epilogue's: two buffers of 32 tokens, or the whole tile's partial sums
    static constexpr int kGroup = 32;
    static constexpr int kEpiBytes = (kSplit ? kTok : 2 * kGroup) * kChan * 4;
    static constexpr int kBars = 2 * kStages + 4 + 2 * kSums + 1;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kScaleBytes + kEpiBytes + 8 * kBars + 16;
    // columns of tensor memory: sums, then each stage's scales of W and A
    static constexpr int kScaleCols = 8 * (1 + kTokChunks);
    static constexpr int kSumCols = (kSums * kTok + 31) / 32 * 32;
    static constexpr int kColumns = 512;
    static_assert(kSumCols + kStages * kScaleCols <= kColumns, "tensor memory");
    static_assert(kABytes % 1024 == 0 && kStageBytes % 1024 == 0, "the swizzle repeats every 1024 bytes");
    // one CTA an SM: two that hold tensor memory and wait for cluster mates
    // could otherwise wait for each other
    static_assert(kSmemBytes > 116 * 1024 && kSmemBytes <= 227 * 1024, "shared memory");
};

// The scales of 512 elements of one row, and of the next 512 if `two`: 16 bytes
// each, in as few loads as the rows' alignment (32, 16 or 4 bytes) allows,
// since every lane reads another row and each load costs a pass over 32 cache
// lines (which the 32-byte form, done with its sector, does not keep).  Words past
// the row read as zero.  Volatile, so that the loads stay where they are issued, a
// round ahead of their use.  Not the non-coherent form, here and for the mix's
// maps: this kernel may start while the one that writes them still runs.
__device__ __forceinline__ void fetch_scales(const uint8_t* row, int pair, bool two, int pitch, int align, uint4& q0,
                                             uint4& q1)
{
    const uint8_t* at = row + 16 * pair;
    if (align == 32 && two) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(q0.x), "=r"(q0.y), "=r"(q0.z), "=r"(q0.w), "=r"(q1.x), "=r"(q1.y), "=r"(q1.z), "=r"(q1.w)
                     : "l"(at));
    } else if (align >= 16) {
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q0.x), "=r"(q0.y), "=r"(q0.z), "=r"(q0.w)
                     : "l"(at));
        if (two)
            asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q1.x), "=r"(q1.y), "=r"(q1.z), "=r"(q1.w)
                         : "l"(at + 16));
    } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 0u;
            if (16 * pair + 4 * j < pitch && (j < 4 || two))
                asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[j]) : "l"(at + 4 * j));
        }
        q0 = make_uint4(w[0], w[1], w[2], w[3]);
        q1 = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Word w of a row's scales without the bytes past its KB blocks: what lies
// there meets code zeros, which a NaN scale would turn into NaN.
__device__ __forceinline__ uint32_t scales_within(uint32_t word, int w, int KB)
{
    const int left = KB - 4 * w;
    return left >= 4 ? word : left <= 0 ? 0u : word & (0xffffffffu >> (8 * (4 - left)));
}

// Two floats in one register pair.  The mix's 160 multiply-adds for a token and
// vector, two channels an instruction: each rounds as fmaf does, and timed in turn
// 16384 x 4096 x 8192 takes 333 us instead of 341, 1000 tokens 40 instead of 42.
__device__ __forceinline__ uint64_t two(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// What the output of eight channels of a token (vector v of N / 8) takes beside
// the product: nothing, or the mix's streams and maps, loaded ahead.
template <bool kMix>
struct StreamVec {
    __device__ __forceinline__ void load(const ProductArgs&, int64_t, int) {}
    __device__ __forceinline__ void emit(const ProductArgs& p, const float (&f)[8], int64_t t, int v) const
    {
        p.out[t * (p.N >> 3) + v] = pack8(f);
    }
};
template <>
struct StreamVec<true> {
    uint4 x[4];
    float h[16], hp[4];
    __device__ __forceinline__ void load(const ProductArgs& p, int64_t t, int v)
    {
        const int NV = p.N >> 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __ldcs(p.X + (t * 4 + j) * NV + v);
        const float4* H = reinterpret_cast<const float4*>(p.H) + 4 * t;
        float4 q[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) q[i] = i < 4 ? H[i] : reinterpret_cast<const float4*>(p.hpost)[t];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            float* to = i < 4 ? h + 4 * i : hp;
            to[0] = q[i].x;
            to[1] = q[i].y;
            to[2] = q[i].z;
            to[3] = q[i].w;
        }
    }
    __device__ __forceinline__ void emit(const ProductArgs& p, const float (&f)[8], int64_t t, int v) const
    {
        const int NV = p.N >> 3;
        uint64_t xf[4][4], ff[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) xf[j][e] = two(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) ff[e] = two(f[2 * e], f[2 * e + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float o[8];
            const uint64_t hh[5] = {two(hp[i], hp[i]), two(h[4 * i], h[4 * i]), two(h[4 * i + 1], h[4 * i + 1]),
                                    two(h[4 * i + 2], h[4 * i + 2]), two(h[4 * i + 3], h[4 * i + 3])};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint64_t s = mul2(hh[0], ff[e]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s = fma2(hh[1 + j], xf[j][e], s);
                asm("mov.b64 {%0, %1}, %2;" : "=f"(o[2 * e]), "=f"(o[2 * e + 1]) : "l"(s));
            }
            __stcs(p.out + (t * 4 + i) * NV + v, pack8(o));
        }
    }
};

// kDiag (a kernel of its own, as the mask costs each product 0.2 to 0.4 us): with a
// limit of the caller's for the waits, and roles that do nothing.
template <class S, bool kMix, bool kDiag>
__global__ void __launch_bounds__(S::kThreads, 1)
mx4_product_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapA,
                   const ProductArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    constexpr int kTok = S::kTok, kStages = S::kStages;
    const uint32_t base = (tc5::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - tc5::smem_addr(smem_raw));
    constexpr int kOffScales = kStages * S::kStageBytes, kOffEpi = kOffScales + S::kScaleBytes,
                  kOffBars = kOffEpi + S::kEpiBytes;
    float* epi = reinterpret_cast<float*>(smem + kOffEpi);
    const uint32_t bars = base + kOffBars;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBars + 8 * S::kBars);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const auto full = [&](int s) { return bars + 8 * s; };
    const auto empty = [&](int s) { return bars + 8 * (kStages + s); };
    const auto scales_full = [&](int b) { return bars + 8 * (2 * kStages + b); };
    const auto scales_empty = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };
    const auto sum_full = [&](int a) { return bars + 8 * (2 * kStages + 4 + a); };
    const auto sum_empty = [&](int a) { return bars + 8 * (2 * kStages + 4 + S::kSums + a); };
    const uint32_t drained = bars + 8 * (2 * kStages + 4 + 2 * S::kSums);  // used when a wait has run out
    constexpr int kOffA = S::kWBytes;  // within a stage

    // shuffled, and voted on where waits decide: uniform for the compiler too.  The
    // operands of the tensor instructions then stay in uniform registers, and the
    // four steps of a K tile issue in about 220 cycles instead of 280.
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        tc5::prefetch_map(&mapW);
        tc5::prefetch_map(&mapA);
        for (int s = 0; s < kStages; ++s) {
            tc5::mbar_init(full(s), 2);  // the codes by TMA, the scales by tensor copy
            tc5::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc5::mbar_init(scales_full(b), 1 + S::kTokChunks);  // the scale warps
            tc5::mbar_init(scales_empty(b), 1);
        }
        for (int a = 0; a < S::kSums; ++a) {
            tc5::mbar_init(sum_full(a), 1);
            tc5::mbar_init(sum_empty(a), kEpiWarps);
        }
        tc5::mbar_init(drained, 2);
        *abort = 0;
        tc5::fence_mbar_init();
    }
    if (warp == 1) tc5::tmem_alloc<S::kColumns>(tc5::smem_addr(tmem_slot));
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();

    // this CTA's output tiles, and its share of K in pairs of tiles
    const int ranks = S::kSplit ? (int)tc5::cluster_size() : 1, rank = S::kSplit ? (int)tc5::cluster_rank() : 0;
    const int pairs = (p.K + 511) / 512;  // 16 bytes of scales
    const int pair0 = pairs * rank / ranks, pair1 = pairs * (rank + 1) / ranks;
    const int k0 = 2 * pair0, k1 = min(2 * pair1, (p.K + 255) / 256);
    const int first = blockIdx.x / ranks, stride = gridDim.x / ranks;
    const uint64_t wait_ns = kDiag ? p.wait_ns : (uint64_t)kProductWaitNs;
    int tiles = p.chan_tiles * p.tok_tiles;
    if (kDiag) {
        const int role = warp == 0 ? MHC_MX4_LOADS : warp == 1 ? MHC_MX4_PRODUCTS : warp == 2 ? MHC_MX4_COPIES
                         : warp == 3 || warp >= 12                                            ? MHC_MX4_SCALES
                                                                                              : 0;
        if ((p.idle & role) != 0) tiles = 0;
    }
    bool ok = true;

    const int mine = first < tiles ? (tiles - 1 - first) / stride + 1 : 0, steps = k1 - k0;  // output tiles, K tiles
    int64_t loads = 0;  // warp 0's, so far
    if (warp == 0) {
        int s = 0, t = first;
        uint32_t phase = 0;
        for (int n = 0; n < mine && ok; ++n, t += stride) {
            const int n0 = t % p.chan_tiles * kChan, t0 = t / p.chan_tiles * kTok;
            for (int k = k0; k < k1; ++k, ++loads) {
                if (!(ok = tc5::mbar_wait_warp(empty(s), phase ^ 1, abort, wait_ns))) break;
                const uint32_t at = base + s * S::kStageBytes;
                if (tc5::elect_one()) {
                    tc5::mbar_expect_tx(full(s), S::kWBytes + S::kABytes);
                    tc5::tma_load_2d(at, &mapW, k * kRowBytes, n0, full(s));
                    tc5::tma_load_2d(at + kOffA, &mapA, k * kRowBytes, t0, full(s));
                }
                __syncwarp();
                s = s + 1 == kStages ? 0 : s + 1;
                phase ^= s == 0;
            }
        }
    } else if (warp == 2) {
        // each K tile's scales from shared into tensor memory, ahead of the products
        int s = 0, buf = 0;
        uint32_t phase = 0, par = 0;
        for (int n = 0; n < mine && ok; ++n) {
            for (int k = 0; k < steps; ++k) {
                const int j = k & (S::kBufTiles - 1);  // in this buffer
                if (j == 0 && !(ok = tc5::mbar_wait_warp(scales_full(buf), par, abort, wait_ns))) break;
                if (!(ok = tc5::mbar_wait_warp(empty(s), phase ^ 1, abort, wait_ns))) break;
                tc5::fence_after_sync();
                const uint32_t at = base + kOffScales + (buf * S::kBufSteps + 2 * j) * S::kScaleStep;
                const uint32_t sw = tmem + S::kSumCols + s * S::kScaleCols;
                const bool last = j + 1 == S::kBufTiles || k + 1 == steps;
                if (tc5::elect_one()) {
#pragma unroll
                    for (int c = 0; c < 2 * (1 + S::kTokChunks); ++c)
                        tc5::copy_scales(sw + 4 * c, tc5::scale_desc(at + 512 * c));
                    tc5::commit(full(s));
                    if (last) tc5::commit(scales_empty(buf));
                }
                __syncwarp();
                s = s + 1 == kStages ? 0 : s + 1;
                phase ^= s == 0;
                buf ^= last;
                par ^= last && buf == 0;
            }
        }
    } else if (warp == 1) {
        // The whole warp waits, one lane issues.  The queue behind it is short
        // (a delay of some 150 cycles between two K tiles is hidden, one of 250 is
        // not), so nothing else is done here.
        constexpr uint32_t inst = tc5::mx4_instruction(kChan, kTok);
        int s = 0;
        uint32_t phase = 0;
        if (mine > 0) ok = tc5::mbar_wait_warp(full(0), 0, abort, wait_ns);
        for (int n = 0; n < mine && ok; ++n) {
            const int a = n % S::kSums;
            if (!(ok = tc5::mbar_wait_warp(sum_empty(a), (n / S::kSums & 1) ^ 1, abort, wait_ns))) break;
            const uint32_t d = tmem + a * kTok;
            for (int k = 0; k < steps; ++k) {
                tc5::fence_after_sync();
                const uint32_t at = base + s * S::kStageBytes;
                const uint32_t sc = tmem + S::kSumCols + s * S::kScaleCols;
                const uint64_t dw = tc5::operand_desc(at), da = tc5::operand_desc(at + kOffA);
                const int here = s;
                s = s + 1 == kStages ? 0 : s + 1;
                phase ^= s == 0;
                // 64 elements a step, 32 bytes along the swizzled row
                const auto step = [&](int q) {
                    const uint32_t sw = sc + 4 * (1 + S::kTokChunks) * (q >> 1);
                    tc5::mma_mx4(d, dw + 2 * q, da + 2 * q, inst | tc5::scale_select(2 * (q & 1)), sw, sw + 4,
                                 k > 0 || q > 0);
                };
                if (tc5::elect_one()) {
                    step(0);
                    step(1);
                    step(2);
                }
                __syncwarp();
                // the next K tile's wait, while the queue holds steps of this one
                if (k + 1 < steps || n + 1 < mine) ok = tc5::mbar_wait_warp(full(s), phase, abort, wait_ns);
                if (tc5::elect_one()) {
                    step(3);
                    tc5::commit(empty(here));
                    if (k + 1 == steps) tc5::commit(sum_full(a));
                }
                __syncwarp();
                if (!ok) break;
            }
        }
    } else if (warp == 3 || warp >= 12) {
        // warp 3: W's rows, the others: 128 of A's each; lane l holds rows l, l + 32,
        // l + 64 and l + 96 of the chunk
        const bool isW = warp == 3;
        const int chunk = isW ? 0 : warp - 11, in_tile = isW ? 0 : 128 * (warp - 12);
        const uint8_t* src = isW ? p.Ws : p.As;
        const int KB = p.K / kMxBlock, pitch = (int)mx_scale_pitch(p.K);
        // of every pair of 512 elements that is fetched together
        const int align = (pitch & 31) == 0 && (reinterpret_cast<uintptr_t>(src) & 31) == 0 && (pair0 & 1) == 0 ? 32
                          : (pitch & 15) == 0                                                                ? 16
                                                                                                             : 4;
        const int64_t rows = isW ? (int64_t)p.N : p.T;
        // the round in work, of four K tiles (two pairs), and the next on its way
        uint4 cur[2][4], next[2][4];
        const auto fetch = [&](int tile, int pair) {
            if (tile >= tiles) return;
            const int64_t r0 =
                isW ? (int64_t)(tile % p.chan_tiles) * kChan : (int64_t)(tile / p.chan_tiles) * kTok + in_tile;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                // rows past the end, or past the tile, stand in for none: what they
                // give is not written
                const uint8_t* row = src + min(r0 + 32 * g + lane, rows - 1) * pitch;
                fetch_scales(row, pair, pair + 1 < pair1, pitch, align, next[0][g], next[1][g]);
            }
        };
        int buf = 0;
        uint32_t par = 0;
        fetch(first, pair0);
        for (int tile = first; tile < tiles && ok; tile += stride) {
            for (int pair = pair0; pair < pair1 && ok; pair += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int g = 0; g < 4; ++g) cur[u][g] = next[u][g];
                if (pair + 2 < pair1)
                    fetch(tile, pair + 2);
                else
                    fetch(tile + stride, pair0);
                if (!(ok = tc5::mbar_wait_warp(scales_empty(buf), par ^ 1, abort, wait_ns))) break;
#pragma unroll
                for (int j = 0; j < S::kBufSteps; ++j) {  // steps of 128 elements, one word of scales a row
                    const int w0 = 4 * pair + j;
                    if (pair + j / 4 >= pair1) break;
                    uint32_t w[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 q = cur[j >> 2][g];
                        w[g] = (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
                        if (4 * (w0 + 1) > KB) w[g] = scales_within(w[g], w0, KB);
                    }
                    uint8_t* at = smem + kOffScales + (buf * S::kBufSteps + j) * S::kScaleStep + 512 * chunk;
                    reinterpret_cast<uint4*>(at)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                tc5::fence_async_shared();
                __syncwarp();
                if (lane == 0) tc5::mbar_arrive(scales_full(buf));
                buf ^= 1;
                par ^= buf == 0;
            }
        }
    } else {
        const int e = threadIdx.x - 128;  // 0..255
        const int quarter = warp & 3, half = (warp - 4) >> 2;  // lanes of tensor memory that a warp may read
        const uint32_t row = (uint32_t)(32 * quarter) << 16;
        // sums that may still be in work, as a wait has run out, are not read
        const auto load_sums = [&](int a, int g, float(&v)[16]) {
            if (ok) {
                tc5::tmem_load(tmem + row + a * kTok + g, v);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __int_as_float(0x7fffffff);
            }
        };
        int n = 0;
        for (int tile = first; tile < tiles; tile += stride, ++n) {
            const int a = n % S::kSums;
            const int v0 = tile % p.chan_tiles * (kChan / 8);
            const int64_t t0 = (int64_t)(tile / p.chan_tiles) * kTok;
            if (ok) ok = tc5::mbar_wait_warp(sum_full(a), n / S::kSums & 1, abort, wait_ns);
            tc5::fence_after_sync();
            if (S::kSplit) {
                // each token in its place, for the cluster to add up
#pragma unroll 1
                for (int g = 16 * half; g < kTok; g += 32) {
                    float v[16];
                    load_sums(a, g, v);
                    float* to = epi + g * kChan + 32 * quarter + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * kChan] = v[i];
                }
            } else {
#pragma unroll 1
                for (int g = 0; g < kTok; g += S::kGroup) {
                    // this thread's eight channels of two tokens of the group
                    const int vec = v0 + (e & 15);
                    StreamVec<kMix> x[2];
                    bool in[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int64_t t = t0 + g + (e >> 4) + 16 * i;
                        in[i] = t < p.T && 8 * vec < p.N;
                        if (in[i]) x[i].load(p, t, vec);
                    }
                    float v[16];
                    load_sums(a, g + 16 * half, v);
                    if (g + S::kGroup >= kTok) {  // the last read of this tile's sums
                        tc5::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc5::mbar_arrive(sum_empty(a));
                    }
                    // two buffers in turn: by the barrier of the next group, all have read this one
                    float* buf = epi + (g & S::kGroup) * kChan;
                    float* to = buf + 16 * half * kChan + 32 * quarter + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * kChan] = v[i];
                    asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!in[i]) continue;
                        const float4* q = reinterpret_cast<const float4*>(buf + ((e >> 4) + 16 * i) * kChan) + 2 * (e & 15);
                        const float4 lo = q[0], hi = q[1];
                        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        x[i].emit(p, f, t0 + g + (e >> 4) + 16 * i, vec);
                    }
                }
            }
        }
    }
    if (!ok) {
        *abort = 1;
        mx4_wait_expired = 1;
    }
    __syncwarp();

    if (S::kSplit) {
        // one tile a cluster: this CTA adds up its share of the tile's vectors
        tc5::cluster_sync();
        const int v0 = first % p.chan_tiles * (kChan / 8);
        const int64_t t0 = (int64_t)(first / p.chan_tiles) * kTok;
        constexpr int kItems = kTok * (kChan / 8);
        for (int i = rank * S::kThreads + threadIdx.x; i < kItems; i += ranks * S::kThreads) {
            const int tok = i >> 4, v = i & 15;
            if (t0 + tok < p.T && 8 * (v0 + v) < p.N) {
                StreamVec<kMix> x;
                x.load(p, t0 + tok, v0 + v);
                float f[8] = {};
                for (int r = 0; r < ranks; ++r) {
                    const uint32_t at = tc5::map_rank(tc5::smem_addr(epi + tok * kChan + 8 * v), r);
                    const float4 lo = tc5::load_cluster(at), hi = tc5::load_cluster(at + 16);
                    const float q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] += q[x];
                }
                x.emit(p, f, t0 + tok, v0 + v);
            }
        }
        tc5::cluster_sync();  // nobody's shared memory goes while it may be read
    }
    tc5::fence_before_sync();
    __syncthreads();
    if (*abort != 0) {
        // A wait of some role has run out, so nothing says that the others' work is
        // done, not even where they had no wait left: before its shared and tensor
        // memory go, the copies in flight (the last kStages at most) and the tensor
        // work are waited for
        const uint64_t t0 = tc5::global_ns();
        const auto left = [&] { return kDrainNs - min(kDrainNs, tc5::global_ns() - t0); };
        if (warp == 0) {
            for (int64_t j = loads > kStages ? loads - kStages : 0; j < loads; ++j)
                tc5::mbar_wait(full((int)(j % kStages)), (uint32_t)(j / kStages) & 1, nullptr, left());
        } else if (warp <= 2) {
            if (tc5::elect_one()) tc5::commit(drained);
            __syncwarp();
            tc5::mbar_wait(drained, 0, nullptr, left());
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc5::fence_after_sync();
        tc5::tmem_free<S::kColumns>(tmem);
    }
}

}  // namespace

cudaError_t launch_premap_fwd_mx4(const uint16_t* X, const float* hpre, uint8_t* codes, uint8_t* scales, int64_t T,
                                  int64_t C, cudaStream_t s)
{
    const int CV = (int)(C / 8), chunks = (CV + kReadThreads - 1) / kReadThreads;
    const int64_t items = T * chunks;
    const int grid = persistent_grid((const void*)premap_fwd_mx4_kernel, kReadThreads, 0, items);
    premap_fwd_mx4_kernel<<<grid, kReadThreads, 0, s>>>((const uint4*)X, hpre, codes, scales, T, chunks, CV);
    return cudaGetLastError();
}

namespace {

// A byte matrix [rows][pitch] read in boxes of box_rows x 128 bytes.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static std::atomic<void*> kept{nullptr};  // the driver's function; the same for every device
    void* f = kept.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        kept.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

bool code_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box_rows)
{
    const EncodeTiled f = encode_tiled();
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {kRowBytes, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return f != nullptr && f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
                             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S, bool kMix, bool kDiag>
cudaError_t product(const uint8_t* A, const uint8_t* W, ProductArgs p, cudaStream_t s)
{
    const auto kernel = mx4_product_kernel<S, kMix, kDiag>;
    static std::atomic<uint64_t> allowed{0};  // devices whose shared-memory limit is set for this kernel
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(allowed.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    p.chan_tiles = (p.N + kChan - 1) / kChan;
    p.tok_tiles = (int)((p.T + S::kTok - 1) / S::kTok);
    const int64_t tiles = (int64_t)p.chan_tiles * p.tok_tiles;
    if (tiles > INT32_MAX / 8) return cudaErrorInvalidValue;
    CUtensorMap mapW, mapA;
    if (!code_map(&mapW, W, p.N, p.K, kChan) || !code_map(&mapA, A, p.T, p.K, S::kTok)) return cudaErrorInvalidValue;

    const int sms = device_sm_count(), pairs = (p.K + 511) / 512;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S::kSplit ? 2 : 1;
    const auto set_ranks = [&](int ranks) {
        cfg.gridDim = dim3((unsigned)(S::kSplit ? tiles * ranks : tiles < sms ? tiles : sms));
        attr[1].val.clusterDim.x = (unsigned)ranks;
    };
    int ranks = 1;
    if (S::kSplit) {
        // CTAs that share a tile: as many as have work, up to 8, while all tiles'
        // clusters fit the GPU at once.  Its SMs do not say how many do: a cluster
        // lies within one GPC (of the B200's 148 SMs, 45 clusters of 3 find room, 26
        // of 5, 15 of 8), so the runtime is asked, once for a size.  With two waves
        // of clusters one token, N = 2048, K = 4096 takes 9.1 us in clusters of 8,
        // in one wave 5.6 in clusters of 6; N = 6144 11.5 in 3 and 6.9 in 2.
        static std::atomic<int> at_once[64][9];  // clusters of that size and one more; 0: not asked
        for (int r = (int)(pairs < 8 ? pairs : 8); r > 1; --r) {
            if (r * tiles > sms) continue;
            set_ranks(r);
            int n = dev < 64 ? at_once[dev][r].load(std::memory_order_relaxed) : 0;
            if (n == 0) {
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                    cudaGetLastError();
                    n = 0;
                }
                ++n;
                if (dev < 64) at_once[dev][r].store(n, std::memory_order_relaxed);
            }
            if (n - 1 >= tiles) {
                ranks = r;
                break;
            }
        }
    }
    set_ranks(ranks);
    return cudaLaunchKernelEx(&cfg, kernel, mapW, mapA, p);
}

using Split16 = ProductShape<16, 9, true>;
using Split64 = ProductShape<64, 6, true>;
// Four stages of 40 KB; with three the products wait for their operands: 115 us
// against 140 at 8192 x 8192 x 4096, with the mix 325 against 388 at 16384 x
// 4096 x 8192, though its loads of the streams have the least L1 beside four.
using Whole192 = ProductShape<192, 4, false>;

// The form by size.  Split forms run one wave, in clusters of as many CTAs as
// that leaves room for, so they are taken while their tiles fit the GPU at once,
// and the narrowest that holds the tokens: at N = 8192, K = 4096 one token takes 7.9 us in tiles of 16 and
// 9.2 in tiles of 64; 200 tokens take 17.6 us in tiles of 64 (256 tiles, two
// waves) and 11.5 whole.  Past one wave the whole form is taken whatever the
// tokens.  For one token and N = 36864 it is the faster one with K = 1024 (10.9 us,
// 11.5 in waves of tiles of 16) but not with K = 4096 (36 and 21) or 7168 (51 and
// 30); from N = 18952 on, that is left.
template <bool kMix, bool kDiag = false>
cudaError_t product_by_size(const uint8_t* A, const uint8_t* W, const ProductArgs& p, cudaStream_t s)
{
    const int64_t chan_tiles = (p.N + kChan - 1) / kChan, sms = device_sm_count();
    if (p.T <= 16 && chan_tiles <= sms) return product<Split16, kMix, kDiag>(A, W, p, s);
    if (chan_tiles * ((p.T + 63) / 64) <= sms) return product<Split64, kMix, kDiag>(A, W, p, s);
    return product<Whole192, kMix, kDiag>(A, W, p, s);
}

}  // namespace

cudaError_t launch_mx4_linear(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws, uint16_t* out,
                              int64_t T, int64_t N, int64_t K, cudaStream_t s)
{
    return product_by_size<false>(
        A, W, ProductArgs{As, Ws, (uint4*)out, nullptr, nullptr, nullptr, T, (int)N, (int)K, 0, 0, 0, 0}, s);
}

cudaError_t launch_mx4_linear_diag(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws,
                                   uint16_t* out, int64_t T, int64_t N, int64_t K, int64_t wait_ns, int idle,
                                   cudaStream_t s)
{
    return product_by_size<false, true>(A, W,
                                        ProductArgs{As, Ws, (uint4*)out, nullptr, nullptr, nullptr, T, (int)N, (int)K,
                                                    0, 0, (uint64_t)wait_ns, idle},
                                        s);
}

cudaError_t launch_mx4_linear_mix(const uint8_t* A, const uint8_t* As, const uint8_t* W, const uint8_t* Ws,
                                  const uint16_t* X, const float* H, const float* hpost, uint16_t* Y, int64_t T,
                                  int64_t C, int64_t K, cudaStream_t s)
{
    return product_by_size<true>(
        A, W, ProductArgs{As, Ws, (uint4*)Y, (const uint4*)X, H, hpost, T, (int)C, (int)K, 0, 0, 0, 0}, s);
}

// The status of the bounded waits since the last call (synchronises the device).
cudaError_t read_wait_status(bool* expired)
{
    int v = 0;
    const int zero = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, mx4_wait_expired, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(mx4_wait_expired, &zero, sizeof zero);
    *expired = v != 0;
    return e;
}

}  // namespace mhc
