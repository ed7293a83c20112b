// mhc_ckpt.cu -- 8-bit checkpoints of the residual streams on sm_100a: packing
// and restoring microscaled rows, the mix forward that writes the checkpoint
// of X and F in the pass that reads them, and the backward kernels that read
// the checkpoint instead of X and F.
//
// The mix's backward needs X and F only for dH_res and dh_post (and dh_pre).
// Kept in bf16 they are 10 C bytes a token between forward and backward, four
// times what a one-stream residual saves; as blocks of 32 channels with 8-bit
// elements (mx_common.cuh) they are 5.16 C.  Y, dX and dF do not depend on the
// checkpoint and equal those of the bf16 path; dH_res, dh_post and dh_pre are
// the gradients at the restored streams.
//
// All are HBM-bound streaming kernels in the layout of mhc_mix.cu: one CTA
// owns a token, a thread moves vectors of 8 channels, 16 bytes of bf16 or 8
// of codes.  Four neighbouring lanes hold a block, so its largest magnitude
// takes two shuffles.  Bytes a token: forward 10 C read, 13.16 C written;
// backward 13.16 C read, 10 C written (28 C in bf16); split backward
// 11.03 C + 22.13 C (38 C in bf16).
#include "birkhoff_math.cuh"
#include "launch.h"
#include "mix_common.cuh"
#include "mx_common.cuh"
#include "pdl.cuh"

namespace mhc {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kFusedTok = 4;  // tokens projected together per CTA round

// ------------------------------------------------------------ pack, restore

// All rows' blocks in one sequence: two lanes hold a block, 16 channels each, a
// CTA 128 blocks side by side, whatever the row length, and a thread goes on
// by the whole grid's stride.  It keeps kPackAhead pieces in flight, and finds
// its row by one division at the start and additions after it.  With 8
// channels a lane the pack was bound by its instructions (118 for 32 vectors,
// 69% of the issue slots, at 78% of the copy bandwidth).
constexpr int kPackThreads = 256;
constexpr int kPackBlocks = kPackThreads / 2;
constexpr int kPackAhead = 2;

struct BlockWalk {
    int64_t r, R, dr;            // row, rows, rows a stride
    int64_t vec, dvec, sc, dsc;  // vector of 8 channels, scale byte: places from the first row's start
    int k, NB, dk;               // block in its row, blocks of a row, blocks a stride
    int vec_wrap, sc_wrap;       // from past a row's last block to the next row's first
    int last;                    // this lane's vectors in a row's last block: 2, 1 or none

    __device__ __forceinline__ BlockWalk(int64_t rows, int CV) : R(rows), NB((CV + 3) >> 2)
    {
        const int64_t first = (int64_t)blockIdx.x * kPackBlocks + (threadIdx.x >> 1);
        const int64_t stride = (int64_t)gridDim.x * kPackBlocks;
        const int sp = (int)mx_scale_pitch((int64_t)CV * 8), off = 2 * (threadIdx.x & 1);
        r = first / NB;
        k = (int)(first - r * NB);
        dr = stride / NB;
        dk = (int)(stride - dr * NB);
        vec = r * CV + 4 * k + off;
        dvec = dr * CV + 4 * dk;
        sc = r * sp + k;
        dsc = dr * sp + dk;
        vec_wrap = CV - 4 * NB;
        sc_wrap = sp - NB;
        last = CV - 4 * (NB - 1) - off;
    }
    __device__ __forceinline__ bool done() const { return r >= R; }
    // vectors that this lane has of the block: 2, 1, or 0 and less
    __device__ __forceinline__ int count() const { return r >= R ? 0 : k < NB - 1 ? 2 : last; }
    __device__ __forceinline__ void next()
    {
        r += dr;
        k += dk;
        vec += dvec;
        sc += dsc;
        if (k >= NB) {
            k -= NB;
            ++r;
            vec += vec_wrap;
            sc += sc_wrap;
        }
    }
};

// Two vectors of 8 channels side by side.  kWide (rows of a multiple of 16
// channels, x on a 32-byte boundary): 32 bytes of bf16, or 16 of 8-bit codes,
// in one access; else vector by vector, of which `n` exist.  Pack of int8 at
// 16384 x 8192: 64 us wide, 68 not; its restore 69 and 78.
template <bool kWide>
__device__ __forceinline__ void load_two(const uint4* p, int n, uint4 (&q)[2])
{
    q[0] = q[1] = make_uint4(0u, 0u, 0u, 0u);
    if (n <= 0) return;
    if constexpr (kWide) {
        asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x), "=r"(q[1].y),
                       "=r"(q[1].z), "=r"(q[1].w)
                     : "l"(p));
    } else {
        q[0] = __ldcs(p);
        if (n > 1) q[1] = __ldcs(p + 1);
    }
}
template <bool kWide>
__device__ __forceinline__ void store_two(uint4* p, int n, const uint4 (&q)[2])
{
    if constexpr (kWide) {
        asm volatile("st.global.cs.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(q[0].x), "r"(q[0].y),
                     "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y), "r"(q[1].z), "r"(q[1].w), "l"(p)
                     : "memory");
    } else {
        __stcs(p, q[0]);
        if (n > 1) __stcs(p + 1, q[1]);
    }
}

template <int kFmt>
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t vec, const uint2 w)
{
    if (kFmt == MHC_MX_E2M1)
        __stcs(reinterpret_cast<uint32_t*>(codes) + vec, w.x);
    else
        __stcs(reinterpret_cast<uint2*>(codes) + vec, w);
}

template <int kFmt>
__device__ __forceinline__ uint2 load_codes(const uint8_t* codes, int64_t vec)
{
    if (kFmt == MHC_MX_E2M1) return make_uint2(__ldcs(reinterpret_cast<const uint32_t*>(codes) + vec), 0u);
    return __ldcs(reinterpret_cast<const uint2*>(codes) + vec);
}

template <int kFmt, bool kWide>
__device__ __forceinline__ void store_two_codes(uint8_t* codes, int64_t vec, int n, const uint2 (&w)[2])
{
    if (!kWide) {
        store_codes<kFmt>(codes, vec, w[0]);
        if (n > 1) store_codes<kFmt>(codes, vec + 1, w[1]);
    } else if (kFmt == MHC_MX_E2M1) {
        __stcs(reinterpret_cast<uint2*>(codes + 4 * vec), make_uint2(w[0].x, w[1].x));
    } else {
        __stcs(reinterpret_cast<uint4*>(codes + 8 * vec), make_uint4(w[0].x, w[0].y, w[1].x, w[1].y));
    }
}
template <int kFmt, bool kWide>
__device__ __forceinline__ void load_two_codes(const uint8_t* codes, int64_t vec, int n, uint2 (&w)[2])
{
    w[0] = w[1] = make_uint2(0u, 0u);
    if (n <= 0) return;
    if (!kWide) {
        w[0] = load_codes<kFmt>(codes, vec);
        if (n > 1) w[1] = load_codes<kFmt>(codes, vec + 1);
    } else if (kFmt == MHC_MX_E2M1) {
        const uint2 q = __ldcs(reinterpret_cast<const uint2*>(codes + 4 * vec));
        w[0].x = q.x, w[1].x = q.y;
    } else {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(codes + 8 * vec));
        w[0] = make_uint2(q.x, q.y), w[1] = make_uint2(q.z, q.w);
    }
}

template <int kFmt, bool kWide>
__global__ void __launch_bounds__(kPackThreads)
mx_pack_kernel(const uint4* x, uint8_t* codes, uint8_t* scales, int64_t R, int CV)
{
    if (kFmt == MHC_MX_E2M1) pdl_release();  // the product's operand
    BlockWalk w(R, CV);
    // a warp goes on while any of its lanes has blocks: all take part in the shuffles
    while (__any_sync(0xffffffffu, !w.done())) {
        uint4 q[kPackAhead][2];
        BlockWalk at = w;
#pragma unroll
        for (int u = 0; u < kPackAhead; ++u) {
            load_two<kWide>(x + w.vec, w.count(), q[u]);
            w.next();
        }
#pragma unroll
        for (int u = 0; u < kPackAhead; ++u) {
            const uint32_t m = max(mx_amax8(q[u][0]), mx_amax8(q[u][1]));
            const int S = mx_scale_byte<kFmt>(max(m, __shfl_xor_sync(0xffffffffu, m, 1)));
            const int n = at.count();
            if (n > 0) {
                uint2 c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f[8];
                    unpack8(q[u][i], f);
                    c[i] = mx_encode8<kFmt>(f, S);
                }
                store_two_codes<kFmt, kWide>(codes, at.vec, n, c);
                if ((threadIdx.x & 1) == 0) mx_store_scale(scales + at.sc, at.k, at.NB, S);
            }
            at.next();
        }
    }
}

template <int kFmt, bool kWide>
__global__ void __launch_bounds__(kPackThreads)
mx_unpack_kernel(const uint8_t* codes, const uint8_t* scales, uint4* x, int64_t R, int CV)
{
    for (BlockWalk w(R, CV); !w.done();) {
        uint2 c[kPackAhead][2];
        int S[kPackAhead];
        BlockWalk at = w;
#pragma unroll
        for (int u = 0; u < kPackAhead; ++u) {
            load_two_codes<kFmt, kWide>(codes, w.vec, w.count(), c[u]);
            if (!w.done()) S[u] = __ldg(scales + w.sc);
            w.next();
        }
#pragma unroll
        for (int u = 0; u < kPackAhead; ++u) {
            const int n = at.count();
            if (n > 0) {
                uint4 q[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f[8];
                    mx_decode8<kFmt>(c[u][i], mx_scale_value(S[u]), f);
                    q[i] = pack8(f);
                }
                store_two<kWide>(x + at.vec, n, q);
            }
            at.next();
        }
    }
}

// ------------------------------------------------- forward with a checkpoint

struct CkptOut {
    uint8_t *Xc, *Xs, *Fc, *Fs;
};

// The inputs come through the backward's prefetch ring (BwdRing in
// mix_common.cuh: its four dY rows are X's here, its Z row is F), two vectors
// ahead and across token boundaries: the arithmetic between a load and its
// stores is long, and with loads straight into registers the kernel ran at
// 62% of the copy bandwidth.
constexpr int kFwdStages = 3;
using FwdRing = BwdRing<kFwdStages, kThreads, false>;

// Streams token t: X, F -> Y and the codes of X and F.
template <int kFmt>
__device__ __forceinline__ void mix_token_fwd_ckpt(const float (&h)[16], const float (&hp)[4], FwdRing& ring, uint4* Y,
                                                   const CkptOut& o, int64_t t, int CV)
{
    const int64_t sp = mx_scale_pitch((int64_t)CV * 8);
    uint4* Yt = Y + t * 4 * CV;
    // the bound depends on the warp only: every lane takes part in the shuffles
    for (int v = threadIdx.x; (v & ~31) < CV; v += kThreads) {
        const bool in = v < CV;
        uint4 r[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) r[j] = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            const uint4* slot = ring.next();
#pragma unroll
            for (int j = 0; j < 5; ++j) r[j] = slot[j * kThreads];
        }
        __syncwarp();
        int S[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) S[j] = mx_scale_byte<kFmt>(mx_block_max(mx_amax8(r[j])));
        if (in) {
            const uint4 x[4] = {r[0], r[1], r[2], r[3]};
            uint4 y[4];
            mix_vec(h, hp, x, r[4], y);
#pragma unroll
            for (int i = 0; i < 4; ++i) __stcs(Yt + (int64_t)i * CV + v, y[i]);
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                float f[8];
                unpack8(r[j], f);
                const int64_t row = j < 4 ? t * 4 + j : t;
                store_codes<kFmt>(j < 4 ? o.Xc : o.Fc, row * CV + v, mx_encode8<kFmt>(f, S[j]));
                if ((v & 3) == 0)
                    mx_store_scale((j < 4 ? o.Xs : o.Fs) + row * sp + (v >> 2), v >> 2, (CV + 3) >> 2, S[j]);
            }
        }
    }
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads)
mix_fwd_ckpt_kernel(const uint4* X, const float* H, const float* hpost, const uint4* F, uint4* Y, CkptOut o,
                    int64_t T, int CV)
{
    extern __shared__ uint4 ring_smem[];
    FwdRing ring(ring_smem, X, nullptr, F, T, CV);
    for (int64_t k = 0; k < ring.tokens(); ++k) {
        const int64_t t = (int64_t)blockIdx.x + k * gridDim.x;
        float h[16], hp[4];
        load_maps(H, hpost, t, h, hp);
        mix_token_fwd_ckpt<kFmt>(h, hp, ring, Y, o, t, CV);
    }
    ring.drain();
}

// Fused projection + mix with the checkpoint: the CTA's next kFusedTok tokens
// are projected together, one thread each, as in proj_mix_fwd_kernel of
// mhc_mix.cu, and then mixed one after the other in the ring's order.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
proj_mix_fwd_ckpt_kernel(const float* logits, const float* hpost, const uint4* X, const uint4* F, uint4* Y,
                         float* Hout, CkptOut o, int64_t T, int CV, int maxit)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float sH[kFusedTok][16];
    FwdRing ring(ring_smem, X, nullptr, F, T, CV);
    const int64_t n = ring.tokens();
    for (int64_t k0 = 0; k0 < n; k0 += kFusedTok) {
        if (threadIdx.x < kFusedTok && k0 + threadIdx.x < n) {
            const int64_t t = (int64_t)blockIdx.x + (k0 + threadIdx.x) * gridDim.x;
            float a[16];
            load16(logits + 16 * t, a);
            newton_project(a, maxit);
            store16(Hout + 16 * t, a);
#pragma unroll
            for (int k = 0; k < 16; ++k) sH[threadIdx.x][k] = a[k];
        }
        __syncthreads();
        for (int k = 0; k < kFusedTok && k0 + k < n; ++k) {
            const int64_t t = (int64_t)blockIdx.x + (k0 + k) * gridDim.x;
            float h[16], hp[4];
#pragma unroll
            for (int q = 0; q < 16; ++q) h[q] = sH[k][q];
            const float4 hq = __ldg(reinterpret_cast<const float4*>(hpost) + t);
            hp[0] = hq.x;
            hp[1] = hq.y;
            hp[2] = hq.z;
            hp[3] = hq.w;
            mix_token_fwd_ckpt<kFmt>(h, hp, ring, Y, o, t, CV);
        }
        __syncthreads();
    }
    ring.drain();
}

// ------------------------------------------------ backward from a checkpoint

// The prefetch ring of the bf16 backward (BwdRing in mix_common.cuh) with the
// X rows as 8-byte vectors of codes and, for kZCodes, the Z row too (F's
// codes; otherwise Z is dx_in in bf16).  Each coded row's scale travels with
// it: the four bytes that hold it, by a copy of their own.  A slot is
// kSlotBytes a thread, laid out row by row across the CTA.
__device__ __forceinline__ void cp_async8(void* smem, const void* gmem)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                     static_cast<unsigned>(__cvta_generic_to_shared(smem))),
                 "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     static_cast<unsigned>(__cvta_generic_to_shared(smem))),
                 "l"(gmem)
                 : "memory");
}

struct CkptIn {
    const uint8_t *Xc, *Xs;  // codes [T][4][C], scales [T][4][pitch]
    const uint8_t *Zc, *Zs;  // F's, or nullptr
    const uint4* Z;          // dx_in, or nullptr
};

constexpr int kStages = 2;
constexpr int kBwdCtas = 4;  // an SM: 128 registers a thread

template <bool kZCodes>
struct CkptRing {
    static constexpr int kCoded = kZCodes ? 5 : 4;
    static constexpr int kVec16 = kZCodes ? 4 : 5;  // dY rows, then dx_in
    static constexpr int kSlotBytes = kVec16 * 16 + kCoded * 8 + kCoded * 4;
    static constexpr int kSmemBytes = kStages * kSlotBytes * kThreads;

    uint8_t* slots;
    const uint4* dY;
    CkptIn in;
    int64_t ntok, ik, sp;
    int CV, rounds, iq, is, cs;

    __device__ __forceinline__ uint4* vec16(int slot, int r) const
    {
        return reinterpret_cast<uint4*>(slots + slot * (kSlotBytes * kThreads)) + r * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ uint2* codes(int slot, int r) const
    {
        return reinterpret_cast<uint2*>(slots + slot * (kSlotBytes * kThreads) + kVec16 * 16 * kThreads) +
               r * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ uint32_t* scale4(int slot, int r) const
    {
        return reinterpret_cast<uint32_t*>(slots + slot * (kSlotBytes * kThreads) +
                                           (kVec16 * 16 + kCoded * 8) * kThreads) +
               r * kThreads + threadIdx.x;
    }

    __device__ __forceinline__ CkptRing(void* smem, const uint4* dY_, const CkptIn& in_, int64_t T, int CV_)
        : slots(static_cast<uint8_t*>(smem)), dY(dY_), in(in_), ik(0), sp(mx_scale_pitch((int64_t)CV_ * 8)), CV(CV_),
          rounds((CV_ + kThreads - 1) / kThreads), iq(0), is(0), cs(0)
    {
        ntok = (int64_t)blockIdx.x < T ? (T - 1 - (int64_t)blockIdx.x) / gridDim.x + 1 : 0;
#pragma unroll
        for (int j = 0; j < kStages - 1; ++j) issue();
    }

    // Tokens of this CTA, and rounds of kThreads vectors in each.  Both, and the
    // ring's place, are the whole CTA's, so that row addresses are uniform; a
    // thread past the row copies nothing.
    __device__ __forceinline__ int64_t tokens() const { return ntok; }
    __device__ __forceinline__ int token_rounds() const { return rounds; }

    __device__ __forceinline__ void issue()
    {
        if (ik < ntok) {
            const int64_t t = (int64_t)blockIdx.x + ik * gridDim.x;
            const unsigned v = threadIdx.x + iq * kThreads;
            if ((int)v < CV) {
                const unsigned w = v >> 4 << 2;
#pragma unroll
                for (int r = 0; r < 4; ++r) cp_async16(vec16(is, r), dY + (t * 4 + r) * CV + v);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    cp_async8(codes(is, r), reinterpret_cast<const uint2*>(in.Xc) + (t * 4 + r) * CV + v);
                    cp_async4(scale4(is, r), in.Xs + (t * 4 + r) * sp + w);
                }
                if (kZCodes) {
                    cp_async8(codes(is, kCoded - 1), reinterpret_cast<const uint2*>(in.Zc) + t * CV + v);
                    cp_async4(scale4(is, kCoded - 1), in.Zs + t * sp + w);
                } else {
                    cp_async16(vec16(is, kVec16 - 1), in.Z + t * CV + v);
                }
            }
            if (++iq == rounds) {
                iq = 0;
                ++ik;
            }
        }
        cp_async_commit();  // an empty group past the end keeps the counting uniform
        is = is + 1 == kStages ? 0 : is + 1;
    }

    // Starts the next copy, waits for the next vector in order and returns its slot.
    __device__ __forceinline__ int next()
    {
        issue();
        cp_async_wait<kStages - 1>();
        const int slot = cs;
        cs = cs + 1 == kStages ? 0 : cs + 1;
        return slot;
    }

    // Row r's eight values at channel vector v.
    template <int kFmt>
    __device__ __forceinline__ void restore(int slot, int r, int v, float (&f)[8]) const
    {
        const int S = (int)((*scale4(slot, r) >> (8 * ((v >> 2) & 3))) & 255u);
        mx_decode8<kFmt>(*codes(slot, r), mx_scale_value(S), f);
    }

    __device__ __forceinline__ void drain() { cp_async_wait<0>(); }
};

// dX, dF, dH, dh_post and the chained projection backward, X and F restored
// from their codes in registers.
template <int kFmt>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
mix_bwd_ckpt_kernel(CkptIn in, const float* H, const float* hpost, const uint4* dY, uint4* dX, float* dH,
                    float* dhpost, uint4* dF, float* dlogits, int64_t T, int CV)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[kWarps * 20];
    __shared__ float tot[20];
    const int tid = threadIdx.x;
    CkptRing<true> ring(ring_smem, dY, in, T, CV);
    for (int64_t k = 0; k < ring.tokens(); ++k) {
        const int64_t t = (int64_t)blockIdx.x + k * gridDim.x;
        if (tid == 0 && k + 1 < ring.tokens()) {
            prefetch_l2(H + 16 * (t + gridDim.x));
            prefetch_l2(hpost + 4 * (t + gridDim.x));
        }
        float h[16], hp[4];
        load_maps(H, hpost, t, h, hp);
        uint4* dXt = dX + t * 4 * CV;
        uint4* dFt = dF + t * CV;
        float acc[20];
#pragma unroll
        for (int q = 0; q < 20; ++q) acc[q] = 0.0f;
        for (int q = 0; q < ring.token_rounds(); ++q) {
            const int slot = ring.next();
            const int v = tid + q * kThreads;
            if (v >= CV) continue;
            float dyf[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack8(*ring.vec16(slot, i), dyf[i]);
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                float xf[8];
                ring.template restore<kFmt>(slot, j, v, xf);
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& a = acc[j < 4 ? 4 * i + j : 16 + i];
                        a = fmaf(dyf[i][e], xf[e], a);
                    }
            }
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float s = (j < 4 ? h[j] : hp[0]) * dyf[0][e];
#pragma unroll
                    for (int i = 1; i < 4; ++i) s = fmaf(j < 4 ? h[4 * i + j] : hp[i], dyf[i][e], s);
                    o[e] = s;
                }
                __stcs(j < 4 ? dXt + (int64_t)j * CV + v : dFt + v, pack8(o));
            }
        }
        block_sum<20>(acc, red, tot);
        if (tid < 16) {
            if (dH) dH[16 * t + tid] = tot[tid];
        } else if (tid < 20) {
            if (dhpost) dhpost[4 * t + tid - 16] = tot[tid];
        }
        if (dlogits != nullptr && tid == 0) {
            float g[16], out[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) g[q] = tot[q];
            implicit_vjp(h, g, out);
            store16(dlogits + 16 * t, out);
        }
        // tot is rewritten only after the next token's first barrier, which
        // every reader above reaches after its read: no barrier needed here
    }
    ring.drain();
}

// Post part of the split backward: dF and dh_post from dY and F's codes.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
mix_post_bwd_ckpt_kernel(const uint4* dY, const uint8_t* Fc, const uint8_t* Fs, const float* hpost, uint4* dF,
                         float* dhpost, int64_t T, int CV)
{
    __shared__ float red[kWarps * 4];
    __shared__ float tot[4];
    const int64_t sp = mx_scale_pitch((int64_t)CV * 8);
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(hpost) + t);
        const float hp[4] = {q.x, q.y, q.z, q.w};
        const uint4* dYt = dY + t * 4 * CV;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int v = threadIdx.x; v < CV; v += kThreads) {
            float ff[8], o[8];
            mx_decode8<kFmt>(load_codes<kFmt>(Fc, t * CV + v), mx_scale_value(__ldg(Fs + t * sp + (v >> 2))), ff);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float dyf[8];
                unpack8(__ldcs(dYt + (int64_t)i * CV + v), dyf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[e] = fmaf(hp[i], dyf[e], o[e]);
                    acc[i] = fmaf(dyf[e], ff[e], acc[i]);
                }
            }
            __stcs(dF + t * CV + v, pack8(o));
        }
        block_sum<4>(acc, red, tot);
        if (threadIdx.x < 4) dhpost[4 * t + threadIdx.x] = tot[threadIdx.x];
    }
}

// Main part of the split backward with the pre-map's: dX, dH, dh_pre and the
// chained projection backward, X restored from its codes in registers.
template <int kFmt>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
mix_premap_bwd_ckpt_kernel(CkptIn in, const float* H, const float* hpre, const uint4* dY, uint4* dX, float* dH,
                           float* dhpre, float* dlogits, int64_t T, int CV)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[kWarps * 20];
    __shared__ float tot[20];
    const int tid = threadIdx.x;
    CkptRing<false> ring(ring_smem, dY, in, T, CV);
    for (int64_t k = 0; k < ring.tokens(); ++k) {
        const int64_t t = (int64_t)blockIdx.x + k * gridDim.x;
        if (tid == 0 && k + 1 < ring.tokens()) {
            prefetch_l2(H + 16 * (t + gridDim.x));
            prefetch_l2(hpre + 4 * (t + gridDim.x));
        }
        float h[16], s[4];
        load_maps(H, hpre, t, h, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = sigmoidf(s[j]);
        uint4* dXt = dX + t * 4 * CV;
        float acc[20];
#pragma unroll
        for (int q = 0; q < 20; ++q) acc[q] = 0.0f;
        for (int u = 0; u < ring.token_rounds(); ++u) {
            const int slot = ring.next();
            const int v = tid + u * kThreads;
            if (v >= CV) continue;
            float dyf[4][8], g[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack8(*ring.vec16(slot, i), dyf[i]);
            unpack8(*ring.vec16(slot, 4), g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float xf[8], o[8];
                ring.template restore<kFmt>(slot, j, v, xf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[4 * i + j] = fmaf(dyf[i][e], xf[e], acc[4 * i + j]);
                    acc[16 + j] = fmaf(g[e], xf[e], acc[16 + j]);
                    float a = s[j] * g[e];
#pragma unroll
                    for (int i = 0; i < 4; ++i) a = fmaf(h[4 * i + j], dyf[i][e], a);
                    o[e] = a;
                }
                __stcs(dXt + (int64_t)j * CV + v, pack8(o));
            }
        }
        block_sum<20>(acc, red, tot);
        if (tid < 16) {
            if (dH) dH[16 * t + tid] = tot[tid];
        } else if (tid < 20) {
            dhpre[4 * t + tid - 16] = sigmoid_grad(hpre[4 * t + tid - 16]) * tot[tid];
        }
        if (dlogits != nullptr && tid == 0) {
            float gH[16], out[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) gH[q] = tot[q];
            implicit_vjp(h, gH, out);
            store16(dlogits + 16 * t, out);
        }
        // as in mix_bwd_ckpt_kernel: the next token's first barrier orders tot
    }
    ring.drain();
}

// CTAs that cover all blocks of R rows, kPackAhead a thread.
int64_t pack_ctas(int64_t R, int CV)
{
    const int64_t blocks = R * ((CV + 3) / 4);
    return (blocks + kPackBlocks * kPackAhead - 1) / (kPackBlocks * kPackAhead);
}

bool wide_rows(const uint16_t* x, int CV) { return CV % 2 == 0 && (reinterpret_cast<uintptr_t>(x) & 31) == 0; }

template <int kFmt>
cudaError_t pack(const uint16_t* x, uint8_t* codes, uint8_t* scales, int64_t R, int CV, cudaStream_t s)
{
    const auto kernel = wide_rows(x, CV) ? mx_pack_kernel<kFmt, true> : mx_pack_kernel<kFmt, false>;
    const int grid = persistent_grid((const void*)kernel, kPackThreads, 0, pack_ctas(R, CV));
    kernel<<<grid, kPackThreads, 0, s>>>((const uint4*)x, codes, scales, R, CV);
    return cudaGetLastError();
}

template <int kFmt>
cudaError_t unpack(const uint8_t* codes, const uint8_t* scales, uint16_t* x, int64_t R, int CV, cudaStream_t s)
{
    const auto kernel = wide_rows(x, CV) ? mx_unpack_kernel<kFmt, true> : mx_unpack_kernel<kFmt, false>;
    const int grid = persistent_grid((const void*)kernel, kPackThreads, 0, pack_ctas(R, CV));
    kernel<<<grid, kPackThreads, 0, s>>>(codes, scales, (uint4*)x, R, CV);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_pack(const uint16_t* x, uint8_t* codes, uint8_t* scales, int64_t R, int64_t C, int format,
                           cudaStream_t s)
{
    const int CV = (int)(C / 8);
    if (format == MHC_MX_INT8) return pack<MHC_MX_INT8>(x, codes, scales, R, CV, s);
    if (format == MHC_MX_E4M3) return pack<MHC_MX_E4M3>(x, codes, scales, R, CV, s);
    return pack<MHC_MX_E2M1>(x, codes, scales, R, CV, s);
}

cudaError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, uint16_t* x, int64_t R, int64_t C,
                             int format, cudaStream_t s)
{
    const int CV = (int)(C / 8);
    if (format == MHC_MX_INT8) return unpack<MHC_MX_INT8>(codes, scales, x, R, CV, s);
    if (format == MHC_MX_E4M3) return unpack<MHC_MX_E4M3>(codes, scales, x, R, CV, s);
    return unpack<MHC_MX_E2M1>(codes, scales, x, R, CV, s);
}

cudaError_t launch_mix_fwd_ckpt(const uint16_t* X, const float* H, const float* hpost, const uint16_t* F, uint16_t* Y,
                                uint8_t* Xc, uint8_t* Xs, uint8_t* Fc, uint8_t* Fs, int64_t T, int64_t C, int format,
                                cudaStream_t s)
{
    const auto kernel = format == MHC_MX_INT8 ? mix_fwd_ckpt_kernel<MHC_MX_INT8> : mix_fwd_ckpt_kernel<MHC_MX_E4M3>;
    constexpr int smem = FwdRing::kSmemBytes;
    static_assert(smem <= 48 * 1024, "ring needs an opt-in");
    const int grid = persistent_grid((const void*)kernel, kThreads, smem, T);
    kernel<<<grid, kThreads, smem, s>>>((const uint4*)X, H, hpost, (const uint4*)F, (uint4*)Y,
                                        CkptOut{Xc, Xs, Fc, Fs}, T, (int)(C / 8));
    return cudaGetLastError();
}

cudaError_t launch_proj_mix_fwd_ckpt(const float* logits, const float* hpost, const uint16_t* X, const uint16_t* F,
                                     uint16_t* Y, float* H, uint8_t* Xc, uint8_t* Xs, uint8_t* Fc, uint8_t* Fs,
                                     int64_t T, int64_t C, int maxit, int format, cudaStream_t s)
{
    const auto kernel =
        format == MHC_MX_INT8 ? proj_mix_fwd_ckpt_kernel<MHC_MX_INT8> : proj_mix_fwd_ckpt_kernel<MHC_MX_E4M3>;
    constexpr int smem = FwdRing::kSmemBytes;
    static_assert(smem + kFusedTok * 64 <= 48 * 1024, "ring needs an opt-in");
    const int grid = persistent_grid((const void*)kernel, kThreads, smem, (T + kFusedTok - 1) / kFusedTok);
    kernel<<<grid, kThreads, smem, s>>>(logits, hpost, (const uint4*)X, (const uint4*)F, (uint4*)Y, H,
                                        CkptOut{Xc, Xs, Fc, Fs}, T, (int)(C / 8), maxit);
    return cudaGetLastError();
}

cudaError_t launch_mix_bwd_ckpt(const uint8_t* Xc, const uint8_t* Xs, const float* H, const float* hpost,
                                const uint8_t* Fc, const uint8_t* Fs, const uint16_t* dY, uint16_t* dX, float* dH,
                                float* dhpost, uint16_t* dF, float* dlogits, int64_t T, int64_t C, int format,
                                cudaStream_t s)
{
    const auto kernel = format == MHC_MX_INT8 ? mix_bwd_ckpt_kernel<MHC_MX_INT8> : mix_bwd_ckpt_kernel<MHC_MX_E4M3>;
    constexpr int smem = CkptRing<true>::kSmemBytes;
    static_assert(smem + kWarps * 20 * 4 + 80 <= 48 * 1024, "ring needs an opt-in");
    const int grid = persistent_grid((const void*)kernel, kThreads, smem, T);
    kernel<<<grid, kThreads, smem, s>>>(CkptIn{Xc, Xs, Fc, Fs, nullptr}, H, hpost, (const uint4*)dY, (uint4*)dX, dH,
                                        dhpost, (uint4*)dF, dlogits, T, (int)(C / 8));
    return cudaGetLastError();
}

cudaError_t launch_mix_post_bwd_ckpt(const uint16_t* dY, const uint8_t* Fc, const uint8_t* Fs, const float* hpost,
                                     uint16_t* dF, float* dhpost, int64_t T, int64_t C, int format, cudaStream_t s)
{
    const auto kernel =
        format == MHC_MX_INT8 ? mix_post_bwd_ckpt_kernel<MHC_MX_INT8> : mix_post_bwd_ckpt_kernel<MHC_MX_E4M3>;
    const int grid = persistent_grid((const void*)kernel, kThreads, 0, T);
    kernel<<<grid, kThreads, 0, s>>>((const uint4*)dY, Fc, Fs, hpost, (uint4*)dF, dhpost, T, (int)(C / 8));
    return cudaGetLastError();
}

cudaError_t launch_mix_premap_bwd_ckpt(const uint8_t* Xc, const uint8_t* Xs, const float* H, const float* hpre,
                                       const uint16_t* dY, const uint16_t* dx_in, uint16_t* dX, float* dH,
                                       float* dhpre, float* dlogits, int64_t T, int64_t C, int format, cudaStream_t s)
{
    const auto kernel =
        format == MHC_MX_INT8 ? mix_premap_bwd_ckpt_kernel<MHC_MX_INT8> : mix_premap_bwd_ckpt_kernel<MHC_MX_E4M3>;
    constexpr int smem = CkptRing<false>::kSmemBytes;
    static_assert(smem + kWarps * 20 * 4 + 80 <= 48 * 1024, "ring needs an opt-in");
    const int grid = persistent_grid((const void*)kernel, kThreads, smem, T);
    kernel<<<grid, kThreads, smem, s>>>(CkptIn{Xc, Xs, nullptr, nullptr, (const uint4*)dx_in}, H, hpre,
                                        (const uint4*)dY, (uint4*)dX, dH, dhpre, dlogits, T, (int)(C / 8));
    return cudaGetLastError();
}

}  // namespace mhc
