// delta.cuh -- the gated delta rule over chunks of C = 64 tokens on the
// tcgen05 tensor cores.
//
// Per batch row, value head h and key head g = h / (H / G), with Gamma_i the
// running log decay inside the chunk, rk_i = 1 / sqrt(|k_i|^2 + 1e-6) and S
// (P x N) the state before the chunk:
//   A_ij = beta_i e^(Gamma_i - Gamma_j) rk_i rk_j (k_i.k_j), j < i
//   T    = (I + A)^-1 diag(beta)                 (unit lower triangular solve)
//   R    = V - diag(e^Gamma rk) K S^T
//   U    = T R                                   (what the tokens really write)
//   Y    = scale rq (e^Gamma Q S^T + M U),  M_ij = e^(Gamma_i - Gamma_j) rk_j (q_i.k_j), j <= i
//   S   <- e^Gamma_last S + U^T diag(e^(Gamma_last - Gamma_j) rk_j) K
// T and M need no state: delta_prep_kernel makes them for every chunk at once.
// delta_walk_kernel then takes the state from chunk to chunk, one block per
// head: R, U, Y and the state's update are four products, each waiting for the
// one before it, so the walk is bound by that chain (about half of it tensor
// products, half the conversions between them), not by bandwidth.
//
// fp16 has no room for small beta (sigmoid(-10) is below its smallest normal
// number), so with theta the power of two above a chunk's largest beta T is
// kept over theta and R times theta; their product is U all the same.
//
// Everything in the walk is kept transposed, so that a tensor-memory lane is
// one value column v (M = 128 lanes): S^T row v, R^T, U^T and Y^T rows are all
// in lane v and belong to one thread, which holds the float32 state row in
// registers.  No value ever crosses a lane; the A operands are what the thread
// itself writes to its lane, and the B operands are the tiles K, Q, T, M as
// they lie in shared memory.  T and M are triangular, so their products go in
// two halves of 32 tokens without the zero block, and each half starts when
// its part of R is there: the conversions of one half run beside the products
// of the other.
//
// A walk takes the chunks of one head one after the other, so few heads leave
// most SMs idle.  Then the sequence is cut into segments: a first pass walks
// every segment but the last without outputs, once from a zero state (its end
// state) and once from the identity without V (its transition, N x N; the
// delta rule's is a full matrix, not a decay), and the walk of segment s enters
// with S_(j+1) = S_j M_j + S_loc,j folded over the segments before it.
//
// Precision.  Operands are fp16 with float32 accumulators.  K and Q enter
// scaled by a power of two per token (largest element in [1/2, 1)): exact, but
// for bits below 2^-25 of the row.  S, R, U (for the state) and T enter as two
// fp16 parts, hi + lo, 21 significant bits; the lo x lo term is dropped.  fp16
// needs values near 1, so each lane carries a power-of-two scale lambda_v: all
// of the walk is linear in lane v, so S, V, R, U and Y simply live in units of
// 1 / lambda_v.  Before each chunk a lane whose largest of |S| and theta |V| has left
// [2^-3, 2^6] rescales; with keys of length at most 1 no product of the chunk
// then exceeds 64 (1 + 64) + 64 sqrt(N) < 2^13, far inside fp16.  Raw keys may
// be longer; an operand that then leaves fp16's range comes out as infinity or
// NaN in y or in the end state (zeros of T and M times infinity are NaN, and S
// keeps one), and where either is not finite the error flag says so.
// Two bf16 parts (no scale needed) came to 4.5e-6 on the final state in a
// float64 model of these roundings, and three to half again as many products;
// measured with fp16 parts: 5e-7.  Y's products take both parts of S, U and M
// too, so Y is rounded once, to bf16: with the leading parts alone it was 4e-4
// off before that, and 3.5e-4 too small (a cut part lies nearer to zero).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "delta_step.cuh"
#include "device_math.cuh"
#include "tc_ops.cuh"

namespace axon {

constexpr int kDlC = 64;                       // tokens per chunk
constexpr int kDlTile = kDlC * kDlC * 2;       // a 64 x 64 fp16 tile: 8 KB
constexpr int kDlVec = 4 * kDlC * 4;           // four rows, a value a token: -theta e^Gamma rk, e^Gamma, e^(Gamma_last - Gamma) rk, scale rq
// Per chunk and value head: T hi, T lo, M hi, vectors.  The three matrices are
// lower triangular, and no product reads their upper right 32 x 32 blocks:
// those hold the three other blocks of M lo (T hi's: rows and columns 0 .. 31,
// T lo's: rows 32 .., columns 0 .., M hi's: rows and columns 32 ..), which as
// a tile of their own would not fit three stages of shared memory.
constexpr int kDlBlob = 3 * kDlTile + kDlVec;

struct DeltaChunkParams {
    DeltaParams d;
    int nC;                      // chunks of L
    unsigned char* kq;           // (B, G, nC): K', then Q': fp16, 64 rows in 64-column blocks, 128-byte swizzle
    unsigned char* blob;         // (B, H, nC): kDlBlob bytes
    int* err;                    // bits: 1 a wait gave up, 2 y or the end state is not finite (told with raw keys only)
    // the sequence in segments of cps chunks, when there are few heads:
    int segs, cps;
    float* sloc;                 // (segs - 1, B, H, P, N): a segment's end state from zeros (the first: from h0)
    unsigned char* tr;           // (segs - 2, B, H): transitions of segments 1 .., fp16 hi and lo tiles (N x N)
    float* trs;                  // (segs - 2, B, H, N): what a transition's row is in units of
    float* h0c;                  // (B, H, P, N): h0 again (h_out may lie over it)
};

// kind::f16 instruction descriptor with fp16 A and B, float32 D
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A pair as hi + lo fp16 parts: hi the leading 11 bits (cut off, so that the
// rest is an exact subtraction), lo the rest rounded.  8.1 cycles a pair and
// warp; rounding hi and subtracting it in the mixed precision fma took 9.6.
__device__ __forceinline__ void split_f16(float2 x, uint32_t& hi, uint32_t& lo) {
    const float h0 = __uint_as_float(__float_as_uint(x.x) & 0xffffe000u), h1 = __uint_as_float(__float_as_uint(x.y) & 0xffffe000u);
    hi = pack_f16(h0, h1);
    lo = pack_f16(x.x - h0, x.y - h1);
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }    // -126 <= e <= 127

// For m > 0 the exponent e with m 2^-e in [1/2, 1); ..
__device__ __forceinline__ int exp_of(float m) { return (int)((__float_as_uint(m) >> 23) & 255u) - 126; }
// .. held to what a float power of two and its inverse can say (m 2^-e < 4).
__device__ __forceinline__ int exp_above(float m) { return min(max(exp_of(m), -126), 126); }
// theta's exponent from the largest b_raw of a chunk (-inf: no token): prep and walk agree to the bit
__device__ __forceinline__ int theta_exp(float b_max) {
    const float beta = delta_beta(b_max);
    return beta > 0.f ? exp_of(beta) : 0;
}
// a b + c with a and b in bf16
__device__ __forceinline__ float fma_bf16(unsigned short a, unsigned short b, float c) {
    float d;
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
    return d;
}
// max(m, |a|, |b|)
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}
// 8 consecutive 32-bit columns into this thread's tensor-memory lane
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
// ---- prep: grid = (nC, G, B), 128 threads.  What bounds it is latency and the
// instruction caches (five blocks an SM in different phases, six at N = 64), so the loops are
// kept short: forward substitution down whole columns, unrolled over
// registers, took 15 to 24 thousand cycles a head where this takes three.
// 4096 tokens of 32 heads on 16 key heads, N = 128: 49 us, 41% of issue slots,
// 65 MB from and to HBM.
template <int N>
struct DeltaPrepSmem {
    static constexpr int LDA = 68;                       // floats a row of A: 16-byte rows without bank conflicts
    static constexpr int LDW = 36;
    static constexpr int KQ_BYTES = 128 * N * 2;
    static constexpr int KQ = 0;                         // [K'; Q'] tile, read by the Gram products only ...
    static constexpr int A = 0;                          // ... then A (float32), in place (I + A)^-1,
    static constexpr int M = kDlC * LDA * 4;             // the M tile,
    static constexpr int W = M + kDlTile;                // and a product on its way
    static constexpr int W_END = W + 32 * LDW * 4;
    static constexpr int V = KQ_BYTES > W_END ? KQ_BYTES : W_END;   // the vectors, two heads
    static constexpr int RK = V + 2 * kDlVec;            // rk'
    static constexpr int RQ = RK + kDlC * 4;             // scale rq'
    static constexpr int GH = RQ + kDlC * 4;             // two heads: Gamma (log2 units), float hi and lo parts
    static constexpr int GL = GH + 2 * kDlC * 4;
    static constexpr int BE = GL + 2 * kDlC * 4;         // beta
    static constexpr int BT = BE + 2 * kDlC * 4;         // beta / theta
    static constexpr int VJ = BT + 2 * kDlC * 4;         // e^(Gamma_r - Gamma_j) rk'_j, r the last of j's 16 tokens
    static constexpr int TOT = VJ + 2 * kDlC * 4;        // doubles: the first warps' totals
    static constexpr int BM = TOT + 16;                  // the warps' largest b_raw
    static constexpr int MB = BM + 16;
    static constexpr int SLOT = MB + 8;
    static constexpr int BYTES = SLOT + 8;
    static constexpr int TOTAL = BYTES + 1024;           // with the alignment pad
    static_assert(M % 16 == 0 && W % 16 == 0 && V % 16 == 0 && TOT % 8 == 0, "alignment");
};

// (I + A)^-1 in place, A strictly lower triangular with zeros above: 16 x 16
// diagonal blocks by forward substitution (a thread a column), then twice
// T21 = -T22 (A21 T11) for blocks of 16 and of 32.  128 threads; ends synchronised.
template <int LDA, int LDW>
__device__ __forceinline__ void delta_invert(float* A, float* W, int tid) {
    if (tid < kDlC) {
        const int o = tid & ~15, j = tid & 15;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float* row = A + (o + i) * LDA + o;
            float acc[4] = {i == j ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < i; k += 4) {             // what the row holds from its diagonal on is 0
                const float4 x4 = *reinterpret_cast<const float4*>(row + k);
                acc[0] = fmaf(-x4.x, t[k], acc[0]);
                if (k + 1 < i) acc[1] = fmaf(-x4.y, t[k + 1], acc[1]);
                if (k + 2 < i) acc[2] = fmaf(-x4.z, t[k + 2], acc[2]);
                if (k + 3 < i) acc[3] = fmaf(-x4.w, t[k + 3], acc[3]);
            }
            t[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) A[(o + i) * LDA + o + j] = t[i];
    }
    __syncthreads();
    {
        const int o = 32 * (tid >> 6), r = (tid & 63) >> 2, c = (tid & 3) * 4;
        float* w = W + (tid >> 6) * 16 * LDW;
        float* row = A + (o + 16 + r) * LDA + o;         // of A21, then of T22 16 columns on
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < 16; k += 4) {
            const float4 x4 = *reinterpret_cast<const float4*>(row + k);
            const float xk[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y = *reinterpret_cast<const float4*>(A + (o + k + q) * LDA + o + c);
                s.x = fmaf(xk[q], y.x, s.x); s.y = fmaf(xk[q], y.y, s.y); s.z = fmaf(xk[q], y.z, s.z); s.w = fmaf(xk[q], y.w, s.w);
            }
        }
        *reinterpret_cast<float4*>(w + r * LDW + c) = s;
        __syncthreads();
        s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < 16; k += 4) {
            const float4 x4 = *reinterpret_cast<const float4*>(row + 16 + k);
            const float xk[4] = {-x4.x, -x4.y, -x4.z, -x4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y = *reinterpret_cast<const float4*>(w + (k + q) * LDW + c);
                s.x = fmaf(xk[q], y.x, s.x); s.y = fmaf(xk[q], y.y, s.y); s.z = fmaf(xk[q], y.z, s.z); s.w = fmaf(xk[q], y.w, s.w);
            }
        }
        *reinterpret_cast<float4*>(row + c) = s;
    }
    __syncthreads();
    {
        const int r = tid >> 2, c = (tid & 3) * 8;
        const int kend = (r & ~7) + 8;                   // T22 is 0 behind its diagonal (warp-uniform)
        float* row = A + (32 + r) * LDA;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {           // W = A21 T11, then T21 = -T22 W
            float2 s[4] = {};
            const float* x = row + 32 * pass;
            const float* y = pass ? W + c : A + c;
            const int ldy = pass ? LDW : LDA;
#pragma unroll 2
            for (int k = 0; k < (pass ? kend : 32); k += 4) {
                const float4 x4 = *reinterpret_cast<const float4*>(x + k);
                const float xk[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 y0 = *reinterpret_cast<const float4*>(y + (k + q) * ldy);
                    const float4 y1 = *reinterpret_cast<const float4*>(y + (k + q) * ldy + 4);
                    const float2 xx = make_float2(xk[q], xk[q]);
                    s[0] = __ffma2_rn(xx, make_float2(y0.x, y0.y), s[0]);
                    s[1] = __ffma2_rn(xx, make_float2(y0.z, y0.w), s[1]);
                    s[2] = __ffma2_rn(xx, make_float2(y1.x, y1.y), s[2]);
                    s[3] = __ffma2_rn(xx, make_float2(y1.z, y1.w), s[3]);
                }
            }
            const float f = pass ? -1.f : 1.f;
            float* out = pass ? row + c : W + r * LDW + c;
            *reinterpret_cast<float4*>(out) = make_float4(f * s[0].x, f * s[0].y, f * s[1].x, f * s[1].y);
            *reinterpret_cast<float4*>(out + 4) = make_float4(f * s[2].x, f * s[2].y, f * s[3].x, f * s[3].y);
            __syncthreads();
        }
    }
}

template <int N>
__global__ void __launch_bounds__(128, 6) delta_prep_kernel(DeltaChunkParams p) {
    using Lay = DeltaPrepSmem<N>;
    constexpr int C = kDlC;
    grid_dep_launch();
    const int c = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const DeltaParams& d = p.d;
    if (c == 0 && g == 0 && b == 0 && tid == 0) *p.err = 0;
    int len = d.L;
    if (d.lengths) len = min(max(__ldg(d.lengths + b), 0), d.L);
    const int t0 = c * C;
    if (t0 >= len) return;                               // whole block
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    unsigned char* sm = smem_raw + pad;
    const uint32_t sb = raw + pad;
    float* rk = reinterpret_cast<float*>(sm + Lay::RK);
    float* rq = reinterpret_cast<float*>(sm + Lay::RQ);

    // ---- rows of K (tile rows 0 .. 63) and Q (64 .. 127) into the tile, eight
    // lanes a row; rows past the end as zeros
    constexpr int PC = N / 64;                           // 16-byte pieces of a lane
    const int l = tid & 7, r0 = tid >> 3;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int t = r0 + 16 * (k & 3), s = k >> 2, ld = s ? d.ldq : d.ldk;
        const bool ok = t0 + t < len;
        const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(s ? d.q : d.k) +
                                   ((size_t)b * d.L + (ok ? t0 + t : 0)) * ld + (size_t)g * N;
#pragma unroll
        for (int i = 0; i < PC; ++i)
            cp_async16(sm + Lay::KQ + i * 16384 + (64 * s + t) * 128 + ((l ^ (t & 7)) << 4), row + 8 * (l + 8 * i), ok);
    }
    cp_async_commit();
    if (w == 0) tmem_alloc(sb + Lay::SLOT, 64);
    if (tid == 0) mbar_init(sb + Lay::MB, 1);
    cp_async_wait_0();
    // each piece in place (its own thread's): the row's largest element to [1/2, 1), fp16
    unsigned char* kq = p.kq + (((size_t)b * d.G + g) * p.nC + c) * Lay::KQ_BYTES;
#pragma unroll 2
    for (int k = 0; k < 8; ++k) {
        const int t = r0 + 16 * (k & 3), s = k >> 2;
        const int in_row = (l ^ (t & 7)) << 4;
        float m = 0.f;
        float f[PC][8];
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(sm + Lay::KQ + i * 16384 + (64 * s + t) * 128 + in_row);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[i][2 * e] = bf16_lo(u[e]);
                f[i][2 * e + 1] = bf16_hi(u[e]);
                m = max_abs3(m, f[i][2 * e], f[i][2 * e + 1]);
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = exp_above(m);
        const float sc = pow2i(-e);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float x0 = f[i][2 * q] * sc, x1 = f[i][2 * q + 1] * sc;
                ss = fmaf(x0, x0, fmaf(x1, x1, ss));
                h[q] = pack_f16(x0, x1);
            }
            const uint4 o = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(sm + Lay::KQ + i * 16384 + (64 * s + t) * 128 + in_row) = o;
            *reinterpret_cast<uint4*>(kq + s * (Lay::KQ_BYTES / 2) + i * 8192 + t * 128 + in_row) = o;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (l == 0) {
            // 1 / sqrt(|k|^2 + eps) in the scaled row's units: |k|^2 = ss 4^e
            const float es = pow2i(e);
            const float f1 = d.norm ? es * rsqrtf(fmaf(ss * es, es, kDeltaEps)) : es;
            (s ? rq : rk)[t] = s ? d.scale * f1 : f1;
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(sm + Lay::SLOT);
    if (w == 0 && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) {
            const uint64_t dsc = umma_desc(sb + Lay::KQ + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
            umma(tbase, dsc, dsc, umma_idesc_f16(128, C, 0, 0), ks > 0);      // [K'; Q'] K'^T
        }
        umma_commit(sb + Lay::MB);
    }
    __syncwarp();
    const bool ok = mbar_wait(sb + Lay::MB, 0u);
    const bool failed = __syncthreads_or(!ok);           // KQ is free from here on: A, M and W lie over it
    const bool drained = !failed || mbar_wait(sb + Lay::MB, 0u);
    tc_fence_after();
    if (failed && tid == 0) atomicOr(p.err, 1);

    const int r = d.H / d.G;
    const int i = tid & 63;                              // this thread's row of A (warps 0, 1) or M (2, 3)
    const bool live = t0 + i < len;
    float* A = reinterpret_cast<float*>(sm + Lay::A);
#pragma unroll 1
    for (int hh = 0; hh < r && !failed; ++hh) {
        const int h = g * r + hh, slot = hh & 1;
        float* vec = reinterpret_cast<float*>(sm + Lay::V) + slot * 4 * C;
        const float* gh = reinterpret_cast<const float*>(sm + Lay::GH) + slot * C;
        const float* gl = reinterpret_cast<const float*>(sm + Lay::GL) + slot * C;
        const float* be = reinterpret_cast<const float*>(sm + Lay::BE) + slot * C;
        const float* bt = reinterpret_cast<const float*>(sm + Lay::BT) + slot * C;
        const float* vj = reinterpret_cast<const float*>(sm + Lay::VJ) + slot * C;
        if (slot == 0) {
            // ---- the rates of two heads (warps 0, 1 and 2, 3), a token a lane.  The
            // running log decay is summed in double: it reaches hundreds, and
            // differences of neighbours count.
            const int mine = tid >> 6, hm = h + mine;
            const bool have = hh + mine < r;
            float lg = 0.f, beta = 0.f, bm = -INFINITY;
            if (live && have) {
                const size_t o = ((size_t)b * d.L + t0 + i) * d.H + hm;
                lg = delta_log2_decay(IoBF16::load(static_cast<const __nv_bfloat16*>(d.dt_raw) + o) + __ldg(d.dt_bias + hm),
                                      delta_exp_a(__ldg(d.A_log + hm)));
                // a decay below 2^-2000 is 0 to a float anyway, and an infinite one would leave inf - inf
                lg = lg < -2000.f ? -2000.f : lg;
                bm = IoBF16::load(static_cast<const __nv_bfloat16*>(d.b_raw) + o);
                beta = delta_beta(bm);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
            float* bms = reinterpret_cast<float*>(sm + Lay::BM);
            if (lane == 0) bms[w] = bm;
            double G = (double)lg;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, G, o);
                if (lane >= o) G += v;
            }
            double* tot = reinterpret_cast<double*>(sm + Lay::TOT) + mine;
            float* gh2 = reinterpret_cast<float*>(sm + Lay::GH) + mine * C;
            float* gl2 = reinterpret_cast<float*>(sm + Lay::GL) + mine * C;
            if ((tid & 63) == 31) *tot = G;
            reinterpret_cast<float*>(sm + Lay::BE)[mine * C + i] = beta;
            __syncthreads();
            if (w & 1) G += *tot;
            const int te = theta_exp(fmaxf(bms[2 * mine], bms[2 * mine + 1]));
            reinterpret_cast<float*>(sm + Lay::BT)[mine * C + i] = beta * pow2i(-te);
            const float hi = (float)G, lo = (float)(G - (double)hi);
            gh2[i] = hi;
            gl2[i] = lo;
            __syncthreads();
            const int r16 = i | 15;
            const float eg = ex2_approx(hi);
            float* v2 = reinterpret_cast<float*>(sm + Lay::V) + mine * 4 * C;
            reinterpret_cast<float*>(sm + Lay::VJ)[mine * C + i] = ex2_approx((gh2[r16] - hi) + (gl2[r16] - lo)) * rk[i];
            v2[i] = -(eg * rk[i]) * pow2i(te);
            v2[C + i] = eg;
            v2[2 * C + i] = ex2_approx((gh2[C - 1] - hi) + (gl2[C - 1] - lo)) * rk[i];
            v2[3 * C + i] = rq[i];
            __syncthreads();
        }
        // ---- row i of A, or of M.  Left of the warp's diagonal blocks of 16 the decay
        // e^(Gamma_i - Gamma_j) = e^(Gamma_i - Gamma_r) e^(Gamma_r - Gamma_j): one
        // exponential a row and block, both factors at most 1.
        const float ghi = gh[i], glo = gl[i];
        const float f = w < 2 ? be[i] * rk[i] : 1.f;
        const int edge = w < 2 ? i : i + 1;              // columns below it belong to the triangle
        const int diag = 32 * (w & 1);                   // the warp's rows are diag .. diag + 31
#pragma unroll 1
        for (int j0 = 0; j0 < diag + 32; j0 += 16) {     // what is right of the diagonal blocks of 32 is not A's or M's (see kDlBlob)
            float x[16];
            tmem_ld16(tbase + ((uint32_t)(32 * w) << 16) + j0, x);
            if (j0 < diag) {
                const float u = ex2_approx((ghi - gh[j0 + 15]) + (glo - gl[j0 + 15])) * f;
#pragma unroll
                for (int q = 0; q < 16; q += 4) {
                    const float4 v4 = *reinterpret_cast<const float4*>(vj + j0 + q);
                    x[q] *= u * v4.x; x[q + 1] *= u * v4.y; x[q + 2] *= u * v4.z; x[q + 3] *= u * v4.w;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; q += 4) {
                    const float4 h4 = *reinterpret_cast<const float4*>(gh + j0 + q);
                    const float4 l4 = *reinterpret_cast<const float4*>(gl + j0 + q);
                    const float4 r4 = *reinterpret_cast<const float4*>(rk + j0 + q);
                    const float hj[4] = {h4.x, h4.y, h4.z, h4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
                    const float rj[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float dec = ex2_approx((ghi - hj[e]) + (glo - lj[e]));
                        x[q + e] = j0 + q + e < edge ? x[q + e] * f * (dec * rj[e]) : 0.f;
                    }
                }
            }
            if (w < 2) {
#pragma unroll
                for (int q = 0; q < 16; q += 4)
                    *reinterpret_cast<float4*>(A + i * Lay::LDA + j0 + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
            } else {
                // M lo: the block at (32, 32) into M's tile, the others beside A's
                // rows 0 .. 31 (bytes 128 .. of a row: M's rows 0 .., then 32 ..), on their way to T's tiles
                const int il = i & 31;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int pc = j0 / 8 + q;
                    uint4 hi, lo;
                    split_f16(make_float2(x[8 * q], x[8 * q + 1]), hi.x, lo.x);
                    split_f16(make_float2(x[8 * q + 2], x[8 * q + 3]), hi.y, lo.y);
                    split_f16(make_float2(x[8 * q + 4], x[8 * q + 5]), hi.z, lo.z);
                    split_f16(make_float2(x[8 * q + 6], x[8 * q + 7]), hi.w, lo.w);
                    *reinterpret_cast<uint4*>(sm + Lay::M + i * 128 + ((pc ^ (i & 7)) << 4)) = hi;
                    *reinterpret_cast<uint4*>(pc >= 4 ? sm + Lay::M + il * 128 + ((pc ^ (il & 7)) << 4)
                                                      : sm + Lay::A + il * (Lay::LDA * 4) + 128 + 2 * diag + 16 * pc) = lo;
                }
            }
        }
        __syncthreads();
        // ---- the blob: T = (I + A)^-1 diag(beta / theta) as fp16 hi and lo tiles, M, the vectors
        unsigned char* blob = p.blob + (((size_t)b * d.H + h) * p.nC + c) * kDlBlob;
        if (w >= 2) {                                    // beside the diagonal blocks' inversion by warps 0 and 1
#pragma unroll
            for (int k = 0; k < kDlTile / 16 / 64; ++k)
                reinterpret_cast<uint4*>(blob + 2 * kDlTile)[i + 64 * k] = *reinterpret_cast<const uint4*>(sm + Lay::M + (i + 64 * k) * 16);
            reinterpret_cast<float4*>(blob + 3 * kDlTile)[i] = reinterpret_cast<const float4*>(vec)[i];
        }
        delta_invert<Lay::LDA, Lay::LDW>(A, reinterpret_cast<float*>(sm + Lay::W), tid);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            const int row = (tid >> 3) + 16 * k, pc = tid & 7;
            const float4 a0 = *reinterpret_cast<const float4*>(A + row * Lay::LDA + 8 * pc);
            const float4 a1 = *reinterpret_cast<const float4*>(A + row * Lay::LDA + 8 * pc + 4);
            const float4 b0 = *reinterpret_cast<const float4*>(bt + 8 * pc), b1 = *reinterpret_cast<const float4*>(bt + 8 * pc + 4);
            uint4 hi, lo;
            split_f16(make_float2(a0.x * b0.x, a0.y * b0.y), hi.x, lo.x);
            split_f16(make_float2(a0.z * b0.z, a0.w * b0.w), hi.y, lo.y);
            split_f16(make_float2(a1.x * b1.x, a1.y * b1.y), hi.z, lo.z);
            split_f16(make_float2(a1.z * b1.z, a1.w * b1.w), hi.w, lo.w);
            if (k < 2 && pc >= 4) {                      // M lo's blocks
                hi = *reinterpret_cast<const uint4*>(sm + Lay::A + row * (Lay::LDA * 4) + 64 + 16 * pc);
                lo = *reinterpret_cast<const uint4*>(sm + Lay::A + row * (Lay::LDA * 4) + 128 + 16 * pc);
            }
            const int off = row * 128 + ((pc ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(blob + off) = hi;
            *reinterpret_cast<uint4*>(blob + kDlTile + off) = lo;
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 0 && __all_sync(0xffffffffu, drained)) tmem_dealloc(tbase, 64);   // unless a late product might still write
}

// ---- the walk: grid = (H, B, segments), 576 threads; without outputs grid =
// (H, B, 2 segments - 3): end states of segments 0 .., then transitions of 1 ...  Warps 0 .. 15 compute: warp w holds
// lanes 32 (w & 3) .. of tensor memory, and the four warps of such a quadrant
// share its lanes' work, thread `part` = w >> 2 of a lane taking a quarter of
// the state row and of the tokens.  (One warp a quadrant, two blocks an SM,
// took 12 thousand cycles a chunk: with one warp a scheduler nothing hides the
// latencies of the conversions.)  Warp 16 copies tiles in and issues products,
// warp 17 finds theta and the columns' largest |v| a chunk ahead.  A chunk takes
// 2.8 us without outputs and 3.3 with (N = P = 128): 4096 tokens of 32 heads in three segments, 70 us
// without and 88 us with outputs, tensor pipe 32% and issue slots 52% busy.
// The second parts of Y's operands and theta are 8 of those 88.
constexpr int kDlThreads = 576;
constexpr int kDlStages = 3;

template <int N, int P>
struct DeltaWalkSmem {
    static constexpr int K_BYTES = kDlC * N * 2;
    static constexpr int V_BYTES = kDlC * P * 2;
    // a stage: all of a chunk's tiles
    static constexpr int K = 0;
    static constexpr int Q = K + K_BYTES;
    static constexpr int T = Q + K_BYTES;                 // T hi, T lo
    static constexpr int M = T + 2 * kDlTile;
    static constexpr int VEC = M + kDlTile;
    static constexpr int V = VEC + kDlVec;                // 64 rows of P bf16
    static constexpr int STAGE = V + V_BYTES;
    static constexpr int VM = kDlStages * STAGE;          // theta times the largest |v| of the columns, per stage; theta
    static constexpr int VMS = P * 4 + 16;
    static constexpr int SMAX = VM + kDlStages * VMS;     // largest |S| of the quarters of a lane's state row
    static constexpr int MB = SMAX + 4 * 128 * 4;
    enum { FULL, VMAX = FULL + kDlStages, X_K0 = VMAX + kDlStages, X_K1, X_Q, U_0, U_1, Y_M, D, D_HI, S_IN, R_IN0, R_IN1, U_IN0,
           U_IN1, Y_OUT, QUAD, DRAIN = QUAD + 4, TR_FULL, BARS = TR_FULL + 2 };
    static constexpr int DEAD = MB + 8 * BARS;            // a wait gave up
    static constexpr int SLOT = DEAD + 4;
    static constexpr int BYTES = SLOT + 4;
    static constexpr int TOTAL = BYTES + 1024;
    static constexpr int TR_BYTES = N * N * 2;            // a part of a transition, in the stages after the first
    static_assert(2 * TR_BYTES <= STAGE, "a transition fits a stage");
    static_assert(TOTAL <= 227 * 1024, "shared memory of a block");
    static_assert(STAGE % 1024 == 0 && VEC % 128 == 0, "swizzled tiles and copies aligned");
    // tensor memory: the A operands hold two fp16 a column; 16 tokens of R, U_w and U (for Y) are 8 columns hi, 8 lo
    static constexpr int S_HI = 0, S_LO = 64, DD = 0;     // the state's increment comes where S was
    static constexpr int XK = 128, XQ = 192;              // K S^T; Q S^T
    static constexpr int R = 256, U = 320, UW = 384, UH = 448;    // M U comes where U was
    static constexpr int COLS = 512;
};

// The warp waits for an mbarrier's phase; gives up after a bounded number of
// polls, or when another warp of the block has.  The same answer in every lane.
__device__ __forceinline__ bool delta_wait(uint32_t mbar, int use, volatile int* dead, int limit = kTcWaitLimit) {
    if (__all_sync(0xffffffffu, mbar_wait(mbar, (uint32_t)(use & 1), 1))) return true;
    bool ok = false;
    for (int k = 0; k < limit && !ok; k += 1024) {
        ok = mbar_wait(mbar, (uint32_t)(use & 1), min(limit - k, 1024));
        if (!ok && *dead) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *dead = 1;
    return ok;
}
// After a wait gave up: tells the host, and whether the products that this
// warp's elected lane has issued are all done (a bounded wait); only then may
// their tensor memory go to another block.
__device__ __forceinline__ bool delta_drain(uint32_t mbar, int* err) {
    if (elect_one()) {
        atomicOr(err, 1);
        umma_commit(mbar);
    }
    __syncwarp();
    return __all_sync(0xffffffffu, mbar_wait(mbar, 0u));
}
// The walk's failure path by itself: warp 0 waits `limit` polls for an mbarrier
// that nothing arrives on, warp 1 (with the walk's own limit) for another until
// warp 0 has given up; then the drain, with no product in flight, and the
// tensor memory is freed.  status[0]: bit 0 warp 0 gave up, 1 warp 1 did, 2
// drained; status[1]: the error flag.  grid = 1, 64 threads.
__global__ void __launch_bounds__(64) delta_wait_probe_kernel(int* status, int limit) {
    __shared__ __align__(8) unsigned long long bars[3];
    __shared__ int dead, slot, got;
    const uint32_t mb = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
    const int w = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(mb + 8 * i, 1);
        dead = 0;
        got = 0;
        status[1] = 0;
        fence_mbar_init();
    }
    if (w == 0) tmem_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(&slot)), 32);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const bool done = delta_wait(mb + 8 * w, 0, &dead, w == 0 ? limit : kTcWaitLimit);
    if (!done && (threadIdx.x & 31) == 0) atomicOr(&got, 1 << w);
    __syncthreads();
    if (w == 0) {
        const bool drained = delta_drain(mb + 16, status + 1);
        if (drained) tmem_dealloc(*reinterpret_cast<volatile int*>(&slot), 32);
        if (threadIdx.x == 0) status[0] = got | (drained ? 4 : 0);
    }
}
// 8 consecutive columns of this thread's tensor-memory lane; 4 into it
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(r[q]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
}

template <int N, int P, bool kFull>
__global__ void __launch_bounds__(kDlThreads, 1) delta_walk_kernel(const __grid_constant__ CUtensorMap tmV, DeltaChunkParams p) {
    using Lay = DeltaWalkSmem<N, P>;
    constexpr int C = kDlC, KS = N / 16, ST = kDlStages;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    unsigned char* sm = smem_raw + pad;
    const uint32_t sb = raw + pad;
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const DeltaParams& d = p.d;
    int len = d.L;
    if (d.lengths) len = min(max(__ldg(d.lengths + b), 0), d.L);
    // this block's chunks: cb .. cb + nC - 1
    const bool trans = !kFull && (int)blockIdx.z >= p.segs - 1;
    const int seg = trans ? blockIdx.z - (p.segs - 1) + 1 : blockIdx.z;
    const int all = (len + C - 1) / C, cb = seg * p.cps, nC = min(p.cps, all - cb);
    if (nC <= 0 && seg > 0) return;                       // whole block; an empty row's state passes through segment 0
    const int nf = kFull && seg > 1 ? seg - 1 : 0;        // transitions to fold into the entering state
    const int lanes = trans ? N : P;
    const int g = h / (d.H / d.G);
    volatile int* dead = reinterpret_cast<volatile int*>(sm + Lay::DEAD);
    auto bar = [&](int i) { return sb + Lay::MB + 8 * i; };

    if (tid == 0) {
        for (int i = 0; i < Lay::BARS; ++i)
            mbar_init(bar(i), i >= Lay::S_IN && i <= Lay::Y_OUT ? lanes / 8 : i >= Lay::QUAD && i < Lay::DRAIN ? 4 : 1);   // warps
        *dead = 0;
        fence_mbar_init();
    }
    grid_dep_wait();                                      // the prep kernel's tiles are written
    fence_proxy_async();
    // only now, or these columns might keep a prep block waiting that this one waits for
    if (w == 16) tmem_alloc(sb + Lay::SLOT, Lay::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(sm + Lay::SLOT);

    if (w == 16) {
        // ---------------- copies and products.  The warp runs the loop together and one
        // lane issues: in a region of one lane only, addresses live in vector
        // registers, and a product costs twice what the tensor core takes for it.
        const unsigned char* kq = p.kq + (((size_t)b * d.G + g) * p.nC + cb) * (2 * Lay::K_BYTES);
        const unsigned char* blob = p.blob + (((size_t)b * d.H + h) * p.nC + cb) * kDlBlob;
        const uint32_t v_bytes = trans ? 0 : Lay::V_BYTES;
        auto load_chunk = [&](int c, int st) {            // V's rows past L read as zeros
            if (elect_one()) {
                const uint32_t full = bar(Lay::FULL + st), dst = sb + st * Lay::STAGE;
                mbar_arrive_expect_tx(full, (kFull ? 2 * Lay::K_BYTES + kDlBlob : Lay::K_BYTES + 2 * kDlTile + kDlVec) + v_bytes);
                const unsigned char* src = blob + (size_t)c * kDlBlob;
                bulk_load(dst + Lay::K, kq + (size_t)c * 2 * Lay::K_BYTES, (kFull ? 2 : 1) * Lay::K_BYTES, full);
                if (!trans) tma_load_3d(dst + Lay::V, &tmV, h * P, (cb + c) * C, b, full);
                if constexpr (kFull) {
                    bulk_load(dst + Lay::T, src, kDlBlob, full);
                } else {
                    bulk_load(dst + Lay::T, src, 2 * kDlTile, full);
                    bulk_load(dst + Lay::VEC, src + 3 * kDlTile, kDlVec, full);
                }
            }
        };
        static_assert(Lay::V - Lay::T == kDlBlob, "T, M and the vectors lie as in the blob");
        int loaded = 0;
        if (nf == 0)
            for (; loaded < min(nC, ST); ++loaded) load_chunk(loaded, loaded);
        else if (nC > 0)
            load_chunk(loaded++, 0);                      // the other stages hold the transitions first
        constexpr uint32_t kId64 = umma_idesc_f16(128, 64, 0, 0);    // B K-major: K', Q', T, M rows
        constexpr uint32_t kId32 = umma_idesc_f16(128, 32, 0, 0);
        constexpr uint32_t kIdS = umma_idesc_f16(128, 64, 0, 1);      // B: K' rows as the K dimension (MN-major)
        // matrix descriptors of the first stage; an offset within shared memory
        // adds to their address field, so a step costs one addition
        const uint64_t d_k = umma_desc(sb + Lay::K, 16, 1024), d_ks = umma_desc(sb + Lay::K, 8192, 1024);
        auto at = [](uint64_t desc, int bytes) { return desc + (uint64_t)(bytes >> 4); };
        auto rows = [](int ks) { return (ks >> 2) * 8192 + (ks & 3) * 32; };     // K step ks of a 64-row tile
        const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
        bool ok = true;
        int folds = 0;                                    // transitions loaded
        if constexpr (kFull) {
            constexpr uint32_t kIdT = umma_idesc_f16(128, N, 0, 1);
            const unsigned char* tr = p.tr + ((size_t)b * d.H + h) * 2 * Lay::TR_BYTES;
            const size_t step = (size_t)d.B * d.H * 2 * Lay::TR_BYTES;
            auto load_tr = [&](int j) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar(Lay::TR_FULL + (j & 1)), 2 * Lay::TR_BYTES);
                    bulk_load(sb + (1 + (j & 1)) * Lay::STAGE, tr + j * step, 2 * Lay::TR_BYTES, bar(Lay::TR_FULL + (j & 1)));
                }
            };
            if (nf > 0) { load_tr(0); folds = 1; }
            for (int j = 0; j < nf; ++j) {                // S M: hi hi, lo hi, hi lo
                if (!(ok = delta_wait(bar(Lay::TR_FULL + (j & 1)), j >> 1, dead) && delta_wait(bar(Lay::S_IN), j, dead))) break;
                tc_fence_after();
                if (j + 1 < nf) { load_tr(j + 1); ++folds; }      // the product that read that stage is done
                const uint64_t t_d = umma_desc(sb + (1 + (j & 1)) * Lay::STAGE, N * 128, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 3 * KS; ++ks)
                        umma_ts(tb + Lay::XK, tb + (ks / KS == 1 ? Lay::S_LO : Lay::S_HI) + 8 * (ks % KS),
                                at(t_d, (ks / KS == 2 ? Lay::TR_BYTES : 0) + (ks % KS) * 2048), kIdT, ks > 0);
                    umma_commit(bar(Lay::D));
                }
            }
            if (nf > 0 && ok) {
                ok = delta_wait(bar(Lay::D), nf - 1, dead);
                if (ok)
                    for (; loaded < min(nC, ST); ++loaded) load_chunk(loaded, loaded);
            }
        }
        for (int c = 0, st = 0, use = 0; c < nC && ok; ++c) {
            const uint64_t k_d = d_k + (uint64_t)(st * (Lay::STAGE >> 4)), ks_d = d_ks + (uint64_t)(st * (Lay::STAGE >> 4));
            if (!(ok = delta_wait(bar(Lay::FULL + st), use, dead) && delta_wait(bar(Lay::S_IN), nf + c, dead))) break;
            tc_fence_after();
            if (elect_one()) {                            // K S^T, both parts of S, 32 tokens at a time
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int ks = 0; ks < 2 * KS; ++ks)
                        umma_ts(tb + Lay::XK + 32 * half, tb + (ks / KS) * Lay::S_LO + 8 * (ks % KS),
                                at(k_d, 4096 * half + rows(ks % KS)), kId32, ks > 0);
                    umma_commit(bar(Lay::X_K0 + half));
                }
            }
            if constexpr (kFull) {
                if (!(ok = c == 0 || delta_wait(bar(Lay::Y_OUT), c - 1, dead))) break;
                tc_fence_after();
                if (elect_one()) {                            // Q S^T, both parts of S
#pragma unroll
                    for (int ks = 0; ks < 2 * KS; ++ks)
                        umma_ts(tb + Lay::XQ, tb + (ks / KS) * Lay::S_LO + 8 * (ks % KS), at(k_d, Lay::Q + rows(ks % KS)),
                                kId64, ks > 0);
                    umma_commit(bar(Lay::X_Q));
                }
            }
            // chunk c - 1 is done with its stage: its increment and its Y have been read
            if (c > 0 && loaded < nC) {
                load_chunk(loaded, st == 0 ? ST - 1 : st - 1);
                ++loaded;
            }
            if (!(ok = delta_wait(bar(Lay::R_IN0), c, dead))) break;
            tc_fence_after();
            if (elect_one()) {                            // U = T R, R's first half: hi hi, lo hi (R lo), hi lo (T lo)
#pragma unroll
                for (int ks = 0; ks < 6; ++ks) {
                    const int q = ks & 1, part = ks >> 1;
                    umma_ts(tb + Lay::U, tb + Lay::R + (part & 1) * 8 + 16 * q, at(k_d, Lay::T + (part >> 1) * kDlTile + q * 32),
                            kId64, ks > 0);
                }
                umma_commit(bar(Lay::U_0));
            }
            if (!(ok = delta_wait(bar(Lay::R_IN1), c, dead))) break;
            tc_fence_after();
            if (elect_one()) {                            // its second half, for the later 32 tokens
#pragma unroll
                for (int ks = 0; ks < 6; ++ks) {
                    const int q = ks & 1, part = ks >> 1;
                    umma_ts(tb + Lay::U + 32, tb + Lay::R + 32 + (part & 1) * 8 + 16 * q,
                            at(k_d, Lay::T + (part >> 1) * kDlTile + 4096 + 64 + q * 32), kId32, 1);
                }
                umma_commit(bar(Lay::U_1));
            }
            // the increment goes where S is: Q S^T has to be done with it
            if (!(ok = (!kFull || delta_wait(bar(Lay::X_Q), c, dead)) && delta_wait(bar(Lay::U_IN0), c, dead))) break;
            tc_fence_after();
            auto increment = [&](int half, int n) {       // U_w^T K, n .. n + 63, 16 tokens a step, hi and lo
#pragma unroll
                for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                    umma_ts(tb + Lay::DD + n, tb + Lay::UW + 8 * ks, at(ks_d, n * 128 + (ks >> 1) * 2048), kIdS, ks > 0);
            };
            if (elect_one()) {
                increment(0, 0);
                if (N == 128) increment(0, 64);
            }
            if (!(ok = delta_wait(bar(Lay::U_IN1), c, dead))) break;
            tc_fence_after();
            if (elect_one()) {
                increment(1, 0);
                umma_commit(bar(Lay::D));                 // the first half of the state's threads can go on
                if (N == 128) {
                    increment(1, 64);
                    umma_commit(bar(Lay::D_HI));
                }
                if constexpr (kFull) {
                    // M U, where U was: hi hi and hi lo (U lo), then lo hi from where M lo's blocks lie
#pragma unroll
                    for (int k2 = 0; k2 < 8; ++k2) {
                        const int ks = k2 & 3;
                        umma_ts(tb + Lay::U + (ks >> 1) * 32, tb + Lay::UH + 16 * ks + 8 * (k2 >> 2),
                                at(k_d, Lay::M + (ks >> 1) * 4096 + ks * 32), ks < 2 ? kId64 : kId32, k2 > 0);
                    }
#pragma unroll
                    for (int k2 = 0; k2 < 6; ++k2) {
                        const int blk = k2 >> 1, q = k2 & 1;          // (0, 0), (32, 0), (32, 32)
                        umma_ts(tb + Lay::U + (blk > 0) * 32, tb + Lay::UH + 16 * (2 * (blk >> 1) + q),
                                at(k_d, (blk == 2 ? Lay::M : Lay::T + blk * kDlTile) + 64 + q * 32), kId32, 1);
                    }
                    umma_commit(bar(Lay::Y_M));
                }
            }
            if (++st == ST) { st = 0; ++use; }
        }
        if (!ok) {
            // copies in flight end before the block does (bounded waits); for products see the end
            for (int i = max(0, loaded - ST); i < loaded; ++i) mbar_wait(bar(Lay::FULL + i % ST), (uint32_t)(i / ST) & 1);
            for (int i = max(0, folds - 2); i < folds; ++i) mbar_wait(bar(Lay::TR_FULL + (i & 1)), (uint32_t)(i >> 1) & 1);
        }
        __syncwarp();
    } else if (w == 17) {
        // ---------------- the largest |v| of each column (bf16 bits order like their values), and theta
        constexpr int PW = P / 64;                        // words (column pairs) a lane
        for (int c = 0, st = 0, use = 0; c < nC && !trans; ++c) {
            const int rows = min(C, len - (cb + c) * C);
            const __nv_bfloat16* bp = static_cast<const __nv_bfloat16*>(d.b_raw) + ((size_t)b * d.L + (cb + c) * C + lane) * d.H + h;
            float bm = fmaxf(lane < rows ? IoBF16::load(bp) : -INFINITY, lane + 32 < rows ? IoBF16::load(bp + (size_t)32 * d.H) : -INFINITY);
            if (!delta_wait(bar(Lay::FULL + st), use, dead)) break;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(sm + st * Lay::STAGE + Lay::V) + lane * PW;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
            const float theta = pow2i(theta_exp(bm));
            uint32_t m[PW];
#pragma unroll
            for (int i = 0; i < PW; ++i) m[i] = 0;
#pragma unroll 8
            for (int t = 0; t < rows; ++t)
#pragma unroll
                for (int i = 0; i < PW; ++i) m[i] = __vmaxu2(m[i], v[t * (P / 2) + i] & 0x7fff7fffu);
            float* vm = reinterpret_cast<float*>(sm + Lay::VM + st * Lay::VMS);
#pragma unroll
            for (int i = 0; i < PW; ++i)
                *reinterpret_cast<float2*>(vm + 2 * PW * lane + 2 * i) = make_float2(theta * bf16_lo(m[i]), theta * bf16_hi(m[i]));
            if (lane == 0) vm[P] = theta;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Lay::VMAX + st));
            if (++st == ST) { st = 0; ++use; }
        }
    } else if ((w & 3) < lanes / 32) {
        // ---------------- four threads a value column
        const int part = w >> 2, v = 32 * (w & 3) + lane;
        constexpr int NQ = N / 4;                         // states of a thread: n = NQ part ..
        const uint32_t tl = tbase + ((uint32_t)(32 * (w & 3)) << 16);
        float2 S[NQ / 2];                                 // lambda times its part of the state row
        float lam = 1.f;                                  // the lane's scale, a power of two
        auto inverse = [](float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); };   // of a power of two: exponents swapped
        const size_t hoff = (((size_t)b * d.H + h) * P + v) * N + NQ * part;
        const size_t hstep = (size_t)d.B * d.H * P * N;   // floats between segments in sloc
        const float* from = seg == 0 ? (kFull && p.h0c ? p.h0c : d.h0) : kFull ? p.sloc : nullptr;
#pragma unroll
        for (int n = 0; n < NQ; n += 4) {
            float4 x = from ? *reinterpret_cast<const float4*>(from + hoff + n) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (!kFull && trans) {                        // the identity
                const int e = v - NQ * part - n;
                x = make_float4(e == 0, e == 1, e == 2, e == 3);
            }
            S[n / 2] = make_float2(x.x, x.y);
            S[n / 2 + 1] = make_float2(x.z, x.w);
            if (!kFull && seg == 0 && p.h0c) *reinterpret_cast<float4*>(p.h0c + hoff + n) = x;
        }
        float* smax = reinterpret_cast<float*>(sm + Lay::SMAX) + v;
        auto arrive = [&](int i) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        // the largest |x| over the lane's four threads: told, then, once all have, read
        auto lane_max = [&](const float2 (&x)[NQ / 2], float& m) {
            m = 0.f;
#pragma unroll
            for (int n = 0; n < NQ / 2; ++n) m = max_abs3(m, x[n].x, x[n].y);
            smax[128 * part] = m;
            arrive(Lay::QUAD + (w & 3));
        };
        auto lane_max_wait = [&](int use, float& m) {
            if (!delta_wait(bar(Lay::QUAD + (w & 3)), use, dead)) return false;
            m = fmaxf(fmaxf(smax[0], smax[128]), fmaxf(smax[256], smax[384]));
            return true;
        };
        bool ok = true;
        if constexpr (kFull) {
            // ---- the state entering this segment: S M_j + S_loc,j over the segments before it
            const float* trs = p.trs + ((size_t)b * d.H + h) * N + NQ * part;
            for (int j = 0; j < nf; ++j) {
                float m;
#pragma unroll
                for (int n = 0; n < NQ; n += 4) {         // to units in which M_j's rows are kept
                    const float4 x = *reinterpret_cast<const float4*>(trs + (size_t)j * d.B * d.H * N + n);
                    S[n / 2] = __fmul2_rn(S[n / 2], make_float2(x.x, x.y));
                    S[n / 2 + 1] = __fmul2_rn(S[n / 2 + 1], make_float2(x.z, x.w));
                }
                lane_max(S, m);
                if (!(ok = lane_max_wait(j, m))) break;
                const int e = m > 0.f ? exp_above(m) : 0;
                const float f = pow2i(-e), back = pow2i(e);
#pragma unroll
                for (int n0 = 0; n0 < NQ / 2; n0 += 8) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) split_f16(__fmul2_rn(S[n0 + q], make_float2(f, f)), hi[q], lo[q]);
                    tmem_st8(tl + Lay::S_HI + NQ / 2 * part + n0, hi);
                    tmem_st8(tl + Lay::S_LO + NQ / 2 * part + n0, lo);
                }
                tmem_st_wait();
                arrive(Lay::S_IN);
                const float* loc = p.sloc + (size_t)(j + 1) * hstep + hoff;
#pragma unroll
                for (int n = 0; n < NQ; n += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(loc + n);
                    S[n / 2] = make_float2(x.x, x.y);
                    S[n / 2 + 1] = make_float2(x.z, x.w);
                }
                if (!(ok = delta_wait(bar(Lay::D), j, dead))) break;
                tc_fence_after();
#pragma unroll
                for (int n0 = 0; n0 < NQ; n0 += 16) {
                    float x[16];
                    tmem_ld16(tl + Lay::XK + NQ * part + n0, x);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        S[n0 / 2 + q] = __ffma2_rn(make_float2(back, back), make_float2(x[2 * q], x[2 * q + 1]), S[n0 / 2 + q]);
                }
            }
        }
        float yl = 0.f;                                   // what Y of the chunk before is in units of
        for (int c = 0, st = 0, use = 0; c <= nC && ok; ++c) {
            const unsigned char* sg = sm + st * Lay::STAGE;
            if (c < nC || trans) {
                // ---- the lane's scale for this chunk, S into the A operand's columns:
                // first in the scale it has, which mostly stands, else once more
                float m;
                lane_max(S, m);
                uint32_t hi[NQ / 2], lo[NQ / 2];
#pragma unroll 1
                for (bool again = false;; again = true) {
#pragma unroll
                    for (int q = 0; q < NQ / 2; ++q) split_f16(S[q], hi[q], lo[q]);
                    if (again) break;
                    // every thread of the lane has read its increment too; V and the vectors are here
                    if (!(ok = lane_max_wait(nf + c, m))) break;
                    float vm = 0.f;
                    if (trans) {
                        if (c < nC && !(ok = delta_wait(bar(Lay::FULL + st), use, dead))) break;
                    } else {
                        if (!(ok = delta_wait(bar(Lay::VMAX + st), use, dead))) break;
                        vm = reinterpret_cast<const float*>(sm + Lay::VM + st * Lay::VMS)[v];
                    }
                    const float both = fmaxf(m, lam * vm);    // infinite or 0 where the product leaves float's range
                    const bool out = both > 64.f || (both < 0.125f && (m > 0.f || vm > 0.f));
                    if (!__any_sync(0xffffffffu, out)) break;
                    const int l = exp_of(lam) - 1;            // by exponents, which stay in range
                    int e = 0;
                    if (out) e = max(m > 0.f ? exp_of(m) : -1000, vm > 0.f ? exp_of(vm) + l : -1000);
                    e = min(max(e, l - 126), l + 126);        // lambda and its inverse stay floats
                    lam = pow2i(l - e);
                    // beyond 2^126 S is 0 (up), or nothing beside V (down: below 2^-120 of it)
                    const float f = pow2i(-min(max(e, -126), 126));
#pragma unroll
                    for (int q = 0; q < NQ / 2; ++q) S[q] = __fmul2_rn(S[q], make_float2(f, f));
                }
                if (!ok) break;
                if (!kFull && c == nC) {                  // the segment's transition: row v, this thread's columns
                    const size_t at = ((size_t)(seg - 1) * d.B + b) * d.H + h;
                    unsigned char* tile = p.tr + at * 2 * Lay::TR_BYTES + (NQ * part / 64) * (N * 128) + v * 128;
#pragma unroll
                    for (int q = 0; q < NQ / 8; ++q) {
                        const int off = (((NQ * part / 8 + q) & 7) ^ (v & 7)) << 4;
                        *reinterpret_cast<uint4*>(tile + off) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                        *reinterpret_cast<uint4*>(tile + Lay::TR_BYTES + off) =
                            make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                    }
                    if (part == 0) p.trs[at * N + v] = inverse(lam);
                    break;
                }
#pragma unroll
                for (int n0 = 0; n0 < NQ / 2; n0 += 8) {
                    tmem_st8(tl + Lay::S_HI + NQ / 2 * part + n0, reinterpret_cast<uint32_t(&)[8]>(hi[n0]));
                    tmem_st8(tl + Lay::S_LO + NQ / 2 * part + n0, reinterpret_cast<uint32_t(&)[8]>(lo[n0]));
                }
                tmem_st_wait();
                arrive(Lay::S_IN);
            }
            // ---- y of chunk c - 1, while K S^T runs: 16 tokens a thread; neighbouring
            // lanes trade tokens, so a lane stores two columns of one token
            if (kFull && c > 0) {
                if (!(ok = delta_wait(bar(Lay::Y_M), c - 1, dead))) break;
                tc_fence_after();
                const int odd = lane & 1, t0 = (cb + c - 1) * C + 16 * part + odd, left = len - t0;
                const size_t ystep = 2 * (size_t)d.H * P;
                __nv_bfloat16* yo = static_cast<__nv_bfloat16*>(d.y) + (((size_t)b * d.L + t0) * d.H + h) * P + (v & ~1);
                // scale rq (e^Gamma Q S^T + M U), times what the lane is in units of
                const float* eg = reinterpret_cast<const float*>(sm + (st == 0 ? ST - 1 : st - 1) * Lay::STAGE + Lay::VEC) + C + 16 * part;
                float2 yv[8];
                {
                    float z[16];
                    tmem_ld16(tl + Lay::U + 16 * part, z);
#pragma unroll
                    for (int q0 = 0; q0 < 8; q0 += 4) {
                        float x[8];
                        tmem_ld8(tl + Lay::XQ + 16 * part + 2 * q0, x);
#pragma unroll
                        for (int q = q0; q < q0 + 4; q += 2) {
                            const float4 e = *reinterpret_cast<const float4*>(eg + 2 * q);
                            const float4 r = *reinterpret_cast<const float4*>(eg + 2 * C + 2 * q);
                            const float* xq = x + 2 * (q - q0);
                            yv[q] = __fmul2_rn(make_float2(r.x, r.y), __ffma2_rn(make_float2(e.x, e.y), make_float2(xq[0], xq[1]),
                                                                                 make_float2(z[2 * q], z[2 * q + 1])));
                            yv[q + 1] = __fmul2_rn(make_float2(r.z, r.w), __ffma2_rn(make_float2(e.z, e.w), make_float2(xq[2], xq[3]),
                                                                                     make_float2(z[2 * q + 2], z[2 * q + 3])));
                        }
                    }
                }
                arrive(Lay::Y_OUT);
                uint32_t o[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float2 a = __fmul2_rn(yv[q], make_float2(yl, yl));
                    const uint32_t mine = pack_bf16(a.x, a.y);
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
                    o[q] = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
                }
                if (!d.norm) {
                    uint32_t big = 0;                     // bf16 bits order like their values, infinity and NaN last
#pragma unroll
                    for (int q = 0; q < 8; ++q) big = __vmaxu2(big, o[q] & 0x7fff7fffu);
                    if ((big & 0xffffu) >= 0x7f80u || big >> 16 >= 0x7f80u) atomicOr(p.err, 2);
                }
                if (len - (cb + c - 1) * C >= C) {        // no token of the chunk is missing
#pragma unroll
                    for (int q = 0; q < 8; ++q) *reinterpret_cast<uint32_t*>(yo + q * ystep) = o[q];
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (2 * q < left) *reinterpret_cast<uint32_t*>(yo + q * ystep) = o[q];
                }
            }
            if (c == nC) break;
            const float* vec = reinterpret_cast<const float*>(sg + Lay::VEC);
            const unsigned short* sv = reinterpret_cast<const unsigned short*>(sg + Lay::V) + v;
            const float theta = trans ? 1.f : reinterpret_cast<const float*>(sm + Lay::VM + st * Lay::VMS)[P];
            const unsigned short lamb = (unsigned short)(__float_as_uint(lam * theta) >> 16);     // a power of two: exact
            const int rows = trans ? 0 : len - (cb + c) * C;      // tokens behind them write nothing
            yl = inverse(lam);
            // ---- R = theta (V - e^Gamma rk K S^T), 8 tokens of each half a thread
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int t0 = 32 * half + 8 * part;
                unsigned short vt[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) vt[q] = rows > 0 ? sv[(t0 + q) * P] : 0;
                if (t0 + 8 > rows) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (t0 + q >= rows) vt[q] = 0;
                }
                if (!(ok = delta_wait(bar(Lay::X_K0 + half), c, dead))) break;
                tc_fence_after();
                float x[8];
                tmem_ld8(tl + Lay::XK + t0, x);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 8; q += 4) {
                    const float4 ek = *reinterpret_cast<const float4*>(vec + t0 + q);
                    float2 a = __fmul2_rn(make_float2(ek.x, ek.y), make_float2(x[q], x[q + 1]));
                    float2 e = __fmul2_rn(make_float2(ek.z, ek.w), make_float2(x[q + 2], x[q + 3]));
                    a.x = fma_bf16(vt[q + 0], lamb, a.x);
                    a.y = fma_bf16(vt[q + 1], lamb, a.y);
                    e.x = fma_bf16(vt[q + 2], lamb, e.x);
                    e.y = fma_bf16(vt[q + 3], lamb, e.y);
                    split_f16(a, hi[q / 2], lo[q / 2]);
                    split_f16(e, hi[q / 2 + 1], lo[q / 2 + 1]);
                }
                const uint32_t r = tl + Lay::R + 32 * half + 16 * (part >> 1) + 4 * (part & 1);
                tmem_st4(r, hi);
                tmem_st4(r + 8, lo);
                tmem_st_wait();
                arrive(Lay::R_IN0 + half);
            }
            if (!ok) break;
            // ---- U for Y, and weighted for the state
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (!(ok = delta_wait(bar(Lay::U_0 + half), c, dead))) break;
                tc_fence_after();
                const int t0 = 32 * half + 8 * part;
                float x[8];
                tmem_ld8(tl + Lay::U + t0, x);
                uint32_t hi[4], lo[4];
                const uint32_t to = 32 * half + 16 * (part >> 1) + 4 * (part & 1);
                if constexpr (kFull) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) split_f16(make_float2(x[2 * q], x[2 * q + 1]), hi[q], lo[q]);
                    tmem_st4(tl + Lay::UH + to, hi);
                    tmem_st4(tl + Lay::UH + to + 8, lo);
                }
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const float4 wk = *reinterpret_cast<const float4*>(vec + 2 * C + t0 + 2 * q);
                    split_f16(__fmul2_rn(make_float2(x[2 * q], x[2 * q + 1]), make_float2(wk.x, wk.y)), hi[q], lo[q]);
                    split_f16(__fmul2_rn(make_float2(x[2 * q + 2], x[2 * q + 3]), make_float2(wk.z, wk.w)), hi[q + 1], lo[q + 1]);
                }
                tmem_st4(tl + Lay::UW + to, hi);
                tmem_st4(tl + Lay::UW + to + 8, lo);
                tmem_st_wait();
                arrive(Lay::U_IN0 + half);
            }
            if (!ok) break;
            // ---- the state after the chunk
            const float el = vec[2 * C - 1];              // e^Gamma of the last token
            const float2 el2 = make_float2(el, el);
            if (!(ok = N == 128 && part >= 2 ? delta_wait(bar(Lay::D_HI), c, dead) : delta_wait(bar(Lay::D), nf + c, dead))) break;
            tc_fence_after();
            if constexpr (NQ == 32) {
                uint32_t x[32];
                tmem_ld32_async(tl + Lay::DD + NQ * part, x);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    S[q] = __ffma2_rn(el2, S[q], make_float2(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1])));
            } else {
                float x[16];
                tmem_ld16(tl + Lay::DD + NQ * part, x);
#pragma unroll
                for (int q = 0; q < 8; ++q) S[q] = __ffma2_rn(el2, S[q], make_float2(x[2 * q], x[2 * q + 1]));
            }
            if (++st == ST) { st = 0; ++use; }
        }
        // the end state: of the segment, or, where the row ends in it, of the row
        float* to = kFull ? (cb + max(nC, 0) == all ? d.h_out : nullptr) : trans ? nullptr : p.sloc + seg * hstep;
        if (ok && to) {
            const float ilam = inverse(lam);
            if (kFull && !d.norm) {
                uint32_t big = 0;
#pragma unroll
                for (int n = 0; n < NQ / 2; ++n)
                    big = max(big, max(__float_as_uint(S[n].x) & 0x7fffffffu, __float_as_uint(S[n].y) & 0x7fffffffu));
                if (big >= 0x7f800000u) atomicOr(p.err, 2);
            }
#pragma unroll
            for (int n = 0; n < NQ; n += 4)
                *reinterpret_cast<float4*>(to + hoff + n) =
                    make_float4(S[n / 2].x * ilam, S[n / 2].y * ilam, S[n / 2 + 1].x * ilam, S[n / 2 + 1].y * ilam);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 16) {
        bool drained = !*dead;                            // else some wait gave up, in this warp or another
        if (!drained) drained = delta_drain(bar(Lay::DRAIN), p.err);
        if (drained) tmem_dealloc(tbase, Lay::COLS);      // a late product must not meet another block's columns
    }
}

}  // namespace axon
