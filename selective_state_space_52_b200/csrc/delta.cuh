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
// Everything in the walk is kept transposed, so that a tensor-memory lane is
// one value column v (M = 128 lanes): S^T row v, R^T, U^T and Y^T rows are all
// in lane v and belong to one thread, which holds the float32 state row in
// registers.  No value ever crosses a lane; the A operands are what the thread
// itself writes to its lane, and the B operands are the tiles K, Q, T, M as
// they lie in shared memory.
//
// Precision.  Operands are fp16 with float32 accumulators.  K and Q enter
// scaled by a power of two per token (largest element in [1/2, 1)): exact, but
// for bits below 2^-25 of the row.  S, R, U (for the state) and T enter as two
// fp16 parts, hi + lo, 22 significant bits; the lo x lo term is dropped.  fp16
// needs values near 1, so each lane carries a power-of-two scale lambda_v: all
// of the walk is linear in lane v, so S, R, U and Y simply live in units of
// 1 / lambda_v; a lane rescales when its largest value leaves [2^-3, 2^6].
// Two bf16 parts (no scale needed) measured 4.5e-6 on the final state in a
// float64 model of these roundings, fp16 parts about 1e-7: the state is a
// float32 output, and the product count is the same.  Y takes one fp16 part of
// S, U and M (2^-12 each, below its bf16 rounding).
#pragma once

#include <cuda_bf16.h>

#include "delta_step.cuh"
#include "device_math.cuh"
#include "tc_ops.cuh"

namespace axon {

constexpr int kDlC = 64;                       // tokens per chunk
constexpr int kDlTile = kDlC * kDlC * 2;       // a 64 x 64 fp16 tile: 8 KB
constexpr int kDlVec = 4 * kDlC * 4;           // ek, eG, wk, oq
constexpr int kDlBlob = 3 * kDlTile + kDlVec;  // per chunk and value head: T hi, T lo, M, vectors

struct DeltaChunkParams {
    DeltaParams d;
    int nC;                      // chunks of L
    unsigned char* kq;           // (B, G, nC): [K'; Q'] fp16, 128 rows in 64-column blocks, 128-byte swizzle
    unsigned char* blob;         // (B, H, nC): kDlBlob bytes
    int* err;                    // set to 1 when a wait gave up
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
// x - (the fp16 in the low / high half of h), float32
__device__ __forceinline__ float f16_rest_lo(uint32_t h, float x) {
    float d;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tsub.f32.f16 %0, a, %2;\n\t}" : "=f"(d) : "r"(h), "f"(x));
    return -d;
}
__device__ __forceinline__ float f16_rest_hi(uint32_t h, float x) {
    float d;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tsub.f32.f16 %0, b, %2;\n\t}" : "=f"(d) : "r"(h), "f"(x));
    return -d;
}
// a pair as hi + lo fp16 parts
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_f16(a, b);
    lo = pack_f16(f16_rest_lo(hi, a), f16_rest_hi(hi, b));
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
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }    // -126 <= e <= 127

// Rows' largest magnitude m > 0: the exponent e with m 2^-e in [1/2, 1),
// held to what a float power of two and its inverse can say.
__device__ __forceinline__ int exp_above(float m) {
    const int e = (int)((__float_as_uint(m) >> 23) & 255u) - 126;
    return min(max(e, -100), 100);
}

// ---- prep: grid = (nC, G, B), 128 threads
template <int N>
struct DeltaPrepSmem {
    static constexpr int LDA = 68;                       // floats a row of A: 16-byte rows without bank conflicts
    static constexpr int KQ = 0;                         // [K'; Q'] tile, read by the Gram products only ...
    static constexpr int A = 0;                          // ... then A (float32), later the T parts over it
    static constexpr int M = kDlC * LDA * 4;             // M tile
    static constexpr int KQ_BYTES = 128 * N * 2;
    static constexpr int V = KQ_BYTES > M + kDlTile ? KQ_BYTES : M + kDlTile;   // vectors ek, eG, wk, oq
    static constexpr int RK = V + kDlVec;                // rk'
    static constexpr int RQ = RK + kDlC * 4;             // scale rq'
    static constexpr int GH = RQ + kDlC * 4;             // Gamma (log2 units), float hi and lo parts
    static constexpr int GL = GH + kDlC * 4;
    static constexpr int BE = GL + kDlC * 4;             // beta
    static constexpr int TOT = BE + kDlC * 4;            // double: the first warp's total
    static constexpr int MB = TOT + 8;
    static constexpr int SLOT = MB + 8;
    static constexpr int BYTES = SLOT + 8;
    static constexpr int TOTAL = BYTES + 1024;           // with the alignment pad
    static_assert(2 * kDlTile <= M, "the T parts fit over A");
    static_assert(M % 16 == 0 && V % 16 == 0 && TOT % 8 == 0, "alignment");
};

// Column j of (I + A)^-1 for the lanes of warps 0 and 1 (j = tid): forward
// substitution down the rows, two products per instruction; A rows are read
// as broadcasts.  Columns of warp 1 are zero above row 32.
__device__ __forceinline__ void delta_invert_column(const float* A, int lda, int j, bool low, float2 (&t)[kDlC / 2]) {
#pragma unroll
    for (int i = 0; i < kDlC / 2; ++i) t[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kDlC; ++i) {
        float2 acc = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        const float* row = A + i * lda;
        if (low || i >= 32) {
            // pairs (k, k + 1) with k < i; A_ii is 0 and the t behind row i are still 0
            if (low) {
#pragma unroll
                for (int k = 0; k < (i < 32 ? i : 32); k += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(row + k);
                    acc = __ffma2_rn(make_float2(a.x, a.y), t[k / 2], acc);
                    if (k + 2 < i) acc1 = __ffma2_rn(make_float2(a.z, a.w), t[k / 2 + 1], acc1);
                }
            }
#pragma unroll
            for (int k = 32; k < i; k += 4) {
                const float4 a = *reinterpret_cast<const float4*>(row + k);
                acc = __ffma2_rn(make_float2(a.x, a.y), t[k / 2], acc);
                if (k + 2 < i) acc1 = __ffma2_rn(make_float2(a.z, a.w), t[k / 2 + 1], acc1);
            }
            const float v = (i == j ? 1.f : 0.f) - ((acc.x + acc.y) + (acc1.x + acc1.y));
            if (i & 1) t[i / 2].y = v;
            else t[i / 2].x = v;
        }
    }
}

template <int N>
__global__ void __launch_bounds__(128) delta_prep_kernel(DeltaChunkParams p) {
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
    if (w == 0) tmem_alloc(sb + Lay::SLOT, 64);
    if (tid == 0) mbar_init(sb + Lay::MB, 1);

    // ---- rows of K (tile rows 0 .. 63) and Q (64 .. 127): eight lanes a row,
    // its largest element to [1/2, 1), fp16 into the tile and to global memory
    {
        constexpr int PC = N / 64;                       // 16-byte pieces of a lane
        const int l = tid & 7, r0 = tid >> 3;
        const __nv_bfloat16* base[2] = {
            static_cast<const __nv_bfloat16*>(d.k) + (size_t)b * d.L * d.ldk + (size_t)g * N,
            static_cast<const __nv_bfloat16*>(d.q) + (size_t)b * d.L * d.ldq + (size_t)g * N};
        const int ld[2] = {d.ldk, d.ldq};
        uint4 v[8][PC];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = r0 + 16 * k, t = t0 + (r & 63), s = k >> 2;
#pragma unroll
            for (int i = 0; i < PC; ++i)
                v[k][i] = t < len ? __ldg(reinterpret_cast<const uint4*>(base[s] + (size_t)t * ld[s]) + l + 8 * i)
                                  : make_uint4(0, 0, 0, 0);
        }
        unsigned char* out = p.kq + (((size_t)b * d.G + g) * p.nC + c) * Lay::KQ_BYTES;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = r0 + 16 * k;
            float m = 0.f;
            float f[PC][8];
#pragma unroll
            for (int i = 0; i < PC; ++i) {
                const uint32_t u[4] = {v[k][i].x, v[k][i].y, v[k][i].z, v[k][i].w};
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
                const int pc = l + 8 * i;
                const int off = (pc >> 3) * 16384 + r * 128 + (((pc & 7) ^ (r & 7)) << 4);
                const uint4 o = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(sm + Lay::KQ + off) = o;
                *reinterpret_cast<uint4*>(out + off) = o;
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (l == 0) {
                // 1 / sqrt(|k|^2 + eps) in the scaled row's units: |k|^2 = ss 4^e
                const float es = pow2i(e);
                const float f1 = d.norm ? es * rsqrtf(fmaf(ss * es, es, kDeltaEps)) : es;
                if (r < C) rk[r] = f1;
                else rq[r - C] = d.scale * f1;
            }
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(sm + Lay::SLOT);
    if (tid == 0) {
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) {
            const uint64_t dsc = umma_desc(sb + Lay::KQ + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
            umma(tbase, dsc, dsc, umma_idesc_f16(128, C, 0, 0), ks > 0);      // [K'; Q'] K'^T
        }
        umma_commit(sb + Lay::MB);
    }
    const bool ok = mbar_wait(sb + Lay::MB, 0u);
    const bool failed = __syncthreads_or(!ok);           // KQ is free from here on: A and M lie over it
    tc_fence_after();
    if (failed && tid == 0) atomicExch(p.err, 1);

    const int r = d.H / d.G;
    const int i = tid & 63;                              // this thread's row of A (warps 0, 1) or M (2, 3)
    const bool live = t0 + i < len;
    float* vec = reinterpret_cast<float*>(sm + Lay::V);
    float* gh = reinterpret_cast<float*>(sm + Lay::GH);
    float* gl = reinterpret_cast<float*>(sm + Lay::GL);
    float* be = reinterpret_cast<float*>(sm + Lay::BE);
    float* A = reinterpret_cast<float*>(sm + Lay::A);
    for (int hh = 0; hh < r && !failed; ++hh) {
        const int h = g * r + hh;
        // ---- rates: warps 0 and 1, a token a lane.  The running log decay is
        // summed in double: it reaches hundreds, and differences of neighbours count.
        double G = 0.0;
        if (w < 2) {
            float lg = 0.f, beta = 0.f;
            if (live) {
                const size_t o = ((size_t)b * d.L + t0 + i) * d.H + h;
                lg = delta_log2_decay(IoBF16::load(static_cast<const __nv_bfloat16*>(d.dt_raw) + o) + __ldg(d.dt_bias + h),
                                      delta_exp_a(__ldg(d.A_log + h)));
                // a decay below 2^-2000 is 0 to a float anyway, and an infinite one would leave inf - inf
                lg = lg < -2000.f ? -2000.f : lg;
                beta = delta_beta(IoBF16::load(static_cast<const __nv_bfloat16*>(d.b_raw) + o));
            }
            G = (double)lg;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, G, o);
                if (lane >= o) G += v;
            }
            if (tid == 31) *reinterpret_cast<double*>(sm + Lay::TOT) = G;
            be[i] = beta;
        }
        __syncthreads();
        if (w < 2) {
            if (w == 1) G += *reinterpret_cast<double*>(sm + Lay::TOT);
            const float hi = (float)G;
            gh[i] = hi;
            gl[i] = (float)(G - (double)hi);
        }
        __syncthreads();
        const float ghi = gh[i], glo = gl[i];
        if (w < 2) {
            const float eg = ex2_approx(ghi);
            vec[i] = eg * rk[i];
            vec[C + i] = eg;
            vec[2 * C + i] = ex2_approx((gh[C - 1] - ghi) + (gl[C - 1] - glo)) * rk[i];
            vec[3 * C + i] = rq[i];
        }
        // ---- row i of A, or of M
        const float f = w < 2 ? be[i] * rk[i] : 1.f;
        const int edge = w < 2 ? i : i + 1;              // columns below it belong to the triangle
#pragma unroll
        for (int j0 = 0; j0 < C; j0 += 16) {
            float x[16];
            if (j0 <= ((w & 1) << 5) + 31) {             // warp-uniform: some row of the warp reaches these columns
                tmem_ld16(tbase + ((uint32_t)(32 * w) << 16) + j0, x);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int j = j0 + q;
                    const float e = ex2_approx((ghi - gh[j]) + (glo - gl[j]));
                    x[q] = j < edge ? x[q] * f * (e * rk[j]) : 0.f;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; ++q) x[q] = 0.f;
            }
            if (w < 2) {
#pragma unroll
                for (int q = 0; q < 16; q += 4)
                    *reinterpret_cast<float4*>(A + i * Lay::LDA + j0 + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int pc = j0 / 8 + q;
                    *reinterpret_cast<uint4*>(sm + Lay::M + i * 128 + ((pc ^ (i & 7)) << 4)) =
                        make_uint4(pack_f16(x[8 * q], x[8 * q + 1]), pack_f16(x[8 * q + 2], x[8 * q + 3]),
                                   pack_f16(x[8 * q + 4], x[8 * q + 5]), pack_f16(x[8 * q + 6], x[8 * q + 7]));
                }
            }
        }
        __syncthreads();
        // ---- T = (I + A)^-1 diag(beta): column j = tid, then its parts over A
        float2 t[C / 2];
        if (w < 2) delta_invert_column(A, Lay::LDA, tid, w == 0, t);
        __syncthreads();
        if (w < 2) {
            const float bj = be[tid];
            const int odd = lane & 1;
#pragma unroll
            for (int q = 0; q < C / 2; ++q) {            // rows 2q, 2q + 1: neighbouring lanes trade halves
                uint32_t hi, lo;
                split_f16(t[q].x * bj, t[q].y * bj, hi, lo);
                const uint32_t oh = __shfl_xor_sync(0xffffffffu, hi, 1), ol = __shfl_xor_sync(0xffffffffu, lo, 1);
                const int row = 2 * q + odd;
                const int off = row * 128 + ((((tid & ~1) >> 3) ^ (row & 7)) << 4) + (tid & 6) * 2;
                *reinterpret_cast<uint32_t*>(sm + Lay::A + off) = odd ? __byte_perm(oh, hi, 0x7632) : __byte_perm(hi, oh, 0x5410);
                *reinterpret_cast<uint32_t*>(sm + Lay::A + kDlTile + off) =
                    odd ? __byte_perm(ol, lo, 0x7632) : __byte_perm(lo, ol, 0x5410);
            }
        }
        __syncthreads();
        // ---- the blob: T hi, T lo, M, vectors (16-byte pieces, coalesced)
        uint4* blob = reinterpret_cast<uint4*>(p.blob + (((size_t)b * d.H + h) * p.nC + c) * kDlBlob);
#pragma unroll
        for (int k = 0; k < 2 * kDlTile / 16 / 128; ++k)
            blob[tid + 128 * k] = *reinterpret_cast<const uint4*>(sm + Lay::A + (tid + 128 * k) * 16);
#pragma unroll
        for (int k = 0; k < kDlTile / 16 / 128; ++k)
            blob[2 * kDlTile / 16 + tid + 128 * k] = *reinterpret_cast<const uint4*>(sm + Lay::M + (tid + 128 * k) * 16);
        if (tid < kDlVec / 16) blob[3 * kDlTile / 16 + tid] = *reinterpret_cast<const uint4*>(sm + Lay::V + tid * 16);
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 0 && !failed) tmem_dealloc(tbase, 64);      // after a failed wait a late product might still write
}

// ---- the walk: grid = (H, B), 160 threads; warps 0 .. P/32 - 1 compute (thread =
// tensor-memory lane = value column), warp 4 copies tiles in and issues products
constexpr int kDlThreads = 160;

template <int N, int P>
struct DeltaWalkSmem {
    static constexpr int KQ_BYTES = 128 * N * 2;
    static constexpr int KQ = 0;                          // two stages
    static constexpr int T = KQ + 2 * KQ_BYTES;           // T hi, T lo
    static constexpr int M = T + 2 * kDlTile;
    static constexpr int V = M + kDlTile;                 // 64 rows of P bf16
    static constexpr int VEC = V + kDlC * P * 2;          // two stages
    static constexpr int MB = VEC + 2 * kDlVec;
    enum { FULL_KQ0, FULL_KQ1, FULL_V, FULL_T, FULL_M, X_K, X_Q, UR, YM, D_A, D_B, S_IN, R_IN, U_IN, Y_OUT, DRAIN, BARS };
    static constexpr int DEAD = MB + 8 * BARS;            // a wait gave up
    static constexpr int SLOT = DEAD + 4;
    static constexpr int BYTES = SLOT + 4;
    static constexpr int TOTAL = BYTES + 1024;
    // tensor memory (256 columns): S hi 0 .. 63, S lo 64 .. 127, K S^T 128 .. 191, Q S^T 192 .. 255;
    // then R hi 64 .. 95, lo 96 .. 127; U 0 .. 63; U_w hi and lo over R, U hi 160 .. 191; Y over Q S^T;
    // the state's increment 0 .. 63 and (n >= 64) 128 .. 191
    static constexpr int COLS = 256;
};

// The warp polls an mbarrier's phase; gives up after a bounded number of
// polls, or when another warp of the block has.  The same answer in every lane.
__device__ __forceinline__ bool delta_wait(uint32_t mbar, int use, volatile int* dead) {
    bool ok = false;
    for (int k = 0; k < 4096 && !ok; ++k) {
        ok = mbar_wait(mbar, (uint32_t)(use & 1), kTcWaitLimit / 4096);
        if (!ok && *dead) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *dead = 1;
    return ok;
}

template <int N, int P>
__global__ void __launch_bounds__(kDlThreads, 2) delta_walk_kernel(DeltaChunkParams p) {
    using Lay = DeltaWalkSmem<N, P>;
    constexpr int C = kDlC, WARPS = P / 32, KS = N / 16;
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
    const int nC = (len + C - 1) / C;
    const int g = h / (d.H / d.G);
    volatile int* dead = reinterpret_cast<volatile int*>(sm + Lay::DEAD);
    auto bar = [&](int i) { return sb + Lay::MB + 8 * i; };

    if (tid == 0) {
        for (int i = 0; i < Lay::BARS; ++i)
            mbar_init(bar(i), i >= Lay::S_IN && i <= Lay::Y_OUT ? WARPS : 1);
        *dead = 0;
        fence_mbar_init();
    }
    grid_dep_wait();                                      // the prep kernel's tiles are written
    fence_proxy_async();
    // only now, or these columns might keep a prep block waiting that this one waits for
    if (w == 4) tmem_alloc(sb + Lay::SLOT, Lay::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(sm + Lay::SLOT);

    if (w == 4) {
        // ---------------- copies and products
        const unsigned char* kq = p.kq + ((size_t)b * d.G + g) * p.nC * Lay::KQ_BYTES;
        const unsigned char* blob = p.blob + ((size_t)b * d.H + h) * p.nC * kDlBlob;
        const __nv_bfloat16* vg = static_cast<const __nv_bfloat16*>(d.v) + (size_t)b * d.L * d.ldv + (size_t)h * P;
        auto load_kq = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Lay::FULL_KQ0 + (c & 1)), Lay::KQ_BYTES);
                bulk_load(sb + Lay::KQ + (c & 1) * Lay::KQ_BYTES, kq + (size_t)c * Lay::KQ_BYTES, Lay::KQ_BYTES,
                          bar(Lay::FULL_KQ0 + (c & 1)));
            }
        };
        auto load_v = [&](int c) {                        // the rows that exist, and the vectors
            const int rows = min(C, len - c * C);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Lay::FULL_V), rows * P * 2 + kDlVec);
                bulk_load(sb + Lay::VEC + (c & 1) * kDlVec, blob + (size_t)c * kDlBlob + 3 * kDlTile, kDlVec, bar(Lay::FULL_V));
            }
            __syncwarp();
            for (int r = lane; r < rows; r += 32)
                bulk_load(sb + Lay::V + r * P * 2, vg + (size_t)(c * C + r) * d.ldv, P * 2, bar(Lay::FULL_V));
        };
        auto load_t = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Lay::FULL_T), 2 * kDlTile);
                bulk_load(sb + Lay::T, blob + (size_t)c * kDlBlob, 2 * kDlTile, bar(Lay::FULL_T));
            }
        };
        auto load_m = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Lay::FULL_M), kDlTile);
                bulk_load(sb + Lay::M, blob + (size_t)c * kDlBlob + 2 * kDlTile, kDlTile, bar(Lay::FULL_M));
            }
        };
        int n_kq = 0, n_v = 0, n_t = 0, n_m = 0;          // copies issued
        if (nC > 0) {
            load_kq(0); load_v(0); load_t(0); load_m(0);
            n_kq = n_v = n_t = n_m = 1;
        }
        constexpr uint32_t kIdN = umma_idesc_f16(128, C, 0, 0);      // B K-major: K', Q', T, M rows
        constexpr uint32_t kIdS = umma_idesc_f16(128, 64, 0, 1);     // B: K' rows as the K dimension (MN-major)
        bool ok = true;
        for (int c = 0; c < nC && ok; ++c) {
            const uint32_t kt = sb + Lay::KQ + (c & 1) * Lay::KQ_BYTES, qt = kt + 8192;
            auto kdesc = [&](uint32_t t, int ks) { return umma_desc(t + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024); };
            ok = delta_wait(bar(Lay::FULL_KQ0 + (c & 1)), c >> 1, dead) && delta_wait(bar(Lay::S_IN), c, dead);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {                              // K S^T, both parts of S
#pragma unroll
                for (int ks = 0; ks < 2 * KS; ++ks)
                    umma_ts(tbase + 128, tbase + (ks / KS) * 64 + 8 * (ks % KS), kdesc(kt, ks % KS), kIdN, ks > 0);
                umma_commit(bar(Lay::X_K));
            }
            // the stage's last reader, the state product of chunk c - 1, is done (its increment has been read)
            if (c + 1 < nC) { load_kq(c + 1); ++n_kq; }
            if (c > 0 && !(ok = delta_wait(bar(Lay::Y_OUT), c - 1, dead))) break;
            tc_fence_after();
            if (lane == 0) {                              // Q S^T, the hi part
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) umma_ts(tbase + 192, tbase + 8 * ks, kdesc(qt, ks), kIdN, ks > 0);
                umma_commit(bar(Lay::X_Q));
            }
            // U goes where S hi is: Q S^T has to be done with it
            if (!(ok = delta_wait(bar(Lay::FULL_T), c, dead) && delta_wait(bar(Lay::R_IN), c, dead) &&
                       delta_wait(bar(Lay::X_Q), c, dead))) break;
            tc_fence_after();
            if (lane == 0) {                              // U = T R: hi hi, lo hi (R lo), hi lo (T lo)
#pragma unroll
                for (int ks = 0; ks < 12; ++ks) {
                    const int q = ks & 3, part = ks >> 2;
                    umma_ts(tbase, tbase + 64 + (part == 1 ? 32 : 0) + 8 * q,
                            umma_desc(sb + Lay::T + (part == 2 ? kDlTile : 0) + q * 32, 16, 1024), kIdN, ks > 0);
                }
                umma_commit(bar(Lay::UR));
            }
            if (c + 1 < nC) { load_v(c + 1); ++n_v; }     // V was read before R came in
            if (!(ok = delta_wait(bar(Lay::FULL_M), c, dead) && delta_wait(bar(Lay::U_IN), c, dead))) break;
            tc_fence_after();
            if (c + 1 < nC) { load_t(c + 1); ++n_t; }     // U was read: the product that read T is done
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)            // Y += M U
                    umma_ts(tbase + 192, tbase + 160 + 8 * ks, umma_desc(sb + Lay::M + ks * 32, 16, 1024), kIdN, 1);
                umma_commit(bar(Lay::YM));
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)            // U_w^T K, n < 64
                    umma_ts(tbase, tbase + 64 + 8 * ks, umma_desc(kt + (ks & 3) * 2048, 16384, 1024), kIdS, ks > 0);
                umma_commit(bar(Lay::D_A));
            }
            // the other half of the increment takes the columns of U hi, once M U has read them
            if (!(ok = delta_wait(bar(Lay::YM), c, dead))) break;
            if (lane == 0 && N == 128) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ts(tbase + 128, tbase + 64 + 8 * ks, umma_desc(kt + 16384 + (ks & 3) * 2048, 16384, 1024), kIdS, ks > 0);
                umma_commit(bar(Lay::D_B));
            }
            if (c + 1 < nC) { load_m(c + 1); ++n_m; }
        }
        if (!ok) {
            // copies and products in flight end before the block does (bounded waits)
            if (lane == 0) {
                atomicExch(p.err, 1);
                umma_commit(bar(Lay::DRAIN));
            }
            __syncwarp();
            mbar_wait(bar(Lay::DRAIN), 0u);
            if (n_kq > 0) mbar_wait(bar(Lay::FULL_KQ0 + ((n_kq - 1) & 1)), (uint32_t)((n_kq - 1) >> 1) & 1);
            if (n_kq > 1) mbar_wait(bar(Lay::FULL_KQ0 + (n_kq & 1)), (uint32_t)((n_kq - 2) >> 1) & 1);
            if (n_v > 0) mbar_wait(bar(Lay::FULL_V), (uint32_t)(n_v - 1) & 1);
            if (n_t > 0) mbar_wait(bar(Lay::FULL_T), (uint32_t)(n_t - 1) & 1);
            if (n_m > 0) mbar_wait(bar(Lay::FULL_M), (uint32_t)(n_m - 1) & 1);
        }
    } else if (w < WARPS) {
        // ---------------- a thread per value column
        const int v = tid;
        const uint32_t tl = tbase + ((uint32_t)(32 * w) << 16);
        float S[N];                                       // lambda times the state row
        float lam = 1.f, ilam = 1.f;                      // the lane's scale and its inverse
        const size_t hoff = (((size_t)b * d.H + h) * P + v) * N;
#pragma unroll
        for (int n = 0; n < N; n += 4) {
            const float4 x = d.h0 ? *reinterpret_cast<const float4*>(d.h0 + hoff + n) : make_float4(0.f, 0.f, 0.f, 0.f);
            S[n] = x.x; S[n + 1] = x.y; S[n + 2] = x.z; S[n + 3] = x.w;
        }
        float mS = 0.f;
        // multiplies the lane by 2^-e, e the exponent of m
        auto rescale = [&](float m) {
            const int e = exp_above(m);
            const float f = pow2i(-e);
            // lambda stays a float power of two whose inverse is one
            if (lam * f < 0x1p-100f || lam * f > 0x1p100f) return 1.f;
            lam *= f;
            ilam *= pow2i(e);
#pragma unroll
            for (int n = 0; n < N; ++n) S[n] *= f;
            mS *= f;
            return f;
        };
        auto store_state = [&]() {                        // S into the A operand's columns
            mS = 0.f;
#pragma unroll
            for (int n = 0; n < N; n += 2) mS = max_abs3(mS, S[n], S[n + 1]);
            if (mS > 64.f || (mS < 0.125f && mS > 0.f)) rescale(mS);
            __syncwarp();
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) split_f16(S[n0 + 2 * q], S[n0 + 2 * q + 1], hi[q], lo[q]);
                tmem_st8(tl + n0 / 2, hi);
                tmem_st8(tl + 64 + n0 / 2, lo);
            }
            tmem_st_wait();
        };
        auto arrive = [&](int i) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        if (nC > 0) {
            store_state();
            arrive(Lay::S_IN);
        }
        bool ok = true;
        for (int c = 0; c < nC; ++c) {
            const float* vec = reinterpret_cast<const float*>(sm + Lay::VEC + (c & 1) * kDlVec);
            const unsigned short* sv = reinterpret_cast<const unsigned short*>(sm + Lay::V) + v;
            const int rows = min(C, len - c * C);
            // ---- R = V - e^Gamma rk (K S^T)
            float fx = 1.f;                               // what the lane was rescaled by since Q S^T
            {
                if (!(ok = delta_wait(bar(Lay::FULL_V), c, dead) && delta_wait(bar(Lay::X_K), c, dead))) break;
                tc_fence_after();
                if (rows < C)                             // tokens that are not there write nothing
                    for (int t = rows; t < C; ++t) const_cast<unsigned short*>(sv)[t * P] = 0;
                // a lane whose values have left the window rescales and does it again
                for (int pass = 0; pass < 2; ++pass) {
                    float m = 0.f;
#pragma unroll
                    for (int t0 = 0; t0 < C; t0 += 16) {
                        float x[16];
                        tmem_ld16(tl + 128 + t0, x);
#pragma unroll
                        for (int q = 0; q < 16; q += 4) {
                            const float4 ek = *reinterpret_cast<const float4*>(vec + t0 + q);
                            const float e4[4] = {ek.x, ek.y, ek.z, ek.w};
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float val = __uint_as_float((uint32_t)sv[(t0 + q + u) * P] << 16);
                                x[q + u] = fmaf(-(e4[u] * fx), x[q + u], lam * val);
                            }
                        }
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            m = max_abs3(m, x[2 * q], x[2 * q + 1]);
                            split_f16(x[2 * q], x[2 * q + 1], hi[q], lo[q]);
                        }
                        tmem_st8(tl + 64 + t0 / 2, hi);
                        tmem_st8(tl + 96 + t0 / 2, lo);
                    }
                    const float mm = fmaxf(m, mS);
                    const bool out = m > 64.f || (mm < 0.125f && mm > 0.f);
                    if (!__any_sync(0xffffffffu, out) || pass) break;
                    if (out) fx = rescale(mm);
                    __syncwarp();
                }
                tmem_st_wait();
                arrive(Lay::R_IN);
            }
            // ---- e^Gamma (Q S^T), back to its columns, while U = T R runs
            {
                if (!(ok = delta_wait(bar(Lay::X_Q), c, dead))) break;
                tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < C; t0 += 16) {
                    float x[16];
                    uint32_t o[16];
                    tmem_ld16(tl + 192 + t0, x);
#pragma unroll
                    for (int q = 0; q < 16; q += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(vec + C + t0 + q);
                        o[q] = __float_as_uint(x[q] * (e.x * fx));
                        o[q + 1] = __float_as_uint(x[q + 1] * (e.y * fx));
                        o[q + 2] = __float_as_uint(x[q + 2] * (e.z * fx));
                        o[q + 3] = __float_as_uint(x[q + 3] * (e.w * fx));
                    }
                    tmem_st16(tl + 192 + t0, o);
                }
            }
            // ---- U: one part for Y; weighted, two parts for the state
            {
                if (!(ok = delta_wait(bar(Lay::UR), c, dead))) break;
                tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < C; t0 += 16) {
                    uint32_t u[8], hi[8], lo[8];
                    float x[16];
                    tmem_ld16(tl + t0, x);
#pragma unroll
                    for (int q = 0; q < 8; ++q) u[q] = pack_f16(x[2 * q], x[2 * q + 1]);
                    tmem_st8(tl + 160 + t0 / 2, u);
#pragma unroll
                    for (int q = 0; q < 8; q += 2) {
                        const float4 wk = *reinterpret_cast<const float4*>(vec + 2 * C + t0 + 2 * q);
                        split_f16(x[2 * q] * wk.x, x[2 * q + 1] * wk.y, hi[q], lo[q]);
                        split_f16(x[2 * q + 2] * wk.z, x[2 * q + 3] * wk.w, hi[q + 1], lo[q + 1]);
                    }
                    tmem_st8(tl + 64 + t0 / 2, hi);
                    tmem_st8(tl + 96 + t0 / 2, lo);
                }
                tmem_st_wait();
                arrive(Lay::U_IN);
            }
            // ---- the state after the chunk
            const float el = vec[2 * C - 1];
            {
                if (!(ok = delta_wait(bar(Lay::D_A), c, dead))) break;
                tc_fence_after();
#pragma unroll
                for (int n0 = 0; n0 < 64; n0 += 16) {
                    float x[16];
                    tmem_ld16(tl + n0, x);
#pragma unroll
                    for (int q = 0; q < 16; ++q) S[n0 + q] = fmaf(el, S[n0 + q], x[q]);
                }
                if constexpr (N == 128) {
                    if (!(ok = delta_wait(bar(Lay::D_B), c, dead))) break;
                    tc_fence_after();
#pragma unroll
                    for (int n0 = 64; n0 < 128; n0 += 16) {
                        float x[16];
                        tmem_ld16(tl + 64 + n0, x);
#pragma unroll
                        for (int q = 0; q < 16; ++q) S[n0 + q] = fmaf(el, S[n0 + q], x[q]);
                    }
                }
            }
            const float yl = ilam;                        // Y is in units of the lane's scale so far
            if (c + 1 < nC) {
                store_state();
                arrive(Lay::S_IN);
            }
            // ---- y, while K S^T of the next chunk runs: neighbouring lanes trade
            // tokens, so a lane stores two columns of one token
            if (!(ok = delta_wait(bar(Lay::YM), c, dead))) break;
            tc_fence_after();
            const int odd = lane & 1;
            __nv_bfloat16* yo = static_cast<__nv_bfloat16*>(d.y) + (((size_t)b * d.L + (size_t)c * C + odd) * d.H + h) * P + (v & ~1);
            const size_t ystep = (size_t)d.H * P;
#pragma unroll
            for (int t0 = 0; t0 < C; t0 += 16) {
                float x[16];
                tmem_ld16(tl + 192 + t0, x);
#pragma unroll
                for (int q = 0; q < 16; q += 4) {
                    const float4 oq = *reinterpret_cast<const float4*>(vec + 3 * C + t0 + q);
                    x[q] *= oq.x * yl; x[q + 1] *= oq.y * yl; x[q + 2] *= oq.z * yl; x[q + 3] *= oq.w * yl;
                }
#pragma unroll
                for (int q = 0; q < 16; q += 2) {
                    const uint32_t mine = pack_bf16(x[q], x[q + 1]);
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
                    const uint32_t o = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
                    if (t0 + q + odd < rows) *reinterpret_cast<uint32_t*>(yo + (t0 + q) * ystep) = o;
                }
            }
            arrive(Lay::Y_OUT);
        }
        if (ok) {
#pragma unroll
            for (int n = 0; n < N; n += 4)
                *reinterpret_cast<float4*>(d.h_out + hoff + n) =
                    make_float4(S[n] * ilam, S[n + 1] * ilam, S[n + 2] * ilam, S[n + 3] * ilam);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 4 && !*dead) tmem_dealloc(tbase, Lay::COLS);   // a late product must not meet another block's columns
}

}  // namespace axon
