// delta_step.cuh -- the gated delta rule token by token, in float32 on the
// CUDA cores: the cached single-token step, and the recurrent prefill (float32
// inputs, whose results bf16 tensor-core products could not give, and short
// bf16 sequences, where the chunked form of delta.cuh has nothing to share).
//
// Per batch row b and value head h (key head g = h / (H / G)), state S (P x N):
//   dt = softplus(dt_raw + dt_bias_h)   (no clip: the delta rule needs no
//   a  = exp(-exp(A_log_h) dt)           smallest step, and a long memory wants
//   beta = sigmoid(b_raw)                decays of exactly 1)
//   rk = 1 / sqrt(|k|^2 + 1e-6), rq likewise (1 without the norm)
//   e_p = beta (v_p - a rk S_p.k),  S_p <- a S_p + (e_p rk) k,
//   y_p = scale rq (a S_p.q + (e_p rk) (k.q))   with the S_p before the update,
// so one pass over a state row gives both products, and the row is read and
// written once.
#pragma once

#include <cuda_bf16.h>

#include "device_math.cuh"
#include "scan_chunked.cuh"   // cp.async helpers
#include "tc_ops.cuh"         // bf16 packing

namespace axon {

constexpr float kDeltaEps = 1e-6f;     // added to |k|^2 and |q|^2

// exp(-v) for v >= 0: the product v log2(e) in two floats, so the argument of
// the MUFU exp2 carries no rounding error that grows with v.
__device__ __forceinline__ float exp_neg(float v) {
    constexpr float kLog2eLo = 1.9259629911e-08f;     // log2(e) - float(log2(e))
    v = fminf(v, 200.0f);                              // exp(-200) is 0 already; inf would give inf - inf
    const float hi = -v * kLog2e;
    const float lo = fmaf(-v, kLog2e, -hi) - v * kLog2eLo;
    return ex2_approx(hi) * fmaf(lo, kLn2, 1.0f);
}
// softplus with the full log1p: log1p_unit's 4e-6 relative error would show in
// the float32 state after long decays.  A NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float softplus_full(float v) {
    return (v < 0.0f ? 0.0f : v) + log1pf(exp_neg(fabsf(v)));
}
// log2 of the decay of one token
__device__ __forceinline__ float delta_log2_decay(float raw, float expA) {
    return -expA * softplus_full(raw) * kLog2e;
}
// One token's decay a, and m = a - 1 for a slow one (a >= 1/2).  A float a near 1
// is up to 2^-25 off, the same way at every token of a like dt, and a state that
// lasts thousands of tokens would show the sum (7e-5 after 4096 tokens, 1e-4 of a
// slower one).  m = -2 e^(-x/2) sinh(x/2) cancels nothing; sinh by its
// series, x/2 <= ln(2)/2: next term below 1e-9.
struct DeltaDecay {
    float a, m;
    __device__ __forceinline__ DeltaDecay(float raw, float expA) {
        const float x = expA * softplus_full(raw), u = 0.5f * x, v = u * u;
        a = ex2_approx(-x * kLog2e);
        m = -x * ex2_approx(-u * kLog2e) * fmaf(v, fmaf(v, fmaf(v, 1.f / 5040.f, 1.f / 120.f), 1.f / 6.f), 1.f);
    }
    __device__ __forceinline__ bool slow() const { return a >= 0.5f; }
    // a as a float whose errors cancel over the tokens t: what 1 + m rounds off,
    // in steps of 2^-24, decides against t times the golden ratio plus a half, mod
    // 1 (evenly spread over any run of tokens; a lone one is rounded to nearest),
    // whether a is one step further.
    __device__ __forceinline__ float at(uint32_t t) const {
        const float r = 1.f + m;
        const float off = (m - (r - 1.f)) * 0x1p24f;                   // exact: within +- 1/2
        const float s = floorf(off + (float)(t * 2654435769u + 0x80000000u >> 8) * 0x1p-24f);
        return slow() ? fmaf(s, 0x1p-24f, r) : a;
    }
};
__device__ __forceinline__ float delta_beta(float b) {
    const float e = exp_neg(fabsf(b));                 // sigmoid without overflow
    const float r = 1.0f / (1.0f + e);
    return b >= 0.0f ? r : (b < 0.0f ? e * r : b);     // NaN stays NaN
}
__device__ __forceinline__ float delta_exp_a(float a_log) {           // exp; NaN stays NaN (exp_neg's clamp would drop it)
    return a_log >= 0.0f ? 1.0f / exp_neg(a_log) : (a_log < 0.0f ? exp_neg(-a_log) : a_log);
}

struct DeltaParams {
    int B, L, H, G, P;
    int ldq, ldk, ldv;           // elements between consecutive tokens
    const void* q;               // (B, L, G, N) io
    const void* k;               // (B, L, G, N) io
    const void* v;               // (B, L, H, P) io
    const void* dt_raw;          // (B, L, H) io
    const void* b_raw;           // (B, L, H) io
    const float* dt_bias;        // (H)
    const float* A_log;          // (H)
    const int* lengths;          // (B) or null
    const float* h0;             // (B, H, P, N) or null
    void* y;                     // (B, L, H, P) io
    float* h_out;                // (B, H, P, N)
    float scale;
    int norm;                    // L2 norm of q and k
};

// 16 values of a lane's share of a q or k row: quads qd + LPR i of the row.
template <class Io, int LPR>
__device__ __forceinline__ void delta_load16(const typename Io::T* row, int qd, float (&r)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float t[4];
        Io::sload4(row + 4 * (qd + LPR * i), t);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[4 * i + j] = t[j];
    }
}

template <int LPR>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int d = LPR / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// One token for B sequences.  LPR = N / 16 lanes share a state row (each
// holds four float4 of it, so a warp's load instruction covers whole 128- or
// 256-byte runs); a lane serves RT rows.  grid = (P / rows, H, B) blocks of
// 128 threads, rows = 4 warps x 32 / LPR x RT.  Bound by the state, read and
// written once: 2 P N 4 bytes a head; all of a lane's state loads are issued
// before the first use.  RT = 1 spreads a small batch over more SMs.
// 64 sequences of 32 heads, N = P = 128, bf16: 44 us, 6.1 TB/s.
template <class Io, int N, int RT>
__global__ void __launch_bounds__(128) delta_step_kernel(DeltaParams p) {
    using T = typename Io::T;
    constexpr int LPR = N / 16, RW = 32 / LPR;
    const int h = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int qd = lane % LPR, rg = lane / LPR;
    const int g = h / (p.H / p.G);
    const int row0 = (blockIdx.x * 4 + w) * RW * RT + rg;       // rows row0 + RW i
    float* st = p.h_out + (((size_t)b * p.H + h) * p.P + row0) * N + 4 * qd;
    float S[RT][16];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(st + (size_t)r * RW * N + 4 * LPR * i);
            S[r][4 * i] = v.x; S[r][4 * i + 1] = v.y; S[r][4 * i + 2] = v.z; S[r][4 * i + 3] = v.w;
        }
    float k[16], q[16], v[RT];
    delta_load16<Io, LPR>(static_cast<const T*>(p.k) + (size_t)b * p.ldk + (size_t)g * N, qd, k);
    delta_load16<Io, LPR>(static_cast<const T*>(p.q) + (size_t)b * p.ldq + (size_t)g * N, qd, q);
    const T* vp = static_cast<const T*>(p.v) + (size_t)b * p.ldv + (size_t)h * p.P + row0;
#pragma unroll
    for (int r = 0; r < RT; ++r) v[r] = Io::load(vp + r * RW);
    const size_t bh = (size_t)b * p.H + h;
    const DeltaDecay dec(Io::load(static_cast<const T*>(p.dt_raw) + bh) + __ldg(p.dt_bias + h), delta_exp_a(__ldg(p.A_log + h)));
    const bool slow = dec.slow();                                   // S + m S, else a S: a call knows no token's number
    const float a = dec.a;
    const float beta = delta_beta(Io::load(static_cast<const T*>(p.b_raw) + bh));
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        kk = fmaf(k[i], k[i], kk);
        qq = fmaf(q[i], q[i], qq);
        kq = fmaf(k[i], q[i], kq);
    }
    kq = lane_sum<LPR>(kq);
    float rk = 1.f, rq = p.scale;
    if (p.norm) {
        rk = rsqrtf(lane_sum<LPR>(kk) + kDeltaEps);
        rq *= rsqrtf(lane_sum<LPR>(qq) + kDeltaEps);
    }
    T* yp = static_cast<T*>(p.y) + bh * p.P + row0;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sk = fmaf(S[r][i], k[i], sk);
            sq = fmaf(S[r][i], q[i], sq);
        }
        sk = lane_sum<LPR>(sk);
        sq = lane_sum<LPR>(sq);
        const float e = beta * (v[r] - a * rk * sk) * rk;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = S[r][4 * i + j];
                s[j] = fmaf(e, k[4 * i + j], slow ? fmaf(dec.m, x, x) : a * x);
            }
            *reinterpret_cast<float4*>(st + (size_t)r * RW * N + 4 * LPR * i) = make_float4(s[0], s[1], s[2], s[3]);
        }
        if (qd == 0) Io::store(yp + r * RW, rq * fmaf(e, kq, a * sq));
    }
}

// The token loop.  A block of 128 threads keeps 4 RW RT rows of one head's
// state in registers and walks the sequence in tiles of kDeltaTile tokens,
// staged in shared memory two tiles deep by cp.async (each tile's copies are
// in flight while the tile before it computes); a tile's decays, betas, norms
// and k.q are computed once, by eight threads a token, then its tokens run
// without a barrier.  grid = (P / rows, H, B).  Bound by the chain through a
// token: two sums over LPR lanes and the update, 0.2 to 0.25 us (515 float32
// tokens of 16 heads, N 64 P 128: 133 us).
constexpr int kDeltaTile = 16;

template <class Io, int N, int RT>
struct DeltaRecurSmem {
    static constexpr int ROWS = 4 * (32 / (N / 16)) * RT;
    static constexpr int QB = kDeltaTile * N * Io::kBytes;          // one tile of q (and of k)
    static constexpr int VB = kDeltaTile * ROWS * Io::kBytes;
    static constexpr int STAGE = 2 * QB + VB;
    static constexpr int SC = 2 * STAGE;                            // float4 (a, beta, rk, rq) per token
    static constexpr int KQ = SC + kDeltaTile * 16;                 // k.q per token
    static constexpr int YT = KQ + kDeltaTile * 4;                  // y of the tile, float32
    static constexpr int TOTAL = YT + kDeltaTile * ROWS * 4;
    static_assert(TOTAL <= 48 * 1024, "static shared memory");
    static_assert(STAGE % 16 == 0, "16-byte copies");
};

template <class Io, int N, int RT>
__global__ void __launch_bounds__(128) delta_recur_kernel(DeltaParams p) {
    using T = typename Io::T;
    using Lay = DeltaRecurSmem<Io, N, RT>;
    constexpr int LPR = N / 16, RW = 32 / LPR, ROWS = Lay::ROWS, TT = kDeltaTile, VE = 16 / Io::kBytes;
    __shared__ __align__(16) unsigned char sm[Lay::TOTAL];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int lane = tid & 31, w = tid >> 5;
    const int qd = lane % LPR, rg = lane / LPR;
    const int g = h / (p.H / p.G);
    const int blk0 = blockIdx.x * ROWS;                             // first row of the block
    const int loc0 = w * RW * RT + rg;                              // this lane's rows: blk0 + loc0 + RW i
    int len = p.L;
    if (p.lengths) len = min(max(__ldg(p.lengths + b), 0), p.L);

    const size_t hoff = (((size_t)b * p.H + h) * p.P + blk0 + loc0) * N + 4 * qd;
    float2 S[RT][8];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = p.h0 ? *reinterpret_cast<const float4*>(p.h0 + hoff + (size_t)r * RW * N + 4 * LPR * i)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            S[r][2 * i] = make_float2(v.x, v.y);
            S[r][2 * i + 1] = make_float2(v.z, v.w);
        }

    const T* qg = static_cast<const T*>(p.q) + (size_t)b * p.L * p.ldq + (size_t)g * N;
    const T* kg = static_cast<const T*>(p.k) + (size_t)b * p.L * p.ldk + (size_t)g * N;
    const T* vg = static_cast<const T*>(p.v) + (size_t)b * p.L * p.ldv + (size_t)h * p.P + blk0;
    T* yg = static_cast<T*>(p.y) + ((size_t)b * p.L * p.H + h) * p.P + blk0;
    auto copy_tile = [&](int t0, int stage) {
        unsigned char* s = sm + stage * Lay::STAGE;
        constexpr int QP = N / VE, VP = ROWS / VE;                  // 16-byte pieces of a row
        for (int i = tid; i < TT * QP; i += 128) {
            const int t = i / QP, c = i % QP;
            const bool ok = t0 + t < len;
            cp_async16(s + i * 16, ok ? qg + (size_t)(t0 + t) * p.ldq + c * VE : qg, ok);
            cp_async16(s + Lay::QB + i * 16, ok ? kg + (size_t)(t0 + t) * p.ldk + c * VE : kg, ok);
        }
        for (int i = tid; i < TT * VP; i += 128) {
            const int t = i / VP, c = i % VP;
            const bool ok = t0 + t < len;
            cp_async16(s + 2 * Lay::QB + i * 16, ok ? vg + (size_t)(t0 + t) * p.ldv + c * VE : vg, ok);
        }
        cp_async_commit();
    };
    const float expA = delta_exp_a(__ldg(p.A_log + h)), bias = __ldg(p.dt_bias + h);
    float4* sc = reinterpret_cast<float4*>(sm + Lay::SC);
    float* skq = reinterpret_cast<float*>(sm + Lay::KQ);
    float* sy = reinterpret_cast<float*>(sm + Lay::YT);

    if (len > 0) copy_tile(0, 0);
    for (int t0 = 0, it = 0; t0 < len; t0 += TT, ++it) {
        const int nt = min(TT, len - t0);
        cp_async_wait_0();
        __syncthreads();                                            // tile landed; the other stage and sy are free
        if (t0 + TT < len) copy_tile(t0 + TT, (it + 1) & 1);
        const T* sq = reinterpret_cast<const T*>(sm + (it & 1) * Lay::STAGE);
        const T* sk = sq + TT * N;
        const T* sv = sk + TT * N;
        {                                                           // eight threads a token
            const int t = tid >> 3, l = tid & 7;
            float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < N / 32; ++i) {
                float a4[4], b4[4];
                Io::sload4(sk + t * N + 4 * (l + 8 * i), a4);
                Io::sload4(sq + t * N + 4 * (l + 8 * i), b4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    kk = fmaf(a4[j], a4[j], kk);
                    qq = fmaf(b4[j], b4[j], qq);
                    kq = fmaf(a4[j], b4[j], kq);
                }
            }
            kk = lane_sum<8>(kk);
            qq = lane_sum<8>(qq);
            kq = lane_sum<8>(kq);
            if (l == 0 && t < nt) {
                const size_t o = ((size_t)b * p.L + t0 + t) * p.H + h;
                const float a = DeltaDecay(Io::load(static_cast<const T*>(p.dt_raw) + o) + bias, expA).at(t0 + t);
                const float beta = delta_beta(Io::load(static_cast<const T*>(p.b_raw) + o));
                sc[t] = make_float4(a, beta, p.norm ? rsqrtf(kk + kDeltaEps) : 1.f,
                                    p.scale * (p.norm ? rsqrtf(qq + kDeltaEps) : 1.f));
                skq[t] = kq;
            }
        }
        __syncthreads();
        float2 k[8], q[8];
        auto token = [&](int t) {
            float r[16];
            delta_load16<Io, LPR>(sk + t * N, qd, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = make_float2(r[2 * i], r[2 * i + 1]);
            delta_load16<Io, LPR>(sq + t * N, qd, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = make_float2(r[2 * i], r[2 * i + 1]);
        };
        for (int t = 0; t < nt; ++t) {
            token(t);
            const float4 c = sc[t];
            const float kq = skq[t];
            float dk[RT], dq[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {                          // two sums each, of pairs: short chains
                float2 a0 = make_float2(0.f, 0.f), a1 = a0, b0 = a0, b1 = a0;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    a0 = __ffma2_rn(S[r][i], k[i], a0);
                    a1 = __ffma2_rn(S[r][i + 1], k[i + 1], a1);
                    b0 = __ffma2_rn(S[r][i], q[i], b0);
                    b1 = __ffma2_rn(S[r][i + 1], q[i + 1], b1);
                }
                dk[r] = (a0.x + a1.x) + (a0.y + a1.y);
                dq[r] = (b0.x + b1.x) + (b0.y + b1.y);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) dk[r] = lane_sum<LPR>(dk[r]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {                          // the decay needs no sum
#pragma unroll
                for (int i = 0; i < 8; ++i) S[r][i] = __fmul2_rn(make_float2(c.x, c.x), S[r][i]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float v = Io::sload(sv + t * ROWS + loc0 + r * RW);
                const float e = c.y * (v - c.x * c.z * dk[r]) * c.z;
#pragma unroll
                for (int i = 0; i < 8; ++i) S[r][i] = __ffma2_rn(make_float2(e, e), k[i], S[r][i]);
                dk[r] = e;
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                dq[r] = lane_sum<LPR>(dq[r]);
                if (qd == 0) sy[t * ROWS + loc0 + r * RW] = c.w * fmaf(dk[r], kq, c.x * dq[r]);
            }
        }
        __syncthreads();                                            // sy complete
        for (int i = tid; i < nt * ROWS; i += 128) {
            const int t = i / ROWS, c = i % ROWS;
            Io::store(yg + (size_t)(t0 + t) * p.H * p.P + c, sy[i]);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(p.h_out + hoff + (size_t)r * RW * N + 4 * LPR * i) =
                make_float4(S[r][2 * i].x, S[r][2 * i].y, S[r][2 * i + 1].x, S[r][2 * i + 1].y);
}

}  // namespace axon
