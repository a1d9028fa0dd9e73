// gated_norm.cuh -- grouped norm of channels-last rows with a SiLU gate or
// activation: the output stage between a recurrent core (one norm per head of
// P channels, gate after the norm; or the gate before a norm over wide groups)
// and the output projection.  Per row and group of D channels
//   t = x, or x act(z) with the gate before the norm
//   n = t / sqrt(mean(t^2) + eps)                      (RMS)
//   n = (t - mean(t)) / sqrt(mean((t - mean(t))^2) + eps)   (group norm)
//   y = n w + b;  gate after: y act(z);  no gate: act(y)    (act: SiLU or none)
// Bound by HBM: each value is read once, kept in registers over the
// statistics (the variance is a second pass over those registers, so it does
// not cancel) and written once.  16-byte loads; float32 inside.
#pragma once

#include <cuda_bf16.h>

#include "device_math.cuh"
#include "tc_ops.cuh"   // bf16 packing

namespace axon {

struct NormParams {
    int rows, C, D;
    int groups;            // rows x C / D
    int ldx, ldz, ldy;     // elements between rows
    const void* x;
    const void* z;         // null: no gate
    const float* w;        // null: 1
    const float* b;        // null: 0
    int per_channel;       // w and b: C values (else D, shared by the groups)
    int centre;            // subtract the mean
    int before;            // the gate goes before the norm
    int act;               // SiLU on the gate, or on y without one
    float eps;
    void* y;
};

template <class Io> struct NormVec;
template <> struct NormVec<IoBF16> {
    static constexpr int VE = 8;
    uint4 v;
    __device__ __forceinline__ void load(const void* p, size_t i) {
        v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(u[i]); f[2 * i + 1] = bf16_hi(u[i]); }
    }
    __device__ __forceinline__ static void store(void* p, size_t i, const float (&f)[8]) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};
template <> struct NormVec<IoF32> {
    static constexpr int VE = 4;
    float4 v;
    __device__ __forceinline__ void load(const void* p, size_t i) {
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
    __device__ __forceinline__ static void store(void* p, size_t i, const float (&f)[4]) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    }
};

// `W` = 1: a group belongs to LG lanes of a warp, each with VPL 16-byte
// pieces (piece lane + LG i); a warp serves 32 / LG groups, U times over, the
// loads of all U issued before the first use.  Blocks are two warps: a block
// gives its registers back when its slower warp is done, and the next one's
// loads start then (65536 x 4096 bf16 in groups of 128 with a gate: 285 us,
// 5650 GB/s; 291 us with blocks of four warps, 318 with eight).  `W` = warps of the block: one
// group per block (LG = 32, U = 1), sums joined through shared memory.
template <class Io, int LG, int VPL, int U, int W>
__global__ void __launch_bounds__(W == 1 ? 64 : 32 * W) gated_norm_kernel(NormParams p) {
    using Vec = NormVec<Io>;
    constexpr int VE = Vec::VE;
    constexpr int GW = 32 / LG;                  // groups a warp serves at once
    static_assert(W == 1 || (LG == 32 && U == 1), "a block's group takes whole warps");
    __shared__ float part[2][W == 1 ? 1 : W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = W == 1 ? lane % LG : (int)threadIdx.x;        // lane's place in its group
    constexpr int STEP = W == 1 ? LG : 32 * W;                   // pieces between a lane's pieces
    const int NG = p.C / p.D, pieces = p.D / VE;
    const int g0 = W == 1 ? ((int)blockIdx.x * 2 + warp) * (GW * U) + lane / LG : (int)blockIdx.x;

    Vec xv[U][VPL], zv[U][VPL];
    int row[U], col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int g = min(g0 + u * GW, p.groups - 1);            // lanes past the last group recompute it and store nothing
        row[u] = g / NG;
        col[u] = (g - row[u] * NG) * p.D;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int pc = gl + STEP * i;
            if (pc < pieces) {
                xv[u][i].load(p.x, (size_t)row[u] * p.ldx + col[u] + pc * VE);
                if (p.z) zv[u][i].load(p.z, (size_t)row[u] * p.ldz + col[u] + pc * VE);
            }
        }
    }
    auto total = [&](float v, int slot) {
#pragma unroll
        for (int d = LG / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if constexpr (W > 1) {
            if (lane == 0) part[slot][warp] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) v += part[slot][i];
        }
        return v;
    };
    const float inv = 1.0f / (float)p.D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float t[VPL][VE], gt[VPL][VE];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (gl + STEP * i >= pieces) continue;
            xv[u][i].get(t[i]);
            if (p.z) {
                zv[u][i].get(gt[i]);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (p.act) gt[i][e] = silu(gt[i][e]);
                    if (p.before) t[i][e] *= gt[i][e];
                }
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                s1 += t[i][e];
                s2 = fmaf(t[i][e], t[i][e], s2);
            }
        }
        float mean = 0.f;
        if (p.centre) {
            mean = total(s1, 0) * inv;
            s2 = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (gl + STEP * i >= pieces) continue;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    t[i][e] -= mean;
                    s2 = fmaf(t[i][e], t[i][e], s2);
                }
            }
        }
        const float rs = rsqrtf(fmaf(total(s2, 1), inv, p.eps));
        const bool live = W > 1 || g0 + u * GW < p.groups;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int pc = gl + STEP * i;
            if (pc >= pieces || !live) continue;
            const int wi = pc * VE + (p.per_channel ? col[u] : 0);
            float wv[VE], bv[VE];
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                const float4 w4 = p.w ? __ldg(reinterpret_cast<const float4*>(p.w + wi + e)) : make_float4(1.f, 1.f, 1.f, 1.f);
                const float4 b4 = p.b ? __ldg(reinterpret_cast<const float4*>(p.b + wi + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
                wv[e] = w4.x; wv[e + 1] = w4.y; wv[e + 2] = w4.z; wv[e + 3] = w4.w;
                bv[e] = b4.x; bv[e + 1] = b4.y; bv[e + 2] = b4.z; bv[e + 3] = b4.w;
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float o = fmaf(t[i][e] * rs, wv[e], bv[e]);
                if (!p.z) o = p.act ? silu(o) : o;
                else if (!p.before) o *= gt[i][e];
                t[i][e] = o;
            }
            Vec::store(p.y, (size_t)row[u] * p.ldy + col[u] + pc * VE, t[i]);
        }
    }
}

}  // namespace axon
