// axon_delta.cu -- C ABI of the gated delta rule and of the grouped gated norm
// (include/axon_ssm.h): argument checks, launch plans, launches of
// delta_step.cuh and gated_norm.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "axon_ssm.h"
#include "delta.cuh"
#include "delta_step.cuh"
#include "gated_norm.cuh"
#include "tensor_map.cuh"

namespace axon {
namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ovl(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}
// bytes from the first to behind the last value of `rows` rows of `cols` values, ld apart
size_t extent(size_t rows, size_t cols, size_t ld, size_t es) { return rows ? ((rows - 1) * ld + cols) * es : 0; }

// Whether two sets of `rows` rows of `cols` values overlap; rows of one stride
// may interleave (slices of one wider row).
bool rows_ovl(const void* a, size_t lda, const void* b, size_t ldb, size_t rows, size_t cols, size_t es) {
    if (!ovl(a, extent(rows, cols, lda, es), b, extent(rows, cols, ldb, es))) return false;
    if (lda != ldb) return true;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const size_t d = (a0 < b0 ? b0 - a0 : a0 - b0) % (lda * es);
    return d < cols * es || d + cols * es > lda * es;
}

int sm_count() {
    static std::atomic<int> cached[64];   // zero-initialised (static storage)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
    if (dev < 64) {
        const int v = cached[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool shape_ok(int H, int G, int P, int N) {
    return G > 0 && H % G == 0 && (P == 64 || P == 128) && (N == 64 || N == 128);
}

// What both delta entry points check alike; `rows` = tokens of all sequences.
axon_status check_delta(size_t rows, int H, int G, int P, int N, axon_dtype io, const void* q, int ldq, const void* k,
                        int ldk, const void* v, int ldv, const void* dt_raw, const void* b_raw, const float* dt_bias,
                        const float* A_log, float scale) {
    if (!shape_ok(H, G, P, N) || (io != AXON_F32 && io != AXON_BF16)) return AXON_ERR_UNSUPPORTED;
    if (!dt_bias || !A_log || !std::isfinite(scale)) return AXON_ERR_INVALID_ARG;
    if (rows > 0 && (!q || !k || !v || !dt_raw || !b_raw)) return AXON_ERR_INVALID_ARG;
    if (ldq < G * N || ldk < G * N || ldv < H * P) return AXON_ERR_INVALID_ARG;
    const int m = io == AXON_BF16 ? 8 : 4;
    if (ldq % m || ldk % m || ldv % m) return AXON_ERR_ALIGNMENT;
    for (const void* t : {q, k, v})
        if (t && !al16(t)) return AXON_ERR_ALIGNMENT;
    // the rates and parameters are read one value at a time
    const uintptr_t gate = reinterpret_cast<uintptr_t>(dt_raw) | reinterpret_cast<uintptr_t>(b_raw);
    const uintptr_t par = reinterpret_cast<uintptr_t>(dt_bias) | reinterpret_cast<uintptr_t>(A_log);
    if ((gate & (io == AXON_BF16 ? 1u : 3u)) || (par & 3u)) return AXON_ERR_ALIGNMENT;
    return AXON_OK;
}

template <class Io, int N>
void launch_step(const DeltaParams& p, cudaStream_t st) {
    constexpr int ROWS1 = 4 * (32 / (N / 16));                      // rows of a block at RT = 1
    // Four rows a lane keep more loads in flight (one row each leaves a third
    // of the bandwidth unused on a large batch); below two blocks an SM that
    // way, the rows are spread over more blocks.
    constexpr int RT = N == 128 ? 4 : 2;
    if ((long long)p.B * p.H * (p.P / (ROWS1 * RT)) >= 2LL * sm_count())
        delta_step_kernel<Io, N, RT><<<dim3((unsigned)(p.P / (ROWS1 * RT)), (unsigned)p.H, (unsigned)p.B), 128, 0, st>>>(p);
    else
        delta_step_kernel<Io, N, 1><<<dim3((unsigned)(p.P / ROWS1), (unsigned)p.H, (unsigned)p.B), 128, 0, st>>>(p);
}
template <class Io, int N>
void launch_recur(const DeltaParams& p, cudaStream_t st) {
    constexpr int ROWS1 = 4 * (32 / (N / 16));
    constexpr int RT = N == 128 ? 4 : 2;
    if ((long long)p.B * p.H * (p.P / (ROWS1 * RT)) >= sm_count())
        delta_recur_kernel<Io, N, RT><<<dim3((unsigned)(p.P / (ROWS1 * RT)), (unsigned)p.H, (unsigned)p.B), 128, 0, st>>>(p);
    else
        delta_recur_kernel<Io, N, 1><<<dim3((unsigned)(p.P / ROWS1), (unsigned)p.H, (unsigned)p.B), 128, 0, st>>>(p);
}

constexpr int kDlMaxSegs = 64;
// Whether bf16 sequences go in chunks: on request (segments > 0), or when that
// is faster.  Measured on the device, in us, with x = B H N P / 128^2: a call
// token by token takes 1 and then max(0.2, 0.13 + 0.0035 x) a token; one chunk
// 22 (N = 128) or 18 (N = 64), most of it the start of two launches, or a SM's
// share of that with many heads, and each further one 3.  Token by token
// against chunks, N = P = 128: B1 H8, 96 tokens 22 and 28, 128 tokens 28 and
// 28, 160 tokens 34 and 31; B8 H16, 32 tokens 23 and 26, 48 tokens 32 and 26;
// B32 H32, 24 tokens 101 and 124, 32 tokens 128 and 125.  N = P = 64: B1 H8,
// 80 tokens 17 and 21, 128 tokens 26 and 21; B32 H32, 48 tokens 55 and 71, 96
// tokens 104 and 117, 128 tokens 139 and 115.
bool chunked(int B, int L, int H, int P, int N, axon_dtype io, int segments) {
    if (io != AXON_BF16 || L <= 0) return false;
    if (segments > 0) return true;
    const double bh = (double)B * H, x = bh * P * N / 16384.0;
    const double first = N == 128 ? std::max(22.0, 0.115 * bh) : std::max(18.0, 0.08 * bh);
    return first + 3.0 * ((L - 1) / kDlC) < 1.0 + L * std::max(0.2, 0.13 + 0.0035 * x);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Segments of whole chunks.  One walk runs on an SM at a time, so a pass takes
// ceil(walks / SMs) rounds of one segment's chunks; a chunk of the pass
// without outputs takes nearly as long as one with them (2.8 and 3.3 us: the same chain of
// products and conversions), a round's start about 2.5 chunks, a fold half of
// one, and the second launch about two.  B1 L4096 H32 measured 261, 248, 193,
// 214, 243 us at 1 to 5 segments; N = P = 64, B2 L2047 H16: 119, 111, 91, 98,
// 102 (three are taken both times).  L counts, not where rows end: lengths lie
// on the device.  `requested` > 0 asks for that many.
struct DeltaPlan {
    int segs, cps;
};
DeltaPlan delta_plan(int B, int L, int H, int requested) {
    const int nC = (L + kDlC - 1) / kDlC;
    const int most = std::min(nC, kDlMaxSegs);
    auto cut = [&](int segs) {
        const int cps = (nC + segs - 1) / segs;
        return DeltaPlan{(nC + cps - 1) / cps, cps};
    };
    if (nC <= 1) return DeltaPlan{1, std::max(nC, 1)};
    if (requested > 0) return cut(std::min(requested, most));
    const long long sms = sm_count(), walks = (long long)B * H;
    DeltaPlan best{1, nC};
    double least = 1e300;
    for (int want = 1; want <= most; ++want) {
        const DeltaPlan p = cut(want);
        const long long full = (p.segs * walks + sms - 1) / sms, state = ((2 * p.segs - 3) * walks + sms - 1) / sms;
        const double t = full * (p.cps + 2.5) + (p.segs > 1 ? state * (p.cps + 2.5) + 0.5 * (p.segs - 2) + 2.0 : 0.0);
        if (t < least) {
            least = t;
            best = p;
        }
    }
    return best;
}

struct DeltaWs {
    size_t err, kq, blob, sloc, tr, trs, h0c, total;
};
DeltaWs delta_ws(int B, int L, int H, int G, int P, int N, const DeltaPlan& plan) {
    const size_t nC = ((size_t)L + kDlC - 1) / kDlC, BH = (size_t)B * H;
    const size_t loc = plan.segs > 1 ? plan.segs - 1 : 0, tr = plan.segs > 2 ? plan.segs - 2 : 0;
    DeltaWs w{};
    w.err = 0;
    w.kq = 256;
    w.blob = w.kq + (size_t)B * G * nC * 128 * N * 2;
    w.sloc = w.blob + up256(BH * nC * kDlBlob);
    w.tr = w.sloc + loc * BH * P * N * 4;
    w.trs = w.tr + tr * BH * 2 * N * N * 2;
    w.h0c = w.trs + up256(tr * BH * N * 4);
    w.total = w.h0c + (plan.segs > 1 ? BH * P * N * 4 : 0);
    return w;
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <class K>
bool allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return true;
}

// V as (channels, tokens, batch rows): boxes of one head's 64 tokens, tokens
// past the end read as zeros.
bool v_map(CUtensorMap* m, const DeltaParams& d) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d.H * d.P, (cuuint64_t)d.L, (cuuint64_t)d.B};
    const cuuint64_t strides[2] = {(cuuint64_t)d.ldv * 2, (cuuint64_t)d.L * d.ldv * 2};
    const cuuint32_t box[3] = {(cuuint32_t)d.P, kDlC, 1}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(d.v), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int P, bool kFull>
bool launch_walk(const CUtensorMap& tmV, const DeltaChunkParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = DeltaWalkSmem<N, P>::TOTAL;
    if (!allow_smem(delta_walk_kernel<N, P, kFull>, smem, done)) return false;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)p.d.H, (unsigned)p.d.B, (unsigned)(kFull ? p.segs : 2 * p.segs - 3));
    c.blockDim = dim3(kDlThreads, 1, 1);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = pdl;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, delta_walk_kernel<N, P, kFull>, tmV, p) == cudaSuccess;
}
template <int N, int P>
axon_status launch_chunked(const DeltaChunkParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> prep_ok{0};
    if (!allow_smem(delta_prep_kernel<N>, DeltaPrepSmem<N>::TOTAL, prep_ok)) return AXON_ERR_CUDA;
    CUtensorMap tmV;
    if (!v_map(&tmV, p.d)) return AXON_ERR_CUDA;
    delta_prep_kernel<N><<<dim3((unsigned)p.nC, (unsigned)p.d.G, (unsigned)p.d.B), 128, DeltaPrepSmem<N>::TOTAL, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return AXON_ERR_CUDA;
    if (p.segs > 1 && !launch_walk<N, P, false>(tmV, p, st)) return AXON_ERR_CUDA;
    if (!launch_walk<N, P, true>(tmV, p, st)) return AXON_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? AXON_OK : AXON_ERR_CUDA;
}

// Lanes a group and pieces a lane: the fewest lanes (4 .. 32) that hold the
// group in one piece each, then more pieces, then whole blocks.
template <class Io>
void launch_norm(const NormParams& p, cudaStream_t st) {
    const int pieces = p.D / NormVec<Io>::VE;
    auto warps = [&](auto kernel, int LG, int U) {
        const int per_block = 2 * (32 / LG) * U;
        kernel<<<(unsigned)((p.groups + per_block - 1) / per_block), 64, 0, st>>>(p);
    };
    if (pieces <= 4) warps(gated_norm_kernel<Io, 4, 1, 4, 1>, 4, 4);
    else if (pieces <= 8) warps(gated_norm_kernel<Io, 8, 1, 4, 1>, 8, 4);
    else if (pieces <= 16) warps(gated_norm_kernel<Io, 16, 1, 4, 1>, 16, 4);
    else if (pieces <= 32) warps(gated_norm_kernel<Io, 32, 1, 4, 1>, 32, 4);
    else if (pieces <= 64) warps(gated_norm_kernel<Io, 32, 2, 2, 1>, 32, 2);
    else if (pieces <= 128) warps(gated_norm_kernel<Io, 32, 4, 1, 1>, 32, 1);
    else if (pieces <= 512) gated_norm_kernel<Io, 32, 2, 1, 8><<<(unsigned)p.groups, 256, 0, st>>>(p);
    else if (pieces <= 1024) gated_norm_kernel<Io, 32, 4, 1, 8><<<(unsigned)p.groups, 256, 0, st>>>(p);
    else gated_norm_kernel<Io, 32, 8, 1, 8><<<(unsigned)p.groups, 256, 0, st>>>(p);
}

}  // namespace
}  // namespace axon

using namespace axon;

extern "C" {

size_t axon_delta_workspace_bytes(int B, int L, int H, int G, int P, int N, axon_dtype io, int segments) {
    if (B <= 0 || L < 0 || H <= 0 || segments < 0 || !shape_ok(H, G, P, N) || !chunked(B, L, H, P, N, io, segments)) return 0;
    return delta_ws(B, L, H, G, P, N, delta_plan(B, L, H, segments)).total;
}

axon_status axon_delta_scan_fwd(int B, int L, int H, int G, int P, int N, axon_dtype io,
                                const void* q, int ldq, const void* k, int ldk, const void* v, int ldv,
                                const void* dt_raw, const void* b_raw, const float* dt_bias, const float* A_log,
                                const int* lengths, const float* h0, float scale, int qk_norm,
                                void* y, float* h_out, int segments, void* workspace, size_t workspace_bytes,
                                axon_stream_t stream) {
    if (B < 0 || L < 0 || H < 0 || segments < 0) return AXON_ERR_INVALID_ARG;
    if (B > 65535 || H > 65535 || (long long)B * L * H > (1LL << 31)) return AXON_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return AXON_OK;
    const size_t rows = (size_t)B * L;
    const axon_status rc = check_delta(rows, H, G, P, N, io, q, ldq, k, ldk, v, ldv, dt_raw, b_raw, dt_bias, A_log, scale);
    if (rc != AXON_OK) return rc;
    if (!h_out || (rows > 0 && !y)) return AXON_ERR_INVALID_ARG;
    if (!al16(y) || !al16(h_out) || !al16(h0) || !al16(workspace) || (reinterpret_cast<uintptr_t>(lengths) & 3u))
        return AXON_ERR_ALIGNMENT;
    const DeltaPlan plan = delta_plan(B, L, H, segments);
    const DeltaWs w = delta_ws(B, L, H, G, P, N, plan);
    const bool by_chunks = chunked(B, L, H, P, N, io, segments);
    const size_t n_ws = by_chunks ? w.total : 0;
    if (workspace_bytes < n_ws) return AXON_ERR_WORKSPACE;
    if (n_ws > 0 && !workspace) return AXON_ERR_INVALID_ARG;
    const size_t es = io == AXON_BF16 ? 2 : 4;
    const size_t n_h = (size_t)B * H * P * N * 4, n_y = rows * H * P * es, n_g = rows * H * es;
    const struct { const void* p; size_t n; } in[] = {
        {q, extent(rows, (size_t)G * N, ldq, es)}, {k, extent(rows, (size_t)G * N, ldk, es)},
        {v, extent(rows, (size_t)H * P, ldv, es)}, {dt_raw, n_g}, {b_raw, n_g},
        {dt_bias, (size_t)H * 4}, {A_log, (size_t)H * 4}, {lengths, (size_t)B * 4}};
    for (const auto& t : in)
        if (ovl(t.p, t.n, y, n_y) || ovl(t.p, t.n, h_out, n_h) || ovl(t.p, t.n, workspace, n_ws)) return AXON_ERR_INVALID_ARG;
    if (ovl(h0, n_h, y, n_y) || ovl(h0, n_h, workspace, n_ws) || ovl(h_out, n_h, y, n_y) ||
        ovl(h_out, n_h, workspace, n_ws) || ovl(y, n_y, workspace, n_ws))
        return AXON_ERR_INVALID_ARG;
    if (h0 != h_out && ovl(h0, n_h, h_out, n_h)) return AXON_ERR_INVALID_ARG;

    DeltaParams p{B, L, H, G, P, ldq, ldk, ldv, q, k, v, dt_raw, b_raw, dt_bias, A_log, lengths, h0, y, h_out, scale, qk_norm != 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (by_chunks) {
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        const bool split = plan.segs > 1;
        const DeltaChunkParams c{p, (L + kDlC - 1) / kDlC, ws + w.kq, ws + w.blob, reinterpret_cast<int*>(ws + w.err),
                                 plan.segs, plan.cps, reinterpret_cast<float*>(ws + w.sloc), ws + w.tr,
                                 reinterpret_cast<float*>(ws + w.trs), split && h0 ? reinterpret_cast<float*>(ws + w.h0c) : nullptr};
        if (N == 128) return P == 128 ? launch_chunked<128, 128>(c, st) : launch_chunked<128, 64>(c, st);
        return P == 128 ? launch_chunked<64, 128>(c, st) : launch_chunked<64, 64>(c, st);
    }
    if (io == AXON_BF16) N == 128 ? launch_recur<IoBF16, 128>(p, st) : launch_recur<IoBF16, 64>(p, st);
    else N == 128 ? launch_recur<IoF32, 128>(p, st) : launch_recur<IoF32, 64>(p, st);
    return cudaGetLastError() == cudaSuccess ? AXON_OK : AXON_ERR_CUDA;
}

axon_status axon_delta_wait_probe(int* status, int limit, axon_stream_t stream) {
    if (!status || (reinterpret_cast<uintptr_t>(status) & 3u) || limit < 1 || limit > (1 << 16)) return AXON_ERR_INVALID_ARG;
    delta_wait_probe_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(status, limit);
    return cudaGetLastError() == cudaSuccess ? AXON_OK : AXON_ERR_CUDA;
}

axon_status axon_delta_step(int B, int H, int G, int P, int N, axon_dtype io,
                            const void* q, int ldq, const void* k, int ldk, const void* v, int ldv,
                            const void* dt_raw, const void* b_raw, const float* dt_bias, const float* A_log,
                            float scale, int qk_norm, float* state, void* y, axon_stream_t stream) {
    if (B < 0 || H < 0) return AXON_ERR_INVALID_ARG;
    if (B > 65535 || H > 65535) return AXON_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return AXON_OK;
    const axon_status rc = check_delta((size_t)B, H, G, P, N, io, q, ldq, k, ldk, v, ldv, dt_raw, b_raw, dt_bias, A_log, scale);
    if (rc != AXON_OK) return rc;
    if (!state || !y) return AXON_ERR_INVALID_ARG;
    if (!al16(state) || !al16(y)) return AXON_ERR_ALIGNMENT;
    const size_t es = io == AXON_BF16 ? 2 : 4, n_h = (size_t)B * H * P * N * 4, n_y = (size_t)B * H * P * es;
    const struct { const void* p; size_t n; } in[] = {
        {q, extent(B, (size_t)G * N, ldq, es)}, {k, extent(B, (size_t)G * N, ldk, es)},
        {v, extent(B, (size_t)H * P, ldv, es)}, {dt_raw, (size_t)B * H * es}, {b_raw, (size_t)B * H * es},
        {dt_bias, (size_t)H * 4}, {A_log, (size_t)H * 4}};
    for (const auto& t : in)
        if (ovl(t.p, t.n, y, n_y) || ovl(t.p, t.n, state, n_h)) return AXON_ERR_INVALID_ARG;
    if (ovl(state, n_h, y, n_y)) return AXON_ERR_INVALID_ARG;

    DeltaParams p{B, 1, H, G, P, ldq, ldk, ldv, q, k, v, dt_raw, b_raw, dt_bias, A_log, nullptr, state, y, state, scale, qk_norm != 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (io == AXON_BF16) N == 128 ? launch_step<IoBF16, 128>(p, st) : launch_step<IoBF16, 64>(p, st);
    else N == 128 ? launch_step<IoF32, 128>(p, st) : launch_step<IoF32, 64>(p, st);
    return cudaGetLastError() == cudaSuccess ? AXON_OK : AXON_ERR_CUDA;
}

axon_status axon_gated_norm_fwd(int rows, int C, int D, axon_dtype io, axon_norm_kind kind, axon_norm_gate gate, int act,
                                const void* x, int ldx, const void* z, int ldz, const float* weight, const float* bias,
                                int per_channel, float eps, void* y, int ldy, axon_stream_t stream) {
    if (rows < 0 || C < 0 || D <= 0 || C % D) return AXON_ERR_INVALID_ARG;
    if ((io != AXON_F32 && io != AXON_BF16) || (kind != AXON_NORM_RMS && kind != AXON_NORM_GROUP) ||
        (gate != AXON_GATE_NONE && gate != AXON_GATE_AFTER && gate != AXON_GATE_BEFORE))
        return AXON_ERR_UNSUPPORTED;
    // the kernel's group index runs past the last group by less than a few hundred
    if (D > 8192 || (long long)rows * (C / D) > (1LL << 31) - 4096) return AXON_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return AXON_ERR_INVALID_ARG;
    if (rows == 0 || C == 0) return AXON_OK;
    const bool gated = gate != AXON_GATE_NONE;
    if (!x || !y || (gated && !z) || ldx < C || ldy < C || (gated && ldz < C)) return AXON_ERR_INVALID_ARG;
    const int m = io == AXON_BF16 ? 8 : 4;
    if (D % m || ldx % m || ldy % m || (gated && ldz % m)) return AXON_ERR_ALIGNMENT;
    if (!al16(x) || !al16(y) || (gated && !al16(z)) || !al16(weight) || !al16(bias)) return AXON_ERR_ALIGNMENT;
    const size_t es = io == AXON_BF16 ? 2 : 4, n_w = (size_t)(per_channel ? C : D) * 4, n_y = extent(rows, C, ldy, es);
    if (!(y == x && ldy == ldx) && rows_ovl(x, ldx, y, ldy, rows, C, es)) return AXON_ERR_INVALID_ARG;
    if (gated && !(y == z && ldy == ldz) && rows_ovl(z, ldz, y, ldy, rows, C, es)) return AXON_ERR_INVALID_ARG;
    if (ovl(weight, n_w, y, n_y) || ovl(bias, n_w, y, n_y)) return AXON_ERR_INVALID_ARG;

    NormParams p{rows, C, D, rows * (C / D), ldx, ldz, ldy, x, gated ? z : nullptr, weight, bias, per_channel != 0,
                 kind == AXON_NORM_GROUP, gate == AXON_GATE_BEFORE, act != 0, eps, y};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (io == AXON_BF16) launch_norm<IoBF16>(p, st);
    else launch_norm<IoF32>(p, st);
    return cudaGetLastError() == cudaSuccess ? AXON_OK : AXON_ERR_CUDA;
}

}  // extern "C"
