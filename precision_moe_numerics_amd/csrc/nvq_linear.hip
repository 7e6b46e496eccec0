// nvq_linear.hip -- the dense product with bias, activation and residual in
// its epilogue, and its backward: the gradient of the pre-activation with the
// bias gradient in one pass, then the two products with it.
//
// That gradient, dz, is rounded to bf16 once, as the operand of both products
// (the bias gradient takes it unrounded): the layer's operands are bf16, and a
// second bf16 term for what the rounding drops would double both products, 133
// of 151 us at 4091 x 1024 x 4096 SwiGLU. It costs 2.3e-3 of the 2-norm of dx
// and a bf16 dw there, where the rounding of the results alone is 1.7e-3, and
// 1.7e-3 of an fp32 dw. Without an activation a caller can split an fp32 dout.
#include "nvq_gemm16.hpp"

#include <algorithm>

namespace nvq {
namespace {
using namespace g16;

// dz of one value pair: dout * act'(z); SwiGLU handles (g, u) itself.
template <int ACT>
__device__ __forceinline__ float act_bwd(float dout, float z) {
    if (ACT == NVQ_ACT_RELU) return z > 0.0f ? dout : 0.0f;
    if (ACT == NVQ_ACT_GELU) {
        const NormTail n(z);
        return dout * (n.phi(z) + z * (0.39894228040143268f * n.e));
    }
    if (ACT == NVQ_ACT_GELU_TANH) {
        const float q = sigmoidf(1.5957691216057308f * (z + 0.044715f * z * z * z));
        // (past |z| = 2^64 the square would be inf, times q (1 - q) = 0)
        return dout * (q + z * q * (1.0f - q) * 1.5957691216057308f * (1.0f + 0.134145f * fminf(z * z, 1e30f)));
    }
    if (ACT == NVQ_ACT_SILU) {
        const float s = sigmoidf(z);
        return dout * (s * (1.0f + z * (1.0f - s)));
    }
    return dout;
}

constexpr int kBwdCols = 512;  // columns of a workgroup: 64 lanes x 8
// Rows of a workgroup, a multiple of its 4 waves: 64, or 16 where that would leave compute units without work (4091 x
// 1024 SwiGLU: 23 us with 64, 128 workgroups; 10 with 16). Each costs one row of partial sums.
inline int bwd_rows(int64_t M, int64_t N) { return (M / 64) * ((N + kBwdCols - 1) / kBwdCols) >= 1024 ? 64 : 16; }
constexpr int kFoldWaves = 16; // row blocks folded side by side

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
                                              bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}

// dz [M, R] = dout * act'(z) in bf16 (R = N, SwiGLU 2 N; not written when dz
// is NULL) and, when part is not NULL, the column sums of the unrounded fp32
// dz over this workgroup's rows: part[row block][R]. A lane owns 8 columns
// and walks rows wave, wave + 4, ...; the four waves' sums are added in order
// through LDS, so the result does not depend on timing.
template <int ACT, bool F32>
__global__ __launch_bounds__(256) void k_act_bwd(const void* __restrict__ dout, const uint16_t* __restrict__ z,
                                                 int64_t M, int N, int rows, uint16_t* __restrict__ dz,
                                                 float* __restrict__ part) {
    constexpr bool GLU = ACT == NVQ_ACT_SWIGLU;
    constexpr int H = GLU ? 2 : 1;
    __shared__ float red[4][64 * 8 * H];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned col_blocks = ((unsigned)N + kBwdCols - 1) / kBwdCols;
    const int64_t rb = blockIdx.x / col_blocks;
    const int c0 = (int)(blockIdx.x % col_blocks) * kBwdCols, c = c0 + lane * 8;
    const int64_t R = (int64_t)N * H;
    const int64_t r0 = rb * rows, r1 = min(r0 + rows, M);
    float sum[H][8] = {};
    if (c < N) {
        for (int64_t r = r0 + wave; r < r1; r += 4) {
            float d[8], g[8], u[8], o[8];
            if (F32) {
                const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(dout) + r * N + c);
                const float4 a = q[0], b = q[1];
                d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w; d[4] = b.x; d[5] = b.y; d[6] = b.z; d[7] = b.w;
            } else {
                load8(static_cast<const uint16_t*>(dout) + r * N + c, d);
            }
            if (ACT != NVQ_ACT_NONE) load8(z + r * R + c, g);
            if (GLU) load8(z + r * R + N + c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (GLU) {
                    const float s = sigmoidf(g[i]);
                    o[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
                    u[i] = d[i] * g[i] * s;
                    sum[H - 1][i] += u[i];
                } else {
                    o[i] = act_bwd<ACT>(d[i], g[i]);
                }
                sum[0][i] += o[i];
            }
            if (dz) {
                store8(dz + r * R + c, o);
                if (GLU) store8(dz + r * R + N + c, u);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[wave][h * 512 + lane * 8 + i] = sum[h][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 512 * H; i += 256) {
        const int col = c0 + (i & 511);
        if (col < N)
            part[rb * R + (int64_t)(i >> 9) * N + col] =
                (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
    }
}

// dbias[c] (+)= sum of part[b][c] over the row blocks: wave w of the workgroup
// adds blocks w, w + 16, .. of 64 columns, then the waves' sums are added in
// order.
__global__ __launch_bounds__(64 * kFoldWaves) void k_fold_bias(const float* __restrict__ part, int64_t nb, int64_t R,
                                                               int accumulate, float* __restrict__ dbias) {
    __shared__ float red[kFoldWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < R) {
#pragma unroll 8
        for (int64_t b = wave; b < nb; b += kFoldWaves) s += part[b * R + c];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= R) return;
#pragma unroll
    for (int w = 1; w < kFoldWaves; ++w) s += red[w][lane];
    dbias[c] = accumulate ? dbias[c] + s : s;
}

template <int ACT>
void launch_act_bwd(const void* dout, bool f32, const uint16_t* z, int64_t M, int64_t N, uint16_t* dz, float* part,
                    hipStream_t s) {
    const int rows = bwd_rows(M, N);
    const dim3 grid((unsigned)((N + kBwdCols - 1) / kBwdCols * ((M + rows - 1) / rows)));
    if (f32) hipLaunchKernelGGL((k_act_bwd<ACT, true>), grid, dim3(256), 0, s, dout, z, M, (int)N, rows, dz, part);
    else hipLaunchKernelGGL((k_act_bwd<ACT, false>), grid, dim3(256), 0, s, dout, z, M, (int)N, rows, dz, part);
}

bool act_ok(int act) { return act >= NVQ_ACT_NONE && act <= NVQ_ACT_SWIGLU; }
bool linear_dims_ok(int64_t M, int64_t N, int64_t K, int act) {
    const bool glu = act == NVQ_ACT_SWIGLU;
    return gemm16_dims_ok(kFwd, glu, M, 1, 0, N, K) && M * N < ((int64_t)1 << 40);
}

size_t bwd_carve(Carver& c, int64_t M, int64_t N, int64_t R, uint16_t** dz, float** part) {
    const int rows = bwd_rows(M, N);
    *dz = c.take<uint16_t>((size_t)(M * R));
    *part = c.take<float>((size_t)((M + rows - 1) / rows * R));
    return c.need;
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" {

int linear_act_bf16(const uint16_t* x, const uint16_t* w, const float* bias, const uint16_t* residual, int64_t M,
                    int64_t N, int64_t K, int act, void* out, int out_dtype, uint16_t* z, nvq_stream_t stream) {
    if (!act_ok(act) || (out_dtype != NVQ_OUT_BF16 && out_dtype != NVQ_OUT_F32)) return NVQ_ERR_UNSUPPORTED;
    if (residual && residual == out && out_dtype != NVQ_OUT_BF16) return NVQ_ERR_UNSUPPORTED;  // rows would overlap others
    if (!linear_dims_ok(M, N, K, act)) return NVQ_ERR_DIM;
    if (!w || (M > 0 && (!x || !out))) return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(out) ||
        !aligned16(z))
        return NVQ_ERR_ALIGN;
    Args p{};
    p.a = x; p.b = w;
    p.a_div = p.b_div = 1;
    p.out = out; p.bias = bias; p.residual = residual; p.z = z;
    p.lda = p.ldb = (int32_t)K;
    p.E = 1; p.rows = (int32_t)M; p.N = (int32_t)N; p.K = (int32_t)K;
    p.out_f32 = out_dtype == NVQ_OUT_F32;
    p.act = act;
    launch_gemm16(kFwd, act == NVQ_ACT_SWIGLU ? kEpiGlu : kEpiAct, p, nullptr, as_stream(stream));
    return launch_status();
}

size_t linear_act_bwd_bf16_workspace_size(int64_t M, int64_t N, int64_t K, int act) {
    (void)K;
    Carver c(nullptr);
    uint16_t* dz;
    float* part;
    M = std::max<int64_t>(M, 0);
    N = std::max<int64_t>(N, 0);
    return bwd_carve(c, M, N, N * (act == NVQ_ACT_SWIGLU ? 2 : 1), &dz, &part);
}

int linear_act_bwd_bf16(const void* dout, int dout_dtype, const uint16_t* x, const uint16_t* w, const uint16_t* z,
                        int64_t M, int64_t N, int64_t K, int act, uint16_t* dx, void* dw, int dw_dtype,
                        int accumulate, float* dbias, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    if (!act_ok(act) || (dout_dtype != NVQ_OUT_BF16 && dout_dtype != NVQ_OUT_F32) ||
        (dw_dtype != NVQ_OUT_BF16 && dw_dtype != NVQ_OUT_F32))
        return NVQ_ERR_UNSUPPORTED;
    const bool glu = act == NVQ_ACT_SWIGLU;
    const int64_t R = glu ? 2 * N : N;
    if (!linear_dims_ok(M, N, K, act) || !gemm16_dims_ok(kDgrad, false, M, 1, 0, K, R) ||
        !gemm16_dims_ok(kWgrad, false, M, 1, R, K, 0) ||
        !grid_ok((N + kBwdCols - 1) / kBwdCols * ((M + bwd_rows(M, N) - 1) / bwd_rows(M, N)), 256))
        return NVQ_ERR_DIM;
    if (!ws || (M > 0 && !dx && !dw && !dbias) || (dx && !w)) return NVQ_ERR_NULL;
    if (M > 0 && (!dout || (dw && !x) || (act != NVQ_ACT_NONE && !z))) return NVQ_ERR_NULL;
    if (!aligned16(dout) || !aligned16(x) || !aligned16(w) || !aligned16(z) || !aligned16(dx) || !aligned16(dw) ||
        !aligned16(dbias) || !aligned256(ws))
        return NVQ_ERR_ALIGN;
    if (ws_bytes < linear_act_bwd_bf16_workspace_size(M, N, K, act)) return NVQ_ERR_WORKSPACE;
    if (M == 0 && !dw && !dbias) return NVQ_OK;
    hipStream_t s = as_stream(stream);
    Carver cv(ws);
    uint16_t* dz;
    float* part;
    bwd_carve(cv, M, N, R, &dz, &part);
    // without an activation a bf16 dout is dz itself
    const bool same = act == NVQ_ACT_NONE && dout_dtype == NVQ_OUT_BF16;
    const bool need_dz = !same && (dx || dw);
    if (M > 0 && (need_dz || dbias)) {
        uint16_t* to = need_dz ? dz : nullptr;
        float* pt = dbias ? part : nullptr;
        const bool f32 = dout_dtype == NVQ_OUT_F32;
        switch (act) {
            case NVQ_ACT_RELU: launch_act_bwd<NVQ_ACT_RELU>(dout, f32, z, M, N, to, pt, s); break;
            case NVQ_ACT_GELU: launch_act_bwd<NVQ_ACT_GELU>(dout, f32, z, M, N, to, pt, s); break;
            case NVQ_ACT_GELU_TANH: launch_act_bwd<NVQ_ACT_GELU_TANH>(dout, f32, z, M, N, to, pt, s); break;
            case NVQ_ACT_SILU: launch_act_bwd<NVQ_ACT_SILU>(dout, f32, z, M, N, to, pt, s); break;
            case NVQ_ACT_SWIGLU: launch_act_bwd<NVQ_ACT_SWIGLU>(dout, f32, z, M, N, to, pt, s); break;
            default: launch_act_bwd<NVQ_ACT_NONE>(dout, f32, z, M, N, to, pt, s); break;
        }
        NVQ_CHECK_LAUNCH();
    }
    if (dbias && (M > 0 || !accumulate))  // (no rows add nothing: old + 0 would turn -0 into +0)
        hipLaunchKernelGGL(k_fold_bias, dim3((unsigned)((R + 63) / 64)), dim3(64 * kFoldWaves), 0, s, part,
                           (M + bwd_rows(M, N) - 1) / bwd_rows(M, N), R, accumulate, dbias);
    const uint16_t* dzp = same ? static_cast<const uint16_t*>(dout) : dz;
    Args p{};
    p.a = dzp;
    p.a_div = p.b_div = 1;
    p.E = 1; p.rows = (int32_t)M;
    if (dx && M > 0) {
        p.b = w; p.out = dx;
        p.lda = (int32_t)R; p.ldb = (int32_t)K;
        p.N = (int32_t)K; p.K = (int32_t)R;
        launch_gemm16(kDgrad, kEpiOut, p, nullptr, s);
    }
    if (dw) {
        p.b = x; p.out = dw;
        p.lda = (int32_t)R; p.ldb = (int32_t)K;
        p.M = (int32_t)R; p.N = (int32_t)K; p.K = 0;
        p.out_f32 = dw_dtype == NVQ_OUT_F32;
        p.accumulate = accumulate != 0;
        launch_gemm16(kWgrad, kEpiOut, p, nullptr, s);
    }
    return launch_status();
}

}  // extern "C"
