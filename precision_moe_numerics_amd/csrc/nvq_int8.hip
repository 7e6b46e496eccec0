// nvq_int8.hip -- the expert layer and the dense product in 8-bit integers:
// symmetric codes with one scale per row (a token, or an output channel of the
// weights), beside the NVFP4, MXFP8 and BF16 forms of the same products. The
// products themselves are the BF16 ones' kernels with int8 operands
// (nvq_gemm16.hpp); here are the quantizer and the host side.
#include "nvq_gemm16.hpp"

#include <algorithm>

namespace nvq {
namespace {
using namespace g16;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ quantize
// Per row: a = max |x|, scale = a / 127, code = 127 x / a to the nearest even.
//
// The quotient q = 127 x / a of two bf16 values decides exactly. 127 x has 15
// significant bits and a has 8, so a quotient that is no tie n + 1/2 lies at
// least 2^-16 of itself away from one, and a tie is an fp32 number. It is found
// from the reciprocal with one correction: q0 = y r, q = q0 + (y - q0 a) r. The
// residual in the middle is exact (24 bits of q0 times 8 of a, of which the
// upper 22 cancel), so q is the fp32 nearest to the quotient to within 2^-45 of
// it before its rounding: a tie comes out as itself and nothing else on or across
// one. a and x are first scaled by the power of two that takes a to [1, 2).
//
// A row that holds an infinity or NaN gets a NaN scale and zero codes: all that
// is computed from it is NaN. An all-zero row gets scale 1.
struct RowQuant {
    float a, r, scale;
    int shift;
    bool live;
    __device__ __forceinline__ explicit RowQuant(uint32_t top) {  // the row's largest |x| as bf16 bits
        const float m = __uint_as_float(top << 16);
        const bool finite = top < 0x7F80u;
        live = finite && top != 0;
        shift = live ? -(int)(__builtin_amdgcn_frexp_expf(m) - 1) : 0;
        a = live ? __builtin_amdgcn_ldexpf(m, shift) : 1.0f;
        r = __builtin_amdgcn_rcpf(a);
        scale = !finite ? __builtin_nanf("") : top ? m / 127.0f : 1.0f;
    }
    // the code in the low byte: adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the mantissa
    __device__ __forceinline__ uint32_t code(float x) const {
        const float y = __builtin_amdgcn_ldexpf(x, shift) * 127.0f;
        const float q0 = y * r;
        const float q = __builtin_fmaf(__builtin_fmaf(-q0, a, y), r, q0);
        return live ? __float_as_uint(q + 12582912.0f) : 0u;
    }
    __device__ __forceinline__ uint2 codes8(u32x4 w) const {
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = code(__uint_as_float(w[i] << 16));
            c[2 * i + 1] = code(__uint_as_float(w[i] & 0xFFFF0000u));
        }
        auto pack = [](const uint32_t* v) {
            const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], 0x04000C0Cu);
            return lo | hi;
        };
        return make_uint2(pack(c), pack(c + 4));
    }
};

// Largest magnitude so far, as pairs of bf16 bits (which order as the values do; NaN above infinity).
__device__ __forceinline__ uint32_t pair_max(uint32_t m, u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u16x2 v = __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu), o = __builtin_bit_cast(u16x2, m);
        m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(v, o));
    }
    return m;
}

// W waves per row (1 or 4, of 4 in the workgroup); a row of up to 512 P W values is read once and held in registers, P = 0
// reads it twice. Rows at or past *limit (not NULL) are left alone. Bound by HBM: 2 bytes read and one written per value.
template <int P, int W>
__global__ __launch_bounds__(256) void k_int8_rows(const uint16_t* __restrict__ x, int64_t R, int C,
                                                   const int32_t* __restrict__ limit, int8_t* __restrict__ codes,
                                                   float* __restrict__ scales) {
    __shared__ uint32_t red[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * (4 / W) + (W == 1 ? wave : 0);
    const int64_t rows = limit ? min(R, (int64_t)max(*limit, 0)) : R;
    if (row >= rows) return;  // whole waves (W = 4: the whole workgroup)
    const int units = C / 8, u0 = W == 1 ? lane : (int)threadIdx.x;
    const u32x4* src = reinterpret_cast<const u32x4*>(x + row * C);
    uint2* dst = reinterpret_cast<uint2*>(codes + row * C);
    constexpr int S = 64 * W;
    u32x4 v[P ? P : 1];
    uint32_t m = 0;
    if (P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            v[i] = (u32x4){0, 0, 0, 0};
            if (u0 + i * S < units) v[i] = src[u0 + i * S];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) m = pair_max(m, v[i]);
    } else {
#pragma unroll 4
        for (int u = u0; u < units; u += S) m = pair_max(m, src[u]);
    }
    uint32_t top = wave_max_u32(max(m & 0xFFFFu, m >> 16));
    if (W > 1) {
        if (lane == 0) red[wave] = top;
        __syncthreads();
        top = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    const RowQuant q(top);
    if (u0 == 0) scales[row] = q.scale;
    if (P) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (u0 + i * S < units) dst[u0 + i * S] = q.codes8(v[i]);
    } else {
#pragma unroll 4
        for (int u = u0; u < units; u += S) dst[u] = q.codes8(src[u]);
    }
}

template <int W>
void launch_rows_w(const uint16_t* x, int64_t R, int C, const int32_t* limit, int8_t* codes, float* scales,
                   hipStream_t s) {
    const dim3 grid((unsigned)((R + 4 / W - 1) / (4 / W)));
    const int per = (C / 8 + 64 * W - 1) / (64 * W);
#define NVQ_ROWS(P_) hipLaunchKernelGGL((k_int8_rows<P_, W>), grid, dim3(256), 0, s, x, R, C, limit, codes, scales)
    if (per <= 1) NVQ_ROWS(1);
    else if (per <= 2) NVQ_ROWS(2);
    else if (W == 1 || per <= 4) NVQ_ROWS(4);  // (W = 1: C <= 2048)
    else if constexpr (W > 1) {
        if (per <= 8) NVQ_ROWS(8);
        else NVQ_ROWS(0);
    }
#undef NVQ_ROWS
}
// A wave per row, or four where rows are long, or few: a wave of its own has less to wait for at the row's end, four have
// more loads under way. us with one, with four: 4 x 4096 3.9, 3.0; 1024 x 1536 3.9, 3.8; 1024 x 2048 4.2, 4.1; 4096 x 1536
// 6.8, 7.3; 4096 x 2048 8.8, 9.0; 32768 x 2048 39, 46; 65536 x 256 20, 43; 4096 x 2560 10.5, 10.1; 4096 x 4096 14.3, 13.1;
// 16384 x 4096 42.6, 38.8 (201 MB: 5.2 TB/s); 16384 x 8192 112, 79.
void launch_int8_rows(const uint16_t* x, int64_t R, int64_t C, const int32_t* limit, int8_t* codes, float* scales,
                      hipStream_t s) {
    if (R <= 1024 || C > 2048) launch_rows_w<4>(x, R, (int)C, limit, codes, scales, s);
    else launch_rows_w<1>(x, R, (int)C, limit, codes, scales, s);
}

// ------------------------------------------------------------------ dequantize
// 16 values per thread: out = code * scale, one fp32 rounding, then bf16 if asked. Bound by HBM: 16384 x 4096 to bf16, 201 MB,
// 38.8 us, 5.2 TB/s (31.5 behind the quantizer, whose codes are still in the caches); to fp32, 335 MB, 87 us, 3.9 TB/s, where a
// lane's four stores lie 64 bytes from its neighbour's.
template <bool F32>
__global__ __launch_bounds__(256) void k_int8_values(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                     uint32_t n16, uint32_t c16, void* __restrict__ out) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= n16) return;
    const float s = scales[u / c16];
    const u32x4 w = reinterpret_cast<const u32x4*>(codes)[u];
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * s;
    if (F32) {
        f32x4* o = static_cast<f32x4*>(out) + (size_t)u * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (f32x4){v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    } else {
        u32x4* o = static_cast<u32x4*>(out) + (size_t)u * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            o[i] = (u32x4){bf16x2_rne(v[8 * i], v[8 * i + 1]), bf16x2_rne(v[8 * i + 2], v[8 * i + 3]),
                           bf16x2_rne(v[8 * i + 4], v[8 * i + 5]), bf16x2_rne(v[8 * i + 6], v[8 * i + 7])};
    }
}

// ------------------------------------------------------------------ host side
// The quantizer's limits; rows are then also within the dequantizer's.
bool rows_ok(int64_t R, int64_t C) {
    return R >= 0 && C >= 16 && C % 16 == 0 && C <= (1 << 22) && R < ((int64_t)1 << 31) && grid_ok(R, 256);
}
bool gemm8_dims_ok(bool glu, int64_t rows, int64_t E, int64_t N, int64_t K) {
    return K >= 16 && K % 16 == 0 && K < (1 << 17) && gemm16_dims_ok(kFwd, glu, rows, E, 0, N, K / 2);
}
bool fc1_dims_ok(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    if (T < 0 || k < 1 || E < 1 || k > E || T > ((int64_t)1 << 31) / k) return false;
    return gemm8_dims_ok(true, T * k, E, d_ff, d) && T * d <= kMaxBytes;
}
bool fwd_dims_ok(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    return fc1_dims_ok(T, d, k, E, d_ff) && gemm8_dims_ok(false, T * k, E, d, d_ff) && rows_ok(T, d) &&
           rows_ok(T * k, d_ff);
}

Args operands(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, int64_t E, int64_t rows,
              int64_t N, int64_t K) {
    Args p{};
    p.a = reinterpret_cast<const uint16_t*>(a);
    p.b = reinterpret_cast<const uint16_t*>(b);
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    p.a_div = p.b_div = 1;
    p.lda = p.ldb = p.K = (int32_t)(K / 2);
    p.E = (int32_t)E; p.rows = (int32_t)rows; p.N = (int32_t)N;
    return p;
}
Args fc1_args(const int8_t* xq, const float* xs, int64_t T, int64_t d, const int32_t* offsets, const int32_t* s2a, int k,
              int64_t E, int64_t d_ff, const int8_t* w1, const float* w1s, uint16_t* h) {
    Args p = operands(xq, xs, w1, w1s, E, T * k, d_ff, d);
    p.a_gather = s2a;
    p.a_div = (uint32_t)k;
    p.a_bytes = T * d;
    p.seg = offsets;
    p.out = h;
    return p;
}
Args fc2_args(const int8_t* hq, const float* hs, int64_t A, int64_t d_ff, const int32_t* offsets, const int32_t* s2a,
              int64_t E, int64_t d, const int8_t* w2, const float* w2s, uint16_t* y) {
    Args p = operands(hq, hs, w2, w2s, E, A, d, d_ff);
    p.seg = offsets;
    p.scatter = s2a;
    p.out = y;
    return p;
}

struct Fwd8 {
    uint32_t* rws;
    void* gws;
    int32_t *offsets, *s2a;
    uint16_t* h;
    int8_t *xq, *hq;
    float *xs, *hs;
};
size_t fwd_carve(Carver& c, int64_t T, int64_t d, int k, int64_t E, int64_t d_ff, const nvq_moe_buffers* b, Fwd8* o) {
    const int64_t A = std::max<int64_t>(T * k, 1), t = std::max<int64_t>(T, 1);
    nvq_moe_buffers z{};
    const nvq_moe_buffers& in = b ? *b : z;
    o->rws = c.take<uint32_t>(route_ws_words(A, E));
    o->gws = c.take<uint8_t>(gemm8_ws_bytes(A, E));
    o->offsets = in.offsets ? in.offsets : c.take<int32_t>((size_t)E + 1);
    o->s2a = in.sorted2assign ? in.sorted2assign : c.take<int32_t>((size_t)A);
    o->h = in.h ? in.h : c.take<uint16_t>((size_t)(A * d_ff));
    o->xq = in.xq_codes ? reinterpret_cast<int8_t*>(in.xq_codes) : c.take<int8_t>((size_t)(t * d));
    o->xs = in.xq_tscale ? in.xq_tscale : c.take<float>((size_t)t);
    o->hq = in.hq_codes ? reinterpret_cast<int8_t*>(in.hq_codes) : c.take<int8_t>((size_t)(A * d_ff));
    o->hs = in.hq_tscale ? in.hq_tscale : c.take<float>((size_t)A);
    return c.need;
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" {

int int8_quantize(const uint16_t* x, int64_t R, int64_t C, int8_t* codes, float* scales, nvq_stream_t stream) {
    if (!rows_ok(R, C)) return NVQ_ERR_DIM;
    if (R > 0 && (!x || !codes || !scales)) return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return NVQ_ERR_ALIGN;
    if (R == 0) return NVQ_OK;
    launch_int8_rows(x, R, C, nullptr, codes, scales, as_stream(stream));
    return launch_status();
}

int int8_dequantize(const int8_t* codes, const float* scales, int64_t R, int64_t C, void* out, int out_dtype,
                    nvq_stream_t stream) {
    if (out_dtype != NVQ_OUT_BF16 && out_dtype != NVQ_OUT_F32) return NVQ_ERR_UNSUPPORTED;
    if (!rows_ok(R, C) || R * (C / 16) >= ((int64_t)1 << 32) - 256) return NVQ_ERR_DIM;
    if (R > 0 && (!codes || !scales || !out)) return NVQ_ERR_NULL;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return NVQ_ERR_ALIGN;
    if (R == 0) return NVQ_OK;
    const uint32_t n16 = (uint32_t)(R * (C / 16)), c16 = (uint32_t)(C / 16);
    const dim3 grid((n16 + 255) / 256);
    hipStream_t s = as_stream(stream);
    if (out_dtype == NVQ_OUT_F32)
        hipLaunchKernelGGL(k_int8_values<true>, grid, dim3(256), 0, s, codes, scales, n16, c16, out);
    else
        hipLaunchKernelGGL(k_int8_values<false>, grid, dim3(256), 0, s, codes, scales, n16, c16, out);
    return launch_status();
}

int linear_act_int8(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales, const float* bias,
                    const uint16_t* residual, int64_t M, int64_t N, int64_t K, int act, void* out, int out_dtype,
                    nvq_stream_t stream) {
    if (act < NVQ_ACT_NONE || act > NVQ_ACT_SWIGLU || (out_dtype != NVQ_OUT_BF16 && out_dtype != NVQ_OUT_F32))
        return NVQ_ERR_UNSUPPORTED;
    if (residual && residual == out && out_dtype != NVQ_OUT_BF16) return NVQ_ERR_UNSUPPORTED;  // rows would overlap others
    const bool glu = act == NVQ_ACT_SWIGLU;
    if (!gemm8_dims_ok(glu, M, 1, N, K) || M * N >= ((int64_t)1 << 40)) return NVQ_ERR_DIM;
    if (!wq || !w_scales || (M > 0 && (!xq || !x_scales || !out))) return NVQ_ERR_NULL;
    if (!aligned16(xq) || !aligned16(x_scales) || !aligned16(wq) || !aligned16(w_scales) || !aligned16(bias) ||
        !aligned16(residual) || !aligned16(out))
        return NVQ_ERR_ALIGN;
    Args p = operands(xq, x_scales, wq, w_scales, 1, M, N, K);
    p.out = out; p.bias = bias; p.residual = residual;
    p.out_f32 = out_dtype == NVQ_OUT_F32;
    p.act = act;
    launch_gemm8(glu ? kEpiGlu : kEpiAct, p, nullptr, as_stream(stream));
    return launch_status();
}

int moe_fc1_swiglu_int8(const int8_t* xq, const float* x_scales, int64_t T, int64_t d, const int32_t* offsets,
                        const int32_t* sorted2assign, int k, int64_t E, int64_t d_ff, const int8_t* w1,
                        const float* w1_scales, uint16_t* h, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    if (!fc1_dims_ok(T, d, k, E, d_ff)) return NVQ_ERR_DIM;
    if (!offsets || !w1 || !w1_scales || !ws || (T > 0 && (!xq || !x_scales || !sorted2assign || !h))) return NVQ_ERR_NULL;
    if (!aligned16(xq) || !aligned16(x_scales) || !aligned16(w1) || !aligned16(w1_scales) || !aligned16(h) ||
        !aligned256(ws))
        return NVQ_ERR_ALIGN;
    if (ws_bytes < gemm8_ws_bytes(T * k, E)) return NVQ_ERR_WORKSPACE;
    launch_gemm8(kEpiGlu, fc1_args(xq, x_scales, T, d, offsets, sorted2assign, k, E, d_ff, w1, w1_scales, h), ws,
                 as_stream(stream));
    return launch_status();
}

int moe_fc2_int8(const int8_t* hq, const float* h_scales, int64_t A, int64_t d_ff, const int32_t* offsets,
                 const int32_t* sorted2assign, int64_t E, int64_t d, const int8_t* w2, const float* w2_scales,
                 uint16_t* y, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    if (!gemm8_dims_ok(false, A, E, d, d_ff)) return NVQ_ERR_DIM;
    if (!offsets || !w2 || !w2_scales || !ws || (A > 0 && (!hq || !h_scales || !sorted2assign || !y))) return NVQ_ERR_NULL;
    if (!aligned16(hq) || !aligned16(h_scales) || !aligned16(w2) || !aligned16(w2_scales) || !aligned16(y) ||
        !aligned256(ws))
        return NVQ_ERR_ALIGN;
    if (ws_bytes < gemm8_ws_bytes(A, E)) return NVQ_ERR_WORKSPACE;
    launch_gemm8(kEpiOut, fc2_args(hq, h_scales, A, d_ff, offsets, sorted2assign, E, d, w2, w2_scales, y), ws,
                 as_stream(stream));
    return launch_status();
}

size_t moe_gemm_int8_workspace_size(int64_t A, int64_t E) { return gemm8_ws_bytes(A, E); }

size_t moe_expert_fwd_int8_workspace_size(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    if (T < 0 || d < 0 || k < 1 || E < 1 || d_ff < 0) return 0;
    Carver c(nullptr);
    Fwd8 o;
    return fwd_carve(c, T, d, k, E, d_ff, nullptr, &o);
}

int moe_expert_fwd_int8(const uint16_t* x, int64_t T, int64_t d, const int32_t* topk_ids, int k, int64_t E,
                        int64_t d_ff, const int8_t* w1, const float* w1_scales, const int8_t* w2,
                        const float* w2_scales, uint16_t* y, const nvq_moe_buffers* bufs, void* ws, size_t ws_bytes,
                        nvq_stream_t stream) {
    if (!fwd_dims_ok(T, d, k, E, d_ff)) return NVQ_ERR_DIM;
    if (!w1 || !w1_scales || !w2 || !w2_scales || !ws || (T > 0 && (!x || !topk_ids || !y))) return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1) || !aligned16(w1_scales) || !aligned16(w2) || !aligned16(w2_scales) ||
        !aligned16(y) || !aligned256(ws))
        return NVQ_ERR_ALIGN;
    if (bufs) {
        if (bufs->xq_scales || bufs->hq_scales || bufs->gu || bufs->gemm_workgroups) return NVQ_ERR_UNSUPPORTED;
        if (!aligned16(bufs->h) || !aligned16(bufs->xq_codes) || !aligned16(bufs->xq_tscale) ||
            !aligned16(bufs->hq_codes) || !aligned16(bufs->hq_tscale))
            return NVQ_ERR_ALIGN;
    }
    Fwd8 m;
    Carver need(nullptr);
    if (ws_bytes < fwd_carve(need, T, d, k, E, d_ff, bufs, &m)) return NVQ_ERR_WORKSPACE;
    if (T == 0 && !(bufs && bufs->offsets)) return NVQ_OK;  // (a caller's offsets become all 0, by the routing)
    Carver cv(ws);
    fwd_carve(cv, T, d, k, E, d_ff, bufs, &m);
    hipStream_t s = as_stream(stream);
    if (T > 0) launch_int8_rows(x, T, d, nullptr, m.xq, m.xs, s);
    launch_route(topk_ids, T * k, E, m.offsets, m.s2a, nullptr, nullptr, 128, m.rws, s);
    if (T == 0) return launch_status();
    launch_gemm8(kEpiGlu, fc1_args(m.xq, m.xs, T, d, m.offsets, m.s2a, k, E, d_ff, w1, w1_scales, m.h), m.gws, s);
    launch_int8_rows(m.h, T * k, d_ff, m.offsets + E, m.hq, m.hs, s);
    launch_gemm8(kEpiOut, fc2_args(m.hq, m.hs, T * k, d_ff, m.offsets, m.s2a, E, d, w2, w2_scales, y), m.gws, s);
    return launch_status();
}

}  // extern "C"
