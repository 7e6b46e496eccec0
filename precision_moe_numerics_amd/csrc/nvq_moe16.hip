// nvq_moe16.hip -- the expert layer in BF16: grouped products (forward, the
// gradients of the rows and of the weights), fc1 with SwiGLU and the whole
// expert forward, beside the NVFP4 and MXFP8 forms of the same layer.
#include "nvq_gemm16.hpp"

#include <algorithm>

using namespace nvq;
using namespace nvq::g16;

// Bytes of a gathered source: one buffer descriptor with 32-bit lane offsets.
static bool gather_ok(const int32_t* gather, int64_t rows, int64_t ld, int32_t div) {
    return !gather || (div >= 1 && rows >= 0 && rows * ld * 2 <= kMaxBytes);
}

static size_t fwd16_carve(Carver& c, int64_t T, int k, int64_t E, int64_t d_ff, const nvq_moe_buffers* b,
                          uint32_t** rws, void** gws, nvq_moe_buffers* out) {
    const int64_t A = std::max<int64_t>(T * k, 1);
    nvq_moe_buffers z{};
    const nvq_moe_buffers& in = b ? *b : z;
    *rws = c.take<uint32_t>(route_ws_words(A, E));
    *gws = c.take<uint8_t>(gemm16_ws_bytes(A, E));
    out->offsets = in.offsets ? in.offsets : c.take<int32_t>((size_t)E + 1);
    out->sorted2assign = in.sorted2assign ? in.sorted2assign : c.take<int32_t>((size_t)A);
    out->h = in.h ? in.h : c.take<uint16_t>((size_t)(A * d_ff));
    out->gu = in.gu;
    return c.need;
}

static bool fc1_dims_ok(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    if (T < 0 || k < 1 || E < 1 || k > E || T > ((int64_t)1 << 31) / k) return false;
    return gemm16_dims_ok(kFwd, true, T * k, E, 0, d_ff, d) && T * d * 2 <= kMaxBytes;
}
static bool fwd16_dims_ok(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    return fc1_dims_ok(T, d, k, E, d_ff) && gemm16_dims_ok(kFwd, false, T * k, E, 0, d, d_ff);
}

static Args fc1_args(const uint16_t* x, int64_t T, int64_t d, const int32_t* offsets, const int32_t* s2a, int k,
                     int64_t E, int64_t d_ff, const uint16_t* w1, uint16_t* h, uint16_t* gu) {
    Args p{};
    p.a = x; p.b = w1;
    p.a_gather = s2a; p.a_div = (uint32_t)k; p.a_bytes = T * d * 2;
    p.seg = offsets;
    p.out = h; p.z = gu;
    p.lda = p.ldb = (int32_t)d;
    p.E = (int32_t)E; p.rows = (int32_t)(T * k); p.N = (int32_t)d_ff; p.K = (int32_t)d;
    return p;
}

extern "C" {

size_t moe_grouped_gemm_bf16_workspace_size(int mode, int64_t E, int64_t R) {
    return mode == NVQ_WGRAD ? 256 : gemm16_ws_bytes(R, E);
}

int moe_grouped_gemm_bf16(int mode, const uint16_t* a, int64_t a_rows, const int32_t* a_gather, int32_t a_div,
                          const uint16_t* b, int64_t b_rows, const int32_t* b_gather, int32_t b_div,
                          const int32_t* seg_offsets, int64_t E, int64_t R, int64_t M, int64_t N, int64_t K,
                          void* out, const int32_t* out_scatter, int out_dtype, int accumulate, void* ws,
                          size_t ws_bytes, nvq_stream_t stream) {
    if (mode != NVQ_FWD && mode != NVQ_DGRAD && mode != NVQ_WGRAD) return NVQ_ERR_UNSUPPORTED;
    if (out_dtype != NVQ_OUT_BF16 && out_dtype != NVQ_OUT_F32) return NVQ_ERR_UNSUPPORTED;
    const bool wg = mode == NVQ_WGRAD;
    if (wg ? out_scatter != nullptr : (accumulate || b_gather)) return NVQ_ERR_UNSUPPORTED;
    const int md = wg ? kWgrad : mode == NVQ_DGRAD ? kDgrad : kFwd;
    if (!gemm16_dims_ok(md, false, R, E, M, N, K)) return NVQ_ERR_DIM;
    const bool rows = R > 0;
    if ((rows && (!a || (wg && !b))) || (!wg && !b) || !seg_offsets || ((rows || wg) && !out) || !ws) return NVQ_ERR_NULL;
    if (!gather_ok(a_gather, a_rows, wg ? M : K, a_div) || !gather_ok(b_gather, b_rows, N, b_div)) return NVQ_ERR_DIM;
    if ((!a_gather && a_rows < R) || (wg && !b_gather && b_rows < R)) return NVQ_ERR_DIM;
    if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned256(ws)) return NVQ_ERR_ALIGN;
    if (ws_bytes < moe_grouped_gemm_bf16_workspace_size(mode, E, R)) return NVQ_ERR_WORKSPACE;
    Args p{};
    p.a = a; p.b = b;
    p.a_gather = a_gather; p.a_div = (uint32_t)std::max(a_div, 1);
    p.b_gather = b_gather; p.b_div = (uint32_t)std::max(b_div, 1);
    p.lda = (int32_t)(wg ? M : K);
    p.ldb = (int32_t)(mode == NVQ_FWD ? K : N);
    p.a_bytes = a_rows * p.lda * 2;
    p.b_bytes = b_rows * p.ldb * 2;
    p.seg = seg_offsets;
    p.scatter = out_scatter;
    p.out = out;
    p.E = (int32_t)E; p.rows = (int32_t)R; p.M = (int32_t)M; p.N = (int32_t)N; p.K = (int32_t)K;
    p.out_f32 = out_dtype == NVQ_OUT_F32;
    p.accumulate = accumulate != 0;
    launch_gemm16(md, kEpiOut, p, ws, as_stream(stream));
    return launch_status();
}

size_t moe_fc1_bf16_workspace_size(int64_t A, int64_t E) { return gemm16_ws_bytes(A, E); }

int moe_fc1_swiglu_bf16(const uint16_t* x, int64_t T, int64_t d, const int32_t* offsets,
                        const int32_t* sorted2assign, int k, int64_t E, int64_t d_ff, const uint16_t* w1,
                        uint16_t* h, uint16_t* gu, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    if (!fc1_dims_ok(T, d, k, E, d_ff)) return NVQ_ERR_DIM;
    if (!offsets || !w1 || !ws || (T > 0 && (!x || !sorted2assign || !h))) return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1) || !aligned16(h) || !aligned16(gu) || !aligned256(ws)) return NVQ_ERR_ALIGN;
    if (ws_bytes < moe_fc1_bf16_workspace_size(T * k, E)) return NVQ_ERR_WORKSPACE;
    launch_gemm16(kFwd, kEpiGlu, fc1_args(x, T, d, offsets, sorted2assign, k, E, d_ff, w1, h, gu), ws,
                  as_stream(stream));
    return launch_status();
}

size_t moe_expert_fwd_bf16_workspace_size(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    (void)d;
    if (T < 0 || k < 1 || E < 1 || d_ff < 0) return 0;
    Carver c(nullptr);
    uint32_t* r;
    void* g;
    nvq_moe_buffers o{};
    return fwd16_carve(c, T, k, E, d_ff, nullptr, &r, &g, &o);
}

int moe_expert_fwd_bf16(const uint16_t* x, int64_t T, int64_t d, const int32_t* topk_ids, int k, int64_t E,
                        int64_t d_ff, const uint16_t* w1, const uint16_t* w2, uint16_t* y,
                        const nvq_moe_buffers* bufs, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    if (!fwd16_dims_ok(T, d, k, E, d_ff)) return NVQ_ERR_DIM;
    if (!w1 || !w2 || !ws || (T > 0 && (!x || !topk_ids || !y))) return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) || !aligned256(ws)) return NVQ_ERR_ALIGN;
    if (bufs) {
        if (bufs->xq_codes || bufs->xq_scales || bufs->xq_tscale || bufs->hq_codes || bufs->hq_scales ||
            bufs->hq_tscale || bufs->gemm_workgroups)
            return NVQ_ERR_UNSUPPORTED;
        if (!aligned16(bufs->h) || !aligned16(bufs->gu)) return NVQ_ERR_ALIGN;
    }
    uint32_t* rws;
    void* gws;
    nvq_moe_buffers m{};
    Carver need(nullptr);
    if (ws_bytes < fwd16_carve(need, T, k, E, d_ff, bufs, &rws, &gws, &m)) return NVQ_ERR_WORKSPACE;
    if (T == 0 && !(bufs && bufs->offsets)) return NVQ_OK;  // (a caller's offsets become all 0, by the routing)
    Carver cv(ws);
    fwd16_carve(cv, T, k, E, d_ff, bufs, &rws, &gws, &m);
    hipStream_t s = as_stream(stream);
    // expert segments, then fc1 + SwiGLU on gathered token rows, then fc2
    // scattered back to (token, slot) order
    launch_route(topk_ids, T * k, E, m.offsets, m.sorted2assign, nullptr, nullptr, 128, rws, s);
    launch_gemm16(kFwd, kEpiGlu, fc1_args(x, T, d, m.offsets, m.sorted2assign, k, E, d_ff, w1, m.h, m.gu), gws, s);
    Args p{};
    p.a = m.h; p.b = w2;
    p.a_div = p.b_div = 1;
    p.seg = m.offsets;
    p.scatter = m.sorted2assign;
    p.out = y;
    p.lda = p.ldb = (int32_t)d_ff;
    p.E = (int32_t)E; p.rows = (int32_t)(T * k); p.N = (int32_t)d; p.K = (int32_t)d_ff;
    launch_gemm16(kFwd, kEpiOut, p, gws, s);
    return launch_status();
}

}  // extern "C"
