// nvq_combine16.hip -- the weighted combine of BF16 expert outputs with its
// backward, and the backward of the two routers: what joins the grouped
// products into a trainable expert layer.
#include "nvq_device.hpp"
#include "nvq_host.hpp"

namespace nvq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kNowhere = 0xFFFFFFE0u;  // past every descriptor: the load returns zeros, reads nothing

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0xFFFFFE00u, 0x00020000);
}

__device__ __forceinline__ void unpack8(i32x4 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float((uint32_t)w[i] << 16);
        v[2 * i + 1] = __uint_as_float((uint32_t)w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ i32x4 pack8(const float (&v)[8]) {
    return (i32x4){(int)bf16x2_rne(v[0], v[1]), (int)bf16x2_rne(v[2], v[3]), (int)bf16x2_rne(v[4], v[5]),
                   (int)bf16x2_rne(v[6], v[7])};
}

constexpr int kSlots = 8;  // slots whose loads are in flight together

// out[t] = residual[t] + sum_s w[t][s] y[t][s], in fp32 in slot order, rounded
// once. One thread owns 8 columns of one token; the slots' loads of a group of
// eight go out together. A dropped slot (id outside [0, E)) loads from past the
// descriptor: zeros without memory traffic, so what its row of y holds (fc2
// never wrote it) does not matter.
__global__ __launch_bounds__(256) void k_combine16(const uint16_t* __restrict__ y, const float* __restrict__ w,
                                                   const int32_t* __restrict__ ids, int E,
                                                   const uint16_t* __restrict__ residual, int64_t T, int k, int C8,
                                                   uint16_t* __restrict__ out) {
    const int64_t u0 = (int64_t)blockIdx.x * 256;
    const int64_t t0 = u0 / C8;  // the workgroup's first token: descriptor base
    const int64_t u = u0 + threadIdx.x;
    if (u >= T * C8) return;
    const int32_t rel = (int32_t)(u - t0 * C8);
    const int dt = rel / C8, c8 = rel % C8;
    const int64_t t = t0 + dt;
    const __amdgpu_buffer_rsrc_t ry = rsrc_of(y + t0 * k * C8 * 8);
    const uint32_t row = (uint32_t)C8 * 16u;
    const uint32_t base = (uint32_t)dt * (uint32_t)k * row + (uint32_t)c8 * 16u;
    float acc[8] = {};
    for (int s0 = 0; s0 < k; s0 += kSlots) {
        i32x4 v[kSlots];
        float ws[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int s = s0 + j;
            bool ok = s < k;
            const int64_t a = t * k + (ok ? s : 0);
            if (ids) ok = ok && (uint32_t)ids[a] < (uint32_t)E;
            ws[j] = ok ? w[a] : 0.0f;
            v[j] = __builtin_amdgcn_raw_buffer_load_b128(ry, ok ? base + (uint32_t)s * row : kNowhere, 0, 2);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(ws[j], f[i], acc[i]);
        }
    }
    if (residual) {
        float f[8];
        unpack8(reinterpret_cast<const i32x4*>(residual)[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    reinterpret_cast<i32x4*>(out)[u] = pack8(acc);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// dy[t][s] = w[t][s] dout[t] in bf16, dw[t][s] = <dout[t], y[t][s]> in fp32:
// y and dout are read once and dy written once. W waves share a token, each
// lane takes every (64 W)-th group of 8 columns; the lanes' partial sums are
// added by a fixed butterfly and the waves' in order. A dropped slot gets
// dy = 0, dw = 0 and its row of y is not read.
template <int W>
__global__ __launch_bounds__(256) void k_combine16_bwd(const uint16_t* __restrict__ dout,
                                                       const uint16_t* __restrict__ y, const float* __restrict__ w,
                                                       const int32_t* __restrict__ ids, int E, int64_t T, int k,
                                                       int C8, uint16_t* __restrict__ dy, float* __restrict__ dw) {
    __shared__ float red[4][kSlots];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t t = (int64_t)blockIdx.x * (4 / W) + wave / W;
    const bool live = t < T;
    if (W == 1 && !live) return;
    const int64_t tt = live ? t : 0;
    const __amdgpu_buffer_rsrc_t ry = rsrc_of(y + tt * k * C8 * 8);
    const uint32_t row = (uint32_t)C8 * 16u;
    const i32x4* dp = reinterpret_cast<const i32x4*>(dout) + tt * C8;
    i32x4* dyp = reinterpret_cast<i32x4*>(dy) + tt * k * C8;
    for (int s0 = 0; s0 < k; s0 += kSlots) {
        float ws[kSlots], sum[kSlots];
        bool ok[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int s = s0 + j;
            ok[j] = live && s < k;
            const int64_t a = tt * k + (s < k ? s : 0);
            if (ids) ok[j] = ok[j] && (uint32_t)ids[a] < (uint32_t)E;
            ws[j] = ok[j] ? w[a] : 0.0f;
            sum[j] = 0.0f;
        }
        for (int c = (wave % W) * 64 + lane; live && c < C8; c += 64 * W) {
            float d[8];
            i32x4 v[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                v[j] = __builtin_amdgcn_raw_buffer_load_b128(
                    ry, ok[j] ? (uint32_t)(s0 + j) * row + (uint32_t)c * 16u : kNowhere, 0, 2);
            unpack8(dp[c], d);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (s0 + j >= k) break;
                float f[8], o[8];
                unpack8(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum[j] = __builtin_fmaf(d[i], f[i], sum[j]);
                    o[i] = ok[j] ? ws[j] * d[i] : 0.0f;
                }
                __builtin_nontemporal_store(pack8(o), dyp + (int64_t)(s0 + j) * C8 + c);
            }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) sum[j] = ok[j] ? wave_sum(sum[j]) : 0.0f;
        if (W > 1) {
            if (s0) __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < kSlots; ++j) red[wave][j] = sum[j];
            __syncthreads();
            if (threadIdx.x < kSlots && s0 + (int)threadIdx.x < k && live)
                dw[t * k + s0 + threadIdx.x] = (red[0][threadIdx.x] + red[1][threadIdx.x]) +
                                               (red[2][threadIdx.x] + red[3][threadIdx.x]);
        } else {
            float mine = sum[0];
#pragma unroll
            for (int j = 1; j < kSlots; ++j) mine = lane == j ? sum[j] : mine;
            if (lane < kSlots && s0 + lane < k) dw[t * k + s0 + lane] = mine;
        }
    }
}

// dlogits of the top-k weights. With D = sum_i w_i dw_i:
//   softmax over the chosen logits: g_j = w_j (dw_j - D);
//   w_j = s_j / S, s_j = sigmoid(logit_j): g_j = w_j (1 - s_j) (dw_j - D).
// One wave per token, lane j the j-th chosen expert. The token's row is laid
// out in LDS (zeros, then the k gradients; ids that occur twice have been added
// up in slot order, so both lanes write the same sum) and written once, 16
// bytes a lane where rows start on 16 bytes. Ids outside [0, E) write nothing.
constexpr int kRouterE = 1024;
template <bool SIGMOID, bool V4>
__global__ __launch_bounds__(256) void k_router_bwd(const float* __restrict__ w, const float* __restrict__ logits,
                                                    const int32_t* __restrict__ ids, const float* __restrict__ dw,
                                                    int64_t T, int E, int k, float* __restrict__ dlogits) {
    __shared__ __attribute__((aligned(16))) float rows[4][kRouterE];
    const int lane = threadIdx.x & 63, wave = (int)(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= T) return;  // whole waves; no barrier below
    float* row = rows[wave];
    int id = -1;
    float wj = 0.0f, dj = 0.0f, f = 1.0f;
    if (lane < k) {
        id = ids[t * k + lane];
        wj = w[t * k + lane];
        dj = dw[t * k + lane];
        if (SIGMOID && (uint32_t)id < (uint32_t)E)  // 1 - sigmoid(v) = 1 / (1 + exp(v))
            f = 1.0f / (1.0f + __expf(logits[t * E + id]));
    }
    for (int c = lane * 4; c < E; c += 256) *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float D = wave_sum(wj * dj);
    const float g = wj * f * (dj - D);
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int idj = __builtin_amdgcn_readlane(id, j);
        const float gj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(g), j));
        sum += idj == id ? gj : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();  // one wave's LDS accesses complete in order
    if (lane < k && (uint32_t)id < (uint32_t)E) row[id] = sum;
    __builtin_amdgcn_wave_barrier();
    float* out = dlogits + t * E;
    if (V4) {
        for (int c = lane * 4; c < E; c += 256)
            *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(row + c);
    } else {
        for (int c = lane; c < E; c += 64) out[c] = row[c];
    }
}

template <bool SIGMOID>
void launch_router_bwd(const float* w, const float* logits, const int32_t* ids, const float* dw, int64_t T, int64_t E,
                       int k, float* dlogits, hipStream_t s) {
    const dim3 grid((unsigned)((T + 3) / 4));
    if (E % 4 == 0 && aligned16(dlogits))
        hipLaunchKernelGGL((k_router_bwd<SIGMOID, true>), grid, dim3(256), 0, s, w, logits, ids, dw, T, (int)E, k,
                           dlogits);
    else
        hipLaunchKernelGGL((k_router_bwd<SIGMOID, false>), grid, dim3(256), 0, s, w, logits, ids, dw, T, (int)E, k,
                           dlogits);
}

// The rows of y that one workgroup addresses from its descriptor's base (the
// tokens its 256 threads touch) below 4 GiB.
bool combine_dims_ok(int64_t T, int k, int64_t C, int64_t E, bool ids) {
    const int64_t i31 = (int64_t)1 << 31;
    if (T < 0 || T >= i31 || k < 1 || k > 1024 || C < 8 || C % 8 != 0 || C > (1 << 20) || (ids && (E < 1 || E >= i31)))
        return false;
    if (T * k >= i31 || (int64_t)k * (256 + 2 * (C / 8)) * 16 > (int64_t)kNowhere) return false;
    return true;
}

bool router_dims_ok(int64_t T, int64_t E, int k) {
    return T >= 0 && k >= 1 && E >= 1 && k <= E && k <= 64 && E <= 1024 && T * E < ((int64_t)1 << 31) &&
           grid_ok((T + 3) / 4, 256);
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" {

int moe_combine_bf16(const uint16_t* y, const float* w, const int32_t* topk_ids, int64_t E, const uint16_t* residual,
                     int64_t T, int k, int64_t C, uint16_t* out, nvq_stream_t stream) {
    if (!combine_dims_ok(T, k, C, E, topk_ids != nullptr)) return NVQ_ERR_DIM;
    if (T > 0 && (!y || !w || !out)) return NVQ_ERR_NULL;
    if (!aligned16(y) || !aligned16(residual) || !aligned16(out)) return NVQ_ERR_ALIGN;
    if (T == 0) return NVQ_OK;
    const int C8 = (int)(C / 8);
    const int64_t grid = (T * C8 + 255) / 256;
    if (!grid_ok(grid, 256)) return NVQ_ERR_DIM;
    hipLaunchKernelGGL(k_combine16, dim3((unsigned)grid), dim3(256), 0, as_stream(stream), y, w, topk_ids, (int)E,
                       residual, T, k, C8, out);
    return launch_status();
}

int moe_combine_bwd_bf16(const uint16_t* dout, const uint16_t* y, const float* w, const int32_t* topk_ids, int64_t E,
                         int64_t T, int k, int64_t C, uint16_t* dy, float* dw, nvq_stream_t stream) {
    if (!combine_dims_ok(T, k, C, E, topk_ids != nullptr)) return NVQ_ERR_DIM;
    if (T > 0 && (!dout || !y || !w || !dy || !dw)) return NVQ_ERR_NULL;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(dy)) return NVQ_ERR_ALIGN;
    if (T == 0) return NVQ_OK;
    const int C8 = (int)(C / 8);
    if (!grid_ok(C8 <= 128 ? (T + 3) / 4 : T, 256)) return NVQ_ERR_DIM;
    hipStream_t s = as_stream(stream);
    if (C8 <= 128)
        hipLaunchKernelGGL(k_combine16_bwd<1>, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, s, dout, y, w, topk_ids,
                           (int)E, T, k, C8, dy, dw);
    else
        hipLaunchKernelGGL(k_combine16_bwd<4>, dim3((unsigned)T), dim3(256), 0, s, dout, y, w, topk_ids, (int)E, T, k,
                           C8, dy, dw);
    return launch_status();
}

int moe_router_softmax_topk_bwd(const float* w, const int32_t* topk_ids, const float* dw, int64_t T, int64_t E,
                                int k, float* dlogits, nvq_stream_t stream) {
    if (!router_dims_ok(T, E, k)) return NVQ_ERR_DIM;
    if (T > 0 && (!w || !topk_ids || !dw || !dlogits)) return NVQ_ERR_NULL;
    if (T == 0) return NVQ_OK;
    launch_router_bwd<false>(w, nullptr, topk_ids, dw, T, E, k, dlogits, as_stream(stream));
    return launch_status();
}

int moe_router_sigmoid_topk_bwd(const float* w, const float* logits, const int32_t* topk_ids, const float* dw,
                                int64_t T, int64_t E, int k, float* dlogits, nvq_stream_t stream) {
    if (!router_dims_ok(T, E, k)) return NVQ_ERR_DIM;
    if (T > 0 && (!w || !logits || !topk_ids || !dw || !dlogits)) return NVQ_ERR_NULL;
    if (T == 0) return NVQ_OK;
    launch_router_bwd<true>(w, logits, topk_ids, dw, T, E, k, dlogits, as_stream(stream));
    return launch_status();
}

}  // extern "C"
