// Attention of one query token per sequence over the paged 8-bit cache
// (q8.cuh), over all of a sequence's tokens (dense) or over each query head's
// selected ones (Loki's last step).
//
//   a_j = scale q . (s_K(j) cK_j),  p = softmax over the row's tokens,
//   out = sum_j p_j s_V(j) cV_j;  a row without tokens gives zeros.
//
// One CTA per (sequence, query head) row: its warps take tokens in turn, a
// lane holds four columns, the softmax runs online in base 2 in fp32, and the
// warps' states are merged in shared memory.
#include "launch.h"
#include "q8.cuh"
#include "tma.cuh"

namespace loki {

constexpr int kQ8Warps = 8;

template <class E>
__global__ void __launch_bounds__(kQ8Warps * 32) k_attend_q8(const AttendQ8Args a) {
    __shared__ float sm_m[kQ8Warps], sm_l[kQ8Warps], sm_acc[kQ8Warps][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x;
    const int b = (int)(r / a.H_q), h = (int)(r % a.H_q), hk = h / (a.H_q / a.H_kv);
    const int D = a.D, c = lane * 4;
    const int64_t cap = (int64_t)a.page_size * a.max_pages;
    int64_t len = a.seq_lens[b];
    len = len < 0 ? 0 : (len > cap ? cap : len);
    const int64_t n = a.idx != nullptr ? a.k : len;
    float q[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < D)
        for (int e = 0; e < 4; ++e)
            q[e] = (a.q_f32 ? static_cast<const float*>(a.q)[r * D + c + e]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[r * D + c + e])) *
                   a.scale_log2;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t t = warp; t < n; t += kQ8Warps) {
        const int64_t j = a.idx != nullptr ? (int64_t)a.idx[r * a.k + t] : t;
        if (j < 0 || j >= len) continue;
        const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + j / a.page_size);
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) atomicExch(a.err, kDevErrBadPage);
            continue;
        }
        const int64_t row = ((int64_t)page * a.H_kv + hk) * a.page_size + j % a.page_size;
        float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
        if (c < D) {
            e4m3x4_to_float(__ldg(reinterpret_cast<const uint32_t*>(a.K_pages + row * D + c)), k);
            e4m3x4_to_float(__ldg(reinterpret_cast<const uint32_t*>(a.V_pages + row * D + c)), v);
        }
        float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
        x = group_sum<32>(x) * __ldg(a.k_scales + row / a.block);
        const float vs = __ldg(a.v_scales + row / a.block);
        const float M = fmaxf(m, x);
        const float al = m == M ? 1.f : exp2f(m - M), p = exp2f(x - M);
        l = l * al + p;
        for (int e = 0; e < 4; ++e) acc[e] = acc[e] * al + p * (v[e] * vs);
        m = M;
    }
    for (int e = 0; e < 4; ++e) sm_acc[warp][c + e] = acc[e];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
    __syncthreads();
    const int col = threadIdx.x;
    if (col >= D) return;
    float M = -INFINITY, L = 0.f, A = 0.f;
    for (int w = 0; w < kQ8Warps; ++w) M = fmaxf(M, sm_m[w]);
    if (M != -INFINITY)
        for (int w = 0; w < kQ8Warps; ++w) {
            const float s = exp2f(sm_m[w] - M);
            L += sm_l[w] * s;
            A += sm_acc[w][col] * s;
        }
    static_cast<typename E::T*>(a.out)[r * D + col] = E::from_float(L > 0.f ? A / L : 0.f);
}

size_t dense_q8_ws_bytes(int, int, int, int64_t, int) { return 256; }
size_t sparse_q8_ws_bytes(int, int, int64_t, int) { return 256; }

cudaError_t launch_attend_q8(Dt out_dt, AttendQ8Args a, cudaStream_t s) {
    a.err = device_error_word();
    if (a.err == nullptr) return cudaErrorInvalidDevice;
    const dim3 grid((unsigned)((int64_t)a.B * a.H_q));
    return out_dt == kF32
               ? launch_kernel(k_attend_q8<ElemF32>, grid, dim3(kQ8Warps * 32), 0, s, false, a)
               : launch_kernel(k_attend_q8<ElemBF16>, grid, dim3(kQ8Warps * 32), 0, s, false, a);
}

}  // namespace loki
