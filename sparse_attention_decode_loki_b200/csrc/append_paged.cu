// Appends to a paged KV-cache with the rotary position embedding on the way:
// the T new keys of every (sequence, KV head) are turned by their position's
// angles, rotated into the head's PCA basis (when there is one) and stored in
// the pages the block table names, in the cache's own type or as 8-bit codes
// with one scale per block of tokens (q8.cuh); the values are stored beside
// them, the first d_lo key columns go to the low-dimensional plane, and the
// step's queries are turned by the same angles.
//
//   pair (a, b) of columns (i, i + r/2), or (2i, 2i + 1) when interleaved, of
//   the token at position j:  a' = a c - b s,  b' = a s + b c,
//   c, s = table[j][i], table[j][r/2 + i];  K~ = rope(K) P.  All in fp32.
//
// An item is the part of one sequence's new tokens that falls into one
// aligned run of `tile` tokens (8 bits: one scale block, so its scale has one
// owner) for one KV head, or a run of query rows. Items are dealt to the grid
// in turn.
#include "launch.h"
#include "q8.cuh"
#include "tma.cuh"

namespace loki {

constexpr int kApThreads = 128;
constexpr int kApRows = 8;  // rows sharing one pass over P

struct ApSpan {
    int64_t lo, hi;    // cache positions of the item's new tokens
    int64_t start;     // first position of the aligned run
    int64_t first;     // the sequence's first appended position
};

// The new tokens of sequence b inside its tile-th aligned run. Tokens outside
// the block table or behind the rope table are left out and flagged.
__device__ __forceinline__ ApSpan append_span(const AppendArgs& a, int b, int64_t tile) {
    const int64_t p0 = a.positions[b];
    int64_t n = a.new_lens != nullptr ? a.new_lens[b] : a.T;
    n = n < 0 ? 0 : (n > a.T ? a.T : n);
    int64_t lo = p0 < 0 ? 0 : p0, hi = p0 + n;
    int64_t lim = (int64_t)a.page_size * a.max_pages;
    if (n > 0 && threadIdx.x == 0 && tile == 0) {
        if (p0 < 0 || hi > lim) atomicExch(a.err, kDevErrBadPage);
        else if (a.rope != nullptr && hi > a.n_pos) atomicExch(a.err, kDevErrRopeRange);
    }
    if (a.rope != nullptr && a.n_pos < lim) lim = a.n_pos;
    hi = hi < lim ? hi : lim;
    ApSpan s;
    s.first = lo;
    s.start = (lo / a.tile + tile) * a.tile;
    s.lo = lo > s.start ? lo : s.start;
    s.hi = hi < s.start + a.tile ? hi : s.start + a.tile;
    return s;
}

// One column of a row at position j after the rotary embedding.
template <class E>
__device__ __forceinline__ float rope_col(const AppendArgs& a, const typename E::T* row, int64_t j,
                                          int c) {
    const float x = E::load1(row + c);
    if (a.rope == nullptr || c >= a.rot_dim) return x;
    const int half = a.rot_dim >> 1;
    const float* cs = a.rope + j * a.rot_dim;
    if (a.interleaved) {
        const float o = E::load1(row + (c ^ 1));
        const float co = __ldg(cs + (c >> 1)), si = __ldg(cs + half + (c >> 1));
        return (c & 1) ? fmaf(o, si, x * co) : fmaf(-o, si, x * co);
    }
    const bool second = c >= half;
    const int i = second ? c - half : c;
    const float o = E::load1(row + (second ? i : c + half));
    const float co = __ldg(cs + i), si = __ldg(cs + half + i);
    return second ? fmaf(o, si, x * co) : fmaf(-o, si, x * co);
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kApThreads / 32; ++w) v = fmaxf(v, red[w]);
    __syncthreads();
    return v;
}

// The rows xs[n][D] into the codes of one scale block: its new scale, older
// codes moved to it when it grew, then the new codes.
__device__ __forceinline__ void store_q8(const float* xs, int n, int D, uint8_t* codes,
                                         float* scale, int first_slot, bool has_old, float* red) {
    float amax = 0.f;
    for (int i = threadIdx.x; i < n * D; i += kApThreads) amax = fmaxf(amax, finite_abs(xs[i]));
    const float grown = pow2_scale(block_max(amax, red));
    const float old = has_old ? *scale : 0.f;
    const float s = has_old ? fmaxf(old, grown) : grown;
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = s;
    if (has_old && s > old) {
        const float f = old / s;
        uint32_t* w = reinterpret_cast<uint32_t*>(codes);
        for (int i = threadIdx.x; i < first_slot * D / 4; i += kApThreads) {
            float v[4];
            e4m3x4_to_float(w[i], v);
            w[i] = to_e4m3x2(v[0] * f, v[1] * f) | to_e4m3x2(v[2] * f, v[3] * f) << 16;
        }
    }
    const float inv = 1.f / s;
    uint32_t* w = reinterpret_cast<uint32_t*>(codes + (int64_t)first_slot * D);
    for (int i = threadIdx.x; i < n * D / 4; i += kApThreads) {
        const float4 v = *reinterpret_cast<const float4*>(xs + 4 * i);
        w[i] = to_e4m3x2(v.x * inv, v.y * inv) | to_e4m3x2(v.z * inv, v.w * inv) << 16;
    }
}

template <class E, bool kQ8>
__global__ void __launch_bounds__(kApThreads) k_append_paged(const AppendArgs a) {
    using Tp = typename E::T;
    extern __shared__ __align__(16) float xs[];  // [tile][D]
    __shared__ float red[kApThreads / 32];
    const int D = a.D, c = threadIdx.x;
    for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
        if (item >= a.kv_items) {  // query rows
            const int64_t r0 = (item - a.kv_items) * kApRows;
            const int64_t rows = (int64_t)a.B * a.H_q * a.T;
            float y[kApRows];
#pragma unroll
            for (int r = 0; r < kApRows; ++r) {
                y[r] = 0.f;
                const int64_t row = r0 + r;
                if (row >= rows || c >= D) continue;
                const int64_t b = row / ((int64_t)a.H_q * a.T), t = row % a.T;
                const int64_t j = (int64_t)a.positions[b] + t;
                const int64_t n = a.new_lens != nullptr ? a.new_lens[b] : a.T;
                if (t >= n || j < 0 || (a.rope != nullptr && j >= a.n_pos)) continue;
                y[r] = rope_col<E>(a, static_cast<const Tp*>(a.q) + row * D, j, c);
            }
            __syncthreads();  // q_out may be q: every column is read before one is written
#pragma unroll
            for (int r = 0; r < kApRows; ++r) {
                const int64_t row = r0 + r;
                if (row >= rows || c >= D) continue;
                const int64_t b = row / ((int64_t)a.H_q * a.T), t = row % a.T;
                const int64_t j = (int64_t)a.positions[b] + t;
                const int64_t n = a.new_lens != nullptr ? a.new_lens[b] : a.T;
                if (t >= n || j < 0 || (a.rope != nullptr && j >= a.n_pos)) continue;
                static_cast<Tp*>(a.q_out)[row * D + c] = E::from_float(y[r]);
            }
            continue;
        }
        const int hk = (int)(item % a.H_kv);
        const int64_t rest = item / a.H_kv;
        const int b = (int)(rest % a.B);
        const ApSpan sp = append_span(a, b, rest / a.B);
        if (sp.lo >= sp.hi) continue;
        const int n = (int)(sp.hi - sp.lo);
        const int64_t t0 = sp.lo - a.positions[b];
        const Tp* Kn = static_cast<const Tp*>(a.K_new) + (((int64_t)b * a.H_kv + hk) * a.T + t0) * D;
        const Tp* Vn = static_cast<const Tp*>(a.V_new) + (((int64_t)b * a.H_kv + hk) * a.T + t0) * D;
        for (int r = 0; r < n; ++r)
            if (c < D) xs[r * D + c] = rope_col<E>(a, Kn + (int64_t)r * D, sp.lo + r, c);
        __syncthreads();
        if (a.P != nullptr) {
            const float* Ph = a.P + (int64_t)hk * D * D + c;
            for (int r0 = 0; r0 < n; r0 += kApRows) {
                float acc[kApRows];
#pragma unroll
                for (int r = 0; r < kApRows; ++r) acc[r] = 0.f;
                if (c < D)
                    for (int i = 0; i < D; ++i) {
                        const float p = __ldg(Ph + (int64_t)i * D);
#pragma unroll
                        for (int r = 0; r < kApRows; ++r)
                            if (r0 + r < n) acc[r] = fmaf(xs[(r0 + r) * D + i], p, acc[r]);
                    }
                __syncthreads();
#pragma unroll
                for (int r = 0; r < kApRows; ++r)
                    if (r0 + r < n && c < D) xs[(r0 + r) * D + c] = acc[r];
            }
            __syncthreads();
        }
        // the page of each row; 8 bits: one page holds the whole block
        auto pool_row = [&](int64_t j) -> int64_t {
            const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + j / a.page_size);
            if (page < 0 || page >= a.n_pages) return -1;
            return ((int64_t)page * a.H_kv + hk) * a.page_size + j % a.page_size;
        };
        for (int r = 0; r < n; ++r) {
            const int64_t row = pool_row(sp.lo + r);
            if (row < 0) {
                if (c == 0) atomicExch(a.err, kDevErrBadPage);
                continue;
            }
            if (a.plane != nullptr && c < a.d_lo)
                static_cast<Tp*>(a.plane)[row * a.d_lo + c] = E::from_float(xs[r * D + c]);
            if (!kQ8 && c < D) {
                static_cast<Tp*>(a.K_pages)[row * D + c] = E::from_float(xs[r * D + c]);
                static_cast<Tp*>(a.V_pages)[row * D + c] = Vn[(int64_t)r * D + c];
            }
        }
        if constexpr (kQ8) {
            const int64_t row = pool_row(sp.start);
            if (row >= 0) {
                const bool has_old = sp.first > sp.start;
                const int slot = (int)(sp.lo - sp.start);
                const int64_t blk = row / a.tile;
                store_q8(xs, n, D, static_cast<uint8_t*>(a.K_pages) + row * D, a.k_scales + blk,
                         slot, has_old, red);
                __syncthreads();
                for (int r = 0; r < n; ++r)
                    if (c < D) xs[r * D + c] = E::load1(Vn + (int64_t)r * D + c);
                __syncthreads();
                store_q8(xs, n, D, static_cast<uint8_t*>(a.V_pages) + row * D, a.v_scales + blk,
                         slot, has_old, red);
            }
        }
        __syncthreads();  // xs is refilled for the next item
    }
}

__global__ void __launch_bounds__(256) k_rope_table(float* __restrict__ table, int64_t n_pos,
                                                    int rot_dim, double base, double pos_scale) {
    const int half = rot_dim >> 1;
    const int64_t n = n_pos * half;
    for (int64_t it = blockIdx.x * 256ll + threadIdx.x; it < n; it += gridDim.x * 256ll) {
        const int64_t j = it / half;
        const int i = (int)(it % half);
        double s, c;
        sincos((double)j * pos_scale * pow(base, -2.0 * i / rot_dim), &s, &c);
        table[j * rot_dim + i] = (float)c;
        table[j * rot_dim + half + i] = (float)s;
    }
}

// ---------------------------------------------------------------------------

template <class E, bool kQ8>
static cudaError_t append_impl(const AppendArgs& a, cudaStream_t s) {
    auto kern = k_append_paged<E, kQ8>;
    const size_t smem = (size_t)a.tile * a.D * sizeof(float);
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 128 * 4);
    if (e != cudaSuccess) return e;
    const int64_t wave = (int64_t)di.sm_count * occupancy((const void*)kern, kApThreads, smem);
    return launch_kernel(kern, dim3((unsigned)min64(a.items, wave * 8)), dim3(kApThreads), smem, s,
                         false, a);
}

cudaError_t launch_append_paged(Dt dt, AppendArgs a, cudaStream_t s) {
    a.err = device_error_word();
    if (a.err == nullptr) return cudaErrorInvalidDevice;
    const bool q8 = a.block > 0;
    a.tile = q8 ? a.block : 16;
    const int64_t tiles = ((int64_t)a.T + a.tile - 2) / a.tile + 1;
    a.kv_items = tiles * a.B * a.H_kv;
    a.items = a.kv_items;
    if (a.q != nullptr) a.items += ((int64_t)a.B * a.H_q * a.T + kApRows - 1) / kApRows;
    if (dt == kF32) return q8 ? append_impl<ElemF32, true>(a, s) : append_impl<ElemF32, false>(a, s);
    return q8 ? append_impl<ElemBF16, true>(a, s) : append_impl<ElemBF16, false>(a, s);
}

cudaError_t launch_rope_table(float* table, int64_t n_pos, int rot_dim, double base,
                              double pos_scale, cudaStream_t s) {
    const int64_t n = n_pos * (rot_dim >> 1);
    return launch_kernel(k_rope_table, dim3((unsigned)min64((n + 255) / 256, 148 * 16)), dim3(256), 0,
                         s, false, table, n_pos, rot_dim, base, pos_scale);
}

}  // namespace loki
