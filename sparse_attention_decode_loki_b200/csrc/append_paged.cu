// Appends to a paged KV-cache with the rotary position embedding on the way
// (append_paged.cuh has the formulas): values, queries and keys without a
// basis as streams; keys of a few tokens against the basis row by row. Longer
// appends rotate their keys in append_basis.cu.
#include "append_paged.cuh"

namespace loki {

// ---------------------------------------------------------------------------
// Streams: keys (no basis), values and queries, one read and one write of each
// row. Bytes bound them.
//
// A warp takes an aligned run of 16 tokens of one head: eight lanes to a row
// (16 columns each), four rows at a time, all loads issued before the first
// use. 8-bit scale blocks of more than 16 tokens belong to block / 16
// neighbouring warps, which share their largest magnitude through shared
// memory; so every scale has one owner and every row is read once. Warps side
// by side take the heads of one run, whose rows of the angle table they share
// in the L1.

constexpr int kStThreads = 256;

enum { kKindKeys, kKindValues, kKindQueries };

template <class E, bool kQ8>
__global__ void __launch_bounds__(kStThreads, 2) k_append_stream(const AppendArgs a) {
    using Tp = typename E::T;
    __shared__ float red[kStThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gw = kQ8 ? a.block >> 4 : 1;  // warps of a task
    const int u = lane & 7;
    const bool lane_on = u < a.D >> 4;
    int64_t task = ((int64_t)blockIdx.x * (kStThreads / 32) + warp) / gw;
    const int sub = warp & (gw - 1);
    int kind = kKindKeys, heads = a.H_kv;
    if (task >= a.key_tasks) {
        task -= a.key_tasks;
        kind = kKindValues;
        if (task >= a.value_tasks) {
            task -= a.value_tasks;
            kind = kKindQueries;
            heads = a.H_q;
        }
    }
    const bool on = task < (kind == kKindKeys ? a.key_tasks : kind == kKindValues ? a.value_tasks : a.query_tasks);
    const int h = (int)(task % heads);
    const int64_t rest = task / heads;
    const int b = (int)(rest % a.B);
    const int64_t ri = rest / a.B;  // which run of the sequence's
    const int run = 16 * gw;
    float x[4][16];
    int row[4];
    bool live[4];
    float amax = 0.f, old = 0.f;
    int64_t first = 0, start = 0, j0 = 0;
    bool any = false, has_old = false;
    int block_row = -1, ca = 0, cb = 0;
    if (on) {
        ApSeq sq = append_seq(a, b, kind == kKindValues && ri == 0 && lane == 0 && sub == 0);
        if (kind == kKindQueries) {  // not bound to the cache's places
            int64_t n = a.new_lens != nullptr ? __ldg(a.new_lens + b) : a.T;
            n = n > a.T ? a.T : n;
            sq.hi = sq.p0 + n;
            if (a.rope != nullptr && a.n_pos < sq.hi) sq.hi = a.n_pos;
        }
        first = sq.lo;
        start = (sq.lo / run + ri) * run;
        j0 = start + sub * 16;
        const void* src = kind == kKindKeys ? a.K_new : kind == kKindValues ? a.V_new : a.q;
        const Tp* rows = static_cast<const Tp*>(src) + ((int64_t)b * heads + h) * a.T * a.D;
        const bool turn = kind != kKindValues && a.rope != nullptr && u < a.rot_dim >> 4;
        unit_cols(turn ? a.rot_dim : 0, a.interleaved, u, &ca, &cb);
        Chunk<E> wa[4], wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = j0 + 4 * i + (lane >> 3);
            live[i] = lane_on && j >= sq.lo && j < sq.hi;
            if (live[i]) {
                const Tp* p = rows + (j - sq.p0) * a.D;
                wa[i].load(p + ca);
                wb[i].load(p + cb);
            }
        }
        any = start < sq.hi && start + run > sq.lo;
        if (kind != kKindQueries) {
            if constexpr (kQ8) {  // one page holds the whole block
                if (any && j0 < (int64_t)a.page_size * a.max_pages) {
                    block_row = pool_row(a, b, h, (int)start);
                    has_old = first > start;
                    if (block_row >= 0 && has_old)
                        old = (kind == kKindKeys ? a.k_scales : a.v_scales)[block_row >> a.block_log2];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    row[i] = live[i] ? pool_row(a, b, h, (int)(j0 + 4 * i + (lane >> 3))) : -1;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!live[i]) continue;
            const int64_t j = j0 + 4 * i + (lane >> 3);
            if (kind == kKindValues && !kQ8) {  // values in their own type: copied, bit by bit
                if (row[i] < 0) continue;
                Tp* o = static_cast<Tp*>(a.V_pages) + (int64_t)row[i] * a.D;
#pragma unroll
                for (int e = 0; e < Chunk<E>::kN; ++e) {
                    reinterpret_cast<uint4*>(o + ca)[e] = wa[i].w[e];
                    reinterpret_cast<uint4*>(o + cb)[e] = wb[i].w[e];
                }
                continue;
            }
            wa[i].get(x[i]);
            wb[i].get(x[i] + 8);
            if (turn) turn_unit(a.rope, a.rot_dim, a.interleaved, j, u, x[i]);
            if (kind == kKindQueries) {
                Tp* o = static_cast<Tp*>(a.q_out) + (((int64_t)b * heads + h) * a.T + (j - sq.p0)) * a.D;
                store_chunk<E>(o + ca, x[i], ca, a.D);
                store_chunk<E>(o + cb, x[i] + 8, cb, a.D);
                continue;
            }
            const int64_t r = kQ8 ? (block_row < 0 ? -1 : block_row + (j - start)) : row[i];
            if (r < 0) continue;
            if (!kQ8) {
                Tp* o = static_cast<Tp*>(a.K_pages) + r * a.D;
                store_chunk<E>(o + ca, x[i], ca, a.D);
                store_chunk<E>(o + cb, x[i] + 8, cb, a.D);
            }
            if (kind == kKindKeys && a.plane != nullptr) {
                Tp* o = static_cast<Tp*>(a.plane) + r * a.d_lo;
                store_chunk<E>(o + ca, x[i], ca, a.d_lo);
                store_chunk<E>(o + cb, x[i] + 8, cb, a.d_lo);
            }
            if constexpr (kQ8) {
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(x[i][e]));
            }
        }
        if constexpr (kQ8) {
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            if (lane == 0) red[warp] = amax;
        }
    }
    if constexpr (kQ8) {
        __syncthreads();  // and every warp has read the old scale
        if (block_row >= 0) {
            for (int w = warp - sub; w < warp - sub + gw; ++w) amax = fmaxf(amax, red[w]);
            const float grown = pow2_scale(amax);
            const float s = has_old ? fmaxf(old, grown) : grown;
            if (sub == 0 && lane == 0)
                (kind == kKindKeys ? a.k_scales : a.v_scales)[block_row >> a.block_log2] = s;
            uint8_t* pages = static_cast<uint8_t*>(kind == kKindKeys ? a.K_pages : a.V_pages);
            const float inv = 1.f / s, f = old / s;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t j = j0 + 4 * i + (lane >> 3);
                uint8_t* o = pages + (block_row + (j - start)) * a.D;
                if (live[i]) {
                    *reinterpret_cast<uint2*>(o + ca) = codes8(x[i], inv);
                    *reinterpret_cast<uint2*>(o + cb) = codes8(x[i] + 8, inv);
                } else if (lane_on && has_old && s > old && j < first) {  // older codes to the new scale
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint2* w = reinterpret_cast<uint2*>(o + (e ? cb : ca));
                        uint2 v = *w;
                        v.x = rescale4(v.x, f);
                        v.y = rescale4(v.y, f);
                        *w = v;
                    }
                }
            }
        }
    }
    // as a programmatic dependent of the keys' kernel: end after it
    griddep_wait();
}

// ---------------------------------------------------------------------------
// Few tokens (a decode step) against the basis. Latency bounds it: one CTA
// per KV head and group of sequences, at most 16 rows. A quarter of a basis
// column sits in each thread's registers, loaded before anything else; a warp
// per row turns it, quantises it and stores it.

constexpr int kRwThreads = 512, kRwRows = 16;

template <class E, bool kQ8, int D>
__global__ void __launch_bounds__(kRwThreads) k_append_rows(const AppendArgs a) {
    using Tp = typename E::T;
    constexpr int DQ = D / 4;
    __shared__ __align__(16) float xs[kRwRows][128];
    __shared__ __align__(16) float part[4][8][128];
    __shared__ float top[2][kRwRows];
    __shared__ int blk[kRwRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= a.kv_ctas) {  // queries: one unit a thread
        const int64_t i = (int64_t)(blockIdx.x - a.kv_ctas) * kRwThreads + threadIdx.x;
        const int64_t r = i >> 3;
        const int u = (int)(i & 7);
        if (r >= (int64_t)a.B * a.H_q * a.T || u >= D >> 4) return;
        const int b = (int)(r / ((int64_t)a.H_q * a.T)), t = (int)(r % a.T);
        const int64_t j = (int64_t)__ldg(a.positions + b) + t;
        const int n = a.new_lens != nullptr ? __ldg(a.new_lens + b) : a.T;
        if (t >= n || j < 0 || (a.rope != nullptr && j >= a.n_pos)) return;
        const bool turn = a.rope != nullptr && u < a.rot_dim >> 4;
        int ca, cb;
        unit_cols(turn ? a.rot_dim : 0, a.interleaved, u, &ca, &cb);
        const Tp* p = static_cast<const Tp*>(a.q) + r * D;
        Chunk<E> wa, wb;
        wa.load(p + ca);
        wb.load(p + cb);
        float x[16];
        wa.get(x);
        wb.get(x + 8);
        if (turn) turn_unit(a.rope, a.rot_dim, a.interleaved, j, u, x);
        Tp* o = static_cast<Tp*>(a.q_out) + r * D;
        store_chunk<E>(o + ca, x, ca, D);
        store_chunk<E>(o + cb, x + 8, cb, D);
        return;
    }
    const int hk = blockIdx.x % a.H_kv, b0 = blockIdx.x / a.H_kv * a.group;
    const int c = threadIdx.x & 127, qd = threadIdx.x >> 7;
    float p[DQ];
    if (c < D) {
        const float* Ph = a.P + ((int64_t)hk * D + qd * DQ) * D + c;
#pragma unroll
        for (int i = 0; i < DQ; ++i) p[i] = __ldg(Ph + i * D);
    }
    // this warp's row
    const int b = b0 + warp / a.T, t = warp % a.T;
    const bool mine = warp < a.group * a.T && b < a.B;
    const int rows = min(a.group, a.B - b0) * a.T;
    bool live = false;
    int64_t j = 0, first = 0;
    int row = -1;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const bool lane_on = lane * 4 < D;
    if (mine) {
        const ApSeq sq = append_seq(a, b, t == 0 && lane == 0 && hk == 0);
        j = sq.p0 + t;
        first = sq.lo;
        live = j >= sq.lo && j < sq.hi;
        const int64_t at = (((int64_t)b * a.H_kv + hk) * a.T + t) * D;
        if (live) {
            if (lane < D >> 4) {
                const bool turn = a.rope != nullptr && lane < a.rot_dim >> 4;
                int ca, cb;
                unit_cols(turn ? a.rot_dim : 0, a.interleaved, lane, &ca, &cb);
                Chunk<E> wa, wb;
                wa.load(static_cast<const Tp*>(a.K_new) + at + ca);
                wb.load(static_cast<const Tp*>(a.K_new) + at + cb);
                float x[16];
                wa.get(x);
                wb.get(x + 8);
                if (turn) turn_unit(a.rope, a.rot_dim, a.interleaved, j, lane, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xs[warp][ca + e] = x[e];
                    xs[warp][cb + e] = x[8 + e];
                }
            }
            row = pool_row(a, b, hk, (int)j);
            if (lane_on) {
                if constexpr (E::kBytes == 4) {
                    const float4 f = __ldcs(reinterpret_cast<const float4*>(static_cast<const Tp*>(a.V_new) + at) + lane);
                    v[0] = f.x;
                    v[1] = f.y;
                    v[2] = f.z;
                    v[3] = f.w;
                } else {
                    const uint2 f = __ldcs(reinterpret_cast<const uint2*>(static_cast<const Tp*>(a.V_new) + at) + lane);
                    v[0] = bf16_lo(f.x);
                    v[1] = bf16_hi(f.x);
                    v[2] = bf16_lo(f.y);
                    v[3] = bf16_hi(f.y);
                }
            }
        }
    }
    if (!live)
        for (int i = lane; i < 128; i += 32) xs[warp][i] = 0.f;
    float old_k = 0.f, old_v = 0.f;
    bool has_old = false;
    if constexpr (kQ8) {
        has_old = live && first > (j & ~(int64_t)(a.block - 1));
        if (row >= 0 && has_old) {
            old_k = a.k_scales[row >> a.block_log2];
            old_v = a.v_scales[row >> a.block_log2];
        }
        if (lane == 0) blk[warp] = row < 0 ? -1 : row >> a.block_log2;
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += 8) {
        float acc[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) acc[r] = 0.f;
        if (c < D) {
#pragma unroll
            for (int i = 0; i < DQ; i += 4) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 f = *reinterpret_cast<const float4*>(&xs[r0 + r][qd * DQ + i]);
                    acc[r] = fmaf(f.x, p[i], acc[r]);
                    acc[r] = fmaf(f.y, p[i + 1], acc[r]);
                    acc[r] = fmaf(f.z, p[i + 2], acc[r]);
                    acc[r] = fmaf(f.w, p[i + 3], acc[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) part[qd][r][c] = acc[r];
        __syncthreads();
        // the rotated rows take their inputs' place: all 512 threads have read them
        for (int i = threadIdx.x; i < 8 * 128; i += kRwThreads) {
            const float* q = &part[0][0][0] + i;
            xs[r0 + (i >> 7)][i & 127] = (q[0] + q[1024]) + (q[2048] + q[3072]);
        }
        __syncthreads();
    }
    float k[4] = {0.f, 0.f, 0.f, 0.f};
    if (lane_on) *reinterpret_cast<float4*>(k) = *reinterpret_cast<const float4*>(&xs[warp][lane * 4]);
    const bool write = row >= 0 && lane_on;
    if (write && a.plane != nullptr && lane * 4 < a.d_lo) {
        Tp* o = static_cast<Tp*>(a.plane) + (int64_t)row * a.d_lo + lane * 4;
        if constexpr (E::kBytes == 4) {
            *reinterpret_cast<float4*>(o) = make_float4(k[0], k[1], k[2], k[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                *reinterpret_cast<__nv_bfloat162*>(o + e) = __floats2bfloat162_rn(k[e], k[e + 1]);
        }
    }
    if constexpr (!kQ8) {
        if (!write) return;
        Tp* ok = static_cast<Tp*>(a.K_pages) + (int64_t)row * D + lane * 4;
        Tp* ov = static_cast<Tp*>(a.V_pages) + (int64_t)row * D + lane * 4;
        if constexpr (E::kBytes == 4) {
            *reinterpret_cast<float4*>(ok) = make_float4(k[0], k[1], k[2], k[3]);
            *reinterpret_cast<float4*>(ov) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            // values: the upper halves of their fp32 words, bit by bit
            __nv_bfloat162 kk[2] = {__floats2bfloat162_rn(k[0], k[1]), __floats2bfloat162_rn(k[2], k[3])};
            const uint2 vv = make_uint2(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x7632),
                                        __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x7632));
            *reinterpret_cast<uint2*>(ok) = *reinterpret_cast<uint2*>(kk);
            *reinterpret_cast<uint2*>(ov) = vv;
        }
    } else {
        float tk = 0.f, tv = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tk = fmaxf(tk, finite_abs(k[e]));
            tv = fmaxf(tv, finite_abs(v[e]));
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            tk = fmaxf(tk, __shfl_xor_sync(0xffffffffu, tk, off));
            tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, off));
        }
        if (lane == 0) {
            top[0][warp] = tk;
            top[1][warp] = tv;
        }
        __syncthreads();  // and every row has read its block's old scales
        if (row < 0) return;
        // rows of this sequence in the same block
        const int r0 = warp - t, own = blk[warp];
        bool lead = true;
        for (int r = r0; r < r0 + a.T; ++r) {
            if (blk[r] != own) continue;
            tk = fmaxf(tk, top[0][r]);
            tv = fmaxf(tv, top[1][r]);
            if (r < warp) lead = false;
        }
        float sk = pow2_scale(tk), sv = pow2_scale(tv);
        if (has_old) {
            sk = fmaxf(sk, old_k);
            sv = fmaxf(sv, old_v);
        }
        uint8_t* ok = static_cast<uint8_t*>(a.K_pages) + (int64_t)row * D;
        uint8_t* ov = static_cast<uint8_t*>(a.V_pages) + (int64_t)row * D;
        if (lane_on) {
            const float ik = 1.f / sk, iv = 1.f / sv;
            reinterpret_cast<uint32_t*>(ok)[lane] =
                to_e4m3x2(k[0] * ik, k[1] * ik) | to_e4m3x2(k[2] * ik, k[3] * ik) << 16;
            reinterpret_cast<uint32_t*>(ov)[lane] =
                to_e4m3x2(v[0] * iv, v[1] * iv) | to_e4m3x2(v[2] * iv, v[3] * iv) << 16;
        }
        if (!lead) return;
        if (lane == 0) {
            a.k_scales[own] = sk;
            a.v_scales[own] = sv;
        }
        if (has_old) {  // the block's older codes, in the rows before this one
            const int n = (int)(j & (a.block - 1)) * (D / 16);
            uint4* bk = reinterpret_cast<uint4*>(ok) - n;
            uint4* bv = reinterpret_cast<uint4*>(ov) - n;
            for (int kv = 0; kv < 2; ++kv) {
                const float s = kv ? sv : sk, old = kv ? old_v : old_k;
                if (!(s > old)) continue;
                uint4* w = kv ? bv : bk;
                const float f = old / s;
                for (int i = lane; i < n; i += 32) {
                    uint4 x = w[i];
                    x.x = rescale4(x.x, f);
                    x.y = rescale4(x.y, f);
                    x.z = rescale4(x.z, f);
                    x.w = rescale4(x.w, f);
                    w[i] = x;
                }
            }
        }
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
static cudaError_t append_impl(AppendArgs a, cudaStream_t s) {
    if (a.P != nullptr && a.T <= kRwRows) {
        // sequences of a CTA: as many as still leave a CTA for every SM
        DevInfo di;
        cudaError_t e = dev_info(&di);
        if (e != cudaSuccess) return e;
        int64_t group = (int64_t)a.B * a.H_kv / di.sm_count;
        group = group < 1 ? 1 : group;
        group = min64(min64(group, kRwRows / a.T), a.B);
        a.group = (int)group;
        const int64_t kv = (a.B + group - 1) / group * a.H_kv;
        const int64_t q = a.q != nullptr ? ((int64_t)a.B * a.H_q * a.T * 8 + kRwThreads - 1) / kRwThreads : 0;
        if (kv + q > 0x7fffffff) return cudaErrorInvalidValue;
        a.kv_ctas = (int)kv;
        auto kern = a.D == 96 ? k_append_rows<E, kQ8, 96> : k_append_rows<E, kQ8, 128>;
        return launch_kernel(kern, dim3((unsigned)(kv + q)), dim3(kRwThreads), 0, s, false, a);
    }
    bool behind = false;
    if (a.P != nullptr) {
        const cudaError_t e = launch_append_basis(E::kBytes == 4 ? kF32 : kBF16, a, s);
        if (e != cudaSuccess) return e;
        behind = true;
    }
    const int gw = kQ8 ? a.block / 16 : 1, run = 16 * gw;
    const int64_t runs = ((int64_t)a.T + run - 2) / run + 1;
    a.key_tasks = a.P == nullptr ? runs * a.B * a.H_kv : 0;
    a.value_tasks = runs * a.B * a.H_kv;
    a.query_tasks = a.q != nullptr ? runs * a.B * a.H_q : 0;
    const int64_t per = kStThreads / 32 / gw;
    const int64_t ctas = (a.key_tasks + a.value_tasks + a.query_tasks + per - 1) / per;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_kernel(k_append_stream<E, kQ8>, dim3((unsigned)ctas), dim3(kStThreads), 0, s, behind, a);
}

cudaError_t launch_append_paged(Dt dt, AppendArgs a, cudaStream_t s) {
    a.err = device_error_word();
    if (a.err == nullptr) return cudaErrorInvalidDevice;
    a.page_log2 = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz(a.page_size) : -1;
    const bool q8 = a.block > 0;
    if (q8) a.block_log2 = __builtin_ctz(a.block);
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
