// Pieces shared by the paged appends with the rotary embedding
// (append_paged.cu: streams and single rows, append_basis.cu: tiles of rows
// against a head's basis).
//
//   pair (a, b) of columns (i, i + r/2), or (2i, 2i + 1) when interleaved, of
//   the token at position j:  a' = a c - b s,  b' = a s + b c,
//   c, s = table[j][i], table[j][r/2 + i];  K~ = rope(K) P.  All in fp32.
//
// A row is cut into units of 16 columns that one lane turns by itself: unit u
// is the column chunks [8u, 8u + 8) and r/2 + the same (pairs of halves), or
// [16u, 16u + 16) (interleaved pairs, and columns behind rot_dim). Either way
// its angles are entries 8u .. 8u + 7 of the table's row.
#pragma once

#include "launch.h"
#include "q8.cuh"
#include "seqs.cuh"
#include "tma.cuh"

namespace loki {

// The appended tokens of sequence b that get written: positions [lo, hi), or
// lo = hi = 0.
// Tokens outside the block table or behind the rope table are left out, and
// flagged when `flag`.
struct ApSeq {
    int64_t p0;  // positions[b]
    int64_t lo, hi;
};

__device__ __forceinline__ ApSeq append_seq(const AppendArgs& a, int b, bool flag) {
    ApSeq s;
    s.p0 = __ldg(a.positions + b);
    int64_t n = a.new_lens != nullptr ? __ldg(a.new_lens + b) : a.T;
    n = n < 0 ? 0 : (n > a.T ? a.T : n);
    s.lo = s.p0 < 0 ? 0 : s.p0;
    s.hi = s.p0 + n;
    int64_t lim = (int64_t)a.page_size * a.max_pages;
    if (flag && n > 0) {
        if (s.p0 < 0 || s.hi > lim) atomicExch(a.err, kDevErrBadPage);
        else if (a.rope != nullptr && s.hi > a.n_pos) atomicExch(a.err, kDevErrRopeRange);
    }
    if (a.rope != nullptr && a.n_pos < lim) lim = a.n_pos;
    s.hi = s.hi < lim ? s.hi : lim;
    if (s.hi <= s.lo) s.lo = s.hi = 0;  // no token: no run and no scale block is touched
    return s;
}

// A row is worked on in aligned runs of 128 positions.
constexpr int kRunRows = 128;

// runs that positions [lo, hi) touch
__device__ __forceinline__ int run_count(int64_t lo, int64_t hi) {
    return hi > lo ? (int)((hi - 1) / kRunRows - lo / kRunRows) + 1 : 0;
}

// the largest finite magnitude of x[0 .. N) and amax
template <int N>
__device__ __forceinline__ float finite_amax(float amax, const float* x) {
    float m = amax;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, fabsf(x[e]));  // (a NaN does not count)
    if (m <= 3.402823466e38f) return m;
#pragma unroll
    for (int e = 0; e < N; ++e) amax = fmaxf(amax, finite_abs(x[e]));
    return amax;
}

// pool row of (sequence b, KV head hk, position j), or -1 (flagged) when its
// page lies outside the pool; 0 <= j < page_size * max_pages
__device__ __forceinline__ int pool_row(const AppendArgs& a, int b, int hk, int j) {
    const int lp = a.page_log2 >= 0 ? j >> a.page_log2 : (int)((uint32_t)j / (uint32_t)a.page_size);
    const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + lp);
    if (page < 0 || page >= a.n_pages) {
        atomicExch(a.err, kDevErrBadPage);
        return -1;
    }
    return (page * a.H_kv + hk) * a.page_size + (j - lp * a.page_size);
}

// first columns of unit u's two chunks
__device__ __forceinline__ void unit_cols(int rot_dim, int interleaved, int u, int* ca, int* cb) {
    const bool halves = !interleaved && u < rot_dim >> 4;
    *ca = halves ? 8 * u : 16 * u;
    *cb = halves ? 8 * u + (rot_dim >> 1) : 16 * u + 8;
}

// eight consecutive elements, as loaded
template <class E>
struct Chunk {
    static constexpr int kN = E::kBytes / 2;  // 16-byte words
    uint4 w[kN];
    __device__ __forceinline__ void load(const typename E::T* p) {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) E::unpack(w[i], f + i * E::kVec);
    }
};

__device__ __forceinline__ uint4 pack16(const float* f, ElemF32) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float* f, ElemBF16) {
    uint4 r;
    uint32_t* w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return r;
}

// eight fp32 to eight elements, each rounded once; the elements at columns
// >= limit (a multiple of one 16-byte word) are not written
template <class E>
__device__ __forceinline__ void store_chunk(typename E::T* p, const float* f, int col, int limit) {
#pragma unroll
    for (int i = 0; i < Chunk<E>::kN; ++i)
        if (col + i * E::kVec < limit) reinterpret_cast<uint4*>(p)[i] = pack16(f + i * E::kVec, E());
}

// the angles of a unit: cos and sin of entries 8u .. 8u + 7 of a table row
struct Angles {
    float c[8], s[8];
    // from shared or global memory
    __device__ __forceinline__ void load(const float* row, int rot_dim, int u) {
        const float4* cp = reinterpret_cast<const float4*>(row + 8 * u);
        const float4* sp = reinterpret_cast<const float4*>(row + (rot_dim >> 1) + 8 * u);
        *reinterpret_cast<float4*>(c) = cp[0];
        *reinterpret_cast<float4*>(c + 4) = cp[1];
        *reinterpret_cast<float4*>(s) = sp[0];
        *reinterpret_cast<float4*>(s + 4) = sp[1];
    }
    // the unit's columns x[0..7] (chunk a) and x[8..15] (chunk b)
    __device__ __forceinline__ void turn(float* x, int interleaved) const {
        if (interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = x[2 * e], q = x[2 * e + 1];
                x[2 * e] = fmaf(-q, s[e], p * c[e]);
                x[2 * e + 1] = fmaf(p, s[e], q * c[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = x[e], q = x[e + 8];
                x[e] = fmaf(-q, s[e], p * c[e]);
                x[e + 8] = fmaf(p, s[e], q * c[e]);
            }
        }
    }
};

__device__ __forceinline__ void turn_unit_from(const float* row, int rot_dim, int interleaved, int u, float* x) {
    Angles g;
    g.load(row, rot_dim, u);
    g.turn(x, interleaved);
}

// the unit turned by the angles of position j (u < rot_dim / 16)
__device__ __forceinline__ void turn_unit(const float* rope, int rot_dim, int interleaved, int64_t j, int u, float* x) {
    turn_unit_from(rope + j * rot_dim, rot_dim, interleaved, u, x);
}

// column c of the row at position j, turned
template <class E>
__device__ __forceinline__ float turned_col(const AppendArgs& a, const typename E::T* row, int64_t j, int c) {
    const float x = E::load1(row + c);
    if (a.rope == nullptr || c >= a.rot_dim) return x;
    const int half = a.rot_dim >> 1;
    const bool second = a.interleaved ? c & 1 : c >= half;
    const int i = a.interleaved ? c >> 1 : second ? c - half : c;
    const float o = E::load1(row + (a.interleaved ? c ^ 1 : second ? i : c + half));
    const float co = __ldg(a.rope + j * a.rot_dim + i), si = __ldg(a.rope + j * a.rot_dim + half + i);
    return second ? fmaf(o, si, x * co) : fmaf(-o, si, x * co);
}

// eight fp32 / s to eight codes
__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
    return make_uint2(to_e4m3x2(f[0] * inv, f[1] * inv) | to_e4m3x2(f[2] * inv, f[3] * inv) << 16,
                      to_e4m3x2(f[4] * inv, f[5] * inv) | to_e4m3x2(f[6] * inv, f[7] * inv) << 16);
}

// four codes moved to a scale 1/f times as large
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    float v[4];
    e4m3x4_to_float(w, v);
    return to_e4m3x2(v[0] * f, v[1] * f) | to_e4m3x2(v[2] * f, v[3] * f) << 16;
}

}  // namespace loki
