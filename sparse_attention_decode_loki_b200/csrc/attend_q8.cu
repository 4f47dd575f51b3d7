// Attention of one query token per sequence over the paged 8-bit cache
// (q8.cuh), over all of a sequence's tokens (dense) or over each query head's
// selected ones (Loki's last step).
//
//   a_j = scale q . (s_K(j) cK_j),  p = softmax over the row's tokens,
//   out = sum_j p_j s_V(j) cV_j;  a row without tokens gives zeros.
//
// Bytes bound it: 2 D of them per token and KV head against 4 D G flop for G
// query heads. fp32 lanes would not keep up from G = 4 on (23 bytes per clock
// and SM at full bandwidth, G products for each), so both contractions run on
// the tensor cores in m16n8k16 instructions whose operands never leave the
// registers: codes are exact in fp16, and a warp's 16-token tile is loaded in
// the order the fragments want.
//
//   scores  [16 tokens x 8] = K [16 x D] q^T,   columns: 4 heads x 2 parts
//   output  [D x 8]         = V^T [D x 16] p^T, columns: 4 heads x 2 parts
//
// An fp32 query or weight is carried as two fp16 parts, value = hi + lo, in
// neighbouring columns (an accumulator's two columns belong to one lane, which
// adds them), after a power of two has brought the row's largest entry to
// 2^14..2^15: 22 bits down to 2^-17 of it; smaller entries are off by 2^-25,
// fp16's last place, at most, which is 2^-39 of the largest. One such
// instruction has room for four heads; five to eight take two. (8-bit operands
// would halve the instructions, but carry four bits of a query at a time.)
//
// Softmax in base 2, in fp32, against references that move rarely: a head's
// weights are u = 2^(x - m) for the sum and w = u s_V 2^-E for the product; m
// and the even number E are raised (and the sums scaled down) only when a
// score lies 8 above m or a weight would pass 2^15, fp16's range. So a tile
// costs one warp vote instead of a maximum over its lanes, and the product
// stays in the tensor cores' accumulators from tile to tile. E is set so that
// the largest weight so far is 1/2 or more: a weight's rounding, 2^-22 of
// itself or 2^-25, is 2^-24 of the largest weighted value at most, whatever
// the scales of the other blocks. 2^-E is held as its root and multiplied in
// twice: it and its inverse would leave fp32 for scales near fp32's ends.
//
// A warp keeps kStages tiles in a ring of its own in shared memory, two of
// them on their way (128 KB in flight per SM): dense tiles, 16 rows of one
// page, come as two bulk copies; selected tokens as cp.async, every lane
// fetching and reading back its own fragments.
//
// Work is dealt in one of two ways (cluster_size chooses). A cluster of CTAs
// takes a unit - a (sequence, KV head), or a (sequence, query head) row when
// tokens are selected - its warps a run of tiles each, and the partials meet in
// shared memory, the CTAs' through distributed shared memory: one kernel. Where
// whole units would leave much of the device empty, the tiles of all units are
// laid end to end and dealt to warps in runs: four fifths of the line to the
// warps that are resident together, the last fifth in runs a quarter as long to
// as many warps behind them, which the SMs that are done first take up (SMs
// differ by 15 % in what the memory gives them; equal runs left the others idle
// for a fifth of the time). A warp that owns a whole unit writes its output,
// others leave partials (fp32 max, sum, D columns per head) that k_q8_combine
// merges. Either way which warp reduces which tiles is fixed by sizes alone.
//
// Measured, inputs in DRAM: 16 ragged sequences to 4096 tokens, 40 heads, 436 MB
// in 71 to 77 us (6.0 TB/s; 69 without any arithmetic in the two-kernel form);
// 4 x 32768 tokens, 8 KV heads for 32, 218 MB in 43 us; 512 selected tokens for
// each of 640 rows, 79 MB of random 128-byte rows in 25 us (21 without
// arithmetic); one sequence of 513 tokens, 32 heads, 6.8 us.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <map>
#include <mutex>
#include <utility>

#include "launch.h"
#include "q8.cuh"
#include "seqs.cuh"
#include "tma.cuh"

namespace loki {

namespace cg = cooperative_groups;

constexpr int kQ8Threads = 128;
constexpr int kClThreads = 256;  // of the cluster kernels
constexpr int kStages = 3;
constexpr int kClusterTiles = 23680;  // up to so many tiles (ten for every resident warp) clusters may be few
constexpr int kQ8MaxWarps = 2 * 148 * 16;  // workspace is laid out for at most this many
constexpr int kTile = 16;
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr float kMost = 3.402823466e38f, kLeast = -kMost;  // kLeast: below every score

// D[16x8] += A[16x16] B[16x8], fp16 in, fp32 out
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// fp16 pair of (x, y), or of what their fp16 roundings leave over
__device__ __forceinline__ uint32_t f16_part(float x, float y, bool rest) {
    __half2 h = __floats2half2_rn(x, y);
    if (rest) {
        const float2 f = __half22float2(h);
        h = __floats2half2_rn(x - f.x, y - f.y);
    }
    return *reinterpret_cast<uint32_t*>(&h);
}

// 2^x to 2 ulp; results below 2^-126 are zero
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// box {D, 16} of a [rows, D] byte matrix, from its row `row` on
__device__ __forceinline__ void tile_load(void* dst, const CUtensorMap* map, int row, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(0), "r"(row), "r"(smem_addr(bar))
        : "memory");
}

// N bytes (4, 8 or 16) to shared memory, zeros when !on
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
    const int n = on ? N : 0;
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src), "n"(N), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile in shared memory. Lane (gid = lane / 4, tig = lane % 4) reads
//   keys:   tokens key_token(gid) and the one eight behind it, the columns
//           key_col(w, tig) .. + 3 as word w;
//   values: tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9, the D / 8 columns
//           from gid D / 8 on.
// Eight lanes that read together so touch rows four or two apart, which the
// 128-byte swizzle of PageStage spreads over all banks.
template <int D>
struct Frag {
    static constexpr int KW = D / 16;             // key words per token
    static constexpr int VW = D / 32;             // value words per token
    static constexpr int KB = D == 128 ? 16 : 8;  // bytes at a time: D = 96 has 24 and 12 a lane and token
    static constexpr int VB = D == 128 ? 16 : 4;
    static constexpr int KC = KW * 4 / KB, VC = VW * 4 / VB;  // of them per token
    __device__ __forceinline__ static int key_col(int w, int tig) {
        return w * 4 / KB * (4 * KB) + tig * KB + w * 4 % KB;
    }
    __device__ __forceinline__ static int key_token(int gid) { return (gid >> 1) + 4 * (gid & 1); }
    __device__ __forceinline__ static int value_token(int i, int tig) { return 2 * tig + (i & 1) + 8 * (i >> 1); }
    template <int N>
    __device__ __forceinline__ static void get(uint32_t* w, const uint8_t* p) {
        if constexpr (N == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (N == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        else *w = *reinterpret_cast<const uint32_t*>(p);
    }
};

// 16 rows of keys and of values as they lie in the page; D = 128: the 16-byte
// chunk c of row r at c ^ (r % 8), as the tensor map's 128-byte swizzle puts it.
template <int D>
struct PageStage : Frag<D> {
    using F = Frag<D>;
    uint8_t k[kTile][D], v[kTile][D];
    __device__ __forceinline__ static int chunk(int c, int row) { return (D == 128 ? c ^ (row & 7) : c) * 16; }
    __device__ __forceinline__ void get_key(int i, int lane, uint32_t* w) const {
        const int r = F::key_token(lane >> 2) + 8 * i;
#pragma unroll
        for (int c = 0; c < F::KC; ++c) {
            const int at = D == 128 ? chunk(4 * c + (lane & 3), r) : c * 4 * F::KB + (lane & 3) * F::KB;
            F::template get<F::KB>(w + c * F::KB / 4, k[r] + at);
        }
    }
    __device__ __forceinline__ void get_value(int i, int lane, uint32_t* w) const {
        const int r = F::value_token(i, lane & 3);
#pragma unroll
        for (int c = 0; c < F::VC; ++c) {
            const int at = D == 128 ? chunk(lane >> 2, r) : (lane >> 2) * (D / 8) + c * F::VB;
            F::template get<F::VB>(w + c * F::VB / 4, v[r] + at);
        }
    }
};

// Selected tokens: each lane's fragments side by side, a scale per token.
template <int D>
struct PickStage : Frag<D> {
    using F = Frag<D>;
    uint8_t k[2][F::KC][32][F::KB];
    uint8_t v[4][F::VC][32][F::VB];
    float ks[kTile], vs[kTile];
    __device__ __forceinline__ void put_key(int i, const uint8_t* row, bool on, int lane) {
#pragma unroll
        for (int c = 0; c < F::KC; ++c) copy_async<F::KB>(k[i][c][lane], row + c * 4 * F::KB + (lane & 3) * F::KB, on);
    }
    __device__ __forceinline__ void put_value(int i, const uint8_t* row, bool on, int lane) {
#pragma unroll
        for (int c = 0; c < F::VC; ++c) copy_async<F::VB>(v[i][c][lane], row + (lane >> 2) * (D / 8) + c * F::VB, on);
    }
    __device__ __forceinline__ void get_key(int i, int lane, uint32_t* w) const {
#pragma unroll
        for (int c = 0; c < F::KC; ++c) F::template get<F::KB>(w + c * F::KB / 4, k[i][c][lane]);
    }
    __device__ __forceinline__ void get_value(int i, int lane, uint32_t* w) const {
#pragma unroll
        for (int c = 0; c < F::VC; ++c) F::template get<F::VB>(w + c * F::VB / 4, v[i][c][lane]);
    }
};

// NT groups of up to four query heads of one KV head: their query fragments,
// softmax state and output accumulators. Lane (gid, tig) accumulates head
// 4 t + tig, columns gid D / 8 .., hi and lo parts apart, in units of 2^(m + E);
// m and lift = 2^(-E / 2) are the same in the eight lanes of a head, l is the
// lane's own tokens' share.
template <int D, int NT>
struct Heads {
    static constexpr int KW = Frag<D>::KW, VW = Frag<D>::VW;
    uint32_t q[NT][KW][2];
    float qs[NT], m[NT], lift[NT], l[NT], acc[NT][2 * VW][4];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t] = kLeast;
            lift[t] = 1.f;
            l[t] = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * VW; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
        }
    }

    // rows row0 .. row0 + G - 1 of q
    __device__ __forceinline__ void load(const AttendQ8Args& a, int64_t row0, int G, int gid, int tig) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int g = 4 * t + (gid >> 1);
            float x[KW][4], top = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const int64_t at = (row0 + g) * D + Frag<D>::key_col(w, tig);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[w][e] = 0.f;
                if (g < G) {
                    if (a.q_f32) {
                        const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
                        x[w][0] = f.x;
                        x[w][1] = f.y;
                        x[w][2] = f.z;
                        x[w][3] = f.w;
                    } else {
                        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at));
                        x[w][0] = bf16_lo(u.x);
                        x[w][1] = bf16_hi(u.x);
                        x[w][2] = bf16_lo(u.y);
                        x[w][3] = bf16_hi(u.y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, finite_abs(x[w][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - exponent of top), within what fp32 can hold and invert
            int e = 14 + 127 - (int)(__float_as_uint(top) >> 23);
            e = e > 126 ? 126 : e;
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            const bool rest = gid & 1;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                q[t][w][0] = f16_part(x[w][0] * up, x[w][1] * up, rest);
                q[t][w][1] = f16_part(x[w][2] * up, x[w][3] * up, rest);
            }
            const float down = __uint_as_float((uint32_t)(127 - e) << 23) * a.scale_log2;
            qs[t] = __shfl_sync(0xffffffffu, down, 8 * tig);
        }
    }

    // One tile: ok0, ok1 and the scales k0 .. v1 are those of the lane's key
    // tokens; of a partial tile only the first `valid` tokens' values count
    // (behind them may lie NaN codes, which a zero weight would not stop).
    template <class S>
    __device__ __forceinline__ void add(const S& f, bool ok0, bool ok1, float k0, float k1, float v0, float v1,
                                        bool partial, int valid, int lane) {
        const int gid = lane >> 2, tig = lane & 3;
        float c[NT][2][4];  // even and odd words: two chains of products
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[t][0][i] = c[t][1][i] = 0.f;
        {
            uint32_t ka[KW], kb[KW];
            f.get_key(0, lane, ka);
            f.get_key(1, lane, kb);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint32_t a0 = e4m3x2_to_f16x2(ka[w] & 0xffffu), a1 = e4m3x2_to_f16x2(kb[w] & 0xffffu);
                const uint32_t a2 = e4m3x2_to_f16x2(ka[w] >> 16), a3 = e4m3x2_to_f16x2(kb[w] >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(c[t][w & 1], a0, a1, a2, a3, q[t][w][0], q[t][w][1]);
            }
        }
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) f.get_value(i, lane, v[i]);
        if (partial) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (Frag<D>::value_token(i, tig) >= valid) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) v[i][w] = 0u;
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // (the scales first: a large query times codes may leave fp32 where the score does not; their own
            // product only where a code other than zero would)
            const float f0 = fminf(qs[t] * k0, kMost), f1 = fminf(qs[t] * k1, kMost);
            const float x0 = ok0 ? ((c[t][0][0] + c[t][1][0]) + (c[t][0][1] + c[t][1][1])) * f0 : -INFINITY;
            const float x1 = ok1 ? ((c[t][0][2] + c[t][1][2]) + (c[t][0][3] + c[t][1][3])) * f1 : -INFINITY;
            float u0 = exp2_fast(x0 - m[t]), u1 = exp2_fast(x1 - m[t]);
            float w0 = u0 * lift[t] * v0 * lift[t], w1 = u1 * lift[t] * v1 * lift[t];
            const float top = fmaxf(x0, x1);
            if (__any_sync(0xffffffffu, top > m[t] + 8.f || fmaxf(w0, w1) > 32768.f)) {
                float M = fmaxf(m[t], top);
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                u0 = exp2_fast(x0 - M);
                u1 = exp2_fast(x1 - M);
                float y = fmaxf(u0 * v0, u1 * v1);
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
                // this tile's largest weighted value lies in 2^(M + E), 2^(M + E + 2), the others' in
                // units of 2^(m + E before)
                int H = max(((int)(__float_as_uint(y) >> 23) - 127) >> 1, -63);  // E / 2
                const int was = 127 - (int)(__float_as_uint(lift[t]) >> 23);
                const float keep = exp2f(m[t] - M);
                if (keep > 0.f) H = max(H, was + ((int)ceilf(m[t] - M) >> 1));
                const float up = __uint_as_float((uint32_t)(127 - H) << 23);
                const float by = __uint_as_float((uint32_t)(127 + was - H) << 23);
                const float down = keep * by * by;  // (2 at most; by reaches 2^75 where keep is 2^-149)
                l[t] *= keep;
#pragma unroll
                for (int i = 0; i < 2 * VW; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][i][e] *= down;
                m[t] = M;
                lift[t] = up;
                w0 = u0 * up * v0 * up;
                w1 = u1 * up * v1 * up;
            }
            l[t] += u0 + u1;
            // column gid of the weights (head gid / 2, part gid % 2) of this lane's value tokens, from
            // the lanes that hold them as key tokens
            const int src = 16 * (tig & 1) + 4 * (tig >> 1) + (gid >> 1);
            const float p0 = __shfl_sync(0xffffffffu, w0, src), p1 = __shfl_sync(0xffffffffu, w0, src + 8);
            const float p2 = __shfl_sync(0xffffffffu, w1, src), p3 = __shfl_sync(0xffffffffu, w1, src + 8);
            pf[t][0] = f16_part(p0, p1, gid & 1);
            pf[t][1] = f16_part(p2, p3, gid & 1);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // bytes (A, B) of one column side by side, two columns a word
                const uint32_t ab = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
                const uint32_t cd = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
                const uint32_t a0 = e4m3x2_to_f16x2(ab & 0xffffu), a1 = e4m3x2_to_f16x2(ab >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(cd & 0xffffu), a3 = e4m3x2_to_f16x2(cd >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(acc[t][2 * w + half], a0, a1, a2, a3, pf[t][0], pf[t][1]);
            }
        }
    }

    // 2^E
    __device__ __forceinline__ float unit(int t) const { return 1.f / (lift[t] * lift[t]); }

    // column i of the lane's, in units of 2^(m + E)
    __device__ __forceinline__ float col(int t, int i) const {
        return acc[t][i >> 1][2 * (i & 1)] + acc[t][i >> 1][2 * (i & 1) + 1];
    }

    // The state of rows row0 .. row0 + G - 1 as output.
    template <class E>
    __device__ __forceinline__ void write(const AttendQ8Args& a, int64_t row0, int G, int gid, int tig) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int g = 4 * t + tig;
            const float L = sum(t);
            if (g >= G) continue;
            typename E::T* o = static_cast<typename E::T*>(a.out) + (row0 + g) * D + gid * (D / 8);
            const float r = L == 0.f ? 0.f : 1.f / L, up = unit(t);
#pragma unroll
            for (int i = 0; i < 4 * VW; ++i) o[i] = E::from_float(col(t, i) * r * up);
        }
    }
    // The state as a partial: (max, sum) at ml[g], columns at pa[g D ..].
    __device__ __forceinline__ void leave(float2* ml, float* pa, int G, int gid, int tig) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int g = 4 * t + tig;
            const float L = sum(t);
            if (g >= G) continue;
            if (gid == 0) ml[g] = make_float2(m[t], L);
            const float r = unit(t);  // to units of 2^m
            float4* o = reinterpret_cast<float4*>(pa + g * D + gid * (D / 8));
#pragma unroll
            for (int i = 0; i < VW; ++i)
                o[i] = make_float4(col(t, 4 * i) * r, col(t, 4 * i + 1) * r, col(t, 4 * i + 2) * r, col(t, 4 * i + 3) * r);
        }
    }
    __device__ __forceinline__ float sum(int t) const {
        float L = l[t];
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        return L;
    }
};

__device__ __forceinline__ int64_t q8_len(const AttendQ8Args& a, int b) {
    const int64_t cap = (int64_t)a.page_size * a.max_pages, n = __ldg(a.seq_lens + b);
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// tiles of sequence b (per KV head)
struct SeqTiles {
    const AttendQ8Args& a;
    __device__ __forceinline__ int64_t operator()(int b) const { return (q8_len(a, b) + kTile - 1) / kTile; }
};

// The line of `total` tiles in runs: a.warps / 2 of `per`, then a.warps / 2 of `tail`.
struct Runs {
    int64_t per, tail, split, total;  // split: where the short runs begin
    int first;                        // warps with long runs
    __device__ __forceinline__ Runs(const AttendQ8Args& a, int64_t n) : total(n), first(a.warps >> 1) {
        per = quot(n * 4, 5 * (int64_t)first);
        per = per < 1 ? 1 : per;
        split = min64(per * first, n);
        tail = quot(n - split + first - 1, first);
        tail = tail < 1 ? 1 : tail;
    }
    __device__ __forceinline__ int64_t begin(int64_t w) const {
        return min64(w < first ? w * per : split + (w - first) * tail, total);
    }
    __device__ __forceinline__ int64_t end(int64_t w) const {
        return w < first ? min64(w * per + per, split) : min64(split + (w - first + 1) * tail, total);
    }
    __device__ __forceinline__ int64_t owner(int64_t tile) const {
        return tile < split ? quot(tile, per) : first + quot(tile - split, tail);
    }
};

// partial `slot` of G heads in the workspace
__device__ __forceinline__ float2* slot_ml(const AttendQ8Args& a, int64_t slot, int G) {
    return static_cast<float2*>(a.ws) + slot * G;
}
__device__ __forceinline__ float* slot_cols(const AttendQ8Args& a, int64_t slot, int G) {
    return reinterpret_cast<float*>(static_cast<float2*>(a.ws) + a.slots * G) + slot * G * a.D;
}

// The cluster's partials of rows row0 .. row0 + G - 1 into the output: each
// CTA merges its warps' in shared memory (which the tiles' rings leave free),
// then takes a share of the outputs over the CTAs' merged ones.
template <class E, int D, int NT>
__device__ __forceinline__ void merge_cluster(const AttendQ8Args& a, Heads<D, NT>& h, uint8_t* smem, int64_t row0, int G) {
    constexpr int W = kClThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* ml = reinterpret_cast<float2*>(smem);       // [W][G], then the CTA's [G]
    float* pa = reinterpret_cast<float*>(ml + 8 * (W + 1) );  // [W][G][D], then the CTA's [G][D]
    __syncthreads();
    h.leave(ml + warp * G, pa + warp * G * D, G, lane >> 2, lane & 3);
    __syncthreads();
    float2* cml = ml + W * G;
    float* cpa = pa + W * G * D;
    for (int i = threadIdx.x; i < G * D; i += kClThreads) {
        const int g = i / D;
        float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * G + g].x);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 x = ml[w * G + g];
            const float s = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
            L = fmaf(x.y, s, L);
            A = fmaf(pa[w * G * D + i], s, A);
        }
        if (a.cluster == 1) {
            static_cast<typename E::T*>(a.out)[row0 * D + i] = E::from_float(L == 0.f ? 0.f : A / L);
        } else {
            cpa[i] = A;
            if (i % D == 0) cml[g] = make_float2(M, L);
        }
    }
    if (a.cluster == 1) return;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int i = cl.block_rank() * kClThreads + threadIdx.x; i < G * D; i += a.cluster * kClThreads) {
        const int g = i / D;
        float M = -INFINITY, L = 0.f, A = 0.f;
        for (int r = 0; r < a.cluster; ++r) M = fmaxf(M, cl.map_shared_rank(cml, r)[g].x);
        for (int r = 0; r < a.cluster; ++r) {
            const float2 x = cl.map_shared_rank(cml, r)[g];
            const float s = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
            L = fmaf(x.y, s, L);
            A = fmaf(cl.map_shared_rank(cpa, r)[i], s, A);
        }
        static_cast<typename E::T*>(a.out)[row0 * D + i] = E::from_float(L == 0.f ? 0.f : A / L);
    }
    cl.sync();  // the others may still read this CTA's
}

// kCl: a cluster per (sequence, KV head), a run of its tiles per warp.
template <class E, int D, int NT, bool kCl>
__global__ void __launch_bounds__(kCl ? kClThreads : kQ8Threads, NT == 1 ? (kCl ? 2 : 4) : (kCl ? 1 : 3))
    k_dense_q8(const AttendQ8Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;  // the swizzle goes by address
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    PageStage<D>* ring = reinterpret_cast<PageStage<D>*>(smem) + warp * kStages;
    __shared__ __align__(8) uint64_t bars[(kCl ? kClThreads : kQ8Threads) / 32][kStages];
    uint64_t* bar = bars[warp];
    if (lane < kStages) mbar_init(bar + lane, 1);
    fence_mbar_init();
    __syncwarp();
    griddep_wait();  // launched early: inputs and workspace may still be in use
    fence_proxy_async_global();             // the tiles come by bulk copies
    if (!kCl) griddep_launch_dependents();  // the merge, which reads the lengths before it waits
    const int64_t wi = (int64_t)blockIdx.x * (kQ8Threads / 32) + warp;
    const int G = a.H_q / a.H_kv;
    int b, hk, len, n, t;  // n: tiles of the unit, t: the next one
    int64_t w, w_end;
    if constexpr (kCl) {
        const int unit = blockIdx.x / a.cluster, cw = blockIdx.x % a.cluster * (kClThreads / 32) + warp;
        b = unit / a.H_kv;
        hk = unit % a.H_kv;
        len = (int)q8_len(a, b);
        n = (len + kTile - 1) / kTile;
        const int cws = a.cluster * (kClThreads / 32), per = (n + cws - 1) / cws;
        w = t = cw * per;
        w_end = min(t + per, n);
    } else {
        int64_t before;
        const SeqTiles tiles{a};
        const Runs runs(a, seqs_total(a.B, tiles) * a.H_kv);  // (seqs_find's lengths come from the L1)
        w = runs.begin(wi);
        w_end = runs.end(wi);
        if (w >= w_end) return;
        b = seqs_find(a.B, w, a.H_kv, tiles, &before);
        if (b < 0) return;
        len = (int)q8_len(a, b);
        n = (len + kTile - 1) / kTile;
        hk = (int)quot(w - before * a.H_kv, n);
        t = (int)(w - before * a.H_kv - (int64_t)hk * n);
    }

    // the copies run kStages - 1 tiles ahead of the arithmetic: lb, lhk, lt, ... are theirs
    int lb = b, lhk = hk, lt = t, llen = len, ln = n;
    int lp = -1, lpage = -1, lnext = -1, loff = 0;  // page index, page and the one behind, first token in it
    const int tk = Frag<D>::key_token(gid);
    auto page = [&](int i) { return __ldg(a.block_table + (int64_t)lb * a.max_pages + min(i, a.max_pages - 1)); };
    // issues the next tile's copies; how many of its tokens count, its scales' index
    struct Tile {
        int valid, blk;
    };
    auto load = [&](int at) -> Tile {
        const int j = lt * kTile;
        if (lp < 0) {
            lp = j / a.page_size;
            loff = j - lp * a.page_size;
            lpage = page(lp);
            lnext = page(lp + 1);
        } else if (loff == a.page_size) {
            ++lp;
            loff = 0;
            lpage = lnext;
            lnext = page(lp + 1);
        }
        Tile x{0, 0};
        if (lpage >= 0 && lpage < a.n_pages) {
            x.valid = min(llen - j, kTile);
            const int row = (lpage * a.H_kv + lhk) * a.page_size + loff;
            x.blk = row >> a.block_log2;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar + at, 2 * kTile * D);
                if constexpr (D == 128) {
                    tile_load(ring[at].k, &kmap, row, bar + at);
                    tile_load(ring[at].v, &vmap, row, bar + at);
                } else {
                    bulk_load(ring[at].k, a.K_pages + (int64_t)row * D, kTile * D, bar + at);
                    bulk_load(ring[at].v, a.V_pages + (int64_t)row * D, kTile * D, bar + at);
                }
            }
        } else if (lane == 0) {
            mbar_arrive(bar + at);  // nothing to wait for
            atomicExch(a.err, kDevErrBadPage);
        }
        loff += kTile;
        if (++lt == ln) {  // the next unit with tokens
            lt = 0;
            lp = -1;
            if (!kCl && ++lhk == a.H_kv) {
                lhk = 0;
                do {
                    if (++lb >= a.B) break;
                    llen = (int)q8_len(a, lb);
                } while (llen == 0);
                ln = (llen + kTile - 1) / kTile;
            }
        }
        return x;
    };

    Tile tile[kStages] = {};  // the one at hand and the ones behind it
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        if (w + i < w_end) tile[i] = load(i);
    float ks = __ldg(a.k_scales + tile[0].blk), vs = __ldg(a.v_scales + tile[0].blk);
    Heads<D, NT> h;
    h.reset();
    h.load(a, (int64_t)b * a.H_q + (int64_t)hk * G, G, gid, tig);
    bool whole = t == 0;
    uint32_t phase = 0;
    bool alive = true;
    for (int at = 0; w < w_end; phase ^= at + 1 == kStages, at = at + 1 == kStages ? 0 : at + 1) {
        fence_proxy_async_shared();
        __syncwarp();  // every lane is done with the stage before this one
        if (w + kStages - 1 < w_end) tile[kStages - 1] = load(at == 0 ? kStages - 1 : at - 1);
        const float ks1 = __ldg(a.k_scales + tile[1].blk), vs1 = __ldg(a.v_scales + tile[1].blk);
        alive = mbar_wait(bar + at, phase, a.err);
        if (!__all_sync(0xffffffffu, alive)) {  // flagged: the copies on their way land (or not) before the ring is left
#pragma unroll 1
            for (int i = 0; i < kStages && w + i < w_end; ++i) {
                const int s = at + i;
                mbar_wait(bar + (s < kStages ? s : s - kStages), phase ^ (s >= kStages), a.err);
            }
            break;
        }
        const int valid = tile[0].valid;
        if (valid > 0)
            h.add(ring[at], tk < valid, tk + 8 < valid, ks, ks, vs, vs, valid < kTile, valid, lane);
        ks = ks1;
        vs = vs1;
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) tile[i] = tile[i + 1];
        ++t;
        ++w;
        if (!kCl && (t == n || w == w_end)) {
            const int64_t unit = (int64_t)b * a.H_kv + hk;
            if (whole && t == n) h.template write<E>(a, unit * G, G, gid, tig);
            else h.leave(slot_ml(a, unit + wi, G), slot_cols(a, unit + wi, G), G, gid, tig);
            if (w == w_end) return;
            t = 0;
            whole = true;
            if (++hk == a.H_kv) {
                hk = 0;
                do {
                    if (++b >= a.B) return;
                    len = (int)q8_len(a, b);
                } while (len == 0);
                n = (len + kTile - 1) / kTile;
            }
            h.reset();
            h.load(a, (int64_t)b * a.H_q + (int64_t)hk * G, G, gid, tig);
        }
    }
    if constexpr (kCl) merge_cluster<E>(a, h, smem, ((int64_t)b * a.H_kv + hk) * G, G);
}

// Selected tokens: a tile is 16 consecutive entries of a row's list; lane l
// looks up entry l % 16 and hands its row number to the lanes that copy it.
// (Rows gathered by tensor map, four to an instruction: the loads alone take no
// less, 22 us, and the whole 28 instead of 25, one sequence 8.2 instead of 7.8:
// the copies start one lookup and one barrier later.)
// kCl: a cluster per (sequence, query head), a run of its tiles per warp.
template <class E, int D, bool kCl>
__global__ void __launch_bounds__(kCl ? kClThreads : kQ8Threads, kCl ? 2 : 4) k_sparse_q8(const AttendQ8Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();  // launched early: inputs and workspace may still be in use
    if (!kCl) griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    PickStage<D>* ring = reinterpret_cast<PickStage<D>*>(smem) + warp * kStages;
    const int64_t wi = (int64_t)blockIdx.x * (kQ8Threads / 32) + warp;
    const int G = a.H_q / a.H_kv;
    const int64_t n = (a.k + kTile - 1) / kTile;
    int64_t w, w_end, r, t;
    if constexpr (kCl) {
        r = blockIdx.x / a.cluster;
        const int cws = a.cluster * (kClThreads / 32);
        const int64_t per = (n + cws - 1) / cws;
        w = t = (blockIdx.x % a.cluster * (kClThreads / 32) + warp) * per;
        w_end = min64(t + per, n);
    } else {
        const Runs runs(a, n * a.B * a.H_q);
        w = runs.begin(wi);
        w_end = runs.end(wi);
        if (w >= w_end) return;
        r = quot(w, n);
        t = w - r * n;
    }
    const int tk = Frag<D>::key_token(gid);

    // entries run kStages tiles ahead of the arithmetic, copies one less
    const int32_t* ip = a.idx + r * a.k + t * kTile + (lane & 15);
    int64_t il = a.k - t * kTile, iw = w_end - w;  // entries left of the row, tiles left of the run
    auto entry = [&]() -> int {
        if (iw-- <= 0) return -1;
        const int j = (lane & 15) < il ? __ldg(ip) : -1;
        if (il <= kTile) {  // on to the next row
            ip += il;
            il = a.k;
        } else {
            ip += kTile;
            il -= kTile;
        }
        return j;
    };
    int64_t lt = n - t;  // tiles left of the copies' row
    int lb = (int)r / a.H_q, lh = (int)r % a.H_q, lhk = lh / G, llen = (int)q8_len(a, lb);
    // issues the copies of the tile with entries j; a bit for each that counts
    auto load = [&](PickStage<D>& x, int j) -> uint32_t {
        uint32_t row = kNoRow;
        if (j >= 0 && j < llen) {
            const uint32_t lp = a.page_log2 >= 0 ? (uint32_t)j >> a.page_log2 : (uint32_t)j / (uint32_t)a.page_size;
            const int page = __ldg(a.block_table + (int64_t)lb * a.max_pages + lp);
            if (page >= 0 && page < a.n_pages)
                row = ((uint32_t)page * a.H_kv + lhk) * a.page_size + ((uint32_t)j - lp * a.page_size);
            else
                atomicExch(a.err, kDevErrBadPage);
        }
        const uint32_t ok = __ballot_sync(0xffffffffu, row != kNoRow) & 0xffffu;
        if (ok != 0) {
            const bool on = row != kNoRow;
            const uint32_t blk = on ? row >> a.block_log2 : 0u;
            if (lane < kTile) copy_async<4>(x.ks + lane, a.k_scales + blk, on);
            else copy_async<4>(x.vs + (lane - kTile), a.v_scales + blk, on);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row, tk + 8 * i);
                x.put_key(i, a.K_pages + (rr != kNoRow ? (int64_t)rr * D : 0), rr != kNoRow, lane);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row, Frag<D>::value_token(i, tig));
                x.put_value(i, a.V_pages + (rr != kNoRow ? (int64_t)rr * D : 0), rr != kNoRow, lane);
            }
        }
        if (--lt == 0) {
            lt = n;
            if (++lh == a.H_q) {
                lh = 0;
                if (++lb < a.B) llen = (int)q8_len(a, lb);
            }
            lhk = lh / G;
        }
        return ok;
    };

    uint32_t ok[kStages] = {};  // of the tile at hand and the ones behind it
    int j = entry();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        const int j0 = j;
        j = entry();
        if (w + i < w_end) ok[i] = load(ring[i], j0);
        copy_commit();
    }
    Heads<D, 1> h;
    h.reset();
    h.load(a, r, 1, gid, tig);
    bool whole = t == 0;
    for (int at = 0; w < w_end; at = at + 1 == kStages ? 0 : at + 1) {
        const int j0 = j;
        j = entry();
        copy_wait<kStages - 2>();
        __syncwarp();  // every lane's copies have landed, and every lane is done with the stage before
        if (w + kStages - 1 < w_end) ok[kStages - 1] = load(ring[at == 0 ? kStages - 1 : at - 1], j0);
        copy_commit();
        if (ok[0] != 0) {
            const PickStage<D>& x = ring[at];
            h.add(x, (ok[0] >> tk) & 1u, (ok[0] >> (tk + 8)) & 1u, x.ks[tk], x.ks[tk + 8], x.vs[tk], x.vs[tk + 8],
                  false, kTile, lane);
        }
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) ok[i] = ok[i + 1];
        ++t;
        ++w;
        if (!kCl && (t == n || w == w_end)) {
            if (whole && t == n) h.template write<E>(a, r, 1, gid, tig);
            else h.leave(slot_ml(a, r + wi, 1), slot_cols(a, r + wi, 1), 1, gid, tig);
            if (w == w_end) return;
            t = 0;
            whole = true;
            ++r;
            h.reset();
            h.load(a, r, 1, gid, tig);
        }
    }
    if constexpr (kCl) merge_cluster<E>(a, h, smem, r, 1);
}

// Merges the partials of one (sequence, query head) row: the W warps take
// partials in turn, four columns a lane. Rows that one warp owned whole are
// written already; rows without tokens get zeros. The lengths are read before
// the wait: they are older than the partials' kernel, every CTA of which has
// waited for all that came before it when it releases this grid. (With the wait
// first a call takes 1.3 to 2.3 us longer.)
template <class E, int D, int W>
__global__ void __launch_bounds__(32 * W) k_q8_combine(const AttendQ8Args a) {
    __shared__ float sm_m[W], sm_l[W];
    __shared__ float4 sm_acc[W][32];
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t unit = r, first, n, total;
    int Gc = 1, g = 0;
    if (a.idx != nullptr) {
        n = (a.k + kTile - 1) / kTile;
        total = n * a.B * a.H_q;
        first = r * n;
    } else {
        Gc = a.H_q / a.H_kv;
        const int b = (int)(r / a.H_q), h = (int)(r % a.H_q);
        int64_t before;
        total = seqs_total(a.B, SeqTiles{a}, b, &before) * a.H_kv;
        n = (q8_len(a, b) + kTile - 1) / kTile;
        g = h % Gc;
        unit = (int64_t)b * a.H_kv + h / Gc;
        first = before * a.H_kv + (h / Gc) * n;
    }
    const Runs runs(a, total);
    const int64_t c0 = runs.owner(first);
    const int np = n == 0 ? 0 : (int)(runs.owner(first + n - 1) - c0 + 1);
    griddep_wait();  // every block: the grid must not end before the partials' writers
    if (np == 1) return;
    const float2* ml = slot_ml(a, unit + c0, Gc) + g;
    const float* pa = slot_cols(a, unit + c0, Gc) + g * D + lane * 4;
    float M = kLeast, L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = lane * 4 < D;
    for (int p0 = warp; p0 < np; p0 += 4 * W) {
        float2 x[4];
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + i * W;
            x[i] = p < np ? ml[(int64_t)p * Gc] : make_float2(kLeast, 0.f);
            y[i] = p < np && on ? *reinterpret_cast<const float4*>(pa + (int64_t)p * Gc * D) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float m = fmaxf(fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), M), keep = exp2f(M - m);
        L *= keep;
        A = make_float4(A.x * keep, A.y * keep, A.z * keep, A.w * keep);
        M = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = exp2f(x[i].x - m);
            L = fmaf(x[i].y, s, L);
            A.x = fmaf(y[i].x, s, A.x);
            A.y = fmaf(y[i].y, s, A.y);
            A.z = fmaf(y[i].z, s, A.z);
            A.w = fmaf(y[i].w, s, A.w);
        }
    }
    sm_acc[warp][lane] = A;
    if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = L;
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= D) return;
    M = sm_m[0];
#pragma unroll
    for (int i = 1; i < W; ++i) M = fmaxf(M, sm_m[i]);
    L = 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float f = exp2f(sm_m[i] - M);
        L = fmaf(sm_l[i], f, L);
        s = fmaf(reinterpret_cast<const float*>(sm_acc[i])[c], f, s);
    }
    static_cast<typename E::T*>(a.out)[r * D + c] = E::from_float(L == 0.f ? 0.f : s / L);
}

// ---------------------------------------------------------------------------

// partials: a (unit, warp) pair for every border between the warps' runs and
// every unit, numbered unit + warp, which grows along the line of tiles
// (an even number: the columns behind the (m, l) pairs start on 16 bytes)
static int64_t q8_slots(int64_t units, int64_t tiles) {
    return (units + min64(kQ8MaxWarps, 2 * tiles) + 1) & ~(int64_t)1;
}

// (none where clusters are sure: the calls still want a workspace, of any size)
static size_t q8_ws_bytes(int64_t units, int64_t tiles, int G, int D) {
    if (tiles <= kClusterTiles) return 1;
    return (size_t)q8_slots(units, tiles) * G * (sizeof(float2) + D * sizeof(float));
}

size_t dense_q8_ws_bytes(int B, int H_q, int H_kv, int64_t S_cap, int D) {
    const int64_t units = (int64_t)B * H_kv;
    return q8_ws_bytes(units, units * ((S_cap + kTile - 1) / kTile), H_q / H_kv, D);
}

size_t sparse_q8_ws_bytes(int B, int H_q, int64_t k, int D) {
    const int64_t rows = (int64_t)B * H_q;
    return q8_ws_bytes(rows, rows * ((k + kTile - 1) / kTile), 1, D);
}

// the kernel's dynamic shared memory and the largest shared split, set once
static cudaError_t allow_smem(const void* f, size_t bytes) {
    const cudaError_t e = prefer_carveout(f, cudaSharedmemCarveoutMaxShared);
    return e != cudaSuccess ? e : allow_dynamic_smem(f, bytes);
}

// cluster 0: none; attr: two. The kernels are launched as programmatic
// dependents of whatever precedes them and wait for it first: that hides their
// launch (a short sequence, call after call: 9.0 -> 6.9 us).
static cudaLaunchConfig_t launch_config(int64_t ctas, int threads, int cluster, size_t smem, cudaStream_t s,
                                        cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cfg;
}

// clusters of 1 .. 8 CTAs of a cluster kernel that the device holds at a time
// (whole clusters have to fit a group of SMs, so sizes like 7 lose places)
struct ClusterSlots {
    int active[9];
};

static cudaError_t cluster_slots(const void* kern, size_t smem, ClusterSlots* out) {
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, ClusterSlots> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    const auto at = known.find({dev, kern});
    if (at != known.end()) {
        *out = at->second;
        return cudaSuccess;
    }
    for (int c = 1; c <= 8; ++c) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = launch_config(c, kClThreads, c, smem, nullptr, attr);
        e = cudaOccupancyMaxActiveClusters(&out->active[c], kern, &cfg);
        if (e != cudaSuccess) return e;
    }
    known[{dev, kern}] = *out;
    return cudaSuccess;
}

// CTAs of a unit's cluster, 0: the two-kernel form. The size that fills most
// of the device while every warp has a tile. One kernel saves the
// second launch and the partials' way through memory, 5 to 10 us; the equal
// runs of the two-kernel form save the places that whole units leave empty.
// Measured, us, cluster / two kernels (H_kv x sequences x tokens):
//   40 x 16 x 4096 ragged 69 / 79, 8 x 4 x 32768 42 / 49, 32 x 4 x 2048 13 / 19;
//   8 x 2 x 65536 (43 % of the places filled) 67 / 55, 40 x 8 x 4096 (54 %)
//   75 / 63, 8 x 1 x 131072 (22 %) 114 / 75; 8 x 1 x 32768 (22 %, but few
//   tiles) 32 / 38. Around the border, even lengths: 9 x 20 x 8192 (61 %) 77 / 69,
//   40 x 5 x 8192 (68 %) 78 / 75, 40 x 15 x 4096 (68 %) 118 / 107, 8 x 13 x 16384
//   (70 %) 80 / 78, 40 x 16 x 4096 (72 %) 119 / 112, 40 x 3 x 16384 (81 %) 82 / 88,
//   8 x 11 x 16384 (89 %, clusters of three) 61 / 67. Ragged lengths shift it
//   down: whole units end apart, and others follow them.
// The tokens are the block table's capacity, the lengths being on the device: a
// wide table over short sequences takes the two kernels where clusters would do
// (8 x 24 x 1000 behind a table of 8192 32 us, of 1024 17; one sequence of 513
// 7.0 to 7.5 us either way).
// Sizes: meeting the other CTAs costs about a tile's time, so two tiles a warp
// stay in one CTA (32 units of 16 tiles 5.7 us, in clusters of 2 to 8 6.1) and
// 64 tiles in four (7.2; in eight 7.6); sizes other than powers of two lose 15 %
// at the same number of tiles a warp (33 tiles: 4 CTAs 7.1, 5 CTAs 7.4; 128: 4
// CTAs 8.9, 5 CTAs 10.8) but fill more (80 units of 1024 tiles: 2 CTAs 65, 3 51).
static int cluster_size(int64_t units, int64_t tiles, const ClusterSlots& slots) {
    constexpr int W = kClThreads / 32;
    const int64_t resident = slots.active[1];
    int best = 1;
    double fill = 0, most = 0;
    for (int c = 1; c <= 8; ++c) {
        const bool useful = c == 1 || (tiles > 2 * W && (c - 1) * W < tiles && (c <= 4 || tiles > 8 * W));
        if (!useful || slots.active[c] < 1 || (c > 1 && units > slots.active[c])) continue;
        const int64_t waves = (units + slots.active[c] - 1) / slots.active[c];
        const double f = (double)(units * c) / (double)(waves * resident);
        const double worth = (c & (c - 1)) == 0 ? f : 0.8 * f;
        if (worth >= most) {
            most = worth;
            fill = f;
            best = c;
        }
    }
    return fill >= 0.7 || units * tiles <= kClusterTiles ? best : 0;
}

// the pages as a [rows, 128] byte matrix, in boxes of one tile
static cudaError_t page_map(CUtensorMap* m, const void* p, int64_t rows) {
    static const PFN_cuTensorMapEncodeTiled encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (PFN_cuTensorMapEncodeTiled)f;
    }();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
    const cuuint32_t box[2] = {128, kTile}, step[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <class E, int D>
static cudaError_t attend_impl(AttendQ8Args& a, cudaStream_t s) {
    const int G = a.H_q / a.H_kv;
    const bool sparse = a.idx != nullptr;
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    const int64_t units = sparse ? (int64_t)a.B * a.H_q : (int64_t)a.B * a.H_kv;
    const int64_t items = sparse ? a.k : (int64_t)a.page_size * a.max_pages;
    const int64_t tiles = (items + kTile - 1) / kTile;
    CUtensorMap kmap = {}, vmap = {};
    if (!sparse && D == 128) {
        const int64_t rows = a.n_pages * a.H_kv * a.page_size;
        e = page_map(&kmap, a.K_pages, rows);
        if (e == cudaSuccess) e = page_map(&vmap, a.V_pages, rows);
        if (e != cudaSuccess) return e;
    }
    auto smem_of = [=](int threads) {
        return threads / 32 * kStages * (sparse ? sizeof(PickStage<D>) : sizeof(PageStage<D>)) + (sparse ? 0 : 1024);
    };
    const size_t csmem = smem_of(kClThreads), smem = smem_of(kQ8Threads);
    const void* ck = sparse   ? (const void*)k_sparse_q8<E, D, true>
                     : G <= 4 ? (const void*)k_dense_q8<E, D, 1, true>
                              : (const void*)k_dense_q8<E, D, 2, true>;
    e = allow_smem(ck, csmem);
    if (e != cudaSuccess) return e;
    ClusterSlots slots;
    e = cluster_slots(ck, csmem, &slots);
    if (e != cudaSuccess) return e;
    a.cluster = cluster_size(units, tiles, slots);
    if (a.cluster > 0 && units * a.cluster <= 0x7fffffff) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = launch_config(units * a.cluster, kClThreads, a.cluster, csmem, s, attr);
        void* args[] = {&a, &kmap, &vmap};
        return cudaLaunchKernelExC(&cfg, ck, args);
    }
    const void* kern = sparse   ? (const void*)k_sparse_q8<E, D, false>
                       : G <= 4 ? (const void*)k_dense_q8<E, D, 1, false>
                                : (const void*)k_dense_q8<E, D, 2, false>;
    e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    const int wpc = kQ8Threads / 32;
    int64_t warps = (int64_t)di.sm_count * occupancy(kern, kQ8Threads, smem) * wpc;
    warps = 2 * min64(min64(warps, kQ8MaxWarps / 2), units * tiles);
    a.warps = (int)warps;
    a.slots = q8_slots(units, units * tiles);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = launch_config((warps + wpc - 1) / wpc, kQ8Threads, 0, smem, s, attr);
    void* args[] = {&a, &kmap, &vmap};
    e = cudaLaunchKernelExC(&cfg, kern, args);
    if (e != cudaSuccess) return e;
    // partials of a unit: a warp to each, within limits
    const bool many = warps > 16 * units;
    return launch_kernel(many ? k_q8_combine<E, D, 16> : k_q8_combine<E, D, 4>,
                         dim3((unsigned)((int64_t)a.B * a.H_q)), dim3(many ? 512 : 128), 0, s, true, a);
}

cudaError_t launch_attend_q8(Dt out_dt, AttendQ8Args a, cudaStream_t s) {
    a.err = device_error_word();
    if (a.err == nullptr) return cudaErrorInvalidDevice;
    a.page_log2 = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz(a.page_size) : -1;
    a.block_log2 = __builtin_ctz(a.block);
    if (a.D == 96) return out_dt == kF32 ? attend_impl<ElemF32, 96>(a, s) : attend_impl<ElemBF16, 96>(a, s);
    return out_dt == kF32 ? attend_impl<ElemF32, 128>(a, s) : attend_impl<ElemBF16, 128>(a, s);
}

}  // namespace loki
