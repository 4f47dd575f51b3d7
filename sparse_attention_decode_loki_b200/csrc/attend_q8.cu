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
// adds them): 22 bits, after a power of two has brought the row's largest entry
// to 2^14..2^15, so entries down to 2^-29 of it keep all 22. One such
// instruction has room for four heads; five to eight take two. (8-bit operands
// would halve the instructions, but carry four bits of a query at a time.)
//
// Softmax in base 2, in fp32, with its maximum taken per tile: the tile's
// weights are relative to its own maximum, and its product joins the running
// sums with one fp32 factor that also carries the values' scale. So scales far
// apart between blocks cost no precision.
//
// The tiles of all (sequence, KV head) units - of all (sequence, query head)
// rows, when tokens are selected - are laid end to end and dealt to the
// resident warps in equal runs. A warp that owns a whole unit writes its
// output, others leave partials (fp32 max, sum, D columns per head) that
// k_q8_combine merges in a fixed order.
#include <cuda_fp16.h>

#include "launch.h"
#include "q8.cuh"
#include "tma.cuh"

namespace loki {

constexpr int kQ8Threads = 128;
constexpr int kQ8MaxWarps = 148 * 16;  // workspace is laid out for at most this many
constexpr int kTile = 16;
constexpr uint32_t kNoRow = 0xffffffffu;

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

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_stream4(const void* p) {
    uint32_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}

// Lane (gid = lane / 4, tig = lane % 4) holds of a tile
//   keys:   tokens tk = 4 (gid / 2) + gid % 2 and tk + 2, the columns
//           key_col(w, tig) .. + 3 as word w;
//   values: tokens 4 tig .. 4 tig + 3, the D / 8 columns from gid D / 8 on.
template <int D>
struct Frag {
    static constexpr int KW = D / 16;  // key words per token
    static constexpr int VW = D / 32;  // value words per token
    uint32_t k[2][KW];
    uint32_t v[4][VW];

    __device__ __forceinline__ static int key_col(int w, int tig) {
        return D == 128 ? (w >> 2) * 64 + tig * 16 + (w & 3) * 4 : (w >> 1) * 32 + tig * 8 + (w & 1) * 4;
    }
    __device__ __forceinline__ void load_key(int i, const uint8_t* row, int tig) {
        if constexpr (D == 128) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 x = ld_stream(row + c * 64 + tig * 16);
                k[i][4 * c] = x.x;
                k[i][4 * c + 1] = x.y;
                k[i][4 * c + 2] = x.z;
                k[i][4 * c + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const uint2 x = ld_stream8(row + c * 32 + tig * 8);
                k[i][2 * c] = x.x;
                k[i][2 * c + 1] = x.y;
            }
        }
    }
    __device__ __forceinline__ void load_value(int i, const uint8_t* row, int gid) {
        if constexpr (D == 128) {
            const uint4 x = ld_stream(row + gid * 16);
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
        } else {
#pragma unroll
            for (int c = 0; c < 3; ++c) v[i][c] = ld_stream4(row + gid * 12 + c * 4);
        }
    }
    __device__ __forceinline__ void zero_key(int i) {
#pragma unroll
        for (int w = 0; w < KW; ++w) k[i][w] = 0u;
    }
    __device__ __forceinline__ void zero_value(int i) {
#pragma unroll
        for (int w = 0; w < VW; ++w) v[i][w] = 0u;
    }
};

// NT groups of up to four query heads of one KV head: their query fragments,
// running softmax state and output accumulators. Lane (gid, tig) accumulates
// head 4 t + tig, columns gid D / 8 ..; m is the same in the eight lanes of a
// head, l is the lane's own tokens' share.
template <int D, int NT>
struct Heads {
    static constexpr int KW = Frag<D>::KW, VW = Frag<D>::VW;
    uint32_t q[NT][KW][2];
    float qs[NT], m[NT], l[NT], acc[NT][4 * VW];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * VW; ++i) acc[t][i] = 0.f;
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

    // One tile: ok0, ok1 and the key scales k0, k1 are those of the lane's key
    // tokens; the values of tokens left out are zero. One value scale for the
    // tile (kOneScale: v0), or one per token (v0, v1).
    template <bool kOneScale>
    __device__ __forceinline__ void add(const Frag<D>& f, bool ok0, bool ok1, float k0, float k1, float v0,
                                        float v1, int gid, int tig) {
        float c[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[t][i] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(f.k[0][w] & 0xffffu), a1 = e4m3x2_to_f16x2(f.k[1][w] & 0xffffu);
            const uint32_t a2 = e4m3x2_to_f16x2(f.k[0][w] >> 16), a3 = e4m3x2_to_f16x2(f.k[1][w] >> 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(c[t], a0, a1, a2, a3, q[t][w][0], q[t][w][1]);
        }
        uint32_t pf[NT][2];
        float keep[NT], gain[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float x0 = ok0 ? (c[t][0] + c[t][1]) * qs[t] * k0 : -INFINITY;
            const float x1 = ok1 ? (c[t][2] + c[t][3]) * qs[t] * k1 : -INFINITY;
            float mt = fmaxf(x0, x1);
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
            const float M = fmaxf(m[t], mt);
            keep[t] = m[t] == M ? 1.f : exp2f(m[t] - M);
            // all of the tile's scores -inf: its weights are zero, not NaN (a
            // NaN score makes p NaN, which l carries to the output)
            const float base = mt == -INFINITY ? 0.f : mt;
            float p0 = exp2f(x0 - base), p1 = exp2f(x1 - base);
            gain[t] = mt == -INFINITY ? 0.f : exp2f(mt - M);
            l[t] = l[t] * keep[t] + gain[t] * (p0 + p1);
            m[t] = M;
            float up = 32768.f;  // largest weight at 2^15
            if constexpr (kOneScale) {
                gain[t] *= v0 * (1.f / 32768.f);
            } else {
                p0 *= v0;
                p1 *= v1;
                float top = fmaxf(p0, p1);
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                int e = 14 + 127 - (int)(__float_as_uint(top) >> 23);
                e = e > 126 ? 126 : e;
                up = __uint_as_float((uint32_t)(e + 127) << 23);
                gain[t] *= __uint_as_float((uint32_t)(127 - e) << 23);
            }
            p0 *= up;
            p1 *= up;
            // column gid of the weights: head gid / 2, part gid % 2, of tokens 4 tig ..
            const int src = 8 * tig + (gid >> 1);
            const float w0 = __shfl_sync(0xffffffffu, p0, src), w1 = __shfl_sync(0xffffffffu, p0, src + 4);
            const float w2 = __shfl_sync(0xffffffffu, p1, src), w3 = __shfl_sync(0xffffffffu, p1, src + 4);
            pf[t][0] = f16_part(w0, w1, gid & 1);
            pf[t][1] = f16_part(w2, w3, gid & 1);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // bytes (A, B) of one column side by side, two columns a word
                const uint32_t ab = __byte_perm(f.v[0][w], f.v[1][w], half ? 0x7362 : 0x5140);
                const uint32_t cd = __byte_perm(f.v[2][w], f.v[3][w], half ? 0x7362 : 0x5140);
                const uint32_t a0 = e4m3x2_to_f16x2(ab & 0xffffu), a1 = e4m3x2_to_f16x2(ab >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(cd & 0xffffu), a3 = e4m3x2_to_f16x2(cd >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float o[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(o, a0, a1, a2, a3, pf[t][0], pf[t][1]);
                    float* A = acc[t] + 4 * w + 2 * half;
                    A[0] = fmaf(gain[t], o[0] + o[1], A[0] * keep[t]);
                    A[1] = fmaf(gain[t], o[2] + o[3], A[1] * keep[t]);
                }
            }
        }
    }

    // The state of rows row0 .. as output (slot < 0) or as the partial `slot`.
    template <class E>
    __device__ __forceinline__ void store(const AttendQ8Args& a, int64_t row0, int G, int64_t slot, int gid,
                                          int tig) {
        float2* ml = static_cast<float2*>(a.ws);
        float* pa = reinterpret_cast<float*>(ml + a.slots * G);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int g = 4 * t + tig;
            float L = l[t];
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
            if (g >= G) continue;
            if (slot < 0) {
                typename E::T* o = static_cast<typename E::T*>(a.out) + (row0 + g) * D + gid * (D / 8);
                const float r = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i) o[i] = E::from_float(acc[t][i] * r);
            } else {
                if (gid == 0) ml[slot * G + g] = make_float2(m[t], L);
                float4* o = reinterpret_cast<float4*>(pa + (slot * G + g) * D + gid * (D / 8));
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    o[i] = make_float4(acc[t][4 * i], acc[t][4 * i + 1], acc[t][4 * i + 2], acc[t][4 * i + 3]);
            }
        }
    }
};

__device__ __forceinline__ int64_t q8_len(const AttendQ8Args& a, int b) {
    const int64_t cap = (int64_t)a.page_size * a.max_pages, n = __ldg(a.seq_lens + b);
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// tiles of the sequences before b (per KV head), and of all
__device__ __forceinline__ void q8_tiles(const AttendQ8Args& a, int b, int64_t* before, int64_t* total) {
    int64_t x = 0, y = 0;
    for (int i = threadIdx.x & 31; i < a.B; i += 32) {
        const int64_t n = (q8_len(a, i) + kTile - 1) / kTile;
        y += n;
        if (i < b) x += n;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    *before = x;
    *total = y;
}

// the sequence of tile w (counting H_kv runs of tiles per sequence)
__device__ __forceinline__ int q8_find(const AttendQ8Args& a, int64_t w, int64_t* before) {
    const int lane = threadIdx.x & 31;
    int64_t carry = 0;
    for (int base = 0; base < a.B; base += 32) {
        int64_t n = base + lane < a.B ? (q8_len(a, base + lane) + kTile - 1) / kTile : 0;
        const int64_t own = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, n, off);
            if (lane >= off) n += o;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, w < a.H_kv * (carry + n));
        if (hit != 0) {
            const int at = __ffs(hit) - 1;
            *before = carry + __shfl_sync(0xffffffffu, n - own, at);
            return base + at;
        }
        carry += __shfl_sync(0xffffffffu, n, 31);
    }
    *before = 0;
    return -1;
}

template <class E, int D, int NT>
__global__ void __launch_bounds__(kQ8Threads, NT == 1 ? 4 : 3) k_dense_q8(const AttendQ8Args a) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int64_t wi = (int64_t)blockIdx.x * (kQ8Threads / 32) + (threadIdx.x >> 5);
    const int G = a.H_q / a.H_kv;
    int64_t before, total;
    q8_tiles(a, 0, &before, &total);
    total *= a.H_kv;
    const int64_t per = (total + a.warps - 1) / a.warps;
    int64_t w = wi * per;
    const int64_t w_end = min64(w + per, total);
    if (w >= w_end) return;
    int b = q8_find(a, w, &before);
    if (b < 0) return;
    int len = (int)q8_len(a, b);
    int n = (len + kTile - 1) / kTile;  // tiles of a unit
    int hk = (int)((w - before * a.H_kv) / n);
    int t = (int)((w - before * a.H_kv) % n);

    // the loads run one tile ahead of the arithmetic: lb, lhk, lt, ... are theirs
    int lb = b, lhk = hk, lt = t, llen = len, ln = n;
    int lp = -1, lpage = -1, loff = 0;  // page index, page, first token in it
    const uint8_t *K = nullptr, *V = nullptr;
    struct Next {
        Frag<D> f;
        float ks, vs;
        int valid;
    } nx, cu;
    const int tk = 4 * (gid >> 1) + (gid & 1);
    auto load = [&](Next& x) {
        const int j = lt * kTile;
        if (lp < 0) {
            lp = j / a.page_size;
            loff = j - lp * a.page_size;
            lpage = __ldg(a.block_table + (int64_t)lb * a.max_pages + lp);
        } else if (loff == a.page_size) {
            ++lp;
            loff = 0;
            lpage = __ldg(a.block_table + (int64_t)lb * a.max_pages + lp);
        }
        if (lpage >= 0 && lpage < a.n_pages) {
            const int64_t row = ((int64_t)lpage * a.H_kv + lhk) * a.page_size + loff;
            K = a.K_pages + row * D;
            V = a.V_pages + row * D;
            x.valid = llen - j;
            x.f.load_key(0, K + tk * D, tig);
            x.f.load_key(1, K + (tk + 2) * D, tig);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.f.load_value(i, V + (4 * tig + i) * D, gid);
            const int64_t blk = row >> a.block_log2;
            x.ks = __ldg(a.k_scales + blk);
            x.vs = __ldg(a.v_scales + blk);
        } else {
            x.valid = 0;
            if (lane == 0) atomicExch(a.err, kDevErrBadPage);
        }
        loff += kTile;
        if (++lt == ln) {  // the next unit with tokens
            lt = 0;
            lp = -1;
            if (++lhk == a.H_kv) {
                lhk = 0;
                do {
                    if (++lb >= a.B) break;
                    llen = (int)q8_len(a, lb);
                } while (llen == 0);
                ln = (llen + kTile - 1) / kTile;
            }
        }
    };

    Heads<D, NT> h;
    h.reset();
    h.load(a, (int64_t)b * a.H_q + (int64_t)hk * G, G, gid, tig);
    bool whole = t == 0;
    load(cu);
    while (true) {
        const bool more = w + 1 < w_end;
        if (more) load(nx);
        if (cu.valid > 0) {
            if (cu.valid < kTile) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * tig + i >= cu.valid) cu.f.zero_value(i);
            }
            h.template add<true>(cu.f, tk < cu.valid, tk + 2 < cu.valid, cu.ks, cu.ks, cu.vs, cu.vs, gid, tig);
        }
        ++t;
        ++w;
        if (t == n || !more) {
            const int64_t unit = (int64_t)b * a.H_kv + hk;
            h.template store<E>(a, unit * G, G, whole && t == n ? -1 : unit + wi, gid, tig);
            if (!more) return;
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
        cu = nx;
    }
}

// Selected tokens: a tile is 16 consecutive entries of a row's list; lane l
// looks up entry l % 16 and hands its row number to the lanes that load it.
template <class E, int D>
__global__ void __launch_bounds__(kQ8Threads, 4) k_sparse_q8(const AttendQ8Args a) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int64_t wi = (int64_t)blockIdx.x * (kQ8Threads / 32) + (threadIdx.x >> 5);
    const int G = a.H_q / a.H_kv;
    const int64_t n = (a.k + kTile - 1) / kTile, total = n * a.B * a.H_q;
    const int64_t per = (total + a.warps - 1) / a.warps;
    int64_t w = wi * per;
    const int64_t w_end = min64(w + per, total);
    if (w >= w_end) return;
    int64_t r = w / n, t = w % n;
    const int tk = 4 * (gid >> 1) + (gid & 1);

    // entries run two tiles ahead of the arithmetic, rows one
    int64_t ir = r, it = t;
    auto entry = [&]() -> int {
        const int64_t e = it * kTile + (lane & 15);
        const int j = e < a.k ? __ldg(a.idx + ir * a.k + e) : -1;
        if (++it == n) {
            it = 0;
            ++ir;
        }
        return j;
    };
    int64_t lr = r, lt = t;
    int lb = (int)(r / a.H_q), lhk = (int)(r % a.H_q) / G, llen = (int)q8_len(a, lb);
    struct Next {
        Frag<D> f;
        float ks, vs;  // of entry lane % 16
        uint32_t ok;   // bit per entry
    } nx, cu;
    auto load = [&](Next& x, int j) {
        uint32_t row = kNoRow;
        x.ks = x.vs = 0.f;
        if (j >= 0 && j < llen) {
            const uint32_t lp = a.page_log2 >= 0 ? (uint32_t)j >> a.page_log2 : (uint32_t)j / (uint32_t)a.page_size;
            const int page = __ldg(a.block_table + (int64_t)lb * a.max_pages + lp);
            if (page >= 0 && page < a.n_pages) {
                row = ((uint32_t)page * a.H_kv + lhk) * a.page_size + ((uint32_t)j - lp * a.page_size);
                x.ks = __ldg(a.k_scales + (row >> a.block_log2));
                x.vs = __ldg(a.v_scales + (row >> a.block_log2));
            } else {
                atomicExch(a.err, kDevErrBadPage);
            }
        }
        x.ok = __ballot_sync(0xffffffffu, row != kNoRow) & 0xffffu;
        if (x.ok != 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row, tk + 2 * i);
                if (rr != kNoRow) x.f.load_key(i, a.K_pages + (int64_t)rr * D, tig);
                else x.f.zero_key(i);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row, 4 * tig + i);
                if (rr != kNoRow) x.f.load_value(i, a.V_pages + (int64_t)rr * D, gid);
                else x.f.zero_value(i);
            }
        }
        if (++lt == n) {
            lt = 0;
            if (++lr < (int64_t)a.B * a.H_q) {
                lb = (int)(lr / a.H_q);
                lhk = (int)(lr % a.H_q) / G;
                llen = (int)q8_len(a, lb);
            }
        }
    };

    Heads<D, 1> h;
    h.reset();
    const int j0 = entry();
    int j1 = w + 1 < w_end ? entry() : -1;
    h.load(a, r, 1, gid, tig);
    bool whole = t == 0;
    load(cu, j0);
    while (true) {
        const bool more = w + 1 < w_end;
        if (more) {
            const int j = j1;
            if (w + 2 < w_end) j1 = entry();
            load(nx, j);
        }
        if (cu.ok != 0) {
            const float k0 = __shfl_sync(0xffffffffu, cu.ks, tk), k1 = __shfl_sync(0xffffffffu, cu.ks, tk + 2);
            const float v0 = __shfl_sync(0xffffffffu, cu.vs, tk), v1 = __shfl_sync(0xffffffffu, cu.vs, tk + 2);
            h.template add<false>(cu.f, (cu.ok >> tk) & 1u, (cu.ok >> (tk + 2)) & 1u, k0, k1, v0, v1, gid, tig);
        }
        ++t;
        ++w;
        if (t == n || !more) {
            h.template store<E>(a, r, 1, whole && t == n ? -1 : r + wi, gid, tig);
            if (!more) return;
            t = 0;
            whole = true;
            ++r;
            h.reset();
            h.load(a, r, 1, gid, tig);
        }
        cu = nx;
    }
}

// Merges the partials of one (sequence, query head) row: the warps take
// partials in turn, four columns a lane. Rows that one warp owned whole are
// written already; rows without tokens get zeros.
template <class E, int D>
__global__ void __launch_bounds__(128) k_q8_combine(const AttendQ8Args a) {
    __shared__ float sm_m[4], sm_l[4];
    __shared__ float4 sm_acc[4][32];
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();  // every block: the grid must not end before the partials' writers
    int64_t unit = r, first, last, per;
    int Gc = 1, g = 0;
    if (a.idx != nullptr) {
        const int64_t n = (a.k + kTile - 1) / kTile;
        per = (n * a.B * a.H_q + a.warps - 1) / a.warps;
        first = r * n;
        last = first + n - 1;
    } else {
        Gc = a.H_q / a.H_kv;
        const int b = (int)(r / a.H_q), h = (int)(r % a.H_q);
        int64_t before, total;
        q8_tiles(a, b, &before, &total);
        const int64_t n = (q8_len(a, b) + kTile - 1) / kTile;
        if (n == 0) {
            if (threadIdx.x < D) static_cast<typename E::T*>(a.out)[r * D + threadIdx.x] = E::from_float(0.f);
            return;
        }
        per = (total * a.H_kv + a.warps - 1) / a.warps;
        g = h % Gc;
        unit = (int64_t)b * a.H_kv + h / Gc;
        first = before * a.H_kv + (h / Gc) * n;
        last = first + n - 1;
    }
    const int64_t c0 = first / per;
    const int np = (int)(last / per - c0 + 1);
    if (np == 1 && first % per + (last - first) < per) return;
    const float2* ml = static_cast<const float2*>(a.ws) + (unit + c0) * Gc + g;
    const float* pa = reinterpret_cast<const float*>(static_cast<const float2*>(a.ws) + a.slots * Gc) +
                      ((unit + c0) * Gc + g) * D;
    float M = -INFINITY;
    for (int p = threadIdx.x; p < np; p += 128) M = fmaxf(M, ml[(int64_t)p * Gc].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) sm_m[warp] = M;
    __syncthreads();
    M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = lane * 4 < D;
#pragma unroll 4
    for (int p = warp; p < np; p += 4) {
        const float2 x = ml[(int64_t)p * Gc];
        const float s = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) y = *reinterpret_cast<const float4*>(pa + (int64_t)p * Gc * D + lane * 4);
        L += x.y * s;
        A.x = fmaf(y.x, s, A.x);
        A.y = fmaf(y.y, s, A.y);
        A.z = fmaf(y.z, s, A.z);
        A.w = fmaf(y.w, s, A.w);
    }
    sm_acc[warp][lane] = A;
    if (lane == 0) sm_l[warp] = L;
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= D) return;
    L = sm_l[0] + sm_l[1] + sm_l[2] + sm_l[3];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += reinterpret_cast<const float*>(sm_acc[i])[c];
    static_cast<typename E::T*>(a.out)[r * D + c] = E::from_float(L == 0.f ? 0.f : s / L);
}

// ---------------------------------------------------------------------------

// partials: a (unit, warp) pair for every border between the warps' runs and
// every unit, numbered unit + warp, which grows along the line of tiles
// (an even number: the columns behind the (m, l) pairs start on 16 bytes)
static int64_t q8_slots(int64_t units, int64_t tiles) {
    return (units + min64(kQ8MaxWarps, tiles) + 1) & ~(int64_t)1;
}

static size_t q8_ws_bytes(int64_t units, int64_t tiles, int G, int D) {
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

template <class E, int D>
static cudaError_t attend_impl(AttendQ8Args& a, cudaStream_t s) {
    const int G = a.H_q / a.H_kv;
    auto kern = a.idx != nullptr ? k_sparse_q8<E, D> : G <= 4 ? k_dense_q8<E, D, 1> : k_dense_q8<E, D, 2>;
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    // no shared memory: the table, scale and index loads want the L1
    e = prefer_carveout((const void*)kern, cudaSharedmemCarveoutMaxL1);
    if (e != cudaSuccess) return e;
    const int64_t units = a.idx != nullptr ? (int64_t)a.B * a.H_q : (int64_t)a.B * a.H_kv;
    const int64_t items = a.idx != nullptr ? a.k : (int64_t)a.page_size * a.max_pages;
    const int64_t tiles = units * ((items + kTile - 1) / kTile);
    const int wpc = kQ8Threads / 32;
    int64_t warps = (int64_t)di.sm_count * occupancy((const void*)kern, kQ8Threads, 0) * wpc;
    warps = min64(min64(warps, kQ8MaxWarps), tiles);
    a.warps = (int)warps;
    a.slots = q8_slots(units, tiles);
    e = launch_kernel(kern, dim3((unsigned)((warps + wpc - 1) / wpc)), dim3(kQ8Threads), 0, s, false, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(k_q8_combine<E, D>, dim3((unsigned)((int64_t)a.B * a.H_q)), dim3(128), 0, s, true, a);
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
