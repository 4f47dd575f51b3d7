// The keys of a longer append to a paged cache: K~ = rope(K) P for tiles of
// 128 tokens of one KV head, on the fifth-generation tensor cores, stored in
// the cache's type or as 8-bit codes with their blocks' scales.
//
// The product is 2 D flop for each of a key's D outputs, and has to come out
// as fp32 would give it (the plane's scores choose tokens by it). Both sides
// are carried as two fp16 parts, x = hi + lo (22 bits, after a power of two
// per row of keys and per column of P has brought the largest entry to
// 2^14..2^15), and three of the four products are taken: hi hi, hi lo, lo hi;
// the fourth lies below 2^-22 of the product. So 6 D flop per output, at the
// fp16 rate with fp32 accumulators in tensor memory.
//
//   A [128 tokens x D]  hi, lo: written by the warps after the rotation
//   B [D columns x D]   hi, lo: P transposed, written once per head
//   both in shared memory, K-major, 128-byte swizzle, 64 columns to an atom;
//   D [128 x D] fp32 in tensor memory, read back one row to a lane.
//
// A persistent CTA takes consecutive tiles with the head slowest, so most keep
// their P. The next tile's keys are loaded while the tensor cores and the
// epilogue work. Rows that hold an infinity or a NaN take the plain fp32 sum
// instead (an infinity has no second part).
#include <cuda_fp16.h>

#include "append_paged.cuh"

namespace loki {

constexpr int kAbThreads = 256, kAbRows = 128;
constexpr int kAbAtom = kAbRows * 128;  // bytes of 128 rows of 64 fp16 columns
constexpr int kAbSmem = 8 * kAbAtom + 1024;

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, eight rows of
// 128 bytes to a group, groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// tensor memory [128 x n] (+)= A B^T, one K step of 16 fp16
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(float* f, uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// exponent e that brings `top` to 2^14..2^15, within what 2^e and 2^-e can be
__device__ __forceinline__ int lift(float top) {
    const int e = 14 + 127 - (int)(__float_as_uint(top) >> 23);
    return e > 126 ? 126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// eight values times `up` as fp16 parts, to chunk `col / 8` of `row` of a
// swizzled matrix pair (hi, lo two atoms apart)
__device__ __forceinline__ void put_parts(uint8_t* m, int row, int col, const float* x, float up) {
    uint4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float p = x[2 * i] * up, q = x[2 * i + 1] * up;
        const __half2 h = __floats2half2_rn(p, q);
        const float2 f = __half22float2(h);
        const __half2 r = __floats2half2_rn(p - f.x, q - f.y);
        (&hi.x)[i] = *reinterpret_cast<const uint32_t*>(&h);
        (&lo.x)[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    const int c = col >> 3;
    uint8_t* at = m + (c >> 3) * kAbAtom + row * 128 + (((c & 7) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = hi;
    *reinterpret_cast<uint4*>(at + 2 * kAbAtom) = lo;
}

// aligned runs of 128 positions that sequence b's written tokens touch
__device__ __forceinline__ int append_runs(const ApSeq& s) {
    return s.hi > s.lo ? (int)((s.hi - 1) / kAbRows - s.lo / kAbRows) + 1 : 0;
}

template <class E, int D, bool kQ8>
__global__ void __launch_bounds__(kAbThreads, 1) k_append_basis(const AppendArgs a) {
    using Tp = typename E::T;
    constexpr int DH = D / 2;  // an epilogue thread's columns
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float col_down[128];
    __shared__ float row_down[kAbRows], red[2][kAbRows / 16];
    __shared__ uint8_t odd_row[kAbRows];
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t tmem_slot;
    uint8_t* A = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    uint8_t* Bm = A + 4 * kAbAtom;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    // this CTA's tiles: heads slowest, then sequences, then their runs
    int64_t R = 0;
    for (int i = lane; i < a.B; i += 32) R += append_runs(append_seq(a, i, false));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) R += __shfl_xor_sync(0xffffffffu, R, off);
    const int64_t total = R * a.H_kv, per = (total + gridDim.x - 1) / gridDim.x;
    int64_t w = blockIdx.x * per;
    const int64_t w_end = min64(w + per, total);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;

    int hk = -1, b = 0, run = 0, runs = 0;
    ApSeq sq{};
    if (w < w_end) {
        hk = (int)(w / R);
        int64_t skip = w % R;
        for (;; ++b) {  // total > w: some sequence holds it
            sq = append_seq(a, b, false);
            runs = append_runs(sq);
            if (skip < runs) break;
            skip -= runs;
        }
        run = (int)skip;
    }

    // keys of a tile as loaded: four rows a thread, unit u of each
    const int u = lane & 7, sub = lane >> 3;
    const bool unit_on = u < D / 16, turn = a.rope != nullptr && u < a.rot_dim >> 4;
    int ca, cb;
    unit_cols(turn ? a.rot_dim : 0, a.interleaved, u, &ca, &cb);
    Chunk<E> wa[4], wb[4];
    bool live[4];
    auto load = [&]() {
        const int64_t start = (sq.lo / kAbRows + run) * kAbRows;
        const Tp* rows = static_cast<const Tp*>(a.K_new) + ((int64_t)b * a.H_kv + hk) * a.T * D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = start + 16 * warp + 4 * i + sub;
            live[i] = unit_on && j >= sq.lo && j < sq.hi;
            if (live[i]) {
                wa[i].load(rows + (j - sq.p0) * D + ca);
                wb[i].load(rows + (j - sq.p0) * D + cb);
            }
        }
    };
    if (w < w_end) load();

    const uint32_t idesc = 1u << 4 | (uint32_t)(D >> 3) << 17 | (uint32_t)(kAbRows >> 4) << 24;
    int held = -1;  // the head whose P is in shared memory
    uint32_t phase = 0;
    while (w < w_end) {
        const int64_t start = (sq.lo / kAbRows + run) * kAbRows, lo = sq.lo, hi = sq.hi, p0 = sq.p0;
        const int tb = b, th = hk;
        if (held != th) {
            held = th;
            const float* Ph = a.P + (int64_t)th * D * D;
            // two threads to a column: its rows' largest magnitude, then its parts
            const int c = tid & 127, half = tid >> 7;
            float x[8], top = 0.f;
            if (c < D)
                for (int i = 0; i < D; ++i) top = fmaxf(top, finite_abs(__ldg(Ph + i * D + c)));
            const int e = lift(top);
            const float up = pow2(e);
            if (half == 0) col_down[c] = pow2(-e);
            if (c < D)
                for (int i = half * DH; i < half * DH + DH; i += 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = __ldg(Ph + (i + k) * D + c);
                    put_parts(Bm, c, i, x, up);
                }
        }
        // rotation, then the rows' parts
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * warp + 4 * i + sub;
            float x[16], top = 0.f;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
            if (live[i]) {
                wa[i].get(x);
                wb[i].get(x + 8);
                if (turn) turn_unit(a.rope, a.rot_dim, a.interleaved, start + r, u, x);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float m = fabsf(x[e]);
                odd |= !(m <= 3.402823466e38f);
                top = fmaxf(top, m);
            }
#pragma unroll
            for (int off = 1; off <= 4; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            odd = (__ballot_sync(0xffffffffu, odd) >> (lane & 24) & 0xffu) != 0;
            const int e = odd ? 0 : lift(top);
            if (u == 0) {
                row_down[r] = pow2(-e);
                odd_row[r] = odd;
            }
            if (unit_on) {
                put_parts(A, r, ca, x, pow2(e));
                put_parts(A, r, cb, x + 8, pow2(e));
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t sa = smem_addr(A), sb = smem_addr(Bm);
#pragma unroll
            for (int pass = 0; pass < 3; ++pass)
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * kAbAtom + (k & 3) * 32;
                    mma_f16_ss(tmem, smem_desc(sa + (pass == 2 ? 2 * kAbAtom : 0) + at),
                               smem_desc(sb + (pass == 1 ? 2 * kAbAtom : 0) + at), idesc, pass + k > 0);
                }
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                             smem_addr(&bar))
                         : "memory");
        }
        // the next tile's keys, meanwhile
        if (++w < w_end) {
            if (++run == runs) {
                run = 0;
                do {
                    if (++b == a.B) {
                        b = 0;
                        ++hk;
                    }
                    sq = append_seq(a, b, false);
                    runs = append_runs(sq);
                } while (runs == 0);
            }
            load();
        }
        // this thread's row of the product, half of its columns
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const int64_t j = start + r;
        const bool mine = j >= lo && j < hi;
        const bool has_row = mine || (kQ8 && j < lo);
        const int block_start = kQ8 ? (int)(j & ~(int64_t)(a.block - 1)) : 0;
        // older rows of a block that receives tokens count too: they may move to a larger scale
        const bool has_new = kQ8 && block_start < hi && block_start + a.block > lo;
        const bool has_old = kQ8 && lo > block_start;
        int row = -1;
        float old = 0.f;
        if (kQ8 ? (has_row && has_new) : mine) row = pool_row(a, tb, th, (int)j);
        if (kQ8 && row >= 0 && has_old) old = a.k_scales[row >> a.block_log2];
        const bool done = mbar_wait(&bar, phase, a.err);
        phase ^= 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        float y[DH];
#pragma unroll
        for (int i = 0; i < DH; i += 16) tmem_ld16(y + i, tmem + ((uint32_t)(warp & 3) << 21) + half * DH + i);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        const float down = row_down[r];
#pragma unroll
        for (int i = 0; i < DH; i += 4) {
            const float4 cd = *reinterpret_cast<const float4*>(&col_down[half * DH + i]);
            y[i] = y[i] * down * cd.x;
            y[i + 1] = y[i + 1] * down * cd.y;
            y[i + 2] = y[i + 2] * down * cd.z;
            y[i + 3] = y[i + 3] * down * cd.w;
        }
        if (mine && odd_row[r]) {
#pragma unroll
            for (int i = 0; i < DH; ++i) y[i] = 0.f;
            const Tp* K = static_cast<const Tp*>(a.K_new) + (((int64_t)tb * a.H_kv + th) * a.T + (j - p0)) * D;
            const float* Ph = a.P + (int64_t)th * D * D + half * DH;
            for (int i = 0; i < D; ++i) {
                const float x = turned_col<E>(a, K, j, i);
#pragma unroll
                for (int c = 0; c < DH; ++c) y[c] = fmaf(x, __ldg(Ph + i * D + c), y[c]);
            }
        }
        if (mine && row >= 0 && a.plane != nullptr) {
            Tp* o = static_cast<Tp*>(a.plane) + (int64_t)row * a.d_lo + half * DH;
#pragma unroll
            for (int i = 0; i < DH; i += E::kVec)
                if (half * DH + i < a.d_lo) *reinterpret_cast<uint4*>(o + i) = pack16(y + i, E());
        }
        if constexpr (!kQ8) {
            if (mine && row >= 0) {
                Tp* o = static_cast<Tp*>(a.K_pages) + (int64_t)row * D + half * DH;
#pragma unroll
                for (int i = 0; i < DH; i += E::kVec) *reinterpret_cast<uint4*>(o + i) = pack16(y + i, E());
            }
        } else {
            float top = 0.f;
            if (mine) {
#pragma unroll
                for (int i = 0; i < DH; ++i) top = fmaxf(top, finite_abs(y[i]));
            }
#pragma unroll
            for (int off = 1; off <= 8; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if ((lane & 15) == 0) red[half][r >> 4] = top;
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        // the tile's reads of tensor and shared memory are over (8 bits: its
        // magnitudes are there, and every row has read its block's old scale)
        if (__syncthreads_or(!done)) break;
        if constexpr (kQ8) {
            if (row >= 0) {
                const int g0 = (r & ~(a.block - 1)) >> 4;
                float top = 0.f;
                for (int g = g0; g < g0 + (a.block >> 4); ++g) top = fmaxf(top, fmaxf(red[0][g], red[1][g]));
                const float grown = pow2_scale(top), s = has_old ? fmaxf(old, grown) : grown;
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.K_pages) + (int64_t)row * D + half * DH);
                if (mine) {
                    const float inv = 1.f / s;
#pragma unroll
                    for (int i = 0; i < DH; i += 16) {
                        const uint2 p = codes8(y + i, inv), q = codes8(y + i + 8, inv);
                        o[i >> 4] = make_uint4(p.x, p.y, q.x, q.y);
                    }
                    if (half == 0 && j == (block_start > lo ? block_start : lo)) a.k_scales[row >> a.block_log2] = s;
                } else if (s > old) {
                    const float f = old / s;
#pragma unroll
                    for (int i = 0; i < DH >> 4; ++i) {
                        uint4 v = o[i];
                        v.x = rescale4(v.x, f);
                        v.y = rescale4(v.y, f);
                        v.z = rescale4(v.z, f);
                        v.w = rescale4(v.w, f);
                        o[i] = v;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem));
}

template <class E, bool kQ8>
static cudaError_t basis_impl(const AppendArgs& a, cudaStream_t s) {
    auto kern = a.D == 96 ? k_append_basis<E, 96, kQ8> : k_append_basis<E, 128, kQ8>;
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAbSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (((int64_t)a.T + kAbRows - 2) / kAbRows + 1) * a.B * a.H_kv;
    return launch_kernel(kern, dim3((unsigned)min64(tiles, di.sm_count)), dim3(kAbThreads), kAbSmem, s, false, a);
}

cudaError_t launch_append_basis(Dt dt, const AppendArgs& a, cudaStream_t s) {
    if (dt == kF32) return a.block > 0 ? basis_impl<ElemF32, true>(a, s) : basis_impl<ElemF32, false>(a, s);
    return a.block > 0 ? basis_impl<ElemBF16, true>(a, s) : basis_impl<ElemBF16, false>(a, s);
}

}  // namespace loki
