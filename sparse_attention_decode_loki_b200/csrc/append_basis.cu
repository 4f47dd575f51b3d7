// The keys of a longer append to a paged cache: K~ = rope(K) P for tiles of
// 128 tokens of one KV head, on the fifth-generation tensor cores, stored in
// the cache's type or as 8-bit codes with their blocks' scales.
//
// The product is 2 D flop for each of a key's D outputs, and has to come out
// as fp32 would give it (the plane's scores choose tokens by it). Both sides
// are carried as two fp16 parts, x = hi + lo (after a power of two per row of
// keys and per column of P has brought the largest entry to 2^14..2^15: 22 bits,
// or 2^-39 of the largest entry where that is more), and three of the four products are taken: lo hi, hi lo, hi hi;
// the fourth lies below 2^-22 of the product. So 6 D flop per output, at the
// fp16 rate with fp32 accumulators in tensor memory.
//
//   A [128 tokens x D]  hi, lo: written by the warps after the rotation
//   B [D columns x D]   hi, lo: P transposed, written once per head
//   both in shared memory, K-major, 128-byte swizzle, 64 columns to an atom;
//   D [128 x D] fp32 in tensor memory, read back one row to a lane.
//
// A persistent CTA of eight warps takes consecutive tiles with the head slowest,
// so most keep their P. In bf16 it leaves half of the SM's registers to the stream
// of values and queries, which runs beside it as a programmatic dependent: both
// wait on latencies most of the time. (fp32 rows in flight take 216 to 255 registers
// a thread, the whole SM: there the stream fills it as the tiles' CTAs end.) Stores go through shared memory (a lane
// holds one row: stored directly, each 16 bytes would touch another line, which
// took 1.5 us a tile). Rows that hold an infinity or a NaN take the plain fp32
// sum instead (an infinity has no second part).
//
// Measured on a 4096-token prompt of 32 heads into 8 bits: 53 us alone, 63 us
// with the stream (27 alone) beside it; 7 us a tile, of which 1.7 us turn and
// split, 1.2 us products, 1.6 us the two passes over the product, 0.7 us copies.
// Latencies of these phases bound it (36 % of issue slots, 13 % of the tensor
// pipe). Two groups of warps with an A each took the whole SM and 55 us; a warp
// of its own for the products caps 17 warps at 96 registers, which spill: 69.
#include <cuda_fp16.h>

#include "append_paged.cuh"

namespace loki {

constexpr int kAbThreads = 256;
constexpr int kAbAtom = kRunRows * 128;  // bytes of 128 rows of 64 fp16 columns
constexpr int kAbSmem = 8 * kAbAtom + 1024;  // and the tile's angles behind them

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

// byte `at` (a multiple of 16) of staged row r of `pitch` bytes: 16-byte chunks
// swizzled, for lanes a row apart as well as for lanes along a row
__device__ __forceinline__ int stage_at(int r, int at, int pitch) { return r * pitch + (at ^ ((r & 7) << 4)); }

template <class E, int D, bool kQ8>
__global__ void __launch_bounds__(kAbThreads, E::kBytes == 2 ? 2 : 1) k_append_basis(const AppendArgs a) {
    using Tp = typename E::T;
    constexpr int DH = D / 2;               // an epilogue thread's columns, and a thread's rows of P
    constexpr int DC = D == 128 ? 32 : 16;  // of the columns at a time
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float col_down[128];
    __shared__ float col_top[2][128];
    __shared__ float row_down[kRunRows], red[2][kRunRows / 16];
    __shared__ int place[kRunRows];  // the tile's rows in the pool, -1: not written
    __shared__ uint8_t odd_row[kRunRows];
    __shared__ __align__(8) uint64_t bar, angle_bar, basis_bar;
    __shared__ uint32_t tmem_slot;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* Bm = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    uint8_t* A = Bm + 4 * kAbAtom;
    float* angles = reinterpret_cast<float*>(A + 4 * kAbAtom);  // [128][rot_dim]
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        mbar_init(&bar, 1);
        mbar_init(&angle_bar, 1);
        mbar_init(&basis_bar, 1);
        fence_mbar_init();
    }
    griddep_wait();  // launched early: inputs and pages may still be in use
    fence_proxy_async_global();  // P and the angles come by bulk copies
    griddep_launch_dependents();  // the stream of values and queries
    // this CTA's tiles: heads slowest, then sequences, then their runs
    auto runs_of = [&](int b) -> int64_t {
        const ApSeq s = append_seq(a, b, false);
        return run_count(s.lo, s.hi);
    };
    const int64_t R = seqs_total(a.B, runs_of), total = R * a.H_kv, per = quot(total + gridDim.x - 1, gridDim.x);
    int64_t w = min64(blockIdx.x * per, total);
    const int64_t w_end = min64(w + per, total);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    constexpr uint32_t idesc = 1u << 4 | (uint32_t)(D >> 3) << 17 | (uint32_t)(kRunRows >> 4) << 24;

    // the tile at hand or next: run `run` of sequence b under head hk
    int hk = 0, b = 0, run = 0, runs = 0;
    ApSeq sq{};
    // its rows as loaded, four a thread, unit u of each, and its angles
    const int u = lane & 7, sub = lane >> 3, rot = a.rope != nullptr ? a.rot_dim : 0;
    const bool unit_on = u < D / 16, turn = u < rot >> 4;
    int ca, cb;
    unit_cols(turn ? rot : 0, a.interleaved, u, &ca, &cb);
    Chunk<E> wa[4], wb[4];
    uint32_t live = 0;
    uint32_t angle_loads = 0;  // thread 0's
    auto load = [&](bool ok) {
        const int64_t start = (sq.lo / kRunRows + run) * kRunRows, j0 = start + 16 * warp + sub;
        const Tp* p = static_cast<const Tp*>(a.K_new) + (((int64_t)b * a.H_kv + hk) * a.T + (j0 - sq.p0)) * D;
        if (rot > 0 && tid == 0 && ok) {  // every reader of the angles before has passed a barrier
            ++angle_loads;
            const uint32_t bytes = (uint32_t)min64(sq.hi - start, kRunRows) * rot * 4;
            mbar_arrive_expect_tx(&angle_bar, bytes);
            bulk_load(angles, a.rope + start * rot, bytes, &angle_bar);
        }
        live = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (unit_on && j0 + 4 * i >= sq.lo && j0 + 4 * i < sq.hi) {
                live |= 1u << i;
                wa[i].load(p + 4 * i * D + ca);
                wb[i].load(p + 4 * i * D + cb);
            }
    };

    uint32_t phase = 0;
    bool alive = true;
    uint32_t heads = 0;
    int64_t ri = 0;  // w's place under its head
    if (w < w_end) {
        hk = (int)quot(w, R);
        ri = w - hk * R;
    }
    for (; alive && w < w_end; ++hk, ri = 0) {  // head by head
        int64_t left = min64(w_end - w, R - ri);  // tiles under this head
        w += left;
        // P, as it is, to where A will be; two threads to a column, half of its rows each: the largest
        // magnitude, then the parts
        fence_proxy_async_shared();
        __syncthreads();  // the last head's product and staged rows are done with
        if (tid == 0) {
            mbar_arrive_expect_tx(&basis_bar, D * D * 4);
            bulk_load(A, a.P + (int64_t)hk * D * D, D * D * 4, &basis_bar);
        }
        int64_t before;
        b = seqs_find(a.B, ri, 1, runs_of, &before);
        sq = append_seq(a, b, false);
        runs = run_count(sq.lo, sq.hi);
        run = (int)(ri - before);
        load(true);
        {
            if (!mbar_wait(&basis_bar, heads & 1, a.err)) alive = false;
            ++heads;
            const int c = tid & 127, i0 = (tid >> 7) * DH;
            const float* Ph = reinterpret_cast<const float*>(A) + i0 * D + c;
            float top = 0.f;
            if (c < D) {
                float x[16];
#pragma unroll 1
                for (int i = 0; i < DH; i += 16) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] = Ph[(i + k) * D];
                    top = finite_amax<16>(top, x);
                }
            }
            col_top[tid >> 7][c] = top;
            __syncthreads();
            const int e = lift(fmaxf(col_top[0][c], col_top[1][c]));
            if (tid < 128) col_down[c] = pow2(-e);
            if (c < D) {
                float x[8];
#pragma unroll 2
                for (int i = 0; i < DH; i += 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = Ph[(i + k) * D];
                    put_parts(Bm, c, i0 + i, x, pow2(e));
                }
            }
            fence_proxy_async_shared();
            alive = !__syncthreads_or(!alive);
        }
        for (; alive && left > 0; --left) {
            const int64_t start = (sq.lo / kRunRows + run) * kRunRows, lo = sq.lo, hi = sq.hi, p0 = sq.p0;
            const int tb = b;
            // rotation, then the rows' parts
            bool done = rot == 0 || mbar_wait(&angle_bar, phase, a.err);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * warp + 4 * i + sub;
                float x[16], top = 0.f, zero = 0.f;  // zero: 0, or NaN where an entry is infinite or NaN
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 0.f;
                if (live >> i & 1u) {
                    wa[i].get(x);
                    wb[i].get(x + 8);
                    if (turn) turn_unit_from(angles + r * rot, rot, a.interleaved, u, x);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    top = fmaxf(top, fabsf(x[e]));
                    zero = fmaf(x[e], 0.f, zero);
                }
#pragma unroll
                for (int off = 1; off <= 4; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const bool odd = (__ballot_sync(0xffffffffu, zero != 0.f) >> (lane & 24) & 0xffu) != 0;
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
            fence_proxy_async_shared();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncthreads();
            if (tid == 0) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sa = smem_addr(A), sb = smem_addr(Bm);
#pragma unroll 1
                for (int pass = 0; pass < 3; ++pass)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = (k >> 2) * kAbAtom + (k & 3) * 32;
                        // lo hi, hi lo, then hi hi: the accumulator truncates at every step, so the small
                        // products come while it is small
                        mma_f16_ss(tmem, smem_desc(sa + (pass == 0 ? 2 * kAbAtom : 0) + at),
                                   smem_desc(sb + (pass == 1 ? 2 * kAbAtom : 0) + at), idesc, pass + k > 0);
                    }
                asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 smem_addr(&bar))
                             : "memory");
            }
            __syncwarp();
            if (left > 1) {  // the next tile, meanwhile
                ++run;
                while (run >= runs) {
                    run = 0;
                    ++b;
                    sq = append_seq(a, b, false);
                    runs = run_count(sq.lo, sq.hi);
                }
                load(done);
            }
            // this thread's row of the product, half of its columns
            const int r = (warp & 3) * 32 + lane, c0 = (warp >> 2) * DH;
            const int64_t j = start + r;
            const bool mine = j >= lo && j < hi;
            const int block_start = kQ8 ? (int)(j & ~(int64_t)(a.block - 1)) : 0;
            // older rows of a block that receives tokens count too: they may move to a larger scale
            const bool has_new = kQ8 && j < hi && block_start + a.block > lo;
            const bool has_old = kQ8 && lo > block_start;
            int row = -1;
            float old = 0.f;
            if (kQ8 ? has_new : mine) row = pool_row(a, tb, hk, (int)j);
            if (kQ8 && row >= 0 && has_old) old = a.k_scales[row >> a.block_log2];
            const bool write = mine && row >= 0;
            done = mbar_wait(&bar, phase, a.err) && done;
            phase ^= 1;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t cols = tmem + ((uint32_t)(warp & 3) << 21);
            const float down = row_down[r];
            const bool odd = mine && odd_row[r];
            // columns c .. c + DC - 1 of the row, times f / down
            auto columns = [&](int c, float* y, float f) {
#pragma unroll
                for (int i = 0; i < DC; i += 16) tmem_ld16(y + i, cols + c + i);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int i = 0; i < DC; i += 4) {
                    const float4 cd = *reinterpret_cast<const float4*>(&col_down[c + i]);
                    y[i] = y[i] * cd.x * f;
                    y[i + 1] = y[i + 1] * cd.y * f;
                    y[i + 2] = y[i + 2] * cd.z * f;
                    y[i + 3] = y[i + 3] * cd.w * f;
                }
                if (!odd) return;
                const Tp* K = static_cast<const Tp*>(a.K_new) + (((int64_t)tb * a.H_kv + hk) * a.T + (j - p0)) * D;
                const float* Ph = a.P + (int64_t)hk * D * D + c;
#pragma unroll
                for (int i = 0; i < DC; ++i) y[i] = 0.f;
#pragma unroll 1
                for (int i = 0; i < D; ++i) {
                    const float x = turned_col<E>(a, K, j, i);
#pragma unroll
                    for (int e = 0; e < DC; ++e) y[e] = fmaf(x, __ldg(Ph + i * D + e), y[e]);
                }
#pragma unroll
                for (int i = 0; i < DC; ++i) y[i] *= f;  // (an odd row's down is 1)
            };
            // The tile's outputs go into A, whose product is done: rows of the cache's type (8 bits: of the
            // plane, as far as they fit in front of the codes).
            uint8_t* stage8 = A + 3 * kAbAtom;
            const int lo_bytes = a.plane != nullptr ? a.d_lo * E::kBytes : 0;
            const int pitch = kQ8 ? (lo_bytes + 127) & ~127 : 128 * E::kBytes;  // whole swizzles
            const bool staged = !kQ8 || pitch * kRunRows <= 3 * kAbAtom;
            float top = 0.f;
#pragma unroll
            for (int c = c0; c < c0 + DH; c += DC) {
                float y[DC];
                columns(c, y, down);
                if (!kQ8 || (c < a.d_lo && staged)) {
#pragma unroll
                    for (int i = 0; i < DC; i += E::kVec)
                        if (!kQ8 || c + i < a.d_lo)
                            *reinterpret_cast<uint4*>(A + stage_at(r, (c + i) * E::kBytes, pitch)) = pack16(y + i, E());
                } else if (write && c < a.d_lo) {
                    Tp* o = static_cast<Tp*>(a.plane) + (int64_t)row * a.d_lo + c;
#pragma unroll
                    for (int i = 0; i < DC; i += 8) store_chunk<E>(o + i, y + i, c + i, a.d_lo);
                }
                if (kQ8 && mine) top = finite_amax<DC>(top, y);
            }
            if constexpr (kQ8) {
#pragma unroll
                for (int off = 1; off <= 8; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if ((lane & 15) == 0) red[warp >> 2][r >> 4] = top;
            }
            if (c0 == 0) place[r] = write ? row : -1;
            // staged (8 bits: magnitudes are there, and every row has read its block's old scale)
            alive = !__syncthreads_or(!done);
            if (!alive) break;
            if constexpr (kQ8) {
                const int g0 = (r & ~(a.block - 1)) >> 4;
                top = 0.f;
                for (int q = g0; q < g0 + (a.block >> 4); ++q) top = fmaxf(top, fmaxf(red[0][q], red[1][q]));
                const float grown = pow2_scale(top), s = has_old ? fmaxf(old, grown) : grown;
                const float f = fminf(down * (1.f / s), 3.402823466e38f);
#pragma unroll
                for (int c = c0; c < c0 + DH; c += DC) {
                    float y[DC];
                    columns(c, y, f);
#pragma unroll
                    for (int i = 0; i < DC; i += 16) {
                        const uint2 p = codes8(y + i, 1.f), q = codes8(y + i + 8, 1.f);
                        *reinterpret_cast<uint4*>(stage8 + stage_at(r, c + i, 128)) = make_uint4(p.x, p.y, q.x, q.y);
                    }
                }
                if (!write && row >= 0 && has_old && s > old) {
                    uint32_t* v = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.K_pages) + (int64_t)row * D + c0);
                    for (int c = 0; c < DH / 4; ++c) v[c] = rescale4(v[c], old / s);
                }
                if (write && c0 == 0 && j == (block_start > lo ? block_start : lo)) a.k_scales[row >> a.block_log2] = s;
                __syncthreads();
            }
            // the staged rows, 16 bytes a lane along the rows
            auto copy_out = [&](const uint8_t* from, int from_pitch, void* pool, int bytes) {
                const int per_row = bytes >> 4;
                int q = tid / per_row, c = tid - q * per_row;
                const int dq = kAbThreads / per_row, dc = kAbThreads - dq * per_row;
                for (; q < kRunRows; q += dq, c += dc) {
                    if (c >= per_row) {
                        c -= per_row;
                        ++q;
                        if (q >= kRunRows) break;
                    }
                    const int to = place[q];
                    if (to >= 0)
                        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(pool) + (int64_t)to * bytes + c * 16) =
                            *reinterpret_cast<const uint4*>(from + stage_at(q, c * 16, from_pitch));
                }
            };
            if constexpr (kQ8) copy_out(stage8, 128, a.K_pages, D);
            else copy_out(A, 128 * E::kBytes, a.K_pages, D * E::kBytes);
            if (lo_bytes > 0 && staged) copy_out(A, pitch, a.plane, lo_bytes);
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncthreads();  // A and place may be written again
        }
    }
    // flagged: copies and products on their way land (or not) before the CTA ends
    if (!alive && tid == 0) {
        mbar_wait(&basis_bar, (heads - 1) & 1, a.err);
        if (angle_loads > 0) mbar_wait(&angle_bar, (angle_loads - 1) & 1, a.err);
        mbar_wait(&bar, phase ^ 1, a.err);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem_slot));
}

template <class E, bool kQ8>
static cudaError_t basis_impl(const AppendArgs& a, cudaStream_t s) {
    auto kern = a.D == 96 ? k_append_basis<E, 96, kQ8> : k_append_basis<E, 128, kQ8>;
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    const int smem = kAbSmem + (a.rope != nullptr ? kRunRows * a.rot_dim * 4 : 0);
    e = allow_dynamic_smem((const void*)kern, kAbSmem + kRunRows * 128 * 4);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (((int64_t)a.T + kRunRows - 2) / kRunRows + 1) * a.B * a.H_kv;
    return launch_kernel(kern, dim3((unsigned)min64(tiles, di.sm_count)), dim3(kAbThreads), smem, s, true, a);
}

cudaError_t launch_append_basis(Dt dt, const AppendArgs& a, cudaStream_t s) {
    if (dt == kF32) return a.block > 0 ? basis_impl<ElemF32, true>(a, s) : basis_impl<ElemF32, false>(a, s);
    return a.block > 0 ? basis_impl<ElemBF16, true>(a, s) : basis_impl<ElemBF16, false>(a, s);
}

}  // namespace loki
