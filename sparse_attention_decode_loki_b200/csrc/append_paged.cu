// Appends to a paged KV-cache with the rotary position embedding on the way
// (append_paged.cuh has the formulas): values, queries and keys without a
// basis as streams; keys of a few tokens against the basis row by row. Longer
// appends rotate their keys in append_basis.cu.
#include "append_paged.cuh"

namespace loki {

// ---------------------------------------------------------------------------
// Longer appends as streams, one read and one write of each row. Bytes bound
// them, and what the loads in flight cost is registers: values and queries
// share a kernel of 64 registers, 32 warps an SM; keys without a basis, which
// are turned and then scaled, have one of their own, a CTA to an SM, which runs
// beside it.
//
// Values and keys: a CTA has an aligned run of 128 positions and goes through
// some heads, a warp has 16 of the positions, eight lanes to a row (16 columns
// each); the next head's rows are loaded before this one's are stored. 8-bit
// scale blocks of more than 16 tokens belong to neighbouring warps, which share
// their largest magnitude through shared memory, so every scale has one owner.
// Queries: a warp has four positions, whose angles stay in its registers while
// it goes through the heads; their rows lie together, 1 KB of bf16 a head, which
// a ring of bulk copies per warp brings.
//
// Measured on two prompts of 8192 and 6144 tokens, 32 query and 8 KV heads, into
// 8 bits, values, queries (279 MB) and keys side by side: 62 us (5.3 TB/s). A
// ring of 3 heads 65, of 4 66; bulk stores as well 64; query loads into
// registers (2 heads ahead) 76, 3 or 4 ahead 84 to 86; rows of all heads in one
// 16-row warp item with the angles in shared memory 103.

constexpr int kStThreads = 256, kStQueryRows = 32, kStQueryStages = 2;

// a warp's 16 positions of a run and their place in the pool but for the head's
// offset (the page is the same for all heads)
template <bool kQ8>
struct RunPlace {
    int64_t j0, block_start;
    int row[kQ8 ? 1 : 4];  // 8 bits: of the scale block's first token; -1: none
    uint32_t live;         // bit i: position j0 + 4 i + lane / 8 is appended and has a place
    bool has_old;          // the block holds older tokens
    __device__ __forceinline__ RunPlace(const AppendArgs& a, const ApSeq& s, int b, int64_t start, bool lane_on) {
        const int sub = threadIdx.x >> 3 & 3;
        j0 = start + 16 * (threadIdx.x >> 5);
        block_start = kQ8 ? j0 & ~(int64_t)(a.block - 1) : 0;
        has_old = kQ8 && s.lo > block_start;
        live = 0;
        if constexpr (kQ8) {  // one page holds the whole block
            row[0] = block_start < s.hi && block_start + a.block > s.lo ? pool_row(a, b, 0, (int)block_start) : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = j0 + 4 * i + sub;
            const bool in = j >= s.lo && j < s.hi;
            if constexpr (!kQ8) row[i] = in ? pool_row(a, b, 0, (int)j) : -1;
            if (lane_on && in && row[kQ8 ? 0 : i] >= 0) live |= 1u << i;
        }
    }
    // pool row of position j0 + 4 i + lane / 8 under a head's offset
    __device__ __forceinline__ int64_t at(int i, int shift) const {
        return kQ8 ? row[0] + shift + (int)(j0 - block_start) + 4 * i + (int)(threadIdx.x >> 3 & 3)
                   : row[kQ8 ? 0 : i] + shift;
    }
};

// The block's new scale from this warp's largest magnitude: shared with the
// block's other warps through red (two sets in turn), stored by the first.
// Every warp of the CTA calls it; old is the scale before.
__device__ __forceinline__ float block_scale(const AppendArgs& a, float amax, float* red, float* scale, bool has_old,
                                             float* old) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gw = a.block >> 4;
    *old = scale != nullptr && has_old ? *scale : 0.f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (gw > 1) {
        if (lane == 0) red[warp] = amax;
        __syncthreads();  // and every warp has read the old scale
        for (int w = warp & ~(gw - 1); w < (warp & ~(gw - 1)) + gw; ++w) amax = fmaxf(amax, red[w]);
    } else {
        __syncwarp();
    }
    const float grown = pow2_scale(amax), s = has_old ? fmaxf(*old, grown) : grown;
    if (scale != nullptr && (warp & (gw - 1)) == 0 && lane == 0) *scale = s;
    return s;
}

// the older codes of a warp's positions, moved from scale `old` to s
__device__ __forceinline__ void rescale_rows(const AppendArgs& a, uint8_t* codes, int64_t j0, int64_t lo, float f) {
    const int u = threadIdx.x & 7, sub = threadIdx.x >> 3 & 3;
    if (u >= a.D >> 4) return;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        if (j0 + 4 * i + sub >= lo) continue;
        uint4* w = reinterpret_cast<uint4*>(codes + (4 * i + sub) * a.D + 16 * u);
        uint4 v = *w;
        v.x = rescale4(v.x, f);
        v.y = rescale4(v.y, f);
        v.z = rescale4(v.z, f);
        v.w = rescale4(v.w, f);
        *w = v;
    }
}

template <class E, bool kQ8>
__global__ void __launch_bounds__(kStThreads, E::kBytes == 2 ? 4 : 2) k_append_stream(const AppendArgs a) {
    using Tp = typename E::T;
    __shared__ float red[2][kStThreads / 32];
    extern __shared__ __align__(16) uint8_t ring[];  // the queries', per warp
    __shared__ __align__(8) uint64_t full[kStThreads / 32][kStQueryStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane & 7, sub = lane >> 3;
    const bool lane_on = u < a.D >> 4;
    // A programmatic dependent of the keys' kernel, which writes nothing that is read or written here.
    // What is read here came before that kernel, and every CTA of it has waited for that work (griddep_wait)
    // before it releases its dependents: it is complete, and no line of it is older, when this grid starts.
    // (A wait of its own would wait for the keys as well. Fences on both sides: 42.0 us instead of 39.3 for
    // four ragged prompts up to 2048 tokens of 32 query and 8 KV heads; every read from the L2: 41.0.)
    if ((int)blockIdx.x >= a.kv_ctas) {
        // CTAs side by side take rows side by side
        const int q = blockIdx.x - a.kv_ctas, blocks = (a.T + kStQueryRows - 1) / kStQueryRows, b = q / blocks % a.B;
        const int t = q % blocks * kStQueryRows + 4 * warp + sub, chunk = q / blocks / a.B;
        const int h0 = chunk * a.q_group, h1 = min(h0 + a.q_group, a.H_q);
        int ca, cb;
        const bool turn = a.rope != nullptr && u < a.rot_dim >> 4;
        unit_cols(turn ? a.rot_dim : 0, a.interleaved, u, &ca, &cb);
        const int64_t step = (int64_t)a.T * a.D, at = (((int64_t)b * a.H_q + h0) * a.T + t) * a.D;
        const Tp* p = static_cast<const Tp*>(a.q) + at;
        Tp* o = static_cast<Tp*>(a.q_out) + at;
        // The warp's rows r0 .. r1 - 1 of its four are appended. They lie together: a bulk copy a head, S
        // heads on their way.
        constexpr int S = kStQueryStages, kSlot = 4 * 128 * E::kBytes;
        uint8_t* const slots = ring + warp * S * kSlot;
        const int t0 = t - sub;
        const int64_t j0 = (int64_t)__ldg(a.positions + b) + t0;
        const int n = a.new_lens != nullptr ? min(__ldg(a.new_lens + b), a.T) : a.T;
        const int r0 = (int)min64(j0 < 0 ? -j0 : 0, 4);
        const int64_t end = min64(min64(4, (int64_t)n - t0), a.rope != nullptr ? a.n_pos - j0 : 4);
        const int r1 = end > r0 ? (int)end : r0, row = a.D * E::kBytes;
        const uint32_t bytes = (r1 - r0) * row;
        if (bytes > 0) {
            if (lane == 0) {
                for (int i = 0; i < S; ++i) mbar_init(&full[warp][i], 1);
                fence_mbar_init();
                fence_proxy_async_global();
            }
            __syncwarp();
            const Tp* src = p + (r0 - sub) * (int64_t)a.D;
            auto issue = [&](int h, int i) {
                mbar_arrive_expect_tx(&full[warp][i], bytes);
                bulk_load(slots + i * kSlot + r0 * row, src + (h - h0) * step, bytes, &full[warp][i]);
            };
            if (lane == 0)
                for (int i = 0; i < S && h0 + i < h1; ++i) issue(h0 + i, i);
            const bool mine = lane_on && sub >= r0 && sub < r1;
            Angles g;
            if (turn && mine) g.load(a.rope + (j0 + sub) * a.rot_dim, a.rot_dim, u);
            int i = 0, h = h0;
            uint32_t phase = 0;
            for (; h < h1; ++h) {
                if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][i], phase, a.err))) break;
                float x[16];
                if (mine) {
                    const uint8_t* in = slots + i * kSlot + sub * row;
#pragma unroll
                    for (int e = 0; e < Chunk<E>::kN; ++e) {
                        E::unpack(reinterpret_cast<const uint4*>(in + ca * E::kBytes)[e], x + e * E::kVec);
                        E::unpack(reinterpret_cast<const uint4*>(in + cb * E::kBytes)[e], x + 8 + e * E::kVec);
                    }
                }
                fence_proxy_async_shared();  // the rows are read before the next head's arrive
                __syncwarp();
                if (lane == 0 && h + S < h1) issue(h + S, i);
                if (mine) {
                    if (turn) g.turn(x, a.interleaved);
                    store_chunk<E>(o + ca, x, ca, a.D);
                    store_chunk<E>(o + cb, x + 8, cb, a.D);
                }
                o += step;
                if (++i == S) i = 0, phase ^= 1;
            }
            // behind a wait that gave up: the copies on their way land (or not) before the CTA may end
            for (int l = h; l < min(h + S, h1); ++l) {
                mbar_wait(&full[warp][i], phase, a.err);
                if (++i == S) i = 0, phase ^= 1;
            }
        }
    } else {
        const int chunk = blockIdx.x % a.chunks, rest = blockIdx.x / a.chunks, b = rest % a.B;
        const ApSeq sq = append_seq(a, b, chunk == 0 && rest < a.B && threadIdx.x == 0);
        const int64_t start = (sq.lo / kRunRows + rest / a.B) * kRunRows;
        if (start < sq.hi) {  // uniform over the CTA
            const RunPlace<kQ8> pl(a, sq, b, start, lane_on);
            const int h0 = chunk * a.group, h1 = min(h0 + a.group, a.H_kv);
            const int64_t step = (int64_t)a.T * a.D;
            const Tp* p = static_cast<const Tp*>(a.V_new) + ((int64_t)b * a.H_kv + h0) * step +
                          (pl.j0 - sq.p0 + sub) * a.D + 16 * u;
            int parity = 0;
            Chunk<E> w[4][2];
            auto load = [&]() {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pl.live >> i & 1u) {
                        w[i][0].load(p + 4 * i * a.D);
                        w[i][1].load(p + 4 * i * a.D + 8);
                    }
                p += step;
            };
            load();
            for (int h = h0; h < h1; ++h) {
                const int shift = h * a.page_size;
                if constexpr (!kQ8) {  // in their own type: copied, bit by bit
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pl.live >> i & 1u) {
                            uint4* o = reinterpret_cast<uint4*>(static_cast<Tp*>(a.V_pages) + pl.at(i, shift) * a.D + 16 * u);
#pragma unroll
                            for (int e = 0; e < Chunk<E>::kN; ++e) {
                                o[e] = w[i][0].w[e];
                                o[Chunk<E>::kN + e] = w[i][1].w[e];
                            }
                        }
                    if (h + 1 < h1) load();
                } else {
                    float amax = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pl.live >> i & 1u) {
                            float x[16];
                            w[i][0].get(x);
                            w[i][1].get(x + 8);
                            amax = finite_amax<16>(amax, x);
                        }
                    float old;
                    float* sc = pl.row[0] < 0 ? nullptr : a.v_scales + ((pl.row[0] + shift) >> a.block_log2);
                    const float s = block_scale(a, amax, red[parity], sc, pl.has_old, &old), inv = 1.f / s;
                    parity ^= 1;
                    uint8_t* o = static_cast<uint8_t*>(a.V_pages) + (pl.at(0, shift) - sub) * a.D;
                    uint4 y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x[16];
                        w[i][0].get(x);
                        w[i][1].get(x + 8);
                        const uint2 ya = codes8(x, inv), yb = codes8(x + 8, inv);
                        y[i] = make_uint4(ya.x, ya.y, yb.x, yb.y);
                    }
                    if (h + 1 < h1) load();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pl.live >> i & 1u) *reinterpret_cast<uint4*>(o + (4 * i + sub) * a.D + 16 * u) = y[i];
                    if (sc != nullptr && pl.has_old && s > old) rescale_rows(a, o, pl.j0, sq.lo, old / s);
                }
            }
        }
    }
    // The grid must end after the keys' kernel, for those who wait for this one: one CTA waits (the
    // others would hold their places on the SMs).
    if (blockIdx.x == gridDim.x - 1) griddep_wait();
}

template <class E, bool kQ8>
__global__ void __launch_bounds__(kStThreads, E::kBytes == 2 ? 2 : 1) k_append_keys(const AppendArgs a) {
    using Tp = typename E::T;
    extern __shared__ __align__(16) float angles[];  // the run's, [128][rot_dim]
    __shared__ float red[2][kStThreads / 32];
    __shared__ __align__(8) uint64_t bar;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane & 7, sub = lane >> 3;
    const bool lane_on = u < a.D >> 4;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    griddep_wait();  // launched early: inputs and pages may still be in use
    fence_proxy_async_global();  // the angles come by bulk copies
    griddep_launch_dependents();
    const int rot = a.rope != nullptr ? a.rot_dim : 0;
    const bool turn = u < rot >> 4;
    int ca, cb;
    unit_cols(turn ? rot : 0, a.interleaved, u, &ca, &cb);
    auto runs_of = [&](int b) -> int64_t {
        const ApSeq s = append_seq(a, b, false);
        return run_count(s.lo, s.hi);
    };
    const int64_t total = seqs_total(a.B, runs_of) * a.H_kv, per = quot(total + gridDim.x - 1, gridDim.x);
    int64_t w = min64(blockIdx.x * per, total);
    const int64_t w_end = min64(w + per, total), step = (int64_t)a.T * a.D;
    int parity = 0;
    uint32_t phase = 0;
    while (w < w_end) {  // run by run, heads fastest
        const int64_t ri = quot(w, a.H_kv);
        int64_t before;
        const int b = seqs_find(a.B, ri, 1, runs_of, &before);
        const int h0 = (int)(w - ri * a.H_kv), h1 = (int)min64(a.H_kv, h0 + (w_end - w));
        w += h1 - h0;
        const ApSeq sq = append_seq(a, b, false);
        const int64_t start = (sq.lo / kRunRows + (ri - before)) * kRunRows;
        fence_proxy_async_shared();
        __syncthreads();  // the run before is done with its angles (and the barrier is set up)
        if (rot > 0 && threadIdx.x == 0) {
            const uint32_t bytes = (uint32_t)min64(sq.hi - start, kRunRows) * rot * 4;
            mbar_arrive_expect_tx(&bar, bytes);
            bulk_load(angles, a.rope + start * rot, bytes, &bar);
        }
        const RunPlace<kQ8> pl(a, sq, b, start, lane_on);
        const Tp* p = static_cast<const Tp*>(a.K_new) + ((int64_t)b * a.H_kv + h0) * step + (pl.j0 - sq.p0 + sub) * a.D;
        Chunk<E> wa[4], wb[4];
        auto load = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (pl.live >> i & 1u) {
                    wa[i].load(p + 4 * i * a.D + ca);
                    wb[i].load(p + 4 * i * a.D + cb);
                }
            p += step;
        };
        load();
        if (rot > 0) {
            const bool ok = mbar_wait(&bar, phase, a.err);
            phase ^= 1;
            if (__syncthreads_or(!ok)) {  // flagged: the copy lands (or not) before the CTA ends
                mbar_wait(&bar, phase ^ 1, a.err);
                return;
            }
        }
        for (int h = h0; h < h1; ++h) {
            const int shift = h * a.page_size;
            float x[4][16], amax = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wa[i].get(x[i]);
                wb[i].get(x[i] + 8);
                if (turn) turn_unit_from(angles + (16 * warp + 4 * i + sub) * rot, rot, a.interleaved, u, x[i]);
                if (!(pl.live >> i & 1u)) continue;
                if (a.plane != nullptr) {
                    Tp* o = static_cast<Tp*>(a.plane) + pl.at(i, shift) * a.d_lo;
                    store_chunk<E>(o + ca, x[i], ca, a.d_lo);
                    store_chunk<E>(o + cb, x[i] + 8, cb, a.d_lo);
                }
                if constexpr (!kQ8) {
                    Tp* o = static_cast<Tp*>(a.K_pages) + pl.at(i, shift) * a.D;
                    store_chunk<E>(o + ca, x[i], ca, a.D);
                    store_chunk<E>(o + cb, x[i] + 8, cb, a.D);
                } else {
                    amax = finite_amax<16>(amax, x[i]);
                }
            }
            if (h + 1 < h1) load();
            if constexpr (kQ8) {
                float old;
                float* sc = pl.row[0] < 0 ? nullptr : a.k_scales + ((pl.row[0] + shift) >> a.block_log2);
                const float s = block_scale(a, amax, red[parity], sc, pl.has_old, &old), inv = 1.f / s;
                parity ^= 1;
                uint8_t* o = static_cast<uint8_t*>(a.K_pages) + (pl.at(0, shift) - sub) * a.D;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pl.live >> i & 1u) {
                        *reinterpret_cast<uint2*>(o + (4 * i + sub) * a.D + ca) = codes8(x[i], inv);
                        *reinterpret_cast<uint2*>(o + (4 * i + sub) * a.D + cb) = codes8(x[i] + 8, inv);
                    }
                if (sc != nullptr && pl.has_old && s > old) rescale_rows(a, o, pl.j0, sq.lo, old / s);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens (a decode step), with or without a basis. Latency bounds it: one
// CTA per KV head and group of sequences, at most 16 rows. A quarter of a
// basis column sits in each thread's registers, loaded before anything else;
// a warp per row turns it, quantises it and stores it. 16 sequences of 40 heads:
// 4.2 us (8 bits 4.9), call after call. Before the launch was hidden behind the
// preceding call: 4.4 (5.2), in two waves of CTAs 8.0 (9.3), in two CTAs an SM of
// 64 registers 6.2 (7.1).

constexpr int kRwThreads = 512, kRwRows = kRwThreads / 32;  // a row to a warp

template <class E, bool kQ8, int D, bool kBasis>
__global__ void __launch_bounds__(kRwThreads) k_append_rows(const AppendArgs a) {
    using Tp = typename E::T;
    constexpr int DQ = D / 4;
    __shared__ __align__(16) float xs[kRwRows][128];
    __shared__ __align__(16) float part[4][8][128];
    __shared__ float top[2][kRwRows];
    __shared__ int blk[kRwRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();  // launched early: inputs and pages may still be in use
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
    if (kBasis && c < D) {
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
        // the row's loads need no position: on their way before it is read
        const int64_t at = (((int64_t)b * a.H_kv + hk) * a.T + t) * D;
        const bool unit_on = lane < D >> 4, turn = unit_on && a.rope != nullptr && lane < a.rot_dim >> 4;
        int ca, cb;
        unit_cols(turn ? a.rot_dim : 0, a.interleaved, lane, &ca, &cb);
        Chunk<E> wa, wb;
        if (unit_on) {
            wa.load(static_cast<const Tp*>(a.K_new) + at + ca);
            wb.load(static_cast<const Tp*>(a.K_new) + at + cb);
        }
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
        const ApSeq sq = append_seq(a, b, t == 0 && lane == 0 && hk == 0);
        j = sq.p0 + t;
        first = sq.lo;
        live = j >= sq.lo && j < sq.hi;
        if (live) {
            row = pool_row(a, b, hk, (int)j);
            if (unit_on) {
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
    for (int r0 = 0; kBasis && r0 < rows; r0 += 8) {
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

template <class E, bool kQ8, int D>
static cudaError_t rows_impl(const AppendArgs& a, int64_t ctas, cudaStream_t s) {
    return launch_kernel(a.P != nullptr ? k_append_rows<E, kQ8, D, true> : k_append_rows<E, kQ8, D, false>,
                         dim3((unsigned)ctas), dim3(kRwThreads), 0, s, true, a);
}

template <class E, bool kQ8>
static cudaError_t append_impl(AppendArgs a, cudaStream_t s) {
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    if (a.T <= kRwRows) {
        // sequences of a CTA: the fewest with which the CTAs are resident together (one to an SM)
        const int64_t q = a.q != nullptr ? ((int64_t)a.B * a.H_q * a.T * 8 + kRwThreads - 1) / kRwThreads : 0;
        int64_t group = 1, kv = (int64_t)a.B * a.H_kv;
        while (kv + q > di.sm_count && group < a.B && (group + 1) * a.T <= kRwRows)
            kv = (a.B + group) / (group + 1) * a.H_kv, ++group;
        a.group = (int)group;
        if (kv + q > 0x7fffffff) return cudaErrorInvalidValue;
        a.kv_ctas = (int)kv;
        return a.D == 96 ? rows_impl<E, kQ8, 96>(a, kv + q, s) : rows_impl<E, kQ8, 128>(a, kv + q, s);
    }
    // keys first; values and queries run beside them as a programmatic dependent
    const int64_t runs = (((int64_t)a.T + kRunRows - 2) / kRunRows + 1) * a.B;
    // heads of a CTA: as many as still leave `waves` CTAs for every place on the device
    auto heads_per_cta = [&](int64_t ctas, int heads, int per_sm, int waves) {
        const int64_t g = ctas * heads / ((int64_t)di.sm_count * per_sm * waves);
        return (int)(g < 1 ? 1 : min64(g, heads));
    };
    if (a.P != nullptr) {
        e = launch_append_basis(E::kBytes == 4 ? kF32 : kBF16, a, s);
    } else {
        // one CTA to an SM, which leaves half of its registers to the stream
        auto kern = k_append_keys<E, kQ8>;
        e = allow_dynamic_smem((const void*)kern, kRunRows * 128 * 4);
        if (e != cudaSuccess) return e;
        const size_t smem = a.rope != nullptr ? (size_t)kRunRows * a.rot_dim * sizeof(float) : 0;
        e = launch_kernel(kern, dim3((unsigned)min64(runs * a.H_kv, di.sm_count)), dim3(kStThreads), smem, s, true, a);
    }
    if (e != cudaSuccess) return e;
    const int per_sm = E::kBytes == 2 ? 4 : 2;
    a.group = heads_per_cta(runs, a.H_kv, per_sm, 3);
    a.chunks = (a.H_kv + a.group - 1) / a.group;
    int64_t q_ctas = 0;
    if (a.q != nullptr) {
        const int64_t rows = ((int64_t)a.T + kStQueryRows - 1) / kStQueryRows * a.B;
        a.q_group = heads_per_cta(rows, a.H_q, per_sm, 3);
        a.q_group = (a.q_group + 3) & ~3;
        a.q_chunks = (a.H_q + a.q_group - 1) / a.q_group;
        q_ctas = rows * a.q_chunks;
    }
    if (runs * a.chunks + q_ctas > 0x7fffffff) return cudaErrorInvalidValue;
    a.kv_ctas = (int)(runs * a.chunks);
    auto kern = k_append_stream<E, kQ8>;
    const size_t ring = a.q != nullptr ? (size_t)kStQueryRows * kStQueryStages * 128 * E::kBytes : 0;
    e = allow_dynamic_smem((const void*)kern, ring);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3((unsigned)(a.kv_ctas + q_ctas)), dim3(kStThreads), ring, s, true, a);
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
