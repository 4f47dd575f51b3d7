// Work of a ragged batch laid end to end: sequence b has n(b) items, and a
// warp finds the total or the sequence that holds an item from the lengths on
// the device. Every lane of the warp takes part and gets the result.
#pragma once

#include <stdint.h>

namespace loki {

// items of the sequences before b (*before), and of all
template <class N>
__device__ __forceinline__ int64_t seqs_total(int B, N n, int b = 0, int64_t* before = nullptr) {
    int64_t x = 0, y = 0;
    for (int i = threadIdx.x & 31; i < B; i += 32) {
        const int64_t v = n(i);
        y += v;
        if (i < b) x += v;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        if (before != nullptr) x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    if (before != nullptr) *before = x;
    return y;
}

// the sequence that holds item x (each counting `copies` times its items), and
// the items before it; -1 behind the last
template <class N>
__device__ __forceinline__ int seqs_find(int B, int64_t x, int copies, N n, int64_t* before) {
    const int lane = threadIdx.x & 31;
    int64_t carry = 0;
    for (int base = 0; base < B; base += 32) {
        const int64_t own = base + lane < B ? n(base + lane) : 0;
        int64_t v = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += o;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, x < copies * (carry + v));
        if (hit != 0) {
            const int at = __ffs(hit) - 1;
            *before = carry + __shfl_sync(0xffffffffu, v - own, at);
            return base + at;
        }
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    *before = 0;
    return -1;
}

// a / b, b > 0: most lines of work are short enough for the 32-bit division
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

}  // namespace loki
