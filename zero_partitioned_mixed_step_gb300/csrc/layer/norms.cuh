// What the two passes over the norms around a block share.
#pragma once

#include "layer.cuh"

namespace zo {

struct Gate {
    const void *p;
    int32_t kind, type;
};

// A token's gate has no elements, and so may be NULL, where there are no rows.
inline bool bad_gate(const void *gate, int kind, int type, int64_t rows)
{
    return kind < ZERO_GATE_NONE || kind > ZERO_GATE_ROWS ||
           (kind != ZERO_GATE_NONE && ((!gate && (kind != ZERO_GATE_ROWS || rows > 0)) || !is_float(type)));
}

inline bool gate_aligned(const void *gate, int kind, int type)
{
    return kind == ZERO_GATE_NONE || aligned(gate, (uintptr_t)type_bytes(type));
}

// w_post times a channel's gate for the 8 columns from c on (1 where there is neither).
template <int W>
__device__ __forceinline__ void post_factors(const void *w_post, int w_type, const Gate &gate, int c, int n, float2 f[4])
{
    if (w_post)
        get_vector<W>(w_post, w_type, c, n, f);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = both(1.0f);
    if (gate.kind == ZERO_GATE_COLS) {
        float2 g[4];
        get_vector<W>(gate.p, gate.type, c, n, g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = mul2(f[i], g[i]);
    }
}

template <int N>
constexpr int kSumPlaces = N <= 2 ? 2 : N <= 4 ? 4 : 8;

// Sums of N values over the threads of a row: G = 16 or 32 lanes, or (0) the CTA's warps,
// at most 16.  The values are shared out between lanes as they are added, so that 6
// take 9 shuffles in a warp and 8 behind the barrier.  `slot`: 16 floats for each of
// kSumPlaces<N> values, zeros where there is no warp, not used again before the next call's
// barrier.
template <int G, int N>
__device__ __forceinline__ void shared_sums(float (&x)[N], float *slot)
{
    constexpr int P = kSumPlaces<N>, L = G ? G : 32;
    float y[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        y[i] = i < N ? x[i] : 0.0f;
    float s = sum_shared<P, L>(y);
    if (!G) {
        constexpr int kShare = 32 / P, kEach = 16 / kShare;  // lanes to a value, warps to a lane
        const int lane = threadIdx.x & 31;
        if (lane % kShare == 0)
            slot[lane / kShare * 16 + (threadIdx.x >> 5)] = s;
        __syncthreads();
        const float *from = slot + lane / kShare * 16 + lane % kShare * kEach;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            s += from[i];
#pragma unroll
        for (int bit = kShare / 2; bit; bit >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, bit);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = __shfl_sync(0xFFFFFFFFu, s, i * (L / P), L);
}

template <int WORDS>
__device__ __forceinline__ void load_shared(uint32_t (&w)[WORDS], uint32_t from)
{
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
    else
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from) : "memory");
}

// Words that the compiler takes for new ones: what was made of them before is made again, not
// held in registers over a barrier (the gradients of the norms, 8192x4096: 65 us, held 72).
template <int WORDS>
__device__ __forceinline__ void renew(uint32_t (&w)[WORDS])
{
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
        asm volatile("" : "+r"(w[i]));
}

}  // namespace zo
