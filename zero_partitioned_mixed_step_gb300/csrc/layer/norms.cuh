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
template <bool W>
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

}  // namespace zo
