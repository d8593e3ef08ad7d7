// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (2011), and the keep decisions
// of dropout drawn from it.
//
// Element i of a tensor takes 16-bit value i % 8 (low half of word 0 first) of
// the block at counter (i / 8, offset) under the key `seed`: one evaluation
// serves the eight elements that a thread loads at once, and a mask is a
// function of (i, seed, offset) alone, so the backward pass draws it again
// instead of reading it.  Sixteen bits per element halve the evaluations that
// 32 would need; the drop probability is rounded to a multiple of 2^-16.
#pragma once

#include <stdint.h>

namespace ct {

struct RngArgs {
    uint64_t seed, offset;
    const uint64_t *dev;   // when set: {seed, offset} read on the device instead
    uint32_t threshold;    // dropped where the 16-bit value is below it
    float scale;           // 65536 / (65536 - threshold); 0 when all is dropped
    uint32_t keys[20];     // the ten rounds' keys of `seed`
};

inline void set_keys(RngArgs &a) {
    for (uint32_t r = 0; r < 10; ++r) {
        a.keys[2 * r] = (uint32_t)a.seed + r * 0x9E3779B9u;
        a.keys[2 * r + 1] = (uint32_t)(a.seed >> 32) + r * 0xBB67AE85u;
    }
}

#ifdef __CUDACC__

// FIXED: the round keys come from the launch's arguments, as operands of the
// rounds themselves; else they are made on the way (20 additions, of about 150
// instructions for eight elements of dropout) from a seed that may lie on the
// device.
template <bool FIXED>
struct Philox {
    const RngArgs &a;
    uint32_t k0, k1, c2, c3;

    __device__ __forceinline__ explicit Philox(const RngArgs &args) : a(args) {
        const uint64_t s = !FIXED && a.dev ? a.dev[0] : a.seed, o = !FIXED && a.dev ? a.dev[1] : a.offset;
        k0 = (uint32_t)s;
        k1 = (uint32_t)(s >> 32);
        c2 = (uint32_t)o;
        c3 = (uint32_t)(o >> 32);
    }

    __device__ __forceinline__ uint4 operator()(uint64_t block) const {
        uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = c2, x3 = c3;
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
            x0 = (uint32_t)(p1 >> 32) ^ x1 ^ (FIXED ? a.keys[2 * r] : k0 + r * 0x9E3779B9u);
            x1 = (uint32_t)p1;
            x2 = (uint32_t)(p0 >> 32) ^ x3 ^ (FIXED ? a.keys[2 * r + 1] : k1 + r * 0xBB67AE85u);
            x3 = (uint32_t)p0;
        }
        return make_uint4(x0, x1, x2, x3);
    }
};

// Dropout of pair j (elements 2j and 2j + 1) of a block.  A 16-bit value h is
// at least t where h << 16, whatever lies below it, is above (t << 16) - 1;
// t = 2^16 keeps nothing.  The launch has t >= 1.
__device__ __forceinline__ float2 drop_pair(uint32_t word, uint32_t limit, float scale, float2 v) {
    v = __fmul2_rn(v, make_float2(scale, scale));
    return make_float2((word << 16) > limit ? v.x : 0.f, word > limit ? v.y : 0.f);
}
__device__ __forceinline__ uint32_t drop_limit(uint32_t threshold) { return (threshold << 16) - 1u; }

// The words for the pairs of a vector of P pairs at element e (a multiple of
// 2 P): a whole block of the generator, or one half of it.
template <bool FIXED, int P>
__device__ __forceinline__ void draw(const Philox<FIXED> &philox, uint64_t e, uint32_t (&w)[P]) {
    const uint4 r = philox(e >> 3);
    if constexpr (P == 4) {
        w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else {
        const bool high = (e >> 2) & 1;
        w[0] = high ? r.z : r.x;
        w[1] = high ? r.w : r.y;
    }
}

#endif

}  // namespace ct
