// slot_exchange.cuh -- how the warps of a row slot meet: their sums, and
// whether one of them gives up.  Included by gbn_device.cuh, after warp_sum(),
// warp_sum2() and named_barrier(); tests/slot_exchange.cpp compiles it with
// those of a CPU, a thread to a warp.
#pragma once

#include <stdint.h>

namespace gbn {

// Floats of reduction scratch per slot: 128, as [buffer][NQ][16 warps].
constexpr int kRedStride = 16;

// The slot's barrier.  Behind it slot_stops() says, uniformly over the slot,
// whether any of its threads came with give_up = true (a wait that ran out).
// `flag` is the slot's, zero at first; `round` is the meeting's own number, from
// 1 on and rising.  The flag holds the round in which a warp gave up: a warp that
// is through one round's barrier may give up in the next before a slower warp
// has read the flag, which then finds another round's number there and comes to
// that round's barrier as well.  Nothing writes over a number before all have
// read it: whoever is through that round's barrier stops there.  (With a mere 1 in the flag
// the slower warp left a row early, and the others waited at a barrier that
// never filled.)
__device__ __forceinline__ void slot_meet(volatile int *flag, int round, bool give_up, int bar_id, int tpr) {
    if (give_up) *flag = round;
    named_barrier(bar_id, tpr);
}
__device__ __forceinline__ bool slot_stops(const volatile int *flag, int round) { return *flag == round; }

// Sums the NQ values of every thread of one row slot (W warps, tpr = 32*W
// threads, named barrier bar_id) and leaves the totals in v on every thread
// of the slot: a butterfly within each warp, then the W warp sums added in
// warp order (read as 16-byte vectors).  `buf` is this slot's scratch of
// NQ*kRedStride floats; consecutive calls must alternate buffers.  Returns
// slot_stops(), with slot_meet()'s flag and round.
template <int NQ>
__device__ __forceinline__ bool slot_reduce(float (&v)[NQ], float *buf, volatile int *flag, int round,
                                            bool give_up, int W, int warp, int lane, int bar_id, int tpr) {
    if constexpr (NQ == 2) {
        warp_sum2(v[0], v[1]);
    } else {
#pragma unroll
        for (int q = 0; q < NQ; ++q) v[q] = warp_sum(v[q]);
    }
    if (W == 1) return __any_sync(0xffffffffu, give_up) != 0;
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) buf[q * kRedStride + warp] = v[q];
    }
    slot_meet(flag, round, give_up, bar_id, tpr);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const float *b = buf + q * kRedStride;
        if (W == 2) {
            const float2 t = *reinterpret_cast<const float2 *>(b);
            v[q] = t.x + t.y;
        } else {
            float s = 0.f;
            for (int w = 0; w < W; w += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(b + w);
                s = w == 0 ? t.x : s + t.x;
                s += t.y;
                s += t.z;
                s += t.w;
            }
            v[q] = s;
        }
    }
    return slot_stops(flag, round);
}

}  // namespace gbn
