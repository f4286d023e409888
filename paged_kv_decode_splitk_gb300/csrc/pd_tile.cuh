// pd_tile.cuh -- what the passes that multiply on the fifth-generation tensor cores
// share: bounded waits and arrivals of a warp, and a softmax thread's work on its
// row of a tile of scores.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "pd_device.cuh"
#include "pd_tcgen05.cuh"

namespace pd {
namespace tile {

// Bounded wait of a whole warp, which also ends when another warp of the CTA
// gave up.  The answer is the same on every lane (the warp goes on to aligned
// instructions together).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    bool ok = dev::mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = dev::global_timer_ns();
        while (!(ok = dev::mbar_try_wait(bar, parity))) {
            if (*gave_up) break;
            if (dev::global_timer_ns() - t0 > 2000000000ull) {
                *gave_up = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The same for one thread.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    if (dev::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = dev::global_timer_ns();
    while (!dev::mbar_try_wait(bar, parity)) {
        if (*gave_up) return false;
        if (dev::global_timer_ns() - t0 > 2000000000ull) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same once for a warp, behind what all its lanes did (32 arrivals at one
// barrier are served one by one).
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) arrive(bar);
}

template <bool KV8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return KV8 ? dev::pack_f16x2(lo, hi) : dev::pack_bf16x2(lo, hi);
}

// Sum of a tile's weights above which a row's reference is raised.
constexpr float kLift = 32768.f;

// Scores of the columns past the live ones become -infinity.
template <int BN>
__device__ __forceinline__ void mask_columns(uint32_t (&x)[BN], int nv) {
#pragma unroll
    for (int i = 0; i < BN; ++i)
        if (i >= nv) x[i] = 0xff800000u;
}

// The largest of a row's scores of a tile.
template <int BN>
__device__ __forceinline__ float largest_of(const uint32_t (&x)[BN]) {
    float m0 = __uint_as_float(x[0]), m1 = __uint_as_float(x[1]);
#pragma unroll
    for (int i = 2; i < BN; i += 2) {
        m0 = fmaxf(m0, __uint_as_float(x[i]));
        m1 = fmaxf(m1, __uint_as_float(x[i + 1]));
    }
    return fmaxf(m0, m1);
}

// The weights 2^(x scale - m) of a row's tile, rounded to pairs of BF16 (f16),
// and their sum before that (scale > 0, so that a masked score weighs 0).
template <int BN, bool KV8>
__device__ __forceinline__ float weigh(const uint32_t (&x)[BN], float scale, float m, uint32_t (&pk)[BN / 2]) {
    const float off = m == -__int_as_float(0x7f800000) ? 0.f : m;
    const uint64_t scale2 = tc::pack_f32x2(scale, scale), off2 = tc::pack_f32x2(-off, -off);
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < BN; i += 2) {
        float a, b;
        tc::unpack_f32x2(tc::fma_f32x2(tc::pack_f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, off2), a, b);
        a = dev::exp2_approx(a);
        b = dev::exp2_approx(b);
        sum[(i / 2) & 3] = tc::add_f32x2(sum[(i / 2) & 3], tc::pack_f32x2(a, b));
        pk[i / 2] = pack2<KV8>(a, b);
    }
    float a, b;
    tc::unpack_f32x2(tc::add_f32x2(tc::add_f32x2(sum[0], sum[1]), tc::add_f32x2(sum[2], sum[3])), a, b);
    return a + b;
}

// Raises the references of the rows that ask for it to `top` at least, by a
// whole number, and scales l and O, which were weighed against the old ones, by
// that power of two.
template <int DPAD>
__device__ __forceinline__ void raise_reference(uint32_t to, float top, bool over, float &m, float &l) {
    const float d = top - m;
    const float k = over && d > 0.f ? ceilf(d) : 0.f;
    const float f = k < 127.f ? __int_as_float((127 - static_cast<int>(k)) << 23) : 0.f;
    m += k;
    l *= f;
#pragma unroll 1
    for (int i = 0; i < DPAD; i += 32) {
        uint32_t x[32];
        tc::ld_32x32(to + i, x);
        tc::wait_ld(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
        tc::st_32x32(to + i, x);
    }
}

constexpr int kConverters = 64;  // threads that turn FP8 tiles into f16 ones

// One landed tile of BN rows of E4M3 codes into an f16 tile (128-byte swizzle), by
// kConverters threads; exact: every E4M3 value is an f16 value.  A quarter-warp
// takes two rows x 64 codes, the second row of the neighbouring 64 codes: its loads
// and its stores each cover the 32 banks once under the swizzle.
template <int DPAD, int BN>
struct Widen {
    static constexpr int CPR = DPAD / 16;                  // 16-code chunks of a row
    static constexpr int KB = CPR / 4;                     // 64-code blocks of a row
    static constexpr int ROWS = kConverters / 8 / KB * 2;  // rows all quarter-warps take at a time
    // a thread's rows share their place in the swizzle, or it flips by half a row
    // from one to the next
    static constexpr int FLIP = ROWS % 8 ? 64 : 0;
    static_assert(ROWS % 4 == 0 && BN % (2 * ROWS) == 0, "rows of a thread");
    int row0, from, to_lo, to_hi;
    __device__ __forceinline__ Widen(int warp, int lane) {
        const int me = warp * 4 + (lane >> 3), j8 = lane & 7;
        row0 = me / KB * 2 + (j8 >> 2);
        const int c = 4 * (KB > 1 ? (me % KB) ^ (j8 >> 2) : 0) + (j8 & 3);
        from = DPAD < 128 ? row0 * DPAD + c * 16 : (c / 8) * (BN * 128) + row0 * 128 + (((c & 7) ^ (row0 & 7)) << 4);
        const int to = (c / 4) * (BN * 128) + row0 * 128, u2 = (2 * c) & 7;
        to_lo = to + ((u2 ^ (row0 & 7)) << 4);
        to_hi = to + (((u2 + 1) ^ (row0 & 7)) << 4);
    }
    // some: rows outside [low, end) become zeros
    __device__ __forceinline__ void operator()(const uint8_t *src, uint8_t *dst, bool some, int low, int end) const {
        // (eight loads before the first store, which the compiler would
        // not move them over)
        constexpr int N = BN / ROWS, BATCH = N < 8 ? N : 8;
#pragma unroll 1
        for (int k0 = 0; k0 < N; k0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                v[k] = *reinterpret_cast<const uint4 *>(src + (k & 1 ? from ^ FLIP : from) + (k0 + k) * (ROWS * (DPAD < 128 ? DPAD : 128)));
            if (some) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = row0 + (k0 + k) * ROWS;
                    if (row >= end || row < low) v[k] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                uint4 lo, hi;
                dev::e4m3x4_to_f16x4(v[k].x, lo.x, lo.y);
                dev::e4m3x4_to_f16x4(v[k].y, lo.z, lo.w);
                dev::e4m3x4_to_f16x4(v[k].z, hi.x, hi.y);
                dev::e4m3x4_to_f16x4(v[k].w, hi.z, hi.w);
                *reinterpret_cast<uint4 *>(dst + (k & 1 ? to_lo ^ FLIP : to_lo) + (k0 + k) * (ROWS * 128)) = lo;
                *reinterpret_cast<uint4 *>(dst + (k & 1 ? to_hi ^ FLIP : to_hi) + (k0 + k) * (ROWS * 128)) = hi;
            }
        }
    }
};

}  // namespace tile
}  // namespace pd
