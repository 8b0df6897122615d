// Device helpers of the attention kernels of kva.h: exponentials, the fp16
// side of an E4M3 cache, bounded waits between the warps of a CTA.
#pragma once

#include "kva_common.cuh"

namespace kvw {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Weights are 2^(s - m) with a reference m that follows the row's maximum only
// when a weight would pass 2^(kSlack + lift): any m will do that keeps the
// weights in range, and the sums are rescaled seldom.  fp16 weights (an E4M3
// cache) lie a further 2^9 higher, the largest between 2^9 and 2^15: fp16 has
// nothing below 2^-25, and at 2^0 that dropped whatever was 2^-25 of the
// largest, while the sum of the weights, in fp32, counted it (one position 18
// above 8191 others: 29 % of what they hold).  Up there each weight is off by
// 2^-11 of itself or 2^-34 of the largest.
constexpr float kSlack = 6.0f;
template <bool F16>
constexpr float weight_lift() {
    return F16 ? 9.0f : 0.0f;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four E4M3 codes -> two f16x2 (low bytes first), exact.
__device__ __forceinline__ void codes_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(lo, hi);
    }
}

// Power of two that brings a row whose largest |value| has the bf16 pattern
// `top` to [2^14, 2^15), and its inverse, as exponents of fp32; both 127 (1.0)
// for a row of zeros or one that holds an infinity or a NaN.  fp16 then holds
// the row's bf16 values exactly down to 2^-31 of the largest.  Rows below
// 2^-112 stop at 2^126, whose inverse is the smallest normal number: they stay
// below 2^14, every bf16 value of theirs exact all the same.
__host__ __device__ __forceinline__ void row_exponents(uint32_t top, uint32_t& up,
                                                       uint32_t& down) {
    const uint32_t e = top >> 7;
    up = top == 0 || e == 255 ? 127u : e < 15 ? 253u : 268u - e;
    down = 254u - up;
}

__device__ __forceinline__ void row_power(uint32_t top, float& up, float& down) {
    uint32_t u, d;
    row_exponents(top, u, d);
    up = __uint_as_float(u << 23);
    down = __uint_as_float(d << 23);
}

// One thread of a converged warp, known to the compiler as one: what it
// issues needs no loop over lanes (an MMA or a copy takes 120 cycles to issue
// without it).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// Bounded wait of a whole warp that ends early when another role gave up;
// the answer is the same for all lanes.  The limit is in cycles of the SM's
// clock, which is read in a few of them; the global timer takes about a
// microsecond, as long as most of these waits.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t* stop,
                                           int64_t limit_cycles) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const int64_t t0 = clock64();
        while (!(ok = mbar_try_wait(bar, parity))) {
            if (*reinterpret_cast<volatile uint32_t*>(stop)) break;
            if (clock64() - t0 > limit_cycles) {
                *reinterpret_cast<volatile uint32_t*>(stop) = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The same without early end, for what has to land before a CTA may go.
__device__ __forceinline__ void drain_phase(uint64_t* bar, uint32_t parity, int64_t limit_cycles) {
    const int64_t t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > limit_cycles) return;
}

// Has the phase of parity `parity` completed?  (Does not wait.)
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// What a kernel of a test build does on purpose: announce its first copies but
// never issue them, or leave its tiles to nobody (the consumers go at once).
enum class Hook { kNone, kWithheld, kAbandoned };

// The last phase of a place that copies land in, before its CTA may go: copies
// that nobody waits for (a consumer that gave up) would land in the shared
// memory of another CTA.  The test build counts those still under way after it.
template <Hook HOOK>
__device__ __forceinline__ void leave_phase(uint64_t* bar, uint32_t parity, int64_t limit_cycles,
                                            uint32_t* err_flags) {
    drain_phase(bar, parity, limit_cycles);
    if constexpr (HOOK == Hook::kAbandoned)
        if ((threadIdx.x & 31u) == 0 && !phase_done(bar, parity)) atomicAdd(err_flags + 1, 1u);
}

// Cycles of a limit in nanoseconds (the clock runs at 2.07 GHz at most).
inline int64_t wait_cycles(uint64_t ns) { return (int64_t)(ns * 2); }

// The same for one thread.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, uint32_t* stop,
                                         int64_t limit_cycles) {
    if (mbar_try_wait(bar, parity)) return true;
    const int64_t t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile uint32_t*>(stop)) return false;
        if (clock64() - t0 > limit_cycles) {
            *reinterpret_cast<volatile uint32_t*>(stop) = 1;
            return false;
        }
    }
    return true;
}

// Four floats of a workspace slot.  Volatile, so that a batch of them is in
// flight before the first is used: the compiler else takes them one by one.
__device__ __forceinline__ float4 load_part(const float* p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p));
    return v;
}

// A ring position: slot and the parity of its present round.
template <int N>
struct RingPos {
    uint32_t slot = 0, parity = 0;
    __device__ __forceinline__ void step() {
        if (++slot == (uint32_t)N) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

}  // namespace kvw
