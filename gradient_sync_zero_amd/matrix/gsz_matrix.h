// What the matrix products take from gfx950 beyond plain loads and stores: the matrix
// instruction, loads straight into LDS, transposing LDS reads, and the waits and
// scheduling that go with them.
#pragma once

#include "gsz_device.h"

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

namespace {

// 16 bytes a lane from the descriptor's base + offset + uniform to LDS, lane l's at lds + 16 l.
// In assembly because the compiler, which cannot tell which LDS reads a builtin load concerns
// where they are the transposing ones, would wait for it before the next of them.  There is
// no result register; whoever reads the LDS calls loads_landed first.  m0 is named as changed, so that no
// value of the compiler's is taken to outlive the statement there; it says that it keeps none in
// reserved registers across such a one, which is what is wanted.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(BufRes res, _Float16* lds, int offset, int uniform) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 : : "s"(at), "v"(offset), "s"(res), "s"(uniform) : "memory", "m0");
}
#pragma clang diagnostic pop
// All but the last PENDING of this wave's loads to LDS are there.
template <int PENDING>
__device__ __forceinline__ void loads_landed() {
    static_assert(PENDING >= 0 && PENDING < 64, "a six-bit count");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(PENDING) : "memory");
}

// ds_read_b64_tr_b16: the 16 lanes of a group give the places of 4 rows of 16 values, 4 lanes
// a row and 4 values a lane; lane l of the group gets column l of the 4 rows.
__device__ __forceinline__ f16x4 read_turned(const _Float16* lds) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lds));
}

// acc + a b for a of 32 x 16 and b of 16 x 32: lane l holds a[l % 32][8 (l / 32) ...], b[8 (l / 32)
// ...][l % 32] and acc[8 (r / 4) + 4 (l / 32) + r % 4][l % 32], r in [0, 16).
__device__ __forceinline__ f32x16 multiply_add(f16x8 a, f16x8 b, f32x16 acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc, 0, 0, 0);
}

// Schedules READS LDS reads evenly among the PRODUCTS matrix instructions around this place.
template <int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int n = 0; n < PRODUCTS; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x100, (READS + PRODUCTS - 1) / PRODUCTS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
}

// Nothing is scheduled across this place.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// What lanes of a wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace
