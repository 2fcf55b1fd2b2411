// The parts of csrc/gsz_device.h and matrix/gsz_matrix.h that the orthogonalising kernels
// use, for the CPU run of those kernels (host_gpu/hip/hip_runtime.h).  A buffer access
// outside its descriptor's range ends the program; other accesses are AddressSanitizer's.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gsz_internal.h"

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

namespace {
constexpr int kBlock = 256, kXcds = 8;
constexpr int64_t kMaxWorkItems = (int64_t)1 << 31;
inline int64_t xcd_remap(int64_t b, int64_t G) {
    const int64_t q = G / kXcds, rem = G % kXcds, x = b % kXcds;
    return x * q + (x < rem ? x : rem) + b / kXcds;
}
inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
inline uint32_t bf16_rne(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x0040u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
inline void widen8(u32x4 w, float a[8]) {
    for (int j = 0; j < 4; ++j) { a[2 * j] = bf16_lo(w[j]); a[2 * j + 1] = bf16_hi(w[j]); }
}

// Every lane's value of any type, by address, while the wave waits.
template <class T, class F> auto with_wave(const T& mine, F f) {
    emu::S.slot[emu::S.cur] = reinterpret_cast<uint64_t>(&mine);
    emu::sync(emu::wave());
    auto r = f([](int lane) -> const T& {
        const int at = (emu::S.cur & ~63) + lane;
        if (at >= emu::S.threads || emu::S.ended[at]) emu::fail("reads a lane that has ended");
        return *reinterpret_cast<const T*>(emu::S.slot[at]);
    });
    emu::sync(emu::wave());
    return r;
}
inline double __shfl_xor(double v, int mask) {
    return with_wave(v, [&](auto of) { return of((emu::S.cur & 63) ^ mask); });
}
inline uint32_t __shfl_xor(uint32_t v, int mask) {
    return with_wave(v, [&](auto of) { return of((emu::S.cur & 63) ^ mask); });
}
inline int lane_id() { return emu::S.cur & 63; }

inline double block_sum(double x) {
    static double part[1024];
    part[emu::S.cur] = x;
    __syncthreads();
    double s = 0.0;
    if (emu::S.cur == 0) for (int k = 0; k < emu::S.threads; ++k) s += part[k];
    __syncthreads();
    return s;
}

struct BufRes { const char* base; uint32_t bytes; };
inline BufRes buf_res(const void* base, int64_t bytes) {
    return {static_cast<const char*>(base), bytes >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)(bytes > 0 ? bytes : 0)};
}
constexpr int kCpNt = 2;
// Dwords outside of the range read as 0, as the hardware has it.
inline u32x4 raw_buffer_load(BufRes r, int off) {
    u32x4 v = {0, 0, 0, 0};
    for (int j = 0; j < 4; ++j) {
        const uint32_t at = (uint32_t)off + 4 * j;
        if (at + 4 > at && (uint64_t)at + 4 <= r.bytes) { uint32_t w; std::memcpy(&w, r.base + at, 4); v[j] = w; }
    }
    return v;
}
#define __builtin_amdgcn_raw_buffer_load_b128(r, off, uniform, policy) raw_buffer_load((r), (off))
inline f32x4 ldf4(const float* p) { f32x4 v; std::memcpy(&v, p, 16); return v; }
inline void stf4(float* p, f32x4 v) { std::memcpy(p, &v, 16); }
inline f32x4 add4(f32x4 a, f32x4 b) { return f32x4{a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w}; }
inline void load_to_lds(BufRes res, _Float16* lds, int offset, int uniform) {
    const uint32_t at = (uint32_t)offset + (uint32_t)uniform;
    if (offset < 0 || uniform < 0) emu::fail("a load to LDS from before its buffer");
    _Float16* first = with_wave(lds, [](auto of) { return of(0); });
    if (first != lds) emu::fail("a load to LDS whose place is not the wave's");
    const u32x4 v = raw_buffer_load(res, (int)at);
    std::memcpy(lds + 8 * lane_id(), &v, 16);
}
template <int PENDING> inline void loads_landed() {}
inline f16x4 read_turned(const _Float16* lds) {
    return with_wave(lds, [](auto of) {
        const int l = lane_id(), group = l & ~15, col = l & 15;
        f16x4 v;
        for (int row = 0; row < 4; ++row) v[row] = of(group + 4 * row + col / 4)[col % 4];
        return v;
    });
}
inline f32x16 multiply_add(f16x8 a, f16x8 b, f32x16 acc) {
    struct Both { f16x8 a, b; } mine{a, b};
    return with_wave(mine, [&](auto of) {
        const int l = lane_id();
        for (int r = 0; r < 16; ++r) {
            const int row = 8 * (r / 4) + 4 * (l / 32) + r % 4;
            float s = 0.0f;
            for (int k = 0; k < 16; ++k) s += (float)of(row + 32 * (k / 8)).a[k % 8] * (float)of(l % 32 + 32 * (k / 8)).b[k % 8];
            acc[r] += s;
        }
        return acc;
    });
}
template <int READS, int PRODUCTS> inline void interleave() {}
inline void in_order() {}
inline void wave_fence() { emu::sync(emu::wave()); }
}  // namespace
