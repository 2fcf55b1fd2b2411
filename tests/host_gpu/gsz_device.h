// The part of csrc/gsz_device.h that the embedding and dropout kernels use, for
// the CPU run of those kernels.
#pragma once
#include <hip/hip_runtime.h>

#include "gsz.h"

namespace gsz {
inline void set_error(const char* fmt, ...) { (void)fmt; }
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

namespace {
constexpr int64_t kMaxWorkItems = (int64_t)1 << 31;
inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
inline void widen8(u32x4 w, float a[8]) {
    a[0] = bf16_lo(w.x); a[1] = bf16_hi(w.x); a[2] = bf16_lo(w.y); a[3] = bf16_hi(w.y);
    a[4] = bf16_lo(w.z); a[5] = bf16_hi(w.z); a[6] = bf16_lo(w.w); a[7] = bf16_hi(w.w);
}
inline f32x4 ldf4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
inline void stf4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
inline f32x4 add4(f32x4 a, f32x4 b) { return f32x4{a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w}; }
}  // namespace
