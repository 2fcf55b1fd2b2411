// Dropout from a counter-based generator: the mask is a function of (seed, step,
// site, element index) and is computed where it is needed, forward and backward,
// and never stored.
//
// Element e of a call belongs to block b = e >> 3.  Philox4x32 with 10 rounds
// (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC'11), key = the two words of the seed, counter = (b low, b high, site, step),
// gives four words, eight 16-bit halves: half e & 7 is the high half h of a
// 32-bit number u.  Its low half l is the same half at the counter with bit 31 of
// word 1 set (b is below 2^61, so the two never meet).  e is dropped iff u < T.
// h alone decides wherever h != T >> 16, so l is drawn only by waves that hold an
// element with h == T >> 16 (one wave in 128): eight exact 32-bit decisions for
// the price of one ten-round block.
#pragma once

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Wunused-function"     // the step's block sum
#include "gsz_device.h"
#pragma clang diagnostic pop

#pragma clang fp contract(off)

namespace {

// ------------------------------------------------ values of either type --

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// 16-byte vectors at any element's place: tensors lie anywhere in a flat bucket,
// and gfx950 takes such accesses whole (unaligned access is part of its HSA ABI).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

// Two fp32 values to bf16, nearest even, the first in the low half
// (v_cvt_pk_bf16_f32; NaN stays a quiet NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)pack_bf16(x, 0.0f); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// Eight consecutive values as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { u32x4 w; };
template <> struct Raw8<float> { f32x4 a, b; };

template <bool NT>
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p) {
    const u32x4_at2* q = reinterpret_cast<const u32x4_at2*>(p);
    return {NT ? __builtin_nontemporal_load(q) : *q};
}
template <bool NT>
__device__ __forceinline__ Raw8<float> load8(const float* p) {
    const f32x4_at4* q = reinterpret_cast<const f32x4_at4*>(p);
    if (NT) return {__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)};
    return {q[0], q[1]};
}
// The first m < 8 of them (m >= 0), 0 in the places of the others.
__device__ __forceinline__ Raw8<uint16_t> load8_part(const uint16_t* p, int m) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = j < m ? p[j] : 0;
    return {u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16}};
}
__device__ __forceinline__ Raw8<float> load8_part(const float* p, int m) {
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = j < m ? p[j] : 0.0f;
    return {f32x4{h[0], h[1], h[2], h[3]}, f32x4{h[4], h[5], h[6], h[7]}};
}
__device__ __forceinline__ void widen(const Raw8<uint16_t>& r, float a[8]) { widen8(r.w, a); }
__device__ __forceinline__ void widen(const Raw8<float>& r, float a[8]) {
    a[0] = r.a.x; a[1] = r.a.y; a[2] = r.a.z; a[3] = r.a.w;
    a[4] = r.b.x; a[5] = r.b.y; a[6] = r.b.z; a[7] = r.b.w;
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, const float a[8]) {
    const u32x4 w = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7])};
    u32x4_at2* q = reinterpret_cast<u32x4_at2*>(p);
    if (NT) __builtin_nontemporal_store(w, q); else *q = w;
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float a[8]) {
    f32x4_at4* q = reinterpret_cast<f32x4_at4*>(p);
    const f32x4 x = {a[0], a[1], a[2], a[3]}, y = {a[4], a[5], a[6], a[7]};
    if (NT) { __builtin_nontemporal_store(x, q); __builtin_nontemporal_store(y, q + 1); }
    else { q[0] = x; q[1] = y; }
}
template <typename T>
__device__ __forceinline__ void store8_part(T* p, const float a[8], int m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) if (j < m) store1(p + j, a[j]);
}

// ------------------------------------------------------ a wave's tile --

// A wave's tile is kTile elements of a row.  A lane's elements of it, so that each of the
// wave's accesses covers whole lines: 8 in a row for bf16 (16 bytes), two groups of 4 for
// fp32.  `T` names the type whose accesses decide (others follow its places).
constexpr int kTile = 512;
template <typename T> struct Cols;
template <> struct Cols<uint16_t> { static constexpr int kPieces = 1, kWidth = 8; };
template <> struct Cols<float> { static constexpr int kPieces = 2, kWidth = 4; };
template <typename T>
__device__ __forceinline__ int64_t piece_col(int p) {
    return p * 64 * Cols<T>::kWidth + Cols<T>::kWidth * (threadIdx.x & 63);
}

template <typename T> struct RowPiece;                // a lane's values of one tile
template <> struct RowPiece<uint16_t> { Raw8<uint16_t> r; };
template <> struct RowPiece<float> { f32x4 a, b; };
template <bool NT>
__device__ __forceinline__ f32x4 load4(const float* p) {
    const f32x4_at4* q = reinterpret_cast<const f32x4_at4*>(p);
    return NT ? __builtin_nontemporal_load(q) : *q;
}
__device__ __forceinline__ f32x4 load4_part(const float* p, int64_t m) {
    return f32x4{m > 0 ? p[0] : 0.0f, m > 1 ? p[1] : 0.0f, m > 2 ? p[2] : 0.0f, m > 3 ? p[3] : 0.0f};
}
// row: the tile's first element; left: elements from there on, and FULL where the tile
// has them all (most do, and the code for the others, eight times
// unrolled, would not fit the instruction cache beside it).
template <bool FULL, bool NT>
__device__ __forceinline__ RowPiece<uint16_t> load_row(const uint16_t* row, int64_t left) {
    const int64_t c = piece_col<uint16_t>(0), m = left - c;
    return {FULL || m >= 8 ? load8<NT>(row + c) : load8_part(row + c, (int)(m > 0 ? m : 0))};
}
template <bool FULL, bool NT>
__device__ __forceinline__ RowPiece<float> load_row(const float* row, int64_t left) {
    const int64_t c = piece_col<float>(0), d = piece_col<float>(1);
    return {FULL || left - c >= 4 ? load4<NT>(row + c) : load4_part(row + c, left - c),
            FULL || left - d >= 4 ? load4<NT>(row + d) : load4_part(row + d, left - d)};
}
__device__ __forceinline__ void widen_row(const RowPiece<uint16_t>& r, float a[8]) { widen(r.r, a); }
__device__ __forceinline__ void widen_row(const RowPiece<float>& r, float a[8]) {
    widen(Raw8<float>{r.a, r.b}, a);
}
// Groups of 4 values of either type (grad and partial rows, at any element).
__device__ __forceinline__ void load4(const float* p, float a[4]) {
    const f32x4 x = *reinterpret_cast<const f32x4_at4*>(p);
    a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float a[4]) {
    const u32x2 w = *reinterpret_cast<const u32x2_at2*>(p);
    a[0] = bf16_lo(w.x); a[1] = bf16_hi(w.x); a[2] = bf16_lo(w.y); a[3] = bf16_hi(w.y);
}
template <bool NT>
__device__ __forceinline__ void store4(float* p, const float a[4]) {
    f32x4_at4* q = reinterpret_cast<f32x4_at4*>(p);
    const f32x4 x = {a[0], a[1], a[2], a[3]};
    if (NT) __builtin_nontemporal_store(x, q); else *q = x;
}
template <bool NT>
__device__ __forceinline__ void store4(uint16_t* p, const float a[4]) {
    u32x2_at2* q = reinterpret_cast<u32x2_at2*>(p);
    const u32x2 x = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
    if (NT) __builtin_nontemporal_store(x, q); else *q = x;
}
// The lane's values of a tile, as fp32.
template <typename T, bool FULL, typename G>
__device__ __forceinline__ void load_old(const G* row, int64_t left, float a[8]) {
    if (Cols<T>::kPieces == 1 && (FULL || left - piece_col<T>(0) >= 8)) {
        widen(load8<false>(row + piece_col<T>(0)), a);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t c = Cols<T>::kPieces == 1 ? piece_col<T>(0) + 4 * h : piece_col<T>(h), m = left - c;
        if (FULL || m >= 4) load4(row + c, a + 4 * h);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j) a[4 * h + j] = j < m ? load1(row + c + j) : 0.0f;
    }
}
template <typename T, bool FULL, bool NT, typename G>
__device__ __forceinline__ void store_row(G* row, int64_t left, const float a[8]) {
    if (Cols<T>::kPieces == 1 && (FULL || left - piece_col<T>(0) >= 8)) {
        store8<NT>(row + piece_col<T>(0), a);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t c = Cols<T>::kPieces == 1 ? piece_col<T>(0) + 4 * h : piece_col<T>(h), m = left - c;
        if (FULL || m >= 4) store4<NT>(row + c, a + 4 * h);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j) if (j < m) store1(row + c + j, a[4 * h + j]);
    }
}

// ------------------------------------------------------------- generator --

// What a call's mask depends on besides the element; rng (device) holds the seed
// and the step.  threshold 0 drops nothing.
struct DropArgs { const uint64_t* rng; uint32_t site, threshold; };
struct DropKey { uint32_t k0, k1, site, step, threshold; };

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
    const uint64_t seed = d.rng[0];
    return {(uint32_t)seed, (uint32_t)(seed >> 32), d.site, (uint32_t)d.rng[1], d.threshold};
}

__device__ __forceinline__ u32x4 philox10(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3,
                                          uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
        const uint32_t y0 = (uint32_t)(b >> 32) ^ x1 ^ k0, y2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x0 = y0; x1 = (uint32_t)b; x2 = y2; x3 = (uint32_t)a;
        k0 += 0x9E3779B9u; k1 += 0xBB67AE85u;
    }
    return u32x4{x0, x1, x2, x3};
}

// u[j] orders as element 8 * block + j's 32-bit number does against the
// threshold: dropped iff u[j] < threshold.
__device__ __forceinline__ void drop_numbers(const DropKey& d, uint64_t block, uint32_t u[8]) {
    const u32x4 r = philox10((uint32_t)block, (uint32_t)(block >> 32), d.site, d.step, d.k0, d.k1);
    // The high halves in place; below them lies what cannot decide.
    u[0] = r.x << 16; u[1] = r.x; u[2] = r.y << 16; u[3] = r.y;
    u[4] = r.z << 16; u[5] = r.z; u[6] = r.w << 16; u[7] = r.w;
    const uint32_t t = d.threshold >> 16;
    bool tie = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) tie |= (u[j] >> 16) == t;
    if (__builtin_expect(tie, 0)) {
        const u32x4 s = philox10((uint32_t)block, (uint32_t)(block >> 32) | 0x80000000u, d.site, d.step, d.k0, d.k1);
        const uint32_t l[8] = {s.x & 0xFFFFu, s.x >> 16, s.y & 0xFFFFu, s.y >> 16,
                               s.z & 0xFFFFu, s.z >> 16, s.w & 0xFFFFu, s.w >> 16};
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = (u[j] & 0xFFFF0000u) | l[j];
    }
}

// a[j] <- 0 where element first + j is dropped (chosen, not multiplied: an infinity or
// NaN in a dropped place leaves 0), first a multiple of 8.
__device__ __forceinline__ void drop8_at(const DropKey& d, const uint32_t u[8], float a[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = u[j] < d.threshold ? 0.0f : a[j];
}
// Bit j: element first + j is dropped.
__device__ __forceinline__ uint32_t dropped8(const DropKey& d, uint64_t first) {
    uint32_t u[8], m = 0;
    drop_numbers(d, first >> 3, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) m |= (uint32_t)(u[j] < d.threshold) << j;
    const uint32_t s = (uint32_t)first & 7;
    if (s != 0) {                                // the eight lie in two blocks
        drop_numbers(d, (first >> 3) + 1, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) m |= (uint32_t)(u[j] < d.threshold) << (8 + j);
        m = m >> s & 0xFFu;
    }
    return m;
}
// a[j] <- 0 where bit j is set.
__device__ __forceinline__ void drop8(uint32_t gone, float a[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (gone >> j & 1) ? 0.0f : a[j];
}

// The lane's values zeroed where dropped; first: element index of the tile's first column.
// Each lane draws the mask of 8 columns in a row; fp32's groups of 4 fetch theirs.
template <typename T>
__device__ __forceinline__ uint32_t dropped_row(const DropKey& d, uint64_t first) {
    const int lane = threadIdx.x & 63;
    const uint32_t m = dropped8(d, first + 8 * lane);
    if (Cols<T>::kPieces == 1) return m;
    const uint32_t lo = (uint32_t)__shfl((int)m, lane >> 1) >> 4 * (lane & 1);
    const uint32_t hi = (uint32_t)__shfl((int)m, 32 + (lane >> 1)) >> 4 * (lane & 1);
    return (lo & 15) | (hi & 15) << 4;
}

// --------------------------------------------------------------- dropout --

// y[e] = (add[e] or 0) + (dropped(e) ? 0 : x[e] * k), e in [0, n): one fp32
// multiplication, one fp32 addition, one rounding to T.  A wave takes one tile, a lane
// draws one generator block.
//
// Bound by memory, the generator's 20 products of 32 bits (v_mad_u64_u32) and 60 other
// instructions for 8 elements just behind it: 512 Mi bf16 elements added to a stream of as
// many in 490 us (6.57 TB/s; 2 GiB copied by torch: 4.9), 48 Mi fp32 from an odd place in 64 us
// (6.3 TB/s; with each lane's 8 values in a row, half a line an access, 74).  One wave per
// block; four took 507 us.  A whole 32-bit word per element would take twice the products.
constexpr int kDropBlock = 64;
template <typename T, bool ADD, bool DROP, bool FULL>
__device__ __forceinline__ void dropout_tile(const T* x, const T* add, T* y, int64_t e, int64_t left,
                                             float k, const DropKey& d) {
    const RowPiece<T> r = load_row<FULL, true>(x + e, left);
    RowPiece<T> q{};
    if (ADD) q = load_row<FULL, true>(add + e, left);
    // The mask needs no data: it is drawn while the loads are on their way.
    // (bf16's lanes use the numbers themselves, which saves packing and unpacking bits.)
    constexpr bool kBits = Cols<T>::kPieces > 1;
    uint32_t gone = 0, u[8];
    if (DROP && kBits) gone = dropped_row<T>(d, (uint64_t)e);
    if (DROP && !kBits) drop_numbers(d, ((uint64_t)e >> 3) + (threadIdx.x & 63), u);
    float a[8], b[8];
    widen_row(r, a);
    if (ADD) widen_row(q, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = a[j] * k;
    if (DROP && kBits) drop8(gone, a);
    if (DROP && !kBits) drop8_at(d, u, a);
    if (ADD) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = b[j] + a[j];
    }
    store_row<T, FULL, true>(y + e, left, a);
}
template <typename T, bool ADD, bool DROP>
__global__ __launch_bounds__(kDropBlock) void k_dropout(const T* x, const T* add, T* y, int64_t n,
                                                        float k, DropArgs da) {
    DropKey d{};
    if (DROP) d = drop_key(da);                      // rng may be NULL otherwise
    const int64_t stride = (int64_t)gridDim.x * kTile;
    for (int64_t e = (int64_t)blockIdx.x * kTile; e < n; e += stride) {
        if (n - e >= kTile) dropout_tile<T, ADD, DROP, true>(x, add, y, e, n - e, k, d);
        else dropout_tile<T, ADD, DROP, false>(x, add, y, e, n - e, k, d);
    }
}

}  // namespace
