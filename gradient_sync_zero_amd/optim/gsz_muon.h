// Orthogonalising updates by Newton-Schulz steps, and the optimizer step built on it.
//
// X0 = U / (|U| + eps); a step takes A = X X^T, S = a I + b A + c A A, X <- S X: three
// products, the first two symmetric (only their lower tiles are computed).  A matrix with
// more rows than columns goes by A = X^T X and X <- X S, so that A has the smaller size.
//
// The iterates are held in fp16 and summed in fp32.  bf16 would cost the same on the matrix
// cores and is eight times coarser: an update of 768 x 2304 comes out 0.9% off the 64-bit
// result (2-norm) in bf16 and 0.09% in fp16, below bf16's own rounding of the result (0.17%).
// The iteration multiplies what is small by 3.4445 a step, roundings in directions that U does not
// have among it: of a U with few directions the result is further off (one: 15%, eight: 4%).  What
// carries that is noise of every direction, 2^-11 of U at first; keeping it down would take X and S in two
// fp16 parts each, three products for one.
// Range: the singular values of X stay near or below 1.2 with the usual coefficients, so X is
// held as 2^13 X, and A and S as 2^12 A, 2^12 S.  Values down to 2^-27 (X) and 2^-26 (A, S)
// then have fp16's full precision, and overflow begins at 8 and 16.  The product of two steps'
// polynomials is held as 2^8 S1 S0, for values up to 256.  a I is part of S (and
// not a X added to the product) so that the rounding of S's diagonal is relative to a + b
// + c after cancellation.
#pragma once

#include "gsz_product.h"

#pragma clang fp contract(off)

namespace {

constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f, kScaleP = 256.0f;
// Elements a block of the norm and of the scaling takes, 8 a lane.
constexpr int kUpdateBlock = 256;
constexpr int64_t kNormTile = 16 * kUpdateBlock;      // two vectors a lane
// Matrices a launch holds: their places travel in the kernel arguments.
constexpr int kMuonBatch = 256;
constexpr int kMostSteps = 16;

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// Where a launch's matrices begin in the flat buffers, elements.
struct Places { int64_t at[kMuonBatch]; };

__device__ __forceinline__ void load8(const float* p, float v[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float v[8]) { widen8(*reinterpret_cast<const u32x4_any*>(p), v); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
// The first m of eight values, 0 for the others.
template <class T>
__device__ __forceinline__ void load8_part(const T* p, int64_t m, float v[8]) {
    if (m >= 8) { load8(p, v); return; }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < m ? load1(p + j) : 0.0f;
}

// What is orthogonalised, eight values of matrix b from its element e on, the first `left` of them
// in the matrix and the others 0.  first() is called once for each value and makes it; again()
// gives it once more.
template <class T>
struct Values {
    const T* x;
    int64_t size;
    __device__ void first(int64_t b, int64_t e, int64_t left, float u[8]) const { load8_part(x + b * size + e, left, u); }
    __device__ void again(int64_t b, int64_t e, int64_t left, float u[8]) const { first(b, e, left, u); }
};

// m <- mu m + g coef; u = g coef + mu m, or m.
struct Momentum {
    float* momentum;
    const float* g;
    const float* coef;
    float mu;
    int nesterov;
    Places places;
    __device__ void direction(const float m[8], const float gc[8], float u[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = nesterov ? gc[j] + mu * m[j] : m[j];
    }
    __device__ void first(int64_t b, int64_t e, int64_t left, float u[8]) const {
        float* p = momentum + places.at[b] + e;
        const float c = *coef;
        float m[8], gc[8];
        load8_part(p, left, m);
        load8_part(g + places.at[b] + e, left, gc);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            gc[j] = gc[j] * c;
            m[j] = mu * m[j] + gc[j];
        }
        direction(m, gc, u);
        if (left >= 8) {
            *reinterpret_cast<f32x4_any*>(p) = f32x4{m[0], m[1], m[2], m[3]};
            *reinterpret_cast<f32x4_any*>(p + 4) = f32x4{m[4], m[5], m[6], m[7]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) if (j < left) p[j] = m[j];
        }
    }
    __device__ void again(int64_t b, int64_t e, int64_t left, float u[8]) const {
        const float c = *coef;
        float m[8], gc[8];
        load8_part(momentum + places.at[b] + e, left, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) gc[j] = 0.0f;
        if (nesterov) load8_part(g + places.at[b] + e, left, gc);
#pragma unroll
        for (int j = 0; j < 8; ++j) gc[j] = gc[j] * c;
        direction(m, gc, u);
    }
};

// Sums of squares, one a block, in fp64 and a fixed order.  Bound by memory: the momentum's pass
// over 24 matrices of 2048 x 2048 (12 bytes an element) 215 us, 5.6 TB/s.
template <class In>
__global__ __launch_bounds__(kUpdateBlock) void k_norm(In in, int64_t size, unsigned tiles, double* partial) {
    const unsigned b = blockIdx.x / tiles, t = blockIdx.x - b * tiles;
    double s = 0.0;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int64_t e = t * kNormTile + n * 8 * kUpdateBlock + 8 * threadIdx.x, left = size - e;
        if (left <= 0) continue;
        float u[8];
        in.first(b, e, left, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = s + (j < left ? (double)u[j] * (double)u[j] : 0.0);
    }
    const double total = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

// 2^13 / (|U| + eps) from |U|^2; NaN where U has a value that is not finite.
__device__ __forceinline__ double norm_scale(double total, double eps) {
    return total - total == 0.0 ? (double)kScaleX / (sqrt(total) + eps) : __builtin_nan("");
}
__global__ __launch_bounds__(kBlock) void k_scale(const double* partial, int64_t tiles, double eps, double* scale) {
    constexpr int kAhead = 16;                       // loads under way: 28672 x 8192 19 us, one by one 88
    double s = 0.0;
    for (int64_t t = threadIdx.x; t < tiles; t += kAhead * kBlock) {
        double p[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) p[j] = t + j * kBlock < tiles ? partial[blockIdx.x * tiles + t + j * kBlock] : 0.0;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) s = s + p[j];
    }
    const double total = block_sum(s);
    if (threadIdx.x == 0) scale[blockIdx.x] = norm_scale(total, eps);
}

// The padded matrices in fp16: eight columns a lane, zeros outside of rows x cols.  Bound by memory:
// 24 momenta of 2048 x 2048 and their gradients (10 bytes an element) 202 us, 5.0 TB/s.  (The scale
// kept for the next launch's reader instead saved about 2 us of 100.)
struct Padded { int64_t rows, cols, ld, vectors; };   // ld = padded columns; vectors: ld / 8 * padded rows
template <class In>
__global__ __launch_bounds__(kUpdateBlock) void k_scaled(In in, Padded p, unsigned tiles, const double* scale, _Float16* x) {
    const unsigned b = blockIdx.x / tiles;
    const int64_t v = (int64_t)(blockIdx.x - b * tiles) * kUpdateBlock + threadIdx.x;
    if (v >= p.vectors) return;
    const int per = (int)(p.ld / 8);
    const int64_t row = v < (int64_t)0xFFFFFFFFu ? (uint32_t)v / (uint32_t)per : v / per;
    const int64_t col = (v - row * per) * 8;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 0.0f;
    if (row < p.rows && col < p.cols) in.again(b, row * p.cols + col, p.cols - col, u);
    const double s = scale[b];
    f16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (_Float16)(float)((double)u[j] * s);
    *reinterpret_cast<f16x8*>(x + b * p.vectors * 8 + v * 8) = h;
}

// ------------------------------------------------------------- epilogues --

// S = a I + b A + c A A, from acc = 2^24 A A and A itself; symmetric.
struct StorePolynomial {
    const _Float16* A;
    _Float16* S;
    int64_t stride, ld;
    float a, b, c;                                      // a 2^12, b, c 2^-12
    template <int FM, int FN>
    __device__ void write(const f32x16 (&acc)[FM][FN], const Place& p) const {
        using St = Staged<FM, FN>;
        const _Float16* in = A + p.matrix * stride;
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t row = p.i + 32 * x + (p.lane & 31), col = p.j + 32 * y + 8 * q + 4 * (p.lane >> 5);
                    f16x4 v = {};
                    if (row < p.rows && col < p.cols) {
                        const f16x4 old = *reinterpret_cast<const f16x4*>(in + row * ld + col);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = (_Float16)(c * acc[x][y][4 * q + e] + b * (float)old[e] + (row == col + e ? a : 0.0f));
                    }
                    St::put(p.lds, x, y, q, p.lane, v);
                }
        wave_fence();
        _Float16* m = S + p.matrix * stride;
        St::rows(p, m, ld);
        if (p.off_diagonal) St::columns(p, m, ld);
    }
};

__device__ __forceinline__ u32x2 pack4_bf16(const float v[4]) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[0], v[1]}), b2)),
                 __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2], v[3]}), b2))};
}

// out = bf16(2^25 O * scale) without the padding.
struct StoreResult {
    uint16_t* out;
    int64_t rows, cols;
    float scale;
    // four values of a row that begin in the matrix
    __device__ void store(int64_t matrix, int64_t row, int64_t col, f32x4 x) const {
        const float v[4] = {x.x * scale, x.y * scale, x.z * scale, x.w * scale};
        const u32x2 w = pack4_bf16(v);
        uint16_t* to = out + (matrix * rows + row) * cols + col;
        if (col + 4 <= cols) {
            *reinterpret_cast<u32x2_any*>(to) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e) if (col + e < cols) to[e] = (uint16_t)((e & 2 ? w.y : w.x) >> 16 * (e & 1));
        }
    }
    template <int FM, int FN>
    __device__ void write(const f32x16 (&acc)[FM][FN], const Place& p) const {
        by_rows(acc, p, [&](int64_t row, int64_t col, f32x4 x) { if (row < rows && col < cols) store(p.matrix, row, col, x); });
    }
};

// theta <- theta (1 - lr wd) - lr scale O; p = bf16(theta).
struct StoreUpdate {
    float* master;
    uint16_t* params;
    Places places;
    int64_t rows, cols;
    float scale, decay, rate;                            // 2^-25, 1 - lr wd, lr * the update's scale
    __device__ void store(int64_t matrix, int64_t row, int64_t col, f32x4 x) const {
        float* w = master + places.at[matrix] + row * cols + col;
        uint16_t* to = params + places.at[matrix] + row * cols + col;
        if (col + 4 <= cols) {
            const f32x4 old = *reinterpret_cast<const f32x4_any*>(w);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = old[e] * decay - rate * (x[e] * scale);
            *reinterpret_cast<f32x4_any*>(w) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<u32x2_any*>(to) = pack4_bf16(v);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (col + e < cols) {
                    const float v = w[e] * decay - rate * (x[e] * scale);
                    w[e] = v;
                    to[e] = (uint16_t)bf16_rne(v);
                }
        }
    }
    template <int FM, int FN>
    __device__ void write(const f32x16 (&acc)[FM][FN], const Place& p) const {
        by_rows(acc, p, [&](int64_t row, int64_t col, f32x4 x) { if (row < rows && col < cols) store(p.matrix, row, col, x); });
    }
};

}  // namespace
