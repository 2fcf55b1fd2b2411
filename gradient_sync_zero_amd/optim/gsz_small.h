// Matrices with a side of at most 128.  Where both are small, one block does the whole of a
// matrix: momentum, norm, all Newton-Schulz steps in LDS, and the update.  18 dependent launches of
// a few microseconds each are what bounds such a matrix otherwise (128 x 128: 75 us, 24 here).
// Where the other side is long, a step is two launches.
//
// X lies in LDS as it does in memory, rows of kSmallPitch or 2 kSmallPitch values, and is read both
// along its rows and down its columns, beside A and S.  16-byte chunk c of
// row r is at c ^ (4 (r & 3) + (r >> 2 & 3)) within its group of 16: sixteen rows read along k, and
// four rows by four chunks read down columns, both meet every bank once.
#pragma once

#include "gsz_muon.h"

#pragma clang fp contract(off)

namespace {

constexpr int kSmallPitch = 128, kSmallSide = 128, kSmallLong = 256, kSmallWaves = 8;

// One of the matrices in LDS.
struct InLds {
    _Float16* at;
    int pitch;
    __device__ static int place(int row, int chunk) { return (chunk & ~15) | ((chunk ^ (4 * (row & 3) + (row >> 2 & 3))) & 15); }
    __device__ _Float16* chunk(int row, int c) const { return at + row * pitch + place(row, c) * 8; }
    // Eight k of a lane's row or, TURNED, column r0 + lane % 32, from k0 + 8 (lane / 32) on.
    template <bool TURNED>
    __device__ f16x8 read(int r0, int k0, int lane) const {
        if (!TURNED) return *reinterpret_cast<const f16x8*>(chunk(r0 + (lane & 31), k0 / 8 + (lane >> 5)));
        const int row = k0 + 8 * (lane >> 5) + (lane >> 2 & 3), c = r0 / 8 + 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
        return __builtin_shufflevector(read_turned(chunk(row, c) + 4 * (lane & 1)), read_turned(chunk(row + 4, c) + 4 * (lane & 1)),
                                       0, 1, 2, 3, 4, 5, 6, 7);
    }
};

template <int FM, int FN>
__device__ __forceinline__ void clear(f32x16 (&acc)[FM][FN]) {
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;
}
// acc += N sixteens of k from k0 on of the FM x FN parts of L R^T at rows i0, columns j0: all of
// their reads are under way before the first product.
template <int N, bool TL, bool TR, int FM, int FN>
__device__ __forceinline__ void small_piece(const InLds& L, const InLds& R, int i0, int j0, int k0, int lane, f32x16 (&acc)[FM][FN]) {
    f16x8 x[N][FM], y[N][FN];
#pragma unroll
    for (int h = 0; h < N; ++h) {
#pragma unroll
        for (int a = 0; a < FM; ++a) x[h][a] = L.read<TL>(i0 + 32 * a, k0 + 16 * h, lane);
#pragma unroll
        for (int b = 0; b < FN; ++b) y[h][b] = R.read<TR>(j0 + 32 * b, k0 + 16 * h, lane);
    }
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b) acc[a][b] = multiply_add(y[h][b], x[h][a], acc[a][b]);
}
// acc += those parts over k in [0, K), K a multiple of 32; N sixteens at a time while there are as many.
template <int N, bool TL, bool TR, int FM, int FN>
__device__ __forceinline__ void small_product(const InLds& L, const InLds& R, int i0, int j0, int K, int lane, f32x16 (&acc)[FM][FN]) {
    int k = 0;
    for (; k + 16 * N <= K; k += 16 * N) small_piece<N, TL, TR>(L, R, i0, j0, k, lane, acc);
    if (N > 2)
        for (; k < K; k += 32) small_piece<2, TL, TR>(L, R, i0, j0, k, lane, acc);
}

// use(row, first of four neighbouring columns, part [a][b], quarter q) for a lane's values of acc.
template <int FM, int FN, class Use>
__device__ __forceinline__ void each_four(int i0, int j0, int lane, Use use) {
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) use(i0 + 32 * a + (lane & 31), j0 + 32 * b + 8 * q + 4 * (lane >> 5), a, b, q);
}

__device__ __forceinline__ void put(const InLds& to, int row, int col, f16x4 v) {
    *reinterpret_cast<f16x4*>(to.chunk(row, col / 8) + (col & 4)) = v;
}
// to[i, j] = fp16(acc scale) for a wave's parts.
template <int FM, int FN>
__device__ __forceinline__ void put_all(const InLds& to, int i0, int j0, int lane, const f32x16 (&acc)[FM][FN], float scale) {
    each_four<FM, FN>(i0, j0, lane, [&](int row, int col, int a, int c, int q) {
        f16x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (_Float16)(acc[a][c][4 * q + e] * scale);
        put(to, row, col, v);
    });
}

// A step's coefficients as the products take them: a 2^12, b, c 2^-12.
struct Coefficients { float a, b, c; };
struct SmallSteps { int count; Coefficients of[kMostSteps]; };

// S = a I + b A + c A A, k x k, beside A or, IN_PLACE, where A was; `mine`: whether the wave has a
// part, at si, sj.  A is there for all waves before, and S after.
template <int N, bool IN_PLACE>
__device__ __forceinline__ void polynomial(const InLds& A, const InLds& S, int k, const Coefficients& f, bool mine, int si, int sj, int lane) {
    f32x16 p[2][1];
    if (mine) {
        clear(p);
        small_product<N, false, false>(A, A, si, sj, k, lane, p);
        each_four<2, 1>(si, sj, lane, [&](int row, int col, int a, int c, int q) {
            const f16x4 old = *reinterpret_cast<const f16x4*>(A.chunk(row, col / 8) + (col & 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) p[a][c][4 * q + e] = f.c * p[a][c][4 * q + e] + f.b * (float)old[e] + (row == col + e ? f.a : 0.0f);
        });
    }
    if (IN_PLACE) __syncthreads();                                   // all of A is read
    if (mine) put_all(S, si, sj, lane, p, 1.0f);
    __syncthreads();
}

// In: the values that are orthogonalised; Out: where the result goes.  `up` is the number of rows,
// `across` of columns; TALL where there are more rows than columns, LONG where the larger side is
// over kSmallPitch.
template <bool TALL, bool LONG, class In, class Out>
__global__ __launch_bounds__(64 * kSmallWaves) void k_small(In in, Out out, int rows, int cols, double eps, SmallSteps steps) {
    constexpr int kSquare = kSmallSide * kSmallPitch, kFN = LONG ? 2 : 1;
    constexpr int kMine = (LONG ? 2 : 1) * kSquare / 8 / (64 * kSmallWaves);     // vectors of X a work-item takes
    __shared__ __align__(16) _Float16 values[(LONG ? 4 : 3) * kSquare];
    __shared__ double part[kSmallWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x;
    const int small = TALL ? cols : rows, large = TALL ? rows : cols;
    const InLds A{values, kSmallPitch}, S{values + kSquare, kSmallPitch};
    const InLds X{values + 2 * kSquare, LONG && !TALL ? 2 * kSmallPitch : kSmallPitch};
    const int up = (rows + 31) / 32 * 32, across = (cols + 31) / 32 * 32;

    const int per = across / 8;
    float u[kMine][8];
    double s = 0.0;
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
        const int v = threadIdx.x + n * 64 * kSmallWaves, row = v / per, col = (v - row * per) * 8, left = row < rows ? cols - col : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[n][j] = 0.0f;
        if (left > 0) in.first(b, (int64_t)row * cols + col, left, u[n]);
    }
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
        const int v = threadIdx.x + n * 64 * kSmallWaves, row = v / per, left = cols - (v - row * per) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= left) u[n][j] = 0.0f;                           // without a value, a momentum's is not 0 times NaN
            s = s + (double)u[n][j] * (double)u[n][j];
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s = s + __shfl_xor(s, o);
    if (lane == 0) part[wave] = s;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) total = total + part[w];
    const double scale = norm_scale(total, eps);
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
        const int v = threadIdx.x + n * 64 * kSmallWaves, row = v / per;
        if (row >= up) continue;
        f16x8 h;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = (_Float16)(float)((double)u[n][j] * scale);
        *reinterpret_cast<f16x8*>(X.chunk(row, v - row * per)) = h;
    }
    __syncthreads();

    // a wave's part of A and S (64 x 32) and of X (64 x 64, or as A's)
    const int si = wave / 4 * 64, sj = wave % 4 * 32;
    const int xi = TALL && LONG ? wave / 2 * 64 : si, xj = LONG ? (TALL ? wave % 2 : wave % 4) * 64 : sj;
    const int k = (small + 31) / 32 * 32, K = (large + 31) / 32 * 32;
    const bool square = si < k && sj < k, whole = xi < up && xj < across;
    for (int t = 0; t < steps.count; ++t) {
        if (square) {
            f32x16 p[2][1];
            clear(p);
            small_product<8, TALL, TALL>(X, X, si, sj, K, lane, p);
            put_all(A, si, sj, lane, p, kScaleA / (kScaleX * kScaleX));
        }
        __syncthreads();
        polynomial<8, false>(A, S, k, steps.of[t], square, si, sj, lane);
        f32x16 x[2][kFN];
        if (whole) {
            clear(x);
            if (TALL) small_product<8, false, false>(X, S, xi, xj, k, lane, x);
            else small_product<8, false, true>(S, X, xi, xj, k, lane, x);
        }
        if (t + 1 == steps.count) {
            if (whole)
                each_four<2, kFN>(xi, xj, lane, [&](int row, int col, int a, int c, int q) {
                    if (row < rows && col < cols)
                        out.store(b, row, col, f32x4{x[a][c][4 * q], x[a][c][4 * q + 1], x[a][c][4 * q + 2], x[a][c][4 * q + 3]});
                });
            break;
        }
        __syncthreads();                                             // all of X is read
        if (whole) put_all(X, xi, xj, lane, x, 1.0f / kScaleA);
        __syncthreads();
    }
}

// ------------------------------------------------------- one side small --

// Matrices with one side of at most kSmallSide and a long other one: X lies in panels of kPanel of
// the long side, k = the small side rounded up to 32.  A step is two launches: the blocks of a
// matrix each take some panels, make S from A for themselves (128^3 products cost less than
// another launch), replace the panels by S X and add up the new panels' part of A; then those
// parts are added up.  26 matrices of 64 x 10048: 151 us, ten dependent launches of 10 to 20 us
// that wait for their panels; as products with their squares 279.  (Pieces of 4 and 8 panels leave
// too few blocks, and a panel loaded ahead of its use took 171 us.)
constexpr int kPanel = 128, kPanelPiece = 2;
struct Panels {
    int rows, cols, k, count, per, parts;    // panels of a matrix; of a block; blocks of a matrix
    _Float16* x;                             // panel p of matrix b, its rows one after the other, at (b count + p) k kPanel
    _Float16* a;                             // A of matrix b as it lies in LDS, at b kSmallSide kSmallPitch
    f32x4* partial;                          // of block n: each wave's parts as its lanes hold them, at n kPartVectors
};
constexpr int kPartVectors = kSmallWaves * 8 * 64;

// FIRST: the panels come from `in`; LAST: the result goes to `out`, and there is no next A.
template <bool TALL, bool FIRST, bool LAST, class In, class Out>
__global__ __launch_bounds__(64 * kSmallWaves) void k_panels(In in, Out out, Panels s, const double* scale, Coefficients step) {
    constexpr int kBlockSize = 64 * kSmallWaves, PN = kPanelPiece;
    __shared__ __align__(16) _Float16 values[2 * kSmallSide * kSmallPitch];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = s.k;
    const int b = blockIdx.x / s.parts, part = blockIdx.x - b * s.parts;
    const InLds X{values, kSmallPitch}, A{values + kSmallSide * kSmallPitch, kSmallPitch};
    const int si = wave / 4 * 64, sj = wave % 4 * 32;
    const bool square = si < k && sj < k, mine = TALL ? sj < k : si < k;
    const int up = TALL ? kPanel : k, vectors = (TALL ? k : kPanel) / 8;     // of a panel: rows, 16-byte vectors a row
    if (!FIRST) {
        const f16x8* from = reinterpret_cast<const f16x8*>(s.a + (int64_t)b * kSmallSide * kSmallPitch);
        for (int v = threadIdx.x; v < k * kSmallPitch / 8; v += kBlockSize) reinterpret_cast<f16x8*>(A.at)[v] = from[v];
        __syncthreads();
        polynomial<PN, true>(A, A, k, step, square, si, sj, lane);
    }
    f32x16 gram[2][1];
    clear(gram);
    const int last = (part + 1) * s.per < s.count ? (part + 1) * s.per : s.count;
    for (int n = part * s.per; n < last; ++n) {
        f16x8* panel = reinterpret_cast<f16x8*>(s.x + ((int64_t)b * s.count + n) * k * kPanel);
        const int row0 = TALL ? n * kPanel : 0, col0 = TALL ? 0 : n * kPanel;
        for (int v = threadIdx.x; v < up * vectors; v += kBlockSize) {
            const int row = v / vectors, c = v - row * vectors;
            f16x8 h;
            if (FIRST) {
                float u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = 0.0f;
                const int left = row0 + row < s.rows ? s.cols - (col0 + 8 * c) : 0;
                if (left > 0) in.again(b, (int64_t)(row0 + row) * s.cols + col0 + 8 * c, left, u);
                const double f = scale[b];
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = (_Float16)(float)((double)u[j] * f);
                panel[v] = h;
            } else {
                h = panel[v];
            }
            *reinterpret_cast<f16x8*>(X.chunk(row, c)) = h;
        }
        __syncthreads();
        if (!FIRST) {
            f32x16 x[2][1];
            if (mine) {
                clear(x);
                if (TALL) small_product<PN, false, false>(X, A, si, sj, k, lane, x);
                else small_product<PN, false, true>(A, X, si, sj, k, lane, x);
                if (LAST)
                    each_four<2, 1>(si, sj, lane, [&](int row, int col, int a, int c, int q) {
                        if (row0 + row < s.rows && col0 + col < s.cols)
                            out.store(b, row0 + row, col0 + col, f32x4{x[a][c][4 * q], x[a][c][4 * q + 1], x[a][c][4 * q + 2], x[a][c][4 * q + 3]});
                    });
            }
            __syncthreads();                                         // all of X is read
            if (LAST) continue;
            if (mine) put_all(X, si, sj, lane, x, 1.0f / kScaleA);
            __syncthreads();
            for (int v = threadIdx.x; v < up * vectors; v += kBlockSize) {
                const int row = v / vectors, c = v - row * vectors;
                panel[v] = *reinterpret_cast<const f16x8*>(X.chunk(row, c));
            }
        }
        if (square) small_product<PN, TALL, TALL>(X, X, si, sj, kPanel, lane, gram);
        if (n + 1 < last) __syncthreads();                           // all of X is read
    }
    if (!LAST && square) {
        f32x4* to = s.partial + (int64_t)blockIdx.x * kPartVectors + wave * 8 * 64 + lane;
        each_four<2, 1>(0, 0, lane, [&](int, int, int a, int c, int q) {
            to[(a * 4 + q) * 64] = f32x4{gram[a][c][4 * q], gram[a][c][4 * q + 1], gram[a][c][4 * q + 2], gram[a][c][4 * q + 3]};
        });
    }
}

// A of each matrix from its blocks' parts, in order: a wave for each 64 of its vectors.
__global__ __launch_bounds__(64) void k_panel_sum(Panels s) {
    constexpr int kPieces = kPartVectors / 64;
    const int lane = threadIdx.x, b = blockIdx.x / kPieces, piece = blockIdx.x - b * kPieces;
    const int wave = piece / 8, a = piece / 4 % 2, q = piece % 4;
    const int row = wave / 4 * 64 + 32 * a + (lane & 31), col = wave % 4 * 32 + 8 * q + 4 * (lane >> 5);
    if (wave / 4 * 64 >= s.k || wave % 4 * 32 >= s.k) return;        // a wave without a part
    const f32x4* from = s.partial + (int64_t)b * s.parts * kPartVectors + piece * 64 + lane;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int n = 0; n < s.parts; n += 8) {                           // eight loads at a time
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = n + j < s.parts ? from[(int64_t)(n + j) * kPartVectors] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = sum[e] + v[j][e];
    }
    f16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (_Float16)(sum[e] * (kScaleA / (kScaleX * kScaleX)));
    const InLds A{s.a + (int64_t)b * kSmallSide * kSmallPitch, kSmallPitch};
    put(A, row, col, h);
}

}  // namespace
