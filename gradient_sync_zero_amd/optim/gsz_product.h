// Batched fp16 matrix products on the matrix cores for the Newton-Schulz steps:
// C[i, j] = sum_k L[i, k] R[j, k], summed in fp32.
//
// A block takes a tile of BM x BN of C, 64 of k at a time.  Each of the two operands
// lies in memory either with k along its rows ("plain": element (i, k) at i * ld + k)
// or with k down its columns ("turned": element (i, k) at k * ld + i), so a product
// with a transpose on either side needs no copy.  The next 64 of k come straight from
// memory into LDS (16 bytes a lane, no registers) while the matrix cores work on the
// present ones: two buffers, one barrier between them.
//
// LDS holds a tile as it lies in memory, in 16-byte chunks whose order within a row is
// permuted so that the lanes of a fragment's read meet every bank equally; the
// loads land in order, so the permutation is in the address that a lane reads from.
//   plain: rows of 64 k; chunk c of row r at place c ^ (r >> 1 & 7).  A lane's eight k
//     of its row are one 16-byte read.
//   turned: 64 rows of BM (or BN) elements; chunk c of row k at c ^ 4 (k & 3) (rows of
//     64: c ^ 2 (k & 2)).  ds_read_b64_tr_b16 gives lane l of 16 the column l of 4 rows of
//     16, so two reads give a lane its eight k.
// All sizes are multiples of the tiles: operands are padded with zeros, which the
// products keep.
#pragma once

#include "gsz_matrix.h"

#pragma clang fp contract(off)

namespace {

constexpr int kStepK = 64;

// One operand of a batched product: matrix b at base + b * stride.
struct Operand { const _Float16* base; int64_t stride; int64_t ld; };

// What an operand's tile of ROWS x 64 (plain) or 64 x ROWS (turned) takes to load and read.
// WAVES waves load it together.
template <int ROWS, bool TURNED, int WAVES>
struct Tile {
    static constexpr int kElems = ROWS * kStepK;
    static constexpr int kLoads = kElems / (512 * WAVES);           // 1 KiB each, per wave
    static constexpr int kChunks = TURNED ? ROWS / 8 : 8;           // 16-byte chunks in a row
    static constexpr int kRowsPerLoad = 64 / kChunks;
    static_assert(kLoads * 512 * WAVES == kElems && WAVES % 2 == 0, "whole loads");

    __device__ static int place(int row, int chunk) {
        return TURNED ? (ROWS == 64 ? chunk ^ (2 * (row & 2)) : chunk ^ (4 * (row & 3))) : chunk ^ (row >> 1 & 7);
    }
    // The bytes that a lane's load is away from its tile's first element (the same for every
    // load of a wave: the permutation repeats after 16 rows or fewer).
    __device__ static int lane_offset(int wave, int lane, int64_t ld) {
        const int row = lane / kChunks, chunk = place(wave * kRowsPerLoad + row, lane % kChunks);
        return (int)(row * ld + chunk * 8) * 2;
    }
    // Loads the tile at `at` (wave-uniform; `left` bytes from there to the matrix's end).
    __device__ static void load(const _Float16* at, int64_t left, int64_t ld, int offset, int wave, _Float16* lds) {
        const BufRes res = buf_res(at, left);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int piece = n * WAVES + wave;
            load_to_lds(res, lds + piece * 512, offset, (int)(piece * kRowsPerLoad * ld * 2));
        }
    }
    // A lane's eight k (16 kk + 8 (lane / 32) ...) of row r0 + lane % 32, r0 a multiple of 32.
    __device__ static f16x8 read(const _Float16* lds, int r0, int kk, int lane) {
        if (!TURNED) {
            const int row = lane & 31, chunk = 2 * kk + (lane >> 5);
            return *reinterpret_cast<const f16x8*>(lds + (r0 + row) * 64 + place(row, chunk) * 8);
        }
        const int row = lane >> 2 & 3, chunk = r0 / 8 + 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
        const _Float16* p = lds + (16 * kk + 8 * (lane >> 5) + row) * ROWS + place(row, chunk) * 8 + 4 * (lane & 1);
        return __builtin_shufflevector(read_turned(p), read_turned(p + 4 * ROWS), 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// The tiles of one launch: `across` tiles of columns by `down` of rows a matrix, or, of a
// symmetric result, those on and below the diagonal.
struct Tiles { int64_t total; int per, down, across; bool half; };

struct TileAt { int64_t matrix; int ti, tj; };

// Blocks of one XCD take neighbouring tiles (they share its L2), columns of 8 tiles of rows.
__device__ __forceinline__ TileAt tile_at(const Tiles& t) {
    const int64_t b = xcd_remap(blockIdx.x, t.total);
    TileAt r;
    r.matrix = b / t.per;
    const int n = (int)(b - r.matrix * t.per);
    if (t.half) {
        int i = (int)((sqrtf(8.0f * n + 1.0f) - 1.0f) * 0.5f);
        while (i * (i + 1) / 2 > n) --i;
        while ((i + 1) * (i + 2) / 2 <= n) ++i;
        r.ti = i;
        r.tj = n - i * (i + 1) / 2;
    } else {
        const int group = n / (8 * t.across), first = group * 8, rows = t.down - first < 8 ? t.down - first : 8;
        const int in = n - group * 8 * t.across;
        r.ti = first + in % rows;
        r.tj = in / rows;
    }
    return r;
}

// The product's tile, handed to the epilogue as its 32 x 32 parts: acc[a][b][r] of a lane is
// C[i0 + 32 a + lane % 32, j0 + 32 b + 8 (r / 4) + 4 (lane / 32) + r % 4], four neighbours of
// a row at a time.
template <int BM, int BN, int WM, int WN, bool TL, bool TR, class Epilogue>
__global__ __launch_bounds__(64 * WM * WN) void k_product(Operand L, Operand R, int64_t rowsL, int64_t rowsR, int64_t K,
                                                          Tiles tiles, Epilogue epilogue) {
    constexpr int kWaves = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    using TileL = Tile<BM, TL, kWaves>;
    using TileR = Tile<BN, TR, kWaves>;
    constexpr int kBuffer = TileL::kElems + TileR::kElems;
    // two variables, so that the compiler sees that the loads of one do not touch the other
    __shared__ __align__(16) _Float16 even[kBuffer], odd[kBuffer];
    static_assert(BM * BN / 2 <= kBuffer, "the epilogue's parts fit");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const TileAt at = tile_at(tiles);
    const int64_t i0 = (int64_t)at.ti * BM, j0 = (int64_t)at.tj * BN;
    const int wi = wave / WN * TM, wj = wave % WN * TN;

    const _Float16* pl = L.base + at.matrix * L.stride + (TL ? i0 : i0 * L.ld);
    const _Float16* pr = R.base + at.matrix * R.stride + (TR ? j0 : j0 * R.ld);
    const _Float16* endL = L.base + at.matrix * L.stride + (TL ? K : rowsL) * L.ld;
    const _Float16* endR = R.base + at.matrix * R.stride + (TR ? K : rowsR) * R.ld;
    const int64_t stepL = TL ? kStepK * L.ld : kStepK, stepR = TR ? kStepK * R.ld : kStepK;
    const int offL = TileL::lane_offset(wave, lane, L.ld), offR = TileR::lane_offset(wave, lane, R.ld);

    f32x16 acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

    auto load = [&](_Float16* buf) {
        TileL::load(pl, (endL - pl) * 2, L.ld, offL, wave, buf);
        TileR::load(pr, (endR - pr) * 2, R.ld, offR, wave, buf + TileL::kElems);
        pl += stepL;
        pr += stepR;
    };
    // One of the four 16-wide pieces of a tile: its fragments, and the products of those.
    f16x8 x[2][FM], y[2][FN];
    auto read = [&](const _Float16* buf, int kk, int set) {
#pragma unroll
        for (int a = 0; a < FM; ++a) x[set][a] = TileL::read(buf, wi + 32 * a, kk, lane);
#pragma unroll
        for (int b = 0; b < FN; ++b) y[set][b] = TileR::read(buf + TileL::kElems, wj + 32 * b, kk, lane);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b) acc[a][b] = multiply_add(y[set][b], x[set][a], acc[a][b]);
        interleave<FM * (TL ? 2 : 1) + FN * (TR ? 2 : 1), FM * FN>();    // the other set's reads among them
    };
    // A tile's last reads are done before the barrier that also says that the next tile is
    // there, so the loads of the tile after that can take its buffer and the next tile's first
    // fragments are read while this tile's last products run.
    const int steps = (int)(K / kStepK);
    auto landed = [&] {
        loads_landed();
        __syncthreads();
    };
    auto tile = [&](_Float16* now, _Float16* next, int t) {
        read(now, 1, 1);
        multiply(0);
        read(now, 2, 0);
        multiply(1);
        read(now, 3, 1);
        multiply(0);
        landed();
        if (t + 2 < steps) load(now);
        if (t + 1 < steps) read(next, 0, 0);
        multiply(1);
    };
    load(even);
    landed();
    if (steps > 1) load(odd);
    read(even, 0, 0);
    for (int t = 0; t < steps; t += 2) {
        tile(even, odd, t);
        if (t + 1 < steps) tile(odd, even, t + 1);
    }
    __syncthreads();                                                    // the buffers are the epilogue's
    epilogue.template write<FM, FN>(acc, at.matrix, i0 + wi, j0 + wj, at.ti != at.tj, lane,
                                    (wave < kWaves / 2 ? even : odd) + wave % (kWaves / 2) * (TM * TN));
}

// ------------------------------------------------------------- epilogues --

// A wave's tile as fp16 through its own part of LDS, so that memory is written in whole rows:
// four neighbours of a row go in as 8 bytes, 16-byte chunks come out.  Rows of TN elements;
// chunk c of row r at c ^ (r >> 1 & 7).
template <int FM, int FN>
struct Staged {
    static constexpr int kRows = 32 * FM, kCols = 32 * FN, kChunks = kCols / 8;
    static_assert(kChunks == 8 || kChunks == 16, "swizzle");
    __device__ static int at(int row, int chunk) { return row * kCols + (chunk ^ (kChunks == 8 ? row >> 1 & 7 : row & 15)) * 8; }
    __device__ static void put(_Float16* lds, int a, int b, int q, int lane, f16x4 v) {
        const int row = 32 * a + (lane & 31);
        *reinterpret_cast<f16x4*>(lds + at(row, 4 * b + q) + 4 * (lane >> 5)) = v;
    }
    // Writes the tile to out (its first element), rows `ld` apart.
    __device__ static void rows(const _Float16* lds, _Float16* out, int64_t ld, int lane) {
        constexpr int kPer = 64 / kChunks;                          // rows an access
#pragma unroll
        for (int n = 0; n < kRows / kPer; ++n) {
            const int row = n * kPer + lane / kChunks, c = lane % kChunks;
            *reinterpret_cast<u32x4*>(out + row * ld + c * 8) = *reinterpret_cast<const u32x4*>(lds + at(row, c));
        }
    }
    // Writes its transpose: row j of out takes column j.
    __device__ static void columns(const _Float16* lds, _Float16* out, int64_t ld, int lane) {
        // a group of 16 lanes turns 8 rows by 16 columns; the groups lie one above the other
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += 32)
#pragma unroll
            for (int c0 = 0; c0 < kCols; c0 += 16) {
                const int row = r0 + 8 * (lane >> 4) + (lane >> 2 & 3), chunk = c0 / 8 + (lane >> 1 & 1);
                const f16x4 x = read_turned(lds + at(row, chunk) + 4 * (lane & 1));
                const f16x4 y = read_turned(lds + at(row + 4, chunk) + 4 * (lane & 1));
                *reinterpret_cast<f16x8*>(out + (int64_t)(c0 + (lane & 15)) * ld + r0 + 8 * (lane >> 4)) =
                    __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            }
    }
};

// out = fp16(acc * scale); a symmetric result's tile is written to both of its places.
template <bool SYMMETRIC>
struct StoreHalf {
    _Float16* out;
    int64_t stride, ld;
    float scale;
    template <int FM, int FN>
    __device__ void write(const f32x16 (&acc)[FM][FN], int64_t matrix, int64_t i, int64_t j, bool off_diagonal, int lane, _Float16* lds) const {
        using S = Staged<FM, FN>;
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    S::put(lds, a, b, q, lane, f16x4{(_Float16)(acc[a][b][4 * q] * scale), (_Float16)(acc[a][b][4 * q + 1] * scale),
                                                    (_Float16)(acc[a][b][4 * q + 2] * scale), (_Float16)(acc[a][b][4 * q + 3] * scale)});
        wave_fence();
        _Float16* m = out + matrix * stride;
        S::rows(lds, m + i * ld + j, ld, lane);
        if (SYMMETRIC && off_diagonal) S::columns(lds, m + j * ld + i, ld, lane);
    }
};

}  // namespace
