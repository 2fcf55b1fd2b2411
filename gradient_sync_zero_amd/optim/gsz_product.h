// Batched fp16 matrix products on the matrix cores for the Newton-Schulz steps:
// C[i, j] = sum_k L[i, k] R[j, k], summed in fp32.
//
// A block takes a tile of BM x BN of C, 64 of k at a time.  Each of the two operands
// lies in memory either with k along its rows ("plain": element (i, k) at i * ld + k)
// or with k down its columns ("turned": element (i, k) at k * ld + i), so a product
// with a transpose on either side needs no copy.  The next 64 of k come straight from
// memory into LDS (16 bytes a lane, no registers) while the matrix cores work on the
// present ones: a barrier for each 64 of k.
//
// LDS holds a tile as it lies in memory, in 16-byte chunks whose order within a row is
// permuted so that the lanes of a fragment's read meet every bank equally; the
// loads land in order, so the permutation is in the address that a lane reads from.
//   plain: rows of 64 k; chunk c of row r at place c ^ (r >> 1 & 7).  A lane's eight k
//     of its row are one 16-byte read.
//   turned: 64 rows of BM (or BN) elements; chunk c of row k at c ^ 4 (k & 3) (rows of
//     64: c ^ 2 (k & 2)).  ds_read_b64_tr_b16 gives lane l of 16 the column l of 4 rows of
//     16, so two reads give a lane its eight k.
// k is a multiple of 64: operands are padded with zeros, which the products keep.  Rows past
// an operand's end are read as zeros (its descriptor's range ends there) and not written.
//
// 8192 x 8192 x 8192: 840 to 870 us, 1.26 to 1.31 PFLOP/s.  The matrix cores are busy for 73 to 75% of the
// time and the clock is down to 1.63 GHz under their load; LDS, 128 bytes a clock, is the next bound.
// (24 of 2048 x 2048 x 2048: 55% at 1.93 GHz, of a symmetric result 39 to 44% at 2.05: the ends of 32
// steps of k, tiles over the diagonal and rounds that are not full.)  Measured and not kept: blocks that stay and run their loads on into the next tile
// (24 of 2048 x 2048 x 2048 401 us against 396), 128 x 128 a wave (its sums spill: half the
// speed), four tiles of 128 in LDS with one block a CU (27.6 us against 28.3 and 14.0 against 13.3).
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
    // Load n of the tile at the descriptor's beginning.
    __device__ static void load(const BufRes& res, int n, int64_t ld, int offset, int wave, _Float16* lds) {
        const int piece = n * WAVES + wave;
        load_to_lds(res, lds + piece * 512, offset, (int)(piece * kRowsPerLoad * ld * 2));
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
// symmetric result, those on and below the diagonal.  The first `whole` are a block's each; of
// the others `parts` blocks take a stretch of k each and leave their sums in `partial`.
struct Tiles { int64_t whole; int per, down, across, parts; bool half; f32x4* partial; };

struct TileAt { int64_t matrix; int ti, tj; };

// Tile n: columns of 8 tiles of rows.
__device__ __forceinline__ TileAt tile_at(const Tiles& t, int64_t index) {
    TileAt r;
    r.matrix = index / t.per;
    const int n = (int)(index - r.matrix * t.per);
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

// A launch's shape: tiles of SIDE x SIDE by WM x WN waves, STAGES tiles of both operands in LDS.
template <int SIDE, int WM_, int WN_, int STAGES_>
struct Form {
    static constexpr int kSide = SIDE, WM = WM_, WN = WN_, kStages = STAGES_, kWaves = WM * WN;
    static constexpr int TM = SIDE / WM, TN = SIDE / WN, FM = TM / 32, FN = TN / 32;
    static constexpr int kBuffer = 2 * SIDE * kStepK;
    static constexpr int kRegion = kStages * kBuffer / kWaves;      // a wave's part of LDS, fp16 values
    // an epilogue stages the wave's tile in fp16, or 32 rows of it in fp32
    static constexpr int kStaged = TM * TN > 64 * TN ? TM * TN : 64 * TN;
    static_assert(kStaged <= kRegion, "the epilogue's parts fit");
};

// A wave's tile of the result: its 32 x 32 parts, acc[a][b][r] of a lane being C[i + 32 a + lane % 32,
// j + 32 b + 8 (r / 4) + 4 (lane / 32) + r % 4], four neighbours of a row at a time.  rows, cols: C's;
// a tile may reach past them.
struct Place { int64_t matrix, i, j, rows, cols; bool off_diagonal; int lane; _Float16* lds; };

template <class F, bool TL, bool TR, class Epilogue>
__global__ __launch_bounds__(64 * F::kWaves) void k_product(Operand L, Operand R, int64_t rows, int64_t cols, int64_t K, Tiles tiles,
                                                            Epilogue epilogue) {
    constexpr int S = F::kStages, FM = F::FM, FN = F::FN, kBuffer = F::kBuffer;
    using TileL = Tile<F::kSide, TL, F::kWaves>;
    using TileR = Tile<F::kSide, TR, F::kWaves>;
    __shared__ __align__(16) _Float16 lds[S * kBuffer];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Blocks of one XCD take neighbouring tiles: they share its L2.
    const int64_t block = blockIdx.x, rest = block - tiles.whole;
    const int64_t index = rest < 0 ? xcd_remap(block, tiles.whole) : tiles.whole + rest / tiles.parts;
    const int part = rest < 0 ? 0 : (int)(rest % tiles.parts), parts = rest < 0 ? 1 : tiles.parts;
    const TileAt at = tile_at(tiles, index);
    const int64_t i0 = (int64_t)at.ti * F::kSide, j0 = (int64_t)at.tj * F::kSide;
    const int wi = wave / F::WN * F::TM, wj = wave % F::WN * F::TN;
    const int all = (int)(K / kStepK), from = (int)((int64_t)all * part / parts), steps = (int)((int64_t)all * (part + 1) / parts) - from;

    const int64_t stepL = TL ? kStepK * L.ld : kStepK, stepR = TR ? kStepK * R.ld : kStepK;
    const _Float16* pl = L.base + at.matrix * L.stride + (TL ? i0 : i0 * L.ld) + from * stepL;
    const _Float16* pr = R.base + at.matrix * R.stride + (TR ? j0 : j0 * R.ld) + from * stepR;
    const _Float16* endL = L.base + at.matrix * L.stride + (TL ? K : rows) * L.ld;
    const _Float16* endR = R.base + at.matrix * R.stride + (TR ? K : cols) * R.ld;
    const int offL = TileL::lane_offset(wave, lane, L.ld), offR = TileR::lane_offset(wave, lane, R.ld);

    f32x16 acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

    // Past the last step the ranges are empty: nothing is read, and the count of loads under way
    // stays the same.
    constexpr int kLoads = TileL::kLoads + TileR::kLoads;
    int loaded = 0;
    BufRes resL, resR;
    auto next_tile = [&] {
        resL = buf_res(pl, loaded < steps ? (endL - pl) * 2 : 0);
        resR = buf_res(pr, loaded < steps ? (endR - pr) * 2 : 0);
        pl += stepL;
        pr += stepR;
        ++loaded;
    };
    auto load = [&](_Float16* buf, int n) {
        if (n < TileL::kLoads) TileL::load(resL, n, L.ld, offL, wave, buf);
        else TileR::load(resR, n - TileL::kLoads, R.ld, offR, wave, buf + TileL::kElems);
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
    // there, so the loads of the tile S further on can take its buffer and the next tile's first
    // fragments are read while this tile's last products run.
    int now = 0;
#pragma unroll
    for (int t = 0; t < S; ++t) {
        next_tile();
#pragma unroll
        for (int n = 0; n < kLoads; ++n) load(lds + t * kBuffer, n);
    }
    loads_landed<(S - 1) * kLoads>();
    __syncthreads();
    read(lds, 0, 0);
    for (int t = 0; t < steps; ++t) {
        _Float16* buf = lds + now;
        now = now + kBuffer == S * kBuffer ? 0 : now + kBuffer;
        read(buf, 1, 1);
        multiply(0);
        read(buf, 2, 0);
        multiply(1);
        read(buf, 3, 1);
        multiply(0);
        loads_landed<(S - 2) * kLoads>();
        __syncthreads();
        next_tile();
        // The next loads go out between the products, a few after each: all of them first kept the
        // matrix cores waiting (8192 cubed 881 -> 850 us, 12 x 768 x 2304 x 768 45.0 -> 42.8; in the
        // first half of the products only 866, a wave's priority raised while it multiplies 890).
        // Where a wave has one product they go first (5 x 832 x 832 x 1536 14.4, after it 15.0).
        constexpr int kProducts = FM * FN;
        if constexpr (kProducts == 1) {
#pragma unroll
            for (int l = 0; l < kLoads; ++l) load(buf, l);
            read(lds + now, 0, 0);
            multiply(1);
        } else {
            read(lds + now, 0, 0);
#pragma unroll
            for (int n = 0; n < kProducts; ++n) {
                acc[n / FN][n % FN] = multiply_add(y[1][n % FN], x[1][n / FN], acc[n / FN][n % FN]);
#pragma unroll
                for (int l = n * kLoads / kProducts; l < (n + 1) * kLoads / kProducts; ++l) load(buf, l);
                in_order();
            }
        }
    }
    loads_landed<0>();
    __syncthreads();                                                    // the buffers are the epilogue's
    if (rest < 0) {
        epilogue.template write<FM, FN>(acc, Place{at.matrix, i0 + wi, j0 + wj, rows, cols, at.ti != at.tj, lane, lds + wave * F::kRegion});
    } else {
        f32x4* to = tiles.partial + (rest * F::kWaves + wave) * (FM * FN * 256) + lane;
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    to[((a * FN + b) * 4 + q) * 64] = f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
    }
}

// Adds up the parts of the tiles that were split, in order, and finishes them: a wave for each
// wave's tile.  Bound by memory and the launch (a few us; 2 x 4096 x 4096 17 us after products of 350).
template <class F, class Epilogue>
__global__ __launch_bounds__(64) void k_join(int64_t rows, int64_t cols, Tiles tiles, Epilogue epilogue) {
    constexpr int FM = F::FM, FN = F::FN;
    __shared__ __align__(16) _Float16 lds[F::kStaged];
    const int lane = threadIdx.x, wave = blockIdx.x % F::kWaves;
    const int64_t split = blockIdx.x / F::kWaves;
    const TileAt at = tile_at(tiles, tiles.whole + split);
    f32x16 acc[FM][FN];
    for (int part = 0; part < tiles.parts; ++part) {
        const f32x4* in = tiles.partial + ((split * tiles.parts + part) * F::kWaves + wave) * (FM * FN * 256) + lane;
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = in[((a * FN + b) * 4 + q) * 64];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[a][b][4 * q + e] = part ? acc[a][b][4 * q + e] + v[e] : v[e];
                }
    }
    epilogue.template write<FM, FN>(acc, Place{at.matrix, (int64_t)at.ti * F::kSide + wave / F::WN * F::TM,
                                               (int64_t)at.tj * F::kSide + wave % F::WN * F::TN, rows, cols, at.ti != at.tj, lane, lds});
}

// ------------------------------------------------------------- epilogues --

// The place of 16-byte chunk `chunk` of a row in a wave's part of LDS, `per` chunks a row, so that
// lanes with a row each and lanes along a row both meet every bank equally.
template <int PER>
__device__ __forceinline__ int staged_chunk(int row, int chunk) {
    static_assert(PER == 4 || PER == 8 || PER == 16, "");
    return row * PER + (chunk ^ (PER == 16 ? row & 15 : PER == 8 ? row >> 1 & 7 : row >> 2 & 3));
}

// A wave's tile as fp16, so that memory is written in whole rows: four neighbours of a row go in
// as 8 bytes, 16-byte chunks come out.
template <int FM, int FN>
struct Staged {
    static constexpr int kRows = 32 * FM, kCols = 32 * FN, kChunks = kCols / 8;
    __device__ static int at(int row, int chunk) { return staged_chunk<kChunks>(row, chunk) * 8; }
    __device__ static void put(_Float16* lds, int a, int b, int q, int lane, f16x4 v) {
        const int row = 32 * a + (lane & 31);
        *reinterpret_cast<f16x4*>(lds + at(row, 4 * b + q) + 4 * (lane >> 5)) = v;
    }
    // Writes the tile to its place in m, rows `ld` apart.
    __device__ static void rows(const Place& p, _Float16* m, int64_t ld) {
        constexpr int kPer = 64 / kChunks;                          // rows an access
        _Float16* out = m + p.i * ld + p.j;
#pragma unroll
        for (int n = 0; n < kRows / kPer; ++n) {
            const int row = n * kPer + p.lane / kChunks, c = p.lane % kChunks;
            if (p.i + row < p.rows && p.j + 8 * c < p.cols)
                *reinterpret_cast<u32x4*>(out + row * ld + c * 8) = *reinterpret_cast<const u32x4*>(p.lds + at(row, c));
        }
    }
    // Writes its transpose to the other side of the diagonal (m is symmetric).
    __device__ static void columns(const Place& p, _Float16* m, int64_t ld) {
        _Float16* out = m + p.j * ld + p.i;
        // a group of 16 lanes turns 8 rows by 16 columns; the groups lie one above the other
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += 32)
#pragma unroll
            for (int c0 = 0; c0 < kCols; c0 += 16) {
                const int row = r0 + 8 * (p.lane >> 4) + (p.lane >> 2 & 3), chunk = c0 / 8 + (p.lane >> 1 & 1);
                const f16x4 x = read_turned(p.lds + at(row, chunk) + 4 * (p.lane & 1));
                const f16x4 y = read_turned(p.lds + at(row + 4, chunk) + 4 * (p.lane & 1));
                const int to = c0 + (p.lane & 15), first = r0 + 8 * (p.lane >> 4);
                if (p.j + to < p.rows && p.i + first < p.cols)
                    *reinterpret_cast<f16x8*>(out + to * ld + first) = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            }
    }
};

// Hands the tile to use(row, column, four values of C) with neighbouring lanes along a row: 32 rows
// at a time through LDS in fp32.
template <int FM, int FN, class Use>
__device__ __forceinline__ void by_rows(const f32x16 (&acc)[FM][FN], const Place& p, Use use) {
    constexpr int kChunks = 8 * FN, kPer = 64 / kChunks;            // 16-byte chunks a row, rows an access
    f32x4* lds = reinterpret_cast<f32x4*>(p.lds);
#pragma unroll
    for (int a = 0; a < FM; ++a) {
        if (a) wave_fence();
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                lds[staged_chunk<kChunks>(p.lane & 31, 8 * b + 2 * q + (p.lane >> 5))] =
                    f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
        wave_fence();
#pragma unroll
        for (int n = 0; n < 32 / kPer; ++n) {
            const int row = n * kPer + p.lane / kChunks, c = p.lane % kChunks;
            use(p.i + 32 * a + row, p.j + 4 * c, lds[staged_chunk<kChunks>(row, c)]);
        }
    }
}

// out = fp16(acc * scale); a symmetric result's tile is written to both of its places.
template <bool SYMMETRIC>
struct StoreHalf {
    _Float16* out;
    int64_t stride, ld;
    float scale;
    template <int FM, int FN>
    __device__ void write(const f32x16 (&acc)[FM][FN], const Place& p) const {
        using S = Staged<FM, FN>;
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    S::put(p.lds, a, b, q, p.lane, f16x4{(_Float16)(acc[a][b][4 * q] * scale), (_Float16)(acc[a][b][4 * q + 1] * scale),
                                                        (_Float16)(acc[a][b][4 * q + 2] * scale), (_Float16)(acc[a][b][4 * q + 3] * scale)});
        wave_fence();
        _Float16* m = out + p.matrix * stride;
        S::rows(p, m, ld);
        if (SYMMETRIC && p.off_diagonal) S::columns(p, m, ld);
    }
};

}  // namespace
