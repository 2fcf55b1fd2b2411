// Embedding lookup with scaling (and dropout), and its gradient by sorted tokens.
#pragma once

#include "gsz_dropout.h"

#pragma clang fp contract(off)

namespace {

// A token as a row of the table, or `rows` (no row) where it is outside [0, rows).
struct Ids { const void* p; int is64; uint32_t rows; };
__device__ __forceinline__ uint32_t row_of(const Ids& ids, int64_t i) {
    if (ids.is64) {
        const int64_t v = static_cast<const int64_t*>(ids.p)[i];
        return v >= 0 && v < (int64_t)ids.rows ? (uint32_t)v : ids.rows;
    }
    const int32_t v = static_cast<const int32_t*>(ids.p)[i];
    return v >= 0 && (uint32_t)v < ids.rows ? (uint32_t)v : ids.rows;
}

// ---------------------------------------------------------------- lookup --

// out[i, c] = id_i is a row and not dropped(i * dim + c) ? table[id_i, c] * c0 : 0.
// A block takes tile_rows rows of vpr = ceil(dim / 8) vectors, about kLookVecs of
// them: kLookUnroll loads of the table in flight per lane, then the stores.
// magic = floor(2^32 / vpr) + 1: (q * magic) >> 32 == q / vpr for q < kLookVecs and
// vpr <= kLookVecs; wider rows come one to a block.
constexpr int kLookBlock = 256, kLookUnroll = 4, kLookVecs = kLookBlock * kLookUnroll;
template <typename T, typename O, bool DROP>
__global__ __launch_bounds__(kLookBlock) void k_lookup(const T* __restrict__ table, Ids ids, int64_t n,
                                                       int64_t dim, int64_t vpr, int tile_rows,
                                                       uint64_t magic, float c0, DropArgs da,
                                                       O* __restrict__ out) {
    DropKey d{};
    if (DROP) d = drop_key(da);
    const int64_t tiles = (n + tile_rows - 1) / tile_rows;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t row0 = tile * tile_rows;
        const int64_t nrows = n - row0 < tile_rows ? n - row0 : tile_rows;
        const int64_t vecs = nrows * vpr;
        for (int64_t q0 = threadIdx.x; q0 < vecs; q0 += kLookVecs) {
            Raw8<T> r[kLookUnroll];
            int64_t row[kLookUnroll], col[kLookUnroll];
            bool is_row[kLookUnroll];
#pragma unroll
            for (int u = 0; u < kLookUnroll; ++u) {
                const int64_t q = q0 + u * kLookBlock;
                is_row[u] = false;
                row[u] = -1;
                if (q < vecs) {
                    const int64_t lr = tile_rows == 1 ? 0 : (int64_t)(((uint64_t)q * magic) >> 32);
                    row[u] = row0 + lr;
                    col[u] = 8 * (q - lr * vpr);
                    const uint32_t v = row_of(ids, row[u]);
                    is_row[u] = v != ids.rows;
                    if (is_row[u]) {
                        const T* p = table + (int64_t)v * dim + col[u];
                        const int64_t left = dim - col[u];
                        r[u] = left >= 8 ? load8<false>(p) : load8_part(p, (int)left);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kLookUnroll; ++u) {
                if (row[u] < 0) continue;
                float a[8] = {};
                if (is_row[u]) {
                    widen(r[u], a);
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = a[j] * c0;
                    if (DROP) drop8(d, (uint64_t)(row[u] * dim + col[u]), a);
                }
                O* p = out + row[u] * dim + col[u];
                const int64_t left = dim - col[u];
                if (left >= 8) store8<true>(p, a);
                else store8_part(p, a, (int)left);
            }
        }
    }
}

// ------------------------------------------------------------------ sort --
//
// The tokens sorted by (row, position): key[s] the s-th row, pos[s] its position;
// tokens without a row sort last with key = rows.

// n <= kRankMax tokens in one launch: token i goes to place
// #{j : key_j < key_i} + #{j < i : key_j == key_i}.  A block holds all keys in LDS
// and places 64 tokens; its waves compare them with a slice of the keys each.
constexpr int kRankMax = 8192, kRankBlock = 512, kRankWaves = kRankBlock / 64;
__global__ __launch_bounds__(kRankBlock) void k_rank(Ids ids, int n, uint32_t* __restrict__ key,
                                                     uint32_t* __restrict__ pos) {
    __shared__ __align__(16) uint32_t all[kRankMax];
    __shared__ uint32_t part[kRankWaves][64];
    const int n4 = (n + 4 * kRankWaves - 1) / (4 * kRankWaves) * (4 * kRankWaves);
    for (int j = threadIdx.x; j < n4; j += kRankBlock) all[j] = j < n ? row_of(ids, j) : 0xFFFFFFFFu;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = blockIdx.x * 64 + lane;
    const uint32_t mine = i < n ? all[i] : 0;
    const int j0 = wave * (n4 / kRankWaves), j1 = j0 + n4 / kRankWaves;
    uint32_t less = 0;
    const u32x4* all4 = reinterpret_cast<const u32x4*>(all);
    for (int j = j0; j < j1; j += 4) {
        const u32x4 k = all4[j >> 2];
        less += (k.x < mine) | ((k.x == mine) & (j < i));
        less += (k.y < mine) | ((k.y == mine) & (j + 1 < i));
        less += (k.z < mine) | ((k.z == mine) & (j + 2 < i));
        less += (k.w < mine) | ((k.w == mine) & (j + 3 < i));
    }
    part[wave][lane] = less;
    __syncthreads();
    if (wave == 0 && i < n) {
        uint32_t s = 0;
#pragma unroll
        for (int w = 0; w < kRankWaves; ++w) s += part[w][lane];
        key[s] = mine;
        pos[s] = (uint32_t)i;
    }
}

// More tokens: stable counting passes over digits of the key, lowest first.
// count[tile][digit] holds how often a digit occurs in a tile of tokens.
constexpr int kSortBlock = 256, kSortWaves = kSortBlock / 64, kSortMaxBins = 1024;
struct Digit { int shift, bins; };       // bins a power of two
__device__ __forceinline__ uint32_t digit_of(const Digit& d, uint32_t key) {
    return (key >> d.shift) & (uint32_t)(d.bins - 1);
}

// Orders a wave's LDS accesses for the compiler (the hardware keeps them in order).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Counts the first digit of each tile, and clears the next pass's counts.
__global__ __launch_bounds__(kSortBlock) void k_count(Ids ids, int64_t n, int64_t tile, Digit d,
                                                      uint32_t* __restrict__ count,
                                                      uint32_t* __restrict__ next) {
    __shared__ uint32_t h[kSortMaxBins];
    for (int b = threadIdx.x; b < d.bins; b += kSortBlock) h[b] = 0;
    __syncthreads();
    const int64_t i1 = (blockIdx.x + 1) * tile < n ? (blockIdx.x + 1) * tile : n;
    for (int64_t i = blockIdx.x * tile + threadIdx.x; i < i1; i += kSortBlock)
        atomicAdd(&h[digit_of(d, row_of(ids, i))], 1u);
    __syncthreads();
    for (int b = threadIdx.x; b < d.bins; b += kSortBlock) {
        count[(int64_t)blockIdx.x * d.bins + b] = h[b];
        next[(int64_t)blockIdx.x * d.bins + b] = 0;
    }
}

// Moves the tokens of one tile to their places by one digit, and counts the next
// digit (dn.bins > 0) where they land; clears the counts after that.  FIRST reads the
// tokens themselves, later passes the sorted pairs.  A wave takes a quarter of the
// tile: it counts its digits, then places them in order from its own bases.
template <bool FIRST>
__global__ __launch_bounds__(kSortBlock) void k_place(Ids ids, const uint32_t* __restrict__ key_in,
                                                      const uint32_t* __restrict__ pos_in, int64_t n,
                                                      int64_t tile, int tiles, Digit d, Digit dn,
                                                      const uint32_t* __restrict__ count,
                                                      uint32_t* __restrict__ next,
                                                      uint32_t* __restrict__ clear,
                                                      uint32_t* __restrict__ key, uint32_t* __restrict__ pos) {
    __shared__ uint32_t base[kSortWaves][kSortMaxBins];
    __shared__ uint32_t sums[kSortBlock];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t0 = blockIdx.x * tile, t1 = t0 + tile < n ? t0 + tile : n;
    const int64_t quarter = (t1 - t0 + kSortWaves - 1) / kSortWaves;
    const int64_t w0 = t0 + wave * quarter < t1 ? t0 + wave * quarter : t1;
    const int64_t w1 = w0 + quarter < t1 ? w0 + quarter : t1;
    if (clear)
        for (int b = threadIdx.x; b < d.bins; b += kSortBlock) clear[(int64_t)blockIdx.x * d.bins + b] = 0;
    for (int b = lane; b < d.bins; b += 64) base[wave][b] = 0;
    __syncthreads();
    for (int64_t i = w0 + lane; i < w1; i += 64)
        atomicAdd(&base[wave][digit_of(d, FIRST ? row_of(ids, i) : key_in[i])], 1u);
    // Thread t sums the digits [t * per, (t + 1) * per) over all tiles, and those of
    // the tiles before this one.
    const int per = (d.bins + kSortBlock - 1) / kSortBlock;
    uint32_t before[kSortMaxBins / kSortBlock], total[kSortMaxBins / kSortBlock], mine = 0;
#pragma unroll
    for (int k = 0; k < kSortMaxBins / kSortBlock; ++k) {
        const int b = threadIdx.x * per + k;
        uint32_t all = 0, prior = 0;
        if (k < per && b < d.bins) {
#pragma unroll 8
            for (int t = 0; t < tiles; ++t) {
                const uint32_t c = count[(int64_t)t * d.bins + b];
                all += c;
                prior += t < (int)blockIdx.x ? c : 0;
            }
        }
        before[k] = prior;
        total[k] = all;
        mine += all;
    }
    sums[threadIdx.x] = mine;
    __syncthreads();
    for (int o = 1; o < kSortBlock; o <<= 1) {
        const uint32_t s = threadIdx.x >= o ? sums[threadIdx.x - o] : 0;
        __syncthreads();
        sums[threadIdx.x] += s;
        __syncthreads();
    }
    uint32_t run = sums[threadIdx.x] - mine;
#pragma unroll
    for (int k = 0; k < kSortMaxBins / kSortBlock; ++k) {
        const int b = threadIdx.x * per + k;
        if (k < per && b < d.bins) {
            uint32_t at = run + before[k];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = base[w][b];
                base[w][b] = at;
                at += c;
            }
            run += total[k];
        }
    }
    __syncthreads();
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < w1;
        const uint32_t k = in ? (FIRST ? row_of(ids, i) : key_in[i]) : 0;
        const uint32_t p = in ? (FIRST ? (uint32_t)i : pos_in[i]) : 0;
        const uint32_t dg = digit_of(d, k);
        // The lanes of this wave with the same digit.
        uint64_t same = __ballot(in);
        for (int bit = 1; bit < d.bins; bit <<= 1) {
            const uint64_t m = __ballot((dg & bit) != 0);
            same &= (dg & bit) ? m : ~m;
        }
        const uint32_t rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        uint32_t at = 0;
        if (in) at = base[wave][dg] + rank;
        wave_fence();
        if (in && rank == 0) base[wave][dg] += __popcll(same);
        wave_fence();
        if (in) {
            key[at] = k;
            pos[at] = p;
            if (dn.bins) atomicAdd(&next[(int64_t)(at / (uint32_t)tile) * dn.bins + digit_of(dn, k)], 1u);
        }
    }
}

// -------------------------------------------------------------- gradient --
//
// grad[v, c] = (old or 0) + c0 * sum of the kept dy[pos, c] over v's tokens.
//
// The sorted tokens are cut into chunks of K; one wave sums the runs of equal
// rows of one chunk over one tile of columns, in fp32, positions rising.  A run
// that lies inside its chunk is finished there.  A run over several chunks leaves
// an fp32 partial sum per chunk: part[2c] where it came from an earlier chunk,
// part[2c + 1] where it starts in c; k_fold and k_join add them in chunk order.

constexpr int kGradBlock = 256, kGradWaves = kGradBlock / 64, kGradCols = 512, kGradUnroll = 8;
constexpr int kMaxChunk = 64;

template <typename G>
__device__ __forceinline__ void grad_write(G* p, const float sum[8], float c0, bool acc, int64_t left) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = sum[j] * c0;
    if (left >= 8) {
        if (acc) {
            float b[8];
            widen(load8<false>(p), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = b[j] + a[j];
        }
        store8<false>(p, a);
    } else {
        if (acc) {
            float b[8];
            widen(load8_part(p, (int)left), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = b[j] + a[j];
        }
        store8_part(p, a, (int)left);
    }
}

// Partial rows are padded to whole vectors.
__device__ __forceinline__ void part_write(float* p, const float sum[8], int64_t left) {
    if (left > 0) store8<false>(p, sum);
}

struct GradShape {
    int64_t dim, pitch;                  // pitch: floats of a partial row
    int64_t n, chunks;
    uint32_t rows;
    int K, col_blocks, acc;
    int64_t sum_blocks;                  // blocks that sum; the rest clear rows
    int clear_rows;                      // rows per clearing block
};

template <typename T, typename G, bool DROP>
__global__ __launch_bounds__(kGradBlock) void k_grad(const T* __restrict__ dy, const uint32_t* __restrict__ key,
                                                     const uint32_t* __restrict__ pos, GradShape s,
                                                     float c0, DropArgs da, G* __restrict__ grad,
                                                     float* __restrict__ part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int64_t)blockIdx.x >= s.sum_blocks) {
        // Clears the rows without a token among clear_rows of them.
        const int64_t r0 = ((int64_t)blockIdx.x - s.sum_blocks) * s.clear_rows;
        const int64_t v = r0 + lane;
        bool missing = lane < s.clear_rows && v < (int64_t)s.rows;
        if (missing) {
            int64_t lo = 0, hi = s.n;    // the first sorted place with key >= v
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (key[mid] < (uint32_t)v) lo = mid + 1; else hi = mid;
            }
            missing = lo >= s.n || key[lo] != (uint32_t)v;
        }
        const float zero[8] = {};
        for (uint64_t m = __ballot(missing); m; m &= m - 1) {
            G* p = grad + (r0 + __builtin_ctzll(m)) * s.dim;
            for (int64_t c = 8 * (int64_t)threadIdx.x; c < s.dim; c += 8 * kGradBlock) {
                if (s.dim - c >= 8) store8<true>(p + c, zero);
                else store8_part(p + c, zero, (int)(s.dim - c));
            }
        }
        return;
    }
    const int64_t chunk = (int64_t)blockIdx.x / s.col_blocks;
    const int64_t c_tile = ((int64_t)(blockIdx.x % s.col_blocks) * kGradWaves + wave) * kGradCols;
    if (c_tile >= s.dim) return;
    // Lanes past the last column stay: every lane holds a key.
    const int64_t c = c_tile + 8 * lane, left = s.dim - c > 0 ? s.dim - c : 0;
    DropKey d{};
    if (DROP) d = drop_key(da);
    const int64_t s0 = chunk * s.K;
    const int m = (int)(s.n - s0 < s.K ? s.n - s0 : s.K);
    // lane l holds the chunk's l-th key and position
    const uint32_t my_key = lane < m ? key[s0 + lane] : s.rows, my_pos = lane < m ? pos[s0 + lane] : 0;
    const uint32_t prev = s0 > 0 ? key[s0 - 1] : s.rows, next = s0 + m < s.n ? key[s0 + m] : s.rows;
    uint32_t cur = __builtin_amdgcn_readfirstlane(my_key);
    if (cur == s.rows) return;                        // from here on no token has a row
    bool from_before = cur == prev;
    float sum[8] = {};
    for (int k0 = 0; k0 < m; k0 += kGradUnroll) {
        Raw8<T> r[kGradUnroll];
        uint32_t kk[kGradUnroll], pp[kGradUnroll];
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const int at = k0 + u < m ? k0 + u : m - 1;
            kk[u] = __builtin_amdgcn_readlane(my_key, at);
            pp[u] = __builtin_amdgcn_readlane(my_pos, at);
            if (k0 + u >= m) kk[u] = s.rows;
            const T* p = dy + (int64_t)pp[u] * s.dim + c;
            r[u] = left >= 8 ? load8<true>(p) : load8_part(p, (int)left);
        }
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            if (kk[u] != cur) {
                if (cur != s.rows) {
                    if (from_before) part_write(part + 2 * chunk * s.pitch + c, sum, left);
                    else grad_write(grad + (int64_t)cur * s.dim + c, sum, c0, s.acc != 0, left);
                }
                from_before = false;
                cur = kk[u];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
            }
            if (kk[u] != s.rows) {
                float a[8];
                widen(r[u], a);
                if (DROP) drop8(d, (uint64_t)pp[u] * (uint64_t)s.dim + (uint64_t)c, a);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = sum[j] + a[j];
            }
        }
    }
    if (cur == s.rows) return;
    if (from_before) part_write(part + 2 * chunk * s.pitch + c, sum, left);
    else if (cur == next) part_write(part + (2 * chunk + 1) * s.pitch + c, sum, left);
    else grad_write(grad + (int64_t)cur * s.dim + c, sum, c0, s.acc != 0, left);
}

// Partial sums of one run are folded kFold at a time: where the aligned group of
// kFold chunks of `step` chunks each lies inside one run, past its first chunk, their
// sum takes the place of the group's first partial.
constexpr int kFold = 32, kJoinCols = 256;
__device__ __forceinline__ bool inside_run(const uint32_t* __restrict__ key, const GradShape& s,
                                           int64_t c, int64_t len) {
    // every token of the chunks [c, c + len) has the row of the token before them
    if (c + len > s.chunks || c == 0) return false;
    const int64_t last = (c + len) * s.K - 1 < s.n ? (c + len) * s.K - 1 : s.n - 1;
    const uint32_t k = key[c * s.K - 1];
    return k != s.rows && key[last] == k;
}
__device__ __forceinline__ f32x4 sum_rows(const float* __restrict__ p, int64_t pitch, int count, f32x4 a) {
    int k = 0;
    for (; k + 8 <= count; k += 8) {
        f32x4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = ldf4(p + (k + u) * pitch);
#pragma unroll
        for (int u = 0; u < 8; ++u) a = add4(a, x[u]);
    }
    for (; k < count; ++k) a = add4(a, ldf4(p + k * pitch));
    return a;
}
__global__ __launch_bounds__(kGradBlock) void k_fold(const uint32_t* __restrict__ key, GradShape s,
                                                     int64_t step, float* __restrict__ part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c0 = (int64_t)(blockIdx.x / s.col_blocks) * kFold * step;
    const int64_t c = ((int64_t)(blockIdx.x % s.col_blocks) * kGradWaves + wave) * kJoinCols + 4 * lane;
    if (c >= s.pitch || !inside_run(key, s, c0, kFold * step)) return;
    float* p = part + 2 * c0 * s.pitch + c;
    stf4(p, sum_rows(p + 2 * step * s.pitch, 2 * step * s.pitch, kFold - 1, ldf4(p)));
}

// Finishes the runs that start in a chunk and go on past it: the sum of the
// chunk's last partial and of the following chunks' first ones, folded groups
// taken whole.
template <typename G>
__global__ __launch_bounds__(kGradBlock) void k_join(const uint32_t* __restrict__ key, GradShape s,
                                                     int64_t max_step, float c0, G* __restrict__ grad,
                                                     const float* __restrict__ part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t chunk = (int64_t)blockIdx.x / s.col_blocks;
    const int64_t c = ((int64_t)(blockIdx.x % s.col_blocks) * kGradWaves + wave) * kJoinCols + 4 * lane;
    if (c >= s.pitch || chunk + 1 >= s.chunks) return;
    const int64_t s1 = (chunk + 1) * s.K;
    const uint32_t k = key[s1 - 1];
    if (k == s.rows || key[s1] != k) return;                         // ends with its chunk
    if (chunk > 0 && key[chunk * s.K - 1] == k) return;              // started earlier
    int64_t lo = s1, hi = s.n;                                       // the first place past the run
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (key[mid] == k) lo = mid + 1; else hi = mid;
    }
    // The run holds the first tokens of chunks [chunk + 1, end) and all of [chunk + 1, whole).
    const int64_t end = (lo + s.K - 1) / s.K, whole = lo == s.n ? s.chunks : lo / s.K;
    f32x4 a = ldf4(part + (2 * chunk + 1) * s.pitch + c);
    for (int64_t at = chunk + 1; at < end;) {
        int64_t step = max_step;                                     // the largest folded group at `at`
        while (step > 1 && (at % step != 0 || at + step > whole)) step /= kFold;
        int64_t limit = step > 1 ? whole : end;                      // equal steps up to the next larger group
        if (step < max_step && limit > (at / (step * kFold) + 1) * (step * kFold))
            limit = (at / (step * kFold) + 1) * (step * kFold);
        const int64_t count = (limit - at) / step;
        a = sum_rows(part + 2 * at * s.pitch + c, 2 * step * s.pitch, (int)count, a);
        at += count * step;
    }
    const int64_t left = s.dim - c;
    G* p = grad + (int64_t)k * s.dim + c;
    const float v[4] = {a.x * c0, a.y * c0, a.z * c0, a.w * c0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < left) store1(p + j, s.acc ? load1(p + j) + v[j] : v[j]);
}

}  // namespace
