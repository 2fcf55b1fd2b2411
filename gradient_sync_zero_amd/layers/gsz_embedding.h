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
//
// A row is vpr = ceil(dim / 8) vectors.  A lane takes up to look_unroll vectors at fixed
// distances, whose loads are in flight together before the first store; the work per
// vector has to stay near the 20 instructions of widening, scaling and rounding, or the
// VALU and not the memory sets the pace (with each lane finding row and column of
// every vector anew, 64 Ki tokens of 8192 columns took 368 us, and the same reads
// without the stores already 211).
// WIDE (vpr > kLookBlock / 2): the rows of a block are the same for all its lanes; a
// row is cut into column blocks of `width` <= kLookBlock vectors, and a block takes
// 2^wide_log2 of them in each of `per` rows: as much of a row as it can, so that
// blocks in order write memory in order.
// Else a block holds `side` rows side by side, lane t being vector t mod vpr of row
// t / vpr, `per` times; magic = floor(2^32 / vpr) + 1, so (t * magic) >> 32 == t / vpr.
// With dropout a lane takes one vector: the generator's 700 cycles a vector leave the
// memory time, and four generators' code does not fit the instruction cache.
//
// Bound by memory: 64 Ki tokens of 8192 bf16 columns (1.07 GB out, 14,000 distinct rows) in
// 246 us; counters show 1.07 GB written and 0.73 GB fetched, 7.3 TB/s, since the L2s do
// not hold the rows until they come again.  Two ways to have them do so fetched 0.45 GB
// and lost: eight column slices, one for each XCD (281 us: rows in pieces of 2 KB; 13%
// faster where the table's rows lie in the memory-side cache), and each row on the XCD of
// its number (266 us with a token to a block, 296 with several: every block first votes on
// the ids of 64 tokens).  8192 tokens of 768 columns with dropout,
// 18 MB: 8.2 us, the generator and the latency of id, row and store.
constexpr int kLookBlock = 256;
constexpr int look_unroll(bool drop) { return drop ? 1 : 4; }
struct LookShape { int64_t n, dim, tiles; uint64_t magic; int vpr, cols, width, wide_log2, side, per; };

template <typename T, typename O, bool DROP, bool WIDE>
__global__ __launch_bounds__(kLookBlock) void k_lookup(const T* __restrict__ table, Ids ids, LookShape s,
                                                       float c0, DropArgs da, O* __restrict__ out) {
    constexpr int U = look_unroll(DROP);
    DropKey d{};
    if (DROP) d = drop_key(da);
    const int tid = threadIdx.x;
    const int64_t blocks = s.tiles * s.cols;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        int64_t tile = b;
        int v = tid, lr = 0;
        if (WIDE) {
            if (tid >= s.width) return;
            tile = s.cols == 1 ? b : b / s.cols;
            v += ((int)(b - tile * s.cols) << s.wide_log2) * s.width;
        } else {
            lr = (int)(((uint64_t)tid * s.magic) >> 32);
            v -= lr * s.vpr;
            if (lr >= s.side) return;
        }
        const int64_t row0 = tile * (s.side * s.per) + lr;
        // The u-th vector's row and first column.
        auto row_at = [&](int u) -> int64_t { return row0 + (WIDE ? u >> s.wide_log2 : u) * s.side; };
        auto col_at = [&](int u) -> int64_t {
            return 8 * (int64_t)(WIDE ? v + (u & ((1 << s.wide_log2) - 1)) * s.width : v);
        };
        const int vectors = WIDE ? s.per << s.wide_log2 : s.per;
        Raw8<T> r[U];
        bool in[U], is_row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row_at(u), col = col_at(u), left = s.dim - col;
            in[u] = is_row[u] = false;
            if (u >= vectors || row >= s.n) continue;
            uint32_t id = row_of(ids, row);
            if (WIDE) id = __builtin_amdgcn_readfirstlane(id);
            in[u] = left > 0;
            is_row[u] = in[u] && id != ids.rows;
            if (is_row[u]) {
                const T* p = table + (int64_t)id * s.dim + col;
                r[u] = left >= 8 ? load8<false>(p) : load8_part(p, (int)left);
            }
        }
        // The mask needs no data: it is drawn while the load is on its way.  Where a row is
        // not a whole number of generator blocks it comes as bits from two of them.
        uint32_t gone = 0, numbers[8];
        const bool bits = (s.dim & 7) != 0;
        if (DROP) {
            const uint64_t first = (uint64_t)(row_at(0) * s.dim + col_at(0));
            if (bits) gone = dropped8(d, first);
            else drop_numbers(d, first >> 3, numbers);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in[u]) continue;
            float a[8] = {};
            if (is_row[u]) {
                widen(r[u], a);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = a[j] * c0;
                if (DROP) {
                    if (bits) drop8(gone, a);
                    else drop8_at(d, numbers, a);
                }
            }
            const int64_t col = col_at(u), left = s.dim - col;
            O* p = out + row_at(u) * s.dim + col;
            if (left >= 8) store8<true>(p, a);
            else store8_part(p, a, (int)left);
        }
    }
}

// ------------------------------------------------------------- clearing --
//
// With accumulate = 0 the rows without a token are cleared.  No launch does only
// that: the blocks that clear ride along with the sort, whose few blocks leave
// the memory idle.  292 MB in three launches of 17.7 us (5.5 TB/s, the sort's own 4-5 us
// a launch hidden).  Clearing part of it beside the sums instead was 2.5% slower on that
// gradient, 6% faster on one of 508 MB and few tokens.

// Clears the rows r0 + i, i a set bit of `missing`, with `threads` threads: neighbours
// as one stretch of memory in whole 16-byte vectors, whatever the rows' alignment (row by
// row at the rows' own places, 31,000 rows of 4097 fp32 took 210 us, 2.5 TB/s).
template <typename G>
__device__ __forceinline__ void clear_rows(G* __restrict__ grad, int64_t dim, int64_t r0, uint64_t missing,
                                           int thread, int threads) {
    while (missing) {
        const int first = __builtin_ctzll(missing);
        const uint64_t rest = ~(missing >> first);
        const int count = rest ? __builtin_ctzll(rest) : 64;
        missing = first + count >= 64 ? 0 : missing >> (first + count) << (first + count);
        G* p = grad + (r0 + first) * dim;
        const int64_t n = count * dim;
        int64_t head = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(G);
        if (head > n) head = n;
        const int64_t vecs = (n - head) * (int64_t)sizeof(G) / 16;
        u32x4* q = reinterpret_cast<u32x4*>(p + head);
        for (int64_t i = thread; i < vecs; i += threads)
            __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, q + i);
        const int64_t tail = head + vecs * (16 / (int64_t)sizeof(G));
        if (thread < head) p[thread] = 0;
        if (thread < n - tail) p[tail + thread] = 0;
    }
}

constexpr int kSortBlock = 512;                       // of the launches that clear beside the sort

// Which part of the table a launch clears: rows [row0, row1), `per` (at most 64) at a time
// for each of its blocks from `first_block` on.  There is a block for every `per` rows, as
// long as the launch can hold so many; tables of over 10^9 narrow rows take several turns.
struct ClearShape { void* grad; int64_t dim, row0, row1; unsigned first_block; int per, f32; };

// owner[v] is some token of row v, if there is one: k_count stores every token's
// position there, and whichever store lands last is as good as another.  The array
// is never cleared: what it holds counts only if that token does have row v.
__device__ __forceinline__ void clear_block(const ClearShape& c, const Ids& ids, int64_t n,
                                            const uint32_t* __restrict__ owner) {
    const int64_t turn = (int64_t)(gridDim.x - c.first_block) * c.per;
    for (int64_t r0 = c.row0 + (int64_t)(blockIdx.x - c.first_block) * c.per; r0 < c.row1; r0 += turn) {
        const int lane = threadIdx.x & 63;
        const int64_t v = r0 + lane;
        bool missing = lane < c.per && v < c.row1;
        if (missing) {
            const uint32_t i = owner[v];
            missing = !(i < (uint64_t)n && row_of(ids, i) == (uint32_t)v);
        }
        const uint64_t m = __ballot(missing);
        if (c.f32) clear_rows(static_cast<float*>(c.grad), c.dim, r0, m, threadIdx.x, kSortBlock);
        else clear_rows(static_cast<uint16_t*>(c.grad), c.dim, r0, m, threadIdx.x, kSortBlock);
    }
}

// ------------------------------------------------------------------ sort --
//
// The tokens sorted by (row, position): key[s] the s-th row, pos[s] its position;
// tokens without a row sort last with key = rows.

// n <= kRankMax tokens in one launch: token i goes to place
// #{j : key_j < key_i} + #{j < i : key_j == key_i}.  A block holds all keys in LDS
// and places kRankTokens tokens; each half of each wave compares them with a slice of
// the keys.  With PACKED (rows < 2^19) a key and its position are one 32-bit number
// and a comparison is two instructions.  Every block also clears the rows without a
// token among clear.per * 64 rows, which it finds among the keys it holds.
// kRankMax is what the LDS holds well; up to there this sort beats the counting passes in
// every call measured: added into 2048 fp32 columns 256 tokens take 13.4 us against 24.9,
// 2048 17.6 against 25.6, 6000 29.1 against 38.9, 8192 34.5 against 37.7; written whole
// with dropout (768 columns) 1024 take 28.2 against 33.0, 8192 36.3 against 40.2.
constexpr int kRankMax = 8192, kRankBits = 13, kRankBlock = 1024, kRankTokens = 32;
constexpr int kRankSlices = kRankBlock / kRankTokens;
constexpr int64_t kRankPackedRows = (int64_t)1 << (32 - kRankBits);
template <bool PACKED>
__global__ __launch_bounds__(kRankBlock) void k_rank(Ids ids, int n, uint32_t* __restrict__ key,
                                                     uint32_t* __restrict__ pos, ClearShape clear) {
    __shared__ __align__(16) uint32_t all[kRankMax];
    __shared__ uint32_t part[kRankSlices][kRankTokens + 1];
    __shared__ uint32_t seen[64][2];
    const int tid = threadIdx.x;
    const int quads = (n + 4 * kRankSlices - 1) / (4 * kRankSlices) * kRankSlices;
    {
        uint32_t k[kRankMax / kRankBlock];            // the loads in flight together
#pragma unroll
        for (int u = 0; u < kRankMax / kRankBlock; ++u) {
            const int j = tid + u * kRankBlock;
            k[u] = j < n ? row_of(ids, j) : 0;
        }
#pragma unroll
        for (int u = 0; u < kRankMax / kRankBlock; ++u) {
            const int j = tid + u * kRankBlock;
            if (j < 4 * quads) all[j] = j >= n ? 0xFFFFFFFFu : PACKED ? k[u] << kRankBits | (uint32_t)j : k[u];
        }
    }
    if (tid < 128) seen[tid >> 1][tid & 1] = 0;
    __syncthreads();
    // The stores that clear leave first and land while the block compares keys.  Each wave
    // has a sixteenth of the block's rows (clear.per is a power of two).
    if (clear.grad) {
        const int64_t r0 = (int64_t)blockIdx.x * clear.per * 64;
        for (int j = tid; j < n; j += kRankBlock) {
            const int64_t v = (int64_t)(PACKED ? all[j] >> kRankBits : all[j]) - r0;
            if (v >= 0 && v < (int64_t)clear.per * 64) atomicOr(&seen[v >> 6][v >> 5 & 1], 1u << (v & 31));
        }
        __syncthreads();
        const int share = clear.per * 64 / (kRankBlock / 64), first = (tid >> 6) * share;
        for (int at = first; at < first + share; at += 64) {
            const int64_t r = r0 + at, left = clear.row1 - r;
            if (left <= 0) break;
            uint64_t m = ~((uint64_t)seen[at >> 6][1] << 32 | seen[at >> 6][0]) >> (at & 63);
            const int64_t most = left < share ? left : share;
            if (most < 64) m &= ((uint64_t)1 << most) - 1;
            if (clear.f32) clear_rows(static_cast<float*>(clear.grad), clear.dim, r, m, tid & 63, 64);
            else clear_rows(static_cast<uint16_t*>(clear.grad), clear.dim, r, m, tid & 63, 64);
        }
    }
    const int t = tid % kRankTokens, slice = tid / kRankTokens;
    const int i = blockIdx.x * kRankTokens + t;
    if ((int64_t)blockIdx.x * kRankTokens < n) {
        const uint32_t mine = i < n ? all[i] : 0;
        const u32x4* all4 = reinterpret_cast<const u32x4*>(all);
        uint32_t less = 0;
#pragma unroll 4
        for (int q = slice; q < quads; q += kRankSlices) {
            const u32x4 k = all4[q];
            if (PACKED) {
                less += k.x < mine;
                less += k.y < mine;
                less += k.z < mine;
                less += k.w < mine;
            } else {
                const int j = 4 * q;
                less += (k.x < mine) | ((k.x == mine) & (j < i));
                less += (k.y < mine) | ((k.y == mine) & (j + 1 < i));
                less += (k.z < mine) | ((k.z == mine) & (j + 2 < i));
                less += (k.w < mine) | ((k.w == mine) & (j + 3 < i));
            }
        }
        part[slice][t] = less;
        __syncthreads();
        if (slice == 0 && i < n) {
            uint32_t s = 0;
#pragma unroll
            for (int w = 0; w < kRankSlices; ++w) s += part[w][t];
            key[s] = PACKED ? mine >> kRankBits : mine;
            pos[s] = (uint32_t)i;
        }
    }
}

// More tokens: stable counting passes over digits of the key, lowest first, a launch
// to count and one to place each.  count[tile][digit]: how often a digit occurs in a
// tile of `rounds` times kSortTile tokens.  64 Ki tokens in four launches of 3.4 to 5 us,
// all latency; tiles of 512 tokens, one per work-item, beat 1024 of four (16 Ki tokens 3 us
// slower, for want of blocks) and 256 (more counts to add up).  Counting the next digit
// while placing this one, with an atomic per token where it lands, saved a launch and cost
// 10 us of atomics on 16 Ki tokens.
constexpr int kSortWaves = kSortBlock / 64, kSortMaxBins = 1024;
constexpr int kSortTile = kSortBlock;
constexpr int kSortBinsPer = kSortMaxBins / kSortBlock;
struct SortPass {
    Ids ids;                              // the tokens themselves (FIRST),
    const uint32_t* key_in;               // or sorted pairs
    const uint32_t* pos_in;
    int64_t n, rounds;
    int tiles, shift, bins;               // bins a power of two
};
__device__ __forceinline__ uint32_t digit_of(const SortPass& s, uint32_t key) {
    return (key >> s.shift) & (uint32_t)(s.bins - 1);
}
// Orders a wave's LDS accesses for the compiler (the hardware keeps them in order).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// FIRST also notes a token of each row in owner (if there is one to note in).
template <bool FIRST>
__global__ __launch_bounds__(kSortBlock) void k_count(SortPass s, uint32_t* __restrict__ count,
                                                      uint32_t* __restrict__ owner, ClearShape clear) {
    if (!FIRST && blockIdx.x >= clear.first_block) return clear_block(clear, s.ids, s.n, owner);
    __shared__ uint32_t h[kSortMaxBins];
    for (int b = threadIdx.x; b < s.bins; b += kSortBlock) h[b] = 0;
    __syncthreads();
    for (int64_t r = 0; r < s.rounds; ++r) {
        const int64_t i = (blockIdx.x * s.rounds + r) * kSortTile + threadIdx.x;
        if (i >= s.n) continue;
        const uint32_t k = FIRST ? row_of(s.ids, i) : s.key_in[i];
        atomicAdd(&h[digit_of(s, k)], 1u);
        if (FIRST && owner && k != s.ids.rows) owner[k] = (uint32_t)i;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < s.bins; b += kSortBlock) count[(int64_t)blockIdx.x * s.bins + b] = h[b];
}

// Moves the tokens of one tile to their places by one digit.  The block sums the
// digit counts of all tiles for its bases; in each round wave w counts its 64 tokens, then
// places them in order from its own bases.
template <bool FIRST>
__global__ __launch_bounds__(kSortBlock) void k_place(SortPass s, const uint32_t* __restrict__ count,
                                                      uint32_t* __restrict__ key, uint32_t* __restrict__ pos,
                                                      const uint32_t* __restrict__ owner, ClearShape clear) {
    if (blockIdx.x >= clear.first_block) return clear_block(clear, s.ids, s.n, owner);
    __shared__ uint32_t base[kSortWaves][kSortMaxBins];
    __shared__ uint32_t next[kSortMaxBins];          // the tile's next place for each digit
    __shared__ uint32_t sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // Thread t sums the digits t, t + kSortBlock, ...: over all tiles, and over
    // those before this one.
    uint32_t before[kSortBinsPer];
    uint32_t carry = 0;
#pragma unroll
    for (int k = 0; k < kSortBinsPer; ++k) {
        if (k * kSortBlock >= s.bins) continue;
        const int b = k * kSortBlock + tid;
        uint32_t all = 0, prior = 0;
        if (b < s.bins) {
#pragma unroll 16
            for (int t = 0; t < s.tiles; ++t) {
                const uint32_t c = count[(int64_t)t * s.bins + b];
                all += c;
                prior += t < (int)blockIdx.x ? c : 0;
            }
        }
        before[k] = prior;
        uint32_t incl = all;                          // inclusive sum over the wave's digits
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t x = __shfl_up(incl, o);
            incl += lane >= o ? x : 0;
        }
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        uint32_t at = carry + incl - all + before[k];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) at += sums[w];
            carry += sums[w];
        }
        if (b < s.bins) next[b] = at;
        __syncthreads();
    }
    for (int64_t r = 0; r < s.rounds; ++r) {
        const int64_t i = (blockIdx.x * s.rounds + r) * kSortTile + tid;
        const bool in = i < s.n;
        uint32_t k = 0, p = 0;
        if (in) {
            k = FIRST ? row_of(s.ids, i) : s.key_in[i];
            p = FIRST ? (uint32_t)i : s.pos_in[i];
        }
        const uint32_t dg = digit_of(s, k);
        for (int b = lane; b < s.bins; b += 64) base[wave][b] = 0;
        wave_fence();
        if (in) atomicAdd(&base[wave][dg], 1u);
        __syncthreads();
        for (int b = tid; b < s.bins; b += kSortBlock) {
            uint32_t at = next[b];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = base[w][b];
                base[w][b] = at;
                at += c;
            }
            next[b] = at;
        }
        __syncthreads();
        uint64_t same = __ballot(in);                 // the lanes with this one's digit
        for (int bit = 1; bit < s.bins; bit <<= 1) {
            const uint64_t m = __ballot((dg & bit) != 0);
            same &= (dg & bit) ? m : ~m;
        }
        if (in) {
            const uint32_t at = base[wave][dg] + __popcll(same & (((uint64_t)1 << lane) - 1));
            key[at] = k;
            pos[at] = p;
        }
        wave_fence();                                 // before the next round clears base
    }
}

// -------------------------------------------------------------- gradient --
//
// grad[v, c] = (old or 0) + c0 * sum of the kept dy[pos, c] over v's tokens.
//
// The sorted tokens are cut into chunks of K; one wave sums the runs of equal rows
// of one chunk over one tile of columns, in fp32, positions rising.  A run that
// starts in a chunk and ends at most K tokens past it is finished by that chunk's
// wave (the next chunk's skips it): without that, most chunks of a Zipf-like text would
// end inside a run and write and read two fp32 rows more.  A longer run leaves an fp32
// partial sum per chunk, part[2c + 1] where it starts in chunk c and part[2c] where it
// came from an earlier one; k_join adds them in chunk order.
//
// Bound by memory, rows of dy read in the tokens' order and not their own: 64 Ki tokens of
// 8192 bf16 columns, 1.07 GB read and 0.26 GB written, in 253 us (5.3 TB/s); 16 Ki tokens
// of 2048 added into fp32 in 35 us (0.18 GB by the counters, 5.0 TB/s).  One wave per block and four rows in flight beat four waves by
// 2-5% and eight rows by 0-4%.

constexpr int kGradBlock = 64, kGradCols = kTile, kGradUnroll = 4;
constexpr int kMaxChunk = 32;                         // a wave holds 2 K keys

struct GradShape {
    int64_t dim, pitch;                  // pitch: floats of a partial row, a multiple of 8
    int64_t n, chunks;
    uint32_t rows;
    int K, tiles;                        // tiles of columns
    int nt;                              // dy is read nontemporally
};

// The tokens [first, last) of a wave's chunk: lane l holds token l's key and position.
struct GradWave { int64_t chunk, c, left; int first, last; bool head_part, tail_part; uint32_t key, pos; };

template <typename T, typename G, bool ACC, bool DROP, bool FULL, bool NT>
__device__ __forceinline__ void grad_wave(const T* __restrict__ dy, const GradShape& s, GradWave w, float c0,
                                          const DropKey& d, G* __restrict__ grad, float* __restrict__ part) {
    float sum[8] = {};
    for (int t = w.first; t < w.last; t += kGradUnroll) {
        RowPiece<T> r[kGradUnroll];
        float old[ACC ? kGradUnroll : 1][8];
        uint32_t kk[kGradUnroll];
        bool ends[kGradUnroll];
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const int at = t + u < w.last ? t + u : w.last - 1;
            kk[u] = __builtin_amdgcn_readlane(w.key, at);
            const uint32_t p = __builtin_amdgcn_readlane(w.pos, at);
            ends[u] = at + 1 == w.last || (uint32_t)__builtin_amdgcn_readlane(w.key, at + 1) != kk[u];
            if (t + u < w.last) {
                const T* row = dy + (int64_t)p * s.dim + w.c;
                r[u] = load_row<FULL, NT>(row, w.left);
            }
            if (ACC && t + u < w.last && ends[u])
                load_old<T, FULL>(grad + (int64_t)kk[u] * s.dim + w.c, w.left, old[u]);
        }
        uint32_t gone = 0;                                           // 8 bits for each u
        if (DROP) {
#pragma unroll 1
            for (int u = 0; u < kGradUnroll && t + u < w.last; ++u) {
                const uint32_t p = __builtin_amdgcn_readlane(w.pos, t + u);
                gone |= dropped_row<T>(d, (uint64_t)p * (uint64_t)s.dim + (uint64_t)w.c) << 8 * u;
            }
        }
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            if (t + u >= w.last) break;
            float a[8];
            widen_row(r[u], a);
            if (DROP) drop8(gone >> 8 * u, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = sum[j] + a[j];
            if (!ends[u]) continue;
            if (w.head_part || (w.tail_part && t + u + 1 == w.last)) {
                store_row<T, FULL, false>(part + (2 * w.chunk + (w.head_part ? 0 : 1)) * s.pitch + w.c, s.pitch - w.c, sum);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[j] = sum[j] * c0;
                    if (ACC) a[j] = old[ACC ? u : 0][j] + a[j];
                }
                store_row<T, FULL, NT && !ACC>(grad + (int64_t)kk[u] * s.dim + w.c, w.left, a);
            }
            w.head_part = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
        }
    }
}

template <typename T, typename G, bool ACC, bool DROP>
__global__ __launch_bounds__(kGradBlock) void k_grad(const T* __restrict__ dy, const uint32_t* __restrict__ key,
                                                     const uint32_t* __restrict__ pos, GradShape s,
                                                     float c0, DropArgs da, G* __restrict__ grad,
                                                     float* __restrict__ part) {
    const int lane = threadIdx.x & 63;
    const int64_t chunk = (int64_t)blockIdx.x / s.tiles;
    if (chunk >= s.chunks) return;
    const int64_t c = ((int64_t)blockIdx.x - chunk * s.tiles) * kGradCols;
    const int64_t s0 = chunk * s.K, s1 = s0 + s.K;
    // Lane l holds the key and position of token s0 + l, l < 2 K.
    uint32_t my_key = s.rows, my_pos = 0;
    if (lane < 2 * s.K && s0 + lane < s.n) { my_key = key[s0 + lane]; my_pos = pos[s0 + lane]; }
    const uint32_t none = 0xFFFFFFFFu;                               // no row's number
    const uint32_t before = s0 > 0 ? key[s0 - 1] : none, long_before = s0 > s.K ? key[s0 - s.K - 1] : none;
    const uint32_t past = s1 + s.K < s.n ? key[s1 + s.K] : none;
    const uint32_t k_first = __builtin_amdgcn_readlane(my_key, 0), k_last = __builtin_amdgcn_readlane(my_key, s.K - 1);
    const uint32_t k_next = __builtin_amdgcn_readlane(my_key, s.K);
    GradWave w{chunk, c, s.dim - c, 0, (int)__popcll(__ballot(lane < s.K && my_key != s.rows)), false, false, my_key, my_pos};
    if (k_first == before) {                                         // a run goes on from the last chunk
        if (long_before != k_first && k_next != k_first)             // that chunk finishes it
            w.first = __popcll(__ballot(lane < s.K && my_key == k_first));
        else w.head_part = true;
    }
    if (k_last == k_next && s.K == w.last) {                         // a run goes on into the next
        if (k_last != before && past != k_last) w.last += __popcll(__ballot(lane >= s.K && my_key == k_last));
        else w.tail_part = k_last != before;
    }
    if (w.first >= w.last) return;
    DropKey d{};
    if (DROP) d = drop_key(da);
    if (w.left < kGradCols) grad_wave<T, G, ACC, DROP, false, false>(dy, s, w, c0, d, grad, part);
    else if (s.nt) grad_wave<T, G, ACC, DROP, true, true>(dy, s, w, c0, d, grad, part);
    else grad_wave<T, G, ACC, DROP, true, false>(dy, s, w, c0, d, grad, part);
}

// Finishes the runs that k_grad left in parts.  A block looks at kJoinChunks chunks and takes
// kJoinCols columns of the runs that start in one of them and leave a tail part: a run
// of at most kJoinWaves parts is one wave's, a longer one the block's, each wave
// summing a stretch of its parts and the first wave those sums, all in order.  5.5 to 14 us,
// the latency of keys, parts and row; blocks of 1024 over 64 chunks took 19 where these
// take 14.
constexpr int kJoinBlock = 512, kJoinWaves = kJoinBlock / 64, kJoinCols = 256, kJoinChunks = 32;
// a + part rows [k, end) of the run that starts in `chunk`, at the lane's columns.
__device__ __forceinline__ f32x4 sum_parts(const float* __restrict__ part, int64_t pitch, int64_t chunk,
                                           int64_t k, int64_t end) {
    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
    auto row = [&](int64_t i) { return ldf4(part + (2 * (chunk + i) + (i == 0)) * pitch); };
    for (; k + 8 <= end; k += 8) {
        f32x4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = row(k + u);
#pragma unroll
        for (int u = 0; u < 8; ++u) a = add4(a, x[u]);
    }
    for (; k < end; ++k) a = add4(a, row(k));
    return a;
}
template <typename G, bool ACC>
__global__ __launch_bounds__(kJoinBlock) void k_join(const uint32_t* __restrict__ key, GradShape s, int tiles,
                                                     float c0, G* __restrict__ grad,
                                                     const float* __restrict__ part) {
    __shared__ f32x4 sums[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t g = (int64_t)blockIdx.x / tiles, c0l = ((int64_t)blockIdx.x % tiles) * kJoinCols;
    const int64_t c = c0l + 4 * lane, cp = c < s.pitch ? c : 0;        // lanes past the row read its start
    const int64_t mine = g * kJoinChunks + lane, e = (mine + 1) * s.K;        // this lane's chunk and its end
    uint32_t k = s.rows;
    bool starts = false, inside = false;                             // a run starts here, or comes from before;
    if (mine < s.chunks && e < s.n) {                                // either way it goes on into the next chunk
        k = key[e - 1];
        const uint32_t next = key[e], before = mine > 0 ? key[e - s.K - 1] : 0xFFFFFFFFu;
        const uint32_t past = e + s.K < s.n ? key[e + s.K] : 0xFFFFFFFFu;
        const bool on = k != s.rows && k == next;
        starts = lane < kJoinChunks && on && k != before && k == past;
        inside = on && k == before;
    }
    const uint64_t through = __ballot(inside);
    int order = 0;
    for (uint64_t m = __ballot(starts); m; m &= m - 1, ++order) {
        const int l = __builtin_ctzll(m);
        const uint32_t row = __builtin_amdgcn_readlane(k, l);
        const int64_t chunk = g * kJoinChunks + l;
        // The chunks of the run: this one, those that it passes through, its last.
        const uint64_t ends = l < 63 ? ~through >> (l + 1) << (l + 1) : 0;
        int64_t parts = (ends ? __builtin_ctzll(ends) : 64) - l + 1;
        while (!ends) {                                              // on past the 64 chunks
            const int64_t j = chunk + parts + lane;
            const uint64_t on = __ballot(j < s.chunks && key[j < s.chunks ? j * s.K : 0] == row);
            const int more = ~on ? __builtin_ctzll(~on) : 64;
            parts += more;
            if (more < 64) break;
        }
        f32x4 a;
        if (parts <= kJoinWaves) {
            if (order % kJoinWaves != wave) continue;
            a = sum_parts(part + cp, s.pitch, chunk, 0, parts);
        } else {
            sums[wave][lane] = sum_parts(part + cp, s.pitch, chunk, parts * wave / kJoinWaves, parts * (wave + 1) / kJoinWaves);
            __syncthreads();
            if (wave == 0) {
                a = sums[0][lane];
                for (int w = 1; w < kJoinWaves; ++w) a = add4(a, sums[w][lane]);
            }
            __syncthreads();
            if (wave != 0) continue;
        }
        float v[4] = {a.x * c0, a.y * c0, a.z * c0, a.w * c0};
        G* p = grad + (int64_t)row * s.dim + c;
        const int64_t left = s.dim - c;
        if (left >= 4) {
            if (ACC) {
                float o[4];
                load4(p, o);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = o[j] + v[j];
            }
            store4<false>(p, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) store1(p + j, ACC ? load1(p + j) + v[j] : v[j]);
        }
    }
}

// ---------------------------------------------------- a few tokens at once --

// n <= kDirectMax tokens in one launch without a sort (64 tokens of 8192 columns added into
// fp32 in 3.8 us; a call of 128 tokens of 4096 columns 7.0 us against 13.2 by sort, sums
// and join, and 17 against 13 where nine in ten are one row's): the wave of (token, tile
// of columns) ends if its row came earlier, else it sums the tokens of its row in order.
// The rule takes no account of the ids, which only the device knows: tokens of one row
// are the dearest here and rare.
// Blocks from clear.first_block on clear the rows that no token has (32,000 rows of 4096
// bf16 columns around 1 to 128 tokens, nine in ten of one row or not, 49 us: 5.3 TB/s).
constexpr int kDirectMax = 128, kDirectUnroll = 8;
template <typename T, typename G, bool ACC, bool DROP>
__global__ __launch_bounds__(kGradBlock) void k_direct(const T* __restrict__ dy, Ids ids, GradShape s, float c0,
                                                       DropArgs da, G* __restrict__ grad, ClearShape clear) {
    const int lane = threadIdx.x & 63;
    const uint32_t k0 = lane < s.n ? row_of(ids, lane) : s.rows, k1 = lane + 64 < s.n ? row_of(ids, lane + 64) : s.rows;
    if (!ACC && blockIdx.x >= clear.first_block) {
        const int64_t turn = (int64_t)(gridDim.x - clear.first_block) * clear.per;
        for (int64_t r0 = (int64_t)(blockIdx.x - clear.first_block) * clear.per; r0 < clear.row1; r0 += turn) {
            const int64_t v = r0 + lane;
            bool missing = lane < clear.per && v < clear.row1;
            for (int j = 0; j < 64; ++j) {
                if ((uint32_t)__builtin_amdgcn_readlane(k0, j) == (uint64_t)v) missing = false;
                if ((uint32_t)__builtin_amdgcn_readlane(k1, j) == (uint64_t)v) missing = false;
            }
            clear_rows(grad, s.dim, r0, __ballot(missing), threadIdx.x, kGradBlock);
        }
        return;
    }
    const int i = (int)((int64_t)blockIdx.x / s.tiles);
    if (i >= s.n) return;
    const int64_t c = ((int64_t)blockIdx.x - (int64_t)i * s.tiles) * kGradCols, left = s.dim - c;
    const uint32_t mine = i < 64 ? __builtin_amdgcn_readlane(k0, i) : __builtin_amdgcn_readlane(k1, i - 64);
    uint64_t m0 = __ballot(k0 == mine), m1 = __ballot(k1 == mine);
    if (mine == s.rows || (m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(m1)) != i) return;
    DropKey d{};
    if (DROP) d = drop_key(da);
    float sum[8] = {}, old[8];
    if (ACC) load_old<T, false>(grad + (int64_t)mine * s.dim + c, left, old);
    while (m0 | m1) {
        uint64_t n0 = m0, n1 = m1;                    // the same tokens once more, for their masks
        RowPiece<T> r[kDirectUnroll];
        int at[kDirectUnroll];
#pragma unroll
        for (int u = 0; u < kDirectUnroll; ++u) {
            at[u] = -1;
            if (m0) { at[u] = __builtin_ctzll(m0); m0 &= m0 - 1; }
            else if (m1) { at[u] = 64 + __builtin_ctzll(m1); m1 &= m1 - 1; }
            if (at[u] >= 0) r[u] = load_row<false, false>(dy + (int64_t)at[u] * s.dim + c, left);
        }
        uint64_t gone = 0;
        if (DROP) {
#pragma unroll 1
            for (int u = 0; u < kDirectUnroll && (n0 | n1); ++u) {
                const int p = n0 ? __builtin_ctzll(n0) : 64 + __builtin_ctzll(n1);
                if (n0) n0 &= n0 - 1; else n1 &= n1 - 1;
                gone |= (uint64_t)dropped_row<T>(d, (uint64_t)p * (uint64_t)s.dim + (uint64_t)c) << 8 * u;
            }
        }
#pragma unroll
        for (int u = 0; u < kDirectUnroll; ++u) {
            if (at[u] < 0) break;
            float a[8];
            widen_row(r[u], a);
            if (DROP) drop8((uint32_t)(gone >> 8 * u), a);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = sum[j] + a[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sum[j] = sum[j] * c0;
        if (ACC) sum[j] = old[j] + sum[j];
    }
    store_row<T, false, false>(grad + (int64_t)mine * s.dim + c, left, sum);
}

}  // namespace
