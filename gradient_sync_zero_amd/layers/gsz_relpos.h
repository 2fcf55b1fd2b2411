// Learned relative position bias: a table of one value per bucket of distances and head,
// added to attention scores, and its gradient.
//
// The bias of (i, j) depends on the distance d = j - i - start alone, so a head's values are
// a line over the diagonals, and each row of scores reads a stretch of it that begins one
// place further left than the row's above.  Both kernels give each lane eight neighbours of
// a row and go down the rows: the bias keeps a window of the line in registers and takes
// one new value a row, the gradient keeps eight diagonals' sums in registers and lets its loads
// move one column a row.  Buckets are intervals of distances: they are looked up once a
// diagonal and tile, never per score.
#pragma once

#include "gsz_dropout.h"

#pragma clang fp contract(off)

namespace {

constexpr int kRelBuckets = 256, kRelBlock = 256;

// first[b]: the smallest distance of bucket b of one direction, non-decreasing; distances from
// first[b] to first[b + 1] - 1 are bucket b's (none where the two are equal), the last one's all
// from first[n - 1].
struct RelMap { int32_t first[kRelBuckets]; int n, both; };

// Where the first query of sequence b stands among the keys.
struct RelStart {
    const void* per;                                 // a number a sequence, or NULL
    int wide;                                        // they are 64 bits wide
    int64_t all;
    __device__ int64_t of(int64_t b) const {
        if (!per) return all;
        const int64_t s = wide ? static_cast<const int64_t*>(per)[b] : static_cast<const int32_t*>(per)[b];
        constexpr int64_t kFar = (int64_t)1 << 40;   // beyond any bucket: keeps sums of places in range
        return s < -kFar ? -kFar : s > kFar ? kFar : s;
    }
};

// The bucket of distance d; first: the map's borders in LDS.
__device__ __forceinline__ int rel_bucket(const int32_t* first, int n, int both, int64_t d) {
    const int64_t a = d > 0 ? (both ? d : 0) : -d;
    const int32_t dist = (int32_t)(a > 0x7FFFFFFF ? 0x7FFFFFFF : a);
    int lo = 0, hi = n - 1;                          // the last bucket that begins at or below dist
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= dist) lo = mid; else hi = mid - 1;
    }
    return both && d > 0 ? lo + n : lo;
}
__device__ __forceinline__ void stage_map(const RelMap& m, int32_t* first) {
    for (int b = threadIdx.x; b < m.n; b += blockDim.x) first[b] = m.first[b];
}

// ------------------------------------------------------------------ bias --

// A tile is `rows` rows by 8 `lanes` columns of one (sequence, head); a block's work-items are
// `lanes` across and `groups` down, each with `per` rows one below the other.
struct BiasShape { int64_t tiles, q, k; int heads, lanes, groups, per, rows, down, across; };
constexpr int kBiasStrip = 8 * kRelBlock + 1024;     // columns + rows of a tile

template <typename T, typename O, bool ADD>
__global__ __launch_bounds__(kRelBlock) void k_relpos_bias(const T* table, RelMap map, RelStart start, BiasShape s, float scale,
                                                           const O* add, O* out) {
    __shared__ int32_t first[kRelBuckets];
    __shared__ float strip[kBiasStrip];
    stage_map(map, first);
    const int x = threadIdx.x % s.lanes, y = threadIdx.x / s.lanes;
    for (int64_t t = blockIdx.x; t < s.tiles; t += gridDim.x) {
        int64_t r = t;
        const int64_t c0 = r % s.across * s.lanes * 8;
        r /= s.across;
        const int64_t i0 = r % s.down * s.rows;
        r /= s.down;
        const int head = (int)(r % s.heads);
        const int64_t d0 = c0 - (i0 + s.rows - 1) - start.of(r / s.heads);
        __syncthreads();                             // the strip's last readers are done, the map is there
        for (int v = threadIdx.x; v < s.rows - 1 + 8 * s.lanes; v += blockDim.x)
            strip[v] = load1(table + (int64_t)rel_bucket(first, map.n, map.both, d0 + v) * s.heads + head) * scale;
        __syncthreads();
        const int64_t col = c0 + 8 * x, left = s.k - col;
        const int first_row = y * s.per;
        if (y >= s.groups || left <= 0) continue;
        const int64_t most = s.q - i0 - first_row;
        const int rows = (int)(most < s.per ? most : s.per);
        const int64_t at = (r * s.q + i0 + first_row) * s.k + col;
        const int place = s.rows - 1 - first_row + 8 * x;      // of the first row's first value
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = strip[place + j];
        const O* pa = ADD ? add + at : nullptr;
        O* po = out + at;
        // the window turns: after n rows its first value is w[-n mod 8]
        int n = 0;
        if (left >= 8) {
            for (; n + 8 <= rows; n += 8) {
                Raw8<O> old[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) if (ADD) old[m] = load8<false>(pa + (int64_t)(n + m) * s.k);
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    if (m) w[8 - m] = strip[place - n - m];
                    else if (n) w[0] = strip[place - n];
                    float v[8], a[8];
                    if (ADD) widen(old[m], a);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = ADD ? a[j] + w[(8 - m + j) & 7] : w[(8 - m + j) & 7];
                    store8<false>(po + (int64_t)(n + m) * s.k, v);
                }
            }
        }
        for (; n < rows; ++n) {
            float v[8], a[8];
            if (ADD) widen(load8_part(pa + (int64_t)n * s.k, (int)(left < 8 ? left : 8)), a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float b = strip[place - n + j];
                v[j] = ADD ? a[j] + b : b;
            }
            store8_part(po + (int64_t)n * s.k, v, (int)(left < 8 ? left : 8));
        }
    }
}

// -------------------------------------------------------------- gradient --

// A tile is `rows` rows of one (sequence, head) and 8 `lanes` of the diagonals that cross
// them; work-items as above.  partial[(head * buckets + b) * tiles of a head + tile]: the tile's sum
// of bucket b.
struct RelGradShape { int64_t tiles, per_head, q, k; int heads, buckets, lanes, groups, per, rows, down, across; };

// Adds the eight values of a row from column c on that are in the row.
template <typename T>
__device__ __forceinline__ void add_part(const T* row, int64_t c, int64_t k, float sum[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) if (c + j >= 0 && c + j < k) sum[j] = sum[j] + load1(row + c + j);
}

template <typename T>
__global__ __launch_bounds__(kRelBlock) void k_relpos_grad(const T* dy, RelMap map, RelStart start, RelGradShape s, float* partial) {
    __shared__ int32_t first[kRelBuckets];
    __shared__ float strip[8 * kRelBlock];
    stage_map(map, first);
    const int x = threadIdx.x % s.lanes, y = threadIdx.x / s.lanes;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int width = 8 * s.lanes;
    for (int64_t t = blockIdx.x; t < s.tiles; t += gridDim.x) {
        int64_t r = t;
        const int64_t across = r % s.across;
        r /= s.across;
        const int64_t i0 = r % s.down * s.rows;
        const int64_t down = r % s.down;
        r /= s.down;
        const int head = (int)(r % s.heads);
        const int64_t b = r / s.heads;
        const int64_t d0 = across * width - (i0 + s.rows - 1);        // the tile's first j - i
        __syncthreads();                             // the strip's last readers are done, the map is there
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
        if (y < s.groups) {
            const int64_t i = i0 + y * s.per, end = s.q - i0 < s.rows ? s.q - i0 : s.rows, most = end - y * s.per;
            const int rows = (int)(most < 0 ? 0 : most < s.per ? most : s.per);
            const T* row = dy + (r * s.q + i) * s.k;
            int64_t c = d0 + 8 * x + i;                               // the row's column of the lane's first diagonal
            int n = 0;
            for (; n + 8 <= rows; n += 8, c += 8, row += 8 * s.k) {
                if (c >= 0 && c + 15 <= s.k) {
                    Raw8<T> v[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) v[m] = load8<true>(row + m * s.k + c + m);
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        float a[8];
                        widen(v[m], a);
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[j] = sum[j] + a[j];
                    }
                } else if (c + 15 > 0 && c < s.k) {
                    for (int m = 0; m < 8; ++m) add_part(row + m * s.k, c + m, s.k, sum);
                }
            }
            for (; n < rows; ++n, ++c, row += s.k) add_part(row, c, s.k, sum);
#pragma unroll
            for (int j = 0; j < 8; ++j) strip[y * width + 8 * x + j] = sum[j];
        }
        __syncthreads();
        // a wave a bucket: the sums of its diagonals, an interval of the tile's
        const int64_t d1 = d0 - start.of(b);                          // distance of the tile's first diagonal
        for (int k = wave; k < s.buckets; k += waves) {
            const bool ahead = map.both && k >= map.n;
            const int f = ahead ? k - map.n : k;
            const int64_t near = first[f], far = f + 1 < map.n ? first[f + 1] : (int64_t)1 << 62;   // distances [near, far)
            int64_t lo, hi;                                           // distances with sign, [lo, hi)
            if (ahead) { lo = near > 1 ? near : 1; hi = far; }
            else { lo = 1 - far; hi = !map.both && near == 0 && far > 0 ? (int64_t)1 << 62 : 1 - near; }
            lo -= d1;
            hi -= d1;
            const int from = (int)(lo < 0 ? 0 : lo > width ? width : lo), to = (int)(hi < 0 ? 0 : hi > width ? width : hi);
            float total = 0.0f;
            for (int g = 0; g < s.groups; ++g)
                for (int v = from + lane; v < to; v += 64) total = total + strip[g * width + v];
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) total = total + __uint_as_float(__shfl_xor(__float_as_uint(total), o));
            if (lane == 0) partial[((int64_t)head * s.buckets + k) * s.per_head + (b * s.down + down) * s.across + across] = total;
        }
    }
}

// grad[b, head] = (grad[b, head] or 0) + scale * the sum of its partial sums: a wave each, in fp64.
template <typename G, bool ACC>
__global__ __launch_bounds__(64) void k_relpos_join(const float* partial, int64_t per_head, int buckets, int heads, double scale, G* grad) {
    const int64_t cells = (int64_t)buckets * heads;
    for (int64_t cell = blockIdx.x; cell < cells; cell += gridDim.x) {       // head * buckets + bucket
        const float* p = partial + cell * per_head;
        double total = 0.0;
        for (int64_t t = threadIdx.x; t < per_head; t += 64) total = total + (double)p[t];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) total = total + __shfl_xor(total, o);
        if (threadIdx.x == 0) {
            G* to = grad + cell % buckets * heads + cell / buckets;
            store1(to, (float)(scale * total + (ACC ? (double)load1(to) : 0.0)));
        }
    }
}

}  // namespace
