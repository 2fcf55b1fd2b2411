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
// top: the largest power of two below n.
struct RelMap { int32_t first[kRelBuckets]; int n, both, top; };

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

// The buckets of N distances d, d + step ...; first: the map's borders in LDS.  The search takes the
// same steps for all, so that their reads are under way together.
template <int N>
__device__ __forceinline__ void rel_buckets(const int32_t* first, const RelMap& map, int64_t d, int step, int out[N]) {
    int32_t dist[N];
    bool ahead[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int64_t e = d + (int64_t)j * step, a = e > 0 ? (map.both ? e : 0) : -e;
        ahead[j] = map.both && e > 0;
        dist[j] = (int32_t)(a > 0x7FFFFFFF ? 0x7FFFFFFF : a);
        out[j] = 0;                                  // the last bucket that begins at or below dist
    }
    for (int half = map.top; half > 0; half >>= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int mid = out[j] + half;
            if (mid < map.n && first[mid] <= dist[j]) out[j] = mid;
        }
#pragma unroll
    for (int j = 0; j < N; ++j) if (ahead[j]) out[j] += map.n;
}
__device__ __forceinline__ void stage_map(const RelMap& m, int32_t* first) {
    for (int b = threadIdx.x; b < m.n; b += blockDim.x) first[b] = m.first[b];
}

// ------------------------------------------------------------------ bias --

// A lane takes the values of 16 bytes of a row (8 bf16 or 4 fp32: neighbouring lanes then write
// whole lines; 8 fp32 a lane, two stores of 16 bytes, took 37 to 58 us where this takes 31).  A
// tile is `rows` rows by that many times `lanes` columns of one (sequence, head); a block's work-items
// are `lanes` across and `groups` down, each with `per` rows one below the other.
//
// The head's bias by diagonal (j - i) is worked out once a tile and laid out in LDS; a lane keeps the
// diagonals of its row in registers and reads one more for the next.  Bound by memory: 4 x 32 heads of 2048 x 2048 bf16 added to, 2.1 GB
// in 390 us, 5.5 TB/s; 16 x 12 rows of 1031 take 8 us, the launch and one tile's chain of reads.
struct BiasShape { int64_t tiles, q, k, total; int buckets, heads, lanes, groups, per, rows, down, across; };
constexpr int kBiasStrip = 8 * kRelBlock + 1024;     // columns + rows of a tile

// 16 bytes of values, as many as a lane takes.
template <typename O> struct Wide;
template <> struct Wide<uint16_t> {
    static constexpr int kWidth = 8;
    u32x4 w;
    template <bool NT> __device__ static Wide load(const uint16_t* p) {
        const u32x4_at2* q = reinterpret_cast<const u32x4_at2*>(p);
        return {NT ? __builtin_nontemporal_load(q) : *q};
    }
    template <bool NT> __device__ void store(uint16_t* p) const {
        u32x4_at2* q = reinterpret_cast<u32x4_at2*>(p);
        if (NT) __builtin_nontemporal_store(w, q); else *q = w;
    }
    __device__ void widen(float a[8]) const { widen8(w, a); }
    __device__ static Wide of(const float a[8]) {
        return {u32x4{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7])}};
    }
    // The first m of them, in pieces of 4, 2 and 1 (a store of each by itself made rows of 1023
    // a half slower than rows of 1024).
    __device__ void store_head(uint16_t* p, int m) const {
        typedef uint32_t u32_at2 __attribute__((aligned(2)));
        int at = 0;
        if (m & 4) { *reinterpret_cast<u32x2_at2*>(p) = u32x2{w.x, w.y}; at = 2; }
        if (m & 2) { *reinterpret_cast<u32_at2*>(p + 2 * at) = at ? w.z : w.x; ++at; }
        if (m & 1) p[2 * at] = (uint16_t)(at == 0 ? w.x : at == 1 ? w.y : at == 2 ? w.z : w.w);
    }
};
template <> struct Wide<float> {
    static constexpr int kWidth = 4;
    f32x4 w;
    template <bool NT> __device__ static Wide load(const float* p) {
        const f32x4_at4* q = reinterpret_cast<const f32x4_at4*>(p);
        return {NT ? __builtin_nontemporal_load(q) : *q};
    }
    template <bool NT> __device__ void store(float* p) const {
        f32x4_at4* q = reinterpret_cast<f32x4_at4*>(p);
        if (NT) __builtin_nontemporal_store(w, q); else *q = w;
    }
    __device__ void widen(float a[4]) const { a[0] = w.x; a[1] = w.y; a[2] = w.z; a[3] = w.w; }
    __device__ static Wide of(const float a[4]) { return {f32x4{a[0], a[1], a[2], a[3]}}; }
    __device__ void store_head(float* p, int m) const {
        typedef float f32x2_at4 __attribute__((ext_vector_type(2), aligned(4)));
        if (m & 2) *reinterpret_cast<f32x2_at4*>(p) = f32x2{w.x, w.y};
        if (m & 1) p[m & 2] = m & 2 ? w.z : w.x;
    }
};

// NT: nontemporal accesses, for more than 128 MiB of scores that are added to, in whole lines of 128
// bytes from a multiple of 64 on.  In us, with them and without:
//   4 x 32 heads of 2048 x 2048 bf16 390, 406; 64 bytes on 408, 415; 16 bytes on 452, 417
//   2 x 32 of 4096 x 4096 727, 757; 8 x 32 of 1024 x 2112 423, 441; 2 x 12 of 2048 x 2048 80, 84
//   rows that are no whole lines: 8 x 32 of 1024 x 2080 457, 443; x 2064 550, 467
//   128 MiB (1 x 16 of 2048 x 2048) 58, 62, but added to in place 58, 46: the last-level cache holds it
//   with nothing to add to, 4 x 32 of 2048 x 2048: 376, 360
// (Buffer descriptors with nontemporal or sc1 stores, 400 and more for the first.)
template <typename T, typename O, bool ADD, bool NT>
__global__ __launch_bounds__(kRelBlock) void k_relpos_bias(const T* table, RelMap map, RelStart start, BiasShape s, float scale,
                                                           const O* add, O* out) {
    constexpr int W = Wide<O>::kWidth;
    __shared__ int32_t first[kRelBuckets];
    __shared__ float value[kRelBuckets];             // the head's, by bucket
    __shared__ float strip[kBiasStrip];
    stage_map(map, first);
    const int x = threadIdx.x % s.lanes, y = threadIdx.x / s.lanes;
    for (int64_t t = blockIdx.x; t < s.tiles; t += gridDim.x) {
        int64_t r = t;
        const int64_t c0 = r % s.across * s.lanes * W;
        r /= s.across;
        const int64_t i0 = r % s.down * s.rows;
        r /= s.down;
        const int head = (int)(r % s.heads);
        const int64_t d0 = c0 - (i0 + s.rows - 1) - start.of(r / s.heads);
        for (int b = threadIdx.x; b < s.buckets; b += blockDim.x) value[b] = load1(table + (int64_t)b * s.heads + head) * scale;
        __syncthreads();                             // the strip's last readers are done, the map and the values are there
        const int diagonals = s.rows - 1 + W * s.lanes;
        for (int v = threadIdx.x; v < diagonals; v += 4 * blockDim.x) {
            int which[4];
            rel_buckets<4>(first, map, d0 + v, blockDim.x, which);
#pragma unroll
            for (int j = 0; j < 4; ++j) if (v + j * (int)blockDim.x < diagonals) strip[v + j * blockDim.x] = value[which[j]];
        }
        __syncthreads();
        const int64_t col = c0 + W * x;
        const int first_row = y * s.per;
        if (y >= s.groups || col >= s.k) continue;
        const int have = (int)(s.k - col < W ? s.k - col : W);
        const int64_t most = s.q - i0 - first_row;
        const int rows = (int)(most < s.per ? most : s.per);
        const int64_t at = (r * s.q + i0 + first_row) * s.k + col;
        const int place = s.rows - 1 - first_row + W * x;      // of the first row's first value
        float w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = strip[place + j];
        // the window turns: after n rows its first value is w[-n mod W]
        auto eight = [&](int n, int count) {
            const int64_t p = at + n * s.k;
            Wide<O> old[8];
            // Values that all lie in the tensor are loaded whole, past the row's end too.
            if (ADD && p + 7 * s.k + W <= s.total) {
#pragma unroll
                for (int m = 0; m < 8; ++m) old[m] = Wide<O>::template load<NT>(add + p + m * s.k);
            } else if (ADD) {
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    if (m < count) {
                        const int64_t left = s.total - (p + m * s.k);
                        float a[8] = {};
                        if (left >= W) old[m] = Wide<O>::template load<NT>(add + p + m * s.k);
                        else {
#pragma unroll
                            for (int j = 0; j < W; ++j) if (j < left) a[j] = load1(add + p + m * s.k + j);
                            old[m] = Wide<O>::of(a);
                        }
                    }
            }
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (m < count) {
                    if (n + m) w[-m & (W - 1)] = strip[place - n - m];
                    float v[W], a[W];
                    if (ADD) old[m].widen(a);
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = ADD ? a[j] + w[(j - m) & (W - 1)] : w[(j - m) & (W - 1)];
                    const Wide<O> to = Wide<O>::of(v);
                    O* o = out + p + m * s.k;
                    if (have == W) to.template store<NT>(o);
                    else to.store_head(o, have);
                }
        };
        int n = 0;
        for (; n + 8 <= rows; n += 8) eight(n, 8);
        if (n < rows) eight(n, rows - n);
    }
}

// -------------------------------------------------------------- gradient --

// A work-item takes blocks of 8 rows by 8 columns, each one block further down and right than
// the last, so that the 15 diagonals it meets stay the same and their sums stay in registers,
// while its loads begin at multiples of 8 columns.  A tile is `rows` rows (8 `per` `groups`, the rest
// of q at the end) of one (sequence, head) and the diagonals that its `lanes` blocks side by side
// cross; groups lie one below the other.  partial[(head * buckets + b) * tiles of a head + tile]:
// the tile's sum of bucket b.  Bound by memory where it is large (2 x 32 heads of 4096 x 4096 bf16, 2.1 GB
// read in 357 us, 6.0 TB/s) and by one round of blocks where it is not (8 x 12 of 1024 x 1024 41 us, 4.9
// TB/s, and 4.5 for the join).
struct RelGradShape { int64_t tiles, per_head, q, k, total; int heads, buckets, lanes, groups, per, rows, down, across; };
constexpr int kRelStrip = 8 * (kRelBlock + 32);      // 8 (lanes + 1) sums for each of up to 32 groups

template <typename T>
__global__ __launch_bounds__(kRelBlock) void k_relpos_grad(const T* dy, RelMap map, RelStart start, RelGradShape s, float* partial) {
    __shared__ int32_t first[kRelBuckets];
    __shared__ float strip[kRelStrip];
    stage_map(map, first);
    const int x = threadIdx.x % s.lanes, y = threadIdx.x / s.lanes;
    const int width = 8 * (s.lanes + 1), blocks = s.per * s.groups;
    for (int64_t t = blockIdx.x; t < s.tiles; t += gridDim.x) {
        int64_t r = t;
        const int64_t across = r % s.across;
        r /= s.across;
        const int64_t down = r % s.down, i0 = down * s.rows;
        r /= s.down;
        const int head = (int)(r % s.heads);
        const int64_t b = r / s.heads;
        // the column block of the tile's first work-item in its first row block, and the first
        // diagonal (j - i) of the strip: that of the block's lower left corner
        const int64_t c0 = across * s.lanes - (blocks - 1), d0 = 8 * c0 - i0 - 7;
        __syncthreads();                             // the strip's last readers are done, the map is there
        float sum[15];
#pragma unroll
        for (int j = 0; j < 15; ++j) sum[j] = 0.0f;
        if (y < s.groups) {
            for (int n = 0; n < s.per; ++n) {
                const int m = y * s.per + n;
                const int64_t i = i0 + 8 * m, c = 8 * (c0 + x + m), rows = s.q - i;
                if (rows <= 0 || c < 0 || c >= s.k) continue;
                const int64_t at = (r * s.q + i) * s.k + c;
                Raw8<T> v[8];
                // Eight values that all lie in the tensor are loaded whole; those past the row's end
                // are another row's and dropped below.
                if (rows >= 8 && at + 7 * s.k + 8 <= s.total) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[l] = load8<true>(dy + at + l * s.k);
                } else {
#pragma unroll
                    for (int l = 0; l < 8; ++l) {
                        const int64_t left = l < rows ? s.total - (at + l * s.k) : 0;
                        v[l] = left >= 8 ? load8<true>(dy + at + l * s.k) : load8_part(dy + at + l * s.k, (int)left);
                    }
                }
                const int have = (int)(s.k - c < 8 ? s.k - c : 8);
#pragma unroll
                for (int l = 0; l < 8; ++l) {
                    float a[8];
                    widen(v[l], a);
                    if (have < 8)
#pragma unroll
                        for (int j = 1; j < 8; ++j) a[j] = j < have ? a[j] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[7 + j - l] = sum[7 + j - l] + a[j];
                }
            }
            // neighbours share seven diagonals: first the places that are a work-item's own to begin
#pragma unroll
            for (int j = 0; j < 8; ++j) strip[y * width + 8 * x + j] = sum[j];
            if (x == s.lanes - 1)
#pragma unroll
                for (int j = 8; j < 16; ++j) strip[y * width + 8 * x + j] = 0.0f;
        }
        __syncthreads();
        if (y < s.groups)
#pragma unroll
            for (int j = 8; j < 15; ++j) strip[y * width + 8 * x + j] += sum[j];
        __syncthreads();
        // the sums of each bucket's diagonals, an interval of the tile's: 64 work-items a bucket, or 16
        const int team = width * s.groups > 512 ? 64 : 16, member = threadIdx.x & (team - 1);
        const int64_t d1 = d0 - start.of(b);                          // distance of the tile's first diagonal
        for (int k = threadIdx.x / team; k < s.buckets; k += blockDim.x / team) {
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
                for (int v = from + member; v < to; v += team) total = total + strip[g * width + v];
            for (int o = team / 2; o > 0; o >>= 1) total = total + __uint_as_float(__shfl_xor(__float_as_uint(total), o));
            if (member == 0) partial[((int64_t)head * s.buckets + k) * s.per_head + (b * s.down + down) * s.across + across] = total;
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
