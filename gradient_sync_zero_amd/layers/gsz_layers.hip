// Host half of the embedding and dropout entry points of include/gsz.h: argument
// checks, launch shapes, workspace layout.  The kernels are in gsz_dropout.h and
// gsz_embedding.h.
#pragma clang fp contract(off)

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "gsz_embedding.h"

using gsz::set_error;

namespace {

int hip_fail(const char* who, hipError_t e) {
    set_error("%s: %s", who, hipGetErrorString(e));
    return GSZ_ERR_HIP;
}

// GSZ_OK where the current device is gfx950.
int check_device(const char* who) {
    static std::atomic<int> known[64];               // 0 unknown, 1 gfx950, -1 other
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(who, e);
    if (dev < 0 || dev >= 64) { set_error("%s: device index %d unsupported", who, dev); return GSZ_ERR_DEVICE; }
    int st = known[dev].load();
    if (st == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess) return hip_fail(who, e);
        st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
        known[dev].store(st);
    }
    if (st != 1) { set_error("%s: device %d is not gfx950 (MI355X); this library targets gfx950 only", who, dev); return GSZ_ERR_DEVICE; }
    return GSZ_OK;
}

int launched(const char* who) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? (int)GSZ_OK : hip_fail(who, e);
}

int64_t value_size(int32_t type) { return type == GSZ_TYPE_BF16 ? 2 : type == GSZ_TYPE_F32 ? 4 : 0; }
int64_t id_size(int32_t type) { return type == GSZ_TYPE_I32 ? 4 : type == GSZ_TYPE_I64 ? 8 : 0; }
bool off_by(const void* p, int64_t align) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)align != 0; }

int bad_arg(const char* who, const char* what) {
    set_error("%s: %s", who, what);
    return GSZ_ERR_INVALID_ARG;
}

// Whether a buffer that a call writes and one that it reads (or writes besides) share a byte.
struct Span { const void* p; int64_t bytes; };
bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
}
Span rng_span(const DropArgs& d) { return {d.threshold ? d.rng : nullptr, 16}; }

// The mask's arguments and the constant scale / (1 - threshold 2^-32), formed in
// double and rounded once.
int check_drop(const char* who, double p, double scale, const uint64_t* rng, uint32_t site,
               DropArgs* da, float* c0) {
    if (!(p >= 0.0 && p < 1.0)) { set_error("%s: dropout probability %g is not in [0, 1)", who, p); return GSZ_ERR_INVALID_ARG; }
    const uint32_t t = (uint32_t)std::floor(p * 4294967296.0);
    const double c = scale / (1.0 - (double)t / 4294967296.0);
    if (!std::isfinite((float)c)) { set_error("%s: scale %g is not finite in fp32", who, c); return GSZ_ERR_INVALID_ARG; }
    if (t && !rng) return bad_arg(who, "dropout needs rng");
    if (t && off_by(rng, 8)) { set_error("%s: rng is not 8-byte aligned", who); return GSZ_ERR_MISALIGNED; }
    *da = DropArgs{rng, site, t};
    *c0 = (float)c;
    return GSZ_OK;
}

// Sizes of an embedding call: rows and n fit the sort's 32-bit keys and positions,
// and element offsets fit 61 bits (a generator block holds 8 elements).
int check_sizes(const char* who, int64_t rows, int64_t dim, int64_t n) {
    if (rows < 0 || dim < 0 || n < 0) return bad_arg(who, "negative size");
    constexpr int64_t kMost = ((int64_t)1 << 31) - 1;
    if (rows > kMost || n > kMost || dim > (int64_t)1 << 29) {
        set_error("%s: rows %lld, dim %lld or n %lld over the limits 2^31 - 1, 2^29 and 2^31 - 1", who,
                  (long long)rows, (long long)dim, (long long)n);
        return GSZ_ERR_SIZE;
    }
    return GSZ_OK;
}

// Blocks of a launch over `tiles` tiles, at most 2^31 work-items.
int grid_for(int64_t tiles, int block) {
    const int64_t cap = kMaxWorkItems / block;
    return (int)(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
}

// ------------------------------------------------------- gradient's plan --

// The counting sort of n > kRankMax tokens: at most kMaxTiles tiles (every block of a pass
// reads the digit counts of all of them) and digits of at most 10 bits.
constexpr int kMaxTiles = 256;
struct SortShape { int64_t rounds; int tiles, bits, passes; };
SortShape sort_shape(int64_t n, int64_t rows) {
    SortShape s{};
    s.rounds = 1;
    while ((n + s.rounds * kSortTile - 1) / (s.rounds * kSortTile) > kMaxTiles) s.rounds *= 2;
    s.tiles = (int)((n + s.rounds * kSortTile - 1) / (s.rounds * kSortTile));
    int bits = 1;
    while (((int64_t)1 << bits) <= rows) ++bits;          // keys [0, rows]
    s.passes = (bits + 9) / 10;
    s.bits = (bits + s.passes - 1) / s.passes;
    return s;
}

int col_tiles(int64_t dim) { return (int)((dim + kGradCols - 1) / kGradCols); }

// Tokens per chunk: as many as leave 4096 waves, 4 at least.  (Chunks of 8 at least: 8192
// tokens of 768 columns 39.0 us against 36.5.  8192 waves: 4096 tokens of 4096 columns
// 26.9 us against 25.7, one row with nine tokens in ten 198 us against 193; 2048 waves:
// 8192 tokens of 4096 columns 49.5 us against 48.1.)
constexpr int kGradMinWaves = 4096, kMinChunk = 4;
int chunk_for(int64_t n, int64_t dim) {
    int K = kMaxChunk;
    while (K > kMinChunk && (n + K - 1) / K * col_tiles(dim) < kGradMinWaves) K /= 2;
    return K;
}
// The most chunks that n tokens or fewer are cut into.  K falls as n does, so a few tokens
// less can be up to twice as many chunks.  With c = ceil(kGradMinWaves / column tiles), n is
// cut by less than kMaxChunk only where ceil(n / 2 K) < c, into ceil(n / K) <= 2 (c - 1) chunks.
int64_t most_chunks(int64_t n, int64_t dim) {
    const int64_t c = dim > 0 ? (kGradMinWaves + col_tiles(dim) - 1) / col_tiles(dim) : 1;
    const int64_t fine = (n + kMinChunk - 1) / kMinChunk, coarse = (n + kMaxChunk - 1) / kMaxChunk;
    const int64_t most = fine < 2 * (c - 1) ? fine : 2 * (c - 1);
    return coarse > most ? coarse : most;
}

// A workspace for n tokens serves every smaller call on the same table: no part of it
// shrinks as n grows.
struct Workspace { size_t key[2], pos[2], count, owner, part, bytes; };
Workspace workspace_for(int64_t n, int64_t rows, int64_t dim) {
    Workspace w{};
    if (n <= kDirectMax) return w;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += (bytes + 255) / 256 * 256; return o; };
    const bool rank = n <= kRankMax;
    for (int k = 0; k < (rank ? 1 : 2); ++k) { w.key[k] = take(4 * n); w.pos[k] = take(4 * n); }
    if (!rank) {
        const int64_t tiles = (n + kSortTile - 1) / kSortTile;
        w.count = take((size_t)4 * (tiles < kMaxTiles ? tiles : kMaxTiles) << sort_shape(n, rows).bits);
        w.owner = take((size_t)4 * rows);
    }
    w.part = take((size_t)8 * most_chunks(n, dim) * ((dim + 7) / 8 * 8));
    w.bytes = at;
    return w;
}

template <class F>
void with_type(int32_t type, F&& f) {
    if (type == GSZ_TYPE_BF16) f(uint16_t{});
    else f(float{});
}
template <class F>
void with_bool(bool b, F&& f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}

}  // namespace

extern "C" int gsz_dropout(const void* x, const void* add, void* y, int64_t n, int32_t type, double p,
                           const uint64_t* rng, uint32_t site, hipStream_t stream) {
    const char* who = "gsz_dropout";
    const int64_t size = value_size(type);
    if (!size) return bad_arg(who, "unknown value type");
    if (n < 0) return bad_arg(who, "negative size");
    if (n > (int64_t)1 << 60) { set_error("%s: n %lld is over 2^60", who, (long long)n); return GSZ_ERR_SIZE; }
    DropArgs da;
    float k;
    int rc = check_drop(who, p, 1.0, rng, site, &da, &k);
    if (rc) return rc;
    if (n > 0 && (!x || !y)) return bad_arg(who, "NULL buffer");
    if (off_by(x, size) || off_by(y, size) || off_by(add, size)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    const Span out{y, n * size};
    if ((y != x && overlap(out, {x, n * size})) || (y != add && overlap(out, {add, n * size})) || overlap(out, rng_span(da)))
        return bad_arg(who, "y overlaps x, add or rng");
    if ((rc = check_device(who))) return rc;
    if (n == 0) return GSZ_OK;
    const int grid = grid_for((n + kTile - 1) / kTile, kDropBlock);
    with_type(type, [&](auto t) {
        using T = decltype(t);
        with_bool(add != nullptr, [&](auto a) {
            with_bool(da.threshold != 0, [&](auto drop) {
                hipLaunchKernelGGL((k_dropout<T, decltype(a)::value, decltype(drop)::value>), dim3(grid),
                                   dim3(kDropBlock), 0, stream, static_cast<const T*>(x),
                                   static_cast<const T*>(add), static_cast<T*>(y), n, k, da);
            });
        });
    });
    return launched(who);
}

extern "C" int gsz_embedding_lookup(const void* table, int32_t table_type, int64_t rows, int64_t dim,
                                    const void* ids, int32_t id_type, int64_t n, double scale, double p,
                                    const uint64_t* rng, uint32_t site, void* out, int32_t out_type,
                                    hipStream_t stream) {
    const char* who = "gsz_embedding_lookup";
    const int64_t ts = value_size(table_type), os = value_size(out_type), is = id_size(id_type);
    if (!ts || !os || !is) return bad_arg(who, "unknown value or id type");
    int rc = check_sizes(who, rows, dim, n);
    if (rc) return rc;
    DropArgs da;
    float c0;
    if ((rc = check_drop(who, p, scale, rng, site, &da, &c0))) return rc;
    const bool work = n > 0 && dim > 0;
    if (work && (!ids || !out || (rows > 0 && !table))) return bad_arg(who, "NULL buffer");
    if (off_by(table, ts) || off_by(out, os) || off_by(ids, is)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    const Span written{out, n * dim * os};
    if (overlap(written, {table, rows * dim * ts}) || overlap(written, {ids, n * is}) || overlap(written, rng_span(da)))
        return bad_arg(who, "out overlaps table, ids or rng");
    if ((rc = check_device(who))) return rc;
    if (!work) return GSZ_OK;
    LookShape l{};
    l.n = n;
    l.dim = dim;
    l.vpr = (int)((dim + 7) / 8);
    const bool wide = l.vpr > kLookBlock / 2;
    // Vectors per lane: fewer where a few thousand blocks are all there is, so that a small
    // call is spread wider (the kernel on one token of 8192 columns 2.5 us with one vector
    // against 3.2 with four; no difference in a call of 8192 tokens of 768 columns, 6.2 us).
    int vectors = look_unroll(da.threshold != 0);
    while (vectors > 1 && n * l.vpr / (kLookBlock * vectors) < 4096) vectors /= 2;
    l.side = wide ? 1 : kLookBlock / l.vpr;
    l.per = vectors;
    l.cols = 1;
    if (wide) {
        const int pieces = (l.vpr + kLookBlock - 1) / kLookBlock;     // of at most kLookBlock vectors
        while (l.per > 1 && 2 << l.wide_log2 <= pieces) { ++l.wide_log2; l.per /= 2; }
        l.width = (l.vpr + pieces - 1) / pieces;
        l.cols = (pieces + (1 << l.wide_log2) - 1) >> l.wide_log2;
    }
    l.magic = ((uint64_t)1 << 32) / (uint64_t)l.vpr + 1;
    l.tiles = (n + (int64_t)l.side * l.per - 1) / ((int64_t)l.side * l.per);
    const int block = ((wide ? l.width : l.side * l.vpr) + 63) / 64 * 64;
    const int grid = grid_for(l.tiles * l.cols, kLookBlock);
    const Ids id{ids, id_type == GSZ_TYPE_I64, (uint32_t)rows};
    with_type(table_type, [&](auto t) {
        with_type(out_type, [&](auto o) {
            with_bool(da.threshold != 0, [&](auto drop) {
                with_bool(wide, [&](auto w) {
                    using T = decltype(t);
                    using O = decltype(o);
                    hipLaunchKernelGGL((k_lookup<T, O, decltype(drop)::value, decltype(w)::value>), dim3(grid),
                                       dim3(block), 0, stream, static_cast<const T*>(table), id, l, c0, da,
                                       static_cast<O*>(out));
                });
            });
        });
    });
    return launched(who);
}

extern "C" int gsz_embedding_workspace_bytes(int64_t n, int64_t rows, int64_t dim, size_t* out) {
    const char* who = "gsz_embedding_workspace_bytes";
    const int rc = check_sizes(who, rows, dim, n);
    if (rc) return rc;
    if (!out) return bad_arg(who, "NULL output");
    *out = workspace_for(n, rows, dim).bytes;
    return GSZ_OK;
}

extern "C" int gsz_embedding_grad(const void* ids, int32_t id_type, int64_t n, const void* dy,
                                  int32_t dy_type, int64_t rows, int64_t dim, double scale, double p,
                                  const uint64_t* rng, uint32_t site, void* grad, int32_t grad_type,
                                  int32_t accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
    const char* who = "gsz_embedding_grad";
    const int64_t ds = value_size(dy_type), gs = value_size(grad_type), is = id_size(id_type);
    if (!ds || !gs || !is) return bad_arg(who, "unknown value or id type");
    if (accumulate != 0 && accumulate != 1) return bad_arg(who, "accumulate is neither 0 nor 1");
    int rc = check_sizes(who, rows, dim, n);
    if (rc) return rc;
    DropArgs da;
    float c0;
    if ((rc = check_drop(who, p, scale, rng, site, &da, &c0))) return rc;
    const Workspace w = workspace_for(n, rows, dim);
    if (n > 0 && dim > 0 && (!ids || !dy)) return bad_arg(who, "NULL buffer");
    if (n > 0 && dim > 0 && w.bytes > 0) {
        if (!ws || ws_bytes < w.bytes) { set_error("%s: workspace of %zu bytes required", who, w.bytes); return GSZ_ERR_SIZE; }
        if (off_by(ws, 16)) { set_error("%s: workspace is not 16-byte aligned", who); return GSZ_ERR_MISALIGNED; }
    }
    if (rows > 0 && dim > 0 && !grad) return bad_arg(who, "NULL buffer");
    if (off_by(dy, ds) || off_by(grad, gs) || off_by(ids, is)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    if (rows == 0 || dim == 0 || (n == 0 && accumulate)) return check_device(who);

    GradShape g{};
    g.dim = dim;
    g.pitch = (dim + 7) / 8 * 8;
    g.n = n;
    g.rows = (uint32_t)rows;
    g.K = chunk_for(n, dim);
    g.chunks = (n + g.K - 1) / g.K;
    g.tiles = col_tiles(dim);
    // dy of 64 MiB and more is read nontemporally: at 32 MiB that took 31.4 us against 27.2,
    // at 64 MiB 64.2 against 68.6 (fp32 gradient) or 47.8 against 46.7 (bf16), at 256 MiB
    // 111 against 126.
    g.nt = n * dim * ds >= (int64_t)64 << 20;
    const bool direct = n <= kDirectMax, rank = !direct && n <= kRankMax, f32 = grad_type == GSZ_TYPE_F32;
    // Rows that a block clears: about 32 KiB beside the sort's or the sums' blocks (2-5%
    // faster than 128 KiB: one block's search for them hides behind others' stores),
    // 256 KiB in whole words of 64 rows for the rank sort's, which hold every key.
    const int64_t row_bytes = dim * gs;
    auto clamp = [](int64_t v, int64_t most) { return (int)(v < 1 ? 1 : v > most ? most : v); };
    int per = rank ? clamp(((int64_t)256 << 10) / (64 * row_bytes), 64) : clamp(((int64_t)32 << 10) / row_bytes, 64);
    while (rank && per & (per - 1)) per &= per - 1;                  // a power of two
    const int64_t rank_max = kMaxWorkItems / kRankBlock, direct_max = kMaxWorkItems / kGradBlock;
    auto clear_for = [&] { return accumulate ? 0 : (rows + (int64_t)per * (rank ? 64 : 1) - 1) / ((int64_t)per * (rank ? 64 : 1)); };
    while (rank && per < 64 && clear_for() > rank_max) per *= 2;
    int64_t clear_blocks = clear_for();                              // the other sort divides them over its launches
    const int64_t sum_blocks = (direct ? n : g.chunks) * g.tiles;
    if (direct && clear_blocks > 0 && clear_blocks > direct_max - sum_blocks)
        clear_blocks = direct_max > sum_blocks ? direct_max - sum_blocks : 1;
    const int join_tiles = (int)((dim + kJoinCols - 1) / kJoinCols);
    const int64_t join_blocks = (g.chunks + kJoinChunks - 1) / kJoinChunks * join_tiles;
    const int64_t rank_blocks = (n + kRankTokens - 1) / kRankTokens > clear_blocks ? (n + kRankTokens - 1) / kRankTokens : clear_blocks;
    const SortShape sh = sort_shape(n, rows);                        // of the counting sort
    const int parts = 2 * sh.passes - 1;                             // its launches that clear
    const int64_t sort_max = kMaxWorkItems / kSortBlock - sh.tiles;  // blocks that each of them has for it
    if (sum_blocks + (direct ? clear_blocks : 0) > direct_max || (!direct && join_blocks > kMaxWorkItems / kJoinBlock) ||
        (rank && rank_blocks > rank_max) || (!direct && !rank && sort_max < 1)) {
        set_error("%s: n %lld by dim %lld needs more than 2^31 work-items", who, (long long)n, (long long)dim);
        return GSZ_ERR_SIZE;
    }
    const Span written{grad, rows * dim * gs}, scratch{ws, (int64_t)w.bytes}, read[] = {{ids, n * is}, {dy, n * dim * ds}, rng_span(da)};
    for (const Span& r : read)
        if (overlap(written, r) || overlap(scratch, r)) return bad_arg(who, "grad or ws overlaps ids, dy or rng");
    if (overlap(written, scratch)) return bad_arg(who, "ws overlaps grad");
    if ((rc = check_device(who))) return rc;

    char* base = static_cast<char*>(ws);
    auto u32 = [&](size_t o) { return reinterpret_cast<uint32_t*>(base + o); };
    const Ids id{ids, id_type == GSZ_TYPE_I64, (uint32_t)rows};
    ClearShape clear{accumulate ? nullptr : grad, dim, 0, rows, 0xFFFFFFFFu, per, f32};
    if (direct) {
        clear.first_block = (unsigned)sum_blocks;
        with_type(dy_type, [&](auto t) {
            with_type(grad_type, [&](auto o) {
                with_bool(accumulate != 0, [&](auto acc) {
                    with_bool(da.threshold != 0, [&](auto drop) {
                        using T = decltype(t);
                        using G = decltype(o);
                        hipLaunchKernelGGL((k_direct<T, G, decltype(acc)::value, decltype(drop)::value>),
                                           dim3((unsigned)(sum_blocks + clear_blocks)), dim3(kGradBlock), 0, stream,
                                           static_cast<const T*>(dy), id, g, c0, da, static_cast<G*>(grad), clear);
                    });
                });
            });
        });
        return launched(who);
    }

    uint32_t* key = u32(w.key[0]);
    uint32_t* pos = u32(w.pos[0]);
    if (rank) {
        with_bool(rows < kRankPackedRows, [&](auto packed) {
            hipLaunchKernelGGL((k_rank<decltype(packed)::value>), dim3((unsigned)rank_blocks), dim3(kRankBlock), 0,
                               stream, id, (int)n, key, pos, clear);
        });
        if ((rc = launched(who))) return rc;
    } else {
        SortPass s{id, nullptr, nullptr, n, sh.rounds, sh.tiles, 0, 1 << sh.bits};
        uint32_t* count = u32(w.count);
        uint32_t* owner = accumulate ? nullptr : u32(w.owner);
        // The launches after the first each clear a part of the rows.
        int part = 0;
        auto next_part = [&]() -> int64_t {                          // its blocks
            clear.first_block = accumulate ? 0xFFFFFFFFu : (unsigned)sh.tiles;
            clear.row0 = clear_blocks * part / parts * per;
            clear.row1 = ++part == parts ? rows : clear_blocks * part / parts * per;
            const int64_t blocks = accumulate ? 0 : (clear.row1 - clear.row0 + per - 1) / per;
            return blocks < sort_max ? blocks : sort_max;
        };
        for (int k = 0; k < sh.passes; ++k) {
            s.shift = k * sh.bits;
            key = u32(w.key[k & 1]);
            pos = u32(w.pos[k & 1]);
            if (k == 0) {
                hipLaunchKernelGGL((k_count<true>), dim3(sh.tiles), dim3(kSortBlock), 0, stream, s, count, owner, clear);
                if ((rc = launched(who))) return rc;
                const int64_t more = next_part();
                hipLaunchKernelGGL((k_place<true>), dim3((unsigned)(sh.tiles + more)), dim3(kSortBlock), 0, stream, s,
                                   count, key, pos, owner, clear);
            } else {
                int64_t more = next_part();
                hipLaunchKernelGGL((k_count<false>), dim3((unsigned)(sh.tiles + more)), dim3(kSortBlock), 0, stream, s,
                                   count, owner, clear);
                if ((rc = launched(who))) return rc;
                more = next_part();
                hipLaunchKernelGGL((k_place<false>), dim3((unsigned)(sh.tiles + more)), dim3(kSortBlock), 0, stream, s,
                                   count, key, pos, owner, clear);
            }
            if ((rc = launched(who))) return rc;
            s.key_in = key;
            s.pos_in = pos;
        }
    }

    float* part = reinterpret_cast<float*>(base + w.part);
    with_type(dy_type, [&](auto t) {
        with_type(grad_type, [&](auto o) {
            with_bool(accumulate != 0, [&](auto acc) {
                with_bool(da.threshold != 0, [&](auto drop) {
                    using T = decltype(t);
                    using G = decltype(o);
                    hipLaunchKernelGGL((k_grad<T, G, decltype(acc)::value, decltype(drop)::value>),
                                       dim3((unsigned)sum_blocks), dim3(kGradBlock), 0, stream,
                                       static_cast<const T*>(dy), key, pos, g, c0, da, static_cast<G*>(grad), part);
                });
            });
        });
    });
    if ((rc = launched(who))) return rc;
    with_type(grad_type, [&](auto o) {
        with_bool(accumulate != 0, [&](auto acc) {
            using G = decltype(o);
            hipLaunchKernelGGL((k_join<G, decltype(acc)::value>), dim3((unsigned)join_blocks), dim3(kJoinBlock), 0,
                               stream, key, g, join_tiles, c0, static_cast<G*>(grad), static_cast<const float*>(part));
        });
    });
    return launched(who);
}
