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

struct SortShape { bool rank; int64_t tile; int tiles, bits, passes; };

SortShape sort_shape(int64_t n, int64_t rows) {
    SortShape s{};
    s.rank = n <= kRankMax;
    if (s.rank) return s;
    // At most 256 tiles: every block of a pass reads the digit counts of all of them.
    s.tile = 1024;
    while ((n + s.tile - 1) / s.tile > 256) s.tile *= 2;
    s.tiles = (int)((n + s.tile - 1) / s.tile);
    int bits = 1;
    while (((int64_t)1 << bits) <= rows) ++bits;          // keys [0, rows]
    s.passes = (bits + 9) / 10;
    s.bits = (bits + s.passes - 1) / s.passes;
    return s;
}

int chunk_for(int64_t n, int64_t dim) {
    const int64_t cols = (dim + kGradCols - 1) / kGradCols;
    int K = kMaxChunk;
    while (K > 8 && (n + K - 1) / K * cols < 4096) K /= 2;
    return K;
}

struct Workspace { size_t key[2], pos[2], count[3], part, bytes; };

Workspace workspace_for(int64_t n, int64_t rows, int64_t dim) {
    Workspace w{};
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += (bytes + 255) / 256 * 256; return o; };
    const SortShape s = sort_shape(n, rows);
    for (int k = 0; k < (s.rank ? 1 : 2); ++k) { w.key[k] = take(4 * n); w.pos[k] = take(4 * n); }
    if (!s.rank)
        for (int k = 0; k < 3; ++k) w.count[k] = take((size_t)4 * s.tiles << s.bits);
    const int64_t chunks = (n + chunk_for(n, dim) - 1) / chunk_for(n, dim), pitch = (dim + 7) / 8 * 8;
    w.part = take((size_t)8 * chunks * pitch);
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
    if ((rc = check_device(who))) return rc;
    if (n == 0) return GSZ_OK;
    const int grid = grid_for((n + 8 * kDropBlock - 1) / (8 * kDropBlock), kDropBlock);
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
    if ((rc = check_device(who))) return rc;
    if (!work) return GSZ_OK;
    const int64_t vpr = (dim + 7) / 8;
    const int tile_rows = vpr >= kLookVecs ? 1 : (int)(kLookVecs / vpr);
    const uint64_t magic = ((uint64_t)1 << 32) / (uint64_t)vpr + 1;
    const int grid = grid_for((n + tile_rows - 1) / tile_rows, kLookBlock);
    const Ids id{ids, id_type == GSZ_TYPE_I64, (uint32_t)rows};
    with_type(table_type, [&](auto t) {
        with_type(out_type, [&](auto o) {
            with_bool(da.threshold != 0, [&](auto drop) {
                using T = decltype(t);
                using O = decltype(o);
                hipLaunchKernelGGL((k_lookup<T, O, decltype(drop)::value>), dim3(grid), dim3(kLookBlock), 0,
                                   stream, static_cast<const T*>(table), id, n, dim, vpr, tile_rows, magic, c0,
                                   da, static_cast<O*>(out));
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
    if (n > 0 && dim > 0) {
        if (!ids || !dy) return bad_arg(who, "NULL buffer");
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
    g.col_blocks = (int)((dim + kGradCols * kGradWaves - 1) / (kGradCols * kGradWaves));
    g.acc = accumulate;
    g.sum_blocks = g.chunks * g.col_blocks;
    // A clearing block writes about 128 KiB.
    const int64_t want = ((int64_t)128 << 10) / (dim * gs);
    g.clear_rows = (int)(want < 1 ? 1 : want > 64 ? 64 : want);
    const int64_t blocks = g.sum_blocks + (accumulate ? 0 : (rows + g.clear_rows - 1) / g.clear_rows);
    GradShape j = g;
    j.col_blocks = (int)((g.pitch + kJoinCols * kGradWaves - 1) / (kJoinCols * kGradWaves));
    if (blocks > kMaxWorkItems / kGradBlock || g.chunks * j.col_blocks > kMaxWorkItems / kGradBlock) {
        set_error("%s: n %lld by dim %lld, or rows %lld, needs more than 2^31 work-items", who, (long long)n, (long long)dim, (long long)rows);
        return GSZ_ERR_SIZE;
    }
    if ((rc = check_device(who))) return rc;

    char* base = static_cast<char*>(ws);
    auto u32 = [&](size_t o) { return reinterpret_cast<uint32_t*>(base + o); };
    const Ids id{ids, id_type == GSZ_TYPE_I64, (uint32_t)rows};
    const uint32_t* key = nullptr;
    const uint32_t* pos = nullptr;
    if (n > 0) {
        const SortShape s = sort_shape(n, rows);
        if (s.rank) {
            hipLaunchKernelGGL(k_rank, dim3((unsigned)((n + 63) / 64)), dim3(kRankBlock), 0, stream, id, (int)n,
                               u32(w.key[0]), u32(w.pos[0]));
            if ((rc = launched(who))) return rc;
            key = u32(w.key[0]);
            pos = u32(w.pos[0]);
        } else {
            const int bins = 1 << s.bits;
            hipLaunchKernelGGL(k_count, dim3(s.tiles), dim3(kSortBlock), 0, stream, id, n, s.tile, Digit{0, bins},
                               u32(w.count[0]), u32(w.count[1]));
            if ((rc = launched(who))) return rc;
            for (int k = 0; k < s.passes; ++k) {
                const Digit d{k * s.bits, bins}, dn{(k + 1) * s.bits, k + 1 < s.passes ? bins : 0};
                uint32_t* clear = k + 2 < s.passes ? u32(w.count[(k + 2) % 3]) : nullptr;
                uint32_t* to_key = u32(w.key[k & 1]);
                uint32_t* to_pos = u32(w.pos[k & 1]);
                with_bool(k == 0, [&](auto first) {
                    hipLaunchKernelGGL((k_place<decltype(first)::value>), dim3(s.tiles), dim3(kSortBlock), 0, stream,
                                       id, key, pos, n, s.tile, s.tiles, d, dn, u32(w.count[k % 3]),
                                       u32(w.count[(k + 1) % 3]), clear, to_key, to_pos);
                });
                if ((rc = launched(who))) return rc;
                key = to_key;
                pos = to_pos;
            }
        }
    }
    float* part = reinterpret_cast<float*>(base + w.part);
    with_type(dy_type, [&](auto t) {
        with_type(grad_type, [&](auto o) {
            with_bool(da.threshold != 0, [&](auto drop) {
                using T = decltype(t);
                using G = decltype(o);
                hipLaunchKernelGGL((k_grad<T, G, decltype(drop)::value>), dim3((unsigned)blocks), dim3(kGradBlock), 0,
                                   stream, static_cast<const T*>(dy), key, pos, g, c0, da, static_cast<G*>(grad), part);
            });
        });
    });
    if ((rc = launched(who))) return rc;
    if (g.chunks < 2) return GSZ_OK;
    int64_t step = 1;
    for (; g.chunks > 2 * kFold * step; step *= kFold) {
        const int64_t groups = (g.chunks + kFold * step - 1) / (kFold * step);
        hipLaunchKernelGGL(k_fold, dim3((unsigned)(groups * j.col_blocks)), dim3(kGradBlock), 0, stream, key, j, step, part);
        if ((rc = launched(who))) return rc;
    }
    with_type(grad_type, [&](auto o) {
        using G = decltype(o);
        hipLaunchKernelGGL((k_join<G>), dim3((unsigned)(g.chunks * j.col_blocks)), dim3(kGradBlock), 0, stream, key, j,
                           step, c0, static_cast<G*>(grad), static_cast<const float*>(part));
    });
    return launched(who);
}
