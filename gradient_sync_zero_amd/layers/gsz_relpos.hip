// Host half of the relative position bias entry points of include/gsz.h: argument checks,
// the buckets' borders, launch shapes, workspace layout.  The kernels are in gsz_relpos.h.
#pragma clang fp contract(off)

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "gsz_relpos.h"

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

int bad_arg(const char* who, const char* what) {
    set_error("%s: %s", who, what);
    return GSZ_ERR_INVALID_ARG;
}

int64_t value_size(int32_t type) { return type == GSZ_TYPE_BF16 ? 2 : type == GSZ_TYPE_F32 ? 4 : 0; }
int64_t id_size(int32_t type) { return type == GSZ_TYPE_I32 ? 4 : type == GSZ_TYPE_I64 ? 8 : 0; }
bool off_by(const void* p, int64_t align) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)align != 0; }

struct Span { const void* p; int64_t bytes; };
bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
}

// Sizes of a call.  Where none is 0 all products of them fit 62 bits.
int check_sizes(const char* who, int64_t batch, int64_t heads, int64_t q, int64_t k, int64_t buckets) {
    if (batch < 0 || heads < 0 || q < 0 || k < 0) return bad_arg(who, "negative size");
    constexpr int64_t kMost = (int64_t)1 << 30;
    if (batch > kMost || heads > 65536 || q > kMost || k > kMost || (double)batch * heads * q * k > 1e15) {
        set_error("%s: batch %lld, heads %lld, q_len %lld or k_len %lld over the limits 2^30, 2^16, 2^30, 2^30 or 1e15 scores", who,
                  (long long)batch, (long long)heads, (long long)q, (long long)k);
        return GSZ_ERR_SIZE;
    }
    if (buckets < 2 || buckets > kRelBuckets) { set_error("%s: buckets %lld is not in [2, %d]", who, (long long)buckets, kRelBuckets); return GSZ_ERR_INVALID_ARG; }
    return GSZ_OK;
}

// The buckets' borders.  Of n buckets a direction the first e = n / 2 hold one distance each; bucket
// e + k begins at the smallest whole number at or past e (D / e)^(k / (n - e)).  The powers are
// products in 64-bit mantissas, off by less than 2^-52 after 256 of them, and a value within 2^-50
// of a whole number is that number: where the power is one exactly (D / e = 16, four of eight
// steps), rounding does not move it up.
int make_map(const char* who, int64_t buckets, int64_t max_distance, int32_t bidirectional, RelMap* m) {
    if (bidirectional != 0 && bidirectional != 1) return bad_arg(who, "bidirectional is neither 0 nor 1");
    const int64_t n = bidirectional ? buckets / 2 : buckets, e = n / 2;
    if (n < 2 || (bidirectional && buckets % 2)) { set_error("%s: %lld buckets do not give 2 or more to each direction", who, (long long)buckets); return GSZ_ERR_INVALID_ARG; }
    if (max_distance <= e || max_distance > (int64_t)1 << 30) {
        set_error("%s: max_distance %lld is not in (%lld, 2^30]", who, (long long)max_distance, (long long)e);
        return GSZ_ERR_INVALID_ARG;
    }
    std::memset(m, 0, sizeof *m);
    m->n = (int)n;
    m->both = bidirectional;
    m->top = 1;
    while (2 * m->top < n) m->top *= 2;
    for (int64_t b = 0; b <= e; ++b) m->first[b] = (int32_t)b;
    const long double ratio = std::exp(std::log((long double)max_distance / e) / (n - e));
    long double t = e;
    for (int64_t k = 1; k < n - e; ++k) {
        t *= ratio;
        const long double near = std::floor(t + 0.5L);
        m->first[e + k] = (int32_t)(std::fabs(t - near) <= near * 0x1p-50L ? near : std::ceil(t));
    }
    return GSZ_OK;
}

int check_start(const char* who, int64_t q_start, const void* starts, int32_t start_type, RelStart* s) {
    const int64_t size = id_size(start_type);
    if (starts && !size) return bad_arg(who, "unknown type of q_starts");
    if (starts && off_by(starts, size)) { set_error("%s: q_starts is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    if (q_start < -((int64_t)1 << 40) || q_start > (int64_t)1 << 40) return bad_arg(who, "q_start is not within 2^40 of 0");
    *s = RelStart{starts, start_type == GSZ_TYPE_I64, q_start};
    return GSZ_OK;
}

int64_t scores(int64_t batch, int64_t heads, int64_t q, int64_t k) { return batch && heads && q && k ? batch * heads * q * k : 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int grid_for(int64_t tiles, int block) {
    const int64_t cap = kMaxWorkItems / block;
    return (int)(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
}

// Across: as many work-items as a row has vectors of 16 bytes, in equal parts where a block does not
// hold them.  Down: the rest of the block, each with up to `most` rows.
BiasShape bias_shape(int64_t batch, int64_t heads, int64_t q, int64_t k, int64_t buckets, int width, int* block) {
    BiasShape s{};
    s.total = batch * heads * q * k;
    s.buckets = (int)buckets;
    s.q = q;
    s.k = k;
    s.heads = (int)heads;
    const int64_t vectors = ceil_div(k, width);
    s.across = (int)ceil_div(vectors, kRelBlock);
    s.lanes = (int)ceil_div(vectors, s.across);
    const int64_t fit = kRelBlock / s.lanes;
    int64_t per = ceil_div(q, fit);
    if (per > 32) per = 32;
    if (per * fit > 1024) per = 1024 / fit;
    s.per = (int)per;
    s.groups = (int)(ceil_div(q, per) < fit ? ceil_div(q, per) : fit);
    s.rows = s.per * s.groups;
    s.down = (int)ceil_div(q, s.rows);
    s.tiles = batch * heads * s.down * s.across;
    *block = (int)(ceil_div((int64_t)s.lanes * s.groups, 64) * 64);
    return s;
}

// Rows a tile: 256, or fewer where that leaves few waves for the card, 32 at least.  (8 x 12 heads of
// 1024 x 1024 bf16: 43.6 us with at least 2048 waves, 54.8 with 4096, 56.3 with 1024.)
constexpr int64_t kRelGradWaves = 2048;
RelGradShape grad_shape(int64_t batch, int64_t heads, int64_t q, int64_t k, int64_t buckets, int* block) {
    RelGradShape s{};
    s.q = q;
    s.k = k;
    s.heads = (int)heads;
    s.buckets = (int)buckets;
    s.total = batch * heads * q * k;
    const int64_t down = ceil_div(q, 8), right = ceil_div(k, 8);
    int64_t rows = 32;                               // row blocks a tile
    while (rows > 4 && batch * heads * ceil_div(down, rows) * ceil_div(right + rows - 1, 64) < kRelGradWaves) rows /= 2;
    if (rows > down) rows = down;
    s.across = (int)ceil_div(right + rows - 1, kRelBlock);
    // as many groups as a block holds (its last row blocks, past `rows`, begin further left)
    for (int64_t groups = rows; ; --groups) {
        s.per = (int)ceil_div(rows, groups);
        s.groups = (int)ceil_div(rows, s.per);
        s.lanes = (int)ceil_div(right + s.per * s.groups - 1, s.across);
        if (s.lanes * s.groups <= kRelBlock) break;  // one group: lanes alone
    }
    s.rows = 8 * s.per * s.groups;
    s.down = (int)ceil_div(q, s.rows);
    s.per_head = batch * s.down * s.across;
    s.tiles = s.per_head * heads;
    *block = (int)(ceil_div((int64_t)s.lanes * s.groups, 64) * 64);
    return s;
}
int64_t partial_bytes(const RelGradShape& s) { return 4 * (int64_t)s.heads * s.buckets * s.per_head; }

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

extern "C" int gsz_relpos_bias(const void* table, int32_t table_type, int64_t buckets, int64_t heads, int64_t max_distance,
                               int32_t bidirectional, int64_t batch, int64_t q_len, int64_t k_len, int64_t q_start,
                               const void* q_starts, int32_t start_type, double scale, const void* add, void* out,
                               int32_t out_type, hipStream_t stream) {
    const char* who = "gsz_relpos_bias";
    const int64_t ts = value_size(table_type), os = value_size(out_type);
    if (!ts || !os) return bad_arg(who, "unknown value type");
    int rc = check_sizes(who, batch, heads, q_len, k_len, buckets);
    if (rc) return rc;
    RelMap map;
    if ((rc = make_map(who, buckets, max_distance, bidirectional, &map))) return rc;
    RelStart start;
    if ((rc = check_start(who, q_start, q_starts, start_type, &start))) return rc;
    const float c = (float)scale;
    if (!std::isfinite(c)) return bad_arg(who, "scale is not finite in fp32");
    const int64_t n = scores(batch, heads, q_len, k_len);
    if (n > 0 && (!table || !out)) return bad_arg(who, "NULL buffer");
    if (off_by(table, ts) || off_by(out, os) || off_by(add, os)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    const Span written{out, n * os};
    if (overlap(written, {table, buckets * heads * ts}) || (add != out && overlap(written, {add, n * os})) ||
        overlap(written, {q_starts, batch * id_size(start_type)}))
        return bad_arg(who, "out overlaps table, add or q_starts");
    if ((rc = check_device(who))) return rc;
    if (n == 0) return GSZ_OK;
    int block;
    const BiasShape s = bias_shape(batch, heads, q_len, k_len, buckets, 16 / (int)os, &block);
    const int grid = grid_for(s.tiles, block);
    const bool stream_past = n * os > (int64_t)128 << 20 && k_len * os % 128 == 0 && !off_by(add, 64) && !off_by(out, 64);
    with_type(table_type, [&](auto t) {
        with_type(out_type, [&](auto o) {
            with_bool(add != nullptr, [&](auto a) {
                using T = decltype(t);
                using O = decltype(o);
                with_bool(decltype(a)::value && stream_past, [&](auto nt) {
                    hipLaunchKernelGGL((k_relpos_bias<T, O, decltype(a)::value, decltype(a)::value && decltype(nt)::value>), dim3(grid),
                                       dim3(block), 0, stream, static_cast<const T*>(table), map, start, s, c,
                                       static_cast<const O*>(add), static_cast<O*>(out));
                });
            });
        });
    });
    return launched(who);
}

extern "C" int gsz_relpos_bias_workspace_bytes(int64_t batch, int64_t heads, int64_t q_len, int64_t k_len, int64_t buckets, size_t* out) {
    const char* who = "gsz_relpos_bias_workspace_bytes";
    const int rc = check_sizes(who, batch, heads, q_len, k_len, buckets);
    if (rc) return rc;
    if (!out) return bad_arg(who, "NULL output");
    int block;
    *out = batch && heads && q_len && k_len ? (size_t)partial_bytes(grad_shape(batch, heads, q_len, k_len, buckets, &block)) : 0;
    return GSZ_OK;
}

extern "C" int gsz_relpos_bias_grad(const void* dy, int32_t dy_type, int64_t buckets, int64_t heads, int64_t max_distance,
                                    int32_t bidirectional, int64_t batch, int64_t q_len, int64_t k_len, int64_t q_start,
                                    const void* q_starts, int32_t start_type, double scale, void* grad, int32_t grad_type,
                                    int32_t accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
    const char* who = "gsz_relpos_bias_grad";
    const int64_t ds = value_size(dy_type), gs = value_size(grad_type);
    if (!ds || !gs) return bad_arg(who, "unknown value type");
    if (accumulate != 0 && accumulate != 1) return bad_arg(who, "accumulate is neither 0 nor 1");
    int rc = check_sizes(who, batch, heads, q_len, k_len, buckets);
    if (rc) return rc;
    RelMap map;
    if ((rc = make_map(who, buckets, max_distance, bidirectional, &map))) return rc;
    RelStart start;
    if ((rc = check_start(who, q_start, q_starts, start_type, &start))) return rc;
    if (!std::isfinite((float)scale)) return bad_arg(who, "scale is not finite in fp32");
    const int64_t n = scores(batch, heads, q_len, k_len);
    if ((n > 0 && !dy) || (heads > 0 && !grad)) return bad_arg(who, "NULL buffer");
    if (off_by(dy, ds) || off_by(grad, gs)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    int block = 64;
    RelGradShape s{};
    s.heads = (int)heads;
    s.buckets = (int)buckets;
    if (n > 0) s = grad_shape(batch, heads, q_len, k_len, buckets, &block);
    const int64_t need = partial_bytes(s);
    if (need > 0) {
        if (!ws || ws_bytes < (size_t)need) { set_error("%s: workspace of %lld bytes required", who, (long long)need); return GSZ_ERR_SIZE; }
        if (off_by(ws, 16)) { set_error("%s: workspace is not 16-byte aligned", who); return GSZ_ERR_MISALIGNED; }
    }
    const Span written{grad, buckets * heads * gs}, scratch{ws, need}, starts{q_starts, batch * id_size(start_type)}, in{dy, n * ds};
    if (overlap(written, in) || overlap(written, starts) || overlap(scratch, in) || overlap(scratch, starts) || overlap(written, scratch))
        return bad_arg(who, "grad or ws overlaps dy, q_starts or the other");
    if ((rc = check_device(who))) return rc;
    if (heads == 0 || (n == 0 && accumulate)) return GSZ_OK;
    float* partial = static_cast<float*>(ws);
    if (n > 0) {
        const int grid = grid_for(s.tiles, block);
        with_type(dy_type, [&](auto t) {
            using T = decltype(t);
            hipLaunchKernelGGL((k_relpos_grad<T>), dim3(grid), dim3(block), 0, stream, static_cast<const T*>(dy), map, start, s, partial);
        });
        if ((rc = launched(who))) return rc;
    }
    const int join = grid_for(buckets * heads, 64);
    with_type(grad_type, [&](auto o) {
        with_bool(accumulate != 0, [&](auto acc) {
            using G = decltype(o);
            hipLaunchKernelGGL((k_relpos_join<G, decltype(acc)::value>), dim3(join), dim3(64), 0, stream, partial, s.per_head,
                               (int)buckets, (int)heads, scale, static_cast<G*>(grad));
        });
    });
    return launched(who);
}
