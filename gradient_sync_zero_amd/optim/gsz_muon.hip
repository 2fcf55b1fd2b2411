// Host half of the orthogonalising entry points of include/gsz.h: argument checks, launch
// shapes, workspace layout.  The kernels are in gsz_muon.h, gsz_product.h
// and gsz_small.h.
#pragma clang fp contract(off)

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <vector>

#include "gsz_small.h"

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
bool off_by(const void* p, int64_t align) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)align != 0; }

struct Span { const void* p; int64_t bytes; };
bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
}

constexpr int64_t kMostSide = (int64_t)1 << 17, kMostElements = (int64_t)1 << 32;

int check_shape(const char* who, int64_t count, int64_t rows, int64_t cols) {
    if (count < 0 || rows < 0 || cols < 0) return bad_arg(who, "negative size");
    if (rows > kMostSide || cols > kMostSide || rows * cols > kMostElements || count > (int64_t)1 << 31 || (double)count * rows * cols > 1e15) {
        set_error("%s: count %lld, rows %lld or cols %lld over the limits 2^31, 2^17, 2^17, 2^32 elements a matrix or 1e15 in all", who,
                  (long long)count, (long long)rows, (long long)cols);
        return GSZ_ERR_SIZE;
    }
    return GSZ_OK;
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// How a call's matrices lie in the workspace: sides padded to kStepK.
struct Shape {
    int64_t rows, cols, small, large;            // as given; the smaller and the larger side, padded
    int64_t padded_rows, padded_cols, norm_tiles;
    bool tall;
};
Shape shape_for(int64_t rows, int64_t cols) {
    Shape s{};
    s.rows = rows;
    s.cols = cols;
    s.tall = rows > cols;
    s.padded_rows = up(rows, kStepK);
    s.padded_cols = up(cols, kStepK);
    s.small = s.tall ? s.padded_cols : s.padded_rows;
    s.large = s.tall ? s.padded_rows : s.padded_cols;
    s.norm_tiles = (rows * cols + kNormTile - 1) / kNormTile;
    return s;
}

// A matrix that one block takes as a whole.
bool fits_a_block(const Shape& s) { return s.small <= kSmallSide && s.large <= kSmallLong; }

// Matrices at a time: their places travel in the kernel arguments, and no launch over their elements,
// eight or more a work-item, comes near 2^32 work-items.
int64_t group_of(int64_t count, const Shape& s) {
    constexpr int64_t kMostAtOnce = (int64_t)1 << 33;
    int64_t most = kMostAtOnce / (s.padded_rows * s.padded_cols);
    most = most < 1 ? 1 : most < kMuonBatch ? most : kMuonBatch;
    return count < most ? count : most;
}

// The parts of split tiles: at most kCus of 256 KiB, or 2 kCus of 64 KiB or 16 KiB.
constexpr int kCus = 256;
constexpr size_t kPartialBytes = (size_t)kCus * 256 * 256 * 4;

// Panels of matrices with a small side: about two blocks a CU, each with as many panels as that takes.
Panels panels_for(int64_t group, const Shape& s) {
    Panels p{};
    const int64_t small = s.tall ? s.cols : s.rows, large = s.tall ? s.rows : s.cols;
    p.rows = (int)s.rows;
    p.cols = (int)s.cols;
    p.k = (int)up(small, 32);
    p.count = (int)((large + kPanel - 1) / kPanel);
    p.per = (int)((group * p.count + 2 * kCus - 1) / (2 * kCus));
    if (p.per > p.count) p.per = p.count;
    p.parts = (p.count + p.per - 1) / p.per;
    return p;
}
// The blocks of the largest number of parts that `group` matrices or fewer have.
int64_t most_parts(int64_t group, const Shape& s) {
    const int64_t panels = (int64_t)panels_for(1, s).count;
    return group * panels < 3 * kCus ? group * panels : 3 * kCus;
}

Coefficients coefficients(const double* q) { return Coefficients{(float)(q[0] * kScaleA), (float)q[1], (float)(q[2] / kScaleA)}; }

// Whether two steps go at once: X <- S1 S0 X with A1 = S0 A0 S0 in place of S0 X and (S0 X)(S0 X)^T.
// That is three more symmetric products of the small side for the two of the long one that a step has
// with X: 3 m^2 (n - m) fewer operations a pair and matrix, and a launch more.  Where those operations
// outweigh it, measured one at a time and in pairs (us for five steps):
//   n >= 8 m: 1 x 129 x 4000 132, 121; 1 x 384 x 3136 144, 136; 20 x 200 x 2000 182, 162
//   n >= 2.5 m: 1 x 768 x 2304 169, 170; 4 x 640 x 1664 175, 171; 1 x 1024 x 4096 235, 224;
//     16 x 640 x 1664 422, 379; 12 x 768 x 2304 510, 449; but 8 x 256 x 1024 110, 112
//   n >= 1.5 m: 24 x 1024 x 1536 1024, 983; but 1 x 1024 x 2048 176, 189; 1 x 2048 x 3200 482, 502;
//     5 x 777 x 1531 245, 250
bool in_pairs(int64_t group, const Shape& s) {
    const int64_t m = s.tall ? s.cols : s.rows, n = s.tall ? s.rows : s.cols;
    const int64_t saved = group * m * m * (n - m);
    return n >= 8 * m || (2 * n >= 5 * m && saved >= (int64_t)1 << 30) || (2 * n >= 3 * m && saved >= (int64_t)1 << 33);
}

struct Workspace { size_t partial, scale, x[2], a, s, t, parts, bytes; };
Workspace workspace_for(int64_t group, const Shape& s) {
    Workspace w{};
    if (fits_a_block(s)) return w;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += (bytes + 255) / 256 * 256; return o; };
    w.partial = take((size_t)8 * group * s.norm_tiles);
    w.scale = take((size_t)8 * group);
    if (s.small <= kSmallSide) {
        const Panels p = panels_for(group, s);
        w.x[0] = take((size_t)2 * group * p.count * p.k * kPanel);
        w.a = take((size_t)2 * group * kSmallSide * kSmallPitch);
        w.parts = take((size_t)16 * most_parts(group, s) * kPartVectors);
        w.bytes = at;
        return w;
    }
    for (int k = 0; k < 2; ++k) w.x[k] = take((size_t)2 * group * s.small * s.large);
    w.a = take((size_t)2 * group * s.small * s.small);
    w.s = take((size_t)2 * group * s.small * s.small);
    if (in_pairs(group, s)) w.t = take((size_t)2 * group * s.small * s.small);
    w.parts = take(kPartialBytes);
    w.bytes = at;
    return w;
}

using Large = Form<256, 2, 4, 2>;                // a block a CU
using Medium = Form<128, 2, 2, 2>;               // two
using Small = Form<64, 2, 2, 4>;                 // two

// What a round of blocks takes, in us: a part for each step of 64 k, from the one where the round
// has few blocks to the one where it has them all, and the rest.  Measured with 1 to 512 blocks of
// 64 to 4096 k and with many rounds.
struct Cost { int side, slots; double few, full, rest; };
constexpr Cost kCosts[] = {{256, kCus, 1.2, 1.75, 8.0}, {128, 2 * kCus, 0.55, 1.1, 4.0}, {64, 2 * kCus, 0.27, 0.42, 2.5}};
struct Choice { int form; int64_t whole, split; int parts; double us; };

// The form and the split that take the least: the tiles of the last, partly filled round may be cut
// along k into as many parts as fill it.  (Two products of 4096 x 4096 x 11008, symmetric: 272 tiles
// of 256 in 493 us, the last 16 of them in 16 parts each 366 us; 20 of 64 x 64 x 10048: 44.5 us, in 20
// parts each 17.6; twelve of 768 x 768 x 768: 25 us in tiles of 256, 13.3 in 128, 18 in 64.)
Choice choose(int64_t group, int64_t M, int64_t N, int64_t K, bool half) {
    Choice best{};
    best.us = 1e30;
    const int64_t steps = K / kStepK;
    for (int f = 0; f < 3; ++f) {
        const Cost& c = kCosts[f];
        const int64_t down = (M + c.side - 1) / c.side, across = (N + c.side - 1) / c.side;
        const int64_t tiles = group * (half ? down * (down + 1) / 2 : down * across);
        const int64_t rounds = tiles / c.slots, tail = tiles % c.slots;
        auto round = [&](int64_t blocks, int64_t k) { return (c.few + (c.full - c.few) * blocks / c.slots) * k + c.rest; };
        const double before = 3.0 + rounds * round(c.slots, steps);
        auto take = [&](int parts, double us) {
            if (us < best.us) best = Choice{f, parts > 1 ? rounds * c.slots : tiles, parts > 1 ? tail : 0, parts, us};
        };
        take(1, before + (tail ? round(tail, steps) : 0.0));
        const int64_t most = tail ? c.slots / tail : 0;
        for (int64_t parts = 2; parts <= most && 2 * parts <= steps; ++parts) {
            // joining: a launch, and the sums written and read back at 4 and 5 TB/s
            const double bytes = (double)parts * tail * c.side * c.side * 4.0;
            take((int)parts, before + round(tail * parts, (steps + parts - 1) / parts) + 5.0 + bytes * (1e6 / 4e12 + 1e6 / 5e12));
        }
    }
    return best;
}

template <class F, bool TL, bool TR, class E>
int launch(const char* who, const Choice& c, int64_t group, Operand L, Operand R, int64_t M, int64_t N, int64_t K, bool half, void* parts,
           const E& e, hipStream_t stream) {
    Tiles t{};
    t.down = (int)((M + F::kSide - 1) / F::kSide);
    t.across = (int)((N + F::kSide - 1) / F::kSide);
    t.half = half;
    t.per = half ? t.down * (t.down + 1) / 2 : t.down * t.across;
    t.whole = c.whole;
    t.parts = c.parts;
    t.partial = static_cast<f32x4*>(parts);
    hipLaunchKernelGGL((k_product<F, TL, TR, E>), dim3((unsigned)(c.whole + c.split * c.parts)), dim3(64 * F::kWaves), 0, stream, L, R, M, N,
                       K, t, e);
    if (int rc = launched(who)) return rc;
    if (c.split == 0) return GSZ_OK;
    hipLaunchKernelGGL((k_join<F, E>), dim3((unsigned)(c.split * F::kWaves)), dim3(64), 0, stream, M, N, t, e);
    return launched(who);
}

// One product over a group: C[i, j] = sum_k L[i, k] R[j, k], i < M, j < N.
template <bool TL, bool TR, class E>
int product(const char* who, int64_t group, Operand L, Operand R, int64_t M, int64_t N, int64_t K, bool half, void* parts, const E& e,
            hipStream_t stream, const Choice* given = nullptr) {
    const Choice c = given ? *given : choose(group, M, N, K, half);
    switch (c.form) {
        case 0: return launch<Large, TL, TR>(who, c, group, L, R, M, N, K, half, parts, e, stream);
        case 1: return launch<Medium, TL, TR>(who, c, group, L, R, M, N, K, half, parts, e, stream);
        default: return launch<Small, TL, TR>(who, c, group, L, R, M, N, K, half, parts, e, stream);
    }
}

// All steps of a group whose scaled matrices lie at w.x[0]; the last product goes to `last`.
template <class E>
int newton_schulz(const char* who, int64_t group, const Shape& s, const Workspace& w, char* base, int steps, const double* ns, const E& last, hipStream_t stream) {
    _Float16* A = reinterpret_cast<_Float16*>(base + w.a);
    _Float16* S = reinterpret_cast<_Float16*>(base + w.s);
    _Float16* T = reinterpret_cast<_Float16*>(base + w.t);
    void* parts = base + w.parts;
    const int64_t size = s.small * s.large, square = s.small * s.small;
    auto small = [&](_Float16* m) { return Operand{m, square, s.small}; };
    // to = scale l r, symmetric
    auto multiply = [&](_Float16* l, _Float16* r, _Float16* to, float scale) {
        return product<false, false>(who, group, small(l), small(r), s.small, s.small, s.small, true, parts, StoreHalf<true>{to, square, s.small, scale}, stream);
    };
    auto polynomial = [&](_Float16* of, _Float16* to, const double* q) {
        const Coefficients f = coefficients(q);
        return product<false, false>(who, group, small(of), small(of), s.small, s.small, s.small, true, parts,
                                     StorePolynomial{of, to, square, s.small, f.a, f.b, f.c}, stream);
    };
    const bool pairs = in_pairs(group, s);
    int rc;
    for (int k = 0, turn = 0; k < steps; ++turn) {
        const double* q = ns + 3 * k;
        _Float16* in = reinterpret_cast<_Float16*>(base + w.x[turn & 1]);
        _Float16* out = reinterpret_cast<_Float16*>(base + w.x[~turn & 1]);
        const Operand x{in, size, s.padded_cols};
        const StoreHalf<true> gram{A, square, s.small, kScaleA / (kScaleX * kScaleX)};
        rc = s.tall ? product<true, true>(who, group, x, x, s.small, s.small, s.large, true, parts, gram, stream)
                    : product<false, false>(who, group, x, x, s.small, s.small, s.large, true, parts, gram, stream);
        if (rc || (rc = polynomial(A, S, q))) return rc;
        // of an odd number of steps the one before the last pair goes alone
        const bool pair = pairs && k + 2 <= steps && !(steps % 2 && k + 3 == steps && steps > 3);
        _Float16* factor = S;
        float scale = kScaleA;
        if (pair) {
            if ((rc = multiply(S, A, T, 1.0f / kScaleA))) return rc;                                 // S0 A0
            if ((rc = multiply(S, T, A, 1.0f / kScaleA))) return rc;                                 // A1
            if ((rc = polynomial(A, T, q + 3))) return rc;                                           // S1
            if ((rc = multiply(T, S, A, kScaleP / (kScaleA * kScaleA)))) return rc;                  // S1 S0
            factor = A;
            scale = kScaleP;
        }
        k += pair ? 2 : 1;
        auto apply = [&](const auto& e) {
            return s.tall ? product<false, false>(who, group, x, small(factor), s.large, s.small, s.small, false, parts, e, stream)
                          : product<false, true>(who, group, small(factor), x, s.small, s.large, s.small, false, parts, e, stream);
        };
        if (k < steps) {
            rc = apply(StoreHalf<false>{out, size, s.padded_cols, 1.0f / scale});
        } else {
            E e = last;
            e.scale = 1.0f / (scale * kScaleX);
            rc = apply(e);
        }
        if (rc) return rc;
    }
    return GSZ_OK;
}

constexpr double kUsual[3] = {3.4445, -4.7750, 2.0315};

// The steps' coefficients: the caller's, or the usual ones for every step.
int check_steps(const char* who, int32_t steps, const double* ns, double eps, double out[3 * kMostSteps]) {
    if (steps < 1 || steps > kMostSteps) { set_error("%s: steps %d is not in [1, %d]", who, (int)steps, kMostSteps); return GSZ_ERR_INVALID_ARG; }
    if (!(eps >= 1e-30 && eps <= 1e30)) { set_error("%s: eps %g is not in [1e-30, 1e30]", who, eps); return GSZ_ERR_INVALID_ARG; }
    for (int k = 0; k < 3 * steps; ++k) {
        out[k] = ns ? ns[k] : kUsual[k % 3];
        if (!(std::fabs(out[k]) <= 1e4)) return bad_arg(who, "a coefficient is not within 1e4 of 0");
    }
    return GSZ_OK;
}

int check_workspace(const char* who, const void* ws, size_t have, size_t need) {
    if (need == 0) return GSZ_OK;
    if (!ws || have < need) { set_error("%s: workspace of %zu bytes required", who, need); return GSZ_ERR_SIZE; }
    if (off_by(ws, 16)) { set_error("%s: workspace is not 16-byte aligned", who); return GSZ_ERR_MISALIGNED; }
    return GSZ_OK;
}

// The norm's launches, as every form but the smallest begins.
template <class In>
int scale_of(const char* who, int64_t m, const Shape& s, const Workspace& w, char* base, double eps, const In& in, hipStream_t stream) {
    double* partial = reinterpret_cast<double*>(base + w.partial);
    hipLaunchKernelGGL((k_norm<In>), dim3((unsigned)(m * s.norm_tiles)), dim3(kUpdateBlock), 0, stream, in, s.rows * s.cols, (unsigned)s.norm_tiles, partial);
    if (int e = launched(who)) return e;
    hipLaunchKernelGGL(k_scale, dim3((unsigned)m), dim3(kBlock), 0, stream, partial, s.norm_tiles, eps, reinterpret_cast<double*>(base + w.scale));
    return launched(who);
}

template <bool TALL, class In, class E>
int panel_steps(const char* who, int64_t m, const Panels& p, const double* scale, int steps, const double* q, const In& in, const E& last,
                hipStream_t stream) {
    const dim3 grid((unsigned)(m * p.parts)), block(64 * kSmallWaves);
    hipLaunchKernelGGL((k_panels<TALL, true, false, In, E>), grid, block, 0, stream, in, last, p, scale, Coefficients{});
    if (int e = launched(who)) return e;
    for (int k = 0; k < steps; ++k) {
        hipLaunchKernelGGL(k_panel_sum, dim3((unsigned)(m * (kPartVectors / 64))), dim3(64), 0, stream, p);
        if (int e = launched(who)) return e;
        const Coefficients c = coefficients(q + 3 * k);
        if (k + 1 < steps) hipLaunchKernelGGL((k_panels<TALL, false, false, In, E>), grid, block, 0, stream, in, last, p, scale, c);
        else hipLaunchKernelGGL((k_panels<TALL, false, true, In, E>), grid, block, 0, stream, in, last, p, scale, c);
        if (int e = launched(who)) return e;
    }
    return GSZ_OK;
}

template <class In, class E>
int run_panels(const char* who, int64_t m, const Shape& s, const Workspace& w, char* base, int steps, const double* q, double eps, const In& in,
               const E& last, hipStream_t stream) {
    if (int e = scale_of(who, m, s, w, base, eps, in, stream)) return e;
    Panels p = panels_for(m, s);
    p.x = reinterpret_cast<_Float16*>(base + w.x[0]);
    p.a = reinterpret_cast<_Float16*>(base + w.a);
    p.partial = reinterpret_cast<f32x4*>(base + w.parts);
    const double* scale = reinterpret_cast<double*>(base + w.scale);
    return s.tall ? panel_steps<true>(who, m, p, scale, steps, q, in, last, stream) : panel_steps<false>(who, m, p, scale, steps, q, in, last, stream);
}

// Orthogonalises m matrices from `in` to `last`.
template <class In, class E>
int run_group(const char* who, int64_t m, const Shape& s, const Workspace& w, char* base, int steps, const double* q, double eps, const In& in,
              const E& last, hipStream_t stream) {
    if (fits_a_block(s)) {
        SmallSteps z{};
        z.count = steps;
        for (int k = 0; k < steps; ++k) z.of[k] = coefficients(q + 3 * k);
        auto go = [&](auto tall, auto is_long) {
            hipLaunchKernelGGL((k_small<decltype(tall)::value, decltype(is_long)::value, In, E>), dim3((unsigned)m), dim3(64 * kSmallWaves), 0, stream,
                               in, last, (int)s.rows, (int)s.cols, eps, z);
        };
        const bool is_long = s.large > kSmallPitch;
        if (s.tall) is_long ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
        else is_long ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
        return launched(who);
    }
    if (s.small <= kSmallSide) return run_panels(who, m, s, w, base, steps, q, eps, in, last, stream);
    if (int e = scale_of(who, m, s, w, base, eps, in, stream)) return e;
    const double* scale = reinterpret_cast<double*>(base + w.scale);
    const Padded p{s.rows, s.cols, s.padded_cols, s.padded_rows * s.padded_cols / 8};
    const unsigned tiles = (unsigned)((p.vectors + kUpdateBlock - 1) / kUpdateBlock);
    hipLaunchKernelGGL((k_scaled<In>), dim3((unsigned)(m * tiles)), dim3(kUpdateBlock), 0, stream, in, p, tiles, scale, reinterpret_cast<_Float16*>(base + w.x[0]));
    if (int e = launched(who)) return e;
    return newton_schulz(who, m, s, w, base, steps, q, last, stream);
}

}  // namespace

extern "C" int gsz_muon_workspace_bytes(int64_t count, int64_t rows, int64_t cols, size_t* out) {
    const char* who = "gsz_muon_workspace_bytes";
    const int rc = check_shape(who, count, rows, cols);
    if (rc) return rc;
    if (!out) return bad_arg(who, "NULL output");
    const Shape s = shape_for(rows, cols);
    *out = count && rows && cols ? workspace_for(group_of(count, s), s).bytes : 0;
    return GSZ_OK;
}

extern "C" int gsz_orthogonalize(const void* x, int32_t type, int64_t count, int64_t rows, int64_t cols, int32_t steps,
                                 const double* ns, double eps, uint16_t* out, void* ws, size_t ws_bytes, hipStream_t stream) {
    const char* who = "gsz_orthogonalize";
    const int64_t size = value_size(type);
    if (!size) return bad_arg(who, "unknown value type");
    int rc = check_shape(who, count, rows, cols);
    if (rc) return rc;
    double q[3 * kMostSteps];
    if ((rc = check_steps(who, steps, ns, eps, q))) return rc;
    const int64_t n = rows * cols;
    if (count == 0 || n == 0) return check_device(who);
    if (!x || !out) return bad_arg(who, "NULL buffer");
    if (off_by(x, size) || off_by(out, 2)) { set_error("%s: a buffer is not aligned to its values", who); return GSZ_ERR_MISALIGNED; }
    const Shape s = shape_for(rows, cols);
    const int64_t group = group_of(count, s);
    const Workspace w = workspace_for(group, s);
    const size_t need = w.bytes;
    if ((rc = check_workspace(who, ws, ws_bytes, need))) return rc;
    const Span in{x, count * n * size}, written{out, count * n * 2}, scratch{ws, (int64_t)need};
    if ((x != out || size != 2) && overlap(written, in)) return bad_arg(who, "out overlaps x");
    if (overlap(scratch, in) || overlap(scratch, written)) return bad_arg(who, "ws overlaps x or out");
    if ((rc = check_device(who))) return rc;

    for (int64_t first = 0; first < count; first += group) {
        const int64_t m = count - first < group ? count - first : group;
        const StoreResult last{out + first * n, rows, cols, 1.0f / (kScaleA * kScaleX)};
        rc = size == 2 ? run_group(who, m, s, w, static_cast<char*>(ws), steps, q, eps, Values<uint16_t>{static_cast<const uint16_t*>(x) + first * n, n}, last, stream)
                       : run_group(who, m, s, w, static_cast<char*>(ws), steps, q, eps, Values<float>{static_cast<const float*>(x) + first * n, n}, last, stream);
        if (rc) return rc;
    }
    return GSZ_OK;
}

extern "C" int gsz_muon_step(const gsz_plan* plan, const int32_t* tensors, int32_t count, int64_t rows, int64_t cols,
                             float* master, float* momentum, const float* g, const float* coef, const gsz_muon_hp* hp,
                             uint16_t* params, void* ws, size_t ws_bytes, hipStream_t stream) {
    const char* who = "gsz_muon_step";
    if (!plan || !hp) return bad_arg(who, "plan or hp is NULL");
    int rc = check_shape(who, count, rows, cols);
    if (rc) return rc;
    double q[3 * kMostSteps];
    if ((rc = check_steps(who, hp->steps, hp->ns, hp->eps, q))) return rc;
    if (hp->nesterov != 0 && hp->nesterov != 1) return bad_arg(who, "nesterov is neither 0 nor 1");
    const float mu = (float)hp->momentum, decay = (float)(1.0 - hp->lr * hp->weight_decay), rate = (float)(hp->lr * hp->scale);
    if (!std::isfinite(mu) || !std::isfinite(decay) || !std::isfinite(rate)) return bad_arg(who, "a hyperparameter is not finite in fp32");
    if (count > 0 && !tensors) return bad_arg(who, "tensors is NULL");
    const int64_t n = rows * cols;
    const int64_t T = (int64_t)plan->numel.size();
    try {
        std::vector<bool> seen((size_t)T, false);
        for (int32_t k = 0; k < count; ++k) {
            const int32_t t = tensors[k];
            if (t < 0 || t >= T) { set_error("%s: tensor %d is not in the plan", who, (int)t); return GSZ_ERR_INVALID_ARG; }
            if (seen[t]) { set_error("%s: tensor %d is given twice", who, (int)t); return GSZ_ERR_INVALID_ARG; }
            seen[t] = true;
            if (plan->numel[t] != n) {
                set_error("%s: tensor %d has %lld elements, not %lld x %lld", who, (int)t, (long long)plan->numel[t], (long long)rows, (long long)cols);
                return GSZ_ERR_SIZE;
            }
        }
    } catch (...) {
        set_error("%s: out of host memory", who);
        return GSZ_ERR_NO_MEMORY;
    }
    if (count == 0 || n == 0) return check_device(who);
    if (!master || !momentum || !g || !coef || !params) return bad_arg(who, "NULL buffer");
    if (off_by(master, 16) || off_by(momentum, 16) || off_by(g, 16) || off_by(params, 16) || off_by(coef, 4)) {
        set_error("%s: a device pointer is not 16-byte aligned", who);
        return GSZ_ERR_MISALIGNED;
    }
    const Shape s = shape_for(rows, cols);
    const int64_t group = group_of(count, s);
    const Workspace w = workspace_for(group, s);
    const size_t need = w.bytes;
    if ((rc = check_workspace(who, ws, ws_bytes, need))) return rc;
    const int64_t len = plan->flat_len;
    const Span spans[] = {{master, len * 4}, {momentum, len * 4}, {params, len * 2}, {ws, (int64_t)need}, {g, len * 4}, {coef, 4}};
    for (int a = 0; a < 4; ++a)
        for (int b = a + 1; b < 6; ++b)
            if (overlap(spans[a], spans[b])) return bad_arg(who, "buffers overlap");
    if ((rc = check_device(who))) return rc;

    for (int64_t first = 0; first < count; first += group) {
        const int m = (int)(count - first < group ? count - first : group);
        Momentum in{momentum, g, coef, mu, hp->nesterov, {}};
        StoreUpdate last{master, params, {}, rows, cols, 1.0f / (kScaleA * kScaleX), decay, rate};
        for (int k = 0; k < m; ++k) in.places.at[k] = last.places.at[k] = plan->tensor_off[tensors[first + k]];
        if ((rc = run_group(who, m, s, w, static_cast<char*>(ws), hp->steps, q, hp->eps, in, last, stream))) return rc;
    }
    return GSZ_OK;
}
