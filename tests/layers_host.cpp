// The embedding and dropout entry points and kernels themselves, run on the CPU
// (host_gpu/hip/hip_runtime.h) in buffers of exactly the documented sizes, against
// a plain reference in double.  Built with AddressSanitizer: an access outside a
// buffer ends the program.
//
//   layers_host op seed   one random case of lookup, grad or dropout
#include "gsz_layers.hip"

#include <memory>
#include <random>

static uint32_t g_key[2], g_step, g_site;
static uint64_t number(uint64_t e) {                  // u(e), from the definition
    uint64_t u = 0;
    for (int top = 0; top < 2; ++top) {
        uint64_t c[4] = {(uint32_t)(e >> 3), (e >> 3 >> 32) | (uint64_t)top << 31, g_site, g_step};
        uint32_t k0 = g_key[0], k1 = g_key[1];
        for (int r = 0; r < 10; ++r, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
            const uint64_t a = 0xD2511F53ull * c[0], b = 0xCD9E8D57ull * c[2];
            c[0] = (b >> 32) ^ c[1] ^ k0; c[1] = (uint32_t)b; c[2] = (a >> 32) ^ c[3] ^ k1; c[3] = (uint32_t)a;
        }
        const uint64_t half = c[(e & 7) >> 1] >> 16 * (e & 1) & 0xFFFF;
        u = u << 16 | half;
    }
    return u;
}
extern "C" __bf16 __truncsfbf2(float f) {              // nearest even
    uint32_t u = __float_as_uint(f);
    uint16_t h = (u & 0x7FFFFFFF) > 0x7F800000 ? (u >> 16) | 0x40 : (u + 0x7FFF + (u >> 16 & 1)) >> 16;
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}

struct Buf {                                           // n values of a type, and nothing after them
    std::unique_ptr<char[]> p;
    int type;
    Buf(int64_t n, int t) : p(new char[n * value_size(t) ? n * value_size(t) : 1]), type(t) {}
    double get(int64_t i) const { return type == GSZ_TYPE_F32 ? ((float*)p.get())[i] : load1((uint16_t*)p.get() + i); }
    void set(int64_t i, double v) {
        if (type == GSZ_TYPE_F32) ((float*)p.get())[i] = (float)v;
        else { uint32_t u = __float_as_uint((float)v); ((uint16_t*)p.get())[i] = (uint16_t)(u >> 16); }
    }
};

int main(int argc, char** argv) {
    const std::string op = argv[1];
    std::mt19937_64 g(std::strtoull(argv[2], nullptr, 10) * 2654435761u + 17);
    auto pick = [&](std::initializer_list<int64_t> v) { return v.begin()[g() % v.size()]; };
    const uint64_t rng[2] = {g(), g()};
    g_key[0] = (uint32_t)rng[0]; g_key[1] = (uint32_t)(rng[0] >> 32); g_step = (uint32_t)rng[1];
    g_site = (uint32_t)g();
    const double p = pick({0, 1}) ? 0.3 : 0.0, scale = pick({0, 1}) ? 1.75 : 1.0;
    const double k = 1.0 / (1.0 - std::floor(p * 4294967296.0) / 4294967296.0);
    const uint64_t T = (uint64_t)std::floor(p * 4294967296.0);
    auto kept = [&](uint64_t e) { return !T || number(e) >= T; };
    auto type = [&] { return (int)pick({GSZ_TYPE_BF16, GSZ_TYPE_F32}); };
    auto value = [&] { return (double)(int64_t)(g() % 17) - 8; };
    int64_t bad = 0, checked = 0;
    auto check = [&](double got, double ref, int t, int64_t terms) {
        ++checked;
        const double tol = (t == GSZ_TYPE_F32 ? 0 : std::ldexp(1.0, -8)) * std::fabs(ref) + 1e-6 * (terms + 1) * (8 + std::fabs(ref));
        if (!(std::fabs(got - ref) <= tol) && ++bad <= 5) std::printf("got %g, want %g\n", got, ref);
    };

    if (op == "dropout") {
        const int64_t n = pick({0, 1, 7, 8, 9, 2047, 2048, 2049, 5000});
        const int t = type();
        const bool add = pick({0, 1}), in_place = pick({0, 1});
        Buf x(n, t), a(n, t), y(n, t);
        std::vector<double> xs(n);
        for (int64_t i = 0; i < n; ++i) { x.set(i, xs[i] = value()); a.set(i, value()); }
        Buf& out = in_place ? x : y;
        if (gsz_dropout(x.p.get(), add ? a.p.get() : nullptr, out.p.get(), n, t, p, T ? rng : nullptr, g_site, nullptr)) return 2;
        for (int64_t i = 0; i < n; ++i) check(out.get(i), (add ? a.get(i) : 0) + (kept(i) ? xs[i] * k : 0), t, 1);
    } else {
        const bool is_grad = op == "grad";
        const int64_t dim = pick({1, 7, 8, 9, 64, 500, 512, 520, 1025, 2060, 8200}), cost = 400000 / dim;
        int64_t n = pick({0, 1, 2, 63, 64, 65, 700, 3000, 8192, 8193, 9001, 20000, 70000, 270001});
        if (n > cost) n = n % (cost + 1);
        if (is_grad && pick({0, 0, 1})) n = n < cost ? cost : n;
        int64_t rows = pick({0, 1, 3, 40, 255, 256, 1000, 1024, 5000, 70000, 1200000});
        if (rows > 2 * cost) rows = rows % (2 * cost + 1);
        const int it = (int)pick({GSZ_TYPE_I32, GSZ_TYPE_I64}), kind = (int)(g() % 4);
        std::vector<int64_t> id(n);
        for (auto& v : id)
            v = kind == 0 || (kind == 1 && g() % 10) ? rows / 2 : kind == 3 ? -1 - (int64_t)(g() % 3) * 7 : (int64_t)(g() % (rows + 2)) - 1;
        std::unique_ptr<char[]> ids(new char[n * id_size(it) ? n * id_size(it) : 1]);
        for (int64_t i = 0; i < n; ++i) {
            if (it == GSZ_TYPE_I64) ((int64_t*)ids.get())[i] = id[i];
            else ((int32_t*)ids.get())[i] = (int32_t)id[i];
        }
        const int bt = type(), st = type();
        Buf big(rows * dim, bt), small(n * dim, st);    // the table or its gradient; the tokens' values
        std::vector<double> want(rows * dim);
        std::vector<int64_t> terms(rows);
        const bool acc = is_grad && pick({0, 1});
        for (int64_t i = 0; i < rows * dim; ++i) { big.set(i, value()); want[i] = acc ? big.get(i) : 0; }
        if (is_grad) {
            for (int64_t i = 0; i < n; ++i)
                for (int64_t c = 0; c < dim; ++c) {
                    const double v = value();
                    small.set(i * dim + c, v);
                    if (id[i] >= 0 && id[i] < rows && kept(i * dim + c)) want[id[i] * dim + c] += v * scale * k;
                }
            for (auto v : id) if (v >= 0 && v < rows) ++terms[v];
            size_t bytes = 0;
            if (gsz_embedding_workspace_bytes(n, rows, dim, &bytes)) return 2;
            void* ws = std::aligned_alloc(256, bytes + 256);       // whole 256-byte units: the end is guarded
            std::free(ws);
            ws = std::aligned_alloc(16, (bytes + 15) / 16 * 16 ? (bytes + 15) / 16 * 16 : 16);
            std::memset(ws, 0xEE, bytes);
            if (gsz_embedding_grad(ids.get(), it, n, small.p.get(), st, rows, dim, scale, p, T ? rng : nullptr, g_site,
                                   big.p.get(), bt, acc, ws, bytes, nullptr)) return 2;
            std::free(ws);
            for (int64_t i = 0; i < rows * dim; ++i) check(big.get(i), want[i], bt, terms[i / dim]);
        } else {
            if (gsz_embedding_lookup(big.p.get(), bt, rows, dim, ids.get(), it, n, scale, p, T ? rng : nullptr, g_site,
                                     small.p.get(), st, nullptr)) return 2;
            for (int64_t i = 0; i < n; ++i)
                for (int64_t c = 0; c < dim; ++c)
                    check(small.get(i * dim + c), id[i] >= 0 && id[i] < rows && kept(i * dim + c) ? big.get(id[i] * dim + c) * scale * k : 0, st, 1);
        }
        std::printf("n %ld rows %ld dim %ld kind %d acc %d: ", (long)n, (long)rows, (long)dim, kind, (int)acc);
    }
    std::printf("%ld values, %ld wrong\n", (long)checked, (long)bad);
    return bad ? 1 : 0;
}
