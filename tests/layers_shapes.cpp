// One lookup or gradient of given sizes, kernels and entry points run on the CPU as in
// layers_host, against a plain reference, in buffers of exactly the documented sizes.
//
//   layers_shapes lookup n rows dim table_type out_type drop seed
//   layers_shapes grad   n rows dim accumulate ids        drop seed
//     ids 0: anywhere, some outside the table; 1: nine in ten the last row; 2: the ends
#define main layers_host_main
#include "layers_host.cpp"
#undef main

int main(int argc, char** argv) {
    const std::string op = argv[1];
    const int64_t n = std::atoll(argv[2]), rows = std::atoll(argv[3]), dim = std::atoll(argv[4]);
    const int a = std::atoi(argv[5]), b = std::atoi(argv[6]);
    const double p = std::atoi(argv[7]) ? 0.3 : 0.0, scale = 2.0;
    std::mt19937_64 g(std::strtoull(argv[8], nullptr, 10));
    const uint64_t rng[2] = {g(), g()};
    g_key[0] = (uint32_t)rng[0]; g_key[1] = (uint32_t)(rng[0] >> 32); g_step = (uint32_t)rng[1];
    g_site = (uint32_t)g();
    const uint64_t T = (uint64_t)std::floor(p * 4294967296.0);
    const double c0 = scale / (1.0 - (double)T / 4294967296.0);
    auto kept = [&](uint64_t e) { return !T || number(e) >= T; };
    std::unique_ptr<int32_t[]> ids(new int32_t[n]);
    for (int64_t i = 0; i < n; ++i) {
        const int64_t ends[] = {0, rows - 1, rows - 2, rows, -1};
        ids[i] = op == "grad" && b == 1 && g() % 10 ? rows - 1 : op == "grad" && b == 2 ? ends[g() % 5] : (int64_t)(g() % (rows + 2)) - 1;
    }
    auto is_row = [&](int64_t i) { return ids[i] >= 0 && ids[i] < rows; };
    int64_t bad = 0, checked = 0;
    auto check = [&](double got, double ref, double tol) {
        ++checked;
        if (!(std::fabs(got - ref) <= tol) && ++bad <= 5) std::printf("got %g, want %g\n", got, ref);
    };
    if (op == "lookup") {
        Buf table(rows * dim, a), out(n * dim, b);
        for (int64_t i = 0; i < rows * dim; ++i) table.set(i, (double)(int64_t)(g() % 17) - 8);
        if (gsz_embedding_lookup(table.p.get(), a, rows, dim, ids.get(), GSZ_TYPE_I32, n, scale, p, T ? rng : nullptr, g_site, out.p.get(), b, nullptr)) return 2;
        for (int64_t i = 0; i < n; ++i)
            for (int64_t c = 0; c < dim; ++c) {
                const double ref = is_row(i) && kept(i * dim + c) ? table.get(ids[i] * dim + c) * c0 : 0;
                // the constant and the product round in fp32, out once
                check(out.get(i * dim + c), ref, std::fabs(ref) * (2.5 * std::ldexp(1.0, -24) + (b == GSZ_TYPE_BF16 ? std::ldexp(1.0, -8) : 0)));
            }
    } else {
        Buf grad(rows * dim, GSZ_TYPE_F32), dy(n * dim, GSZ_TYPE_BF16);
        std::vector<double> want(rows * dim), size(rows * dim);
        std::vector<int64_t> terms(rows);
        for (int64_t i = 0; i < rows * dim; ++i) { grad.set(i, (double)(g() % 5)); want[i] = a ? grad.get(i) : 0; }
        for (int64_t i = 0; i < n; ++i) {
            if (is_row(i)) ++terms[ids[i]];
            for (int64_t c = 0; c < dim; ++c) {
                dy.set(i * dim + c, (double)(int64_t)(g() % 17) - 8);
                if (!is_row(i) || !kept(i * dim + c)) continue;
                want[ids[i] * dim + c] += dy.get(i * dim + c) * c0;
                size[ids[i] * dim + c] += std::fabs(dy.get(i * dim + c) * c0);
            }
        }
        size_t bytes = 0;
        if (gsz_embedding_workspace_bytes(n, rows, dim, &bytes)) return 2;
        std::unique_ptr<char, void (*)(void*)> ws((char*)std::aligned_alloc(16, (bytes + 16) / 16 * 16), std::free);
        std::memset(ws.get(), 0xEE, bytes);
        if (gsz_embedding_grad(ids.get(), GSZ_TYPE_I32, n, dy.p.get(), GSZ_TYPE_BF16, rows, dim, scale, p, T ? rng : nullptr, g_site,
                               grad.p.get(), GSZ_TYPE_F32, a, ws.get(), bytes, nullptr)) return 2;
        for (int64_t i = 0; i < rows * dim; ++i)
            check(grad.get(i), want[i], (size[i] * (terms[i / dim] + 3) + std::fabs(want[i])) * 1.1 * std::ldexp(1.0, -24));
    }
    std::printf("%ld values, %ld wrong\n", (long)checked, (long)bad);
    return bad ? 1 : 0;
}
