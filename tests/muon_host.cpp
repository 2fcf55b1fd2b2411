// The orthogonalising entry points and kernels themselves, run on the CPU (host_gpu/,
// host_matrix/) in buffers of exactly the documented sizes, against a plain reference in
// double.  Built with AddressSanitizer: an access outside a buffer ends the program.
//
//   muon_host count rows cols type steps seed      orthogonalises; type 0 bf16, 1 fp32
//   muon_host count rows cols step nesterov seed   a whole update ("step": the word)
#include "gsz_muon.hip"
#include "plan.cpp"

#include <memory>
#include <random>
#include <string>

extern "C" __bf16 __truncsfbf2(float f) {
    const uint16_t h = (uint16_t)bf16_rne(f);
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}

using M = std::vector<double>;
static M turned(const M& x, int64_t r, int64_t c) {
    M y(x.size());
    for (int64_t i = 0; i < r; ++i) for (int64_t j = 0; j < c; ++j) y[j * r + i] = x[i * c + j];
    return y;
}
static M orthogonal(M x, int64_t r, int64_t c, int steps, double eps) {
    const bool tall = r > c;
    if (tall) { x = turned(x, r, c); std::swap(r, c); }
    double s = 0;
    for (double v : x) s += v * v;
    for (double& v : x) v /= std::sqrt(s) + eps;
    for (int k = 0; k < steps; ++k) {
        M A(r * r), S(r * r), y(r * c);
        for (int64_t i = 0; i < r; ++i) for (int64_t j = 0; j < r; ++j) {
            double t = 0;
            for (int64_t l = 0; l < c; ++l) t += x[i * c + l] * x[j * c + l];
            A[i * r + j] = t;
        }
        for (int64_t i = 0; i < r; ++i) for (int64_t j = 0; j < r; ++j) {
            double t = 0;
            for (int64_t l = 0; l < r; ++l) t += A[i * r + l] * A[l * r + j];
            S[i * r + j] = -4.7750 * A[i * r + j] + 2.0315 * t + (i == j ? 3.4445 : 0.0);
        }
        for (int64_t i = 0; i < r; ++i) for (int64_t l = 0; l < r; ++l) for (int64_t j = 0; j < c; ++j) y[i * c + j] += S[i * r + l] * x[l * c + j];
        x = y;
    }
    return tall ? turned(x, r, c) : x;
}
static double off(const M& got, const M& want) {
    double d = 0, n = 0;
    for (size_t i = 0; i < got.size(); ++i) { d += (got[i] - want[i]) * (got[i] - want[i]); n += want[i] * want[i]; }
    return std::sqrt(d / (n > 0 ? n : 1));
}
static float bf(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

int main(int argc, char** argv) {
    (void)argc;
    const int64_t count = std::atoll(argv[1]), rows = std::atoll(argv[2]), cols = std::atoll(argv[3]), n = rows * cols;
    const std::string kind = argv[4];
    std::mt19937_64 gen(std::strtoull(argv[6], nullptr, 10) + 99);
    std::normal_distribution<double> normal;
    size_t bytes = 0;
    if (gsz_muon_workspace_bytes(count, rows, cols, &bytes)) return 2;
    std::unique_ptr<char[]> raw(new char[bytes + 16]);
    char* ws = raw.get() + (16 - reinterpret_cast<uintptr_t>(raw.get()) % 16) % 16;
    std::memset(ws, 0xFF, bytes);                        // NaNs: nothing may count on zeros
    double worst = 0;
    if (kind != "step") {
        const int type = std::atoi(argv[4]), steps = std::atoi(argv[5]);
        std::unique_ptr<char[]> x(new char[count * n * value_size(type)]);
        std::unique_ptr<uint16_t[]> out(new uint16_t[count * n]);
        M all(count * n);
        for (int64_t i = 0; i < count * n; ++i) {
            const float v = (float)normal(gen);
            if (type == GSZ_TYPE_F32) { reinterpret_cast<float*>(x.get())[i] = v; all[i] = v; }
            else { const uint16_t h = (uint16_t)bf16_rne(v); reinterpret_cast<uint16_t*>(x.get())[i] = h; all[i] = bf(h); }
        }
        const int rc = gsz_orthogonalize(x.get(), type, count, rows, cols, steps, nullptr, 1e-7, out.get(), ws, bytes, nullptr);
        if (rc) { std::printf("refused: %d\n", rc); return 2; }
        for (int64_t b = 0; b < count; ++b) {
            M got(n), in(all.begin() + b * n, all.begin() + (b + 1) * n);
            for (int64_t i = 0; i < n; ++i) got[i] = bf(out[b * n + i]);
            worst = std::max(worst, off(got, orthogonal(in, rows, cols, steps, 1e-7)));
        }
    } else {
        const int nesterov = std::atoi(argv[5]);
        std::vector<int64_t> numel;
        std::vector<int32_t> list;
        for (int64_t b = 0; b < count; ++b) { numel.push_back(n); list.push_back((int32_t)numel.size() - 1); numel.push_back(3 + b); }
        gsz_plan* plan;
        if (gsz_plan_create(numel.data(), (int32_t)numel.size(), 1000, 2, 8, &plan)) return 2;
        const int64_t len = plan->flat_len;
        struct Free { void operator()(void* p) const { std::free(p); } };
        std::vector<std::unique_ptr<void, Free>> all;
        auto bytes_of = [&](int64_t size) { all.emplace_back(std::aligned_alloc(16, size)); return all.back().get(); };
        auto floats = [&](double std) {
            float* p = static_cast<float*>(bytes_of(len * 4));
            for (int64_t i = 0; i < len; ++i) p[i] = (float)(std * normal(gen));
            return p;
        };
        float *w = floats(0.02), *m = floats(1.0), *g = floats(0.3), coef = 0.75f;
        uint16_t* p = static_cast<uint16_t*>(bytes_of(len * 2));
        for (int64_t i = 0; i < len; ++i) p[i] = 0x1234;
        const std::vector<float> w0(w, w + len), m0(m, m + len);
        gsz_muon_hp hp{0.02, 0.95, 0.1, 0.2 * std::sqrt((double)std::max(rows, cols)), 1e-7, nullptr, 5, nesterov};
        const int rc = gsz_muon_step(plan, list.data(), (int32_t)count, rows, cols, w, m, g, &coef, &hp, p, ws, bytes, nullptr);
        if (rc) { std::printf("refused: %d\n", rc); return 2; }
        std::vector<bool> touched(len, false);
        for (int32_t t : list) {
            const int64_t at = plan->tensor_off[t];
            M u(n), dw(n), want(n);
            for (int64_t i = 0; i < n; ++i) {
                const double gc = (double)g[at + i] * coef, mm = 0.95 * m0[at + i] + gc;
                if (std::fabs(m[at + i] - mm) > 1e-6 * (std::fabs(mm) + std::fabs(gc))) { std::printf("momentum\n"); return 1; }
                u[i] = nesterov ? gc + 0.95 * mm : mm;
                touched[at + i] = true;
            }
            const M o = orthogonal(u, rows, cols, 5, 1e-7);
            for (int64_t i = 0; i < n; ++i) {
                dw[i] = w[at + i] - (double)w0[at + i] * (1.0 - 0.02 * 0.1);
                want[i] = -0.02 * hp.scale * o[i];
                if (p[at + i] != bf16_rne(w[at + i])) { std::printf("parameter\n"); return 1; }
            }
            worst = std::max(worst, off(dw, want));
        }
        for (int64_t i = 0; i < len; ++i)
            if (!touched[i] && (w[i] != w0[i] || m[i] != m0[i] || p[i] != 0x1234)) { std::printf("wrote outside\n"); return 1; }
        gsz_plan_destroy(plan);
    }
    std::printf("off by %.3g\n", worst);
    return worst < 6e-3 ? 0 : 1;
}
