// The relative position bias entry points and kernels themselves, run on the CPU
// (host_gpu/, host_matrix/) in buffers of exactly the documented sizes, against a plain
// reference in double.  Built with AddressSanitizer: an access outside a buffer ends the program.
//
//   relpos_host bias|grad batch heads q k buckets max_distance both seed
//   relpos_host map buckets max_distance both      prints the buckets' borders
#include "gsz_relpos.hip"
#include "plan.cpp"

#include <memory>
#include <random>
#include <string>
#include <vector>

extern "C" __bf16 __truncsfbf2(float f) {              // nearest even
    uint32_t u = __float_as_uint(f);
    uint16_t h = (u & 0x7FFFFFFF) > 0x7F800000 ? (u >> 16) | 0x40 : (u + 0x7FFF + (u >> 16 & 1)) >> 16;
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}
// n values of a type at place `shift` of their buffer; nothing after them but the rest of the last
// four bytes (reads of whole 4-byte words stay on the page).
struct Buf {
    std::unique_ptr<char[]> raw;
    char* p;
    int type;
    Buf(int64_t n, int t, int shift = 0) : raw(new char[((n + shift) * value_size(t) + 3) / 4 * 4]), p(raw.get() + shift * value_size(t)), type(t) {}
    double get(int64_t i) const { return type == GSZ_TYPE_F32 ? ((float*)p)[i] : load1((uint16_t*)p + i); }
    void set(int64_t i, double v) {
        if (type == GSZ_TYPE_F32) ((float*)p)[i] = (float)v;
        else { uint32_t u = __float_as_uint((float)v); ((uint16_t*)p)[i] = (uint16_t)(u >> 16); }
    }
};

int main(int argc, char** argv) {
    const std::string op = argv[1];
    if (op == "map") {
        RelMap m;
        if (make_map("map", std::atoll(argv[2]), std::atoll(argv[3]), std::atoi(argv[4]), &m)) return 2;
        for (int b = 0; b < m.n; ++b) std::printf("%d ", m.first[b]);
        return 0;
    }
    const int64_t batch = std::atoll(argv[2]), heads = std::atoll(argv[3]), q = std::atoll(argv[4]), k = std::atoll(argv[5]),
                  buckets = std::atoll(argv[6]), far = std::atoll(argv[7]);
    const int both = std::atoi(argv[8]);
    std::mt19937_64 g(std::strtoull(argv[9], nullptr, 10) * 2654435761u + 17);
    auto value = [&] { return (double)(int64_t)(g() % 17) - 8; };
    auto type = [&] { return g() % 2 ? GSZ_TYPE_BF16 : GSZ_TYPE_F32; };
    const int64_t n = batch * heads * q * k, cells = buckets * heads;
    std::vector<int64_t> starts(batch);
    for (auto& s : starts) s = (int64_t)(g() % (2 * k + 2 * q)) - q;
    const bool each = g() % 2;
    const int64_t start = starts.empty() ? 0 : starts[0];
    const double scale = g() % 2 ? 1.0 : 0.5;
    auto bucket = [&](int64_t d) -> int64_t {
        const int64_t half = both ? buckets / 2 : buckets, e = half / 2, dist = both ? std::abs(d) : d < 0 ? -d : 0;
        int64_t b = dist < e ? dist : std::min(half - 1, e + (int64_t)std::floor(std::log((double)dist / e) / std::log((double)far / e) * (half - e) + 1e-9));
        return both && d > 0 ? b + half : b;
    };
    int64_t bad = 0;
    if (op == "bias") {
        const int shift = (int)(g() % 9);
        Buf table(cells, type(), shift), out(n, type(), shift), add(n, out.type, 2 * shift);
        for (int64_t i = 0; i < cells; ++i) table.set(i, value());
        for (int64_t i = 0; i < n; ++i) add.set(i, value());
        const bool with = g() % 2, same = with && g() % 2;
        const int rc = gsz_relpos_bias(table.p, table.type, buckets, heads, far, both, batch, q, k, start, each ? starts.data() : nullptr,
                                       GSZ_TYPE_I64, scale, with ? add.p : nullptr, same ? add.p : out.p, out.type, nullptr);
        if (rc) { std::printf("refused %d\n", rc); return 2; }
        if (same) return 0;
        for (int64_t b = 0, at = 0; b < batch; ++b) for (int64_t h = 0; h < heads; ++h) for (int64_t i = 0; i < q; ++i) for (int64_t j = 0; j < k; ++j, ++at) {
            const double want = (with ? add.get(at) : 0.0) + scale * table.get(bucket(j - i - (each ? starts[b] : start)) * heads + h);
            if (out.get(at) != want && ++bad < 5) std::printf("%ld %ld %ld %ld: %g, not %g\n", (long)b, (long)h, (long)i, (long)j, out.get(at), want);
        }
    } else {
        Buf dy(n, type(), (int)(g() % 9)), grad(cells, GSZ_TYPE_F32);
        const int acc = (int)(g() % 2);
        std::vector<double> want(cells, 0.0);
        for (int64_t i = 0; i < cells; ++i) { grad.set(i, value()); if (acc) want[i] = grad.get(i); }
        for (int64_t b = 0, at = 0; b < batch; ++b) for (int64_t h = 0; h < heads; ++h) for (int64_t i = 0; i < q; ++i) for (int64_t j = 0; j < k; ++j, ++at) {
            dy.set(at, value());
            want[bucket(j - i - (each ? starts[b] : start)) * heads + h] += scale * dy.get(at);
        }
        size_t bytes = 0;
        if (gsz_relpos_bias_workspace_bytes(batch, heads, q, k, buckets, &bytes)) return 2;
        std::vector<char> raw(1);
        std::unique_ptr<char[]> ws(new char[bytes ? bytes : 1]);
        std::memset(ws.get(), 0xFF, bytes);
        const int rc = gsz_relpos_bias_grad(dy.p, dy.type, buckets, heads, far, both, batch, q, k, start, each ? starts.data() : nullptr,
                                            GSZ_TYPE_I64, scale, grad.p, grad.type, acc, ws.get(), bytes, nullptr);
        if (rc) { std::printf("refused %d\n", rc); return 2; }
        for (int64_t i = 0; i < cells; ++i)
            if (grad.get(i) != want[i] && ++bad < 5) std::printf("bucket %ld head %ld: %g, not %g\n", (long)(i / heads), (long)(i % heads), grad.get(i), want[i]);
    }
    if (bad) std::printf("%ld wrong\n", (long)bad);
    return bad != 0;
}
