// The relative position bias added to scores in place: the entry point and kernels themselves, run on
// the CPU (host_gpu/, host_matrix/) in buffers of exactly the documented sizes, against a plain
// reference computed from a copy of the scores.  Built with AddressSanitizer.
//
//   relpos_in_place_host batch heads q k buckets max_distance both type shift seed
#include "gsz_relpos.hip"
#include "plan.cpp"

#include <memory>
#include <random>
#include <vector>

extern "C" __bf16 __truncsfbf2(float f) {              // nearest even
    uint32_t u = __float_as_uint(f);
    uint16_t h = (u & 0x7FFFFFFF) > 0x7F800000 ? (u >> 16) | 0x40 : (u + 0x7FFF + (u >> 16 & 1)) >> 16;
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}
static double get(const char* p, int type, int64_t i) {
    return type == GSZ_TYPE_F32 ? reinterpret_cast<const float*>(p)[i] : load1(reinterpret_cast<const uint16_t*>(p) + i);
}
static void set(char* p, int type, int64_t i, double v) {
    if (type == GSZ_TYPE_F32) reinterpret_cast<float*>(p)[i] = (float)v;
    else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(__float_as_uint((float)v) >> 16);
}

int main(int argc, char** argv) {
    if (argc != 11) return 3;
    int64_t a[11];
    for (int k = 1; k < 11; ++k) a[k] = std::atoll(argv[k]);
    const int64_t batch = a[1], heads = a[2], q = a[3], k = a[4], buckets = a[5], far = a[6], n = batch * heads * q * k, cells = buckets * heads;
    const int both = (int)a[7], type = (int)a[8], shift = (int)a[9];
    std::mt19937_64 g(a[10] * 2654435761u + 5);
    auto value = [&] { return (double)(int64_t)(g() % 17) - 8; };   // sums are exact in bf16
    // nothing before the scores but `shift` values, nothing after them but the rest of four bytes
    const int64_t size = value_size(type);
    std::unique_ptr<char[]> raw(new char[((n + shift) * size + 3) / 4 * 4]), table(new char[(cells * size + 3) / 4 * 4]);
    char* scores = raw.get() + shift * size;
    for (int64_t i = 0; i < cells; ++i) set(table.get(), type, i, value());
    for (int i = 0; i < shift; ++i) set(raw.get(), type, i, 3.0);
    for (int64_t i = 0; i < n; ++i) set(scores, type, i, i % 11 == 7 ? -INFINITY : value());
    const std::vector<char> before(scores, scores + n * size);
    std::vector<int32_t> starts(batch);
    for (auto& s : starts) s = (int32_t)(g() % (2 * k + 2 * q)) - (int32_t)q;
    const bool each = g() % 2;
    const int rc = gsz_relpos_bias(table.get(), type, buckets, heads, far, both, batch, q, k, starts[0], each ? starts.data() : nullptr, GSZ_TYPE_I32,
                                   0.5, scores, scores, type, nullptr);
    if (rc) { std::printf("refused %d\n", rc); return 2; }
    auto bucket = [&](int64_t d) -> int64_t {
        const int64_t half = both ? buckets / 2 : buckets, e = half / 2, dist = both ? std::abs(d) : d < 0 ? -d : 0;
        const int64_t b = dist < e ? dist : std::min(half - 1, e + (int64_t)std::floor(std::log((double)dist / e) / std::log((double)far / e) * (half - e) + 1e-9));
        return both && d > 0 ? b + half : b;
    };
    int64_t bad = 0, at = 0;
    for (int64_t b = 0; b < batch; ++b) for (int64_t h = 0; h < heads; ++h) for (int64_t i = 0; i < q; ++i) for (int64_t j = 0; j < k; ++j, ++at) {
        const double want = get(before.data(), type, at) + 0.5 * get(table.get(), type, bucket(j - i - starts[each ? b : 0]) * heads + h);
        const double got = get(scores, type, at);
        if (!(got == want) && ++bad < 5) std::printf("%ld %ld %ld %ld: %g, not %g\n", (long)b, (long)h, (long)i, (long)j, got, want);
    }
    for (int i = 0; i < shift; ++i) if (get(raw.get(), type, i) != 3.0) { std::printf("wrote before\n"); ++bad; }
    return bad != 0;
}
