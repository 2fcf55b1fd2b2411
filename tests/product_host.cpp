// The products of the orthogonalising update run on the CPU (host_gpu/, host_matrix/) in each of
// their forms and splits, against a plain reference: whole numbers, so the results are equal.
// Built with AddressSanitizer: an access outside a buffer ends the program.
//
//   product_host form parts split turned_left turned_right symmetric M N K
#include "gsz_muon.hip"
#include "plan.cpp"

#include <random>

extern "C" __bf16 __truncsfbf2(float f) {
    const uint16_t h = (uint16_t)bf16_rne(f);
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}

template <bool TL, bool TR>
static int run(int form, int parts, int64_t split, bool half, int64_t M, int64_t N, int64_t K) {
    std::mt19937 g(1);
    auto values = [&](int64_t n) {
        std::vector<_Float16> v(n);
        for (auto& x : v) x = (_Float16)(float)((int)(g() % 17) - 8);
        return v;
    };
    constexpr int64_t kCount = 2;
    const std::vector<_Float16> l = values(kCount * M * K), r = values(kCount * N * K);
    std::vector<_Float16> c(kCount * M * N, (_Float16)77.0f);
    const Operand L{l.data(), M * K, TL ? M : K}, R{half ? l.data() : r.data(), half ? M * K : N * K, TR ? N : K};
    const int64_t side = kCosts[form].side, down = (M + side - 1) / side, across = (N + side - 1) / side;
    const int64_t tiles = kCount * (half ? down * (down + 1) / 2 : down * across);
    if (split > tiles) split = tiles;
    const Choice choice{form, tiles - split, split, parts, 0.0};
    std::vector<f32x4> partial(split * parts * side * side / 4 + 1);
    auto go = [&](const auto& e) { return product<TL, TR>("product", kCount, L, R, M, N, K, half, partial.data(), e, nullptr, &choice); };
    if (half ? go(StoreHalf<true>{c.data(), M * N, N, 1.0f / 16}) : go(StoreHalf<false>{c.data(), M * N, N, 1.0f / 16})) return 2;
    int64_t bad = 0;
    for (int64_t b = 0; b < kCount; ++b)
        for (int64_t i = 0; i < M; ++i)
            for (int64_t j = 0; j < N; ++j) {
                float s = 0.0f;
                for (int64_t k = 0; k < K; ++k)
                    s += (float)L.base[b * L.stride + (TL ? k * L.ld + i : i * L.ld + k)] * (float)R.base[b * R.stride + (TR ? k * R.ld + j : j * R.ld + k)];
                if ((float)c[(b * M + i) * N + j] != (float)(_Float16)(s / 16) && ++bad < 4)
                    std::printf("%ld %ld %ld: %g, not %g\n", (long)b, (long)i, (long)j, (double)c[(b * M + i) * N + j], s / 16);
            }
    std::printf("%ld wrong\n", (long)bad);
    return bad != 0;
}

int main(int, char** a) {
    const int form = std::atoi(a[1]), parts = std::atoi(a[2]), tl = std::atoi(a[4]), tr = std::atoi(a[5]), half = std::atoi(a[6]);
    const int64_t split = std::atoll(a[3]), M = std::atoll(a[7]), N = std::atoll(a[8]), K = std::atoll(a[9]);
    if (tl) return run<true, true>(form, parts, split, half, M, N, K);
    return tr ? run<false, true>(form, parts, split, half, M, N, K) : run<false, false>(form, parts, split, half, M, N, K);
}
