// The embedding and dropout entry points at the limits of their sizes, on the CPU.
//
//   layers_limits sizes     calls at both sides of each documented limit, their launches
//                           only counted: each has 1 to 2^31 work-items
//   layers_limits op seed   a random case of layers_host, under the smallest limit of
//                           work-items per launch that the call takes: what has a block of
//                           its own otherwise is gone over by a few, and must come out alike
#include <hip/hip_runtime.h>

#include "gsz_device.h"

// A refused call of layers_host ends with its workspace still allocated.
extern "C" const char* __asan_default_options() { return "detect_leaks=0"; }

static int64_t g_most = (int64_t)1 << 31;
static bool g_run = true;
static void launch_checked(unsigned grid, unsigned block, std::function<void()> body) {
    if (grid < 1 || block < 1 || (int64_t)grid * block > g_most) emu::fail("a launch of no or too many work-items");
    if (g_run) emu::launch(grid, block, body);
}
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
    launch_checked((grid).x, (block).x, [=] { (kernel)(__VA_ARGS__); })
#define kMaxWorkItems g_most
#define main layers_host_main
#include "layers_host.cpp"
#undef main

static int sizes() {
    g_run = false;
    auto at = [](int bit) { return reinterpret_cast<void*>((uintptr_t)1 << bit); };      // no launch runs: never read
    void* const p = at(20);
    const int64_t K = 1 << 10, M = K * K, G = K * M, kRows = 2 * G - 1;
    struct Case { int64_t n, rows, dim; int acc, type, want; };
    const Case cases[] = {
        // any number of rows, cleared or not, on every path
        {0, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {4, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {4, kRows, 1, 0, GSZ_TYPE_F32, GSZ_OK},
        {128, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {4, kRows, 1, 1, GSZ_TYPE_BF16, GSZ_OK}, {4, kRows, 8192, 0, GSZ_TYPE_F32, GSZ_OK},
        {129, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {8192, kRows, 64, 0, GSZ_TYPE_F32, GSZ_OK}, {700, 256 * M, 2048, 0, GSZ_TYPE_BF16, GSZ_OK},
        {8193, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {9000, 1900 * M, 1, 0, GSZ_TYPE_F32, GSZ_OK}, {70000, kRows, 100, 0, GSZ_TYPE_BF16, GSZ_OK},
        {9000, kRows, 1, 1, GSZ_TYPE_F32, GSZ_OK}, {9000, kRows + 1, 1, 1, GSZ_TYPE_F32, GSZ_ERR_SIZE},
        // n <= 128: n * column tiles of 512
        {128, 10, 128 * M, 1, GSZ_TYPE_BF16, GSZ_OK}, {128, 10, 128 * M + 1, 1, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
        {128, 10, 128 * M - 512, 0, GSZ_TYPE_BF16, GSZ_OK}, {128, 10, 128 * M, 0, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
        {1, 10, 512 * M, 0, GSZ_TYPE_F32, GSZ_OK}, {31, 3, 512 * M, 0, GSZ_TYPE_F32, GSZ_OK}, {33, 3, 512 * M, 1, GSZ_TYPE_F32, GSZ_ERR_SIZE},
        // more: chunks of 32 tokens * column tiles
        {G, 10, 512, 0, GSZ_TYPE_BF16, GSZ_OK}, {G, kRows, 1, 0, GSZ_TYPE_BF16, GSZ_OK}, {G + 1, 10, 1, 1, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
        {G / 2, 10, 513, 1, GSZ_TYPE_BF16, GSZ_OK}, {G / 2 + 1, 10, 513, 1, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
        {K, 10, 512 * M, 1, GSZ_TYPE_BF16, GSZ_OK}, {K + 1, 10, 512 * M, 1, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
        {kRows, 10, 1, 1, GSZ_TYPE_BF16, GSZ_ERR_SIZE},
    };
    int bad = 0;
    for (const Case& c : cases) {
        const int rc = gsz_embedding_grad(p, GSZ_TYPE_I32, c.n, at(44), GSZ_TYPE_BF16, c.rows, c.dim, 1.0, 0.0, nullptr, 0, at(61), c.type,
                                          c.acc, at(62), ~(size_t)0 >> 1, nullptr);
        if (rc != c.want && ++bad)
            std::printf("gradient of %ld tokens, %ld rows of %ld, accumulate %d: %d, want %d\n", (long)c.n, (long)c.rows, (long)c.dim, c.acc, rc, c.want);
    }
    const int64_t lookups[][3] = {{kRows, kRows, 512 * M}, {kRows, kRows, 1}, {1, 1, 512 * M}, {kRows, 1, 8192}, {kRows, 1, 1023}};
    for (auto& l : lookups)
        for (double drop : {0.0, 0.5})
            if (gsz_embedding_lookup(at(61), GSZ_TYPE_BF16, l[1], l[2], at(40), GSZ_TYPE_I64, l[0], 1.0, drop, (uint64_t*)p, 0, at(62), GSZ_TYPE_F32, nullptr) != GSZ_OK && ++bad)
                std::printf("lookup of %ld tokens of %ld columns refused\n", (long)l[0], (long)l[2]);
    for (int64_t n : {(int64_t)1, kRows, (int64_t)1 << 60})
        if (gsz_dropout(at(61), at(61), at(61), n, GSZ_TYPE_F32, 0.5, (uint64_t*)p, 0, nullptr) != GSZ_OK && ++bad) std::printf("dropout of %ld refused\n", (long)n);
    // Buffers side by side: 16 values; 200 tokens on 10 rows of 8.
    char* const b = static_cast<char*>(at(30));
    size_t bytes = 0;
    gsz_embedding_workspace_bytes(200, 10, 8, &bytes);
    const bool taken =
        gsz_dropout(b, b + 64, b + 32, 16, GSZ_TYPE_BF16, 0.5, (uint64_t*)(b + 96), 0, nullptr) == GSZ_OK &&
        gsz_dropout(b + 64, b, b + 32, 16, GSZ_TYPE_BF16, 0.5, (uint64_t*)(b - 16), 0, nullptr) == GSZ_OK &&
        gsz_dropout(b, b + 32, b + 32, 16, GSZ_TYPE_BF16, 0.5, (uint64_t*)(b + 64), 0, nullptr) == GSZ_OK &&
        gsz_dropout(b, b + 2, b, 16, GSZ_TYPE_BF16, 0.0, (uint64_t*)b, 0, nullptr) == GSZ_ERR_INVALID_ARG &&
        gsz_embedding_lookup(b, GSZ_TYPE_BF16, 10, 8, b + 160 + 64, GSZ_TYPE_I64, 4, 1.0, 0.5, (uint64_t*)(b + 256), 0, b + 160, GSZ_TYPE_BF16, nullptr) == GSZ_OK &&
        gsz_embedding_grad(b, GSZ_TYPE_I64, 200, b + 1760, GSZ_TYPE_BF16, 10, 8, 1.0, 0.0, (uint64_t*)(b + 1600), 0, b + 1600, GSZ_TYPE_BF16, 0,
                           b + 4960, bytes, nullptr) == GSZ_OK &&
        gsz_embedding_grad(b, GSZ_TYPE_I64, 4, b + 32, GSZ_TYPE_BF16, 10, 8, 1.0, 0.0, nullptr, 0, b + 96, GSZ_TYPE_BF16, 0, b, 8, nullptr) == GSZ_OK;
    if (!taken && ++bad) std::printf("buffers that only touch, or are not read, refused\n");
    return bad ? 1 : 0;
}

int main(int argc, char** argv) {
    if (std::string(argv[1]) == "sizes") return sizes();
    // The sums of a gradient have a block each: more work-items until they fit.
    for (g_most = kRankBlock; g_most <= (int64_t)1 << 31; g_most *= 2) {
        const int rc = layers_host_main(argc, argv);
        if (rc != 2) return rc;
    }
    return 2;
}
