// The orthogonalising entry points and kernels themselves, run on the CPU (host_gpu/,
// host_matrix/) on values from a file, in buffers of exactly the documented sizes and a workspace
// of NaNs; what they give goes to another file, for the caller to compare.
//
//   muon_values_host orthogonalize count rows cols type steps in out
//     in: the matrices, type 0 bf16 or 1 fp32; out: bf16
//   muon_values_host step count rows cols nesterov in out
//     a plan of count matrices with 3, 4 ... elements after each; in: master, momentum, g of the plan's
//     length; out: master, momentum, params (0x1234 before the call)
#include "gsz_muon.hip"
#include "plan.cpp"

#include <cstdlib>
#include <memory>
#include <string>

extern "C" __bf16 __truncsfbf2(float f) {
    const uint16_t h = (uint16_t)bf16_rne(f);
    __bf16 b;
    std::memcpy(&b, &h, 2);
    return b;
}

// Memory of just these bytes, 16-byte aligned.
struct Bytes {
    char* p;
    explicit Bytes(size_t n, int fill = 0) {
        void* at;
        if (posix_memalign(&at, 16, n)) std::exit(3);
        p = static_cast<char*>(at);
        std::memset(p, fill, n);
    }
    ~Bytes() { std::free(p); }
    Bytes(const Bytes&) = delete;
};
struct File {
    FILE* f;
    File(const char* name, const char* mode) : f(std::fopen(name, mode)) { if (!f) std::exit(3); }
    ~File() { std::fclose(f); }
    void read(void* p, size_t n) { if (std::fread(p, 1, n, f) != n) std::exit(3); }
    void write(const void* p, size_t n) { if (std::fwrite(p, 1, n, f) != n) std::exit(3); }
};

int main(int argc, char** argv) {
    if (argc < 8) return 3;
    const int64_t count = std::atoll(argv[2]), rows = std::atoll(argv[3]), cols = std::atoll(argv[4]), n = rows * cols;
    const int last = std::atoi(argv[5]);
    size_t need = 0;
    if (gsz_muon_workspace_bytes(count, rows, cols, &need)) return 2;
    Bytes ws(need, 0xFF);
    if (std::string(argv[1]) == "orthogonalize") {
        Bytes x(count * n * value_size(last)), out(count * n * 2, 0xFF);
        File(argv[7], "rb").read(x.p, count * n * value_size(last));
        if (gsz_orthogonalize(x.p, last, count, rows, cols, std::atoi(argv[6]), nullptr, 1e-7, reinterpret_cast<uint16_t*>(out.p), ws.p, need, nullptr))
            return 2;
        File(argv[8], "wb").write(out.p, count * n * 2);
        return 0;
    }
    std::vector<int64_t> numel;
    std::vector<int32_t> list;
    for (int64_t b = 0; b < count; ++b) {
        list.push_back((int32_t)numel.size());
        numel.push_back(n);
        numel.push_back(3 + b);
    }
    gsz_plan* plan;
    if (gsz_plan_create(numel.data(), (int32_t)numel.size(), 1000, 2, 8, &plan)) return 2;
    const size_t len = (size_t)plan->flat_len;
    Bytes w(len * 4), m(len * 4), g(len * 4), p(len * 2);
    File in(argv[6], "rb");
    for (Bytes* b : {&w, &m, &g}) in.read(b->p, len * 4);
    for (size_t i = 0; i < len; ++i) reinterpret_cast<uint16_t*>(p.p)[i] = 0x1234;
    const float coef = 0.75f;
    const gsz_muon_hp hp{0.02, 0.95, 0.1, 0.2 * std::sqrt((double)std::max(rows, cols)), 1e-7, nullptr, 5, last};
    const int rc = gsz_muon_step(plan, list.data(), (int32_t)count, rows, cols, reinterpret_cast<float*>(w.p), reinterpret_cast<float*>(m.p),
                                 reinterpret_cast<float*>(g.p), &coef, &hp, reinterpret_cast<uint16_t*>(p.p), ws.p, need, nullptr);
    gsz_plan_destroy(plan);
    if (rc) return 2;
    File to(argv[7], "wb");
    to.write(w.p, len * 4);
    to.write(m.p, len * 4);
    to.write(p.p, len * 2);
    return 0;
}
