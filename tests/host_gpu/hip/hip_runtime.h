// Runs HIP kernels on the CPU, one fiber per work-item, for tests of their
// indexing under AddressSanitizer.  Work-items of a block take turns at barriers
// and at wave operations; a wave operation that some live lanes of the wave never
// reach, or that reads a lane that has ended, ends the program.
#pragma once
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define __align__(n) __attribute__((aligned(n)))

typedef void* hipStream_t;
enum hipError_t { hipSuccess = 0 };
struct hipDeviceProp_t { char gcnArchName[16]; int multiProcessorCount; };
inline hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
inline hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) { std::strcpy(p->gcnArchName, "gfx950"); p->multiProcessorCount = 256; return hipSuccess; }
inline hipError_t hipGetLastError() { return hipSuccess; }
inline const char* hipGetErrorString(hipError_t) { return ""; }

struct dim3 { unsigned x; dim3(unsigned v = 1) : x(v) {} };

// Saves the registers a call keeps, stores the stack pointer in *from and goes on
// where the stack `to` left off (x86-64; no system call, unlike swapcontext).
extern "C" void emu_switch(void** from, void* to);
asm(".text\n.globl emu_switch\n.type emu_switch,@function\nemu_switch:\n"
    "push %rbp\npush %rbx\npush %r12\npush %r13\npush %r14\npush %r15\n"
    "mov %rsp,(%rdi)\nmov %rsi,%rsp\n"
    "pop %r15\npop %r14\npop %r13\npop %r12\npop %rbx\npop %rbp\nret\n");

namespace emu {
constexpr int kMaxThreads = 1024;
constexpr size_t kStack = 64 << 10;
struct Group { int alive = 0, arrived = 0; uint64_t gen = 0; };
struct Thread { void* sp = nullptr; bool done = true; };
struct State {
    Thread t[kMaxThreads];
    std::vector<char> stacks;
    void* back;
    Group block, wave[kMaxThreads / 64];
    uint64_t slot[kMaxThreads];
    bool ended[kMaxThreads];
    int cur = 0, threads = 0;
    uint64_t moves = 0;
    unsigned bx = 0, gx = 0, dimx = 0;
    std::function<void()> body;
};
inline State S;
inline void fail(const char* why) { std::fprintf(stderr, "emulated kernel: %s (block %u, work-item %d)\n", why, S.bx, S.cur); std::abort(); }
inline void yield() { emu_switch(&S.t[S.cur].sp, S.back); }
inline void arrive(Group& g) { if (g.arrived == g.alive && g.alive) { g.arrived = 0; ++g.gen; ++S.moves; } }
inline void sync(Group& g) {
    const uint64_t gen = g.gen;
    ++g.arrived;
    arrive(g);
    while (g.gen == gen) yield();
}
inline Group& wave() { return S.wave[S.cur >> 6]; }
inline void entry() {
    S.body();
    S.t[S.cur].done = true;
    S.ended[S.cur] = true;
    ++S.moves;
    --S.block.alive;
    --wave().alive;
    arrive(S.block);
    arrive(wave());
    yield();
}
template <class F> void launch(unsigned grid, unsigned block, F body) {
    if (block > kMaxThreads) fail("block too large");
    if (S.stacks.empty()) S.stacks.resize(kStack * kMaxThreads);
    S.body = body;
    S.gx = grid; S.dimx = block; S.threads = (int)block;
    for (S.bx = 0; S.bx < grid; ++S.bx) {
        S.block = Group{(int)block, 0, 0};
        for (unsigned w = 0; w * 64 < block; ++w) S.wave[w] = Group{(int)(block - w * 64 < 64 ? block - w * 64 : 64), 0, 0};
        for (unsigned i = 0; i < block; ++i) {
            S.ended[i] = S.t[i].done = false;
            // as emu_switch leaves a stack: six registers, then where to go on
            void** top = reinterpret_cast<void**>((reinterpret_cast<uintptr_t>(S.stacks.data()) + kStack * (i + 1)) & ~(uintptr_t)15);
            top[-1] = nullptr;
            top[-2] = reinterpret_cast<void*>(entry);
            S.t[i].sp = top - 8;
        }
        for (int left = (int)block; left > 0;) {
            left = 0;
            const uint64_t before = S.moves;
            for (unsigned i = 0; i < block; ++i) {
                if (S.t[i].done) continue;
                ++left;
                S.cur = (int)i;
                emu_switch(&S.back, S.t[i].sp);
            }
            if (left && S.moves == before) fail("work-items wait for each other");
        }
    }
}
struct Idx { int which; operator unsigned() const { return which == 0 ? (unsigned)S.cur : which == 1 ? S.bx : which == 2 ? S.gx : S.dimx; } };
struct Dim { Idx x; };
inline uint64_t exchange(uint64_t v, std::function<uint64_t()> read) {
    S.slot[S.cur] = v;
    sync(wave());
    const uint64_t r = read();
    sync(wave());
    return r;
}
inline uint32_t read_lane(uint32_t v, int lane) {
    const int at = (S.cur & ~63) + lane;
    return (uint32_t)exchange(v, [at] { if (at >= S.threads || S.ended[at]) fail("reads a lane that has ended"); return S.slot[at]; });
}
}  // namespace emu

static const emu::Dim threadIdx{{0}}, blockIdx{{1}}, gridDim{{2}}, blockDim{{3}};
inline void __syncthreads() { emu::sync(emu::S.block); }
inline uint64_t __ballot(bool b) {
    return emu::exchange(b, [] {
        uint64_t m = 0;
        const int w = emu::S.cur & ~63;
        for (int l = 0; l < 64 && w + l < emu::S.threads; ++l) if (!emu::S.ended[w + l] && emu::S.slot[w + l]) m |= (uint64_t)1 << l;
        return m;
    });
}
inline int __popcll(uint64_t x) { return __builtin_popcountll(x); }
inline uint32_t atomicAdd(uint32_t* p, uint32_t v) { const uint32_t o = *p; *p += v; return o; }
inline uint32_t atomicOr(uint32_t* p, uint32_t v) { const uint32_t o = *p; *p |= v; return o; }
inline float __uint_as_float(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
inline uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
inline uint32_t __umulhi(uint32_t a, uint32_t b) { return (uint32_t)((uint64_t)a * b >> 32); }
inline uint32_t __shfl(uint32_t v, int lane) { return emu::read_lane(v, lane); }
inline uint32_t __shfl_up(uint32_t v, int delta) {
    const int lane = emu::S.cur & 63;
    return emu::read_lane(v, lane >= delta ? lane - delta : lane);
}
#define __builtin_amdgcn_fence(...) ((void)0)
#define __builtin_amdgcn_wave_barrier() emu::sync(emu::wave())
#define __builtin_amdgcn_readlane(v, lane) emu::read_lane((v), (lane))
#define __builtin_amdgcn_readfirstlane(v) emu::read_lane((v), 0)
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
    emu::launch((grid).x, (block).x, [=] { (kernel)(__VA_ARGS__); })
