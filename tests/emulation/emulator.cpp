// Fibers of one workgroup (x86-64).  A wave runs on until all its lanes stand at the workgroup's
// barrier, then the next wave in the given order does: of two waves' accesses with no barrier
// between them, one comes first in the ascending order and the other in the descending one.
#include <hip/hip_runtime.h>
#undef asm
#undef volatile

Index threadIdx, blockIdx, gridDim, blockDim;

extern "C" {
void emulator_switch(void **from, void *to);
extern char __start_emulated_lds[], __stop_emulated_lds[];
}
asm(R"(
.globl emulator_switch
emulator_switch:
  pushq %rbp
  pushq %rbx
  pushq %r12
  pushq %r13
  pushq %r14
  pushq %r15
  movq %rsp, (%rdi)
  movq %rsi, %rsp
  popq %r15
  popq %r14
  popq %r13
  popq %r12
  popq %rbx
  popq %rbp
  ret
)");

namespace {

constexpr int kItems = 256, kWaves = kItems / 64, kStack = 256 << 10;
struct Fiber {
    void *sp;
    char *stack;
    bool done, waits;         // waits: at the barrier
};
Fiber fibers[kItems];
void *main_sp;
int current;
bool descending;
const std::function<void()> *body;
emulator::Slot slots[kWaves][64];
int arrived[kWaves], phase[kWaves];

void yield() { emulator_switch(&fibers[current].sp, main_sp); }

void entry()
{
    (*body)();
    fibers[current].done = true;
    yield();
    abort();
}

}  // namespace

namespace emulator {

void fail(const char *what)
{
    fprintf(stderr, "emulator: %s (workgroup %u, work-item %u)\n", what, blockIdx.x, threadIdx.x);
    abort();
}

int lane_id() { return current & 63; }
Slot &slot(int lane) { return slots[current / 64][lane]; }

void wave_sync()
{
    const int w = current / 64, before = phase[w];
    if (++arrived[w] == 64) {
        arrived[w] = 0;
        ++phase[w];
        return;
    }
    while (phase[w] == before) yield();
}

void barrier()
{
    fibers[current].waits = true;
    yield();
}

void launch(dim3 grid, dim3 block, const std::function<void()> &fn)
{
    body = &fn;
    const int items = (int)block.x, waves = (items + 63) / 64;
    if (items > kItems || items % 64 != 0) fail("a workgroup of other sizes");
    gridDim = {grid.x, 1, 1};
    blockDim = {block.x, 1, 1};
    for (unsigned g = 0; g < grid.x; ++g) {
        memset(__start_emulated_lds, 0xff, __stop_emulated_lds - __start_emulated_lds);
        for (int w = 0; w < waves; ++w) arrived[w] = 0;
        for (int i = 0; i < items; ++i) {
            Fiber &f = fibers[i];
            if (!f.stack) f.stack = (char *)aligned_alloc(64, kStack);
            void **sp = (void **)(f.stack + kStack - 64);
            *--sp = nullptr;
            *--sp = (void *)entry;
            for (int k = 0; k < 6; ++k) *--sp = nullptr;
            f.sp = sp;
            f.done = f.waits = false;
        }
        for (bool live = true; live;) {
            live = false;
            for (int k = 0; k < waves; ++k) {
                const int w = descending ? waves - 1 - k : k;
                int idle = 0;
                for (bool runs = true; runs; ++idle) {
                    runs = false;
                    for (int i = 64 * w; i < 64 * w + 64; ++i) {
                        if (fibers[i].done || fibers[i].waits) continue;
                        runs = true;
                        current = i;
                        threadIdx = {(unsigned)i, 0, 0};
                        blockIdx = {g, 0, 0};
                        emulator_switch(&main_sp, fibers[i].sp);
                    }
                    if (idle > (1 << 24)) fail("lanes that wait for each other");
                }
                if (arrived[w] != 0) fail("lanes at a barrier while others exchange values");
            }
            for (int i = 0; i < items; ++i) {
                live = live || !fibers[i].done;
                fibers[i].waits = false;
            }
        }
    }
}

}  // namespace emulator

// the library's record of the last HIP error
namespace ssd { int hip_status(hipError_t e) { return e == hipSuccess ? 0 : 5; } }

extern "C" void emulator_descending(int on) { descending = on != 0; }
