// Layer norm's host code behind a runtime of this file's own: two host threads call
// kernels that want different amounts of shared memory for the first time, at once.
// The runtime keeps each kernel's limit as a driver does and refuses launches
// above it.  Linked to the library's object by tests/test_shared_memory_opt_in.py.
//
//   program first|last    which of the two has the larger request's answer: the thread
//                         that goes on first, or the other
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <thread>

#include "../block_scaled_mxfp4_gb300/csrc/dense.h"

namespace {

std::mutex m;
std::condition_variable changed;
std::map<const void *, int> limit;               // bytes that a kernel may use
std::set<size_t> asked;                          // bytes of the launches
int inside = 0, applied = 0, refused = 0;
bool larger_last = false, racing = false;
constexpr auto kLong = std::chrono::milliseconds(300);

}  // namespace

extern "C" {

cudaError_t cudaGetDevice(int *dev)
{
    *dev = 0;
    return cudaSuccess;
}

// The first two requests of a race wait for one another (for a while: a lock may keep the second out); the
// larger takes effect first, and neither goes on before both have.
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute, int value)
{
    static int largest;
    std::unique_lock<std::mutex> lock(m);
    if (!racing || inside >= 2) {
        limit[f] = value;
        return cudaSuccess;
    }
    largest = inside == 0 || value > largest ? value : largest;
    ++inside;
    changed.notify_all();
    changed.wait_for(lock, kLong, [] { return inside >= 2; });
    const bool large = value == largest;
    if (!large)
        changed.wait_for(lock, kLong, [] { return applied >= 1; });
    limit[f] = value;
    ++applied;
    changed.notify_all();
    changed.wait_for(lock, kLong, [] { return applied >= 2; });
    lock.unlock();
    if (large == larger_last)
        std::this_thread::sleep_for(kLong / 4);  // the other one goes on meanwhile
    return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    std::unique_lock<std::mutex> lock(m);
    asked.insert(c->dynamicSmemBytes);
    const int most = limit.count(f) ? limit[f] : 48 << 10;
    if (c->dynamicSmemBytes <= static_cast<size_t>(most))
        return cudaSuccess;
    ++refused;
    return cudaErrorInvalidValue;
}

// What a translation unit of nvcc's registers; nothing is launched here.
void **__cudaRegisterFatBinary(void *)
{
    static void *handle[1];
    return handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return 1; }
cudaError_t __cudaGetKernel(void **, const void *) { return cudaErrorInvalidValue; }
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaErrorInvalidValue; }
cudaError_t cudaMemcpyFromSymbol(void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaErrorInvalidValue; }
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaErrorInvalidValue; }

}  // extern "C"

namespace mxfp4 {
cudaError_t launch_sum_partials(float *, int64_t, float *, int64_t, const float *, int, cudaStream_t) { return cudaSuccess; }
}  // namespace mxfp4

static cudaError_t call(bool backward, int N, int width)
{
    mxfp4::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.T = 100000;
    a.N = N;
    a.width = width;
    a.blocks = mxfp4::norm_backward_blocks(a.T, N);
    return backward ? mxfp4::launch_layer_norm_backward(a, nullptr) : mxfp4::launch_layer_norm(a, 152, nullptr);
}

int main(int, char **argv)
{
    larger_last = !std::strcmp(argv[1], "last");
    int bad = 0;
    for (const bool backward : {false, true})
        for (const int width : {8, 1}) {
            const int n[2] = {2056, 8192 - (width == 1)};
            cudaError_t first[2], second[2];
            asked.clear();
            inside = applied = 0;
            racing = true;
            std::thread other([&] { first[1] = call(backward, n[1], width); });
            first[0] = call(backward, n[0], width);
            other.join();
            racing = false;
            for (int i = 0; i < 2; ++i)
                second[i] = call(backward, n[i], width);
            for (int i = 0; i < 2; ++i)
                if (first[i] != cudaSuccess || second[i] != cudaSuccess) {
                    std::printf("%s, rows of %d, accesses of %d: %d, later %d\n", backward ? "gradients" : "norm", n[i], width, first[i],
                                second[i]);
                    ++bad;
                }
            if (asked.size() != 2) {
                std::printf("the two calls want the same\n");
                ++bad;
            }
        }
    std::printf("%d refused\n", refused);
    return bad != 0;
}
