// csrc/q8_smem.h against a stand-in for the CUDA runtime (no device, no libcudart):
// the limit that stands after calls from two threads is the largest asked for.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

#include "q8_smem.h"

static std::mutex mu;
static std::condition_variable cv;
static int limit_now = 48 * 1024, calls = 0;
static bool small_inside = false, big_set = false;
static const int kBig = 200 * 1024, kSmall = 100 * 1024;

extern "C" cudaError_t cudaGetDevice(int* dev) { *dev = 0; return cudaSuccess; }
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
    std::unique_lock<std::mutex> lk(mu);
    ++calls;
    if (bytes == kSmall) {   // the smaller request takes its time: a larger one may come in between
        small_inside = true;
        cv.notify_all();
        cv.wait_for(lk, std::chrono::milliseconds(300), [] { return big_set; });
    }
    limit_now = bytes;       // replaces the limit, as the runtime does
    if (bytes == kBig) big_set = true;
    cv.notify_all();
    return cudaSuccess;
}

static void kernel() {}

int main() {
    std::thread small([] { q8::set_smem(kernel, kSmall); });
    {
        std::unique_lock<std::mutex> lk(mu);
        cv.wait(lk, [] { return small_inside; });
    }
    std::thread big([] { q8::set_smem(kernel, kBig); });
    small.join();
    big.join();
    q8::set_smem(kernel, 150 * 1024);   // below the largest: nothing to do
    const bool ok = limit_now == kBig && calls == 2;
    std::printf("%s limit %d after %d calls\n", ok ? "ok" : "FAIL", limit_now, calls);
    return ok ? 0 : 1;
}
