// Two host threads call smr_expert_down with one workspace; the launches are
// stand-ins that say what was launched, in which order. (A host program: the
// CUDA runtime's device queries are stand-ins too.)
#include <cuda_runtime.h>

#include <chrono>
#include <cstdio>
#include <mutex>
#include <thread>

#include "smr.h"
#include "smr_launch.h"

static std::mutex print_lock;
static void say(const char *what, const void *x) {
    const std::lock_guard<std::mutex> one(print_lock);
    std::printf("%s %zu\n", what, reinterpret_cast<size_t>(x));
}

extern "C" cudaError_t cudaGetDevice(int *dev) { return *dev = 0, cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr attr, int) {
    *v = attr == cudaDevAttrComputeCapabilityMajor ? 10 : 3;
    return cudaSuccess;
}

namespace smr {
bool expert_rows_fp32(int64_t, int, int) { return true; }
cudaError_t launch_expert_product(const FfnLaunch &a, cudaStream_t) {
    say("product", a.hdr);
    std::this_thread::sleep_for(std::chrono::milliseconds(3));
    return cudaSuccess;
}
cudaError_t launch_expert_combine(const CombineLaunch &a, cudaStream_t) {
    say("sum", static_cast<const char *>(a.y) - 256 - 16 * 1024 * 8);
    return cudaSuccess;
}
}  // namespace smr

int main() {
    auto work = [](size_t at) {
        void *ptr = reinterpret_cast<void *>(0x10000);
        smr_expert_down_args a{};
        a.num_tokens = 2, a.width = 2, a.H = 64, a.I = 64, a.num_experts = 4, a.block_size = 64, a.num_logical = 4;
        a.x = a.w = ptr, a.out = ptr, a.topk_ids = static_cast<int32_t *>(ptr), a.topk_weights = static_cast<float *>(ptr);
        a.sorted_token_ids = a.expert_ids = a.num_tokens_post_padded = static_cast<int32_t *>(ptr);
        a.sorted_cap = 256;
        for (int i = 0; i < 10; ++i)
            if (smr_expert_down(&a, reinterpret_cast<void *>(at), 1 << 20, nullptr) != SMR_OK) say(smr_last_error(), nullptr);
    };
    std::thread t1(work, 0x100000), t2(work, 0x100000);
    t1.join(), t2.join();
    return 0;
}
