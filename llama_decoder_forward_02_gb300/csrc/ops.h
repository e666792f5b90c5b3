// Argument checks and error returns shared by the C entry points that run one
// operator a call.
#pragma once
#include <string>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "../../include/llm.h"

namespace llm {

void set_global_error(const char *msg);

inline int32_t refuse(const char *who, const char *why) {
    set_global_error((std::string(who) + ": " + why).c_str());
    return LLM_ERR_INVALID;
}

inline int32_t launched(const char *who, cudaError_t e) {
    if (!e) return LLM_OK;
    set_global_error((std::string(who) + ": " + cudaGetErrorString(e)).c_str());
    return LLM_ERR_COMPUTE;
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The kernels of these calls wait for the previous one before they touch
// memory, so their launches may overlap its end (programmatic dependent
// launch): calls in a row then follow each other without the gap of a launch,
// 2 to 4 us.
inline Launch overlapped(void *stream) { return Launch{(cudaStream_t)stream, true, nullptr}; }

inline int current_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// What is wrong with the shape of one layer's heads and cache, or null.
inline const char *shape_error(int T, int H, int Hkv, int hd, int n_ctx, int n_seq) {
    if (T < 1) return "T must be positive";
    if (hd != 32 && hd != 64 && hd != 128) return "head_dim must be 32, 64 or 128";
    if (Hkv < 1 || H < 1 || H % Hkv) return "n_head must be a positive multiple of n_head_kv";
    if (H > 4096) return "n_head must be at most 4096";
    if (n_ctx < 1 || n_seq < 1) return "n_ctx and n_seq must be positive";
    if (n_ctx > (1 << 30)) return "n_ctx must be at most 2^30";
    if ((double)n_seq * Hkv * n_ctx * hd > 0x1p46) return "the cache has more than 2^46 elements";
    return nullptr;
}

}  // namespace llm
