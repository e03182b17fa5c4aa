// Checks that the host entries of the operators around the attention share, and what they read off a plan.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_step.h"

namespace bsp {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int ilog2(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// Device (or managed) memory of the current device, aligned to `align` bytes.
inline bool device_ptr(const void* p, size_t align) {
    if (!p || (reinterpret_cast<uintptr_t>(p) & (align - 1))) return false;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (a.type == cudaMemoryTypeManaged) return true;
    int dev = 0;
    return a.type == cudaMemoryTypeDevice && cudaGetDevice(&dev) == cudaSuccess && a.device == dev;
}
inline bool optional_ptr(const void* p, size_t align) { return !p || device_ptr(p, align); }

// The plan's workspace is on the current device, where the kernel is going to read it.
inline bool plan_here(const bsp_plan_t* plan) { return device_ptr(plan->ws_device, 16); }

inline int32_t* status_word(const bsp_plan_t* plan) { return static_cast<int32_t*>(plan->ws_device); }
inline const int32_t* image_header(const bsp_plan_t* plan) {
    return reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan->ws_device) + kStatusBytes);
}
inline const int32_t* section(const bsp_plan_t* plan, uint64_t off) {
    return reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan->ws_device) + off);
}
// What the staged image's header says of this plan.
inline PlanShape plan_shape(const bsp_plan_t* plan) {
    const bsp_geometry& geo = plan->geo;
    return PlanShape{{static_cast<int32_t>(plan->generation), static_cast<int32_t>(plan->generation >> 32)},
                     plan->batch, plan->beam_width, plan->kind, plan->total_rows,
                     static_cast<int32_t>(plan->off_pages - kStatusBytes), geo.num_q_heads, geo.num_kv_heads,
                     geo.page_size, geo.head_dim};
}

inline bsp_status launched(cudaError_t e) {
    if (e == cudaSuccess) return BSP_OK;
    cudaGetLastError();
    return BSP_ERR_CUDA;
}

}  // namespace bsp
