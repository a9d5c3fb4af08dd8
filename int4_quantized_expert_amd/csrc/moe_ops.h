// moe_ops.h — launches and workspaces of the routing and linear operators (k_route.hip, k_linear.hip), which the C
// entries in moe_ops.hip call.
#pragma once
#include "moe_internal.h"

namespace moe {

// routing from logits and its gradients
size_t route_ws_bytes(int E, int T);
hipError_t launch_moe_route(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                            const float* bias, const uint8_t* valid, int32_t* ids, float* w, int32_t* load, float* imp,
                            void* ws, hipStream_t st);
hipError_t launch_moe_route_grad(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                                 const uint8_t* valid, const int32_t* ids, const float* dw, const float* dimp, void* dz,
                                 int64_t ld_d, hipStream_t st);
// slots whose id, taken as unsigned, is not below id_end are dropped
hipError_t launch_slot_grad(const float* eout, const int32_t* ids, const float* dy, int T, int K, int H, uint32_t id_end,
                            float* dw, hipStream_t st);
// product over weight codes with its epilogue
size_t linear_ws_bytes(const moe_linear_config& c, int64_t T);
hipError_t launch_linear(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                         const void* x, int64_t ldx, int T, int dtype, const void* res, int64_t ldr, void* y,
                         int64_t ldy, void* ws, hipStream_t st);

}  // namespace moe
