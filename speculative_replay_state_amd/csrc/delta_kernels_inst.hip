// One checkpoint type's kernels of the gated delta rule (SSU_INST_ST = 0 fp32,
// 1 bf16, 2 fp16): the build compiles this file once per type.
#include "delta_kernels.cuh"

#ifndef SSU_INST_ST
#error "SSU_INST_ST must name the state type to instantiate"
#endif

namespace ssu {

template hipError_t delta_step_st<SSU_INST_ST>(const DCache &, const DStep &, int, hipStream_t);
template hipError_t delta_flush_st<SSU_INST_ST>(const DCache &, const int32_t *, const int32_t *, int, hipStream_t);
template hipError_t delta_init_st<SSU_INST_ST>(const DCache &, const float *, int64_t, const int32_t *, int,
                                               hipStream_t);
template hipError_t delta_read_st<SSU_INST_ST>(const DCache &, float *, int64_t, const int32_t *, int, hipStream_t);

}  // namespace ssu
