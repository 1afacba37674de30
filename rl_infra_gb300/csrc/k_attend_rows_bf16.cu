// k_attend_rows_bf16.cu -- attend_rows.cuh for caches of bfloat16 (a file for each type: they compile side by side).
#include "attend_rows.cuh"

namespace gbper {
namespace attend {

cudaError_t attend_rows_bf16(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    return rows_t<__nv_bfloat16>(a, PER_TYPE_BF16, dev, st, bytes);
}

}  // namespace attend
}  // namespace gbper
