// k_attend_rows_f32.cu -- attend_rows.cuh for caches of binary32 (a file for each type: they compile side by side).
#include "attend_rows.cuh"

namespace gbper {
namespace attend {

cudaError_t attend_rows_f32(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    return rows_t<float>(a, PER_TYPE_F32, dev, st, bytes);
}

}  // namespace attend
}  // namespace gbper
