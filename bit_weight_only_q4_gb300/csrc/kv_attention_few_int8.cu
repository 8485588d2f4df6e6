// The attention kernel for few query rows over int8 caches.
#include "kv_attention_few.cuh"

namespace q4 {

KvKernel kv_few_kernel_int8(const DeviceInfo &dev, int head_dim, int rows)
{
    return head_dim == 64 ? kf_describe<Q4_CACHE_INT8, 64>(dev, rows) : kf_describe<Q4_CACHE_INT8, 128>(dev, rows);
}

}  // namespace q4
