// stage_tc.cu -- host side of the tensor-core products: tensor maps, and the
// record of waits that ran out.
#include <mutex>
#include <vector>

#include "stage_product.cuh"

namespace pps {
namespace {

std::mutex g_wait_mu;
std::vector<uint64_t (*)()> &wait_readers() {
    static std::vector<uint64_t (*)()> v;
    return v;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        (void)cudaGetLastError();
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

}  // namespace

int register_wait_reader(uint64_t (*reader)()) {
    std::lock_guard<std::mutex> lk(g_wait_mu);
    wait_readers().push_back(reader);
    return 0;
}

int encode_map(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t ld, int box_inner,
               int box_rows) {
    const EncodeTiled fn = encoder();
    if (!fn) return PP_ERR_CUDA;
    if (rows == 1) ld = round_up(inner, 8);  // there is no second row: any stride will do
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r =
        fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PP_OK : PP_ERR_CUDA;
}

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;
    }
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return 152;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

namespace {

__global__ void __launch_bounds__(256) k_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H,
                                                   const int64_t *target, int64_t V, uint16_t *out, int64_t ld) {
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        bool in = true;
        if (target) {
            const int64_t g = target[t];
            in = g >= 0 && g < V;
        }
        for (int64_t h = threadIdx.x; h < ld; h += blockDim.x) out[t * ld + h] = in && h < H ? x[t * stride + h] : 0;
    }
}

}  // namespace

int launch_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H, const int64_t *target, int64_t V,
                     uint16_t *out, int64_t ld, cudaStream_t stream) {
    k_copy_rows<<<(unsigned)(T < 152 * 32 ? T : 152 * 32), 256, 0, stream>>>(x, stride, T, H, target, V, out, ld);
    PPS_CUDA_TRY(cudaGetLastError());
    return PP_OK;
}

}  // namespace pps

extern "C" int pp_stage_wait_failure(uint64_t *first_failure) {
    if (!first_failure) return PP_ERR_ARG;
    uint64_t first = 0;
    std::lock_guard<std::mutex> lk(pps::g_wait_mu);
    PPS_CUDA_TRY(cudaDeviceSynchronize());
    for (uint64_t (*reader)() : pps::wait_readers()) {
        const uint64_t w = reader();
        if (!first) first = w;
    }
    *first_failure = first;
    return PP_OK;
}
