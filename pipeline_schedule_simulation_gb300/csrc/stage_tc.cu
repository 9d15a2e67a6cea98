// stage_tc.cu -- host side of the tensor-core products: tensor maps, and the
// record of waits that ran out.
#include "stage_kept.cuh"
#include "stage_product.cuh"

namespace pps {
namespace {

// Units register while the library is loaded, before or after this one.
WaitRecords &wait_records() {
    static WaitRecords r;
    return r;
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

int register_wait_reader(WaitReader *r) {
    wait_records().add(r);
    return 0;
}

int encode_map(CUtensorMap *map, const Matrix &m, int64_t rows, int64_t cols, bool panels, int box_rows,
               int box_panels) {
    const EncodeTiled fn = encoder();
    if (!fn) return PP_ERR_CUDA;
    // a row's stride is of no account where there is one row
    const int64_t ld = rows == 1 ? round_up(m.ld, 8) : m.ld;
    const cuuint64_t dims[3] = {panels ? 64 : (cuuint64_t)cols, (cuuint64_t)rows,
                                panels ? (cuuint64_t)ceil_div(cols, 64) : 1};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, panels ? (cuuint64_t)m.panel * 2 : (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_panels}, step[3] = {1, 1, 1};
    const CUresult r =
        fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(m.p), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PP_OK : PP_ERR_CUDA;
}

ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool by_64, bool may_split) {
    const int64_t sms = sm_count(), blocks = ceil_div(K, kTileK);
    const double start = 6;  // slices that a tile's start and end cost
    // a slice's 512 cycles at about 1.8 GHz, in bytes of memory traffic
    const double part_cost = 8. * (double)M * (double)N / 1.9e6;
    ProductPlan best{};
    double least = 0;
    const auto consider = [&](int cg, int64_t tile_n) {
        ProductPlan p;
        p.cg = cg, p.tile_n = (int)tile_n;
        p.mt = ceil_div(M, kHalf * cg), p.nt = ceil_div(N, tile_n);
        const int64_t tiles = p.mt * p.nt, units = sms / cg;
        const double slice = cg == 2 ? 1. : (256. + 2. * (double)tile_n) / 512.;
        int64_t parts = may_split ? units / tiles : 1;
        if (parts > blocks / 4) parts = blocks / 4;
        for (int64_t s : {(int64_t)1, parts}) {
            if (s < 1) continue;
            s = ceil_div(blocks, ceil_div(blocks, s));  // no part is empty
            const double cost = (double)ceil_div(tiles * s, units) * ((double)ceil_div(blocks, s) * slice + start) +
                                (s > 1 ? (double)s * part_cost + start : 0.);
            p.splits = (int)s;
            if (best.cg == 0 || cost < least) best = p, least = cost;
        }
    };
    if (M > kHalf) consider(2, 256);
    const int64_t mt = ceil_div(M, kHalf), to = by_64 ? 64 : 16;
    for (int64_t waves = 1; waves <= 4; ++waves) {
        const int64_t columns = sms * waves / mt;  // column tiles that fill the SMs
        if (columns < 1) continue;
        const int64_t n = round_up(ceil_div(N, columns), to);
        if (n <= 256) consider(1, n);
    }
    consider(1, 128);
    consider(1, 256);
    return best;
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

// A thread copies 8 columns of 4 rows.
constexpr int kCopyRows = 4;
template <bool VEC>
__global__ void __launch_bounds__(256) k_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H,
                                                   const int64_t *target, int64_t V, int *clear, uint16_t *out,
                                                   int64_t ld, int64_t panel) {
    let_next_start();
    after_previous();
    const int64_t per = (H + 63) / 64 * 8, u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, g = u / per;
    if (clear)
        for (int64_t i = u; i < V; i += (int64_t)gridDim.x * blockDim.x) clear[i] = -1;
    const int64_t t = g * kCopyRows, c = (u - g * per) * 8, left = H - c;
    Raw8 r[kCopyRows];
#pragma unroll
    for (int i = 0; i < kCopyRows; ++i) {
        bool in = t + i < T && left > 0;
        if (in && target) {
            const int64_t v = target[t + i];
            in = v >= 0 && v < V;
        }
        r[i] = Raw8{};
        if (in) r[i] = load8<VEC>(x + (t + i) * stride + c, left);
    }
#pragma unroll
    for (int i = 0; i < kCopyRows; ++i)
        if (t + i < T) store8<true>(out + (t + i) * ld + c / 64 * panel + c % 64, 8, r[i]);
}

}  // namespace

int launch_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H, const int64_t *target, int64_t V,
                     int *clear, uint16_t *out, int64_t ld, int64_t panel, cudaStream_t stream) {
    const int64_t grid = ceil_div(ceil_div(T, kCopyRows) * ceil_div(H, 64) * 8, 256);
    return launch_after(rows_aligned(x, stride, T, 2) ? k_copy_rows<true> : k_copy_rows<false>, grid, 256, 0, stream, 1, x,
                        stride, T, H, target, V, clear, out, ld, panel);
}

static int take_waits(uint64_t *record) { return wait_records().take(record); }

}  // namespace pps

extern "C" int pp_stage_wait_failure(uint64_t *first_failure) {
    if (!first_failure) return PP_ERR_ARG;
    *first_failure = 0;
    PPS_CUDA_TRY(cudaDeviceSynchronize());
    const int e = pps::take_waits(first_failure);
    if (e) (void)cudaGetLastError();
    return e ? PP_ERR_CUDA : PP_OK;
}
