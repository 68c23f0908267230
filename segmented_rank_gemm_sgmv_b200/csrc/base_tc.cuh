// What the two tensor-core kernels of the base products share.
#pragma once
#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "experts.h"
#include "ptx.cuh"

namespace sgmv {

constexpr int kTcRows = 128;           // rows of W in a tile
constexpr int kStageK = 128;           // K values of an operand stage
constexpr int kCodesK = 256;           // K values of a stage of codes: 128 bytes of a row

// mbar_try_wait that lets the hardware suspend the thread for up to 0.1 ms: many warps wait here at a time, and their
// polling would take the issue slots of those that work.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}
// Wait for a phase; gives up after kWaitLimitCycles, or when another thread of the block has (*abort_flag).
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
    if (mbar_try_wait_long(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_long(bar, parity) && !*abort_flag)
        if (clock64() - t0 > kWaitLimitCycles) {
            atomicOr(err, kErrTimeout);
            *abort_flag = 1;
        }
}

__device__ __forceinline__ void tma_load_3d(void* dst_smem, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst_smem)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One lane of a converged warp.  MMAs under this election have their operands in uniform registers; under a branch on
// the lane number each took about 200 cycles to issue, elected one by one about 100.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// The scales or zero points of N consecutive groups of a row, as loaded; `left`: groups of the row from the first on,
// `vec`: at least N, aligned to their size.
template <int N>
__device__ __forceinline__ void load_scales(uint32_t (&w)[N], const void* scales, int64_t at, int left, bool f32, bool vec) {
    if (vec) {
        if constexpr (N == 2) {
            if (f32) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(static_cast<const uint32_t*>(scales) + at);
            else w[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(scales) + at);
        } else {
            if (f32) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(scales) + at);
            else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(scales) + at);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) {
            if (f32) w[i] = static_cast<const uint32_t*>(scales)[at + i];
            else w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(scales)[at + i] << (i % 2 * 16);
        }
}
template <int N>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[N], int i, bool f32) {
    return f32 ? __uint_as_float(w[i]) : i % 2 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
}
template <int N>
__device__ __forceinline__ uint32_t load_zeros(const uint8_t* zeros, int64_t at, int left, bool vec) {
    if (vec) return N == 2 ? *reinterpret_cast<const uint16_t*>(zeros + at) : *reinterpret_cast<const uint32_t*>(zeros + at);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) w |= (uint32_t)zeros[at + i] << (8 * i);
    return w;
}

// The unit that blockIdx.y stands for among those of all experts in order: an expert's rows in units of even size, at
// most `most` rows.  Returns false if there is none; *e, *row and *row_end are then unset.  By all N threads of the
// block; offsets that do not ascend from 0 to at most a.rows are reported to *err, and no row outside y is named.
template <int N>
__device__ __forceinline__ bool find_unit(const BaseArgs& a, int most, unsigned int* err, int* e, int* row, int* row_end) {
    __shared__ int s_sum[N / 32];
    __shared__ int s_found[3];
    const int tid = threadIdx.x, lane = tid % 32, each = (a.experts + N - 1) / N;
    const int e0 = min(a.experts, tid * each), e1 = min(a.experts, e0 + each);
    if (tid == 0) s_found[0] = -1;
    const auto units_of = [&](int i, int* first, int* n) {
        const int lo = a.offsets[i], hi = a.offsets[i + 1];
        if (blockIdx.x + blockIdx.y == 0 && (lo < 0 || hi < lo || hi > a.rows || (i == 0 && lo != 0))) atomicOr(err, kErrExpert);
        *first = max(lo, 0);
        *n = max(min(hi, a.rows) - *first, 0);
        return (*n + most - 1) / most;
    };
    int units = 0, first, n;
    for (int i = e0; i < e1; ++i) units += units_of(i, &first, &n);
    int upto = units;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) s_sum[tid / 32] = upto;
    __syncthreads();
    for (int w = 0; w < tid / 32; ++w) upto += s_sum[w];
    int k = (int)blockIdx.y - (upto - units);
    if (k >= 0 && k < units)
        for (int i = e0; i < e1; ++i) {
            const int u = units_of(i, &first, &n);
            if (k < u) {
                s_found[0] = i;
                s_found[1] = first + (int)((int64_t)n * k / u);
                s_found[2] = first + (int)((int64_t)n * (k + 1) / u);
                break;
            }
            k -= u;
        }
    __syncthreads();
    *e = s_found[0];
    *row = s_found[1];
    *row_end = s_found[2];
    return s_found[0] >= 0;
}

// Allows `kern` its shared memory, once a kernel and device (the call takes about a microsecond), and refuses a build
// whose registers a thread differ from `registers`: setmaxnreg waits for good where a block has fewer at launch than its
// warpgroups ask for.
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kern, int smem, int registers, std::atomic<uint64_t>* done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
    if (attr.numRegs != registers) return cudaErrorInvalidConfiguration;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done->fetch_or(bit, std::memory_order_relaxed);
    return cudaSuccess;
}

// A tensor map with the 128-byte swizzle; what lies past an end reads as 0.
inline cudaError_t encode_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
// The codes, [experts][d_out][d_in / 2] bytes, in boxes of 128 rows of 128 bytes.
inline cudaError_t encode_codes(CUtensorMap* map, const BaseArgs& a) {
    const cuuint64_t row_bytes = a.d_in / 2;
    const cuuint64_t dims[3] = {row_bytes, (cuuint64_t)a.d_out, (cuuint64_t)a.experts}, strides[2] = {row_bytes, row_bytes * a.d_out};
    const cuuint32_t box[3] = {128, kTcRows, 1};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.codes, dims, strides, box);
}
}  // namespace sgmv
