// Base products from 4-bit weights with group scales, y = W x: one matrix for all rows, or one per
// expert over rows sorted by expert.
#include <algorithm>
#include <string>

#include "experts.h"
#include "ptx.cuh"

namespace sgmv {

__device__ unsigned int g_err_base;

namespace {

constexpr int kSimpleWarps = 8;

__device__ __forceinline__ float load_scale(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i]
               : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Expert of row r: the last e with offsets[e] <= r (offsets ascend); -1 past the last row.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int experts, int r) {
    if (r >= offsets[experts]) return -1;
    int lo = 0, hi = experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (offsets[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// The first block reports offsets that do not ascend from 0 to at most `rows`.
__device__ __forceinline__ void check_offsets(const BaseArgs& a) {
    if (!a.offsets || blockIdx.x + blockIdx.y > 0) return;
    for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) {
        const int o = a.offsets[e];
        if (e == 0 ? o != 0 : o < a.offsets[e - 1] || o > a.rows) atomicOr(&g_err_base, kErrExpert);
    }
}

// One output a warp: y[r][n] = sum_g s[n][g] sum_{c in g} (q[n][c] - z[n][g]) x[r][c], in fp32.
template <bool YF32>
__global__ void __launch_bounds__(kSimpleWarps * 32) base_simple_kernel(BaseArgs a, bool scale_f32) {
    check_offsets(a);
    const int n = blockIdx.x * kSimpleWarps + threadIdx.x / 32, r = blockIdx.y, lane = threadIdx.x % 32;
    if (n >= a.d_out) return;
    int e = 0;
    int64_t xr = r;
    if (a.offsets) {
        e = expert_of(a.offsets, a.experts, r);
        if (e < 0) return;
    }
    if (a.slot_of) {
        const int slot = a.slot_of[r];
        xr = slot / a.k;
        if (slot < 0 || xr >= a.x_rows) {
            if (lane == 0) atomicOr(&g_err_base, kErrRows);
            return;
        }
    }
    const int64_t row = (int64_t)e * a.d_out + n;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.codes + row * (a.d_in / 2));
    const uint16_t* x = a.x + xr * a.ldx;
    const int64_t g0 = row * (a.d_in / a.group);
    float acc = 0.0f;
    for (int u = lane; u < a.d_in / 8; u += 32) {
        const int64_t g = g0 + u * 8 / a.group;
        const float z = a.zeros ? (float)a.zeros[g] : 8.0f;
        uint32_t codes = q[u];
        if (!a.zeros) codes ^= 0x88888888u;   // two's complement to excess 8
        float f[8], s = 0.0f;
        unpack8(*reinterpret_cast<const uint4*>(x + u * 8), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf((float)((codes >> (4 * i)) & 15u) - z, f[i], s);
        acc = fmaf(load_scale(a.scales, g, scale_f32), s, acc);
    }
    for (int o = 16; o > 0; o /= 2) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) {
        if (YF32) static_cast<float*>(a.y)[r * a.ldy + n] = acc;
        else static_cast<uint16_t*>(a.y)[r * a.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
    }
}

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

sgmv_status product_impl(const char* who_, BaseArgs a, int32_t scale_dtype, int32_t y_dtype, cudaStream_t stream) {
    const std::string who(who_);
    if (a.rows < 0 || a.x_rows < 0 || a.d_in < 1 || a.d_out < 1)
        return fail(SGMV_ERR_INVALID, who + ": the numbers of rows must be >= 0, d_in and d_out >= 1");
    if (a.group != 32 && a.group != 64 && a.group != 128)
        return fail(SGMV_ERR_INVALID, who + ": group must be 32, 64 or 128");
    if (a.d_in % a.group) return fail(SGMV_ERR_INVALID, who + ": d_in must be a multiple of group");
    if ((scale_dtype != 0 && scale_dtype != 1) || (y_dtype != 0 && y_dtype != 1))
        return fail(SGMV_ERR_INVALID, who + ": scale_dtype and y_dtype must be 0 (bf16) or 1 (fp32)");
    if (a.rows == 0) return SGMV_OK;
    if (!a.x || !a.codes || !a.scales || !a.y) return fail(SGMV_ERR_INVALID, who + ": x, codes, scales and y are required");
    if (a.ldx < a.d_in || a.ldx % 8 || !aligned(a.x, 16))
        return fail(SGMV_ERR_INVALID, who + ": x rows must be 16-byte aligned, ldx >= d_in");
    if (!aligned(a.codes, 16)) return fail(SGMV_ERR_INVALID, who + ": codes must be 16-byte aligned");
    if (!aligned(a.scales, scale_dtype ? 4 : 2)) return fail(SGMV_ERR_INVALID, who + ": scales must be aligned to their type");
    if (a.ldy < a.d_out || !aligned(a.y, y_dtype ? 4 : 2))
        return fail(SGMV_ERR_INVALID, who + ": y must be aligned to its type, ldy >= d_out");
    const dim3 grid((a.d_out + kSimpleWarps - 1) / kSimpleWarps, a.rows);
    if (y_dtype) base_simple_kernel<true><<<grid, kSimpleWarps * 32, 0, stream>>>(a, scale_dtype == 1);
    else base_simple_kernel<false><<<grid, kSimpleWarps * 32, 0, stream>>>(a, scale_dtype == 1);
    SGMV_CUDA_TRY(cudaGetLastError());
    return SGMV_OK;
}

}  // namespace

cudaError_t read_clear_errors_base(uint32_t* bits, cudaStream_t stream) {
    unsigned int h = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&h, g_err_base, sizeof(h), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_err_base, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *bits |= h;
    return e;
}

}  // namespace sgmv

using namespace sgmv;

extern "C" sgmv_status sgmv_base_product(const void* x, int64_t ldx, int32_t T, int32_t d_in, int32_t d_out,
                                         const void* codes, const void* scales, int32_t scale_dtype,
                                         const uint8_t* zeros, int32_t group, void* y, int64_t ldy, int32_t y_dtype,
                                         sgmv_stream_t stream) {
    const BaseArgs a{static_cast<const uint16_t*>(x), ldx, static_cast<const uint8_t*>(codes), scales, zeros, y, ldy,
                     nullptr, nullptr, T, T, 1, 1, d_in, d_out, group};
    return product_impl("base_product", a, scale_dtype, y_dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sgmv_status sgmv_base_product_experts(const void* x, int64_t ldx, int32_t x_rows, int32_t d_in,
                                                 int32_t d_out, int32_t n_experts, const void* codes,
                                                 const void* scales, int32_t scale_dtype, const uint8_t* zeros,
                                                 int32_t group, const int32_t* offsets, const int32_t* slot_of,
                                                 int32_t k, int32_t rows, void* y, int64_t ldy, int32_t y_dtype,
                                                 sgmv_stream_t stream) {
    const char* who = "base_product_experts";
    if (n_experts < 1 || n_experts > kMaxExperts)
        return fail(SGMV_ERR_INVALID, "base_product_experts: the number of experts must be in 1..4096");
    if (rows > 0 && (!offsets || !aligned(offsets, 4) || (slot_of && !aligned(slot_of, 4))))
        return fail(SGMV_ERR_INVALID, "base_product_experts: offsets are required; offsets and slot_of 4-byte aligned");
    if (slot_of ? (k < 1 || k > kMaxExpertsPerToken) : x_rows < rows)
        return fail(SGMV_ERR_INVALID, "base_product_experts: slot_of needs k in 1..64; without it x has a row for every row of y");
    const BaseArgs a{static_cast<const uint16_t*>(x), ldx, static_cast<const uint8_t*>(codes), scales, zeros, y, ldy,
                     offsets, slot_of, rows, x_rows, slot_of ? k : 1, n_experts, d_in, d_out, group};
    return product_impl(who, a, scale_dtype, y_dtype, reinterpret_cast<cudaStream_t>(stream));
}
