// Base products from 4-bit weights for many rows of x: tcgen05 tensor cores, fp32 accumulation per group.
#include <algorithm>
#include <cstring>

#include "base_tc.cuh"

namespace sgmv {

__device__ unsigned int g_err_base_tc;

namespace {

// y^T = W x^T in tiles of 128 rows of W and NTOK rows of x.  tcgen05.mma takes the codes less their zero points,
// exact in bf16, as its A operand and x as B, and sums one group of K values at a time into tensor memory; the
// epilogue warps fetch each group's sums and add them, times the row's fp32 scale, to totals in registers, so that
// no scale is ever rounded to bf16.  The converted codes go straight to tensor memory (a thread holds a row, which is
// a lane there): through shared memory they made its bandwidth the bound, at 61 % of the MMA rate.
//
// Everything that hands an accumulator over (waits, fences, the issue of 8 MMAs) takes about 1000 cycles, as long as
// the MMAs of 128 x 256 x 128.  So there are two lanes, each an MMA warp, an accumulator of at most 128 columns and a
// set of epilogue warps: with more than 128 rows of x they take half of the rows each, else alternate groups, whose
// totals are added at the end.
//
// What bounds it: with 256 rows of x, shared memory (x written and read once, 1152 cycles for 128 K values) and the
// tensor cores (1024); with groups of 32 and with few rows, the handing over, the conversion and the stream of codes.
// 4096 rows, 8192 x 8192, groups of 128: 462 us, 1.19 PFLOP/s (floor 336 us): a tile of 70 us is 62 of stages, 3 until
// the first accumulator, 1 to put the totals together and 3 to write y.  256 rows, 8192 x 8192: 40 us; 256 rows,
// 14336 x 4096, groups of 32: 91 us (floor 18), a handover for every 32 K values.  32 rows, 8192 x 28672: 48 us, 2.6 TB/s.
//
// Roles: warp 0 streams codes (TMA, stages of 128 rows x 256 values), 2 copies x (TMA), 1 and 3 issue the MMAs, 4 or 8
// warps convert (of 8, half take each stage), the rest are the epilogue.  K is split over the CTAs of a cluster when
// there are few tiles.  All totals meet in shared memory in a fixed order.
template <int G, int NTOK>
struct TcConfig {
    static constexpr int kConvert = NTOK == 256 ? 4 : NTOK == 128 || G < 128 ? 8 : 16;       // warps
    static constexpr int kEpilogue = NTOK == 256 ? 16 : 8;
    static constexpr int kThreads = (4 + kConvert + kEpilogue) * 32;
    static constexpr int kRegisters = NTOK == 256 ? 80 : kConvert == 8 ? 96 : 72;     // a thread at launch
    static constexpr int kPassCols = NTOK < 128 ? NTOK : 128;        // columns of an accumulator
    static constexpr int kCols = kPassCols / (kEpilogue / 8);        // of them, an epilogue warp's
    static constexpr int kStages = NTOK <= 64 ? 6 : 3;               // of 128 K values
    static constexpr int kCodeStages = NTOK == 256 ? 2 : 3;          // of 256 K values
    static constexpr int kB = NTOK * 256, kCodes = 128 * 128;
    static constexpr int kSmem = 1024 + kStages * kB + kCodeStages * kCodes;
    static constexpr int kTmemA = 2 * kPassCols, kTmem = kTmemA + kStages * 64 <= 256 ? 256 : 512;    // columns
    static constexpr int kRedStride = 132;                           // floats of a row of totals
    static_assert(2 * kPassCols * kRedStride * 4 <= kSmem - 1024, "the totals fit into the operands' memory");
    static_assert(kSmem <= 227 * 1024 && kTmemA + kStages * 64 <= 512, "the stages fit");
};
// D[tmem] (+)= A[tmem] * B[smem]^T: A has a lane a row and two consecutive K values a column.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// setmaxnreg to N registers a thread, more (inc) or fewer than now; by whole warpgroups.  At the end all go back to the
// launch's count, lest the epilogue of the block is compiled for the least of them (its spills took 15 us): the warps
// that had taken registers give them up before the block's barrier, the others take theirs after it, since before it
// some might still be waiting for registers themselves.
template <int N, bool inc>
__device__ __forceinline__ void set_registers() {
    if constexpr (inc) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Eight codes (value i in bits 4i..4i+3) less the zero point, as eight bf16 in order.  bf16 128 + n has the bits
// 0x4300 | n for n < 128, so inserting the code and subtracting 128 + z is exact.  `flip` is 0x08080808 for two's
// complement codes (n ^ 8 is the value plus 8; then z is 8).
__device__ __forceinline__ void convert8(uint32_t c, uint32_t flip, uint32_t z2, uint32_t* out) {
    const uint32_t even = (c & 0x0f0f0f0fu) ^ flip, odd = ((c >> 4) & 0x0f0f0f0fu) ^ flip;
    const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
    uint32_t p[4] = {__byte_perm(lo, 0x43u, 0x4140), __byte_perm(lo, 0x43u, 0x4342), __byte_perm(hi, 0x43u, 0x4140),
                     __byte_perm(hi, 0x43u, 0x4342)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&p[i]), *reinterpret_cast<const __nv_bfloat162*>(&z2));
        out[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

template <int G, int NTOK, bool Z>
__global__ void __launch_bounds__(TcConfig<G, NTOK>::kThreads, 1)
    base_tc_kernel(BaseArgs a, const __grid_constant__ CUtensorMap codes_map,
                   const __grid_constant__ CUtensorMap x_map, bool scale_f32, bool y_f32, bool vec, int n_split) {
    using C = TcConfig<G, NTOK>;
    constexpr int kSpan = G == 32 ? 128 : 256, kGroups = kSpan / G;  // K values whose scales are loaded together
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages], s_cfull[C::kCodeStages], s_cempty[C::kCodeStages],
        s_afull[2], s_aempty[2], s_done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_xrow[NTOK];         // -1: the row of y is not written
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
    const int rank = blockIdx.x % n_split, n0 = (int)(blockIdx.x / n_split) * kTcRows;
    uint8_t* stages = smem_raw + (1024 - smem_u32(smem_raw) % 1024) % 1024;  // [kStages][2][NTOK] rows of 64 values of x
    uint8_t* codes = stages + C::kStages * C::kB;                            // [kCodeStages][128] rows of 256 codes

    // the unit: up to NTOK consecutive rows of y of one matrix
    int e = 0, row0 = blockIdx.y * NTOK, row_end = min(a.rows, (int)(blockIdx.y + 1) * NTOK);
    if (a.offsets && !find_unit<C::kThreads>(a, NTOK, &g_err_base_tc, &e, &row0, &row_end)) return;
    const int n_tok = row_end - row0;
    // this CTA's code stages of K (256 values) and operand stages (128)
    const int all = (a.d_in + 255) / 256;
    const int c0 = (int)((int64_t)all * rank / n_split), c1 = (int)((int64_t)all * (rank + 1) / n_split);
    const int k_begin = c0 * 256, k_end = min(a.d_in, c1 * 256), n_k = (k_end - k_begin + kStageK - 1) / kStageK;
    const int n_pad = (n_tok + 15) / 16 * 16;    // columns of the MMAs
    const bool halves = n_pad > C::kPassCols;    // the lanes take half of the rows each, else alternate groups
    const int half = (n_pad / 2 + 15) / 16 * 16; // then the first lane's rows
    const bool alone = !halves && G == kStageK;  // then each stage is one lane's
    const int groups = a.d_in / G;

    const auto copy_codes = [&](int i) {
        mbar_arrive_expect_tx(&s_cfull[i % C::kCodeStages], C::kCodes);
        tma_load_3d(codes + i % C::kCodeStages * C::kCodes, &codes_map, (c0 + i) * 128, n0, e, &s_cfull[i % C::kCodeStages]);
    };
    const auto copy_x = [&](int kt) {
        const int s = kt % C::kStages;
        mbar_arrive_expect_tx(&s_full[s], C::kB);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            tma_load_2d(stages + s * C::kB + i * NTOK * 128, &x_map, k_begin + kt * kStageK + i * 64, row0, &s_full[s]);
    };
    if (tid < NTOK) {
        int r = -1;
        if (tid < n_tok) {
            r = row0 + tid;
            if (a.slot_of) {
                const int slot = a.slot_of[r];
                if (slot < 0 || slot / a.k >= a.x_rows) r = -1;       // reported by the gather
            }
        }
        s_xrow[tid] = r;
    }
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&s_full[i], 128 + 1);
            mbar_init(&s_empty[i], alone ? 1 : 2);
        }
        for (int i = 0; i < C::kCodeStages; ++i) {
            mbar_init(&s_cfull[i], 1);
            mbar_init(&s_cempty[i], C::kConvert == 4 ? 128 : 256);           // the threads that read a stage
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_afull[i], 1);
            mbar_init(&s_aempty[i], C::kEpilogue / 2);
        }
        mbar_init(&s_done, 2);
        s_abort = 0;
        fence_mbar_init();
        for (int i = 0; i < min(C::kCodeStages, c1 - c0); ++i) copy_codes(i);      // the first copies start here
        for (int kt = 0; kt < min(C::kStages, n_k); ++kt) copy_x(kt);
    }
    if (warp == 1) {
        tmem_alloc(&s_tmem, C::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    // waits give up together: whoever runs out of time stops the others' waits too
    volatile int* abort_flag = &s_abort;
    const auto wait = [&](uint64_t* bar, uint32_t parity) { wait_or_abort(bar, parity, abort_flag, &g_err_base_tc); };

    float* red = reinterpret_cast<float*>(stages);                   // [2 kPassCols][kRedStride] totals

    if (warp < 4) {
        // registers at launch: 7 warpgroups of 72 = 40 + 4 x 56 + 2 x 120; 5 of 96 = 48 + 2 x 56 + 2 x 160; 6 of 80 =
        // 40 + 56 + 4 x 96
        if constexpr (C::kConvert == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            if (elect_one()) {
                int i = min(C::kCodeStages, c1 - c0);
                for (; i < c1 - c0; ++i) {
                    wait(&s_cempty[i % C::kCodeStages], (i / C::kCodeStages - 1) & 1);
                    if (*abort_flag) break;
                    copy_codes(i);
                }
                for (int j = max(0, i - C::kCodeStages); j < i; ++j)         // no copy is left in flight
                    mbar_wait(&s_cfull[j % C::kCodeStages], (j / C::kCodeStages) & 1, &g_err_base_tc);
            }
        } else if (warp == 1 || warp == 3) {
            const int ln = warp / 2;     // 0 or 1
            const uint64_t bdesc = smem_desc_sw128(smem_u32(stages), 16, 1024) + (halves ? ln * half * (128 / 16) : 0);
            const uint32_t idesc = idesc_bf16_f32(128, halves ? (ln ? n_pad - half : half) : n_pad, false, false);
            const uint32_t d = tmem + ln * C::kPassCols;
            int n = 0, g = 0;            // this lane's groups begun; the stage's first group
            for (int kt = alone ? ln : 0; kt < n_k; kt += alone ? 2 : 1) {
                const int s = kt % C::kStages;
                wait(&s_full[s], (kt / C::kStages) & 1);
                tc_fence_after();
                const int n_groups = min(kStageK, k_end - k_begin - kt * kStageK) / G;
                const uint32_t at = tmem + C::kTmemA + s * 64;
                const uint64_t bd = bdesc + (uint64_t)(s * (C::kB / 16));
#pragma unroll
                for (int gi = 0; gi < kStageK / G; ++gi) {
                    if (gi >= n_groups) break;
                    if (!halves && !alone && (g + gi) % 2 != ln) continue;
                    if (n > 0) {
                        wait(&s_aempty[ln], (n - 1) & 1);
                        tc_fence_after();
                    }
                    ++n;
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < G / 16; ++i) {
                            const int ks = gi * (G / 16) + i;
                            tc_mma_bf16_ts(d, at + ks * 8, bd + (ks / 4) * (NTOK * 128 / 16) + ks % 4 * 2, idesc, i > 0);
                        }
                        tc_commit(&s_afull[ln]);
                    }
                    __syncwarp();
                }
                g += n_groups;
                if (elect_one()) tc_commit(&s_empty[s]);     // arrives at once where this lane had no group
                __syncwarp();
            }
            if (elect_one()) tc_commit(&s_done);     // no MMA is left in flight
            mbar_wait(&s_done, 0, &g_err_base_tc);
        } else if (warp == 2) {
            const bool copier = elect_one();
            int n_x = min(C::kStages, n_k);          // stages asked for
            for (; copier && n_x < n_k; ++n_x) {
                wait(&s_empty[n_x % C::kStages], (n_x / C::kStages - 1) & 1);
                if (*abort_flag) break;
                copy_x(n_x);
            }
            if (*abort_flag)             // no copy is left in flight
                for (int kt = max(0, n_x - C::kStages); kt < n_x; ++kt) mbar_wait(&s_full[kt % C::kStages], (kt / C::kStages) & 1, &g_err_base_tc);
        }
        __syncwarp();
        named_bar_sync(2, C::kThreads);
        set_registers<C::kRegisters, true>();
    } else if (warp < 4 + C::kConvert) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int r = (tid - 128) % 128, part = (warp - 4) / 4;      // a row; of two sets of warps each takes alternate stages
        constexpr int kParts = C::kConvert / 4;
        const int64_t zrow = ((int64_t)e * a.d_out + min(n0 + r, a.d_out - 1)) * groups;
        const auto zeros_at = [&](int k) {
            const int g = min(k, a.d_in - 1) / kSpan * kGroups;
            return load_zeros<kGroups>(a.zeros, zrow + g, groups - g, vec);
        };
        uint32_t z_now = 0, z_next = Z ? zeros_at(k_begin + part * kStageK) : 0;
        int z_span = -1;                 // the span that z_now is of
        const uint32_t to = tmem + C::kTmemA + ((uint32_t)(warp % 4 * 32) << 16);
        for (int kt = part; kt < n_k; kt += kParts) {
            const int k = k_begin + kt * kStageK;
            if (Z && k / kSpan != z_span) {
                z_span = k / kSpan;
                z_now = z_next;
                z_next = zeros_at(k + max(kSpan, kParts * kStageK));    // of this warp's next span
            }
            const int s = kt % C::kStages, ci = kt / 2, cs = ci % C::kCodeStages;
            wait(&s_cfull[cs], (ci / C::kCodeStages) & 1);
            const uint8_t* cp = codes + cs * C::kCodes + r * 128;
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(cp + ((kt % 2 * 4 + i) ^ (r & 7)) * 16);
            if (kt >= C::kStages) wait(&s_empty[s], (kt / C::kStages - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t z2 = Z ? (0x4300u | (z_now >> ((k + 32 * i) % kSpan / G * 8) & 0xffu)) * 0x10001u : 0x43084308u;
                uint32_t w[16];
                convert8(v[i].x, Z ? 0u : 0x08080808u, z2, w);
                convert8(v[i].y, Z ? 0u : 0x08080808u, z2, w + 4);
                convert8(v[i].z, Z ? 0u : 0x08080808u, z2, w + 8);
                convert8(v[i].w, Z ? 0u : 0x08080808u, z2, w + 12);
                tmem_st_x16(to + s * 64 + i * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&s_full[s]);
            if (kParts > 1 || kt % 2 == 1) mbar_arrive(&s_cempty[cs]);
        }
        named_bar_sync(2, C::kThreads);
        set_registers<C::kRegisters, true>();
    } else {
        if constexpr (NTOK == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        else if constexpr (C::kConvert == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        const int ew = warp - 4 - C::kConvert, ln = ew / (C::kEpilogue / 2);
        const int erow = (warp % 4) * 32 + lane, ecol = ew % (C::kEpilogue / 2) / 4 * C::kCols;     // of the lane's accumulator
        const int cols = (halves ? (ln ? n_pad - half : half) : n_pad) - ecol;      // of this warp's that are used
        float total[C::kCols];
        const int64_t srow = ((int64_t)e * a.d_out + min(n0 + erow, a.d_out - 1)) * groups;
#pragma unroll
        for (int i = 0; i < C::kCols; ++i) total[i] = 0.0f;
        const int g0 = k_begin / G, g1 = k_end / G;
        uint32_t now[kGroups], next[kGroups];
        load_scales(next, a.scales, srow + g0, groups - g0, scale_f32, vec);
        int n = 0;                       // groups done
        for (int gs = g0; gs < g1; gs += kGroups) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) now[i] = next[i];
            if (gs + kGroups < g1) load_scales(next, a.scales, srow + gs + kGroups, groups - gs - kGroups, scale_f32, vec);
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi) {
                if (gs + gi >= g1) break;
                if (!halves && gi % 2 != ln) continue;               // a span begins at an even group
                const float sc = scale_of(now, gi, scale_f32);
                wait(&s_afull[ln], n++ & 1);
                tc_fence_after();
                const uint32_t from = tmem + ln * C::kPassCols + ecol + ((uint32_t)(warp % 4 * 32) << 16);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 32) {
                    if (c >= cols) break;
                    uint32_t v0[16], v1[16];
                    tmem_ld_x16(from + c, v0);
                    if (C::kCols > 16) tmem_ld_x16(from + c + 16, v1);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) total[c + i] = fmaf(sc, __uint_as_float(v0[i]), total[c + i]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) total[c + 16 + i] = fmaf(sc, __uint_as_float(v1[i]), total[c + 16 + i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_aempty[ln]);
            }
        }
        named_bar_sync(1, C::kEpilogue * 32);        // both lanes' last MMAs are complete: the totals take the stages' memory
#pragma unroll
        for (int i = 0; i < C::kCols; ++i)
            if (i < cols) red[(ln * C::kPassCols + ecol + i) * C::kRedStride + erow] = total[i];
        set_registers<C::kRegisters, false>();
        named_bar_sync(2, C::kThreads);
    }
    // the totals of the lanes and of the cluster's CTAs, in a fixed order
    if (n_split > 1) cluster_sync();
    // (a warp a row: the registers straight to y, 64 bytes of a row at a time, took 4.5 us more for 256 rows)
    const uint32_t base = smem_u32(red);
    const int n = n0 + lane * 4;
    const bool dead = *abort_flag, wide = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % (y_f32 ? 16 : 8) == 0 && n + 4 <= a.d_out;
    for (int t = rank * (C::kThreads / 32) + warp; t < n_tok; t += n_split * (C::kThreads / 32)) {
        const int at = halves && t >= half ? C::kPassCols + t - half : t;    // of the totals' rows
        const uint32_t at0 = (at * C::kRedStride + lane * 4) * 4, at1 = at0 + C::kPassCols * C::kRedStride * 4;
        float4 v;
        if (n_split == 1) {
            v = *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(red) + at0);
            if (!halves) v = add4(v, *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(red) + at1));
        } else {
            float4 u[8], w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                u[c] = w[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c < n_split) {
                    const uint32_t from = map_cluster(base, c);
                    u[c] = ld_cluster_v4(from + at0);
                    if (!halves) w[c] = ld_cluster_v4(from + at1);
                }
            }
            v = add4(u[0], w[0]);
#pragma unroll
            for (int c = 1; c < 8; ++c) v = add4(v, add4(u[c], w[c]));
        }
        if (s_xrow[t] < 0 || dead) continue;
        const int64_t to = (int64_t)(row0 + t) * a.ldy + n;
        if (wide) {
            if (y_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.y) + to) = v;
            else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + to) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            continue;
        }
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= a.d_out) break;
            if (y_f32) static_cast<float*>(a.y)[to + i] = f[i];
            else static_cast<uint16_t*>(a.y)[to + i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
        }
    }
    if (n_split > 1) {
        cluster_arrive_relaxed();        // every CTA of the cluster has read the totals
        cluster_wait_acquire();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// x in boxes of 64 values of `rows` rows; with slots, it has been gathered into a row for each row of y.
cudaError_t encode_x(CUtensorMap* map, const BaseArgs& a, int rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)a.d_in, (cuuint64_t)(a.slot_of ? a.rows : a.x_rows)}, strides[1] = {(cuuint64_t)a.ldx * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.x, dims, strides, box);
}

template <int G, int NTOK, bool Z>
cudaError_t launch_t(const BaseArgs& a, bool scale_f32, bool y_f32, cudaStream_t stream) {
    using C = TcConfig<G, NTOK>;
    auto kern = base_tc_kernel<G, NTOK, Z>;
    static std::atomic<uint64_t> done{0};
    cudaError_t err = prepare_kernel(kern, C::kSmem, C::kRegisters, &done);
    if (err != cudaSuccess) return err;
    CUtensorMap map, x_map;
    if ((err = encode_codes(&map, a)) != cudaSuccess || (err = encode_x(&x_map, a, NTOK)) != cudaSuccess) return err;
    const int tiles = (a.d_out + kTcRows - 1) / kTcRows, k_stages = (a.d_in + 255) / 256;
    const int64_t units = a.offsets ? (int64_t)a.rows / NTOK + std::min(a.rows, a.experts) : ((int64_t)a.rows + NTOK - 1) / NTOK;
    // the split of K that takes the fewest rounds of 148 CTAs, each counted with four code stages' worth of fixed cost
    int split = 1;
    double best = 0;
    for (int c = 1; c <= std::min(8, k_stages); ++c) {
        const double cost = (double)((tiles * units * c + 147) / 148) * ((k_stages + c - 1) / c + 4);
        if (c == 1 || cost < 0.97 * best) best = cost, split = c;
        if (a.offsets) break;
    }
    constexpr int kSpan = G == 32 ? 128 : 256;
    const auto at = [](const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const bool vec = a.d_in % kSpan == 0 && at(a.scales, 16) && at(a.zeros, 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)units);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, map, x_map, scale_f32, y_f32, vec, split);
}

template <int G, bool Z>
cudaError_t launch_g(const BaseArgs& a, int64_t per, bool scale_f32, bool y_f32, cudaStream_t stream) {
    if (per <= 32) return launch_t<G, 32, Z>(a, scale_f32, y_f32, stream);
    if (per <= 64) return launch_t<G, 64, Z>(a, scale_f32, y_f32, stream);
    if (per <= 128) return launch_t<G, 128, Z>(a, scale_f32, y_f32, stream);
    return launch_t<G, 256, Z>(a, scale_f32, y_f32, stream);
}

}  // namespace

cudaError_t launch_base_tc(const BaseArgs& a, int64_t per, bool scale_f32, bool y_f32, cudaStream_t stream) {
    if (a.zeros)
        return a.group == 128  ? launch_g<128, true>(a, per, scale_f32, y_f32, stream)
               : a.group == 64 ? launch_g<64, true>(a, per, scale_f32, y_f32, stream)
                               : launch_g<32, true>(a, per, scale_f32, y_f32, stream);
    return a.group == 128  ? launch_g<128, false>(a, per, scale_f32, y_f32, stream)
           : a.group == 64 ? launch_g<64, false>(a, per, scale_f32, y_f32, stream)
                           : launch_g<32, false>(a, per, scale_f32, y_f32, stream);
}

cudaError_t read_clear_errors_base_tc(uint32_t* bits, cudaStream_t stream) {
    unsigned int h = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&h, g_err_base_tc, sizeof(h), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_err_base_tc, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *bits |= h;
    return e;
}

}  // namespace sgmv
