// Base products from 4-bit weights with group scales, y = W x: one matrix for all rows, or one per
// expert over rows sorted by expert.
#include <algorithm>
#include <string>
#include <type_traits>

#include "experts.h"
#include "ptx.cuh"

namespace sgmv {

__device__ unsigned int g_err_base;

namespace {

// Values of a row in a stage of a warp's ring: as many as leave registers for the scales of two stages.
template <int G> __host__ __device__ constexpr int stage_k() { return G == 32 ? 256 : 512; }

// The first block reports offsets that do not ascend from 0 to at most `rows`.
__device__ __forceinline__ void check_offsets(const BaseArgs& a) {
    if (!a.offsets || blockIdx.x + blockIdx.y > 0) return;
    for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) {
        const int o = a.offsets[e];
        if (e == 0 ? o != 0 : o < a.offsets[e - 1] || o > a.rows) atomicOr(&g_err_base, kErrExpert);
    }
}

__device__ __forceinline__ void cp_async16_to(uint32_t dst_smem, const void* src_gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src_gmem) : "memory");
}
// mma_bf16_16816 as a function of its registers, which the compiler may move among other instructions.
__device__ __forceinline__ void mma_rows(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_y(const BaseArgs& a, bool y_f32, int64_t row, int col, float v) {
    if (y_f32) static_cast<float*>(a.y)[row * a.ldy + col] = v;
    else static_cast<uint16_t*>(a.y)[row * a.ldy + col] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Expert of row r, by one warp: the last e with offsets[e] <= r, 32 candidates a step.
__device__ __forceinline__ int expert_of_row(const int32_t* offsets, int experts, int r) {
    int lo = 0, n = experts;
    while (n > 1) {
        const int step = (n + 31) / 32, i = (int)(threadIdx.x % 32) * step;
        const bool below = i < n && offsets[lo + i] <= r;
        const int last = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0) * step;
        lo += last;
        n = min(step, n - last);
    }
    return lo;
}

// Row of x for row r of y, or -1 (reported).
__device__ __forceinline__ int x_row_of(const BaseArgs& a, int r) {
    if (!a.slot_of) return r;
    const int slot = a.slot_of[r];
    const int t = slot / a.k;
    if (slot >= 0 && t < a.x_rows) return t;
    atomicOr(&g_err_base, kErrRows);
    return -1;
}

// Eight codes (value i in bits 4i..4i+3) less the zero point, as the bf16 pairs (0,4), (1,5), (2,6), (3,7).
// bf16 128 + n has the bits 0x4300 | n for n < 128, so inserting the code and subtracting 128 + z is exact.
// `magic` is 0x43004300, or 0x43084308 for two's complement codes (n ^ 8 is the value plus 8; z is 8).
__device__ __forceinline__ void codes_to_bf16(uint32_t c, uint32_t magic, uint32_t z2, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0x6a;" : "=r"(v) : "r"(c >> (4 * i)), "r"(magic));   // (c & mask) ^ magic
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&z2));
        p[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// y = W x for up to 8 NT rows of x at a time, on warp-level tensor-core products.
//
// What bounds it is the stream of codes (each is read once; x is small and comes from L2) and, close behind,
// the conversion of the codes: eight take seven integer operations and four subtractions, all at half rate.
// The 16 rows of an m16n8k16 product are 16 rows of W and its 8 columns are 8 rows of x, so that one conversion
// serves up to 8 NT outputs.  The K order inside a product is free as long as both operands agree: of every 32
// values of a row, lane q = lane % 4 of a product's operands takes 8q .. 8q+7, which are one 32-bit word of codes
// (what ldmatrix gives it of a 16-byte unit) and one 16-byte unit of x, whose eight values are stored in the
// pairs' order.  All values of a product are in one group, whose sum is scaled in fp32 and added to the total.
//
// A cluster of n_split CTAs (they split K) takes a run of 16-row tiles of W.  Of a CTA's share of K, each of its 8
// warps takes the same stages of every tile, so that its x is in one place; it streams its codes through a ring of
// its own (16-byte cp.async, two stages, each refilled as soon as its codes are in registers; no barrier with other
// warps).  At the end of a tile the warps leave their sums in shared memory; they take turns in adding them, in a
// fixed order, and the CTAs' sums meet at the end through distributed shared memory.
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = kWarps * 8192;   // two stages of 16 rows x 512 values a warp
constexpr int kPartBufs = 2;           // tiles whose sums are in shared memory at a time
constexpr int kPartStride = 20;        // floats: the four rows of x that a store touches fall on different banks
constexpr int kXPad = 64;              // bytes between rows of x: two rows' 64-byte reads fall on different banks

// The scales and zero points of a lane's two rows in one stage, as loaded.
template <int G, bool Z, bool SF32>
struct StageGroups {
    static constexpr int kGroups = stage_k<G>() / G;
    static constexpr int kWords = kGroups * (SF32 ? 4 : 2) / 4;
    static constexpr int kZeroWords = Z ? (kGroups + 3) / 4 : 1;
    uint32_t scale[2][kWords];
    uint32_t zero[2][kZeroWords];

    __device__ __forceinline__ float scale_of(int r, int i) const {
        if constexpr (SF32) return __uint_as_float(scale[r][i]);
        else return i % 2 ? bf16hi(scale[r][i / 2]) : bf16lo(scale[r][i / 2]);
    }
    __device__ __forceinline__ uint32_t zero_pair(int r, int i, uint32_t magic) const {      // bf16 128 + z, twice
        if constexpr (Z) return (0x4300u | (zero[r][i / 4] >> (i % 4 * 8) & 0xffu)) * 0x10001u;
        else return magic;
    }
    // ps, pz: the stage's first scale and zero point; `left`: groups of the row from there on; `vec`: whole stages,
    // aligned to their size
    __device__ __forceinline__ void load(int r, const uint8_t* ps, const uint8_t* pz, int left, bool vec) {
        if (vec) {
            if constexpr (kWords == 1) {
                scale[r][0] = *reinterpret_cast<const uint32_t*>(ps);
            } else if constexpr (kWords == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(ps);
                scale[r][0] = v.x; scale[r][1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 v = reinterpret_cast<const uint4*>(ps)[i];
                    scale[r][4 * i] = v.x; scale[r][4 * i + 1] = v.y; scale[r][4 * i + 2] = v.z; scale[r][4 * i + 3] = v.w;
                }
            }
            if constexpr (Z) {
                if constexpr (kGroups == 4) zero[r][0] = *reinterpret_cast<const uint32_t*>(pz);
                else {
                    const uint2 v = *reinterpret_cast<const uint2*>(pz);
                    zero[r][0] = v.x; zero[r][1] = v.y;
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) scale[r][i] = 0;
#pragma unroll
        for (int i = 0; i < kZeroWords; ++i) zero[r][i] = 0;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            if (i < left) {
                if constexpr (SF32) scale[r][i] = reinterpret_cast<const uint32_t*>(ps)[i];
                else scale[r][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(ps)[i] << (i % 2 * 16);
                if constexpr (Z) zero[r][i / 4] |= (uint32_t)pz[i] << (i % 4 * 8);
            }
    }
};

enum : int { kUnitDense = 0, kUnitExpert = 1, kUnitRow = 2 };

template <int G, int NT, bool Z, bool SF32>
__global__ void __launch_bounds__(kThreads, 2)
    base_rows_kernel(BaseArgs a, bool y_f32, int unit, int n_split, int tokens, int tiles_each, int x_stride, bool vec) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int s_xrow[8 * NT];
    __shared__ int s_unit[3];
    __shared__ __align__(8) uint64_t s_full[kPartBufs], s_empty[kPartBufs];
    constexpr int KS = stage_k<G>(), kCopies = KS / 64;              // 16-byte copies of a lane in a stage
    check_offsets(a);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const int rank = blockIdx.x % n_split;
    const int tile0 = (int)(blockIdx.x / n_split) * tiles_each;
    const int n_tiles = min(tiles_each, (a.d_out + 15) / 16 - tile0);
    // this CTA's stages of K, and this warp's
    const int all_stages = (a.d_in + KS - 1) / KS;
    const int st0 = (int)((int64_t)all_stages * rank / n_split), st1 = (int)((int64_t)all_stages * (rank + 1) / n_split);
    const int per_warp = (st1 - st0 + kWarps - 1) / kWarps, n_warps = (st1 - st0 + per_warp - 1) / per_warp;
    const int ws0 = st0 + warp * per_warp, n_ws = max(0, min(st1 - ws0, per_warp));
    const int kPart = tokens * kPartStride;                          // floats of a warp's sums
    float* s_part = reinterpret_cast<float*>(smem + kRing);          // [bufs][warps][tokens][kPartStride]
    uint8_t* xs = smem + kRing + kPartBufs * kWarps * kPart * 4;     // [tokens][x_stride]
    float* s_out = reinterpret_cast<float*>(xs + tokens * x_stride); // [tiles][tokens][16]
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPartBufs; ++i) {
            mbar_init(&s_full[i], n_warps);
            mbar_init(&s_empty[i], 1);
        }
        fence_mbar_init();
    }

    int e = 0, row = blockIdx.y * tokens, row_end = a.rows, row_step = gridDim.y * tokens;
    if (unit == kUnitExpert) {
        e = blockIdx.y;
        row = max(a.offsets[e], 0);
        row_end = min(a.offsets[e + 1], a.rows);
        row_step = tokens;
    } else if (unit == kUnitRow) {       // a row starts a unit if it is a multiple of `tokens` into its expert
        if (warp == 0) {
            const int r = blockIdx.y, f = expert_of_row(a.offsets, a.experts, r);
            const int first = a.offsets[f], end = min(a.offsets[f + 1], a.rows);
            if (lane == 0) {
                const bool mine = first >= 0 && r >= first && r < end && (r - first) % tokens == 0;
                s_unit[0] = f;
                s_unit[1] = mine ? r : 0;
                s_unit[2] = mine ? min(end, r + tokens) : 0;
            }
        }
        __syncthreads();
        e = s_unit[0];
        row = s_unit[1];
        row_end = s_unit[2];
        row_step = tokens;
    }

    uint32_t n_done = 0;                 // tiles of earlier rounds of the loop below
    for (; row < row_end; row += row_step, n_done += n_tiles) {
        const int n_tok = min(tokens, row_end - row);
        // codes: lane l copies the even or odd 16-byte units of row l / 2; unit u of row r is stored at u ^ (r % 8)
        const int64_t row_bytes = a.d_in / 2;
        const int cr = lane / 2;
        const uint32_t ring = smem_u32(smem) + warp * 8192;
        const uint32_t copy_at = ring + cr * (KS / 2);
        const int copy_flip = (lane % 2 ^ cr % 8) * 16;
        const uint8_t* copy_from = a.codes + ((int64_t)e * a.d_out + tile0 * 16 + cr) * row_bytes + ws0 * (KS / 2) + lane % 2 * 16;
        int copy_left = min(a.d_out, (tile0 + n_tiles) * 16) - tile0 * 16 - cr, copy_s = 0;   // rows of this lane's from the next stage's on
        uint32_t copy_slot = 0;
        const int64_t next_row = 16 * row_bytes - (n_ws - 1) * (KS / 2);
        const auto copy_stage = [&] {
            if (copy_left > 0) {
                const int units = a.d_in / 32 - (ws0 + copy_s) * (KS / 32) - lane % 2;       // of the row from this lane's first on
#pragma unroll
                for (int j = 0; j < kCopies; ++j)
                    if (2 * j < units)
                        cp_async16_to(copy_at + copy_slot + j / 4 * 128 + ((j % 4 * 32) ^ copy_flip), copy_from + j * 32);
            }
            cp_async_commit();
            copy_slot ^= 4096;
            if (++copy_s == n_ws) {
                copy_s = 0;
                copy_left -= 16;
                copy_from += next_row;
            } else {
                copy_from += KS / 2;
            }
        };
        __syncthreads();                 // the barriers are set up; s_xrow and x are free
        if (n_ws > 0) {
            copy_stage();
            copy_stage();
        }
        if ((int)threadIdx.x < n_tok) s_xrow[threadIdx.x] = x_row_of(a, row + threadIdx.x);
        __syncthreads();
        {                                // x in the pairs' order, a batch of loads at a time; a warp takes whole rows in turn
            const int units = (min(st1 * KS, a.d_in) - st0 * KS) / 8;
            const int t0 = n_tok >= kWarps ? warp : 0, dt = n_tok >= kWarps ? kWarps : 1;
            const int u0 = n_tok >= kWarps ? lane : threadIdx.x, du = n_tok >= kWarps ? 32 : kThreads;
            for (int t = t0; t < n_tok; t += dt) {
                const uint4* from = reinterpret_cast<const uint4*>(a.x + (int64_t)max(s_xrow[t], 0) * a.ldx + st0 * KS);
                uint4* to = reinterpret_cast<uint4*>(xs + t * x_stride);
                for (int u = u0; u < units; u += 4 * du) {
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = __ldg(from + min(u + j * du, units - 1));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (u + j * du < units)
                            to[u + j * du] = make_uint4(__byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                                                        __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
                }
            }
        }
        __syncthreads();
        const int groups = a.d_in / G;
        // adds the warps' sums of a tile
        const auto finish = [&](int tile) {
            const uint32_t n = n_done + tile, buf = n % kPartBufs;
            mbar_wait(&s_full[buf], (n / kPartBufs) & 1, &g_err_base);
            const float* part = s_part + buf * kWarps * kPart;
            for (int i = lane; i < n_tok * 16; i += 32) {
                const int t = i / 16, r = i % 16, col = (tile0 + tile) * 16 + r;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (w < n_warps) v += part[w * kPart + t * kPartStride + r];
                if (n_split > 1) s_out[(tile * tokens + t) * 16 + r] = v;
                else if (col < a.d_out && s_xrow[t] >= 0) store_y(a, y_f32, row + t, col, v);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[buf]);
        };
        if (n_ws > 0) {
            using Groups = StageGroups<G, Z, SF32>;
            constexpr int kScale = SF32 ? 4 : 2;
            const uint8_t* xp[NT];       // columns without a row of x repeat the last one
#pragma unroll
            for (int j = 0; j < NT; ++j) xp[j] = xs + min(8 * j + g, n_tok - 1) * x_stride + (ws0 - st0) * (KS * 2) + q * 16;
            // the row and unit that this lane addresses for ldmatrix
            const uint32_t read_at = ring + lane % 16 * (KS / 2), read_flip = (lane / 16 ^ lane % 8) * 16;
            const uint8_t *scale_at[2], *zero_at[2];                 // the next stage whose groups to load
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t at = ((int64_t)e * a.d_out + tile0 * 16 + g + 8 * r) * groups + ws0 * Groups::kGroups;
                scale_at[r] = static_cast<const uint8_t*>(a.scales) + at * kScale;
                zero_at[r] = Z ? a.zeros + at : nullptr;
            }
            int load_left = min(a.d_out, (tile0 + n_tiles) * 16) - tile0 * 16 - g, load_s = 0;
            const int64_t next_groups = 16 * groups - (n_ws - 1) * Groups::kGroups;
            const auto load_groups = [&](Groups& gr) {
                const int left = vec ? Groups::kGroups : groups - (ws0 + load_s) * Groups::kGroups;
                const bool last = ++load_s == n_ws;
                const int64_t step = last ? next_groups : Groups::kGroups;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (load_left > 8 * r) gr.load(r, scale_at[r], zero_at[r], left, vec);
                    scale_at[r] += step * kScale;
                    if constexpr (Z) zero_at[r] += step;
                }
                if (last) {
                    load_s = 0;
                    load_left -= 16;
                }
            };
            // known to the compiler only as a value: as a constant it would be moved into a register at every use
            const uint32_t magic = a.zeros ? 0x43004300u : 0x43084308u;
            Groups ahead[2] = {};
            load_groups(ahead[0]);
            float total[NT][4];
            const int items = n_tiles * n_ws;
            int s = 0, tile = 0, turn = n_warps - 1;                 // turn: the warp that adds the tile before
            uint32_t slot = 0;
            for (int i0 = 0; i0 < items; i0 += 2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (i0 + h >= items) break;
                    if (s == 0) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int v = 0; v < 4; ++v) total[j][v] = 0.0f;
                    }
                    load_groups(ahead[h ^ 1]);
                    cp_async_wait<1>();
                    __syncwarp();        // the stage's codes are there
                    uint32_t code[KS / 16];                          // word w of rows g, g + 8: 2 w, 2 w + 1
#pragma unroll
                    for (int i = 0; i < KS / 64; ++i)
                        ldsm_x4(read_at + slot + i / 4 * 128 + ((i % 4 * 32) ^ read_flip), *reinterpret_cast<uint32_t(*)[4]>(&code[4 * i]));
                    __syncwarp();        // every lane has them
                    copy_stage();
                    const int here = vec ? Groups::kGroups : groups - (ws0 + s) * Groups::kGroups;
                    const int xo = s * (KS * 2);
                    float sum[NT][4];
#pragma unroll
                    for (int w = 0; w < KS / 32; ++w) {
                        constexpr int kWords = G / 32;               // words of a lane in one group
                        const int gr = w / kWords;
                        if (w % kWords == 0) {
                            if (gr >= here) break;
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int v = 0; v < 4; ++v) sum[j][v] = 0.0f;
                        }
                        uint32_t p0[4], p1[4];
                        codes_to_bf16(code[2 * w], magic, ahead[h].zero_pair(0, gr, magic), p0);
                        codes_to_bf16(code[2 * w + 1], magic, ahead[h].zero_pair(1, gr, magic), p1);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint4 v = *reinterpret_cast<const uint4*>(xp[j] + xo + w * 64);
                            mma_rows(sum[j], p0[0], p1[0], p0[1], p1[1], v.x, v.y);
                            mma_rows(sum[j], p0[2], p1[2], p0[3], p1[3], v.z, v.w);
                        }
                        if (w % kWords == kWords - 1) {
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int v = 0; v < 4; ++v) total[j][v] = fmaf(ahead[h].scale_of(v / 2, gr), sum[j][v], total[j][v]);
                        }
                    }
                    slot ^= 4096;
                    if (++s == n_ws) {   // the tile's end
                        s = 0;
                        const uint32_t n = n_done + tile, buf = n % kPartBufs;
                        if (n >= kPartBufs) mbar_wait(&s_empty[buf], (n / kPartBufs - 1) & 1, &g_err_base);
                        float* part = s_part + (buf * kWarps + warp) * kPart + 2 * q * kPartStride + g;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                if (8 * j + 2 * q + v % 2 < n_tok) part[(8 * j + v % 2) * kPartStride + v / 2 * 8] = total[j][v];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_full[buf]);
                        if (turn == warp && tile > 0) finish(tile - 1);
                        if (++turn == n_warps) turn = 0;
                        ++tile;
                    }
                }
            }
            cp_async_wait<0>();
            if (turn == warp) finish(n_tiles - 1);
        }
        if (n_split > 1) {               // the CTAs' sums, in a fixed order
            cluster_sync();
            const uint32_t base = smem_u32(s_out);
            for (int i = rank * kThreads + threadIdx.x; i < n_tiles * n_tok * 16; i += n_split * kThreads) {
                const int tile = i / (n_tok * 16), t = i / 16 % n_tok, r = i % 16, col = (tile0 + tile) * 16 + r;
                const uint32_t at = base + ((tile * tokens + t) * 16 + r) * 4;
                float v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = c < n_split ? ld_cluster_f32(map_cluster(at, c)) : 0.0f;
#pragma unroll
                for (int c = 1; c < 8; ++c) v[0] += v[c];
                if (col < a.d_out && s_xrow[t] >= 0) store_y(a, y_f32, row + t, col, v[0]);
            }
            cluster_arrive_relaxed();    // every CTA of the cluster has read the sums
            cluster_wait_acquire();
        }
    }
}

template <int G, int NT, bool Z, bool SF32>
cudaError_t launch_rows_t(const BaseArgs& a, bool y_f32, cudaStream_t stream) {
    auto kern = base_rows_kernel<G, NT, Z, SF32>;
    constexpr int KS = stage_k<G>(), kMost = 227 * 1024, kHalf = kMost / 2 - 1024;
    const int tiles = (a.d_out + 15) / 16, stages = (a.d_in + KS - 1) / KS;
    int unit = kUnitDense, tokens = (int)std::min<int64_t>(8 * NT, a.rows);
    // K is split over 2 CTAs, or over as many as it takes for two of them to share an SM; where x is too large even
    // for that, and for one, a unit takes fewer rows of x
    const auto smem_of = [&](int split, int each) {
        const int x_stride = (stages + split - 1) / split * KS * 2 + kXPad;
        return kRing + kPartBufs * kWarps * tokens * kPartStride * 4 + tokens * x_stride + (split > 1 ? each * tokens * 64 : 0);
    };
    int split = std::min(2, stages);
    while (split < std::min(8, stages) && smem_of(split, 4) > kHalf) split = std::min(2 * split, stages);
    while (tokens > 1 && smem_of(split, 4) > kMost) tokens = (tokens + 1) / 2;
    int units = (int)std::min<int64_t>(65535, ((int64_t)a.rows + tokens - 1) / tokens), active = units;
    if (a.offsets) {
        unit = a.rows < a.experts ? kUnitRow : kUnitExpert;
        units = active = std::min(a.rows, a.experts);
    }
    const int clusters = 2 * 148 / split;
    int each = std::max(1, (int)(((int64_t)tiles * active + clusters - 1) / clusters));
    while (each > 1 && smem_of(split, each) > std::max(kHalf, smem_of(split, 4))) each = (each + 1) / 2;
    const int smem = smem_of(split, each), x_stride = (stages + split - 1) / split * KS * 2 + kXPad;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const auto at = [](const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const bool vec = a.d_in % KS == 0 && at(a.scales, 16) && at(a.zeros, 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles + each - 1) / each * split), (unsigned)units);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, y_f32, unit, split, tokens, each, x_stride, vec);
}
template <int G, int NT>
cudaError_t launch_rows_z(const BaseArgs& a, bool scale_f32, bool y_f32, cudaStream_t stream) {
    if (a.zeros) return scale_f32 ? launch_rows_t<G, NT, true, true>(a, y_f32, stream) : launch_rows_t<G, NT, true, false>(a, y_f32, stream);
    return scale_f32 ? launch_rows_t<G, NT, false, true>(a, y_f32, stream) : launch_rows_t<G, NT, false, false>(a, y_f32, stream);
}
template <int G>
cudaError_t launch_rows(const BaseArgs& a, int64_t per, bool scale_f32, bool y_f32, cudaStream_t stream) {
    return per <= 8 ? launch_rows_z<G, 1>(a, scale_f32, y_f32, stream) : launch_rows_z<G, 2>(a, scale_f32, y_f32, stream);
}

// Rows of a matrix, on average.
int64_t rows_each(int64_t rows, int64_t experts) { return (rows + experts - 1) / experts; }
// From this many rows a matrix on, the tensor-core kernel is the faster.
constexpr int kTcFrom = 17;

// Rows slot_of[r] / k of x to rows r of a workspace, for the tensor-core kernel, whose copies of x take consecutive
// rows (four rows a copy, from anywhere, took 2.5 times as long as this and the product together).
__global__ void __launch_bounds__(256) base_gather_kernel(BaseArgs a, uint4* to) {
    const int units = a.d_in / 8, r = blockIdx.x, slot = a.slot_of[r];
    if (slot < 0 || slot / a.k >= a.x_rows) {
        if (threadIdx.x == 0 && r < a.offsets[a.experts]) atomicOr(&g_err_base, kErrRows);
        return;
    }
    const uint4* from = reinterpret_cast<const uint4*>(a.x + (int64_t)(slot / a.k) * a.ldx);
    for (int i = threadIdx.x; i < units; i += 256) to[(int64_t)r * units + i] = from[i];
}

cudaError_t launch_product(BaseArgs a, bool scale_f32, bool y_f32, void* workspace, cudaStream_t stream) {
    const int64_t per = a.offsets ? rows_each(a.rows, a.experts) : a.rows;
    if (per >= kTcFrom) {
        if (a.slot_of) {
            base_gather_kernel<<<a.rows, 256, 0, stream>>>(a, static_cast<uint4*>(workspace));
            if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
            a.x = static_cast<const uint16_t*>(workspace);
            a.ldx = a.d_in;
        }
        return launch_base_tc(a, per, scale_f32, y_f32, stream);
    }
    return a.group == 128  ? launch_rows<128>(a, per, scale_f32, y_f32, stream)
           : a.group == 64 ? launch_rows<64>(a, per, scale_f32, y_f32, stream)
                           : launch_rows<32>(a, per, scale_f32, y_f32, stream);
}

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

sgmv_status product_impl(const char* who_, const BaseArgs& a, int32_t scale_dtype, int32_t y_dtype, void* workspace, cudaStream_t stream) {
    const std::string who(who_);
    if (a.rows < 0 || a.x_rows < 0 || a.d_in < 1 || a.d_out < 1)
        return fail(SGMV_ERR_INVALID, who + ": the numbers of rows must be >= 0, d_in and d_out >= 1");
    if (a.group != 32 && a.group != 64 && a.group != 128)
        return fail(SGMV_ERR_INVALID, who + ": group must be 32, 64 or 128");
    if (a.d_in % a.group) return fail(SGMV_ERR_INVALID, who + ": d_in must be a multiple of group");
    if ((scale_dtype != 0 && scale_dtype != 1) || (y_dtype != 0 && y_dtype != 1))
        return fail(SGMV_ERR_INVALID, who + ": scale_dtype and y_dtype must be 0 (bf16) or 1 (fp32)");
    if (a.d_in > kMaxBaseK) return fail(SGMV_ERR_UNSUPPORTED, who + ": d_in must be at most 524288");
    if (a.rows == 0) return SGMV_OK;
    if (!a.x || !a.codes || !a.scales || !a.y) return fail(SGMV_ERR_INVALID, who + ": x, codes, scales and y are required");
    if (a.ldx < a.d_in || a.ldx % 8 || !aligned(a.x, 16))
        return fail(SGMV_ERR_INVALID, who + ": x rows must be 16-byte aligned, ldx >= d_in");
    if (!aligned(a.codes, 16)) return fail(SGMV_ERR_INVALID, who + ": codes must be 16-byte aligned");
    if (!aligned(a.scales, scale_dtype ? 4 : 2)) return fail(SGMV_ERR_INVALID, who + ": scales must be aligned to their type");
    if (a.ldy < a.d_out || !aligned(a.y, y_dtype ? 4 : 2))
        return fail(SGMV_ERR_INVALID, who + ": y must be aligned to its type, ldy >= d_out");
    SGMV_CUDA_TRY(launch_product(a, scale_dtype == 1, y_dtype == 1, workspace, stream));
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
    return product_impl("base_product", a, scale_dtype, y_dtype, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int64_t sgmv_base_product_experts_workspace(int32_t rows, int32_t d_in, int32_t n_experts) {
    if (rows < 0 || d_in < 1 || n_experts < 1 || n_experts > kMaxExperts) return -1;
    return rows_each(rows, n_experts) >= kTcFrom ? (int64_t)rows * d_in * 2 : 0;
}

extern "C" sgmv_status sgmv_base_product_experts(const void* x, int64_t ldx, int32_t x_rows, int32_t d_in,
                                                 int32_t d_out, int32_t n_experts, const void* codes,
                                                 const void* scales, int32_t scale_dtype, const uint8_t* zeros,
                                                 int32_t group, const int32_t* offsets, const int32_t* slot_of,
                                                 int32_t k, int32_t rows, void* y, int64_t ldy, int32_t y_dtype,
                                                 void* workspace, int64_t workspace_bytes, sgmv_stream_t stream) {
    const char* who = "base_product_experts";
    if (n_experts < 1 || n_experts > kMaxExperts)
        return fail(SGMV_ERR_INVALID, "base_product_experts: the number of experts must be in 1..4096");
    if (rows > 0 && (!offsets || !aligned(offsets, 4) || (slot_of && !aligned(slot_of, 4))))
        return fail(SGMV_ERR_INVALID, "base_product_experts: offsets are required; offsets and slot_of 4-byte aligned");
    if (slot_of ? (k < 1 || k > kMaxExpertsPerToken || (rows > 0 && x_rows < 1)) : x_rows < rows)
        return fail(SGMV_ERR_INVALID, "base_product_experts: slot_of needs k in 1..64 and a row of x; without it x has a row for every row of y");
    const BaseArgs a{static_cast<const uint16_t*>(x), ldx, static_cast<const uint8_t*>(codes), scales, zeros, y, ldy,
                     offsets, slot_of, rows, x_rows, slot_of ? k : 1, n_experts, d_in, d_out, group};
    const int64_t need = slot_of ? sgmv_base_product_experts_workspace(rows, d_in, n_experts) : 0;
    if (need > 0 && (!workspace || !aligned(workspace, 16)))
        return fail(SGMV_ERR_INVALID, "base_product_experts: a workspace is required, 16-byte aligned");
    if (need > workspace_bytes)
        return fail(SGMV_ERR_CAPACITY, "base_product_experts: the workspace is smaller than sgmv_base_product_experts_workspace says");
    return product_impl(who, a, scale_dtype, y_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
}
