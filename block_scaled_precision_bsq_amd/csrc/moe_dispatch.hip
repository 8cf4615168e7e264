// Expert-sorted order of routed tokens (dispatch), and the weighted sum of
// each token's expert outputs (combine) with its backward.
//
// Dispatch is a stable counting sort of the T x k choices by expert.  A
// wave ranks 64 consecutive choices at a time: a ballot per bit of the expert
// number gives each lane the set of lanes with the same expert, whose lowest
// lane advances the expert's counter.  Every wave owns a contiguous range of
// choices and its own counters, so the order never depends on timing.  Choices
// without an expert (a negative or too large id) are bucket E: they take the
// rows past offsets[E], whose source row is -1.
// Up to DISPATCH_ONE_BLOCK choices run as one workgroup; more run as a
// counting launch and a placing launch, whose workgroups each add up the
// counts before them (a few hundred bytes per workgroup and expert, from L2)
// instead of waiting for a third launch in between.  131072 choices of 384
// experts: 3.2 and 8.1 us, bound by dependent steps (the counts, a scan, one
// counter per rank), not by their 1.5 MB; 128 choices in 3.6 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "moe_common.h"

namespace bsq {

constexpr int DISPATCH_MAX_E = 1024;
constexpr int DISPATCH_WAVES = 16;
constexpr int DISPATCH_ONE_BLOCK = 4096;
constexpr int DISPATCH_MAX_BLOCKS = 128;
// choices per workgroup while there are workgroups to take them (131072 choices:
// the call 13.0 us; with 2048 or 1024 15.5)
constexpr int DISPATCH_BLOCK = 4096;
constexpr int DISPATCH_AHEAD = 4;  // rounds of 64 choices that a wave holds in registers

struct DispatchArgs {
    const int32_t* ids;
    int64_t n;  // choices
    int K, E;
    int64_t per_wave;  // a multiple of 64
    int32_t* offsets;
    int32_t* row_index;
    int32_t* slot;
    int32_t* counts;  // [blocks][E + 1], two-launch form
};

__device__ __forceinline__ int dispatch_bucket(const DispatchArgs& a, int64_t i) {
    const int id = a.ids[i];
    return (uint32_t)id < (uint32_t)a.E ? id : a.E;
}

// Counts of this workgroup's choices.
__global__ __launch_bounds__(1024) void k_moe_dispatch_count(DispatchArgs a) {
    __shared__ int32_t s_n[DISPATCH_MAX_E + 1];
    for (int e = threadIdx.x; e <= a.E; e += 1024) s_n[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * DISPATCH_WAVES * a.per_wave;
    const int64_t hi = min(a.n, lo + DISPATCH_WAVES * a.per_wave);
    for (int64_t i = lo + threadIdx.x; i < hi; i += 1024) atomicAdd(&s_n[dispatch_bucket(a, i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += 1024) a.counts[(int64_t)blockIdx.x * (a.E + 1) + e] = s_n[e];
}

__global__ __launch_bounds__(1024) void k_moe_dispatch_place(DispatchArgs a) {
    // the waves' counters: counts at first, then the next slot of each bucket
    __shared__ int32_t s_w[DISPATCH_WAVES][DISPATCH_MAX_E + 1];
    __shared__ int32_t s_part[DISPATCH_WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = gridDim.x;
    int32_t* mine = s_w[wave];
    const int64_t lo = ((int64_t)blockIdx.x * DISPATCH_WAVES + wave) * a.per_wave;
    const int64_t hi = min(a.n, lo + a.per_wave);
    auto bucket = [&](int64_t i) { return i < hi ? dispatch_bucket(a, i) : -1; };
    // the wave's first choices and (thread e) the workgroups' counts of expert e
    // are on their way together
    int ahead[DISPATCH_AHEAD];
#pragma unroll
    for (int k = 0; k < DISPATCH_AHEAD; ++k) ahead[k] = bucket(lo + 64 * k + lane);
    const int e = threadIdx.x;
    int before = 0, total = 0;
    if (nb > 1 && e < a.E) {
#pragma unroll 32
        for (int b = 0; b < nb; ++b) {
            const int c = a.counts[(int64_t)b * (a.E + 1) + e];
            before += b < (int)blockIdx.x ? c : 0;
            total += c;
        }
    }
    int before_e = 0;  // of bucket E, by lane
    if (wave == 0)
        for (int b = lane; b < (int)blockIdx.x; b += 64) before_e += a.counts[(int64_t)b * (a.E + 1) + a.E];
    for (int i = lane; i <= a.E; i += 64) mine[i] = 0;
    // (a wave's own counters: its LDS operations are in order)
#pragma unroll
    for (int k = 0; k < DISPATCH_AHEAD; ++k)
        if (ahead[k] >= 0) atomicAdd(&mine[ahead[k]], 1);
    for (int64_t i = lo + 64 * DISPATCH_AHEAD + lane; i < hi; i += 64) atomicAdd(&mine[dispatch_bucket(a, i)], 1);
    __syncthreads();
    // thread e: the workgroup's counts, those of the workgroups before it and
    // of all, and the waves' counters turned into positions within the expert
    if (nb == 1 && e < a.E)
        for (int w = 0; w < DISPATCH_WAVES; ++w) total += s_w[w][e];
    const int incl = wave_scan_i32(total);
    if (lane == 63) s_part[wave] = incl;
    __syncthreads();
    int base = incl - total, routed = 0;
    for (int w = 0; w < DISPATCH_WAVES; ++w) {
        base += w < wave ? s_part[w] : 0;
        routed += s_part[w];
    }
    if (blockIdx.x == 0) {
        if (e < a.E) a.offsets[e] = base;
        if (e == 0) a.offsets[a.E] = routed;
    }
    if (e < a.E) {
        int run = base + before;
        for (int w = 0; w < DISPATCH_WAVES; ++w) {
            const int c = s_w[w][e];
            s_w[w][e] = run;
            run += c;
        }
    }
    if (wave == 0) {
        // bucket E starts after every routed choice
        int run = routed + __builtin_amdgcn_readlane(wave_scan_i32(before_e), 63);
        if (lane == 0)
            for (int w = 0; w < DISPATCH_WAVES; ++w) {
                const int c = s_w[w][a.E];
                s_w[w][a.E] = run;
                run += c;
            }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(a.E);
    auto place = [&](int64_t i, int x) {
        const bool in = x >= 0;
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (x >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const uint64_t below = same & ((1ull << lane) - 1);
        const int leader = in ? __builtin_ctzll(same) : lane;
        int first = 0;
        if (in && lane == leader) first = atomicAdd(&mine[x], __builtin_popcountll(same));
        first = __shfl(first, leader, 64);
        if (in) {
            const int pos = first + __builtin_popcountll(below);
            a.row_index[pos] = x < a.E ? (int32_t)((uint32_t)i / (uint32_t)a.K) : -1;
            a.slot[i] = x < a.E ? pos : -1;
        }
    };
#pragma unroll
    for (int k = 0; k < DISPATCH_AHEAD; ++k)
        if (lo + 64 * k < hi) place(lo + 64 * k + lane, ahead[k]);
    for (int64_t i0 = lo + 64 * DISPATCH_AHEAD; i0 < hi; i0 += 64) place(i0 + lane, bucket(i0 + lane));
}

struct CombineArgs {
    const void* ye;
    int64_t M, ld_ye;
    const int32_t* slot;
    const float* weights;
    int64_t T, width;
    int K;
    void* y;       // forward: output; backward: null
    const void* dy;
    int64_t ld_y;  // pitch of y / dy
    const int32_t* offsets;
    int E;
    void* dye;
    int64_t ld_d;
    float* dweights;
};

// Eight elements as binary32.
template <bool F32>
__device__ __forceinline__ void ld8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    }
}
template <bool F32>
__device__ __forceinline__ void st8(void* p, int64_t at, const float (&v)[8]) {
    if constexpr (F32) {
        float* o = static_cast<float*>(p) + at;
        st_stream16(o, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        st_stream16(o + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
        st_stream16(static_cast<uint16_t*>(p) + at, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
}

// y[t] = sum_j w[t][j] ye[slot[t][j]], j ascending, binary32, rounded once.
// A thread owns 8 columns of one token, so a token's K row pieces are in
// flight together; a workgroup covers 1024 columns.  Bound by the bytes of the
// gathered rows: 4096 tokens of 7168 bf16 columns, top 8, 95 us, 5.4 TB/s past
// L2; 16 tokens 4.3 us.
template <bool F32>
__global__ __launch_bounds__(128) void k_moe_combine(CombineArgs a) {
    const int64_t t = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 1024 + threadIdx.x * 8;
    if (c >= a.width) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (a.M > 0) {
        for (int j0 = 0; j0 < a.K; j0 += 8) {
            float v[8][8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // a choice without a row reads row 0 and drops it, so the
                // eight loads issue without a branch between them
                const int x = j0 + j < a.K ? a.slot[t * a.K + j0 + j] : -1;
                const bool ok = (uint64_t)(int64_t)x < (uint64_t)a.M;
                w[j] = ok ? (a.weights ? a.weights[t * a.K + j0 + j] : 1.0f) : 0.0f;
                ld8<F32>(a.ye, (ok ? (int64_t)x : 0) * a.ld_ye + c, v[j]);
                if (!ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], v[j][i], acc[i]);
        }
    }
    st8<F32>(a.y, t * a.ld_y + c, acc);
}

// dye[slot[t][j]] = w[t][j] dy[t] and dw[t][j] = <dy[t], ye[slot[t][j]]>: a
// workgroup per token reads dy[t] once for up to 8 choices.  Rows that no
// choice owns (past offsets[E]) become zero in the workgroups past the tokens.
// Bound by its bytes, a read and a write of every routed row: 4096 tokens of 7168
// bf16 columns, top 8, 177 us, 5.5 TB/s.
constexpr int COMBINE_TAIL_BLOCKS = 64;
template <bool F32>
__global__ __launch_bounds__(256) void k_moe_combine_bwd(CombineArgs a) {
    __shared__ float s_dw[4][8];
    if ((int64_t)blockIdx.x >= a.T) {
        if (a.offsets == nullptr) return;
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int64_t first = max(0, a.offsets[a.E]);
        for (int64_t r = first + ((int64_t)blockIdx.x - a.T); r < a.M; r += COMBINE_TAIL_BLOCKS)
            for (int64_t c = threadIdx.x * 8; c < a.width; c += 2048) st8<F32>(a.dye, r * a.ld_d + c, zero);
        return;
    }
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < a.K; j0 += 8) {
        int64_t s[8];
        float w[8], dw[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = j0 + j < a.K;
            const int x = in ? a.slot[t * a.K + j0 + j] : -1;
            s[j] = (uint64_t)(int64_t)x < (uint64_t)a.M ? x : -1;
            w[j] = in ? (a.weights ? a.weights[t * a.K + j0 + j] : 1.0f) : 0.0f;
            dw[j] = 0.0f;
        }
        for (int64_t c = threadIdx.x * 8; c < a.width; c += 2048) {
            float g[8];
            ld8<F32>(a.dy, t * a.ld_y + c, g);
            if (a.dweights && a.M > 0) {
                float v[8][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) ld8<F32>(a.ye, max(s[j], (int64_t)0) * a.ld_ye + c, v[j]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[j] = s[j] >= 0 ? fmaf(g[i], v[j][i], dw[j]) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (s[j] < 0) continue;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = w[j] * g[i];
                st8<F32>(a.dye, s[j] * a.ld_d + c, o);
            }
        }
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = wave_sum_f32(dw[j]);
                if (lane == 0) s_dw[wave][j] = x;
            }
            __syncthreads();
            const int j = threadIdx.x;
            if (j < 8 && j0 + j < a.K)
                a.dweights[t * a.K + j0 + j] = (s_dw[0][j] + s_dw[1][j]) + (s_dw[2][j] + s_dw[3][j]);
            __syncthreads();
        }
    }
}

namespace {

int dispatch_blocks(int64_t n) {
    if (n <= DISPATCH_ONE_BLOCK) return 1;
    const int64_t b = (n + DISPATCH_BLOCK - 1) / DISPATCH_BLOCK;
    return (int)(b < DISPATCH_MAX_BLOCKS ? b : DISPATCH_MAX_BLOCKS);
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace bsq

extern "C" {

size_t bsq_moe_dispatch_workspace_size(int64_t tokens, int32_t top_k, int32_t num_experts) {
    if (tokens < 0 || top_k < 1 || num_experts < 1 || num_experts > bsq::DISPATCH_MAX_E) return 0;
    return ((size_t)bsq::dispatch_blocks(tokens * top_k) * (num_experts + 1) * 4 + 255) / 256 * 256;
}

bsq_status bsq_moe_dispatch(const int32_t* expert_ids, int64_t tokens, int32_t top_k, int32_t num_experts,
                            int32_t* offsets, int32_t* row_index, int32_t* slot, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    if (tokens < 0 || top_k < 1 || num_experts < 1) return BSQ_ERR_INVALID_ARG;
    if (!offsets || !workspace || (tokens > 0 && (!expert_ids || !row_index || !slot))) return BSQ_ERR_INVALID_ARG;
    // slots are 32-bit, and a wave's range of choices stays a 32-bit count
    if (num_experts > bsq::DISPATCH_MAX_E || tokens >= ((int64_t)1 << 31) / top_k) return BSQ_ERR_UNSUPPORTED;
    if (!bsq::al(expert_ids, 4) || !bsq::al(offsets, 4) || !bsq::al(row_index, 4) || !bsq::al(slot, 4) ||
        !bsq::al(workspace, 256))
        return BSQ_ERR_UNSUPPORTED;
    if (workspace_bytes < bsq_moe_dispatch_workspace_size(tokens, top_k, num_experts))
        return BSQ_ERR_WORKSPACE_TOO_SMALL;
    const int64_t n = tokens * top_k;
    const int blocks = bsq::dispatch_blocks(n);
    const int64_t waves = (int64_t)blocks * bsq::DISPATCH_WAVES;
    const int64_t per_wave = ((n + waves - 1) / waves + 63) / 64 * 64;
    bsq::DispatchArgs a{expert_ids, n, top_k, num_experts, per_wave, offsets, row_index, slot,
                        static_cast<int32_t*>(workspace)};
    if (blocks > 1) {
        hipLaunchKernelGGL(bsq::k_moe_dispatch_count, dim3(blocks), dim3(1024), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return BSQ_ERR_HIP;
    }
    hipLaunchKernelGGL(bsq::k_moe_dispatch_place, dim3(blocks), dim3(1024), 0, stream, a);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

bsq_status bsq_moe_combine(const void* ye, bsq_dtype dtype, int64_t m_total, int64_t width, int64_t ld_ye,
                           const int32_t* slot, const float* weights, int64_t tokens, int32_t top_k, void* y,
                           int64_t ld_y, hipStream_t stream) {
    if (m_total < 0 || width < 0 || tokens < 0 || top_k < 1) return BSQ_ERR_INVALID_ARG;
    if (dtype != BSQ_BF16 && dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (tokens == 0 || width == 0) return BSQ_OK;
    if (!slot || !y || (m_total > 0 && (!ye || ld_ye < width)) || ld_y < width) return BSQ_ERR_INVALID_ARG;
    if (width % 8 || ld_ye % 8 || ld_y % 8 || !bsq::al(ye, 16) || !bsq::al(y, 16) || !bsq::al(slot, 4) ||
        !bsq::al(weights, 4))
        return BSQ_ERR_UNSUPPORTED;
    if (width > ((int64_t)1 << 24) || tokens >= (int64_t)1 << 24 || m_total >= (int64_t)1 << 31)
        return BSQ_ERR_UNSUPPORTED;
    bsq::CombineArgs a{ye, m_total, ld_ye, slot, weights, tokens, width, top_k, y, nullptr, ld_y,
                       nullptr, 0, nullptr, 0, nullptr};
    const dim3 grid((unsigned)tokens, (unsigned)((width + 1023) / 1024));
    if (dtype == BSQ_F32) hipLaunchKernelGGL((bsq::k_moe_combine<true>), grid, dim3(128), 0, stream, a);
    else hipLaunchKernelGGL((bsq::k_moe_combine<false>), grid, dim3(128), 0, stream, a);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

bsq_status bsq_moe_combine_bwd(const void* dy, bsq_dtype dtype, int64_t tokens, int64_t width, int64_t ld_dy,
                               const void* ye, int64_t m_total, int64_t ld_ye, const int32_t* slot,
                               const float* weights, int32_t top_k, const int32_t* offsets, int32_t num_experts,
                               void* dye, int64_t ld_dye, float* dweights, hipStream_t stream) {
    if (m_total < 0 || width < 0 || tokens < 0 || top_k < 1 || num_experts < 0) return BSQ_ERR_INVALID_ARG;
    if (dtype != BSQ_BF16 && dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (tokens > 0 && (!slot || !dy || ld_dy < width)) return BSQ_ERR_INVALID_ARG;
    if (m_total > 0 && (!dye || ld_dye < width || (dweights && (!ye || ld_ye < width)))) return BSQ_ERR_INVALID_ARG;
    if (width == 0 || width % 8 || ld_dy % 8 || ld_dye % 8 || (ye && ld_ye % 8) || !bsq::al(dy, 16) ||
        !bsq::al(ye, 16) || !bsq::al(dye, 16) || !bsq::al(slot, 4) || !bsq::al(weights, 4) ||
        !bsq::al(offsets, 4) || !bsq::al(dweights, 4))
        return BSQ_ERR_UNSUPPORTED;
    if (width > ((int64_t)1 << 24) || tokens >= ((int64_t)1 << 24) - bsq::COMBINE_TAIL_BLOCKS ||
        m_total >= (int64_t)1 << 31)
        return BSQ_ERR_UNSUPPORTED;
    bsq::CombineArgs a{ye, m_total, ld_ye, slot, weights, tokens, width, top_k, nullptr, dy, ld_dy,
                       offsets, num_experts, dye, ld_dye, dweights};
    const dim3 grid((unsigned)(tokens + bsq::COMBINE_TAIL_BLOCKS));
    if (dtype == BSQ_F32) hipLaunchKernelGGL((bsq::k_moe_combine_bwd<true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((bsq::k_moe_combine_bwd<false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

}  // extern "C"
