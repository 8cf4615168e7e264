// Top-k routing of router logits with the balance loss, forward and backward.
//
// Per token t with logits l (binary32) and selection bias b: the k largest
// keys l_e + b_e choose the experts, ties to the lowest index.  p = softmax(l);
// the weights are p of the chosen experts, or the softmax over the chosen
// ones, times `scale`.  With f_e tokens choosing expert e, V tokens that
// choose any and P_e = (1/V) sum_t p_te the balance loss is
//   L = coef * E / (k V) * sum_e f_e P_e,
// and, f being constant, dL/dl_te = p_te (u_e - sum_i p_ti u_i) with
// u_e = coef * E f_e / (k V^2).
//
// One wave per token: lane l holds experts [l*VPL, (l+1)*VPL) in registers, so
// a key's position orders first by lane: the winner of a round is the lowest
// lane that holds the wave's maximum, and the lowest of its entries.  The
// kernel reads the logits once; a round of the selection costs a six-step lane
// reduction, a ballot and VPL compares, which bounds the kernel rather than
// its bytes (figures at the launcher).
// Token sums never go through atomics: a wave adds the probabilities of its
// tokens in registers, a workgroup its waves in order, and k_moe_route_finish
// the workgroups in order in binary64.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "moe_common.h"

#include <type_traits>

namespace bsq {

constexpr int ROUTE_MAX_E = 1024;
constexpr int ROUTE_MAX_K = 64;
// Up to this many tokens one workgroup of 16 waves does everything in one
// launch; more run workgroups of 4 waves and the finishing launch.
constexpr int ROUTE_ONE_BLOCK = 64;
constexpr int ROUTE_MAX_BLOCKS = 512;
constexpr int ROUTE_BLOCK_TOKENS = 16;  // at least this many tokens per workgroup

struct RouteArgs {
    const void* logits;
    int64_t T, ld;
    int E, K;
    const float* bias;
    const uint8_t* mask;
    int normalize;
    float scale, coef;
    int32_t* ids;
    float* weights;
    float* lse;
    int32_t* counts;  // [E + 1]
    float* loss;
    // workspace of the two-launch form
    float* part_p;    // [blocks][E]
    int32_t* part_n;  // [blocks][E]
    int32_t* part_v;  // [blocks] tokens with a choice
    double* part_l;   // [finishing workgroups]
    int32_t* ticket;
};

// NaN counts as -inf and +inf as the largest finite value.
__device__ __forceinline__ float route_canon(float x) { return x == x ? fminf(x, 3.402823466e38f) : -INFINITY; }

// The lane's VPL logits of one row; entries past E are -inf.  PAIRS: E and
// the pitch are even and the base is aligned to two elements.
template <bool F32, int VPL, bool PAIRS>
__device__ __forceinline__ void route_load(const void* logits, int64_t at, int e0, int E, float (&v)[VPL]) {
    if constexpr (PAIRS && VPL % 2 == 0) {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) {
            float a = -INFINITY, b = -INFINITY;
            if (e0 + j < E) {
                if constexpr (F32) {
                    const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(logits) + at + e0 + j);
                    a = w.x;
                    b = w.y;
                } else {
                    const uint32_t w =
                        *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(logits) + at + e0 + j);
                    a = bf16_lo(w);
                    b = bf16_hi(w);
                }
            }
            v[j] = route_canon(a);
            v[j + 1] = route_canon(b);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float a = -INFINITY;
            if (e0 + j < E) {
                if constexpr (F32)
                    a = static_cast<const float*>(logits)[at + e0 + j];
                else
                    a = bits_bf16(static_cast<const uint16_t*>(logits)[at + e0 + j]);
            }
            v[j] = route_canon(a);
        }
    }
}

// Binary64 sum of one value per thread over the workgroup, in thread order
// within a wave tree and wave order across; the result is valid in thread 0.
__device__ __forceinline__ double block_sum_f64(double x, double* s_w) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
    if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = x;
    __syncthreads();
    double r = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w) r += s_w[w];
    return r;
}

template <bool F32, int VPL, bool PAIRS>
__global__ __launch_bounds__(1024) void k_moe_route(RouteArgs a) {
    __shared__ float s_p[ROUTE_MAX_E];
    __shared__ int32_t s_n[ROUTE_MAX_E];
    __shared__ int32_t s_v;
    __shared__ double s_w[16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nw = blockDim.x >> 6;
    const int e0 = lane * VPL;
    float bias[VPL], psum[VPL];
    int cnt[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        bias[j] = (a.bias != nullptr && e0 + j < a.E) ? a.bias[e0 + j] : 0.0f;
        psum[j] = 0.0f;
        cnt[j] = 0;
    }
    int live_rows = 0;
    for (int64_t t = (int64_t)blockIdx.x * nw + wave; t < a.T; t += (int64_t)gridDim.x * nw) {
        const bool on = a.mask == nullptr || a.mask[t] != 0;
        float v[VPL], key[VPL];
        if (on) {
            route_load<F32, VPL, PAIRS>(a.logits, t * a.ld, e0, a.E, v);
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) v[j] = -INFINITY;
        }
        float lm = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const float k = v[j] + bias[j];
            key[j] = k == k ? k : -INFINITY;
            lm = fmaxf(lm, v[j]);
        }
        const float m = wave_max_f32(lm);
        const float mm = m > -INFINITY ? m : 0.0f;
        float p[VPL], ls = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            p[j] = expf(v[j] - mm);
            ls += p[j];
        }
        const float sum = wave_sum_f32(ls);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) p[j] *= inv;

        // the lane's best entry: key, position and what is read off it
        float bk;
        int bj;
        auto best = [&]() {
            bk = key[0];
            bj = 0;
#pragma unroll
            for (int j = 1; j < VPL; ++j)
                if (key[j] > bk) {
                    bk = key[j];
                    bj = j;
                }
        };
        best();
        int id = -1;           // lane r < K: the r-th choice
        float lsel = -INFINITY, psel = 0.0f;
        for (int r = 0; r < a.K; ++r) {
            const float top = wave_max_f32(bk);
            if (!(top > -INFINITY)) break;
            const int w = __builtin_ctzll(__ballot(bk == top));
            float bv = v[0], bp = p[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) {
                bv = bj == j ? v[j] : bv;
                bp = bj == j ? p[j] : bp;
            }
            const int we = __builtin_amdgcn_readlane(e0 + bj, w);
            const float wv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), w));
            const float wp = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bp), w));
            if (lane == r) {
                id = we;
                lsel = wv;
                psel = wp;
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (e0 + j == we) {
                    key[j] = -INFINITY;
                    cnt[j] += 1;
                }
            best();
        }
        const bool live = __builtin_amdgcn_readlane(id, 0) >= 0;
        live_rows += live ? 1 : 0;
        if (live) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) psum[j] += p[j];
        }
        float w = psel;
        if (a.normalize && live) {
            // softmax over the chosen logits: no underflow when a bias lifts
            // experts whose share of the whole softmax is below binary32
            const float ms = wave_max_f32(lsel);
            const float ex = id >= 0 ? expf(lsel - ms) : 0.0f;
            w = ex / wave_sum_f32(ex);
        }
        if (lane < a.K) {
            a.ids[t * a.K + lane] = id;
            a.weights[t * a.K + lane] = id >= 0 ? w * a.scale : 0.0f;
        }
        if (lane == 0) a.lse[t] = live ? logf(sum) + m : -INFINITY;
    }
    // the workgroup's sums, wave by wave
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        s_p[e] = 0.0f;
        s_n[e] = 0;
    }
    if (threadIdx.x == 0) s_v = 0;
    for (int w = 0; w < nw; ++w) {
        __syncthreads();
        if (w == wave) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (e0 + j < a.E) {
                    s_p[e0 + j] += psum[j];
                    s_n[e0 + j] += cnt[j];
                }
            if (lane == 0) s_v += live_rows;
        }
    }
    __syncthreads();
    if (gridDim.x == 1) {
        double x = 0.0;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            a.counts[e] = s_n[e];
            x += (double)s_n[e] * (double)s_p[e];
        }
        x = block_sum_f64(x, s_w);
        if (threadIdx.x == 0) {
            const double n = s_v > 0 ? (double)s_v : 1.0;
            a.counts[a.E] = s_v;
            a.loss[0] = (float)((double)a.coef * a.E / a.K * x / (n * n));
        }
    } else {
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            a.part_p[(int64_t)blockIdx.x * a.E + e] = s_p[e];
            a.part_n[(int64_t)blockIdx.x * a.E + e] = s_n[e];
        }
        if (threadIdx.x == 0) {
            a.part_v[blockIdx.x] = s_v;
            if (blockIdx.x == 0) *a.ticket = 0;
        }
    }
}

// Sums of the workgroups' parts: a workgroup of 1024 threads takes 64 experts,
// 16 threads each, and leaves its share of sum_e f_e P_e; the last workgroup
// to arrive (a ticket) adds the shares in order.
__global__ __launch_bounds__(1024) void k_moe_route_finish(RouteArgs a, int blocks) {
    __shared__ double s_p[16][64];
    __shared__ int32_t s_n[16][64];
    __shared__ double s_w[16];
    __shared__ int s_last;
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    double p = 0.0;
    int n = 0;
    if (e < a.E) {
#pragma unroll 4
        for (int b = part; b < blocks; b += 16) {
            p += (double)a.part_p[(int64_t)b * a.E + e];
            n += a.part_n[(int64_t)b * a.E + e];
        }
    }
    s_p[part][lane] = p;
    s_n[part][lane] = n;
    __syncthreads();
    double x = 0.0;
    if (part == 0 && e < a.E) {
        double tp = 0.0;
        int tn = 0;
        for (int i = 0; i < 16; ++i) {
            tp += s_p[i][lane];
            tn += s_n[i][lane];
        }
        a.counts[e] = tn;
        x = (double)tn * tp;
    }
    x = block_sum_f64(x, s_w);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&a.part_l[blockIdx.x], x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int before = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last || part != 0) return;
    int v = 0;
    for (int b = lane; b < blocks; b += 64) v += a.part_v[b];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    if (lane == 0) {
        double s = 0.0;
        for (int b = 0; b < (int)gridDim.x; ++b)
            s += __hip_atomic_load(&a.part_l[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const double nv = v > 0 ? (double)v : 1.0;
        a.counts[a.E] = v;
        a.loss[0] = (float)((double)a.coef * a.E / a.K * s / (nv * nv));
    }
}

struct RouteBwdArgs {
    const void* logits;
    int64_t T, ld;
    int E, K;
    const int32_t* ids;
    const float* weights;
    const float* lse;
    const int32_t* counts;
    const float* dweights;  // may be null: no gradient of the weights
    const float* dloss;     // may be null: no gradient of the loss
    int normalize;
    float scale, coef;
    void* dlogits;
    int64_t ldd;
};

// One wave per token, experts in registers as in k_moe_route; lse only tells
// the tokens that went nowhere.  Weights of the softmax over the chosen experts, q = w / scale:
//   dl_e += w_e (dw_e - sum_i q_i dw_i) for chosen e;
// weights taken from p: u_e += scale dw_e for chosen e.
template <bool F32, int VPL, bool PAIRS>
__global__ __launch_bounds__(256) void k_moe_route_bwd(RouteBwdArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = lane * VPL;
    float u[VPL];
    {
        const double nv = a.counts[a.E] > 0 ? (double)a.counts[a.E] : 1.0;
        const double c = a.dloss ? (double)a.dloss[0] * a.coef * a.E / a.K / (nv * nv) : 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) u[j] = e0 + j < a.E ? (float)(c * a.counts[e0 + j]) : 0.0f;
    }
    const float rscale = a.scale != 0.0f ? 1.0f / a.scale : 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
        float d[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
        if (a.lse[t] > -INFINITY) {
            float v[VPL], g[VPL];
            route_load<F32, VPL, PAIRS>(a.logits, t * a.ld, e0, a.E, v);
            int id = -1;
            float x = 0.0f;  // lane r < K: what its choice adds
            if (lane < a.K && a.dweights) {
                id = a.ids[t * a.K + lane];
                if (id >= 0) {
                    const float dw = a.dweights[t * a.K + lane];
                    x = a.normalize ? a.weights[t * a.K + lane] * dw : a.scale * dw;
                }
            }
            if (a.normalize && a.dweights) {
                const float dot = wave_sum_f32(x);  // sum_i w_i dw_i = scale sum_i q_i dw_i
                if (id >= 0) x -= a.weights[t * a.K + lane] * rscale * dot;
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) g[j] = 0.0f;
            if (a.dweights) {
                for (int r = 0; r < a.K; ++r) {
                    const int we = __builtin_amdgcn_readlane(id, r);
                    const float wx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), r));
#pragma unroll
                    for (int j = 0; j < VPL; ++j) g[j] += (e0 + j == we) ? wx : 0.0f;
                }
            }
            // the softmax again rather than exp(l - lse): at a maximum of large
            // magnitude lse does not hold the logarithm of the sum
            float lm = v[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) lm = fmaxf(lm, v[j]);
            const float m = wave_max_f32(lm);
            float p[VPL], up[VPL], ls = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] = expf(v[j] - m);
                ls += p[j];
            }
            const float inv = 1.0f / wave_sum_f32(ls);
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] *= inv;
                up[j] = a.normalize ? u[j] : u[j] + g[j];
                dot += p[j] * up[j];
            }
            const float s = wave_sum_f32(dot);
#pragma unroll
            for (int j = 0; j < VPL; ++j) d[j] = p[j] * (up[j] - s) + (a.normalize ? g[j] : 0.0f);
        }
        const int64_t at = t * a.ldd;
        if constexpr (F32) {
            float* o = static_cast<float*>(a.dlogits) + at;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (e0 + j < a.E) o[e0 + j] = d[j];
        } else {
            uint16_t* o = static_cast<uint16_t*>(a.dlogits) + at;
            if (PAIRS && VPL % 2 == 0) {
#pragma unroll
                for (int j = 0; j + 1 < VPL; j += 2)
                    if (e0 + j < a.E) *reinterpret_cast<uint32_t*>(o + e0 + j) = pack_bf16x2(d[j], d[j + 1]);
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (e0 + j < a.E) o[e0 + j] = bf16_rne(d[j]);
            }
        }
    }
}

namespace {

int route_blocks(int64_t T) {
    if (T <= ROUTE_ONE_BLOCK) return 1;
    const int64_t b = (T + ROUTE_BLOCK_TOKENS - 1) / ROUTE_BLOCK_TOKENS;
    return (int)(b < ROUTE_MAX_BLOCKS ? b : ROUTE_MAX_BLOCKS);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Calls f with the number of experts a lane holds.
template <class F>
void with_vpl(int E, F f) {
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 128) f(std::integral_constant<int, 2>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else if (E <= 384) f(std::integral_constant<int, 6>{});
    else if (E <= 512) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}

}  // namespace
}  // namespace bsq

extern "C" {

size_t bsq_moe_route_workspace_size(int64_t tokens, int32_t num_experts) {
    if (tokens < 0 || num_experts < 1 || num_experts > bsq::ROUTE_MAX_E) return 0;
    const size_t b = (size_t)bsq::route_blocks(tokens);
    return bsq::up256(b * num_experts * 4) * 2 + bsq::up256(b * 4) + 256 + 256;
}

bsq_status bsq_moe_route(const void* logits, bsq_dtype dtype, int64_t tokens, int32_t num_experts, int64_t ld,
                         int32_t top_k, const float* bias, const uint8_t* mask, int32_t normalize, float scale,
                         float loss_coef, int32_t* expert_ids, float* weights, float* lse, int32_t* counts,
                         float* loss, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (tokens < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts) return BSQ_ERR_INVALID_ARG;
    if (dtype != BSQ_BF16 && dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (!counts || !loss || !workspace) return BSQ_ERR_INVALID_ARG;
    if (tokens > 0 && (!logits || !expert_ids || !weights || !lse || ld < num_experts)) return BSQ_ERR_INVALID_ARG;
    if (num_experts > bsq::ROUTE_MAX_E || top_k > bsq::ROUTE_MAX_K || tokens >= (int64_t)1 << 31)
        return BSQ_ERR_UNSUPPORTED;
    const int z = dtype == BSQ_F32 ? 4 : 2;
    if (!bsq::aligned_to(logits, z) || !bsq::aligned_to(bias, 4) || !bsq::aligned_to(expert_ids, 4) ||
        !bsq::aligned_to(weights, 4) || !bsq::aligned_to(lse, 4) || !bsq::aligned_to(counts, 4) ||
        !bsq::aligned_to(loss, 4) || !bsq::aligned_to(workspace, 256))
        return BSQ_ERR_UNSUPPORTED;
    if (workspace_bytes < bsq_moe_route_workspace_size(tokens, num_experts)) return BSQ_ERR_WORKSPACE_TOO_SMALL;
    const int blocks = bsq::route_blocks(tokens);
    char* ws = static_cast<char*>(workspace);
    const size_t pe = bsq::up256((size_t)blocks * num_experts * 4);
    bsq::RouteArgs a{logits, tokens, ld, num_experts, top_k, bias, mask, normalize, scale, loss_coef,
                     expert_ids, weights, lse, counts, loss,
                     reinterpret_cast<float*>(ws), reinterpret_cast<int32_t*>(ws + pe),
                     reinterpret_cast<int32_t*>(ws + 2 * pe),
                     reinterpret_cast<double*>(ws + 2 * pe + bsq::up256((size_t)blocks * 4)),
                     reinterpret_cast<int32_t*>(ws + 2 * pe + bsq::up256((size_t)blocks * 4) + 256)};
    const bool pairs = num_experts % 2 == 0 && ld % 2 == 0 && bsq::aligned_to(logits, 2 * z);
    const dim3 grid(blocks), block(blocks == 1 ? 1024 : 256);
    bsq::with_vpl(num_experts, [&](auto V) {
        constexpr int VPL = decltype(V)::value;
        if (dtype == BSQ_F32) {
            if (pairs) hipLaunchKernelGGL((bsq::k_moe_route<true, VPL, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((bsq::k_moe_route<true, VPL, false>), grid, block, 0, stream, a);
        } else {
            if (pairs) hipLaunchKernelGGL((bsq::k_moe_route<false, VPL, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((bsq::k_moe_route<false, VPL, false>), grid, block, 0, stream, a);
        }
    });
    if (hipGetLastError() != hipSuccess) return BSQ_ERR_HIP;
    if (blocks > 1) {
        hipLaunchKernelGGL(bsq::k_moe_route_finish, dim3((num_experts + 63) / 64), dim3(1024), 0, stream, a, blocks);
        if (hipGetLastError() != hipSuccess) return BSQ_ERR_HIP;
    }
    return BSQ_OK;
}

bsq_status bsq_moe_route_bwd(const void* logits, bsq_dtype dtype, int64_t tokens, int32_t num_experts, int64_t ld,
                             int32_t top_k, const int32_t* expert_ids, const float* weights, const float* lse,
                             const int32_t* counts, const float* dweights, const float* dloss, int32_t normalize,
                             float scale, float loss_coef, void* dlogits, int64_t ld_d, hipStream_t stream) {
    if (tokens < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts) return BSQ_ERR_INVALID_ARG;
    if (dtype != BSQ_BF16 && dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (tokens == 0) return BSQ_OK;
    if (!logits || !expert_ids || !weights || !lse || !counts || !dlogits || ld < num_experts || ld_d < num_experts)
        return BSQ_ERR_INVALID_ARG;
    if (num_experts > bsq::ROUTE_MAX_E || top_k > bsq::ROUTE_MAX_K || tokens >= (int64_t)1 << 31)
        return BSQ_ERR_UNSUPPORTED;
    const int z = dtype == BSQ_F32 ? 4 : 2;
    if (!bsq::aligned_to(logits, z) || !bsq::aligned_to(dlogits, z) || !bsq::aligned_to(expert_ids, 4) ||
        !bsq::aligned_to(weights, 4) || !bsq::aligned_to(lse, 4) || !bsq::aligned_to(counts, 4) ||
        !bsq::aligned_to(dweights, 4) || !bsq::aligned_to(dloss, 4))
        return BSQ_ERR_UNSUPPORTED;
    bsq::RouteBwdArgs a{logits, tokens, ld, num_experts, top_k, expert_ids, weights, lse, counts, dweights, dloss,
                        normalize, scale, loss_coef, dlogits, ld_d};
    const bool pairs = num_experts % 2 == 0 && ld % 2 == 0 && ld_d % 2 == 0 && bsq::aligned_to(logits, 2 * z) &&
                       bsq::aligned_to(dlogits, 2 * z);
    const int64_t blocks = (tokens + 3) / 4;
    const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048)), block(256);
    bsq::with_vpl(num_experts, [&](auto V) {
        constexpr int VPL = decltype(V)::value;
        if (dtype == BSQ_F32) {
            if (pairs) hipLaunchKernelGGL((bsq::k_moe_route_bwd<true, VPL, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((bsq::k_moe_route_bwd<true, VPL, false>), grid, block, 0, stream, a);
        } else {
            if (pairs) hipLaunchKernelGGL((bsq::k_moe_route_bwd<false, VPL, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((bsq::k_moe_route_bwd<false, VPL, false>), grid, block, 0, stream, a);
        }
    });
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

}  // extern "C"
