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
// One wave per token, the experts in registers: lane l holds experts 128 c + 2 l
// and 128 c + 2 l + 1 of every chunk c of 128, so loads and stores cover whole
// lines.  Keys are compared as integers in the order of their values, which
// makes a step of a wave maximum one instruction.  Every lane keeps the best
// two of its keys: a round of the selection is a wave maximum of the first ones
// and a pop in the lane that has it; only a lane that gives a third expert
// looks at its keys again.  The instructions bound the kernel, not its bytes:
// 16384 x 384 binary32, top 8, take 22 us (25 MB, 5 us at the copy rate), of
// which about 7 are the launch and the sums at its end; with a scan of all keys in
// every round 25 us, and 43 us with entries in lane order, position tracking in
// every round and two workgroups' worth of waves.  More waves do not help
// (512 workgroups: 26.5 us): their starts and partial sums cost more.
// Token sums never go through float atomics: a wave adds the probabilities of
// its tokens in registers, a workgroup its waves in order, and
// k_moe_route_finish (5 us) the workgroups in order in binary64.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "moe_common.h"

#include <type_traits>

namespace bsq {

constexpr int ROUTE_MAX_E = 1024;
constexpr int ROUTE_MAX_K = 64;
// Up to this many tokens one workgroup does everything in one launch; more run
// up to ROUTE_MAX_BLOCKS workgroups and the finishing launch.
constexpr int ROUTE_ONE_BLOCK = 64;
constexpr int ROUTE_MAX_BLOCKS = 256;
constexpr int ROUTE_WAVES = 16;  // per workgroup: as many tokens at a time

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
    uint2* part;      // [blocks][E]: sum of probabilities (f32), tokens
    int32_t* part_v;  // [blocks] tokens with a choice
    double* part_l;   // [finishing workgroups]
    int32_t* ticket;
};

// NaN counts as -inf and +inf as the largest finite value.
__device__ __forceinline__ float route_canon(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f); }

// Position of the lane's entry j (VPL 1: experts up to 64, one a lane).
template <int VPL>
__device__ __forceinline__ int route_pos(int lane, int j) { return VPL == 1 ? lane : 128 * (j >> 1) + 2 * lane + (j & 1); }

// The lane's VPL logits of one row; entries past E are -inf.  PAIRS: E and
// the pitch are even and the base is aligned to two elements.
template <bool F32, int VPL, bool PAIRS>
__device__ __forceinline__ void route_load(const void* logits, int64_t at, int lane, int E, float (&v)[VPL]) {
    if constexpr (PAIRS && VPL > 1) {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) {
            const int e = route_pos<VPL>(lane, j);
            v[j] = v[j + 1] = -INFINITY;
            if (e < E) {
                if constexpr (F32) {
                    const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(logits) + at + e);
                    v[j] = w.x;
                    v[j + 1] = w.y;
                } else {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(logits) + at + e);
                    v[j] = bf16_lo(w);
                    v[j + 1] = bf16_hi(w);
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = route_pos<VPL>(lane, j);
            v[j] = -INFINITY;
            if (e < E)
                v[j] = F32 ? static_cast<const float*>(logits)[at + e]
                           : bits_bf16(static_cast<const uint16_t*>(logits)[at + e]);
        }
    }
}

// Integers in the order of the keys (which are never -0, a bias being no -0).
// The image of -inf, which NaN counts as too, is an entry that is not there.
constexpr int KEY_NONE = (int)0x807FFFFFu;
__device__ __forceinline__ int route_key(float k) {
    const int b = __float_as_int(fmaxf(k, -INFINITY));
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}

// The lane's best two entries still to be chosen, in the order of the choice
// (key descending, position ascending), and their positions.  A second entry
// of KEY_LOST stands for the ones of the lane that have not been looked for.
constexpr int KEY_LOST = (int)0x80000000u;
struct RouteBest {
    int k1, k2, p1, p2;
};
template <int VPL>
__device__ __forceinline__ RouteBest route_best(const int (&key)[VPL], int lane) {
    RouteBest b{key[0], KEY_NONE, 0, 0};
#pragma unroll
    for (int j = 1; j < VPL; ++j) {
        const int x = key[j], at = route_pos<VPL>(0, j);
        const bool first = x > b.k1, second = x > b.k2;
        b.p2 = first ? b.p1 : (second ? at : b.p2);
        b.p1 = first ? at : b.p1;
        b.k2 = max(min(b.k1, x), b.k2);
        b.k1 = max(b.k1, x);
    }
    b.p1 += VPL == 1 ? lane : 2 * lane;
    b.p2 += 2 * lane;
    return b;
}

// Takes the first choice `top` (the maximum over the lanes, some real key) and
// returns its position.  `key` is only looked at where a lane gives a third one.
template <int VPL>
__device__ __forceinline__ int route_take(RouteBest& b, const int (&key)[VPL], int top, int lane) {
    uint64_t who = __ballot(b.k1 == top);
    int l = __builtin_ctzll(who), e = __builtin_amdgcn_readlane(b.p1, l);
    if (who & (who - 1)) {  // a tie across lanes: the lowest position, whose lane it gives
        e = -wave_max_i32(b.k1 == top ? -b.p1 : KEY_LOST);
        l = VPL == 1 ? e : (e & 127) >> 1;
    }
    const bool me = lane == l;
    b.k1 = me ? b.k2 : b.k1;
    if constexpr (VPL > 1) {
        b.p1 = me ? b.p2 : b.p1;
        if (VPL > 2 && __builtin_amdgcn_readlane(b.k1, l) == KEY_LOST) {
            int left[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                left[j] = ((key[j] < top) | ((key[j] == top) & (route_pos<VPL>(lane, j) > e))) ? key[j] : KEY_NONE;
            const RouteBest n = route_best<VPL>(left, lane);
            b.k1 = me ? n.k1 : b.k1;
            b.p1 = me ? n.p1 : b.p1;
            b.k2 = me ? n.k2 : b.k2;
            b.p2 = me ? n.p2 : b.p2;
        } else {
            b.k2 = me ? (VPL > 2 ? KEY_LOST : KEY_NONE) : b.k2;
        }
    } else {
        b.k1 = me ? KEY_NONE : b.k1;
    }
    return e;
}

// For every lane the entry v at position e of another lane's (any value where e is not a position).
template <int VPL>
__device__ __forceinline__ float route_fetch(const float (&v)[VPL], int e) {
    float r = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int from = VPL == 1 ? e : (e & 127) >> 1;
        const float x = __int_as_float(__builtin_amdgcn_ds_bpermute(4 * from, __float_as_int(v[j])));
        r = (VPL == 1 || (2 * (e >> 7) + (e & 1)) == j) ? x : r;
    }
    return r;
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
__global__ __launch_bounds__(64 * ROUTE_WAVES) void k_moe_route(RouteArgs a) {
    constexpr int NE = VPL == 1 ? 64 : 64 * VPL;
    __shared__ float s_p[ROUTE_WAVES][NE];
    __shared__ int32_t s_n[NE];
    __shared__ int32_t s_v[ROUTE_WAVES];
    __shared__ double s_w[ROUTE_WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t step = (int64_t)gridDim.x * ROUTE_WAVES;
    int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + wave;
    // the next token's logits and mask byte are on their way while one is worked on
    float next[VPL];
    uint8_t next_mask = 1;
    auto fetch = [&](int64_t i) {
        if (i >= a.T) return;
        route_load<F32, VPL, PAIRS>(a.logits, i * a.ld, lane, a.E, next);
        if (a.mask) next_mask = a.mask[i];
    };
    fetch(t);
    for (int e = threadIdx.x; e < NE; e += 64 * ROUTE_WAVES) s_n[e] = 0;
    float bias[VPL], psum[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = route_pos<VPL>(lane, j);
        bias[j] = (a.bias != nullptr && e < a.E) ? a.bias[e] + 0.0f : 0.0f;  // (-0 becomes 0)
        psum[j] = 0.0f;
    }
    __syncthreads();
    int live_rows = 0;
    for (; t < a.T; t += step) {
        float v[VPL];
        const bool on = next_mask != 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[j] = on ? route_canon(next[j]) : -INFINITY;
        fetch(t + step);
        float lm = v[0];
        int key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            key[j] = route_key(v[j] + bias[j]);
            lm = max_num(lm, v[j]);
        }
        RouteBest best = route_best<VPL>(key, lane);
        int id = -1;  // lane r < K: the r-th choice
        for (int r = 0; r < a.K; ++r) {
            const int top = wave_max_i32(best.k1);
            if (top <= KEY_NONE) break;
            const int e = route_take<VPL>(best, key, top, lane);
            id = lane == r ? e : id;
        }
        const bool live = __builtin_amdgcn_readlane(id, 0) >= 0;
        float sum = 0.0f, m = 0.0f, w = 0.0f;
        if (live) {
            ++live_rows;
            m = wave_max_f32(lm);
            float p[VPL], ls = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] = exp_neg(v[j] - m);
                ls += p[j];
            }
            sum = wave_sum_f32(ls);
            const float inv = 1.0f / sum;
#pragma unroll
            for (int j = 0; j < VPL; ++j) psum[j] = fmaf(p[j], inv, psum[j]);
            const float at = route_fetch<VPL>(v, id);  // (all lanes: a lane that is off has nothing to give)
            w = id >= 0 ? exp_neg(at - m) : 0.0f;
            if (!a.normalize) {
                w *= inv;
            } else {
                // the softmax over the chosen logits, about their own maximum where a
                // bias lifts experts whose share of the whole softmax is all but nothing
                if (__ballot(id >= 0 && !(w > 0x1p-100f))) {
                    const float lsel = id >= 0 ? at : -INFINITY;
                    const float ms = wave_max_f32(lsel);
                    w = id >= 0 ? exp_neg(lsel - ms) : 0.0f;
                }
                const float of = a.K <= 16 ? row_sum_f32(w) : wave_sum_f32(w);
                w /= of;
            }
            if (id >= 0) atomicAdd(&s_n[id], 1);
        }
        if (lane < a.K) {
            a.ids[t * a.K + lane] = id;
            a.weights[t * a.K + lane] = id >= 0 ? w * a.scale : 0.0f;
        }
        if (lane == 0) a.lse[t] = live ? fmaf(__builtin_amdgcn_logf(sum), 0.693147182f, m) : -INFINITY;
    }
    // the workgroup's sums, its waves in order
#pragma unroll
    for (int j = 0; j < VPL; ++j) s_p[wave][route_pos<VPL>(lane, j)] = psum[j];
    if (lane == 0) s_v[wave] = live_rows;
    __syncthreads();
    int live_all = 0;
#pragma unroll
    for (int w = 0; w < ROUTE_WAVES; ++w) live_all += s_v[w];
    double x = 0.0;
    for (int e = threadIdx.x; e < a.E; e += 64 * ROUTE_WAVES) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < ROUTE_WAVES; ++w) p += s_p[w][e];
        const int n = s_n[e];
        if (gridDim.x == 1) {
            a.counts[e] = n;
            x += (double)n * (double)p;
        } else {
            a.part[(int64_t)blockIdx.x * a.E + e] = make_uint2(__float_as_uint(p), (uint32_t)n);
        }
    }
    if (gridDim.x == 1) {
        x = block_sum_f64(x, s_w);
        if (threadIdx.x == 0) {
            const double n = live_all > 0 ? (double)live_all : 1.0;
            a.counts[a.E] = live_all;
            a.loss[0] = (float)((double)a.coef * a.E / a.K * x / (n * n));
        }
    } else if (threadIdx.x == 0) {
        a.part_v[blockIdx.x] = live_all;
        if (blockIdx.x == 0) *a.ticket = 0;
    }
}

// Sums of the workgroups' parts: 256 threads take 16 experts, 16 threads each,
// and leave their share of sum_e f_e P_e; the last workgroup to arrive (a
// ticket) adds the shares in order.
constexpr int FINISH_E = 16;
__global__ __launch_bounds__(256) void k_moe_route_finish(RouteArgs a, int blocks) {
    __shared__ double s_p[16][FINISH_E];
    __shared__ int32_t s_n[16][FINISH_E];
    __shared__ int s_last;
    const int i = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int e = blockIdx.x * FINISH_E + i;
    double p = 0.0;
    int n = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int b = part; b < blocks; b += 16) {
            const uint2 w = a.part[(int64_t)b * a.E + e];
            p += (double)__uint_as_float(w.x);
            n += (int)w.y;
        }
    }
    s_p[part][i] = p;
    s_n[part][i] = n;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    double x = 0.0;
    if (part == 0 && e < a.E) {
        double tp = 0.0;
        int tn = 0;
        for (int k = 0; k < 16; ++k) {
            tp += s_p[k][i];
            tn += s_n[k][i];
        }
        a.counts[e] = tn;
        x = (double)tn * tp;
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&a.part_l[blockIdx.x], x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int before = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == (int)gridDim.x - 1;
    }
    if (!__builtin_amdgcn_readfirstlane(s_last)) return;
    const int lane = threadIdx.x;
    int v = 0;
    for (int b = lane; b < blocks; b += 64) v += a.part_v[b];
    double s = lane < (int)gridDim.x ? __hip_atomic_load(&a.part_l[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        v += __shfl_xor(v, off, 64);
        s += __shfl_xor(s, off, 64);
    }
    if (lane == 0) {
        const double nv = v > 0 ? (double)v : 1.0;
        a.counts[a.E] = v;
        a.loss[0] = (float)((double)a.coef * a.E / a.K * s / (nv * nv));
    }
}
static_assert(ROUTE_MAX_E / FINISH_E <= 64, "one lane a share");

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
// What the choices add goes to the lanes that hold their experts through the
// wave's row of LDS, which is all zero between tokens.  16384 x 384 binary32
// take 13 us (50 MB, 3.8 TB/s).
template <bool F32, int VPL, bool PAIRS>
__global__ __launch_bounds__(256) void k_moe_route_bwd(RouteBwdArgs a) {
    constexpr int NE = VPL == 1 ? 64 : 64 * VPL;
    __shared__ float s_g[4][NE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* g_row = s_g[wave];
    float u[VPL];
    {
        const double nv = a.counts[a.E] > 0 ? (double)a.counts[a.E] : 1.0;
        const double c = a.dloss ? (double)a.dloss[0] * a.coef * a.E / a.K / (nv * nv) : 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = route_pos<VPL>(lane, j);
            u[j] = e < a.E ? (float)(c * a.counts[e]) : 0.0f;
            g_row[e] = 0.0f;
        }
    }
    const float rscale = a.scale != 0.0f ? 1.0f / a.scale : 0.0f;
    const int64_t step = (int64_t)gridDim.x * 4;
    int64_t t = (int64_t)blockIdx.x * 4 + wave;
    float next[VPL], next_w = 0.0f, next_dw = 0.0f;
    int next_id = -1;
    bool next_on = false;
    auto fetch = [&](int64_t i) {
        next_on = i < a.T && a.lse[i] > -INFINITY;
        if (!next_on) return;
        route_load<F32, VPL, PAIRS>(a.logits, i * a.ld, lane, a.E, next);
        next_id = -1;
        if (lane < a.K && a.dweights) {
            next_id = a.ids[i * a.K + lane];
            next_w = a.weights[i * a.K + lane];
            next_dw = a.dweights[i * a.K + lane];
        }
    };
    fetch(t);
    for (; t < a.T; t += step) {
        float d[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
        if (next_on) {
            float v[VPL], g[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) v[j] = route_canon(next[j]);
            const int id = (uint32_t)next_id < (uint32_t)a.E ? next_id : -1;
            const float w = next_w;
            float x = 0.0f;  // lane r < K: what its choice adds
            if (id >= 0) x = a.normalize ? w * next_dw : a.scale * next_dw;
            fetch(t + step);
            if (a.dweights) {
                if (a.normalize) {
                    const float dot = wave_sum_f32(x);  // sum_i w_i dw_i = scale sum_i q_i dw_i
                    if (id >= 0) x -= w * rscale * dot;
                }
                if (id >= 0) atomicAdd(&g_row[id], x);
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < VPL; ++j) g[j] = g_row[route_pos<VPL>(lane, j)];
            __builtin_amdgcn_wave_barrier();
            if (id >= 0) g_row[id] = 0.0f;
            // the softmax again rather than exp(l - lse): at a maximum of large
            // magnitude lse does not hold the logarithm of the sum
            float lm = v[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) lm = max_num(lm, v[j]);
            const float m = wave_max_f32(lm);
            float p[VPL], up[VPL], ls = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] = exp_neg(v[j] - m);
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
        } else {
            fetch(t + step);
        }
        const int64_t at = t * a.ldd;
#pragma unroll
        for (int j = 0; j < VPL; j += (PAIRS && VPL > 1) ? 2 : 1) {
            const int e = route_pos<VPL>(lane, j);
            if (e >= a.E) continue;
            if constexpr (PAIRS && VPL > 1) {
                if constexpr (F32)
                    st_stream8(static_cast<float*>(a.dlogits) + at + e, make_uint2(__float_as_uint(d[j]), __float_as_uint(d[j + 1])));
                else
                    st_stream4(static_cast<uint16_t*>(a.dlogits) + at + e, pack_bf16x2(d[j], d[j + 1]));
            } else if constexpr (F32) {
                static_cast<float*>(a.dlogits)[at + e] = d[j];
            } else {
                static_cast<uint16_t*>(a.dlogits)[at + e] = bf16_rne(d[j]);
            }
        }
    }
}

namespace {

int route_blocks(int64_t T) {
    if (T <= ROUTE_ONE_BLOCK) return 1;
    const int64_t b = (T + ROUTE_WAVES - 1) / ROUTE_WAVES;
    return (int)(b < ROUTE_MAX_BLOCKS ? b : ROUTE_MAX_BLOCKS);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Calls f with the number of experts a lane holds (one, or two of every 128).
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
    return bsq::up256(b * num_experts * 8) + bsq::up256(b * 4) + 512 + 256;
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
    const size_t pe = bsq::up256((size_t)blocks * num_experts * 8), pv = bsq::up256((size_t)blocks * 4);
    bsq::RouteArgs a{logits, tokens, ld, num_experts, top_k, bias, mask, normalize, scale, loss_coef,
                     expert_ids, weights, lse, counts, loss,
                     reinterpret_cast<uint2*>(ws), reinterpret_cast<int32_t*>(ws + pe),
                     reinterpret_cast<double*>(ws + pe + pv), reinterpret_cast<int32_t*>(ws + pe + pv + 512)};
    const bool pairs = num_experts % 2 == 0 && ld % 2 == 0 && bsq::aligned_to(logits, 2 * z);
    const dim3 grid(blocks), block(64 * bsq::ROUTE_WAVES);
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
        hipLaunchKernelGGL(bsq::k_moe_route_finish, dim3((num_experts + bsq::FINISH_E - 1) / bsq::FINISH_E),
                           dim3(256), 0, stream, a, blocks);
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
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024)), block(256);
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
