// Losses of an output head's product over the whole vocabulary, and their gradients.
//
//   z[t][v] = scale * sum_h x[t][h] w[v][h],  lse[t] = log sum_v exp z[t][v],  p = exp(z - lse)
//   cross entropy   loss[t] = lse[t] - z[t][label[t]]
//   distillation    loss[t] = sum_k q[t][k] (log q[t][k] - z[t][id[t][k]] + lse[t])
//   gradient of z   g[t][v] = (dloss Q + dlse) p[t][v] - dloss sum_{k: id = v} q[t][k],  Q = sum_k q[t][k]
//                   (cross entropy: one entry, the label, with q = 1)
//   dx = scale g w,  dw = scale g^T x
//
// (Sizes in comments: tokens x vocabulary x hidden, or (tokens, vocabulary, hidden) of one call
// replayed in a graph; times in microseconds unless said.)
//
// The logits exist only in accumulators: the forward reduces a tile's 256 columns to a
// maximum and a sum of exponentials per row, and the backward forms them again, a
// piece of the vocabulary at a time, to write that piece's g for the other two products.
// Rows without a target are left out: k_rows lists the others, and a dense copy of
// their x, padded with zeros, is what the products read.
//
// For bf16 gradients g is rounded to bf16, an error of the size of the output's own rounding
// (the two together are 1.4 of it, by the norm), and of a pair of bf16 for up to PAIR tokens,
// where the few large entries of g, those of the targets, do not average out. For f32 gradients it is
// split into three bf16 parts, which hold all of its 24 bits.
//
// dx is formed transposed, since its columns layout operand (w) is the one that a wave reads
// less of, and dw takes a transposed copy of x.
//
// A row's loss and lse are the same bits whatever else the call holds: a logit is
// one chain of MFMAs along k in every form, and parts of its sum are merged
// in one order: the 16 values of a lane, then a binary tree over runs of 32, 64 .. 4096
// columns, then those runs one after the other.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/bsq.h"
#include "device_common.h"
#include "gemm_pipe.h"
#include "moe_common.h"
#include "vocab_gemm.h"

namespace bsq {

constexpr float LOG2E = 1.44269504f;
constexpr int RUN = 4096;       // columns of a tree of parts of a sum
constexpr int MAX_LIST = 1024;  // entries of a token's list

// Which tokens have a target (backward: and a gradient).
struct Live {
    const int32_t* labels;  // cross entropy, or
    const float* qsum;      // distillation: [T] sum of a list's weights
    const float *dloss, *dlse;
    int back;
    int64_t V, T;
    __device__ __forceinline__ bool operator()(int64_t t) const {
        bool on = labels ? (uint64_t)(int64_t)labels[t] < (uint64_t)V : qsum[t] != 0.0f;
        if (back) on &= (dloss && dloss[t] != 0.0f) || (dlse && dlse[t] != 0.0f);
        return on;
    }
};

struct HeadArgs {
    // operands
    const uint8_t* w;
    int64_t ldw;             // bytes
    int64_t V, H, T;
    const uint8_t* x;        // dense rows with a target, [Tp][Hp], zero past them; direct: the caller's
    int64_t ldx;             // bytes
    int64_t Hp, Tp;
    float scale;
    float far_key;           // 2^(far - 20) of the pairs
    Live live;
    // rows (not direct)
    const int32_t* count;    // rows with a target
    const int32_t* rows;     // their tokens
    // targets (cross entropy: live.labels)
    int K;                   // distillation: entries of a list, sorted by id:
    const int32_t* sid;      //   ids
    const int32_t* sslot;    //   places in the caller's list
    const float* sq;         //   weights q
    const uint16_t* tab;     //   [T][blocks + 1] first entry of each block of columns
    int64_t blocks;
    // forward
    float2* part;            // [blocks of columns][Tp] pairs of the sums of exponentials (merge)
    float* zat;              // cross entropy: [Tp] unscaled logit of the label
    float* logits;           // distillation: [T][K] logits of the list
    // backward
    const float* lse;
    int64_t v0, vc;          // the piece's first column and width (a multiple of 256)
    uint16_t* g;             // [terms][Tp][vc] bf16 parts of g
    int terms;
};

// ------------------------------------------------------------ rows with a target

struct RowsArgs {
    Live live;
    int64_t T, Tp, H, Hp;
    const uint16_t* x;
    int64_t ldx;
    int32_t *count, *rows, *pos;
    uint16_t *xc, *xt;      // xt: the copy transposed, [Hp][Tp], or null
};

constexpr int ROWS_ITEMS = 4;
constexpr int ROWS_SELF = 256 * ROWS_ITEMS;  // tokens up to which every workgroup of the copy lists them by itself

// Exclusive prefix of `n` over the workgroup; *total: the sum.
template <int WAVES>
__device__ __forceinline__ int block_scan(int n, int* s_sum, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int incl = wave_scan_i32(n);
    __syncthreads();
    if (lane == 63) s_sum[wave] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        if (i < wave) before += s_sum[i];
        total += s_sum[i];
    }
    return before + incl - n;
}

// One workgroup: the list of the rows with a target, for more than ROWS_SELF tokens.  Bound by the latency of a
// round of loads (4096 tokens 5 us, 16384 16): next to the product of so many it is nothing, and one
// workgroup needs no order among several.
__global__ __launch_bounds__(1024) void k_rows(RowsArgs a) {
    __shared__ int s_sum[16];
    int done = 0;
    for (int64_t base = 0; base < a.T; base += 1024 * ROWS_ITEMS) {
        const int64_t t0 = base + (int64_t)threadIdx.x * ROWS_ITEMS;
        unsigned on = 0;
#pragma unroll
        for (int i = 0; i < ROWS_ITEMS; ++i)
            if (t0 + i < a.T && a.live(t0 + i)) on |= 1u << i;
        int total;
        int at = done + block_scan<16>(__builtin_popcount(on), s_sum, total);
#pragma unroll
        for (int i = 0; i < ROWS_ITEMS; ++i)
            if (t0 + i < a.T) {
                const bool o = (on >> i) & 1;
                a.pos[t0 + i] = o ? at : -1;
                if (o) a.rows[at++] = (int32_t)(t0 + i);
            }
        done += total;
    }
    if (threadIdx.x == 0) *a.count = done;
}

// A dense copy of every row, for few tokens at a pitch that the products' 32-bit offsets do not reach
// (the last positions of long sequences, say).
__global__ __launch_bounds__(256) void k_pack_rows(const uint16_t* x, int64_t ldx, int64_t H, uint16_t* to, int64_t ld) {
    const int64_t h = 8 * ((int64_t)blockIdx.y * 256 + threadIdx.x);
    if (h < H) *reinterpret_cast<uint4*>(to + blockIdx.x * ld + h) = *reinterpret_cast<const uint4*>(x + blockIdx.x * ldx + h);
}

// Dense copy, and its transpose for dw: 64 rows x 64 columns a workgroup, zeros behind the
// last row up to a multiple of 256.  dw reduces over rows, and the operand of which a wave reads more
// has to be contiguous along the reduction; the transpose goes through LDS in pairs of columns.
// Bound by bytes: 4096 x 7168, both copies, 21 us (8.3 TB/s with what the caches hold, 115 MB written).
template <bool SELF>
__global__ __launch_bounds__(256) void k_copy_rows(RowsArgs a) {
    __shared__ int s_sum[4];
    __shared__ int s_row[64];
    __shared__ uint32_t s_t[64][33];
    const int64_t r0 = (int64_t)blockIdx.x * 64, h0 = (int64_t)blockIdx.y * 64;
    int count;
    if constexpr (SELF) {
        const int t0 = threadIdx.x * ROWS_ITEMS;
        unsigned on = 0;
#pragma unroll
        for (int i = 0; i < ROWS_ITEMS; ++i)
            if (t0 + i < a.T && a.live(t0 + i)) on |= 1u << i;
        int at = block_scan<4>(__builtin_popcount(on), s_sum, count);
#pragma unroll
        for (int i = 0; i < ROWS_ITEMS; ++i)
            if (t0 + i < a.T) {
                const bool o = (on >> i) & 1;
                if (blockIdx.x == 0 && blockIdx.y == 0) {
                    a.pos[t0 + i] = o ? at : -1;
                    if (o) a.rows[at] = t0 + i;
                }
                if (o && at >= r0 && at < r0 + 64) s_row[at - r0] = t0 + i;
                at += o;
            }
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.count = count;
    } else {
        count = *a.count;
        if (threadIdx.x < 64 && r0 + threadIdx.x < count) s_row[threadIdx.x] = a.rows[r0 + threadIdx.x];
    }
    __syncthreads();
    if (r0 >= (count + 255) / 256 * 256) return;
#pragma unroll
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i >> 3, c = i & 7;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + r < count && h0 + 8 * c < a.H)
            v = *reinterpret_cast<const uint4*>(a.x + (int64_t)s_row[r] * a.ldx + h0 + 8 * c);
        *reinterpret_cast<uint4*>(a.xc + (r0 + r) * a.Hp + h0 + 8 * c) = v;
        s_t[r][4 * c] = v.x;
        s_t[r][4 * c + 1] = v.y;
        s_t[r][4 * c + 2] = v.z;
        s_t[r][4 * c + 3] = v.w;
    }
    if (!a.xt) return;
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int c = i >> 3, r = 8 * (i & 7);  // column c of rows r .. r + 7
        uint32_t w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            w[v] = __builtin_amdgcn_perm(s_t[r + 2 * v + 1][c >> 1], s_t[r + 2 * v][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
        *reinterpret_cast<uint4*>(a.xt + (h0 + c) * a.Tp + r0 + r) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ----------------------------------------------------- lists of the teacher's entries

struct ListArgs {
    const int32_t* ids;
    const void* tl;          // teacher logits, f32 or bf16
    int tl_f32;
    const float* tlse;       // or null: normalized over the list
    float tscale;
    int64_t T, V;
    int K;
    int block;               // columns of a block of the table
    int64_t blocks;
    int32_t *sid, *sslot;
    float* sq;
    uint16_t* tab;
    float* qsum;
    float* logits;           // cleared, where not null
};

// A wave per token: weights, the present entries sorted by id (by rank: K^2 / 64 comparisons), and the
// table of where each block of columns begins.  Sorted lists let a tile of the logits read only the
// entries of its own columns.  4096 lists of 128 take 23 us, 8192 of 32 14, beside products of 0.9 ms.
__global__ __launch_bounds__(256) void k_lists(ListArgs a) {
    __shared__ int32_t s_key[4][MAX_LIST], s_sorted[4][MAX_LIST];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    const bool live = t < a.T;
    const int K = live ? a.K : 0;
    auto value = [&](int k) {  // scaled teacher logit of entry k, or -inf
        const int64_t i = t * a.K + k;
        if ((uint64_t)(int64_t)a.ids[i] >= (uint64_t)a.V) return -INFINITY;
        return a.tscale * (a.tl_f32 ? static_cast<const float*>(a.tl)[i] : bits_bf16(static_cast<const uint16_t*>(a.tl)[i]));
    };
    float top = -INFINITY, sum = 0.0f;
    for (int k = lane; k < K; k += 64) {
        const int32_t id = a.ids[t * a.K + k];
        s_key[wave][k] = (uint64_t)(int64_t)id < (uint64_t)a.V ? id : 0x7FFFFFFF;
        top = fmaxf(top, value(k));
        if (a.logits) a.logits[t * a.K + k] = 0.0f;
    }
    if (a.tlse) {
        top = live ? a.tlse[t] : 0.0f;
    } else {
        top = wave_max_f32(top);
        if (top == -INFINITY) top = 0.0f;
    }
    auto weight = [&](int k) {
        const float v = value(k);
        return v == -INFINITY ? 0.0f : expf(v - top);
    };
    for (int k = lane; k < K; k += 64) sum += weight(k);
    sum = wave_sum_f32(sum);
    const float div = a.tlse || sum == 0.0f ? 1.0f : sum;
    float q = 0.0f;
    __syncthreads();
    int n = 0;
    for (int k = lane; k < K; k += 64) {
        const int32_t key = s_key[wave][k];
        const bool on = key != 0x7FFFFFFF;
        int rank = 0;
        for (int j = 0; j < K; ++j) {
            const int32_t o = s_key[wave][j];
            rank += o < key || (o == key && j < k);
        }
        if (on) {
            const float w = weight(k) / div;
            q += w;
            s_sorted[wave][rank] = key;
            a.sid[t * a.K + rank] = key;
            a.sslot[t * a.K + rank] = k;
            a.sq[t * a.K + rank] = w;
            ++n;
        }
    }
    q = wave_sum_f32(q);
    n = __builtin_amdgcn_readlane(wave_scan_i32(n), 63);
    if (live && lane == 0) a.qsum[t] = q;
    __syncthreads();
    if (live)
        for (int64_t b = lane; b <= a.blocks; b += 64) {
            const int64_t first = b * a.block;
            int lo = 0, hi = n;  // entries below `first`
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_sorted[wave][mid] < first) lo = mid + 1;
                else hi = mid;
            }
            a.tab[t * (a.blocks + 1) + b] = (uint16_t)lo;
        }
}

// --------------------------------------------------------------- the logits' tiles

// A part of a row's sum of exponentials is a pair (2^-20 R, s): s = sum 2^(kappa z - R), kappa = scale
// log2(e), z unscaled, R the whole number next to the part's largest kappa z (NOTHING in its place where
// there is none).  One rounding gives an exponent's argument, and merging two parts is exact but for the addition.
// Where the largest kappa z is beyond FAR in size, the rounding of R itself, more than 32, is too much for an exponent, and
// different z are 64 or more apart (2^-24 of their size).  There s = sum 2^(kappa (z - m)) with m the largest z, which is how
// many are equal to it, and R is 2^f m, 2^f being the least power of two from kappa on: exact, beyond FAR as well, and of
// different m still 64 or more apart.  (R is held as 2^-20 of it, which every finite m leaves in binary32 up to a scale of
// 2^19.)  Logits of -1e10 and the lowest finite values, which mask parts of a vocabulary, are of this kind.
constexpr float NOTHING = -3e38f, FAR = 1073741824.0f, KEY = 1.0f / (1 << 20), MOST = 3.40282347e38f;
constexpr float LARGE = 65536.0f;  // of R, from where on roundings of the logits' size show in a sum
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
    const float r = max_num(a.x, b.x);
    auto scaled = [&](float2 x) { return ldexpf(x.y, (int)(max_num(x.x - r, -512.0f * KEY) * (1 / KEY))); };
    return make_float2(r, scaled(a) + scaled(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
// The pair of 16 values.
__device__ __forceinline__ float2 pair16(const float (&x)[16], float kappa, float far_key) {
    const float m = max3(max3(max3(x[0], x[1], x[2]), x[3], x[4]), max3(max3(x[5], x[6], x[7]), x[8], x[9]),
                         max3(max3(x[10], x[11], x[12]), max3(x[13], x[14], x[15]), x[15]));
    const float y = __builtin_rintf(m * kappa), r = max_num(y, NOTHING);
    float e[16], key = max_num(y * KEY, NOTHING);
#pragma unroll
    for (int v = 0; v < 16; ++v) e[v] = fmaf(x[v], kappa, -r);
    const bool far = !(fabsf(r) <= FAR) && m > -INFINITY;
    if (__builtin_expect(__ballot(far) != 0, 0)) {
        const float k = kappa < MOST ? kappa : MOST;
#pragma unroll
        for (int v = 0; v < 16; ++v) e[v] = far ? (x[v] - m) * k : e[v];
        key = far ? fminf(fmaxf(m * far_key, NOTHING), -NOTHING) : key;
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) e[v] = __builtin_amdgcn_exp2f(e[v]);
#pragma unroll
    for (int n = 1; n < 16; n *= 2)
#pragma unroll
        for (int v = 0; v < 16; v += 2 * n) e[v] += e[v + n];
    return make_float2(key, e[0]);
}

// The tile of workgroup wg: an XCD (every eighth workgroup) takes an eighth of them,
// row by row of groups of 4 row tiles, so that the tiles it runs at once share operands.
// (Grids stay below 2^23 workgroups.)
__device__ __forceinline__ bool pick_tile(uint32_t wg, int64_t nq_, int64_t np_, int64_t& q, int64_t& p) {
    const uint32_t nq = (uint32_t)nq_, np = (uint32_t)np_;
    const uint32_t n = nq * np, share = (n + 7) / 8, i = wg >> 3, t = (wg & 7) * share + i;
    if (i >= share || t >= n) return false;
    const uint32_t g = t / (4 * np), first = 4 * g, r = t - first * np;
    const uint32_t m = nq - first < 4 ? nq - first : 4, c = r / m;
    q = first + (r - c * m);
    p = c;
    return true;
}

// A tile of logits and, in its accumulators, what becomes of them.  Bound by the matrix cores for many
// tokens: 4096 x 131072 x 7168 4.9 ms (1570 TFLOP/s; the matrix units 92% busy, the clock at the power limit; the
// library's bare product 5.18 ms), 16384 x 32768 x 2048 1.55 ms (1420: a tile's exponentials take 7 of its 50 us, and
// nothing overlaps them); by w for few: (64, 131072, 7168) 324 us, 5.8 TB/s, (48, 32768, 2048) 24, 5.6.  A workgroup that
// goes on to another tile and fetches its first stages ahead of the exponentials was no faster (1556 and 1573, 122 and
// 124 for 1237 x 50021 x 1000): the next workgroup starts as early, and the kept state spills.
// DIRECT: on the caller's x (any number of rows of tiles); rows without a target are zeros.
template <class Loop, bool BACK, bool LIST, bool DIRECT>
__global__ __launch_bounds__(64 * Loop::WAVES, 1) void k_logits(HeadArgs a) {
    constexpr int TP = Loop::TP, TQ = Loop::TQ, NP = Loop::NP, NQ = Loop::NQ, WP = Loop::WP;
    __shared__ __align__(1024) uint8_t smem[Loop::LDS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % WP, wq = wave / WP;
    const int count = DIRECT ? (int)a.T : *a.count;
    const int64_t vend = BACK ? (a.v0 + a.vc < a.V ? a.v0 + a.vc : a.V) : a.V;
    const int64_t np = BACK ? a.vc / TP : (a.V + TP - 1) / TP;
    int64_t tq, tp;
    if (!pick_tile(blockIdx.x, (count + TQ - 1) / TQ, np, tq, tp)) return;
    const int64_t q0 = tq * TQ, p0 = (BACK ? a.v0 : 0) + tp * TP;
    float4v acc[NP][NQ];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
    const int64_t pr = vend - p0 < TP ? (vend - p0 > 0 ? vend - p0 : 0) : TP;
    const Side P{a.w + p0 * a.ldw, pr ? (pr - 1) * a.ldw + 2 * a.H : 0, 128, (uint32_t)a.ldw, (uint32_t)pr,
                 (uint32_t)(2 * a.H - 2 * (a.Hp - 64))};
    // (a piece's tiles past the vocabulary are zero)
    const int stages = pr ? (int)(a.Hp / 64) : 0;
    if constexpr (DIRECT) {
        const int64_t rows = a.T - q0 < TQ ? a.T - q0 : TQ;
        const Side Q{a.x + q0 * a.ldx, (rows - 1) * a.ldx + 2 * a.H, 128, (uint32_t)a.ldx, (uint32_t)rows, P.tail};
        Loop::run(acc, smem, stages, 1, [&](int) { return P; }, [&](int) { return Q; }, [&](int r) { return a.live(q0 + r); });
    } else {
        const Side Q{a.x + q0 * a.ldx, TQ * a.ldx, 128, (uint32_t)a.ldx, TQ, 128};
        Loop::run(acc, smem, stages, 1, [&](int) { return P; }, [&](int) { return Q; });
    }

    const float kappa = a.scale * LOG2E;
    const int g = lane >> 4;
    // values of this lane: v of acc[i][j] is column base + 64 (i / 4) + 4 (i % 4) + v
    const int base = (int)p0 + 16 * NP * wp + 16 * g;
    auto value = [](int i, int v) { return 64 * (i >> 2) + 4 * (i & 3) + v; };
    // what the rows of this lane need, all loads of a kind together: a chain of them a row
    // takes a microsecond
    int token[NQ], at_[NQ], end_[NQ];
    float lse_[NQ], d_[NQ], c_[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int64_t q = q0 + 16 * (NQ * wq + j) + (lane & 15);
        token[j] = q < count ? (int)q : -1;
        if constexpr (!DIRECT) {
            const int row = a.rows[q < count ? q : 0];
            token[j] = q < count ? row : -1;
        }
    }
    if constexpr (DIRECT) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
            if (token[j] >= 0 && !a.live(token[j])) token[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int64_t t = token[j] >= 0 ? token[j] : 0;
        if constexpr (!LIST) {
            at_[j] = a.live.labels[t];
        } else {
            // (the table ends with the vocabulary)
            const uint16_t* tab = a.tab + t * (a.blocks + 1) + (pr ? p0 / TP : 0);
            at_[j] = tab[0];
            end_[j] = token[j] >= 0 && pr ? tab[1] : 0;
        }
        if constexpr (BACK) {
            lse_[j] = token[j] >= 0 ? a.lse[t] : 0.0f;
            d_[j] = a.live.dloss ? a.live.dloss[t] : 0.0f;
            c_[j] = LIST ? a.live.qsum[t] : 1.0f;
        }
    }
    if constexpr (BACK) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const float s = a.live.dlse ? a.live.dlse[token[j] >= 0 ? token[j] : 0] : 0.0f;
            c_[j] = token[j] < 0 ? 0.0f : a.scale * ((d_[j] == 0.0f ? 0.0f : d_[j] * c_[j]) + s);
            d_[j] = token[j] < 0 ? 0.0f : a.scale * d_[j];
        }
    }
    if constexpr (BACK) {
        // rows without a target, and those behind the last: their x is zero, which an infinite w makes a NaN of
        if (DIRECT || q0 + TQ > count) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = token[j] < 0 ? 0.0f : acc[i][j][v];
        }
    }
    // f(value, entry's x): for each entry of the list of row j that one of this lane's values stands
    // for; x(e): what is loaded of entry e
    auto hits = [&](int j, auto x, auto f) {
        if constexpr (!LIST) {
            const int d = at_[j] - base;
            const bool mine = token[j] >= 0 && d >= 0 && d < 16 * NP && (d & 63) < 16;
            if (__ballot(mine) && mine) f(d, x(0));
        } else {
            const int64_t list = (int64_t)(token[j] >= 0 ? token[j] : 0) * a.K;
            for (int e = at_[j]; __ballot(e < end_[j]); e += 4) {
                int id[4];
                decltype(x(0)) y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = e + u < end_[j] ? e + u : 0;
                    id[u] = a.sid[list + k];
                    y[u] = x(list + k);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int d = id[u] - base;
                    const bool mine = e + u < end_[j] && d >= 0 && d < 16 * NP && (d & 63) < 16;
                    if (__ballot(mine) && mine) f(d, y[u]);
                }
            }
        }
    };
    float k_[NQ];  // exponents of e are fmaf(acc, k_, -lse_)
#pragma unroll
    for (int j = 0; j < NQ; ++j) k_[j] = a.scale;
    // columns past the end (the last tile's)
    const int end = (int)vend - base;
    if (p0 + TP > vend) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (value(i, v) >= end) acc[i][j][v] = -INFINITY;  // (its exponential is 0)
    }
    if constexpr (BACK) {
        // Where lse is large, z is rounded as the forward rounds the largest logit into it, whose p so is 1, and no p is more.
        bool large = false;
#pragma unroll
        for (int j = 0; j < NQ; ++j) large |= !(fabsf(lse_[j]) <= LARGE / 2);
        if (__builtin_expect(__ballot(large) != 0, 0)) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                if (!(fabsf(lse_[j]) <= LARGE / 2)) {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float d = a.scale * acc[i][j][v] - lse_[j];
                            acc[i][j][v] = d > 0.0f && lse_[j] > -INFINITY ? 0.0f : d;
                        }
                    k_[j] = 1.0f;
                    lse_[j] = 0.0f;
                }
        }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        if constexpr (!BACK) {
            hits(j, [&](int64_t e) { return LIST ? a.sslot[e] : 0; }, [&](int d, int slot) {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) z = d == value(i, v) ? acc[i][j][v] : z;
                if constexpr (LIST) a.logits[(int64_t)token[j] * a.K + slot] = z;  // (k_finish scales it)
                else a.zat[q0 + 16 * (NQ * wq + j) + (lane & 15)] = z;
            });
            float2 u[NP / 4];
#pragma unroll
            for (int n = 0; n < NP / 4; ++n) {
                float x[16];
#pragma unroll
                for (int v = 0; v < 16; ++v) x[v] = acc[4 * n + v / 4][j][v & 3];
                u[n] = pair16(x, kappa, a.far_key);
                // with the lanes 16, then 32 away: the runs of 32 and of 64 columns
                Pair32 pm = swap16(__float_as_uint(u[n].x)), ps = swap16(__float_as_uint(u[n].y));
                u[n] = merge(make_float2(__uint_as_float(pm.a), __uint_as_float(ps.a)),
                             make_float2(__uint_as_float(pm.b), __uint_as_float(ps.b)));
                pm = swap32(__float_as_uint(u[n].x));
                ps = swap32(__float_as_uint(u[n].y));
                u[n] = merge(make_float2(__uint_as_float(pm.a), __uint_as_float(ps.a)),
                             make_float2(__uint_as_float(pm.b), __uint_as_float(ps.b)));
            }
            if constexpr (NP == 8) u[0] = merge(u[0], u[1]);
            static_assert(NP == 4 || NP == 8, "one or two runs of 64 columns a wave");
            if (g == 0) reinterpret_cast<float2*>(smem)[wp * TQ + 16 * (NQ * wq + j) + lane] = u[0];
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[i][j][v] = c_[j] * __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], k_[j], -lse_[j]) * LOG2E);
            if (__ballot(d_[j] != 0.0f))
                hits(j, [&](int64_t e) { return LIST ? a.sq[e] : 1.0f; }, [&](int at, float w) {
                    if (d_[j] == 0.0f) return;
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] -= at == value(i, v) ? d_[j] * w : 0.0f;
                });
        }
    }
    if constexpr (BACK) {
        for (int n = 0; n < a.terms; ++n) {
            uint16_t* to = a.g + (n * a.Tp + q0) * a.vc + (p0 - a.v0);
            store_tile<Loop, uint16_t, false>(acc, smem, TP, [&](int q) { return q0 + q < a.Tp ? to + q * a.vc : nullptr; });
            if (n + 1 < a.terms) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const uint32_t lo = pack_bf16x2(acc[i][j][0], acc[i][j][1]), hi = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
                        acc[i][j] -= float4v{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
                    }
            }
        }
    }
    if constexpr (!BACK) {
        __syncthreads();
        for (int i = threadIdx.x; i < TQ; i += 64 * Loop::WAVES) {
            const float2* s = reinterpret_cast<const float2*>(smem);
            float2 u = s[i];
            if constexpr (WP == 2) u = merge(u, s[TQ + i]);
            static_assert(WP <= 2, "one merge over the waves");
            if (q0 + i < a.Tp) a.part[tp * a.Tp + q0 + i] = u;
        }
    }
}

// ---------------------------------------------------------- the forward's last step

struct FinishArgs {
    const float2* part;
    int64_t blocks, Tp, T;
    float scale;
    float far_unit;          // 2^(20 - far) of the pairs
    double unit;             // scale / kappa
    Live live;
    const int32_t* pos;      // null: direct
    const float* zat;
    int K;
    const int32_t* sslot;
    const float* sq;
    const uint16_t* tab;
    float *logits, *loss, *lse;
};

// LEAF columns a pair.  A workgroup takes TOK tokens; a thread the tree of 16 pairs of one token,
// and every thread then merges the token's runs.  Bound by latency (4 us for 16 tokens, a kernel's least; 4096 x
// 131072, 17 MB of pairs, 13): TOK adjacent tokens make a 32- or 64-byte piece of every block's row.
template <int LEAF, bool LIST>
__global__ __launch_bounds__(256) void k_finish(FinishArgs a) {
    constexpr int TOK = LEAF == 256 ? 8 : 4, SLOTS = 256 / TOK, SUB = RUN / LEAF / 16;
    __shared__ float2 s_run[SLOTS][TOK];
    const int tk = threadIdx.x % TOK, g = threadIdx.x / TOK;
    const int64_t t = (int64_t)blockIdx.x * TOK + tk;
    auto place = [&](int64_t t) -> int { return t >= a.T ? -1 : a.pos ? a.pos[t] : a.live(t) ? (int)t : -1; };
    const int pos = place(t);
    const float kappa = a.scale * LOG2E;
    const float2 none = make_float2(NOTHING, 0.0f);
    float2 all = none;
    for (int64_t b0 = 0; b0 < a.blocks; b0 += 16 * SLOTS) {
        float2 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t b = b0 + 16 * g + i;
            x[i] = pos >= 0 && b < a.blocks ? a.part[b * a.Tp + pos] : none;
        }
#pragma unroll
        for (int n = 1; n < 16; n *= 2)
#pragma unroll
            for (int i = 0; i < 16; i += 2 * n) x[i] = merge(x[i], x[i + n]);
        s_run[g][tk] = x[0];
        __syncthreads();
        const int64_t left = (a.blocks - b0 + 15) / 16;
        for (int i = 0; i < SLOTS && i < left; i += SUB) {
            float2 u = s_run[i][tk];
            if constexpr (SUB >= 2) u = merge(u, s_run[i + 1][tk]);
            if constexpr (SUB == 4) u = merge(u, merge(s_run[i + 2][tk], s_run[i + 3][tk]));
            all = merge(all, u);
        }
        __syncthreads();
    }
    constexpr float LN2 = 0.693147181f, HUGE_Z = 1e38f;
    const float ln = logf(all.y);
    // lse of a pair's (key, ln s).  Beyond LARGE the roundings of kappa and of R ln 2 would show beside ln s: 64 bits, or the
    // largest logit as it is rounded by itself.
    auto lse_of = [&](float key, float ln) {
        const float R = key / KEY;
        if (fabsf(R) > LARGE && key > NOTHING) {
            const double top = fabsf(R) > FAR ? (double)(a.scale * (key * a.far_unit)) : R * a.unit;
            return (float)(top + ln);
        }
        return fmaf(R, LN2, ln);
    };
    // lse - z of an unscaled logit, as the sum's own term of it was formed (its product with kappa may leave binary32, though)
    auto loss_of = [&](float key, float ln, float z) {
        const float R = key / KEY;
        if (fabsf(R) > FAR && key > NOTHING) return ln - a.scale * (z - key * a.far_unit);
        return fabsf(z * kappa) < HUGE_Z ? ln - LN2 * fmaf(z, kappa, -R) : lse_of(key, ln) - a.scale * z;
    };
    if constexpr (!LIST) {
        if (g == 0 && t < a.T) {
            a.lse[t] = pos >= 0 ? lse_of(all.x, ln) : -INFINITY;
            const float loss = pos >= 0 ? loss_of(all.x, ln, a.zat[pos]) : 0.0f;
            a.loss[t] = loss < 0.0f ? 0.0f : loss;  // (not below 0 by a rounding)
        }
    } else {
        // a wave per token: its lanes share the list, whose logits are unscaled so far
        __shared__ float s_m[TOK], s_l[TOK];
        if (g == 0) {
            s_m[tk] = all.x;
            s_l[tk] = ln;
        }
        __syncthreads();
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int k = threadIdx.x >> 6; k < TOK; k += 4) {
            const int64_t u = (int64_t)blockIdx.x * TOK + k;
            const int at = place(u);
            float sum = 0.0f;
            if (at >= 0) {
                const int n = a.tab[u * (a.blocks + 1) + a.blocks];
                for (int e = lane; e < n; e += 64) {
                    float* to = a.logits + u * a.K + a.sslot[u * a.K + e];
                    const float q = a.sq[u * a.K + e], z = *to;
                    *to = a.scale * z;
                    if (q != 0.0f) sum += q * (logf(q) + loss_of(s_m[k], s_l[k], z));
                }
            }
            sum = wave_sum_f32(sum);
            if (lane == 0 && u < a.T) {
                a.loss[u] = at >= 0 ? sum : 0.0f;
                a.lse[u] = at >= 0 ? lse_of(s_m[k], s_l[k]) : -INFINITY;
            }
        }
    }
}

// ---------------------------------------------------------- the gradients' products

// dx transposed: out[h][t] over a part of the piece's columns, added to a sum in 32 bits.
// STACKED: the parts of g are rows one below the other (of the caller's tokens), and so w is
// read once for all of them; else passes.
struct DxArgs {
    float* part;       // [splits][Hp][pitch]
    int64_t pitch;     // Tp, stacked: terms * Tp
    int splits, first; // first: the sums begin here
    int terms;
};

template <class Loop, bool STACKED>
__device__ __forceinline__ void dx_tile(const HeadArgs& h, const DxArgs& a, uint8_t* smem, uint32_t wg) {
    constexpr int TP = Loop::TP, TQ = Loop::TQ, NP = Loop::NP, NQ = Loop::NQ, WP = Loop::WP;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % WP, wq = wave / WP;
    const int64_t nh = (h.Hp + TQ - 1) / TQ;
    int64_t tp, tqs;
    if (!pick_tile(wg, ((STACKED ? a.pitch : *h.count) + TP - 1) / TP, nh * a.splits, tp, tqs)) return;
    const int64_t split = tqs / nh, p0 = tp * TP, q0 = (tqs - split * nh) * TQ;
    const int64_t all = h.vc / 64, each = (all + a.splits - 1) / a.splits;
    const int64_t s0 = split * each, s1 = s0 + each < all ? s0 + each : all;
    const int n = s1 > s0 ? (int)(s1 - s0) : 0;
    const int64_t rows = STACKED && a.pitch - p0 < TP ? a.pitch - p0 : TP;  // of g
    // this lane's rows of h, and its 4 adjacent rows of g in each tile
    const int64_t row = q0 + 16 * NQ * wq + (lane & 15);
    static_assert(!Loop::PERM, "tile i's rows follow tile i - 1's");
    float4v acc[NP][NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    // the small parts of g first, so that only the last pass rounds sums of full size
    const int64_t v = h.v0 + 64 * s0, hc = h.H - q0 < TQ ? (h.H > q0 ? h.H - q0 : 0) : TQ;
    Loop::run(
        acc, smem, n, STACKED ? 1 : a.terms,
        [&](int pass) {
            const uint16_t* g = h.g + ((STACKED ? 0 : (a.terms - 1 - pass) * h.Tp) + p0) * h.vc + 64 * s0;
            return Side{reinterpret_cast<const uint8_t*>(g), (rows * h.vc - 64 * s0) * 2, 128, (uint32_t)(2 * h.vc), (uint32_t)rows, 128};
        },
        [&](int) {
            return Side{h.w + v * h.ldw + 2 * q0, hc && h.V > v ? (h.V - v - 1) * h.ldw + 2 * hc : 0, 64 * h.ldw,
                        (uint32_t)h.ldw, (uint32_t)hc, 0};
        });
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        float* out = a.part + (split * h.Hp + row + 16 * j) * a.pitch + p0 + 16 * NP * wp + 4 * (lane >> 4);
        if (row + 16 * j < h.Hp) {
            auto on = [&](int i) { return !STACKED || 16 * (NP * wp + i) < rows; };
            if (!a.first) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    if (on(i)) acc[i][j] += *reinterpret_cast<const float4v*>(out + 16 * i);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (on(i)) *reinterpret_cast<float4v*>(out + 16 * i) = acc[i][j];
        }
    }
}

// dw: out[v][h] over the rows with a target, from their transposed copy.
struct DwArgs {
    const uint16_t* xt;  // [Hp][Tp]
    void* dw;
    int64_t ld;
    int terms;
};

template <class Loop, bool F32>
__device__ __forceinline__ void dw_tile(const HeadArgs& h, const DwArgs& a, uint8_t* smem, uint32_t wg) {
    constexpr int TP = Loop::TP, TQ = Loop::TQ, NP = Loop::NP, NQ = Loop::NQ;
    const int count = *h.count;
    int64_t tq, tp;
    if (!pick_tile(wg, h.vc / TQ, (h.Hp + TP - 1) / TP, tq, tp)) return;
    const int64_t q0 = tq * TQ, p0 = tp * TP;
    if (h.v0 + q0 >= h.V) return;
    const int n = (count + 63) / 64;
    float4v acc[NP][NQ];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j) acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t hc = h.Hp - p0 < TP ? h.Hp - p0 : TP, rows = 64 * (int64_t)n;
    Loop::run(
        acc, smem, n, a.terms,
        [&](int) {
            return Side{reinterpret_cast<const uint8_t*>(a.xt + p0 * h.Tp), hc * h.Tp * 2, 128, (uint32_t)(2 * h.Tp), (uint32_t)hc, 128};
        },
        [&](int pass) {
            return Side{reinterpret_cast<const uint8_t*>(h.g + (a.terms - 1 - pass) * h.Tp * h.vc + q0),
                        ((rows - 1) * h.vc + TQ) * 2, 128 * h.vc, (uint32_t)(2 * h.vc), TQ, 0};
        });
    typedef std::conditional_t<F32, float, uint16_t> O;
    O* out = static_cast<O*>(a.dw) + (h.v0 + q0) * a.ld + p0;
    const int64_t left = h.V - h.v0 - q0;
    store_tile<Loop, O, true>(acc, smem, h.H - p0, [&](int q) { return q < left ? out + q * a.ld : nullptr; });
}

// Both products of a piece in one launch: the first dx_grid workgroups are dx's, whose tiles are
// longer, the others dw's, which fill what those leave.  Bound by the matrix cores: both products of half of
// 4096 x 131072 x 7168 5.0 ms (1530 TFLOP/s, the matrix units 89% busy); the library's products of these
// two forms reach 887 and 1139.
template <class Loop, bool F32>
__global__ __launch_bounds__(64 * Loop::WAVES, 1) void k_grads(HeadArgs h, DxArgs x, DwArgs w, uint32_t dx_grid) {
    __shared__ __align__(1024) uint8_t smem[Loop::LDS];
    if (blockIdx.x < dx_grid) dx_tile<Loop, false>(h, x, smem, blockIdx.x);
    else dw_tile<Loop, F32>(h, w, smem, blockIdx.x - dx_grid);
}

// dx alone of 65 to 128 tokens: (100, 131072, 7168) 1310 us with dw, where 256 x 128 tiles beside dw, which read
// g twice as often, took 1655.
template <class Loop>
__global__ __launch_bounds__(64 * Loop::WAVES, 1) void k_dx_stacked(HeadArgs h, DxArgs x) {
    __shared__ __align__(1024) uint8_t smem[Loop::LDS];
    dx_tile<Loop, true>(h, x, smem, blockIdx.x);
}

// Rows of `bytes` bytes (a multiple of 16) at a pitch, zero.
__global__ __launch_bounds__(256) void k_zero(void* to, int64_t rows, int64_t bytes, int64_t pitch) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t b = 16 * threadIdx.x; b < bytes; b += 16 * 256)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(to) + r * pitch + b) = make_uint4(0, 0, 0, 0);
}

// dw of up to 64 KT tokens, on the caller's x: bound by its output.  A workgroup keeps 256
// columns of x as fragments and goes through 64-row tiles of dw, from `first` to `last`: the next tile's g
// is on its way while one is formed, and a tile goes out as whole lines through LDS: through what held its g
// (SHARE) where that makes a workgroup smaller, as it costs a barrier.
template <bool F32, int TERMS, int KT>
struct ThinDw {
    typedef Operand<256, true> OX;
    typedef Operand<64, true> OG;
    static constexpr int NP = 4, NQ = 4, ESZ = F32 ? 4 : 2, OUT = 64 * 256 * ESZ;
    static constexpr int G = TERMS * KT * OG::BYTES, MORE = OUT > G ? OUT : G;
    static constexpr bool SHARE = 2 * MORE < OUT + 2 * G;
    static constexpr int RING = SHARE ? 0 : OUT, BUF = SHARE ? MORE : G, LDS = RING + 2 * BUF;  // two buffers of g
    static_assert(OUT >= OX::BYTES && LDS <= 163840, "the columns of x fit where a tile goes out");

    __device__ static void run(const HeadArgs& h, const DwArgs& a, uint8_t* smem, int64_t p0, int first, int last) {
        const int lane = threadIdx.x & 63, g = lane >> 4;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        const int64_t hc = h.H - p0 < 256 ? h.H - p0 : 256;
        if (first >= last || hc <= 0) return;
        Feed<64, true, false, 2> feed_g[TERMS * KT];
#pragma unroll
        for (int u = 0; u < TERMS * KT; ++u) {
            const int term = u / KT, k0 = 64 * (u % KT);
            const int64_t row = term * h.Tp + k0, rows = h.Tp - k0 < 64 ? h.Tp - k0 : 64;
            feed_g[u].start(
                [&](int) {
                    return Side{reinterpret_cast<const uint8_t*>(h.g + row * h.vc + 64 * (int64_t)first),
                                ((rows - 1) * h.vc + 64 * (int64_t)(last - first)) * 2, 128, (uint32_t)(2 * h.vc), 64, 0};
                },
                last - first, 1, wave, lane, [&](int r) { return r < rows; });
        }
        auto send = [&](int i) {
#pragma unroll
            for (int u = 0; u < TERMS * KT; ++u) {
                feed_g[u].issue(0, lds0 + (uint32_t)(RING + (i & 1) * BUF + u * OG::BYTES), lane);
                feed_g[u].issue(1, lds0 + (uint32_t)(RING + (i & 1) * BUF + u * OG::BYTES), lane);
                feed_g[u].next([&](int) { return Side{}; });
            }
        };
        send(0);
        constexpr uint32_t X = SHARE ? BUF : 0;
        const uint32_t part_x[2] = {OX::lane_part(NP * wave, lane), 0}, part_g[2] = {OG::lane_part(0, lane), 0};
        bf16x8 P[KT][2][NP];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const int64_t k0 = 64 * k, rows = h.T - k0 < 64 ? h.T - k0 : 64;
            Feed<256, true, false, 8> feed_x;
            feed_x.start(
                [&](int) {
                    return Side{h.x + k0 * h.ldx + 2 * p0, rows > 0 ? (rows - 1) * h.ldx + 2 * hc : 0, 0, (uint32_t)h.ldx, (uint32_t)hc, 0};
                },
                1, 1, wave, lane, [&](int r) { return r < rows && h.live(k0 + r); });
#pragma unroll
            for (int i = 0; i < 8; ++i) feed_x.issue(i, lds0 + X, lane);
            wait_vmcnt<0>();
            block_barrier();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < NP; ++i) P[k][kk][i] = OX::frag(part_x, lds0 + X, i, kk);
            wait_lgkmcnt0();
            block_barrier();
        }
        constexpr int ROWB = 256 * ESZ, CHUNKS = ROWB / 16, STORES = 64 * CHUNKS / 256;
        for (int i = 0; i < last - first; ++i) {
            if (i > 0) wait_vmcnt<STORES>();  // this tile's g has landed (the last tile's stores may not have)
            block_barrier();
            const uint32_t at = lds0 + (uint32_t)(RING + (i & 1) * BUF);
            __attribute__((address_space(3))) uint8_t* lds = (__attribute__((address_space(3))) uint8_t*)(uintptr_t)(SHARE ? at : lds0);
            // The next tile's g (of the other buffer every wave has read what it needs): here, or
            // behind the products where there is no barrier before the tile goes out.  (100, 131072, 7168):
            // 1309 us, behind them 1390; (48, 32768, 2048), without SHARE: 95.0 here, 90.7 behind.
            if (SHARE && i + 1 < last - first) send(i + 1);
            float4v acc[NP][NQ];
#pragma unroll
            for (int x = 0; x < NP; ++x)
#pragma unroll
                for (int j = 0; j < NQ; ++j) acc[x][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = TERMS * KT - 1; u >= 0; --u) {
                bf16x8 Q[2][NQ];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int j = 0; j < NQ; ++j) Q[kk][j] = OG::frag(part_g, at + (uint32_t)(u * OG::BYTES), j, kk);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
#pragma unroll
                        for (int x = 0; x < NP; ++x) acc[x][j] = mfma16(P[u % KT][kk][x], Q[kk][j], acc[x][j]);
            }
            if (!SHARE && i + 1 < last - first) send(i + 1);
            if constexpr (SHARE) {
                wait_lgkmcnt0();
                block_barrier();  // (every wave has read g)
            }
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    const int q = 16 * j + (lane & 15);
                    const uint32_t b = (uint32_t)((64 * wave + 16 * x + 4 * g) * ESZ);
                    const uint32_t to = (uint32_t)(q * ROWB) + (((b >> 4) ^ (uint32_t)(q & 15)) << 4) + (b & 15u);
                    if constexpr (F32)
                        *(__attribute__((address_space(3))) float4v*)(lds + to) = acc[x][j];
                    else
                        *(__attribute__((address_space(3))) u32x2*)(lds + to) =
                            u32x2{pack_bf16x2(acc[x][j][0], acc[x][j][1]), pack_bf16x2(acc[x][j][2], acc[x][j][3])};
                }
            wait_lgkmcnt0();
            block_barrier();
            // (every store goes out, those past an edge to nowhere: the wait above counts them)
            const int64_t v = h.v0 + 64 * (int64_t)(first + i);
            const int64_t rows = h.V - v < 64 ? h.V - v : 64;
            const __amdgpu_buffer_rsrc_t ro = make_rsrc(uniform_ptr(static_cast<uint8_t*>(a.dw) + (v * a.ld + p0) * ESZ), 0x7FFFFFFFu);
#pragma unroll
            for (int k = 0; k < STORES; ++k) {
                const int item = k * 256 + threadIdx.x, q = item / CHUNKS, c = item % CHUNKS;
                const u32x4 x = *(const __attribute__((address_space(3))) u32x4*)(lds + q * ROWB + ((c ^ (q & 15)) << 4));
                const bool ok = q < rows && c * (16 / ESZ) < hc;
                __builtin_amdgcn_raw_buffer_store_b128(x, ro, ok ? (int)((uint32_t)q * (uint32_t)(a.ld * ESZ) + 16u * (uint32_t)c) : (int)OOB, 0, 2);
            }
            wait_lgkmcnt0();
            block_barrier();
        }
        wait_vmcnt<0>();
    }
};

// Both products of few tokens in one launch, bound by w, which dx reads, and dw: (48, 32768, 2048), 134 MB of
// each, 56 us (4.8 TB/s; a large copy 4.7).  The first dx_grid workgroups form dx from the stacked parts of
// g, the others dw, workgroup i the tiles from each * (i / blocks) on of column block i % blocks.
// (Without DX: dw alone.)
template <class DX, class DW>
__global__ __launch_bounds__(256, 1) void k_thin_grads(HeadArgs h, DxArgs x, DwArgs w, uint32_t dx_grid, int blocks, int tiles, int each) {
    constexpr bool BOTH = !std::is_void_v<DX>;
    constexpr int LDS = [] { if constexpr (BOTH) return DX::LDS > DW::LDS ? DX::LDS : DW::LDS; else return DW::LDS; }();
    __shared__ __align__(1024) uint8_t smem[LDS];
    if (BOTH && blockIdx.x < dx_grid) {
        if constexpr (BOTH) dx_tile<DX, true>(h, x, smem, blockIdx.x);
    } else {
        const int i = (int)(blockIdx.x - dx_grid), c = i / blocks, first = c * each;
        DW::run(h, w, smem, 256 * (int64_t)(i - c * blocks), first, first + each < tiles ? first + each : tiles);
    }
}

// dx of every token: the sums of the splits (and of the parts of g, where they are rows), transposed
// and rounded once; zeros where there is no target.  A workgroup takes 64 rows with a target, and the tokens
// of the same numbers that have none, 16 columns at a time: four tokens of a column a thread, and where those
// are fewer than the threads, several share the splits, and their sums are added in order.
// (48 tokens, 2048 columns, 32 sums: 6 us; with 64 columns a workgroup 12, with four times the rows of 16
// splits 27 instead of 12.  4096 x 2048, one sum each: the same.)
struct DxFinish {
    const float* part;
    int64_t Hp, pitch, stride;  // stride: from one part of g to the next
    int splits, terms;
    Live live;
    const int32_t *count, *rows, *pos;  // null: direct
    int64_t T, H;
    void* dx;
    int64_t ld;
};
template <bool F32>
__global__ __launch_bounds__(256) void k_dx_finish(DxFinish a) {
    __shared__ float s_t[64][17];
    __shared__ float4v s_part[256];
    const int64_t t0 = (int64_t)blockIdx.x * 64;
    const int64_t n = a.count ? *a.count : a.T;
    const int quads = (int)((a.stride - t0 < 64 ? a.stride - t0 : 64) / 4), items = 16 * quads, share = 256 / items;
    const int k = (int)threadIdx.x / items, it = (int)threadIdx.x - k * items, h = it / quads, q = 4 * (it - h * quads);
    // what this thread writes: 8 columns of a token with a sum, or of one without
    const int c = 8 * (threadIdx.x & 1), r = (threadIdx.x >> 1) & 63;
    bool zero = threadIdx.x >= 128, on;
    int64_t t = t0 + r;
    if (a.count) {
        on = zero ? t < a.T && a.pos[t] < 0 : t < n;
        if (on && !zero) t = a.rows[t];
    } else {
        on = !zero && t < a.T;
        zero = on && !a.live(t);
    }
    for (int64_t h0 = 16 * (int64_t)blockIdx.y; h0 < a.Hp; h0 += 16 * (int64_t)gridDim.y) {
        if (t0 < n) {
            float4v x = {0.0f, 0.0f, 0.0f, 0.0f};
            if (k < share) {
                // (the small parts of g first)
                for (int u = a.terms - 1; u >= 0; --u) {
                    const float* part = a.part + (h0 + h) * a.pitch + u * a.stride + t0 + q;
#pragma unroll 8
                    for (int s = k; s < a.splits; s += share) x += *reinterpret_cast<const float4v*>(part + s * a.Hp * a.pitch);
                }
            }
            if (share > 1) {
                s_part[threadIdx.x] = x;
                __syncthreads();
                if (k == 0)
                    for (int j = 1; j < share; ++j) x += s_part[threadIdx.x + j * items];
            }
            if (k == 0) {
#pragma unroll
                for (int v = 0; v < 4; ++v) s_t[q + v][h] = x[v];
            }
        }
        __syncthreads();
        if (on && h0 + c < a.H) {
            float x[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) x[v] = zero ? 0.0f : s_t[r][c + v];
            if constexpr (F32) {
                float4v* o = reinterpret_cast<float4v*>(static_cast<float*>(a.dx) + t * a.ld + h0 + c);
                o[0] = float4v{x[0], x[1], x[2], x[3]};
                o[1] = float4v{x[4], x[5], x[6], x[7]};
            } else {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dx) + t * a.ld + h0 + c) =
                    make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- host side

namespace {

// Tiles of the logits (columns x rows), of dx (rows of g x columns of h) and of dw (columns of h x rows of w).
// Logits64 has four stages of ring, two workgroups a compute unit: with three (64, 4096, 5000) takes 41.0 in place of
// 38.4 and (6, 68684, 936) 37.8 in place of 41.0, with six 41.6 and 55.0.
typedef TileLoop<4, 1, 1, 4, false, true, 4> Logits64;
typedef TileLoop<4, 1, 1, 4, false, true, 4, true> Logits64Stream;
typedef TileLoop<4, 4, 2, 2, false, true, 2> Logits128;
typedef TileLoop<4, 4, 2, 2, false, true, 2, true> Logits128Stream;
typedef WideLoop<false, true> Logits256;
template <int ROWS>  // of the stacked parts of g: up to 64 with 256 columns, else with 128
using Stacked = TileLoop<(ROWS > 64 ? ROWS / 32 : ROWS / 16), 4, (ROWS > 64 ? 2 : 1), (ROWS > 64 ? 2 : 4), true, false, 2>;
typedef TileLoop<4, 4, 2, 2, true, false, 2> Grad128;
typedef WideLoop<true, false> Grad256;

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tokens: 256 rows of the transposed copy stay below 2^31 bytes, and dw, a sum of tokens / 32 matrix instructions
// one after the other, keeps an error of about sqrt(tokens / 32) 2^-23 = 2e-5 of its size.
constexpr int64_t MAX_TOKENS = (int64_t)1 << 20, MAX_VOCAB = (int64_t)1 << 29, MAX_HIDDEN = (int64_t)1 << 20;
// Within these every grid has less than 2^23 tiles (and less than 2^32 threads).
constexpr int64_t MAX_LOGITS = (int64_t)1 << 38, MAX_X = (int64_t)1 << 35, MAX_W = (int64_t)1 << 38;
constexpr int64_t MAX_PITCH = (int64_t)1 << 21;     // 256 rows of it stay below 2^31 bytes
constexpr int64_t THIN = 128;                       // tokens up to which the products may take the caller's x (plan)
constexpr int64_t PAIR = 256;                       // tokens up to which g is a pair of bf16 for bf16 outputs
// Of g, which stays behind the last-level cache at any size: small pieces cost uneven last rounds of tiles. 8192 x 32768 x 2048
// with f32 gradients: 7867 us with 256 MiB, 5432 with 512, 5418 with 1024; 16384 x 32768 x 2048: 4842, 4752, 4696.
constexpr int64_t PIECE_BYTES = (int64_t)512 << 20;
constexpr int64_t CUS = 256;
constexpr int64_t LAST_LEVEL_CACHE = (int64_t)256 << 20;

// How a call is laid out in its workspace; every part starts on 256 bytes.
struct Plan {
    int64_t Tp, Hp, blocks, vc;
    int block;     // columns of a tile of the logits: 64, 128, 256
    int dx_tile, dw_tile;
    int splits;
    bool thin;
    size_t count, rows, pos, xc, xt, part, zat, sid, sslot, sq, tab, qsum, g, dx, bytes;
};

// Size of the tiles of an m x n output with a short reduction: the large ones where they fill most of the compute units.
// Logits of 128 and 256: (400, 8000, 1024) 25.8 and 32.9 us, (3000, 2000, 4096) 75 and 87; (400, 32000, 4096) 146 and 101,
// (800, 16000, 1024) 46 and 40.  dw: (400, 8000, 1024) 37.6 and 40.4, (1500, 4000, 2048) 73.6 and 74.5.
int tile_of(int64_t m, int64_t n) {
    return up(m, 256) / 256 * (up(n, 256) / 256) >= CUS * 3 / 4 ? 256 : 128;
}
// Columns of a tile of the logits.  64 and 128: (80, 8000, 2048) 25.3 and 35.1 us, (200, 4588, 736) 18.5 and 22.4; (100, 32000,
// 2048) 46.6 and 37.9, (200, 16384, 2048) 47.0 and 37.8; 128 and 256 of 65 to 128 tokens: (100, 131072, 7168) 368 and 416.
int logits_tile(int64_t T, int64_t V) {
    if (T <= 64 || up(T, 64) / 64 * (up(V, 64) / 64) <= 2 * CUS) return 64;
    return T <= 128 ? 128 : tile_of(T, V);
}

Plan plan(int64_t T, int64_t H, int64_t V, int K, unsigned flags, int terms, int dx_terms) {
    Plan p{};
    size_t at = 0;
    auto take = [&](int64_t n) {
        const size_t r = at;
        at += (size_t)up(n, 256);
        return r;
    };
    // The gradients of more than 64 tokens only where the work of dx, in stages of 256 x 256 tiles, is large, else a
    // copy pays.  (128, 20000, 512): 65 us on x, 51 with the copy; (100, 11000, 1344): 71, 69; (70, 40000, 1024): 103,
    // 115; (100, 131072, 7168): 1310, 1846.  Up to 64 always: (50, 8000, 600): 31, 37; (64, 20000, 512): 41, 45.  The
    // forward always: (100, 131072, 7168) 338, 370.
    p.thin = T <= THIN / 2 || (T <= THIN && (!flags || up(V, 256) / 64 * (up(H, 256) / 256) >= 8 * CUS));
    p.Tp = !p.thin ? up(T, 256) : T <= 16 ? up(T, 16) : T <= 32 ? 32 : T <= 64 ? 64 : 128;
    p.Hp = up(H, 64);
    p.block = logits_tile(T, V);
    p.blocks = (V + p.block - 1) / p.block;
    if (p.thin) {
        p.xc = take(2 * T * p.Hp);
    } else {
        p.count = take(4);
        p.rows = take(4 * p.Tp);
        p.pos = take(4 * p.Tp);
        p.xc = take(2 * p.Tp * p.Hp);
        if (flags & BSQ_WGRAD) p.xt = take(2 * p.Hp * p.Tp);
    }
    if (K) {
        p.sid = take(4 * T * K);
        p.sslot = take(4 * T * K);
        p.sq = take(4 * T * K);
        p.tab = take(2 * T * (p.blocks + 1));
        p.qsum = take(4 * T);
    }
    if (!flags) {
        p.part = take(8 * p.blocks * p.Tp);
        p.zat = take(4 * p.Tp);
    } else {
        // pieces of about the same width
        const int64_t most = std::max<int64_t>(256, PIECE_BYTES / (2 * terms * std::max<int64_t>(p.Tp, 16)) / 256 * 256);
        const int64_t pieces = (V + most - 1) / most;
        p.vc = up((V + pieces - 1) / pieces, 256);
        p.g = take(2 * terms * p.Tp * p.vc);
        p.dw_tile = tile_of(p.vc, H);
        if (flags & BSQ_DGRAD) {
            const int64_t steps = p.vc / 64;
            // dx: a tile's reduction is long, so its work counts, not the tiles.  128 and 256: (400, 8000, 1024), 512 stages
            // of such tiles, 49.0 and 54.6 us; (200, 16384, 2048), 2048 of them, 85.6 and 84.7; (1500, 4000, 2048), 3024,
            // 93.4 and 86.6.
            const int64_t work = steps * (up(p.Hp, 256) / 256), rows = dx_terms * p.Tp;
            int64_t down = 1;  // rows of tiles
            if (!p.thin) {
                p.dx_tile = work * (up(T, 256) / 256) >= 8 * CUS ? 256 : 128;
                down = up(T, p.dx_tile) / p.dx_tile;
            } else if (p.Tp > 64) {
                p.dx_tile = 256;
                down = up(rows, 256) / 256;
            } else {
                p.dx_tile = rows > 64 ? 128 : 256;  // (Stacked's)
            }
            const int64_t tiles = down * (up(p.Hp, p.dx_tile) / p.dx_tile);
            const int64_t places = p.thin || p.dx_tile == 256 ? CUS : 2 * CUS;
            // Stages a split: fewer make the sum over the splits dearer than they save.  For 4 and 8,
            // (10, 11000, 1344) takes 41.9 and 37.4 us, (50, 8000, 600) 40.3 and 33.8, (400, 9000, 1024) 68.6 and
            // 68.4; for 16 (1, 46563, 864) takes 67.2 in place of 62.3.
            const int64_t least = 8;
            p.splits = (int)std::min<int64_t>(std::max<int64_t>(1, places / std::max<int64_t>(tiles, 1)), std::max<int64_t>(1, steps / least));
            p.dx = take(4 * p.splits * p.Tp * (p.thin ? dx_terms : 1) * p.Hp);
        }
    }
    p.bytes = at;
    return p;
}

bool sizes_ok(int64_t T, int64_t H, int64_t V, int64_t K) {
    return T <= MAX_TOKENS && H <= MAX_HIDDEN && V <= MAX_VOCAB && K <= MAX_LIST && H % 8 == 0 && T * V <= MAX_LOGITS &&
           T * H <= MAX_X && V * H <= MAX_W;
}

// Everything a call may ask for.
struct Call {
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw, T, H, V;
    float scale;
    const int32_t* labels;                                                 // cross entropy
    const int32_t* ids; const void* tl; int tl_f32; const float* tlse; float tscale; int K;  // distillation
    float *loss, *lse, *logits;                                            // forward
    const float *lse_in, *dloss, *dlse;                                    // backward
    bool list, back;
    unsigned flags;
    void* dx; int64_t lddx; int dx_f32;
    void* dw; int64_t lddw; int dw_f32;
};

#define BSQ_TRY(...) do { const bsq_status st_ = (__VA_ARGS__); if (st_ != BSQ_OK) return st_; } while (0)

template <class... A, class... B>
bsq_status go(void (*kernel)(A...), dim3 grid, int threads, hipStream_t s, B... args) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, args...);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}
dim3 wide(int64_t n) { return dim3((unsigned)up(n, 8)); }

template <bool BACK, bool LIST>
bsq_status logits(const HeadArgs& h, const Plan& p, int64_t columns, hipStream_t s) {
    const int64_t tile = p.block, n = (h.T + tile - 1) / tile * ((columns + tile - 1) / tile);
    if (p.thin) {
        // Weights that do not stay in the last-level cache until the next read: (64, 131072, 7168) 342.6 us, 361.0 without
        // the hint; with it (48, 32768, 2048), whose 134 MB do stay, takes 37.3 in place of 32.8.
        const bool stream = h.V * h.ldw > LAST_LEVEL_CACHE;
        if (tile == 64 && stream) return go(k_logits<Logits64Stream, BACK, LIST, true>, wide(n), 256, s, h);
        if (tile == 64) return go(k_logits<Logits64, BACK, LIST, true>, wide(n), 256, s, h);
        if (stream) return go(k_logits<Logits128Stream, BACK, LIST, true>, wide(n), 256, s, h);
        return go(k_logits<Logits128, BACK, LIST, true>, wide(n), 256, s, h);
    }
    if (tile == 64) return go(k_logits<Logits64, BACK, LIST, false>, wide(n), 256, s, h);
    if (tile == 128) return go(k_logits<Logits128, BACK, LIST, false>, wide(n), 256, s, h);
    return go(k_logits<Logits256, BACK, LIST, false>, wide(n), 512, s, h);
}

template <bool LIST>
bsq_status finish(const FinishArgs& f, int block, hipStream_t s) {
    const unsigned g8 = (unsigned)((f.T + 7) / 8), g4 = (unsigned)((f.T + 3) / 4);
    if (block == 64) return go(k_finish<64, LIST>, dim3(g4), 256, s, f);
    if (block == 128) return go(k_finish<128, LIST>, dim3(g4), 256, s, f);
    return go(k_finish<256, LIST>, dim3(g8), 256, s, f);
}

template <class DX, class DW>
bsq_status thin_grads(const HeadArgs& h, const DxArgs& x, const DwArgs& w, const Plan& p, unsigned flags, hipStream_t s) {
    int64_t dx = 0, lds = DW::LDS;
    if constexpr (!std::is_void_v<DX>) {
        if (flags & BSQ_DGRAD) dx = up(up(p.Hp, DX::TQ) / DX::TQ * p.splits, 8);
        lds = std::max<int64_t>(lds, DX::LDS);
    }
    const int64_t tiles = (std::min(h.vc, h.V - h.v0) + 63) / 64, blocks = up(p.Hp, 256) / 256;
    // dw: as many workgroups as run at once
    const int64_t at_once = CUS * (163840 / lds), each = std::max<int64_t>(1, (tiles * blocks + at_once - 1) / at_once);
    const int64_t dw = flags & BSQ_WGRAD ? (tiles + each - 1) / each * blocks : 0;
    return go(k_thin_grads<DX, DW>, dim3((unsigned)(dx + dw)), 256, s, h, x, w, (uint32_t)dx, (int)blocks, (int)tiles, (int)each);
}

template <bool F32>
bsq_status grads(const HeadArgs& h, const DxArgs& x, const DwArgs& w, const Plan& p, unsigned flags, hipStream_t s) {
    if (p.thin) {
        constexpr int TERMS = F32 ? 3 : 2;  // parts of g that dw takes
        typedef ThinDw<F32, TERMS, 1> DW;
        const int64_t rows = x.pitch;
        if (p.Tp <= 64) {
            if (rows > 128) return thin_grads<Stacked<192>, DW>(h, x, w, p, flags, s);
            if (rows > 64) return thin_grads<Stacked<128>, DW>(h, x, w, p, flags, s);
            if (rows > 32) return thin_grads<Stacked<64>, DW>(h, x, w, p, flags, s);
            return thin_grads<Stacked<32>, DW>(h, x, w, p, flags, s);
        }
        typedef ThinDw<F32, TERMS, 2> DW2;
        if (flags & BSQ_DGRAD)
            BSQ_TRY(go(k_dx_stacked<Grad256>, wide((rows + 255) / 256 * (up(p.Hp, 256) / 256) * p.splits), 512, s, h, x));
        return flags & BSQ_WGRAD ? thin_grads<void, DW2>(h, x, w, p, flags, s) : BSQ_OK;
    }
    auto both = [&](auto kernel, int64_t tile, int threads, unsigned which) {
        const int64_t dx = which & BSQ_DGRAD ? up((h.T + tile - 1) / tile * (up(p.Hp, tile) / tile) * p.splits, 8) : 0;
        const int64_t dw = which & BSQ_WGRAD ? up(h.vc / tile * (up(p.Hp, tile) / tile), 8) : 0;
        return go(kernel, wide(dx + dw), threads, s, h, x, w, (uint32_t)dx);
    };
    unsigned big = 0;  // the products that take 256 x 256 tiles
    if ((flags & BSQ_DGRAD) && p.dx_tile == 256) big |= BSQ_DGRAD;
    if ((flags & BSQ_WGRAD) && p.dw_tile == 256) big |= BSQ_WGRAD;
    if (big) BSQ_TRY(both(k_grads<Grad256, F32>, 256, 512, big));
    if (flags & ~big) return both(k_grads<Grad128, F32>, 128, 256, flags & ~big);
    return BSQ_OK;
}

bsq_status run(const Call& c, void* workspace, size_t workspace_bytes, hipStream_t s) {
    const int low = c.T <= PAIR ? 2 : 1, dx_terms = c.dx_f32 ? 3 : low, dw_terms = c.dw_f32 ? 3 : low;
    const int terms = std::max(c.flags & BSQ_DGRAD ? dx_terms : low, c.flags & BSQ_WGRAD ? dw_terms : low);
    const Plan p = plan(c.T, c.H, c.V, c.K, c.flags, terms, dx_terms);
    if (workspace_bytes < p.bytes) return BSQ_ERR_WORKSPACE_TOO_SMALL;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool list = c.K > 0;
    auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    uint16_t* tab = reinterpret_cast<uint16_t*>(ws + p.tab);

    if (c.T > 0 && list) {
        const ListArgs a{c.ids, c.tl, c.tl_f32, c.tlse, c.tscale, c.T, c.V, c.K, p.block, p.blocks, i32(p.sid),
                         i32(p.sslot), f32(p.sq), tab, f32(p.qsum), c.logits};
        BSQ_TRY(go(k_lists, dim3((unsigned)((c.T + 3) / 4)), 256, s, a));
    }
    HeadArgs h{};
    h.w = static_cast<const uint8_t*>(c.w);
    h.ldw = 2 * c.ldw;
    h.V = c.V; h.H = c.H; h.T = c.T; h.Hp = p.Hp; h.Tp = p.Tp;
    h.scale = c.scale;
    h.live = Live{c.labels, list ? f32(p.qsum) : nullptr, c.dloss, c.dlse, c.flags != 0, c.V, c.T};
    h.K = c.K; h.sid = i32(p.sid); h.sslot = i32(p.sslot); h.sq = f32(p.sq); h.tab = tab; h.blocks = p.blocks;
    if (p.thin) {
        h.x = static_cast<const uint8_t*>(c.x);
        h.ldx = 2 * c.ldx;
        if (c.T > 0 && c.ldx > MAX_PITCH) {
            BSQ_TRY(go(k_pack_rows, dim3((unsigned)c.T, (unsigned)((c.H + 2047) / 2048)), 256, s, static_cast<const uint16_t*>(c.x),
                       c.ldx, c.H, reinterpret_cast<uint16_t*>(ws + p.xc), p.Hp));
            h.x = ws + p.xc;
            h.ldx = 2 * p.Hp;
        }
    } else {
        h.x = ws + p.xc;
        h.ldx = 2 * p.Hp;
        h.count = i32(p.count);
        h.rows = i32(p.rows);
        const RowsArgs r{h.live, c.T, p.Tp, c.H, p.Hp, static_cast<const uint16_t*>(c.x), c.ldx, i32(p.count), i32(p.rows),
                         i32(p.pos), reinterpret_cast<uint16_t*>(ws + p.xc),
                         c.flags & BSQ_WGRAD ? reinterpret_cast<uint16_t*>(ws + p.xt) : nullptr};
        const dim3 grid((unsigned)(p.Tp / 64), (unsigned)(p.Hp / 64));
        if (c.T <= ROWS_SELF) {
            BSQ_TRY(go(k_copy_rows<true>, grid, 256, s, r));
        } else {
            BSQ_TRY(go(k_rows, dim3(1), 1024, s, r));
            BSQ_TRY(go(k_copy_rows<false>, grid, 256, s, r));
        }
    }

    if (!c.flags) {
        h.part = reinterpret_cast<float2*>(ws + p.part);
        h.zat = f32(p.zat);
        h.logits = c.logits;
        const float kappa = c.scale * LOG2E;
        const int far = (int)std::ceil(std::log2((double)c.scale * LOG2E));
        h.far_key = std::ldexp(1.0f, far - 20);
        const float far_unit = std::ldexp(1.0f, 20 - far);
        const double unit = (double)c.scale / kappa;
        BSQ_TRY(list ? logits<false, true>(h, p, c.V, s) : logits<false, false>(h, p, c.V, s));
        const FinishArgs f{h.part, p.blocks, p.Tp, c.T, c.scale, far_unit, unit, h.live, p.thin ? nullptr : i32(p.pos), h.zat, c.K, h.sslot, h.sq,
                           tab, c.logits, c.loss, c.lse};
        return list ? finish<true>(f, p.block, s) : finish<false>(f, p.block, s);
    }

    h.lse = c.lse_in;
    h.g = reinterpret_cast<uint16_t*>(ws + p.g);
    h.vc = p.vc;  // (the last piece's columns past the vocabulary are zero)
    h.terms = terms;
    if (c.T == 0) {  // dw is zero
        return c.flags & BSQ_WGRAD ? go(k_zero, dim3((unsigned)std::min<int64_t>(c.V, 65536)), 256, s, c.dw, c.V,
                                        c.H * (c.dw_f32 ? 4 : 2), c.lddw * (c.dw_f32 ? 4 : 2))
                                   : BSQ_OK;
    }
    const DwArgs w{reinterpret_cast<const uint16_t*>(ws + p.xt), c.dw, c.lddw, dw_terms};
    for (h.v0 = 0; h.v0 < c.V; h.v0 += p.vc) {
        BSQ_TRY(list ? logits<true, true>(h, p, p.vc, s) : logits<true, false>(h, p, p.vc, s));
        const DxArgs x{f32(p.dx), p.Tp * (p.thin ? dx_terms : 1), p.splits, h.v0 == 0, dx_terms};
        BSQ_TRY(c.dw_f32 ? grads<true>(h, x, w, p, c.flags, s) : grads<false>(h, x, w, p, c.flags, s));
    }
    if (c.flags & BSQ_DGRAD) {
        const DxFinish f{f32(p.dx), p.Hp, p.Tp * (p.thin ? dx_terms : 1), p.Tp, p.splits, p.thin ? dx_terms : 1, h.live,
                         h.count, h.rows, p.thin ? nullptr : i32(p.pos), c.T, c.H, c.dx, c.lddx};
        const int64_t rows = (c.T + 63) / 64;
        const dim3 grid((unsigned)rows, (unsigned)std::min<int64_t>(p.Hp / 16, std::max<int64_t>(1, 32768 / rows)));
        return c.dx_f32 ? go(k_dx_finish<true>, grid, 256, s, f) : go(k_dx_finish<false>, grid, 256, s, f);
    }
    return BSQ_OK;
}

bool grad_type(bsq_dtype t) { return t == BSQ_BF16 || t == BSQ_F32; }

// What a call's arguments have to be, all of it before anything is enqueued: first what is invalid, then
// what is not supported.
bsq_status check(const Call& c, const void* workspace, bsq_dtype teacher, bsq_dtype dx_dtype, bsq_dtype dw_dtype) {
    const bool back = c.back, dg = c.flags & BSQ_DGRAD, wg = c.flags & BSQ_WGRAD, some = c.T > 0;
    if (c.T < 0 || c.H <= 0 || c.V <= 0 || !(c.scale > 0.0f && c.scale < INFINITY)) return BSQ_ERR_INVALID_ARG;
    if (!workspace || !c.w || (some && !c.x) || c.ldx < c.H || c.ldw < c.H) return BSQ_ERR_INVALID_ARG;
    if (c.list) {
        if (c.K < 1 || !(c.tscale > 0.0f && c.tscale < INFINITY) || !grad_type(teacher)) return BSQ_ERR_INVALID_ARG;
        if (some && (!c.ids || !c.tl || (!back && !c.logits))) return BSQ_ERR_INVALID_ARG;
    } else if (some && !c.labels) {
        return BSQ_ERR_INVALID_ARG;
    }
    if (!back && some && (!c.loss || !c.lse)) return BSQ_ERR_INVALID_ARG;
    if (back) {
        if (c.flags == 0 || (c.flags & ~(BSQ_DGRAD | BSQ_WGRAD)) || (some && !c.lse_in)) return BSQ_ERR_INVALID_ARG;
        if (dg && (!grad_type(dx_dtype) || (some && !c.dx) || c.lddx < c.H)) return BSQ_ERR_INVALID_ARG;
        if (wg && (!grad_type(dw_dtype) || !c.dw || c.lddw < c.H)) return BSQ_ERR_INVALID_ARG;
    }
    if (!sizes_ok(c.T, c.H, c.V, c.K) || c.ldx % 8 || c.ldw % 8 || c.ldw > MAX_PITCH) return BSQ_ERR_UNSUPPORTED;
    if (!al(c.x, 16) || !al(c.w, 16) || !al(workspace, 256)) return BSQ_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)c.labels, (const void*)c.ids, (const void*)c.tlse, (const void*)c.loss, (const void*)c.lse,
                          (const void*)c.logits, (const void*)c.lse_in, (const void*)c.dloss, (const void*)c.dlse})
        if (!al(p, 4)) return BSQ_ERR_UNSUPPORTED;
    if (!al(c.tl, c.tl_f32 ? 4 : 2)) return BSQ_ERR_UNSUPPORTED;
    if (dg && (!al(c.dx, 16) || c.lddx % 8)) return BSQ_ERR_UNSUPPORTED;
    if (wg && (!al(c.dw, 16) || c.lddw % 8 || c.lddw > MAX_PITCH)) return BSQ_ERR_UNSUPPORTED;
    return BSQ_OK;
}

}  // namespace
}  // namespace bsq

extern "C" {

size_t bsq_linear_loss_workspace_size(int64_t tokens, int64_t hidden, int64_t vocab, int32_t top_k, unsigned flags,
                                      bsq_dtype grad_dtype) {
    if (tokens < 0 || hidden <= 0 || vocab <= 0 || top_k < 0 || (flags & ~(BSQ_DGRAD | BSQ_WGRAD))) return 0;
    if (!bsq::sizes_ok(tokens, hidden, vocab, top_k)) return 0;
    const int low = tokens <= bsq::PAIR ? 2 : 1;
    auto bytes = [&](int terms, int dx_terms) { return bsq::plan(tokens, hidden, vocab, top_k, flags, terms, dx_terms).bytes; };
    size_t n = bytes(low, low);
    // (any mix of the two types: fewer rows of dx can be split further, and then need more)
    if (grad_dtype == BSQ_F32) n = std::max({n, bytes(3, low), bytes(3, 3)});
    return n ? n : 256;
}

bsq_status bsq_linear_ce(const void* x_bf16, int64_t ld_x, const void* w_bf16, int64_t ld_w, const int32_t* labels,
                         int64_t tokens, int64_t hidden, int64_t vocab, float scale, float* loss, float* lse,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
    bsq::Call c{};
    c.x = x_bf16; c.ldx = ld_x; c.w = w_bf16; c.ldw = ld_w; c.T = tokens; c.H = hidden; c.V = vocab; c.scale = scale;
    c.labels = labels; c.loss = loss; c.lse = lse;
    BSQ_TRY(bsq::check(c, workspace, BSQ_F32, BSQ_F32, BSQ_F32));
    if (tokens == 0) return BSQ_OK;
    return bsq::run(c, workspace, workspace_bytes, stream);
}

bsq_status bsq_linear_ce_bwd(const void* x_bf16, int64_t ld_x, const void* w_bf16, int64_t ld_w, const int32_t* labels,
                             int64_t tokens, int64_t hidden, int64_t vocab, float scale, const float* lse,
                             const float* dloss, const float* dlse, void* dx, bsq_dtype dx_dtype, int64_t ld_dx, void* dw,
                             bsq_dtype dw_dtype, int64_t ld_dw, unsigned flags, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    bsq::Call c{};
    c.x = x_bf16; c.ldx = ld_x; c.w = w_bf16; c.ldw = ld_w; c.T = tokens; c.H = hidden; c.V = vocab; c.scale = scale;
    c.labels = labels; c.lse_in = lse; c.dloss = dloss; c.dlse = dlse; c.flags = flags;
    c.dx = dx; c.lddx = ld_dx; c.dx_f32 = dx_dtype == BSQ_F32; c.dw = dw; c.lddw = ld_dw; c.dw_f32 = dw_dtype == BSQ_F32;
    c.back = true;
    BSQ_TRY(bsq::check(c, workspace, BSQ_F32, dx_dtype, dw_dtype));
    return bsq::run(c, workspace, workspace_bytes, stream);
}

bsq_status bsq_linear_distill(const void* x_bf16, int64_t ld_x, const void* w_bf16, int64_t ld_w, const int32_t* teacher_ids,
                              const void* teacher_logits, bsq_dtype teacher_dtype, const float* teacher_lse, int32_t top_k,
                              int64_t tokens, int64_t hidden, int64_t vocab, float scale, float teacher_scale, float* loss,
                              float* lse, float* logits, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    bsq::Call c{};
    c.x = x_bf16; c.ldx = ld_x; c.w = w_bf16; c.ldw = ld_w; c.T = tokens; c.H = hidden; c.V = vocab; c.scale = scale;
    c.ids = teacher_ids; c.tl = teacher_logits; c.tl_f32 = teacher_dtype == BSQ_F32; c.tlse = teacher_lse;
    c.tscale = teacher_scale; c.K = top_k; c.loss = loss; c.lse = lse; c.logits = logits;
    c.list = true;
    BSQ_TRY(bsq::check(c, workspace, teacher_dtype, BSQ_F32, BSQ_F32));
    if (tokens == 0) return BSQ_OK;
    return bsq::run(c, workspace, workspace_bytes, stream);
}

bsq_status bsq_linear_distill_bwd(const void* x_bf16, int64_t ld_x, const void* w_bf16, int64_t ld_w,
                                  const int32_t* teacher_ids, const void* teacher_logits, bsq_dtype teacher_dtype,
                                  const float* teacher_lse, int32_t top_k, int64_t tokens, int64_t hidden, int64_t vocab,
                                  float scale, float teacher_scale, const float* lse, const float* dloss, const float* dlse,
                                  void* dx, bsq_dtype dx_dtype, int64_t ld_dx, void* dw, bsq_dtype dw_dtype, int64_t ld_dw,
                                  unsigned flags, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    bsq::Call c{};
    c.x = x_bf16; c.ldx = ld_x; c.w = w_bf16; c.ldw = ld_w; c.T = tokens; c.H = hidden; c.V = vocab; c.scale = scale;
    c.ids = teacher_ids; c.tl = teacher_logits; c.tl_f32 = teacher_dtype == BSQ_F32; c.tlse = teacher_lse;
    c.tscale = teacher_scale; c.K = top_k; c.lse_in = lse; c.dloss = dloss; c.dlse = dlse; c.flags = flags;
    c.dx = dx; c.lddx = ld_dx; c.dx_f32 = dx_dtype == BSQ_F32; c.dw = dw; c.lddw = ld_dw; c.dw_f32 = dw_dtype == BSQ_F32;
    c.list = c.back = true;
    BSQ_TRY(bsq::check(c, workspace, teacher_dtype, dx_dtype, dw_dtype));
    return bsq::run(c, workspace, workspace_bytes, stream);
}

}  // extern "C"
