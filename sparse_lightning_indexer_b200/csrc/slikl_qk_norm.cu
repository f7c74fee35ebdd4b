// q and k from the projections' outputs (norm of each head, position rotation, 8-bit checkpoint)
// and the gradient back to them: slikl_qk_norm_rope, slikl_qk_norm_rope_grad and
// slikl_grad_projected (formulas and contract in include/slikl.h).
//
// Both kernels are bound by HBM: an element costs 2 + 2 bytes (1 more each way for a checkpoint)
// against some twenty instructions. A head row of D values is held by D/16 threads, 16 values each,
// as two 8-value chunks that the rotation by halves pairs with each other: thread l of the first
// rot_dim/16 takes chunks l and l + rot_dim/16, the others two neighbouring chunks behind the
// rotated dims. So every load and store is 16 bytes a thread (8 for e4m3), the rotation needs no
// exchange between threads, and the norm's sums cross at most 8 lanes by shuffles. Statistics,
// products and sums are fp32; y and dx are rounded once.
#include <cuda_fp8.h>
#include <float.h>

#include <algorithm>

#include "slikl_sm100.cuh"

namespace slikl {
namespace {

using sm100::pack2;
using sm100::unpack2;

// Division of a row number below 2^31 by a fixed number: n / d = (n * m) >> (31 + s) with
// m = floor(2^(31+s) / d) + 1 and 2^(s-1) < d <= 2^s. The error of m is at most d, so that of the
// product is below n * d < 2^(31+s), too small to reach the next quotient.
struct FastDiv {
    uint32_t d, m, s;
};

FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    if (d > 1) f.m = (uint32_t)((1ull << (31 + f.s)) / d + 1);
    return f;
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
    return f.d == 1 ? n : __umulhi(n, f.m) >> (f.s - 1);
}

struct Side {
    uint32_t rows;            // head rows T * N
    FastDiv N, S;
    int norm;
    int64_t x_stride, dx_stride;
    const void *x;
    const uint8_t *x8;
    const float *x8_scale;
    const int32_t *positions;
    const float *gain, *bias;
    void *y;
    uint8_t *keep8;
    float *keep8_scale;
    const void *dy;
    void *dx;
};

struct Args {
    Side side[2];             // q, k
    uint32_t blocks_q;        // blocks of the q side; the others are the k side's
    uint32_t blocks_k;
    int rot, pairs;           // rotated dims; neighbours (1) or halves (0)
    uint32_t table_rows;
    float eps;
    const float *cos_sin;
    uint32_t *status;
    float *partial;           // gradient: [4][blocks][D] sums of dgain, dbias of q, dgain, dbias of k
};

constexpr int kThreads = 256;
constexpr int kGradBlocks = 592;      // most blocks of the gradient kernel (the workspace's size)

// What one thread of a head row is responsible for.
struct Lane {
    int ca, cb;               // first dims of its two chunks of 8
    int ta, tb;               // their places in the table's cosines (angle of the chunk's first
                              // value; 8 from ta for halves, 4 from ta and 4 from tb for pairs)
    bool turns;               // rotated dims
};

__device__ __forceinline__ Lane lane_of(int l, int rot, int pairs) {
    Lane t;
    const int half = rot / 16;
    t.turns = l < half;
    t.ca = t.turns ? 8 * l : rot + 16 * (l - half);
    t.cb = t.turns ? t.ca + rot / 2 : t.ca + 8;
    t.ta = pairs ? 4 * l : 8 * l;
    t.tb = pairs ? 4 * l + rot / 4 : t.ta + 4;
    return t;
}

// Position of head row r's token; false for padding and (flagged) for a bad position.
__device__ __forceinline__ bool position_of(const Args &a, const Side &s, uint32_t token,
                                            uint32_t &pos) {
    if (s.positions) {
        const int32_t p = s.positions[token];
        pos = (uint32_t)p;
        if (p < 0 || (a.rot && pos >= a.table_rows)) {
            if (p != -1 && a.status) set_status(a.status, SLIKL_DEV_BAD_POSITION);
            return false;
        }
        return true;
    }
    pos = token - div_by(token, s.S) * s.S.d;
    if (a.rot && pos >= a.table_rows) {
        if (a.status) set_status(a.status, SLIKL_DEV_BAD_POSITION);
        return false;
    }
    return true;
}

__device__ __forceinline__ void load_angles(const Args &a, const Lane &t, uint32_t pos, float *c,
                                            float *s) {
    if (!t.turns) return;
    const float *row = a.cos_sin + (int64_t)pos * a.rot;
    const float4 c0 = *reinterpret_cast<const float4 *>(row + t.ta);
    const float4 c1 = *reinterpret_cast<const float4 *>(row + t.tb);
    const float4 s0 = *reinterpret_cast<const float4 *>(row + a.rot / 2 + t.ta);
    const float4 s1 = *reinterpret_cast<const float4 *>(row + a.rot / 2 + t.tb);
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
    c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
    s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
}

// v[0..8) is the thread's first chunk, v[8..16) its second; sign -1 turns back.
__device__ __forceinline__ void turn(float *v, const float *c, const float *s, int pairs,
                                     float sign) {
    if (pairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = v[2 * i], y = v[2 * i + 1], sn = sign * s[i];
            v[2 * i] = x * c[i] - y * sn;
            v[2 * i + 1] = y * c[i] + x * sn;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = v[i], y = v[i + 8], sn = sign * s[i];
            v[i] = x * c[i] - y * sn;
            v[i + 8] = y * c[i] + x * sn;
        }
    }
}

template <typename T>
__device__ __forceinline__ void widen(const uint4 &a, const uint4 &b, float *v) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void widen8(const uint2 &a, const uint2 &b, float scale, float *v) {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * scale;
        v[2 * i + 1] = f.y * scale;
    }
}

template <typename T>
__device__ __forceinline__ void narrow_store(T *row, const Lane &t, const float *v) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(row + t.ca) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(row + t.cb) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Sum (or maximum) over the threads of a head row; every one gets the same bits.
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int TPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// x -> (x - m) r in place; returns r. The variance is taken about the mean, not as a difference
// of moments, so that a mean far above the deviation costs no digits.
template <int D, int NORM>
__device__ __forceinline__ float normalise(float *x, float eps) {
    if (NORM == SLIKL_NORM_NONE) return 1.f;
    constexpr int TPR = D / 16;
    if (NORM == SLIKL_NORM_LAYER) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m += x[i];
        m = row_sum<TPR>(m) * (1.f / D);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] -= m;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) q = fmaf(x[i], x[i], q);
    const float r = rsqrtf(fmaf(row_sum<TPR>(q), 1.f / D, eps));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= r;
    return r;
}

// The row of x (or of its checkpoint) as the thread's 16 values.
template <typename T, int D, bool SRC8>
struct Raw {
    uint4 a, b;
    uint2 a8, b8;
    float scale;
    __device__ __forceinline__ void load(const Side &s, uint32_t row, uint32_t token,
                                         const Lane &t) {
        if (SRC8) {
            const uint8_t *p = s.x8 + (int64_t)row * D;
            a8 = *reinterpret_cast<const uint2 *>(p + t.ca);
            b8 = *reinterpret_cast<const uint2 *>(p + t.cb);
            scale = s.x8_scale[row];
        } else {
            const T *p = static_cast<const T *>(s.x) + (int64_t)token * s.x_stride +
                         (row - token * s.N.d) * D;
            a = *reinterpret_cast<const uint4 *>(p + t.ca);
            b = *reinterpret_cast<const uint4 *>(p + t.cb);
        }
    }
    __device__ __forceinline__ void values(float *v) const {
        if (SRC8) widen8(a8, b8, scale, v);
        else widen<T>(a, b, v);
    }
};

__device__ __forceinline__ void load16(const float *p, const Lane &t, float *v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 *q = reinterpret_cast<const float4 *>(p + (h ? t.cb : t.ca));
        const float4 u = q[0], w = q[1];
        v[8 * h] = u.x; v[8 * h + 1] = u.y; v[8 * h + 2] = u.z; v[8 * h + 3] = u.w;
        v[8 * h + 4] = w.x; v[8 * h + 5] = w.y; v[8 * h + 6] = w.z; v[8 * h + 7] = w.w;
    }
}

// One e4m3 checkpoint row: scale = max|x| / 448, values x / scale (a product with the scale's
// reciprocal, which may round a value halfway between two codes the other way). Every lane of the
// warp has to come here (the maximum crosses lanes); rows that are not `in` are not stored.
template <int D>
__device__ __forceinline__ void keep_row(const Side &s, uint32_t row, const Lane &t, int l,
                                         bool in, bool live, const float *x) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
    top = row_max<D / 16>(top);
    if (!in) return;
    // a row of subnormal bf16 values keeps a normal scale, so that its reciprocal is finite
    const float scale = live && top > 0.f ? fmaxf(top / 448.f, FLT_MIN) : 0.f;
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    uint32_t w[4] = {0, 0, 0, 0};
    if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t two = __nv_cvt_float2_to_fp8x2(
                make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            w[i >> 1] |= two << (16 * (i & 1));
        }
    }
    uint8_t *p = s.keep8 + (int64_t)row * D;
    *reinterpret_cast<uint2 *>(p + t.ca) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(p + t.cb) = make_uint2(w[2], w[3]);
    if (l == 0) s.keep8_scale[row] = scale;
}

// Forward: each warp takes kFwdUnroll * 512 / D consecutive head rows, all of them loaded before
// the first is worked on.
constexpr int kFwdUnroll = 2;

template <typename T, int D, int NORM, bool SRC8>
__device__ __forceinline__ void forward_rows(const Args &a, const Side &s, uint32_t block) {
    constexpr int TPR = D / 16, RPW = 32 / TPR;
    const int lane = threadIdx.x & 31, l = lane % TPR;
    const Lane t = lane_of(l, a.rot, a.pairs);
    const uint32_t first = (block * (kThreads / 32) + (threadIdx.x >> 5)) * (RPW * kFwdUnroll) +
                           lane / TPR;
    Raw<T, D, SRC8> raw[kFwdUnroll];
    uint32_t token[kFwdUnroll];
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
        // rows behind the last one are worked on as copies of it and not stored
        const uint32_t row = min(first + u * RPW, s.rows - 1);
        token[u] = div_by(row, s.N);
        raw[u].load(s, row, token[u], t);
    }
    float gain[16], bias[16];
    if (NORM != SLIKL_NORM_NONE && s.gain) load16(s.gain, t, gain);
    if (NORM == SLIKL_NORM_LAYER && s.bias) load16(s.bias, t, bias);
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
        const uint32_t row = first + u * RPW;
        const bool in = row < s.rows;
        uint32_t pos = 0;
        const bool live = position_of(a, s, token[u], pos);
        float v[16];
        raw[u].values(v);
        if (!SRC8 && s.keep8) keep_row<D>(s, row, t, l, in, live, v);
        if (!s.y) continue;
        normalise<D, NORM>(v, a.eps);
        if (NORM != SLIKL_NORM_NONE && s.gain) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= gain[i];
        }
        if (NORM == SLIKL_NORM_LAYER && s.bias) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += bias[i];
        }
        if (!in) continue;
        if (!live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
        } else if (t.turns) {
            float c[8], sn[8];
            load_angles(a, t, pos, c, sn);
            turn(v, c, sn, a.pairs, 1.f);
        }
        narrow_store<T>(static_cast<T *>(s.y) + (int64_t)row * D, t, v);
    }
}

template <typename T, int D, bool SRC8>
__device__ __forceinline__ void forward_side(const Args &a, const Side &s, uint32_t block) {
    if (s.norm == SLIKL_NORM_RMS) forward_rows<T, D, SLIKL_NORM_RMS, SRC8>(a, s, block);
    else if (s.norm == SLIKL_NORM_LAYER) forward_rows<T, D, SLIKL_NORM_LAYER, SRC8>(a, s, block);
    else forward_rows<T, D, SLIKL_NORM_NONE, SRC8>(a, s, block);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_forward(const __grid_constant__ Args a) {
    const bool k = blockIdx.x >= a.blocks_q;
    const Side &s = a.side[k];
    const uint32_t block = blockIdx.x - (k ? a.blocks_q : 0);
    if (s.x) forward_side<T, D, false>(a, s, block);
    else forward_side<T, D, true>(a, s, block);
}

// Gradient: a block takes a contiguous share of the side's rows, its warps side by side, with the
// next rows' loads in flight while the present ones are worked on. The sums of dgain and dbias
// stay in registers over the whole share, are added over the block in a fixed order and stored;
// qk_grad_sums adds the blocks' sums, again in a fixed order.
template <typename T, int D, int NORM, bool SRC8>
__device__ __forceinline__ void gradient_rows(const Args &a, const Side &s, uint32_t block,
                                              uint32_t blocks, float *partial, float *smem) {
    constexpr int TPR = D / 16, RPW = 32 / TPR, WARPS = kThreads / 32, TILE = WARPS * RPW;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % TPR;
    const Lane t = lane_of(l, a.rot, a.pairs);
    const uint32_t tiles = (s.rows + TILE - 1) / TILE;
    const uint32_t begin = (uint32_t)((uint64_t)tiles * block / blocks);
    const uint32_t end = (uint32_t)((uint64_t)tiles * (block + 1) / blocks);
    float gain[16], dgain[16], dbias[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) gain[i] = 1.f, dgain[i] = 0.f, dbias[i] = 0.f;
    if (NORM != SLIKL_NORM_NONE && s.gain) load16(s.gain, t, gain);

    Raw<T, D, SRC8> x, x_next;
    uint4 ga, gb, ga_next, gb_next;
    uint32_t token = 0, token_next = 0;
    auto fetch = [&](uint32_t tile) {
        const uint32_t row = min(tile * TILE + warp * RPW + lane / TPR, s.rows - 1);
        token_next = div_by(row, s.N);
        if (NORM != SLIKL_NORM_NONE) x_next.load(s, row, token_next, t);
        const T *g = static_cast<const T *>(s.dy) + (int64_t)row * D;
        ga_next = *reinterpret_cast<const uint4 *>(g + t.ca);
        gb_next = *reinterpret_cast<const uint4 *>(g + t.cb);
    };
    if (begin < end) fetch(begin);
    for (uint32_t tile = begin; tile < end; ++tile) {
        x = x_next, ga = ga_next, gb = gb_next, token = token_next;
        const uint32_t row = tile * TILE + warp * RPW + lane / TPR;
        const bool in = row < s.rows;
        uint32_t pos = 0;
        const bool live = position_of(a, s, token, pos);
        float g[16];
        widen<T>(ga, gb, g);
        if (live && t.turns) {
            float c[8], sn[8];
            load_angles(a, t, pos, c, sn);
            turn(g, c, sn, a.pairs, -1.f);
        }
        if (tile + 1 < end) fetch(tile + 1);
        if (NORM != SLIKL_NORM_NONE) {
            float v[16];
            x.values(v);
            const float r = normalise<D, NORM>(v, a.eps);
            const bool counts = in && live;
            float su = 0.f, sv = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (counts) {
                    dgain[i] = fmaf(g[i], v[i], dgain[i]);
                    if (NORM == SLIKL_NORM_LAYER) dbias[i] += g[i];
                }
                g[i] *= gain[i];
                su += g[i];
                sv = fmaf(g[i], v[i], sv);
            }
            sv = row_sum<TPR>(sv) * (1.f / D);
            su = NORM == SLIKL_NORM_LAYER ? row_sum<TPR>(su) * (1.f / D) : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = r * (g[i] - su - v[i] * sv);
        }
        if (!in) continue;
        if (!live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = 0.f;
        }
        narrow_store<T>(static_cast<T *>(s.dx) + (int64_t)token * s.dx_stride +
                            (row - token * s.N.d) * D, t, g);
    }
    if constexpr (NORM != SLIKL_NORM_NONE) {
#pragma unroll
        for (int which = 0; which < (NORM == SLIKL_NORM_LAYER ? 2 : 1); ++which) {
            float *acc = which ? dbias : dgain;
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int o = 16; o >= TPR; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (lane < TPR) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    smem[warp * D + t.ca + i] = acc[i];
                    smem[warp * D + t.cb + i] = acc[8 + i];
                }
            }
            __syncthreads();
            if (threadIdx.x < D) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) sum += smem[w * D + threadIdx.x];
                partial[((int64_t)which * kGradBlocks + block) * D + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

template <typename T, int D, bool SRC8>
__device__ __forceinline__ void gradient_side(const Args &a, const Side &s, uint32_t block,
                                              uint32_t blocks, float *partial, float *smem) {
    if (s.norm == SLIKL_NORM_RMS)
        gradient_rows<T, D, SLIKL_NORM_RMS, SRC8>(a, s, block, blocks, partial, smem);
    else if (s.norm == SLIKL_NORM_LAYER)
        gradient_rows<T, D, SLIKL_NORM_LAYER, SRC8>(a, s, block, blocks, partial, smem);
    else
        gradient_rows<T, D, SLIKL_NORM_NONE, SRC8>(a, s, block, blocks, partial, smem);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) qk_gradient(const __grid_constant__ Args a) {
    __shared__ float smem[(kThreads / 32) * D];
    const bool k = blockIdx.x >= a.blocks_q;
    const Side &s = a.side[k];
    const uint32_t block = blockIdx.x - (k ? a.blocks_q : 0);
    const uint32_t blocks = k ? a.blocks_k : a.blocks_q;
    float *partial = a.partial + (k ? 2 * kGradBlocks * D : 0);
    if (s.x || s.norm == SLIKL_NORM_NONE)
        gradient_side<T, D, false>(a, s, block, blocks, partial, smem);
    else
        gradient_side<T, D, true>(a, s, block, blocks, partial, smem);
}

struct Sums {
    float *out[4];            // dgain, dbias of q, of k; null where not asked for
    uint32_t blocks[4];
    const float *partial;
    int D;
};

// One block adds 32 columns of one of the four sums over the blocks' partial sums.
__global__ void __launch_bounds__(1024) qk_grad_sums(Sums a) {
    __shared__ float smem[32][33];
    const int which = blockIdx.y, col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    if (!a.out[which]) return;
    float sum = 0.f;
    for (uint32_t b = part; b < a.blocks[which]; b += 32)
        sum += a.partial[((int64_t)which * kGradBlocks + b) * a.D + col];
    smem[part][threadIdx.x & 31] = sum;
    __syncthreads();
    if (part == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += smem[i][threadIdx.x];
        a.out[which][col] = sum;
    }
}

// --- host side ---------------------------------------------------------------------------------

bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

slikl_status check_side(const slikl_qk_problem *p, const slikl_qk_side &s) {
    if (s.T < 0 || s.N < 1 || s.N > 128 || s.T >= (int64_t(1) << 31) ||
        s.T * s.N >= (int64_t(1) << 31) || s.reserved != 0)
        return SLIKL_ERR_PARAM_INVALID;
    if (s.norm != SLIKL_NORM_NONE && s.norm != SLIKL_NORM_RMS && s.norm != SLIKL_NORM_LAYER)
        return SLIKL_ERR_PARAM_INVALID;
    for (int64_t st : {s.x_stride, s.dx_stride})
        if (st != 0 && (st < s.N * p->D || st % 8 != 0 || st >= (int64_t(1) << 31)))
            return SLIKL_ERR_PARAM_INVALID;
    return SLIKL_OK;
}

slikl_status check_problem(const slikl_qk_problem *p) {
    if (!p) return SLIKL_ERR_PARAM_NULLPTR;
    if (p->dtype != SLIKL_FP16 && p->dtype != SLIKL_BF16) return SLIKL_ERR_PARAM_INVALID;
    if (p->rot_layout != SLIKL_ROT_HALVES && p->rot_layout != SLIKL_ROT_PAIRS)
        return SLIKL_ERR_PARAM_INVALID;
    if (p->D != 64 && p->D != 128) return SLIKL_ERR_PARAM_INVALID;
    if (p->rot_dim < 0 || p->rot_dim > p->D || p->rot_dim % 16 != 0) return SLIKL_ERR_PARAM_INVALID;
    if (p->rot_dim && (p->table_rows < 1 || p->table_rows >= (int64_t(1) << 31)))
        return SLIKL_ERR_PARAM_INVALID;
    if (!(p->eps > 0.f) || !(p->eps <= FLT_MAX) || p->reserved != 0) return SLIKL_ERR_PARAM_INVALID;
    const slikl_status st = check_side(p, p->q);
    return st != SLIKL_OK ? st : check_side(p, p->k);
}

slikl_status check_side_tensors(const slikl_qk_problem *p, const slikl_qk_side &s,
                                const slikl_qk_side_tensors &t, bool gradient) {
    const bool norm = s.norm != SLIKL_NORM_NONE, layer = s.norm == SLIKL_NORM_LAYER;
    if ((t.gain && !norm) || (t.bias && !layer)) return SLIKL_ERR_PARAM_INVALID;
    if (misaligned(t.gain, 16) || misaligned(t.bias, 16)) return SLIKL_ERR_PARAM_INVALID;
    if (gradient) {
        if ((t.dgain && !norm) || (t.dbias && !layer)) return SLIKL_ERR_PARAM_INVALID;
        if (misaligned(t.dgain, 4) || misaligned(t.dbias, 4)) return SLIKL_ERR_PARAM_INVALID;
    }
    if (s.T == 0) return SLIKL_OK;
    if (!t.positions && p->rot_dim && (s.S < 1 || s.S >= (int64_t(1) << 31)))
        return SLIKL_ERR_PARAM_INVALID;
    if (misaligned(t.positions, 4) || misaligned(t.x, 16)) return SLIKL_ERR_PARAM_INVALID;
    const bool reads_x = !gradient || norm;
    if (reads_x && !t.x) {
        if (!t.x8 || !t.x8_scale) return SLIKL_ERR_PARAM_NULLPTR;
        if (misaligned(t.x8, 16) || misaligned(t.x8_scale, 4)) return SLIKL_ERR_PARAM_INVALID;
    }
    if (gradient) {
        if (!t.dy || !t.dx) return SLIKL_ERR_PARAM_NULLPTR;
        if (misaligned(t.dy, 16) || misaligned(t.dx, 16)) return SLIKL_ERR_PARAM_INVALID;
        return SLIKL_OK;
    }
    if (!t.y && !t.keep8) return SLIKL_ERR_PARAM_NULLPTR;
    if (!t.keep8 != !t.keep8_scale) return SLIKL_ERR_PARAM_NULLPTR;
    if (t.keep8 && !t.x) return SLIKL_ERR_PARAM_INVALID;
    if (misaligned(t.y, 16) || misaligned(t.keep8, 16) || misaligned(t.keep8_scale, 4))
        return SLIKL_ERR_PARAM_INVALID;
    return SLIKL_OK;
}

slikl_status check_tensors(const slikl_qk_problem *p, const slikl_qk_tensors *t, bool gradient) {
    if (!t) return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(t->status, 4)) return SLIKL_ERR_PARAM_INVALID;
    if (p->rot_dim && (p->q.T || p->k.T)) {
        if (!t->cos_sin) return SLIKL_ERR_PARAM_NULLPTR;
        if (misaligned(t->cos_sin, 16)) return SLIKL_ERR_PARAM_INVALID;
    }
    const slikl_status st = check_side_tensors(p, p->q, t->q, gradient);
    return st != SLIKL_OK ? st : check_side_tensors(p, p->k, t->k, gradient);
}

Side make_side(const slikl_qk_problem *p, const slikl_qk_side &s, const slikl_qk_side_tensors &t) {
    Side d{};
    d.rows = (uint32_t)(s.T * s.N);
    d.N = fast_div((uint32_t)s.N);
    d.S = fast_div(s.S >= 1 && s.S < (int64_t(1) << 31) ? (uint32_t)s.S : 0x7fffffffu);
    d.norm = s.norm;
    d.x_stride = s.x_stride ? s.x_stride : s.N * p->D;
    d.dx_stride = s.dx_stride ? s.dx_stride : s.N * p->D;
    d.x = t.x;
    d.x8 = static_cast<const uint8_t *>(t.x8);
    d.x8_scale = t.x8_scale;
    d.positions = t.positions;
    d.gain = t.gain;
    d.bias = t.bias;
    d.y = t.y;
    d.keep8 = static_cast<uint8_t *>(t.keep8);
    d.keep8_scale = t.keep8_scale;
    d.dy = t.dy;
    d.dx = t.dx;
    return d;
}

Args make_args(const slikl_qk_problem *p, const slikl_qk_tensors *t) {
    Args a{};
    a.side[0] = make_side(p, p->q, t->q);
    a.side[1] = make_side(p, p->k, t->k);
    a.rot = (int)p->rot_dim;
    a.pairs = p->rot_layout == SLIKL_ROT_PAIRS;
    a.table_rows = (uint32_t)p->table_rows;
    a.eps = p->eps;
    a.cos_sin = t->cos_sin;
    a.status = t->status;
    return a;
}

bool on_sm100() {
    int dev = 0, major = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
           major == 10;
}

slikl_status run_forward(const slikl_qk_problem *p, const slikl_qk_tensors *t, cudaStream_t st) {
    Args a = make_args(p, t);
    const uint32_t per_block = (kThreads / 32) * kFwdUnroll * (uint32_t)(512 / p->D);
    a.blocks_q = (a.side[0].rows + per_block - 1) / per_block;
    a.blocks_k = (a.side[1].rows + per_block - 1) / per_block;
    const uint32_t blocks = a.blocks_q + a.blocks_k;
    if (blocks == 0) return SLIKL_OK;
    auto kernel = p->dtype == SLIKL_BF16
                      ? (p->D == 128 ? qk_forward<__nv_bfloat16, 128> : qk_forward<__nv_bfloat16, 64>)
                      : (p->D == 128 ? qk_forward<__half, 128> : qk_forward<__half, 64>);
    kernel<<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SLIKL_OK : SLIKL_ERR_CUDA;
}

slikl_status run_gradient(const slikl_qk_problem *p, const slikl_qk_tensors *t, float *partial,
                          cudaStream_t st) {
    Args a = make_args(p, t);
    a.partial = partial;
    const uint32_t tile = (kThreads / 32) * (uint32_t)(512 / p->D);
    const uint32_t tq = (a.side[0].rows + tile - 1) / tile, tk = (a.side[1].rows + tile - 1) / tile;
    const uint32_t most = 296;       // two blocks on each multiprocessor
    if (tq + tk <= most) {
        a.blocks_q = tq;
        a.blocks_k = tk;
    } else {                         // in proportion to the work, one at least for a side with rows
        const uint32_t share = (uint32_t)((uint64_t)most * tk / ((uint64_t)tq + tk));
        a.blocks_k = tk == 0 ? 0 : std::min(tk, std::max(share, 1u));
        a.blocks_q = std::min(tq, most - a.blocks_k);
    }
    if (a.blocks_q + a.blocks_k > 0) {
        auto kernel =
            p->dtype == SLIKL_BF16
                ? (p->D == 128 ? qk_gradient<__nv_bfloat16, 128> : qk_gradient<__nv_bfloat16, 64>)
                : (p->D == 128 ? qk_gradient<__half, 128> : qk_gradient<__half, 64>);
        kernel<<<a.blocks_q + a.blocks_k, kThreads, 0, st>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    Sums sums{{t->q.dgain, t->q.dbias, t->k.dgain, t->k.dbias},
              {a.blocks_q, a.blocks_q, a.blocks_k, a.blocks_k},
              partial, (int)p->D};
    if (sums.out[0] || sums.out[1] || sums.out[2] || sums.out[3]) {
        qk_grad_sums<<<dim3((unsigned)p->D / 32, 4), 1024, 0, st>>>(sums);
        if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    return SLIKL_OK;
}

size_t grad_workspace(const slikl_qk_problem *p) {
    return align256(sizeof(float) * 4 * kGradBlocks * (size_t)p->D);
}

// slikl_grad_projected's workspace: slikl_grad_ex's (its status word first), then q, k, dq, dk,
// then the gradient's partial sums.
struct ProjectedLayout {
    size_t q, k, dq, dk, partial, total;
};

slikl_status check_projected(const slikl_problem *pr, const slikl_qk_problem *qk,
                             const slikl_options *options, ProjectedLayout *L) {
    size_t grad = 0;
    slikl_status st = slikl_grad_workspace_size_ex(pr, options, &grad);
    if (st != SLIKL_OK) return st;
    st = check_problem(qk);
    if (st != SLIKL_OK) return st;
    const int64_t T1 = pr->layout_q == SLIKL_BSND ? pr->B * pr->S1 : pr->T1;
    const int64_t T2 = pr->layout_k == SLIKL_BSND ? pr->B * pr->S2 : pr->T2;
    if (qk->dtype != pr->dtype || qk->D != pr->D || qk->q.T != T1 || qk->q.N != pr->N1 ||
        qk->k.T != T2 || qk->k.N != 1)
        return SLIKL_ERR_PARAM_INVALID;
    const size_t qb = align256((size_t)T1 * pr->N1 * pr->D * 2), kb = align256((size_t)T2 * pr->D * 2);
    L->q = align256(grad);
    L->k = L->q + qb;
    L->dq = L->k + kb;
    L->dk = L->dq + qb;
    L->partial = L->dk + kb;
    L->total = L->partial + grad_workspace(qk);
    return SLIKL_OK;
}

}  // namespace
}  // namespace slikl

using namespace slikl;

extern "C" {

slikl_status slikl_qk_norm_rope(const slikl_qk_problem *problem, const slikl_qk_tensors *tensors,
                                void *stream) {
    slikl_status st = check_problem(problem);
    if (st != SLIKL_OK) return st;
    st = check_tensors(problem, tensors, false);
    if (st != SLIKL_OK) return st;
    if (!on_sm100()) return SLIKL_ERR_CUDA;
    return run_forward(problem, tensors, static_cast<cudaStream_t>(stream));
}

slikl_status slikl_qk_norm_rope_grad_workspace_size(const slikl_qk_problem *problem,
                                                    size_t *workspace_bytes) {
    if (!workspace_bytes) return SLIKL_ERR_INNER_NULLPTR;
    const slikl_status st = check_problem(problem);
    if (st != SLIKL_OK) return st;
    *workspace_bytes = grad_workspace(problem);
    return SLIKL_OK;
}

slikl_status slikl_qk_norm_rope_grad(const slikl_qk_problem *problem,
                                     const slikl_qk_tensors *tensors, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    slikl_status st = check_problem(problem);
    if (st != SLIKL_OK) return st;
    st = check_tensors(problem, tensors, true);
    if (st != SLIKL_OK) return st;
    if (!workspace) return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(workspace, 256)) return SLIKL_ERR_PARAM_INVALID;
    if (workspace_bytes < grad_workspace(problem)) return SLIKL_ERR_WORKSPACE_TOO_SMALL;
    if (!on_sm100()) return SLIKL_ERR_CUDA;
    return run_gradient(problem, tensors, static_cast<float *>(workspace),
                        static_cast<cudaStream_t>(stream));
}

slikl_status slikl_grad_projected_workspace_size(const slikl_problem *problem,
                                                 const slikl_qk_problem *qk,
                                                 const slikl_options *options,
                                                 size_t *workspace_bytes) {
    if (!workspace_bytes) return SLIKL_ERR_INNER_NULLPTR;
    ProjectedLayout L;
    const slikl_status st = check_projected(problem, qk, options, &L);
    if (st != SLIKL_OK) return st;
    *workspace_bytes = L.total;
    return SLIKL_OK;
}

slikl_status slikl_grad_projected(const slikl_problem *problem, const slikl_qk_problem *qk,
                                  const slikl_tensors *tensors, const slikl_qk_tensors *qk_tensors,
                                  void *workspace, size_t workspace_bytes, void *stream,
                                  const slikl_options *options) {
    ProjectedLayout L;
    slikl_status st = check_projected(problem, qk, options, &L);
    if (st != SLIKL_OK) return st;
    if (!tensors || !qk_tensors || !workspace) return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(workspace, 256)) return SLIKL_ERR_PARAM_INVALID;
    if (workspace_bytes < L.total) return SLIKL_ERR_WORKSPACE_TOO_SMALL;
    char *ws = static_cast<char *>(workspace);
    slikl_tensors tn = *tensors;
    tn.q = ws + L.q;
    tn.k = ws + L.k;
    tn.dq = ws + L.dq;
    tn.dk = ws + L.dk;
    slikl_qk_tensors qt = *qk_tensors;
    qt.q.y = ws + L.q;
    qt.k.y = ws + L.k;
    qt.q.dy = tn.dq;
    qt.k.dy = tn.dk;
    qt.q.keep8 = qt.k.keep8 = nullptr;
    qt.q.keep8_scale = qt.k.keep8_scale = nullptr;
    // the gradient pass, behind slikl_grad_ex's clearing of the status word, reports positions
    qt.status = nullptr;
    st = check_tensors(qk, &qt, false);
    if (st != SLIKL_OK) return st;
    st = check_tensors(qk, &qt, true);
    if (st != SLIKL_OK) return st;
    // slikl_grad_ex's own checks, before this call's first launch
    st = check_index_call(problem, &tn, options, true);
    if (st != SLIKL_OK) return st;
    if (!on_sm100()) return SLIKL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = run_forward(qk, &qt, s);
    if (st != SLIKL_OK) return st;
    st = slikl_grad_ex(problem, &tn, workspace, L.q, stream, options);
    if (st != SLIKL_OK) return st;
    qt.status = reinterpret_cast<uint32_t *>(workspace);
    return run_gradient(qk, &qt, reinterpret_cast<float *>(ws + L.partial), s);
}

}  // extern "C"
