// q and k from the projections' outputs (norm of each head, position rotation, 8-bit checkpoint)
// and the gradient back to them: slikl_qk_norm_rope, slikl_qk_norm_rope_grad and
// slikl_grad_projected (formulas and contract in include/slikl.h).
//
// Both kernels are bound by HBM: an element costs 2 + 2 bytes (1 more each way for a checkpoint)
// against some twenty instructions. A head row of D values is held by D/16 threads, 16 values each,
// as two 8-value chunks that the rotation by halves pairs with each other: thread l of the first
// rot_dim/16 takes chunks l and l + rot_dim/16, the others pair the two halves of the dims behind
// the rotated ones alike. So every load and store is 16 bytes a thread (8 for e4m3) and neighbours
// share its 32-byte sectors (two neighbouring chunks a thread, which split each sector over two
// instructions, took 36 us to copy 134 MB where this takes 22), the rotation needs no exchange
// between threads, and the norm's sums cross at most 8 lanes by shuffles. Statistics, products and
// sums are fp32; y and dx are rounded once.
//
// HBM wants some 40 KB in flight on each multiprocessor. Registers cannot hold that beside the
// row being worked on (two blocks of 256 threads with two rows a thread reached half the copy
// rate), so each thread copies its chunks of the rows to come into a ring in shared memory that
// it alone reads back: asynchronous copies, several rows deep, and no barrier at all. Next to that
// the issue slots count (a row of 16 values a thread took 420 instructions in the gradient, which
// kept it at half the copy rate; it is 224 now): arithmetic runs on pairs of fp32 values, addresses
// are stepped along the warp's rows instead of computed, and two rows of a token share what is not
// arithmetic. Measured on B200 on the device, as replays of a graph (of the measured copy rate): 4096 rows of
// 64 heads of 128 with their checkpoint 33 us (82 %), 34117 rows of 32 heads in fp16 110 to 115 us (78 to
// 82 %, by the machine), the gradient of 4096 rows 42 us (75 %), that of 32768 rows of 16 heads at their
// checkpoint 83 us (68 %).
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
    uint32_t per_warp, longer;   // groups of rows of each warp; one more for the first `longer`
    int two;                  // groups of two rows a thread, all of one token
    FastDiv N, S;
    int norm;
    uint32_t x_stride, dx_stride;   // bytes from one row to the next
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
    int rot;                  // rotated dims
    uint32_t table_rows;
    float eps;
    const float *cos_sin;
    uint32_t *status;
    float *partial;           // gradient: [4][blocks][D] sums of dgain, dbias of q, dgain, dbias of k
};

constexpr int kThreads = 128;
constexpr int kFwdPerSm = 6, kGradPerSm = 3;   // blocks that a multiprocessor's registers hold
constexpr int kMaxSms = 256;
constexpr int kGradBlocks = kMaxSms * kGradPerSm;   // most blocks of the gradient kernel (the
                                                    // workspace's size)

// What one thread of a head row is responsible for.
struct Lane {
    int ca, cb;               // first dims of its two chunks of 8
    int ta, tb;               // their places in the table's cosines (angle of the chunk's first
                              // value; 8 from ta for halves, 4 from ta and 4 from tb for pairs)
    bool turns;               // rotated dims
};

template <bool PAIRS>
__device__ __forceinline__ Lane lane_of(int l, int rot, int D) {
    Lane t;
    const int half = rot / 16;
    t.turns = l < half;
    t.ca = t.turns ? 8 * l : rot + 8 * (l - half);
    t.cb = t.ca + (t.turns ? rot : D - rot) / 2;
    t.ta = PAIRS ? 4 * l : 8 * l;
    t.tb = PAIRS ? 4 * l + rot / 4 : t.ta + 4;
    return t;
}

// Two fp32 values and what one instruction does to both.
union Pair {
    unsigned long long w;
    float2 f;
};
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    p.f = make_float2(x, y);
    return p;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.w) : "l"(a.w), "l"(b.w));
    return d;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.w) : "l"(a.w), "l"(b.w));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.w) : "l"(a.w), "l"(b.w), "l"(c.w));
    return d;
}
__device__ __forceinline__ float both(Pair a) { return a.f.x + a.f.y; }

// The thread's 16 values as eight pairs, v[i] meeting v[i + 4] in the rotation for i < 4. Halves: v
// holds neighbours, the first chunk's in [0, 4) and the second's in [4, 8). PAIRS: word p of the two
// chunks (eight words of two 16-bit values) holds the two values that angle p turns; the low ones of
// words 2i and 2i + 1 are v[i], the high ones v[i + 4]. So both layouts are turned by the same
// code, and differ in where a value comes from alone.
template <bool PAIRS>
__device__ __forceinline__ float2 word(const Pair *v, int p) {
    if (!PAIRS) return v[p].f;
    return p & 1 ? make_float2(v[p / 2].f.y, v[p / 2 + 4].f.y)
                 : make_float2(v[p / 2].f.x, v[p / 2 + 4].f.x);
}
template <bool PAIRS>
__device__ __forceinline__ void set_word(Pair *v, int p, float2 f) {
    if (!PAIRS) {
        v[p].f = f;
    } else if (p & 1) {
        v[p / 2].f.y = f.x;
        v[p / 2 + 4].f.y = f.y;
    } else {
        v[p / 2].f.x = f.x;
        v[p / 2 + 4].f.x = f.y;
    }
}

// Cosines and sines of the thread's eight angles: c[i], s[i] belong to v[i] and v[i + 4].
struct Angles {
    Pair c[4], s[4];
};

__device__ __forceinline__ void load_angles(const Args &a, const Lane &t, int32_t pos, Angles &g) {
    const float *row = a.cos_sin + (int64_t)pos * a.rot;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 c = *reinterpret_cast<const float4 *>(row + (h ? t.tb : t.ta));
        const float4 s = *reinterpret_cast<const float4 *>(row + a.rot / 2 + (h ? t.tb : t.ta));
        g.c[2 * h] = pair(c.x, c.y), g.c[2 * h + 1] = pair(c.z, c.w);
        g.s[2 * h] = pair(s.x, s.y), g.s[2 * h + 1] = pair(s.z, s.w);
    }
}

// What turns scaled values and applies the gain in one go, v -> v c + w s with w the value's partner
// in the rotation, formed once a token: c the gain times the cosine, s the partner's gain times
// plus or minus the sine (1 and 0 where nothing turns).
struct Turner {
    Pair c[8], s[8];
};

__device__ __forceinline__ void form_turner(const Args &a, const Lane &t, const Pair *gain,
                                            int32_t pos, Turner &o) {
    Angles g;
#pragma unroll
    for (int i = 0; i < 4; ++i) g.c[i] = pair(1.f, 1.f), g.s[i] = pair(0.f, 0.f);
    if (t.turns) load_angles(a, t, pos, g);
    const Pair minus = pair(-1.f, -1.f), none = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.c[i] = gain[i] * g.c[i];
        o.c[i + 4] = gain[i + 4] * g.c[i];
        // (where nothing turns the partner's gain stays out of it, infinite or NaN as it may be)
        o.s[i] = t.turns ? gain[i + 4] * g.s[i] * minus : none;
        o.s[i + 4] = t.turns ? gain[i] * g.s[i] : none;
    }
}

__device__ __forceinline__ void turn(Pair *v, const Turner &o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Pair x = v[i], y = v[i + 4];
        v[i] = fma2(x, o.c[i], y * o.s[i]);
        v[i + 4] = fma2(y, o.c[i + 4], x * o.s[i + 4]);
    }
}

// Turns the values by the angles, or (BACK) by minus the angles.
template <bool BACK>
__device__ __forceinline__ void turn(Pair *v, const Angles &g) {
    const Pair minus = pair(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Pair x = v[i], y = v[i + 4], xs = x * g.s[i], ys = y * g.s[i];
        v[i] = fma2(x, g.c[i], BACK ? ys : ys * minus);
        v[i + 4] = fma2(y, g.c[i], BACK ? xs * minus : xs);
    }
}

template <typename T, bool PAIRS>
__device__ __forceinline__ void widen(const uint4 &a, const uint4 &b, Pair *v) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int p = 0; p < 8; ++p) set_word<PAIRS>(v, p, unpack2<T>(w[p]));
}

template <bool PAIRS>
__device__ __forceinline__ void widen8(const uint2 &a, const uint2 &b, float scale, Pair *v) {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[p >> 1] >> (16 * (p & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        set_word<PAIRS>(v, p, __half22float2(__half2(h)));
    }
    const Pair s = pair(scale, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * s;
}

// Stores the thread's 16 values as 16-bit ones; `first`: where its first chunk goes.
template <typename T, bool PAIRS>
__device__ __forceinline__ void narrow_store(char *first, const Lane &t, const Pair *v) {
    uint32_t w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const float2 f = word<PAIRS>(v, p);
        w[p] = pack2<T>(f.x, f.y);
    }
    *reinterpret_cast<uint4 *>(first) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(first + 2 * (t.cb - t.ca)) = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void zero_store(char *first, const Lane &t) {
    *reinterpret_cast<uint4 *>(first) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(first + 2 * (t.cb - t.ca)) = make_uint4(0, 0, 0, 0);
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

// Two sums at once, so that one's shuffles fill the other's latency.
template <int TPR>
__device__ __forceinline__ void row_sums(float &v, float &w) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, v, o), y = __shfl_xor_sync(0xffffffffu, w, o);
        v += x;
        w += y;
    }
}
// Sums over the thread's values, as two running ones.
__device__ __forceinline__ Pair sum8(const Pair *v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
__device__ __forceinline__ Pair dot8(const Pair *v, const Pair *w) {
    Pair a = v[0] * w[0], b = v[1] * w[1];
#pragma unroll
    for (int i = 2; i < 8; i += 2) a = fma2(v[i], w[i], a), b = fma2(v[i + 1], w[i + 1], b);
    return a + b;
}

// Takes the row's mean off x (layer norm) and returns r. The variance is taken about the mean, not
// as a difference of moments, so that a mean far above the deviation costs no digits.
template <int D, int NORM>
__device__ __forceinline__ float centre(Pair *x, float eps) {
    constexpr int TPR = D / 16;
    if (NORM == SLIKL_NORM_LAYER) {
        const float mean = row_sum<TPR>(both(sum8(x))) * (-1.f / D);
        const Pair less = pair(mean, mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] + less;
    }
    return rsqrtf(fmaf(row_sum<TPR>(both(dot8(x, x))), 1.f / D, eps));
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// A stage of the threads' rings: U rows of x (two 16-byte chunks each, or two 8-byte ones and the
// scale of a checkpoint) and of dy (two 16-byte chunks), and their position. Neighbouring threads'
// chunks are neighbours, so no access has a bank conflict.
template <bool SRC8, bool GRAD, int U>
struct Stage {
    uint4 x[U][SRC8 ? 1 : 2][kThreads];    // (a checkpoint's two 8-byte chunks are x[u][0][i])
    uint4 dy[GRAD ? U : 1][GRAD ? 2 : 1][GRAD ? kThreads : 1];
    float scale[SRC8 ? U : 1][SRC8 ? kThreads : 1];
    int32_t pos[kThreads];                 // -1: the rows take no part, and their values are zero
};
// Rows a thread has on the way beside those it works on: three one at a time, four (forward) or two
// (gradient: x and dy of each) two at a time.
template <bool GRAD, int U>
constexpr int kStages = U == 1 ? 4 : GRAD ? 2 : 3;
template <bool SRC8, bool GRAD, int U>
using Ring = Stage<SRC8, GRAD, U>[kStages<GRAD, U>];
template <bool GRAD>
constexpr size_t kRingBytes = std::max({sizeof(Ring<false, GRAD, 1>), sizeof(Ring<true, GRAD, 1>),
                                        sizeof(Ring<false, GRAD, 2>), sizeof(Ring<true, GRAD, 2>)});

// The rows of a warp: groups of U * RPW rows next to one another (RPW = 512 / D), an equal share of
// the side's groups. `row` is the thread's (first) row in the group, which it steps through together
// with its token and head; its second one, with U = 2, is RPW rows on and of the same token: that
// form is taken where a token's heads are a multiple of 2 * RPW, and shares the work that is not
// arithmetic between two rows (a plain copy's step of four rows: 145 instructions, 116 shared). Rows behind the
// side's last one are worked on like padding, and not stored.
template <int RPW, int U>
struct Walk {
    uint32_t row, token, head;
    int32_t steps;
    uint32_t dt, dh;          // a step is dt tokens and dh heads
    __device__ __forceinline__ Walk(const Side &s, uint32_t block, int sub) {
        const uint32_t warp = block * (kThreads / 32) + (threadIdx.x >> 5);
        steps = (int32_t)(s.per_warp + (warp < s.longer));
        row = (warp * s.per_warp + min(warp, s.longer)) * (RPW * U) + sub;
        token = div_by(row, s.N);
        head = row - token * s.N.d;
        dt = U == 2 ? 0 : div_by(RPW, s.N);
        dh = U == 2 ? 2 * RPW : RPW - dt * s.N.d;
    }
    // Whether the step led to another token.
    __device__ __forceinline__ bool step(const Side &s) {
        row += RPW * U;
        if (U == 1) token += dt;
        head += dh;
        if (head < s.N.d) return U == 1 && dt != 0;
        head -= s.N.d;
        ++token;
        return true;
    }
};

// Copies the rows to come into the ring. Rows that take no part arrive as zeros, so that the work on
// them needs no branches: their y, checkpoint and dx come out as zero and they add zero to every sum.
template <typename T, int D, bool SRC8, bool GRAD, bool READS_X, int U>
struct Fetch {
    static constexpr int RPW = 512 / D;
    Walk<RPW, U> w;
    const char *x, *dy;       // the thread's first chunk of row 0
    int32_t pos;              // of the walk's token, read a step early; -1: takes no part
    bool fresh;               // not looked at yet
    uint32_t stage;

    __device__ __forceinline__ Fetch(const Args &a, const Side &s, const Lane &t,
                                     const Walk<RPW, U> &from)
        : w(from), stage(0) {
        x = SRC8 ? reinterpret_cast<const char *>(s.x8) + t.ca
                 : static_cast<const char *>(s.x) + 2 * t.ca;
        dy = static_cast<const char *>(s.dy) + 2 * t.ca;
        find_position(s);
    }
    __device__ __forceinline__ void find_position(const Side &s) {
        pos = -1;
        fresh = true;
        if (w.row < s.rows)
            pos = s.positions ? s.positions[w.token]
                              : (int32_t)(w.token - div_by(w.token, s.S) * s.S.d);
    }
    // Starts the copies of the walk's rows and steps on. A token's position is checked, a bad one
    // flagged, and its angles are brought near, once. (They are loaded when the row is worked on, often
    // once for many heads; keys of one head need new ones each row, and without the prefetch their
    // side took twice as long as the queries'.)
    __device__ __forceinline__ void next(Ring<SRC8, GRAD, U> &ring, const Args &a, const Side &s,
                                         const Lane &t) {
        auto &to = ring[stage];
        if (++stage == kStages<GRAD, U>) stage = 0;
        const int i = threadIdx.x;
        if (fresh) {
            fresh = false;
            if (pos < 0 || (a.rot && (uint32_t)pos >= a.table_rows)) {
                if (pos != -1 && a.status) set_status(a.status, SLIKL_DEV_BAD_POSITION);
                pos = -1;
            } else if (t.turns) {
                const float *row = a.cos_sin + (int64_t)pos * a.rot + t.ta;
                asm volatile("prefetch.global.L1 [%0];" ::"l"(row));
                asm volatile("prefetch.global.L1 [%0];" ::"l"(row + a.rot / 2));
            }
        }
        to.pos[i] = pos;
        const uint32_t apart = t.cb - t.ca;
        if (pos >= 0) {                        // (never behind the last row)
            if (READS_X && SRC8) {
                const char *p = x + (uint64_t)w.row * D;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t at = sm100::smem_u32(&to.x[u][0][i]);
                    cp_async8(at, p + u * RPW * D);
                    cp_async8(at + 8, p + u * RPW * D + apart);
                    cp_async4(sm100::smem_u32(&to.scale[u][i]), s.x8_scale + w.row + u * RPW);
                }
            } else if (READS_X) {
                const char *p = x + (uint64_t)w.token * s.x_stride + w.head * (2 * D);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    sm100::cp_async16(sm100::smem_u32(&to.x[u][0][i]), p + u * RPW * 2 * D, 16);
                    sm100::cp_async16(sm100::smem_u32(&to.x[u][SRC8 ? 0 : 1][i]),
                                      p + u * RPW * 2 * D + 2 * apart, 16);
                }
            }
            if (GRAD) {
                const char *p = dy + (uint64_t)w.row * (2 * D);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    sm100::cp_async16(sm100::smem_u32(&to.dy[GRAD ? u : 0][0][i]), p + u * RPW * 2 * D, 16);
                    sm100::cp_async16(sm100::smem_u32(&to.dy[GRAD ? u : 0][GRAD ? 1 : 0][i]),
                                      p + u * RPW * 2 * D + 2 * apart, 16);
                }
            }
        } else {
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                to.x[u][0][i] = zero;
                if (SRC8) to.scale[SRC8 ? u : 0][SRC8 ? i : 0] = 0.f;
                else to.x[u][SRC8 ? 0 : 1][i] = zero;
                if (GRAD) to.dy[GRAD ? u : 0][0][GRAD ? i : 0] = to.dy[GRAD ? u : 0][GRAD ? 1 : 0][GRAD ? i : 0] = zero;
            }
        }
        cp_async_commit();
        if (w.step(s)) find_position(s);
    }
};

template <typename T, bool PAIRS, bool SRC8, bool GRAD, int U>
__device__ __forceinline__ void source(const Stage<SRC8, GRAD, U> &from, int u, Pair *v) {
    const int i = threadIdx.x;
    const uint4 x = from.x[u][0][i];
    if (SRC8) widen8<PAIRS>(make_uint2(x.x, x.y), make_uint2(x.z, x.w), from.scale[SRC8 ? u : 0][SRC8 ? i : 0], v);
    else widen<T, PAIRS>(x, from.x[u][SRC8 ? 0 : 1][i], v);
}

// The thread's 16 of D fp32 values (a gain or a bias).
template <bool PAIRS>
__device__ __forceinline__ void load16(const float *p, const Lane &t, Pair *v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 *q = reinterpret_cast<const float4 *>(p + (h ? t.cb : t.ca));
        const float4 u = q[0], w = q[1];
        set_word<PAIRS>(v, 4 * h, make_float2(u.x, u.y));
        set_word<PAIRS>(v, 4 * h + 1, make_float2(u.z, u.w));
        set_word<PAIRS>(v, 4 * h + 2, make_float2(w.x, w.y));
        set_word<PAIRS>(v, 4 * h + 3, make_float2(w.z, w.w));
    }
}

// Largest magnitude of a chunk's eight 16-bit values, NaN aside, in both halves of the word.
template <typename T>
__device__ __forceinline__ uint32_t top_of(const uint4 &a, const uint4 &b);
template <>
__device__ __forceinline__ uint32_t top_of<__nv_bfloat16>(const uint4 &a, const uint4 &b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[i])));
    return reinterpret_cast<const uint32_t &>(m);
}
template <>
__device__ __forceinline__ uint32_t top_of<__half>(const uint4 &a, const uint4 &b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __half2 m = __habs2(reinterpret_cast<const __half2 &>(w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(reinterpret_cast<const __half2 &>(w[i])));
    return reinterpret_cast<const uint32_t &>(m);
}

// One e4m3 checkpoint row: scale = max|x| / 448, values x / scale. The scale is the quotient correctly
// rounded: the product with 1/448 and one step by its exact residual (division by a known divisor, Brisebarre,
// Muller and Raina, IEEE Trans. Computers 53 (2004); a test tries every 16-bit maximum). With the operator
// / in its place registers spilled: 8 tokens took 3.4 us instead of 2.8. The values are products with the
// reciprocal, which __fdividef gives to 2 units, so that one within 2^-21 of the middle between
// two codes may go to either. Every lane of the warp has to come here (the maximum crosses lanes); rows
// that are not `in` are not stored. `top`: top_of the thread's values.
template <typename T, int D, bool PAIRS>
__device__ __forceinline__ void keep_row(const Side &s, uint32_t row, const Lane &t, int l,
                                         bool in, uint32_t top, const Pair *x) {
    const float2 two = unpack2<T>(top);
    const float m = row_max<D / 16>(fmaxf(two.x, two.y));
    if (!in) return;
    // a row of subnormal bf16 values keeps a normal scale, so that its reciprocal is finite
    const float near = m * (1.f / 448.f), off = fmaf(-448.f, near, m);
    const float exact = m <= FLT_MAX ? fmaf(off, 1.f / 448.f, near) : m;
    const float scale = m > 0.f ? fmaxf(exact, FLT_MIN) : 0.f;
    const float inv = m > 0.f ? __fdividef(1.f, scale) : 0.f;
    const Pair by = pair(inv, inv);
    Pair q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[i] * by;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(word<PAIRS>(q, 2 * i), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(word<PAIRS>(q, 2 * i + 1), __NV_SATFINITE, __NV_E4M3);
        w[i] = __byte_perm(lo, hi, 0x5410);
    }
    uint8_t *p = s.keep8 + t.ca + (uint64_t)row * D;
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(p + (t.cb - t.ca)) = make_uint2(w[2], w[3]);
    if (l == 0) s.keep8_scale[row] = scale;
}

template <typename T, int D, bool PAIRS, int NORM, bool SRC8, int U>
__device__ __forceinline__ void forward_rows(const Args &a, const Side &s, uint32_t block,
                                             void *smem) {
    constexpr int TPR = D / 16, RPW = 32 / TPR;
    auto &ring = *static_cast<Ring<SRC8, false, U> *>(smem);
    const int l = (threadIdx.x & 31) % TPR;
    const Lane t = lane_of<PAIRS>(l, a.rot, D);
    const Walk<RPW, U> walk(s, block, (threadIdx.x & 31) / TPR);
    const int32_t steps = walk.steps;
    uint32_t row = walk.row, stage = 0;
    Fetch<T, D, SRC8, false, true, U> fetch(a, s, t, walk);
#pragma unroll
    for (int i = 0; i < kStages<false, U> - 1; ++i) {
        if (i < steps) fetch.next(ring, a, s, t);
        else cp_async_commit();
    }
    // without a bias the gain goes into the rotation, and both together into a Turner; a layer norm
    // (of keys of one head, mostly) takes gain, bias and angles one after another
    constexpr bool LAYER = NORM == SLIKL_NORM_LAYER;
    Turner turner;
    Angles angles;
    int32_t turned_to = -1;               // the position that they belong to
#pragma unroll
    for (int j = 0; j < 8; ++j) turner.c[j] = turner.s[j] = pair(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) angles.c[j] = angles.s[j] = pair(0.f, 0.f);
    for (int32_t i = 0; i < steps; ++i, row += RPW * U) {
        sm100::cp_async_wait<kStages<false, U> - 2>();
        const auto &now = ring[stage];
        if (++stage == kStages<false, U>) stage = 0;
        const int32_t pos = now.pos[threadIdx.x];
        if (pos >= 0 && pos != turned_to) {
            turned_to = pos;
            if (LAYER) {
                if (t.turns) load_angles(a, t, pos, angles);
            } else {
                Pair gain[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) gain[j] = pair(1.f, 1.f);
                if (s.gain) load16<PAIRS>(s.gain, t, gain);
                form_turner(a, t, gain, pos, turner);
            }
        }
        if (i + kStages<false, U> - 1 < steps) fetch.next(ring, a, s, t);
        else cp_async_commit();
        char *y = static_cast<char *>(s.y) + 2 * t.ca + (uint64_t)row * (2 * D);
        const bool in = U == 2 || row < s.rows;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pair v[8];
            source<T, PAIRS>(now, u, v);
            if (!SRC8 && s.keep8)
                keep_row<T, D, PAIRS>(s, row + u * RPW, t, l, in,
                               top_of<T>(now.x[u][0][threadIdx.x], now.x[u][SRC8 ? 0 : 1][threadIdx.x]), v);
            if (!s.y) continue;
            if (NORM != SLIKL_NORM_NONE) {
                const float r = centre<D, NORM>(v, a.eps);
                const Pair by = pair(r, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * by;
            }
            if (!in) continue;
            if (LAYER) {
                if (pos < 0) {            // the bias is not zero
                    zero_store(y + u * RPW * 2 * D, t);
                    continue;
                }
                if (s.gain) {
                    Pair gain[8];
                    load16<PAIRS>(s.gain, t, gain);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * gain[j];
                }
                if (s.bias) {
                    Pair bias[8];
                    load16<PAIRS>(s.bias, t, bias);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] + bias[j];
                }
                if (t.turns) turn<false>(v, angles);
            } else if (NORM != SLIKL_NORM_NONE || t.turns) {
                // (without a norm the dims that do not turn stay out of it: their partner, times zero,
                // may be infinite)
                turn(v, turner);
            }
            narrow_store<T, PAIRS>(y + u * RPW * 2 * D, t, v);
        }
    }
}

template <typename T, int D, bool PAIRS, bool SRC8, int U>
__device__ __forceinline__ void forward_side(const Args &a, const Side &s, uint32_t block,
                                             void *smem) {
    if (s.norm == SLIKL_NORM_RMS)
        forward_rows<T, D, PAIRS, SLIKL_NORM_RMS, SRC8, U>(a, s, block, smem);
    else if (s.norm == SLIKL_NORM_LAYER)
        forward_rows<T, D, PAIRS, SLIKL_NORM_LAYER, SRC8, U>(a, s, block, smem);
    else
        forward_rows<T, D, PAIRS, SLIKL_NORM_NONE, SRC8, U>(a, s, block, smem);
}

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kFwdPerSm) qk_forward(const __grid_constant__ Args a) {
    __shared__ __align__(16) unsigned char smem[kRingBytes<false>];
    const bool k = blockIdx.x >= a.blocks_q;
    const Side &s = a.side[k];
    const uint32_t block = blockIdx.x - (k ? a.blocks_q : 0);
    if (s.x) {
        if (s.two) forward_side<T, D, PAIRS, false, 2>(a, s, block, smem);
        else forward_side<T, D, PAIRS, false, 1>(a, s, block, smem);
    } else {
        if (s.two) forward_side<T, D, PAIRS, true, 2>(a, s, block, smem);
        else forward_side<T, D, PAIRS, true, 1>(a, s, block, smem);
    }
}

// Gradient: the sums of dgain and dbias stay in registers over a warp's rows, are added over the
// block in a fixed order and stored; qk_grad_sums adds the blocks' sums, again in a fixed order.
// With x less its mean, h = dz gain:
//   dbias += dz,  dgain += (dz x) r,  dx = r (h - [mean(h)]) - x r^3 mean(h x)
template <typename T, int D, bool PAIRS, int NORM, bool SRC8, int U>
__device__ __forceinline__ void gradient_rows(const Args &a, const Side &s, uint32_t block,
                                              float *partial, void *ring_smem, float4 *gains) {
    constexpr int TPR = D / 16, RPW = 32 / TPR, WARPS = kThreads / 32;
    constexpr bool X = NORM != SLIKL_NORM_NONE;        // without a norm x is not needed
    constexpr bool LAYER = NORM == SLIKL_NORM_LAYER;
    auto &ring = *static_cast<Ring<SRC8, true, U> *>(ring_smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Lane t = lane_of<PAIRS>(lane % TPR, a.rot, D);
    Walk<RPW, U> at(s, block, lane / TPR);
    const int32_t steps = at.steps;
    uint32_t stage = 0;
    Fetch<T, D, SRC8, true, X, U> fetch(a, s, t, at);
#pragma unroll
    for (int i = 0; i < kStages<true, U> - 1; ++i) {
        if (i < steps) fetch.next(ring, a, s, t);
        else cp_async_commit();
    }
    // the thread's gains, as its four 16-byte pieces in a row with the other threads' same pieces:
    // registers are short here, and every row reads each gain once
    if (X && threadIdx.x < TPR) {
        Pair gain[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) gain[j] = pair(1.f, 1.f);
        if (s.gain) load16<PAIRS>(s.gain, t, gain);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            gains[j * TPR + threadIdx.x] =
                make_float4(gain[2 * j].f.x, gain[2 * j].f.y, gain[2 * j + 1].f.x, gain[2 * j + 1].f.y);
    }
    __syncthreads();
    Pair dgain[8], dbias[8];
    Angles angles;
    int32_t turned_to = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) angles.c[i] = angles.s[i] = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dgain[i] = dbias[i] = pair(0.f, 0.f);
    for (int32_t i = 0; i < steps; ++i, at.step(s)) {
        sm100::cp_async_wait<kStages<true, U> - 2>();
        const auto &now = ring[stage];
        if (++stage == kStages<true, U>) stage = 0;
        const int32_t pos = now.pos[threadIdx.x];
        if (t.turns && pos >= 0 && pos != turned_to) {
            load_angles(a, t, pos, angles);
            turned_to = pos;
        }
        if (i + kStages<true, U> - 1 < steps) fetch.next(ring, a, s, t);
        else cp_async_commit();
        char *dx = static_cast<char *>(s.dx) + 2 * t.ca + (uint64_t)at.token * s.dx_stride +
                   at.head * (2 * D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pair g[8], v[8];
            widen<T, PAIRS>(now.dy[u][0][threadIdx.x], now.dy[u][1][threadIdx.x], g);
            if (X) source<T, PAIRS>(now, u, v);
            if (t.turns) turn<true>(g, angles);
            if (X) {
                // two rounds of sums over the row's threads, each of two sums side by side: the means
                // of x and h (layer only), then x^2 and h x
                float lift = 0.f;
                Pair e[8];
                if (LAYER) {
                    const float m = both(sum8(v));
                    float sx = m, sh;
                    Pair sum = pair(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 w = gains[j * TPR + lane % TPR];
                        sum = fma2(g[2 * j], pair(w.x, w.y), sum);
                        sum = fma2(g[2 * j + 1], pair(w.z, w.w), sum);
                    }
                    sh = both(sum);
                    row_sums<TPR>(sx, sh);
                    lift = sh * (-1.f / D);
                    const Pair less = pair(sx * (-1.f / D), sx * (-1.f / D));
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[j] = v[j] + less;
                        dbias[j] = dbias[j] + g[j];
                    }
                }
                Pair sum = pair(0.f, 0.f), more = sum;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w = gains[j * TPR + lane % TPR];
                    e[2 * j] = g[2 * j] * v[2 * j];
                    e[2 * j + 1] = g[2 * j + 1] * v[2 * j + 1];
                    sum = fma2(e[2 * j], pair(w.x, w.y), sum);
                    more = fma2(e[2 * j + 1], pair(w.z, w.w), more);
                    g[2 * j] = g[2 * j] * pair(w.x, w.y);            // h from here on
                    g[2 * j + 1] = g[2 * j + 1] * pair(w.z, w.w);
                }
                float sq = both(dot8(v, v)), sh = both(sum + more);
                row_sums<TPR>(sq, sh);
                const float r = rsqrtf(fmaf(sq, 1.f / D, a.eps));
                // (r^3 by itself may be infinite where a row of zeros meets a tiny eps)
                const float m = sh * (-1.f / D) * r * r * r;
                const Pair by = pair(r, r), along = pair(m, m), up = pair(r * lift, r * lift);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dgain[j] = fma2(e[j], by, dgain[j]);
                    g[j] = fma2(v[j], along, LAYER ? fma2(g[j], by, up) : g[j] * by);
                }
            }
            if (U == 2 || at.row < s.rows) narrow_store<T, PAIRS>(dx + u * RPW * 2 * D, t, g);
        }
    }
    // the ring's memory serves the sum over the block's warps once every warp is done with it
    sm100::cp_async_wait<0>();
    __syncthreads();
    float *smem = static_cast<float *>(ring_smem);
    if constexpr (NORM != SLIKL_NORM_NONE) {
#pragma unroll
        for (int which = 0; which < (NORM == SLIKL_NORM_LAYER ? 2 : 1); ++which) {
            float acc[16];                // by the values' places in the two chunks
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float2 f = word<PAIRS>(which ? dbias : dgain, p);
                acc[2 * p] = f.x;
                acc[2 * p + 1] = f.y;
            }
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

template <typename T, int D, bool PAIRS, bool SRC8, int U>
__device__ __forceinline__ void gradient_side(const Args &a, const Side &s, uint32_t block,
                                              float *partial, void *smem, float4 *gains) {
    if (s.norm == SLIKL_NORM_RMS)
        gradient_rows<T, D, PAIRS, SLIKL_NORM_RMS, SRC8, U>(a, s, block, partial, smem, gains);
    else if (s.norm == SLIKL_NORM_LAYER)
        gradient_rows<T, D, PAIRS, SLIKL_NORM_LAYER, SRC8, U>(a, s, block, partial, smem, gains);
    else
        gradient_rows<T, D, PAIRS, SLIKL_NORM_NONE, SRC8, U>(a, s, block, partial, smem, gains);
}

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kGradPerSm) qk_gradient(const __grid_constant__ Args a) {
    __shared__ __align__(16) unsigned char smem[kRingBytes<true>];
    __shared__ float4 gains[D / 4];
    let_next_start();         // qk_grad_sums
    const bool k = blockIdx.x >= a.blocks_q;
    const Side &s = a.side[k];
    const uint32_t block = blockIdx.x - (k ? a.blocks_q : 0);
    float *partial = a.partial + (k ? 2 * kGradBlocks * D : 0);
    if (s.x || s.norm == SLIKL_NORM_NONE) {
        if (s.two) gradient_side<T, D, PAIRS, false, 2>(a, s, block, partial, smem, gains);
        else gradient_side<T, D, PAIRS, false, 1>(a, s, block, partial, smem, gains);
    } else {
        if (s.two) gradient_side<T, D, PAIRS, true, 2>(a, s, block, partial, smem, gains);
        else gradient_side<T, D, PAIRS, true, 1>(a, s, block, partial, smem, gains);
    }
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
    await_previous();
    const int which = blockIdx.y, col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    if (!a.out[which]) return;
    // eight loads on the way at once: one after another they took 4 us
    float sums[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float *from = a.partial + (int64_t)which * kGradBlocks * a.D + col;
    for (uint32_t b = part; b < a.blocks[which]; b += 256)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (b + 32 * i < a.blocks[which]) sums[i] += from[(int64_t)(b + 32 * i) * a.D];
    float sum = ((sums[0] + sums[1]) + (sums[2] + sums[3])) + ((sums[4] + sums[5]) + (sums[6] + sums[7]));
    smem[part][threadIdx.x & 31] = sum;
    __syncthreads();
    if (part == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += smem[i][threadIdx.x];
        a.out[which][col] = sum;
    }
}

// Positions of the rows of a slikl_grad_projected call with used lengths: those that the caller gives (or t
// % S), and -1 for the rows behind a batch's used ones, whose x, like the gradient's own padding rows, may
// hold anything: without a position a NaN there would reach dgain as 0 * NaN.
struct UsedRows {
    int64_t T, S, batch, B;   // rows; S of slikl_qk_side; rows of a batch (0: cu), batches
    const int32_t *cu, *used, *positions;
    int32_t *out;             // null: this side has no used lengths
};

__global__ void __launch_bounds__(256) used_positions(UsedRows q, UsedRows k) {
    const UsedRows &s = blockIdx.y ? k : q;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (!s.out || t >= s.T) return;
    int64_t b, local;
    if (s.batch) {
        b = t / s.batch;
        local = t - b * s.batch;
    } else {                  // the last batch that starts at t or before
        int64_t lo = 0, hi = s.B;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (s.cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
        local = t - s.cu[b];
    }
    s.out[t] = local >= s.used[b] ? -1 : s.positions ? s.positions[t] : (int32_t)(t % s.S);
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
    d.x_stride = (uint32_t)(2 * (s.x_stride ? s.x_stride : s.N * p->D));
    d.dx_stride = (uint32_t)(2 * (s.dx_stride ? s.dx_stride : s.N * p->D));
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
    a.table_rows = (uint32_t)p->table_rows;
    a.eps = p->eps;
    a.cos_sin = t->cos_sin;
    a.status = t->status;
    return a;
}

// Multiprocessors of the current device; 0 where it cannot run these kernels.
int sm100_multiprocessors() {
    int dev = 0, major = 0, sms = 0;
    const bool ok =
        cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    return ok && major == 10 ? sms : 0;
}

// Blocks of both sides, as many as the multiprocessors hold, in proportion to what their rows take; a
// side with rows gets one at least. A row of a token with few heads, for which angles come from the
// table, takes 1 + few / N times as long as one of many heads (measured over shares on B200: with
// few = 0.6 the varlen forward took 122 us, with 3 110; the gradient at the checkpoint 94 with 0.6,
// 84 with 1.1 and 2, 88 with 3), and a layer norm 1.25 times as long as an RMS norm (with 1, 1.25 and 1.6
// the gradient at the checkpoint took 84.9, 83.4 and 86.4 us, the forward with its checkpoint 33.1,
// 32.9 and 33.6). A small call gets a group of rows for each warp, so that it spreads over all multiprocessors.
void share_blocks(Args &a, int64_t D, int sms, int per_sm, double few) {
    const uint32_t most = (uint32_t)(std::min(sms, kMaxSms) * per_sm), warps = kThreads / 32;
    const uint32_t rpw = (uint32_t)(512 / D);
    uint32_t groups[2], blocks[2];
    double cost[2];
    for (int i = 0; i < 2; ++i) {
        Side &s = a.side[i];
        // two rows a thread where a token's heads allow it and every warp still gets a group
        s.two = s.N.d % (2 * rpw) == 0 && s.rows >= 2 * rpw * warps * most;
        const uint32_t per = rpw << s.two;
        groups[i] = (s.rows + per - 1) / per;
        blocks[i] = (groups[i] + warps - 1) / warps;
        cost[i] = s.rows * (s.two ? 1.0 : 1.0 + few / s.N.d) * (s.norm == SLIKL_NORM_LAYER ? 1.25 : 1.0);
    }
    if ((uint64_t)blocks[0] + blocks[1] > most) {
        const uint32_t share = (uint32_t)(most * (cost[1] / (cost[0] + cost[1])) + 0.5);
        const uint32_t least_q = blocks[0] ? 1 : 0, least_k = blocks[1] ? 1 : 0;
        blocks[1] = std::min(blocks[1], std::min(std::max(share, least_k), most - least_q));
        blocks[0] = std::min(blocks[0], most - blocks[1]);
    }
    for (int i = 0; i < 2; ++i)
        if (blocks[i]) {
            a.side[i].per_warp = groups[i] / (blocks[i] * warps);
            a.side[i].longer = groups[i] % (blocks[i] * warps);
        }
    a.blocks_q = blocks[0];
    a.blocks_k = blocks[1];
}

using Kernel = void (*)(Args);
struct Forward {
    template <typename T, int D, bool PAIRS>
    Kernel get() const { return qk_forward<T, D, PAIRS>; }
};
struct Gradient {
    template <typename T, int D, bool PAIRS>
    Kernel get() const { return qk_gradient<T, D, PAIRS>; }
};
template <typename T, typename K>
Kernel pick_of(const slikl_qk_problem &p, const K &k) {
    const bool pairs = p.rot_layout == SLIKL_ROT_PAIRS;
    if (p.D == 128) return pairs ? k.template get<T, 128, true>() : k.template get<T, 128, false>();
    return pairs ? k.template get<T, 64, true>() : k.template get<T, 64, false>();
}
template <typename K>
Kernel pick(const slikl_qk_problem &p, const K &k) {
    return p.dtype == SLIKL_BF16 ? pick_of<__nv_bfloat16>(p, k) : pick_of<__half>(p, k);
}

slikl_status run_forward(const slikl_qk_problem *p, const slikl_qk_tensors *t, int sms,
                         cudaStream_t st) {
    Args a = make_args(p, t);
    share_blocks(a, p->D, sms, kFwdPerSm, 3.0);
    const uint32_t blocks = a.blocks_q + a.blocks_k;
    if (blocks == 0) return SLIKL_OK;
    const auto kernel = pick(*p, Forward{});
    kernel<<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SLIKL_OK : SLIKL_ERR_CUDA;
}

slikl_status run_gradient(const slikl_qk_problem *p, const slikl_qk_tensors *t, float *partial,
                          int sms, cudaStream_t st) {
    Args a = make_args(p, t);
    a.partial = partial;
    share_blocks(a, p->D, sms, kGradPerSm, 1.5);
    if (a.blocks_q + a.blocks_k > 0) {
        const auto kernel = pick(*p, Gradient{});
        kernel<<<a.blocks_q + a.blocks_k, kThreads, 0, st>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    Sums sums{{t->q.dgain, t->q.dbias, t->k.dgain, t->k.dbias},
              {a.blocks_q, a.blocks_q, a.blocks_k, a.blocks_k},
              partial, (int)p->D};
    if (sums.out[0] || sums.out[1] || sums.out[2] || sums.out[3]) {
        if (launch_next(qk_grad_sums, dim3((unsigned)p->D / 32, 4), 1024, 0, st, sums) != cudaSuccess)
            return SLIKL_ERR_CUDA;
    }
    return SLIKL_OK;
}

size_t grad_workspace(const slikl_qk_problem *p) {
    return align256(sizeof(float) * 4 * kGradBlocks * (size_t)p->D);
}

// slikl_grad_projected's workspace: slikl_grad_ex's (its status word first), then q, k, dq, dk, the
// rows' positions (where there are used lengths), then the gradient's partial sums.
struct ProjectedLayout {
    size_t q, k, dq, dk, pos_q, pos_k, partial, total;
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
    L->pos_q = L->dk + kb;
    L->pos_k = L->pos_q + align256(sizeof(int32_t) * (size_t)T1);
    L->partial = L->pos_k + align256(sizeof(int32_t) * (size_t)T2);
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
    const int sms = sm100_multiprocessors();
    if (!sms) return SLIKL_ERR_CUDA;
    return run_forward(problem, tensors, sms, static_cast<cudaStream_t>(stream));
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
    const int sms = sm100_multiprocessors();
    if (!sms) return SLIKL_ERR_CUDA;
    return run_gradient(problem, tensors, static_cast<float *>(workspace), sms,
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
    const int sms = sm100_multiprocessors();
    if (!sms) return SLIKL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (options && (options->seq_used_q || options->seq_used_k)) {
        auto rows = [&](const slikl_qk_side &side, slikl_qk_side_tensors &t, const int32_t *used, int layout,
                        int64_t batch, const int32_t *cu, size_t at) {
            UsedRows u{side.T, std::max<int64_t>(1, side.S), layout == SLIKL_BSND ? batch : 0, problem->B, cu, used,
                       t.positions, nullptr};
            if (used && side.T > 0) t.positions = u.out = reinterpret_cast<int32_t *>(ws + at);
            return u;
        };
        const UsedRows uq = rows(qk->q, qt.q, options->seq_used_q, problem->layout_q, problem->S1, tn.cu_seqlens_q, L.pos_q);
        const UsedRows uk = rows(qk->k, qt.k, options->seq_used_k, problem->layout_k, problem->S2, tn.cu_seqlens_k, L.pos_k);
        const int64_t most = std::max(uq.out ? uq.T : 0, uk.out ? uk.T : 0);
        if (most > 0) {
            used_positions<<<dim3((unsigned)((most + 255) / 256), 2), 256, 0, s>>>(uq, uk);
            if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
        }
    }
    st = run_forward(qk, &qt, sms, s);
    if (st != SLIKL_OK) return st;
    st = slikl_grad_ex(problem, &tn, workspace, L.q, stream, options);
    if (st != SLIKL_OK) return st;
    qt.status = reinterpret_cast<uint32_t *>(workspace);
    return run_gradient(qk, &qt, reinterpret_cast<float *>(ws + L.partial), sms, s);
}

}  // extern "C"
