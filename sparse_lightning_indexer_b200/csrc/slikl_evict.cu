// Cutting a cache to the key rows with the highest scores (slikl_evict; contract in
// include/slikl.h).
//
// evict_choose finds, for each sequence, the score of the last row that stays by a radix select
// over order-preserving integers (four passes of 8 bits), then walks the rows in
// order and writes the kept ones behind one another. It is bound by latency: a pass over the scores,
// which L2 holds, and the barriers between. So a long sequence is shared by a cluster of eight blocks,
// whose histograms and counts the others read from its shared memory (one block took 127 us for
// sequences of up to 131072 rows; with three passes of 11 bits each block's reads of the others' 2048
// bins, and their prefix sums, took two thirds of a pass; 21 us now). evict_copy moves the caches' rows, bound by HBM.
#include <cooperative_groups.h>

#include <algorithm>

#include "slikl_common.cuh"

namespace slikl {
namespace {

constexpr int kChoose = 1024;         // threads of evict_choose
constexpr int kBins = 256;

struct EvictArgs {
    int layout_k, n_caches;
    int64_t B, S2, T2;
    int32_t budget, sinks, recent;
    const float *scores;
    const int32_t *cu_k, *used_k;
    int32_t *kept, *lengths;
    float *scores_out;
    uint32_t *status;
    slikl_evict_cache caches[SLIKL_EVICT_MAX_CACHES];
};

// Rows [base, base + n) of the key tensor in use by sequence b.
struct Sequence {
    int64_t base;
    int32_t n;
};

__device__ Sequence sequence_of(const EvictArgs &a, int64_t b, bool report) {
    Sequence q{b * a.S2, (int32_t)a.S2};
    uint32_t bad = 0;
    if (a.layout_k == SLIKL_TND) {
        const int64_t k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        const bool fits = k0 >= 0 && k1 >= k0 && k1 <= a.T2;
        q.base = fits ? k0 : 0;
        q.n = fits ? (int32_t)(k1 - k0) : 0;
        if (!fits || (b == 0 && k0 != 0) || (b == a.B - 1 && k1 != a.T2))
            bad |= SLIKL_DEV_BAD_CU_SEQLENS_K;
    }
    if (a.used_k) {
        const int32_t u = a.used_k[b];
        if (u < 0 || u > q.n) bad |= SLIKL_DEV_BAD_SEQ_USED;
        q.n = max(0, min(u, q.n));
    }
    if (report && bad && a.status) set_status(a.status, bad);
    return q;
}

// Larger scores have larger numbers; +0 and -0 the same one, NaN the lowest.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The score that an order number stands for, where it is one: not for NaN and zero, which have several.
__device__ __forceinline__ float score_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// CS blocks share a sequence; a tile of a block's slice is ROUNDS rows for each of its threads, which hold
// their order numbers in registers: row 32 k of a warp's share (32 ROUNDS neighbours) and the lane's place.
// The usual slice is one tile, read once; a longer one is read again for every pass.
template <int CS, int ROUNDS>
__global__ void __launch_bounds__(kChoose) __cluster_dims__(CS, 1, 1) evict_choose(EvictArgs a) {
    namespace cg = cooperative_groups;
    constexpr bool SMALL = CS == 1 && ROUNDS == 1;
    constexpr uint32_t SHARE = 32 * ROUNDS, TILE = kChoose * ROUNDS;
    __shared__ int bins[SMALL ? 1 : 4][SMALL ? 1 : kBins];   // of each pass: the other blocks may still
                                                             // read an earlier one
    __shared__ int more[2][32];
    __shared__ uint32_t found_bin;
    __shared__ int found_above, counts[2];
    let_next_start();                    // evict_copy
    auto cluster = cg::this_cluster();
    const uint32_t rank = CS == 1 ? 0 : cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.x / CS;
    const Sequence q = sequence_of(a, b, threadIdx.x == 0 && rank == 0);
    const uint32_t n = q.n, budget = a.budget, stay = min(n, budget);
    const bool all = n <= budget;
    const uint32_t lo = all ? 0 : a.sinks, hi = all ? 0 : n - a.recent;   // rows that scores decide on
    const uint32_t wanted = all ? 0 : budget - a.sinks - a.recent;
    const float *scores = a.scores + q.base;
    const uint32_t per = (n + CS - 1) / CS, slice0 = min(n, rank * per), slice1 = min(n, slice0 + per);
    const bool once = slice1 - slice0 <= TILE;
    const uint32_t first = slice0 + warp * SHARE + lane;     // the thread's first row of the first tile

    uint32_t order[ROUNDS], decided = 0;      // bit k: row k is one that scores decide on
    auto read_tile = [&](uint32_t j) {
        decided = 0;
        float x[ROUNDS];
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)          // (all on the way at once: no load behind a branch)
            x[k] = scores[min(j + 32 * k, slice1 - 1)];
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            order[k] = order_of(x[k]);
            decided |= (uint32_t)(j + 32 * k >= lo && j + 32 * k < min(hi, slice1)) << k;
        }
    };
    if (slice0 < slice1) read_tile(first);

    // the order number of the wanted-th of them, and how many rows with that number stay
    uint32_t prefix = 0;
    int left = wanted, above_mine = 0;
    if (wanted > 0 && SMALL && once) {
        // a row a thread: the number bit by bit, a barrier that counts for each
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t next = prefix | 1u << bit;
            if (__syncthreads_count(decided && order[0] >= next) >= (int)wanted) prefix = next;
        }
        left -= __syncthreads_count(decided && order[0] > prefix);
    } else if (wanted > 0 && !SMALL) {
        uint32_t mask = 0;
        for (int i = threadIdx.x; i < 4 * kBins; i += kChoose) bins[0][i] = 0;
        __syncthreads();
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (uint32_t j = 0; j < slice1 - slice0; j += TILE) {
                if (!once) read_tile(first + j);
#pragma unroll
                for (int k = 0; k < ROUNDS; ++k)
                    if ((decided >> k & 1) && (order[k] & mask) == prefix)
                        atomicAdd(&bins[pass][order[k] >> shift & 255], 1);
            }
            if (CS == 1) __syncthreads();
            else cluster.sync();
            // thread i < 256 holds bin 255 - i: the prefix runs from the highest bin
            const int bin = kBins - 1 - (int)threadIdx.x;
            int h = 0, mine = 0, x = 0;
            if (threadIdx.x < kBins) {
                mine = bins[pass][bin];
                if (CS == 1) {
                    h = mine;
                } else {
#pragma unroll
                    for (int r = 0; r < CS; ++r) h += *cluster.map_shared_rank(&bins[pass][bin], r);
                }
                x = h;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) more[0][warp] = x;
            }
            __syncthreads();
            if (threadIdx.x < kBins) {
                int above = x - h;
                for (int w = 0; w < warp; ++w) above += more[0][w];
                if (above < left && left <= above + h) {
                    found_bin = bin;
                    found_above = above;
                }
            }
            __syncthreads();
            if (threadIdx.x < kBins && bin > (int)found_bin) above_mine += mine;
            prefix |= found_bin << shift;
            mask |= 255u << shift;
            left -= found_above;
        }
    }
    // rows before this block's slice that stay whatever the ties (counts[0]) or tie for the last
    // places (counts[1])
    int sure = 0, tied = 0;
    if (CS > 1) {
        // (above_mine: of the first 256 threads, eight warps)
        const int sum = __reduce_add_sync(0xffffffffu, above_mine);
        if (lane == 0) more[1][warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            const uint32_t from = max(lo, slice0), to = min(hi, slice1);
            int total = (int)(slice1 - slice0 - (from < to ? to - from : 0));
            for (int w = 0; w < kBins / 32; ++w) total += more[1][w];
            counts[0] = total;
            counts[1] = wanted > 0 ? bins[SMALL ? 0 : 3][SMALL ? 0 : prefix & 255] : 0;
        }
        cluster.sync();
        for (int r = 0; r < (int)rank; ++r) {
            const int *c = cluster.map_shared_rank(counts, r);
            sure += c[0];
            tied += c[1];
        }
    }

    int32_t *kept = a.kept + b * budget;
    float *out = a.scores_out ? a.scores_out + b * budget : nullptr;
    for (uint32_t j0 = 0; j0 < slice1 - slice0; j0 += TILE) {
        if (!once) read_tile(first + j0);
        uint32_t is_sure = 0, is_tied = 0;       // bit k: this lane's row of round k
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const bool d = decided >> k & 1;
            const bool s = d ? wanted > 0 && order[k] > prefix : first + j0 + 32 * k < slice1 &&
                               !(first + j0 + 32 * k >= lo && first + j0 + 32 * k < hi);
            const bool t = d && wanted > 0 && order[k] == prefix;
            is_sure |= (uint32_t)s << k;
            is_tied |= (uint32_t)t << k;
        }
        const int n_sure = __reduce_add_sync(0xffffffffu, __popc(is_sure));
        const int n_tied = __reduce_add_sync(0xffffffffu, __popc(is_tied));
        __syncthreads();
        if (lane == 0) more[0][warp] = n_sure, more[1][warp] = n_tied;
        __syncthreads();
        const int c_sure = more[0][lane], c_tied = more[1][lane];
        int g = sure + __reduce_add_sync(0xffffffffu, lane < warp ? c_sure : 0);
        int e = tied + __reduce_add_sync(0xffffffffu, lane < warp ? c_tied : 0);
        sure += __reduce_add_sync(0xffffffffu, c_sure);
        tied += __reduce_add_sync(0xffffffffu, c_tied);
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const bool s = is_sure >> k & 1, t = is_tied >> k & 1;
            const uint32_t bs = __ballot_sync(0xffffffffu, s), bt = __ballot_sync(0xffffffffu, t);
            const uint32_t below = (1u << lane) - 1;
            const int before = e + __popc(bt & below);
            if (s || (t && before < left)) {
                const int place = g + __popc(bs & below) + min(before, left);
                const uint32_t j = first + j0 + 32 * k;
                kept[place] = (int32_t)j;
                if (out) {
                    const float x = score_of(order[k]);
                    out[place] = x == 0.f || x != x ? scores[j] : x;
                }
            }
            g += __popc(bs);
            e += __popc(bt);
        }
    }
    for (uint32_t j = stay + rank * kChoose + threadIdx.x; j < budget; j += CS * kChoose) {
        kept[j] = -1;
        if (out) out[j] = 0.f;
    }
    if (CS == 1) __syncthreads();         // every thread has read seq_used_k, which lengths may be (a
                                          // cluster has met above)
    if (threadIdx.x == 0 && rank == 0) a.lengths[b] = (int32_t)stay;
    if (CS > 1) cluster.sync();           // the others may still read this block's counts
}

constexpr int kCopy = 256, kCopyRows = 2, kCopyChunks = 4;

// Threads that share a row of so many 16-byte chunks: a power of two, about four chunks each.
__host__ __device__ inline uint32_t row_threads(uint32_t chunks) {
    uint32_t n = 1;
    while (n < 32 && n * kCopyChunks < chunks) n *= 2;
    return n;
}

// Copies a sequence's kept rows of one cache; grid (groups of rows, caches, sequences). A thread has
// two rows on the way at once, four chunks of each.
__global__ void __launch_bounds__(kCopy) evict_copy(EvictArgs a) {
    await_previous();
    const slikl_evict_cache &c = a.caches[blockIdx.y];
    const uint32_t chunks = (uint32_t)(c.row_bytes / 16), tpr = row_threads(chunks);
    const uint32_t col = threadIdx.x & (tpr - 1), mine = threadIdx.x / tpr, across = kCopy / tpr;
    for (int64_t b = blockIdx.z; b < a.B; b += gridDim.z) {
        const int32_t *kept = a.kept + b * a.budget;
        const int64_t base = a.layout_k == SLIKL_BSND ? b * a.S2 : a.cu_k[b];
        const uint4 *in = static_cast<const uint4 *>(c.in) + base * chunks;
        uint4 *out = static_cast<uint4 *>(c.out) + b * a.budget * chunks;
        for (uint32_t row = blockIdx.x * across * kCopyRows + mine; row < (uint32_t)a.budget;
             row += gridDim.x * across * kCopyRows) {
            const uint32_t next = row + across;
            const int32_t j0 = kept[row], j1 = next < (uint32_t)a.budget ? kept[next] : -1;
            const uint4 *p0 = in + (int64_t)j0 * chunks, *p1 = in + (int64_t)j1 * chunks;
            uint4 *q0 = out + (int64_t)row * chunks, *q1 = out + (int64_t)next * chunks;
            for (uint32_t k = col; k < chunks; k += kCopyChunks * tpr) {
                uint4 v0[kCopyChunks], v1[kCopyChunks];
#pragma unroll
                for (int i = 0; i < kCopyChunks; ++i) {
                    if (j0 >= 0 && k + i * tpr < chunks) v0[i] = p0[k + i * tpr];
                    if (j1 >= 0 && k + i * tpr < chunks) v1[i] = p1[k + i * tpr];
                }
#pragma unroll
                for (int i = 0; i < kCopyChunks; ++i) {
                    if (j0 >= 0 && k + i * tpr < chunks) q0[k + i * tpr] = v0[i];
                    if (j1 >= 0 && k + i * tpr < chunks) q1[k + i * tpr] = v1[i];
                }
            }
        }
    }
}

// --- host side ---------------------------------------------------------------------------------

bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

// Bytes of one tensor; none where the pointer is null.
struct Range {
    const void *p;
    int64_t n;
};

bool overlap(const Range &r, const Range &q) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(r.p), y = reinterpret_cast<uintptr_t>(q.p);
    return r.p && q.p && r.n > 0 && q.n > 0 && x < y + (uint64_t)q.n && y < x + (uint64_t)r.n;
}

}  // namespace
}  // namespace slikl

using namespace slikl;

extern "C" {

slikl_status slikl_evict(const slikl_evict_problem *problem, const slikl_evict_tensors *tensors,
                         void *stream) {
    if (!problem || !tensors) return SLIKL_ERR_PARAM_NULLPTR;
    const slikl_evict_problem &p = *problem;
    const int64_t limit = int64_t(1) << 31;
    if ((p.layout_k != SLIKL_BSND && p.layout_k != SLIKL_TND) || p.n_caches < 0 ||
        p.n_caches > SLIKL_EVICT_MAX_CACHES || p.B < 1 || p.B >= limit / 8 || p.budget < 1 ||
        p.budget >= limit || p.B * p.budget >= limit || p.sinks < 0 || p.recent < 0 ||
        p.sinks > p.budget || p.recent > p.budget - p.sinks)
        return SLIKL_ERR_PARAM_INVALID;
    int64_t T2 = p.T2;
    if (p.layout_k == SLIKL_BSND) {
        if (p.S2 < 1 || p.S2 >= limit || p.B * p.S2 >= limit) return SLIKL_ERR_PARAM_INVALID;
        T2 = p.B * p.S2;
    } else if (p.S2 < 0 || T2 < 0 || T2 >= limit) {
        return SLIKL_ERR_PARAM_INVALID;
    }
    const slikl_evict_tensors &t = *tensors;
    if ((T2 > 0 && !t.scores) || !t.kept || !t.lengths ||
        (p.layout_k == SLIKL_TND && !t.cu_seqlens_k))
        return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(t.scores, 4) || misaligned(t.cu_seqlens_k, 4) || misaligned(t.seq_used_k, 4) ||
        misaligned(t.kept, 4) || misaligned(t.lengths, 4) || misaligned(t.scores_out, 4) ||
        misaligned(t.status, 4))
        return SLIKL_ERR_PARAM_INVALID;
    for (int i = 0; i < p.n_caches; ++i) {
        const slikl_evict_cache &c = t.caches[i];
        if (c.row_bytes < 16 || c.row_bytes % 16 != 0 || c.row_bytes >= limit)
            return SLIKL_ERR_PARAM_INVALID;
        if ((T2 > 0 && !c.in) || !c.out) return SLIKL_ERR_PARAM_NULLPTR;
        if (misaligned(c.in, 16) || misaligned(c.out, 16)) return SLIKL_ERR_PARAM_INVALID;
    }
    // Scores, lengths and rows are read while others are written, and evict_copy follows the row numbers
    // of `kept` wherever they lead: nothing written may lie in an input or in another output. (A
    // sequence's length is written behind the last read of its used length.)
    const int64_t places = p.B * p.budget;
    Range in[3 + SLIKL_EVICT_MAX_CACHES] = {{t.scores, T2 * 4},
                                            {p.layout_k == SLIKL_TND ? t.cu_seqlens_k : nullptr, (p.B + 1) * 4},
                                            {t.lengths == t.seq_used_k ? nullptr : t.seq_used_k, p.B * 4}};
    Range out[4 + SLIKL_EVICT_MAX_CACHES] = {{t.kept, places * 4}, {t.lengths, p.B * 4},
                                             {t.scores_out, places * 4}, {t.status, 4}};
    for (int i = 0; i < p.n_caches; ++i) {
        in[3 + i] = {t.caches[i].in, T2 * t.caches[i].row_bytes};
        out[4 + i] = {t.caches[i].out, places * t.caches[i].row_bytes};
    }
    for (int i = 0; i < 4 + p.n_caches; ++i) {
        for (int j = 0; j < 3 + p.n_caches; ++j)
            if (overlap(out[i], in[j])) return SLIKL_ERR_PARAM_INVALID;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SLIKL_ERR_PARAM_INVALID;
    }
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        major != 10)
        return SLIKL_ERR_CUDA;

    EvictArgs a{};
    a.layout_k = p.layout_k;
    a.n_caches = p.n_caches;
    a.B = p.B;
    a.S2 = p.layout_k == SLIKL_BSND ? p.S2 : 0;
    a.T2 = T2;
    a.budget = (int32_t)p.budget;
    a.sinks = (int32_t)p.sinks;
    a.recent = (int32_t)p.recent;
    a.scores = t.scores;
    a.cu_k = t.cu_seqlens_k;
    a.used_k = t.seq_used_k;
    a.kept = t.kept;
    a.lengths = t.lengths;
    a.scores_out = t.scores_out;
    a.status = t.status;
    int64_t blocks = 0;
    for (int i = 0; i < p.n_caches; ++i) {
        a.caches[i] = t.caches[i];
        const int64_t rows = kCopyRows * (kCopy / row_threads((uint32_t)(t.caches[i].row_bytes / 16)));
        blocks = std::max(blocks, (p.budget + rows - 1) / rows);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Sequences of up to 8192 rows, eight a thread, go through one block: a cluster's barriers cost more
    // than they share out. (The one-row form is right for a length that breaks the promise only with
    // its passes, which it lacks: it is for lengths that the tensors themselves bound.)
    const int64_t range = p.layout_k == SLIKL_BSND ? p.S2 : p.S2 > 0 ? std::min(p.S2, T2) : T2;
    const int64_t bound = p.layout_k == SLIKL_BSND ? p.S2 : T2;
    if (bound <= kChoose) evict_choose<1, 1><<<(unsigned)p.B, kChoose, 0, s>>>(a);
    else if (range <= 8192) evict_choose<1, 8><<<(unsigned)p.B, kChoose, 0, s>>>(a);
    else evict_choose<8, 16><<<(unsigned)p.B * 8, kChoose, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    if (p.n_caches > 0) {
        const dim3 grid((unsigned)blocks, (unsigned)p.n_caches, (unsigned)std::min<int64_t>(p.B, 65535));
        if (launch_next(evict_copy, grid, kCopy, 0, s, a) != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    return SLIKL_OK;
}

}  // extern "C"
