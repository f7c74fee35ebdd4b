// Cutting a cache to the key rows with the highest scores (slikl_evict; contract in
// include/slikl.h).
//
// evict_choose finds, for each sequence, the score of the last row that stays by a radix select
// over order-preserving integers (three passes of 11, 11 and 10 bits), then walks the rows in
// order and writes the kept ones behind one another. evict_copy moves the caches' rows.
#include "slikl_common.cuh"

namespace slikl {
namespace {

constexpr int kChoose = 1024;         // threads of evict_choose
constexpr int kBins = 2048;

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

// Exclusive prefix of v over the block and the block's total.
__device__ int block_prefix(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kChoose) evict_choose(EvictArgs a) {
    __shared__ int bins[kBins];
    __shared__ int warp_sums[32];
    __shared__ uint32_t found_bin;
    __shared__ int found_above;
    const int64_t b = blockIdx.x;
    const Sequence q = sequence_of(a, b, threadIdx.x == 0);
    const int32_t n = q.n, stay = min(n, a.budget);
    const bool all = n <= a.budget;
    const int32_t lo = all ? 0 : a.sinks, hi = all ? 0 : n - a.recent;   // rows that scores decide on
    const int32_t wanted = all ? 0 : a.budget - a.sinks - a.recent;
    const float *scores = a.scores + q.base;

    // the order number of the wanted-th of them, and how many rows with that number stay
    uint32_t prefix = 0, mask = 0;
    int left = wanted;
    if (wanted > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
            for (int i = threadIdx.x; i < kBins; i += kChoose) bins[i] = 0;
            __syncthreads();
            for (int32_t j = lo + threadIdx.x; j < hi; j += kChoose) {
                const uint32_t o = order_of(scores[j]);
                if ((o & mask) == prefix) atomicAdd(&bins[(o >> shift) & ((1u << width) - 1)], 1);
            }
            __syncthreads();
            // thread i holds bins 2047 - 2i and 2046 - 2i: the prefix runs from the highest bin
            const int h0 = bins[kBins - 1 - 2 * threadIdx.x], h1 = bins[kBins - 2 - 2 * threadIdx.x];
            int total;
            const int above = block_prefix(h0 + h1, warp_sums, total);
            if (above < left && left <= above + h0 + h1) {
                const bool first = left <= above + h0;
                found_bin = kBins - 1 - 2 * threadIdx.x - (first ? 0 : 1);
                found_above = above + (first ? 0 : h0);
            }
            __syncthreads();
            prefix |= found_bin << shift;
            mask |= ((1u << width) - 1) << shift;
            left -= found_above;
            __syncthreads();
        }
    }

    int32_t *kept = a.kept + b * a.budget;
    float *out = a.scores_out ? a.scores_out + b * a.budget : nullptr;
    int at = 0, equals = 0;
    for (int32_t j0 = 0; j0 < n; j0 += kChoose) {
        const int32_t j = j0 + threadIdx.x;
        const float x = j < n ? scores[j] : 0.f;
        const bool decided = j >= lo && j < hi;
        const uint32_t o = order_of(x);
        const bool equal = decided && wanted > 0 && o == prefix;
        int total;
        const int rank = equals + block_prefix(equal, warp_sums, total);
        equals += total;
        const bool stays = j < n && (!decided || (wanted > 0 && (o > prefix || (equal && rank < left))));
        const int place = at + block_prefix(stays, warp_sums, total);
        at += total;
        if (stays) {
            kept[place] = j;
            if (out) out[place] = x;
        }
    }
    for (int32_t j = stay + threadIdx.x; j < a.budget; j += kChoose) {
        kept[j] = -1;
        if (out) out[j] = 0.f;
    }
    if (threadIdx.x == 0) a.lengths[b] = stay;
}

__global__ void __launch_bounds__(256) evict_copy(EvictArgs a) {
    const slikl_evict_cache &c = a.caches[blockIdx.y];
    const int64_t chunks = c.row_bytes / 16, total = a.B * a.budget * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / chunks, part = i - row * chunks, b = row / a.budget;
        const int32_t j = a.kept[row];
        if (j < 0) continue;
        const int64_t base = a.layout_k == SLIKL_BSND ? b * a.S2 : a.cu_k[b];
        static_cast<uint4 *>(c.out)[row * chunks + part] =
            static_cast<const uint4 *>(c.in)[(base + j) * chunks + part];
    }
}

// --- host side ---------------------------------------------------------------------------------

bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

bool overlap(const void *p, int64_t n, const void *q, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && x < y + (uint64_t)m && y < x + (uint64_t)n;
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
        p.n_caches > SLIKL_EVICT_MAX_CACHES || p.B < 1 || p.B >= limit || p.budget < 1 ||
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
    const int64_t places = p.B * p.budget;
    if (t.scores_out && overlap(t.scores, T2 * 4, t.scores_out, places * 4))
        return SLIKL_ERR_PARAM_INVALID;
    for (int i = 0; i < p.n_caches; ++i) {
        const slikl_evict_cache &c = t.caches[i];
        if (c.row_bytes < 16 || c.row_bytes % 16 != 0 || c.row_bytes >= limit)
            return SLIKL_ERR_PARAM_INVALID;
        if ((T2 > 0 && !c.in) || !c.out) return SLIKL_ERR_PARAM_NULLPTR;
        if (misaligned(c.in, 16) || misaligned(c.out, 16)) return SLIKL_ERR_PARAM_INVALID;
    }
    // rows are copied while others are still to be read: nothing written may lie in an input, and
    // no two outputs may share memory
    for (int i = 0; i < p.n_caches; ++i) {
        const slikl_evict_cache &c = t.caches[i];
        for (int j = 0; j < p.n_caches; ++j) {
            const slikl_evict_cache &d = t.caches[j];
            if (overlap(c.out, places * c.row_bytes, d.in, T2 * d.row_bytes) ||
                (i != j && overlap(c.out, places * c.row_bytes, d.out, places * d.row_bytes)))
                return SLIKL_ERR_PARAM_INVALID;
        }
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
    int64_t most = 0;
    for (int i = 0; i < p.n_caches; ++i) {
        a.caches[i] = t.caches[i];
        most = most > t.caches[i].row_bytes ? most : t.caches[i].row_bytes;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    evict_choose<<<(unsigned)p.B, kChoose, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    if (p.n_caches > 0) {
        const int64_t blocks = (places * (most / 16) + 255) / 256;
        evict_copy<<<dim3((unsigned)(blocks < 148 * 16 ? blocks : 148 * 16), (unsigned)p.n_caches),
                     256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    return SLIKL_OK;
}

}  // extern "C"
