// The weight that a call's query rows put on each key row (slikl_key_weights; formula and
// contract in include/slikl.h).
//
// Weights are summed as 64-bit integers, so the order of the additions does not change the result. The
// floor is the read of the slots (an index and a weight, 8 bytes each); what has to be kept from
// bounding the call instead is the scattered additions. 64-bit additions to global memory, one a
// slot, run at 128 G/s on B200 however far apart the keys are (147 us for 16.8 M slots over 131072
// keys, seven times the floor) and slower on few keys. So sums are kept in shared memory, as 32-bit
// additions that return what was there; a carry out of the low word and the high word of a large weight
// go their own way. All rows of a batch name the same keys, so a block reads a
// stretch of the batch's slots without looking where rows begin. Two forms:
//   weights_direct  few slots a batch (a decoding step): a block owns a chunk of a batch's keys, reads
//                   all of the batch's slots, keeps both words and writes the chunk's result: one
//                   launch and no workspace;
//   weights_split   else: blocks share a batch's slots, keep the low words of up to 55296 keys (larger
//                   ranges are covered by several blocks that read the same slots, from L2 mostly)
//                   and add them to 64-bit sums in the workspace once, which weights_clear has set to
//                   zero; weights_finish makes the result. Each starts up while the one before it runs.
// Measured on B200 on the device (replays of a graph): 4 to 5 us for 32 rows of 2048 slots over 8192 keys
// each, 19 us for 8.4 M slots over 4096 keys, a quarter of them empty (58.7 MB, which take 9.1 us at the copy
// rate), 68 us for 16.8 M over 131072 (floor 21; three blocks read each slot). The
// split form is bound by its instructions (issue slots 58 %, the integer pipe 56 % in use) and by the
// latency of its loads between them; more loads on their way, by registers or through shared memory,
// were no faster.
#include <float.h>

#include <algorithm>

#include "slikl_common.cuh"

namespace slikl {
namespace {

struct WeightArgs {
    int layout_q, layout_k, K;
    int64_t B, S1, S2, T1, T2;
    const int32_t *idx, *cu_q, *cu_k, *used_q, *used_k;
    const float *weights, *scores;
    float *out;
    double decay;
    float one;                // 2^u: the units of a weight of 1
    unsigned long long *sums; // [T2], in units
    uint32_t *bad_k;          // weights_clear's finding that cu_seqlens_k is unusable; null: it has not looked
    int64_t first_batch;      // of weights_split's grid
    uint32_t *status;
};

__device__ __forceinline__ void flag(const WeightArgs &a, uint32_t bit) {
    if (a.status) set_status(a.status, bit);
}

// A batch's slots [begin, end) of its rows in use, and the keys that they may name: rows [base, base +
// used) of the key tensor, of the `count` that the batch has. Empty where cu_seqlens is unusable.
struct Batch {
    int64_t begin, end, base;
    int32_t count, used;
};

__device__ Batch batch_of(const WeightArgs &a, int64_t b) {
    Batch r{0, 0, 0, 0, 0};
    if (a.layout_k == SLIKL_BSND) {
        r.base = b * a.S2;
        r.count = (int32_t)a.S2;
    } else {
        const int64_t k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        if (k0 < 0 || k1 < k0 || k1 > a.T2) return r;
        r.base = k0;
        r.count = (int32_t)(k1 - k0);
    }
    r.used = a.used_k ? max(0, min(a.used_k[b], r.count)) : r.count;
    int64_t q0, qn;
    if (a.layout_q == SLIKL_BSND) {
        q0 = b * a.S1;
        qn = a.S1;
    } else {
        q0 = a.cu_q[b];
        qn = a.cu_q[b + 1] - q0;
        if (q0 < 0 || qn < 0 || q0 + qn > a.T1) return r;
    }
    if (a.used_q) qn = max((int64_t)0, min((int64_t)a.used_q[b], qn));
    r.begin = q0 * a.K;
    r.end = (q0 + qn) * a.K;
    return r;
}

// A weight, times 2^u in fp32 (exact), as an integer; bad ones are flagged and cut to [0, 2].
__device__ __forceinline__ uint64_t units(const WeightArgs &a, float x) {
    if (!(x >= 0.f && x <= 2.f * a.one)) {
        flag(a, SLIKL_DEV_BAD_WEIGHT);
        x = x > 0.f ? 2.f * a.one : 0.f;
    }
    return (uint64_t)__float2ll_rn(x);
}

// Four slots a thread, v their keys in the chunk (at least `named` where a slot does not count) and w
// their weights: added to the low words. Of the 32 words behind the chunk, the lane's takes what does
// not count, as zero, so that the usual step has no branch. more(key, n) adds n times 2^32. Weights of
// 2^(32-u) and more, bad ones and carries are seen to behind the additions.
template <typename F>
__device__ __forceinline__ void add_four(const WeightArgs &a, const uint32_t *v, const float *w,
                                         uint32_t named, uint32_t keys, uint32_t *low, const F &more) {
    const uint32_t small = __float_as_uint(4294967296.f);     // bits of 0 <= x < 2^32 are below
    float x[4];
    const uint32_t spare = keys + (threadIdx.x & 31);
    uint32_t most = 0, carries = 0;
    bool some = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) some |= v[k] < named;
    // (rows are sorted more often than not, and all of a warp's slots outside the chunk then)
    if (!__any_sync(0xffffffffu, some)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = v[k] < named ? w[k] * a.one : 0.f;
        most = max(most, __float_as_uint(x[k]));
    }
    if (most < small) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = __float2uint_rn(x[k]);
            carries |= (uint32_t)(atomicAdd(low + (v[k] < named ? v[k] : spare), lo) > ~lo) << k;
        }
        if (!carries) return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (v[k] >= named || (most < small && !(carries >> k & 1))) continue;
        uint32_t hi = 1;
        if (most >= small) {
            const uint64_t u = units(a, x[k]);
            const uint32_t lo = (uint32_t)u;
            hi = (uint32_t)(u >> 32) + (atomicAdd(low + v[k], lo) > ~lo);
        }
        if (hi) more(v[k], hi);
    }
}

// Whether this thread sees cu_seqlens_k break its contract (0 .. T2, non-decreasing). All batches' key ranges
// are empty then, as in the gradient: ranges that overlap or leave rows out have no meaning.
__device__ __forceinline__ bool sees_bad_keys(const WeightArgs &a) {
    bool bad = false;
#pragma unroll 4
    for (int64_t b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int64_t k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        bad |= k1 < k0 || (b == 0 && k0 != 0) || (b == a.B - 1 && k1 != a.T2);
    }
    return bad;
}

// Adds the slots of [begin, end) that name a key of [first, first + keys) to the low words. Flags
// indices that break the contract. A step is four slots a thread, a block's width apart; loads run
// ahead, the indices two steps and the weights, read only where the slot counts, one.
template <int THREADS, typename F>
__device__ __forceinline__ void add_some(const WeightArgs &a, const Batch &r, int64_t begin, int64_t end,
                                         int32_t first, int32_t keys, uint32_t *low, const F &more) {
    constexpr uint32_t STEP = 4 * THREADS;
    const uint32_t named = (uint32_t)max(0, min(keys, r.used - first));
    const uint32_t slots = (uint32_t)(end - begin);
    const int32_t *idx = a.idx + begin;
    const float *weights = a.weights + begin;
    uint32_t largest = 0;     // of the indices plus one
    auto indices = [&](uint32_t i, uint32_t *v) {
        const int32_t *p = idx + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k * THREADS < slots ? p[k * THREADS] : -1;
    };
    auto load = [&](uint32_t i, uint32_t *v, float *w) {
        const float *p = weights + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            largest = max(largest, v[k] + 1);
            v[k] -= first;
            w[k] = v[k] < named ? p[k * THREADS] : 0.f;
        }
    };
    uint32_t v[3][4], i = threadIdx.x;
    float w[2][4];
    indices(i, v[0]);
    indices(i + STEP, v[1]);
    load(i, v[0], w[0]);
    for (uint32_t all = 0; all < slots; all += 6 * STEP, i += 6 * STEP) {   // the same steps for all threads
#pragma unroll
        for (int j = 0; j < 6; ++j) {
            if (j && all + j * STEP >= slots) break;
            indices(i + (j + 2) * STEP, v[(j + 2) % 3]);
            load(i + (j + 1) * STEP, v[(j + 1) % 3], w[(j + 1) % 2]);
            add_four(a, v[j % 3], w[j % 2], named, keys, low, more);
        }
    }
    if (largest > (uint32_t)r.count) flag(a, SLIKL_DEV_INDEX_OUT_OF_RANGE);
}

// What the per-batch arrays promise, looked at once by the first block of weights_finish.
__device__ void check_batches(const WeightArgs &a) {
    for (int64_t b = threadIdx.x; b < a.B; b += blockDim.x) {
        int64_t qn = a.S1, kn = a.S2;
        if (a.layout_q == SLIKL_TND) {
            const int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
            qn = c1 - c0;
            if (qn < 0 || (b == 0 && c0 != 0) || (b == a.B - 1 && c1 != a.T1))
                flag(a, SLIKL_DEV_BAD_CU_SEQLENS_Q);
        }
        if (a.layout_k == SLIKL_TND) {
            const int64_t c0 = a.cu_k[b], c1 = a.cu_k[b + 1];
            kn = c1 - c0;
            if (kn < 0 || (b == 0 && c0 != 0) || (b == a.B - 1 && c1 != a.T2))
                flag(a, SLIKL_DEV_BAD_CU_SEQLENS_K);
        }
        if ((a.used_q && (a.used_q[b] < 0 || a.used_q[b] > qn)) ||
            (a.used_k && (a.used_k[b] < 0 || a.used_k[b] > kn)))
            flag(a, SLIKL_DEV_BAD_SEQ_USED);
    }
}

__device__ __forceinline__ float finished(const WeightArgs &a, unsigned long long sum, int64_t key) {
    // both products and their sum in fp64: the history loses no more than its own fp32 rounding
    double s = (double)(long long)sum * (1.0 / (double)a.one);
    if (a.scores) s += a.decay * (double)a.scores[key];
    return (float)s;
}

constexpr int kDirectThreads = 512, kDirectKeys = 2048;
constexpr int kSplitThreads = 1024, kSplitKeys = 55296;       // 216 KB of low words

// Whether cu_seqlens_k is usable: each block of the direct form looks itself, one load a thread, at up to 512
// batches; for more weights_clear has looked (1024 batches of 2048 keys 17.5 us instead of 18.5, 8192 of
// 256 82 instead of 133; 15.5 and 74 without a look).
constexpr int kMostLooks = 512;

// grid (chunks of keys, batches).
__global__ void __launch_bounds__(kDirectThreads) weights_direct(WeightArgs a, int chunk) {
    __shared__ uint32_t low[kDirectKeys + 32], high[kDirectKeys];
    const int64_t b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0 && a.status) check_batches(a);
    const Batch r = batch_of(a, b);
    if (a.layout_k == SLIKL_TND) {
        if (blockIdx.x > 0 && (int64_t)blockIdx.x * chunk >= r.count) return;
        bool bad;
        if (a.bad_k) {
            await_previous();
            bad = *a.bad_k != 0;
        } else {
            bad = sees_bad_keys(a);
        }
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0)
                for (int64_t key = b * kDirectThreads + threadIdx.x; key < a.T2; key += a.B * kDirectThreads)
                    a.out[key] = finished(a, 0, key);
            return;
        }
    }
    for (int64_t first = (int64_t)blockIdx.x * chunk; first < r.count;
         first += (int64_t)gridDim.x * chunk) {
        const int32_t keys = (int32_t)min((int64_t)chunk, r.count - first);
        for (int i = threadIdx.x; i < keys; i += kDirectThreads) low[i] = high[i] = 0;
        __syncthreads();
        add_some<kDirectThreads>(a, r, r.begin, r.end, (int32_t)first, keys, low,
                                 [&](uint32_t k, uint32_t n) { atomicAdd(&high[k], n); });
        __syncthreads();
        for (int i = threadIdx.x; i < keys; i += kDirectThreads) {
            const int64_t key = r.base + first + i;
            a.out[key] = finished(a, (unsigned long long)high[i] << 32 | low[i], key);
        }
        __syncthreads();
    }
}

// A kernel instead of a memset: weights_split starts while it runs.
__global__ void __launch_bounds__(512) weights_clear(WeightArgs a, int64_t pairs) {
    let_next_start();         // weights_split, weights_finish
    ulonglong2 *sums = reinterpret_cast<ulonglong2 *>(a.sums);
    for (int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x; i < pairs; i += (int64_t)gridDim.x * 512)
        sums[i] = make_ulonglong2(0, 0);
    if (a.bad_k && blockIdx.x == 0) {
        const int bad = __syncthreads_or(sees_bad_keys(a));
        if (threadIdx.x == 0) *a.bad_k = bad != 0;
    }
}

// grid (chunks of keys, splits of the slots, batches). Blocks next to one another read the same slots.
__global__ void __launch_bounds__(kSplitThreads) weights_split(WeightArgs a, int chunk) {
    extern __shared__ uint32_t low[];
    let_next_start();         // weights_finish
    const Batch r = batch_of(a, a.first_batch + blockIdx.z);
    const int64_t slots = r.end - r.begin;
    const int64_t begin = r.begin + slots * blockIdx.y / gridDim.y;
    const int64_t end = r.begin + slots * (blockIdx.y + 1) / gridDim.y;
    for (int64_t first = (int64_t)blockIdx.x * chunk; begin < end && first < r.used;
         first += (int64_t)gridDim.x * chunk) {
        const int32_t keys = (int32_t)min((int64_t)chunk, r.used - first);
        unsigned long long *sums = a.sums + r.base + first;
        for (int i = threadIdx.x; i < keys; i += kSplitThreads) low[i] = 0;
        await_previous();     // carries go to the sums
        __syncthreads();
        const auto more = [&](uint32_t k, uint32_t n) { atomicAdd(sums + k, (unsigned long long)n << 32); };
        add_some<kSplitThreads>(a, r, begin, end, (int32_t)first, keys, low, more);
        __syncthreads();
        for (int i = threadIdx.x; i < keys; i += kSplitThreads)
            if (low[i]) atomicAdd(sums + i, (unsigned long long)low[i]);
        __syncthreads();
    }
    await_previous();         // for blocks without slots too: weights_finish waits for this kernel alone
}

__global__ void __launch_bounds__(256) weights_finish(WeightArgs a) {
    await_previous();
    if (blockIdx.x == 0 && a.status) check_batches(a);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool none = a.bad_k && *a.bad_k;
    if (i < a.T2) a.out[i] = finished(a, none ? 0 : a.sums[i], i);
}

// --- host side ---------------------------------------------------------------------------------

// The problem with the fields that this operator does not read set to supported values.
slikl_problem index_problem(const slikl_problem &p) {
    slikl_problem q = p;
    q.dtype = SLIKL_BF16;
    q.deterministic = 0;
    q.N1 = 1;
    q.D = 64;
    return q;
}

struct Layout {
    size_t sums, bad_k, total;
};

Layout make_workspace(int64_t T2) {
    Layout L;
    L.sums = 0;
    L.bad_k = align256(sizeof(unsigned long long) * (size_t)T2);
    L.total = L.bad_k + 256;
    return L;
}

bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

}  // namespace
}  // namespace slikl

using namespace slikl;

extern "C" {

slikl_status slikl_key_weights_workspace_size(const slikl_problem *problem,
                                              size_t *workspace_bytes) {
    if (!workspace_bytes) return SLIKL_ERR_INNER_NULLPTR;
    if (!problem) return SLIKL_ERR_PARAM_NULLPTR;
    const slikl_problem pr = index_problem(*problem);
    size_t unused = 0;
    slikl_options scatter{};
    scatter.dk_path = SLIKL_DK_SCATTER;
    const slikl_status st = slikl_grad_workspace_size_ex(&pr, &scatter, &unused);
    if (st != SLIKL_OK) return st;
    *workspace_bytes = make_workspace(pr.layout_k == SLIKL_BSND ? pr.B * pr.S2 : pr.T2).total;
    return SLIKL_OK;
}

slikl_status slikl_key_weights(const slikl_problem *problem,
                               const slikl_key_weights_tensors *tensors, double decay,
                               void *workspace, size_t workspace_bytes, void *stream,
                               const slikl_options *options) {
    if (!problem || !tensors) return SLIKL_ERR_PARAM_NULLPTR;
    const slikl_problem pr = index_problem(*problem);
    slikl_tensors tn{};
    tn.sparse_indices = tensors->sparse_indices;
    tn.cu_seqlens_q = tensors->cu_seqlens_q;
    tn.cu_seqlens_k = tensors->cu_seqlens_k;
    slikl_status st = check_index_call(&pr, &tn, options, false);
    if (st != SLIKL_OK) return st;
    const int64_t T1 = pr.layout_q == SLIKL_BSND ? pr.B * pr.S1 : pr.T1;
    const int64_t T2 = pr.layout_k == SLIKL_BSND ? pr.B * pr.S2 : pr.T2;
    if (!(decay >= 0.0) || decay > DBL_MAX) return SLIKL_ERR_PARAM_INVALID;
    if ((T1 > 0 && !tensors->weights) || (T2 > 0 && !tensors->out) || !workspace)
        return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(tensors->weights, 4) || misaligned(tensors->scores, 4) ||
        misaligned(tensors->out, 4) || misaligned(tensors->status, 4) || misaligned(workspace, 256))
        return SLIKL_ERR_PARAM_INVALID;
    const Layout L = make_workspace(T2);
    if (workspace_bytes < L.total) return SLIKL_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0, major = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10)
        return SLIKL_ERR_CUDA;
    if (T2 == 0) return SLIKL_OK;

    WeightArgs a{};
    a.layout_q = pr.layout_q;
    a.layout_k = pr.layout_k;
    a.K = (int)pr.topk;
    a.B = pr.B;
    a.S1 = pr.S1;
    a.S2 = pr.S2;
    a.T1 = T1;
    a.T2 = T2;
    a.idx = tensors->sparse_indices;
    a.cu_q = tensors->cu_seqlens_q;
    a.cu_k = tensors->cu_seqlens_k;
    a.used_q = options ? options->seq_used_q : nullptr;
    a.used_k = options ? options->seq_used_k : nullptr;
    a.weights = tensors->weights;
    a.scores = decay == 0.0 ? nullptr : tensors->scores;
    a.out = tensors->out;
    a.decay = decay;
    int bits = 0;                    // ceil(log2(slots)): the sum stays below 2^(1 + bits + u) <= 2^62
    while ((int64_t(1) << bits) < T1 * pr.topk) ++bits;
    const int u = 61 - bits < 40 ? 61 - bits : 40;
    a.one = (float)(int64_t(1) << u);
    a.sums = reinterpret_cast<unsigned long long *>(static_cast<char *>(workspace) + L.sums);
    if (pr.layout_k == SLIKL_TND)
        a.bad_k = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + L.bad_k);
    a.status = tensors->status;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // longest key range: known, promised, or all keys
    const int64_t range = std::min(pr.S2 > 0 ? pr.S2 : T2, T2);
    // A block of the direct form reads every slot of its batch, so that form is for few of them: up to
    // 65536 a batch on average. Measured on the device with equal batches, direct / split: 8192 slots of one
    // batch of 4096 keys 5.2 / 7.3 us, 16384 7.2 / 8.1, 32768 10.3 / 8.2, 65536 17.5 / 8.2; of 32 batches of
    // 8192 keys 7.2 / 9.3, 9.5 / 9.8, 14.4 / 11.6, 24.6 / 16.4: they meet near 20000 slots, above which the
    // direct form saves the host two launches. Neither form looks at how uneven batches are, and the longest
    // sets the time: 8192 rows beside 31 sequences of 128 (2048 slots a row) 1755 us where 32 equal ones take
    // 173, a prompt of 3000 rows beside 127 single tokens 1700 us (direct).
    if (T1 * pr.topk <= 65536 * pr.B && pr.B <= 65535) {
        // chunks of 256 to 2048 keys, two blocks a multiprocessor where there are as many
        int64_t chunk = 256;
        while (chunk < kDirectKeys && pr.B * ((range + chunk - 1) / chunk) > 2 * sms) chunk *= 2;
        const int64_t chunks = std::min<int64_t>((range + chunk - 1) / chunk, 1 << 20);
        const dim3 grid((unsigned)chunks, (unsigned)pr.B);
        if (a.bad_k && pr.B > kMostLooks) {
            weights_clear<<<1, 512, 0, s>>>(a, 0);
            if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
            return launch_next(weights_direct, grid, kDirectThreads, 0, s, a, (int)chunk) == cudaSuccess
                       ? SLIKL_OK
                       : SLIKL_ERR_CUDA;
        }
        a.bad_k = nullptr;
        weights_direct<<<grid, kDirectThreads, 0, s>>>(a, (int)chunk);
        return cudaGetLastError() == cudaSuccess ? SLIKL_OK : SLIKL_ERR_CUDA;
    }
    const int64_t pairs = (T2 + 1) / 2;
    weights_clear<<<(unsigned)std::min<int64_t>((pairs + 511) / 512, 2 * sms), 512, 0, s>>>(a, pairs);
    if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    if (T1 > 0) {
        const int64_t chunks = (range + kSplitKeys - 1) / kSplitKeys;
        const int64_t chunk = (range + chunks - 1) / chunks;
        const size_t smem = sizeof(uint32_t) * (size_t)(chunk + 32);
        // as many splits as fill the multiprocessors, each of 4096 slots at least
        const int64_t splits =
            std::max<int64_t>(1, std::min(sms / (chunks * pr.B), (T1 * pr.topk / pr.B + 4095) / 4096));
        if (cudaFuncSetAttribute(weights_split, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(sizeof(uint32_t) * (kSplitKeys + 32))) != cudaSuccess)
            return SLIKL_ERR_CUDA;
        WeightArgs part = a;
        // the grid's third dimension holds 65535 batches
        for (int64_t b = 0; b < pr.B; b += 65535) {
            part.first_batch = b;
            const dim3 grid((unsigned)chunks, (unsigned)splits, (unsigned)std::min<int64_t>(pr.B - b, 65535));
            if (launch_next(weights_split, grid, kSplitThreads, smem, s, part, (int)chunk) != cudaSuccess)
                return SLIKL_ERR_CUDA;
        }
    }
    const dim3 grid((unsigned)((T2 + 255) / 256));
    return launch_next(weights_finish, grid, 256, 0, s, a) == cudaSuccess ? SLIKL_OK : SLIKL_ERR_CUDA;
}

}  // extern "C"
