// The weight that a call's query rows put on each key row (slikl_key_weights; formula and
// contract in include/slikl.h).
//
// Weights are summed as 64-bit integers, so the order of the additions does not change the result.
// The floor is the read of the slots (an index and a weight, 8 bytes each).
#include "slikl_common.cuh"

namespace slikl {
namespace {

struct WeightArgs {
    int layout_q, layout_k, K;
    int64_t B, S1, S2, T1, T2;
    const int32_t *idx, *cu_q, *cu_k, *used_q, *used_k;
    const float *weights, *scores;
    float *out;
    float decay;
    float one;                // 2^u: the units of a weight of 1
    unsigned long long *sums; // [T2], in units
    uint32_t *status;
};

__device__ __forceinline__ void flag(const WeightArgs &a, uint32_t bit) {
    if (a.status) set_status(a.status, bit);
}

// The keys that query row t's slots may name: rows [base, base + used) of the key tensor, of the
// `count` that its batch has.
struct RowKeys {
    int64_t base;
    int32_t count, used;
    bool in_use;              // a row whose indices are read
};

__device__ RowKeys row_keys(const WeightArgs &a, int64_t t) {
    RowKeys r{0, 0, 0, false};
    int64_t b, q0, q1;
    if (a.layout_q == SLIKL_BSND) {
        b = t / a.S1;
        q0 = b * a.S1;
        q1 = q0 + a.S1;
    } else {
        int64_t lo = 0, hi = a.B - 1;       // the last batch that begins at or before t
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (a.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
        }
        b = lo;
        q0 = a.cu_q[b];
        q1 = a.cu_q[b + 1];
        if (t < q0 || t >= q1) return r;
    }
    if (a.used_q && t - q0 >= a.used_q[b]) return r;
    if (a.layout_k == SLIKL_BSND) {
        r.base = b * a.S2;
        r.count = (int32_t)a.S2;
    } else {
        const int64_t k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        if (k0 < 0 || k1 < k0 || k1 > a.T2) return r;
        r.base = k0;
        r.count = (int32_t)(k1 - k0);
    }
    r.in_use = true;
    r.used = r.count;
    if (a.used_k) r.used = max(0, min(a.used_k[b], r.count));
    return r;
}

// A weight in units of 2^-u.
__device__ __forceinline__ unsigned long long units(const WeightArgs &a, float w) {
    if (!(w >= 0.f && w <= 2.f)) {
        flag(a, SLIKL_DEV_BAD_WEIGHT);
        w = w > 2.f ? 2.f : 0.f;
    }
    return (unsigned long long)__float2ll_rn(w * a.one);
}

// Whether a slot of a row in use names one of its keys; flags an index that breaks the contract.
__device__ __forceinline__ bool names_key(const WeightArgs &a, const RowKeys &r, int32_t v) {
    if (v < -1 || v >= r.count) flag(a, SLIKL_DEV_INDEX_OUT_OF_RANGE);
    return v >= 0 && v < r.used;
}

__global__ void __launch_bounds__(256) weights_scatter(WeightArgs a) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < a.T1;
         t += (int64_t)gridDim.x * 8) {
        const RowKeys r = row_keys(a, t);
        if (!r.in_use) continue;
        const int64_t o = t * a.K;
        for (int j = lane; j < a.K; j += 32) {
            const int32_t v = a.idx[o + j];
            if (names_key(a, r, v)) atomicAdd(a.sums + r.base + v, units(a, a.weights[o + j]));
        }
    }
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
    if (a.scores) s += (double)a.decay * (double)a.scores[key];
    return (float)s;
}

__global__ void __launch_bounds__(256) weights_finish(WeightArgs a) {
    if (blockIdx.x == 0 && a.status) check_batches(a);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < a.T2) a.out[i] = finished(a, a.sums[i], i);
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
    size_t sums, total;
};

Layout make_workspace(int64_t T2) {
    Layout L;
    L.sums = 0;
    L.total = align256(sizeof(unsigned long long) * (size_t)T2) + 256;
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
                               const slikl_key_weights_tensors *tensors, float decay,
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
    if (!(decay >= 0.f) || decay > 3.4e38f) return SLIKL_ERR_PARAM_INVALID;
    if ((T1 > 0 && !tensors->weights) || (T2 > 0 && !tensors->out) || !workspace)
        return SLIKL_ERR_PARAM_NULLPTR;
    if (misaligned(tensors->weights, 4) || misaligned(tensors->scores, 4) ||
        misaligned(tensors->out, 4) || misaligned(tensors->status, 4) || misaligned(workspace, 256))
        return SLIKL_ERR_PARAM_INVALID;
    const Layout L = make_workspace(T2);
    if (workspace_bytes < L.total) return SLIKL_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        major != 10)
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
    a.scores = decay == 0.f ? nullptr : tensors->scores;
    a.out = tensors->out;
    a.decay = decay;
    int bits = 0;                    // ceil(log2(slots)): the sum stays below 2^(1 + bits + u) <= 2^62
    while ((int64_t(1) << bits) < T1 * pr.topk) ++bits;
    const int u = 61 - bits < 40 ? 61 - bits : 40;
    a.one = (float)(int64_t(1) << u);
    a.sums = reinterpret_cast<unsigned long long *>(static_cast<char *>(workspace) + L.sums);
    a.status = tensors->status;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(a.sums, 0, sizeof(*a.sums) * (size_t)T2, s) != cudaSuccess)
        return SLIKL_ERR_CUDA;
    if (T1 > 0) {
        const int64_t blocks = (T1 + 7) / 8;
        weights_scatter<<<(unsigned)(blocks < 148 * 8 ? blocks : 148 * 8), 256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SLIKL_ERR_CUDA;
    }
    weights_finish<<<(unsigned)((T2 + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SLIKL_OK : SLIKL_ERR_CUDA;
}

}  // extern "C"
