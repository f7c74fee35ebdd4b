// Argument marshalling of the operators around slikl_grad for torch tensors: checks types, shapes,
// strides and devices, allocates outputs and workspaces with torch's allocator on the current
// stream, fills the structs of include/slikl.h and calls libslikl.so. In C++ because these
// operators are called for a handful of rows too: the same marshalling in Python took 20 to 40 us a
// call, ten times what such a call takes on the GPU.
//
// Functions return (status code, outputs..); a refused argument raises ValueError.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>

#include "slikl.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;
using MaybeStream = std::optional<c10::Stream>;

namespace {

template <typename... A>
[[noreturn]] void refuse(A &&...parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw py::value_error(s.str());
}

std::string placed(const std::string &name, const char *side) { return side ? name + "_" + side : name; }

// Device address of a contiguous tensor on this device with this type (and shape).
template <typename P = void>
P *address(const Tensor &t, const std::string &name, const at::Device &dev, at::ScalarType type,
           std::optional<at::IntArrayRef> shape = std::nullopt) {
    if (t.device() != dev || t.scalar_type() != type || !t.is_contiguous() ||
        (shape && t.sizes() != *shape)) {
        std::ostringstream want;
        if (shape) want << " of shape " << *shape;
        refuse(name, " must be a contiguous ", c10::toString(type), " tensor on ", dev, want.str(), ", not ",
               c10::toString(t.scalar_type()), " ", t.sizes(), " on ", t.device());
    }
    return static_cast<P *>(t.data_ptr());
}

// (torch::empty and select go through the dispatcher, 1.2 us each time)
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// A contiguous tensor of this shape in t's memory, `offset` elements in.
Tensor part_of(const Tensor &t, int64_t offset, at::IntArrayRef shape) {
    Tensor v = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
    v.unsafeGetTensorImpl()->set_storage_offset(t.storage_offset() + offset);
    v.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return v;
}

// Elements from one row to the next of t [B, S, N, D] or [T, N, D] whose heads are dense.
int64_t row_stride(const Tensor &t, const std::string &name) {
    const auto shape = t.sizes();
    const auto st = t.strides();
    const int64_t n = t.dim(), N = shape[n - 2], D = shape[n - 1], dense = N * D;
    if (t.is_contiguous()) return dense;
    if (st[n - 1] != 1 || (N > 1 && st[n - 2] != D))
        refuse(name, ": the heads of a row must be contiguous");
    int64_t row = dense;
    if (n == 3) {
        if (shape[0] > 1) row = st[0];
    } else if (shape[1] > 1) {
        row = st[1];
        if (shape[0] > 1 && st[0] != shape[1] * row)
            refuse(name, ": the batches must follow one another at the rows' stride");
    } else if (shape[0] > 1) {
        row = st[0];
    }
    if (row < dense || row % 8)
        refuse(name, ": row stride ", row, " is not a multiple of 8 of at least N*D = ", dense);
    return row;
}

int code_of(at::ScalarType t) {
    if (t == at::kBFloat16) return SLIKL_BF16;
    if (t == at::kHalf) return SLIKL_FP16;
    refuse("float16 or bfloat16 is wanted, not ", c10::toString(t));
}

// What a call gets of one side: x, or the values of its checkpoint with their scale.
struct SideArgs {
    Maybe x, scale, positions, gain, bias;
    int norm, layout;       // slikl codes; -1 for a name that is none
};

struct Call {
    slikl_qk_problem pr{};
    slikl_qk_tensors tn{};
    at::ScalarType dtype = at::kBFloat16;
    at::Device dev = at::kCPU;
    std::optional<at::IntArrayRef> shape[2];
};

void enter_side(Call &c, const char *name, const SideArgs &in, slikl_qk_side &side,
                slikl_qk_side_tensors &t, int which) {
    side.N = 1;
    if (!in.x) return;
    const Tensor &x = *in.x;
    const auto shape = x.sizes();
    if (in.norm < 0) refuse("norm_", name, " must be none, rms or layer");
    if (in.layout != SLIKL_BSND && in.layout != SLIKL_TND) refuse("layout_", name, " must be BSND or TND");
    const bool bsnd = in.layout == SLIKL_BSND;
    if (x.dim() != (bsnd ? 4 : 3) || shape.back() != c.pr.D || x.device() != c.dev)
        refuse("x_", name, " must be ", bsnd ? "[B,S,N,D]" : "[T,N,D]", " rows on ", c.dev, " with D = ", c.pr.D);
    if (in.scale) {
        t.x8 = address(x, placed("x", name) + ".values", c.dev, at::kFloat8_e4m3fn);
        t.x8_scale = address<const float>(*in.scale, placed("x", name) + ".scale", c.dev, at::kFloat,
                                          shape.slice(0, shape.size() - 1));
    } else {
        if (x.scalar_type() != c.dtype) refuse("q and k must share one type, float16 or bfloat16");
        side.x_stride = row_stride(x, placed("x", name));
        t.x = x.data_ptr();
    }
    c.shape[which] = shape;
    side.norm = in.norm;
    side.N = shape[shape.size() - 2];
    side.T = bsnd ? shape[0] * shape[1] : shape[0];
    side.S = bsnd ? std::max<int64_t>(1, shape[1]) : 1;
    if (in.positions) {
        t.positions = address<const int32_t>(*in.positions, placed("pos", name), c.dev, at::kInt);
        if (in.positions->numel() != side.T) refuse("pos_", name, " must have ", side.T, " entries");
    } else if (c.pr.rot_dim && side.T && !bsnd) {
        refuse("TND needs pos_", name);
    }
    const int64_t d[1] = {c.pr.D};
    if (in.gain) t.gain = address<const float>(*in.gain, placed("gain", name), c.dev, at::kFloat, at::IntArrayRef(d));
    if (in.bias) t.bias = address<const float>(*in.bias, placed("bias", name), c.dev, at::kFloat, at::IntArrayRef(d));
}

Call enter(const SideArgs &q, const SideArgs &k, std::optional<at::ScalarType> type, const Maybe &cos_sin,
           int rot_layout, double eps, const Maybe &status) {
    Call c;
    const Maybe &some = q.x ? q.x : k.x;
    if (!some) refuse("x_q and x_k are both None");
    c.dev = some->device();
    if (!c.dev.is_cuda()) refuse("tensors must be CUDA tensors");
    c.dtype = type ? *type : some->scalar_type();
    if (some->dim() < 2 || rot_layout < 0) refuse("[.., N, D] tensors and rot_layout halves or pairs are wanted");
    c.pr.dtype = code_of(c.dtype);
    c.pr.rot_layout = rot_layout;
    c.pr.D = some->sizes().back();
    c.pr.eps = (float)eps;
    if (cos_sin) {
        if (cos_sin->dim() != 2) refuse("cos_sin must be [positions, rotated dims]");
        c.pr.table_rows = cos_sin->size(0);
        c.pr.rot_dim = cos_sin->size(1);
        c.tn.cos_sin = address<const float>(*cos_sin, "cos_sin", c.dev, at::kFloat);
    }
    enter_side(c, "q", q, c.pr.q, c.tn.q, 0);
    enter_side(c, "k", k, c.pr.k, c.tn.k, 1);
    const int64_t one[1] = {1};
    if (status) c.tn.status = address<uint32_t>(*status, "status", c.dev, at::kInt, at::IntArrayRef(one));
    return c;
}

// For its life the tensors' device is the current one, and `stream`, where given, the current stream: what
// is allocated then belongs to it too.
struct On {
    c10::cuda::OptionalCUDAStreamGuard stream;
    c10::cuda::OptionalCUDAGuard device;
    On(const at::Device &dev, const MaybeStream &s) {
        if (s && s->device() != dev) refuse("stream is of ", s->device(), ", the tensors are on ", dev);
        if (s) stream.reset_stream(*s);
        device.set_device(dev);
    }
};

void *stream_of(const at::Device &dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Outputs q, k, and of each the checkpoint's values and scale where `keep`; `plain` = false: no q, k.
py::tuple qk_forward(Maybe x_q, Maybe scale_q, Maybe x_k, Maybe scale_k, std::optional<at::ScalarType> type,
                     Maybe cos_sin, Maybe pos_q, Maybe pos_k, Maybe gain_q, Maybe gain_k, Maybe bias_q,
                     Maybe bias_k, int norm_q, int norm_k, int rot_layout, double eps, int layout_q,
                     int layout_k, bool plain, bool keep, Maybe out_q, Maybe out_k, Maybe status,
                     MaybeStream stream) {
    Call c = enter({x_q, scale_q, pos_q, gain_q, bias_q, norm_q, layout_q},
                   {x_k, scale_k, pos_k, gain_k, bias_k, norm_k, layout_k}, type, cos_sin, rot_layout, eps, status);
    const On on(c.dev, stream);
    Maybe y[2], kept[2], scale[2];
    for (int i = 0; i < 2; ++i) {
        if (!c.shape[i]) continue;
        slikl_qk_side_tensors &t = i ? c.tn.k : c.tn.q;
        const Maybe &given = i ? out_k : out_q;
        if (plain) {
            if (given) {
                t.y = address(*given, i ? "k" : "q", c.dev, c.dtype, *c.shape[i]);
                y[i] = given;
            } else {
                y[i] = fresh(*c.shape[i], c.dtype, c.dev);
                t.y = y[i]->data_ptr();
            }
        }
        if (keep) {
            kept[i] = fresh(*c.shape[i], at::kFloat8_e4m3fn, c.dev);
            scale[i] = fresh(c.shape[i]->slice(0, c.shape[i]->size() - 1), at::kFloat, c.dev);
            t.keep8 = kept[i]->data_ptr();
            t.keep8_scale = scale[i]->data_ptr<float>();
        }
    }
    const int rc = slikl_qk_norm_rope(&c.pr, &c.tn, stream_of(c.dev));
    return py::make_tuple(rc, y[0], y[1], kept[0], scale[0], kept[1], scale[1]);
}

// dx of both sides (given ones are checked) and one tensor whose rows are the sums asked for: dgain and
// dbias of q, then of k.
struct Grads {
    Maybe dx[2], sum[4];
};

Grads enter_gradients(Call &c, const Maybe &out_q, const Maybe &out_k) {
    Grads g;
    const int nq = c.shape[0] ? c.pr.q.norm : 0, nk = c.shape[1] ? c.pr.k.norm : 0;
    Tensor sums;
    if (nq + nk) sums = fresh({nq + nk, c.pr.D}, at::kFloat, c.dev);
    int64_t row = 0;
    for (int i = 0; i < 2; ++i) {
        if (!c.shape[i]) continue;
        slikl_qk_side &side = i ? c.pr.k : c.pr.q;
        slikl_qk_side_tensors &t = i ? c.tn.k : c.tn.q;
        const Maybe &given = i ? out_k : out_q;
        const char *name = i ? "dx_k" : "dx_q";
        if (given) {
            if (given->device() != c.dev || given->scalar_type() != c.dtype || given->sizes() != *c.shape[i])
                refuse(name, " must be ", c10::toString(c.dtype), " ", *c.shape[i], " on ", c.dev);
            side.dx_stride = row_stride(*given, name);
            g.dx[i] = given;
        } else {
            g.dx[i] = fresh(*c.shape[i], c.dtype, c.dev);
        }
        t.dx = g.dx[i]->data_ptr();
        for (int which = 0; which < side.norm; ++which) {
            g.sum[2 * i + which] = part_of(sums, c.pr.D * row++, {c.pr.D});
            float *p = g.sum[2 * i + which]->data_ptr<float>();
            if (which) t.dbias = p;
            else t.dgain = p;
        }
    }
    return g;
}

Tensor workspace_of(const Maybe &given, size_t bytes, const at::Device &dev) {
    if (given && given->numel() * given->element_size() >= (int64_t)bytes) {
        if (given->device() != dev || !given->is_contiguous()) refuse("workspace must be a contiguous tensor on ", dev);
        return *given;
    }
    return fresh({(int64_t)bytes}, at::kByte, dev);
}

size_t bytes_of(const Tensor &t) { return t.numel() * t.element_size(); }

py::tuple qk_gradient(Maybe dq, Maybe dk, Maybe x_q, Maybe scale_q, Maybe x_k, Maybe scale_k,
                      std::optional<at::ScalarType> type, Maybe cos_sin, Maybe pos_q, Maybe pos_k, Maybe gain_q,
                      Maybe gain_k, int norm_q, int norm_k, int rot_layout, double eps, int layout_q,
                      int layout_k, Maybe out_q, Maybe out_k, Maybe workspace, Maybe status,
                      MaybeStream stream) {
    Call c = enter({x_q, scale_q, pos_q, gain_q, {}, norm_q, layout_q}, {x_k, scale_k, pos_k, gain_k, {}, norm_k, layout_k},
                   type, cos_sin, rot_layout, eps, status);
    const On on(c.dev, stream);
    for (int i = 0; i < 2; ++i) {
        if (!c.shape[i]) continue;
        const Maybe &dy = i ? dk : dq;
        const char *name = i ? "dk" : "dq";
        if (!dy) refuse(name, " is missing");
        (i ? c.tn.k : c.tn.q).dy = address(*dy, name, c.dev, c.dtype, *c.shape[i]);
    }
    Grads g = enter_gradients(c, out_q, out_k);
    size_t bytes = 0;
    int rc = slikl_qk_norm_rope_grad_workspace_size(&c.pr, &bytes);
    Tensor ws;
    if (rc == SLIKL_OK) {
        ws = workspace_of(workspace, bytes, c.dev);
        rc = slikl_qk_norm_rope_grad(&c.pr, &c.tn, ws.data_ptr(), bytes_of(ws), stream_of(c.dev));
    }
    return py::make_tuple(rc, g.dx[0], g.dx[1], g.sum[0], g.sum[1], g.sum[2], g.sum[3], ws);
}

// The number of batches, on which both sides have to agree.
int64_t batches(int layout_q, int layout_k, int64_t rows_q, int64_t rows_k, const Maybe &cu_q, const Maybe &cu_k) {
    const int64_t q = layout_q == SLIKL_BSND ? rows_q : cu_q ? cu_q->numel() - 1 : -1;
    const int64_t k = layout_k == SLIKL_BSND ? rows_k : cu_k ? cu_k->numel() - 1 : -1;
    if (q != k || q < 0) refuse("queries and keys must have the same number of batches (TND: cu_seqlens)");
    return q;
}

const int32_t *lengths(const Maybe &t, const char *name, const at::Device &dev, int64_t n) {
    const int64_t shape[1] = {n};
    return t ? address<const int32_t>(*t, name, dev, at::kInt, at::IntArrayRef(shape)) : nullptr;
}

py::tuple grad_projected(Tensor x_q, Maybe scale_q, Tensor x_k, Maybe scale_k, std::optional<at::ScalarType> type,
                         Tensor w, Tensor p, Tensor idx, Maybe cos_sin, Maybe pos_q, Maybe pos_k, Maybe gain_q,
                         Maybe gain_k, Maybe bias_q, Maybe bias_k, int norm_q, int norm_k, int rot_layout,
                         double eps, int layout_q, int layout_k, Maybe cu_q, Maybe cu_k, bool deterministic,
                         int dk_path, int64_t key_range_bound, bool loss, Maybe used_q, Maybe used_k, Maybe out_q,
                         Maybe out_k, Maybe workspace, MaybeStream stream) {
    Call c = enter({x_q, scale_q, pos_q, gain_q, bias_q, norm_q, layout_q},
                   {x_k, scale_k, pos_k, gain_k, bias_k, norm_k, layout_k}, type, cos_sin, rot_layout, eps, {});
    const On on(c.dev, stream);
    const auto sq = *c.shape[0], sk = *c.shape[1];
    if (idx.dim() < 1) refuse("sparse_indices must be [.., 1, topk]");
    slikl_problem pr{};
    pr.dtype = c.pr.dtype;
    pr.layout_q = layout_q;
    pr.layout_k = layout_k;
    pr.deterministic = deterministic;
    pr.B = batches(layout_q, layout_k, sq[0], sk[0], cu_q, cu_k);
    pr.S1 = layout_q == SLIKL_BSND ? sq[1] : 0;
    pr.S2 = layout_k == SLIKL_BSND ? sk[1] : key_range_bound;
    pr.T1 = c.pr.q.T;
    pr.T2 = c.pr.k.T;
    pr.N1 = c.pr.q.N;
    pr.D = c.pr.D;
    pr.topk = idx.sizes().back();
    std::vector<int64_t> rows(sq.begin(), sq.end() - 1), slots(sq.begin(), sq.end() - 2);
    slots.insert(slots.end(), {1, pr.topk});
    slikl_tensors tn{};
    tn.w = address<const float>(w, "w", c.dev, at::kFloat, at::IntArrayRef(rows));
    tn.attn_softmax_l1norm = address<const float>(p, "attn_softmax_l1norm", c.dev, at::kFloat, at::IntArrayRef(slots));
    tn.sparse_indices = address<const int32_t>(idx, "sparse_indices", c.dev, at::kInt, at::IntArrayRef(slots));
    if (layout_q == SLIKL_TND) tn.cu_seqlens_q = address<const int32_t>(*cu_q, "cu_seqlens_q", c.dev, at::kInt);
    if (layout_k == SLIKL_TND) tn.cu_seqlens_k = address<const int32_t>(*cu_k, "cu_seqlens_k", c.dev, at::kInt);
    slikl_options opt{};
    opt.dk_path = dk_path;
    opt.seq_used_q = lengths(used_q, "seq_used_q", c.dev, pr.B);
    opt.seq_used_k = lengths(used_k, "seq_used_k", c.dev, pr.B);
    Grads g = enter_gradients(c, out_q, out_k);
    Tensor dw = fresh(rows, at::kFloat, c.dev), y = fresh(slots, at::kFloat, c.dev);
    tn.dw = dw.data_ptr<float>();
    tn.softmax_out = y.data_ptr<float>();
    Maybe losses;
    if (loss) {
        losses = fresh({pr.T1}, at::kFloat, c.dev);
        opt.loss = losses->data_ptr<float>();
    }
    size_t bytes = 0;
    int rc = slikl_grad_projected_workspace_size(&pr, &c.pr, &opt, &bytes);
    Tensor ws;
    if (rc == SLIKL_OK) {
        ws = workspace_of(workspace, bytes, c.dev);
        rc = slikl_grad_projected(&pr, &c.pr, &tn, &c.tn, ws.data_ptr(), bytes_of(ws), stream_of(c.dev), &opt);
    }
    return py::make_tuple(rc, g.dx[0], g.dx[1], g.sum[0], g.sum[1], g.sum[2], g.sum[3], dw, y, losses, ws);
}

py::tuple key_weights(Tensor weights, Tensor idx, Tensor scores, double decay, int layout_q, int layout_k,
                      Maybe cu_q, Maybe cu_k, Maybe used_q, Maybe used_k, int64_t key_range_bound, Maybe out,
                      Maybe workspace, Maybe status, MaybeStream stream) {
    const at::Device dev = scores.device();
    if (!dev.is_cuda() || layout_q < 0 || layout_k < 0) refuse("CUDA tensors and layouts BSND or TND are wanted");
    const auto shape = idx.sizes(), rows = scores.sizes();
    if (idx.dim() != (layout_q == SLIKL_BSND ? 4 : 3) || shape[shape.size() - 2] != 1 ||
        scores.dim() != (layout_k == SLIKL_BSND ? 2 : 1))
        refuse("sparse_indices must be [B,S1,1,topk] / [T1,1,topk], scores [B,S2] / [T2]");
    const On on(dev, stream);
    slikl_problem pr{};
    pr.layout_q = layout_q;
    pr.layout_k = layout_k;
    pr.topk = shape.back();
    pr.B = batches(layout_q, layout_k, shape[0], rows[0], cu_q, cu_k);
    slikl_key_weights_tensors tn{};
    if (layout_q == SLIKL_BSND) {
        pr.S1 = shape[1];
    } else {
        pr.T1 = shape[0];
        tn.cu_seqlens_q = address<const int32_t>(*cu_q, "cu_seqlens_q", dev, at::kInt);
    }
    if (layout_k == SLIKL_BSND) {
        pr.S2 = rows[1];
    } else {
        pr.T2 = rows[0];
        pr.S2 = key_range_bound;
        tn.cu_seqlens_k = address<const int32_t>(*cu_k, "cu_seqlens_k", dev, at::kInt);
    }
    slikl_options opt{};
    opt.seq_used_q = lengths(used_q, "seq_used_q", dev, pr.B);
    opt.seq_used_k = lengths(used_k, "seq_used_k", dev, pr.B);
    tn.sparse_indices = address<const int32_t>(idx, "sparse_indices", dev, at::kInt);
    tn.weights = address<const float>(weights, "weights", dev, at::kFloat, shape);
    tn.scores = address<const float>(scores, "scores", dev, at::kFloat);
    const int64_t one[1] = {1};
    if (status) tn.status = address<uint32_t>(*status, "status", dev, at::kInt, at::IntArrayRef(one));
    Tensor result = out ? *out : fresh(rows, at::kFloat, dev);
    tn.out = address<float>(result, "out", dev, at::kFloat, rows);
    size_t bytes = 0;
    int rc = slikl_key_weights_workspace_size(&pr, &bytes);
    Tensor ws;
    if (rc == SLIKL_OK) {
        ws = workspace_of(workspace, bytes, dev);
        rc = slikl_key_weights(&pr, &tn, decay, ws.data_ptr(), bytes_of(ws), stream_of(dev), &opt);
    }
    return py::make_tuple(rc, result, ws);
}

py::tuple evict(Tensor scores, std::vector<Tensor> caches, int64_t budget, int64_t sinks, int64_t recent,
                int layout_k, Maybe cu_k, Maybe used_k, int64_t key_range_bound, Maybe out_kept, Maybe out_lengths,
                Maybe out_scores, std::optional<std::vector<Tensor>> out_caches, Maybe status,
                MaybeStream stream) {
    const at::Device dev = scores.device();
    if (!dev.is_cuda() || layout_k < 0) refuse("CUDA tensors and layout BSND or TND are wanted");
    const bool bsnd = layout_k == SLIKL_BSND;
    const auto rows = scores.sizes();
    const size_t lead = rows.size();
    if (lead != (bsnd ? 2u : 1u) || (!bsnd && !cu_k)) refuse("scores must be [B,S2], or [T2] with cu_seqlens_k");
    if (budget < 1 || budget >> 31 || caches.size() > SLIKL_EVICT_MAX_CACHES)
        refuse("budget must be at least 1 and below 2^31, and caches at most ", SLIKL_EVICT_MAX_CACHES);
    if (out_caches && out_caches->size() != caches.size()) refuse("out['caches'] must have a tensor for each cache");
    const On on(dev, stream);
    slikl_evict_problem pr{};
    slikl_evict_tensors tn{};
    pr.layout_k = layout_k;
    pr.n_caches = (int32_t)caches.size();
    pr.budget = budget;
    pr.sinks = sinks;
    pr.recent = recent;
    pr.B = bsnd ? rows[0] : cu_k->numel() - 1;
    pr.S2 = bsnd ? rows[1] : key_range_bound;
    pr.T2 = bsnd ? 0 : rows[0];
    tn.scores = address<const float>(scores, "scores", dev, at::kFloat);
    if (!bsnd) tn.cu_seqlens_k = address<const int32_t>(*cu_k, "cu_seqlens_k", dev, at::kInt);
    tn.seq_used_k = lengths(used_k, "seq_used_k", dev, pr.B);
    const int64_t one[1] = {1}, batch[1] = {pr.B}, places[2] = {pr.B, budget};
    if (status) tn.status = address<uint32_t>(*status, "status", dev, at::kInt, at::IntArrayRef(one));
    Tensor kept, lens;
    if (!out_kept && !out_lengths && pr.B >= 0) {     // one allocation for both
        const Tensor both = fresh({pr.B * (budget + 1)}, at::kInt, dev);
        kept = part_of(both, 0, places);
        lens = part_of(both, pr.B * budget, batch);
    } else {
        kept = out_kept ? *out_kept : fresh(places, at::kInt, dev);
        lens = out_lengths ? *out_lengths : fresh(batch, at::kInt, dev);
    }
    Tensor best = out_scores ? *out_scores : fresh(places, at::kFloat, dev);
    tn.kept = address<int32_t>(kept, "kept", dev, at::kInt, at::IntArrayRef(places));
    tn.lengths = address<int32_t>(lens, "lengths", dev, at::kInt, at::IntArrayRef(batch));
    tn.scores_out = address<float>(best, "scores (out)", dev, at::kFloat, at::IntArrayRef(places));
    py::list outs;
    for (size_t i = 0; i < caches.size(); ++i) {
        const Tensor &c = caches[i];
        const std::string name = "cache " + std::to_string(i);
        if ((size_t)c.dim() < lead || c.sizes().slice(0, lead) != rows) refuse(name, " must have scores' rows");
        std::vector<int64_t> shape(places, places + 2);
        int64_t bytes = c.element_size();
        for (const int64_t n : c.sizes().slice(lead)) {
            shape.push_back(n);
            bytes *= n;
        }
        Tensor o = out_caches ? (*out_caches)[i] : at::zeros(shape, c.options());
        tn.caches[i].in = address(c, name, dev, c.scalar_type());
        tn.caches[i].out = address(o, "out " + name, dev, c.scalar_type(), at::IntArrayRef(shape));
        tn.caches[i].row_bytes = bytes;
        outs.append(o);
    }
    const int rc = slikl_evict(&pr, &tn, stream_of(dev));
    return py::make_tuple(rc, kept, lens, best, outs);
}

}  // namespace

PYBIND11_MODULE(_slikl_torch, m) {
    m.def("qk_forward", &qk_forward);
    m.def("qk_gradient", &qk_gradient);
    m.def("grad_projected", &grad_projected);
    m.def("key_weights", &key_weights);
    m.def("evict", &evict);
    m.def("row_stride", &row_stride);
}
