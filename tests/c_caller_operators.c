/* Prints the sizes and field offsets of the structs that the operators around slikl_grad take, as
 * a C99 compiler lays them out, and phase-1 answers, for comparison with the Python binding. */
#include <stddef.h>
#include <stdio.h>
#include <string.h>

#include "slikl.h"

#define SIZE(t) printf("size %s %d\n", #t, (int)sizeof(t))
#define FIELD(t, f) printf("field %s %s %d\n", #t, #f, (int)offsetof(t, f))

int main(void) {
    slikl_qk_problem qk;
    slikl_problem pr;
    size_t n = 0;
    SIZE(slikl_qk_side);
    FIELD(slikl_qk_side, T); FIELD(slikl_qk_side, S); FIELD(slikl_qk_side, N);
    FIELD(slikl_qk_side, x_stride); FIELD(slikl_qk_side, dx_stride);
    FIELD(slikl_qk_side, norm); FIELD(slikl_qk_side, reserved);
    SIZE(slikl_qk_problem);
    FIELD(slikl_qk_problem, dtype); FIELD(slikl_qk_problem, rot_layout); FIELD(slikl_qk_problem, D);
    FIELD(slikl_qk_problem, rot_dim); FIELD(slikl_qk_problem, table_rows);
    FIELD(slikl_qk_problem, eps); FIELD(slikl_qk_problem, reserved); FIELD(slikl_qk_problem, q);
    FIELD(slikl_qk_problem, k);
    SIZE(slikl_qk_side_tensors);
    FIELD(slikl_qk_side_tensors, x); FIELD(slikl_qk_side_tensors, x8);
    FIELD(slikl_qk_side_tensors, x8_scale); FIELD(slikl_qk_side_tensors, positions);
    FIELD(slikl_qk_side_tensors, gain); FIELD(slikl_qk_side_tensors, bias);
    FIELD(slikl_qk_side_tensors, y); FIELD(slikl_qk_side_tensors, keep8);
    FIELD(slikl_qk_side_tensors, keep8_scale); FIELD(slikl_qk_side_tensors, dy);
    FIELD(slikl_qk_side_tensors, dx); FIELD(slikl_qk_side_tensors, dgain);
    FIELD(slikl_qk_side_tensors, dbias);
    SIZE(slikl_qk_tensors);
    FIELD(slikl_qk_tensors, q); FIELD(slikl_qk_tensors, k); FIELD(slikl_qk_tensors, cos_sin);
    FIELD(slikl_qk_tensors, status);
    SIZE(slikl_key_weights_tensors);
    FIELD(slikl_key_weights_tensors, sparse_indices); FIELD(slikl_key_weights_tensors, weights);
    FIELD(slikl_key_weights_tensors, cu_seqlens_q); FIELD(slikl_key_weights_tensors, cu_seqlens_k);
    FIELD(slikl_key_weights_tensors, scores); FIELD(slikl_key_weights_tensors, out);
    FIELD(slikl_key_weights_tensors, status);
    SIZE(slikl_evict_problem);
    FIELD(slikl_evict_problem, layout_k); FIELD(slikl_evict_problem, n_caches);
    FIELD(slikl_evict_problem, B); FIELD(slikl_evict_problem, S2); FIELD(slikl_evict_problem, T2);
    FIELD(slikl_evict_problem, budget); FIELD(slikl_evict_problem, sinks);
    FIELD(slikl_evict_problem, recent);
    SIZE(slikl_evict_cache);
    FIELD(slikl_evict_cache, in); FIELD(slikl_evict_cache, out); FIELD(slikl_evict_cache, row_bytes);
    SIZE(slikl_evict_tensors);
    FIELD(slikl_evict_tensors, scores); FIELD(slikl_evict_tensors, cu_seqlens_k);
    FIELD(slikl_evict_tensors, seq_used_k); FIELD(slikl_evict_tensors, kept);
    FIELD(slikl_evict_tensors, lengths); FIELD(slikl_evict_tensors, scores_out);
    FIELD(slikl_evict_tensors, status); FIELD(slikl_evict_tensors, caches);

    memset(&qk, 0, sizeof(qk));
    memset(&pr, 0, sizeof(pr));
    qk.dtype = pr.dtype = SLIKL_BF16;
    qk.D = pr.D = 128;
    qk.rot_dim = 64;
    qk.table_rows = 4096;
    qk.eps = 1e-6f;
    qk.q.T = qk.k.T = qk.q.S = qk.k.S = pr.S1 = pr.S2 = 4096;
    qk.q.N = pr.N1 = 64;
    qk.k.N = pr.B = 1;
    qk.q.norm = SLIKL_NORM_RMS;
    qk.k.norm = SLIKL_NORM_LAYER;
    pr.topk = 2048;
    printf("rc %d ", (int)slikl_qk_norm_rope_grad_workspace_size(&qk, &n));
    printf("%lu\n", (unsigned long)n);
    printf("rc %d ", (int)slikl_grad_projected_workspace_size(&pr, &qk, NULL, &n));
    printf("%lu\n", (unsigned long)n);
    printf("rc %d ", (int)slikl_key_weights_workspace_size(&pr, &n));
    printf("%lu\n", (unsigned long)n);
    return 0;
}
