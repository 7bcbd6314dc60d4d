// fa_api.cu -- the C ABI (include/fa.h): argument checks, launch set-up,
// status strings and the device error word.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

int device_sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev >= 0 && dev < 64) {
        int v = cached[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    int n = 1;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n < 1) n = 1;
    if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

int encode_tensor_map_3d(void *map, const void *base, int elem_bytes, uint64_t dim0,
                         uint64_t dim1, uint64_t dim2, uint64_t stride1_bytes,
                         uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2,
                         int swizzle_bytes) {
    auto fn = encode_fn();
    if (!fn) return -1;
    CUtensorMapDataType dt;
    switch (elem_bytes) {
    case 1: dt = CU_TENSOR_MAP_DATA_TYPE_UINT8; break;
    case 2: dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; break;
    case 4: dt = CU_TENSOR_MAP_DATA_TYPE_FLOAT32; break;
    default: return -1;
    }
    CUtensorMapSwizzle sw;
    switch (swizzle_bytes) {
    case 0: sw = CU_TENSOR_MAP_SWIZZLE_NONE; break;
    case 32: sw = CU_TENSOR_MAP_SWIZZLE_32B; break;
    case 64: sw = CU_TENSOR_MAP_SWIZZLE_64B; break;
    case 128: sw = CU_TENSOR_MAP_SWIZZLE_128B; break;
    default: return -1;
    }
    cuuint64_t dims[3] = {dim0, dim1, dim2};
    cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
    cuuint32_t box[3] = {box0, box1, box2};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(static_cast<CUtensorMap *>(map), dt, 3,
                    const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE,
                    sw,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? 0 : -1;
}

// Diagnostic kernel for the watchdog: waits on a barrier that nothing ever
// arrives on.  The bounded wait gives up after ~1 s, records the timeout in
// the device error word and the kernel returns normally.
__global__ void watchdog_probe_kernel() {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag);
}

}  // namespace fa

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int map_rc(int rc) {
    switch (rc) {
    case 0: return FA_OK;
    case -2: return FA_ERR_UNSUPPORTED;
    case -4: return FA_ERR_WORKSPACE;
    default: return FA_ERR_CUDA;
    }
}

int check_common(int Hq, int Hkv, int d, int causal, int window, float scale, int o_dtype) {
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_FP32) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (window > 0 && !causal) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace

extern "C" {

}  // extern "C"

namespace {

int fwd_dense(const void *q, const void *k, const void *v, void *o, float *lse,
              const float *sinks, int B, int Hq, int Hkv, int N, int d, int causal, int window,
              float scale, int o_dtype, void *stream, const int *doc = nullptr,
              int n_sink = 0) {
    if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, o_dtype);
    if (rc) return rc;
    if (B == 0 || N == 0) return FA_OK;
    if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
    if ((long long)B * N > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3)))
        return FA_ERR_ALIGNMENT;
    fa::PrefillArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.cu_seqlens = nullptr;
    a.num_seqs = B;
    a.seqlen = N;
    a.total_tokens = B * N;
    a.max_seqlen = N;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.o_fp32 = o_dtype == FA_OUT_FP32;
    a.sinks = sinks;
    a.doc = doc;
    a.n_sink = n_sink;
    return map_rc(fa::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

int fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
               const float *sinks, const int *cu_seqlens, int num_seqs, int total_tokens,
               int max_seqlen, int Hq, int Hkv, int d, int causal, int window, float scale,
               int o_dtype, void *stream, int n_sink = 0) {
    if (num_seqs < 0 || total_tokens < 0 || max_seqlen < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, o_dtype);
    if (rc) return rc;
    if (num_seqs == 0 || total_tokens == 0 || max_seqlen == 0) return FA_OK;
    if (!q || !k || !v || !o || !cu_seqlens) return FA_ERR_INVALID_ARG;
    if (total_tokens > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(cu_seqlens) & 3) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3)))
        return FA_ERR_ALIGNMENT;
    fa::PrefillArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.cu_seqlens = cu_seqlens;
    a.num_seqs = num_seqs;
    a.seqlen = 0;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.o_fp32 = o_dtype == FA_OUT_FP32;
    a.sinks = sinks;
    a.n_sink = n_sink;
    return map_rc(fa::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
           int Hkv, int N, int d, int causal, int window, float scale, int o_dtype,
           void *stream) {
    return fwd_dense(q, k, v, o, lse, nullptr, B, Hq, Hkv, N, d, causal, window, scale,
                     o_dtype, stream);
}

int fa_fwd_sink_tokens(const void *q, const void *k, const void *v, void *o, float *lse,
                       int B, int Hq, int Hkv, int N, int d, int window, int n_sink,
                       float scale, int o_dtype, void *stream) {
    if (window <= 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
    return fwd_dense(q, k, v, o, lse, nullptr, B, Hq, Hkv, N, d, 1, window, scale, o_dtype,
                     stream, nullptr, n_sink);
}

int fa_fwd_varlen_sink_tokens(const void *q, const void *k, const void *v, void *o, float *lse,
                              const int *cu_seqlens, int num_seqs, int total_tokens,
                              int max_seqlen, int Hq, int Hkv, int d, int window, int n_sink,
                              float scale, int o_dtype, void *stream) {
    if (window <= 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
    return fwd_varlen(q, k, v, o, lse, nullptr, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                      Hq, Hkv, d, 1, window, scale, o_dtype, stream, n_sink);
}

int fa_fwd_sinks(const void *q, const void *k, const void *v, void *o, float *lse,
                 const float *sinks, int B, int Hq, int Hkv, int N, int d, int causal,
                 int window, float scale, int o_dtype, void *stream) {
    if (!sinks) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(sinks) & 3) return FA_ERR_ALIGNMENT;
    return fwd_dense(q, k, v, o, lse, sinks, B, Hq, Hkv, N, d, causal, window, scale,
                     o_dtype, stream);
}

int fa_fwd_doc(const void *q, const void *k, const void *v, void *o, float *lse,
               const int *doc_ids, int B, int Hq, int Hkv, int N, int d, int causal,
               int window, float scale, int o_dtype, void *stream) {
    if (!doc_ids) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(doc_ids) & 3) return FA_ERR_ALIGNMENT;
    return fwd_dense(q, k, v, o, lse, nullptr, B, Hq, Hkv, N, d, causal, window, scale,
                     o_dtype, stream, doc_ids);
}

int fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                  const int *cu_seqlens, int num_seqs, int total_tokens, int max_seqlen,
                  int Hq, int Hkv, int d, int causal, int window, float scale, int o_dtype,
                  void *stream) {
    return fwd_varlen(q, k, v, o, lse, nullptr, cu_seqlens, num_seqs, total_tokens,
                      max_seqlen, Hq, Hkv, d, causal, window, scale, o_dtype, stream);
}

int fa_fwd_varlen_sinks(const void *q, const void *k, const void *v, void *o, float *lse,
                        const float *sinks, const int *cu_seqlens, int num_seqs,
                        int total_tokens, int max_seqlen, int Hq, int Hkv, int d, int causal,
                        int window, float scale, int o_dtype, void *stream) {
    if (!sinks) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(sinks) & 3) return FA_ERR_ALIGNMENT;
    return fwd_varlen(q, k, v, o, lse, sinks, cu_seqlens, num_seqs, total_tokens,
                      max_seqlen, Hq, Hkv, d, causal, window, scale, o_dtype, stream);
}

int fa_fwd_paged(const void *q, const void *k_cache, const void *v_cache,
                 const int *block_table, const int *cu_seqlens_q, const int *seq_lens_k,
                 void *o, float *lse, const float *sinks, int num_seqs, int total_q,
                 int max_seqlen_q, int num_pages, int Hq, int Hkv, int d, int page_size,
                 int max_pages_per_seq, int causal, int window, float scale, int o_dtype,
                 void *stream) {
    if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || num_pages < 0 ||
        max_pages_per_seq <= 0)
        return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, o_dtype);
    if (rc) return rc;
    if (page_size != 16) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return FA_OK;
    if (num_pages == 0) return FA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens_q || !seq_lens_k || !o)
        return FA_ERR_INVALID_ARG;
    if (total_q > INT32_MAX / 2 || (long long)num_pages * page_size > INT32_MAX / 2 ||
        (long long)max_pages_per_seq * page_size > INT32_MAX / 2)
        return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3) ||
        (reinterpret_cast<uintptr_t>(cu_seqlens_q) & 3) ||
        (reinterpret_cast<uintptr_t>(seq_lens_k) & 3) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) ||
        (sinks && (reinterpret_cast<uintptr_t>(sinks) & 3)))
        return FA_ERR_ALIGNMENT;
    fa::PrefillArgs a{};
    a.q = q; a.k = k_cache; a.v = v_cache; a.o = o; a.lse = lse;
    a.cu_seqlens = cu_seqlens_q;
    a.num_seqs = num_seqs;
    a.seqlen = 0;
    a.total_tokens = total_q;
    a.max_seqlen = max_seqlen_q;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.o_fp32 = o_dtype == FA_OUT_FP32;
    a.sinks = sinks;
    a.paged = 1;
    a.block_table = block_table;
    a.seq_lens_k = seq_lens_k;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    return map_rc(fa::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_bwd_workspace_bytes(int total_tokens, int Hq, int d) {
    return fa::bwd_workspace_bytes(total_tokens, Hq, d);
}

}  // extern "C"

namespace {

int bwd_common(const void *q, const void *k, const void *v, const void *o, const void *dout,
               const float *lse, void *dq, void *dk, void *dv, int Hq, int Hkv, int d,
               int causal, int window, float scale, long long total, void *workspace,
               size_t workspace_bytes) {
    int rc = check_common(Hq, Hkv, d, causal, window, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
    if (total > INT32_MAX / 2 || total * Hq > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        (reinterpret_cast<uintptr_t>(lse) & 3))
        return FA_ERR_ALIGNMENT;
    const size_t need = fa::bwd_workspace_bytes(total, Hq, d);
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    return FA_OK;
}

}  // namespace

extern "C" {

}  // extern "C"

namespace {

int bwd_dense_call(const void *q, const void *k, const void *v, const void *o,
                   const void *dout, const float *lse, const float *sinks, void *dq, void *dk,
                   void *dv, float *dsinks, int B, int Hq, int Hkv, int N, int d, int causal,
                   int window, float scale, void *workspace, size_t workspace_bytes,
                   void *stream) {
    if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (B == 0 || N == 0) return FA_OK;
    rc = bwd_common(q, k, v, o, dout, lse, dq, dk, dv, Hq, Hkv, d, causal, window, scale,
                    (long long)B * N, workspace, workspace_bytes);
    if (rc) return rc;
    fa::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.cu_seqlens = nullptr;
    a.num_seqs = B;
    a.seqlen = N;
    a.total_tokens = B * N;
    a.max_seqlen = N;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.workspace = workspace;
    a.sinks = sinks;
    a.dsinks = dsinks;
    return map_rc(fa::launch_bwd(a, static_cast<cudaStream_t>(stream)));
}

int bwd_varlen_call(const void *q, const void *k, const void *v, const void *o,
                    const void *dout, const float *lse, const float *sinks, void *dq, void *dk,
                    void *dv, float *dsinks, const int *cu_seqlens, int num_seqs,
                    int total_tokens, int max_seqlen, int Hq, int Hkv, int d, int causal,
                    int window, float scale, void *workspace, size_t workspace_bytes,
                    void *stream) {
    if (num_seqs < 0 || total_tokens < 0 || max_seqlen < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (num_seqs == 0 || total_tokens == 0 || max_seqlen == 0) return FA_OK;
    if (!cu_seqlens) return FA_ERR_INVALID_ARG;
    rc = bwd_common(q, k, v, o, dout, lse, dq, dk, dv, Hq, Hkv, d, causal, window, scale,
                    total_tokens, workspace, workspace_bytes);
    if (rc) return rc;
    if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3) return FA_ERR_ALIGNMENT;
    fa::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.cu_seqlens = cu_seqlens;
    a.num_seqs = num_seqs;
    a.seqlen = 0;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.workspace = workspace;
    a.sinks = sinks;
    a.dsinks = dsinks;
    return map_rc(fa::launch_bwd(a, static_cast<cudaStream_t>(stream)));
}

int check_sink_pair(const float *sinks, const float *dsinks) {
    if (!sinks || !dsinks) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(sinks) & 3) || (reinterpret_cast<uintptr_t>(dsinks) & 3))
        return FA_ERR_ALIGNMENT;
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout,
           const float *lse, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int N, int d,
           int causal, int window, float scale, void *workspace, size_t workspace_bytes,
           void *stream) {
    return bwd_dense_call(q, k, v, o, dout, lse, nullptr, dq, dk, dv, nullptr, B, Hq, Hkv, N,
                          d, causal, window, scale, workspace, workspace_bytes, stream);
}

int fa_bwd_sinks(const void *q, const void *k, const void *v, const void *o, const void *dout,
                 const float *lse, const float *sinks, void *dq, void *dk, void *dv,
                 float *dsinks, int B, int Hq, int Hkv, int N, int d, int causal, int window,
                 float scale, void *workspace, size_t workspace_bytes, void *stream) {
    const int rc = check_sink_pair(sinks, dsinks);
    if (rc) return rc;
    return bwd_dense_call(q, k, v, o, dout, lse, sinks, dq, dk, dv, dsinks, B, Hq, Hkv, N, d,
                          causal, window, scale, workspace, workspace_bytes, stream);
}

int fa_bwd_varlen(const void *q, const void *k, const void *v, const void *o,
                  const void *dout, const float *lse, void *dq, void *dk, void *dv,
                  const int *cu_seqlens, int num_seqs, int total_tokens, int max_seqlen,
                  int Hq, int Hkv, int d, int causal, int window, float scale, void *workspace,
                  size_t workspace_bytes, void *stream) {
    return bwd_varlen_call(q, k, v, o, dout, lse, nullptr, dq, dk, dv, nullptr, cu_seqlens,
                           num_seqs, total_tokens, max_seqlen, Hq, Hkv, d, causal, window,
                           scale, workspace, workspace_bytes, stream);
}

int fa_bwd_varlen_sinks(const void *q, const void *k, const void *v, const void *o,
                        const void *dout, const float *lse, const float *sinks, void *dq,
                        void *dk, void *dv, float *dsinks, const int *cu_seqlens, int num_seqs,
                        int total_tokens, int max_seqlen, int Hq, int Hkv, int d, int causal,
                        int window, float scale, void *workspace, size_t workspace_bytes,
                        void *stream) {
    const int rc = check_sink_pair(sinks, dsinks);
    if (rc) return rc;
    return bwd_varlen_call(q, k, v, o, dout, lse, sinks, dq, dk, dv, dsinks, cu_seqlens,
                           num_seqs, total_tokens, max_seqlen, Hq, Hkv, d, causal, window,
                           scale, workspace, workspace_bytes, stream);
}

size_t fa_decode_workspace_bytes(int num_seqs, int Hq, int d, int page_size,
                                 int max_pages_per_seq) {
    return fa::decode_workspace_bytes(num_seqs, Hq, d, page_size, max_pages_per_seq);
}

}  // extern "C"

namespace {

int decode_impl_call(const void *q, const void *k_cache, const void *v_cache,
                     const int *block_table, const int *seq_lens, void *o, float *lse,
                     const float *sinks, int num_seqs, int num_pages, int Hq, int Hkv, int d,
                     int page_size, int max_pages_per_seq, float scale, void *workspace,
                     size_t workspace_bytes, void *stream, const float *k_scale = nullptr,
                     const float *v_scale = nullptr) {
    if (num_seqs < 0 || num_pages < 0 || max_pages_per_seq <= 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, 0, 0, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (page_size != 16) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return FA_OK;
    if (num_pages == 0) return FA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3) ||
        (reinterpret_cast<uintptr_t>(seq_lens) & 3) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3)))
        return FA_ERR_ALIGNMENT;
    const size_t need = fa::decode_workspace_bytes(num_seqs, Hq, d, page_size, max_pages_per_seq);
    if (need == 0) return FA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    fa::DecodeArgs a{};
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    a.block_table = block_table; a.seq_lens = seq_lens;
    a.o = o; a.lse = lse;
    a.num_seqs = num_seqs; a.num_pages = num_pages;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.page_size = page_size;
    a.max_pages = max_pages_per_seq;
    a.scale = scale;
    a.workspace = workspace;
    a.sinks = sinks;
    a.fp8 = k_scale != nullptr;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.workspace_bytes = workspace_bytes;
    return map_rc(fa::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fa_decode_paged(const void *q, const void *k_cache, const void *v_cache,
                    const int *block_table, const int *seq_lens, void *o, float *lse,
                    int num_seqs, int num_pages, int Hq, int Hkv, int d, int page_size,
                    int max_pages_per_seq, float scale, void *workspace, size_t workspace_bytes,
                    void *stream) {
    return decode_impl_call(q, k_cache, v_cache, block_table, seq_lens, o, lse, nullptr,
                            num_seqs, num_pages, Hq, Hkv, d, page_size, max_pages_per_seq,
                            scale, workspace, workspace_bytes, stream);
}

int fa_decode_paged_fp8(const void *q, const void *k_cache, const void *v_cache,
                        const float *k_scale, const float *v_scale, const int *block_table,
                        const int *seq_lens, void *o, float *lse, const float *sinks,
                        int num_seqs, int num_pages, int Hq, int Hkv, int d, int page_size,
                        int max_pages_per_seq, float scale, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (!k_scale || !v_scale) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_scale) & 3) || (reinterpret_cast<uintptr_t>(v_scale) & 3) ||
        (sinks && (reinterpret_cast<uintptr_t>(sinks) & 3)))
        return FA_ERR_ALIGNMENT;
    return decode_impl_call(q, k_cache, v_cache, block_table, seq_lens, o, lse, sinks,
                            num_seqs, num_pages, Hq, Hkv, d, page_size, max_pages_per_seq,
                            scale, workspace, workspace_bytes, stream, k_scale, v_scale);
}

int fa_decode_paged_sinks(const void *q, const void *k_cache, const void *v_cache,
                          const int *block_table, const int *seq_lens, void *o, float *lse,
                          const float *sinks, int num_seqs, int num_pages, int Hq, int Hkv,
                          int d, int page_size, int max_pages_per_seq, float scale,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (!sinks) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(sinks) & 3) return FA_ERR_ALIGNMENT;
    return decode_impl_call(q, k_cache, v_cache, block_table, seq_lens, o, lse, sinks,
                            num_seqs, num_pages, Hq, Hkv, d, page_size, max_pages_per_seq,
                            scale, workspace, workspace_bytes, stream);
}

size_t fa_fp8_workspace_bytes(int B, int N, int Hkv) {
    if (B <= 0 || N <= 0 || Hkv <= 0) return 0;
    return (size_t)B * Hkv * (size_t)((N + 127) / 128) * sizeof(float);
}

int fa_fp8_prepare(const void *q, const void *k, const void *v, const float *signs,
                   void *q8, void *k8, void *vt8, float *q_scale, float *k_scale,
                   float *v_scale, int B, int N, int Hq, int Hkv, int d, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (d != 128) return (d == 64) ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return FA_OK;
    if (!q || !k || !v || !q8 || !k8 || !vt8 || !q_scale || !k_scale || !v_scale)
        return FA_ERR_INVALID_ARG;
    if ((long long)B * N > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    const size_t need = fa_fp8_workspace_bytes(B, N, Hkv);
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q8) || !aligned16(k8) ||
        !aligned16(vt8) || (signs && !aligned16(signs)) ||
        (reinterpret_cast<uintptr_t>(q_scale) & 3) || (reinterpret_cast<uintptr_t>(k_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(v_scale) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 3))
        return FA_ERR_ALIGNMENT;
    fa::Fp8PrepArgs a{};
    a.q = q; a.k = k; a.v = v; a.signs = signs;
    a.q8 = q8; a.k8 = k8; a.vt8 = vt8;
    a.q_scale = q_scale; a.k_scale = k_scale; a.v_scale = v_scale;
    a.v_block_max = static_cast<float *>(workspace);
    a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.vt_stride = (N + 15) / 16 * 16;
    return map_rc(fa::launch_fp8_prepare(a, static_cast<cudaStream_t>(stream)));
}

int fa_fwd_fp8(const void *q8, const void *k8, const void *vt8, const float *q_scale,
               const float *k_scale, const float *v_scale, void *o, float *lse, int B,
               int Hq, int Hkv, int N, int d, int causal, int window, float scale,
               int o_dtype, void *stream) {
    if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, causal, window, scale, o_dtype);
    if (rc) return rc;
    if (d != 128) return FA_ERR_UNSUPPORTED;
    if (B == 0 || N == 0) return FA_OK;
    if (!q8 || !k8 || !vt8 || !o || !q_scale || !k_scale || !v_scale) return FA_ERR_INVALID_ARG;
    if ((long long)B * N > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q8) || !aligned16(k8) || !aligned16(vt8) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) ||
        (reinterpret_cast<uintptr_t>(q_scale) & 3) || (reinterpret_cast<uintptr_t>(k_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(v_scale) & 3))
        return FA_ERR_ALIGNMENT;
    fa::PrefillArgs a{};
    a.q = q8; a.k = k8; a.v = vt8; a.o = o; a.lse = lse;
    a.cu_seqlens = nullptr;
    a.num_seqs = B;
    a.seqlen = N;
    a.total_tokens = B * N;
    a.max_seqlen = N;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.causal = causal;
    a.window = window > 0 ? window : 0;
    a.scale = scale;
    a.o_fp32 = o_dtype == FA_OUT_FP32;
    a.q_scale = q_scale; a.k_scale = k_scale; a.v_scale = v_scale;
    a.vt_stride = (N + 15) / 16 * 16;
    return map_rc(fa::launch_prefill_fp8(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Sequences whose bookkeeping one block keeps in shared memory (32 KiB).
constexpr int kMaxCacheSlots = 8192;

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

int check_cache(const void *k, const void *v, const float *ks, const float *vs, int elem_bytes,
                int num_pages, int Hkv, int d, int page_size, int max_pages) {
    if (num_pages < 0 || Hkv <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
    if (elem_bytes != 1 && elem_bytes != 2) return FA_ERR_INVALID_ARG;
    if (page_size != 16 || (d != 64 && d != 128) || Hkv > 65536) return FA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > INT32_MAX / 2 ||
        (long long)max_pages * page_size > INT32_MAX / 2)
        return FA_ERR_UNSUPPORTED;
    if (num_pages == 0 || !k || !v) return FA_ERR_INVALID_ARG;
    // E4M3 codes come with both scales, bf16 values with none
    if ((elem_bytes == 1) != (ks != nullptr) || (elem_bytes == 1) != (vs != nullptr))
        return FA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned4(ks) || !aligned4(vs)) return FA_ERR_ALIGNMENT;
    return FA_OK;
}

fa::CachePages cache_pages(void *k, void *v, float *ks, float *vs, int elem_bytes, int num_pages,
                           int Hkv, int d) {
    fa::CachePages c;
    c.k = k; c.v = v; c.k_scale = ks; c.v_scale = vs;
    c.num_pages = num_pages; c.Hkv = Hkv; c.d = d; c.elem_bytes = elem_bytes;
    return c;
}

}  // namespace

extern "C" {

int fa_cache_fork(void *k_cache, void *v_cache, float *k_scale, float *v_scale, int elem_bytes,
                  const int *block_table, const int *seq_lens, int num_slots, const int *parents,
                  int num_new, const int *free_pages, const int *free_count, int free_capacity,
                  int *block_table_out, int *seq_lens_out, int *free_count_out, int num_pages, int Hkv, int d,
                  int page_size, int max_pages_per_seq, void *stream) {
    if (num_slots < 0 || num_new < 0 || free_capacity < 0) return FA_ERR_INVALID_ARG;
    const int rc = check_cache(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d,
                               page_size, max_pages_per_seq);
    if (rc) return rc;
    if (num_slots > kMaxCacheSlots || num_new > kMaxCacheSlots) return FA_ERR_UNSUPPORTED;
    if (!free_pages || !free_count || !free_count_out) return FA_ERR_INVALID_ARG;
    if (num_slots > 0 && (!block_table || !seq_lens)) return FA_ERR_INVALID_ARG;
    if (num_new > 0 && (!parents || !block_table_out || !seq_lens_out)) return FA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(parents) ||
        !aligned4(free_pages) || !aligned4(free_count) || !aligned4(block_table_out) ||
        !aligned4(seq_lens_out) || !aligned4(free_count_out))
        return FA_ERR_ALIGNMENT;
    const size_t row = (size_t)max_pages_per_seq * 4;
    if (overlap(block_table, num_slots * row, block_table_out, num_new * row) ||
        overlap(seq_lens, (size_t)num_slots * 4, seq_lens_out, (size_t)num_new * 4) ||
        overlap(free_count, 4, free_count_out, 4))
        return FA_ERR_INVALID_ARG;
    return map_rc(fa::launch_cache_fork(
        cache_pages(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d), block_table,
        seq_lens, num_slots, parents, num_new, free_pages, free_count, free_capacity,
        block_table_out, seq_lens_out, free_count_out, max_pages_per_seq, static_cast<cudaStream_t>(stream)));
}

int fa_cache_append(const void *k_new, const void *v_new, const int *cu_new, int num_seqs,
                    int total_new, void *k_cache, void *v_cache, int *block_table,
                    const int *seq_lens, const int *free_pages, const int *free_count,
                    int free_capacity, int *seq_lens_out, int *free_count_out, int num_pages, int Hkv, int d,
                    int page_size, int max_pages_per_seq, void *stream) {
    if (num_seqs < 0 || total_new < 0 || (num_seqs == 0 && total_new > 0) || free_capacity < 0)
        return FA_ERR_INVALID_ARG;
    const int rc = check_cache(k_cache, v_cache, nullptr, nullptr, 2, num_pages, Hkv, d, page_size,
                               max_pages_per_seq);
    if (rc) return rc;
    if (num_seqs > kMaxCacheSlots || total_new > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!free_pages || !free_count || !free_count_out) return FA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!cu_new || !block_table || !seq_lens || !seq_lens_out))
        return FA_ERR_INVALID_ARG;
    if (total_new > 0 && (!k_new || !v_new)) return FA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(cu_new) || !aligned4(block_table) ||
        !aligned4(seq_lens) || !aligned4(free_pages) || !aligned4(free_count) ||
        !aligned4(seq_lens_out) || !aligned4(free_count_out))
        return FA_ERR_ALIGNMENT;
    if (overlap(seq_lens, (size_t)num_seqs * 4, seq_lens_out, (size_t)num_seqs * 4) ||
        overlap(free_count, 4, free_count_out, 4))
        return FA_ERR_INVALID_ARG;
    return map_rc(fa::launch_cache_append(
        cache_pages(k_cache, v_cache, nullptr, nullptr, 2, num_pages, Hkv, d), k_new, v_new, cu_new,
        num_seqs, total_new, block_table, seq_lens, free_pages, free_count, free_capacity, seq_lens_out,
        free_count_out, max_pages_per_seq, static_cast<cudaStream_t>(stream)));
}

int fa_cache_copy_pages(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                        int elem_bytes, const int *src, const int *dst, int n, int num_pages,
                        int Hkv, int d, int page_size, void *stream) {
    if (n < 0) return FA_ERR_INVALID_ARG;
    const int rc = check_cache(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d,
                               page_size, 1);
    if (rc) return rc;
    if (n == 0) return FA_OK;
    if (!src || !dst) return FA_ERR_INVALID_ARG;
    if (!aligned4(src) || !aligned4(dst)) return FA_ERR_ALIGNMENT;
    return map_rc(fa::launch_cache_copy(
        cache_pages(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d), src, dst, n,
        static_cast<cudaStream_t>(stream)));
}

size_t fa_cache_collect_workspace_bytes(int num_pages) {
    return fa::cache_collect_workspace_bytes(num_pages);
}

int fa_cache_collect(const int *block_table, const int *seq_lens, int num_seqs,
                     int max_pages_per_seq, int num_pages, int page_size, int *free_pages,
                     int *free_count, void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || max_pages_per_seq <= 0 || num_pages <= 0) return FA_ERR_INVALID_ARG;
    if (page_size != 16 || num_seqs > 65535 || (long long)num_pages * page_size > INT32_MAX / 2 ||
        (long long)max_pages_per_seq * page_size > INT32_MAX / 2)
        return FA_ERR_UNSUPPORTED;
    if (!free_pages || !free_count || (num_seqs > 0 && (!block_table || !seq_lens)))
        return FA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(free_pages) ||
        !aligned4(free_count))
        return FA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < fa::cache_collect_workspace_bytes(num_pages))
        return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    return map_rc(fa::launch_cache_collect(block_table, seq_lens, num_seqs, max_pages_per_seq,
                                           num_pages, free_pages, free_count, workspace,
                                           static_cast<cudaStream_t>(stream)));
}

size_t fa_cache_compact_workspace_bytes(int num_pages) {
    return fa::cache_compact_workspace_bytes(num_pages);
}

int fa_cache_compact(void *k_cache, void *v_cache, float *k_scale, float *v_scale, int elem_bytes,
                     const int *block_table, const int *seq_lens, int num_seqs,
                     int *block_table_out, int *free_pages, int *free_count, int num_pages, int Hkv,
                     int d, int page_size, int max_pages_per_seq, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (num_seqs < 0) return FA_ERR_INVALID_ARG;
    const int rc = check_cache(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d,
                               page_size, max_pages_per_seq);
    if (rc) return rc;
    if (num_seqs > 65535) return FA_ERR_UNSUPPORTED;
    if (!free_pages || !free_count ||
        (num_seqs > 0 && (!block_table || !seq_lens || !block_table_out)))
        return FA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(block_table_out) ||
        !aligned4(free_pages) || !aligned4(free_count))
        return FA_ERR_ALIGNMENT;
    const size_t bytes = (size_t)num_seqs * max_pages_per_seq * 4;
    if (block_table != block_table_out && overlap(block_table, bytes, block_table_out, bytes))
        return FA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < fa::cache_compact_workspace_bytes(num_pages))
        return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    return map_rc(fa::launch_cache_compact(
        cache_pages(k_cache, v_cache, k_scale, v_scale, elem_bytes, num_pages, Hkv, d), block_table,
        seq_lens, num_seqs, max_pages_per_seq, block_table_out, free_pages, free_count, workspace,
        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Pointers and sizes that the cross-attention calls share.
int check_cross(const void *q, const void *k, const void *v, const void *o, const float *lse,
                const int *seq_lens_k, const int *cu_q, const int *cu_k, bool packed,
                long long total_q, long long total_k) {
    if (packed && (!cu_q || !cu_k)) return FA_ERR_INVALID_ARG;
    if (total_q > 0 && (!q || !o)) return FA_ERR_INVALID_ARG;
    if (total_k > 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
    if (total_q > INT32_MAX / 2 || total_k > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
        !aligned4(seq_lens_k) || !aligned4(cu_q) || !aligned4(cu_k))
        return FA_ERR_ALIGNMENT;
    return FA_OK;
}

// Dense (cu_q = cu_k = NULL: num_seqs sequences of Nq queries and Nk keys) or packed.
int fwd_cross_call(const void *q, const void *k, const void *v, void *o, float *lse,
                   const int *seq_lens_k, const int *cu_q, const int *cu_k, bool packed,
                   int num_seqs, long long total_q, long long total_k, int max_q, int max_k, int Hq,
                   int Hkv, int d, float scale, int o_dtype, void *stream) {
    if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0)
        return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, 0, 0, scale, o_dtype);
    if (rc) return rc;
    if (num_seqs == 0 || total_q == 0) return FA_OK;
    rc = check_cross(q, k, v, o, lse, seq_lens_k, cu_q, cu_k, packed, total_q, total_k);
    if (rc) return rc;
    fa::PrefillArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.cu_seqlens = cu_q;
    a.num_seqs = num_seqs;
    a.seqlen = packed ? 0 : max_q;
    a.total_tokens = (int)total_q;
    a.max_seqlen = max_q;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.scale = scale;
    a.o_fp32 = o_dtype == FA_OUT_FP32;
    a.cross = 1;
    a.cu_seqlens_k = cu_k;
    a.seq_lens_k = seq_lens_k;
    a.seqlen_k = packed ? 0 : max_k;
    a.total_k = (int)total_k;
    a.max_seqlen_k = max_k;
    return map_rc(fa::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

int bwd_cross_call(const void *q, const void *k, const void *v, const void *o, const void *dout,
                   const float *lse, void *dq, void *dk, void *dv, const int *seq_lens_k,
                   const int *cu_q, const int *cu_k, bool packed, int num_seqs, long long total_q,
                   long long total_k, int max_q, int max_k, int Hq, int Hkv, int d, float scale,
                   void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0)
        return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, 0, 0, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (num_seqs == 0 || (total_q == 0 && total_k == 0)) return FA_OK;
    rc = check_cross(q, k, v, o, lse, seq_lens_k, cu_q, cu_k, packed, total_q, total_k);
    if (rc) return rc;
    if (total_q > 0 && (!dout || !lse || !dq)) return FA_ERR_INVALID_ARG;
    if (total_k > 0 && (!dk || !dv)) return FA_ERR_INVALID_ARG;
    if (total_q * Hq > INT32_MAX / 2) return FA_ERR_UNSUPPORTED;
    if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FA_ERR_ALIGNMENT;
    if (total_q > 0) {
        if (!workspace || workspace_bytes < fa::bwd_workspace_bytes(total_q, Hq, d))
            return FA_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    }
    fa::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.cu_seqlens = cu_q;
    a.num_seqs = num_seqs;
    a.seqlen = packed ? 0 : max_q;
    a.total_tokens = (int)total_q;
    a.max_seqlen = max_q;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d;
    a.scale = scale;
    a.workspace = workspace;
    a.cross = 1;
    a.cu_seqlens_k = cu_k;
    a.seq_lens_k = seq_lens_k;
    a.seqlen_k = packed ? 0 : max_k;
    a.total_k = (int)total_k;
    a.max_seqlen_k = max_k;
    return map_rc(fa::launch_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fa_fwd_cross(const void *q, const void *k, const void *v, void *o, float *lse,
                 const int *seq_lens_k, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                 int o_dtype, void *stream) {
    if (B < 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
    return fwd_cross_call(q, k, v, o, lse, seq_lens_k, nullptr, nullptr, false, B, (long long)B * Nq,
                          (long long)B * Nk, Nq, Nk, Hq, Hkv, d, scale, o_dtype, stream);
}

int fa_fwd_varlen_cross(const void *q, const void *k, const void *v, void *o, float *lse,
                        const int *cu_seqlens_q, const int *cu_seqlens_k, int num_seqs, int total_q,
                        int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int d,
                        float scale, int o_dtype, void *stream) {
    return fwd_cross_call(q, k, v, o, lse, nullptr, cu_seqlens_q, cu_seqlens_k, true, num_seqs,
                          total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, o_dtype,
                          stream);
}

int fa_bwd_cross(const void *q, const void *k, const void *v, const void *o, const void *dout,
                 const float *lse, void *dq, void *dk, void *dv, const int *seq_lens_k, int B, int Hq,
                 int Hkv, int Nq, int Nk, int d, float scale, void *workspace,
                 size_t workspace_bytes, void *stream) {
    if (B < 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
    return bwd_cross_call(q, k, v, o, dout, lse, dq, dk, dv, seq_lens_k, nullptr, nullptr, false, B,
                          (long long)B * Nq, (long long)B * Nk, Nq, Nk, Hq, Hkv, d, scale, workspace,
                          workspace_bytes, stream);
}

int fa_bwd_varlen_cross(const void *q, const void *k, const void *v, const void *o,
                        const void *dout, const float *lse, void *dq, void *dk, void *dv,
                        const int *cu_seqlens_q, const int *cu_seqlens_k, int num_seqs, int total_q,
                        int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int d,
                        float scale, void *workspace, size_t workspace_bytes, void *stream) {
    return bwd_cross_call(q, k, v, o, dout, lse, dq, dk, dv, nullptr, cu_seqlens_q, cu_seqlens_k,
                          true, num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d,
                          scale, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

constexpr int kSharedMaxGroup = 128;   // query heads per KV head

// Sequences that one launch of decode_cross takes: blocks of 256 rows bound it.
int cross_batch(int B, long long rows_per_seq) {
    const long long pairs = (rows_per_seq + 255) / 256;
    const long long most = fa::kSharedMaxItems / pairs;
    return (int)std::min<long long>(B, std::min<long long>(most, fa::kSharedMaxSeqs));
}

// Sizes decode_cross can take: rows of a sequence in one launch's items, and
// the plan's cost (below) within 32 bits.
bool cross_fits(int Hq, int Hkv, int Nq, int Nk) {
    const int G = Hq / Hkv;
    const long long rows = (long long)Nq * G;
    return G <= kSharedMaxGroup && rows <= 256ll * fa::kSharedMaxItems &&
           fa::kSharedMaxItems * 8ll * (Nk / 128 + 2) <= INT32_MAX / 2;
}

}  // namespace

extern "C" {

size_t fa_decode_shared_workspace_bytes(int num_seqs, int Hq, int Hkv, int d) {
    if (num_seqs <= 0 || num_seqs > fa::kSharedMaxSeqs || Hkv <= 0 || Hq <= 0 || Hq % Hkv ||
        Hq / Hkv > kSharedMaxGroup || (d != 64 && d != 128))
        return 0;
    return fa::shared_workspace_bytes((long long)num_seqs * (Hq / Hkv), Hkv, d, true);
}

int fa_decode_shared(const void *q, const void *k_cache, const void *v_cache,
                     const int *block_table, const int *seq_lens, const int *cu_groups,
                     const int *prefix_lens, void *o, float *lse, const float *sinks, int num_seqs,
                     int num_groups, int num_pages, int Hq, int Hkv, int d, int page_size,
                     int max_pages_per_seq, float scale, void *workspace, size_t workspace_bytes,
                     void *stream) {
    if (num_seqs < 0 || num_groups < 0 || num_groups > num_seqs || num_pages < 0 ||
        max_pages_per_seq <= 0)
        return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, 0, 0, scale, FA_OUT_BF16);
    if (rc) return rc;
    const int G = Hq / Hkv;
    if (page_size != 16 || num_seqs > fa::kSharedMaxSeqs || G > kSharedMaxGroup)
        return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return FA_OK;
    if (num_pages == 0) return FA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o ||
        (num_groups > 0 && (!cu_groups || !prefix_lens)))
        return FA_ERR_INVALID_ARG;
    // 32-bit row coordinates, page counts and plan costs (at most 8 per block of 8 pages, 5 per item)
    const long long items = 2ll * num_seqs + (long long)num_seqs * G / 256 + 1;
    if ((long long)num_pages * page_size > INT32_MAX / 2 || max_pages_per_seq >= 1 << 22 ||
        items * 8 * (max_pages_per_seq / 8 + 2) > INT32_MAX / 2)
        return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
        !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(cu_groups) ||
        !aligned4(prefix_lens) || !aligned4(lse) || !aligned4(sinks))
        return FA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < fa_decode_shared_workspace_bytes(num_seqs, Hq, Hkv, d))
        return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    fa::SharedArgs a{};
    a.q = q; a.k = k_cache; a.v = v_cache;
    a.block_table = block_table; a.lens = seq_lens;
    a.cu_groups = cu_groups; a.prefix_lens = prefix_lens;
    a.o = o; a.lse = lse; a.sinks = sinks;
    a.paged = 1;
    a.S = num_seqs;
    a.num_groups = num_groups;
    a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.Nq = 1;
    a.scale = scale;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return map_rc(fa::launch_shared(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_decode_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
    if (B <= 0 || Nq <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || (d != 64 && d != 128) ||
        !cross_fits(Hq, Hkv, Nq, 0))
        return 0;
    const long long rows = (long long)Nq * (Hq / Hkv);
    return fa::shared_workspace_bytes(cross_batch(B, rows) * rows, Hkv, d, false);
}

int fa_decode_cross(const void *q, const void *k, const void *v, const int *seq_lens_k, void *o,
                    float *lse, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                    void *workspace, size_t workspace_bytes, void *stream) {
    if (B < 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
    int rc = check_common(Hq, Hkv, d, 0, 0, scale, FA_OUT_BF16);
    if (rc) return rc;
    if (B == 0 || Nq == 0) return FA_OK;
    rc = check_cross(q, k, v, o, lse, seq_lens_k, nullptr, nullptr, false, (long long)B * Nq,
                     (long long)B * Nk);
    if (rc) return rc;
    if (!cross_fits(Hq, Hkv, Nq, Nk)) return FA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < fa_decode_cross_workspace_bytes(B, Hq, Hkv, Nq, d))
        return FA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return FA_ERR_ALIGNMENT;
    const int batch = cross_batch(B, (long long)Nq * (Hq / Hkv));
    for (int s0 = 0; s0 < B; s0 += batch) {    // (one launch after the other uses the workspace)
        const size_t q0 = (size_t)s0 * Nq * Hq, k0 = (size_t)s0 * Nk * Hkv * d * 2;
        fa::SharedArgs a{};
        a.q = static_cast<const char *>(q) + q0 * d * 2;
        a.k = k ? static_cast<const char *>(k) + k0 : nullptr;
        a.v = v ? static_cast<const char *>(v) + k0 : nullptr;
        a.lens = seq_lens_k ? seq_lens_k + s0 : nullptr;
        a.o = static_cast<char *>(o) + q0 * d * 2;
        a.lse = lse ? lse + q0 : nullptr;
        a.S = std::min(batch, B - s0);
        a.S_all = B - s0;
        a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.Nq = Nq; a.Nk = Nk;
        a.scale = scale;
        a.workspace = workspace; a.workspace_bytes = workspace_bytes;
        rc = map_rc(fa::launch_shared(a, static_cast<cudaStream_t>(stream)));
        if (rc) return rc;
    }
    return FA_OK;
}

const char *fa_status_string(int status) {
    switch (status) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration";
    case FA_ERR_ALIGNMENT: return "pointer not aligned";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_CUDA: return "CUDA runtime error";
    case FA_ERR_TIMEOUT: return "device-side wait timed out";
    case FA_ERR_PAGES: return "no free cache page left";
    default: return "unknown status";
    }
}

int fa_check_device_error(void *stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return FA_ERR_CUDA;
    int word = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&word, fa::g_device_error, sizeof word) != cudaSuccess)
        return FA_ERR_CUDA;
    if (word && cudaMemcpyToSymbol(fa::g_device_error, &zero, sizeof zero) != cudaSuccess)
        return FA_ERR_CUDA;
    if (word == fa::kDevErrTimeout) return FA_ERR_TIMEOUT;
    if (word == fa::kDevErrInput) return FA_ERR_INVALID_ARG;
    if (word == fa::kDevErrPages) return FA_ERR_PAGES;
    return word ? FA_ERR_CUDA : FA_OK;
}

int fa_selftest_watchdog(void *stream) {
    fa::watchdog_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>();
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_version(void) { return 100; }

}  // extern "C"
