// C ABI of the node-level operators around a convolution: the type embedding,
// the block norm and the gradient norm with clipping (contracts in
// include/eqconv.h).  Arguments are checked here; nothing allocates per call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <utility>
#include <vector>

#include "eqc_elem.cuh"
#include "eqc_layers.h"
#include "eqc_plan.h"
#include "eqconv.h"

using eqc::aligned_to;
using eqc::check_device;
using eqc::cuda_status;
using eqc::type_bytes;

namespace {

constexpr int kMaxEmbedC = 65536;
constexpr int kMaxNormC = 16384;

int layer_plan(eqconv_plan_t* out, const eqc::LayerSpec& spec, int C, int D) {
    eqconv_plan_s* p = new (std::nothrow) eqconv_plan_s();
    eqc::LayerSpec* s = new (std::nothrow) eqc::LayerSpec(spec);
    if (!p || !s) {
        delete p;
        delete s;
        return EQCONV_ERR_CUDA;
    }
    p->C = C;
    p->lin = p->lout = spec.L;
    p->D_in = p->D_out = D;
    p->D_sh = 1;
    p->node_product = true;   // not a convolution plan
    p->layer = s;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess) e = cudaMalloc(&p->d_status, sizeof(unsigned));
    if (e == cudaSuccess) {
        e = cudaMemset(p->d_status, 0, sizeof(unsigned));
        if (e != cudaSuccess) cudaFree(p->d_status);
    }
    if (e != cudaSuccess) {
        delete p;
        delete s;
        return cuda_status(e, "plan creation");
    }
    *out = p;
    return EQCONV_OK;
}

const eqc::LayerSpec* embedding(eqconv_plan_t plan) { return plan && plan->layer && !plan->layer->norm ? plan->layer : nullptr; }
const eqc::LayerSpec* block_norm(eqconv_plan_t plan) { return plan && plan->layer && plan->layer->norm ? plan->layer : nullptr; }

// The checks that both directions of the embedding share.
int embed_args(eqconv_plan_t plan, int64_t N, const void* ids, int id_bits, float scale, int64_t row_stride,
               eqc::EmbedArgs& a) {
    const eqc::LayerSpec* s = embedding(plan);
    if (!s || N < 0 || N > INT32_MAX - 1 || (id_bits != 32 && id_bits != 64) || row_stride < 0)
        return EQCONV_ERR_INVALID_ARG;
    const int rc = check_device(plan);
    if (rc != EQCONV_OK) return rc;
    if (N > 0 && (!ids || !aligned_to(ids, id_bits / 8))) return EQCONV_ERR_INVALID_ARG;
    a.V = s->V;
    a.padding = s->padding;
    a.C = plan->C;
    a.in_type = s->in_type;
    a.out_type = s->out_type;
    a.id_bits = id_bits;
    a.N = N;
    a.ids = ids;
    a.scale = scale;
    a.status = plan->d_status;
    return EQCONV_OK;
}

// Both ranges of bytes, half open, have a byte in common.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
    return na > 0 && nb > 0 && p < q + nb && q < p + na;
}

int norm_args(eqconv_plan_t plan, int N, const void* x, const void* b, const void* gate, const float* w_post,
              const float* w_pre, float scale, eqc::BlockNormArgs& a) {
    const eqc::LayerSpec* s = block_norm(plan);
    if (!s || N < 0) return EQCONV_ERR_INVALID_ARG;
    const int rc = check_device(plan);
    if (rc != EQCONV_OK) return rc;
    const size_t es = type_bytes(s->in_type);
    const bool post = w_post != nullptr;
    if (!post && !w_pre) return EQCONV_ERR_INVALID_ARG;
    if (N > 0 && (!x || (post && !b) || (post && s->gate != EQCONV_GATE_NONE && !gate))) return EQCONV_ERR_INVALID_ARG;
    if ((!post && (b || gate)) || (s->gate == EQCONV_GATE_NONE && gate)) return EQCONV_ERR_INVALID_ARG;
    if (!aligned_to(x, es) || !aligned_to(b, es) || !aligned_to(gate, es) || !aligned_to(w_post, 4) ||
        !aligned_to(w_pre, 4))
        return EQCONV_ERR_INVALID_ARG;
    a.N = N;
    a.L = s->L;
    a.C = plan->C;
    a.type = s->in_type;
    a.gate_kind = s->gate;
    a.eps = s->eps;
    a.scale = scale;
    a.x = x;
    a.b = b;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.status = plan->d_status;
    return EQCONV_OK;
}

// A tensor fits one launch (2^30 chunks of 32 KB, its start up to 15 bytes into the first).
constexpr int64_t kMaxTensorBytes = (int64_t(1) << 45) - 16;

int check_tensors(int n, const eqconv_tensor_t* t) {
    if (n < 0 || (n > 0 && !t)) return EQCONV_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const size_t es = type_bytes(t[i].type);
        if (!es || t[i].n < 0 || t[i].n > kMaxTensorBytes / (int64_t)es) return EQCONV_ERR_INVALID_ARG;
        if (t[i].n > 0 && (!t[i].in || !aligned_to(t[i].in, es))) return EQCONV_ERR_INVALID_ARG;
    }
    return EQCONV_OK;
}

// Every output is its own input or overlaps no other tensor of the list.
int check_outputs(int n, const eqconv_tensor_t* t) {
    struct Range {
        uintptr_t from, to;
        bool write;
    };
    std::vector<Range> r;
    r.reserve(2 * (size_t)n);
    for (int i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        const size_t es = type_bytes(t[i].type);
        if (!t[i].out || !aligned_to(t[i].out, es)) return EQCONV_ERR_INVALID_ARG;
        const uintptr_t in = reinterpret_cast<uintptr_t>(t[i].in), out = reinterpret_cast<uintptr_t>(t[i].out);
        const size_t bytes = (size_t)t[i].n * es;
        r.push_back({out, out + bytes, true});
        if (in != out) r.push_back({in, in + bytes, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
    uintptr_t written = 0, touched = 0;   // ends of what was written and of all seen so far
    for (const Range& a : r) {
        if (a.from < written || (a.write && a.from < touched)) return EQCONV_ERR_INVALID_ARG;
        if (a.write) written = std::max(written, a.to);
        touched = std::max(touched, a.to);
    }
    return EQCONV_OK;
}

}  // namespace

extern "C" {

int eqconv_embedding_plan_create(eqconv_plan_t* out, int64_t n_types, int C, int table_type, int out_type,
                                 int64_t padding) {
    if (!out) return EQCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (n_types < 1 || C < 1 || padding < -1 || padding >= n_types || !type_bytes(table_type) ||
        !type_bytes(out_type))
        return EQCONV_ERR_INVALID_ARG;
    if (n_types > INT32_MAX - 2 || C > kMaxEmbedC || (out_type != table_type && table_type != EQCONV_F32))
        return EQCONV_ERR_UNSUPPORTED;
    eqc::LayerSpec s{};
    s.V = n_types;
    s.padding = padding;
    s.in_type = table_type;
    s.out_type = out_type;
    return layer_plan(out, s, C, 1);
}

int eqconv_embedding(eqconv_plan_t plan, int64_t N, const void* ids, int id_bits, const void* table,
                     int64_t table_stride, float scale, void* y, int64_t y_stride, eqconv_stream_t stream) {
    eqc::EmbedArgs a{};
    const int rc = embed_args(plan, N, ids, id_bits, scale, table_stride, a);
    if (rc != EQCONV_OK) return rc;
    if (N == 0) return EQCONV_OK;
    if (!table || !y || !aligned_to(table, type_bytes(a.in_type)) || !aligned_to(y, type_bytes(a.out_type)) ||
        y_stride < a.C || (a.V > 1 && table_stride < a.C))
        return EQCONV_ERR_INVALID_ARG;
    return cuda_status(eqc::embed_forward(a, table, table_stride, y, y_stride, (cudaStream_t)stream), "embedding");
}

size_t eqconv_embedding_workspace_bytes(eqconv_plan_t plan, int64_t N) {
    const eqc::LayerSpec* s = embedding(plan);
    if (!s || N < 0 || N > INT32_MAX - 1) return 0;
    return eqc::embed_workspace(s->V, plan->C, N);
}

int eqconv_embedding_backward(eqconv_plan_t plan, int64_t N, const void* ids, int id_bits, const void* gy,
                              int64_t gy_stride, float scale, void* dtable, void* workspace, size_t workspace_bytes,
                              eqconv_stream_t stream) {
    eqc::EmbedArgs a{};
    const int rc = embed_args(plan, N, ids, id_bits, scale, gy_stride, a);
    if (rc != EQCONV_OK) return rc;
    if ((N > 0 && (!gy || !aligned_to(gy, type_bytes(a.out_type)))) || !dtable ||
        !aligned_to(dtable, type_bytes(a.in_type)))
        return EQCONV_ERR_INVALID_ARG;
    const size_t need = eqc::embed_workspace(a.V, a.C, N);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))) return EQCONV_ERR_WORKSPACE;
    return cuda_status(eqc::embed_backward(a, gy, gy_stride, dtable, workspace, (cudaStream_t)stream),
                       "embedding backward");
}

int eqconv_block_norm_plan_create(eqconv_plan_t* out, const char* irreps, int C, int type, int gate, float eps) {
    if (!out) return EQCONV_ERR_INVALID_ARG;
    *out = nullptr;
    const int L = eqc::natural_prefix(irreps);
    if (L == -1 || C < 1 || !type_bytes(type) || gate < EQCONV_GATE_NONE || gate > EQCONV_GATE_TANH || !(eps > 0.f) ||
        std::isinf(eps))
        return EQCONV_ERR_INVALID_ARG;
    if (L == -2 || C > kMaxNormC) return EQCONV_ERR_UNSUPPORTED;
    eqc::LayerSpec s{};
    s.norm = true;
    s.in_type = s.out_type = type;
    s.L = L;
    s.gate = gate;
    s.eps = eps;
    return layer_plan(out, s, C, (L + 1) * (L + 1));
}

int eqconv_block_norm(eqconv_plan_t plan, int N, const void* x, const void* b, const void* gate, const float* w_post,
                      const float* w_pre, float scale, void* x_out, void* h, float* stats, eqconv_stream_t stream) {
    eqc::BlockNormArgs a{};
    const int rc = norm_args(plan, N, x, b, gate, w_post, w_pre, scale, a);
    if (rc != EQCONV_OK) return rc;
    if ((!w_post && x_out) || (!w_pre && h)) return EQCONV_ERR_INVALID_ARG;
    if (N == 0) return EQCONV_OK;
    const size_t es = type_bytes(a.type);
    if ((w_post && !x_out) || (w_pre && !h) || !aligned_to(x_out, es) || !aligned_to(h, es) || !aligned_to(stats, 4))
        return EQCONV_ERR_INVALID_ARG;
    const int64_t bytes = (int64_t)N * (a.L + 1) * (a.L + 1) * a.C * (int64_t)es;
    const int64_t gbytes = gate ? (int64_t)N * (a.L + 1) * a.C * (int64_t)es : 0;
    for (const void* o : {(const void*)x_out, (const void*)h})
        if (o && (overlap(o, bytes, x, bytes) || (b && overlap(o, bytes, b, bytes)) || overlap(o, bytes, gate, gbytes)))
            return EQCONV_ERR_INVALID_ARG;
    if (x_out && h && overlap(x_out, bytes, h, bytes)) return EQCONV_ERR_INVALID_ARG;
    a.x_out = x_out;
    a.h = h;
    a.stats = stats;
    return cuda_status(eqc::block_norm_forward(a, (cudaStream_t)stream), "block norm");
}

size_t eqconv_block_norm_workspace_bytes(eqconv_plan_t plan, int N) {
    const eqc::LayerSpec* s = block_norm(plan);
    if (!s || N < 0) return 0;
    return eqc::block_norm_workspace(s->L, plan->C, N);
}

int eqconv_block_norm_backward(eqconv_plan_t plan, int N, const void* x, const void* b, const void* gate,
                               const float* w_post, const float* w_pre, float scale, const float* stats,
                               const void* g_x, const void* g_h, void* dx, void* db, void* dgate, float* dw_post,
                               float* dw_pre, void* workspace, size_t workspace_bytes, eqconv_stream_t stream) {
    eqc::BlockNormArgs a{};
    const int rc = norm_args(plan, N, x, b, gate, w_post, w_pre, scale, a);
    if (rc != EQCONV_OK) return rc;
    const size_t es = type_bytes(a.type);
    if ((!w_post && (g_x || db || dgate || dw_post)) || (!w_pre && (g_h || dw_pre)) || (!gate && dgate && N > 0) ||
        !aligned_to(dw_post, 4) || !aligned_to(dw_pre, 4))
        return EQCONV_ERR_INVALID_ARG;
    if (N > 0) {
        if (!dx || !stats || (w_post && !db) || (gate && !dgate)) return EQCONV_ERR_INVALID_ARG;
        for (const void* p : {(const void*)g_x, (const void*)g_h, (const void*)dx, (const void*)db, (const void*)dgate})
            if (!aligned_to(p, es)) return EQCONV_ERR_INVALID_ARG;
        const int64_t bytes = (int64_t)N * (a.L + 1) * (a.L + 1) * a.C * (int64_t)es;
        const int64_t gbytes = (int64_t)N * (a.L + 1) * a.C * (int64_t)es;
        const std::pair<const void*, int64_t> ins[] = {
            {x, bytes}, {b, b ? bytes : 0}, {gate, gate ? gbytes : 0}, {g_x, g_x ? bytes : 0}, {g_h, g_h ? bytes : 0}};
        const std::pair<const void*, int64_t> outs[] = {{dx, bytes}, {db, db ? bytes : 0}, {dgate, dgate ? gbytes : 0}};
        for (int i = 0; i < 3; ++i) {
            for (const auto& in : ins)
                if (overlap(outs[i].first, outs[i].second, in.first, in.second)) return EQCONV_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (overlap(outs[i].first, outs[i].second, outs[j].first, outs[j].second))
                    return EQCONV_ERR_INVALID_ARG;
        }
        if (!workspace || workspace_bytes < eqc::block_norm_workspace(a.L, a.C, N) || !aligned_to(workspace, 16))
            return EQCONV_ERR_WORKSPACE;
    }
    a.stats = const_cast<float*>(stats);
    a.g_x = g_x;
    a.g_h = g_h;
    a.dx = dx;
    a.db = db;
    a.dgate = dgate;
    a.dw_post = dw_post;
    a.dw_pre = dw_pre;
    a.part = static_cast<float*>(workspace);
    return cuda_status(eqc::block_norm_backward(a, (cudaStream_t)stream), "block norm backward");
}

size_t eqconv_clip_workspace_bytes(int n, const eqconv_tensor_t* tensors) {
    if (check_tensors(n, tensors) != EQCONV_OK) return 0;
    return eqc::clip_workspace(n, tensors);
}

int eqconv_gradient_norm(int n, const eqconv_tensor_t* tensors, float* norm, void* workspace, size_t workspace_bytes,
                         eqconv_stream_t stream) {
    const int rc = check_tensors(n, tensors);
    if (rc != EQCONV_OK) return rc;
    if (!norm || !aligned_to(norm, 4)) return EQCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < eqc::clip_workspace(n, tensors) || !aligned_to(workspace, 16))
        return EQCONV_ERR_WORKSPACE;
    return cuda_status(eqc::clip_gradients(n, tensors, false, 0.f, 0.f, norm, workspace, (cudaStream_t)stream),
                       "gradient norm");
}

int eqconv_clip_gradients(int n, const eqconv_tensor_t* tensors, float max_norm, float eps, float* norm,
                          void* workspace, size_t workspace_bytes, eqconv_stream_t stream) {
    int rc = check_tensors(n, tensors);
    if (rc != EQCONV_OK) return rc;
    if (!(max_norm >= 0.f) || !(eps > 0.f) || std::isinf(eps) || !norm || !aligned_to(norm, 4))
        return EQCONV_ERR_INVALID_ARG;
    try {
        rc = check_outputs(n, tensors);
    } catch (const std::bad_alloc&) {
        return EQCONV_ERR_CUDA;   // host memory
    }
    if (rc != EQCONV_OK) return rc;
    if (!workspace || workspace_bytes < eqc::clip_workspace(n, tensors) || !aligned_to(workspace, 16))
        return EQCONV_ERR_WORKSPACE;
    return cuda_status(eqc::clip_gradients(n, tensors, true, max_norm, eps, norm, workspace, (cudaStream_t)stream),
                       "clip gradients");
}

}  // extern "C"
