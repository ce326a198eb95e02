// Host side of the block norm: the shape of a launch, and the weight gradients'
// last sum (kernels in eqc_bnorm.cuh, instances in eqc_bnorm_<type>.cu).
#include "eqc_bnorm_staged.cuh"

namespace eqc {
namespace bn {

cudaError_t run_f32(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);
cudaError_t run_bf16(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);
cudaError_t run_f16(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);
cudaError_t staged_f32(const StagedParams& s, const Staged& h, int grid, bool bwd, cudaStream_t st);
cudaError_t staged_bf16(const StagedParams& s, const Staged& h, int grid, bool bwd, cudaStream_t st);
cudaError_t staged_f16(const StagedParams& s, const Staged& h, int grid, bool bwd, cudaStream_t st);

namespace {

// dw[l, c]: the CTAs' partial rows in CTA order, 8 equal runs of them by the
// block's 8 warps and the warps' sums in order.  rows: degrees a CTA has sums
// of (L + 1, or 1 where CTAs first[l] .. first[l + 1] work on degree l).
__global__ void __launch_bounds__(256) bn_dw_reduce(const BnParams p, int rows, float* dw_post, float* dw_pre) {
    wait_for_last();
    __shared__ float s[8][32];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x, l = blockIdx.y;
    float* dw = blockIdx.z ? dw_pre : dw_post;
    if (!dw) return;
    const int from = rows == 1 ? p.first[l] : 0, to = rows == 1 ? p.first[l + 1] : p.first[p.L + 1];
    const int share = (to - from + 7) / 8;
    const int t0 = from + w * share, t1 = t0 + share < to ? t0 + share : to;
    float v = 0.f;
    if (c < p.C)
#pragma unroll 8
        for (int t = t0; t < t1; ++t)
            v += p.part[(((int64_t)t * 2 + blockIdx.z) * rows + (rows == 1 ? 0 : l)) * p.C + c];
    s[w][x] = v;
    __syncthreads();
    if (w != 0 || c >= p.C) return;
    for (int i = 1; i < 8; ++i) v += s[i][x];
    dw[l * p.C + c] = v;
}

BnParams params_of(const BlockNormArgs& a) {
    BnParams p{};
    p.N = a.N;
    p.C = a.C;
    p.L = a.L;
    p.gate_kind = a.gate_kind;
    p.eps = a.eps;
    p.scale = a.scale;
    p.x = a.x;
    p.b = a.b;
    p.gate = a.gate;
    p.w_post = a.w_post;
    p.w_pre = a.w_pre;
    p.x_out = a.x_out;
    p.h = a.h;
    p.stats = a.stats;
    p.g_x = a.g_x;
    p.g_h = a.g_h;
    p.dx = a.dx;
    p.db = a.db;
    p.dgate = a.dgate;
    p.part = a.part;
    return p;
}

// The bytes that all tensors start on, 16 at most.
int common_start(const BlockNormArgs& a) {
    uintptr_t all = 16;
    for (const void* q : {a.x, a.b, a.gate, (const void*)a.x_out, (const void*)a.h, a.g_x, a.g_h,
                          (const void*)a.dx, (const void*)a.db, (const void*)a.dgate, (const void*)a.w_post,
                          (const void*)a.w_pre})
        all |= reinterpret_cast<uintptr_t>(q);
    return (int)(all & (~all + 1));
}

// The staged launch of these arguments (slots 0: none).
Staged staged_for_args(const BlockNormArgs& a, bool bwd) {
    const int tensors = bwd ? 2 * (a.g_h != nullptr) + (a.b != nullptr) + (a.g_x != nullptr) : 1 + (a.b != nullptr);
    if (!tensors) return Staged{};
    return staged_shape(a.N, a.L, a.C, type_bytes(a.type), tensors, a.gate != nullptr, bwd,
                        common_start(a) == 16);
}

// rows: of the partial sums a CTA leaves (see bn_dw_reduce).
cudaError_t run(BnParams& p, const BlockNormArgs& a, bool bwd, cudaStream_t st, int* rows) {
    const Staged h = staged_for_args(a, bwd);
    if (h.slots) {
        StagedParams s{};
        const int es = type_bytes(a.type), node = (a.L + 1) * (a.L + 1) * a.C * es, gate = (a.L + 1) * a.C * es;
        p.width = h.width;
        s.slots = h.slots;
        s.nodes = h.nodes;
        s.batch = h.batch;
        s.ring = h.ring;
        s.total = ((int64_t)a.N + h.nodes - 1) / h.nodes;
        int o = 0;
        const auto place = [&](bool there, const void* from, int bytes) {
            if (!there) return 0;
            s.from[s.tensors] = static_cast<const unsigned char*>(from);
            s.bytes[s.tensors] = bytes;
            s.offset[s.tensors] = o;
            o += (int)part_bytes((int64_t)bytes * h.nodes, h.apart);
            return s.tensors++;
        };
        s.i_x = place(!bwd || a.g_h, a.x, node);
        s.i_b = place(a.b, a.b, node);
        s.i_gx = place(bwd && a.g_x, a.g_x, node);
        s.i_gh = place(bwd && a.g_h, a.g_h, node);
        s.i_g = place(a.gate, a.gate, gate);
        s.slot_bytes = o;
        s.ends = 16 / (gate * h.nodes) + 2;
        s.status = a.status;
        const int64_t most = (int64_t)kSMs * h.ctas;
        const int grid = (int)(s.total < most ? s.total : most);
        p.first[p.L + 1] = grid;
        s.p = p;
        *rows = a.L + 1;
        switch (a.type) {
            case EQCONV_F32: return staged_f32(s, h, grid, bwd, st);
            case EQCONV_BF16: return staged_bf16(s, h, grid, bwd, st);
            default: return staged_f16(s, h, grid, bwd, st);
        }
    }
    const Shape s = shape_of(a.L, a.C, type_bytes(a.type), bwd, common_start(a));
    *rows = 1;
    switch (a.type) {
        case EQCONV_F32: return run_f32(p, s, bwd, st);
        case EQCONV_BF16: return run_bf16(p, s, bwd, st);
        default: return run_f16(p, s, bwd, st);
    }
}

}  // namespace
}  // namespace bn

cudaError_t block_norm_forward(const BlockNormArgs& a, cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    bn::BnParams p = bn::params_of(a);
    int rows = 0;
    return bn::run(p, a, false, st, &rows);
}

size_t block_norm_workspace(int L, int C, int N) {
    // the most CTAs of any shape that C and the tensors' starts allow
    int most = bn::cta_cap(bn::Shape{0, 0, 0});
    for (const int es : {2, 4})
        for (const int pieces : {16, 8}) {
            const int k = bn::cta_cap(bn::shape_of(L, C, es, true, pieces));
            if (k > most) most = k;
        }
    int64_t ctas = (int64_t)bn::kSMs * most;
    if (ctas > (int64_t)N * (L + 1)) ctas = (int64_t)N * (L + 1);
    // or, with the sums of all degrees, one CTA an SM, or several of wide nodes (64 threads at least)
    int64_t staged = (int64_t)bn::kSMs * (L > 0 ? 4 : C < 2048 ? 16 : 2);
    if (staged > N) staged = N;
    const int64_t r = ctas + L + 1 > staged * (L + 1) ? ctas + L + 1 : staged * (L + 1);
    return (size_t)r * 2 * C * sizeof(float);
}

cudaError_t block_norm_backward(const BlockNormArgs& a, cudaStream_t st) {
    cudaError_t err;
    const size_t wbytes = (size_t)(a.L + 1) * a.C * sizeof(float);
    if (a.N == 0) {
        if (a.dw_post && (err = cudaMemsetAsync(a.dw_post, 0, wbytes, st)) != cudaSuccess) return err;
        if (a.dw_pre && (err = cudaMemsetAsync(a.dw_pre, 0, wbytes, st)) != cudaSuccess) return err;
        return cudaSuccess;
    }
    bn::BnParams p = bn::params_of(a);
    int rows = 0;
    if ((err = bn::run(p, a, true, st, &rows)) != cudaSuccess || (!a.dw_post && !a.dw_pre)) return err;
    err = launch_after(bn::bn_dw_reduce, dim3((a.C + 31) / 32, a.L + 1, 2), 256, st, p, rows, a.dw_post, a.dw_pre);
    count_launch();
    return err;
}

}  // namespace eqc
