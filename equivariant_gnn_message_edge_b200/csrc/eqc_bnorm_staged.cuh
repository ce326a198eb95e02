// Block norm, staged: whole nodes come to shared memory by bulk copies, a ring
// of slots ahead of the threads that work on them.  A node's rows of all
// degrees are contiguous in every tensor, so a slot is one copy per tensor; the
// copies of the next slots run while the current ones are summed and written,
// which is what the register-resident kernels of eqc_bnorm.cuh lack (their
// loads, sums and stores follow one another in each warp).  Used where two
// slots fit.  Rows that are no whole 16 bytes, or start off that boundary, are
// copied with the bytes around them up to the boundary (they are other nodes'),
// and a thread's channels are then `width` apart instead of neighbours, so that
// every element is read alone and a warp's lanes still lie side by side.
//
// A worker is a warp (32 / width nodes at a time, each warp with slots of its own)
// or, for wide nodes, the whole CTA (one node a slot).  Its threads own V
// channels of every row of the node.
//
// Bound by memory for fp32 (32768 lmax2 nodes of 128 channels: forward 111 us,
// 5.9 TB/s; backward 171 us, 5.9 TB/s).  16-bit nodes have half the bytes and
// the same arithmetic, conversions and waits per element (the same nodes in
// bf16: 56 us, 5.8 TB/s, and 133 us, 3.8 TB/s).
#pragma once

#include "eqc_bnorm.cuh"
#include "eqc_bulk.cuh"

namespace eqc {
namespace bn {

constexpr int kMaxSlots = 16;

struct StagedParams {
    BnParams p;
    int slots, nodes;          // slots of the ring, nodes a slot
    int batch;                 // of which a worker takes nodes / batch at a time
    int64_t total;             // slots' worth of nodes in all
    // the tensors of a slot: where they come from, their bytes a node, their place in the slot
    int tensors;
    const unsigned char* from[5];
    int bytes[5], offset[5];
    int i_x, i_b, i_gx, i_gh, i_g;       // which of them is which
    int slot_bytes, ring;      // bytes of a slot; where the ring begins in shared memory
    int ends;                  // the first and last slots whose pieces may reach over a tensor's ends
    unsigned* status;
};

struct Ring {
    unsigned char* base;
    uint64_t* full;            // a phase: one arrival per tensor, and its bytes
};

// The 16-byte pieces that hold tensor t of the nodes of one slot.
struct Window {
    const unsigned char* at;   // the first piece
    uint32_t lead, bytes;      // the nodes begin `lead` bytes into it; all bytes are there
    bool inside;               // every piece lies in the tensor
};
__device__ __forceinline__ Window window(const StagedParams& s, int t, int64_t g) {
    const int64_t n0 = g * s.nodes, left = s.p.N - n0, nodes = left < s.nodes ? left : s.nodes;
    const unsigned char* p = s.from[t] + n0 * s.bytes[t];
    Window w;
    w.lead = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    w.at = p - w.lead;
    w.bytes = (w.lead + (uint32_t)(nodes * s.bytes[t]) + 15) & ~15u;
    w.inside = w.at >= s.from[t] && w.at + w.bytes <= s.from[t] + (int64_t)s.p.N * s.bytes[t];
    return w;
}

// Copies of sequence number k of this CTA into its slot: tensor t by lane t,
// so that the warp that does it is held up by one copy's instructions only.
__device__ __forceinline__ void fill(const StagedParams& s, const Ring& r, int k, int lane) {
    const int64_t g = blockIdx.x + (int64_t)k * gridDim.x;
    if (g >= s.total || lane >= s.tensors) return;
    const Window w = window(s, lane, g);
    const int slot = k % s.slots;
    bulk::expect(r.full + slot, w.inside ? w.bytes + EQC_TEST_BULK_DEFICIT : 0);
    if (w.inside) bulk::copy(r.base + (int64_t)slot * s.slot_bytes + s.offset[lane], w.at, w.bytes, r.full + slot);
}

// What a worker that gave up at sequence number k does (by one thread, when all
// of them have left their loop): reports it, and waits, each time within the
// limit, for the copies on their way, so that they end before the CTA's memory
// does.  They are those of k and of the worker's next numbers, `step` apart, up
// to a ring's length.
__device__ __forceinline__ void give_up(const StagedParams& s, const Ring& r, int k, int step, int mine) {
    atomicOr(s.status, 4u);
    for (int j = k; j < mine && j < k + s.slots; j += step) bulk::wait(r.full + j % s.slots, (uint32_t)(j / s.slots) & 1u);
}

// How far into its first piece the nodes of a slot begin.
__device__ __forceinline__ uint32_t lead_of(const StagedParams& s, int t, int64_t g) {
    return ((uint32_t)reinterpret_cast<uintptr_t>(s.from[t]) + (uint32_t)g * s.nodes * s.bytes[t]) & 15u;
}

// The first and last nodes' pieces that reach over the tensor's ends are
// copied element by element, by the threads that wait for the slot (`lane` of
// `lanes`).  True if there were any: the caller then waits for the others.
template <class T>
__device__ __forceinline__ bool fill_ends(const StagedParams& s, const Ring& r, int k, int lane, int lanes) {
    const int64_t g = blockIdx.x + (int64_t)k * gridDim.x;
    if (g >= s.ends && g + s.ends < s.total) return false;
    bool any = false;
    for (int t = 0; t < s.tensors; ++t) {
        const Window w = window(s, t, g);
        if (w.inside) continue;
        any = true;
        const int64_t n0 = g * s.nodes, left = s.p.N - n0, nodes = left < s.nodes ? left : s.nodes;
        const T* from = reinterpret_cast<const T*>(w.at + w.lead);
        T* to = reinterpret_cast<T*>(r.base + (int64_t)(k % s.slots) * s.slot_bytes + s.offset[t] + w.lead);
        for (int i = lane; i < (int)(nodes * s.bytes[t] / sizeof(T)); i += lanes) to[i] = from[i];
    }
    if (any) bulk::fence_writes();       // the slot's next copies come behind these
    return any;
}

// A thread's V channels of a row: neighbours from `first` (on the vector's
// boundary), or (APART) first, first + step, ... below C, zeros behind C.
template <int V, bool APART>
struct Lanes {
    int first, step, C;
    template <class T>
    __device__ __forceinline__ void load(F2 (&v)[V / 2], const T* row) const {
        if constexpr (!APART) {
            load2<T, V>(v, row + first);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const int c = first + 2 * i * step, d = c + step;
                v[i] = F2(c < C ? to_float(row[c]) : 0.f, d < C ? to_float(row[d]) : 0.f);
            }
        }
    }
    template <class T>
    __device__ __forceinline__ void store(T* row, const F2 (&v)[V / 2]) const {
        if constexpr (!APART) {
            store2<T, V>(row + first, v);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const int c = first + 2 * i * step, d = c + step;
                float x, y;
                v[i].split(x, y);
                if (c < C) row[c] = from_float<T>(x);
                if (d < C) row[d] = from_float<T>(y);
            }
        }
    }
};

// What one worker sees of its node: the tensors' slot parts.
template <class T>
struct View {
    const T *x, *b, *gx, *gh, *g;
};

template <class T, int V, int L, bool APART>
__device__ __forceinline__ void fwd_node(const BnParams& p, const View<T>& s, const float* w, const Lanes<V, APART>& q,
                                         bool own, bool live, int64_t row, int64_t srow, bool lead,
                                         WorkerSum<L + 1>& sum) {
    constexpr int H = V / 2;
    const bool post = p.b != nullptr, pre = p.w_pre != nullptr, gated = p.gate != nullptr;
    float sb[L + 1], sy[L + 1];
#pragma unroll
    for (int l = 0; l <= L; ++l) sb[l] = sy[l] = 0.f;
    if (post) {
#pragma unroll
        for (int l = 0; l <= L; ++l)
            if (own) {
                F2 v(0.f);
#pragma unroll
                for (int m = 0; m < 2 * l + 1; ++m) {
                    F2 b[H];
                    q.load(b, s.b + (l * l + m) * p.C);
#pragma unroll
                    for (int i = 0; i < H; ++i) v = fma2(b[i], b[i], v);
                }
                sb[l] = v.sum();
            }
        sum(sb);
    }
    F2 k[L + 1][H];                  // y = x + k b
#pragma unroll
    for (int l = 0; l <= L; ++l) {
        if (post) sb[l] = rsqrtf(sb[l] * (1.f / ((2 * l + 1) * (float)p.C)) + p.eps);
        if (!own) continue;
        if (post) {
            q.load(k[l], w + l * p.C);
#pragma unroll
            for (int i = 0; i < H; ++i) k[l][i] = mul2(k[l][i], F2(p.scale * sb[l]));
            if (gated) {
                F2 g[H], a[H], da[H];
                q.load(g, s.g + l * p.C);
                gate_values<V, sizeof(T) == 2>(p.gate_kind, g, a, da);
#pragma unroll
                for (int i = 0; i < H; ++i) k[l][i] = mul2(k[l][i], a[i]);
            }
        }
        F2 v(0.f);
#pragma unroll
        for (int m = 0; m < 2 * l + 1; ++m) {
            F2 y[H];
            q.load(y, s.x + (l * l + m) * p.C);
            if (post) {
                F2 b[H];
                q.load(b, s.b + (l * l + m) * p.C);
#pragma unroll
                for (int i = 0; i < H; ++i) y[i] = fma2(k[l][i], b[i], y[i]);
                if (live) q.store(static_cast<T*>(p.x_out) + row + (l * l + m) * p.C, y);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) v = fma2(y[i], y[i], v);
        }
        sy[l] = v.sum();
    }
    if (pre) {
        sum(sy);
#pragma unroll
        for (int l = 0; l <= L; ++l) {
            sy[l] = rsqrtf(sy[l] * (1.f / ((2 * l + 1) * (float)p.C)) + p.eps);
            if (!own) continue;
            F2 wi[H];
            q.load(wi, w + (L + 1 + l) * p.C);
#pragma unroll
            for (int i = 0; i < H; ++i) wi[i] = mul2(wi[i], F2(sy[l]));
#pragma unroll
            for (int m = 0; m < 2 * l + 1; ++m) {
                F2 y[H];
                q.load(y, s.x + (l * l + m) * p.C);
                if (post) {
                    F2 b[H];
                    q.load(b, s.b + (l * l + m) * p.C);
#pragma unroll
                    for (int i = 0; i < H; ++i) y[i] = fma2(k[l][i], b[i], y[i]);
                }
#pragma unroll
                for (int i = 0; i < H; ++i) y[i] = mul2(y[i], wi[i]);
                if (live) q.store(static_cast<T*>(p.h) + row + (l * l + m) * p.C, y);
            }
        }
    }
    if (p.stats && lead && live)
#pragma unroll
        for (int l = 0; l <= L; ++l) {
            if (post) p.stats[srow + l] = sb[l];
            if (pre) p.stats[(int64_t)p.N * (L + 1) + srow + l] = sy[l];
        }
}

// With f = scale a(gate) w_post, bs = b s_b and p = g_h w_pre, the mean that db
// needs is linear in the mean that t needs:
//   sum f bs t = sum f bs (g_x + s_y p) - s_y m1 sum f bs y,   m1 = s_y^2 mean(p y)
// so one round of sums serves both, and t, dx and db follow in one pass.
template <class T, int V, int L, bool APART>
__device__ __forceinline__ void bwd_node(const BnParams& p, const View<T>& s, const float* w, const Lanes<V, APART>& q,
                                         bool own, bool live, int64_t row, int64_t grow, const float (&sb)[L + 1],
                                         const float (&sy)[L + 1], F2 (&dwo)[L + 1][V / 2], F2 (&dwi)[L + 1][V / 2],
                                         WorkerSum<3 * (L + 1)>& sum) {
    constexpr int H = V / 2;
    // Rows in a loop where their code, element by element, would not stay in the instruction caches (20000 lmax2 nodes
    // of 81 channels 231 -> 168 us); side by side otherwise (128 channels: 169 us, 195 us in a loop).
    constexpr int kRows = APART && L >= 2 ? 1 : 2 * L + 1;
    const bool post = p.b != nullptr, pre = p.g_h != nullptr, gated = p.gate != nullptr, more = p.g_x != nullptr;
    F2 sa[L + 1][H], da[L + 1][H];     // scale a(gate), scale a'(gate)
    float sums[3 * (L + 1)];           // per degree: p y, f bs y, f bs (g_x + s_y p)
#pragma unroll
    for (int l = 0; l <= L; ++l) {
        sums[3 * l] = sums[3 * l + 1] = sums[3 * l + 2] = 0.f;
        if (!own) continue;
        if (gated) {
            F2 g[H];
            q.load(g, s.g + l * p.C);
            gate_values<V, sizeof(T) == 2>(p.gate_kind, g, sa[l], da[l]);
        }
        F2 wi[H], k[H], v0(0.f), v1(0.f), v2(0.f);
        if (pre) q.load(wi, w + (L + 1 + l) * p.C);
        if (post) q.load(k, w + l * p.C);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            sa[l][i] = gated ? mul2(sa[l][i], F2(p.scale)) : F2(p.scale);
            da[l][i] = gated ? mul2(da[l][i], F2(p.scale)) : F2(0.f);
            if (post) k[i] = mul2(mul2(k[i], sa[l][i]), F2(sb[l]));
        }
#pragma unroll kRows
        for (int m = 0; m < 2 * l + 1; ++m) {
            const int r = l * l + m;
            F2 b[H], t[H];
            if (post) q.load(b, s.b + r * p.C);
            if (post && more) q.load(t, s.gx + r * p.C);
            else
#pragma unroll
                for (int i = 0; i < H; ++i) t[i] = F2(0.f);
            if (pre) {
                F2 gh[H], y[H];
                q.load(y, s.x + r * p.C);
                q.load(gh, s.gh + r * p.C);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const F2 pp = mul2(gh[i], wi[i]);
                    if (post) {
                        const F2 fb = mul2(k[i], b[i]);
                        y[i] = add2(fb, y[i]);
                        v1 = fma2(fb, y[i], v1);
                        v2 = fma2(fb, fma2(pp, F2(sy[l]), t[i]), v2);
                    }
                    v0 = fma2(pp, y[i], v0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) v2 = fma2(mul2(k[i], b[i]), t[i], v2);
            }
        }
        sums[3 * l] = v0.sum();
        sums[3 * l + 1] = v1.sum();
        sums[3 * l + 2] = v2.sum();
    }
    sum(sums);
#pragma unroll
    for (int l = 0; l <= L; ++l) {
        if (!own) continue;
        const float inv_m = 1.f / ((2 * l + 1) * (float)p.C);
        const float m1 = sums[3 * l] * inv_m * sy[l] * sy[l] * sy[l];           // with t's factor s_y
        const float m2 = (sums[3 * l + 2] - m1 * sums[3 * l + 1]) * inv_m * sb[l] * sb[l];
        F2 wi[H], wo[H], k[H], tb[H], gy[H];      // wi: s_y w_pre
        if (pre) q.load(wi, w + (L + 1 + l) * p.C);
        if (post) q.load(wo, w + l * p.C);
        const F2 n1(-m1), n2(-m2), s1(sy[l]), s0(sb[l]);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            tb[i] = gy[i] = F2(0.f);
            if (pre) wi[i] = mul2(wi[i], s1);
            if (post) k[i] = mul2(mul2(wo[i], sa[l][i]), s0);
        }
#pragma unroll kRows
        for (int m = 0; m < 2 * l + 1; ++m) {
            const int r = l * l + m;
            F2 t[H], b[H];
            if (post) q.load(b, s.b + r * p.C);
            if (more) q.load(t, s.gx + r * p.C);
            else
#pragma unroll
                for (int i = 0; i < H; ++i) t[i] = F2(0.f);
            if (pre) {
                F2 gh[H], y[H];
                q.load(y, s.x + r * p.C);
                q.load(gh, s.gh + r * p.C);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if (post) y[i] = fma2(k[i], b[i], y[i]);
                    t[i] = fma2(gh[i], wi[i], fma2(y[i], n1, t[i]));
                    gy[i] = fma2(gh[i], y[i], gy[i]);
                }
            }
            if (live) q.store(static_cast<T*>(p.dx) + row + r * p.C, t);
            if (post) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    tb[i] = fma2(t[i], b[i], tb[i]);
                    t[i] = fma2(k[i], t[i], mul2(b[i], n2));
                }
                if (live) q.store(static_cast<T*>(p.db) + row + r * p.C, t);
            }
        }
        F2 dg[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            if (post) {
                const F2 u = mul2(tb[i], s0);
                if (live) dwo[l][i] = fma2(sa[l][i], u, dwo[l][i]);
                dg[i] = mul2(mul2(da[l][i], wo[i]), u);
            }
            if (live && pre) dwi[l][i] = fma2(gy[i], s1, dwi[l][i]);
        }
        if (gated && live) q.store(static_cast<T*>(p.dgate) + grow + l * p.C, dg);
    }
}

// Shared memory: [w_post, w_pre: 2 (L + 1) C floats] [ring of slots].
template <class T, int V, int L, bool BWD, bool CTA, bool APART>
__global__ void __launch_bounds__(CTA ? 256 : BWD ? 256 : 512, 1) bn_staged_kernel(const StagedParams s) {
    if constexpr (BWD) let_next_start();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kMaxSlots];
    __shared__ float red[CTA ? 2 * (BWD ? 3 : 1) * (L + 1) * 16 : 1];
    constexpr int D = (L + 1) * (L + 1);
    const BnParams& p = s.p;
    float* w = reinterpret_cast<float*>(smem);
    const Ring ring{smem + s.ring, full};
    const int workers = CTA ? 1 : blockDim.x / 32, worker = CTA ? 0 : threadIdx.x / 32;
    const int lane = CTA ? threadIdx.x : threadIdx.x & 31;
    const int width = CTA ? (int)blockDim.x : p.width;
    const int sub = CTA ? 0 : lane / width, x0 = lane - sub * width;
    const Lanes<V, APART> q{APART ? x0 : x0 * V, width, p.C};
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.slots; ++i) bulk::init(full + i, s.tensors);
        bulk::fence_init();
    }
    for (int i = threadIdx.x; i < (L + 1) * p.C; i += blockDim.x) {
        w[i] = p.w_post ? p.w_post[i] : 0.f;
        w[(L + 1) * p.C + i] = p.w_pre ? p.w_pre[i] : 0.f;
    }
    __syncthreads();
    if (threadIdx.x < 32)
        for (int k = 0; k < s.slots; ++k) fill(s, ring, k, threadIdx.x);
    const bool own = q.first < p.C;
    F2 dwo[BWD ? L + 1 : 1][V / 2], dwi[BWD ? L + 1 : 1][V / 2];
#pragma unroll
    for (int l = 0; l < (BWD ? L + 1 : 1); ++l)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dwo[l][i] = dwi[l][i] = F2(0.f);
    WorkerSum<BWD ? 3 * (L + 1) : L + 1> sum{red, width, 0};
    const int mine = s.total > blockIdx.x ? (int)((s.total - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
    // a node's statistics are fetched while the worker's last node is worked on
    float sb_next[BWD ? L + 1 : 1], sy_next[BWD ? L + 1 : 1];
    const int each = CTA ? 1 : 32 / width;       // nodes a worker takes at a time
    const auto first_of = [&](int k) { return (blockIdx.x + (int64_t)k * gridDim.x) * s.nodes + sub; };
    const auto fetch = [&](int64_t n) {
#pragma unroll
        for (int l = 0; l < (BWD ? L + 1 : 1); ++l) {
            sb_next[l] = n < p.N && p.b ? __ldg(p.stats + n * (L + 1) + l) : 0.f;
            sy_next[l] = n < p.N && p.g_h ? __ldg(p.stats + ((int64_t)p.N + n) * (L + 1) + l) : 0.f;
        }
    };
    if constexpr (BWD)
        if (worker < mine) fetch(first_of(worker));
    int k = worker;
    for (; k < mine; k += workers) {
        const int slot = k % s.slots;
        // a worker's threads give up together: a warp's here, a CTA's at the barrier that ends the slot
        const bool there = bulk::wait(full + slot, (uint32_t)(k / s.slots) & 1u);
        if constexpr (!CTA)
            if (!__all_sync(0xffffffffu, there)) break;
        if constexpr (APART)
            if (fill_ends<T>(s, ring, k, lane, CTA ? blockDim.x : 32)) {
                if constexpr (CTA) __syncthreads();
                else __syncwarp();
            }
        const unsigned char* base = ring.base + (int64_t)slot * s.slot_bytes;
        const auto at = [&](int t) {
            const uint32_t lead = APART ? lead_of(s, t, blockIdx.x + (int64_t)k * gridDim.x) : 0;
            return base + s.offset[t] + lead;
        };
        const unsigned char *xs = at(s.i_x), *bs = at(s.i_b), *gxs = at(s.i_gx), *ghs = at(s.i_gh), *gs = at(s.i_g);
        const int batch = L == 0 && !CTA ? s.batch : 1;
        for (int m = 0; m < batch; ++m) {
            const int64_t n = first_of(k) + m * each;
            if (n - sub >= p.N) break;           // for all lanes alike
            const bool live = n < p.N;
            const int node = (m * each + sub) * D * p.C, group = (m * each + sub) * (L + 1) * p.C;
            const auto of = [&](const unsigned char* q, int i) { return reinterpret_cast<const T*>(q) + i; };
            const View<T> v{of(xs, node), of(bs, node), of(gxs, node), of(ghs, node), of(gs, group)};
            const int64_t row = n * D * p.C, grow = n * (L + 1) * p.C;
            if constexpr (BWD) {
                float sb[L + 1], sy[L + 1];
#pragma unroll
                for (int l = 0; l <= L; ++l) sb[l] = sb_next[l], sy[l] = sy_next[l];
                fetch(m + 1 < batch ? n + each : first_of(k + workers));
                bwd_node<T, V, L, APART>(p, v, w, q, own, live, row, grow, sb, sy, dwo, dwi, sum);
            } else {
                fwd_node<T, V, L, APART>(p, v, w, q, own, live, row, n * (L + 1), x0 == 0, sum);
            }
        }
        // everyone has read the slot: its next copies may come
        if constexpr (CTA) {
            if (!__syncthreads_and(there)) break;
        } else {
            __syncwarp();
        }
        if (lane < 32) fill(s, ring, k + s.slots, lane);
    }
    if (k < mine && lane == 0) give_up(s, ring, k, workers, mine);
    if constexpr (BWD) {
        float* part = p.part + (int64_t)blockIdx.x * 2 * (L + 1) * p.C;
        if constexpr (CTA) {
#pragma unroll
            for (int l = 0; l <= L; ++l)
                if (own) {
                    q.store(part + l * p.C, dwo[l]);
                    q.store(part + (L + 1 + l) * p.C, dwi[l]);
                }
        } else {
            // the warps' sums in order, and within a warp its nodes', one degree and kind at a time
            __syncthreads();      // every slot has been read
            float* t = reinterpret_cast<float*>(smem + s.ring);
#pragma unroll
            for (int l = 0; l <= L; ++l)
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    const int groups = workers * (32 / width), mine_at = (threadIdx.x / width) * width * V;
                    Lanes<V, APART>{q.first, q.step, width * V}.store(t + mine_at, which ? dwi[l] : dwo[l]);
                    __syncthreads();
                    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
                        float v = 0.f;
                        for (int g = 0; g < groups; ++g) v += t[(g * width) * V + c];
                        part[(which * (L + 1) + l) * p.C + c] = v;
                    }
                    __syncthreads();
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Wide rows (L = 0, more than 32 vectors across): a CTA takes a row out of its
// slot into registers (8 channels a thread), frees the slot at its first
// barrier, and does all arithmetic from registers, once per element: every
// factor of a channel is formed once and the weights stay in registers.  fp32
// rows are bound by memory (8191 x 4096: 116 and 165 us, 5.8 and 6.5 TB/s).
// 16-bit rows (74 and 126 us, 4.5 and 4.3 TB/s) are bound by latency: a
// scheduler has 8 warps forward and 4 backward, issues in 62 and 54 % of the
// cycles, and they wait for shared memory, results and the barriers of the
// row's sums; no pipe is busy for more than 37 %.

// Sums of K values over the CTA; red: [2][K][16], zeros behind the last warp.
// Returns whether `ok` holds for every thread.
template <int K>
struct CtaSum {
    float* red;
    int flip;
    __device__ __forceinline__ bool operator()(float (&v)[K], bool ok) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        float* r = red + flip * K * 16;
        flip ^= 1;       // the next sums' buffer: one barrier a round is enough
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < K; ++i) r[i * 16 + (threadIdx.x >> 5)] = v[i];
        ok = __syncthreads_and(ok);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            F2 q[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) load2<float, 4>(q[j], r + i * 16 + 4 * j);
            v[i] = add2(add2(add2(q[0][0], q[0][1]), add2(q[1][0], q[1][1])),
                        add2(add2(q[2][0], q[2][1]), add2(q[3][0], q[3][1])))
                       .sum();
        }
        return ok;
    }
};

template <class T, int V, int J, bool BWD, bool APART>
__global__ void __launch_bounds__(512, BWD || J * V > 8 ? 1 : 2) bn_row_kernel(const StagedParams s) {
    if constexpr (BWD) let_next_start();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kMaxSlots];
    constexpr int K = BWD ? 3 : 1;
    __shared__ __align__(16) float red[2 * K * 16];
    const BnParams& p = s.p;
    const Ring ring{smem, full};
    const bool post = p.b != nullptr, gated = p.gate != nullptr;
    const bool pre = BWD ? p.g_h != nullptr : p.w_pre != nullptr, more = p.g_x != nullptr;
    const float inv_m = 1.f / (float)p.C;
    for (int i = threadIdx.x; i < 2 * K * 16; i += blockDim.x) red[i] = 0.f;
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.slots; ++i) bulk::init(full + i, s.tensors);
        bulk::fence_init();
    }
    __syncthreads();
    if (threadIdx.x < 32)
        for (int k = 0; k < s.slots; ++k) fill(s, ring, k, threadIdx.x);
    constexpr int H = V / 2;
    bool own[J];
    Lanes<V, APART> q[J];
    F2 wo[J][H], wi[J][H], dwo[J][H], dwi[J][H];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        q[j] = Lanes<V, APART>{(int)(APART ? threadIdx.x + j * V * blockDim.x : (threadIdx.x + j * blockDim.x) * V),
                               (int)blockDim.x, p.C};
        own[j] = q[j].first < p.C;
        if (own[j] && post) q[j].load(wo[j], p.w_post);
        if (own[j] && pre) q[j].load(wi[j], p.w_pre);
#pragma unroll
        for (int i = 0; i < H; ++i) dwo[j][i] = dwi[j][i] = F2(0.f);
    }
    CtaSum<K> sum{red, 0};
    const F2 scale(p.scale);
    const int mine = s.total > blockIdx.x ? (int)((s.total - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
    // a row's statistics are fetched while the row before is worked on
    float sb_next = 0.f, sy_next = 0.f;
    const auto fetch = [&](int64_t n) {
        if (post && n < p.N) sb_next = __ldg(p.stats + n);
        if (pre && n < p.N) sy_next = __ldg(p.stats + p.N + n);
    };
    if constexpr (BWD) fetch(blockIdx.x);
    int k = 0;
    for (int slot = 0, turn = 0; k < mine; ++k) {
        const int64_t n = blockIdx.x + (int64_t)k * gridDim.x;
        float sb = sb_next, sy = sy_next;
        if constexpr (BWD) fetch(n + gridDim.x);
        const bool there = bulk::wait(full + slot, (uint32_t)turn & 1u);      // all give up together, at the first sums
        if constexpr (APART)
            if (fill_ends<T>(s, ring, k, threadIdx.x, blockDim.x)) __syncthreads();
        const unsigned char* base = ring.base + (int64_t)slot * s.slot_bytes;
        const auto at = [&](int t) {
            const uint32_t lead = APART ? lead_of(s, t, n) : 0;
            return reinterpret_cast<const T*>(base + s.offset[t] + lead);
        };
        const auto to = [&](void* y) { return static_cast<T*>(y) + n * p.C; };
        const auto release = [&] {       // behind a barrier: every thread has read the slot (and written its ends)
            if (threadIdx.x < 32) fill(s, ring, k + s.slots, threadIdx.x);
        };
        // y: x, then x_out; bs: b, then b / rms(b); sa, da: scale a(gate), scale a'(gate)
        F2 y[J][H], bs[J][H], sa[J][H], da[J][H];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!own[j]) continue;
            if (!BWD || pre) q[j].load(y[j], at(s.i_x));
            if (post) q[j].load(bs[j], at(s.i_b));
            if (gated) {
                F2 g[H];
                q[j].load(g, at(s.i_g));
                gate_values<V, sizeof(T) == 2>(p.gate_kind, g, sa[j], da[j]);
#pragma unroll
                for (int i = 0; i < H; ++i) sa[j][i] = mul2(sa[j][i], scale);
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) sa[j][i] = scale;
            }
        }
        if constexpr (!BWD) {
            if (post) {
                F2 v(0.f);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (own[j])
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            v = fma2(bs[j][i], bs[j][i], v);
                            sa[j][i] = mul2(sa[j][i], wo[j][i]);
                        }
                float total[1] = {v.sum()};
                if constexpr (!BWD)
                    if (!sum(total, there)) break;
                sb = rsqrtf(total[0] * inv_m + p.eps);
                release();
            }
            F2 v(0.f);
            const F2 s0(sb);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (own[j]) {
                    if (post) {
#pragma unroll
                        for (int i = 0; i < H; ++i) y[j][i] = fma2(sa[j][i], mul2(bs[j][i], s0), y[j][i]);
                        q[j].store(to(p.x_out), y[j]);
                    }
#pragma unroll
                    for (int i = 0; i < H; ++i) v = fma2(y[j][i], y[j][i], v);
                }
            if (pre) {
                float total[1] = {v.sum()};
                if constexpr (!BWD)
                    if (!sum(total, there)) break;
                sy = rsqrtf(total[0] * inv_m + p.eps);
                if (!post) release();
                const F2 s1(sy);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (own[j]) {
#pragma unroll
                        for (int i = 0; i < H; ++i) y[j][i] = mul2(mul2(y[j][i], s1), wi[j][i]);
                        q[j].store(to(p.h), y[j]);
                    }
            }
            if (p.stats && threadIdx.x == 0) {
                if (post) p.stats[n] = sb;
                if (pre) p.stats[p.N + n] = sy;
            }
        } else {
            // one round of sums, as in bwd_node: p y, f bs y, f bs (g_x + s_y p)
            F2 gx[J][H], gh[J][H], v0(0.f), v1(0.f), v2(0.f);
            const F2 s0(sb), s1(sy);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j]) continue;
                if (more) q[j].load(gx[j], at(s.i_gx));
                else
#pragma unroll
                    for (int i = 0; i < H; ++i) gx[j][i] = F2(0.f);
                if (pre) q[j].load(gh[j], at(s.i_gh));
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    F2 fb;
                    if (post) {
                        bs[j][i] = mul2(bs[j][i], s0);
                        fb = mul2(mul2(sa[j][i], wo[j][i]), bs[j][i]);
                    }
                    if (pre) {
                        // t but for the mean's share, in the place of g_x
                        const F2 pp = mul2(gh[j][i], wi[j][i]);
                        gx[j][i] = fma2(pp, s1, gx[j][i]);
                        if (post) {
                            y[j][i] = add2(fb, y[j][i]);
                            v1 = fma2(fb, y[j][i], v1);
                        }
                        v0 = fma2(pp, y[j][i], v0);
                        dwi[j][i] = fma2(mul2(gh[j][i], y[j][i]), s1, dwi[j][i]);
                    }
                    if (post) v2 = fma2(fb, gx[j][i], v2);
                }
            }
            float total[3] = {v0.sum(), v1.sum(), v2.sum()};
            if constexpr (BWD)
                if (!sum(total, there)) break;
            release();
            const float m1 = total[0] * inv_m * sy * sy * sy;           // with t's factor s_y
            const F2 n1(-m1), n2(-((total[2] - m1 * total[1]) * inv_m));
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j]) continue;
                if (pre)
#pragma unroll
                    for (int i = 0; i < H; ++i) gx[j][i] = fma2(n1, y[j][i], gx[j][i]);
                q[j].store(to(p.dx), gx[j]);
                if (!post) continue;
                F2 dg[H];
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const F2 tb = mul2(gx[j][i], bs[j][i]);
                    dwo[j][i] = fma2(sa[j][i], tb, dwo[j][i]);
                    if (gated) dg[i] = mul2(mul2(da[j][i], scale), mul2(wo[j][i], tb));
                    gx[j][i] = mul2(s0, fma2(mul2(sa[j][i], wo[j][i]), gx[j][i], mul2(bs[j][i], n2)));
                }
                if (gated) q[j].store(to(p.dgate), dg);
                q[j].store(to(p.db), gx[j]);
            }
        }
        if (++slot == s.slots) {
            slot = 0;
            ++turn;
        }
    }
    if (k < mine && threadIdx.x == 0) give_up(s, ring, k, 1, mine);
    if constexpr (BWD) {
        float* part = p.part + (int64_t)blockIdx.x * 2 * p.C;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (own[j]) {
                q[j].store(part, dwo[j]);
                q[j].store(part + p.C, dwi[j]);
            }
    }
}

// How a staged launch is cut; slots 0: not staged.
struct Staged {
    int V, J, width, threads, slots, nodes, batch, ctas, smem, ring;
    bool row;          // the kernel for wide rows
    bool apart;        // a thread's channels are `width` apart
};

// Bytes of a tensor's part of a slot: whole 16-byte pieces.
inline int64_t part_bytes(int64_t bytes, bool apart) { return apart ? (bytes + 30) / 16 * 16 : bytes; }

// Two slots an SM at least, of what its shared memory holds.  tensors: as large
// as x; gated: the gate too; aligned: all start on 16 bytes.
inline Staged staged_shape(int64_t N, int L, int C, int es, int tensors, bool gated, bool bwd, bool aligned) {
    Staged s{};
    const int room = 224 * 1024, wbytes = (2 * (L + 1) * C * 4 + 15) / 16 * 16;
    s.apart = !aligned || C * es % 16 != 0;
    s.batch = 1;
    // 16 bytes of neighbours a thread; 8 of 16-bit ones where more would not stay in registers (backward, L = 3:
    // 16384 nodes of 128 bf16 channels 146 us, 194 us with 16 bytes), and four single channels where they lie apart
    s.V = L == 0 || (!s.apart && (L <= 2 || !bwd)) ? 16 / es : 4;
    s.J = 1;
    const int vecs = (C + s.V - 1) / s.V;
    const auto slot = [&](int nodes) {
        const int64_t rows = (int64_t)(L + 1) * C * es * nodes;
        return part_bytes(rows * (L + 1), s.apart) * tensors + (gated ? part_bytes(rows, s.apart) : 0);
    };
    if (vecs <= 32) {
        s.width = 1;
        while (s.width < vecs) s.width *= 2;
        s.ctas = 1;
        s.ring = wbytes;
        // rows (L = 0) are small: so many a slot that the slots of all warps fill the shared memory, while there are
        // rows for all (131072 fp32 rows of 128: 79 us forward and 135 us backward, with one row a slot 120 and 182 us)
        const int most = bwd ? 8 : 16, each = 32 / s.width;
        const int64_t full = (room - wbytes) / most / slot(each), some = N / ((int64_t)148 * most * each);
        s.batch = (int)(full < some ? full : some);
        s.batch = L > 0 || s.batch < 1 ? 1 : s.batch > 16 ? 16 : s.batch;
        s.nodes = each * s.batch;
        const int64_t fit = (room - wbytes) / slot(s.nodes);
        s.slots = (int)(fit < kMaxSlots ? fit : kMaxSlots);
        if (s.slots < 2) return Staged{};
        // Every warp has slots of its own (the slots are a multiple of the warps): a slot's next copies are then
        // waited for by the warp that issued them, so no warp can meet a slot two phases behind, whose barrier would
        // show the parity of the phase it wants.
        // One slot a warp is best where that gives no more than 8 warps backward (222 registers a thread; lmax2: 8
        // slots of 8 warps 170 us, 10 of 5 warps 219 us) or 16 forward (108 us; 16 slots of 8 warps 109 us).
        const int warps = s.slots < most ? s.slots : most;
        s.slots = s.slots / warps * warps;
        s.threads = 32 * warps;
    } else if (L == 0) {
        // 8 channels a thread, 16 for the widest 16-bit rows; 512 threads an SM (128 registers each) backward and
        // for the widest, 1024 else
        s.row = true;
        s.J = s.V == 4 || vecs > 512 ? 2 : 1;
        if (vecs > 512 * s.J) return Staged{};
        s.width = s.threads = ((vecs + s.J - 1) / s.J + 31) / 32 * 32;
        s.nodes = 1;
        s.ctas = (bwd || s.J * s.V > 8 ? 512 : 1024) / s.threads;
        int64_t fit = (room / s.ctas - 1536) / slot(1);      // barriers and what the system keeps of each CTA
        while (fit < 2 && s.ctas > 1) fit = (room / --s.ctas - 1536) / slot(1);
        s.slots = (int)(fit < 4 ? fit : 4);
        if (s.slots < 2) return Staged{};
    } else {
        // one node a CTA; CTAs up to 256 threads an SM backward (up to 255 registers each) and 512 forward, with one
        // slot each where no more fit: one CTA's copies then run beside the others' work
        if (vecs > 256) return Staged{};
        s.width = s.threads = (vecs + 31) / 32 * 32;
        s.nodes = 1;
        s.ring = wbytes;
        const auto slots = [&] { return (room / s.ctas - 1536 - wbytes) / slot(1); };
        s.ctas = (bwd ? 256 : 512) / s.threads;
        while (slots() < 1 && s.ctas > 1) --s.ctas;
        if (slots() < 1 || slots() * s.ctas < 2) return Staged{};
        s.slots = (int)(slots() < 4 ? slots() : 4);
    }
    s.smem = s.ring + (int)slot(s.nodes) * s.slots;
    // where a warp has a node, the weight gradients are summed over the warps in the ring's place, which takes
    // threads * V floats: 8 KB, more than the ring of the narrowest rows
    if (bwd && s.width <= 32 && s.smem < s.ring + s.threads * s.V * 4) s.smem = s.ring + s.threads * s.V * 4;
    return s;
}

// Lets a kernel have the shared memory of an SM, once per device.
template <class K>
cudaError_t allow_smem(K kernel, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <class T, int V, int L, bool BWD, bool CTA, bool APART>
cudaError_t launch_staged(const StagedParams& s, const Staged& h, int grid, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(bn_staged_kernel<T, V, L, BWD, CTA, APART>, done);
    if (e != cudaSuccess) return e;
    bn_staged_kernel<T, V, L, BWD, CTA, APART><<<grid, h.threads, h.smem, st>>>(s);
    count_launch();
    return cudaGetLastError();
}

template <class T, int V, int J, bool BWD, bool APART>
cudaError_t launch_row(const StagedParams& s, const Staged& h, int grid, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(bn_row_kernel<T, V, J, BWD, APART>, done);
    if (e != cudaSuccess) return e;
    bn_row_kernel<T, V, J, BWD, APART><<<grid, h.threads, h.smem, st>>>(s);
    count_launch();
    return cudaGetLastError();
}

template <class T, bool BWD, bool APART>
cudaError_t staged_for(const StagedParams& s, const Staged& h, int grid, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T), V = APART ? 4 : W;
    const bool cta = h.width > 32;
    if (h.row) {
        if constexpr (W == 8)
            if (h.J == 1) return launch_row<T, W, 1, BWD, APART>(s, h, grid, st);
        return launch_row<T, W, 2, BWD, APART>(s, h, grid, st);
    }
    switch (s.p.L) {
        case 0:
            return launch_staged<T, W, 0, BWD, false, APART>(s, h, grid, st);
        case 1:
            return cta ? launch_staged<T, V, 1, BWD, true, APART>(s, h, grid, st)
                       : launch_staged<T, V, 1, BWD, false, APART>(s, h, grid, st);
        case 2:
            return cta ? launch_staged<T, V, 2, BWD, true, APART>(s, h, grid, st)
                       : launch_staged<T, V, 2, BWD, false, APART>(s, h, grid, st);
        default:
            return cta ? launch_staged<T, BWD ? 4 : V, 3, BWD, true, APART>(s, h, grid, st)
                       : launch_staged<T, BWD ? 4 : V, 3, BWD, false, APART>(s, h, grid, st);
    }
}

}  // namespace bn
}  // namespace eqc
