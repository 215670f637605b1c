// decode_combine.cu -- the split-KV combine kernel and its launch: it writes the decode
// output from the warp partials the decode grid(s) leave in the workspace.
#include <algorithm>

#include "decode_impl.cuh"

namespace kvq {
namespace decode {

// ---------------------------------------------------------------------------
// Combine: the warp partials of each (sequence, query head) row into its output.
// ---------------------------------------------------------------------------
// One source of partials: a decode grid's workspace region and how that grid listed
// each sequence's pages and laid out its partials.
struct CSource {
    const float* ws_ml;
    const float* ws_o;
    const int32_t* ws_pre;  // the pages prefix the grid publishes (used above kCombineLocalB)
    int32_t Hg, ns;         // head groups of the grid's units, query heads per unit
    int32_t C, W;           // the grid's CTAs, and warps per CTA (partials per CTA and segment)
    int32_t max_blocks, window, sinks, len_sub;  // as in KParams
};

struct CParams {
    CSource src[2];
    int32_t nsrc;  // 1, or 2 for the mixed-precision decode (INT4 history, FP16 recent tokens)
    const int32_t* seq_lens;
    float* out;
    float* out_host;  // device address of mapped pinned host memory that also receives out, or nullptr
    int32_t B, Hq, lg_p;
    // MODE 1: (max, 1 / sum) of each row, written by the combine (the second -1 where a part of the
    // row failed); the decode grid's scores [B][Hq][score_ld], the accumulated weights
    // [B][Hkv][weights_ld], the query heads per kv head, the chunks of positions a kv head is cut
    // into, and the bound the lengths are cut to
    float2* stat;
    const float* scores;
    float* weights;
    float decay;
    int32_t score_ld, weights_ld, r, chunks, len_max;
    // MODE 2 (Hq counts virtual heads, two per output row)
    const float* lambda;
    const float* norm_weight;
    float norm_eps, out_scale;
};

constexpr int kCombineMaxWarps = 16;
constexpr int kCombineLocalB = 256;   // up to this batch the row metadata is computed before the wait

// MODE 1: CTA size of the weights, and the scores a thread has in flight: 16, a position's R of
// them for each of 16 / R positions, R the query heads per kv head rounded up to 1, 2, 4 or 8;
// 8 positions at R = 1, where the old weights are as many loads again (8 x 32 heads of 8193
// positions, a call: 59.4 us with 16, 58.5 with 8; at R = 4 45.6 with 16, 46.4 with 8).  A
// chunk is what a CTA's threads cover.
constexpr int kAddThreads = 256;
__host__ __device__ constexpr int add_rows(int r) { return r <= 2 ? r : (r <= 4 ? 4 : 8); }
__host__ __device__ constexpr int add_per_thread(int r) { return r == 1 ? 8 : 16 / add_rows(r); }
__host__ __device__ constexpr int add_positions(int r) { return kAddThreads * add_per_thread(r); }

// Where a row's partials lie: n of them from `base` on, made by CTAs cf, cf + 1, .. of U units.
struct RowPartials {
    int n;
    long long base, cf, U;
};

// The attention weight of one chunk of positions, from wt on, of kv head wh of sequence b:
//     weights[b][wh][t] = decay * weights[b][wh][t] + sum over the kv head's r rows of 2^(z - M) / L,
// z the scores the decode grid stored, in row order (results do not depend on timing).  M and
// 1 / L of the rows come from the combine (stat), or with WITH_ROWS from the (max, sum) pairs of
// their partials, by one warp per row.  A kv head of which a part failed (a copy that did not
// arrive: scores that were not stored) keeps its weights as they were.  Bound by latency: a
// thread's scores, its old weights and the rows' statistics are all in flight together, and the
// scores, written just before, mostly still lie in the L2.  s_m, s_inv: r floats each.
template <int R, bool WITH_ROWS>
__device__ __forceinline__ void add_weights(const CParams& p, int b, int wh, int wt, const RowPartials& rp, float* s_m,
                                            float* s_inv) {
    constexpr int K = add_per_thread(R);
    const CSource& s = p.src[0];
    const int hq = wh * p.r;
    const int Lb = min(min(p.seq_lens[b], p.len_max),
                       static_cast<int>(min(static_cast<long long>(s.max_blocks) << p.lg_p, 0x7fffffffLL)));
    if (wt >= Lb) return;  // the whole CTA
    const int t0 = wt + static_cast<int>(threadIdx.x);
    float* w = p.weights + (static_cast<long long>(b) * (p.Hq / p.r) + wh) * p.weights_ld + t0;
    const float* zp = p.scores + (static_cast<long long>(b) * p.Hq + hq) * p.score_ld + t0;
    float z[K][R], old[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const bool in = t0 + k * kAddThreads < Lb;
#pragma unroll
        for (int i = 0; i < R; ++i)
            z[k][i] = in && i < p.r ? __ldcg(zp + static_cast<long long>(i) * p.score_ld + k * kAddThreads) : 0.f;
        old[k] = in && p.decay != 0.f ? w[k * kAddThreads] : 0.f;
    }
    if constexpr (WITH_ROWS) {
        const int g = threadIdx.x >> 5, lane = threadIdx.x & 31;  // 8 warps, r <= 8 rows
        if (g < p.r) {
            const bool dense = rp.U >= s.C;  // every CTA slice of the decode grid holds units
            const float* ml0 = s.ws_ml + (rp.base * s.ns + (hq + g) % s.ns) * 2;
            float M = -INFINITY, L = 0.f;
            bool failed = false;
            for (int j = lane; j < rp.n; j += 32) {
                const long long k = rp.cf + j / s.W;
                if (!dense && slice_start(k, rp.U, s.C) >= slice_start(k + 1, rp.U, s.C)) continue;
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(ml0 + static_cast<long long>(j) * s.ns * 2));
                const float mn = fmaxf(M, ml.x);
                failed |= ml.y < 0.f;
                if (mn == -INFINITY) continue;
                L = L * fast_exp2(M - mn) + ml.y * fast_exp2(ml.x - mn);
                M = mn;
            }
            float Mx = M;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, off));
            L = M == -INFINITY ? 0.f : L * fast_exp2(M - Mx);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
            failed = __any_sync(0xffffffffu, failed);
            if (lane == 0) {
                s_m[g] = Mx;
                s_inv[g] = failed ? -1.f : (L > 0.f ? 1.f / L : 0.f);
            }
        }
    } else if (static_cast<int>(threadIdx.x) < p.r) {
        const float2 st = __ldcg(p.stat + static_cast<long long>(b) * p.Hq + hq + threadIdx.x);
        s_m[threadIdx.x] = st.x;
        s_inv[threadIdx.x] = st.y;
    }
    __syncthreads();
    if (s_inv[0] < 0.f) return;  // (a warp takes all rows of a kv head or fails for all of them)
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < p.r) sum = fmaf(fast_exp2(z[k][i] - s_m[i]), s_inv[i], sum);
        if (t0 + k * kAddThreads < Lb) w[k * kAddThreads] = fmaf(p.decay, old[k], sum);
    }
}

// The weights as a third kernel, one CTA per kv head and chunk.  8 x 32 heads of 8193 positions
// (25 MB): 6.7 us on its own.  Tried and slower for the whole call on that shape (60 us): the
// same work in further CTAs of the combine's launch, which then either hold the combine's
// registers or hold the merge to theirs (65 to 78 us with 64 to 40 registers; see MODE 3 for
// where it pays), and run beside the combine with M and L from the partials (63 us).
template <int R>
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(CParams p) {
    __shared__ float s_m[8], s_inv[8];
    asm volatile("griddepcontrol.launch_dependents;");
    const unsigned head = blockIdx.x / p.chunks, heads = p.Hq / p.r;
    const int wt = static_cast<int>(blockIdx.x - head * p.chunks) * add_positions(R);
    const int b = static_cast<int>(head / heads), wh = static_cast<int>(head % heads);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    add_weights<R, false>(p, b, wh, wt, RowPartials{}, s_m, s_inv);
}

// One CTA per output row (b, hq).  In source s the row's partials sit at W * (cf + seg) + j
// for j < W * (cl - cf + 1), where CTAs cf..cl of that grid hold the units of segment
// seg = (b, hq / ns); when some CTA slices are empty (fewer units than CTAs) their partials
// do not exist.  Warp w of the CTA takes partials w, w + nw, ..., NB at a time, keeping
// a running maximum M and sum L and an unnormalised output (lane l: dimensions 4f .. 4f + 3
// for f = l, l + 32, ... below D / 4),
// over the sources in turn; the warps' results are then merged with weights 2^(M_w - max M).
// Sequences without positions have no partials and get zeros.  This is the split-KV
// combine of flash decoding: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// NSRC: sources of partials (p.nsrc), a template parameter so the one-source combine
// carries no code for a second.
// NB: partials a warp loads together, 8 or 4.  The 4-partial instance, held to 64
// registers (at head_dim 256 it may take more, which its rows need), serves the rows of
// many partials (16-warp CTAs): at up to 128 registers such a CTA would hold a whole SM's
// register file and keep the next call's decode CTAs off that SM until it leaves; at 64
// it holds half.  Rows of 4- and 8-warp CTAs (up to 64 partials) load 8 at a time, in
// one round.
// MODE 1 (attention with weights) also leaves each row's maximum and reciprocal sum for the
// weights' kernel.  MODE 3 (the same, small calls) has the weights' CTAs in its own launch,
// behind those of the rows: one launch less, which is what a call that leaves the device half
// empty spends its time on (8 heads of 513 positions: 12.5 us a call in a stream, 14 with the
// third launch; on the device 10.3 either way).
// MODE 2 (differential attention) has one CTA per query head: even warps merge its first map's
// row, odd warps the second's, then o = o1 - lambda o2, the optional RMS norm over the row,
// which warp 0 holds whole, and the output scale.
template <int D, int NSRC, int NB, int MODE = 0>
__global__ void __launch_bounds__(MODE == 3 ? kAddThreads : kCombineMaxWarps * 32,
                                  MODE == 3 ? 2 : (NB == 8 || D == 256 ? 1 : 2))
combine_kernel(CParams p) {
    static_assert(D == 64 || D == 128 || D == 256, "head_dim 64, 128 or 256");
    static_assert(NB == 8 || NB == 4, "8 partials a batch, or 4 for the 4-warp CTAs");
    constexpr int NV = (D / 4 + 31) / 32;                 // float4 of the row per lane
    constexpr int NA = NB == 4 ? 1 : (NV == 1 ? 4 : 2);  // independent sums per float4 (shorter fma chains)
    auto lane_has = [](int lane, int v) { return D / 4 >= 32 || lane + 32 * v < D / 4; };
    // the next decode call may start its set-up; it waits for this grid before it
    // touches the workspace
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float s_m[kCombineMaxWarps], s_l[kCombineMaxWarps];
    __shared__ float4 s_o[kCombineMaxWarps][D / 4];
    __shared__ int s_red[2][2][kCombineMaxWarps];
    __shared__ bool s_failed[kCombineMaxWarps];  // MODE 1: a partial that the warp took has failed
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int nw = blockDim.x >> 5;
    const int rows_b = MODE == 2 ? p.Hq / 2 : p.Hq;  // output rows per sequence
    int b = static_cast<int>(blockIdx.x / rows_b);
    int hrow = static_cast<int>(blockIdx.x - static_cast<long long>(b) * rows_b);
    const bool adds = MODE == 3 && b >= p.B;  // a CTA of the weights: kv head hrow / r, positions from wt on
    int wt = 0;
    if (adds) {
        const unsigned k = blockIdx.x - static_cast<unsigned>(p.B) * rows_b;
        const unsigned head = k / p.chunks, heads = p.Hq / p.r;
        wt = static_cast<int>(k - head * p.chunks) * add_positions(p.r);
        b = static_cast<int>(head / heads);
        hrow = static_cast<int>(head % heads) * p.r;
    }
    const int hq = MODE == 2 ? 2 * hrow : hrow;  // (both maps' virtual heads, and a kv head's rows, share a segment)
    // the warps that merge this warp's row: all of them, or in MODE 2 every other one
    const int map = MODE == 2 ? warp & 1 : 0, sub = MODE == 2 ? warp >> 1 : warp, nsub = MODE == 2 ? nw >> 1 : nw;

    // Pages of sequence i as source s listed them, and the row's range of partials.
    auto pages_of = [&](const CSource& s, int i) {
        int L = p.seq_lens[i] - s.len_sub;
        if constexpr (MODE == 1 || MODE == 3) L = min(L, p.len_max);
        return seq_span(L, p.lg_p, s.max_blocks, s.window, s.sinks).np;
    };
    auto row_range = [&](const CSource& s, int pb_, int np_, int tot_, long long& cf_, long long& base_,
                         long long& U_) {
        const int hg = hq / s.ns;
        U_ = static_cast<long long>(s.Hg) * tot_;
        const long long sf = static_cast<long long>(s.Hg) * pb_ + static_cast<long long>(hg) * np_;
        cf_ = slice_of(sf, U_, s.C);
        const long long cl = slice_of(sf + np_ - 1, U_, s.C);
        base_ = static_cast<long long>(s.W) * (cf_ + static_cast<long long>(b) * s.Hg + hg);
        return s.W * static_cast<int>(cl - cf_ + 1);
    };
    int n[2] = {0, 0};
    long long cf[2] = {0, 0}, base[2] = {0, 0}, U[2] = {1, 1};

    // The row's pages prefix: for small batches from seq_lens (a read-only input) while
    // the decode grids still run; else from the prefix each decode grid publishes.
    const bool local = p.B <= kCombineLocalB;
    if (local) {
#pragma unroll
        for (int si = 0; si < NSRC; ++si) {
            int before = 0, all = 0;
            for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
                const int n_i = pages_of(p.src[si], i);
                all += n_i;
                if (i < b) before += n_i;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                before += __shfl_xor_sync(0xffffffffu, before, off);
                all += __shfl_xor_sync(0xffffffffu, all, off);
            }
            if (lane == 0) {
                s_red[si][0][warp] = before;
                s_red[si][1][warp] = all;
            }
        }
        __syncthreads();
#pragma unroll
        for (int si = 0; si < NSRC; ++si) {
            int pb = 0, tot = 0;
            for (int w = 0; w < nw; ++w) {
                pb += s_red[si][0][w];
                tot += s_red[si][1][w];
            }
            const int np = pages_of(p.src[si], b);
            if (np > 0) n[si] = row_range(p.src[si], pb, np, tot, cf[si], base[si], U[si]);
        }
    }

    // the partials (and the published prefixes) are written by the decode grids ahead of this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!local) {
#pragma unroll
        for (int si = 0; si < NSRC; ++si) {
            const int32_t* pre = p.src[si].ws_pre;
            const int pb = __ldcg(pre + b);
            const int np = __ldcg(pre + b + 1) - pb;
            const int tot = __ldcg(pre + p.B);
            if (np > 0) n[si] = row_range(p.src[si], pb, np, tot, cf[si], base[si], U[si]);
        }
    }

    if constexpr (MODE == 3) {
        if (adds) {
            const int wh = hrow / p.r;
            const RowPartials rp{n[0], base[0], cf[0], U[0]};
            switch (add_rows(p.r)) {
                case 1: add_weights<1, true>(p, b, wh, wt, rp, s_m, s_l); break;
                case 2: add_weights<2, true>(p, b, wh, wt, rp, s_m, s_l); break;
                case 4: add_weights<4, true>(p, b, wh, wt, rp, s_m, s_l); break;
                default: add_weights<8, true>(p, b, wh, wt, rp, s_m, s_l); break;
            }
            return;  // the whole CTA
        }
    }

    float M = -INFINITY, L = 0.f;
    bool failed = false;
    float4 acc[NV][NA];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[v][a] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int si = 0; si < NSRC; ++si) {
        const CSource& s = p.src[si];
        const int sl = hq - (hq / s.ns) * s.ns + map;
        const bool dense = U[si] >= s.C;  // every CTA slice holds units
        const long long stride_ml = static_cast<long long>(s.ns) * 2;
        const long long stride_o = static_cast<long long>(s.ns) * D;
        const float* ml0 = s.ws_ml + (base[si] * s.ns + sl) * 2;
        const float* o0 = s.ws_o + (base[si] * s.ns + sl) * D + 4 * lane;
        for (int j0 = sub; j0 < n[si]; j0 += NB * nsub) {
            float2 ml[NB];
            float4 ov[NB][NV];
#pragma unroll
            for (int kk = 0; kk < NB; ++kk) {
                const int j = j0 + kk * nsub;
                bool have = j < n[si];
                if (have && !dense) {
                    const long long k = cf[si] + j / s.W;
                    have = slice_start(k, U[si], s.C) < slice_start(k + 1, U[si], s.C);
                }
                ml[kk] = have ? __ldcg(reinterpret_cast<const float2*>(ml0 + j * stride_ml)) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    ov[kk][v] = have && lane_has(lane, v) ? __ldcg(reinterpret_cast<const float4*>(o0 + j * stride_o) + 32 * v)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mb = M;
#pragma unroll
            for (int kk = 0; kk < NB; ++kk) {
                mb = fmaxf(mb, ml[kk].x);
                if constexpr (MODE == 1) failed |= ml[kk].y < 0.f;
            }
            if (mb == -INFINITY) continue;  // only empty partials so far
            if (mb > M) {  // a larger running maximum: rescale what has been summed
                const float f = fast_exp2(M - mb);
                L *= f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int a = 0; a < NA; ++a) {
                        acc[v][a].x *= f;
                        acc[v][a].y *= f;
                        acc[v][a].z *= f;
                        acc[v][a].w *= f;
                    }
                M = mb;
            }
#pragma unroll
            for (int kk = 0; kk < NB; ++kk) {
                const float f = fast_exp2(ml[kk].x - M);
                L = fmaf(f, ml[kk].y, L);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float4& A = acc[v][kk % NA];
                    A.x = fmaf(f, ov[kk][v].x, A.x);
                    A.y = fmaf(f, ov[kk][v].y, A.y);
                    A.z = fmaf(f, ov[kk][v].z, A.z);
                    A.w = fmaf(f, ov[kk][v].w, A.w);
                }
            }
        }
    }
    if (lane == 0) {
        s_m[warp] = M;
        s_l[warp] = L;
        if constexpr (MODE == 1) s_failed[warp] = failed;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float4 t = acc[v][0];
#pragma unroll
        for (int a = 1; a < NA; ++a) {
            t.x += acc[v][a].x;
            t.y += acc[v][a].y;
            t.z += acc[v][a].z;
            t.w += acc[v][a].w;
        }
        if (lane_has(lane, v)) s_o[warp][lane + 32 * v] = t;
    }
    __syncthreads();
    // the row of map `m` (lane l: float4 l, l + 32, ..)
    auto merge = [&](int m, float4 (&res)[NV], float& Mx, float& inv) {
        constexpr int step = MODE == 2 ? 2 : 1;
        Mx = -INFINITY;
        for (int w = m; w < nw; w += step) Mx = fmaxf(Mx, s_m[w]);
        float Ls = 0.f;
        if (Mx != -INFINITY)
            for (int w = m; w < nw; w += step) Ls = fmaf(fast_exp2(s_m[w] - Mx), s_l[w], Ls);
        inv = Ls > 0.f ? 1.f / Ls : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            res[v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!lane_has(lane, v) || Mx == -INFINITY) continue;
            for (int w = m; w < nw; w += step) {
                const float f = fast_exp2(s_m[w] - Mx);
                const float4 ow = s_o[w][lane + 32 * v];
                res[v].x = fmaf(f, ow.x, res[v].x);
                res[v].y = fmaf(f, ow.y, res[v].y);
                res[v].z = fmaf(f, ow.z, res[v].z);
                res[v].w = fmaf(f, ow.w, res[v].w);
            }
            res[v] = make_float4(res[v].x * inv, res[v].y * inv, res[v].z * inv, res[v].w * inv);
        }
    };
    float4 res[NV];
    float Mx, inv;
    if constexpr (MODE == 2) {
        __shared__ float4 s_second[D / 4];
        if (warp < 2) merge(warp, res, Mx, inv);
        if (warp == 1) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (lane_has(lane, v)) s_second[lane + 32 * v] = res[v];
        }
        __syncthreads();
        if (warp != 0) return;
        const float lam = p.lambda[hrow];
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!lane_has(lane, v)) continue;
            const float4 o2 = s_second[lane + 32 * v];
            res[v] = make_float4(fmaf(-lam, o2.x, res[v].x), fmaf(-lam, o2.y, res[v].y), fmaf(-lam, o2.z, res[v].z),
                                 fmaf(-lam, o2.w, res[v].w));
            ss += res[v].x * res[v].x + res[v].y * res[v].y + res[v].z * res[v].z + res[v].w * res[v].w;
        }
        float f = p.out_scale;
        if (p.norm_weight != nullptr) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            f *= rsqrtf(ss * (1.f / D) + p.norm_eps);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!lane_has(lane, v)) continue;
            float4 w = make_float4(f, f, f, f);
            if (p.norm_weight != nullptr) {
                w = reinterpret_cast<const float4*>(p.norm_weight)[lane + 32 * v];
                w = make_float4(w.x * f, w.y * f, w.z * f, w.w * f);
            }
            // no positions: zeros, whatever norm_eps is
            res[v] = n[0] > 0 ? make_float4(res[v].x * w.x, res[v].y * w.y, res[v].z * w.z, res[v].w * w.w)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    } else {
        if (warp != 0) return;
        merge(0, res, Mx, inv);
    }
    const long long row = static_cast<long long>(b) * rows_b + hrow;
    if constexpr (MODE == 1) {
        failed = __any_sync(0xffffffffu, lane < nw && s_failed[lane]);
        if (lane == 0) p.stat[row] = make_float2(Mx, failed ? -1.f : inv);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (!lane_has(lane, v)) continue;
        reinterpret_cast<float4*>(p.out + row * D)[lane + 32 * v] = res[v];
        if (p.out_host != nullptr) reinterpret_cast<float4*>(p.out_host + row * D)[lane + 32 * v] = res[v];
    }
}

}  // namespace decode

namespace {

// The partials one decode grid (arguments a, plan) leaves in its workspace.
decode::CSource source_of(const DecodeArgs& a, const DecodePlan& plan) {
    decode::CSource s;
    s.ws_ml = reinterpret_cast<const float*>(a.workspace + plan.ws_ml_offset);
    s.ws_o = reinterpret_cast<const float*>(a.workspace + plan.ws_o_offset);
    s.ws_pre = reinterpret_cast<const int32_t*>(a.workspace + plan.ws_pre_offset);
    s.Hg = a.Hkv / plan.hk;
    s.ns = plan.hk * (a.Hq / a.Hkv);
    s.C = plan.ctas;
    s.W = 4;
    s.max_blocks = a.max_blocks;
    s.window = a.window;
    s.sinks = a.sinks;
    s.len_sub = a.len_sub;
    return s;
}

template <int MODE>
cudaError_t launch_one(const cudaLaunchConfig_t& cfg, const decode::CParams& p, int d, bool light) {
    constexpr int NB = MODE == 3 ? 4 : 8;  // (MODE 3: always the light one)
    switch (d) {
        case 64: return light ? cudaLaunchKernelEx(&cfg, decode::combine_kernel<64, 1, 4, MODE>, p)
                              : cudaLaunchKernelEx(&cfg, decode::combine_kernel<64, 1, NB, MODE>, p);
        case 128: return light ? cudaLaunchKernelEx(&cfg, decode::combine_kernel<128, 1, 4, MODE>, p)
                               : cudaLaunchKernelEx(&cfg, decode::combine_kernel<128, 1, NB, MODE>, p);
        case 256: return light ? cudaLaunchKernelEx(&cfg, decode::combine_kernel<256, 1, 4, MODE>, p)
                               : cudaLaunchKernelEx(&cfg, decode::combine_kernel<256, 1, NB, MODE>, p);
        default: return cudaErrorInvalidValue;
    }
}

// with_weights: the weights' CTAs in the same launch (MODE 3)
cudaError_t launch(const decode::CParams& p, DecodeMode mode, int d, int warps, cudaStream_t stream,
                   bool with_weights = false) {
    long long rows = static_cast<long long>(p.B) * (mode == DecodeMode::kDiff ? p.Hq / 2 : p.Hq);
    if (with_weights) {
        rows += static_cast<long long>(p.B) * (p.Hq / p.r) * p.chunks;
        warps = decode::kAddThreads / 32;
    } else if (mode == DecodeMode::kDiff) {
        warps = std::min(2 * warps, decode::kCombineMaxWarps);  // two rows
    }
    if (rows <= 0) return cudaSuccess;
    if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    // Launched while the decode grid runs (programmatic dependent launch); the kernel
    // waits with griddepcontrol.wait before it reads the workspace.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    cfg.blockDim = dim3(static_cast<unsigned>(warps) * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err;
    // The 64-register instance; in the weights and differential modes also where the rows' CTAs
    // of the other one (16 warps on each of 152 SMs) would not all be resident at once
    // (attention with weights, 32 x 8 kv heads of up to 4096 positions, 1024 rows: 39.3 -> 36.7 us), and at head_dim 256
    // (differential, 8 x 16 heads of 4097 positions: 40.3 -> 39.1 us; never slower).
    const bool light = warps == 16 || (mode != DecodeMode::kPlain && (rows * warps > 152 * 16 || d == 256));
    if (p.nsrc == 2) err = cudaLaunchKernelEx(&cfg, decode::combine_kernel<128, 2, 8>, p);  // mixed: head_dim 128 only
    else if (with_weights) err = launch_one<3>(cfg, p, d, true);
    else if (mode == DecodeMode::kWeights) err = launch_one<1>(cfg, p, d, light);
    else if (mode == DecodeMode::kDiff) err = launch_one<2>(cfg, p, d, light);
    else err = launch_one<0>(cfg, p, d, light);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

int lg2(int P) {
    int l = 0;
    while ((1 << l) < P) ++l;
    return l;
}

}  // namespace

cudaError_t launch_combine(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
    decode::CParams p{};
    p.src[0] = source_of(a, plan);
    p.nsrc = 1;
    p.seq_lens = a.seq_lens;
    p.out = a.out;
    p.out_host = a.out_host;
    p.B = a.B;
    p.Hq = a.Hq;
    p.lg_p = lg2(a.L.P);
    p.stat = reinterpret_cast<float2*>(a.workspace + plan.ws_stat_offset);
    p.scores = reinterpret_cast<const float*>(a.workspace + plan.ws_score_offset);
    p.weights = a.weights;
    p.decay = a.decay;
    p.score_ld = plan.score_ld;
    p.weights_ld = a.weights_ld;
    p.r = a.Hq / a.Hkv;
    p.chunks = static_cast<int32_t>((static_cast<long long>(a.max_len) + decode::add_positions(p.r) - 1) /
                                    decode::add_positions(p.r));
    p.len_max = a.max_len;
    p.lambda = a.lambda;
    p.norm_weight = a.norm_weight;
    p.norm_eps = a.norm_eps;
    p.out_scale = a.out_scale;
    const long long adders = static_cast<long long>(a.B) * a.Hkv * p.chunks;
    const bool weights = a.mode == DecodeMode::kWeights && adders > 0;
    // everything behind the decode grid in one launch where it is no more CTAs than the device's 152 SMs
    const bool one = weights && static_cast<long long>(a.B) * a.Hq + adders <= 152;
    cudaError_t err = launch(p, a.mode, a.L.d, plan.combine_warps, stream, one);
    if (err != cudaSuccess || !weights || one) return err;
    // launched while the combine runs; the kernel waits for it before it reads the workspace
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(adders));
    cfg.blockDim = dim3(decode::kAddThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (decode::add_rows(p.r)) {
        case 1: err = cudaLaunchKernelEx(&cfg, decode::add_weights_kernel<1>, p); break;
        case 2: err = cudaLaunchKernelEx(&cfg, decode::add_weights_kernel<2>, p); break;
        case 4: err = cudaLaunchKernelEx(&cfg, decode::add_weights_kernel<4>, p); break;
        default: err = cudaLaunchKernelEx(&cfg, decode::add_weights_kernel<8>, p); break;
    }
    return err != cudaSuccess ? err : cudaGetLastError();
}

// The mixed-precision decode: the partials of the INT4 grid (a0, plan0) and of the FP16
// grid (a1, plan1) merged per row.
cudaError_t launch_combine2(const DecodeArgs& a0, const DecodePlan& plan0, const DecodeArgs& a1,
                            const DecodePlan& plan1, cudaStream_t stream) {
    decode::CParams p{};
    p.src[0] = source_of(a0, plan0);
    p.src[1] = source_of(a1, plan1);
    p.nsrc = 2;
    p.seq_lens = a0.seq_lens;
    p.out = a0.out;
    p.B = a0.B;
    p.Hq = a0.Hq;
    p.lg_p = lg2(a0.L.P);
    const int warps = std::max(plan0.combine_warps, plan1.combine_warps);
    return launch(p, DecodeMode::kPlain, a0.L.d, warps, stream);
}

}  // namespace kvq
