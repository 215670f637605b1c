// chunk_few.cu -- chunk attention where a sequence has few lines (rows times the query heads of a kv head):
// drafted tokens, single tokens, short parts.
//
// The kernel of chunk_attention.cu puts lines along M, 128 at a time; with 8 or 32 of them most of its
// softmax and products are of rows nobody asked for.  Here both products are transposed, as in
// latent_attention.cu: S^T [128 positions, NC lines] = K Q^T and O^T [dimensions, NC lines] += V^T P^T, so
// that lines are columns, 16 or 32 of them, and an MMA of 128 x 16 x 16 takes 40 cycles instead of 64.
// What is left is the way of the keys and values: copied, dequantized, multiplied, tile after tile, with
// the products of two tiles in flight.
//
// Measured on four sequences over 32761 positions, 32 heads on 8 kv heads of 128 (in brackets the kernel of
// chunk_attention.cu): one row each 69 us (111), 8 rows 76 (112); 80 where four channels of the keys are 20 times
// larger and references move.  The pages are 140 MB, 20.8 us at the copy
// rate: a tile of 128 positions takes 2500 cycles of an SM where its copy would take 700.  It is bounded by
// the work on a tile (two thirds of the issue slots; unpack and multiply at half rate, 64 KB of stores into shared
// memory, the softmax's barriers) and by shared memory, which leaves room for three packed tiles in flight:
// with two it took 90.  Keys and values by the same eight warps took 94.
//
// Warps of a CTA (one per SM): 0-7 softmax, 8-15 dequantize the keys (and bring the queries), 16-23 the
// values, 24 the products, 25 the packed pages.
#include <cmath>

#include "chunk_shared.cuh"
#include "kvq_columns.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 896;
constexpr int kSmWarps = 8, kMmaWarp = 24, kPageWarp = 25;
constexpr int kRing = 2;  // operand tiles of keys, and as many of values
constexpr uint32_t kTmem = 256;  // columns: outputs from 0, two score tiles from 64

template <int D, int NC>
struct Shape {
    static constexpr int kOperand = kTile * D * 2;
    static constexpr int kQChunk = NC * 128;                     // [NC][64] f16
    static constexpr int kQ = (D / 64) * kQChunk;
    // operand tiles, weights of two tiles ([128][NC] f16 in rows of 128 bytes), queries, packed tiles
    static constexpr int kP = 2 * kRing * kOperand, kQAt = kP + 2 * kChunk, kPackedAt = kQAt + kQ;
};

template <int NC>
struct Ctl {
    TileBars tiles;
    // scores and weights by buffer; the output with tile i in o_done[i % 2], so that whoever waits for it has seen
    // the phase before (scores of tile i complete: the output with tile i - 2, too)
    uint64_t q_full, q_free, s_full[2], p_full[2], o_done[2], last;
    long long warp_sum[kThreads / 32];
    Start start;
    uint32_t tmem;
    int stop;
    Walk walk[kPageWarp + 1];
    alignas(16) float ref[NC];    // the reference maximum, or 0 where nothing is seen yet
    alignas(16) float scale[NC];  // factors of a rescaling, or of the output
    float m[NC];                  // reference maximum of the scores (of z / scale)
    int lim[NC];                  // positions a line sees
    float part[4][NC];            // by warp
};

template <int D, int NC>
__global__ void __launch_bounds__(kThreads, 1) chunk_few_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ uint8_t smem_raw[];
    using Z = Shape<D, NC>;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t ring_s = smem_u32(smem), p_s = ring_s + Z::kP, q_s = ring_s + Z::kQAt;
    const int packed_bytes = (kTile >> p.lg_p) * p.L.bytes;
    Ctl<NC>* ctl = reinterpret_cast<Ctl<NC>*>(smem + Z::kPackedAt + kPacked * packed_bytes);
    volatile int* stop = &ctl->stop;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPacked; ++i) {
            mbar_init(smem_u32(&ctl->tiles.pk_full[i]), 1);
            mbar_init(smem_u32(&ctl->tiles.pk_empty[i]), 2 * kDqWarps);
        }
        for (int i = 0; i < 2 * kRing; ++i) {
            mbar_init(smem_u32(&ctl->tiles.kv_full[i]), kDqWarps + (i == kRing ? p.withheld : 0));
            mbar_init(smem_u32(&ctl->tiles.kv_empty[i]), 1);
        }
        mbar_init(smem_u32(&ctl->q_full), kDqWarps);
        mbar_init(smem_u32(&ctl->q_free), 1);
        mbar_init(smem_u32(&ctl->last), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->s_full[i]), 1);
            mbar_init(smem_u32(&ctl->p_full[i]), kSmWarps);
            mbar_init(smem_u32(&ctl->o_done[i]), 1);
        }
        ctl->stop = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&ctl->tmem), kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    find_start<kThreads>(p, &ctl->start, ctl->warp_sum);  // (has barriers of the CTA)
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Start st = ctl->start;
    Walk& walk = ctl->walk[min(warp, kPageWarp)];
    if (st.units > 0 && warp <= kPageWarp) walk.begin(p, st);
    const Segment& g = walk.g;

    if (warp < kSmWarps) {
        regs_more<96>();
        // ---- softmax: position `t` of a tile, columns c0 .. c0 + HC - 1; the thread's tensor-memory lane is also a
        // dimension of the output
        constexpr int HC = NC / 2;
        const int t = threadIdx.x & 127, side = warp / 4, c0 = side * HC;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t s_t = tmem + lanes + 64 + c0, o_t = tmem + lanes;
        uint32_t n_b0 = 0, n_b1 = 0;  // tiles of earlier segments, by buffer
        auto phase = [&](int i) { return ((i & 1 ? n_b1 : n_b0) + (i >> 1)) & 1; };
        while (st.units > 0 && walk.next(p)) {
            const int n = g.k1 - g.k0;
            if (side == 0 && t < NC) {
                ctl->lim[t] = g.ahead + (g.line0 + min(t, g.lines - 1)) / p.per_row + 1;
                ctl->m[t] = -INFINITY;
                ctl->ref[t] = 0.f;
            }
            softmax_barrier();
            const int lim0 = ctl->lim[0];  // the least
            float l[HC];
#pragma unroll
            for (int i = 0; i < HC; ++i) l[i] = 0.f;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int pos = (g.k0 + i) * kTile + t, buf = i & 1;
                wait_or_stop(smem_u32(&ctl->s_full[buf]), phase(i), stop, p);
                tc_fence_after();
                uint32_t s[HC];
                auto fetch = [&]() {
                    load_columns<HC>(s_t + 64 * buf, s);
                    if ((g.k0 + i + 1) * kTile > lim0) {
#pragma unroll
                        for (int x = 0; x < HC; ++x)
                            if (pos >= ctl->lim[c0 + x]) s[x] = 0xff800000u;
                    }
                };
                // The scores less their references.  (The difference before the product: exact at the maximum, however
                // large the scores are; a fused s c - m c would leave the rounding of m c)
                auto less = [&]() -> float {
                    float top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < HC; x += 4) {
                        const float4 r = *reinterpret_cast<const float4*>(&ctl->ref[c0 + x]);
                        const float a = __uint_as_float(s[x]) - r.x, b = __uint_as_float(s[x + 1]) - r.y;
                        const float c = __uint_as_float(s[x + 2]) - r.z, d = __uint_as_float(s[x + 3]) - r.w;
                        top = fmaxf(fmaxf(fmaxf(top, a), fmaxf(b, c)), d);
                        s[x] = __float_as_uint(a);
                        s[x + 1] = __float_as_uint(b);
                        s[x + 2] = __float_as_uint(c);
                        s[x + 3] = __float_as_uint(d);
                    }
                    return top;
                };
                fetch();
                // are the references still within 2^kLag of every score? (see latent_attention.cu)
                if (any_of_softmax(less() * p.c > kLag || i == 0)) {
                    fetch();
#pragma unroll
                    for (int x = 0; x < HC; ++x) {
                        const float r = warp_max(__uint_as_float(s[x]));
                        if (lane == x) ctl->part[warp & 3][c0 + x] = r;
                    }
                    softmax_barrier();
                    if (side == 0 && t < NC) {
                        const float most = fmaxf(fmaxf(ctl->part[0][t], ctl->part[1][t]), fmaxf(ctl->part[2][t], ctl->part[3][t]));
                        const float m = ctl->m[t];
                        const float to = m == -INFINITY || (most - m) * p.c > kLag ? fmaxf(most, m) : m;
                        ctl->scale[t] = to == m ? 1.f : fast_exp2((m - to) * p.c);
                        ctl->m[t] = to;
                        ctl->ref[t] = to == -INFINITY ? 0.f : to;
                    }
                    softmax_barrier();
                    less();
                    if (i > 0) {
                        wait_or_stop(smem_u32(&ctl->o_done[buf ^ 1]), phase(i - 1), stop, p);  // the output so far
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < HC; ++x) l[x] *= ctl->scale[c0 + x];
#pragma unroll 1
                        for (int x = side; x < NC / 16; x += 2) {
                            uint32_t o[16];
                            tmem_ld16(o_t + 16 * x, o);
                            tmem_wait_ld();
                            tmem_touch(o);
                            const float* f = &ctl->scale[16 * x];
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f[y]);
                            tmem_st16(o_t + 16 * x, o);
                        }
                        tmem_wait_st();
                    }
                }
                // the weights, in rows of a position
#pragma unroll
                for (int x = 0; x < HC; x += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 8; y += 4) {
                        const float a = fast_exp2(fmaf(__uint_as_float(s[x + y]), p.c, kUp));
                        const float b = fast_exp2(fmaf(__uint_as_float(s[x + y + 1]), p.c, kUp));
                        const float c = fast_exp2(fmaf(__uint_as_float(s[x + y + 2]), p.c, kUp));
                        const float d = fast_exp2(fmaf(__uint_as_float(s[x + y + 3]), p.c, kUp));
                        l[x + y] += a;
                        l[x + y + 1] += b;
                        l[x + y + 2] += c;
                        l[x + y + 3] += d;
                        w[y / 2] = pack_h2(a, b);
                        w[y / 2 + 1] = pack_h2(c, d);
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p_s + buf * kChunk + swizzled(t, (c0 + x) / 8)),
                                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[buf]));
            }
            // ---- the segment's result
            const bool whole = g.k0 == 0 && g.k1 == g.nt;
            warp_sums<HC>(l, lane);
            ctl->part[warp & 3][c0 + first_column<HC>(lane)] = l[0];
            softmax_barrier();
            const int slot = partial_slot(g);
            if (side == 0 && t < NC) {
                const float sum = (ctl->part[0][t] + ctl->part[1][t]) + (ctl->part[2][t] + ctl->part[3][t]);
                ctl->scale[t] = !whole ? 1.f : sum > 0.f ? 2.f / sum : 0.f;
                if (!whole) {
                    p.part_ml[(static_cast<long long>(slot) * NC + t) * 2] = ctl->m[t];
                    p.part_ml[(static_cast<long long>(slot) * NC + t) * 2 + 1] = sum;
                }
            }
            softmax_barrier();
            wait_or_stop(smem_u32(&ctl->o_done[(n - 1) & 1]), phase(n - 1), stop, p);
            tc_fence_after();
            n_b0 += (n + 1) / 2;
            n_b1 += n / 2;
            const int dim = dim_of(t);
#pragma unroll 1
            for (int x = side; x < NC / 16; x += 2) {
                uint32_t o[16];
                tmem_ld16(o_t + 16 * x, o);
                tmem_wait_ld();
                tmem_touch(o);
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const int c = 16 * x + y;
                    if (c < g.lines && t < D) {
                        if (whole) {
                            const int line = g.line0 + c, tok = line / p.r;
                            p.out[((static_cast<long long>(g.row0) + tok) * p.Hq + g.h * p.r + line - tok * p.r) * D + dim] =
                                __float2half_rn(__uint_as_float(o[y]) * ctl->scale[c]);
                        } else {
                            p.part_o[(static_cast<long long>(slot) * NC + c) * D + dim] = __uint_as_float(o[y]);
                        }
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            softmax_barrier();
        }
    } else if (warp < kSmWarps + 2 * kDqWarps) {
        regs_less<64>();
        // ---- dequantize: eight warps the keys (and the queries), eight the values
        const int is_v = warp >= kSmWarps + kDqWarps, dw = (warp - kSmWarps) % kDqWarps, tid = threadIdx.x - 32 * kSmWarps;
        uint32_t n_pk = 0, n_q = 0;
        while (st.units > 0 && walk.next(p)) {
            const int n = g.k1 - g.k0, end0 = g.vis - g.k0 * kTile;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++n_pk) {
                dequantize_tile<D, true>(p, ctl->tiles, smem + Z::kPackedAt, packed_bytes, ring_s, n_pk, end0 - i * kTile, is_v, dw,
                                         kRing * is_v + n_pk % kRing, n_pk / kRing, stop);
                if (i > 0 || is_v) continue;
                // the item's queries, their dimensions in the order the unpack leaves
                if (n_q > 0) wait_or_stop(smem_u32(&ctl->q_free), (n_q - 1) & 1, stop, p);
                ++n_q;
#pragma unroll 4
                for (int j = tid; j < NC * (D / 8); j += 32 * kDqWarps) {
                    const int c = j / (D / 8), piece = j % (D / 8);
                    const int line = g.line0 + c, tok = line / p.r;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (c < g.lines)
                        x = __ldg(reinterpret_cast<const uint4*>(
                                      p.q + ((static_cast<long long>(g.row0) + tok) * p.Hq + g.h * p.r + line - tok * p.r) * D) +
                                  piece);
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(q_s + (piece / 8) * Z::kQChunk + swizzled(c, piece % 8)),
                                 "r"(prmt(x.x, x.z, 0x5410) ^ p.q_flip), "r"(prmt(x.x, x.z, 0x7632) ^ p.q_flip),
                                 "r"(prmt(x.y, x.w, 0x5410) ^ p.q_flip), "r"(prmt(x.y, x.w, 0x7632) ^ p.q_flip)
                                 : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full));
            }
        }
    } else {
        regs_less<56>();
        if (warp == kMmaWarp) {
            // ---- the products
            constexpr uint32_t kIdS = mma_idesc(kTile, NC, false, false), kIdO = mma_idesc(128, NC, true, true);
            const uint32_t tm = uniform(tmem);
            bool live = true;  // false once a wait has been given up: nothing more is issued
            uint32_t n_k = 0, n_v = 0, n_seg = 0, n_b0 = 0, n_b1 = 0;
            auto take = [&](uint32_t& n, uint32_t first) -> uint32_t {  // the next operand tile of keys or values
                const uint32_t stage = first + n % kRing;
                live &= wait_or_stop(smem_u32(&ctl->tiles.kv_full[stage]), (n / kRing) & 1, stop, p);
                ++n;
                return stage;
            };
            while (uniform(st.units > 0 && walk.next(p))) {
                const int n = uniform(g.k1 - g.k0);
                live &= wait_or_stop(smem_u32(&ctl->q_full), n_seg & 1, stop, p);
                ++n_seg;
                // turn i: the output with value tile i, then the scores with key tile i + 2 (it starts with scores alone)
#pragma unroll 1
                for (int i = -2; i < n; ++i) {
                    const int buf = i & 1;
                    if (i >= 0) {
                        const uint32_t v = take(n_v, kRing);
                        live &= wait_or_stop(smem_u32(&ctl->p_full[buf]), ((buf ? n_b1 : n_b0) + (i >> 1)) & 1, stop, p);
                        tc_fence_after();
                        // (64 dimensions: the second half of M is the next operand tile's bytes, whatever they are; the
                        // rows of the output it gives are not read)
                        const uint32_t a = desc_lo(ring_s + v * Z::kOperand, kChunk), b = desc_lo(p_s + buf * kChunk, kChunk);
                        if (elect_one() && live) {
#pragma unroll
                            for (int x = 0; x < kTile / 16; ++x)
                                mma_ss(tm, smem_desc(a + (x * 2048 >> 4)), smem_desc(b + (x * 2048 >> 4)), kIdO, i > 0 || x > 0);
                            mma_commit(smem_u32(&ctl->tiles.kv_empty[v]));
                            mma_commit(smem_u32(&ctl->o_done[buf]));
                        }
                        __syncwarp();
                    }
                    if (i + 2 < n) {
                        const uint32_t k = take(n_k, 0);
                        tc_fence_after();
                        const uint32_t a = desc_lo(ring_s + k * Z::kOperand, 16), b = desc_lo(q_s, 16);
                        if (elect_one() && live) {
#pragma unroll
                            for (int x = 0; x < D / 16; ++x)
                                mma_ss(tm + 64 + 64 * buf, smem_desc(a + (((x / 4) * kChunk + (x % 4) * 32) >> 4)),
                                       smem_desc(b + (((x / 4) * Z::kQChunk + (x % 4) * 32) >> 4)), kIdS, x > 0);
                            mma_commit(smem_u32(&ctl->s_full[buf]));
                            mma_commit(smem_u32(&ctl->tiles.kv_empty[k]));
                            if (i + 3 == n) mma_commit(smem_u32(&ctl->q_free));
                        }
                        __syncwarp();
                    }
                }
                n_b0 += (n + 1) / 2;
                n_b1 += n / 2;
            }
        } else if (warp == kPageWarp) {
            load_pages(p, ctl->tiles, walk, ring_s + Z::kPackedAt, packed_bytes, st.units > 0, stop);
        }
    }
    tc_fence_before();
    __syncthreads();
    finish_products(warp == kMmaWarp, smem_u32(&ctl->last), stop);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, kTmem);
    }
}

// The items cut between CTAs.
template <int D, int NC>
__global__ void __launch_bounds__(256) chunk_few_merge_kernel(const __grid_constant__ ChunkParams p, int ctas) {
    __shared__ MergeShare share;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // lanes hold 4 dimensions of a line each (D = 64: half of the lanes)
    merge_items<1>(
        p, p.c, ctas, 1, &share,
        [&](long long slot, int line, int, float& m, float& l, float4& o, int lane) {
            const long long at = slot * NC + line;
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            m = ml.x;
            l = ml.y;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * lane < D) o = reinterpret_cast<const float4*>(p.part_o + at * D)[lane];
        },
        [&](const MergeDesc& d, int line, int, float l, const float4& o, int lane) {
            if (4 * lane >= D) return;
            const float inv = l > 0.f ? 2.f / l : 0.f;
            const long long at = static_cast<long long>(d.line0) + line, row = at / p.r;
            reinterpret_cast<uint2*>(p.out + (row * p.Hq + d.h * p.r + (at - row * p.r)) * D)[lane] =
                make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
        });
}

template <int D, int NC>
cudaError_t launch(ChunkParams p, int ctas, cudaStream_t stream) {
    p.per_row = p.r;
    p.step = NC;
    static_assert(1024 + Shape<D, NC>::kPackedAt + kPacked * kTile * (D + D / 8) + sizeof(Ctl<NC>) <= 232448, "");  // groups of 32
    const size_t smem = 1024 + Shape<D, NC>::kPackedAt + static_cast<size_t>(kPacked) * (kTile >> p.lg_p) * p.L.bytes + sizeof(Ctl<NC>);
    cudaError_t e = cudaFuncSetAttribute(chunk_few_kernel<D, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, chunk_few_kernel<D, NC>, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(4 * ctas));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, chunk_few_merge_kernel<D, NC>, p, ctas);
}

}  // namespace

cudaError_t launch_chunk_few(ChunkParams p, int head_dim, int lines, int ctas, cudaStream_t stream) {
    if (head_dim == 64)
        return lines <= 16 ? launch<64, 16>(p, ctas, stream) : launch<64, 32>(p, ctas, stream);
    return lines <= 16 ? launch<128, 16>(p, ctas, stream) : launch<128, 32>(p, ctas, stream);
}

}  // namespace kvq
