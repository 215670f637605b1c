// latent_attention.cu -- attention whose keys and values are one shared latent vector per token
// (absorbed form), over the packed latent cache, on the tcgen05 tensor cores.
//
// For a line (a row's query head) at position p:  z_t = scale (q_l . c_t + q_r . k_t),
// o = sum_{t <= p} softmax(z)_t c_t, with c_t the latent (4 bits, dequantized) and k_t the rotary key.
//
// Tiles.  Both products are formed transposed, positions and latent dimensions along M:
//   S^T [128 positions, NC lines]  = [C R] [Q_l Q_r]^T        (K = latent and rotary dimensions)
//   O^T [128 dimensions, NC lines] += C^T P^T, L / 128 times  (K = positions)
// so that the lines are a column count of 16, 32 or 64 (a decode step of 16 heads fills 16 columns, not 16
// of 128 rows), the output of 64 lines takes L / 128 x 64 = 256 of tensor memory's 512 columns, and one
// dequantized tile serves both products: rows of 64 dimensions are a K-major operand of the first and an
// MN-major one of the second.  A tile of 128 positions is 144 KB in shared memory and single: its halves
// of 256 dimensions are refilled as the second product lets them go.
//
// Warps of a CTA (one per SM):
//   0-7    softmax: two threads have a position, half of the lines' scores each in registers.
//   8-15   dequantize: packed rows go from memory to registers a tile ahead, eight lanes 128 bytes of a row.
//   16     issues the MMAs.
// Work is shared out as in kvq_units.cuh; an item is NC lines of one sequence.
//
// Rounding.  As in chunk_attention.cu: latents and weights are f16 operands, everything else fp32.  Latents are held
// halved (chunk_shared.cuh), so the rotary queries are too: below 2^-13 in size, to multiples of 2^-23 (2^-24 of a
// key's size in a score, where the rounding of the latents is 2^-12 of a query's).
//
// What bounds it.  One tile is in shared memory, so its steps stand in a row: refill of the halves (the
// unpacking of 128 x 512 values), 36 MMAs for the scores, the softmax, 32 for the output.  Measured, L =
// 512, the cache in memory (in brackets: in L2, from the call before): 32 sequences of 1024 to 8192 positions with 128
// heads 96 us (86; 41 GFLOP, 68 MB: tensor cores 20% busy, 35% of the issue slots); one of 131072 positions with 16
// heads 47 us (39; 52 MB), of which the merge of 152 parts is 5.  A second tile of 128 positions would take 144 KB that
// are not there at L = 512; at L = 256 (72 KB) there is room for one, and at 512 for two of 64 positions, which has
// not been tried.
#include <cuda_fp16.h>

#include <cmath>

#include "kvq_columns.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tcgen05.cuh"
#include "kvq_units.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 640;
constexpr int kSmWarps = 8, kDqWarps = 8, kMmaWarp = 16;
constexpr int kRope = 64;              // rotary dimensions
constexpr int kChunk = kTile * 128;    // bytes of a chunk [128][64] f16

struct LatentParams : Units {  // per_row: query heads
    const uint8_t* pool;
    const __half* q;
    const int32_t* block_table;
    __half* out;
    float* part_ml;  // [2 gridDim.x][NC][2]: reference maximum (of the scores) and sum
    float* part_o;   // [2 gridDim.x][NC][L]
    int32_t max_blocks, num_pages, lg_p, lg_g;
    float c;          // 2 |scale| log2(e): latents are held halved, and so are the rotary queries
    uint32_t q_flip;  // sign bits of a negative scale
    LatentLayout lay;
};

template <int L, int NC>
struct Shape {
    static constexpr int kChunks = L / 64 + 1;             // the last one: rotary keys
    static constexpr int kGroups = L / 128;                // outputs of 128 dimensions
    static constexpr int kHalves = L / 256;                // runs of four latent chunks, refilled together
    static constexpr int kQChunk = NC * 128;               // bytes of a chunk of queries [NC][64] f16
    static constexpr int kQ = kChunks * kQChunk;
    static constexpr int kK = kChunks * kChunk;
    // weights [128][NC] f16 in rows of 128 bytes: in place of the rotary keys where memory is short (the scores are
    // complete by the time there are weights)
    static constexpr bool kOwnP = kQ + kK + kChunk + 8192 <= 231424;
    static constexpr int kBytes = kQ + kK + (kOwnP ? kChunk : 0);
    static constexpr uint32_t kS = kGroups * NC;           // tensor memory: outputs, then scores
    static constexpr uint32_t kTmem = kS + NC <= 128 ? 128 : kS + NC <= 256 ? 256 : 512;
};

template <int NC>
struct Ctl {
    uint64_t full[3], free[3];  // halves of the latent chunks; [2]: the rotary chunk (the weights, where they share)
    uint64_t q_full, q_free, s_full, p_full, o_done, last;
    long long warp_sum[kThreads / 32];
    Start start;
    uint32_t tmem;
    int stop;
    Walk walk[kMmaWarp + 1];
    alignas(16) float ref[NC];    // the reference maximum, or 0 where nothing is seen yet
    alignas(16) float scale[NC];  // factors of a rescaling, or of the output
    float m[NC];                  // reference maximum of the scores (of z / scale)
    int lim[NC];                  // positions a line sees
    float part[4][NC];            // by warp
};

template <int L, int NC>
__global__ void __launch_bounds__(kThreads, 1) latent_kernel(const __grid_constant__ LatentParams p) {
    extern __shared__ uint8_t smem_raw[];
    using Z = Shape<L, NC>;
    constexpr int G = Z::kGroups;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t k_s = smem_u32(smem), q_s = k_s + Z::kK;
    const uint32_t p_s = Z::kOwnP ? q_s + Z::kQ : k_s + (Z::kChunks - 1) * kChunk;
    Ctl<NC>* ctl = reinterpret_cast<Ctl<NC>*>(smem + Z::kBytes);
    volatile int* stop = &ctl->stop;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), i < 2 ? kDqWarps / Z::kHalves : kDqWarps + p.withheld);
            mbar_init(smem_u32(&ctl->free[i]), 1);
        }
        mbar_init(smem_u32(&ctl->q_full), kDqWarps);
        mbar_init(smem_u32(&ctl->q_free), 1);
        mbar_init(smem_u32(&ctl->last), 1);
        mbar_init(smem_u32(&ctl->s_full), 1);
        mbar_init(smem_u32(&ctl->p_full), kSmWarps);
        mbar_init(smem_u32(&ctl->o_done), 1);
        ctl->stop = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&ctl->tmem), Z::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    find_start<kThreads>(p, &ctl->start, ctl->warp_sum);  // (has barriers of the CTA)
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Start st = ctl->start;
    Walk& walk = ctl->walk[min(warp, kMmaWarp)];
    if (st.units > 0 && warp <= kMmaWarp) walk.begin(p, st);
    const Segment& g = walk.g;

    if (warp < kSmWarps) {
        regs_more<104>();
        // ---- softmax: position `t` of a tile, columns c0 .. c0 + HC - 1; the thread's tensor-memory lane is also a
        // dimension of the outputs
        constexpr int HC = NC / 2;
        const int t = threadIdx.x & 127, side = warp / 4, c0 = side * HC;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t s_t = tmem + lanes + Z::kS + c0, o_t = tmem + lanes;
        uint32_t n_tile = 0, n_seg = 0;
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
            for (int i = 0; i < n; ++i, ++n_tile) {
                const int pos = (g.k0 + i) * kTile + t;
                wait_or_stop(smem_u32(&ctl->s_full), n_tile & 1, stop, p);
                tc_fence_after();
                uint32_t s[HC];
                auto fetch = [&]() {
                    load_columns<HC>(s_t, s);
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
                // Are the references still within 2^kLag of every score?  (Nothing is reduced over the positions then: of
                // a few hundred tiles a few move a reference)
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
#pragma unroll
                        for (int x = 0; x < HC; ++x) l[x] *= ctl->scale[c0 + x];
#pragma unroll 1
                        for (int x = side; x < G * NC / 16; x += 2) {  // (the products into O that came before S are complete)
                            uint32_t o[16];
                            tmem_ld16(o_t + 16 * x, o);
                            tmem_wait_ld();
                            tmem_touch(o);
                            const float* f = &ctl->scale[16 * x % NC];
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
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p_s + swizzled(t, (c0 + x) / 8)), "r"(w[0]), "r"(w[1]),
                                 "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full));
            }
            // ---- the segment's result
            const bool whole = g.k0 == 0 && g.k1 == g.nt;
            warp_sums<HC>(l, lane);
            ctl->part[warp & 3][c0 + first_column<HC>(lane)] = l[0];
            softmax_barrier();
            const long long line0 = static_cast<long long>(g.row0) * p.per_row + g.line0;
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
            wait_or_stop(smem_u32(&ctl->o_done), n_seg & 1, stop, p);
            ++n_seg;
            tc_fence_after();
            const int dim = dim_of(t);
#pragma unroll 1
            for (int x = side; x < G * NC / 16; x += 2) {
                uint32_t o[16];
                tmem_ld16(o_t + 16 * x, o);
                tmem_wait_ld();
                tmem_touch(o);
                const int c = 16 * x % NC, d = 16 * x / NC * 128 + dim;
                if (whole) {
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (c + y < g.lines)
                            p.out[(line0 + c + y) * L + d] = __float2half_rn(__uint_as_float(o[y]) * ctl->scale[c + y]);
                } else {
                    float* to = p.part_o + (static_cast<long long>(slot) * NC + c) * L + d;
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (c + y < g.lines) to[y * L] = __uint_as_float(o[y]);
                }
                __syncwarp();
            }
            tc_fence_before();
            softmax_barrier();
        }
    } else if (warp < kSmWarps + kDqWarps) {
        regs_more<104>();
        // ---- dequantize.  A warp takes four positions of one half (256 dimensions) at a time: eight lanes read 128
        // bytes of a row's codes, 16 each (32 dimensions, half of a chunk)
        constexpr int WPH = kDqWarps / Z::kHalves;   // warps of a half
        constexpr int JOBS = kTile / (4 * WPH);      // positions of a lane
        const int tid = threadIdx.x - 32 * kSmWarps, dw = warp - kSmWarps;
        const int half = dw / WPH, q = lane & 7, hf = q & 1;
        const int t0 = (dw % WPH) * 4 + (lane >> 3);  // the lane's positions: t0 + 4 WPH job
        const int r0 = dw * 4 + (lane >> 3);          // of the rotary keys: r0 + 32 job, 16 bytes each
        const int per = kTile >> p.lg_p, lg_p = p.lg_p;
        // A lane's four 16-byte pieces of f16 lie in one chunk; the eight lanes' chunks start on the same banks, so each
        // pair of lanes starts with another piece (its words turned accordingly) and no bank is met twice
        const int turn = q >> 1;
        uint32_t to[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            to[x] = k_s + (4 * half + (q >> 1)) * kChunk + t0 * 128 + (((4 * hf + ((x + turn) & 3)) ^ (t0 & 7)) << 4);
        struct Tile {
            const int32_t* table;
            const __half* q;  // the item's queries, where the tile is its first of this CTA (else nullptr)
            int tile, vis, lines;
            bool there;
        };
        int k = 0, k1 = 0;
        auto next_tile = [&](Tile& x) {
            x.q = nullptr;
            if (++k >= k1) {
                x.there = walk.next(p);
                if (!x.there) return;
                k = g.k0;
                k1 = g.k1;
                x.vis = g.vis;
                x.lines = g.lines;
                x.table = p.block_table + static_cast<long long>(g.b) * p.max_blocks;
                x.q = p.q + (static_cast<long long>(g.row0) * p.per_row + g.line0) * (L + kRope);
            }
            x.tile = k;
        };
        auto pages_of = [&](const Tile& x) -> int {  // lane l: page l of the tile
            const int first = x.tile * per + lane;
            return x.there && lane < per && (first << lg_p) < x.vis ? __ldg(x.table + first) : 0;
        };
        // the packed rows of a tile
        uint4 codes[JOBS], keys[4];
        uint32_t scales[JOBS];
        auto load = [&](const Tile& x, int pages) {
            const int end = x.there ? x.vis - x.tile * kTile : 0;  // positions that exist
            if (x.there && (pages < 0 || pages >= p.num_pages)) {
                raise_flag(p.status, KVQ_FLAG_BAD_PAGE);
                pages = 0;
            }
            const int mask = (1 << lg_p) - 1;
#pragma unroll
            for (int j = 0; j < JOBS; ++j) {
                const int t = t0 + 4 * WPH * j;
                const uint8_t* src = p.pool + static_cast<long long>(__shfl_sync(0xffffffffu, pages, t >> lg_p)) * p.lay.bytes;
                codes[j] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                scales[j] = 0;
                if (t < end) {
                    const int slot = t & mask;
                    codes[j] = __ldg(reinterpret_cast<const uint4*>(src + slot * (L / 2)) + 8 * half + q);
                    scales[j] = __ldg(reinterpret_cast<const uint16_t*>(src + p.lay.scales) +
                                      ((slot * L + 256 * half + 32 * q) >> p.lg_g));
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = r0 + 32 * j;
                const uint8_t* src = p.pool + static_cast<long long>(__shfl_sync(0xffffffffu, pages, t >> lg_p)) * p.lay.bytes;
                keys[j] = make_uint4(0, 0, 0, 0);
                if (t < end) keys[j] = __ldg(reinterpret_cast<const uint4*>(src + p.lay.rope + (t & mask) * (2 * kRope)) + q);
            }
        };
        auto store = [&](uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
        };
        uint32_t n_tile = 0, n_q = 0;
        Tile cur{}, nxt{};
        cur.there = false;
        if (st.units > 0) {
            next_tile(cur);
            nxt = cur;
            load(cur, pages_of(cur));
            if (cur.there) next_tile(nxt);
        }
        int pages = pages_of(nxt);
#pragma unroll 1
        while (cur.there) {
            if (cur.q != nullptr) {
                // the item's queries, latent dimensions in the order the unpack leaves, the rotary part halved
                if (n_q > 0) wait_or_stop(smem_u32(&ctl->q_free), (n_q - 1) & 1, stop, p);
                ++n_q;
                constexpr int PIECES = (L + kRope) / 8;
#pragma unroll 6
                for (int i = tid; i < NC * PIECES; i += 32 * kDqWarps) {
                    const int line = i / PIECES, piece = i - line * PIECES;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (line < cur.lines) x = __ldg(reinterpret_cast<const uint4*>(cur.q + static_cast<long long>(line) * (L + kRope)) + piece);
                    x.x ^= p.q_flip;
                    x.y ^= p.q_flip;
                    x.z ^= p.q_flip;
                    x.w ^= p.q_flip;
                    const uint32_t at = q_s + (piece / 8) * Z::kQChunk + swizzled(line, piece % 8);
                    if (piece < L / 8)
                        store(at, prmt(x.x, x.z, 0x5410), prmt(x.x, x.z, 0x7632), prmt(x.y, x.w, 0x5410), prmt(x.y, x.w, 0x7632));
                    else
                        store(at, h2_mul(x.x, 0x38003800u), h2_mul(x.y, 0x38003800u), h2_mul(x.z, 0x38003800u),
                              h2_mul(x.w, 0x38003800u));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full));
            }
            if (n_tile > 0) wait_or_stop(smem_u32(&ctl->free[half]), (n_tile - 1) & 1, stop, p);
#pragma unroll
            for (int j = 0; j < JOBS; ++j) {
                // half of the codes, so that 7 scales stay finite
                const uint32_t sc = scales[j] | scales[j] << 16;
                const bool one = turn & 1, two = turn & 2;
                const uint32_t a = one ? codes[j].y : codes[j].x, b = one ? codes[j].z : codes[j].y;
                const uint32_t c = one ? codes[j].w : codes[j].z, d = one ? codes[j].x : codes[j].w;
                const uint32_t ws[4] = {two ? c : a, two ? d : b, two ? a : c, two ? b : d};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t lo = ws[x], hi = ws[x] >> 8;
                    store(to[x] + 4 * WPH * 128 * j, h2_mul(unpack_lo_half(lo), sc), h2_mul(unpack_hi_half(lo), sc),
                          h2_mul(unpack_lo_half(hi), sc), h2_mul(unpack_hi_half(hi), sc));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->full[half]));
            if (n_tile > 0) wait_or_stop(smem_u32(&ctl->free[2]), (n_tile - 1) & 1, stop, p);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                store(k_s + (Z::kChunks - 1) * kChunk + swizzled(r0 + 32 * j, q), keys[j].x, keys[j].y, keys[j].z, keys[j].w);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->full[2]));
            // the next tile's rows (here and not between the stores: the fences above would wait for loads in flight)
            load(nxt, pages);
            Tile far = nxt;
            if (nxt.there) next_tile(far);
            pages = pages_of(far);
            ++n_tile;
            cur = nxt;
            nxt = far;
        }
    } else {
        regs_less<64>();
        if (warp == kMmaWarp) {
            // ---- the products
            constexpr uint32_t kIdS = mma_idesc(kTile, NC, false, false), kIdO = mma_idesc(128, NC, true, true);
            const uint32_t tm = uniform(tmem);
            bool live = true;  // false once a wait has been given up: nothing more is issued
            uint32_t n_tile = 0, n_seg = 0;
            while (uniform(st.units > 0 && walk.next(p))) {
                const int n = uniform(g.k1 - g.k0);
                live &= wait_or_stop(smem_u32(&ctl->q_full), n_seg & 1, stop, p);
                ++n_seg;
#pragma unroll 1
                for (int i = 0; i < n; ++i, ++n_tile) {
#pragma unroll 1
                    for (int c = 0; c <= Z::kHalves; ++c) {  // four chunks, four chunks, the rotary one
                        live &= wait_or_stop(smem_u32(&ctl->full[c < Z::kHalves ? c : 2]), n_tile & 1, stop, p);
                        tc_fence_after();
                        const uint32_t a = desc_lo(k_s + 4 * c * kChunk, 16), b = desc_lo(q_s + 4 * c * Z::kQChunk, 16);
                        if (elect_one() && live) {
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                if (x < 4 || c < Z::kHalves)
                                    mma_ss(tm + Z::kS, smem_desc(a + (((x / 4) * kChunk + (x % 4) * 32) >> 4)),
                                           smem_desc(b + (((x / 4) * Z::kQChunk + (x % 4) * 32) >> 4)), kIdS, c > 0 || x > 0);
                        }
                        __syncwarp();
                    }
                    if (elect_one() && live) {
                        mma_commit(smem_u32(&ctl->s_full));
                        if (i + 1 == n) mma_commit(smem_u32(&ctl->q_free));
                    }
                    __syncwarp();
                    live &= wait_or_stop(smem_u32(&ctl->p_full), n_tile & 1, stop, p);
                    tc_fence_after();
                    if (elect_one() && live) {
#pragma unroll 1
                        for (int m = 0; m < G; ++m) {
                            const uint32_t a = desc_lo(k_s + 2 * m * kChunk, kChunk), b = desc_lo(p_s, kChunk);
#pragma unroll
                            for (int x = 0; x < kTile / 16; ++x)
                                mma_ss(tm + m * NC, smem_desc(a + (x * 2048 >> 4)), smem_desc(b + (x * 2048 >> 4)), kIdO,
                                       i > 0 || x > 0);
                            if (m & 1) mma_commit(smem_u32(&ctl->free[m / 2]));
                        }
                        mma_commit(smem_u32(&ctl->free[2]));
                        if (i + 1 == n) mma_commit(smem_u32(&ctl->o_done));
                    }
                    __syncwarp();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    finish_products(warp == kMmaWarp, smem_u32(&ctl->last), stop);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, Z::kTmem);
    }
}

// The items cut between CTAs.
template <int L, int NC>
__global__ void __launch_bounds__(256) latent_merge_kernel(const __grid_constant__ LatentParams p, int ctas) {
    __shared__ MergeShare share;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    merge_items<L / 128>(
        p, p.c, ctas, 1, &share,
        [&](long long slot, int line, int e, float& m, float& l, float4& o, int lane) {
            const long long at = slot * NC + line;
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            m = ml.x;
            l = ml.y;
            o = reinterpret_cast<const float4*>(p.part_o + at * L)[32 * e + lane];
        },
        [&](const MergeDesc& d, int line, int e, float l, const float4& o, int lane) {
            const float inv = l > 0.f ? 2.f / l : 0.f;
            reinterpret_cast<uint2*>(p.out + (static_cast<long long>(d.line0) + line) * L)[32 * e + lane] =
                make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
        });
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <int L, int NC>
cudaError_t launch(LatentParams p, int ctas, cudaStream_t stream) {
    p.step = NC;
    const size_t smem = 1024 + Shape<L, NC>::kBytes + sizeof(Ctl<NC>);
    cudaError_t e =
        cudaFuncSetAttribute(latent_kernel<L, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
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
    e = cudaLaunchKernelEx(&cfg, latent_kernel<L, NC>, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(4 * ctas));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_merge_kernel<L, NC>, p, ctas);
}

}  // namespace

size_t latent_workspace_bytes(const LatentAttnArgs& a) {
    const size_t sms = static_cast<size_t>(attention_ctas());
    if (sms == 0) return 0;
    return 256 + align256(sms * sizeof(MergeDesc)) + 2 * sms * 64 * (2 + a.lay.L) * sizeof(float);
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, cudaStream_t stream) {
    const int sms = attention_ctas();
    LatentParams p{};
    p.pool = a.pool;
    p.q = a.q;
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.cu_rows = a.cu_rows;
    p.out = a.out;
    p.status = reinterpret_cast<uint32_t*>(a.workspace);
    p.desc = reinterpret_cast<MergeDesc*>(a.workspace + 256);
    p.part_ml = reinterpret_cast<float*>(a.workspace + 256 + align256(sms * sizeof(MergeDesc)));
    p.part_o = p.part_ml + 2ll * sms * 64 * 2;
    p.rows = a.rows;
    p.B = a.B;
    p.heads = 1;
    p.per_row = a.H;
    p.max_blocks = a.max_blocks;
    p.num_pages = a.num_pages;
    p.lg_p = a.lg_p;
    p.lg_g = a.lay.G == 32 ? 5 : a.lay.G == 64 ? 6 : 7;
    const long long table = static_cast<long long>(a.max_blocks) << a.lg_p;
    p.most = static_cast<int32_t>(table < a.max_len ? table : a.max_len);
    p.wait_ns = a.wait_limit_ns > 0 ? a.wait_limit_ns : kWaitNs;
    p.withheld = a.wait_limit_ns > 0;
    // (at least 1e-30: a hidden score is -infinity, which zero times is not a number)
    p.c = std::fmax(2.f * std::fabs(a.softmax_scale) * 1.4426950408889634f, 1e-30f);
    p.q_flip = a.softmax_scale < 0.f ? 0x80008000u : 0u;
    p.lay = a.lay;
    // As many lines to an item as a sequence has on average: an MMA of 16, 32 and 64 columns takes 40, 41 and 48
    // cycles, but unused columns cost shared memory for their queries and the softmax's time
    const long long lines = static_cast<long long>(a.rows) * a.H / a.B;
    const int nc = lines <= 16 ? 16 : lines <= 32 ? 32 : 64;
    if (a.lay.L == 256)
        return nc == 16 ? launch<256, 16>(p, sms, stream) : nc == 32 ? launch<256, 32>(p, sms, stream) : launch<256, 64>(p, sms, stream);
    return nc == 16 ? launch<512, 16>(p, sms, stream) : nc == 32 ? launch<512, 32>(p, sms, stream) : launch<512, 64>(p, sms, stream);
}

}  // namespace kvq
