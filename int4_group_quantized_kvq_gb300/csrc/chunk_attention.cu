// chunk_attention.cu -- causal attention of a ragged batch of query rows (prompts, parts of prompts,
// a few drafted tokens) over the packed INT4 cache, on the tcgen05 tensor cores.
//
// For a row at position p:  z_t = scale q . k_t,  o = sum_{t <= p} softmax(z)_t v_t.
//
// Tiles.  128 rows of M are the r query heads of 128 / r tokens that share a kv head; 128 positions are
// a key/value tile.  An item is two such row tiles of one (sequence, kv head), which share every key and
// value tile (the dequantization is paid once for 256 rows); where an item has no second row tile, its
// two streams take alternate key/value tiles instead and merge at the end.  A unit is one key/value
// tile of an item; every CTA takes an equal run of the list of units, so causal prompts, uneven batches
// and single long sequences spread evenly.  An item cut between CTAs leaves partial results (maximum,
// sum, unnormalised output) that a second kernel merges in order.
//
// Warps of a CTA (one per SM):
//   0-3, 4-7   softmax of stream 0 and 1: a thread has a row.  Scores come from tensor memory, weights go
//              back there (as the f16 A operand of the second product, over the scores' columns).
//   8-15       dequantize packed tiles into f16 operand tiles (shared memory, a ring of kRing), and bring the
//              items' queries there.
//   16, 17     issue the MMAs of stream 0 and 1: S = Q K^T (both from shared memory), O += P V (P from tensor
//              memory).  A warp for each, so that one stream's waits and bookkeeping do not hold up the other.
//   18         copies packed pages into shared memory (bulk copies, a ring of kPacked tiles).
//
// Rounding.  Operands are f16: code x scale (chunk_shared.cuh) and the weights (11 of their bits; the sum
// that divides takes them unrounded).  Scores, maxima, sums and outputs are fp32 throughout.
//
// What bounds it.  A pair of tiles (one key/value tile, both streams) takes the tensor cores 32 MMAs of 64
// cycles, 2048; the exponential unit 32768 values at 32 a cycle, 1024; the half-rate pipe (64 lanes a cycle)
// about 1500 for the maxima, the conversions and the unpacking of keys and values.  It takes about 5000 in
// all.  Measured (8192 tokens of one prompt, 32 heads on 8 kv heads of 128): 609 us, 903 TFLOP/s, tensor
// cores 39% busy, 56% of the issue slots.  A stream's scores, softmax and output follow one another, and with two
// streams the waits between them are not filled: neither pipe is full.  (At head_dim 128 tensor memory has no room
// for a third buffer of scores; at 64, where half of the products wait for the same softmax, 128 columns are free.)
// Tried and not kept: 64-position steps with two score buffers a stream (848 -> 991 us at the time); the
// softmax loops unrolled whole (848 instead of 703: instruction fetch); 128 scores in registers at once
// (spills, which go to L2).
#include <cuda_fp16.h>

#include <cmath>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "chunk_shared.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 640;
constexpr int kRing = 3;  // operand tiles
constexpr uint32_t kTmem = 512;
// Up to so many lines to a sequence, on average, lines are columns (chunk_few.cu).  Both sides for even batches, in
// us, lines as columns first: four sequences of 32761 positions, 8 kv heads of 128, with 4 lines 69 and 111, with 32
// lines 76 and 112, with 36 (two items) 134 and 113, with 64 134 and 114; 16 of 8000 positions with 32 lines 77 and
// 112; 24 short sequences of 4 to 12 lines, 21 and 24.  The average is what the host knows: all rows of the arrays,
// those behind the last sequence too, over the batch.  It is a poor guide where they are uneven: 16 single tokens over
// 4096 positions take 42, in arrays padded to 2048 rows 64; 64 of them and a prompt of 2048 rows 342, where apart they
// take 127 and 83; 63 and a part of 400 rows 241, apart 125 and 58.
constexpr int kFewLines = 32;

struct Ctl {
    TileBars tiles;
    // o_done: a stream's output of a segment of two row tiles, for that stream alone; o_both: both streams' of a segment
    // of one, for both.  (A stream that waited for the other's o_done in some segments would skip phases of it, and
    // a wait by parity knows a phase only from the one before)
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_done[2], o_both, turn, last[2];
    long long warp_sum[kThreads / 32];
    Start start;
    uint32_t tmem;
    int stop;
    Walk walk[kThreads / 32];
    float ml[2][kTile][2];
};

template <int D>
struct Sizes {
    static constexpr int kOperand = kTile * D * 2;           // bytes of an operand tile
    static constexpr int kQ = 2 * kOperand;
};

// Eight output columns (in the order the unpack leaves: 0 4 1 5 2 6 3 7) as 16 bytes in dimension order.
__device__ __forceinline__ uint4 columns_to_halves(const float (&v)[8]) {
    return make_uint4(pack_h2(v[0], v[2]), pack_h2(v[4], v[6]), pack_h2(v[1], v[3]), pack_h2(v[5], v[7]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ uint8_t smem_raw[];
    using Z = Sizes<D>;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_u32(smem), ring_s = q_s + Z::kQ, packed_s = ring_s + kRing * Z::kOperand;
    const int packed_bytes = (kTile >> p.lg_p) * p.L.bytes;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + Z::kQ + kRing * Z::kOperand + kPacked * packed_bytes);
    volatile int* stop = &ctl->stop;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPacked; ++i) {
            mbar_init(smem_u32(&ctl->tiles.pk_full[i]), 1);
            mbar_init(smem_u32(&ctl->tiles.pk_empty[i]), kDqWarps);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&ctl->tiles.kv_full[i]), kDqWarps + (i == 1 ? p.withheld : 0));
            mbar_init(smem_u32(&ctl->tiles.kv_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->q_full[i]), kDqWarps);
            mbar_init(smem_u32(&ctl->q_free[i]), 2 - i);
            mbar_init(smem_u32(&ctl->s_full[i]), 1);
            mbar_init(smem_u32(&ctl->p_full[i]), 4);
            mbar_init(smem_u32(&ctl->o_done[i]), 1);
            mbar_init(smem_u32(&ctl->last[i]), 1);
        }
        mbar_init(smem_u32(&ctl->o_both), 2);
        mbar_init(smem_u32(&ctl->turn), 1);
        ctl->stop = 0;
        fence_mbar_init();
    }
    if (warp == 16) tmem_alloc(smem_u32(&ctl->tmem), kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    find_start<kThreads>(p, &ctl->start, ctl->warp_sum);  // (has barriers of the CTA)
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Start st = ctl->start;

    Walk& walk = ctl->walk[warp];
    if (st.units > 0) walk.begin(p, st);
    const Segment& g = walk.g;

    if (warp < 8) {
        regs_more<136>();
        // ---- softmax of stream sw, row `row` of the stream's row tile
        const int sw = warp / 4;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t s_t = tmem + lanes + 128u * sw, o_t = tmem + lanes + 256u;
        const int tok_in = row / p.r;  // token within the row tile
        uint32_t n_s = 0, n_two = 0, n_one = 0;  // score tiles; segments of two row tiles, and of one
        while (st.units > 0 && walk.next(p)) {
            const int n = g.k1 - g.k0;
            const bool two = g.lines > p.T;                    // a second row tile (else the streams alternate)
            const int tok = (two ? sw * p.T : 0) + tok_in;     // token of the item
            const bool valid = tok_in < p.T && tok < g.lines;
            int seen = valid ? g.ahead + g.line0 + tok + 1 - g.k0 * kTile : 0;  // columns the row sees, from tile k0 on
            float m = -INFINITY, l = 0.f;  // the maximum the weights are taken against (of z / scale), their sum
            bool begun = false;
            if (!two && sw == 1) seen -= kTile;
            for (int i = two ? 0 : sw; i < n; i += two ? 1 : 2, seen -= two ? kTile : 2 * kTile) {
                wait_or_stop(smem_u32(&ctl->s_full[sw]), n_s & 1, stop, p);
                ++n_s;
                tc_fence_after();
                // Two passes over the scores, 64 columns at a time: the maximum, then the weights.  (128 scores in
                // registers at once would spill, and a spill goes to L2, shared memory leaving no L1 to speak of.)
                // The loops are not unrolled further: five warps with five programs share a scheduler, and longer
                // code keeps them waiting for instructions
                const bool part = __any_sync(0xffffffffu, seen < kTile);
                uint32_t a[32], b[32];
                auto fetch = [&](int x) {
                    tmem_ld32(s_t + 64 * x, a);
                    tmem_ld32(s_t + 64 * x + 32, b);
                    tmem_wait_ld();
                    tmem_touch(a);
                    tmem_touch(b);
                    if (part) {
                        const int to = seen - 64 * x;
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            if (y >= to) a[y] = 0xff800000u;
                            if (32 + y >= to) b[y] = 0xff800000u;
                        }
                    }
                };
                float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    fetch(x);
#pragma unroll
                    for (int y = 0; y < 32; y += 2) {
                        top0 = fmaxf(fmaxf(top0, __uint_as_float(a[y])), __uint_as_float(a[y + 1]));
                        top1 = fmaxf(fmaxf(top1, __uint_as_float(b[y])), __uint_as_float(b[y + 1]));
                    }
                }
                const float top = fmaxf(top0, top1);
                // (kvq_units.cuh: when the reference follows the maximum)
                const bool move = (top - m) * p.c > kLag || m == -INFINITY;
                const float m_new = move ? fmaxf(top, m) : m;
                if (begun && __any_sync(0xffffffffu, move && m_new != m)) {
                    const float f = m_new == -INFINITY ? 1.f : fast_exp2((m - m_new) * p.c);
                    l *= f;
#pragma unroll 1
                    for (int x = 0; x < D / 16; ++x) {  // (the products into O that came before S are complete)
                        uint32_t o[16];
                        tmem_ld16(o_t + D * sw + 16 * x, o);
                        tmem_wait_ld();
                        tmem_touch(o);
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tmem_st16(o_t + D * sw + 16 * x, o);
                    }
                }
                m = m_new;
                begun = true;
                // The difference before the product: exact at the maximum however large the scores are, where a fused
                // s c - m c would leave the rounding of m c (2% of a long prompt's time; a branch for large scores alone
                // took the same)
                const float ref = m == -INFINITY ? 0.f : -m;
                const uint64_t c2 = pair_of(p.c, p.c), ref2 = pair_of(ref, ref), up2 = pair_of(kUp, kUp);
                uint64_t sums = 0, sums1 = 0;  // two sums each
                // the second half first: the weights, two to a column, go to columns 64 .. 127, over scores that
                // are in registers by now
#pragma unroll 1
                for (int x = 1; x >= 0; --x) {
                    fetch(x);
                    auto weigh = [&](uint32_t (&v)[32], uint64_t& sum, uint32_t to) {
                        uint32_t w[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const uint64_t z = fma_pair(add_pair(pair_of(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])), ref2), c2, up2);
                            float p0, p1;
                            split_pair(z, p0, p1);
                            p0 = fast_exp2(p0);
                            p1 = fast_exp2(p1);
                            sum = add_pair(sum, pair_of(p0, p1));
                            w[y] = pack_h2(p0, p1);
                        }
                        tmem_st16(to, w);
                    };
                    weigh(a, sums, s_t + 64 + 32 * x);
                    weigh(b, sums1, s_t + 80 + 32 * x);
                }
                float l0, l1, l2, l3;
                split_pair(sums, l0, l1);
                split_pair(sums1, l2, l3);
                l += (l0 + l1) + (l2 + l3);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[sw]));
            }
            // ---- the segment's result
            const bool whole = g.k0 == 0 && g.k1 == g.nt;
            const int slot = partial_slot(g);
            const int prow = (two ? sw * kTile : 0) + row;  // row of a partial result
            float* pml = p.part_ml + (static_cast<long long>(slot) * 256 + prow) * 2;
            float* po = p.part_o + (static_cast<long long>(slot) * 256 + prow) * D;
            __half* out = p.out + (static_cast<long long>(g.row0 + g.line0 + tok) * p.Hq + g.h * p.r + (row - tok_in * p.r)) * D;
            auto put = [&](const uint32_t (&o)[32], int x, float f) {  // 32 columns of the row
                if (valid && whole) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float v[8];
#pragma unroll
                        for (int z = 0; z < 8; ++z) v[z] = __uint_as_float(o[8 * y + z]) * f;
                        reinterpret_cast<uint4*>(out)[4 * x + y] = columns_to_halves(v);
                    }
                } else if (valid) {
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        reinterpret_cast<uint4*>(po)[8 * x + y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
                __syncwarp();
            };
            if (two) {
                wait_or_stop(smem_u32(&ctl->o_done[sw]), n_two & 1, stop, p);
                ++n_two;
                tc_fence_after();
                const float inv = l > 0.f ? 2.f / l : 0.f;
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t o[32];
                    tmem_ld32(o_t + D * sw + 32 * x, o);
                    tmem_wait_ld();
                    tmem_touch(o);
                    put(o, x, inv);
                }
                if (valid && !whole) {
                    pml[0] = m;
                    pml[1] = l;
                }
                tc_fence_before();
            } else {
                // both streams hold a part of the same rows: lane by lane the same tensor-memory lane
                const bool both = n > 1;
                wait_or_stop(smem_u32(&ctl->o_both), n_one & 1, stop, p);
                ++n_one;
                tc_fence_after();
                ctl->ml[sw][row][0] = m;
                ctl->ml[sw][row][1] = l;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const float m0 = ctl->ml[0][row][0], m1 = ctl->ml[1][row][0];
                const float mm = fmaxf(m0, m1);
                const float a0 = m0 == -INFINITY ? 0.f : fast_exp2((m0 - mm) * p.c);
                const float a1 = m1 == -INFINITY ? 0.f : fast_exp2((m1 - mm) * p.c);
                const float ll = ctl->ml[0][row][1] * a0 + ctl->ml[1][row][1] * a1;
                const float f = whole ? (ll > 0.f ? 2.f / ll : 0.f) : 1.f;
#pragma unroll 1
                for (int x = sw * (D / 64); x < (sw + 1) * (D / 64); ++x) {  // each stream's warps half of the columns
                    uint32_t o[32], u[32];
                    tmem_ld32(o_t + 32 * x, o);
                    if (both) tmem_ld32(o_t + D + 32 * x, u);
                    tmem_wait_ld();
                    tmem_touch(o);
                    if (both) tmem_touch(u);
#pragma unroll
                    for (int y = 0; y < 32; ++y) {
                        float v = __uint_as_float(o[y]) * a0;
                        if (both) v = fmaf(__uint_as_float(u[y]), a1, v);
                        o[y] = __float_as_uint(v);
                    }
                    put(o, x, f);
                }
                if (valid && !whole && sw == 0) {
                    pml[0] = mm;
                    pml[1] = ll;
                }
                tc_fence_before();
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
        }
    } else if (warp < 8 + kDqWarps) {
        regs_less<72>();
        // ---- dequantize
        const int dw = warp - 8;
        uint32_t n_ring = 0, n_pk = 0, n_q0 = 0, n_q1 = 0;
        while (st.units > 0 && walk.next(p)) {
            const int n = g.k1 - g.k0;
            const int end0 = g.vis - g.k0 * kTile;
            auto dequant = [&](int i, int is_v) {
                dequantize_tile<D, false>(p, ctl->tiles, smem + Z::kQ + kRing * Z::kOperand, packed_bytes, ring_s, n_pk + i,
                                          end0 - i * kTile, is_v, dw, n_ring % kRing, n_ring / kRing, stop);
                ++n_ring;
            };
            // the item's row tile qs into shared memory, its dimensions in the order the unpack leaves (n_q: how many
            // have been there before)
            auto queries = [&](int qs, uint32_t n_q) {
                constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes of a row, rows a warp takes at a time
                constexpr int LOADS = kTile / (RPW * kDqWarps) / 2;
                const int rows = min(g.lines - qs * p.T, p.T) * p.r;
                const __half* src = p.q + (static_cast<long long>(g.row0 + g.line0 + qs * p.T) * p.Hq + g.h * p.r) * D;
                const int piece = lane % LPR;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int row0 = half * (kTile / 2) + dw * RPW + lane / LPR;
                    uint4 x[LOADS];
#pragma unroll
                    for (int i = 0; i < LOADS; ++i) {
                        const int row = row0 + i * RPW * kDqWarps;
                        const int tok = row / p.r;
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (row < rows)
                            x[i] = __ldg(reinterpret_cast<const uint4*>(src + (static_cast<long long>(tok) * p.Hq + row - tok * p.r) * D) +
                                         piece);
                    }
                    if (n_q > 0 && half == 0) wait_or_stop(smem_u32(&ctl->q_free[qs]), (n_q - 1) & 1, stop, p);
#pragma unroll
                    for (int i = 0; i < LOADS; ++i) {
                        const int row = row0 + i * RPW * kDqWarps;
                        const uint32_t at = q_s + qs * Z::kOperand + (piece / 8) * kChunk + swizzled(row, piece % 8);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(prmt(x[i].x, x[i].z, 0x5410) ^ p.q_flip),
                                     "r"(prmt(x[i].x, x[i].z, 0x7632) ^ p.q_flip), "r"(prmt(x[i].y, x[i].w, 0x5410) ^ p.q_flip),
                                     "r"(prmt(x[i].y, x[i].w, 0x7632) ^ p.q_flip)
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full[qs]));
            };
            // in the order of the products.  Two row tiles: K0 V0 K1 V1 ..; one, whose streams' next scores come
            // before the other's output: K0 K1 V0 K2 V1 ..
            const bool two = g.lines > p.T;
#pragma unroll 1
            for (int t = 0; t < 2 * n; ++t) {
                int i = t >> 1, is_v = t & 1;
                if (!two && t < 2 * n - 1) {
                    is_v = t >= 2 && !(t & 1);
                    i = t < 2 ? t : t & 1 ? (t + 1) >> 1 : (t - 2) >> 1;
                }
                dequant(i, is_v);
                if (t == 0) {
                    queries(0, n_q0);
                    ++n_q0;
                    if (two) {
                        queries(1, n_q1);
                        ++n_q1;
                    }
                }
            }
            n_pk += n;
        }
    } else {
        regs_less<64>();
        if (warp < 18) {
            // ---- the products of stream sw
            constexpr uint32_t kIdS = mma_idesc(kTile, kTile, false, false), kIdO = mma_idesc(kTile, D, false, true);
            // (The path between two products has as few trips to shared memory as can be: each takes 250 cycles in
            // the traffic of the other warps, as long as the MMAs still queued.)
            const uint32_t tm = uniform(tmem), sw = uniform(warp - 16);
            bool live = true;  // false once a wait has been given up: nothing more is issued
            uint32_t n_ring = 0, n_q0 = 0, n_q1 = 0, n_p = 0, n_turn = 0;
            auto take = [&]() -> uint32_t {  // the next operand tile, in order
                const uint32_t stage = n_ring % kRing;
                live &= wait_or_stop(smem_u32(&ctl->tiles.kv_full[stage]), (n_ring / kRing) & 1, stop, p);
                ++n_ring;
                tc_fence_after();
                return stage;
            };
            while (uniform(st.units > 0 && walk.next(p))) {
                const int n = uniform(g.k1 - g.k0);
                const bool two = uniform(g.lines > p.T);
                // Two row tiles: turn i is the output with value tile i and the scores with key tile i + 1, of both
                // streams.  One: the output with value tile i and the scores with key tile i + 2, of stream i % 2; the
                // other stream lets the tiles go.  (It starts with turns that have scores alone.)
                // The streams issue in turn, a turn's products as one block: the streams' softmaxes then alternate
                // with the products.  Mixed products would end together, and then both softmaxes run at once while
                // the tensor cores wait.
                // Turns alternate strictly (stream 1 takes an empty one behind an odd number of alternating tiles): a
                // stream that waits for the other's turn has then seen the one before it.
                const int ahead = two ? 1 : 2, turns = two ? n : n + (n & 1);
                live &= wait_or_stop(smem_u32(&ctl->q_full[0]), n_q0 & 1, stop, p);
                ++n_q0;
                if (two && sw == 1) {
                    live &= wait_or_stop(smem_u32(&ctl->q_full[1]), n_q1 & 1, stop, p);
                    ++n_q1;
                }
#pragma unroll 1
                for (int i = -ahead; i < turns; ++i) {
                    const bool mine = two || (i & 1) == static_cast<int>(sw);
                    const bool out = i >= 0 && i < n, in = i + ahead < n;
                    const uint32_t v = out ? take() : 0, k = in ? take() : 0;
                    if (mine) {
                        if (out) {
                            live &= wait_or_stop(smem_u32(&ctl->p_full[sw]), n_p & 1, stop, p);
                            ++n_p;
                        }
                        const uint32_t turn = n_turn + (two ? 2 * (i + 1) + sw : i + 2);
                        if (turn > 0) live &= wait_or_stop(smem_u32(&ctl->turn), (turn - 1) & 1, stop, p);
                        tc_fence_after();
                        if (elect_one()) {
                            if (live && out) {
                                const uint32_t a = tm + 128u * sw + 64, d = tm + 256u + D * sw;
                                const uint32_t b = desc_lo(ring_s + v * Z::kOperand, kChunk);
                                const bool first = i < ahead;
#pragma unroll
                                for (int x = 0; x < kTile / 16; ++x)
                                    mma_ts(d, a + 8 * x, smem_desc(b + (x * 2048 >> 4)), kIdO, !first || x > 0);
                                mma_commit(smem_u32(&ctl->tiles.kv_empty[v]));
                                if (two && !in) mma_commit(smem_u32(&ctl->o_done[sw]));
                            }
                            if (live && in) {
                                const uint32_t a = desc_lo(q_s + (two ? sw : 0) * Z::kOperand, 16);
                                const uint32_t b = desc_lo(ring_s + k * Z::kOperand, 16);
                                const uint32_t d = tm + 128u * sw;
#pragma unroll
                                for (int x = 0; x < D / 16; ++x) {
                                    const uint32_t off = ((x / 4) * kChunk + (x % 4) * 32) >> 4;
                                    mma_ss(d, smem_desc(a + off), smem_desc(b + off), kIdS, x > 0);
                                }
                                mma_commit(smem_u32(&ctl->s_full[sw]));
                                mma_commit(smem_u32(&ctl->tiles.kv_empty[k]));
                            }
                            if (live && !two && i + 2 >= turns) mma_commit(smem_u32(&ctl->o_both));  // the stream's last turn
                            mbar_arrive(smem_u32(&ctl->turn));
                        }
                    } else if (elect_one()) {
                        if (out) mbar_arrive(smem_u32(&ctl->tiles.kv_empty[v]));
                        if (in) mbar_arrive(smem_u32(&ctl->tiles.kv_empty[k]));
                    }
                    if (i + ahead + 1 == n && elect_one() && live) {  // no more scores of the item
                        mma_commit(smem_u32(&ctl->q_free[0]));
                        if (two && sw == 1) mma_commit(smem_u32(&ctl->q_free[1]));
                    }
                    __syncwarp();
                }
                n_turn += two ? 2 * (n + 1) : turns + 2;
            }
        } else if (warp == 18) {
            // ---- packed pages
            load_pages(p, ctl->tiles, walk, packed_s, packed_bytes, st.units > 0, stop);
        }
    }
    tc_fence_before();
    __syncthreads();
    finish_products(warp == 16 || warp == 17, smem_u32(&ctl->last[warp & 1]), stop);
    if (warp == 16) {
        tc_fence_after();
        tmem_free(tmem, kTmem);
    }
}

// The items cut between CTAs.
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const __grid_constant__ ChunkParams p, int ctas) {
    __shared__ MergeShare share;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // lanes hold 4 columns of a row each (D = 64: half of the lanes)
    merge_items<1>(
        p, p.c, ctas, p.r, &share,
        [&](long long slot, int line, int, float& m, float& l, float4& o, int lane) {
            const int tok = line / p.r;
            const long long at = slot * 256 + (tok / p.T) * kTile + (tok % p.T) * p.r + line - tok * p.r;
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            m = ml.x;
            l = ml.y;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * lane < D) o = reinterpret_cast<const float4*>(p.part_o + at * D)[lane];
        },
        [&](const MergeDesc& d, int line, int, float l, const float4& o, int lane) {
            if (4 * lane >= D) return;
            const float inv = l > 0.f ? 2.f / l : 0.f;
            const int tok = line / p.r;
            // columns 4 lane .. of the 8 that share 16 bytes: dimensions 0 4 1 5 or 2 6 3 7
            __half* out = p.out + (static_cast<long long>(d.line0 + tok) * p.Hq + d.h * p.r + line - tok * p.r) * D + (lane & ~1) * 4 +
                          (lane & 1) * 2;
            *reinterpret_cast<uint32_t*>(out) = pack_h2(o.x * inv, o.z * inv);
            *reinterpret_cast<uint32_t*>(out + 4) = pack_h2(o.y * inv, o.w * inv);
        });
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <int D>
cudaError_t launch(const ChunkParams& p, int ctas, cudaStream_t stream) {
    const size_t smem = 1024 + Sizes<D>::kQ + kRing * Sizes<D>::kOperand +
                        static_cast<size_t>(kPacked) * (kTile >> p.lg_p) * p.L.bytes + sizeof(Ctl);
    cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
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
    e = cudaLaunchKernelEx(&cfg, chunk_kernel<D>, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(4 * ctas));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D>, p, ctas);
}

}  // namespace

int attention_ctas() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms < kMaxCtas ? sms : kMaxCtas;
}

size_t chunk_workspace_bytes(const ChunkArgs& a) {
    const size_t sms = static_cast<size_t>(attention_ctas());
    if (sms == 0) return 0;
    return 256 + align256(sms * sizeof(MergeDesc)) + 2 * sms * 256 * (2 + a.L.d) * sizeof(float);
}

cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t stream) {
    const int sms = attention_ctas();
    ChunkParams p{};
    p.pool = a.pool;
    p.q = a.q;
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.cu_rows = a.cu_rows;
    p.out = a.out;
    p.status = reinterpret_cast<uint32_t*>(a.workspace);
    p.desc = reinterpret_cast<MergeDesc*>(a.workspace + 256);
    p.part_ml = reinterpret_cast<float*>(a.workspace + 256 + align256(sms * sizeof(MergeDesc)));
    p.part_o = p.part_ml + 2ll * sms * 256 * 2;
    p.rows = a.rows;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.r = a.Hq / a.Hkv;
    p.T = kTile / p.r;
    p.heads = a.Hkv;
    p.per_row = 1;
    p.step = 2 * p.T;
    p.max_blocks = a.max_blocks;
    p.num_pages = a.num_pages;
    p.lg_p = a.lg_p;
    p.lg_gk = a.L.Gk == 32 ? 5 : a.L.Gk == 64 ? 6 : 7;
    p.lg_gv = a.L.Gv == 32 ? 5 : a.L.Gv == 64 ? 6 : 7;
    const long long table = static_cast<long long>(a.max_blocks) << a.lg_p;
    p.most = static_cast<int32_t>(table < a.max_len ? table : a.max_len);
    p.wait_ns = a.wait_limit_ns > 0 ? a.wait_limit_ns : kWaitNs;
    p.withheld = a.wait_limit_ns > 0;
    // (at least 1e-30: a hidden score is -infinity, which zero times is not a number)
    p.c = std::fmax(2.f * std::fabs(a.softmax_scale) * 1.4426950408889634f, 1e-30f);
    p.q_flip = a.softmax_scale < 0.f ? 0x80008000u : 0u;
    p.L = a.L;
    // Few lines to a sequence (on average): lines as columns instead of rows of 128
    const long long lines = static_cast<long long>(a.rows) * p.r / a.B;
    if (lines <= kFewLines) return launch_chunk_few(p, a.L.d, static_cast<int>(lines), sms, stream);
    return a.L.d == 64 ? launch<64>(p, sms, stream) : launch<128>(p, sms, stream);
}

}  // namespace kvq
