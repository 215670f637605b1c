// chunk_shared.cuh -- what the two kernels of chunk attention share: their parameters, and the way of a
// tile of 128 positions from its packed pages into f16 operand tiles.
#pragma once

#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tcgen05.cuh"
#include "kvq_units.cuh"

namespace kvq {

constexpr int kDqWarps = 8;
constexpr int kMaxRing = 4;          // operand tiles (K or V) in shared memory, at most
constexpr int kPacked = 3;           // packed tiles in shared memory
constexpr int kChunk = kTile * 128;  // bytes of a chunk [128][64] f16

struct ChunkParams : Units {  // an item: the tokens of two row tiles
    const uint8_t* pool;
    const __half* q;
    const int32_t* block_table;
    __half* out;
    float* part_ml;   // [2 gridDim.x][256][2]: reference maximum (of the scores) and sum
    float* part_o;    // [2 gridDim.x][256][D]
    int32_t Hq, Hkv, r, T, max_blocks, num_pages, lg_p, lg_gk, lg_gv;  // T: tokens of a row tile
    float c;          // 2 |scale| log2(e): keys are held halved
    uint32_t q_flip;  // sign bits of a negative scale
    BlockLayout L;
};

// The barriers of the rings: packed tiles (copied, read), operand tiles (written, multiplied).
struct TileBars {
    uint64_t pk_full[kPacked], pk_empty[kPacked];
    uint64_t kv_full[kMaxRing], kv_empty[kMaxRing];
};

// The keys (is_v 0) or values of packed tile n_tile, `end` of whose positions exist, into operand tile
// `stage`, which was written `use` times before; by warp dw of kDqWarps.  APART: keys and values have
// warps of their own (else the same ones dequantize a tile's keys, later its values).
//
// code x scale has 15 significant bits and is rounded to the 11 of f16, the operands' type: a relative
// 2^-12 at most on average over a key's dimensions, which moves a score by about 2^-12 of its own spread.
// (Exact operands would take a second product for the scales' lower bits, or one product per group.)  Half of
// it is what is held (7 scales may pass fp16's largest), so elements below 2^-13 in size are rounded to multiples of
// 2^-23; the scale itself is not rounded.
template <int D, bool APART>
__device__ __forceinline__ void dequantize_tile(const ChunkParams& p, TileBars& tiles, const uint8_t* packed, int packed_bytes,
                                                uint32_t ring_s, uint32_t n_tile, int end, int is_v, int dw, uint32_t stage,
                                                uint32_t use, volatile int* stop) {
    constexpr int PARTS = D / 32;  // 16-byte pieces of a row's codes
    constexpr int kOperand = kTile * D * 2;
    const int lane = threadIdx.x & 31;
    const uint32_t pk = n_tile % kPacked;
    if (APART || is_v == 0) wait_or_stop(smem_u32(&tiles.pk_full[pk]), (n_tile / kPacked) & 1, stop, p);
    const uint8_t* src = packed + pk * packed_bytes;
    const uint32_t dst = ring_s + stage * kOperand;
    const int lg_g = is_v ? p.lg_gv : p.lg_gk;
    const int codes_off = is_v ? p.L.v_codes : 0, scales_off = is_v ? p.L.v_scales : p.L.k_scales;
    const int mask = (1 << p.lg_p) - 1;
    constexpr int JOBS = kTile * PARTS / (32 * kDqWarps);
    // 8 tokens x 4 pieces a warp: eight lanes of a piece read 128 bytes apart by rows (no bank twice)
    // and write 8 rows' swizzled pieces (no bank twice)
    uint32_t f[JOBS][16];
#pragma unroll
    for (int w = 0; w < JOBS; ++w) {
        const int job = (w * kDqWarps + dw) * 32 + lane;
        const int t = (job / (8 * PARTS)) * 8 + (job & 7);
        const int part = ((job >> 3) + (t & 7) * PARTS / 8) % PARTS;
        const uint8_t* blk = src + (t >> p.lg_p) * p.L.bytes;
        const int slot = t & mask;
        uint4 w4 = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        uint32_t s2 = 0;
        if (t < end) {
            w4 = *reinterpret_cast<const uint4*>(blk + codes_off + slot * (D / 2) + part * 16);
            s2 = *reinterpret_cast<const uint16_t*>(blk + scales_off + (((slot * D + part * 32) >> lg_g) << 1));
        }
        // half of the codes, so that 7 scales stay finite
        const uint32_t sc = s2 | s2 << 16;
        const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t lo = ws[x], hi = ws[x] >> 8;
            f[w][4 * x] = h2_mul(unpack_lo_half(lo), sc);
            f[w][4 * x + 1] = h2_mul(unpack_hi_half(lo), sc);
            f[w][4 * x + 2] = h2_mul(unpack_lo_half(hi), sc);
            f[w][4 * x + 3] = h2_mul(unpack_hi_half(hi), sc);
        }
    }
    // only now the operand tile has to be free: the products wait for the stores alone
    if (use > 0) wait_or_stop(smem_u32(&tiles.kv_empty[stage]), (use & 1) ^ 1, stop, p);
#pragma unroll
    for (int w = 0; w < JOBS; ++w) {
        const int job = (w * kDqWarps + dw) * 32 + lane;
        const int t = (job / (8 * PARTS)) * 8 + (job & 7);
        const int part = ((job >> 3) + (t & 7) * PARTS / 8) % PARTS;
        const uint32_t base = dst + (part / 2) * kChunk + t * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t at = base + ((((part & 1) * 4 + x) ^ (t & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(f[w][4 * x]),
                         "r"(f[w][4 * x + 1]), "r"(f[w][4 * x + 2]), "r"(f[w][4 * x + 3])
                         : "memory");
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(smem_u32(&tiles.kv_full[stage]));
        if (APART || is_v) mbar_arrive(smem_u32(&tiles.pk_empty[pk]));
    }
}

// Packed pages into the ring, by one warp: all of a CTA's segments (any: there are some).
__device__ __forceinline__ void load_pages(const ChunkParams& p, TileBars& tiles, Walk& walk, uint32_t packed_s, int packed_bytes,
                                           bool any, volatile int* stop) {
    const int lane = threadIdx.x & 31;
    uint32_t n_pk = 0, n_copied = 0;
    const int per = kTile >> p.lg_p;  // pages of a tile
    const Segment& g = walk.g;
    while (any && walk.next(p)) {
        const int pages = (max(g.vis, 0) + (1 << p.lg_p) - 1) >> p.lg_p;  // the item's
        const int32_t* table = p.block_table + static_cast<long long>(g.b) * p.max_blocks;
        int base = g.k0 * per;  // lane l holds page base + l, and the one 32 later
        auto look = [&](int at) -> int { return at < pages ? __ldg(table + at) : 0; };
        int cur = look(base + lane), nxt = look(base + 32 + lane);
        for (int i = g.k0; i < g.k1; ++i, ++n_pk) {
            const uint32_t pk = n_pk % kPacked;
            if (n_pk >= kPacked)
                wait_or_stop(smem_u32(&tiles.pk_empty[pk]), ((n_pk / kPacked) & 1) ^ 1, stop, p);
            const int first = i * per;
            if (first - base >= 32) {
                base += 32;
                cur = nxt;
                nxt = look(base + 32 + lane);
            }
            const int count = max(0, min(per, pages - first));
            const uint32_t bar = smem_u32(&tiles.pk_full[pk]);
            const bool go = !__shfl_sync(0xffffffffu, *stop, 0);  // one answer: what is announced is copied
            if (go) n_copied = n_pk + 1;
            if (lane == 0 && go) {
                if (count > 0) mbar_arrive_expect_tx(bar, count * p.L.bytes);
                else mbar_arrive(bar);
            }
            __syncwarp();
            int page = __shfl_sync(0xffffffffu, cur, (first - base + lane) & 31);
            if (lane < count && go) {
                if (page < 0 || page >= p.num_pages) {
                    raise_flag(p.status, KVQ_FLAG_BAD_PAGE);
                    page = 0;
                }
                bulk_g2s(packed_s + pk * packed_bytes + lane * p.L.bytes,
                         p.pool + (static_cast<long long>(page) * p.Hkv + g.h) * p.L.bytes, p.L.bytes, bar);
            }
            __syncwarp();
        }
    }
    // No copy of this CTA may be in flight when it leaves.  (Given up: of the tiles that were copied, whose phases
    // alone tell the last copies apart from those before)
    for (uint32_t i = n_copied > kPacked ? n_copied - kPacked : 0; i < n_copied; ++i)
        mbar_wait(smem_u32(&tiles.pk_full[i % kPacked]), (i / kPacked) & 1, kWaitNs);
}

// Chunk attention where a sequence has few lines (rows times the query heads of a kv head): chunk_few.cu.
// Lines of an item: 16 or 32.
cudaError_t launch_chunk_few(ChunkParams p, int head_dim, int lines, int ctas, cudaStream_t stream);

}  // namespace kvq
