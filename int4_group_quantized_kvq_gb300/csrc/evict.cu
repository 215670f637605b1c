// evict.cu -- eviction from a paged cache by accumulated attention weight: the choice of the
// positions each kv head keeps, and the move of their rows to the front of the sequence.
//
// Neither kernel signals its dependents early: the lengths and the pool they write may be the
// inputs that the next decode call reads before its own wait.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// Select
// ---------------------------------------------------------------------------
// A weight as an unsigned key of the same order: NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

constexpr int kSelectThreads = 1024;

// One CTA per (sequence, kv head).  Of n > keep positions the first `sinks` and the last
// `recent` stay, and of those between, the k = keep - sinks - recent of largest weight: a
// radix descent over the keys finds the k-th largest T and how many keys equal to T belong
// (four passes, a histogram of 8 bits each), then one pass in position order writes the
// positions with key > T and the first ones with key == T.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(EvictSelectArgs p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ uint32_t s_gt[32], s_eq[32];
    const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = p.seq_lens[b];
    n = n < 0 ? 0 : n;
    if (n > p.max_len) {
        n = p.max_len;
        if (h == 0 && tid == 0) raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
    }
    if (h == 0 && tid == 0) p.new_lens[b] = min(n, p.keep);
    const float* w = p.weights + static_cast<long long>(blockIdx.x) * p.weights_ld;
    int32_t* kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
    if (n <= p.keep) {
        for (int i = tid; i < p.keep; i += kSelectThreads) kept[i] = i < n ? i : -1;
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;
    const int k = p.keep - p.sinks - p.recent;
    for (int i = tid; i < lo; i += kSelectThreads) kept[i] = i;
    for (int i = tid; i < p.recent; i += kSelectThreads) kept[lo + k + i] = hi + i;
    if (k == 0) return;

    uint32_t prefix = 0, left = static_cast<uint32_t>(k);
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t above = shift == 24 ? 0u : ~0u << (shift + 8);
        for (int t = lo + tid; t < hi; t += kSelectThreads) {
            const uint32_t key = weight_key(w[t]);
            if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8 l down to 248 - 8 l; the digit where the count from
            // the top reaches `left`
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
            uint32_t before = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += y;
            }
            before -= sum;
            if (before < left && before + sum >= left) {
                uint32_t need = left - before;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (need > 0 && need <= c[j]) {
                        s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - j) << shift);
                        s_left = need;
                        need = 0;
                    } else if (need > 0) {
                        need -= c[j];
                    }
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }

    // in position order: keys above T, and the first `left` equal to it
    uint32_t gt_done = 0, eq_done = 0;
    for (int t0 = lo; t0 < hi; t0 += kSelectThreads) {
        const int t = t0 + tid;
        const uint32_t key = t < hi ? weight_key(w[t]) : 0u;
        const bool gt = t < hi && key > prefix, eq = t < hi && key == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_gt[warp] = __popc(mg);
            s_eq[warp] = __popc(me);
        }
        __syncthreads();
        uint32_t bg = gt_done, be = eq_done, ag = 0, ae = 0;
        for (int v = 0; v < 32; ++v) {
            const uint32_t xg = s_gt[v], xe = s_eq[v];
            if (v < warp) {
                bg += xg;
                be += xe;
            }
            ag += xg;
            ae += xe;
        }
        const uint32_t below = (1u << lane) - 1u;
        bg += __popc(mg & below);
        be += __popc(me & below);
        if (gt || (eq && be < left)) kept[lo + bg + min(be, left)] = t;
        gt_done += ag;
        eq_done += ae;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 512;
constexpr int kCompactRows = 64;  // rows moved together

// One CTA per (sequence, kv head), kCompactRows rows at a time through shared memory: every
// row of the chunk is read before one is written.  The kept positions ascend, so kept[i] >= i
// and a chunk's writes (positions below its own end) never reach a row that a later chunk
// still has to read; in place and other pages are one path.
__global__ void __launch_bounds__(kCompactThreads) evict_compact_kernel(EvictCompactArgs p) {
    extern __shared__ __align__(16) uint8_t buf[];
    __shared__ long long s_src[kCompactRows], s_dst[kCompactRows];
    __shared__ float s_w[kCompactRows];
    const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
    const int tid = threadIdx.x;
    const int P = 1 << p.lg_p;
    const bool first = h == 0 && tid == 0;
    long long n = p.seq_lens[b];
    n = n < 0 ? 0 : n;
    long long cap = static_cast<long long>(p.max_blocks) << p.lg_p;
    if (p.weights && cap > p.weights_ld) cap = p.weights_ld;
    if (n > cap) {
        n = cap;
        if (first) raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
    }
    const int m = static_cast<int>(min(n, static_cast<long long>(p.keep)));
    const int32_t* kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
    float* w = p.weights ? p.weights + static_cast<long long>(blockIdx.x) * p.weights_ld : nullptr;
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.max_blocks;
    const int32_t* dtable = p.dst_table + static_cast<long long>(b) * p.dst_max_blocks;
    int row = 0;
    for (int i = 0; i < 4; ++i) row += p.row_bytes[i];
    const int row_pad = (row + 15) & ~15;
    for (int i0 = 0; i0 < m; i0 += kCompactRows) {
        const int rows = min(kCompactRows, m - i0);
        if (tid < rows) {
            const int i = i0 + tid, t = kept[i];
            long long src = -1, dst = -1;
            float x = 0.f;
            if (t < 0 || t >= n || (i >> p.lg_p) >= p.dst_max_blocks) {
                raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
            } else {
                const int sp = table[t >> p.lg_p], dp = dtable[i >> p.lg_p];
                if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) {
                    raise_flag(p.status, KVQ_FLAG_BAD_PAGE);
                } else if (sp != dp || (t & (P - 1)) != (i & (P - 1))) {
                    src = ((static_cast<long long>(sp) * p.Hkv + h) << 6) | (t & (P - 1));
                    dst = ((static_cast<long long>(dp) * p.Hkv + h) << 6) | (i & (P - 1));
                }
                if (w) x = w[t];
            }
            s_src[tid] = src;
            s_dst[tid] = dst;
            s_w[tid] = x;
        }
        __syncthreads();
        // codes in 16-byte words, scales in 2-byte ones
        for (int pass = 0; pass < 2; ++pass) {
            int off = 0;
            for (int sec = 0; sec < 4; ++sec) {
                const int rb = p.row_bytes[sec];
                const int unit = sec < 2 ? 16 : 2;
                const int words = rb / unit;
                for (int e = tid; e < rows * words; e += kCompactThreads) {
                    const int rr = e / words, ww = e - rr * words;
                    const long long at = pass == 0 ? s_src[rr] : s_dst[rr];
                    if (at < 0) continue;
                    uint8_t* g = p.pool + (at >> 6) * p.block_bytes + p.sec_off[sec] + (at & 63) * rb + ww * unit;
                    uint8_t* s = buf + rr * row_pad + off + ww * unit;
                    if (unit == 16) {
                        if (pass == 0) *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(g);
                        else *reinterpret_cast<uint4*>(g) = *reinterpret_cast<const uint4*>(s);
                    } else {
                        if (pass == 0) *reinterpret_cast<uint16_t*>(s) = *reinterpret_cast<const uint16_t*>(g);
                        else *reinterpret_cast<uint16_t*>(g) = *reinterpret_cast<const uint16_t*>(s);
                    }
                }
                off += rb;
            }
            if (pass == 0) __syncthreads();
        }
        if (w && tid < rows) w[i0 + tid] = s_w[tid];
        __syncthreads();
    }
    if (w)
        for (long long i = m + tid; i < n; i += kCompactThreads) w[i] = 0.f;
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs& a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv;
    if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    evict_select_kernel<<<static_cast<unsigned>(rows), kSelectThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_evict_compact(const EvictCompactArgs& a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv;
    if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    int row = 0;
    for (int i = 0; i < 4; ++i) row += a.row_bytes[i];
    const int smem = kCompactRows * ((row + 15) & ~15);
    evict_compact_kernel<<<static_cast<unsigned>(rows), kCompactThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvq
