// evict.cu -- eviction from a paged cache by accumulated attention weight: the choice of the
// positions each kv head keeps, and the move of their rows to the front of the sequence.
//
// Both kernels give one thread-block cluster to each (sequence, kv head), so that a few long
// sequences still fill the device, and are launched while the kernel ahead on the stream
// finishes (programmatic dependent launch, with a wait before anything is read).  Neither
// signals its own dependents early: the lengths and the pool they write may be the inputs
// that the next decode call reads before its own wait.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Select
// ---------------------------------------------------------------------------
// A weight as an unsigned key of the same order: NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

constexpr int kSelKeys = 8;     // keys a thread holds in registers; a longer slice is read again in each pass
constexpr int kSelBins = 2048;  // 11 bits a pass

// Of n > keep positions the first `sinks` and the last `recent` stay, and of the ones between
// (lo .. hi - 1) the k = keep - sinks - recent of largest weight.  A radix descent finds the
// k-th largest key T and how many keys equal to T belong: three passes over digits of 11, 11
// and 10 bits from the top, each a histogram of the keys that share the digits found so far.
// Then the positions with key > T and the first ones with key == T are written in order.
//
// The cluster's CTAs take equal slices of the positions.  A thread holds its keys in registers,
// read once; the CTAs' histograms are added through distributed shared memory by every CTA for
// itself, one cluster barrier per pass (a histogram per pass, so none is cleared while another
// CTA may read it).  The first digit spans sign, exponent and two mantissa bits: accumulated
// weights lie within a few binades, and with 8 bits almost all keys of a warp would meet in
// one or two counters.  Bound by latency (the chain of barriers and passes, not the bytes):
// 4 x 8 rows of 32768 positions 69.7 us a call with one CTA a row and four 8-bit passes over
// the L2, 11.5 so, 17.9 with one CTA a row and 32 keys a thread.
template <int CL, int T>
__global__ void __launch_bounds__(T) evict_select_kernel(EvictSelectArgs p) {
    constexpr int kWarps = T / 32;
    static_assert(kWarps >= kSelKeys && kWarps <= 32, "a warp per round of keys, a lane per warp");
    __shared__ __align__(16) uint32_t hist[3][kSelBins];
    __shared__ uint32_t s_warp[32], s_digit, s_left;
    __shared__ uint32_t s_gt[kSelKeys][kWarps], s_eq[kSelKeys][kWarps];
    __shared__ uint32_t s_cta[2];
    const int rank = CL > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int row = blockIdx.x / CL;
    const int h = row % p.Hkv, b = row / p.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 3 * kSelBins; i += T) hist[0][i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int n = p.seq_lens[b];
    n = n < 0 ? 0 : n;
    const bool first = h == 0 && rank == 0 && tid == 0;
    if (n > p.max_len) {
        n = p.max_len;
        if (first) raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
    }
    const float* w = p.weights + static_cast<long long>(row) * p.weights_ld;
    int32_t* kept = p.kept + static_cast<long long>(row) * p.keep;
    const int all = CL * T, me = rank * T + tid;
    if (n <= p.keep) {  // (the whole cluster)
        for (int i = me; i < p.keep; i += all) kept[i] = i < n ? i : -1;
        if (first) p.new_lens[b] = n;
        return;
    }
    if (first) p.new_lens[b] = p.keep;
    const int lo = p.sinks, hi = n - p.recent;
    const int k = p.keep - p.sinks - p.recent;
    for (int i = me; i < lo; i += all) kept[i] = i;
    for (int i = me; i < p.recent; i += all) kept[lo + k + i] = hi + i;
    if (k == 0) return;  // (the whole cluster)

    const int slice = (hi - lo + CL - 1) / CL;
    const int t0 = min(lo + rank * slice, hi), t1 = min(t0 + slice, hi);
    uint32_t key[kSelKeys];
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
        const int t = t0 + j * T + tid;
        key[j] = t < t1 ? weight_key(w[t]) : 0u;
    }
    const int rest = t0 + kSelKeys * T + tid;  // this thread's first position past its registers
    __syncthreads();

    uint32_t prefix = 0, left = static_cast<uint32_t>(k);
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const int bins = pass == 2 ? 1024 : kSelBins;
        const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);  // bits above this pass's digit start here
        auto count = [&](uint32_t x) {
            if (pass == 0 || (x >> above) == (prefix >> above)) atomicAdd(&hist[pass][(x >> shift) & (bins - 1)], 1u);
        };
#pragma unroll
        for (int j = 0; j < kSelKeys; ++j)
            if (t0 + j * T + tid < t1) count(key[j]);
        for (int t = rest; t < t1; t += T) count(weight_key(w[t]));
        if (CL > 1) cg::this_cluster().sync();
        else __syncthreads();
        // thread i holds NB bins, the i-th NB from the top; c[j] counts the j-th of them from the top
        constexpr int NB = kSelBins / T;
        uint32_t c[NB], sum = 0;
        const int top = bins - 1 - tid * NB;  // (the last pass has half as many bins: the upper threads none)
#pragma unroll
        for (int j = 0; j < NB; ++j) c[j] = 0;
        if (top > 0) {
#pragma unroll
            for (int r = 0; r < CL; ++r) {
                const uint32_t* from = CL > 1 ? cg::this_cluster().map_shared_rank(&hist[pass][0], r) : &hist[pass][0];
#pragma unroll
                for (int j = 0; j < NB; j += 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(from + top - j - 1);
                    c[j] += v.y;
                    c[j + 1] += v.x;
                }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) sum += c[j];
        }
        uint32_t before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += y;
        }
        if (lane == 31) s_warp[warp] = before;
        before -= sum;
        __syncthreads();
        uint32_t x = lane < kWarps ? s_warp[lane] : 0u;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (warp > 0) before += __shfl_sync(0xffffffffu, x, warp - 1);
        if (before < left && before + sum >= left) {  // exactly one thread
            uint32_t need = left - before;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (need > 0 && need <= c[j]) {
                    s_digit = static_cast<uint32_t>(top - j);
                    s_left = need;
                }
                need = need > c[j] ? need - c[j] : 0;
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        left = s_left;
    }

    // how many of this CTA's keys are above T and equal to it, and the same of the CTAs before it
    uint32_t g = 0, e = 0;
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
        const bool in = t0 + j * T + tid < t1;
        const uint32_t mg = __ballot_sync(0xffffffffu, in && key[j] > prefix);
        const uint32_t m2 = __ballot_sync(0xffffffffu, in && key[j] == prefix);
        if (lane == 0) {
            s_gt[j][warp] = __popc(mg);
            s_eq[j][warp] = __popc(m2);
        }
    }
    uint32_t done_gt = 0, done_eq = 0;  // before this CTA, then before the chunk being written
    if (CL > 1) {
        for (int t = rest; t < t1; t += T) {
            const uint32_t x = weight_key(w[t]);
            g += x > prefix;
            e += x == prefix;
        }
        if (tid < 2) s_cta[tid] = 0;
        __syncthreads();
        if (warp < kSelKeys && lane < kWarps) {
            g += s_gt[warp][lane];
            e += s_eq[warp][lane];
        }
        g = __reduce_add_sync(0xffffffffu, g);
        e = __reduce_add_sync(0xffffffffu, e);
        if (lane == 0 && (g | e) != 0) {
            atomicAdd(&s_cta[0], g);
            atomicAdd(&s_cta[1], e);
        }
        cg::this_cluster().sync();
        for (int r = 0; r < rank; ++r) {
            const uint32_t* from = cg::this_cluster().map_shared_rank(&s_cta[0], r);
            done_gt += from[0];
            done_eq += from[1];
        }
        // (this CTA has read the others' shared memory: the last wait below is for the rest)
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    // in position order, kSelKeys rounds of T positions at a time: an entry of
    // s_gt, s_eq counts a warp's 32 positions, entries ordered as positions are
    for (int c0 = t0;; c0 += kSelKeys * T) {
        uint32_t mg[kSelKeys], m2[kSelKeys];
#pragma unroll
        for (int j = 0; j < kSelKeys; ++j) {
            const int t = c0 + j * T + tid;
            const uint32_t x = c0 == t0 ? key[j] : (t < t1 ? weight_key(w[t]) : 0u);
            mg[j] = __ballot_sync(0xffffffffu, t < t1 && x > prefix);
            m2[j] = __ballot_sync(0xffffffffu, t < t1 && x == prefix);
            if (c0 != t0 && lane == 0) {
                s_gt[j][warp] = __popc(mg[j]);
                s_eq[j][warp] = __popc(m2[j]);
            }
        }
        __syncthreads();
        // warps 0 .. kSelKeys - 1 turn a round's counts into sums before each warp, lane order;
        // the rounds' totals are added by every thread below
        if (warp < kSelKeys) {
            uint32_t a = lane < kWarps ? s_gt[warp][lane] : 0u, q = lane < kWarps ? s_eq[warp][lane] : 0u;
            const uint32_t a0 = a, q0 = q;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t ya = __shfl_up_sync(0xffffffffu, a, off), yq = __shfl_up_sync(0xffffffffu, q, off);
                if (lane >= off) {
                    a += ya;
                    q += yq;
                }
            }
            if (lane < kWarps) {
                s_gt[warp][lane] = a - a0;
                s_eq[warp][lane] = q - q0;
            }
            if (lane == 31) {
                s_warp[warp] = a;
                s_warp[kSelKeys + warp] = q;
            }
        }
        __syncthreads();
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int j = 0; j < kSelKeys; ++j) {
            const bool gt = (mg[j] >> lane) & 1u, eq = (m2[j] >> lane) & 1u;
            const uint32_t bg = done_gt + s_gt[j][warp] + __popc(mg[j] & below);
            const uint32_t be = done_eq + s_eq[j][warp] + __popc(m2[j] & below);
            if (gt || (eq && be < left)) kept[lo + bg + min(be, left)] = c0 + j * T + tid;
            done_gt += s_warp[j];
            done_eq += s_warp[kSelKeys + j];
        }
        if (c0 + kSelKeys * T >= t1) break;
        __syncthreads();
    }
    // no CTA leaves while another may read its shared memory
    if (CL > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
constexpr int kCmpThreads = 512;
constexpr int kCmpWords = 8;      // 16-byte code words a thread holds between its loads and its stores
constexpr int kCmpMaxRows = kCmpThreads;  // rows a CTA moves in a round: one per thread

// A row's scales of one kind: 2, 4, 8 or 16 bytes, as stored.
__device__ __forceinline__ uint4 load_piece(const uint8_t* g, int bytes) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (bytes == 4) v.x = *reinterpret_cast<const uint32_t*>(g);
    else if (bytes == 2) v.x = *reinterpret_cast<const uint16_t*>(g);
    else if (bytes == 8) *reinterpret_cast<uint2*>(&v) = *reinterpret_cast<const uint2*>(g);
    else v = *reinterpret_cast<const uint4*>(g);
    return v;
}
__device__ __forceinline__ void store_piece(uint8_t* g, int bytes, const uint4& v) {
    if (bytes == 4) *reinterpret_cast<uint32_t*>(g) = v.x;
    else if (bytes == 2) *reinterpret_cast<uint16_t*>(g) = static_cast<uint16_t>(v.x);
    else if (bytes == 8) *reinterpret_cast<uint2*>(g) = make_uint2(v.x, v.y);
    else *reinterpret_cast<uint4*>(g) = v;
}

// A cluster moves the kept rows of its (sequence, kv head) in rounds: every CTA loads its share
// of the round's rows into registers, the cluster's barrier, then the stores.  Kept positions
// ascend, so kept[i] >= i: a round's stores reach only positions below the round's end, no row
// that a later round has to read, and within the round everything has been read; the move in
// place needs no second buffer, and the move into other pages is the same path.  A thread owns
// a row's lookups, scales and weight, and 16-byte words of codes across the CTA's rows, whose
// source and destination it finds in shared memory as byte offsets.  The bound is HBM: every
// row is read once (in 64-byte accesses that its 64 code bytes, not aligned to them, half fill:
// 2.2 times its bytes on 8 x 32 x 2048 rows of 134 bytes, ncu) and written once.
// One CTA per (sequence, kv head) with chunks of 64 rows through shared memory took 173 us for
// those rows (its chain of small round trips), and 332 us for 4 x 8 x 4095 of 264; so 42.7 and
// 16.7 us.
__global__ void __launch_bounds__(kCmpThreads, 2) evict_compact_kernel(EvictCompactArgs p, int32_t rows_cta, int32_t lg_w) {
    // offset of a row's K codes in the pool, where it comes from and where it goes; -1: it stays
    __shared__ long long s_src[kCmpMaxRows], s_dst[kCmpMaxRows];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
    const int row = blockIdx.x / size;
    const int h = row % p.Hkv, b = row / p.Hkv;
    const int tid = threadIdx.x;
    const int P = 1 << p.lg_p;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t* kept = p.kept + static_cast<long long>(row) * p.keep;
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.max_blocks;
    const int32_t* dtable = p.dst_table + static_cast<long long>(b) * p.dst_max_blocks;
    // this thread's row of the round at `base`: its position and its two pages, looked up a round
    // ahead (the kept list and the tables do not change); t -1: a bad entry.  Bounded by `keep`, so
    // that the first lookup does not wait for the length.
    int t_next = -1, sp_next = 0, dp_next = 0;
    auto look_up = [&](long long base) {
        const long long i = base + static_cast<long long>(rank) * rows_cta + tid;
        t_next = -1;
        if (tid >= rows_cta || i >= p.keep) return;
        const bool in = (i >> p.lg_p) < p.dst_max_blocks;
        if (in) dp_next = dtable[i >> p.lg_p];
        t_next = kept[i];
        if (!in || t_next < 0 || (t_next >> p.lg_p) >= p.max_blocks) t_next = -1;
        else sp_next = table[t_next >> p.lg_p];
    };
    look_up(0);
    long long n = p.seq_lens[b];
    n = n < 0 ? 0 : n;
    long long cap = static_cast<long long>(p.max_blocks) << p.lg_p;
    if (p.weights && cap > p.weights_ld) cap = p.weights_ld;
    if (n > cap) {
        n = cap;
        if (h == 0 && rank == 0 && tid == 0) raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
    }
    const int m = static_cast<int>(min(n, static_cast<long long>(p.keep)));
    float* w = p.weights ? p.weights + static_cast<long long>(row) * p.weights_ld : nullptr;
    // a row's code words: 2^lg_w of K, then as many of V
    const int half_mask = (1 << lg_w) - 1;
    for (long long base = 0; base < m; base += static_cast<long long>(size) * rows_cta) {
        const long long r0 = base + static_cast<long long>(rank) * rows_cta;
        const int rows = r0 < m ? static_cast<int>(min(static_cast<long long>(rows_cta), m - r0)) : 0;
        // this thread's row: its weight (0 if it is skipped) and scales, and where the scales go
        float wv = 0.f;
        uint4 ks = make_uint4(0, 0, 0, 0), vs = ks;
        uint8_t* to = nullptr;  // the destination block, or nullptr
        int to_slot = 0;
        if (tid < rows) {
            const int t = t_next, sp = sp_next, dp = dp_next;
            long long src = -1, dst = -1;
            if (t < 0 || t >= n) {
                raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
            } else {
                const int ss = t & (P - 1), ds = (static_cast<int>(r0) + tid) & (P - 1);
                const bool pages = sp >= 0 && sp < p.num_pages && dp >= 0 && dp < p.num_pages;
                if (w && pages) wv = w[t];
                if (!pages) {
                    raise_flag(p.status, KVQ_FLAG_BAD_PAGE);
                } else if (sp != dp || ss != ds) {
                    src = (static_cast<long long>(sp) * p.Hkv + h) * p.block_bytes;
                    dst = (static_cast<long long>(dp) * p.Hkv + h) * p.block_bytes;
                    const uint8_t* from = p.pool + src;
                    to = p.pool + dst;
                    to_slot = ds;
                    ks = load_piece(from + p.sec_off[2] + ss * p.row_bytes[2], p.row_bytes[2]);
                    vs = load_piece(from + p.sec_off[3] + ss * p.row_bytes[3], p.row_bytes[3]);
                    src += ss * p.row_bytes[0];
                    dst += ds * p.row_bytes[0];
                }
            }
            s_src[tid] = src;
            s_dst[tid] = dst;
        }
        __syncthreads();
        uint4 v[kCmpWords];
#pragma unroll
        for (int k = 0; k < kCmpWords; ++k) {
            const int e = tid + k * kCmpThreads, rr = e >> (lg_w + 1);
            const int off = ((e >> lg_w) & 1) * p.sec_off[1] + ((e & half_mask) << 4);
            v[k] = make_uint4(0, 0, 0, 0);
            if (rr < rows && s_src[rr] >= 0) v[k] = *reinterpret_cast<const uint4*>(p.pool + s_src[rr] + off);
        }
        look_up(base + static_cast<long long>(size) * rows_cta);
        cluster.sync();  // the round has been read
#pragma unroll
        for (int k = 0; k < kCmpWords; ++k) {
            const int e = tid + k * kCmpThreads, rr = e >> (lg_w + 1);
            const int off = ((e >> lg_w) & 1) * p.sec_off[1] + ((e & half_mask) << 4);
            if (rr < rows && s_dst[rr] >= 0) *reinterpret_cast<uint4*>(p.pool + s_dst[rr] + off) = v[k];
        }
        if (to != nullptr) {
            store_piece(to + p.sec_off[2] + to_slot * p.row_bytes[2], p.row_bytes[2], ks);
            store_piece(to + p.sec_off[3] + to_slot * p.row_bytes[3], p.row_bytes[3], vs);
        }
        if (w && tid < rows) w[r0 + tid] = wv;
        __syncthreads();
    }
    // (every round's weights have been read: the last barrier)
    if (w)
        for (long long i = m + rank * kCmpThreads + tid; i < n; i += static_cast<long long>(size) * kCmpThreads) w[i] = 0.f;
}

// A launch of `rows` clusters of `cluster` CTAs behind the kernel ahead on the stream.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), long long rows, int cluster, int threads, cudaStream_t stream,
                            Args... args) {
    if (rows * cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs& a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv;
    // Rows that 256 threads hold in registers take a CTA of that size, several to an SM.
    // Longer ones take CTAs of 1024 threads, one to an SM, and the largest cluster that leaves no
    // more of them than the 152 SMs and every thread a position.  (A cluster's CTAs have to find
    // their SMs in one GPC, so close to that bound the last clusters may start behind others.)
    if (a.max_len <= 256 * kSelKeys) return launch_clusters(evict_select_kernel<1, 256>, rows, 1, 256, stream, a);
    int cl = 1;
    while (cl < 8 && rows * cl * 2 <= 152 && a.max_len > 1024 * cl) cl *= 2;
    switch (cl) {
        case 1: return launch_clusters(evict_select_kernel<1, 1024>, rows, 1, 1024, stream, a);
        case 2: return launch_clusters(evict_select_kernel<2, 1024>, rows, 2, 1024, stream, a);
        case 4: return launch_clusters(evict_select_kernel<4, 1024>, rows, 4, 1024, stream, a);
        default: return launch_clusters(evict_select_kernel<8, 1024>, rows, 8, 1024, stream, a);
    }
}

cudaError_t launch_evict_compact(const EvictCompactArgs& a, cudaStream_t stream) {
    // rows a CTA holds: its threads' code words over a row's (K and V, 16 bytes each)
    int lg_w = 0;
    while ((16 << lg_w) < a.row_bytes[0]) ++lg_w;
    const int rows_cta = std::min((kCmpThreads * kCmpWords) >> (lg_w + 1), kCmpMaxRows);
    // the smallest cluster that moves a sequence in one round, at most 8 (the portable size)
    int cl = 1;
    while (cl < 8 && cl * rows_cta < a.keep) cl *= 2;
    return launch_clusters(evict_compact_kernel, static_cast<long long>(a.B) * a.Hkv, cl, kCmpThreads, stream, a,
                           static_cast<int32_t>(rows_cta), static_cast<int32_t>(lg_w));
}

}  // namespace kvq
