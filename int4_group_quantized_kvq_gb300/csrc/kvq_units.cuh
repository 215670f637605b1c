// kvq_units.cuh -- how the attention kernels over ragged batches of rows share their work out: equal runs
// of units per CTA, items cut between CTAs, and where their partial results meet.
//
// A sequence has n rows (the last n of its len positions), each of per_row lines (query heads that read
// one key/value head, where the kernel's items are counted in those); an item is `step` lines of one
// (sequence, key/value head), and a unit one tile of 128 positions that an item attends to.  The list of
// units is ordered (sequence, head, item, tile).
#pragma once

#include <cstdint>

#include "kvq_device.cuh"

namespace kvq {

constexpr int kTile = 128;     // positions of a tile
constexpr int kItemUnits = 2;  // what an item costs a CTA besides its tiles (queries in, output out), in units

// A softmax weight is 2^(z + kUp), z the score in powers of two less a reference: the running maximum, which is
// followed when a score exceeds it by more than kLag (outputs are rescaled a few times a row instead of every tile).
// The largest weight of a row lies in [2^kUp, 2^(kUp + kLag)], inside f16; those down to 2^-21 of the largest keep 11
// bits, those down to 2^-32 some.  (At kUp 0 all below 2^-25 were lost, while the sum that divides held them; the time
// is the same.  A closer reference leaves more bits and costs rescalings: kLag 4 and kUp 11 took 628 us instead of
// 608 for a prompt of 8192 tokens and 86 instead of 80 for drafts over 32761 positions)
constexpr float kUp = 7.f, kLag = 8.f;

// Where a CTA's run of units starts, and how long it is.
struct Start {
    int b, h, j, k;
    long long units;
};

// Merging of an item whose units lie in several CTAs, described by the CTA of its second part.
struct MergeDesc {
    int32_t parts;  // 0: nothing to merge
    int32_t line0, lines, h;  // line0 counts all rows' lines
};

struct Units {
    const int32_t* seq_lens;
    const int32_t* cu_rows;
    uint32_t* status;
    MergeDesc* desc;  // [gridDim.x]
    int32_t rows, B, heads, per_row, step;
    int32_t most;      // the longest sequence
    uint32_t wait_ns;  // bound of every wait
    // A test of that bound: 1 adds an arrival that nobody makes to what an operand tile's barrier waits for
    uint32_t withheld;
};

struct Seq {
    int row0, n, len;  // first row, rows, positions
};
__device__ __forceinline__ Seq sequence(const Units& p, int b) {
    Seq s;
    const int c0 = min(max(__ldg(p.cu_rows + b), 0), p.rows), c1 = min(max(__ldg(p.cu_rows + b + 1), 0), p.rows);
    s.row0 = c0;
    s.n = max(0, c1 - c0);
    s.len = min(max(__ldg(p.seq_lens + b), 0), p.most);
    return s;
}
// (rows times lines are below 2^31)
__device__ __forceinline__ uint32_t lines_of(const Units& p, const Seq& s) { return static_cast<uint32_t>(s.n) * p.per_row; }
// Positions the last line of item j can see, and the item's tiles (one at least: rows that see nothing
// are written too).
__device__ __forceinline__ int visible(const Units& p, const Seq& s, uint32_t j) {
    uint32_t end = min((j + 1) * p.step, lines_of(p, s));
    if (p.per_row != 1) end = (end + p.per_row - 1) / p.per_row;
    return s.len - s.n + static_cast<int>(end);
}
__device__ __forceinline__ int tiles_of(int vis) { return max(1, (vis + kTile - 1) / kTile); }

// A segment: the tiles [k0, k1) of one item.
struct Segment {
    int b, h, k0, k1, nt, vis;
    int line0, lines;  // within the sequence
    int row0, ahead;   // the sequence's first row, and positions before that row's
};

// Walks a CTA's segments; every role walks the same ones.  The state lies in shared memory, a copy for
// each warp: kept in registers it would cost each two dozen.
struct Walk {
    long long left;
    int b, h, j, k;
    Seq s;
    Segment g;
    __device__ __forceinline__ void begin(const Units& p, const Start& st) {
        left = st.units;
        b = st.b;
        h = st.h;
        j = st.j;
        k = st.k;
        s = sequence(p, b);
        __syncwarp();
    }
    __device__ __forceinline__ bool next(const Units& p) {
        __syncwarp();
        long long room = left;
        int cj = j, ch = h, cb = b;
        const int ck = k;
        Seq cs = s;
        if (room <= 0) return false;
        if (static_cast<uint32_t>(cj) * p.step >= lines_of(p, cs)) {  // the next head or sequence
            cj = 0;
            if (++ch == p.heads) {
                ch = 0;
                do {
                    if (++cb >= p.B) return false;
                    cs = sequence(p, cb);
                } while (cs.n == 0);
            }
        }
        const int vis = visible(p, cs, cj), nt = tiles_of(vis);
        if (ck == 0) room -= kItemUnits;
        const int k1 = static_cast<int>(min(static_cast<long long>(nt), ck + room));
        __syncwarp();
        if (k1 <= ck) {  // not a tile of it
            left = 0;
            return false;
        }
        const int line0 = cj * p.step;
        g = Segment{cb, ch, ck, k1, nt, vis, line0, min(p.step, static_cast<int>(lines_of(p, cs)) - line0), cs.row0,
                    cs.len - cs.n};
        left = room - (k1 - ck);
        k = 0;
        j = cj + 1;
        h = ch;
        b = cb;
        s = cs;
        __syncwarp();
        return true;
    }
};

// c U / C (in 32 bits where that is enough: a 64-bit division takes a microsecond's fifth).
__device__ __forceinline__ long long slice(long long c, long long U, long long C) {
    if (U < (1 << 23) && C < 512) return static_cast<uint32_t>(c) * static_cast<uint32_t>(U) / static_cast<uint32_t>(C);
    return c * U / C;
}

// The CTA's run of units: all threads (with barriers of the CTA).  A thread counts the units of a sequence
// per head.  warp_sum: THREADS / 32 numbers in shared memory.
template <int THREADS>
__device__ __forceinline__ void find_start(const Units& p, Start* start, long long* warp_sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const long long cta = blockIdx.x;
    auto count = [&](int b) -> long long {
        if (b >= p.B) return 0;
        const Seq s = sequence(p, b);
        long long u = 0;
        for (uint32_t j = 0; j * p.step < lines_of(p, s); ++j) u += tiles_of(visible(p, s, j)) + kItemUnits;
        if (u > 0 && blockIdx.x == 0 && __ldg(p.seq_lens + b) > p.most) raise_flag(p.status, KVQ_FLAG_BAD_POSITION);
        return u * p.heads;
    };
    long long mine = 0, first = 0;
    for (int b = tid; b < p.B; b += THREADS) {
        const long long u = count(b);
        if (b == tid) first = u;
        mine += u;
    }
    if (tid == 0) {
        *start = Start{0, 0, 0, 0, 0};
        p.desc[cta].parts = 0;
    }
    auto block_scan = [&](long long v, long long& total) -> long long {  // inclusive
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += t;
        }
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll 4
        for (int w = 0; w < THREADS / 32; ++w) {
            const long long t = warp_sum[w];
            if (w < warp) before += t;
            total += t;
        }
        return v + before;
    };
    long long U;
    long long incl = block_scan(mine, U);
    const long long C = min(static_cast<long long>(gridDim.x), U);
    if (cta >= C) return;  // (the whole CTA)
    const long long u0 = slice(cta, U, C), u1 = slice(cta + 1, U, C);
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const long long v = b0 == 0 ? first : count(b0 + tid);
        if (p.B > THREADS) {  // (else the first scan has it)
            long long total;
            __syncthreads();
            incl = base + block_scan(v, total);
            base += total;
        }
        const long long excl = incl - v;
        if (u0 >= excl && u0 < incl) {  // one thread
            const int b = b0 + tid;
            const Seq s = sequence(p, b);
            int h = 0;
            long long rem = u0 - excl;
            if (p.heads > 1) {
                const long long per = v / p.heads;
                h = static_cast<int>(rem < (1ll << 31) ? static_cast<uint32_t>(rem) / static_cast<uint32_t>(per) : rem / per);
                rem -= h * per;
            }
            int j = 0, nt;
            while (true) {
                nt = tiles_of(visible(p, s, j));
                if (rem < nt + kItemUnits) break;
                rem -= nt + kItemUnits;
                ++j;
            }
            // a boundary within an item's first kItemUnits leaves all its tiles to this CTA
            const long long i0 = u0 - rem + kItemUnits;  // where the item's tiles start in the list
            const int k = static_cast<int>(max(0ll, u0 - i0));
            *start = Start{b, h, j, k, u1 - (k > 0 ? u0 : i0 - kItemUnits)};
            // this CTA starts inside an item: is its part the item's second one?
            if (k > 0 && slice(cta - 1, U, C) <= i0) {
                // the CTAs that start before the item's end (an estimate, and at most a step or two from it)
                long long c = cta + 1;
                if (U < (1 << 23) && C < 512) c = max(c, static_cast<long long>(static_cast<uint32_t>(i0 + nt) * static_cast<uint32_t>(C) / static_cast<uint32_t>(U)));
                while (c > cta + 1 && slice(c - 1, U, C) >= i0 + nt) --c;
                while (c < C && slice(c, U, C) < i0 + nt) ++c;
                p.desc[cta] = MergeDesc{static_cast<int>(c - cta) + 1, s.row0 * p.per_row + j * p.step,
                                        min(p.step, static_cast<int>(lines_of(p, s)) - j * p.step), h};
            }
        }
        if (base > u0) break;
    }
    __syncthreads();
}

// The slot of a CTA's partial result of a segment: slot 0 where it starts inside an item, else slot 1 (its
// last segment).  The parts of a cut item are slot 1 of the CTA ahead of the descriptor's and slot 0 of
// the descriptor's and those behind it.
__device__ __forceinline__ int partial_slot(const Segment& g) { return 2 * blockIdx.x + (g.k0 == 0 ? 1 : 0); }

constexpr int kMaxCtas = 256;  // of an attention grid

// The merges of a call, shared out over a grid of 256-thread CTAs in pieces of 128 dimensions of a line: a
// warp merges a piece of an item of few parts, a CTA one of many (its warps take the parts in turn).
// `first` counts the units of work ahead of each descriptor's: eight pieces, or one.
struct MergeShare {
    int first[kMaxCtas + 1];
    int warp_sum[8];
    float ml[8][2];
    float4 sums[8][32];
};
constexpr int kFewParts = 8;

// A line has E pieces, four dimensions of one to a lane.  fetch(slot, line, e, m, l, o, lane) reads a part,
// put(desc, line, e, l, o, lane) writes what is merged; lines: `mult` times the descriptor's.  c: a maximum's factor
// to powers of two, which the difference of two maxima takes (that is exact or nearly, however large they are).
template <int E, class FETCH, class PUT>
__device__ __forceinline__ void merge_items(const Units& p, float c, int ctas, int mult, MergeShare* share, FETCH fetch, PUT put) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    int mine = 0;
    if (tid < ctas) {
        const MergeDesc d = p.desc[tid];
        if (d.parts > 0) mine = d.parts > kFewParts ? d.lines * mult * E : (d.lines * mult * E + 7) / 8;
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
    }
    if (lane == 31) share->warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += share->warp_sum[w];
    share->first[tid] = incl - mine;
    if (tid == 255) share->first[256] = incl;
    __syncthreads();
    const int total = share->first[256];
    auto add = [&](float& m, float& l, float4& o, float mk, float lk, const float4& ok) {
        const float mn = fmaxf(m, mk), at = mn == -INFINITY ? 0.f : mn;  // (a part that saw nothing: weight 0)
        const float a = fast_exp2((m - at) * c), ak = fast_exp2((mk - at) * c);
        l = l * a + lk * ak;
        o.x = o.x * a + ok.x * ak;
        o.y = o.y * a + ok.y * ak;
        o.z = o.z * a + ok.z * ak;
        o.w = o.w * a + ok.w * ak;
        m = mn;
    };
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int lo = 0, hi = 255;  // the last descriptor whose units start at or before u: it has some
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (share->first[mid] <= u) lo = mid;
            else hi = mid - 1;
        }
        const MergeDesc d = p.desc[lo];
        const bool wide = d.parts > kFewParts;
        const int piece = wide ? u - share->first[lo] : (u - share->first[lo]) * 8 + warp;
        const int line = piece / E, e = piece - line * E;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (line < d.lines * mult) {
#pragma unroll 4
            for (int k = wide ? warp : 0; k < d.parts; k += wide ? 8 : 1) {
                float mk, lk;
                float4 ok;
                fetch(k == 0 ? 2 * (lo - 1) + 1 : 2 * (lo + k - 1), line, e, mk, lk, ok, lane);
                add(m, l, o, mk, lk, ok);
            }
            if (!wide) put(d, line, e, l, o, lane);
        }
        if (!wide) continue;
        share->sums[warp][lane] = o;
        if (lane == 0) {
            share->ml[warp][0] = m;
            share->ml[warp][1] = l;
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < 8; ++w) add(m, l, o, share->ml[w][0], share->ml[w][1], share->sums[w][lane]);
            put(d, line, e, l, o, lane);
        }
        __syncthreads();
    }
}

}  // namespace kvq
