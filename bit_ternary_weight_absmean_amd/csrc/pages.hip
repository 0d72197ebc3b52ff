// The pages of a cache: giving sequences pages for new tokens, sharing and dropping them, bringing the pages in use
// together, and copying pages (bt_pages_grow, _fork, _compact, _copy).
//
// State: table [B, W] (the pages of each sequence, in order; -1 behind them), length [B] in tokens, refs [P] (how many
// tables hold a page; 0: free) and a bound `first` below which every page is in use. All of it is on the device and
// read there, so that a step that changes it can be captured and replayed. Every entry taken from it or from the
// caller's lists is checked against the arrays before it is used as an index.
//
// Determinism: free pages are taken lowest index first, in the order of the sequences; the only atomics add and take
// minima of integers, whose order does not matter. Counts rise in one launch and fall in a later one (fork), so a
// page is seen to reach 0 exactly when it is free.
//
// Bound by launches and, where pages are copied, by their bytes (each read once and written once).
#include "bt_internal.h"
#include "pages.h"
#include "wave.h"

namespace bt {
namespace {

constexpr int kPlan = 1024;         // threads of the one workgroup that hands out pages
constexpr int kPlanWaves = kPlan / 64;
constexpr int kCopyBytes = 16384;   // of a page, by one workgroup at a time

__device__ inline int pages_for(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }
__device__ inline int rank_in(uint64_t mask) { return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0)); }

struct Range {
    int from, n;
};
// The new tokens of sequence b, kept inside [0, T) whatever the offsets say.
__device__ inline Range new_tokens(const PagesArgs &a, int b)
{
    const int from = min(max(a.q_start[b], 0), a.T);
    return {from, min(max(a.q_start[b + 1], from), a.T) - from};
}

__device__ inline int length_of(const PagesArgs &a, int b)
{
    return (int)min((int64_t)max(a.length[b], 0), (int64_t)a.W << a.page_shift);
}

// Sum over the workgroup of v, and the sum over the threads before this one.
__device__ inline int block_scan(int v, int *lds, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(sum, d);
        sum += lane >= d ? up : 0;
    }
    __syncthreads();  // lds may still be read from before
    if (lane == 63)
        lds[wave] = sum;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        before += w < wave ? lds[w] : 0;
        total += lds[w];
    }
    return before + sum - v;
}

// Copies 16 * n16 bytes of page src to page dst in every layer: task i of count * layers * pieces.
__device__ inline void copy_piece(const PagesArgs &a, int64_t src, int64_t dst, int layer, int piece)
{
    const char *from = a.pool + layer * a.layer_stride + src * a.page_bytes;
    char *to = a.pool + layer * a.layer_stride + dst * a.page_bytes;
    const int64_t lo = (int64_t)piece * kCopyBytes, hi = min(lo + kCopyBytes, a.page_bytes);
    constexpr int U = kCopyBytes / 16 / 256;
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = lo + (u * 256 + threadIdx.x) * 16;
        if (at < hi)
            x[u] = *reinterpret_cast<const uint4 *>(from + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = lo + (u * 256 + threadIdx.x) * 16;
        if (at < hi)
            *reinterpret_cast<uint4 *>(to + at) = x[u];
    }
}

template <typename Pair>
__device__ inline void copy_pages(const PagesArgs &a, int64_t count, Pair pair)
{
    const int pieces = (int)((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
    const int64_t per = (int64_t)a.layers * pieces;
    for (int64_t task = blockIdx.x; task < count * per; task += gridDim.x) {
        const int64_t i = task / per;
        const int rest = (int)(task % per);
        int64_t src, dst;
        if (pair(i, src, dst))
            copy_piece(a, src, dst, rest / pieces, rest % pieces);
    }
}

unsigned copy_grid(const PagesArgs &a, int64_t count)
{
    const int64_t tasks = count * a.layers * ((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
    return (unsigned)(tasks < 1 ? 1 : tasks > 4096 ? 4096 : tasks);
}

// ---------------------------------------------------------------------------------- grow
//
// Workspace: [0] pages handed out, [1] pages copied, then per sequence the end of its demand (inclusive sum) and
// the page slot it starts at, then the list of copied pages (from, to), then the free pages.

struct GrowSpace {
    int *counts, *end, *slot, *from, *to, *free;
};
__device__ __host__ inline GrowSpace grow_space(int *ws, int64_t B)
{
    return {ws, ws + 4, ws + 4 + B, ws + 4 + 2 * B, ws + 4 + 3 * B, ws + 4 + 4 * B};
}

__global__ __launch_bounds__(kPlan) void k_pages_plan(PagesArgs a)
{
    __shared__ int lds[kPlanWaves];
    __shared__ int freed;
    const GrowSpace ws = grow_space(a.ws, a.B);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    if (tid == 0)
        freed = a.P;
    // what every sequence needs
    int asked = 0;
    for (int c = 0; c < a.B; c += kPlan) {
        const int b = c + tid;
        int need = 0, slot = -1;
        if (b < a.B) {
            const int n = new_tokens(a, b).n, len = length_of(a, b);
            const int have = pages_for(len, a.page_shift), want = pages_for((int64_t)len + n, a.page_shift);
            if (n > 0 && want <= a.W) {
                bool copy = false;
                if (len & ((1 << a.page_shift) - 1)) {
                    const int tail = a.table[(int64_t)b * a.W + have - 1];
                    copy = tail >= 0 && tail < a.P && a.refs[tail] > 1;
                }
                need = want - have + copy;
                slot = have - copy;
            }
        }
        int total;
        const int before = block_scan(need, lds, total);
        if (b < a.B) {
            ws.end[b] = asked + before + need;
            ws.slot[b] = slot;
        }
        asked += total;
    }
    // the first `asked` free pages
    constexpr int kPer = 8, kStep = kPlan * kPer;
    int found = 0, base = asked > 0 ? min(max(*a.first, 0), a.P) : a.P;
    for (; base < a.P && found < asked; base += kStep) {
        const int mine = base + wave * 64 * kPer;
        uint64_t free[kPer];
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int page = mine + i * 64 + lane;
            free[i] = __ballot(page < a.P && a.refs[page] == 0);
            n += __popcll(free[i]);
        }
        __syncthreads();
        if (lane == 0)
            lds[wave] = n;
        __syncthreads();
        int at = found;
        for (int w = 0; w < kPlanWaves; ++w) {
            at += w < wave ? lds[w] : 0;
            found += lds[w];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = at + rank_in(free[i]);
            if ((free[i] >> lane & 1) && k < asked)
                ws.free[k] = mine + i * 64 + lane;
            at += __popcll(free[i]);
        }
    }
    __syncthreads();  // the lists, for all of the workgroup
    // who gets them: those whose demand ends within what was found
    int taken = 0, copies = 0;
    for (int c = 0; c < a.B; c += kPlan) {
        const int b = c + tid;
        int need = 0, copy = 0, from = 0, to = 0;
        if (b < a.B) {
            const int end = ws.end[b], slot = ws.slot[b], n = new_tokens(a, b).n;
            need = end - (b ? ws.end[b - 1] : 0);
            const bool fits = slot >= 0 && (need == 0 || end <= found);
            a.granted[b] = fits ? n : 0;
            if (fits) {
                const int len = length_of(a, b);
                copy = slot < pages_for(len, a.page_shift);
                if (copy) {
                    from = a.table[(int64_t)b * a.W + slot];
                    to = ws.free[end - need];
                    if (atomicSub(a.refs + from, 1) == 1)
                        atomicMin(&freed, from);
                }
                a.length[b] = len + n;
            } else {
                ws.slot[b] = -1;
                need = 0;
            }
        }
        int total;
        const int at = copies + block_scan(copy, lds, total);
        if (copy) {
            ws.from[at] = from;
            ws.to[at] = to;
        }
        copies += total;
        block_scan(need, lds, total);
        taken += total;
    }
    __syncthreads();
    if (tid == 0) {
        ws.counts[0] = taken;
        ws.counts[1] = copies;
        if (asked > 0) {
            const int next = taken > 0 ? ws.free[taken - 1] + 1 : found > 0 ? ws.free[0] : a.P;
            *a.first = min(next, freed);
        }
    }
}

// First index i in [0, n) with x[i] > v (n: none); x does not fall.
__device__ inline int first_above(const int *x, int n, int v)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (x[mid] > v)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__global__ __launch_bounds__(256) void k_pages_grow(PagesArgs a)
{
    const GrowSpace ws = grow_space(a.ws, a.B);
    const int taken = ws.counts[0], copies = ws.counts[1];
    const int id = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
    for (int k = id; k < taken; k += step) {
        const int b = first_above(ws.end, a.B, k);
        if (b >= a.B)
            continue;
        const int start = b ? ws.end[b - 1] : 0, page = ws.free[k];
        a.table[(int64_t)b * a.W + ws.slot[b] + k - start] = page;
        a.refs[page] = 1;
    }
    const int mask = (1 << a.page_shift) - 1;
    for (int t = id; t < a.T; t += step) {
        const int b = first_above(a.q_start + 1, a.B, t);
        int row = -1, at = -1;
        if (b < a.B) {
            const Range r = new_tokens(a, b);
            if (t >= r.from && t < r.from + r.n) {
                at = length_of(a, b) - a.granted[b] + t - r.from;
                const int slot = ws.slot[b];
                if (slot >= 0) {
                    const int p = at >> a.page_shift, start = b ? ws.end[b - 1] : 0;
                    // what this launch writes to the table is taken from the list
                    const int page = p >= slot && start + p - slot < ws.end[b] ? ws.free[start + p - slot]
                                                                              : a.table[(int64_t)b * a.W + p];
                    row = page < 0 ? -1 : page << a.page_shift | (at & mask);
                }
            }
        }
        a.rows[t] = row;
        a.positions[t] = at;
    }
    copy_pages(a, copies, [&](int64_t i, int64_t &src, int64_t &dst) {
        src = ws.from[i];
        dst = ws.to[i];
        return true;
    });
}

// ---------------------------------------------------------------------------------- fork
//
// One workgroup per sequence. First launch: the rows as they will be, from the parents' rows as they are, and the
// counts up. Second: the counts of what a sequence held down, and its new row.
// Workspace: the new lengths, the new rows.

__device__ inline bool fork_source(const PagesArgs &a, int b, int &p)
{
    p = a.parent[b];
    return p >= 0 && p < a.B;
}

__global__ __launch_bounds__(256) void k_fork_take(PagesArgs a)
{
    const int b = blockIdx.x;
    int p;
    const bool from = fork_source(a, b, p);
    if (from && p == b)
        return;
    const int len = from ? length_of(a, p) : 0, n = pages_for(len, a.page_shift);
    int *rows = a.ws + a.B + (int64_t)b * a.W;
    for (int i = threadIdx.x; i < n; i += 256) {
        const int page = a.table[(int64_t)p * a.W + i];
        rows[i] = page;
        if (page >= 0 && page < a.P)
            atomicAdd(a.refs + page, 1);
    }
    if (threadIdx.x == 0)
        a.ws[b] = len;
}

__global__ __launch_bounds__(256) void k_fork_give(PagesArgs a)
{
    const int b = blockIdx.x;
    int p;
    if (fork_source(a, b, p) && p == b)
        return;
    const int old = pages_for(length_of(a, b), a.page_shift), len = a.ws[b], n = pages_for(len, a.page_shift);
    const int *rows = a.ws + a.B + (int64_t)b * a.W;
    int *table = a.table + (int64_t)b * a.W;
    for (int i = threadIdx.x; i < max(old, n); i += 256) {
        if (i < old) {
            const int page = table[i];
            if (page >= 0 && page < a.P && atomicSub(a.refs + page, 1) == 1)
                atomicMin(a.first, page);
        }
        table[i] = i < n ? rows[i] : -1;
    }
    __syncthreads();  // all have read the length
    if (threadIdx.x == 0)
        a.length[b] = len;
}

// ------------------------------------------------------------------------------- compact
//
// With L pages in use, the k-th one at or past L goes to the k-th free one below L. A page in use has a rank (how
// many are in use before it), a free page i has i - rank free ones before it: segments of pages need no more than
// the counts of those before them. The pages that move are those with the last ranks.
// Workspace: [0] L, [1] moves, then counts of the segments, then for each free page below L (in order) its index, for
// each rank its page (those that move), for each page its rank (those that move; -1).

constexpr int kSegment = 4096;

struct CompactSpace {
    int *counts, *segment, *hole, *mover, *rank;
};
__device__ __host__ inline CompactSpace compact_space(int *ws, int64_t P)
{
    int *segment = ws + 4, *hole = segment + (P + kSegment - 1) / kSegment;
    return {ws, segment, hole, hole + P, hole + 2 * P};
}

__global__ __launch_bounds__(kPlan) void k_compact_count(PagesArgs a)
{
    __shared__ int lds[kPlanWaves];
    const int base = blockIdx.x * kSegment;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSegment / kPlan; ++i) {
        const int page = base + i * kPlan + (int)threadIdx.x;
        n += page < a.P && a.refs[page] > 0;
    }
    int total;
    block_scan(n, lds, total);
    if (threadIdx.x == 0)
        compact_space(a.ws, a.P).segment[blockIdx.x] = total;
}

__global__ __launch_bounds__(kPlan) void k_compact_list(PagesArgs a)
{
    __shared__ int lds[kPlanWaves];
    const CompactSpace ws = compact_space(a.ws, a.P);
    const int segments = (a.P + kSegment - 1) / kSegment, base = blockIdx.x * kSegment;
    int live = 0, rank = 0, total;
    for (int i = threadIdx.x; i < segments; i += kPlan) {
        live += ws.segment[i];
        rank += i < (int)blockIdx.x ? ws.segment[i] : 0;
    }
    block_scan(live, lds, total);
    live = total;
    block_scan(rank, lds, total);
    rank = total;
    if (live == 0 && blockIdx.x == 0 && threadIdx.x == 0)
        ws.counts[0] = ws.counts[1] = 0;
    for (int i = 0; i < kSegment / kPlan; ++i) {
        const int page = base + i * kPlan + (int)threadIdx.x;
        const int used = page < a.P && a.refs[page] > 0;
        const int r = rank + block_scan(used, lds, total);
        rank += total;
        if (page >= a.P)
            continue;
        if (page < live && !used)
            ws.hole[page - r] = page;
        if (page >= live) {
            ws.rank[page] = used ? r : -1;
            if (used)
                ws.mover[r] = page;
        }
        if (page == live - 1) {
            ws.counts[0] = live;
            ws.counts[1] = live - r - used;
        }
    }
}

__global__ __launch_bounds__(256) void k_compact_move(PagesArgs a)
{
    const CompactSpace ws = compact_space(a.ws, a.P);
    const int live = ws.counts[0], moves = ws.counts[1], stay = live - moves;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = id; i < (int64_t)a.B * a.W; i += step) {
        const int page = a.table[i];
        if (page >= live && page < a.P) {
            const int r = ws.rank[page];
            if (r >= stay && r < live)
                a.table[i] = ws.hole[r - stay];
        }
    }
    for (int64_t i = id; i < moves; i += step) {
        const int src = ws.mover[stay + i], dst = ws.hole[i];
        a.refs[dst] = a.refs[src];
        a.refs[src] = 0;
    }
    if (id == 0)
        *a.first = live;
    copy_pages(a, moves, [&](int64_t i, int64_t &src, int64_t &dst) {
        src = ws.mover[stay + i];
        dst = ws.hole[i];
        return true;
    });
}

// ---------------------------------------------------------------------------------- copy

__global__ __launch_bounds__(256) void k_pages_copy(PagesArgs a, const int *src, const int *dst, int64_t n)
{
    copy_pages(a, n, [&](int64_t i, int64_t &from, int64_t &to) {
        from = src[i];
        to = dst[i];
        return from >= 0 && from < a.P && to >= 0 && to < a.P && from != to;
    });
}

}  // namespace

size_t pages_workspace_bytes(int64_t B, int64_t W, int64_t P)
{
    const int64_t grow = 4 + 4 * B + P, fork = B + B * W;
    const int64_t compact = 4 + (P + kSegment - 1) / kSegment + 3 * P;
    const int64_t most = grow > fork ? grow : fork;
    return (size_t)(4 * (most > compact ? most : compact));
}

hipError_t launch_pages_grow(const PagesArgs &a, hipStream_t s)
{
    k_pages_plan<<<1, kPlan, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    const int64_t tokens = ((int64_t)a.T + 255) / 256;
    const unsigned copies = copy_grid(a, a.B), all = tokens > 4096 ? 4096u : (unsigned)(tokens < 1 ? 1 : tokens);
    k_pages_grow<<<copies > all ? copies : all, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PagesArgs &a, hipStream_t s)
{
    k_fork_take<<<(unsigned)a.B, 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    k_fork_give<<<(unsigned)a.B, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t s)
{
    const unsigned segments = (unsigned)((a.P + kSegment - 1) / kSegment);
    k_compact_count<<<segments, kPlan, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    k_compact_list<<<segments, kPlan, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    const int64_t cells = ((int64_t)a.B * a.W + 255) / 256;
    const unsigned copies = copy_grid(a, a.P / 2), all = cells > 4096 ? 4096u : (unsigned)(cells < 1 ? 1 : cells);
    k_compact_move<<<copies > all ? copies : all, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_copy(const PagesArgs &a, const int *src, const int *dst, int64_t n, hipStream_t s)
{
    k_pages_copy<<<copy_grid(a, n), 256, 0, s>>>(a, src, dst, n);
    return hipGetLastError();
}

}  // namespace bt
