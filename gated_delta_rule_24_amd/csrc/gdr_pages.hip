// Pages of the cache as several continuations of one prompt hold them: rows of
// the block table forked from other rows, with the pages that more than one row is
// about to write copied, fresh pages dealt out and dropped ones free again
// (gdr_kv_fork); and used pages moved to the lowest places (gdr_kv_compact).
//
// The tables alone say what is in use: each call counts, for every page, the
// entries that name it.  Nothing is kept between calls that could go astray, a
// call made twice gives the same result, and which pages are dealt out does not
// depend on the order in which workgroups run: the j-th wanted page, row by row, is
// the j-th lowest free one.
#include "gdr_device.h"
#include "gdr_generation.h"
#include "gdr_launch.h"

namespace gdr {

namespace {

constexpr int kPage = 64;
constexpr int kThreads = 256;
constexpr int kPagesPerBlock = 4096;                  // pages that a workgroup counts
constexpr int kEntriesPerBlock = 2048;                // entries of one row that a workgroup copies
constexpr int kPiece = 16 * kThreads;                 // bytes that a workgroup copies at once; a side of a page is whole ones
constexpr int kForkPieces = 1, kMovePieces = 4;       // that it copies together
constexpr int kCopyWorkgroups = 4096;                 // compact: workgroups that take the moved pages in turn

// A page's counters: entries that name it in the low half, rows that will write
// into it in the high half; and N - n of the lowest such row n.
struct ForkSpace {
    unsigned long long* count;  // [n_pages]
    int* lowest;                // [n_pages]
    int* block_free;            // free pages of each 4,096
    int* want;                  // [N] pages wanted; bit 30: the first is a copy
    int* source;                // [N] the page to copy, and to where, or -1
    int* place;
};
constexpr int kCopyBit = 1 << 30;

__host__ __device__ inline size_t up16(size_t n) { return (n + 15) / 16 * 16; }
inline int blocks_of(long long n, long long per) { return (int)((n + per - 1) / per); }

ForkSpace fork_space(void* ws, int N, int n_pages) {
    char* at = static_cast<char*>(ws);
    ForkSpace s;
    auto take = [&](size_t bytes) { char* x = at; at += up16(bytes); return x; };
    s.count = reinterpret_cast<unsigned long long*>(take(8 * (size_t)n_pages));
    s.lowest = reinterpret_cast<int*>(take(4 * (size_t)n_pages));
    s.block_free = reinterpret_cast<int*>(take(4 * (size_t)blocks_of(n_pages, kPagesPerBlock)));
    s.want = reinterpret_cast<int*>(take(4 * (size_t)N));
    s.source = reinterpret_cast<int*>(take(4 * (size_t)N));
    s.place = reinterpret_cast<int*>(take(4 * (size_t)N));
    return s;
}

// What row n continues: its row of the table, or -1, and its tokens (held inside
// the table's width, so that no content of cache_len leads out of it).
__device__ __forceinline__ int row_of(const PagesParams& p, int n, int& len) {
    const int from = p.parent ? p.parent[n] : n;
    if ((unsigned)from >= (unsigned)p.N_in) { len = 0; return -1; }
    const long long most = (long long)p.max_pages * kPage;
    const int l = p.cache_len[from];
    len = l < 0 ? 0 : l > most ? (int)most : l;
    return from;
}
__device__ __forceinline__ int room_of(const PagesParams& p, int n) {
    const int r = p.room ? p.room[n] : p.room_all;
    return r < 0 ? 0 : r;
}
__device__ __forceinline__ int pages_of(long long tokens) { return (int)((tokens + kPage - 1) / kPage); }

__global__ __launch_bounds__(kThreads) void pages_clear(uint4* at, long long n) {
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads)
        at[i] = make_uint4(0, 0, 0, 0);
}

// sum over the workgroup, in every thread
__device__ __forceinline__ int block_sum(int x, int* s) {
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) sum += s[w];
    return sum;
}
// sum over the threads before this one; `all` the workgroup's
__device__ __forceinline__ int block_before(int x, int* s, int& all) {
    int run = x;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(run, o, 64);
        if ((int)(threadIdx.x & 63) >= o) run += y;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) s[threadIdx.x >> 6] = run;
    __syncthreads();
    int base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < (int)(threadIdx.x >> 6)) base += s[w];
        all += s[w];
    }
    return base + run - x;
}

// PIECES pieces of a page from one place to another, part `part` of the keys' bytes, then the
// values'; and (part 0) the scales.  Loads without a branch: with one, each waited for the last.
template <int PIECES>
__device__ __forceinline__ void copy_part(const PagesParams& p, int from, int to, int part) {
    const size_t side = (size_t)p.Hkv * kPage * p.d;
    const int each = (int)(side / kPiece), at = 16 * threadIdx.x;
    uint4 x[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int c = min(part * PIECES + i, 2 * each - 1);
        const uint8_t* src = c < each ? p.k_cache + from * side + (size_t)c * kPiece : p.v_cache + from * side + (size_t)(c - each) * kPiece;
        x[i] = *reinterpret_cast<const uint4*>(src + at);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int c = part * PIECES + i;
        if (c >= 2 * each) break;
        uint8_t* dst = c < each ? p.k_cache + to * side + (size_t)c * kPiece : p.v_cache + to * side + (size_t)(c - each) * kPiece;
        *reinterpret_cast<uint4*>(dst + at) = x[i];
    }
    if (part == 0)
        for (int h = threadIdx.x; h < p.Hkv; h += kThreads) {
            p.k_scale[(size_t)to * p.Hkv + h] = p.k_scale[(size_t)from * p.Hkv + h];
            p.v_scale[(size_t)to * p.Hkv + h] = p.v_scale[(size_t)from * p.Hkv + h];
        }
}
int copy_parts(int Hkv, int d, int pieces) { return blocks_of(2LL * Hkv * kPage * d, (long long)pieces * kPiece); }

}  // namespace

// The new rows, and for every page the entries that name it.  One workgroup per
// 2,048 entries of a row.
__global__ __launch_bounds__(kThreads) void fork_rows(PagesParams p, ForkSpace s, int chunks) {
    const int n = blockIdx.x / chunks, begin = (blockIdx.x % chunks) * kEntriesPerBlock;
    int len;
    const int from = row_of(p, n, len);
    const int pages = pages_of(len), written = len % kPage != 0 && room_of(p, n) > 0 ? len / kPage : -1;
    const int end = min(begin + kEntriesPerBlock, p.max_pages);
    for (int i = begin + threadIdx.x; i < end; i += kThreads) {
        int page = -1;
        if (i < pages) {
            page = p.block_table[(size_t)from * p.max_pages + i];
            if ((unsigned)page >= (unsigned)p.n_pages) page = -1;
        }
        p.table_out[(size_t)n * p.max_pages + i] = page;
        if (page >= 0) {
            atomicAdd(&s.count[page], i == written ? (1ull << 32) + 1 : 1ull);
            if (i == written) atomicMax(&s.lowest[page], p.N - n);
        }
    }
    if (begin == 0 && threadIdx.x == 0) p.len_out[n] = len;
}

// Free pages of each 4,096, and the pages that each row wants.
__global__ __launch_bounds__(kThreads) void fork_count(PagesParams p, ForkSpace s) {
    __shared__ int s_sum[kThreads / 64];
    const int first = blockIdx.x * kPagesPerBlock;
    if (first < p.n_pages) {
        int free = 0;
#pragma unroll
        for (int i = 0; i < kPagesPerBlock / kThreads; ++i) {
            const int page = first + i * kThreads + (int)threadIdx.x;
            if (page < p.n_pages) free += s.count[page] == 0 && !(p.held && p.held[page]);
        }
        free = block_sum(free, s_sum);
        if (threadIdx.x == 0) s.block_free[blockIdx.x] = free;
    }
    const int n = blockIdx.x * kThreads + threadIdx.x;
    if (n < p.N) {
        int len, want = 0;
        const int from = row_of(p, n, len), room = room_of(p, n);
        if (from >= 0 && room > 0) {
            const int have = pages_of(len);
            want = min(pages_of((long long)len + room), p.max_pages) - have;
            if (len % kPage != 0) {
                const int page = p.table_out[(size_t)n * p.max_pages + len / kPage];
                if (page >= 0) {
                    // alone, or the lowest of rows that all write: this row keeps it
                    const unsigned long long c = s.count[page];
                    const bool keeps = (uint32_t)c == (uint32_t)(c >> 32) && s.lowest[page] == p.N - n && !(p.held && p.held[page]);
                    if (!keeps) want = (want + 1) | kCopyBit;
                }
            }
        }
        s.want[n] = want;
        s.place[n] = -1;
    }
}

// The j-th wanted page is the j-th lowest free one.  A workgroup ranks the free
// pages among its 4,096 and looks up whose wish each rank is, in the running sums of
// the rows' wishes, which it makes for itself (in LDS, for up to 2,048 runs of rows).
constexpr int kRuns = 2048;
__global__ __launch_bounds__(kThreads) void fork_assign(PagesParams p, ForkSpace s, int blocks) {
    __shared__ int s_sum[kThreads / 64];
    __shared__ int s_before[kRuns];                   // wishes of the rows before run i
    const int tid = threadIdx.x;
    const int per = (p.N + kRuns - 1) / kRuns, runs = (p.N + per - 1) / per;
    int total = 0;
    for (int i0 = 0; i0 < runs; i0 += kThreads) {
        const int i = i0 + tid;
        int x = 0, all;
        if (i < runs)
            for (int n = i * per; n < min((i + 1) * per, p.N); ++n) x += s.want[n] & ~kCopyBit;
        const int before = block_before(x, s_sum, all);
        if (i < runs) s_before[i] = total + before;
        total += all;
    }
    __syncthreads();
    int base = 0, free_all = 0;
    for (int b0 = 0; b0 < blocks; b0 += kThreads) {
        const int b = b0 + tid;
        const int f = b < blocks ? s.block_free[b] : 0;
        base += block_sum(b < (int)blockIdx.x ? f : 0, s_sum);
        free_all += block_sum(f, s_sum);
    }
    // what rows do not get
    for (int i = blockIdx.x * kThreads + tid; i < runs; i += gridDim.x * kThreads) {
        int at = s_before[i];
        for (int n = i * per; n < min((i + 1) * per, p.N); ++n) {
            const int w = s.want[n] & ~kCopyBit;
            at += w;
            p.missing[n] = max(0, min(w, at - free_all));
        }
    }
    // this thread's pages: 16 in a row, so that their ranks follow each other
    constexpr int kRow = kPagesPerBlock / kThreads;
    const int first = blockIdx.x * kPagesPerBlock + tid * kRow;
    uint32_t mine = 0;
    if (base < total) {
#pragma unroll
        for (int i = 0; i < kRow; ++i)
            if (first + i < p.n_pages && s.count[first + i] == 0 && !(p.held && p.held[first + i])) mine |= 1u << i;
    }
    int all;
    int rank = base + block_before(__popc(mine), s_sum, all);
    for (; mine && rank < total; mine &= mine - 1, ++rank) {
        const int page = first + __ffs(mine) - 1;
        int lo = 0, hi = runs - 1;                    // the last run that starts at or before this rank
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_before[mid] <= rank) lo = mid;
            else hi = mid - 1;
        }
        int n = lo * per, before = s_before[lo], w = s.want[n];
        while (rank >= before + (w & ~kCopyBit)) {    // (ends: this run's wishes pass `rank`)
            before += w & ~kCopyBit;
            w = s.want[++n];
        }
        int len;
        row_of(p, n, len);
        int entry = pages_of(len) + rank - before;
        if (w & kCopyBit) --entry;                    // the copied page's own place first
        int* at = p.table_out + (size_t)n * p.max_pages + entry;
        if ((w & kCopyBit) && rank == before) {
            s.source[n] = *at;
            s.place[n] = page;
        }
        *at = page;
    }
}

// One piece a workgroup: 110 pages of 128 KiB behind 256 rows take 6.2 us, 4.7 TB/s.  (Consecutive
// workgroups go to the 8 XCDs and there to the 4 shader engines by turns.  With 16 for a
// row, not 32, the rows that copy, mostly every other one, fell on half of them: 17.6.)
__global__ __launch_bounds__(kThreads) void fork_copy(PagesParams p, ForkSpace s, int parts) {
    const int n = blockIdx.x / parts, to = s.place[n], from = s.source[n];   // (without a place, no page: not read)
    if (to >= 0) copy_part<kForkPieces>(p, from, to, blockIdx.x % parts);
}

// The same for caches and tables that one workgroup has soon read: the counters are in
// LDS, and a call is this kernel and the copies.  (256 rows of 40 pages: five launches take 41 us a
// call, two 20.5; of 130, 44 and 28; of 157, next to the limit, 42 and 30; past it, of 200, 42.5 and
// 34 and of 272, 44 and 40.6: the limit is not where they cross but keeps clear of the counters' 16
// bits.  4 rows of 17 pages: 29 and 19.)  Compaction of 120 rows of 66 pages: 101 and 86; of 250 rows of
// 80 pages 37.9 and 39.6, of 160 pages 39 and 51.
constexpr int kSmallThreads = 1024;
constexpr int kMine = 12;                             // pages a thread
constexpr int kSmallPages = kMine * kSmallThreads, kSmallRows = 2048;   // (LDS: 8 bytes a page, 16 a row)
constexpr int kForkEntries = 40 * kSmallThreads;      // (counters of 16 bits)
constexpr int kCompactEntries = 20 * kSmallThreads;
bool small_tables(int N, int n_pages, int max_pages, int entries) {
    return n_pages <= kSmallPages && N <= kSmallRows && (long long)N * max_pages <= entries;
}

// sum over the threads of 1,024 before this one; `all` the workgroup's
__device__ __forceinline__ int wide_before(int x, int* s, int& all) {
    int run = x;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(run, o, 64);
        if ((int)(threadIdx.x & 63) >= o) run += y;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) s[threadIdx.x >> 6] = run;
    __syncthreads();
    int base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kSmallThreads / 64; ++w) {
        if (w < (int)(threadIdx.x >> 6)) base += s[w];
        all += s[w];
    }
    return base + run - x;
}

// Bit i: page first + i is held.  (All loads at once, before the first wait.)
__device__ __forceinline__ uint32_t held_bits(const PagesParams& p, int first) {
    if (!p.held) return 0;
    uint32_t h[kMine], bits = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) h[i] = p.held[min(first + i, p.n_pages - 1)];
#pragma unroll
    for (int i = 0; i < kMine; ++i) bits |= h[i] ? 1u << i : 0;
    return bits;
}

// Every entry of the rows' tables, eight at a time a thread (their loads do not wait for
// each other): f(place, row, entry of the row, the page it names or -1).
template <typename F>
__device__ __forceinline__ void entries_of(const PagesParams& p, const int* len, const int* from, const F& f) {
    constexpr int kAtOnce = 8;
    const int entries = p.N * p.max_pages;
    for (int at0 = threadIdx.x; at0 < entries; at0 += kAtOnce * kSmallThreads) {
        int n[kAtOnce], i[kAtOnce], page[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int at = min(at0 + j * kSmallThreads, entries - 1);
            n[j] = at / p.max_pages;
            i[j] = at - n[j] * p.max_pages;
            page[j] = -1;
            if (i[j] < pages_of(len[n[j]])) page[j] = p.block_table[from ? (size_t)from[n[j]] * p.max_pages + i[j] : (size_t)at];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (at0 + j * kSmallThreads < entries)
                f(at0 + j * kSmallThreads, n[j], i[j], (unsigned)page[j] < (unsigned)p.n_pages ? page[j] : -1);
    }
}

size_t fork_small_lds(int N, int n_pages) { return 8 * (size_t)n_pages + 16 * (size_t)N; }

__global__ __launch_bounds__(kSmallThreads) void fork_small(PagesParams p, ForkSpace s) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ int s_sum[kSmallThreads / 64];
    uint32_t* count = reinterpret_cast<uint32_t*>(smem);             // [n_pages] entries that name it, and rows that write into it << 16
    int* lowest = reinterpret_cast<int*>(count + p.n_pages);         // [n_pages]
    int* from = lowest + p.n_pages;                                  // [N] the row continued; then 1: the first page is a copy
    int* len = from + p.N;                                           // [N]
    int* before = len + p.N;                                         // [N] the entry it writes into, or -1; then the pages wanted by the rows before
    int* into = before + p.N;                                        // [N] the page it writes into, or -1
    const int tid = threadIdx.x;
    const int mine = (p.n_pages + kSmallThreads - 1) / kSmallThreads, first = tid * mine;
    const uint32_t held = held_bits(p, first);
    for (int n = tid; n < p.N; n += kSmallThreads) {
        int l;
        from[n] = row_of(p, n, l);
        len[n] = l;
        before[n] = l % kPage != 0 && room_of(p, n) > 0 ? l / kPage : -1;
        into[n] = -1;
        p.len_out[n] = l;
        s.place[n] = -1;
    }
    for (int i = tid; i < 2 * p.n_pages; i += kSmallThreads) count[i] = 0;
    __syncthreads();
    entries_of(p, len, from, [&](int at, int n, int i, int page) {
        p.table_out[at] = page;
        if (page >= 0) {
            const bool written = i == before[n];
            atomicAdd(&count[page], written ? 0x10001u : 1u);
            if (written) {
                atomicMax(&lowest[page], p.N - n);
                into[n] = page;
            }
        }
    });
    __syncthreads();
    // what each row wants: `per` rows a thread, one after the other
    const int per = (p.N + kSmallThreads - 1) / kSmallThreads, first_row = min(tid * per, p.N), end_row = min(first_row + per, p.N);
    int want_all = 0;
    for (int n = first_row; n < end_row; ++n) {
        const int l = len[n], room = room_of(p, n), page = into[n];
        int want = 0;
        bool copy = false;
        if (from[n] >= 0 && room > 0) {
            want = min(pages_of((long long)l + room), p.max_pages) - pages_of(l);
            if (page >= 0) {
                // alone, or the lowest of rows that all write: this row keeps it
                const uint32_t c = count[page];
                copy = !((c & 0xffff) == c >> 16 && lowest[page] == p.N - n && !(p.held && p.held[page]));
            }
        }
        want += copy;
        from[n] = copy;
        before[n] = want;
        want_all += want;
    }
    int total, free_all;
    int run = wide_before(want_all, s_sum, total);
    for (int n = first_row; n < end_row; ++n) {
        const int want = before[n];
        before[n] = run;
        run += want;
    }
    // the free pages among this thread's and their ranks
    uint32_t free = 0;
    for (int i = 0; i < mine; ++i)
        if (first + i < p.n_pages && count[first + i] == 0 && !(held >> i & 1)) free |= 1u << i;
    int rank = wide_before(__popc(free), s_sum, free_all);
    for (int n = first_row; n < end_row; ++n) {
        const int end = n + 1 < end_row ? before[n + 1] : run;
        p.missing[n] = max(0, min(end - before[n], end - free_all));
    }
    for (; free && rank < total; free &= free - 1, ++rank) {
        const int page = first + __ffs(free) - 1;
        int lo = 0, hi = p.N - 1;                     // the last row that starts at or before this rank: it wants some
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before[mid] <= rank) lo = mid;
            else hi = mid - 1;
        }
        const int n = lo, k = rank - before[n], copy = from[n];
        if (copy && k == 0) {
            s.source[n] = into[n];
            s.place[n] = page;
        }
        p.table_out[(size_t)n * p.max_pages + pages_of(len[n]) + k - copy] = page;
    }
}

size_t kv_fork_workspace(int N, int n_pages) {
    return up16(8 * (size_t)n_pages) + up16(4 * (size_t)n_pages) + up16(4 * (size_t)blocks_of(n_pages, kPagesPerBlock)) +
           3 * up16(4 * (size_t)N);
}

long long kv_fork_workgroups(int N, int Hkv, int d, int n_pages, int max_pages) {
    const long long rows = (long long)N * blocks_of(max_pages, kEntriesPerBlock), copies = (long long)N * copy_parts(Hkv, d, kForkPieces);
    const long long pages = blocks_of(n_pages, kPagesPerBlock);
    return rows > copies ? (rows > pages ? rows : pages) : copies > pages ? copies : pages;
}

hipError_t launch_kv_fork(const PagesParams& p, hipStream_t st) {
    const ForkSpace s = fork_space(p.workspace, p.N, p.n_pages);
    const int parts = copy_parts(p.Hkv, p.d, kForkPieces);
    if (small_tables(p.N, p.n_pages, p.max_pages, kForkEntries)) {
        static std::atomic<unsigned long long> done{0};
        const hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&fork_small), (int)fork_small_lds(kSmallRows, kSmallPages), done);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(fork_small, dim3(1), dim3(kSmallThreads), (unsigned)fork_small_lds(p.N, p.n_pages), st, p, s);
        hipLaunchKernelGGL(fork_copy, dim3((unsigned)(p.N * (long long)parts)), dim3(kThreads), 0, st, p, s, parts);
        return hipGetLastError();
    }
    const long long vecs = (long long)(up16(8 * (size_t)p.n_pages) + up16(4 * (size_t)p.n_pages)) / 16;
    const dim3 block(kThreads);
    hipLaunchKernelGGL(pages_clear, dim3((unsigned)(vecs < 1024 * kThreads ? blocks_of(vecs, kThreads) : 1024)), block, 0, st,
                       reinterpret_cast<uint4*>(s.count), vecs);
    const int chunks = blocks_of(p.max_pages, kEntriesPerBlock);
    hipLaunchKernelGGL(fork_rows, dim3((unsigned)(p.N * (long long)chunks)), block, 0, st, p, s, chunks);
    const int blocks = blocks_of(p.n_pages, kPagesPerBlock), row_blocks = blocks_of(p.N, kThreads);
    hipLaunchKernelGGL(fork_count, dim3((unsigned)(blocks > row_blocks ? blocks : row_blocks)), block, 0, st, p, s);
    hipLaunchKernelGGL(fork_assign, dim3((unsigned)blocks), block, 0, st, p, s, blocks);
    hipLaunchKernelGGL(fork_copy, dim3((unsigned)(p.N * (long long)parts)), block, 0, st, p, s, parts);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------
//
// The j-th lowest free page takes the j-th highest page in use (one that nobody
// else holds) while that is the higher of the two: from some j on it is not, so the
// moves are a prefix of the pairs, and a source is never a destination.

namespace {
struct CompactSpace {
    int* named;                 // [n_pages] 1: some entry names it
    int* block_free;            // of each 4,096 pages: the free ones, those that may move
    int* block_used;
    int* free_list;             // [n_pages] free pages, ascending
    int* used_list;             // [n_pages] pages that may move, descending
    int* rank;                  // [n_pages] a page's place in used_list
    int* counts;                // [2] lengths of the lists
};
size_t compact_take(void* ws, int n_pages, CompactSpace* out) {
    char* at = static_cast<char*>(ws);
    auto take = [&](size_t n) { char* x = at; at += up16(4 * n); return reinterpret_cast<int*>(x); };
    CompactSpace s;
    const size_t blocks = blocks_of(n_pages, kPagesPerBlock);
    s.named = take(n_pages);
    s.block_free = take(blocks);
    s.block_used = take(blocks);
    s.free_list = take(n_pages);
    s.used_list = take(n_pages);
    s.rank = take(n_pages);
    s.counts = take(2);
    if (out) *out = s;
    return (size_t)(at - static_cast<char*>(ws));
}
}  // namespace

__global__ __launch_bounds__(kThreads) void compact_rows(PagesParams p, CompactSpace s, int chunks) {
    const int n = blockIdx.x / chunks, begin = (blockIdx.x % chunks) * kEntriesPerBlock;
    int len;
    row_of(p, n, len);
    const int end = min(begin + kEntriesPerBlock, pages_of(len));
    for (int i = begin + threadIdx.x; i < end; i += kThreads) {
        const int page = p.block_table[(size_t)n * p.max_pages + i];
        if ((unsigned)page < (unsigned)p.n_pages) s.named[page] = 1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.used[0] = 0;
}

__global__ __launch_bounds__(kThreads) void compact_count(PagesParams p, CompactSpace s) {
    __shared__ int s_sum[kThreads / 64];
    int free = 0, used = 0, top = 0;
#pragma unroll
    for (int i = 0; i < kPagesPerBlock / kThreads; ++i) {
        const int page = blockIdx.x * kPagesPerBlock + i * kThreads + (int)threadIdx.x;
        if (page < p.n_pages) {
            if (p.held && p.held[page]) top = page + 1;
            else if (s.named[page]) ++used;
            else ++free;
        }
    }
    free = block_sum(free, s_sum);
    used = block_sum(used, s_sum);
    for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o, 64));
    if ((threadIdx.x & 63) == 0 && top > 0) atomicMax(p.used, top);
    if (threadIdx.x == 0) { s.block_free[blockIdx.x] = free; s.block_used[blockIdx.x] = used; }
}

__global__ __launch_bounds__(kThreads) void compact_lists(PagesParams p, CompactSpace s, int blocks) {
    __shared__ int s_sum[kThreads / 64];
    const int tid = threadIdx.x;
    int free_before = 0, used_behind = 0, free_all = 0, used_all = 0;
    for (int b0 = 0; b0 < blocks; b0 += kThreads) {
        const int b = b0 + tid;
        const int f = b < blocks ? s.block_free[b] : 0, u = b < blocks ? s.block_used[b] : 0;
        free_before += block_sum(b < (int)blockIdx.x ? f : 0, s_sum);
        used_behind += block_sum(b > (int)blockIdx.x ? u : 0, s_sum);
        free_all += block_sum(f, s_sum);
        used_all += block_sum(u, s_sum);
    }
    constexpr int kRow = kPagesPerBlock / kThreads;
    const int first = blockIdx.x * kPagesPerBlock + tid * kRow;
    uint32_t free = 0, used = 0;
#pragma unroll
    for (int i = 0; i < kRow; ++i) {
        const int page = first + i;
        if (page < p.n_pages) {
            const bool held = p.held && p.held[page];
            if (held) s.rank[page] = INT_MAX;
            else if (s.named[page]) used |= 1u << i;
            else free |= 1u << i;
        }
    }
    int all;
    int f = free_before + block_before(__popc(free), s_sum, all);
    int u = block_before(__popc(used), s_sum, all);
    u = used_behind + all - u - 1;                    // of this thread's lowest page that may move
    for (; free; free &= free - 1) s.free_list[f++] = first + __ffs(free) - 1;
    for (; used; used &= used - 1, --u) {
        const int page = first + __ffs(used) - 1;
        s.used_list[u] = page;
        s.rank[page] = u;
    }
    if (blockIdx.x == 0 && tid == 0) { s.counts[0] = free_all; s.counts[1] = used_all; }
}

// The same for caches and tables that one workgroup has soon read: which pages are named, the
// lists and the ranks are in LDS, the rows follow at once, and what is left to another
// kernel are the moves.
size_t compact_small_lds(int N, int n_pages) { return 4 * (size_t)((n_pages + 31) / 32) + 4 * (size_t)N + 6 * (size_t)n_pages; }

__global__ __launch_bounds__(kSmallThreads) void compact_small(PagesParams p, CompactSpace s) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ int s_sum[kSmallThreads / 64];
    __shared__ int s_top;
    uint32_t* named = reinterpret_cast<uint32_t*>(smem);             // a bit a page
    int* len = reinterpret_cast<int*>(named + (p.n_pages + 31) / 32);                   // [N]
    uint16_t* free_list = reinterpret_cast<uint16_t*>(len + p.N);    // [n_pages] free pages, ascending
    uint16_t* used_list = free_list + p.n_pages;                     // [n_pages] pages that may move, descending
    uint16_t* place = used_list + p.n_pages;                         // [n_pages] where a page is afterwards
    const int tid = threadIdx.x;
    const int mine = (p.n_pages + kSmallThreads - 1) / kSmallThreads, first = tid * mine;
    const uint32_t held = held_bits(p, first);
    for (int i = tid; i < (p.n_pages + 31) / 32; i += kSmallThreads) named[i] = 0;
    for (int n = tid; n < p.N; n += kSmallThreads) {
        int l;
        row_of(p, n, l);
        len[n] = l;
    }
    if (tid == 0) s_top = 0;
    __syncthreads();
    entries_of(p, len, nullptr, [&](int, int, int, int page) {
        // (rows behind one prompt name the same pages: most find the bit there)
        if (page >= 0 && !(named[page >> 5] >> (page & 31) & 1)) atomicOr(&named[page >> 5], 1u << (page & 31));
    });
    __syncthreads();
    // this thread's pages, in a row
    uint32_t free = 0, used = 0;
    int top = 0;
    for (int i = 0; i < mine; ++i) {
        const int page = first + i;
        if (page < p.n_pages) {
            place[page] = (uint16_t)page;
            if (held >> i & 1) top = page + 1;
            else if (named[page >> 5] >> (page & 31) & 1) used |= 1u << i;
            else free |= 1u << i;
        }
    }
    int free_all, used_all;
    int f = wide_before(__popc(free), s_sum, free_all), u = wide_before(__popc(used), s_sum, used_all);
    u = used_all - u - 1;                             // of this thread's lowest page that may move
    for (; free; free &= free - 1) free_list[f++] = (uint16_t)(first + __ffs(free) - 1);
    for (; used; used &= used - 1) used_list[u--] = (uint16_t)(first + __ffs(used) - 1);
    __syncthreads();
    for (int j = tid; j < used_all; j += kSmallThreads) {
        int page = used_list[j];
        if (j < free_all && free_list[j] < page) {
            s.free_list[j] = free_list[j];
            s.used_list[j] = page;
            place[page] = free_list[j];
            page = free_list[j];
        } else if (j < free_all) {                    // (the first of these ends the moves)
            s.free_list[j] = s.used_list[j] = 0;
        }
        top = max(top, page + 1);
    }
    for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) atomicMax(&s_top, top);
    __syncthreads();
    entries_of(p, len, nullptr, [&](int at, int, int, int page) { p.table_out[at] = page >= 0 ? (int)place[page] : -1; });
    if (tid == 0) {
        p.used[0] = s_top;
        s.counts[0] = free_all;
        s.counts[1] = used_all;
    }
}

// The moves, 16 KiB a workgroup at a time, and (rows > 0) the rows that follow them.  HBM bounds them:
// 1,240 pages of 128 KiB take 61 to 66 us, 4.9 to 5.3 TB/s (8 KiB 65, 4 KiB 70, 32 KiB 95).
__global__ __launch_bounds__(kThreads) void compact_move(PagesParams p, CompactSpace s, int parts, int chunks, int rows) {
    const int free = s.counts[0], used = s.counts[1], pairs = min(free, used);
    if ((int)blockIdx.x < rows) {
        const int n = blockIdx.x / chunks, begin = (blockIdx.x % chunks) * kEntriesPerBlock;
        int len;
        row_of(p, n, len);
        const int pages = pages_of(len), end = min(begin + kEntriesPerBlock, p.max_pages);
        for (int i = begin + threadIdx.x; i < end; i += kThreads) {
            const size_t at = (size_t)n * p.max_pages + i;
            int page = -1;
            if (i < pages) {
                page = p.block_table[at];
                if ((unsigned)page >= (unsigned)p.n_pages) {
                    page = -1;
                } else {
                    const int j = s.rank[page];
                    if (j < pairs && s.free_list[j] < page) page = s.free_list[j];
                }
            }
            p.table_out[at] = page;
        }
        return;
    }
    // moves are a prefix of the pairs: the first that is none ends the walk
    const long long items = (long long)pairs * parts, step = (long long)gridDim.x - rows;
    for (long long it = (long long)blockIdx.x - rows; it < items; it += step) {
        const int j = (int)(it / parts);
        const int to = s.free_list[j], from = s.used_list[j];
        if (to >= from) break;
        copy_part<kMovePieces>(p, from, to, (int)(it % parts));
    }
    // pages up to the last in use: the last destination, or the first that stays
    if (rows > 0 && (int)blockIdx.x == rows) {
        for (int j = threadIdx.x; j <= pairs; j += kThreads) {
            const bool moves = j < pairs && s.free_list[j] < s.used_list[j];
            const bool before = j == 0 || s.free_list[j - 1] < s.used_list[j - 1];
            if (!moves && before) {                   // one j: the number of moves
                int top = j > 0 ? s.free_list[j - 1] + 1 : 0;
                if (j < used) top = max(top, s.used_list[j] + 1);
                if (top > 0) atomicMax(p.used, top);
            }
        }
    }
}

size_t kv_compact_workspace(int n_pages) { return compact_take(nullptr, n_pages, nullptr); }

long long kv_compact_workgroups(int N, int n_pages, int max_pages) {
    return (long long)N * blocks_of(max_pages, kEntriesPerBlock) + kCopyWorkgroups;
}

hipError_t launch_kv_compact(const PagesParams& p, hipStream_t st) {
    CompactSpace s;
    compact_take(p.workspace, p.n_pages, &s);
    const dim3 block(kThreads);
    const int parts = copy_parts(p.Hkv, p.d, kMovePieces);
    // at most half the pages move
    const long long items = ((long long)p.n_pages / 2) * parts;
    const int movers = items < 1 ? 1 : items < kCopyWorkgroups ? (int)items : kCopyWorkgroups;
    if (small_tables(p.N, p.n_pages, p.max_pages, kCompactEntries)) {
        static std::atomic<unsigned long long> done{0};
        const hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&compact_small), (int)compact_small_lds(kSmallRows, kSmallPages), done);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(compact_small, dim3(1), dim3(kSmallThreads), (unsigned)compact_small_lds(p.N, p.n_pages), st, p, s);
        hipLaunchKernelGGL(compact_move, dim3((unsigned)movers), block, 0, st, p, s, parts, 1, 0);
        return hipGetLastError();
    }
    const long long vecs = (long long)up16(4 * (size_t)p.n_pages) / 16;
    hipLaunchKernelGGL(pages_clear, dim3((unsigned)(vecs < 1024 * kThreads ? blocks_of(vecs, kThreads) : 1024)), block, 0, st,
                       reinterpret_cast<uint4*>(s.named), vecs);
    const int chunks = blocks_of(p.max_pages, kEntriesPerBlock), blocks = blocks_of(p.n_pages, kPagesPerBlock);
    const int rows = p.N * chunks;
    hipLaunchKernelGGL(compact_rows, dim3((unsigned)rows), block, 0, st, p, s, chunks);
    hipLaunchKernelGGL(compact_count, dim3((unsigned)blocks), block, 0, st, p, s);
    hipLaunchKernelGGL(compact_lists, dim3((unsigned)blocks), block, 0, st, p, s, blocks);
    hipLaunchKernelGGL(compact_move, dim3((unsigned)(rows + movers)), block, 0, st, p, s, parts, chunks, rows);
    return hipGetLastError();
}

}  // namespace gdr
