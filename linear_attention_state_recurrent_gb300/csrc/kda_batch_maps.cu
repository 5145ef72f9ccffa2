// kda_batch_maps: running order, cu_seqlens, state slots, block table and slot map of a step
// from the requests' lengths.
//
// Everything is integers and small; what counts is latency, so it is one launch without a
// workspace: every CTA scans the lengths of all requests for itself (they sit in L2) and
// then fills its own 2 * blockDim token rows. A request's rows start at the scan of the
// query lengths in running order: decodes (one token each) come first, so decode number d
// starts at row d and another request at D + the tokens of the non-decodes before it. Pages
// are handed out by a second scan, in the given order. 128 decodes take 3.8 us and a step of 4096
// requests and 262,144 rows 8.3 us; bound by the chain of load, scan, scan, load, store.
#include <climits>
#include <cstdint>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_layer.h"
#include "kda_pdl.cuh"

namespace kda {
namespace {

constexpr int kItems = 4;       // requests per thread and step of the scan
constexpr int kRows = 2;        // token rows per thread
constexpr int kMaxThreads = 1024;
constexpr int64_t kMostCtas = 512;
constexpr uint32_t kErrPages = 8u, kErrLengths = 16u;

// Exclusive prefix of v over the block and the block's total (blockDim.x a multiple of 32).
// `part` holds one value per warp; a barrier separates two uses of it.
template <typename V>
__device__ __forceinline__ V block_exclusive(V v, V *part, V *total)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    V inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    V w = lane < warps ? part[lane] : V(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const V before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : V(0)) + inc - v;
}

struct Lens {
    int32_t q, c;
    bool bad;
};

__device__ __forceinline__ Lens load_lens(const BatchMapsParams &p, int r)
{
    Lens l{0, 0, false};
    if (r >= p.R) return l;
    l.q = __ldg(p.qlen + r);
    l.c = __ldg(p.clen + r);
    if (l.q < 0 || l.c < 0 || static_cast<int64_t>(l.q) + l.c > INT32_MAX) l = Lens{0, 0, true};
    return l;
}

// Division by the page size, a shift where it is a power of two (shift >= 0).
struct PageSize {
    uint32_t size;
    int shift;
    __device__ __forceinline__ uint32_t floor(uint32_t n) const { return shift >= 0 ? n >> shift : n / size; }
    __device__ __forceinline__ uint32_t ceil(uint32_t n) const { return floor(n + size - 1u); }   // n below 2^31, as the size
};

__global__ void __launch_bounds__(kMaxThreads) batch_maps_kernel(const BatchMapsParams p, const PageSize page_of, const int share)
{
    extern __shared__ int32_t own[];   // per token row of this CTA: request (-1: not its first row here)
    const int rows = kRows * blockDim.x;
    int32_t *own_start = own + rows, *own_base = own + 2 * rows;   // its first row, its first new page's number,
    int32_t *own_context = own + 3 * rows;                         // and its context
    __shared__ int64_t part[32];
    const int64_t T0 = static_cast<int64_t>(blockIdx.x) * rows;
    const int64_t N = p.num_tokens;
    uint32_t err = 0;
    pdl_wait_then_release();

    // everything the first step reads is asked for at once; of the outputs per request a CTA writes a share
    const int32_t free_count = __ldg(p.free_count);
    const int step = kItems * blockDim.x, mine0 = blockIdx.x * share, mine1 = mine0 + share;
    auto slot_of = [&](int r) { return r >= mine0 && r < mine1 && r < p.R ? __ldg(p.slots + r * p.slot_stride) : 0; };
    Lens first[kItems];
    int32_t first_slot[kItems];
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        first[i] = load_lens(p, threadIdx.x * kItems + i);
        first_slot[i] = slot_of(threadIdx.x * kItems + i);
    }
    for (int i = threadIdx.x; i < rows; i += blockDim.x) own[i] = -1;
    int64_t D = 0;
    if (p.R > step) {
        // the decodes, all of them, before anything can be placed (one step knows them from its scan)
        int32_t nd = 0, all;
#pragma unroll
        for (int i = 0; i < kItems; i++) nd += first[i].q == 1;
        for (int r0 = step; r0 < p.R; r0 += step)
#pragma unroll
            for (int i = 0; i < kItems; i++) nd += load_lens(p, r0 + threadIdx.x * kItems + i).q == 1;
        block_exclusive(nd, reinterpret_cast<int32_t *>(part), &all);
        D = all;
    }

    int64_t d_done = 0, t_done = 0;
    uint32_t p_done = 0;   // pages: at most one per token and request
    for (int r0 = 0; r0 < p.R; r0 += step) {
        Lens l[kItems];
        int32_t slot[kItems];
        // decodes above bit 44, the others' tokens below it: 4096 requests of less than 2^31
        // tokens at most in one step
        int64_t mine = 0;
        uint32_t pages = 0, pages_of[kItems];
#pragma unroll
        for (int i = 0; i < kItems; i++) {
            l[i] = r0 == 0 ? first[i] : load_lens(p, r0 + threadIdx.x * kItems + i);
            slot[i] = r0 == 0 ? first_slot[i] : slot_of(r0 + threadIdx.x * kItems + i);
            mine += l[i].q == 1 ? (int64_t(1) << 44) : l[i].q;
        }
        int64_t total;
        int64_t before = block_exclusive(mine, part, &total);
        if (p.R <= step) D = total >> 44;
        int64_t d = d_done + (before >> 44), t = t_done + (before & ((int64_t(1) << 44) - 1));
        int64_t start_of[kItems];
#pragma unroll
        for (int i = 0; i < kItems; i++) {
            const int r = r0 + threadIdx.x * kItems + i;
            pages_of[i] = 0;
            if (r >= p.R) continue;
            const bool dec = l[i].q == 1;
            const int64_t s = dec ? d : D + (r - d);
            const int64_t start = dec ? d : D + t;
            const int64_t end = start + l[i].q;
            if (dec) d++; else t += l[i].q;
            start_of[i] = start;
            if (l[i].bad || end > N) err |= kErrLengths;
            // cut off at the capacity
            const int64_t cs = start < N ? start : N, ce = end < N ? end : N;
            if (r >= mine0 && r < mine1) {
                p.order[s] = r;
                p.cu[s + 1] = static_cast<int32_t>(ce);
                p.state_indices[s] = slot[i];
            }
            l[i].q = static_cast<int32_t>(ce - cs);
            int64_t old = page_of.ceil(l[i].c), now = page_of.ceil(l[i].c + l[i].q);
            if (now > p.width) { if (l[i].q > 0) err |= kErrPages; now = p.width; }
            pages_of[i] = now > old ? static_cast<uint32_t>(now - old) : 0;
            pages += pages_of[i];
        }
        uint32_t ptotal;
        uint32_t base = p_done + block_exclusive(pages, reinterpret_cast<uint32_t *>(part), &ptotal);
#pragma unroll
        for (int i = 0; i < kItems; i++) {
            const int r = r0 + threadIdx.x * kItems + i;
            if (r < p.R && l[i].q > 0 && start_of[i] < T0 + rows && start_of[i] + l[i].q > T0) {
                const int o = static_cast<int>(start_of[i] > T0 ? start_of[i] - T0 : 0);
                own[o] = r;
                own_start[o] = static_cast<int32_t>(start_of[i]);
                own_base[o] = static_cast<int32_t>(base);
                own_context[o] = l[i].c;
            }
            base += pages_of[i];
        }
        d_done += total >> 44;
        t_done += total & ((int64_t(1) << 44) - 1);
        p_done += ptotal;
    }
    const int64_t fc = max(int64_t(0), min(static_cast<int64_t>(free_count), p.num_free));
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.cu[0] = 0;
        *p.num_decodes = static_cast<int32_t>(D);
        *p.free_left = static_cast<int32_t>(fc > p_done ? fc - p_done : 0);
        if (p_done > fc) err |= kErrPages;
    }
    __syncthreads();

    // each row's request starts at the nearest marked row at or before it
    int head[kRows], last = -1;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const int o = threadIdx.x * kRows + i;
        if (own[o] >= 0) last = o;
        head[i] = last;
    }
    int inc = last;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = max(inc, u);
    }
    int *wpart = reinterpret_cast<int *>(part);
    if (lane == 31) wpart[warp] = inc;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) before = -1;
    if (warp > 0) {   // the warps before this one, of 32 at most
        int w = lane < warp ? wpart[lane] : -1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
        before = max(before, w);
    }
    const int64_t live = D + t_done < N ? D + t_done : N;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const int64_t t = T0 + threadIdx.x * kRows + i;
        if (t >= N) break;
        int64_t slot = -1;
        int32_t pos = 0;
        if (t < live) {
            const int o = head[i] >= 0 ? head[i] : before;
            const int r = own[o];
            const int32_t c = own_context[o];
            pos = c + static_cast<int32_t>(t - own_start[o]);
            const int32_t j = page_of.floor(pos), old = page_of.ceil(c), off = pos - j * p.page;
            int32_t page = -1;
            if (j < p.width) {
                int32_t *entry = p.table + r * p.table_stride + j;
                if (j < old) {
                    page = *entry;
                } else {
                    const int64_t k = static_cast<int64_t>(static_cast<uint32_t>(own_base[o])) + (j - old);
                    if (k < fc) page = __ldg(p.free_pages + (fc - 1 - k));
                    if (off == 0) *entry = page;   // a new page's first position is one of the query's
                }
            }
            if (page >= 0 && page < p.num_pages) slot = static_cast<int64_t>(page) * p.page + off;
            else err |= kErrPages;
        }
        p.positions[t] = pos;
        p.slot_map[t] = slot;
    }
    if (err && p.err) atomicOr(p.err, err);
}

}  // namespace

cudaError_t launch_batch_maps(const BatchMapsParams &p, cudaStream_t stream)
{
    // Enough threads for one step of the scan, and no more, as a barrier costs by the warp (64 requests with 45,000
    // rows: 4.1 us, in the widest CTAs 6.7), unless that takes more CTAs than three or four for each SM, all of which
    // scan for themselves (512 requests with 500,000 rows: 10.6 us, without this bound 12.0).
    const int64_t scan = (p.R + kItems - 1) / kItems;
    int64_t threads = scan <= 64 ? 64 : (scan + 31) / 32 * 32;
    while (threads < kMaxThreads && p.num_tokens > kMostCtas * kRows * threads) threads *= 2;
    if (threads > kMaxThreads) threads = kMaxThreads;
    const int64_t per = kRows * threads;
    const int64_t grid = p.num_tokens > 0 ? (p.num_tokens + per - 1) / per : 1;
    PageSize page{static_cast<uint32_t>(p.page), -1};
    for (int i = 0; i < 31; i++)
        if (p.page == 1 << i) page.shift = i;
    const int share = static_cast<int>((p.R + grid - 1) / grid);
    return launch_pdl(batch_maps_kernel, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)),
                      static_cast<size_t>(4 * per * sizeof(int32_t)), stream, p, page, share);
}

}  // namespace kda
