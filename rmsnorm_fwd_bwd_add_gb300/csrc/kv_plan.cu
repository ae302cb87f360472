// kv_plan.cu -- block tables and slot maps of a paged KV cache, built on the GPU
// from the requests' lengths: rmsnorm_kv_release gives finished requests'
// blocks back to the pool's stack of free ones, rmsnorm_kv_plan takes the
// blocks this step's new tokens need and writes each token's position, cache
// slot and request, as rmsnorm_rope_kv_append takes them.
//
// Both are a scan over the requests followed by copies, a few kilobytes in
// all: bound by latency, that is by the number of dependent trips to memory.  One
// CTA scans (KV_PER requests a thread), lists the requests that move blocks, and
// moves all their blocks together, KV_BATCH loads in flight a thread, whatever
// request they belong to (a warp per request took 41 us to give back 80 requests
// of 128 blocks each among 4000, and 32 us to hand out 1400 single blocks).  The
// tokens are written by a second kernel over all SMs, or by the same CTA, from
// shared memory, when they are few.  Release and plan of 250 requests with a token
// each take 10.5 us of GPU time together, of 4000 with up to 64 tokens 25 us.
// Everything is in request order: the results are the same on every run.
//
// Lengths and block ids are device data and are checked there: a negative
// length, a stack that runs over or an id outside the pool sets
// RMSNORM_DEVSTATUS_BAD_INDEX, and nothing is read or written out of range.
#include "rmsnorm.h"

#include <algorithm>
#include <climits>

#include "checks.h"
#include "common.cuh"
#include "launch_util.h"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
int record_cuda_error(cudaError_t e);
}  // namespace rmsn

namespace {

using namespace rmsn;

constexpr int KV_NT = 1024;
constexpr int KV_PER = 4;                      // consecutive requests a thread scans
constexpr int KV_TILE = KV_NT * KV_PER;        // requests a pass of the CTA
constexpr int KV_BATCH = 4;                    // block ids a thread keeps in flight
constexpr int KV_TOKEN_NT = 256;
constexpr int KV_TOKENS = 2 * KV_TOKEN_NT;     // tokens a CTA of the second kernel writes
constexpr int KV_FUSED_TOKENS = 4096;          // the scanning CTA writes up to so many itself
constexpr unsigned int BAD_INDEX = RMSNORM_DEVSTATUS_BAD_INDEX;

struct KvArgs {
    const int32_t *lens, *new_lens;
    const uint8_t *finished;
    int32_t *table;
    int64_t ld_table, width, block;
    int32_t *free_blocks;          // the stack: entries [0, *free_count) are free block ids
    const int32_t *free_count;
    int64_t num_blocks;            // the stack's capacity; ids are below it
    int32_t *lens_out, *free_count_out;
    int64_t *starts, *positions, *slots;
    int32_t *requests;
    uint8_t *granted;
    int64_t B, T;
    unsigned int *status;
};

// Inclusive sums over the CTA of N sequences of KV_PER values a thread, in order;
// total[n] is the sum of all.  `sums` holds N int64 a warp; the CTA passes two
// barriers, whatever N.
template <int N>
__device__ __forceinline__ void cta_scan(int64_t (&v)[N][KV_PER], int64_t (*sums)[2], int64_t (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t own[N], run[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int k = 1; k < KV_PER; ++k) v[n][k] += v[n][k - 1];
        own[n] = run[n] = v[n][KV_PER - 1];
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t u = __shfl_up_sync(0xffffffffu, run[n], off);
            if (lane >= off) run[n] += u;
        }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) {
#pragma unroll
        for (int n = 0; n < N; ++n) sums[warp][n] = run[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        int64_t w = sums[lane][n];  // KV_NT / 32 == 32 warps
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += u;
        }
        total[n] = __shfl_sync(0xffffffffu, w, 31);
        const int64_t warps_before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
        const int64_t before = run[n] - own[n] + (warp ? warps_before : 0);
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) v[n][k] += before;
    }
}

// The requests of a tile that move blocks, in order.  A scanned word carries
// both a request's place in the list (its top bits) and its first block's place
// among all of them.
constexpr int KV_COUNT_SHIFT = 48;  // a tile moves fewer than 2^12 * 2^31 < 2^48 blocks
struct Moves {
    uint32_t first[KV_TILE]; // place of an entry's first block among the tile's (saturated)
    int32_t from[KV_TILE];   // index of its first block in its table row
    uint16_t req[KV_TILE];   // its request within the tile
};

struct PlanShared {
    int64_t sums[KV_NT / 32][2];
    unsigned long long last;
    union {
        Moves moves;
        struct {               // for the tokens, once the blocks are moved
            int64_t starts[KV_TILE + 1];
            int32_t base[KV_TILE];  // length before the step, or -1 - length if not granted
        } map;
    };
};

constexpr int64_t KV_BLOCKS = ((int64_t)1 << KV_COUNT_SHIFT) - 1;

__device__ __forceinline__ int64_t move_word(int64_t n) { return n + (n > 0 ? (int64_t)1 << KV_COUNT_SHIFT : 0); }

// Request k of this thread, whose inclusive sum of words is v, moves n blocks from
// block `from` of its row on.  The list may be read once the CTA has passed a
// barrier.
__device__ __forceinline__ void list_move(Moves &mv, int64_t v, int64_t n, int32_t from, int k) {
    const int at = (int)(v >> KV_COUNT_SHIFT) - 1;
    mv.first[at] = (uint32_t)min((v & KV_BLOCKS) - n, (int64_t)UINT32_MAX);
    mv.from[at] = from;
    mv.req[at] = (uint16_t)(threadIdx.x * KV_PER + k);
}

// The last i < n with a[i] <= x (a ascending, a[0] <= x).
template <typename A> __device__ __forceinline__ int last_at_most(const A *a, int n, A x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Moves the tile's `total` (below 2^31) blocks: load(row pointer at the block, its
// place), then store(row pointer, place, id), KV_BATCH of the first ahead of the
// second.
template <typename F, typename G>
__device__ __forceinline__ void move_blocks(const KvArgs &a, const Moves &mv, int entries, uint32_t total, int64_t b0,
                                            F load, G store) {
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += KV_NT * KV_BATCH) {
        int32_t *at[KV_BATCH];
        int32_t id[KV_BATCH];
#pragma unroll
        for (int i = 0; i < KV_BATCH; ++i) {
            const uint32_t e = e0 + i * KV_NT;
            if (e < total) {
                const int k = last_at_most(mv.first, entries, e);
                at[i] = a.table + (b0 + mv.req[k]) * a.ld_table + (mv.from[k] + (int64_t)(e - mv.first[k]));
                id[i] = load(at[i], e);
            }
        }
#pragma unroll
        for (int i = 0; i < KV_BATCH; ++i) {
            const uint32_t e = e0 + i * KV_NT;
            if (e < total) store(at[i], e, id[i]);
        }
    }
}

// The free count as loaded, clamped to what the stack holds.
__device__ __forceinline__ int64_t stack_top(const KvArgs &a, int64_t n) {
    if ((n < 0 || n > a.num_blocks) && threadIdx.x == 0) atomicOr(a.status, BAD_INDEX);
    return min(max(n, (int64_t)0), a.num_blocks);
}

// ceil(len / block), both below 2^31 (in 32 bits: the 64-bit divisions of the scan
// alone were a third of its instructions)
__device__ __forceinline__ int64_t blocks_of(uint32_t len, const KvArgs &a) {
    return (len + (uint32_t)a.block - 1u) / (uint32_t)a.block;
}

__global__ void __launch_bounds__(KV_NT) kv_release_kernel(const KvArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    PlanShared &sh = *reinterpret_cast<PlanShared *>(smem);
    griddep_wait();
    griddep_launch_dependents();
    const int32_t count = *a.free_count;  // in flight with the first requests' loads
    int64_t pushed = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += KV_TILE) {
        int32_t len[KV_PER];
        bool done[KV_PER];
        const int64_t b = b0 + threadIdx.x * KV_PER;
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            len[k] = b + k < a.B ? a.lens[b + k] : 0;
            done[k] = b + k < a.B && a.finished[b + k];
        }
        int64_t n[KV_PER], v[1][KV_PER], sum[1];
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            n[k] = done[k] && len[k] > 0 ? blocks_of((uint32_t)len[k], a) : 0;
            if (len[k] < 0 || n[k] > a.width) {  // such a request gives nothing back
                atomicOr(a.status, BAD_INDEX);
                n[k] = 0;
            }
            if (b + k < a.B) a.lens_out[b + k] = done[k] ? 0 : len[k];
            v[0][k] = move_word(n[k]);
        }
        cta_scan<1>(v, sh.sums, sum);
#pragma unroll
        for (int k = 0; k < KV_PER; ++k)
            if (n[k] > 0) list_move(sh.moves, v[0][k], n[k], 0, k);
        __syncthreads();
        const int entries = (int)(sum[0] >> KV_COUNT_SHIFT);
        const int64_t total = sum[0] & KV_BLOCKS, base = stack_top(a, count) + pushed;
        // what the stack has no room for is not pushed
        const int64_t room = max((int64_t)0, a.num_blocks - base);
        if (total > room && threadIdx.x == 0) atomicOr(a.status, BAD_INDEX);
        move_blocks(a, sh.moves, entries, (uint32_t)min(total, room), b0, [](const int32_t *p, uint32_t) { return *p; },
                    [&](const int32_t *, uint32_t e, int32_t id) {
                        if (id < 0 || id >= a.num_blocks) atomicOr(a.status, BAD_INDEX);
                        a.free_blocks[base + e] = id;
                    });
        pushed += total;
        __syncthreads();  // the list may be written again
    }
    __syncthreads();  // every thread has read the count it may overwrite
    if (threadIdx.x == 0) *a.free_count_out = (int32_t)min(stack_top(a, count) + pushed, a.num_blocks);
}

// Position, slot and request of token t, which is request `req`'s token number
// `off`; `base` is its length before the step, or -1 - length if not granted.
__device__ __forceinline__ void write_token(const KvArgs &a, int64_t t, int64_t req, int64_t off, int32_t base) {
    int64_t slot = -1;
    const bool ok = base >= 0;
    const int64_t pos = (ok ? (int64_t)base : -1 - (int64_t)base) + off;
    if (ok) {  // pos < 2^31
        const uint32_t blk = (uint32_t)pos / (uint32_t)a.block;
        const int32_t id = a.table[req * a.ld_table + blk];
        if (id < 0 || (a.free_count && id >= a.num_blocks)) atomicOr(a.status, BAD_INDEX);
        else slot = (int64_t)id * a.block + ((uint32_t)pos - blk * (uint32_t)a.block);
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
    a.requests[t] = (int32_t)req;
}

__device__ __forceinline__ void write_padding(const KvArgs &a, int64_t t) {
    a.positions[t] = 0;
    a.slots[t] = -1;
    a.requests[t] = -1;
}

// The scan over the requests; with `tokens` (one tile), the same CTA writes the
// tokens.
__global__ void __launch_bounds__(KV_NT) kv_plan_kernel(const KvArgs a, bool tokens) {
    extern __shared__ __align__(16) unsigned char smem[];
    PlanShared &sh = *reinterpret_cast<PlanShared *>(smem);
    griddep_wait();
    griddep_launch_dependents();
    const bool pool = a.free_count != nullptr;
    const int32_t count = pool ? *a.free_count : 0;  // in flight with the first requests' loads
    int64_t total_new = 0, total_need = 0, popped = 0;  // so far: tokens, blocks asked for, blocks taken
    int64_t start[KV_PER];
    int32_t base[KV_PER];  // for the tokens of the last tile
    for (int64_t b0 = 0; b0 < a.B; b0 += KV_TILE) {
        const int64_t b = b0 + threadIdx.x * KV_PER;
        int32_t len[KV_PER], add[KV_PER];
        bool valid[KV_PER];
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            valid[k] = b + k < a.B;
            len[k] = valid[k] ? a.lens[b + k] : 0;
            add[k] = valid[k] ? a.new_lens[b + k] : 0;
        }
        int64_t need[KV_PER], v[2][KV_PER], sum[2];  // v: tokens, words of blocks
        int32_t have[KV_PER];
        bool fits[KV_PER];
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            if (len[k] < 0 || add[k] < 0) {
                atomicOr(a.status, BAD_INDEX);
                valid[k] = false;
                add[k] = 0;
            }
            const int64_t all = (int64_t)len[k] + add[k];
            valid[k] = valid[k] && all <= INT_MAX;
            const int64_t h = valid[k] ? blocks_of((uint32_t)len[k], a) : 0;
            const int64_t want = valid[k] ? blocks_of((uint32_t)all, a) : 0;
            fits[k] = valid[k] && want <= a.width;
            need[k] = fits[k] && pool ? want - h : 0;
            have[k] = (int32_t)min(h, (int64_t)INT_MAX);
            v[0][k] = add[k];
            v[1][k] = move_word(need[k]);
        }
        cta_scan<2>(v, sh.sums, sum);
        if (total_new + sum[0] > a.T) {  // the last requests' tokens do not fit: their blocks do not count
            int64_t again[1][KV_PER], sum1[1];
#pragma unroll
            for (int k = 0; k < KV_PER; ++k) {
                fits[k] = fits[k] && total_new + v[0][k] <= a.T;
                need[k] = fits[k] ? need[k] : 0;
                again[0][k] = move_word(need[k]);
            }
            cta_scan<1>(again, sh.sums, sum1);
#pragma unroll
            for (int k = 0; k < KV_PER; ++k) v[1][k] = again[0][k];
            sum[1] = sum1[0];
        }
        // Requests that need blocks are granted in order until the stack runs out, so
        // the tile's blocks are the next ones off the stack, and the list's entries
        // the first so many.
        const int64_t top = pool ? stack_top(a, count) : 0;
        int64_t granted_word = 0;
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            const bool ok = fits[k] && (need[k] == 0 || total_need + (v[1][k] & KV_BLOCKS) <= top);
            start[k] = total_new + v[0][k] - add[k];
            base[k] = ok ? len[k] : -1 - max(len[k], 0);
            if (ok && need[k] > 0) {
                list_move(sh.moves, v[1][k], need[k], have[k], k);
                granted_word = v[1][k];
            }
            if (b + k < a.B) {
                a.starts[b + k] = start[k];
                a.granted[b + k] = ok ? 1 : 0;
                a.lens_out[b + k] = ok ? len[k] + add[k] : len[k];
            }
        }
        total_new += sum[0];
        int64_t moved = sum[1];
        if (total_need + (moved & KV_BLOCKS) > top) {  // not all of them were: the last one's word
            if (threadIdx.x == 0) sh.last = 0;
            __syncthreads();
            if (granted_word) atomicMax(&sh.last, (unsigned long long)granted_word);
            __syncthreads();
            moved = (int64_t)sh.last;
        }
        total_need += sum[1] & KV_BLOCKS;
        const int entries = (int)(moved >> KV_COUNT_SHIFT);
        const int64_t total = moved & KV_BLOCKS;
        __syncthreads();
        const int64_t from = top - 1 - popped;
        move_blocks(a, sh.moves, entries, (uint32_t)total, b0,
                    [&](const int32_t *, uint32_t e) { return a.free_blocks[from - e]; },
                    [&](int32_t *p, uint32_t, int32_t id) {
                        if (id < 0 || id >= a.num_blocks) atomicOr(a.status, BAD_INDEX);
                        *p = id;
                    });
        popped += total;
        __syncthreads();  // the list may be written again
    }
    __syncthreads();  // every thread has read the count it may overwrite
    if (threadIdx.x == 0) {
        a.starts[a.B] = total_new;
        if (pool) *a.free_count_out = (int32_t)(stack_top(a, count) - popped);
    }
    if (tokens) {
        const int n = (int)a.B;
#pragma unroll
        for (int k = 0; k < KV_PER; ++k) {
            const int b = threadIdx.x * KV_PER + k;
            if (b < n) {
                sh.map.starts[b] = start[k];
                sh.map.base[b] = base[k];
            }
        }
        __syncthreads();  // with the table entries written above
        for (int64_t t = threadIdx.x; t < a.T; t += KV_NT) {
            if (t < total_new) {
                const int req = last_at_most(sh.map.starts, n, t);
                write_token(a, t, req, t - sh.map.starts[req], sh.map.base[req]);
            } else {
                write_padding(a, t);
            }
        }
    }
}

// The last request whose first token is at or before t, by a whole warp: 32
// probes a step.
__device__ __forceinline__ int64_t request_of(const KvArgs &a, int64_t t) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = a.B;  // in [lo, lo + n)
    while (n > 1) {
        const int64_t step = (n + 31) / 32;
        const int64_t at = lo + lane * step;
        const bool below = lane * step < n && a.starts[at] <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));  // lane 0 always is
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// A CTA writes KV_TOKENS consecutive tokens.  Two warps find its first and last
// requests; their starts go to shared memory, where every token finds its own.
__global__ void __launch_bounds__(KV_TOKEN_NT) kv_tokens_kernel(const KvArgs a) {
    constexpr int CAP = 2048;  // requests a CTA's tokens usually span fewer of
    __shared__ int64_t s_starts[CAP + 1];
    __shared__ int32_t s_base[CAP];
    __shared__ int64_t s_range[2];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t total = a.starts[a.B];
    const int warp = threadIdx.x >> 5;
    for (int64_t t0 = (int64_t)blockIdx.x * KV_TOKENS; t0 < a.T; t0 += (int64_t)gridDim.x * KV_TOKENS) {
        const int64_t t1 = min(min(t0 + KV_TOKENS, a.T), total);  // its live tokens end
        if (warp < 2 && t0 < t1) {
            const int64_t r = request_of(a, warp == 0 ? t0 : t1 - 1);
            if ((threadIdx.x & 31) == 0) s_range[warp] = r;
        }
        __syncthreads();
        const int64_t lo = t0 < t1 ? s_range[0] : 0, n = t0 < t1 ? s_range[1] - lo + 1 : 0;
        const bool fits = n <= CAP;
        auto base_of = [&](int64_t req, int64_t s0, int64_t s1) -> int32_t {
            const int32_t len = a.lens_out[req];
            return a.granted[req] ? (int32_t)(len - (s1 - s0)) : -1 - max(len, 0);
        };
        if (fits) {
            for (int i = threadIdx.x; i < n; i += KV_TOKEN_NT) {
                const int64_t s0 = a.starts[lo + i], s1 = a.starts[lo + i + 1];
                s_starts[i] = s0;
                s_base[i] = base_of(lo + i, s0, s1);
            }
        }
        __syncthreads();
        for (int64_t t = t0 + threadIdx.x; t < min(t0 + KV_TOKENS, a.T); t += KV_TOKEN_NT) {
            if (t >= total) {
                write_padding(a, t);
            } else if (fits) {
                const int i = last_at_most(s_starts, (int)n, t);
                write_token(a, t, lo + i, t - s_starts[i], s_base[i]);
            } else {
                const int64_t req = lo + last_at_most(a.starts + lo, (int)n, t);
                const int64_t s0 = a.starts[req];
                write_token(a, t, req, t - s0, base_of(req, s0, a.starts[req + 1]));
            }
        }
        __syncthreads();  // the starts are written again
    }
}

struct Buf {
    const void *p;
    size_t n;
    bool out;
    int same;  // index of the buffer it may coincide with, or -1
};

// Every written buffer is apart from every other one, but for an output that
// is its input.
bool buffers_ok(const Buf *b, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && b[i].out && overlaps(b[i].p, b[i].n, b[j].p, b[j].n) &&
                !((b[i].same == j || b[j].same == i) && b[i].p == b[j].p))
                return false;
    return true;
}

bool shapes_ok(int64_t B, int64_t width, int64_t ld_table, int64_t block, int64_t num_blocks) {
    return B >= 0 && width >= 0 && ld_table >= width && block > 0 && num_blocks >= 0;
}

bool sizes_ok(int64_t B, int64_t ld_table, int64_t block, int64_t num_blocks) {
    return B <= ((int64_t)1 << 31) - 2 && num_blocks < INT_MAX && block <= INT_MAX &&
           (ld_table == 0 || B <= (INT64_MAX / 8) / ld_table);
}

size_t table_bytes(int64_t B, int64_t width, int64_t ld_table) {
    return B > 0 && width > 0 ? ((size_t)(B - 1) * ld_table + width) * 4 : 0;
}

bool al(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace

extern "C" int rmsnorm_kv_release(const int32_t *lens, const uint8_t *finished, const int32_t *block_table,
                                  int64_t ld_table, int64_t table_width, int64_t block_size,
                                  int32_t *free_blocks, const int32_t *free_count, int64_t num_blocks,
                                  int32_t *lens_out, int32_t *free_count_out, int64_t B, void *stream) {
    if (!shapes_ok(B, table_width, ld_table, block_size, num_blocks)) return RMSNORM_ERR_INVALID_ARG;
    if (!sizes_ok(B, ld_table, block_size, num_blocks)) return RMSNORM_ERR_UNSUPPORTED;
    if (!free_count || !free_count_out || (num_blocks > 0 && !free_blocks) ||
        (B > 0 && (!lens || !finished || !lens_out || (table_width > 0 && !block_table))))
        return RMSNORM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)block_table, (const void *)free_blocks,
                          (const void *)free_count, (const void *)lens_out, (const void *)free_count_out})
        if (!al(p, 4)) return RMSNORM_ERR_INVALID_ARG;
    const size_t nb = (size_t)B;
    const Buf bufs[] = {{lens, nb * 4, false, 3}, {finished, nb, false, -1},
                        {block_table, table_bytes(B, table_width, ld_table), false, -1},
                        {lens_out, nb * 4, true, 0}, {free_blocks, (size_t)num_blocks * 4, true, -1},
                        {free_count, 4, false, 6}, {free_count_out, 4, true, 5}};
    if (!buffers_ok(bufs, 7)) return RMSNORM_ERR_INVALID_ARG;
    KvArgs a{};
    const int st = current_status_word(&a.status);
    if (st != RMSNORM_OK) return st;
    a.lens = lens; a.finished = finished;
    a.table = const_cast<int32_t *>(block_table);  // read only here
    a.ld_table = ld_table; a.width = table_width; a.block = block_size;
    a.free_blocks = free_blocks; a.free_count = free_count; a.num_blocks = num_blocks;
    a.lens_out = lens_out; a.free_count_out = free_count_out;
    a.B = B;
    static std::atomic<uint64_t> smem_mask{0};
    cudaError_t e = allow_max_dynamic_smem((const void *)kv_release_kernel, smem_mask);
    if (e == cudaSuccess)
        e = launch_pdl(kv_release_kernel, dim3(1), dim3(KV_NT), sizeof(PlanShared), static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

extern "C" int rmsnorm_kv_plan(const int32_t *lens, const int32_t *new_lens, int32_t *block_table,
                               int64_t ld_table, int64_t table_width, int64_t block_size,
                               const int32_t *free_blocks, const int32_t *free_count, int64_t num_blocks,
                               int32_t *lens_out, int32_t *free_count_out, int64_t *starts,
                               int64_t *positions, int64_t *slots, int32_t *requests, uint8_t *granted,
                               int64_t B, int64_t T, void *stream) {
    if (!shapes_ok(B, table_width, ld_table, block_size, num_blocks) || T < 0) return RMSNORM_ERR_INVALID_ARG;
    if (!sizes_ok(B, ld_table, block_size, num_blocks) || T > INT_MAX) return RMSNORM_ERR_UNSUPPORTED;
    if ((free_count != nullptr) != (free_count_out != nullptr) || (free_blocks && !free_count) ||
        (free_count && num_blocks > 0 && !free_blocks))
        return RMSNORM_ERR_INVALID_ARG;
    if (!starts || (B > 0 && (!lens || !new_lens || !lens_out || !granted || (table_width > 0 && !block_table))) ||
        (T > 0 && (!positions || !slots || !requests)))
        return RMSNORM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)new_lens, (const void *)block_table,
                          (const void *)free_blocks, (const void *)free_count, (const void *)lens_out,
                          (const void *)free_count_out, (const void *)requests})
        if (!al(p, 4)) return RMSNORM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)starts, (const void *)positions, (const void *)slots})
        if (!al(p, 8)) return RMSNORM_ERR_INVALID_ARG;
    const size_t nb = (size_t)B, nt = (size_t)T;
    const Buf bufs[] = {{lens, nb * 4, false, 3}, {new_lens, nb * 4, false, -1},
                        {block_table, table_bytes(B, table_width, ld_table), true, -1},
                        {lens_out, nb * 4, true, 0},
                        {free_blocks, (size_t)num_blocks * 4, false, -1},
                        {free_count, 4, false, 6}, {free_count_out, 4, true, 5},
                        {starts, (nb + 1) * 8, true, -1}, {positions, nt * 8, true, -1},
                        {slots, nt * 8, true, -1}, {requests, nt * 4, true, -1}, {granted, nb, true, -1}};
    if (!buffers_ok(bufs, 12)) return RMSNORM_ERR_INVALID_ARG;
    KvArgs a{};
    int sm = 0;
    int st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&a.status);
    if (st != RMSNORM_OK) return st;
    a.lens = lens; a.new_lens = new_lens;
    a.table = block_table; a.ld_table = ld_table; a.width = table_width; a.block = block_size;
    a.free_blocks = const_cast<int32_t *>(free_blocks);  // read only here
    a.free_count = free_count; a.num_blocks = num_blocks;
    a.lens_out = lens_out; a.free_count_out = free_count_out;
    a.starts = starts; a.positions = positions; a.slots = slots; a.requests = requests; a.granted = granted;
    a.B = B; a.T = T;
    const bool fused = T <= KV_FUSED_TOKENS && B <= KV_TILE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    static std::atomic<uint64_t> smem_mask{0};
    cudaError_t e = allow_max_dynamic_smem((const void *)kv_plan_kernel, smem_mask);
    if (e == cudaSuccess) e = launch_pdl(kv_plan_kernel, dim3(1), dim3(KV_NT), sizeof(PlanShared), s, a, fused);
    if (e == cudaSuccess && !fused) {
        const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((T + KV_TOKENS - 1) / KV_TOKENS, (int64_t)sm * 8));
        e = launch_pdl(kv_tokens_kernel, dim3(grid), dim3(KV_TOKEN_NT), 0, s, a);
    }
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}
