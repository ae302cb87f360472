// kv_plan.cu -- block tables and slot maps of a paged KV cache, built on the GPU
// from the requests' lengths: rmsnorm_kv_release gives finished requests'
// blocks back to the pool's stack of free ones, rmsnorm_kv_plan takes the
// blocks this step's new tokens need and writes each token's position, cache
// slot and request, as rmsnorm_rope_kv_append takes them.
//
// Both are a scan over the requests followed by copies, a few kilobytes in
// all: bound by latency.  One CTA scans (a request a thread, tiles of KV_NT
// requests with a carry) and moves the blocks, a warp per request that has any;
// the tokens are written by a second kernel over all SMs, or by the same CTA
// when they are few.  Everything is in request order: the results are the same
// on every run.
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
constexpr int KV_TOKEN_NT = 256;
constexpr int KV_FUSED_TOKENS = 4096;
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

// Inclusive sum of v over the CTA's threads in thread order; *total is the
// CTA's sum.  `sums` holds an int64 a warp; the CTA passes two barriers.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *sums, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t w = lane < KV_NT / 32 ? sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v + (warp ? before : 0);
}

// The free count, clamped to what the stack holds.
__device__ __forceinline__ int64_t stack_top(const KvArgs &a) {
    const int64_t n = *a.free_count;
    if ((n < 0 || n > a.num_blocks) && threadIdx.x == 0) atomicOr(a.status, BAD_INDEX);
    return min(max(n, (int64_t)0), a.num_blocks);
}

__global__ void __launch_bounds__(KV_NT) kv_release_kernel(const KvArgs a) {
    __shared__ int64_t sums[KV_NT / 32];
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t top = stack_top(a);
    int64_t pushed = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += KV_NT) {
        const int64_t b = b0 + threadIdx.x;
        const int64_t len = b < a.B ? a.lens[b] : 0;
        const bool done = b < a.B && a.finished[b];
        int64_t n = done && len > 0 ? (len + a.block - 1) / a.block : 0;
        if (len < 0 || n > a.width) {  // such a request gives nothing back
            atomicOr(a.status, BAD_INDEX);
            n = 0;
        }
        int64_t total;
        const int64_t first = top + pushed + cta_scan(n, sums, &total) - n;
        pushed += total;
        for (unsigned todo = __ballot_sync(0xffffffffu, n > 0); todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1;
            const int64_t nj = __shfl_sync(0xffffffffu, n, j), at = __shfl_sync(0xffffffffu, first, j);
            const int32_t *row = a.table + (b - lane + j) * a.ld_table;
            for (int64_t i = lane; i < nj; i += 32) {
                const int32_t id = row[i];
                if (id < 0 || id >= a.num_blocks || at + i >= a.num_blocks) atomicOr(a.status, BAD_INDEX);
                if (at + i < a.num_blocks) a.free_blocks[at + i] = id;
            }
        }
        if (b < a.B) a.lens_out[b] = done ? 0 : (int32_t)len;
    }
    __syncthreads();  // every thread has read the count it may overwrite
    if (threadIdx.x == 0) *a.free_count_out = (int32_t)min(top + pushed, a.num_blocks);
    griddep_launch_dependents();
}

// Position, slot and request of token t.
__device__ __forceinline__ void write_token(const KvArgs &a, int64_t t, int64_t total) {
    int64_t pos = 0, slot = -1;
    int32_t req = -1;
    if (t < total) {
        int64_t lo = 0, hi = a.B;  // the last request whose first token is at or before t
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.starts[mid] <= t) lo = mid; else hi = mid;
        }
        const int64_t s0 = a.starts[lo], s1 = a.starts[lo + 1];
        const bool ok = a.granted[lo] != 0;
        req = (int32_t)lo;
        pos = (int64_t)a.lens_out[lo] - (ok ? s1 - s0 : 0) + (t - s0);
        if (ok) {
            const int64_t blk = pos / a.block;
            const int32_t id = a.table[lo * a.ld_table + blk];
            if (id < 0 || (a.free_count && id >= a.num_blocks)) atomicOr(a.status, BAD_INDEX);
            else slot = (int64_t)id * a.block + (pos - blk * a.block);
        } else {
            pos = max(pos, (int64_t)0);
        }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
    a.requests[t] = req;
}

// The scan over the requests; with `tokens`, the same CTA writes the tokens.
__global__ void __launch_bounds__(KV_NT) kv_plan_kernel(const KvArgs a, bool tokens) {
    __shared__ int64_t sums[KV_NT / 32];
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const bool pool = a.free_count != nullptr;
    const int64_t top = pool ? stack_top(a) : 0;
    int64_t total_new = 0, total_need = 0, popped = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += KV_NT) {
        const int64_t b = b0 + threadIdx.x;
        int64_t len = 0, add = 0;
        bool valid = b < a.B;
        if (valid) {
            len = a.lens[b];
            add = a.new_lens[b];
            if (len < 0 || add < 0) {
                atomicOr(a.status, BAD_INDEX);
                valid = false;
                add = 0;
            }
        }
        int64_t tile_new, tile_need;
        const int64_t end = total_new + cta_scan(add, sums, &tile_new);
        const int64_t have = valid ? (len + a.block - 1) / a.block : 0;
        const int64_t want = valid ? (len + add + a.block - 1) / a.block : 0;
        const bool fits = valid && want <= a.width && end <= a.T && len + add <= INT_MAX;
        const int64_t need = fits && pool ? want - have : 0;
        const int64_t cum = total_need + cta_scan(need, sums, &tile_need);
        const bool ok = fits && (need == 0 || cum <= top);
        total_new += tile_new;
        total_need += tile_need;
        const int64_t take = ok ? need : 0;
        if (take) popped = max(popped, cum);
        for (unsigned todo = __ballot_sync(0xffffffffu, take > 0); todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1;
            const int64_t n = __shfl_sync(0xffffffffu, take, j);
            const int64_t from = top - 1 - (__shfl_sync(0xffffffffu, cum, j) - n);
            int32_t *row = a.table + (b - lane + j) * a.ld_table + __shfl_sync(0xffffffffu, have, j);
            for (int64_t i = lane; i < n; i += 32) {
                const int32_t id = a.free_blocks[from - i];
                if (id < 0 || id >= a.num_blocks) atomicOr(a.status, BAD_INDEX);
                row[i] = id;
            }
        }
        if (b < a.B) {
            a.starts[b] = end - add;
            a.granted[b] = ok ? 1 : 0;
            a.lens_out[b] = (int32_t)(ok ? len + add : len);
        }
    }
    // blocks taken: the furthest any granted request reached
    for (int off = 16; off > 0; off >>= 1) popped = max(popped, __shfl_xor_sync(0xffffffffu, popped, off));
    __syncthreads();
    if (lane == 0) sums[threadIdx.x >> 5] = popped;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < KV_NT / 32; ++w) popped = max(popped, sums[w]);
        a.starts[a.B] = total_new;
        if (pool) *a.free_count_out = (int32_t)(top - popped);
    }
    griddep_launch_dependents();
    if (tokens) {
        __syncthreads();  // this CTA's own writes above
        for (int64_t t = threadIdx.x; t < a.T; t += KV_NT) write_token(a, t, total_new);
    }
}

__global__ void __launch_bounds__(KV_TOKEN_NT) kv_tokens_kernel(const KvArgs a) {
    griddep_wait();
    const int64_t total = a.starts[a.B];
    for (int64_t t = (int64_t)blockIdx.x * KV_TOKEN_NT + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * KV_TOKEN_NT)
        write_token(a, t, total);
    griddep_launch_dependents();
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
    const cudaError_t e = launch_pdl(kv_release_kernel, dim3(1), dim3(KV_NT), 0,
                                     static_cast<cudaStream_t>(stream), a);
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
    const bool fused = T <= KV_FUSED_TOKENS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(kv_plan_kernel, dim3(1), dim3(KV_NT), 0, s, a, fused);
    if (e == cudaSuccess && !fused) {
        const int grid = (int)std::min<int64_t>((T + KV_TOKEN_NT - 1) / KV_TOKEN_NT, (int64_t)sm * 8);
        e = launch_pdl(kv_tokens_kernel, dim3(grid), dim3(KV_TOKEN_NT), 0, s, a);
    }
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}
