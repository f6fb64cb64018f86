// slots.hip -- the slots of a state pool: states copied, slots counted and acquired, the pool
// compacted.
//
// A pool [layers][slots] of equal states and a count of uses per slot (0: free). A state is
// moved whole, so the copies are bound by memory, two bytes of traffic a byte: 16-byte loads
// and stores with the non-temporal hint (nothing is read twice), 16 KB a workgroup. 96 states of 2 MB:
// 402 MB in 71 us, 5.6 TB/s (32 KB a workgroup 103 us, 8 KB 71, without the hint 77); the call with its
// release and acquire 78 us. 144 states moved by compaction: 118 us.
// The index work is a few thousand whole numbers at most: one workgroup, prefix sums by
// ballots, every result independent of the order in which threads run.
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int NT = 512, PER = 2;
constexpr size_t CHUNK = (size_t)NT * PER * 16;      // bytes a workgroup moves at a time

// One chunk of a state; from == nullptr: zeros.
__device__ __forceinline__ void move_chunk(const char *from, char *to, size_t chunk, size_t bytes, int t) {
    const size_t at = chunk * CHUNK + (size_t)t * 16;
    u32x4 x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        x[i] = u32x4{0u, 0u, 0u, 0u};
        const size_t b = at + (size_t)i * NT * 16;
        if (from && b < bytes) x[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(from + b));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const size_t b = at + (size_t)i * NT * 16;
        if (b < bytes) __builtin_nontemporal_store(x[i], reinterpret_cast<u32x4 *>(to + b));
    }
}

__global__ __launch_bounds__(NT) void copy_kernel(const char *from, char *to, const int32_t *__restrict__ src,
                                                  const int32_t *__restrict__ dst, int layers, int from_slots, int to_slots,
                                                  size_t bytes, unsigned chunks) {
    const unsigned item = blockIdx.x / chunks, chunk = blockIdx.x % chunks, i = item / layers, layer = item % layers;
    const int s = src[i], d = dst[i];
    if (d < 0 || d >= to_slots) return;
    const char *p = s >= 0 && s < from_slots ? from + ((size_t)layer * from_slots + s) * bytes : nullptr;
    move_chunk(p, to + ((size_t)layer * to_slots + d) * bytes, chunk, bytes, threadIdx.x);
}

// uses[which[i]] += add for every i; a count that would fall below zero is zero.
__global__ __launch_bounds__(1024) void count_kernel(int32_t *uses, const int32_t *__restrict__ which, int n, int slots, int add) {
    for (int i = threadIdx.x; i < n; i += 1024) {
        const int s = which[i];
        if (s >= 0 && s < slots) atomicAdd(&uses[s], add);
    }
    if (add > 0) return;
    __threadfence();                         // every count is final before the first is looked at
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 1024) {
        const int s = which[i];
        if (s >= 0 && s < slots) atomicMax(&uses[s], 0);
    }
}

// How many threads before this one in the workgroup, and in all, hold true.
__device__ __forceinline__ int rank_of(bool x, int *waves, int t, int &all) {
    const unsigned long long b = __ballot(x);
    __syncthreads();                         // the last sums have been read
    if ((t & 63) == 0) waves[t >> 6] = __popcll(b);
    __syncthreads();
    int before = __popcll(b & ((1ull << (t & 63)) - 1));
    all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if (w < (t >> 6)) before += waves[w];
        all += waves[w];
    }
    return before;
}

__global__ __launch_bounds__(1024) void acquire_kernel(int32_t *uses, int slots, int32_t *taken, int n) {
    __shared__ int waves[16];
    const int t = threadIdx.x;
    int found = 0;
    for (int s0 = 0; s0 < slots && found < n; s0 += 1024) {
        const int s = s0 + t;
        const bool free = s < slots && uses[s] <= 0;
        int all;
        const int r = found + rank_of(free, waves, t, all);
        if (free && r < n) {
            taken[r] = s;
            uses[s] = 1;
        }
        found += all;
    }
    for (int i = found + t; i < n; i += 1024) taken[i] = -1;
}

// Which live slots move where: those at or behind the count of live ones, in ascending order, to the
// free ones before it. moved[s]: a slot's new place (-1: it was free); moves: [0] how many, then
// pairs (from, to). Counts go with their slots; entries of table follow.
__global__ __launch_bounds__(1024) void plan_kernel(int32_t *uses, int slots, int32_t *moved, int32_t *moves, int32_t *count,
                                                    int32_t *table, int table_n) {
    __shared__ int waves[16];
    const int t = threadIdx.x;
    int live = 0;
    for (int s0 = 0; s0 < slots; s0 += 1024) {
        int all;
        rank_of(s0 + t < slots && uses[s0 + t] > 0, waves, t, all);
        live += all;
    }
    int from = 0, to = 0;
    for (int s0 = 0; s0 < slots; s0 += 1024) {
        const int s = s0 + t;
        const bool in = s < slots, used = in && uses[s] > 0;
        int all;
        const bool mover = used && s >= live;
        int r = from + rank_of(mover, waves, t, all);
        from += all;
        if (mover) moves[1 + 2 * r] = s;
        const bool hole = in && !used && s < live;
        r = to + rank_of(hole, waves, t, all);
        to += all;
        if (hole) moves[2 + 2 * r] = s;
        if (in) moved[s] = used ? s : -1;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = t; i < from; i += 1024) {
        const int s = moves[1 + 2 * i], d = moves[2 + 2 * i];
        moved[s] = d;
        uses[d] = uses[s];
        uses[s] = 0;
    }
    if (t == 0) {
        moves[0] = from;
        *count = live;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = t; i < table_n; i += 1024) {
        const int s = table[i];
        if (s >= 0 && s < slots) table[i] = moved[s];
    }
}

__global__ __launch_bounds__(NT) void moves_kernel(char *pool, const int32_t *__restrict__ moves, int slots, int layers,
                                                   size_t bytes, unsigned chunks) {
    const unsigned long long all = (unsigned long long)moves[0] * layers * chunks;
    for (unsigned long long u = blockIdx.x; u < all; u += gridDim.x) {
        const unsigned chunk = u % chunks, i = u / chunks / layers, layer = u / chunks % layers;
        char *base = pool + (size_t)layer * slots * bytes;
        move_chunk(base + (size_t)moves[1 + 2 * i] * bytes, base + (size_t)moves[2 + 2 * i] * bytes, chunk, bytes, threadIdx.x);
    }
}

}  // namespace

// a copy's workgroups times their threads stay below 2^32
bool slots_copy_fits(long long n, int layers, size_t slot_bytes) {
    const double chunks = (double)(slot_bytes / CHUNK + 1);
    return (double)n * layers * chunks < (double)(1 << 23);
}

// compaction's workgroups take chunks in turn, so only its counts have to fit
bool slots_compact_fits(int slots, size_t slot_bytes) { return slots < (1 << 25) && slot_bytes / CHUNK < (1u << 31); }

hipError_t launch_slots_copy(const SlotsCopyArgs &a) {
    const unsigned chunks = (unsigned)((a.slot_bytes + CHUNK - 1) / CHUNK);
    hipLaunchKernelGGL(copy_kernel, dim3((unsigned)a.n * a.layers * chunks), dim3(NT), 0, a.stream, a.from, a.to, a.src, a.dst,
                       a.layers, a.from_slots, a.to_slots, a.slot_bytes, chunks);
    return hipGetLastError();
}

hipError_t launch_slots_count(int32_t *uses, const int32_t *which, int n, int slots, int add, hipStream_t stream) {
    hipLaunchKernelGGL(count_kernel, dim3(1), dim3(1024), 0, stream, uses, which, n, slots, add);
    return hipGetLastError();
}

hipError_t launch_slots_acquire(int32_t *uses, int slots, int32_t *taken, int n, hipStream_t stream) {
    hipLaunchKernelGGL(acquire_kernel, dim3(1), dim3(1024), 0, stream, uses, slots, taken, n);
    return hipGetLastError();
}

hipError_t launch_slots_compact(const SlotsCompactArgs &a) {
    int32_t *moves = a.moved + a.slots;
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(1024), 0, a.stream, a.uses, a.slots, a.moved, moves, a.count, a.table, a.table_n);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned chunks = (unsigned)((a.slot_bytes + CHUNK - 1) / CHUNK);
    // at most half of the slots move; workgroups beyond eight a CU take more than one chunk
    const unsigned long long most = (unsigned long long)(a.slots / 2) * a.layers * chunks;
    if (most == 0) return hipSuccess;
    hipLaunchKernelGGL(moves_kernel, dim3((unsigned)(most < 2048 ? most : 2048)), dim3(NT), 0, a.stream, a.pool, moves, a.slots,
                       a.layers, a.slot_bytes, chunks);
    return hipGetLastError();
}

}  // namespace kda
