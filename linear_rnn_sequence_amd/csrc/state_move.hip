// Moves of states between the slots of a pool: pool[dst[i]] = old pool[src[i]]
// for all i at once (copies, forks, permutations, compaction, zeroing).
//
// Targets may be other pairs' sources, so every source has to be read before
// any target is written.  The slots are cut into pieces of at most 8 KiB at the
// same place in every slot; a workgroup takes one piece of all n pairs, loads
// its n sources into registers (at most 64 KiB: 512 threads x 8 x 16 bytes),
// waits for all of them, and writes.  No two workgroups touch the same bytes,
// so nothing else has to be ordered, and each byte is read and written once.
// The list of pairs is read and resolved (bounds, and which of several pairs
// with the same target is the last) once per workgroup, which then walks over
// pieces of all layers; four workgroups per CU overlap one's loads with
// another's stores.  48 moves of 32 layers with 655 KB a slot, a quarter of them zeroes,
// read 0.70 GB and write 1.01 GB in 346 us, 4.9 TB/s; 64 moves of 12 layers with 197 KB whose
// sources repeat read 0.11 GB and write 0.15 GB in 49 us, 5.3 TB/s; a large copy reaches
// 6.6 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gated_delta.h"

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kPer = 8;                // pieces of 16 bytes a thread holds
constexpr int kMax = STATE_MOVE_MAX;
constexpr int kTable = 2 * kMax;       // hash table of targets, at most half full
static_assert((kTable & (kTable - 1)) == 0, "power of two");
static_assert(kMax * 64 <= kThreads * kPer * 16, "64-byte pieces of the most pairs fit");

struct MoveArgs {
    char *pool;
    size_t layer_bytes, slot_bytes;
    const int *src, *dst;
    int layers, slots, n;
    int lanes;             // threads per piece: piece bytes / 16, a power of two
    unsigned pieces;       // per slot
};

__global__ __launch_bounds__(kThreads) void state_move_kernel(MoveArgs p) {
    __shared__ int sKey[kTable], sLast[kTable];
    // the pairs as they were read once (targets out of range: -1): were they read again for the
    // search below, a list that is written meanwhile would make it look for what is not there
    __shared__ int sSrc[kMax], sDst[kMax];
    const int tid = threadIdx.x;
    for (int i = tid; i < kTable; i += kThreads) {
        sKey[i] = -1;
        sLast[i] = -1;
    }
    __syncthreads();
    auto valid = [&](int s, int d) { return d >= 0 && d < p.slots && s >= -1 && s < p.slots; };
    auto hash = [](int d) { return (int)(((unsigned)d * 2654435761u) >> 16) & (kTable - 1); };
    for (int i = tid; i < p.n; i += kThreads) {
        const int s = p.src[i], d = p.dst[i];
        sSrc[i] = s;
        sDst[i] = valid(s, d) ? d : -1;
        if (!valid(s, d)) continue;
        int h = hash(d);
        // ends: at most kMax of the kTable places are ever taken
        for (;;) {
            const int old = atomicCAS(&sKey[h], -1, d);
            if (old == -1 || old == d) break;
            h = (h + 1) & (kTable - 1);
        }
        atomicMax(&sLast[h], i);
    }
    __syncthreads();
    // this thread's part of up to kPer pairs
    const int sub = tid & (p.lanes - 1), row0 = tid / p.lanes, rows = kThreads / p.lanes;
    long long from[kPer], to[kPer];  // byte offsets in a layer; from -1: zeros, to -1: no pair
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = row0 + j * rows;
        from[j] = to[j] = -1;
        if (i >= p.n) continue;
        const int s = sSrc[i], d = sDst[i];
        if (d < 0) continue;
        int h = hash(d);
        while (sKey[h] != d) h = (h + 1) & (kTable - 1);  // it was put there above
        if (sLast[h] != i) continue;
        to[j] = (long long)d * (long long)p.slot_bytes + sub * 16;
        from[j] = s < 0 ? -1 : (long long)s * (long long)p.slot_bytes + sub * 16;
    }
    const unsigned long long all = (unsigned long long)p.pieces * p.layers;
    for (unsigned long long w = blockIdx.x; w < all; w += gridDim.x) {
        const size_t in_slot = (size_t)(w % p.pieces) * p.lanes * 16;
        char *base = p.pool + (size_t)(w / p.pieces) * p.layer_bytes + in_slot;
        const bool inside = in_slot + sub * 16 < p.slot_bytes;
        u32x4 x[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            x[j] = u32x4{0u, 0u, 0u, 0u};
            if (inside && from[j] >= 0)
                x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(base + from[j]));
        }
        // the sources are in registers before any wave passes the barrier
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (inside && to[j] >= 0)
                __builtin_nontemporal_store(x[j], reinterpret_cast<u32x4 *>(base + to[j]));
    }
}

}  // namespace

extern "C" rwkv7_status state_move(void *pool, int layers, size_t layer_bytes, int slots,
                                   size_t slot_bytes, const int *src, const int *dst, int n,
                                   void *stream) {
    if (layers < 1 || slots < 1 || n < 0 || n > STATE_MOVE_MAX) return RWKV7_ERR_SHAPE;
    if (slot_bytes == 0 || slot_bytes % 16 || slot_bytes > SIZE_MAX / 4 / (size_t)slots)
        return RWKV7_ERR_SHAPE;
    const size_t one = slot_bytes * (size_t)slots;
    if (layers == 1) layer_bytes = one;
    if (layer_bytes % 16 || layer_bytes < one || layer_bytes > SIZE_MAX / 4 / (size_t)layers)
        return RWKV7_ERR_SHAPE;
    if (n == 0) return RWKV7_OK;
    if (!pool || !src || !dst) return RWKV7_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pool) & 15u) return RWKV7_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3u)
        return RWKV7_ERR_ALIGN;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(pool);
    const uintptr_t hi = lo + layer_bytes * (size_t)(layers - 1) + one;
    for (const int *x : {src, dst}) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x);
        if (a < hi && lo < a + (size_t)n * 4) return RWKV7_ERR_ALIAS;
    }
    MoveArgs a{};
    a.pool = static_cast<char *>(pool);
    a.layer_bytes = layer_bytes;
    a.slot_bytes = slot_bytes;
    a.src = src; a.dst = dst;
    a.layers = layers; a.slots = slots; a.n = n;
    a.lanes = kThreads;  // the largest piece that fits all pairs and is not mostly behind the slot
    while (a.lanes > 4 && ((size_t)n * a.lanes > (size_t)kThreads * kPer ||
                           (size_t)a.lanes * 16 >= 2 * slot_bytes))
        a.lanes /= 2;
    const size_t pieces = (slot_bytes + (size_t)a.lanes * 16 - 1) / ((size_t)a.lanes * 16);
    if (pieces > 0x7fffffffu) return RWKV7_ERR_SHAPE;
    a.pieces = (unsigned)pieces;
    const unsigned long long all = (unsigned long long)pieces * (unsigned)layers;
    const unsigned blocks = (unsigned)(all < 1024 ? all : 1024);  // four workgroups per CU
    hipLaunchKernelGGL(state_move_kernel, dim3(blocks), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP;
}
