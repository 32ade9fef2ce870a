// gmm_route: the lists of an assignment, a stable counting sort of its T = n m
// entries by component.
//
// slot(e) = offsets[k] + #{e' < e : idx[e'] = k}, k = idx[e]: the count splits
// into whole chunks before e's (hist, scanned over chunks), whole waves of its
// own chunk (counters in LDS), groups of 64 entries before its own in its
// wave (the same counter, advanced group by group) and the lanes below it with
// its key (one ballot per bit of the key).  Nothing depends on the order of
// atomics: they only count.
//
// A workgroup of eight waves sorts a chunk of up to 8192 (16384) entries, its
// keys in registers, in LDS first, so that entry[] leaves in runs.  A small
// assignment is one chunk and one launch; larger ones take three: count per
// chunk, scan over chunks, place.  1e7 points in two of 256 lists:
// 18 + 6 + 76 us; the two passes over idx and the writes are 320 MB, 63 us at
// the rate of a copy, and placing waits for its LDS counters group by group.
// 96 entries: 4.6 us, the latency of a load, two scans and a store.

#include "experts_internal.h"

namespace gmm {

namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// Keys a lane holds, by the number of lists: the more lists, the longer the chunk whose
// counters they share (hist is 4 K bytes a chunk).  Counters are 16 bits.
constexpr int kKeysFew = 16, kKeysMany = 32, kManyLists = 1024;

int64_t chunk_for(int k) { return (int64_t)kThreads * (k > kManyLists ? kKeysMany : kKeysFew); }

__device__ __forceinline__ bool in_lists(int key, int K) { return (unsigned)key < (unsigned)K; }

// Lanes of the wave that hold this lane's key (valid lanes only).
__device__ __forceinline__ uint64_t same_key(int key, bool valid, int bits) {
    uint64_t mask = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool bit = (key >> b) & 1;
        const uint64_t set = __ballot(bit);
        mask &= bit ? set : ~set;
    }
    return mask;
}

// Exclusive scan over keys of a per-key LDS array, in place; returns the
// sum.  All threads call it.
__device__ int scan_keys(int* a, int K, int* scratch) {
    const int t = threadIdx.x, nt = blockDim.x, per = (K + nt - 1) / nt;
    const int lo = min(t * per, K), hi = min(lo + per, K);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += a[i];
    // inclusive scan of the threads' sums
    int v = sum;
    const int lane = t & 63, wave = t >> 6;
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    if (lane == 63) scratch[wave] = v;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < nt / 64; ++w) {
        if (w < wave) before += scratch[w];
        total += scratch[w];
    }
    int run = before + v - sum;
    for (int i = lo; i < hi; ++i) {
        const int c = a[i];
        a[i] = run;
        run += c;
    }
    __syncthreads();
    return total;
}

// Counts of every key in every chunk: hist [K][stride], a key's chunks side by
// side, so that the scan reads and writes whole lines.
__global__ __launch_bounds__(1024) void k_route_count(const int32_t* __restrict__ idx, int64_t rows,
                                                      int64_t chunk, int K, int stride, int* __restrict__ hist) {
    __shared__ int h[GMM_MAX_LISTS];
    const int t = threadIdx.x, nt = blockDim.x;
    for (int i = t; i < K; i += nt) h[i] = 0;
    __syncthreads();
    const int64_t c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, rows);
    for (int64_t e = c0 + t; e < c1; e += 8 * nt) {   // eight loads in flight
        int key[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) key[u] = e + u * nt < c1 ? idx[e + u * nt] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (in_lists(key[u], K)) atomicAdd(&h[key[u]], 1);
    }
    __syncthreads();
    for (int i = t; i < K; i += nt) hist[(int64_t)i * stride + blockIdx.x] = h[i];
}

// hist -> exclusive sums over the chunks; total[key].  One workgroup a key.
__global__ __launch_bounds__(256) void k_route_scan(int* __restrict__ hist, int chunks, int stride,
                                                    int* __restrict__ total) {
    constexpr int U = 8;
    __shared__ int part[2][4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int* row = hist + (int64_t)blockIdx.x * stride;
    int before = 0;   // the strips so far
    for (int c0 = 0, turn = 0; c0 < chunks; c0 += 256 * U, turn ^= 1) {
        int v[U], sum = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + t * U + u;
            v[u] = c < chunks ? row[c] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) sum += v[u];
        int upto = sum;
        for (int o = 1; o < 64; o <<= 1) {
            const int w = __shfl_up(upto, o);
            if (lane >= o) upto += w;
        }
        if (lane == 63) part[turn][wave] = upto;
        __syncthreads();
        int run = before + upto - sum;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) run += part[turn][w];
            before += part[turn][w];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + t * U + u;
            if (c < chunks) row[c] = run;
            run += v[u];
        }
    }
    if (t == 0) total[blockIdx.x] = before;
}

// One chunk: hist and total from the kernels above, or null for an assignment of one chunk.
template <int KEYS, int KMAX>
__global__ __launch_bounds__(kThreads) void k_route_place(const int32_t* __restrict__ idx, int64_t rows, int K,
                                                          int bits, int stride, const int* __restrict__ hist,
                                                          const int* __restrict__ total, int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ entry, int32_t* __restrict__ slot) {
    constexpr int kChunk = kThreads * KEYS;
    __shared__ uint32_t cnt32[kWaves * KMAX / 2];   // [wave][key], 16 bits each
    __shared__ int to[KMAX];                        // global minus local position of a key's entries
    __shared__ uint16_t sorted[kChunk] __attribute__((aligned(4))), key_of[kChunk];
    __shared__ int scratch[kWaves];
    static_assert(sizeof(int) * KMAX <= sizeof(sorted), "local");
    int* local = (int*)sorted;   // the chunk's counts, then their exclusive sums; before the keys are placed
    uint16_t* cnt = (uint16_t*)cnt32;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t c0 = (int64_t)blockIdx.x * kChunk;
    const int here = (int)min((int64_t)kChunk, rows - c0);
    const int run = ((here + kWaves - 1) / kWaves + 63) / 64 * 64;   // entries of a wave
    const int a = wave * run, b = min(a + run, here);

    int key[KEYS];
#pragma unroll
    for (int g = 0; g < KEYS; ++g) {
        const int e = a + 64 * g + lane;
        key[g] = 64 * g < run && e < b ? idx[c0 + e] : -1;
    }
    for (int i = t; i < kWaves * KMAX / 2; i += kThreads) cnt32[i] = 0;
    for (int i = t; i < K; i += kThreads) to[i] = total != nullptr ? total[i] : 0;
    __syncthreads();
#pragma unroll
    for (int g = 0; g < KEYS; ++g)
        if (in_lists(key[g], K)) {
            const int at = wave * KMAX + key[g];
            atomicAdd(&cnt32[at >> 1], 1u << (16 * (at & 1)));
        }
    int all = 0;
    if (total != nullptr) all = scan_keys(to, K, scratch);   // the lists' first slots
    __syncthreads();
    for (int i = t; i < K; i += kThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) n += cnt[w * KMAX + i];
        local[i] = n;
    }
    __syncthreads();
    const int listed = scan_keys(local, K, scratch);
    if (total == nullptr) all = listed;
    if (blockIdx.x == 0) {
        for (int i = t; i < K; i += kThreads) offsets[i] = total != nullptr ? to[i] : local[i];
        if (t == 0) offsets[K] = all;
        __syncthreads();
    }
    for (int i = t; i < K; i += kThreads) {
        // the waves' counts become their first local positions
        int n = local[i];
        to[i] = total != nullptr ? to[i] + hist[(int64_t)i * stride + blockIdx.x] - n : 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = cnt[w * KMAX + i];
            cnt[w * KMAX + i] = (uint16_t)n;
            n += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < KEYS; ++g) {
        if (64 * g >= run) continue;
        const int e = a + 64 * g + lane;
        const bool valid = in_lists(key[g], K);
        const uint64_t same = same_key(key[g], valid, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int pos = -1;
        if (valid) pos = cnt[wave * KMAX + key[g]] + rank;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid && rank == 0) cnt[wave * KMAX + key[g]] = (uint16_t)(pos + __popcll(same));
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid) {
            sorted[pos] = (uint16_t)e;
            key_of[pos] = (uint16_t)key[g];
        }
        if (e < b) slot[c0 + e] = valid ? to[key[g]] + pos : -1;
    }
    __syncthreads();
    for (int i = t; i < listed; i += kThreads) entry[to[key_of[i]] + i] = (int32_t)(c0 + sorted[i]);
    for (int64_t i = all + (int64_t)blockIdx.x * kThreads + t; i < rows; i += (int64_t)gridDim.x * kThreads) entry[i] = -1;
}

__global__ void k_route_empty(int K, int32_t* offsets) {
    for (int i = threadIdx.x; i <= K; i += blockDim.x) offsets[i] = 0;
}

}  // namespace

gmm_status check_shape(int64_t n, int64_t m, int64_t k) {
    if (n < 0 || m < 1 || m > GMM_MAX_TOPM || k < 1 || k > GMM_MAX_LISTS) return GMM_E_ARG;
    if (n > kMaxEntries || n * m > kMaxEntries) return GMM_E_ARG;
    return GMM_OK;
}

gmm_status check_routes(const gmm_routes* r) {
    if (r == nullptr) return GMM_E_ARG;
    const gmm_status st = check_shape(r->n, r->m, r->k);
    if (st != GMM_OK) return st;
    if (r->n > 0 && (r->offsets == nullptr || r->entry == nullptr || r->slot == nullptr)) return GMM_E_ARG;
    return GMM_OK;
}

gmm_status check_width(int64_t d, int32_t dtype) {
    if (d < 1 || d > kMaxWidth || dtype < GMM_F32 || dtype > GMM_F16) return GMM_E_ARG;
    return GMM_OK;
}

gmm_status check_stride(int64_t ld, int64_t d) { return ld < d || ld > kMaxStride ? GMM_E_ARG : GMM_OK; }

}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_route_workspace_bytes(int64_t n, int32_t m, int32_t k, size_t* bytes) {
    if (bytes == nullptr) return GMM_E_ARG;
    const gmm_status st = check_shape(n, m, k);
    if (st != GMM_OK) return st;
    const int64_t rows = n * m;
    *bytes = 0;
    const int64_t chunk = chunk_for(k);
    if (rows > chunk) {
        const int64_t chunks = (rows + chunk - 1) / chunk;
        *bytes = sizeof(int) * (size_t)(chunks + 1) * k;
    }
    return GMM_OK;
}

gmm_status gmm_route(int64_t n, int32_t m, int32_t k, const int32_t* idx, void* ws, size_t ws_bytes,
                     int32_t* offsets, int32_t* entry, int32_t* slot, hipStream_t stream) {
    size_t need = 0;
    const gmm_status st = gmm_route_workspace_bytes(n, m, k, &need);
    if (st != GMM_OK) return st;
    const int64_t rows = n * m;
    if (offsets == nullptr || (rows > 0 && (idx == nullptr || entry == nullptr || slot == nullptr))) return GMM_E_ARG;
    if (need > 0) {
        if (ws == nullptr || (uintptr_t)ws % 256 != 0) return GMM_E_ARG;
        if (ws_bytes < need) return GMM_E_WORKSPACE;
    }
    if (rows == 0) {
        hipLaunchKernelGGL(k_route_empty, dim3(1), dim3(256), 0, stream, k, offsets);
        return launched();
    }
    int bits = 0;
    while ((1 << bits) < k) ++bits;
    const int64_t chunk = chunk_for(k);
    const int chunks = (int)((rows + chunk - 1) / chunk);
    int *hist = nullptr, *total = nullptr;
    if (need > 0) {
        hist = (int*)ws;
        total = hist + (int64_t)chunks * k;
        hipLaunchKernelGGL(k_route_count, dim3(chunks), dim3(1024), 0, stream, idx, rows, chunk, k, chunks, hist);
        hipLaunchKernelGGL(k_route_scan, dim3(k), dim3(256), 0, stream, hist, chunks, chunks, total);
    }
    auto place = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(chunks), dim3(kThreads), 0, stream, idx, rows, k, bits, chunks, (const int*)hist,
                           (const int*)total, offsets, entry, slot);
    };
    if (k <= 256) place(k_route_place<kKeysFew, 256>);
    else if (k <= kManyLists) place(k_route_place<kKeysFew, kManyLists>);
    else place(k_route_place<kKeysMany, GMM_MAX_LISTS>);
    return launched();
}

}  // extern "C"
