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
// One workgroup does the whole sort of a small assignment in one launch;
// larger ones take three: count per chunk, scan over chunks, place.

#include "experts_internal.h"

namespace gmm {

namespace {

constexpr int kSmallEntries = 8192;    // one workgroup up to here
constexpr int kCounters = 16384;       // 16-bit counters in LDS: waves x lists
constexpr int kMinChunk = 4096, kMaxChunk = 49152;   // entries per chunk; counters are 16 bits
constexpr int kChunks = 1024;          // chunks aimed at

int waves_for(int k) {
    int w = 16;
    while (w > 1 && w * ((k + 1) & ~1) > kCounters) w >>= 1;
    return w;
}

int64_t chunk_for(int64_t rows) {
    int64_t c = (rows + kChunks - 1) / kChunks;
    c = (c + kMinChunk - 1) / kMinChunk * kMinChunk;
    return c > kMaxChunk ? kMaxChunk : c;
}

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

// Entries [c0, c1) of one workgroup: per-wave counts of its keys into cnt
// [waves][kp] (16 bits each).
__device__ __forceinline__ void count_waves(const int32_t* __restrict__ idx, int64_t c0, int64_t c1,
                                            int64_t run, int K, int kp, uint32_t* cnt) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t a = c0 + wave * run, b = min(a + run, c1);
    for (int64_t e = a + lane; e < b; e += 64) {
        const int key = idx[e];
        if (in_lists(key, K)) {
            const int at = wave * kp + key;
            atomicAdd(&cnt[at >> 1], 1u << (16 * (at & 1)));
        }
    }
}

// Turns the waves' counts into the waves' offsets within the workgroup, per
// key; the workgroup's count goes to total[key] when it is asked for.
__device__ __forceinline__ void prefix_waves(uint16_t* cnt, int waves, int K, int kp, int* total) {
    for (int key = threadIdx.x; key < K; key += blockDim.x) {
        int run = 0;
        for (int w = 0; w < waves; ++w) {
            const int c = cnt[w * kp + key];
            cnt[w * kp + key] = (uint16_t)run;
            run += c;
        }
        if (total != nullptr) total[key] = run;
    }
}

__device__ __forceinline__ void place(const int32_t* __restrict__ idx, int64_t c0, int64_t c1, int64_t run,
                                      int K, int kp, int bits, uint16_t* cnt, const int* base,
                                      int32_t* __restrict__ entry, int32_t* __restrict__ slot) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t a = c0 + wave * run, b = min(a + run, c1);
    for (int64_t e0 = a; e0 < b; e0 += 64) {
        const int64_t e = e0 + lane;
        const bool there = e < b;
        const int key = there ? idx[e] : -1;
        const bool valid = in_lists(key, K);
        const uint64_t same = same_key(key, valid, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int pos = -1;
        if (valid) pos = base[key] + cnt[wave * kp + key] + rank;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid && rank == 0) cnt[wave * kp + key] += (uint16_t)__popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid) entry[pos] = (int32_t)e;
        if (there) slot[e] = pos;
    }
}

// The whole sort in one workgroup.
__global__ __launch_bounds__(1024) void k_route_small(const int32_t* __restrict__ idx, int rows, int K, int kp,
                                                      int bits, int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ entry, int32_t* __restrict__ slot) {
    __shared__ uint32_t cnt[kCounters / 2];
    __shared__ int base[GMM_MAX_LISTS];
    __shared__ int scratch[16];
    const int t = threadIdx.x, nt = blockDim.x, waves = nt / 64;
    for (int i = t; i < waves * kp / 2; i += nt) cnt[i] = 0;
    __syncthreads();
    const int64_t run = ((rows + waves - 1) / waves + 63) / 64 * 64;
    count_waves(idx, 0, rows, run, K, kp, cnt);
    __syncthreads();
    prefix_waves((uint16_t*)cnt, waves, K, kp, base);
    __syncthreads();
    const int total = scan_keys(base, K, scratch);
    for (int i = t; i < K; i += nt) offsets[i] = base[i];
    if (t == 0) offsets[K] = total;
    place(idx, 0, rows, run, K, kp, bits, (uint16_t*)cnt, base, entry, slot);
    for (int i = total + t; i < rows; i += nt) entry[i] = -1;
}

// Counts of every key in every chunk: hist [chunks][K].
__global__ __launch_bounds__(1024) void k_route_count(const int32_t* __restrict__ idx, int64_t rows,
                                                      int64_t chunk, int K, int* __restrict__ hist) {
    __shared__ int h[GMM_MAX_LISTS];
    const int t = threadIdx.x, nt = blockDim.x;
    for (int i = t; i < K; i += nt) h[i] = 0;
    __syncthreads();
    const int64_t c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, rows);
    for (int64_t e = c0 + t; e < c1; e += nt) {
        const int key = idx[e];
        if (in_lists(key, K)) atomicAdd(&h[key], 1);
    }
    __syncthreads();
    for (int i = t; i < K; i += nt) hist[(int64_t)blockIdx.x * K + i] = h[i];
}

// hist -> exclusive sums over the chunks, per key; total[key].  64 keys a
// workgroup, 16 waves on a part of the chunks each.
__global__ __launch_bounds__(1024) void k_route_scan(int* __restrict__ hist, int chunks, int K,
                                                     int* __restrict__ total) {
    __shared__ int part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int key = blockIdx.x * 64 + lane;
    const bool there = key < K;
    const int per = (chunks + 15) / 16, lo = min(wave * per, chunks), hi = min(lo + per, chunks);
    int sum = 0;
    for (int c = lo; c < hi; ++c) sum += there ? hist[(int64_t)c * K + key] : 0;
    part[wave][lane] = sum;
    __syncthreads();
    int run = 0, all = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < wave) run += part[w][lane];
        all += part[w][lane];
    }
    if (!there) return;
    if (wave == 0) total[key] = all;
    for (int c = lo; c < hi; ++c) {
        const int v = hist[(int64_t)c * K + key];
        hist[(int64_t)c * K + key] = run;
        run += v;
    }
}

__global__ __launch_bounds__(1024) void k_route_place(const int32_t* __restrict__ idx, int64_t rows, int64_t chunk,
                                                      int K, int kp, int bits, const int* __restrict__ hist,
                                                      const int* __restrict__ total, int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ entry, int32_t* __restrict__ slot) {
    __shared__ uint32_t cnt[kCounters / 2];
    __shared__ int base[GMM_MAX_LISTS];
    __shared__ int scratch[16];
    const int t = threadIdx.x, nt = blockDim.x, waves = nt / 64;
    for (int i = t; i < waves * kp / 2; i += nt) cnt[i] = 0;
    for (int i = t; i < K; i += nt) base[i] = total[i];
    __syncthreads();
    const int64_t c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, rows);
    const int64_t run = ((c1 - c0 + waves - 1) / waves + 63) / 64 * 64;
    count_waves(idx, c0, c1, run, K, kp, cnt);
    const int all = scan_keys(base, K, scratch);
    if (blockIdx.x == 0) {
        for (int i = t; i < K; i += nt) offsets[i] = base[i];
        if (t == 0) offsets[K] = all;
        __syncthreads();
    }
    for (int i = t; i < K; i += nt) base[i] += hist[(int64_t)blockIdx.x * K + i];
    __syncthreads();
    prefix_waves((uint16_t*)cnt, waves, K, kp, nullptr);
    __syncthreads();
    place(idx, c0, c1, run, K, kp, bits, (uint16_t*)cnt, base, entry, slot);
    for (int64_t i = all + (int64_t)blockIdx.x * nt + t; i < rows; i += (int64_t)gridDim.x * nt) entry[i] = -1;
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
    if (rows > kSmallEntries) {
        const int64_t chunk = chunk_for(rows), chunks = (rows + chunk - 1) / chunk;
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
    const int kp = (k + 1) & ~1, waves = waves_for(k);
    int bits = 0;
    while ((1 << bits) < k) ++bits;
    if (need == 0) {
        hipLaunchKernelGGL(k_route_small, dim3(1), dim3(64 * waves), 0, stream, idx, (int)rows, k, kp, bits, offsets,
                           entry, slot);
        return launched();
    }
    const int64_t chunk = chunk_for(rows);
    const int chunks = (int)((rows + chunk - 1) / chunk);
    int* hist = (int*)ws;
    int* total = hist + (int64_t)chunks * k;
    hipLaunchKernelGGL(k_route_count, dim3(chunks), dim3(1024), 0, stream, idx, rows, chunk, k, hist);
    hipLaunchKernelGGL(k_route_scan, dim3((k + 63) / 64), dim3(1024), 0, stream, hist, chunks, k, total);
    hipLaunchKernelGGL(k_route_place, dim3(chunks), dim3(64 * waves), 0, stream, idx, rows, chunk, k, kp, bits, hist,
                       total, offsets, entry, slot);
    return launched();
}

}  // extern "C"
