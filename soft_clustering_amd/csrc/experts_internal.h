// Shared by the kernels behind include/gmm_experts.h: storage types, 16-byte
// pieces of a row, the map from workgroups to lists.
#pragma once

#include "common.h"
#include "gmm_experts.h"

namespace gmm {

constexpr int64_t kMaxWidth = 1 << 20, kMaxStride = 1 << 22;
constexpr int64_t kMaxEntries = 1 << 30;   // entries and slots are 32-bit, grids of them stay in range

// fp32 -> storage type, round to nearest even.
__device__ __forceinline__ void from_f32(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_f32(float v, bf16_t* o) { o->bits = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void from_f32(float v, _Float16* o) { *o = (_Float16)v; }

template <typename T> __device__ __forceinline__ uint4 pack16(const float* v) {
    constexpr int E = Vec16<T>::kElems;
    T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) from_f32(v[i], t + i);
    return __builtin_bit_cast(uint4, t);
}

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfrag8 __attribute__((ext_vector_type(8)));

// c += A . B on 16 x 16 blocks: lane l gives row l % 16 of A and column l % 16 of B, quarter
// l / 16 of the contraction (32 elements, fp32: 16), and holds column l % 16, rows 4 (l / 16) + r.
template <typename T> __device__ __forceinline__ f32x4 mma16(const uint4& a, const uint4& b, f32x4 c);
template <> __device__ __forceinline__ f32x4 mma16<_Float16>(const uint4& a, const uint4& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<bf16_t>(const uint4& a, const uint4& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfrag8, a), __builtin_bit_cast(bfrag8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<float>(const uint4& a, const uint4& b, f32x4 c) {
    c = mfma16x16x4(__uint_as_float(a.x), __uint_as_float(b.x), c);
    c = mfma16x16x4(__uint_as_float(a.y), __uint_as_float(b.y), c);
    c = mfma16x16x4(__uint_as_float(a.z), __uint_as_float(b.z), c);
    return mfma16x16x4(__uint_as_float(a.w), __uint_as_float(b.w), c);
}

static __device__ __constant__ uint4 zero_piece = {0, 0, 0, 0};

// 16 bytes of global memory at an alignment.  The address space is named because the compiler loses it where
// an address comes from a select with zero_piece, and a generic load holds up LDS and the loads behind it.
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
template <int ALIGN> struct Words4;
template <> struct Words4<1> { typedef words4 type __attribute__((aligned(1))); };
template <> struct Words4<2> { typedef words4 type __attribute__((aligned(2))); };
template <> struct Words4<4> { typedef words4 type __attribute__((aligned(4))); };
template <> struct Words4<16> { typedef words4 type __attribute__((aligned(16))); };
template <int ALIGN> __device__ __forceinline__ uint4 load16(const void* p) {
    const words4 v = *(const __attribute__((address_space(1))) typename Words4<ALIGN>::type*)p;
    return make_uint4(v.x, v.y, v.z, v.w);
}

// The 16 bytes from byte c of a row of `width` >= 16 on, at the alignment given, in two steps so
// that many loads can be in flight: the load itself (of the row's last 16 bytes where fewer are left, of zeros
// where there is none), and the bits that lie before c, to be dropped later.
struct Loose {
    uint4 v;
    int drop;
};
template <int ALIGN>
__device__ __forceinline__ Loose load_loose(const char* row, bool there, int64_t c, int64_t width, const char* zero) {
    there = there && c < width;
    const int64_t from = min(c, width - 16);
    Loose l;
    l.v = load16<ALIGN>(there ? row + from : zero);
    l.drop = there ? 8 * (int)(c - from) : 0;
    return l;
}
__device__ __forceinline__ uint4 settle(const Loose& l) {
    uint64_t v[2] = {l.v.x | (uint64_t)l.v.y << 32, l.v.z | (uint64_t)l.v.w << 32};
    const bool far = l.drop >= 64;
    const int by = l.drop & 63;
    const uint64_t lo = far ? v[1] : v[0], hi = far ? 0 : v[1];
    v[0] = (lo >> by) | (by ? hi << (64 - by) : 0);
    v[1] = hi >> by;
    return make_uint4((uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32));
}

// 16 bytes of a row of less than 16, from element c on; zero beyond the row.
template <typename T> __device__ __forceinline__ uint4 load_narrow(const T* row, bool there, int c, int width) {
    constexpr int E = Vec16<T>::kElems;
    T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (there && c + i < width) t[i] = row[c + i];
        else from_f32(0.0f, t + i);
    }
    return __builtin_bit_cast(uint4, t);
}

// 16 bytes of a row from element c on, at any alignment of the elements; zero beyond it.  NARROW: the row may
// be of less than 16 bytes.  A kernel of its own, as the compiler waits for a load at the end of the
// branch it is in: with both forms in one loop each step waited for the memory once per piece.
template <typename T, bool NARROW>
__device__ __forceinline__ Loose load_piece(const T* row, bool there, int c, int width, const char* zero) {
    constexpr int S = (int)sizeof(T);
    if (NARROW && width * S < 16) return Loose{load_narrow(row, there, c, width), 0};
    return load_loose<S>((const char*)row, there, (int64_t)c * S, (int64_t)width * S, zero);
}

// 16 bytes from each lane's address to LDS bytes lds + 16 lane, asynchronously: the wave that
// issued it waits with wait_pieces() before the barrier that hands the tile over.  Written as asm
// because the compiler, which tracks the builtin form as an LDS store, would wait
// for the pieces of the next step before it reads those of this one.
__device__ __forceinline__ void fetch_piece(const void* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_pieces() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// Its address in vector registers, so that a loop with waits in it does not load it again.
__device__ __forceinline__ const char* zero_address() {
    const char* p = (const char*)&zero_piece;
    asm volatile("" : "+v"(p));
    return p;
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p);
}


// Workgroup -> rows of one list.  Row block `t` of a launch is either block
// (t - t0_k) of the list k with the largest t0_k = offsets[k] / BM + k not
// above t (a list of c rows spans at most the ceil(c / BM) blocks up to
// t0_{k+1}, so rows / BM + K blocks cover every list without any host
// knowledge of the lengths), or, with by_slot, the block that starts at slot
// t (only every BM-th slot of a list starts one; fewer workgroups where there are
// fewer rows than lists).  Each wave finds k for itself: 256 candidates at once, four a
// lane, after a first step over every 64th list where there are more.  Every offset is
// clamped to [0, rows]: whatever the array holds, the slots stay inside the row buffers.
struct ListRows {
    int k;        // list, -1: nothing to do
    int s0, s1;   // slots [s0, s1): from the block's first to the list's end
    int first;    // the list's first slot
};

__device__ __forceinline__ int clamped_offset(const int32_t* offsets, int k, int rows) {
    return min(max(offsets[k], 0), rows);
}

__device__ __forceinline__ ListRows find_rows(const int32_t* __restrict__ offsets, int K, int rows, int t,
                                              int bm, bool by_slot) {
    const int lane = threadIdx.x & 63;
    auto before = [&](int k, int o) { return k < K && (by_slot ? o : o / bm + k) <= t; };   // list k starts by block t
    int k0 = 0;
    if (K > 256) {
        const int k = lane * 64;
        const int o = clamped_offset(offsets, min(k, K), rows);
        k0 = max(__popcll(__ballot(before(k, o))) - 1, 0) * 64;
    }
    int o[4], count = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = clamped_offset(offsets, min(k0 + 4 * lane + q, K), rows);
#pragma unroll
    for (int q = 0; q < 4; ++q) count += __popcll(__ballot(before(k0 + 4 * lane + q, o[q])));
    const int i = __builtin_amdgcn_readfirstlane(count) - 1;   // the list is k0 + i
    ListRows r = {-1, 0, 0, 0};
    if (i < 0) return r;
    auto window = [&](int at) {
        const int l = at >> 2, q = at & 3;
        const int lo = q & 1 ? __builtin_amdgcn_readlane(o[1], l) : __builtin_amdgcn_readlane(o[0], l);
        const int hi = q & 1 ? __builtin_amdgcn_readlane(o[3], l) : __builtin_amdgcn_readlane(o[2], l);
        return q & 2 ? hi : lo;
    };
    const int a = window(i), b = i < 255 ? window(i + 1) : clamped_offset(offsets, min(k0 + 256, K), rows);
    int s0;
    if (by_slot) {
        if ((t - a) % bm != 0) return r;
        s0 = t;
    } else {
        const int64_t start = a + (int64_t)(t - (a / bm + k0 + i)) * bm;
        if (start >= b) return r;
        s0 = (int)start;
    }
    if (s0 >= b) return r;
    r.k = k0 + i;
    r.s0 = __builtin_amdgcn_readfirstlane(s0);
    r.s1 = __builtin_amdgcn_readfirstlane(b);
    r.first = __builtin_amdgcn_readfirstlane(a);
    return r;
}

inline int64_t row_blocks(int64_t rows, int64_t k, int bm, bool* by_slot) {
    const int64_t by_list = rows / bm + k;
    *by_slot = rows < by_list;
    return *by_slot ? rows : by_list;
}

inline bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }
inline int elem_size(int dtype) { return dtype == GMM_F32 ? 4 : 2; }

// Argument checks shared by the calls on lists.
gmm_status check_routes(const gmm_routes* r);
gmm_status check_shape(int64_t n, int64_t m, int64_t k);
gmm_status check_width(int64_t d, int32_t dtype);
gmm_status check_stride(int64_t ld, int64_t d);

inline gmm_status launched() { return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP; }

}  // namespace gmm
