// gmm_dispatch, gmm_combine and their gradients: rows of the points to the
// lists and back.
//
// All four walk the points and use slot[] alone, so a point's own row crosses
// the memory once whatever m is, and the m rows by slot once each:
//
//   dispatch            y[slot] = x[p]                       read d, write m d
//   dispatch_backward   dx[p] = sum_i dy[slot_i]             read m d, write d
//   combine             out[p] = sum_i g_i z[slot_i]         read m d, write d
//   combine_backward    dz[slot_i] = g_i dout[p],            read (1 + m) d, write m d
//                       dg_i = <dout[p], z[slot_i]>
//
// Sums run over the columns in order and over the row in fp32.  A group of
// 2^q lanes holds one point, 16 bytes of its row per lane and step, at any alignment of the
// elements; the last piece of a row that is no whole number of them starts early, and what it shares with
// the one before is computed and written twice, alike.  Rows shorter than 16 bytes go
// element by element.  All are bound by the memory: 1e6 points, m = 2: dispatch 64 fp32
// 137 us (5.7 TB/s), combine_backward 128 bf16 256 us (5.1 TB/s).

#include <algorithm>

#include "experts_internal.h"

namespace gmm {

namespace {

struct RowArgs {
    int64_t n;
    int64_t rows;        // n * m
    int m, d;
    const int32_t* slot;
    const float* gamma;
    const void* by_point;   // x, dout
    int64_t ldp;
    const void* by_slot;    // dy, z
    int64_t lds;
    void* out_point;        // dx, out
    int64_t ldop;
    void* out_slot;         // y, dz
    int64_t ldos;
    float* dgamma;
};

// How a row is cut.
enum Cut {
    CUT_ELEMENTS,   // one element a piece
    CUT_ANY,        // 16 bytes, the last piece early, any alignment
    CUT_WHOLE       // 16 bytes, aligned, no rest
};

template <typename T, int CUT> struct Piece {
    static constexpr int kElems = CUT == CUT_ELEMENTS ? 1 : Vec16<T>::kElems;
    // first element of piece c of a row of d
    __device__ __forceinline__ static int first(int c, int d) {
        return CUT == CUT_ANY ? min(c * kElems, d - kElems) : c * kElems;
    }
    __device__ __forceinline__ static uint4 raw(const T* p) {
        uint4 v;
        if constexpr (CUT == CUT_WHOLE) v = *(const uint4*)p;
        else __builtin_memcpy(&v, p, 16);
        return v;
    }
    __device__ __forceinline__ static void put(T* p, const uint4& v) {
        if constexpr (CUT == CUT_WHOLE) *(uint4*)p = v;
        else __builtin_memcpy(p, &v, 16);
    }
    __device__ __forceinline__ static void load(const T* p, float* v) {
        if constexpr (CUT == CUT_ELEMENTS) v[0] = to_f32(*p);
        else Vec16<T>::unpack(raw(p), v);
    }
    __device__ __forceinline__ static void store(T* p, const float* v) {
        if constexpr (CUT == CUT_ELEMENTS) from_f32(v[0], p);
        else put(p, pack16<T>(v));
    }
};

// y[slot] = x[p].
template <typename T, int CUT>
__global__ __launch_bounds__(256) void k_dispatch(const RowArgs a, int lanes_log2) {
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    using P = Piece<T, CUT>;
    const int pieces = (a.d + P::kElems - 1) / P::kElems;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        const T* x = (const T*)a.by_point + p * a.ldp;
        for (int c = c0; c < pieces; c += lanes) {
            const int e = P::first(c, a.d);
            if constexpr (CUT == CUT_ELEMENTS) {
                const T v = x[e];
                for (int i = 0; i < a.m; ++i) {
                    const int s = a.slot[p * a.m + i];
                    if (s >= 0 && s < a.rows) ((T*)a.out_slot + s * a.ldos)[e] = v;
                }
            } else {
                const uint4 v = P::raw(x + e);
                for (int i = 0; i < a.m; ++i) {
                    const int s = a.slot[p * a.m + i];
                    if (s >= 0 && s < a.rows) P::put((T*)a.out_slot + s * a.ldos + e, v);
                }
            }
        }
    }
}

// out[p] = sum_i g_i z[slot_i]; WEIGHTED false: g = 1.
template <typename T, int CUT, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const RowArgs a, int lanes_log2) {
    using P = Piece<T, CUT>;
    constexpr int E = P::kElems;
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const int pieces = (a.d + E - 1) / E;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        T* out = (T*)a.out_point + p * a.ldop;
        for (int c = c0; c < pieces; c += lanes) {
            const int e = P::first(c, a.d);
            float acc[E];
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] = 0.0f;
            for (int i = 0; i < a.m; ++i) {
                const int s = a.slot[p * a.m + i];
                if (s < 0 || s >= a.rows) continue;
                float v[E];
                P::load((const T*)a.by_slot + s * a.lds + e, v);
                const float g = WEIGHTED ? a.gamma[p * a.m + i] : 1.0f;
#pragma unroll
                for (int j = 0; j < E; ++j) acc[j] = WEIGHTED ? fmaf(g, v[j], acc[j]) : acc[j] + v[j];
            }
            P::store(out + e, acc);
        }
    }
}

// dz[slot_i] = g_i dout[p], dg_i = <dout[p], z[slot_i]>; either output may be
// absent.
template <typename T, int CUT>
__global__ __launch_bounds__(256) void k_combine_backward(const RowArgs a, int lanes_log2) {
    using P = Piece<T, CUT>;
    constexpr int E = P::kElems;
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const int pieces = (a.d + E - 1) / E;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        const T* dout = (const T*)a.by_point + p * a.ldp;
        for (int i = 0; i < a.m; ++i) {
            const int s = a.slot[p * a.m + i];
            const bool there = s >= 0 && s < a.rows;
            float dot = 0.0f;
            if (there) {
                const float g = a.gamma[p * a.m + i];
                for (int c = c0; c < pieces; c += lanes) {
                    const int e = P::first(c, a.d);
                    float v[E], z[E];
                    P::load(dout + e, v);
                    if (a.dgamma != nullptr) {
                        P::load((const T*)a.by_slot + s * a.lds + e, z);
#pragma unroll
                        for (int j = 0; j < E; ++j)   // an early piece's first elements are the one before's
                            if (CUT != CUT_ANY || e + j >= c * E) dot = fmaf(v[j], z[j], dot);
                    }
                    if (a.out_slot != nullptr) {
#pragma unroll
                        for (int j = 0; j < E; ++j) v[j] *= g;
                        P::store((T*)a.out_slot + s * a.ldos + e, v);
                    }
                }
            }
            if (a.dgamma != nullptr) {
                for (int o = lanes >> 1; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
                if (c0 == 0) a.dgamma[p * a.m + i] = dot;
            }
        }
    }
}

constexpr int64_t kMaxGrid = 1 << 22;   // workgroups; more points than they hold are walked

enum RowOp { ROW_DISPATCH, ROW_SUM, ROW_COMBINE, ROW_COMBINE_BACKWARD };

template <typename T, int CUT> gmm_status launch_op(RowOp op, const RowArgs& a, hipStream_t stream) {
    const int pieces = (a.d + Piece<T, CUT>::kElems - 1) / Piece<T, CUT>::kElems;
    int lg = 0;
    while (lg < 6 && (1 << lg) < pieces) ++lg;
    const int per = 256 >> lg;
    const dim3 grid(std::min<int64_t>((a.n + per - 1) / per, kMaxGrid));
    switch (op) {
        case ROW_DISPATCH: hipLaunchKernelGGL((k_dispatch<T, CUT>), grid, dim3(256), 0, stream, a, lg); break;
        case ROW_SUM: hipLaunchKernelGGL((k_combine<T, CUT, false>), grid, dim3(256), 0, stream, a, lg); break;
        case ROW_COMBINE: hipLaunchKernelGGL((k_combine<T, CUT, true>), grid, dim3(256), 0, stream, a, lg); break;
        default: hipLaunchKernelGGL((k_combine_backward<T, CUT>), grid, dim3(256), 0, stream, a, lg);
    }
    return launched();
}

bool whole_pieces(const void* p, int64_t ld, int es) { return p == nullptr || (aligned16(p) && ld * es % 16 == 0); }

template <typename T> gmm_status launch_type(RowOp op, const RowArgs& a, hipStream_t stream) {
    const int es = (int)sizeof(T);
    const bool whole = (int64_t)a.d * es % 16 == 0 && whole_pieces(a.by_point, a.ldp, es) &&
                       whole_pieces(a.by_slot, a.lds, es) && whole_pieces(a.out_point, a.ldop, es) &&
                       whole_pieces(a.out_slot, a.ldos, es);
    if (whole) return launch_op<T, CUT_WHOLE>(op, a, stream);
    return a.d * es >= 16 ? launch_op<T, CUT_ANY>(op, a, stream) : launch_op<T, CUT_ELEMENTS>(op, a, stream);
}

gmm_status run_rows(RowOp op, int dtype, const RowArgs& a, hipStream_t stream) {
    switch (dtype) {
        case GMM_F32: return launch_type<float>(op, a, stream);
        case GMM_BF16: return launch_type<bf16_t>(op, a, stream);
        default: return launch_type<_Float16>(op, a, stream);
    }
}

gmm_status start(const gmm_routes* r, int64_t d, int32_t dtype, RowArgs* a) {
    gmm_status st = check_routes(r);
    if (st == GMM_OK) st = check_width(d, dtype);
    if (st != GMM_OK) return st;
    *a = RowArgs{};
    a->n = r->n;
    a->rows = r->n * r->m;
    a->m = r->m;
    a->d = (int)d;
    a->slot = r->slot;
    return GMM_OK;
}

}  // namespace

}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_dispatch(const gmm_routes* routes, int64_t d, int32_t dtype, const void* x, int64_t ldx, void* y,
                        int64_t ldy, hipStream_t stream) {
    RowArgs a;
    gmm_status st = start(routes, d, dtype, &a);
    if (st != GMM_OK) return st;
    if ((st = check_stride(ldx, d)) != GMM_OK || (st = check_stride(ldy, d)) != GMM_OK) return st;
    if (a.n == 0) return GMM_OK;
    if (x == nullptr || y == nullptr) return GMM_E_ARG;
    a.by_point = x, a.ldp = ldx, a.out_slot = y, a.ldos = ldy;
    return run_rows(ROW_DISPATCH, dtype, a, stream);
}

gmm_status gmm_dispatch_backward(const gmm_routes* routes, int64_t d, int32_t dtype, const void* dy, int64_t lddy,
                                 void* dx, int64_t lddx, hipStream_t stream) {
    RowArgs a;
    gmm_status st = start(routes, d, dtype, &a);
    if (st != GMM_OK) return st;
    if ((st = check_stride(lddy, d)) != GMM_OK || (st = check_stride(lddx, d)) != GMM_OK) return st;
    if (a.n == 0) return GMM_OK;
    if (dy == nullptr || dx == nullptr) return GMM_E_ARG;
    a.by_slot = dy, a.lds = lddy, a.out_point = dx, a.ldop = lddx;
    return run_rows(ROW_SUM, dtype, a, stream);
}

gmm_status gmm_combine(const gmm_routes* routes, int64_t d, int32_t dtype, const void* z, int64_t ldz,
                       const float* gamma, void* out, int64_t ldo, hipStream_t stream) {
    RowArgs a;
    gmm_status st = start(routes, d, dtype, &a);
    if (st != GMM_OK) return st;
    if ((st = check_stride(ldz, d)) != GMM_OK || (st = check_stride(ldo, d)) != GMM_OK) return st;
    if (a.n == 0) return GMM_OK;
    if (z == nullptr || gamma == nullptr || out == nullptr) return GMM_E_ARG;
    a.by_slot = z, a.lds = ldz, a.gamma = gamma, a.out_point = out, a.ldop = ldo;
    return run_rows(ROW_COMBINE, dtype, a, stream);
}

gmm_status gmm_combine_backward(const gmm_routes* routes, int64_t d, int32_t dtype, const void* dout, int64_t lddo,
                                const void* z, int64_t ldz, const float* gamma, void* dz, int64_t lddz, float* dgamma,
                                hipStream_t stream) {
    RowArgs a;
    gmm_status st = start(routes, d, dtype, &a);
    if (st != GMM_OK) return st;
    if ((st = check_stride(lddo, d)) != GMM_OK) return st;
    if (dgamma != nullptr && (st = check_stride(ldz, d)) != GMM_OK) return st;
    if (dz != nullptr && (st = check_stride(lddz, d)) != GMM_OK) return st;
    if (a.n == 0 || (dz == nullptr && dgamma == nullptr)) return GMM_OK;
    if (dout == nullptr || gamma == nullptr || (dgamma != nullptr && z == nullptr)) return GMM_E_ARG;
    a.by_point = dout, a.ldp = lddo, a.gamma = gamma, a.out_slot = dz, a.ldos = lddz, a.dgamma = dgamma;
    if (dgamma != nullptr) a.by_slot = z, a.lds = ldz;
    return run_rows(ROW_COMBINE_BACKWARD, dtype, a, stream);
}

}  // extern "C"
