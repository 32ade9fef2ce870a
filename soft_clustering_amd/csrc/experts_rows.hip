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
// 2^q lanes holds one point, 16 bytes of its row per lane and step.

#include <algorithm>
#include <type_traits>

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

// The E elements of piece c of a row (VEC: 16 bytes; else one element).
template <typename T, bool VEC> struct Piece {
    static constexpr int kElems = VEC ? Vec16<T>::kElems : 1;
    __device__ __forceinline__ static void load(const T* row, int c, float* v) {
        if constexpr (VEC) Vec16<T>::unpack(((const uint4*)row)[c], v);
        else v[0] = to_f32(row[c]);
    }
    __device__ __forceinline__ static void store(T* row, int c, const float* v) {
        if constexpr (VEC) ((uint4*)row)[c] = pack16<T>(v);
        else from_f32(v[0], row + c);
    }
};

// y[slot] = x[p].
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_dispatch(const RowArgs a, int lanes_log2) {
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const int pieces = VEC ? a.d / Vec16<T>::kElems : a.d;
    using V = typename std::conditional<VEC, uint4, T>::type;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        const V* x = (const V*)((const T*)a.by_point + p * a.ldp);
        for (int c = c0; c < pieces; c += lanes) {
            const V v = x[c];
            for (int i = 0; i < a.m; ++i) {
                const int s = a.slot[p * a.m + i];
                if (s >= 0 && s < a.rows) ((V*)((T*)a.out_slot + s * a.ldos))[c] = v;
            }
        }
    }
}

// out[p] = sum_i g_i z[slot_i]; WEIGHTED false: g = 1.
template <typename T, bool VEC, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const RowArgs a, int lanes_log2) {
    using P = Piece<T, VEC>;
    constexpr int E = P::kElems;
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const int pieces = a.d / E;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        T* out = (T*)a.out_point + p * a.ldop;
        for (int c = c0; c < pieces; c += lanes) {
            float acc[E];
    #pragma unroll
            for (int j = 0; j < E; ++j) acc[j] = 0.0f;
            for (int i = 0; i < a.m; ++i) {
                const int s = a.slot[p * a.m + i];
                if (s < 0 || s >= a.rows) continue;
                float v[E];
                P::load((const T*)a.by_slot + s * a.lds, c, v);
                const float g = WEIGHTED ? a.gamma[p * a.m + i] : 1.0f;
    #pragma unroll
                for (int j = 0; j < E; ++j) acc[j] = WEIGHTED ? fmaf(g, v[j], acc[j]) : acc[j] + v[j];
            }
            P::store(out, c, acc);
        }
    }
}

// dz[slot_i] = g_i dout[p], dg_i = <dout[p], z[slot_i]>; either output may be
// absent.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_combine_backward(const RowArgs a, int lanes_log2) {
    using P = Piece<T, VEC>;
    constexpr int E = P::kElems;
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1);
    const int64_t p0 = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const int pieces = a.d / E;
    for (int64_t p = p0; p < a.n; p += (int64_t)gridDim.x * (256 >> lanes_log2)) {
        const T* dout = (const T*)a.by_point + p * a.ldp;
        for (int i = 0; i < a.m; ++i) {
            const int s = a.slot[p * a.m + i];
            const bool there = s >= 0 && s < a.rows;
            float dot = 0.0f;
            if (there) {
                const float g = a.gamma[p * a.m + i];
                for (int c = c0; c < pieces; c += lanes) {
                    float v[E], z[E];
                    P::load(dout, c, v);
                    if (a.dgamma != nullptr) {
                        P::load((const T*)a.by_slot + s * a.lds, c, z);
    #pragma unroll
                        for (int j = 0; j < E; ++j) dot = fmaf(v[j], z[j], dot);
                    }
                    if (a.out_slot != nullptr) {
    #pragma unroll
                        for (int j = 0; j < E; ++j) v[j] *= g;
                        P::store((T*)a.out_slot + s * a.ldos, c, v);
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

template <typename T, bool VEC> gmm_status launch_op(RowOp op, const RowArgs& a, hipStream_t stream) {
    const int pieces = VEC ? a.d / Vec16<T>::kElems : a.d;
    int lg = 0;
    while (lg < 6 && (1 << lg) < pieces) ++lg;
    const int per = 256 >> lg;
    const int64_t grid = std::min<int64_t>((a.n + per - 1) / per, kMaxGrid);
    switch (op) {
        case ROW_DISPATCH: hipLaunchKernelGGL((k_dispatch<T, VEC>), dim3(grid), dim3(256), 0, stream, a, lg); break;
        case ROW_SUM: hipLaunchKernelGGL((k_combine<T, VEC, false>), dim3(grid), dim3(256), 0, stream, a, lg); break;
        case ROW_COMBINE: hipLaunchKernelGGL((k_combine<T, VEC, true>), dim3(grid), dim3(256), 0, stream, a, lg); break;
        default: hipLaunchKernelGGL((k_combine_backward<T, VEC>), dim3(grid), dim3(256), 0, stream, a, lg);
    }
    return launched();
}

bool whole_pieces(const void* p, int64_t ld, int es) { return p == nullptr || (aligned16(p) && ld * es % 16 == 0); }

gmm_status run_rows(RowOp op, int dtype, const RowArgs& a, hipStream_t stream) {
    const int es = elem_size(dtype);
    const bool vec = (int64_t)a.d * es % 16 == 0 && whole_pieces(a.by_point, a.ldp, es) &&
                     whole_pieces(a.by_slot, a.lds, es) && whole_pieces(a.out_point, a.ldop, es) &&
                     whole_pieces(a.out_slot, a.ldos, es);
    switch (dtype) {
        case GMM_F32: return vec ? launch_op<float, true>(op, a, stream) : launch_op<float, false>(op, a, stream);
        case GMM_BF16: return vec ? launch_op<bf16_t, true>(op, a, stream) : launch_op<bf16_t, false>(op, a, stream);
        default: return vec ? launch_op<_Float16, true>(op, a, stream) : launch_op<_Float16, false>(op, a, stream);
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
