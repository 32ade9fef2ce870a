// gmm_linear and its gradients: one linear model per component on the rows of
// its list, as matrix products on the matrix cores.
//
//   y[s]  = W_k x_s + b_k       contraction over d_in, both operands contiguous along it
//   dx[s] = W_k^T dy[s]         contraction over d_out; W_k is contiguous along the output
//   dW_k  = sum_s dy[s] x_s^T   contraction over the list's rows; neither is contiguous along it
//   db_k  = sum_s dy[s]
//
// A workgroup of four waves computes a 128 x 128 tile, each wave 64 x 64 as 2 x 2
// blocks of v_mfma_f32_32x32x16 (16-bit storage) or v_mfma_f32_32x32x2_f32, fp32 accumulators.
// Operand tiles go through LDS in 16-byte pieces, 128 bytes of the contraction (64 or 32 elements)
// a step, two buffers.  An operand contiguous along the contraction is kept
// [row][128 bytes], its pieces XOR-swizzled by the row, and read a fragment (8 or 4 elements) at a time; one that is
// contiguous along the output is kept [contraction][128 columns] and read with
// ds_read_b64_tr_b16 (16-bit) or element by element (fp32).
//
// Workgroup -> rows: find_rows (experts_internal.h); the host never learns the lists' lengths.

#include "experts_internal.h"

namespace gmm {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfrag8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kTile = 128;        // rows and columns of a workgroup's tile
constexpr int kTileBytes = kTile * 128;   // one operand, one step

// acc += A . B on one fragment pair: 16 bytes of each lane's row, 16 (or 8) of
// the contraction.  A's rows become the accumulator's rows: lane l holds column l % 32 and
// rows 8 (r / 4) + 4 (l / 32) + r % 4.
template <typename T> __device__ __forceinline__ f32x16 mma(const uint4& a, const uint4& b, f32x16 c);
template <> __device__ __forceinline__ f32x16 mma<_Float16>(const uint4& a, const uint4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x16 mma<bf16_t>(const uint4& a, const uint4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bfrag8, a), __builtin_bit_cast(bfrag8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x16 mma<float>(const uint4& a, const uint4& b, f32x16 c) {
    // the lanes' halves hold elements 0-3 and 4-7 of the contraction: MFMA e takes {e, 4 + e}
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
}

template <typename T> __device__ __forceinline__ uint4 ones();
template <> __device__ __forceinline__ uint4 ones<float>() {
    const uint32_t u = 0x3F800000u;
    return make_uint4(u, u, u, u);
}
template <> __device__ __forceinline__ uint4 ones<bf16_t>() {
    const uint32_t u = 0x3F803F80u;
    return make_uint4(u, u, u, u);
}
template <> __device__ __forceinline__ uint4 ones<_Float16>() {
    const uint32_t u = 0x3C003C00u;
    return make_uint4(u, u, u, u);
}

// 16 bytes of a row from element c on, of `width` elements; zero beyond it.
// VEC: width and c are multiples of the piece.
template <typename T, bool VEC> __device__ __forceinline__ uint4 load_piece(const T* row, int c, int width) {
    constexpr int E = Vec16<T>::kElems;
    if constexpr (VEC) {
        return c < width ? *(const uint4*)(row + c) : make_uint4(0, 0, 0, 0);
    } else {
        T t[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (c + i < width) t[i] = row[c + i];
            else from_f32(0.0f, t + i);
        }
        return __builtin_bit_cast(uint4, t);
    }
}

// Four consecutive outputs of a row from column c on.
template <typename T, bool VEC> __device__ __forceinline__ void store4(T* row, int c, int width, const float* v) {
    T t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) from_f32(v[i], t + i);
    if constexpr (VEC) {
        if (c < width) __builtin_memcpy(__builtin_assume_aligned(row + c, 4 * sizeof(T)), t, 4 * sizeof(T));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < width) row[c + i] = t[i];
    }
}

// ---- operand tiles in LDS

// [row][128 bytes]: piece p of a row sits at p ^ (row & 7).
struct RowTile {
    __device__ __forceinline__ static int at(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }
    // lane's fragment of step j (of four) for row block `r0`
    __device__ __forceinline__ static uint4 frag(const char* t, int r0, int j) {
        const int lane = threadIdx.x & 63;
        return *(const uint4*)(t + at(r0 + (lane & 31), 2 * j + (lane >> 5)));
    }
};

// [contraction][128 columns]: rows of 256 or 512 bytes.
template <typename T> struct ColTile {
    static constexpr int kRows = 128 / (int)sizeof(T);           // contraction elements of a step
    static constexpr int kPieces = 8 * (int)sizeof(T);           // 16-byte pieces of a row
    // Pairs of pieces (the 16 columns of a transposed read) move by a number
    // that differs between the 8 rows one read touches.
    __device__ __forceinline__ static int swz(int row) {
        return sizeof(T) == 2 ? 2 * ((row & 3) | ((row >> 1) & 4)) : 0;
    }
    __device__ __forceinline__ static int at(int row, int piece) {
        return row * (kPieces * 16) + ((piece ^ swz(row)) << 4);
    }
    __device__ __forceinline__ static uint4 frag(const char* t, int c0, int j) {
        const int lane = threadIdx.x & 63;
        if constexpr (sizeof(T) == 2) {
            const int g = lane >> 4, i = lane & 15;
            const int col = c0 + 16 * (g & 1) + 4 * (i & 3), row = 16 * j + 8 * (g >> 1) + (i >> 2);
            uint2 v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const char* p = t + at(row + 4 * u, col >> 3) + 2 * (col & 7);
                v[u] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)((lds_char*)p)));
            }
            return make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
        } else {
            const int row = 8 * j + 4 * (lane >> 5), col = c0 + (lane & 31);
            const float* p = (const float*)(t + at(row, 0)) + col;
            constexpr int W = kPieces * 4;
            return make_uint4(__float_as_uint(p[0]), __float_as_uint(p[W]), __float_as_uint(p[2 * W]),
                              __float_as_uint(p[3 * W]));
        }
    }
};

struct LinArgs {
    const int32_t* offsets;
    const int32_t* entry;
    int rows;            // n * m
    int n;               // points
    int m;
    int K;
    bool by_slot;
    bool gather;         // rows of a are the points' (entry[s] / m), else by slot
    const void* a;       // x or dy
    int64_t lda;
    const void* w;       // [K, d_out, d_in]
    int d_in, d_out;
    const float* bias;
    void* c;             // y or dx
    int64_t ldc;
};

// Row of x behind a slot, or -1.
__device__ __forceinline__ int64_t source_row(const int32_t* __restrict__ entry, int s, int m, int rows) {
    const int e = entry[s];
    return e >= 0 && e < rows ? e / m : -1;
}

// y = x W^T + b (BACK false) or dx = dy W (BACK true) on one 128 x 128 tile.
template <typename T, bool VEC, bool BACK>
__global__ __launch_bounds__(256) void k_linear(const LinArgs a) {
    constexpr int E = Vec16<T>::kElems, KS = 8 * E;   // elements of a piece, of a step
    __shared__ char lds[2][2][kTileBytes] __attribute__((aligned(16)));
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, blockIdx.x, kTile, a.by_slot);
    if (lr.k < 0) return;
    const int kd = BACK ? a.d_out : a.d_in, nd = BACK ? a.d_in : a.d_out;   // contraction, output width
    const int n0 = blockIdx.y * kTile;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    const T* w = (const T*)a.w + (int64_t)lr.k * a.d_in * a.d_out;

    // this thread's four pieces of each operand tile
    const T* arow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int s = lr.s0 + (t >> 3) + 32 * j;
        int64_t row = -1;
        if (s < lr.s1) row = a.gather ? source_row(a.entry, s, a.m, a.rows) : s;
        arow[j] = row >= 0 ? (const T*)a.a + row * a.lda : nullptr;
    }
    uint4 ra[4], rb[4];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = t + 256 * j;
            ra[j] = arow[j] != nullptr ? load_piece<T, VEC>(arow[j], k0 + (q & 7) * E, kd) : make_uint4(0, 0, 0, 0);
            if constexpr (!BACK) {
                const int r = n0 + (q >> 3);
                rb[j] = r < nd ? load_piece<T, VEC>(w + (int64_t)r * kd, k0 + (q & 7) * E, kd) : make_uint4(0, 0, 0, 0);
            } else {
                constexpr int P = ColTile<T>::kPieces;
                const int r = k0 + q / P;
                rb[j] = r < kd ? load_piece<T, VEC>(w + (int64_t)r * nd, n0 + (q % P) * E, nd) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = t + 256 * j;
            *(uint4*)(lds[buf][0] + RowTile::at(q >> 3, q & 7)) = ra[j];
            constexpr int P = ColTile<T>::kPieces;
            *(uint4*)(lds[buf][1] + (BACK ? ColTile<T>::at(q / P, q % P) : RowTile::at(q >> 3, q & 7))) = rb[j];
        }
    };

    f32x16 acc[2][2] = {};
    fetch(0);
    int buf = 0;
    for (int k0 = 0; k0 < kd; k0 += KS, buf ^= 1) {
        put(buf);
        __syncthreads();
        if (k0 + KS < kd) fetch(k0 + KS);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = RowTile::frag(lds[buf][0], wm + 32 * i, j);
                fb[i] = BACK ? ColTile<T>::frag(lds[buf][1], wn + 32 * i, j) : RowTile::frag(lds[buf][1], wn + 32 * i, j);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[i][h] = mma<T>(fb[h], fa[i], acc[i][h]);
        }
    }

    // lane: slot lane % 32, four consecutive outputs per register group
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lr.s0 + wm + 32 * i + (lane & 31);
        if (s >= lr.s1) continue;
        T* row = (T*)a.c + (int64_t)s * a.ldc;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = n0 + wn + 32 * h + 8 * q + 4 * (lane >> 5);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = acc[i][h][4 * q + e];
                    if (!BACK && a.bias != nullptr && c + e < nd) v[e] += a.bias[(int64_t)lr.k * nd + c + e];
                }
                store4<T, VEC>(row, c, nd, v);
            }
    }
}

// ---- gradient of the weights

struct GradArgs {
    const int32_t* offsets;
    const int32_t* entry;
    int rows, m, K;
    bool by_slot, gather;
    int chunk;              // rows of a list one workgroup sums
    const void* x;
    int64_t ldx;
    const void* dy;
    int64_t ldy;
    int d_in, d_out;
    float* dw;
    float* db;
    float* part;            // slots of d_out * d_in + d_out sums
};

// First partial slot of a list of more than one chunk that starts at slot a:
// such a list of c rows takes the ceil(c / chunk) slots up to the next list's first one,
// since floor(2 b / chunk) - floor(2 a / chunk) >= ceil(2 c / chunk) - 1 >= ceil(c / chunk) for c > chunk.
__device__ __host__ __forceinline__ int64_t first_slot(int64_t a, int chunk) { return 2 * a / chunk; }

// dW (and db) over one chunk of one list, a 128 (d_out) x 128 (d_in) tile.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_linear_dw(const GradArgs a) {
    constexpr int E = Vec16<T>::kElems, P = ColTile<T>::kPieces, KS = ColTile<T>::kRows;
    __shared__ char lds[2][2][kTileBytes] __attribute__((aligned(16)));
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, blockIdx.z, a.chunk, a.by_slot);
    if (lr.k < 0) return;
    const int i0 = blockIdx.x * kTile, o0 = blockIdx.y * kTile;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wi = (wave & 1) * 64, wo = (wave >> 1) * 64;
    const int first = clamped_offset(a.offsets, lr.k, a.rows);
    const int s1 = min((int64_t)lr.s0 + a.chunk, (int64_t)lr.s1);
    const bool with_db = a.db != nullptr && blockIdx.x == 0 && wi == 0;

    uint4 rx[4], ry[4];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = t + 256 * j, s = s0 + q / P;
            rx[j] = ry[j] = make_uint4(0, 0, 0, 0);
            if (s < s1) {
                const int64_t row = a.gather ? source_row(a.entry, s, a.m, a.rows) : s;
                if (row >= 0) rx[j] = load_piece<T, VEC>((const T*)a.x + row * a.ldx, i0 + (q % P) * E, a.d_in);
                ry[j] = load_piece<T, VEC>((const T*)a.dy + (int64_t)s * a.ldy, o0 + (q % P) * E, a.d_out);
            }
        }
    };
    f32x16 acc[2][2] = {}, sum[2] = {};
    fetch(lr.s0);
    int buf = 0;
    for (int s0 = lr.s0; s0 < s1; s0 += KS, buf ^= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = t + 256 * j;
            *(uint4*)(lds[buf][0] + ColTile<T>::at(q / P, q % P)) = rx[j];
            *(uint4*)(lds[buf][1] + ColTile<T>::at(q / P, q % P)) = ry[j];
        }
        __syncthreads();
        if (s0 + KS < s1) fetch(s0 + KS);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 fx[2], fy[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fx[i] = ColTile<T>::frag(lds[buf][0], wi + 32 * i, j);
                fy[i] = ColTile<T>::frag(lds[buf][1], wo + 32 * i, j);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[i][h] = mma<T>(fx[i], fy[h], acc[i][h]);
                if (with_db) sum[h] = mma<T>(ones<T>(), fy[h], sum[h]);
            }
        }
    }

    // a list of one chunk writes its gradient, a longer one a partial slot
    float* dw = a.dw + (int64_t)lr.k * a.d_out * a.d_in;
    float* db = with_db ? a.db + (int64_t)lr.k * a.d_out : nullptr;
    if (lr.s1 - first > a.chunk) {
        const int64_t slot = first_slot(first, a.chunk) + (lr.s0 - first) / a.chunk;
        dw = a.part + slot * ((int64_t)a.d_out * a.d_in + a.d_out);
        db = with_db ? dw + (int64_t)a.d_out * a.d_in : nullptr;
    }
    // lane: output o = lane % 32, four consecutive inputs per register group
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int o = o0 + wo + 32 * h + (lane & 31);
        if (o >= a.d_out) continue;
        if (with_db && lane < 32) db[o] = sum[h][0];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = i0 + wi + 32 * i + 8 * q + 4 * (lane >> 5);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][h][4 * q + e];
                store4<float, false>(dw + (int64_t)o * a.d_in, c, a.d_in, v);
            }
    }
}

// The partial slots of the lists of several chunks, summed in order; zeros for
// the empty lists.
__global__ __launch_bounds__(256) void k_linear_dw_join(const GradArgs a) {
    const int k = blockIdx.y;
    const int s0 = clamped_offset(a.offsets, k, a.rows), s1 = clamped_offset(a.offsets, k + 1, a.rows);
    const int64_t c = (int64_t)s1 - s0;
    if (c > 0 && c <= a.chunk) return;
    const int64_t wide = (int64_t)a.d_out * a.d_in, slot = wide + a.d_out;
    const int chunks = c <= 0 ? 0 : (int)((c + a.chunk - 1) / a.chunk);
    const float* part = a.part + first_slot(s0, a.chunk) * slot;
    const int64_t all = a.db != nullptr ? slot : wide;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        float v = 0.0f;
        for (int q = 0; q < chunks; ++q) v += part[q * slot + i];
        if (i < wide) a.dw[k * wide + i] = v;
        else a.db[(int64_t)k * a.d_out + (i - wide)] = v;
    }
}

__global__ __launch_bounds__(256) void k_zero(float* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// Rows of a list per workgroup of the weights' gradient: about 1024
// workgroups over all tiles, at least 512 rows.
int chunk_rows(int64_t rows, const gmm_linear_desc* d) {
    const int64_t tiles = ((d->d_in + kTile - 1) / kTile) * ((d->d_out + kTile - 1) / kTile);
    int64_t chunk = (rows * tiles / 1024 + 511) / 512 * 512;
    if (chunk < 512) chunk = 512;
    const int64_t most = ((int64_t)1 << 30);
    return (int)(chunk > most ? most : chunk);
}

gmm_status check_desc(const gmm_linear_desc* d) {
    if (d == nullptr) return GMM_E_ARG;
    gmm_status st = check_width(d->d_in, d->dtype);
    if (st == GMM_OK) st = check_width(d->d_out, d->dtype);
    if (st == GMM_OK && d->sorted_rows != 0 && d->sorted_rows != 1) st = GMM_E_ARG;
    return st;
}

template <typename T, bool VEC, bool BACK> gmm_status launch_linear(const LinArgs& a, int64_t k, hipStream_t stream) {
    LinArgs b = a;
    const int64_t blocks = row_blocks(a.rows, k, kTile, &b.by_slot);
    const int nd = BACK ? a.d_in : a.d_out;
    hipLaunchKernelGGL((k_linear<T, VEC, BACK>), dim3(blocks, (nd + kTile - 1) / kTile), dim3(256), 0, stream, b);
    return launched();
}

template <bool BACK> gmm_status run_linear(const LinArgs& a, int64_t k, int dtype, bool vec, hipStream_t stream) {
    switch (dtype) {
        case GMM_F32:
            return vec ? launch_linear<float, true, BACK>(a, k, stream) : launch_linear<float, false, BACK>(a, k, stream);
        case GMM_BF16:
            return vec ? launch_linear<bf16_t, true, BACK>(a, k, stream) : launch_linear<bf16_t, false, BACK>(a, k, stream);
        default:
            return vec ? launch_linear<_Float16, true, BACK>(a, k, stream)
                       : launch_linear<_Float16, false, BACK>(a, k, stream);
    }
}

template <typename T, bool VEC> gmm_status launch_dw(const GradArgs& a, hipStream_t stream) {
    GradArgs b = a;
    const int64_t blocks = row_blocks(a.rows, a.K, a.chunk, &b.by_slot);
    const dim3 grid((a.d_in + kTile - 1) / kTile, (a.d_out + kTile - 1) / kTile, blocks);
    hipLaunchKernelGGL((k_linear_dw<T, VEC>), grid, dim3(256), 0, stream, b);
    const int64_t wide = (int64_t)a.d_out * a.d_in;
    const int64_t parts = (wide + a.d_out + 1023) / 1024;
    hipLaunchKernelGGL(k_linear_dw_join, dim3(parts < 256 ? parts : 256, a.K), dim3(256), 0, stream, b);
    return launched();
}

}  // namespace

}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_linear(const gmm_routes* routes, const gmm_linear_desc* desc, const void* x, const void* w,
                      const float* bias, void* y, hipStream_t stream) {
    gmm_status st = check_routes(routes);
    if (st == GMM_OK) st = check_desc(desc);
    if (st != GMM_OK) return st;
    if ((st = check_stride(desc->ldx, desc->d_in)) != GMM_OK || (st = check_stride(desc->ldy, desc->d_out)) != GMM_OK)
        return st;
    if (routes->n == 0) return GMM_OK;
    if (x == nullptr || w == nullptr || y == nullptr) return GMM_E_ARG;
    LinArgs a = {routes->offsets, routes->entry, (int)(routes->n * routes->m), (int)routes->n, routes->m, routes->k,
                 false, desc->sorted_rows == 0, x, desc->ldx, w, (int)desc->d_in, (int)desc->d_out, bias, y, desc->ldy};
    const int es = elem_size(desc->dtype);
    const bool vec = desc->d_in * es % 16 == 0 && desc->ldx * es % 16 == 0 && aligned16(x) && aligned16(w) &&
                     desc->d_out * es % 16 == 0 && desc->ldy * es % 16 == 0 && aligned16(y);
    return run_linear<false>(a, routes->k, desc->dtype, vec, stream);
}

gmm_status gmm_linear_backward_workspace_bytes(int64_t n, int32_t m, int32_t k, const gmm_linear_desc* desc,
                                               size_t* bytes) {
    if (bytes == nullptr) return GMM_E_ARG;
    gmm_status st = check_shape(n, m, k);
    if (st == GMM_OK) st = check_desc(desc);
    if (st != GMM_OK) return st;
    const int64_t rows = n * m;
    const int chunk = chunk_rows(rows, desc);
    *bytes = 0;
    if (rows > chunk) *bytes = sizeof(float) * (size_t)(first_slot(rows, chunk) + 1) * desc->d_out * (desc->d_in + 1);
    return GMM_OK;
}

gmm_status gmm_linear_backward(const gmm_routes* routes, const gmm_linear_desc* desc, const void* dy, const void* x,
                               const void* w, void* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
    gmm_status st = check_routes(routes);
    if (st == GMM_OK) st = check_desc(desc);
    if (st != GMM_OK) return st;
    if ((st = check_stride(desc->ldy, desc->d_out)) != GMM_OK) return st;
    if (dx != nullptr && (st = check_stride(desc->lddx, desc->d_in)) != GMM_OK) return st;
    if (dw != nullptr && (st = check_stride(desc->ldx, desc->d_in)) != GMM_OK) return st;
    if (db != nullptr && dw == nullptr) return GMM_E_ARG;
    const int64_t rows = routes->n * routes->m;
    if (rows > 0 && (dy == nullptr || (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr))) return GMM_E_ARG;
    size_t need = 0;
    if (dw != nullptr) {
        st = gmm_linear_backward_workspace_bytes(routes->n, routes->m, routes->k, desc, &need);
        if (st != GMM_OK) return st;
        if (need > 0 && (ws == nullptr || (uintptr_t)ws % 256 != 0)) return GMM_E_ARG;
        if (ws_bytes < need) return GMM_E_WORKSPACE;
    }
    const int es = elem_size(desc->dtype);
    const bool wide = desc->d_in * es % 16 == 0 && desc->d_out * es % 16 == 0;
    const bool dy_vec = desc->ldy * es % 16 == 0 && aligned16(dy);
    if (dx != nullptr && rows > 0) {
        LinArgs a = {routes->offsets, routes->entry, (int)rows, (int)routes->n, routes->m, routes->k, false, false, dy,
                     desc->ldy, w, (int)desc->d_in, (int)desc->d_out, nullptr, dx, desc->lddx};
        const bool vec = wide && dy_vec && aligned16(w) && desc->lddx * es % 16 == 0 && aligned16(dx);
        if ((st = run_linear<true>(a, routes->k, desc->dtype, vec, stream)) != GMM_OK) return st;
    }
    if (dw == nullptr) return GMM_OK;
    if (rows == 0) {   // every list is empty
        const int64_t per = (int64_t)routes->k * desc->d_out;
        hipLaunchKernelGGL(k_zero, dim3(1024), dim3(256), 0, stream, dw, per * desc->d_in);
        if (db != nullptr) hipLaunchKernelGGL(k_zero, dim3(64), dim3(256), 0, stream, db, per);
        return launched();
    }
    GradArgs g = {routes->offsets, routes->entry, (int)rows, routes->m, routes->k, false, desc->sorted_rows == 0,
                  chunk_rows(rows, desc), x, desc->ldx, dy, desc->ldy, (int)desc->d_in, (int)desc->d_out, dw, db,
                  (float*)ws};
    const bool vec = wide && dy_vec && desc->ldx * es % 16 == 0 && aligned16(x);
    switch (desc->dtype) {
        case GMM_F32: return vec ? launch_dw<float, true>(g, stream) : launch_dw<float, false>(g, stream);
        case GMM_BF16: return vec ? launch_dw<bf16_t, true>(g, stream) : launch_dw<bf16_t, false>(g, stream);
        default: return vec ? launch_dw<_Float16, true>(g, stream) : launch_dw<_Float16, false>(g, stream);
    }
}

}  // extern "C"
