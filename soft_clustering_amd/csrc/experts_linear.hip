// gmm_linear and its gradients: one linear model per component on the rows of
// its list, as matrix products on the matrix cores.
//
//   y[s]  = W_k x_s + b_k       contraction over d_in, both operands contiguous along it
//   dx[s] = W_k^T dy[s]         contraction over d_out; W_k is contiguous along the output
//   dW_k  = sum_s dy[s] x_s^T   contraction over the list's rows; neither is contiguous along it
//   db_k  = sum_s dy[s]
//
// A workgroup computes a tile of 64 x 64 blocks, one a wave, each as 2 x 2
// blocks of v_mfma_f32_32x32x16 (16-bit storage) or v_mfma_f32_32x32x2_f32,
// fp32 accumulators.  Operand tiles go through LDS in 16-byte pieces, 64 or 128
// bytes of the contraction a step, two or three steps at a time: the pieces of
// the next steps are fetched while one is multiplied, straight into LDS
// (global_load_lds) where rows allow 16-byte pieces, through registers where
// they do not.  An operand contiguous along the contraction is kept [row][step],
// its pieces XOR-swizzled by the row, and read a fragment (8 or 4 elements) at a
// time; one that is contiguous along the output is kept [contraction][columns]
// and read with ds_read_b64_tr_b16 (16-bit) or element by element (fp32).
// Pieces beyond a row's end, a list's end or the contraction come from 16 zero
// bytes, so they add nothing.
//
// Measured (bf16): 32768 rows in 8 lists, 1024 -> 2048: forward 143 us
// (960 TFLOP/s), dx 136 (1010), dw 173 (795); in 64 lists 201, 187, 269: the
// weights' 268 MB and their gradient's 537 MB pass the memory too.  Bound there
// by LDS reads and the barrier of each step; 2e6 rows in 256 lists, 128 -> 128,
// fp16, 225 us: bound by the memory, where the gathered rows pass twice (a
// point's two lists lie far apart).  fp32 is bound by its products (a sixteenth
// of the 16-bit rate) and, on short chunks, by latency.
//
// Workgroup -> rows: find_rows (experts_internal.h); the host never learns the lists' lengths.

#include <type_traits>

#include "experts_internal.h"

namespace gmm {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;
typedef __attribute__((address_space(3))) char lds_char;

// A workgroup: its waves along the rows and along the columns of its tile, the
// bytes of the contraction a step takes, the steps in LDS (one multiplied, the others on their way)
// and the workgroups a compute unit is meant to hold.  NARROW: rows may be of less than 16 bytes.
template <int WM_, int WN_, int STEP, int STAGES, int HELD, bool NARROW = false> struct Shape {
    static constexpr bool kNarrow = NARROW;
    static constexpr int WM = WM_, WN = WN_, kStep = STEP, kStages = STAGES, kHeld = HELD;
    static constexpr int kThreads = 64 * WM * WN, kM = 64 * WM, kN = 64 * WN;
    static constexpr int kFrags = kStep / 32;   // fragments of a step
    static constexpr int kABytes = kM * kStep, kBBytes = kN * kStep;   // one operand, one step
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kWavesPerSimd = HELD * WM * WN / 4;
    static constexpr int kWaves = WM * WN;
    static constexpr int kAJ = kABytes / 1024 / kWaves, kBJ = kBBytes / 1024 / kWaves;   // wave loads a step
};

// e / m for 0 <= e < 2^30, 1 <= m <= 16, magic = 2^34 / m + 1: the excess of
// magic is at most 1, so e magic / 2^34 exceeds e / m by less than 1 / 16, and
// e / m lies at least 1 / m below the next whole number (m = 16: magic's excess over 2^30 is
// exactly 1 and e / 2^34 < 1 / 16).
__host__ __device__ __forceinline__ uint64_t magic_of(int m) { return ((uint64_t)1 << 34) / m + 1; }
__device__ __forceinline__ int over_m(int e, uint64_t magic) { return (int)((uint64_t)(uint32_t)e * magic >> 34); }

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

// Sum of the elements a lane holds of a fragment: half of the contraction of row lane % 32.
template <typename T> __device__ __forceinline__ float add_elements(const uint4& frag) {
    float v[Vec16<T>::kElems];
    Vec16<T>::unpack(frag, v);
#pragma unroll
    for (int w = Vec16<T>::kElems / 2; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) v[i] += v[i + w];
    return v[0];
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

// [row][kStep bytes]: pieces XOR-swizzled so that the 8 rows that one LDS cycle of
// a fragment read touches lie in 8 different places of the 256 bytes of banks.
template <int kStep> struct RowTile {
    static constexpr int kPieces = kStep / 16, kRowsPerLoad = 64 / kPieces;
    __device__ __forceinline__ static int swz(int row) { return kPieces == 8 ? row & 7 : (row >> 2) & 3; }
    __device__ __forceinline__ static int at(int row, int piece) { return row * kStep + ((piece ^ swz(row)) << 4); }
    // lane's fragment j of the step for row block `r0`
    __device__ __forceinline__ static uint4 frag(const char* t, int r0, int j) {
        const int lane = threadIdx.x & 63;
        return *(const uint4*)(t + at(r0 + (lane & 31), 2 * j + (lane >> 5)));
    }
};

// [contraction][N columns].
template <typename T, int N, int kStep> struct ColTile {
    static constexpr int kRows = kStep / (int)sizeof(T);         // contraction elements of a step
    static constexpr int kPieces = N * (int)sizeof(T) / 16;      // 16-byte pieces of a row
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
    int K;
    uint64_t magic;      // of m
    bool by_slot;
    bool gather;         // rows of a are the points' (entry[s] / m), else by slot
    const void* a;       // x or dy
    int64_t lda;
    const void* w;       // [K, d_out, d_in]
    int d_in, d_out;
    const float* bias;
    void* c;             // y or dx
    int64_t ldc;
    int row_blocks, col_blocks, col_step;
};

// Row of x behind an entry, or -1.
__device__ __forceinline__ int source_row(int e, uint64_t magic, int rows) {
    return e >= 0 && e < rows ? over_m(e, magic) : -1;
}

// Workgroup -> tile.  Workgroups go round the 8 XCDs; consecutive tiles (the columns of a
// row block, then the next row block of the same list) stay on one, whose L2 then
// serves the rows to all column blocks and the list's weights to all row blocks.
__device__ __forceinline__ int tile_of(int block, int tiles) {
    const int per = (tiles + 7) >> 3;
    return (block & 7) * per + (block >> 3);
}

// y = x W^T + b (BACK false) or dx = dy W (BACK true) on one tile.  VIN: rows along d_in (x, W, dx) are whole
// aligned pieces; VOUT: rows along d_out (y, dy) are.  An operand whose rows are not goes through registers,
// one step ahead; a result whose rows are not leaves from the accumulators.
template <typename T, bool VIN, bool VOUT, bool BACK, typename S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void k_linear(const LinArgs a) {
    constexpr bool AV = BACK ? VOUT : VIN, BV = VIN, CV = BACK ? VIN : VOUT;   // the operands' and the result's rows
    constexpr int WM = S::WM, kStep = S::kStep, kStages = S::kStages, kFrags = S::kFrags;
    using RT = RowTile<kStep>;
    using CT = ColTile<T, S::kN, kStep>;
    constexpr int E = Vec16<T>::kElems, KS = kStep / (int)sizeof(T);   // elements of a piece, of a step
    constexpr int AJ = S::kAJ, BJ = S::kBJ, kStage = S::kStage;
    constexpr int kOut = S::kWaves * 32 * 64 * (int)sizeof(T);   // the epilogue's rows
    __shared__ char lds[kStages * kStage > kOut ? kStages * kStage : kOut] __attribute__((aligned(16)));
    const int tile = tile_of(blockIdx.x, a.row_blocks * a.col_blocks);
    if (tile >= a.row_blocks * a.col_blocks) return;
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, tile / a.col_blocks, S::kM, a.by_slot);
    if (lr.k < 0) return;
    const int kd = BACK ? a.d_out : a.d_in, nd = BACK ? a.d_in : a.d_out;   // contraction, output width
    const int n0 = tile % a.col_blocks * a.col_step, n1 = min(n0 + a.col_step, nd);   // this tile's outputs
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave % WM * 64, wn = wave / WM * 64;
    const T* w = (const T*)a.w + (int64_t)lr.k * a.d_in * a.d_out;

    // Wave load j covers the RA tile rows from RA (wave AJ + j) on; the piece that sits at
    // place p of a row is p ^ swz(row), the same for every j (RA rows are a whole period).
    constexpr int PA = RT::kPieces, RA = RT::kRowsPerLoad;
    const int ca = ((lane % PA) ^ RT::swz(lane / PA)) * E;
    // Each wave load has its own pointer, advanced by the step; where a lane has no row or
    // column it stays on the zero piece.
    const char* zero = zero_address();
    const char *pa[AJ], *pb[BJ];
    int64_t sa[AJ], sb[BJ];   // bytes a step
    bool there_a[AJ], there_b[BJ];
    int rb[BJ];               // BACK: contraction row within the step
    int e[AJ];
    if (a.gather) {
#pragma unroll
        for (int j = 0; j < AJ; ++j) e[j] = a.entry[min(lr.s0 + RA * (wave * AJ + j) + lane / PA, lr.s1 - 1)];
    }
#pragma unroll
    for (int j = 0; j < AJ; ++j) {
        const int s = lr.s0 + RA * (wave * AJ + j) + lane / PA;
        const int row = a.gather ? source_row(e[j], a.magic, a.rows) : s;
        there_a[j] = s < lr.s1 && row >= 0;
        pa[j] = there_a[j] ? (const char*)((const T*)a.a + (int64_t)row * a.lda + (AV ? ca : 0)) : zero;
        sa[j] = there_a[j] ? kStep : 0;
    }
    constexpr int RI = 64 / CT::kPieces;   // BACK: tile rows of a wave load
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
        if constexpr (!BACK) {
            const int r = n0 + RA * (wave * BJ + j) + lane / PA;
            there_b[j] = r < n1;
            pb[j] = there_b[j] ? (const char*)(w + (int64_t)r * kd + (BV ? ca : 0)) : zero;
            sb[j] = there_b[j] ? kStep : 0;
            rb[j] = 0;
        } else {
            rb[j] = (wave * BJ + j) * RI + lane / CT::kPieces;
            const int c = n0 + ((lane % CT::kPieces) ^ CT::swz(rb[j])) * E;
            there_b[j] = c < n1;
            pb[j] = there_b[j] ? (const char*)(w + (int64_t)rb[j] * nd + (BV ? c : 0)) : zero;
            sb[j] = there_b[j] ? (int64_t)KS * nd * (int)sizeof(T) : 0;
        }
    }
    const uint32_t base = lds_address(lds);
    Loose ra[AV ? 1 : AJ], rl[BV ? 1 : BJ];
    // the pieces of the step at k0, the next one not yet fetched: into buffer `buf` or into registers
    auto fetch = [&](int k0, int buf) {
        const uint32_t to = base + buf * kStage;
        const bool whole = k0 + KS <= kd;
#pragma unroll
        for (int j = 0; j < AJ; ++j) {
            if constexpr (AV) {
                fetch_piece(whole || k0 + ca < kd ? pa[j] : zero, to + (wave * AJ + j) * 1024);
                pa[j] += sa[j];
            } else {
                ra[j] = load_piece<T, S::kNarrow>((const T*)pa[j], there_a[j], k0 + ca, kd, zero);
            }
        }
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            if constexpr (BV) {
                fetch_piece(whole || k0 + (BACK ? rb[j] : ca) < kd ? pb[j] : zero, to + S::kABytes + (wave * BJ + j) * 1024);
            } else if constexpr (BACK) {
                const int c = n0 + ((lane % CT::kPieces) ^ CT::swz(rb[j])) * E;
                rl[j] = load_piece<T, S::kNarrow>((const T*)pb[j], there_b[j] && k0 + rb[j] < kd, c, nd, zero);
            } else {
                rl[j] = load_piece<T, S::kNarrow>((const T*)pb[j], there_b[j], k0 + ca, kd, zero);
            }
            if (BV || BACK) pb[j] += sb[j];
        }
    };
    auto put = [&](int buf) {   // what came into registers
        char* to = lds + buf * kStage + lane * 16;
        if constexpr (!AV) {
#pragma unroll
            for (int j = 0; j < AJ; ++j) *(uint4*)(to + (wave * AJ + j) * 1024) = settle(ra[j]);
        }
        if constexpr (!BV) {
#pragma unroll
            for (int j = 0; j < BJ; ++j) *(uint4*)(to + S::kABytes + (wave * BJ + j) * 1024) = settle(rl[j]);
        }
    };

    // blocks of columns with outputs (16-bit pieces: not worth the branches)
    constexpr bool kAll = AV && BV && sizeof(T) == 2;
    const bool live[2] = {kAll || n0 + wn < n1, kAll || n0 + wn + 32 < n1};
    f32x16 acc[2][2] = {};
    if (!BACK && a.bias != nullptr) {   // sums start from the bias
        const float* bias = a.bias + (int64_t)lr.k * nd;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if constexpr (CV) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = n0 + wn + 32 * h + 8 * q + 4 * (lane >> 5);
                    float b[4];
                    __builtin_memcpy(b, bias + (c < nd ? c : 0), sizeof(b));
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][h][4 * q + e] = acc[1][h][4 * q + e] = b[e];
                }
            } else {
                const float b = bias[min(n0 + wn + 32 * h + (lane & 31), nd - 1)];
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][h][r] = acc[1][h][r] = b;
            }
    }
    const int steps = (kd + KS - 1) / KS;
    constexpr int kAhead = AV && BV ? kStages - 1 : 1;   // steps on their way (registers hold one)
    for (int i = 0; i < kAhead && i < steps; ++i) fetch(i * KS, i);
    int buf = 0;
    for (int i = 0; i < steps; ++i) {
        // this step's pieces are in LDS, and every wave has read the last step's
        if (kAhead > 1 && i + kAhead - 1 < steps) wait_pieces<(kAhead - 1) * (AJ + BJ)>();
        else if (AV || BV) wait_pieces<0>();
        put(buf);
        __syncthreads();
        if (i + kAhead < steps) fetch((i + kAhead) * KS, buf + kAhead < kStages ? buf + kAhead : buf + kAhead - kStages);
        const char* ta = lds + buf * kStage;
        const char* tb = ta + S::kABytes;
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            uint4 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = RT::frag(ta, wm + 32 * i, j);
                fb[i] = BACK ? CT::frag(tb, wn + 32 * i, j) : RT::frag(tb, wn + 32 * i, j);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (live[h]) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)   // CV: lanes along the slots, else along the columns
                        acc[i][h] = CV ? mma<T>(fb[h], fa[i], acc[i][h]) : mma<T>(fa[i], fb[h], acc[i][h]);
                }
        }
        buf = buf + 1 < kStages ? buf + 1 : 0;
    }

    if constexpr (CV) {
        // lane: slot lane % 32, four consecutive outputs per register group;
        // through LDS, so that a row leaves in whole pieces: the wave's 64 x 64 block, two halves of
        // 32 rows, pieces swizzled by the row
        constexpr int RB = 64 * (int)sizeof(T), PR = RB / 16;   // bytes, pieces of a row
        __syncthreads();
        char* mine = lds + wave * (32 * RB);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    T v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) from_f32(acc[i][h][4 * q + e], v + e);
                    const int r = lane & 31, c = (32 * h + 8 * q + 4 * (lane >> 5)) * (int)sizeof(T);
                    __builtin_memcpy(__builtin_assume_aligned(mine + r * RB + (((c >> 4) ^ (r & (PR - 1))) << 4) + (c & 15),
                                                              4 * sizeof(T)), v, 4 * sizeof(T));
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            constexpr int U = 32 * PR / 64, RU = 64 / PR;
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = RU * u + lane / PR;
                v[u] = *(const uint4*)(mine + r * RB + (((lane % PR) ^ (r & (PR - 1))) << 4));
            }
            const int s = lr.s0 + wm + 32 * i + lane / PR, c = n0 + wn + lane % PR * E;
            T* to = (T*)a.c + (int64_t)s * a.ldc + c;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + RU * u < lr.s1 && c < n1) *(uint4*)(to + (int64_t)(RU * u) * a.ldc) = v[u];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    } else {
        // lane: output lane % 32, slots 8 (r / 4) + 4 (lane / 32) + r % 4: a register's store covers 32
        // outputs of two rows
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int s = lr.s0 + wm + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (s >= lr.s1) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = n0 + wn + 32 * h + (lane & 31);
                    if (c < n1) from_f32(acc[i][h][r], (T*)a.c + (int64_t)s * a.ldc + c);
                }
            }
    }
}

// ---- few rows

constexpr int kFewRows = 16, kFewOutputs = 16, kFewWaves = 4;

// y = x W^T + b on 16 outputs of up to 16 rows of a list: nothing to share between
// workgroups, so no LDS tiles.  The waves split the contraction, every lane streams its row of
// W_k and of x into 16 x 16 products, and the four partial blocks are summed in order.
template <typename T, bool VIN, bool VOUT, bool NARROW>
__global__ __launch_bounds__(64 * kFewWaves) void k_linear_few(const LinArgs a) {
    constexpr int E = Vec16<T>::kElems, KS = 4 * E;   // contraction of a product
    constexpr int kAhead = 4;                         // products whose pieces are in flight
    __shared__ f32x4 part[kFewWaves][64];
    const int row_block = blockIdx.x / a.col_blocks, n0 = blockIdx.x % a.col_blocks * kFewOutputs;
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, row_block, kFewRows, a.by_slot);
    if (lr.k < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = lr.s0 + (lane & 15), o = n0 + (lane & 15);
    int row = s < lr.s1 ? s : -1;
    if (a.gather) {
        const int e = a.entry[min(s, lr.s1 - 1)];
        row = s < lr.s1 ? source_row(e, a.magic, a.rows) : -1;
    }
    const T* w = (const T*)a.w + ((int64_t)lr.k * a.d_out + min(o, a.d_out - 1)) * a.d_in;
    const T* x = (const T*)a.a + (int64_t)max(row, 0) * a.lda;
    const bool has_w = o < a.d_out, has_x = row >= 0;
    f32x4 acc = {};
    const int mine = (lane >> 4) * E;
    const char* zero = zero_address();
    auto piece = [&](const T* p, bool there, int k) {
        if constexpr (VIN) return Loose{load16<16>(there && k < a.d_in ? (const char*)(p + k) : zero), 0};
        else return load_piece<T, NARROW>(p, there, k, a.d_in, zero);
    };
    for (int k0 = wave * KS; k0 < a.d_in; k0 += kAhead * kFewWaves * KS) {
        Loose fw[kAhead], fx[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            fw[u] = piece(w, has_w, k0 + u * kFewWaves * KS + mine);
            fx[u] = piece(x, has_x, k0 + u * kFewWaves * KS + mine);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            acc = VIN ? mma16<T>(fw[u].v, fx[u].v, acc) : mma16<T>(settle(fw[u]), settle(fx[u]), acc);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0 || s >= lr.s1) return;
    const int c = n0 + 4 * (lane >> 4);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = acc[e];
#pragma unroll
        for (int q = 1; q < kFewWaves; ++q) v[e] += part[q][lane][e];
        if (a.bias != nullptr) v[e] += a.bias[(int64_t)lr.k * a.d_out + min(c + e, a.d_out - 1)];
    }
    store4<T, VOUT>((T*)a.c + (int64_t)s * a.ldc, c, a.d_out, v);
}

constexpr int kBackRows = 8, kBackWaves = 8, kBackOutputs = 512;   // slots, waves, outputs of W in LDS at a time

// dx = dy W on up to 8 rows of a list: a lane owns 16 bytes of columns (VIN) or one, the lanes of a wave that
// the columns leave over and the waves split the contraction, and the partial sums are added in a
// fixed order.  The rows of W_k pass once, whole; dy waits in LDS as [output][slot].
template <typename T, bool VIN>
__global__ __launch_bounds__(64 * kBackWaves) void k_linear_few_back(const LinArgs a, int lanes_log2) {
    constexpr int V = VIN ? Vec16<T>::kElems : 1, kAhead = 4;
    __shared__ __align__(16) float dy[kBackOutputs][kBackRows];
    __shared__ float part[kBackWaves][64 * V];
    const int row_block = blockIdx.x / a.col_blocks, lanes = 1 << lanes_log2;
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, row_block, kBackRows, a.by_slot);
    if (lr.k < 0) return;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, subs = 64 >> lanes_log2;
    const int c = (blockIdx.x % a.col_blocks * lanes + (lane & (lanes - 1))) * V, sub = lane >> lanes_log2;
    const int n = min(kBackRows, lr.s1 - lr.s0);
    const T* w = (const T*)a.w + (int64_t)lr.k * a.d_out * a.d_in + (c < a.d_in ? c : 0);
    float acc[kBackRows][V] = {};
    for (int o0 = 0; o0 < a.d_out; o0 += kBackOutputs) {
        const int here = min(kBackOutputs, a.d_out - o0);
        __syncthreads();   // the last outputs are through
        for (int i = t; i < kBackOutputs * kBackRows; i += 64 * kBackWaves) {
            const int r = i / kBackOutputs, o = i % kBackOutputs;
            dy[o][r] = r < n && o < here ? to_f32(((const T*)a.a)[(int64_t)(lr.s0 + r) * a.lda + o0 + o]) : 0.0f;
        }
        __syncthreads();
        const int stride = kBackWaves * subs;
        for (int o = wave * subs + sub; o < here; o += kAhead * stride) {
            float v[kAhead][V];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const T* row = w + (int64_t)(o0 + min(o + u * stride, here - 1)) * a.d_in;
                if constexpr (VIN) Vec16<T>::unpack(*(const uint4*)row, v[u]);
                else v[u][0] = to_f32(*row);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (o + u * stride < here) {
#pragma unroll
                    for (int r = 0; r < kBackRows; ++r)
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[r][e] = fmaf(dy[o + u * stride][r], v[u][e], acc[r][e]);
                }
        }
    }
    for (int r = 0; r < n; ++r) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float sum = 0.0f;   // acc[r][e]
#pragma unroll
            for (int q = 0; q < kBackRows; ++q) sum = q == r ? acc[q][e] : sum;
            for (int m = lanes; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
            if (sub == 0) part[wave][(lane & (lanes - 1)) * V + e] = sum;
        }
        __syncthreads();
        for (int i = t; i < lanes * V; i += 64 * kBackWaves) {
            const int to = blockIdx.x % a.col_blocks * lanes * V + i;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < kBackWaves; ++q) sum += part[q][i];
            if (to < a.d_in) from_f32(sum, (T*)a.c + (int64_t)(lr.s0 + r) * a.ldc + to);
        }
        __syncthreads();
    }
}

// ---- gradient of the weights

struct GradArgs {
    const int32_t* offsets;
    const int32_t* entry;
    int rows, K;
    uint64_t magic;
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
    int row_blocks, in_blocks, out_blocks, in_step, out_step;
};

// First partial slot of a list of more than one chunk that starts at slot a:
// such a list of c rows takes the ceil(c / chunk) slots up to the next list's first one,
// since floor(2 b / chunk) - floor(2 a / chunk) >= ceil(2 c / chunk) - 1 >= ceil(c / chunk) for c > chunk.
__device__ __host__ __forceinline__ int64_t first_slot(int64_t a, int chunk) { return 2 * a / chunk; }

// dW (and db) over one chunk of one list, one tile: 64 WM of d_in x 64 WN of d_out.
template <typename T, bool VIN, bool VOUT, typename S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void k_linear_dw(const GradArgs a) {
    constexpr int WM = S::WM, kStages = S::kStages, kFrags = S::kFrags;
    using XT = ColTile<T, S::kM, S::kStep>;
    using YT = ColTile<T, S::kN, S::kStep>;
    constexpr int E = Vec16<T>::kElems, KS = XT::kRows;
    constexpr int XJ = S::kAJ, YJ = S::kBJ, kStage = S::kStage;
    constexpr int XR = 64 / XT::kPieces, YR = 64 / YT::kPieces;   // tile rows of a wave load
    __shared__ char lds[kStages * kStage] __attribute__((aligned(16)));
    __shared__ int source[2 * S::kThreads];
    const int per_row = a.in_blocks * a.out_blocks;
    // The lists' lengths differ, so each XCD takes an eighth of the tiles of every chunk (a run of
    // them, which shares rows of x and dy); with fewer than 8 tiles, each tile goes round the XCDs.
    const int per = (per_row + 7) >> 3, b = blockIdx.x;
    const int block = per_row < 8 ? b / per_row : (b >> 3) / per;
    const int tile = per_row < 8 ? (b % per_row + (int)((int64_t)block * per_row >> 3)) % per_row : (b & 7) * per + (b >> 3) % per;
    if (block >= a.row_blocks || tile >= per_row) return;
    const ListRows lr = find_rows(a.offsets, a.K, a.rows, block, a.chunk, a.by_slot);
    if (lr.k < 0) return;
    const int i0 = tile % a.in_blocks * a.in_step, o0 = tile / a.in_blocks * a.out_step;
    const int i1 = min(i0 + a.in_step, a.d_in), o1 = min(o0 + a.out_step, a.d_out);   // this tile's weights
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wi = wave % WM * 64, wo = wave / WM * 64;
    const int first = lr.first;
    const int s1 = min((int64_t)lr.s0 + a.chunk, (int64_t)lr.s1);
    const bool with_db = a.db != nullptr && i0 == 0 && wi == 0;

    const uint32_t base = lds_address(lds);
    Loose rx[VIN ? 1 : XJ], ry[VOUT ? 1 : YJ];
    // Rows of x behind the slots, one slot a thread and segment of kThreads slots, two segments in
    // LDS: an entry loaded in every step would be waited for behind the pieces on their way.
    constexpr int R = S::kThreads, SPR = R / KS;   // slots, steps of a segment
    auto entry_of = [&](int seg) {
        const int64_t s = lr.s0 + (int64_t)seg * R + t;
        if (s >= s1) return -1;
        return a.gather ? a.entry[s] : (int)s;
    };
    auto keep = [&](int seg, int e) {
        if (a.gather) e = source_row(e, a.magic, a.rows);
        source[(seg & 1) * R + t] = e;
    };
    keep(0, entry_of(0));
    __syncthreads();
    const char* zero = zero_address();
    int cx[XJ];           // column of this lane's piece of x
    const char* py[YJ];   // dy, advanced by the step
    int64_t sy[YJ];
    int cy[YJ], rowy[YJ];
#pragma unroll
    for (int j = 0; j < XJ; ++j)
        cx[j] = i0 + ((lane % XT::kPieces) ^ XT::swz((wave * XJ + j) * XR + lane / XT::kPieces)) * E;
#pragma unroll
    for (int j = 0; j < YJ; ++j) {
        rowy[j] = lr.s0 + (wave * YJ + j) * YR + lane / YT::kPieces;
        cy[j] = o0 + ((lane % YT::kPieces) ^ YT::swz((wave * YJ + j) * YR + lane / YT::kPieces)) * E;
        const bool there = cy[j] < o1;
        py[j] = there ? (const char*)((const T*)a.dy + (int64_t)rowy[j] * a.ldy + (VOUT ? cy[j] : 0)) : zero;
        sy[j] = there ? (int64_t)KS * a.ldy * (int)sizeof(T) : 0;
    }
    // the step at slot s0, the next one not yet fetched; its rows of x are in from[]
    auto fetch = [&](int s0, int buf) {
        const uint32_t to = base + buf * kStage;
        const bool whole = s0 + KS <= s1;
#pragma unroll
        for (int j = 0; j < XJ; ++j) {
            const int from = source[(s0 - lr.s0 + (wave * XJ + j) * XR + lane / XT::kPieces) & (2 * R - 1)];
            const bool there = from >= 0 && cx[j] < i1;
            const char* row = (const char*)((const T*)a.x + (int64_t)from * a.ldx);
            if constexpr (VIN) fetch_piece(there ? row + cx[j] * (int)sizeof(T) : zero, to + (wave * XJ + j) * 1024);
            else rx[j] = load_piece<T, S::kNarrow>((const T*)row, there, cx[j], a.d_in, zero);
        }
#pragma unroll
        for (int j = 0; j < YJ; ++j) {
            const bool there = whole || s0 - lr.s0 + rowy[j] < s1;
            if constexpr (VOUT) fetch_piece(there ? py[j] : zero, to + S::kABytes + (wave * YJ + j) * 1024);
            else ry[j] = load_piece<T, S::kNarrow>((const T*)py[j], there, cy[j], a.d_out, zero);
            py[j] += sy[j];
        }
    };
    auto put = [&](int buf) {   // what came into registers
        char* to = lds + buf * kStage + lane * 16;
        if constexpr (!VIN) {
#pragma unroll
            for (int j = 0; j < XJ; ++j) *(uint4*)(to + (wave * XJ + j) * 1024) = settle(rx[j]);
        }
        if constexpr (!VOUT) {
#pragma unroll
            for (int j = 0; j < YJ; ++j) *(uint4*)(to + S::kABytes + (wave * YJ + j) * 1024) = settle(ry[j]);
        }
    };

    // blocks with gradients (16-bit pieces: not worth the branches)
    constexpr bool kAll = VIN && VOUT && sizeof(T) == 2;
    const bool live[2] = {kAll || i0 + wi < i1, kAll || i0 + wi + 32 < i1};
    const bool live_o[2] = {kAll || o0 + wo < o1, kAll || o0 + wo + 32 < o1};
    f32x16 acc[2][2] = {};
    float sum[2] = {};
    const int steps = (s1 - lr.s0 + KS - 1) / KS;
    constexpr int kAhead = VIN && VOUT ? kStages - 1 : 1;
    for (int i = 0; i < kAhead && i < steps; ++i) fetch(lr.s0 + i * KS, i);
    int buf = 0, next = -1;   // next: the entry of this thread's slot in the segment after the one being fetched
    static_assert(SPR - 3 >= kAhead && (R & (R - 1)) == 0, "a segment is loaded and kept while its forerunner is fetched");
    for (int i = 0; i < steps; ++i) {
        if (kAhead > 1 && i + kAhead - 1 < steps) wait_pieces<(kAhead - 1) * (XJ + YJ)>();
        else if (VIN || VOUT) wait_pieces<0>();
        put(buf);
        // the last step of a segment is about to be fetched: every wave is past the segment before it
        const int f = i + kAhead;
        if (f % SPR == SPR - 1) keep(f / SPR + 1, next);
        __syncthreads();
        if (f < steps) {
            fetch(lr.s0 + f * KS, buf + kAhead < kStages ? buf + kAhead : buf + kAhead - kStages);
            if (f % SPR == SPR - 3) next = entry_of(f / SPR + 1);
        }
        const char* tx = lds + buf * kStage;
        const char* ty = tx + S::kABytes;
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            uint4 fx[2], fy[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fx[i] = XT::frag(tx, wi + 32 * i, j);
                fy[i] = YT::frag(ty, wo + 32 * i, j);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (live[i] && live_o[h]) acc[i][h] = mma<T>(fy[h], fx[i], acc[i][h]);
            if (with_db) {
#pragma unroll
                for (int h = 0; h < 2; ++h) sum[h] += add_elements<T>(fy[h]);
            }
        }
        buf = buf + 1 < kStages ? buf + 1 : 0;
    }

    // a list of one chunk writes its gradient, a longer one a partial slot
    float* dw = a.dw + (int64_t)lr.k * a.d_out * a.d_in;
    float* db = with_db ? a.db + (int64_t)lr.k * a.d_out : nullptr;
    if (lr.s1 - first > a.chunk) {
        const int64_t slot = first_slot(first, a.chunk) + (lr.s0 - first) / a.chunk;
        dw = a.part + slot * ((int64_t)a.d_out * a.d_in + a.d_out);
        db = with_db ? dw + (int64_t)a.d_out * a.d_in : nullptr;
    }
    if (with_db) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float all = halves_sum(sum[h]);
            const int o = o0 + wo + 32 * h + (lane & 31);
            if (lane < 32 && o < o1) db[o] = all;
        }
    }
    // lane: input i = lane % 32, so that a register's store covers 128 bytes of two rows; outputs
    // 8 (r / 4) + 4 (lane / 32) + r % 4
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int o = o0 + wo + 32 * h + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
            if (o >= o1) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = i0 + wi + 32 * i + (lane & 31);
                if (c < i1) dw[(int64_t)o * a.d_in + c] = acc[i][h][r];
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
        int q = 0;
        for (; q + 8 <= chunks; q += 8) {   // eight loads in flight, added in order
            float p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) p[u] = part[(q + u) * slot + i];
#pragma unroll
            for (int u = 0; u < 8; ++u) v += p[u];
        }
        for (; q < chunks; ++q) v += part[q * slot + i];
        if (i < wide) a.dw[k * wide + i] = v;
        else a.db[(int64_t)k * a.d_out + (i - wide)] = v;
    }
}

__global__ __launch_bounds__(256) void k_zero(float* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// Rows of a list per workgroup of the weights' gradient: 1024 workgroups at most over all
// tiles, and rows enough that writing and reading a partial slot (8 bytes a weight) costs no
// more than reading the rows, as long as that leaves 256 workgroups (fp32, whose products take sixteen
// times as long: 512; 60032 rows in 37 lists, 128 x 128: 54 us with 256, 38 with 512).
int chunk_rows(int64_t rows, const gmm_linear_desc* d) {
    const int64_t tiles = ((d->d_in + 127) / 128) * ((d->d_out + 127) / 128);
    const int64_t most_groups = rows * tiles / 1024, least_groups = rows * tiles / (d->dtype == GMM_F32 ? 512 : 256);
    int64_t chunk = 8 * d->d_in * d->d_out / ((d->d_in + d->d_out) * elem_size(d->dtype));
    if (chunk > least_groups) chunk = least_groups;
    if (chunk < most_groups) chunk = most_groups;
    chunk = (chunk / 128 + 1) * 128;
    const int64_t most = (int64_t)1 << 30;
    return (int)(chunk > most ? most : chunk);
}

int blocks_of(int width, int tile) { return (width + tile - 1) / tile; }

// Columns of each of a width's tiles: as even as blocks of 32 allow (130: 96 and 34, not 128 and 2).
int step_of(int width, int tile) {
    const int blocks = blocks_of(width, tile);
    return ((width + blocks - 1) / blocks + 31) / 32 * 32;
}

gmm_status check_desc(const gmm_linear_desc* d) {
    if (d == nullptr) return GMM_E_ARG;
    gmm_status st = check_width(d->d_in, d->dtype);
    if (st == GMM_OK) st = check_width(d->d_out, d->dtype);
    if (st == GMM_OK && d->sorted_rows != 0 && d->sorted_rows != 1) st = GMM_E_ARG;
    return st;
}

// Tiles of a launch, or GMM_E_ARG where they do not fit a grid.
gmm_status grid_of(int64_t tiles, int* grid) {
    if (tiles > ((int64_t)1 << 24) - 8) return GMM_E_ARG;   // a grid holds fewer than 2^32 threads
    *grid = (int)((tiles + 7) / 8 * 8);
    return GMM_OK;
}

template <typename T, bool VIN, bool VOUT, bool BACK, typename S>
gmm_status launch_shape(const LinArgs& a, hipStream_t stream) {
    LinArgs b = a;
    int grid;
    b.row_blocks = (int)row_blocks(a.rows, a.K, S::kM, &b.by_slot);
    const int nd = BACK ? a.d_in : a.d_out;
    b.col_blocks = blocks_of(nd, S::kN);
    b.col_step = step_of(nd, S::kN);
    const gmm_status st = grid_of((int64_t)b.row_blocks * b.col_blocks, &grid);
    if (st != GMM_OK) return st;
    hipLaunchKernelGGL((k_linear<T, VIN, VOUT, BACK, S>), dim3(grid), dim3(S::kThreads), 0, stream, b);
    return launched();
}

template <typename T, bool VIN, bool VOUT, bool NARROW = false> gmm_status launch_few(const LinArgs& a, hipStream_t stream) {
    LinArgs b = a;
    int grid;
    b.row_blocks = (int)row_blocks(a.rows, a.K, kFewRows, &b.by_slot);
    b.col_blocks = blocks_of(a.d_out, kFewOutputs);
    const gmm_status st = grid_of((int64_t)b.row_blocks * b.col_blocks, &grid);
    if (st != GMM_OK) return st;
    hipLaunchKernelGGL((k_linear_few<T, VIN, VOUT, NARROW>), dim3(b.row_blocks * b.col_blocks), dim3(64 * kFewWaves), 0, stream, b);
    return launched();
}

template <typename T, bool VIN> gmm_status launch_few_back(const LinArgs& a, hipStream_t stream) {
    LinArgs b = a;
    int grid, lg = 0;
    const int pieces = VIN ? a.d_in / Vec16<T>::kElems : a.d_in, line = VIN ? 8 : 128 / (int)sizeof(T);
    while ((1 << lg) < line && (1 << lg) < pieces) ++lg;   // at most a line of W's row a workgroup
    b.row_blocks = (int)row_blocks(a.rows, a.K, kBackRows, &b.by_slot);
    b.col_blocks = blocks_of(pieces, 1 << lg);
    const gmm_status st = grid_of((int64_t)b.row_blocks * b.col_blocks, &grid);
    if (st != GMM_OK) return st;
    hipLaunchKernelGGL((k_linear_few_back<T, VIN>), dim3(b.row_blocks * b.col_blocks), dim3(64 * kBackWaves), 0, stream, b, lg);
    return launched();
}

// Small: 128 x 128 tiles, several workgroups a compute unit, whose waits hide behind each
// other.  Large: 256 x 256, half the operand traffic a product, one workgroup a compute unit.
using Small = Shape<2, 2, 64, 2, 3>;
using Narrow = Shape<2, 2, 64, 2, 3, true>;
using Large = Shape<4, 4, 128, 2, 1>;
using LargeGrad = Shape<4, 4, 64, 3, 1>;

// Large pays where its tiles go twice round the 256 compute units, a tile of a
// short contraction counting for less (bf16, even lists, us, Small / Large: 64 lists of 512 rows,
// 1024 -> 2048: 245 / 200; 256 of 1024, 256 -> 256: 88 / 75; 256 of 512, 256 -> 256:
// 32 / 39; 8 of 512, 1024 -> 1024: 18 / 31).  fp32 is bound by its products.
bool large_tiles(const LinArgs& a, int kd, int nd) {
    const int64_t tiles = ((int64_t)a.rows + 255) / 256 * blocks_of(nd, 256);
    return nd > 128 && tiles * (kd < 512 ? kd : 512) >= 512 * 512;
}

// Without tiles (k_linear_few, k_linear_few_back), where a tile would stand alone and its steps
// wait for each other (us, few / Small.  Forward, 16-bit: 1 list of 64 rows, 1024 -> 1024: 6 / 14; 16
// lists of 8: 10 / 17, of 32: 21 / 17; 256 of 4, 128 -> 128: 8.5 / 6.1.  Forward, fp32: 16 of 32, 1024 -> 1024: 37 /
// 78, of 128: 121 / 77; 1 of 1024: 64 / 78.  dx, 16-bit: 16 of 1: 13 / 17, of 4: 23 / 17; 3 of 1, 25 -> 1557: 18 / 29.
// dx, fp32: 16 of 8: 29 / 80; 64 of 16, 512 -> 512: 56 / 43; 4 of 100, 77 -> 2000: 28 / 166; 256 of 4,
// 128 -> 128: 20 / 14).
template <typename T, bool BACK> bool few_rows(const LinArgs& a) {
    const int64_t k = a.K;
    if (!BACK) return sizeof(T) == 2 ? a.rows <= 4 * k || a.rows <= 128 : a.rows <= 32 * k || a.rows <= 512;
    if (sizeof(T) == 2) return a.rows <= k && a.d_out >= 512;
    return a.rows <= 512 || (a.rows <= 4 * k && a.d_out >= 512);
}

template <typename T> bool narrow_rows(int width) { return width * (int)sizeof(T) < 16; }

template <typename T, bool VIN, bool VOUT, bool BACK> gmm_status launch_linear(const LinArgs& a, hipStream_t stream) {
    const bool narrow = narrow_rows<T>(a.d_in) || (BACK && narrow_rows<T>(a.d_out));   // among the operands
    if (few_rows<T, BACK>(a)) {
        if constexpr (BACK) return launch_few_back<T, VIN>(a, stream);
        if constexpr (!BACK && !VIN)
            if (narrow) return launch_few<T, VIN, VOUT, true>(a, stream);
        if constexpr (!BACK) return launch_few<T, VIN, VOUT>(a, stream);
    }
    if constexpr (!VIN || (BACK && !VOUT))
        if (narrow) return launch_shape<T, VIN, VOUT, BACK, Narrow>(a, stream);
    if constexpr (VIN && VOUT && sizeof(T) == 2)
        if (large_tiles(a, BACK ? a.d_out : a.d_in, BACK ? a.d_in : a.d_out))
            return launch_shape<T, VIN, VOUT, BACK, Large>(a, stream);
    return launch_shape<T, VIN, VOUT, BACK, Small>(a, stream);
}

template <bool BACK, typename T> gmm_status linear_of(const LinArgs& a, bool vin, bool vout, hipStream_t stream) {
    if (vin) return vout ? launch_linear<T, true, true, BACK>(a, stream) : launch_linear<T, true, false, BACK>(a, stream);
    return vout ? launch_linear<T, false, true, BACK>(a, stream) : launch_linear<T, false, false, BACK>(a, stream);
}

template <bool BACK> gmm_status run_linear(const LinArgs& a, int dtype, bool vin, bool vout, hipStream_t stream) {
    switch (dtype) {
        case GMM_F32: return linear_of<BACK, float>(a, vin, vout, stream);
        case GMM_BF16: return linear_of<BACK, bf16_t>(a, vin, vout, stream);
        default: return linear_of<BACK, _Float16>(a, vin, vout, stream);
    }
}

template <typename T, bool VIN, bool VOUT, typename S> gmm_status launch_dw_shape(const GradArgs& a, hipStream_t stream) {
    GradArgs b = a;
    int grid;
    b.row_blocks = (int)row_blocks(a.rows, a.K, a.chunk, &b.by_slot);
    b.in_blocks = blocks_of(a.d_in, S::kM), b.out_blocks = blocks_of(a.d_out, S::kN);
    b.in_step = step_of(a.d_in, S::kM), b.out_step = step_of(a.d_out, S::kN);
    const int64_t per = (int64_t)b.in_blocks * b.out_blocks;
    const gmm_status st = grid_of(b.row_blocks * (per < 8 ? per : (per + 7) / 8 * 8), &grid);
    if (st != GMM_OK) return st;
    hipLaunchKernelGGL((k_linear_dw<T, VIN, VOUT, S>), dim3(grid), dim3(S::kThreads), 0, stream, b);
    return launched();
}

// 256 x 256 tiles of the weights' gradient where lists average 512 rows and the
// tiles fill the compute units (bf16, us, Small / LargeGrad: 64 lists of 512, 1024 x 2048: 298 / 255; 8 of 4096:
// 205 / 154; 64 of 256, 512 x 512: 37 / 41; 256 of 2048, 128 x 256: 175 / 187).
bool large_grad(const GradArgs& a) {
    const int64_t tiles = (int64_t)blocks_of(a.d_in, 256) * blocks_of(a.d_out, 256);
    return a.d_in >= 256 && a.d_out >= 256 && a.rows >= 512 * (int64_t)a.K && (a.rows / a.chunk + a.K) * tiles >= 256;
}

// Large tiles exist for whole 16-bit rows.
template <typename T, bool VEC> struct GradShape {
    using L = typename std::conditional<VEC && sizeof(T) == 2, LargeGrad, Small>::type;
};

template <typename T, bool VIN, bool VOUT> gmm_status launch_dw(const GradArgs& a, hipStream_t stream) {
    gmm_status st;
    using N = typename std::conditional<VIN && VOUT, Small, Narrow>::type;
    if (VIN && VOUT && sizeof(T) == 2 && large_grad(a)) st = launch_dw_shape<T, VIN, VOUT, typename GradShape<T, VIN && VOUT>::L>(a, stream);
    else if (narrow_rows<T>(a.d_in) || narrow_rows<T>(a.d_out)) st = launch_dw_shape<T, VIN, VOUT, N>(a, stream);
    else st = launch_dw_shape<T, VIN, VOUT, Small>(a, stream);
    if (st != GMM_OK) return st;
    const int64_t wide = (int64_t)a.d_out * a.d_in;
    const int64_t parts = (wide + a.d_out + 255) / 256;
    hipLaunchKernelGGL(k_linear_dw_join, dim3(parts < 256 ? parts : 256, a.K), dim3(256), 0, stream, a);
    return launched();
}

template <typename T> gmm_status dw_of(const GradArgs& a, bool vin, bool vout, hipStream_t stream) {
    if (vin) return vout ? launch_dw<T, true, true>(a, stream) : launch_dw<T, true, false>(a, stream);
    return vout ? launch_dw<T, false, true>(a, stream) : launch_dw<T, false, false>(a, stream);
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
    LinArgs a = {routes->offsets, routes->entry, (int)(routes->n * routes->m), routes->k, magic_of(routes->m), false,
                 desc->sorted_rows == 0, x, desc->ldx, w, (int)desc->d_in, (int)desc->d_out, bias, y, desc->ldy, 0, 0, 0};
    const int es = elem_size(desc->dtype);
    const bool vin = desc->d_in * es % 16 == 0 && desc->ldx * es % 16 == 0 && aligned16(x) && aligned16(w);
    const bool vout = desc->d_out * es % 16 == 0 && desc->ldy * es % 16 == 0 && aligned16(y);
    return run_linear<false>(a, desc->dtype, vin, vout, stream);
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
    const bool whole_in = desc->d_in * es % 16 == 0;
    const bool vout = desc->d_out * es % 16 == 0 && desc->ldy * es % 16 == 0 && aligned16(dy);
    if (dx != nullptr && rows > 0) {
        LinArgs a = {routes->offsets, routes->entry, (int)rows, routes->k, magic_of(routes->m), false, false, dy,
                     desc->ldy, w, (int)desc->d_in, (int)desc->d_out, nullptr, dx, desc->lddx, 0, 0, 0};
        const bool vin = whole_in && aligned16(w) && desc->lddx * es % 16 == 0 && aligned16(dx);
        if ((st = run_linear<true>(a, desc->dtype, vin, vout, stream)) != GMM_OK) return st;
    }
    if (dw == nullptr) return GMM_OK;
    if (rows == 0) {   // every list is empty
        const int64_t per = (int64_t)routes->k * desc->d_out;
        hipLaunchKernelGGL(k_zero, dim3(1024), dim3(256), 0, stream, dw, per * desc->d_in);
        if (db != nullptr) hipLaunchKernelGGL(k_zero, dim3(64), dim3(256), 0, stream, db, per);
        return launched();
    }
    GradArgs g = {routes->offsets, routes->entry, (int)rows, routes->k, magic_of(routes->m), false,
                  desc->sorted_rows == 0, chunk_rows(rows, desc), x, desc->ldx, dy, desc->ldy, (int)desc->d_in,
                  (int)desc->d_out, dw, db, (float*)ws, 0, 0, 0, 0, 0};
    const bool vin = whole_in && desc->ldx * es % 16 == 0 && aligned16(x);
    switch (desc->dtype) {
        case GMM_F32: return dw_of<float>(g, vin, vout, stream);
        case GMM_BF16: return dw_of<bf16_t>(g, vin, vout, stream);
        default: return dw_of<_Float16>(g, vin, vout, stream);
    }
}

}  // extern "C"
