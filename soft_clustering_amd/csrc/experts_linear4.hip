// gmm_linear4 and gmm_quantize4: the components' models in 4 bits, for one
// point or a few.
//
//   out[p, o] = sum_i g_i (sum_j (q_kj - 8) s_k,j/group x[p, j] + b_k),  k = idx[p, i]
//
// Bound by the codes' bytes and the latency of the first ones, so each listed
// component's codes are read once a group of up to 16 points, whatever number
// of them list it.  A workgroup owns 16 outputs of such a group and every
// component it lists; its eight waves split the contraction into pieces of 128
// to 512 columns and, where there are fewer, the components.  A wave holds its
// columns of x in registers and streams the components' codes past them, up to
// eight components in flight: 16 points by 16 outputs on v_mfma_f32_16x16x32,
// whether they list the component or not (the products are free beside the
// bytes).  The codes become 16-bit floats by bit operations, exactly; one
// product chain covers one group of columns, and its fp32 result is scaled,
// weighted with gamma where the point lists the component, and added in fp32.
// The halves of a word of codes are nibbles i and i + 4, so x takes the same
// order.  fp16: 0x6400 | q is 1024 + q, less 1032.  bf16: 0x4300 | q is
// 128 + q, and a second product with -136 takes the offset off.  fp32 rows are
// split into three bf16 parts, which hold all 24 bits, and meet q - 8 in bf16.
//
// Measured: one point in two of 16 models 4096 -> 4096 (bf16, groups of 128)
// 8.4 us, 17 MB of codes; 24 points in four of 64 models 1024 -> 2048 (fp16,
// groups of 64) 32 us.  Lanes that hold different rows of weights load from
// different lines, 64 cycles an instruction; so codes and x come into LDS row
// by row, and the scales are staged there for all components of a phase: with
// loads straight into the operands' registers the batch took 51 us, 20 of them
// for the scales.

#include <type_traits>

#include "experts_internal.h"

namespace gmm {

namespace {

constexpr int kOutputs = 16, kPoints = 16, kWaves = 8, kThreads = 64 * kWaves;
constexpr int kEntries = kPoints * GMM_MAX_TOPM;   // entries of a workgroup

constexpr int kRing = 8192;      // bytes of LDS of a wave
constexpr int kScales = 16384;   // scales of a phase in LDS

// This wave's LDS reads and writes so far are done before its next ones, the asynchronous loads among them.
__device__ __forceinline__ void drain() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

struct Lin4Args {
    int n, m, K, d_in, d_out, groups;
    int points;   // of a workgroup
    const void* x;
    int64_t ldx;
    const int32_t* idx;
    const float* gamma;
    const uint8_t* codes;
    const bf16_t* scales;
    const float* bias;
    void* out;
    int64_t ldo;
};

// Eight values in the order of the codes' words: (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 code_order(const uint4& v) {
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100), __builtin_amdgcn_perm(v.z, v.x, 0x07060302),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100), __builtin_amdgcn_perm(v.w, v.y, 0x07060302));
}

// The constants of the codes' conversion, in registers: v_and_or_b32 takes no two literals.
struct Bits {
    uint32_t low, high, one;   // nibbles 0 and 4 of a word, nibbles 1 and 5, the exponent
};
__device__ __forceinline__ Bits bits_of(uint32_t one) {
    Bits b = {0x000F000Fu, 0x00F000F0u, one};
    asm volatile("" : "+v"(b.low), "+v"(b.high), "+v"(b.one));
    return b;
}
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) { return (v & mask) | bits; }

// q - 8 of a word of codes in fp16: 1024 + q - 1032, and (1024 + 16 q) / 16 - 72, all exact.
__device__ __forceinline__ uint4 codes_f16(uint32_t q, const Bits& b) {
    typedef _Float16 half2v __attribute__((ext_vector_type(2)));
    const half2v less = {(_Float16)-1032.0f, (_Float16)-1032.0f}, less16 = {(_Float16)-72.0f, (_Float16)-72.0f},
                 by16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const half2v lo = __builtin_bit_cast(half2v, and_or(q, b.low, b.one)),
                     hi = __builtin_bit_cast(half2v, and_or(q, b.high, b.one));
        w[2 * i] = __builtin_bit_cast(uint32_t, lo + less);
        w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(hi, by16, less16));
        q >>= 8;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Products of one word of codes with the eight values of x it meets.
template <typename T> struct Codes;
template <> struct Codes<_Float16> {
    static constexpr int kTerms = 1;
    static constexpr uint32_t kOne = 0x64006400u;   // 1024
    __device__ __forceinline__ static void take(const uint4* v, uint4* f) { f[0] = code_order(v[0]); }
    __device__ __forceinline__ static f32x4 mul(const uint4* f, uint32_t q, const Bits& b, f32x4 d) {
        return mma16<_Float16>(f[0], codes_f16(q, b), d);
    }
};
__device__ __forceinline__ uint4 codes_bf16(uint32_t q, const Bits& b) {
    return make_uint4(and_or(q, b.low, b.one), and_or(q >> 4, b.low, b.one), and_or(q >> 8, b.low, b.one),
                      and_or(q >> 12, b.low, b.one));
}
__device__ __forceinline__ f32x4 mul_bf16(const uint4& f, const uint4& w, f32x4 d) {
    const uint32_t off = 0xC308C308u;
    return mma16<bf16_t>(f, make_uint4(off, off, off, off), mma16<bf16_t>(f, w, d));
}
template <> struct Codes<bf16_t> {
    static constexpr int kTerms = 1;
    static constexpr uint32_t kOne = 0x43004300u;   // 128
    __device__ __forceinline__ static void take(const uint4* v, uint4* f) { f[0] = code_order(v[0]); }
    __device__ __forceinline__ static f32x4 mul(const uint4* f, uint32_t q, const Bits& b, f32x4 d) {
        return mul_bf16(f[0], codes_bf16(q, b), d);
    }
};
template <> struct Codes<float> {
    static constexpr int kTerms = 3;
    static constexpr uint32_t kOne = 0x64006400u;
    __device__ __forceinline__ static void take(const uint4* raw, uint4* f) {
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) Vec16<float>::unpack(raw[h], v + 4 * h);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            bf16_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                from_f32(v[i], b + i);
                const float rest = v[i] - to_f32(b[i]);
                v[i] = isfinite(rest) ? rest : 0.0f;   // an infinity or NaN is all in the first part
            }
            f[u] = code_order(__builtin_bit_cast(uint4, b));
        }
    }
    __device__ __forceinline__ static f32x4 mul(const uint4* f, uint32_t q, const Bits& b, f32x4 d) {
        // q - 8 itself in bf16: an offset taken off afterwards would cost fp32 sums four of their bits
        const uint4 h = codes_f16(q, b);
        float v[8];
        Vec16<_Float16>::unpack(h, v);
        const uint4 w = pack16<bf16_t>(v);
        return mma16<bf16_t>(f[0], w, mma16<bf16_t>(f[1], w, mma16<bf16_t>(f[2], w, d)));
    }
};

// A wave's share of LDS: pieces of x, then codes on their way; rows of BYTES bytes whose 16-byte
// places are XORed with the row, so that the 16 rows a fragment read touches lie in
// different banks.  VEC: straight from memory, else through registers.
template <bool VEC, int BYTES> struct Rows {
    static constexpr int kPlaces = BYTES / 16, kPerLoad = BYTES >= 1024 ? 1 : 1024 / BYTES;   // rows of a wave load
    __device__ __forceinline__ static int at(int row, int byte) {
        return row * BYTES + (((byte >> 4) ^ (row & (kPlaces < 16 ? kPlaces - 1 : 15))) << 4) + (byte & 15);
    }
    // rows [r0, r0 + kPerLoad): this lane's row `from`, nullptr: zeros; bytes [c, c + BYTES) of `width`
    __device__ __forceinline__ static void load(char* lds, uint32_t address, int r0, const char* from, int64_t c, int64_t width) {
        const int lane = threadIdx.x & 63, r = r0 + lane / kPlaces;
        const int64_t b = c + (((lane % kPlaces) ^ (r & (kPlaces < 16 ? kPlaces - 1 : 15))) << 4);
        if constexpr (VEC) {
            fetch_piece(from != nullptr && b < width ? from + b : (const char*)&zero_piece, address + r0 * BYTES);
        } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (from != nullptr && width >= 16) {
                v = settle(load_loose<1>(from, true, b, width, (const char*)&zero_piece));
            } else if (from != nullptr) {
                uint8_t t[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) t[i] = b + i < width ? from[b + i] : 0;
                v = __builtin_bit_cast(uint4, t);
            }
            *(uint4*)(lds + r0 * BYTES + lane * 16) = v;
        }
    }
};

// PIECE: columns of a wave's piece of the contraction.
template <typename T, bool VEC, int GROUP, int PIECE>
__global__ __launch_bounds__(kThreads, 2) void k_linear4(const Lin4Args a) {
    using C = Codes<T>;
    using XRows = Rows<VEC, PIECE * (int)sizeof(T)>;
    using QRows = Rows<VEC, PIECE / 2>;
    constexpr int GC = PIECE / GROUP, WORDS = GROUP / 32;   // groups of a piece; words of a lane and group
    constexpr int kUnit = kOutputs * PIECE / 2;             // bytes of a component's codes
    constexpr int kAhead = kRing / kUnit;                   // components in LDS or on their way
    constexpr int kLoads = kUnit / 1024;                    // wave loads of a component
    constexpr int kXRows = kRing / (PIECE * (int)sizeof(T)) < kPoints ? kRing / (PIECE * (int)sizeof(T)) : kPoints;
    __shared__ __align__(16) char ring[kWaves][kRing];
    __shared__ __align__(32) bf16_t scale[kScales];              // [component of the phase][output][padded groups]
    __shared__ __align__(16) int key[kEntries];                  // components of the entries
    __shared__ int place[kEntries], unit[kEntries];              // of a leader; the components in order of appearance
    __shared__ __align__(16) float weight[kEntries][kPoints];    // per component: the points' gamma
    __shared__ uint32_t listing[kEntries];                       // and the points that list it
    __shared__ float part[kWaves][kPoints][kOutputs];
    __shared__ int starts_of[kEntries / 64];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int p0 = blockIdx.y * a.points, n = min(a.points, a.n - p0), entries = n * a.m;
    const int32_t* idx = a.idx + p0 * a.m;
    const float* gamma = a.gamma + p0 * a.m;

    // ---- the components these points list: a component's first entry leads it
    int k_mine = -1;
    float g_mine = 0.0f;
    if (t < kEntries) {
        if (t < entries) {
            const int k = idx[t];
            g_mine = gamma[t];
            k_mine = (unsigned)k < (unsigned)a.K ? k : -1;
        }
        key[t] = k_mine;
        listing[t] = 0;
    }
    for (int i = t; i < entries * kPoints; i += kThreads) (&weight[0][0])[i] = 0.0f;
    __syncthreads();
    int lead = t;
    if (t < kEntries && k_mine >= 0)
        for (int e = t & ~3; e >= 0; e -= 4) {
            const int4 k4 = *(const int4*)(key + e);
            lead = k4.w == k_mine ? min(lead, e + 3) : lead;
            lead = k4.z == k_mine ? min(lead, e + 2) : lead;
            lead = k4.y == k_mine ? min(lead, e + 1) : lead;
            lead = k4.x == k_mine ? min(lead, e) : lead;
        }
    const bool leads = t < kEntries && k_mine >= 0 && lead == t;
    const uint64_t starts = __ballot(leads);
    if (t < kEntries && lane == 0) starts_of[wave] = __popcll(starts);
    __syncthreads();
    int units = 0, before = 0;
    for (int w = 0; w < kEntries / 64; ++w) {
        if (w < wave) before += starts_of[w];
        units += starts_of[w];
    }
    if (leads) {
        place[t] = before + __popcll(starts & ((1ull << lane) - 1));
        unit[place[t]] = k_mine;
    }
    __syncthreads();
    if (t < kEntries && k_mine >= 0) {
        const int u = place[lead], p = t / a.m, i = t - p * a.m;
        bool first = true;   // of its point's columns with this component
        for (int j = 0; j < i; ++j) first = first && key[p * a.m + j] != k_mine;
        if (first) {
            float g = g_mine;
            for (int j = i + 1; j < a.m; ++j)
                if (key[p * a.m + j] == k_mine) g += gamma[p * a.m + j];
            weight[u][p] = g;
            atomicOr(&listing[u], 1u << p);
        }
    }

    // ---- products, in phases of as many components as have their scales in LDS
    const int o0 = blockIdx.x * kOutputs, quarter_c = lane >> 4;
    const int pieces = (a.d_in + PIECE - 1) / PIECE;
    int split = 1;   // waves on one piece, each on every split-th component
    while (2 * split * pieces <= kWaves) split *= 2;
    const int64_t bytes = (a.d_in + 1) / 2;
    const int padded = (a.groups + GC - 1) / GC * GC, per_unit = kOutputs * padded;
    const bool scales_fit = per_unit <= kScales;   // else (very wide rows) they are read from memory
    const int phase = scales_fit ? kScales / per_unit : kEntries;
    const Bits bits = bits_of(C::kOne);
    char* mine = ring[wave];
    const uint32_t mine_at = lds_address(mine);
    float out[4] = {};
    for (int v0 = 0; v0 < units; v0 += phase) {
        const int v1 = min(v0 + phase, units);
        if (scales_fit) {
            __syncthreads();   // every wave is through with the last phase's
            for (int i = t; i < (v1 - v0) * per_unit; i += kThreads) {
                const int u = i / per_unit, r = i % per_unit / padded, g = i % padded;
                const int64_t from = (int64_t)unit[v0 + u] * a.d_out + min(o0 + r, a.d_out - 1);
                scale[i] = a.scales[from * a.groups + min(g, a.groups - 1)];
            }
        }
        __syncthreads();
        for (int item = wave; item < pieces * split; item += kWaves) {
            const int piece = item / split, first = v0 + item % split;
            if (first >= v1) continue;
            // x: the points' rows of the piece through the ring into fragments; zeros for no point
            uint4 f[GC][WORDS][C::kTerms];
#pragma unroll
            for (int g = 0; g < GC; ++g)
#pragma unroll
                for (int w = 0; w < WORDS; ++w)
#pragma unroll
                    for (int z = 0; z < C::kTerms; ++z) f[g][w][z] = make_uint4(0, 0, 0, 0);
            for (int q0 = 0; q0 < n; q0 += kXRows) {
                drain();   // the last reads of the ring, before it is written again
#pragma unroll
                for (int r = 0; r < kXRows; r += XRows::kPerLoad) {
                    const int p = q0 + r + lane / XRows::kPlaces;
                    if (q0 + r < n)
                        XRows::load(mine, mine_at, r, p < n ? (const char*)((const T*)a.x + (int64_t)(p0 + p) * a.ldx) : nullptr,
                                    (int64_t)piece * PIECE * (int)sizeof(T), (int64_t)a.d_in * (int)sizeof(T));
                }
                wait_pieces<0>();
                drain();
                const int r = (lane & 15) - q0;
                if (r >= 0 && r < kXRows && q0 + r < n) {
#pragma unroll
                    for (int g = 0; g < GC; ++g)
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) {
                            constexpr int LOADS = 8 / Vec16<T>::kElems;
                            uint4 raw[LOADS];
#pragma unroll
                            for (int h = 0; h < LOADS; ++h) {
                                const int c = g * GROUP + quarter_c * (GROUP / 4) + 8 * w + h * Vec16<T>::kElems;
                                raw[h] = *(const uint4*)(mine + XRows::at(r, c * (int)sizeof(T)));
                            }
                            C::take(raw, f[g][w]);
                        }
                }
            }
            drain();
            auto fetch = [&](int u, int slot) {   // component u's codes; past the last one, that one again
                const int64_t from = (int64_t)__builtin_amdgcn_readfirstlane(unit[min(u, v1 - 1)]) * a.d_out + o0;
#pragma unroll
                for (int l = 0; l < kLoads; ++l) {
                    const int r = l * QRows::kPerLoad + lane / QRows::kPlaces;
                    QRows::load(mine + slot * kUnit, mine_at + slot * kUnit, l * QRows::kPerLoad,
                                (const char*)a.codes + (from + min(r, a.d_out - 1 - o0)) * bytes, (int64_t)piece * PIECE / 2, bytes);
                }
            };
#pragma unroll
            for (int h = 0; h < kAhead - 1; ++h) fetch(first + h * split, h);
            int slot = 0;
            for (int u = first; u < v1; u += split) {
                // the slot read in the last turn takes the component kAhead - 1 turns ahead
                fetch(u + (kAhead - 1) * split, slot == 0 ? kAhead - 1 : slot - 1);
                wait_pieces<(kAhead - 1) * kLoads>();
                const float4 g4 = *(const float4*)&weight[u][4 * quarter_c];
                const uint32_t on = listing[u];
                const float gw[4] = {g4.x, g4.y, g4.z, g4.w};
                bf16_t s[GC];
                const int gp = piece * GC;
                if (scales_fit) {
                    __builtin_memcpy(s, __builtin_assume_aligned(&scale[(u - v0) * per_unit + (lane & 15) * padded + gp], 2 * GC), 2 * GC);
                } else {
                    const int64_t from = (int64_t)unit[u] * a.d_out + min(o0 + (lane & 15), a.d_out - 1);
#pragma unroll
                    for (int g = 0; g < GC; ++g) s[g] = a.scales[from * a.groups + min(gp + g, a.groups - 1)];
                }
                const char* codes = mine + slot * kUnit;
                f32x4 y = {};
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    uint32_t q[WORDS];
                    __builtin_memcpy(q, __builtin_assume_aligned(codes + QRows::at(lane & 15, g * GROUP / 2 + quarter_c * 4 * WORDS), 4 * WORDS),
                                     4 * WORDS);
                    f32x4 d = {};
#pragma unroll
                    for (int w = 0; w < WORDS; ++w) d = C::mul(f[g][w], q[w], bits, d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = fmaf(to_f32(s[g]), d[i], y[i]);
                }
                // lane: output lane % 16, points 4 (lane / 16) + i.  The bits of y taken away where the point
                // does not list the component, not a product with 0: y may be NaN
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t keep = (uint32_t)((int32_t)(on << (31 - 4 * quarter_c - i)) >> 31);
                    out[i] = fmaf(gw[i], __uint_as_float(__float_as_uint(y[i]) & keep), out[i]);
                }
                drain();
                slot = slot + 1 < kAhead ? slot + 1 : 0;
            }
            wait_pieces<0>();   // the codes fetched past the last component
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][4 * quarter_c + i][lane & 15] = out[i];
    __syncthreads();
    for (int i = t; i < n * kOutputs; i += kThreads) {
        const int p = i / kOutputs, c = i % kOutputs;
        if (o0 + c >= a.d_out) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][p][c];
        if (a.bias != nullptr)
            for (int e = p * a.m; e < (p + 1) * a.m; ++e)
                if (key[e] >= 0) v = fmaf(gamma[e], a.bias[(int64_t)key[e] * a.d_out + o0 + c], v);
        from_f32(v, (T*)a.out + (int64_t)(p0 + p) * a.ldo + o0 + c);
    }
}

// One wave a group: its scale, its codes two columns a lane.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize4(const T* __restrict__ w, int64_t rows, int d_in, int group,
                                                   int groups, uint8_t* __restrict__ codes,
                                                   bf16_t* __restrict__ scales) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t g = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); g < rows * groups; g += waves) {
        const int64_t row = g / groups;
        const int c0 = (int)(g % groups) * group, c1 = min(c0 + group, d_in);
        const T* r = w + row * d_in;
        const int c = c0 + 2 * lane;
        float v[2] = {c < c1 ? to_f32(r[c]) : 0.0f, c + 1 < c1 ? to_f32(r[c + 1]) : 0.0f};
        float top = fmaxf(fabsf(v[0]), fabsf(v[1]));
        const bool finite = __ballot(!(isfinite(v[0]) && isfinite(v[1]))) == 0;
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        bf16_t s;
        from_f32(finite ? __fdiv_rn(top, 7.0f) : __builtin_nanf(""), &s);
        const float scale = to_f32(s);
        uint32_t q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float f = finite && scale != 0.0f ? rintf(__fdiv_rn(v[e], scale)) : 0.0f;
            f = fminf(fmaxf(f, -8.0f), 7.0f);
            q[e] = (uint32_t)((int)f + 8);
        }
        if (c < c1) codes[row * ((d_in + 1) / 2) + (c >> 1)] = (uint8_t)(q[0] | q[1] << 4);
        if (lane == 0) scales[g] = s;
    }
}

bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

template <typename T, bool VEC> gmm_status launch_linear4(const Lin4Args& a, int group, hipStream_t stream) {
    Lin4Args b = a;
    const int tiles = (a.d_out + kOutputs - 1) / kOutputs;
    // fewer points a workgroup where that takes more workgroups to fill the compute units
    b.points = kPoints;
    while (b.points > 4 && (int64_t)tiles * ((a.n + b.points - 1) / b.points) < 256) b.points /= 2;
    const dim3 grid(tiles, (a.n + b.points - 1) / b.points);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, b); };
    auto by_group = [&](auto piece) {
        constexpr int P = decltype(piece)::value;
        if (group == 32) go(k_linear4<T, VEC, 32, P>);
        else if (group == 64) go(k_linear4<T, VEC, 64, P>);
        else go(k_linear4<T, VEC, 128, P>);
    };
    // the widest pieces that still give every wave a piece of some component (us at 512 / 256 / 128 columns:
    // one point, two models 4096 -> 4096: 8.4 / 9.7 / 12.4; 24 points, 1024 -> 2048: 33 / 32 / 38): each costs a component's
    // bookkeeping once (fp32's three parts of x fill the registers at 256)
    const int listed = (a.n < b.points ? a.n : b.points) * a.m;
    auto fills = [&](int piece) { return (int64_t)((a.d_in + piece - 1) / piece) * listed >= kWaves; };
    if constexpr (sizeof(T) == 2) {
        if (fills(512)) {
            by_group(std::integral_constant<int, 512>());
            return launched();
        }
    }
    if (fills(256)) {
        by_group(std::integral_constant<int, 256>());
        return launched();
    }
    by_group(std::integral_constant<int, 128>());
    return launched();
}

template <typename T>
gmm_status launch_quantize4(const void* w, int64_t rows, int d_in, int group, uint8_t* codes, void* scales,
                            hipStream_t stream) {
    const int groups = (d_in + group - 1) / group;
    const int64_t blocks = (rows * groups + 3) / 4;
    hipLaunchKernelGGL(k_quantize4<T>, dim3(blocks < 65536 ? blocks : 65536), dim3(256), 0, stream, (const T*)w, rows,
                       d_in, group, groups, codes, (bf16_t*)scales);
    return launched();
}

}  // namespace

}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_quantize4(int64_t rows, int64_t d_in, int32_t group, int32_t dtype, const void* w, uint8_t* codes,
                         void* scales, hipStream_t stream) {
    const gmm_status st = check_width(d_in, dtype);
    if (st != GMM_OK) return st;
    if (rows < 0 || rows > ((int64_t)1 << 32) || !group_ok(group)) return GMM_E_ARG;
    if (rows == 0) return GMM_OK;
    if (w == nullptr || codes == nullptr || scales == nullptr) return GMM_E_ARG;
    switch (dtype) {
        case GMM_F32: return launch_quantize4<float>(w, rows, (int)d_in, group, codes, scales, stream);
        case GMM_BF16: return launch_quantize4<bf16_t>(w, rows, (int)d_in, group, codes, scales, stream);
        default: return launch_quantize4<_Float16>(w, rows, (int)d_in, group, codes, scales, stream);
    }
}

gmm_status gmm_linear4(int64_t n, int32_t m, int32_t k, int64_t d_in, int64_t d_out, int32_t group, int32_t dtype,
                       const void* x, int64_t ldx, const int32_t* idx, const float* gamma, const uint8_t* codes,
                       const void* scales, const float* bias, void* out, int64_t ldo, hipStream_t stream) {
    gmm_status st = check_shape(n, m, k);
    if (st == GMM_OK) st = check_width(d_in, dtype);
    if (st == GMM_OK) st = check_width(d_out, dtype);
    if (st == GMM_OK) st = check_stride(ldx, d_in);
    if (st == GMM_OK) st = check_stride(ldo, d_out);
    if (st != GMM_OK) return st;
    if (n > GMM_LINEAR4_MAX_N || !group_ok(group)) return GMM_E_ARG;
    if (n == 0) return GMM_OK;
    if (x == nullptr || idx == nullptr || gamma == nullptr || codes == nullptr || scales == nullptr || out == nullptr)
        return GMM_E_ARG;
    const int es = elem_size(dtype);
    const bool vec = d_in % 32 == 0 && aligned16(x) && ldx * es % 16 == 0 && aligned16(codes);
    Lin4Args a = {(int)n, m, k, (int)d_in, (int)d_out, (int)((d_in + group - 1) / group), 0, x, ldx, idx, gamma,
                  codes, (const bf16_t*)scales, bias, out, ldo};
    switch (dtype) {
        case GMM_F32: return vec ? launch_linear4<float, true>(a, group, stream) : launch_linear4<float, false>(a, group, stream);
        case GMM_BF16: return vec ? launch_linear4<bf16_t, true>(a, group, stream) : launch_linear4<bf16_t, false>(a, group, stream);
        default: return vec ? launch_linear4<_Float16, true>(a, group, stream) : launch_linear4<_Float16, false>(a, group, stream);
    }
}

}  // extern "C"
