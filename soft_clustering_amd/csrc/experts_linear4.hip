// gmm_linear4 and gmm_quantize4: the components' models in 4 bits, for one
// point or a few.
//
//   out[p, o] = sum_i g_i (sum_j (q_kj - 8) s_k,j/group x[p, j] + b_k),  k = idx[p, i]
//
// A wave owns one output o of one point and walks the point's components: 16
// bytes of codes (32 columns, one scale) a lane and step, fp32 sums.

#include "experts_internal.h"

namespace gmm {

namespace {

struct Lin4Args {
    int n, m, K, d_in, d_out, group, groups;
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

__device__ __forceinline__ float wave_sum(float v) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_linear4(const Lin4Args a) {
    constexpr int E = Vec16<T>::kElems;
    const int lane = threadIdx.x & 63;
    const int o = blockIdx.x * 4 + (threadIdx.x >> 6), p = blockIdx.y;
    if (o >= a.d_out) return;
    const T* x = (const T*)a.x + (int64_t)p * a.ldx;
    float out = 0.0f;
    for (int i = 0; i < a.m; ++i) {
        const int k = a.idx[p * a.m + i];
        if ((unsigned)k >= (unsigned)a.K) continue;
        const int64_t row = (int64_t)k * a.d_out + o;
        const uint8_t* codes = a.codes + row * ((a.d_in + 1) / 2);
        const bf16_t* scales = a.scales + row * a.groups;
        float sum = 0.0f;
        if constexpr (VEC) {
            for (int c = lane; c < a.d_in / 32; c += 64) {
                const uint4 q4 = ((const uint4*)codes)[c];
                const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
                float dot = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float v[8];
#pragma unroll
                    for (int h = 0; h < 8 / E; ++h) Vec16<T>::unpack(((const uint4*)(x + 32 * c + 8 * u))[h], v + h * E);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = fmaf((float)((int)(q[u] >> (4 * j) & 15) - 8), v[j], dot);
                }
                sum = fmaf(to_f32(scales[32 * c / a.group]), dot, sum);
            }
        } else {
            for (int j = lane; j < a.d_in; j += 64) {
                const int q = (codes[j >> 1] >> (4 * (j & 1)) & 15) - 8;
                sum = fmaf(to_f32(scales[j / a.group]) * (float)q, to_f32(x[j]), sum);
            }
        }
        sum = wave_sum(sum);
        if (a.bias != nullptr) sum += a.bias[row];
        out = fmaf(a.gamma[p * a.m + i], sum, out);
    }
    if (lane == 0) from_f32(out, (T*)a.out + (int64_t)p * a.ldo + o);
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

template <typename T> gmm_status launch_linear4(const Lin4Args& a, bool vec, hipStream_t stream) {
    const dim3 grid((a.d_out + 3) / 4, a.n);
    if (vec) hipLaunchKernelGGL((k_linear4<T, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_linear4<T, false>), grid, dim3(256), 0, stream, a);
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
    const bool vec = d_in % 32 == 0 && aligned16(codes) && aligned16(x) && ldx * es % 16 == 0;
    Lin4Args a = {(int)n, m, k, (int)d_in, (int)d_out, group, (int)((d_in + group - 1) / group), x, ldx, idx, gamma,
                  codes, (const bf16_t*)scales, bias, out, ldo};
    switch (dtype) {
        case GMM_F32: return launch_linear4<float>(a, vec, stream);
        case GMM_BF16: return launch_linear4<bf16_t>(a, vec, stream);
        default: return launch_linear4<_Float16>(a, vec, stream);
    }
}

}  // extern "C"
