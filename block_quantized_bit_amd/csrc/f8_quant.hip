// e4m3 quantizers: activations per 1 x 128 block (rows), per 128 x 1 block
// (columns, written transposed), weights per 128 x 128 block, and the
// transposition of weight codes. They read their input once and write one byte
// per value, which is all that they have to do: 4096 x 4096 values take 11 us in
// bfloat16 and 18 in float32 at the rate of a large copy (4.8 TB/s).
//   rows     15 and 16 us (in a cache); between two products that leave the caches
//            dirty 16 us in bfloat16 (two or four blocks a lane group were slower)
//   columns  20 and 19 us: two barriers and a turn through LDS for each 128 x 64
//   weights  26 and 23 us: loads of one value a lane, 64 registers of them held
//            until the block's maximum is known; not tuned, run once a step at most
//   codes' transposition 13 us (7 at the copy's rate), one byte at a time from LDS
// The three operands of both gradients of 1024 x 4096 x 4096 in one launch 13 us.
#include "f8.h"
#include "kernels_wide.h"
#include "wide.h"

namespace q4 {

namespace {

// 8 consecutive values of a row of `left` more. VEC: 16-byte loads (rows that
// start on 16 bytes, a length that is a multiple of 8); else element loads with
// a bound.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* x, long long at, int left, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (left <= 0) return;
    if (VEC) {
        load8_aligned<BF16>(x, at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) v[i] = load_as_float<BF16>(x, at + i);
    }
}

struct Job {
    int M, K, blocks_x;  // blocks_x: workgroups along K (columns)
    const void* x;
    long long stride;
    uint8_t* codes;
    float* scales;
};

// Rows. 16 lanes share a block of 128: 8 consecutive values a lane, so that
// the maximum is one DPP row reduction.
template <bool BF16, bool VEC>
__device__ __forceinline__ void quantize_rows(const Job& j, int group) {
    const unsigned kb = (j.K + 127) / 128;
    const unsigned t = threadIdx.x & 15;
    const unsigned blk = (unsigned)group * 16 + (threadIdx.x >> 4);  // (row, block), the block fastest: below 2^28
    const bool live = blk < j.M * kb;
    const int m = live ? (int)(blk / kb) : 0;
    const int b = live ? (int)(blk - m * kb) : 0;
    const int k0 = 128 * b + 8 * (int)t;
    float v[8];
    load8<BF16, VEC>(j.x, m * j.stride + k0, live ? j.K - k0 : 0, v);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = row_max16(amax);
    if (!live) return;
    const float s = amax / F8_TOP;
    const float inv = f8_inverse(s);
    *reinterpret_cast<uint2*>(j.codes + (long long)m * ((long long)kb * 128) + k0) = make_uint2(f8_codes4(v, s, inv), f8_codes4(v + 4, s, inv));
    if (t == 0) j.scales[(long long)b * j.M + m] = s;
}

// Columns. A workgroup takes 128 tokens of 64 channels. Thread (q, e) holds the
// 4 x 8 block of tokens 4 q ... and channels 8 e ...; the 32 threads of a channel
// combine their maxima by lane exchanges and LDS, and each makes one word of
// four tokens' codes for each of its channels, which LDS gathers into the
// channels' rows.
template <bool BF16, bool VEC>
__device__ __forceinline__ void quantize_cols(const Job& j, int group, float (*top)[64], uint32_t (*turn)[33]) {
    const int tid = threadIdx.x, e = tid & 7, q = tid >> 3;  // a wavefront: 8 token quads of all 8 channel groups
    const int bx = group % j.blocks_x, by = group / j.blocks_x;
    const int k0 = bx * 64 + 8 * e, m0 = by * 128 + 4 * q;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        load8<BF16, VEC>(j.x, (long long)(m0 + i) * j.stride + k0, m0 + i < j.M ? j.K - k0 : 0, v[i]);
    float amax[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        amax[c] = fmaxf(fmaxf(fabsf(v[0][c]), fabsf(v[1][c])), fmaxf(fabsf(v[2][c]), fabsf(v[3][c])));
#pragma unroll
        for (int off = 8; off < 64; off <<= 1) amax[c] = fmaxf(amax[c], __shfl_xor(amax[c], off, 64));
    }
    if ((tid & 63) < 8)
#pragma unroll
        for (int c = 0; c < 8; ++c) top[tid >> 6][8 * e + c] = amax[c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int ch = 8 * e + c;
        const float s = fmaxf(fmaxf(top[0][ch], top[1][ch]), fmaxf(top[2][ch], top[3][ch])) / F8_TOP;
        const float col[4] = {v[0][c], v[1][c], v[2][c], v[3][c]};
        turn[ch][q] = f8_codes4(col, s, f8_inverse(s));
        if (q == 0 && k0 + c < j.K) j.scales[(long long)by * j.K + k0 + c] = s;
    }
    __syncthreads();
    // a channel's 128 codes: four threads of 32 bytes
    const int ch = tid >> 2, w0 = 8 * (tid & 3), k = bx * 64 + ch;
    if (k >= j.K) return;
    const int Mp = (j.M + 127) / 128 * 128;
    uint4* out = reinterpret_cast<uint4*>(j.codes + (long long)k * Mp + by * 128 + 4 * w0);
    out[0] = make_uint4(turn[ch][w0], turn[ch][w0 + 1], turn[ch][w0 + 2], turn[ch][w0 + 3]);
    out[1] = make_uint4(turn[ch][w0 + 4], turn[ch][w0 + 5], turn[ch][w0 + 6], turn[ch][w0 + 7]);
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void f8_rows_quant_kernel(Job j) {
    quantize_rows<BF16, VEC>(j, blockIdx.x);
}

// The operands of both gradients in one launch: workgroups of the first job
// (columns), then of the second (columns), then of the third (rows). Jobs
// without workgroups are left out.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void f8_cols_quant_kernel(Job a, int na, Job b, int nb, Job r) {
    __shared__ float top[4][64];
    __shared__ uint32_t turn[64][33];
    const int id = blockIdx.x;
    if (id < na)
        quantize_cols<BF16, VEC>(a, id, top, turn);
    else if (id < na + nb)
        quantize_cols<BF16, VEC>(b, id - na, top, turn);
    else
        quantize_rows<BF16, VEC>(r, id - na - nb);
}

// Weights. One workgroup per 128 x 128 block; thread (r, g) takes columns
// 4 l ... of rows r, r + 8, ...
template <bool BF16>
__global__ __launch_bounds__(256) void f8_weights_quant_kernel(int N, int K, int kb, const void* __restrict__ w,
                                                               uint8_t* __restrict__ wq, float* __restrict__ ws) {
    __shared__ float top[4];
    const int l = threadIdx.x & 31, r0 = threadIdx.x >> 5;
    const int k0 = blockIdx.x * 128 + 4 * l;
    const int n0 = blockIdx.y * 128 + r0;
    float v[16][4];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 8 * i, k = k0 + j;
            v[i][j] = (n < N && k < K) ? load_as_float<BF16>(w, (long long)n * K + k) : 0.0f;
            amax = fmaxf(amax, fabsf(v[i][j]));
        }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = amax;
    __syncthreads();
    const float s = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) / F8_TOP;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int n = n0 + 8 * i;
        if (n < N)
            *reinterpret_cast<uint32_t*>(wq + (long long)n * kb * 128 + k0) =
                f8_pack4(f8_quotient(v[i][0], s), f8_quotient(v[i][1], s), f8_quotient(v[i][2], s),
                         f8_quotient(v[i][3], s));
    }
    if (threadIdx.x == 0) ws[(long long)blockIdx.y * kb + blockIdx.x] = s;
}

// Codes [N][Kp] -> [K][Np], 128 x 128 bytes a workgroup through LDS.
__global__ __launch_bounds__(256) void f8_transpose_kernel(int N, int K, int kb, int nb,
                                                           const uint8_t* __restrict__ wq,
                                                           const float* __restrict__ ws, uint8_t* __restrict__ wqt,
                                                           float* __restrict__ wst) {
    __shared__ uint8_t tile[128][132];
    const int kt = blockIdx.x, nt = blockIdx.y;
    const int l = threadIdx.x & 31, r0 = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = r0 + 8 * i, n = nt * 128 + r;
        const uint32_t p =
            n < N ? *reinterpret_cast<const uint32_t*>(wq + (long long)n * kb * 128 + kt * 128 + 4 * l) : 0u;
        *reinterpret_cast<uint32_t*>(&tile[r][4 * l]) = p;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int c = r0 + 8 * i, k = kt * 128 + c;
        if (k < K) {
            const uint32_t p = (uint32_t)tile[4 * l][c] | ((uint32_t)tile[4 * l + 1][c] << 8) |
                               ((uint32_t)tile[4 * l + 2][c] << 16) | ((uint32_t)tile[4 * l + 3][c] << 24);
            *reinterpret_cast<uint32_t*>(wqt + (long long)k * nb * 128 + nt * 128 + 4 * l) = p;
        }
    }
    if (threadIdx.x == 0) wst[(long long)kt * nb + nt] = ws[(long long)nt * kb + kt];
}

}  // namespace

namespace {

bool vec_ok(const Job& j, int size) {
    return !j.x || (j.K % 8 == 0 && (j.stride * size) % 16 == 0 && ((uintptr_t)j.x & 15) == 0);
}
unsigned rows_grid(const Job& j) { return j.x ? (unsigned)(((long long)j.M * ((j.K + 127) / 128) * 16 + 255) / 256) : 0; }
unsigned cols_grid(Job& j) {
    j.blocks_x = (j.K + 63) / 64;
    return j.x ? (unsigned)((long long)j.blocks_x * ((j.M + 127) / 128)) : 0;
}

hipError_t launch_cols(Job a, Job b, Job r, bool bf16, hipStream_t stream) {
    const int size = bf16 ? 2 : 4;
    const unsigned na = cols_grid(a), nb = cols_grid(b), nr = rows_grid(r);
    const bool vec = vec_ok(a, size) && vec_ok(b, size) && vec_ok(r, size);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(na + nb + nr), dim3(256), 0, stream, a, (int)na, b, (int)nb, r);
    };
    if (bf16)
        vec ? go(f8_cols_quant_kernel<true, true>) : go(f8_cols_quant_kernel<true, false>);
    else
        vec ? go(f8_cols_quant_kernel<false, true>) : go(f8_cols_quant_kernel<false, false>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize_rows(int M, int K, bool bf16, const void* x, long long stride, uint8_t* xq, float* xs,
                                   hipStream_t stream) {
    const Job j = {M, K, 0, x, stride, xq, xs};
    const bool vec = vec_ok(j, bf16 ? 2 : 4);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(rows_grid(j)), dim3(256), 0, stream, j); };
    if (bf16)
        vec ? go(f8_rows_quant_kernel<true, true>) : go(f8_rows_quant_kernel<true, false>);
    else
        vec ? go(f8_rows_quant_kernel<false, true>) : go(f8_rows_quant_kernel<false, false>);
    return hipGetLastError();
}

hipError_t launch_f8_quantize_cols(int M, int K, bool bf16, const void* x, long long stride, uint8_t* xt, float* xts,
                                   hipStream_t stream) {
    return launch_cols({M, K, 0, x, stride, xt, xts}, {}, {}, bf16, stream);
}

hipError_t launch_f8_quantize_backward(int M, int K, int N, bool bf16, const void* dy, long long dy_stride,
                                       const void* x, long long x_stride, uint8_t* dyq, float* dys, uint8_t* dyt,
                                       float* dyts, uint8_t* xt, float* xts, bool need_dx, bool need_dw,
                                       hipStream_t stream) {
    if (!need_dw) return launch_f8_quantize_rows(M, N, bf16, dy, dy_stride, dyq, dys, stream);
    Job r = {};
    if (need_dx) r = {M, N, 0, dy, dy_stride, dyq, dys};
    return launch_cols({M, N, 0, dy, dy_stride, dyt, dyts}, {M, K, 0, x, x_stride, xt, xts}, r, bf16, stream);
}

hipError_t launch_f8_quantize_weights(int N, int K, bool bf16, const void* w, uint8_t* wq, float* ws,
                                      hipStream_t stream) {
    const int kb = (K + 127) / 128;
    const dim3 grid(kb, (N + 127) / 128);
    if (bf16)
        hipLaunchKernelGGL((f8_weights_quant_kernel<true>), grid, dim3(256), 0, stream, N, K, kb, w, wq, ws);
    else
        hipLaunchKernelGGL((f8_weights_quant_kernel<false>), grid, dim3(256), 0, stream, N, K, kb, w, wq, ws);
    return hipGetLastError();
}

hipError_t launch_f8_transpose(int N, int K, const uint8_t* wq, const float* ws, uint8_t* wqt, float* wst,
                               hipStream_t stream) {
    const int kb = (K + 127) / 128, nb = (N + 127) / 128;
    hipLaunchKernelGGL(f8_transpose_kernel, dim3(kb, nb), dim3(256), 0, stream, N, K, kb, nb, wq, ws, wqt, wst);
    return hipGetLastError();
}

}  // namespace q4
