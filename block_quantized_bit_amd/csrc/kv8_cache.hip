// Storing into and reading from the 8-bit paged key/value cache (kv8.h).
// One workgroup handles one page of one head of K or of V: it alone reads and
// writes that page's codes and scale, so a scale that grows and the old codes'
// rounding under the new one need no atomics. Prompts of 13 000 tokens, 8 heads of
// 128: 16 us to read back (4.9 TB/s, bound by memory), 33 us to store (54 MB read,
// twice, the second time from a cache, 27 MB written; 17 us at a copy's rate). What
// the storing waits for is not found: the second reading it is not, since keeping
// the rows in registers took 32.6 us. 64 single tokens 5 us: the launch and loads
// that depend on each other.
#include <type_traits>

#include "kernels_wide.h"
#include "kv8_dev.h"

namespace q4 {

namespace {

__device__ __forceinline__ float tame(float v) {
    return v != v ? 0.0f : fminf(fmaxf(v, -3.402823466e38f), 3.402823466e38f);
}

template <int FMT>
__device__ __forceinline__ float kv_top() { return FMT == KV8_INT8 ? 127.0f : 448.0f; }

// Four codes of four quotients.
template <int FMT>
__device__ __forceinline__ uint32_t kv_round4(float a, float b, float c, float d) {
    constexpr float t = FMT == KV8_INT8 ? 127.0f : 448.0f;
    a = fminf(fmaxf(a, -t), t);
    b = fminf(fmaxf(b, -t), t);
    c = fminf(fmaxf(c, -t), t);
    d = fminf(fmaxf(d, -t), t);
    if (FMT == KV8_E4M3) return f8_pack4(a, b, c, d);
    return ((uint32_t)(int)rintf(a) & 0xFFu) | (((uint32_t)(int)rintf(b) & 0xFFu) << 8) |
           (((uint32_t)(int)rintf(c) & 0xFFu) << 16) | ((uint32_t)(int)rintf(d) << 24);
}

template <int FMT>
__device__ __forceinline__ void kv_values4(uint32_t w, float (&v)[4]) {
    if (FMT == KV8_INT8) {
        v[0] = (float)(int)(int8_t)(w & 0xFFu);
        v[1] = (float)(int)(int8_t)((w >> 8) & 0xFFu);
        v[2] = (float)(int)(int8_t)((w >> 16) & 0xFFu);
        v[3] = (float)((int)w >> 24);
    } else {
        const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
        v[0] = (float)a[0];
        v[1] = (float)a[1];
        v[2] = (float)b[0];
        v[3] = (float)b[1];
    }
}

// Bytes of `fresh` where the mask has ones, of `old` elsewhere.
__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t fresh, uint32_t old) {
    return (fresh & mask) | (old & ~mask);
}
// Mask of the bytes j = 0..3 with lo <= first + j < hi.
__device__ __forceinline__ uint32_t byte_range(int first, int lo, int hi) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (first + j >= lo && first + j < hi) m |= 0xFFu << (8 * j);
    return m;
}

// Eight consecutive values, by 16-byte loads where rows allow it.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* p, long long at, float (&v)[8]) {
    if (VEC) {
        load8_aligned<BF16>(p, at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = load_as_float<BF16>(p, at + i);
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* out, long long at, const float (&v)[8]) {
    if (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Tokens lie along d in the packed rows and in a K page, and along the slots in
// a V page. A thread takes 8 values of one token (K), or the 4 x 8 block of four
// slots and eight d (V), whose eight words of four codes it turns in registers;
// consecutive threads take consecutive slots of a d's row.
template <int FMT, bool BF16, bool VEC>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8 c, int total, int max_new,
                                                         const void* __restrict__ k_new, long long k_stride,
                                                         const void* __restrict__ v_new, long long v_stride) {
    __shared__ float part[4];
    const int h = blockIdx.y;
    const int b = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const Kv8Span s = kv8_span(c, b, total, max_new);
    // positions of this workgroup's page that get tokens
    const int first = max(s.begin, 0);
    const int p = first / c.P + (int)blockIdx.x;
    if (p >= c.max_pages) return;
    const int lo = max(first, p * c.P), hi = min(s.end, p * c.P + c.P);
    if (lo >= hi) return;
    const int pg = c.table[(long long)b * c.max_pages + p];
    if (pg < 0 || pg >= c.pages) return;

    const int tid = threadIdx.x;
    const int D = c.D, n = hi - lo, d8 = D >> 3;
    const void* src = is_v ? v_new : k_new;
    const long long stride = is_v ? v_stride : k_stride;
    const long long at0 = (long long)(s.row0 + lo - s.begin) * stride + (long long)h * D;

    float amax = 0.0f;
    for (int t = tid; t < n * d8; t += 256) {
        const int i = t / d8, d = 8 * (t - i * d8);
        float v[8];
        load8<BF16, VEC>(src, at0 + i * stride + d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(tame(v[j])));
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    float* scale = (is_v ? c.v_scale : c.k_scale) + (long long)pg * c.H + h;
    const bool holds = lo > p * c.P;
    const float s_old = holds ? *scale : 0.0f;
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float s_mine = amax / kv_top<FMT>();
    const float s_new = s_mine > s_old ? s_mine : s_old;
    const bool grew = holds && s_new > s_old && s_old > 0.0f;
    const float ratio = s_old / s_new;  // used where grew
    if (tid == 0) *scale = s_new;

    const int lo_s = lo - p * c.P, hi_s = hi - p * c.P;  // slots
    // codes of four values: the float32 quotients by s_new, rounded (divisions only near a tie)
    const float inv = FMT == KV8_E4M3 ? f8_inverse(s_new) : act_inverse(s_new);
    const auto codes4 = [&](float a, float b, float c, float d) -> uint32_t {
        if (s_new == 0.0f) return 0u;
        const float v[4] = {tame(a), tame(b), tame(c), tame(d)};
        if (FMT == KV8_E4M3) return f8_codes4(v, s_new, inv);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= ((uint32_t)act_code(v[i], s_new, inv) & 0xFFu) << (8 * i);
        return w;
    };
    const auto again = [&](uint32_t w) {
        float v[4];
        kv_values4<FMT>(w, v);
        return kv_round4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
    };
    uint8_t* page = (is_v ? c.v_codes : c.k_codes) + ((long long)pg * c.H + h) * c.P * D;
    if (grew) {
        // the codes the page held, under the new scale: whole rows of K, the first lo_s slots of V's rows
        const int words = is_v ? (lo_s + 3) >> 2 : lo_s * (D >> 2);
        for (int t = tid; t < (is_v ? words * D : words); t += 256) {
            const int row = is_v ? t / words : 0, q = t - row * words;
            uint32_t* cell = reinterpret_cast<uint32_t*>(page + (long long)row * c.P) + q;
            *cell = is_v ? pick(byte_range(4 * q, 0, lo_s), again(*cell), *cell) : again(*cell);
        }
        __syncthreads();  // the last of those words may get new codes below
    }
    if (n < 8) {
        // a few tokens: a value a thread
        for (int t = tid; t < n * D; t += 256) {
            const int i = t / D, d = t - i * D;
            const uint32_t w = codes4(load_as_float<BF16>(src, at0 + i * stride + d), 0.0f, 0.0f, 0.0f);
            page[is_v ? (long long)d * c.P + lo_s + i : (long long)(lo_s + i) * D + d] = (uint8_t)w;
        }
        return;
    }
    if (!is_v) {
        for (int t = tid; t < n * d8; t += 256) {
            const int i = t / d8, d = 8 * (t - i * d8);
            float v[8];
            load8<BF16, VEC>(src, at0 + i * stride + d, v);
            reinterpret_cast<uint2*>(page)[lo_s * d8 + t] = make_uint2(codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7]));
        }
        return;
    }
    const int q0 = lo_s >> 2, quads = ((hi_s + 3) >> 2) - q0;
    for (int t = tid; t < quads * d8; t += 256) {
        const int e = t / quads, slot = 4 * (q0 + t - e * quads);  // values 8 e ..., slots slot ...
        uint32_t* cell = reinterpret_cast<uint32_t*>(page + (long long)8 * e * c.P + slot);
        const int step = c.P >> 2;  // words between two d
        const uint32_t fresh_part = byte_range(slot, lo_s, hi_s);
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = min(max(slot + i - lo_s, 0), n - 1);  // the others' bytes stay as they are
            load8<BF16, VEC>(src, at0 + at * stride + 8 * e, v[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t fresh = codes4(v[0][j], v[1][j], v[2][j], v[3][j]);
            cell[j * step] = fresh_part == 0xFFFFFFFFu ? fresh : pick(fresh_part, fresh, cell[j * step]);
        }
    }
}

template <int FMT, bool BF16>
__global__ __launch_bounds__(256) void kv8_read_kernel(Kv8 c, int total, int max_new, void* __restrict__ k_out,
                                                       void* __restrict__ v_out) {
    const int h = blockIdx.y;
    const int b = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const Kv8Span s = kv8_span(c, b, total, max_new);
    const int p0 = s.begin >= 0 ? s.begin / c.P : -((c.P - 1 - s.begin) / c.P);
    const int p = p0 + (int)blockIdx.x;
    const int lo = max(s.begin, p * c.P), hi = min(s.end, p * c.P + c.P);
    if (lo >= hi) return;
    const int D = c.D, d8 = D >> 3, tid = threadIdx.x, n = hi - lo;
    const int pg = p >= 0 && p < c.max_pages ? c.table[(long long)b * c.max_pages + p] : -1;
    const bool live = pg >= 0 && pg < c.pages;
    const long long page = live ? ((long long)pg * c.H + h) * c.P * D : 0;
    const float scale = live ? (is_v ? c.v_scale : c.k_scale)[(long long)pg * c.H + h] : 0.0f;
    void* out = is_v ? v_out : k_out;
    const long long row = ((long long)(s.row0 + lo - s.begin) * c.H + h) * D, step = (long long)c.H * D;
    const int lo_s = lo - p * c.P;
    if (!live) {
        const float zero[8] = {};
        for (int t = tid; t < n * d8; t += 256) store8<BF16>(out, row + t / d8 * step + 8 * (t % d8), zero);
        return;
    }
    const auto value = [&](uint32_t lo_w, uint32_t hi_w, float (&v)[8]) {
        float a[4], z[4];
        kv_values4<FMT>(lo_w, a);
        kv_values4<FMT>(hi_w, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j] * scale;
            v[4 + j] = z[j] * scale;
        }
    };
    if (!is_v) {
        const uint2* src = reinterpret_cast<const uint2*>(c.k_codes + page) + lo_s * d8;
        for (int t = tid; t < n * d8; t += 256) {
            const int i = t / d8;
            const uint2 w = src[t];
            float v[8];
            value(w.x, w.y, v);
            store8<BF16>(out, row + i * step + 8 * (t - i * d8), v);
        }
        return;
    }
    // four slots of eight d a thread, turned in registers
    const int q0 = lo_s >> 2, quads = ((lo_s + n + 3) >> 2) - q0;
    for (int t = tid; t < quads * d8; t += 256) {
        const int e = t / quads, slot = 4 * (q0 + t - e * quads);
        const uint32_t* cell = reinterpret_cast<const uint32_t*>(c.v_codes + page + (long long)8 * e * c.P + slot);
        float x[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) kv_values4<FMT>(cell[j * (c.P >> 2)], x[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = slot + i - lo_s;
            if (at < 0 || at >= n) continue;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[j][i] * scale;
            store8<BF16>(out, row + at * step + 8 * e, v);
        }
    }
}

}  // namespace

// Pages that max_new consecutive tokens can touch.
static int pages_touched(int max_new, int P) { return (max_new + P - 2) / P + 1; }

hipError_t launch_kv8_append(const Kv8& c, int format, int total, int max_new, bool bf16, const void* k_new,
                             long long k_stride, const void* v_new, long long v_stride, hipStream_t stream) {
    const dim3 grid(pages_touched(max_new, c.P), c.H, 2 * c.B);
    const int size = bf16 ? 2 : 4;
    const bool vec = (((uintptr_t)k_new | (uintptr_t)v_new) & 15) == 0 && (k_stride * size) % 16 == 0 && (v_stride * size) % 16 == 0;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, c, total, max_new, k_new, k_stride, v_new, v_stride);
    };
    auto by_type = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (vec)
            bf16 ? go(kv8_append_kernel<F, true, true>) : go(kv8_append_kernel<F, false, true>);
        else
            bf16 ? go(kv8_append_kernel<F, true, false>) : go(kv8_append_kernel<F, false, false>);
    };
    if (format == KV8_INT8)
        by_type(std::integral_constant<int, KV8_INT8>());
    else
        by_type(std::integral_constant<int, KV8_E4M3>());
    return hipGetLastError();
}

hipError_t launch_kv8_read(const Kv8& c, int format, int total, int max_new, bool bf16, void* k_out, void* v_out,
                           hipStream_t stream) {
    const dim3 grid(pages_touched(max_new, c.P), c.H, 2 * c.B);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, c, total, max_new, k_out, v_out);
    };
    if (format == KV8_INT8)
        bf16 ? go(kv8_read_kernel<KV8_INT8, true>) : go(kv8_read_kernel<KV8_INT8, false>);
    else
        bf16 ? go(kv8_read_kernel<KV8_E4M3, true>) : go(kv8_read_kernel<KV8_E4M3, false>);
    return hipGetLastError();
}

}  // namespace q4
