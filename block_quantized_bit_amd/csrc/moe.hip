// Routed gated MLP on 4-bit experts for a few tokens (moe.h), in two launches.
//
// The work is bound by the bytes of the chosen experts' weights, so both
// kernels stream each of them once and keep everything else small:
//   up    a workgroup takes one chosen expert and one block of bs hidden rows
//         (the gate row and the up row of each). It routes by itself (the
//         top_k of T x E logits is cheaper than a launch), quantizes the
//         expert's tokens into LDS, and ends with the block's hidden values,
//         which it can therefore quantize itself: the next kernel reads codes.
//   down  a workgroup takes a few rows of W2 of all chosen experts, and adds
//         the experts of a token in their order, with no atomics.
// The integer dots are v_dot4_i32_i8 on nibbles masked out of 16-byte loads,
// as in the decode GEMV: one lane owns whole 32-code pieces of a row, so a
// block's scales enter once per piece. Several tokens of an affine expert go
// through the int8 matrix cores instead.
// One token, 8 of 128 experts (2048 x 768, Q4_0): 13.2 us, 7.9 + 5.2 in the two
// kernels, for 21 MB. Sixteen tokens, 2 of 8 experts (4096 x 14336, affine 128):
// 224 us, 123 (3.9 TB/s) + 99 (2.4 TB/s). The second kernel's 99 us is the same
// with v_dot4 or the matrix cores, with twice the loads in flight, with rotated
// starts and with fewer cache lines a load: the reason is not found. (Not tried:
// the tokens' codes in LDS, as in the first kernel.)
#include <type_traits>

#include "kernels_wide.h"
#include "moe.h"
#include "wide.h"

namespace q4 {

namespace {

constexpr uint32_t OUT = 0x80000000u;  // beyond every buffer range: reads as zero
constexpr int ONCE = 2;                // non-temporal: each weight byte is read once
constexpr int MOST_PAIRS = 64 * 16;
// Tokens of an expert that share one reading of its weights: 8 sums a row in
// registers, or the 16 columns of a matrix instruction (affine, see MatrixSteps).
constexpr int DOT_BATCH = 8, MATRIX_BATCH = 16;

__device__ __forceinline__ int dot32(const uint4& w, const uint4& xa, const uint4& xb) {
    int d = 0;
    d = __builtin_amdgcn_sdot4((int)lo_nibbles(w.x), (int)xa.x, d, false);
    d = __builtin_amdgcn_sdot4((int)lo_nibbles(w.y), (int)xa.y, d, false);
    d = __builtin_amdgcn_sdot4((int)lo_nibbles(w.z), (int)xa.z, d, false);
    d = __builtin_amdgcn_sdot4((int)lo_nibbles(w.w), (int)xa.w, d, false);
    d = __builtin_amdgcn_sdot4((int)hi_nibbles(w.x), (int)xb.x, d, false);
    d = __builtin_amdgcn_sdot4((int)hi_nibbles(w.y), (int)xb.y, d, false);
    d = __builtin_amdgcn_sdot4((int)hi_nibbles(w.z), (int)xb.z, d, false);
    d = __builtin_amdgcn_sdot4((int)hi_nibbles(w.w), (int)xb.w, d, false);
    return d;
}

__device__ __forceinline__ float wave_max(float v) {
    v = row_max16(v);
    const int b = __builtin_bit_cast(int, v);
    const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}

// The chosen experts of one token, by one wavefront: lane + 64 j is an expert.
// sel and weight [top_k]; -1 and 0 where fewer are left.
template <int J>
__device__ __forceinline__ void route(const float* __restrict__ logits, int E, int top_k, bool renorm, int lane,
                                      int* sel, float* weight) {
    const float none = -__builtin_inff();
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 64 * j;
        const float x = e < E ? logits[e] : none;
        v[j] = x == x ? x : none;
    }
    float most = v[0];
#pragma unroll
    for (int j = 1; j < J; ++j) most = fmaxf(most, v[j]);
    most = wave_max(most);
    float all = 0.0f;
    if (!renorm && most != none) {
#pragma unroll
        for (int j = 0; j < J; ++j) all += expf(v[j] - most);
        all = wave_sum(all);
    }
    float mine_w = 0.0f;
    int mine_e = -1;
    float sum = 0.0f;
    float top = most;
    for (int k = 0; k < top_k; ++k) {
        if (k > 0) {
            float m = v[0];
#pragma unroll
            for (int j = 1; j < J; ++j) m = fmaxf(m, v[j]);
            top = wave_max(m);
        }
        if (top == none) break;
        int e = -1;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const unsigned long long hit = __ballot(v[j] == top);
            if (e < 0 && hit) e = 64 * j + __builtin_ctzll(hit);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (lane + 64 * j == e) v[j] = none;
        const float w = expf(top - most);
        sum += w;
        if (lane == k) {
            mine_e = e;
            mine_w = w;
        }
    }
    const float by = renorm ? sum : all;
    if (lane < top_k) {
        sel[lane] = mine_e;
        weight[lane] = mine_e >= 0 ? mine_w / by : 0.0f;
    }
}

struct Moe {
    int T, H, I, E, k;
    int renorm;
    int wide;  // scales and biases start on 16 bytes
    const void* x;
    const float* logits;
    const uint8_t* w13;
    const uint16_t* s13;
    const uint16_t* b13;
    const uint8_t* w2;
    const uint16_t* s2;
    const uint16_t* b2;
    void* y;
    // workspace
    int8_t* hq;       // [pairs][I], pair = t * k + j
    uint2* hs;        // [pairs][I / bs]: scale (float32) and code sum (int32)
    int* sel;         // [pairs]
    float* weight;    // [pairs]
    int* slots;       // [1 + pairs]: number of chosen experts, then their indices, rising
};

// A lane's weights for U pieces of R rows: piece c of a row is 32 codes, lane
// part `lc` of LPR takes pieces c0 + lc, c0 + LPR + lc, ... The loads are issued
// by load() and may be on their way while other work is done. Rows past the
// range and pieces past the row read as zeros.
template <int FMT, int G, int R, int LPR, int U>
struct Piece {
    static constexpr int CPG = G / 32;
    uint4 w[U][R];
    uint16_t s[U][R], b[U][R];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs,
                                         __amdgpu_buffer_rsrc_t rb, const uint32_t (&row)[R], int nchunks, int c0,
                                         int lc) {
        const int ngroups = nchunks / CPG;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * LPR + lc;
            const bool in = c < nchunks;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                w[u][i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                        rw, in ? row[i] * (16u * nchunks) + 16u * c : OUT, 0, ONCE));
                const uint32_t at = in ? 2u * (row[i] * ngroups + c / CPG) : OUT;
                s[u][i] = __builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
                if (FMT == 1) b[u][i] = __builtin_amdgcn_raw_buffer_load_b16(rb, at, 0, 0);
            }
        }
    }

    // acc[i][n] += row i's product with activation n; act(n, c, group, ...) gives the codes, scale and code sum
    template <int NT, typename Act>
    __device__ __forceinline__ void multiply(int nchunks, int c0, int lc, Act act, float (&acc)[R][NT]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * LPR + lc;
            const int cc = c < nchunks ? c : nchunks - 1;  // past the row: zero codes and scales
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 xa, xb;
                float xs;
                int xm;
                act(n, cc, cc / CPG, xa, xb, xs, xm);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int d = dot32(w[u][i], xa, xb);
                    if (FMT == 0) {
                        acc[i][n] += (half_to_float(s[u][i]) * xs) * (float)(d - 8 * xm);
                    } else {
                        acc[i][n] += xs * (bf16_to_float(s[u][i]) * (float)d);
                        const float t = xs * (bf16_to_float(b[u][i]) * (float)xm);
                        acc[i][n] += c % CPG == 0 ? t : 0.0f;
                    }
                }
            }
        }
    }
};

// acc over all pieces of the rows; `p` holds the first ones' loads. (No second set
// of registers for the next pieces' loads: the wavefronts that a CU holds in their
// place hide the loads.)
template <int FMT, int G, int R, int LPR, int U, int NT, typename Act>
__device__ __forceinline__ void row_products(Piece<FMT, G, R, LPR, U>& p, __amdgpu_buffer_rsrc_t rw,
                                             __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rb,
                                             const uint32_t (&row)[R], int nchunks, int lc, Act act,
                                             float (&acc)[R][NT]) {
    for (int c0 = 0; c0 < nchunks; c0 += U * LPR) {
        if (c0 > 0) p.load(rw, rs, rb, row, nchunks, c0, lc);
        p.multiply(nchunks, c0, lc, act, acc);
    }
}

__device__ __forceinline__ float add_swapped(uint32_t a, uint32_t b) { return __uint_as_float(a) + __uint_as_float(b); }

// Sum over aligned groups of LPR lanes: DPP inside a row of 16, lane swaps between rows.
template <int LPR>
__device__ __forceinline__ float group_total(float v) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false));
    if (LPR >= 32) {
        const uint32_t x = __float_as_uint(v);
        const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        v = add_swapped(a[0], a[1]);
    }
    if (LPR >= 64) {
        const uint32_t x = __float_as_uint(v);
        const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        v = add_swapped(a[0], a[1]);
    }
    return v;
}

// f(number of tokens to compute) for n tokens: the next larger of the built ones.
template <int MOST, typename F>
__device__ __forceinline__ void by_tokens(int n, F f) {
    if (MOST == 1 || n == 1) return f(std::integral_constant<int, 1>());
    if constexpr (MOST > 1) {
        if (n == 2) return f(std::integral_constant<int, 2>());
        if (n <= 4) return f(std::integral_constant<int, 4>());
        if (n <= 6) return f(std::integral_constant<int, 6>());
        f(std::integral_constant<int, 8>());
    }
}

// Four steps of sixteen weight rows against up to sixteen tokens on the int8
// matrix cores; a step is 128 codes of k, for affine groups of 64 or 128. Lane
// (r, q) holds piece q of a step's four of weight row r (low nibbles: 16
// consecutive k, high nibbles the next 16) and the same 32 codes of token r; the
// sum over the lane groups that the instruction takes is then the whole step's,
// or with the other groups' codes zeroed one group of 64. A lane of the result
// has one weight row (r) and the four tokens 4 q ..., so a weight's scale is one
// value a lane; the scales of the four steps come in one load each where rows
// of them start on its size (single 2-byte loads take more of the caches'
// throughput than the weights themselves).
template <int G>
struct MatrixSteps {
    static constexpr int U = 4;
    static constexpr int PARTS = 128 / G;        // groups a step
    static constexpr int WORDS = U * PARTS / 2;  // of two scales
    uint4 w[U];
    uint32_t s[WORDS], b[WORDS];

    // steps t0 .. t0 + 3 of weight row `row`; t0 is a multiple of four. wide: nchunks is a multiple of 16.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs,
                                         __amdgpu_buffer_rsrc_t rb, uint32_t row, int nchunks, bool wide, int t0,
                                         int end, int q) {
        const int ngroups = nchunks / (G / 32);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = 4 * (t0 + u) + q;
            w[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rw, t0 + u < end && c < nchunks ? row * (16u * nchunks) + 16u * c : OUT, 0, ONCE));
        }
        const int grp = PARTS * t0;
        if (wide) {
            const uint32_t at = 2u * (row * ngroups + grp);
            if (WORDS == 2) {
                const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0));
                const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rb, at, 0, 0));
                s[0] = x.x; s[1] = x.y;
                b[0] = y.x; b[1] = y.y;
            } else {
                const uint4 x = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
                const uint4 y = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rb, at, 0, 0));
                s[0] = x.x; s[1] = x.y; s[2 % WORDS] = x.z; s[3 % WORDS] = x.w;
                b[0] = y.x; b[1] = y.y; b[2 % WORDS] = y.z; b[3 % WORDS] = y.w;
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
            const uint32_t lo = grp + 2 * j < ngroups ? 2u * (row * ngroups + grp + 2 * j) : OUT;
            const uint32_t hi = grp + 2 * j + 1 < ngroups ? 2u * (row * ngroups + grp + 2 * j + 1) : OUT;
            s[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, lo, 0, 0) |
                   ((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, hi, 0, 0) << 16);
            b[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, lo, 0, 0) |
                   ((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, hi, 0, 0) << 16);
        }
    }

    // acc[i] += the row's products with tokens 4 q + i, steps before `end`. codes(c, lo, hi): piece c of this
    // lane's token; sums(group, xs, xm): scales and code sums of tokens 4 q ...
    template <typename Codes, typename Sums>
    __device__ __forceinline__ void multiply(int nchunks, int t0, int end, int q, Codes codes, Sums sums,
                                             v4f& acc) const {
        const int ngroups = nchunks / (G / 32);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t0 + u >= end) break;
            v4i xa, xb;
            codes(min(4 * (t0 + u) + q, nchunks - 1), xa, xb);
            const v4i lo = {(int)lo_nibbles(w[u].x), (int)lo_nibbles(w[u].y), (int)lo_nibbles(w[u].z), (int)lo_nibbles(w[u].w)};
            const v4i hi = {(int)hi_nibbles(w[u].x), (int)hi_nibbles(w[u].y), (int)hi_nibbles(w[u].z), (int)hi_nibbles(w[u].w)};
#pragma unroll
            for (int j = 0; j < PARTS; ++j) {
                const int keep = PARTS == 1 || (q >> 1) == j ? -1 : 0;
                v4i d = {0, 0, 0, 0};
                d = __builtin_amdgcn_mfma_i32_16x16x64_i8(xa, lo & keep, d, 0, 0, 0);
                d = __builtin_amdgcn_mfma_i32_16x16x64_i8(xb, hi & keep, d, 0, 0, 0);
                float xs[4];
                int xm[4];
                sums(min(PARTS * (t0 + u) + j, ngroups - 1), xs, xm);
                const int at = PARTS * u + j;
                const float sw = bf16_to_float(at & 1 ? s[at / 2] >> 16 : s[at / 2] & 0xFFFFu);
                const float bw = bf16_to_float(at & 1 ? b[at / 2] >> 16 : b[at / 2] & 0xFFFFu);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = fmaf(xs[i], fmaf(sw, (float)d[i], bw * (float)xm[i]), acc[i]);
            }
        }
    }
};

// ---- gate and up --------------------------------------------------------------------

// Sixteen lanes share a row, so that a wavefront's load covers four rows (of two
// hidden values: gate and up of each) and a row's sum needs four lane additions;
// wavefronts with few rows take more pieces at a time instead.
template <int G>
struct Up {
    static constexpr int WAVES = G == 32 ? 16 : 8;
    static constexpr int ROWS = 2 * G / WAVES;              // weight rows of a wavefront: 4, 16, 32
    static constexpr int R = ROWS < 16 ? ROWS / 4 : 4;      // loads of four rows at a time: 1, 4, 4
    static constexpr int U = R == 1 ? 4 : 1;
};

// MATRIX: tokens on the matrix instructions (affine, more than one token in the
// call), else v_dot4.
template <int FMT, int G, bool XBF16, int J, bool MATRIX>
__global__ __launch_bounds__(64 * Up<G>::WAVES) void moe_up_kernel(Moe a, int batch) {
    constexpr int WAVES = Up<G>::WAVES, NT = 64 * WAVES;
    constexpr int L = 16;        // lanes a block of G while quantizing
    constexpr int EPT = G / L;   // 2, 4 or 8 values a lane
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int sel[MOST_PAIRS];
    __shared__ float weight[MOST_PAIRS];
    __shared__ int used[512];
    __shared__ int mine[64];  // pairs of this workgroup's expert
    constexpr int BATCH = MATRIX ? MATRIX_BATCH : DOT_BATCH;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.k;
    const int H = a.H, nchunks = H / 32, ngroups = H / G;
    const int pitch = H + 16;  // rows of tokens start on different banks
    int8_t* xq = reinterpret_cast<int8_t*>(lds);                          // [batch][pitch]
    float* xs = reinterpret_cast<float*>(lds + (size_t)batch * pitch);    // [H / G][BATCH]
    int* xm = reinterpret_cast<int*>(xs + (size_t)BATCH * ngroups);       // [H / G][BATCH]
    float* hid = reinterpret_cast<float*>(xm + (size_t)BATCH * ngroups);  // [gate, up][batch][G]

    // int8 codes of n tokens: 16 lanes a block; token(i) is the i-th one's row of x
    const auto quantize = [&](int n, auto token, int thread, int threads) {
        const int items = n * ngroups * L;
        for (int i0 = 0; i0 < items; i0 += threads) {
            const bool live = i0 + thread < items;  // whole blocks of 16 lanes
            const int it = live ? i0 + thread : items - 1;
            const int tk = it / (ngroups * L), at = it - tk * (ngroups * L);
            const int grp = at / L, k0 = grp * G + (at & (L - 1)) * EPT;
            const long long src = (long long)token(tk) * H + k0;
            float v[EPT];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                v[j] = load_as_float<XBF16>(a.x, src + j);
                top = max(top, magnitude(v[j]));
            }
            const float amax = __uint_as_float(row_max16(top));  // a NaN if there is one: it makes the scale NaN
            const float s = amax / 127.0f;
            const float inv = act_inverse(s);
            int q[EPT], sum = 0;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                q[j] = amax != 0.0f ? act_code(v[j], s, inv) : 0;
                sum += q[j];
            }
#pragma unroll
            for (int off = 1; off < L; off <<= 1) sum += __shfl_xor(sum, off, 64);
            if (!live) continue;
#pragma unroll
            for (int j = 0; j < EPT; ++j) xq[tk * pitch + k0 + j] = (int8_t)q[j];
            if ((at & (L - 1)) == 0) {
                xs[grp * BATCH + tk] = amax != 0.0f ? s : 0.0f;
                xm[grp * BATCH + tk] = sum;
            }
        }
    };

    for (int e = tid; e < a.E; e += NT) used[e] = 0;
    __syncthreads();
    for (int t = wave; t < a.T; t += WAVES) {
        route<J>(a.logits + (long long)t * a.E, a.E, a.k, a.renorm != 0, lane, sel + t * a.k, weight + t * a.k);
        if (lane < a.k && sel[t * a.k + lane] >= 0) used[sel[t * a.k + lane]] = 1;
    }
    // a single token is every expert's: the other wavefronts quantize it while the first one routes
    if (a.T == 1 && wave > 0) quantize(1, [](int) { return 0; }, tid - 64, NT - 64);
    __syncthreads();

    // the slot-th used expert, and the pairs it has; every wavefront finds them for itself
    const int slot = blockIdx.y;
    int before = 0, expert = -1;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 64 * j;
        const unsigned long long hit = __ballot(e < a.E && used[e]);
        const int n = __popcll(hit);
        if (expert < 0 && slot < before + n) {
            unsigned long long rest = hit;
            for (int i = before; i < slot; ++i) rest &= rest - 1;
            expert = 64 * j + __builtin_ctzll(rest);
        }
        if (blockIdx.x == 0 && slot == 0 && wave == 0 && (hit >> lane & 1))
            a.slots[1 + before + __popcll(hit & ((1ull << lane) - 1))] = e;
        before += n;
    }
    if (blockIdx.x == 0 && slot == 0) {
        if (tid == 0) a.slots[0] = before;
        for (int p = tid; p < pairs; p += NT) {
            a.sel[p] = sel[p];
            a.weight[p] = weight[p];
        }
    }
    expert = __builtin_amdgcn_readfirstlane(expert);
    if (expert < 0) return;
    int count = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
        const int p = p0 + lane;
        const unsigned long long hit = __ballot(p < pairs && sel[p] == expert);
        // all wavefronts write the same
        if (hit >> lane & 1) mine[count + __popcll(hit & ((1ull << lane) - 1))] = p;
        count += __popcll(hit);
    }

    const uint32_t rows = 2u * a.I;
    const __amdgpu_buffer_rsrc_t rw = buffer_of(a.w13 + (size_t)expert * rows * (H / 2), rows * (uint32_t)(H / 2));
    const __amdgpu_buffer_rsrc_t rs = buffer_of(a.s13 + (size_t)expert * rows * ngroups, rows * ngroups * 2u);
    const __amdgpu_buffer_rsrc_t rb =
        buffer_of(FMT == 1 ? a.b13 + (size_t)expert * rows * ngroups : nullptr, FMT == 1 ? rows * ngroups * 2u : 0u);
    const int h0 = blockIdx.x * G;  // I is a multiple of G: the block is whole
    constexpr int R = Up<G>::R;
    // lane group 2 j + (0 gate, 1 up) of load i: hidden row r0 + 2 i + j
    const int which = (lane >> 4) & 1, pair_row = lane >> 5;
    const auto rows_at = [&](int r0, uint32_t (&row)[R]) {
#pragma unroll
        for (int i = 0; i < R; ++i) row[i] = which * a.I + h0 + r0 + 2 * i + pair_row;
    };
    const int r_first = wave * (G / WAVES), r_end = r_first + G / WAVES;

    const auto up_by_dots = [&](int first, int n) {
        // the first weights are on their way while the tokens are quantized
        Piece<FMT, G, R, 16, Up<G>::U> piece;
        uint32_t row[R];
        rows_at(r_first, row);
        piece.load(rw, rs, rb, row, nchunks, 0, lane & 15);
        if (a.T > 1) {
            quantize(n, [&](int i) { return mine[first + i] / a.k; }, tid, NT);
            __syncthreads();
        }
        by_tokens<FMT == 1 ? 1 : 8>(n, [&](auto nt) {
            constexpr int N = decltype(nt)::value;
            const auto act = [&](int i, int c, int grp, uint4& xa, uint4& xb, float& s, int& m) {
                const int tk = min(i, n - 1);
                const uint4* p = reinterpret_cast<const uint4*>(xq + tk * pitch + 32 * c);
                xa = p[0];
                xb = p[1];
                s = xs[grp * BATCH + tk];
                m = xm[grp * BATCH + tk];
            };
#pragma unroll 1
            for (int r0 = r_first; r0 < r_end; r0 += 2 * R) {
                if (r0 > r_first) {
                    rows_at(r0, row);
                    piece.load(rw, rs, rb, row, nchunks, 0, lane & 15);
                }
                float acc[R][N] = {};
                row_products(piece, rw, rs, rb, row, nchunks, lane & 15, act, acc);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        const float v = group_total<16>(acc[i][t]);
                        if ((lane & 15) == 0 && t < n) hid[(which * batch + t) * G + r0 + 2 * i + pair_row] = v;
                    }
            }
        });
    };

    for (int first = 0; first < count; first += batch) {
        const int n = min(batch, count - first);
        if (first > 0) __syncthreads();
        if constexpr (MATRIX) {
            quantize(n, [&](int i) { return mine[first + i] / a.k; }, tid, NT);
            __syncthreads();
            // a wavefront's rows in tiles of sixteen: gate rows, then up rows (of its 16 hidden values for
            // groups of 128, of its 8 for groups of 64)
            constexpr int HID = G / WAVES, TILES = 2 * HID / 16;
            const int r = lane & 15, q = lane >> 4;
            uint32_t row[TILES];
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const int at = 16 * i + r;
                row[i] = (at / HID) * a.I + h0 + r_first + at % HID;
            }
            const auto codes = [&](int c, v4i& lo, v4i& hi) {
                const v4i* p = reinterpret_cast<const v4i*>(xq + min(r, n - 1) * pitch + 32 * c);
                lo = p[0];
                hi = p[1];
            };
            const auto sums = [&](int grp, float (&s)[4], int (&m)[4]) {
                const float4 f = *reinterpret_cast<const float4*>(xs + grp * BATCH + 4 * q);
                const int4 k = *reinterpret_cast<const int4*>(xm + grp * BATCH + 4 * q);
                s[0] = f.x; s[1] = f.y; s[2] = f.z; s[3] = f.w;
                m[0] = k.x; m[1] = k.y; m[2] = k.z; m[3] = k.w;
            };
            v4f acc[TILES];
#pragma unroll
            for (int i = 0; i < TILES; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            const int steps = (nchunks + 3) / 4;
            const bool wide = a.wide && nchunks % 16 == 0;
            for (int t0 = 0; t0 < steps; t0 += MatrixSteps<G>::U) {
                MatrixSteps<G> w[TILES];
#pragma unroll
                for (int i = 0; i < TILES; ++i) w[i].load(rw, rs, rb, row[i], nchunks, wide, t0, steps, q);
#pragma unroll
                for (int i = 0; i < TILES; ++i) w[i].multiply(nchunks, t0, steps, q, codes, sums, acc[i]);
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 16 * i + r;
                    if (4 * q + e < n) hid[((at / HID) * batch + 4 * q + e) * G + r_first + at % HID] = acc[i][e];
                }
        } else {
            up_by_dots(first, n);
        }
        __syncthreads();

        // the block's hidden values are one quantization block of each token: 16 lanes each
        for (int it = tid; it < n * L; it += NT) {
            const int tk = it / L, k0 = (it & (L - 1)) * EPT;
            float v[EPT];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const float g = hid[tk * G + k0 + j], u = hid[(batch + tk) * G + k0 + j];
                v[j] = g / (1.0f + expf(-g)) * u;
                top = max(top, magnitude(v[j]));
            }
            const float amax = __uint_as_float(row_max16(top));
            const float s = amax / 127.0f;
            const float inv = act_inverse(s);
            const int pair = mine[first + tk];
            int sum = 0;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const int q = amax != 0.0f ? act_code(v[j], s, inv) : 0;
                sum += q;
                a.hq[(size_t)pair * a.I + h0 + k0 + j] = (int8_t)q;
            }
#pragma unroll
            for (int off = 1; off < L; off <<= 1) sum += __shfl_xor(sum, off, 64);
            if ((it & (L - 1)) == 0) {
                a.hs[(size_t)pair * (a.I / G) + blockIdx.x] =
                    make_uint2(__float_as_uint(amax != 0.0f ? s : 0.0f), (uint32_t)sum);
            }
        }
    }
}

// ---- down -----------------------------------------------------------------------------

constexpr int DOWN_WAVES = 8;

// LPR lanes share a row's pieces. A workgroup has ROWS rows of W2, a wavefront
// takes all of them of one expert, or a part where there are fewer experts than
// wavefronts. More rows share the reading of the hidden codes, fewer give more
// workgroups.
template <int FMT, int G, int LPR, int ROWS_WG, bool YBF16>
__global__ __launch_bounds__(64 * DOWN_WAVES) void moe_down_kernel(Moe a) {
    constexpr int NT = 64 * DOWN_WAVES;
    constexpr int RPL = 64 / LPR;  // rows a load instruction covers
    constexpr int R = ROWS_WG / 4, U = 4 / R;
    constexpr int ROWS = R * RPL;  // of a wavefront: ROWS_WG, or a half or a quarter
    extern __shared__ float part[];                     // [pairs][ROWS_WG]: products of every pair
    __shared__ int sel[MOST_PAIRS];
    __shared__ int list[DOWN_WAVES][64];                // pairs of the expert a wavefront works on

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.k;
    const int n0 = blockIdx.x * ROWS_WG;
    const int I = a.I, nchunks = I / 32, ngroups = I / G;
    for (int p = tid; p < pairs; p += NT) sel[p] = a.sel[p];
    const int nslots = __builtin_amdgcn_readfirstlane(a.slots[0]);
    __syncthreads();

    constexpr int PER = ROWS_WG / ROWS;
    for (int item = wave; item < nslots * PER; item += DOWN_WAVES) {
        const int expert = __builtin_amdgcn_readfirstlane(a.slots[1 + item / PER]);
        const int r0 = n0 + item % PER * ROWS;
        int count = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const unsigned long long hit = __ballot(p < pairs && sel[p] == expert);
            if (hit >> lane & 1) list[wave][count + __popcll(hit & ((1ull << lane) - 1))] = p;
            count += __popcll(hit);
        }
        const __amdgpu_buffer_rsrc_t rw = buffer_of(a.w2 + (size_t)expert * a.H * (I / 2), (uint32_t)a.H * (I / 2));
        const __amdgpu_buffer_rsrc_t rs = buffer_of(a.s2 + (size_t)expert * a.H * ngroups, (uint32_t)a.H * ngroups * 2u);
        const __amdgpu_buffer_rsrc_t rb = buffer_of(FMT == 1 ? a.b2 + (size_t)expert * a.H * ngroups : nullptr,
                                                    FMT == 1 ? (uint32_t)a.H * ngroups * 2u : 0u);
        uint32_t row[R];
#pragma unroll
        for (int i = 0; i < R; ++i) row[i] = r0 + i * RPL + lane / LPR;  // H is a multiple of 32: inside
        const auto run = [&](auto nt, int first, int n) {
            constexpr int N = decltype(nt)::value;
            int pair[N];
#pragma unroll
            for (int i = 0; i < N; ++i) pair[i] = list[wave][first + min(i, n - 1)];
            const auto act = [&](int i, int c, int grp, uint4& xa, uint4& xb, float& s, int& m) {
                const uint4* p = reinterpret_cast<const uint4*>(a.hq + (size_t)pair[i] * I + 32 * c);
                xa = p[0];
                xb = p[1];
                const uint2 t = a.hs[(size_t)pair[i] * ngroups + grp];
                s = __uint_as_float(t.x);
                m = (int)t.y;
            };
            float acc[R][N] = {};
            Piece<FMT, G, R, LPR, U> piece;
            piece.load(rw, rs, rb, row, nchunks, 0, lane % LPR);
            row_products(piece, rw, rs, rb, row, nchunks, lane % LPR, act, acc);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const float v = group_total<LPR>(acc[q][i]);
                    if (lane % LPR == 0 && i < n) part[pair[i] * ROWS_WG + row[q] - n0] = v;
                }
        };
        for (int first = 0; first < count; first += 8) {
            const int n = min(8, count - first);
            by_tokens<8>(n, [&](auto nt) { run(nt, first, n); });
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * ROWS_WG; i += NT) {
        const int t = i / ROWS_WG, q = i % ROWS_WG;
        float v = 0.0f;
        for (int j = 0; j < a.k; ++j)
            if (sel[t * a.k + j] >= 0) v = fmaf(a.weight[t * a.k + j], part[(t * a.k + j) * ROWS_WG + q], v);
        const size_t at = (size_t)t * a.H + n0 + q;
        if (YBF16)
            static_cast<uint16_t*>(a.y)[at] = (uint16_t)bf16_bits(v);
        else
            static_cast<float*>(a.y)[at] = v;
    }
}

// The same on the matrix cores, for affine experts with several tokens each:
// sixteen rows a workgroup, one expert and half of k a wavefront.
constexpr int MATRIX_WAVES = 16, HALVES = 2;
constexpr size_t CU_LDS = 160 * 1024;
static_assert((MOST_PAIRS + MATRIX_WAVES * 64) * 4 + HALVES * MOST_PAIRS * 16 * 4 <= CU_LDS, "lists and sums of any call");

template <int G, bool YBF16>
__global__ __launch_bounds__(64 * MATRIX_WAVES) void moe_down_matrix_kernel(Moe a, int stage) {
    constexpr int NT = 64 * MATRIX_WAVES, U = MatrixSteps<G>::U;
    extern __shared__ __attribute__((aligned(16))) float part[];  // [HALVES][pairs][16], then `staged` [pairs][I / G]
    __shared__ int sel[MOST_PAIRS];
    __shared__ int list[MATRIX_WAVES][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.k;
    const int n0 = blockIdx.x * 16;
    const int I = a.I, nchunks = I / 32, ngroups = I / G;
    for (int p = tid; p < pairs; p += NT) sel[p] = a.sel[p];
    const int nslots = __builtin_amdgcn_readfirstlane(a.slots[0]);
    uint2* staged = reinterpret_cast<uint2*>(part + HALVES * pairs * 16);  // scales and code sums, if they fit
    if (stage)
        for (int p = tid; p < pairs * ngroups; p += NT) staged[p] = a.hs[p];
    __syncthreads();

    const int r = lane & 15, q = lane >> 4;
    const int steps = (nchunks + 3) / 4, half = ((steps + HALVES - 1) / HALVES + U - 1) / U * U;
    const bool wide = a.wide && nchunks % 16 == 0;
    for (int item = wave; item < nslots * HALVES; item += MATRIX_WAVES) {
        const int expert = __builtin_amdgcn_readfirstlane(a.slots[1 + item / HALVES]);
        const int h = item % HALVES;
        const int from = h * half, to = min(steps, from + half);
        int count = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const unsigned long long hit = __ballot(p < pairs && sel[p] == expert);
            if (hit >> lane & 1) list[wave][count + __popcll(hit & ((1ull << lane) - 1))] = p;
            count += __popcll(hit);
        }
        const __amdgpu_buffer_rsrc_t rw = buffer_of(a.w2 + (size_t)expert * a.H * (I / 2), (uint32_t)a.H * (I / 2));
        const __amdgpu_buffer_rsrc_t rs = buffer_of(a.s2 + (size_t)expert * a.H * ngroups, (uint32_t)a.H * ngroups * 2u);
        const __amdgpu_buffer_rsrc_t rb = buffer_of(a.b2 + (size_t)expert * a.H * ngroups, (uint32_t)a.H * ngroups * 2u);
        for (int first = 0; first < count; first += 16) {
            const int n = min(16, count - first);
            const int8_t* mine = a.hq + (size_t)list[wave][first + min(r, n - 1)] * I;
            int at[4];  // scales of tokens 4 q + i
#pragma unroll
            for (int i = 0; i < 4; ++i) at[i] = list[wave][first + min(4 * q + i, n - 1)] * ngroups;
            const auto codes = [&](int c, v4i& lo, v4i& hi) {
                const v4i* p = reinterpret_cast<const v4i*>(mine + 32 * c);
                lo = p[0];
                hi = p[1];
            };
            const auto sums = [&](int grp, float (&s)[4], int (&m)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 t = stage ? staged[at[i] + grp] : a.hs[at[i] + grp];
                    s[i] = __uint_as_float(t.x);
                    m[i] = (int)t.y;
                }
            };
            v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int t0 = from; t0 < to; t0 += U) {
                MatrixSteps<G> w;
                w.load(rw, rs, rb, n0 + r, nchunks, wide, t0, to, q);
                w.multiply(nchunks, t0, to, q, codes, sums, acc);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * q + i < n) part[(h * pairs + list[wave][first + 4 * q + i]) * 16 + r] = acc[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 16; i += NT) {
        const int t = i / 16, c = i % 16;
        float v = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = t * a.k + j;
            if (sel[p] >= 0) v = fmaf(a.weight[p], part[p * 16 + c] + part[(pairs + p) * 16 + c], v);
        }
        const size_t at = (size_t)t * a.H + n0 + c;
        if (YBF16)
            static_cast<uint16_t*>(a.y)[at] = (uint16_t)bf16_bits(v);
        else
            static_cast<float*>(a.y)[at] = v;
    }
}

template <int FMT, int G, bool BF16>
hipError_t launch(const Moe& a, hipStream_t stream) {
    const int slots = min(a.E, a.T * a.k);  // most experts chosen
    // tokens of an expert whose codes the LDS holds at a time: about twice the mean, so that a CU can hold two
    // workgroups (an expert with more tokens has its weights read again, mostly from a cache)
    const bool matrix = FMT == 1 && a.T > 1;
    const int columns = matrix ? MATRIX_BATCH : DOT_BATCH;
    const size_t fixed = (size_t)columns * (a.H / G) * 8, per = a.H + 16 + 2 * G * 4;
    int batch = 4;
    while (batch < columns && batch * a.E < 2 * a.T * a.k) batch *= 2;
    while (batch > 1 && batch * per + fixed > 96 * 1024) batch /= 2;
    if (a.T == 1) batch = 1;
    const size_t lds = batch * per + fixed;
    const dim3 grid(a.I / G, slots);
    auto up = [&](auto kernel) -> hipError_t {
        const hipError_t e = lds > 16384 ? ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds) : hipSuccess;
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, grid, dim3(64 * Up<G>::WAVES), lds, stream, a, batch);
        return hipGetLastError();
    };
    auto by_experts = [&](auto m) -> hipError_t {
        constexpr bool MATRIX = decltype(m)::value;
        if (a.E <= 64) return up(moe_up_kernel<FMT, G, BF16, 1, MATRIX>);
        if (a.E <= 128) return up(moe_up_kernel<FMT, G, BF16, 2, MATRIX>);
        return up(moe_up_kernel<FMT, G, BF16, 8, MATRIX>);
    };
    hipError_t e;
    if constexpr (FMT == 1)
        e = matrix ? by_experts(std::true_type()) : by_experts(std::false_type());
    else
        e = by_experts(std::false_type());
    if (e != hipSuccess) return e;
    auto down = [&](auto kernel, int rows) -> hipError_t {
        const size_t bytes = (size_t)a.T * a.k * rows * 4;
        const hipError_t e = bytes > 16384 ? ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes) : hipSuccess;
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, dim3(a.H / rows), dim3(64 * DOWN_WAVES), bytes, stream, a);
        return hipGetLastError();
    };
    if constexpr (FMT == 1)
        if (a.T * a.k >= 2 * slots) {  // two tokens an expert: what v_dot4 costs for two, the instruction costs for any
            auto kernel = moe_down_matrix_kernel<G, BF16>;
            // scales and code sums are staged where they fit beside the sums (at most 128 KiB) and the lists of pairs;
            // up to 48 KiB
            const size_t pairs = (size_t)a.T * a.k, sums = HALVES * pairs * 16 * 4, staged = pairs * (a.I / G) * 8;
            const size_t lists = (MOST_PAIRS + MATRIX_WAVES * 64) * sizeof(int);
            const int stage = staged <= 48 * 1024 && lists + sums + staged <= CU_LDS;
            const size_t bytes = sums + (stage ? staged : 0);
            e = bytes > 16384 ? ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes) : hipSuccess;
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(kernel, dim3(a.H / 16), dim3(64 * MATRIX_WAVES), bytes, stream, a, stage);
            return hipGetLastError();
        }
    auto by_rows = [&](auto lpr) {
        constexpr int LPR = decltype(lpr)::value;
        // H is a multiple of 32
        return a.H >= 16 * 256 ? down(moe_down_kernel<FMT, G, LPR, 16, BF16>, 16)
                               : down(moe_down_kernel<FMT, G, LPR, 8, BF16>, 8);
    };
    if (slots > 4) return by_rows(std::integral_constant<int, 16>());
    if (slots > 2) return by_rows(std::integral_constant<int, 32>());
    return by_rows(std::integral_constant<int, 64>());
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t moe_q4_workspace(int T, int I, int k, int bs) {
    const size_t pairs = (size_t)T * k;
    return align256(pairs * I) + align256(pairs * (I / bs) * 8) + 2 * align256(pairs * 4) + align256((1 + pairs) * 4);
}

hipError_t launch_moe_q4(int T, int H, int I, int E, int k, int bs, int fmt, bool bf16, const void* x,
                         const float* logits, const uint8_t* w13, const void* s13, const void* b13, const uint8_t* w2,
                         const void* s2, const void* b2, bool renorm, void* y, void* work, hipStream_t stream) {
    const size_t pairs = (size_t)T * k;
    Moe a;
    a.T = T; a.H = H; a.I = I; a.E = E; a.k = k;
    a.renorm = renorm;
    a.wide = (((uintptr_t)s13 | (uintptr_t)b13 | (uintptr_t)s2 | (uintptr_t)b2) & 15) == 0;
    a.x = x;
    a.logits = logits;
    a.w13 = w13;
    a.s13 = static_cast<const uint16_t*>(s13);
    a.b13 = static_cast<const uint16_t*>(b13);
    a.w2 = w2;
    a.s2 = static_cast<const uint16_t*>(s2);
    a.b2 = static_cast<const uint16_t*>(b2);
    a.y = y;
    uint8_t* p = static_cast<uint8_t*>(work);
    const auto take = [&](size_t bytes) {
        uint8_t* at = p;
        p += align256(bytes);
        return at;
    };
    a.hq = reinterpret_cast<int8_t*>(take(pairs * I));
    a.hs = reinterpret_cast<uint2*>(take(pairs * (I / bs) * 8));
    a.sel = reinterpret_cast<int*>(take(pairs * 4));
    a.weight = reinterpret_cast<float*>(take(pairs * 4));
    a.slots = reinterpret_cast<int*>(take((1 + pairs) * 4));
    if (fmt == 0) return bf16 ? launch<0, 32, true>(a, stream) : launch<0, 32, false>(a, stream);
    if (bs == 64) return bf16 ? launch<1, 64, true>(a, stream) : launch<1, 64, false>(a, stream);
    return bf16 ? launch<1, 128, true>(a, stream) : launch<1, 128, false>(a, stream);
}

}  // namespace q4
