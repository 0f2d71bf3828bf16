// Attention over the 8-bit paged cache (kv8.h).
//
// A query row is a (token, head of the group) pair of one key/value head; a
// tile of 16 RT rows shares every key and value byte it reads. A wavefront
// works on chunks of 64 tokens with v_mfma_f32_16x16x32_f16 (for float32 results the
// second product is v_mfma_f32_16x16x32_bf16):
//   S^T = K Q^T   A = keys (rows: tokens), B = queries (columns)
//   O^T = V^T P^T A = V^T (rows: d), B = probabilities (columns: queries)
// Column r of both results belongs to lane r (mod 16), so the softmax runs
// along a lane's own registers and over the four lanes of a column. Lane
// group g (lanes 16 g ...) takes the 16 consecutive tokens 16 g ... of a chunk:
// row 4 g' + i of the t-th key tile is token 16 g' + 4 t + i, which makes a
// lane's results of the first product exactly its operand of the second (the
// order of tokens inside a sum is free), and V^T, stored [d][token], is read
// with one 16-byte load for each 16 tokens of a d. No operand passes LDS.
// Bound: the cache's bytes, read once: 64 sequences of 4096 to 16384 tokens, 8
// key/value heads of 128, 288 us, 4.7 TB/s (a large copy moves 4.77 TB/s here). A
// long sequence is cut into splits, which a second launch joins: one sequence of
// 1000 tokens 9.9 us, most of it launches and three dependent loads.
//
// Numbers. Codes are exact in f16 and bfloat16. Queries are scaled per row by a
// power of two into f16's range: bfloat16 queries are exact there (values more
// than 2^22 below the row's largest are rounded), float32 ones are split into two
// f16 halves. Products accumulate in float32. The page scales enter in float32:
// the key scale multiplies the scores, the value scale vs the probabilities, which
// are the weights of the second product. Their running reference is
//     m = max_t (s_t + max(log2 vs_t, -80)) - LOW,
// not the largest score alone: p_t = 2^(s_t - m) and the weight p_t vs_t are then
// bounded whatever the scales of other pages are, and both sums (of p_t, and of
// p_t vs_t v_t) are in units of 2^m.
// For bfloat16 results a weight is one f16: 2^-12 of itself, against 2^-9 of the
// result's rounding. LOW = 11 and a reference that lags by at most 2^4 hold the
// largest weight between 2^11 and 2^15, so that weights keep their eleven bits down
// to 2^-25 of it, and what is lost below is 2^-36 of it: where one token of small
// value takes nearly all of the weight, the result is the other tokens'. (p_t stays
// below 2^95, and a sum over 2^30 tokens finite.)
// For float32 results a weight is three bfloat16 pieces (eight bits each, cut, not
// rounded), which hold a float32 exactly at any size; there LOW = 0 and the
// reference may lag by 2^8.
#include <algorithm>
#include <type_traits>

#include "kernels_wide.h"
#include "kv8_dev.h"

namespace q4 {

namespace {

constexpr float NEG = -__builtin_inff();
constexpr int CHUNK = 64;

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// 8 codes -> 8 f16, exactly. int8: the byte + 128 under 0x64 is the f16 value
// 1024 + 128 + code.
template <int FMT>
__device__ __forceinline__ h8 codes_f16(uint32_t lo, uint32_t hi) {
    if (FMT == KV8_E4M3) {
        const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
        const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
        const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
        const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
        return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    const h2 bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    const h2 a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)) + bias;
    const h2 b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)) + bias;
    const h2 c = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)) + bias;
    const h2 d = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)) + bias;
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The upper 16 bits of two float32 values: bfloat16, the rest cut off.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// 8 codes -> 8 bfloat16, exactly (seven and four bits).
template <int FMT>
__device__ __forceinline__ b8 codes_bf16(uint32_t lo, uint32_t hi) {
    uint32_t w[4];
    if (FMT == KV8_E4M3) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = (i < 2 ? lo : hi) >> (16 * (i & 1));
            w[i] = upper_halves((float)(int8_t)(c & 0xFFu), (float)(int8_t)(c >> 8 & 0xFFu));
        }
    }
    return __builtin_bit_cast(b8, make_uint4(w[0], w[1], w[2], w[3]));
}

// The operands of the second product: f16, and one piece a weight, for bfloat16
// results; bfloat16, and three pieces a weight, for float32 ones.
template <bool WIDE>
struct Second;
template <>
struct Second<false> {
    static constexpr int PIECES = 1;
    static constexpr float LOW = 11.0f, LAG = 4.0f;  // see the head of the file
    typedef h8 Op;
    template <int FMT>
    static __device__ __forceinline__ Op values(uint32_t lo, uint32_t hi) { return codes_f16<FMT>(lo, hi); }
    static __device__ __forceinline__ void weights(const float (&w)[8], Op (&p)[PIECES]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[0][i] = (_Float16)w[i];
    }
    static __device__ __forceinline__ v4f product(Op v, Op p, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p, c, 0, 0, 0);
    }
};
template <>
struct Second<true> {
    static constexpr int PIECES = 3;
    static constexpr float LOW = 0.0f, LAG = 8.0f;
    typedef b8 Op;
    template <int FMT>
    static __device__ __forceinline__ Op values(uint32_t lo, uint32_t hi) { return codes_bf16<FMT>(lo, hi); }
    static __device__ __forceinline__ void weights(const float (&w)[8], Op (&p)[PIECES]) {
        float left[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) left[i] = w[i];
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = upper_halves(left[2 * i], left[2 * i + 1]);
            p[q] = __builtin_bit_cast(Op, make_uint4(x[0], x[1], x[2], x[3]));
            if (q + 1 < PIECES)
#pragma unroll
                for (int i = 0; i < 8; ++i) left[i] -= __uint_as_float(__float_as_uint(left[i]) & 0xFFFF0000u);  // exact
        }
    }
    static __device__ __forceinline__ v4f product(Op v, Op p, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p, c, 0, 0, 0);
    }
};

struct Attend {
    int total, max_new, max_kv, heads, group;  // group = heads / Hkv
    int window;
    int chunks_per_split, splits;
    const void* q;
    long long q_stride;
    bool q_vec;  // its rows start on 16 bytes
    float scale2;  // softmax scale * log2(e)
    void* out;
    float* lse;
    float* part_o;   // [splits][total * heads][D]
    float2* part_ml; // [splits][total * heads]
};

constexpr float LN2 = 0.6931471805599453f;

// Logarithm of a row's sum l 2^m: -infinity only for a row that sees no key (a NaN query has no maximum either, but
// its sum is NaN).
__device__ __forceinline__ float log_of_sum(float m, float l) {
    return l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
}
// Rows of a sequence and head that the first kernel takes: 40 rows over a window of 512 keys took it 12 us, the
// kernel for many rows 18 us.
constexpr int FEW_ROWS = 64;

// Query row `at` of a sequence's rows: its position, its row in the output, and
// this lane group's part as f16 under a power of two; qs is the score of a unit
// product, without the sign of the softmax scale, which the query carries. Step
// k of the first product takes d = D/4 g + 8 k ... (a lane's codes contiguous in
// memory), or with BY_STEP d = 32 k + 8 g ... (the order in LDS).
template <int D, bool WIDE, bool BY_STEP>
__device__ __forceinline__ void load_query(const Kv8& c, const Attend& a, const Kv8Span& s, int h, int at, int g,
                                           int& qpos, long long& orow, float& qs, h8 (&qf)[D / 32][WIDE ? 2 : 1]) {
    const int i = at / a.group, hh = at - i * a.group;
    qpos = s.begin + i;
    orow = (long long)(s.row0 + i) * a.heads + h * a.group + hh;
    const long long qat = (long long)(s.row0 + i) * a.q_stride + (long long)(h * a.group + hh) * D;
    float v[D / 4];
    const auto part = [&](int k) { return qat + (BY_STEP ? 32 * k + 8 * g : (D / 4) * g + 8 * k); };
    if (a.q_vec) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) load8_aligned<!WIDE>(a.q, part(k), v + 8 * k);
    } else {
#pragma unroll
        for (int j = 0; j < D / 4; ++j) v[j] = load_as_float<!WIDE>(a.q, part(j / 8) + j % 8);
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 4; ++j) amax = fmaxf(amax, fabsf(v[j]));
    amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    // 2^(8 - exponent of amax): the largest value falls in 128 .. 256
    int e;
    frexpf(amax, &e);
    e = amax > 0.0f && amax < __builtin_inff() ? 8 - e : 0;
    qs = ldexpf(fabsf(a.scale2), -e);
#pragma unroll
    for (int j = 0; j < D / 4; ++j) {
        float x = ldexpf(a.scale2 < 0.0f ? -v[j] : v[j], e);
        if (WIDE) __asm__("" : "+v"(x));
        const _Float16 hi = (_Float16)x;
        qf[j / 8][0][j % 8] = hi;
        if (WIDE) qf[j / 8][WIDE ? 1 : 0][j % 8] = (_Float16)(x - (float)hi);
    }
}

// Maximum over the four lanes of a column (r, r + 16, r + 32, r + 48). A swap of
// a register with a copy of itself leaves the even rows in one result and the
// odd ones in the other.
__device__ __forceinline__ float column_max(float v) {
    uint32_t x = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const uint32_t a0 = a[0], a1 = a[1];
    x = __float_as_uint(fmaxf(__uint_as_float(a0), __uint_as_float(a1)));
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const uint32_t b0 = b[0], b1 = b[1];
    return fmaxf(__uint_as_float(b0), __uint_as_float(b1));
}

// Moves a column's running reference m up to `top` - LOW and its sums with it, but
// only once some column of the wavefront is more than 2^LAG behind: most chunks
// leave the sums alone.
template <bool WIDE, int DT>
__device__ __forceinline__ void move_reference(float& m, float top, float& l, v4f (&o)[DT]) {
    top -= Second<WIDE>::LOW;
    if (!__any(top > m + Second<WIDE>::LAG)) return;
    const float to = fmaxf(m, top);
    const float f = __builtin_amdgcn_exp2f(m - (to == NEG ? 0.0f : to));
    m = to;
    l *= f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] *= f;
}

// FMT: format of the codes; D: head size; RT: row tiles of 16; WIDE: float32
// queries (two f16 halves) and results. The W wavefronts of a workgroup
// share its rows and take every W-th chunk. (Eight wavefronts without splits, one
// launch instead of two, were no faster for one sequence of 1000 tokens, 12.0
// against 11.0 us: a CU alone does not draw its 256 KB fast enough.)
template <int FMT, int D, int RT, bool WIDE>
__global__ __launch_bounds__(256) void kv8_attn_kernel(Kv8 c, Attend a) {
    constexpr int KS = D / 32;         // steps of the first product
    constexpr int DT = D / 16;         // row tiles of the second
    constexpr int KL = D / 64;         // 16-byte loads of a lane's part of a key
    constexpr int W = 4;
    constexpr int HALVES = WIDE ? 2 : 1;
    using S2 = Second<WIDE>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int b = blockIdx.x / c.H, h = blockIdx.x - b * c.H;
    const int split = blockIdx.y, tile = blockIdx.z;

    const Kv8Span s = kv8_span(c, b, a.total, a.max_new);
    const int rows = (s.end - s.begin) * a.group;  // rows of this sequence and head
    const int row0 = tile * (16 * RT);
    if (row0 >= rows) return;

    // chunks that some row of the tile sees
    const int lo_row = row0;
    const int hi_row = min(row0 + 16 * RT, rows) - 1;
    const int last = min(s.begin + hi_row / a.group, a.max_kv - 1);  // last position seen
    const int first = a.window > 0 ? max(0, s.begin + lo_row / a.group - a.window + 1) : 0;
    const int chunk0 = first / CHUNK;
    const int chunk_end = last >= 0 ? last / CHUNK + 1 : 0;
    const int from = chunk0 + split * a.chunks_per_split;
    const int to = min(chunk_end, from + a.chunks_per_split);
    const int pos_min = s.begin + lo_row / a.group, pos_max = s.begin + hi_row / a.group;

    const int32_t* table = c.table + (long long)b * c.max_pages;
    const int shift = 31 - __builtin_clz(c.P);
    // pages of the 16 tokens whose scores this lane holds, and of those whose keys it loads; asked for one turn ahead
    const int mine = 16 * g, mine_k = 16 * (r >> 2);
    int pg_asked = 0, kpg_asked = 0;
    const auto ask = [&](int ch) {
        pg_asked = table[min(ch * CHUNK + mine, last) >> shift];
        kpg_asked = table[min(ch * CHUNK + mine_k, last) >> shift];
    };
    if (from + wave < to) ask(from + wave);

    // this lane's query rows (one a column tile), rows past the end repeat the last
    int qpos[RT];
    long long orow[RT];
    bool live[RT];
    float qs[RT];  // score of a unit product: the row's power of two * softmax scale
    h8 qf[RT][KS][HALVES];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rho = row0 + 16 * t + r;
        live[t] = rho < rows;
        load_query<D, WIDE, false>(c, a, s, h, min(rho, rows - 1), g, qpos[t], orow[t], qs[t], qf[t]);
    }

    float m[RT], l[RT];
    v4f o[RT][DT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = NEG;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][d][e] = 0.0f;
    }

    for (int ch = from + wave; ch < to; ch += W) {
        const int base = ch * CHUNK;
        const int tok = base + mine, ktok = base + mine_k;
        const bool has = tok <= last && pg_asked >= 0 && pg_asked < c.pages;
        const int pg = has ? pg_asked : 0;
        const int kpg = ktok <= last && kpg_asked >= 0 && kpg_asked < c.pages ? kpg_asked : 0;
        ask(ch + W);

        const uint8_t* kp = c.k_codes + (((long long)kpg * c.H + h) * c.P + (ktok & (c.P - 1)) + (r & 3)) * D + (D / 4) * g;
        const uint8_t* vp = c.v_codes + ((long long)pg * c.H + h) * c.P * D + (long long)r * c.P + (tok & (c.P - 1));
        uint4 kc[4][KL];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int q = 0; q < KL; ++q) kc[t][q] = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 16 * q);
        uint4 vc[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) vc[d] = *reinterpret_cast<const uint4*>(vp + (long long)16 * d * c.P);
        const long long sat = (long long)pg * c.H + h;
        const float ks = has ? c.k_scale[sat] : 0.0f;
        const float vs = has ? c.v_scale[sat] : 0.0f;

        // S^T: 16 scores a lane and row tile
        v4f st[RT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int u = 0; u < RT; ++u) st[u][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint4 w = kc[t][k / 2];
                const h8 kf = (k & 1) ? codes_f16<FMT>(w.z, w.w) : codes_f16<FMT>(w.x, w.y);
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int q = 0; q < HALVES; ++q)
                        st[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[u][k][q], st[u][t], 0, 0, 0);
            }
        }

        // a chunk at an end of some row's range, or with a missing page, is masked
        const bool masked = base + CHUNK - 1 > min(pos_min, a.max_kv - 1) ||
                            (a.window > 0 && base <= pos_max - a.window) || __any(!has);
        if (masked) {
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int pos = tok + 4 * t + e;
                        const bool see = has && pos <= qpos[u] && pos < a.max_kv &&
                                         (a.window <= 0 || pos > qpos[u] - a.window);
                        st[u][t][e] = see ? st[u][t][e] * (ks * qs[u]) : NEG;
                    }
            // what lies behind the last token was never written: no NaN may meet a zero weight
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                uint32_t w[4] = {vc[d].x, vc[d].y, vc[d].z, vc[d].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int left = has ? last + 1 - (tok + 4 * q) : 0;  // valid bytes
                    w[q] = left >= 4 ? w[q] : left <= 0 ? 0u : w[q] & ((1u << (8 * left)) - 1u);
                }
                vc[d] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[u][t][e] *= ks * qs[u];
        }

        const float lv = fmaxf(__builtin_amdgcn_logf(vs), -80.0f);
        typename S2::Op pf[RT][2][S2::PIECES];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            float top = NEG;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, st[u][t][e]);
            top = column_max(top + lv);
            move_reference<WIDE>(m[u], top, l[u], o[u]);
            const float ref = m[u] == NEG ? 0.0f : m[u];
            float sum = 0.0f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = __builtin_amdgcn_exp2f(st[u][2 * half + j / 4][j % 4] - ref);
                    sum += p;
                    w[j] = p * vs;
                }
                S2::weights(w, pf[u][half]);
            }
            l[u] += sum;
        }

        // O^T
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const auto v0 = S2::template values<FMT>(vc[d].x, vc[d].y), v1 = S2::template values<FMT>(vc[d].z, vc[d].w);
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int q = 0; q < S2::PIECES; ++q) {
                    o[u][d] = S2::product(v0, pf[u][0][q], o[u][d]);
                    o[u][d] = S2::product(v1, pf[u][1][q], o[u][d]);
                }
        }
    }

    // sums over the lanes of a column
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        l[u] += __shfl_xor(l[u], 16, 64);
        l[u] += __shfl_xor(l[u], 32, 64);
    }

    // join the wavefronts in a fixed order
    __shared__ float ml[W][RT][16][2];
    constexpr int DH = D < 128 ? D : 128;  // columns joined at a time
    __shared__ float so[W][16][DH + 4];
    if (g == 0)
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            ml[wave][u][r][0] = m[u];
            ml[wave][u][r][1] = l[u];
        }
    __syncthreads();
    float top[RT], f[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        top[u] = ml[0][u][r][0];
#pragma unroll
        for (int w = 1; w < W; ++w) top[u] = fmaxf(top[u], ml[w][u][r][0]);
        const float ref = top[u] == NEG ? 0.0f : top[u];
        f[u] = __builtin_amdgcn_exp2f(m[u] - ref);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += ml[w][u][r][1] * __builtin_amdgcn_exp2f(ml[w][u][r][0] - ref);
        l[u] = sum;
        m[u] = top[u];
    }
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
        for (int part = 0; part < D / DH; ++part) {
            if (u + part > 0) __syncthreads();
#pragma unroll
            for (int d = 0; d < DH / 16; ++d) {
                const v4f x = o[u][part * (DH / 16) + d];
                *reinterpret_cast<float4*>(&so[wave][r][16 * d + 4 * g]) =
                    make_float4(x[0] * f[u], x[1] * f[u], x[2] * f[u], x[3] * f[u]);
            }
            __syncthreads();
            // wavefront w finishes the d tiles w, w + W, ... of this part
            for (int d = wave; d < DH / 16; d += W) {
                const int in = 16 * d + 4 * g, at = part * DH + in;
                float4 v = *reinterpret_cast<const float4*>(&so[0][r][in]);
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(&so[w][r][in]);
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                }
                if (!live[u]) continue;
                if (a.splits > 1) {
                    *reinterpret_cast<float4*>(a.part_o + ((long long)split * a.total * a.heads + orow[u]) * D + at) = v;
                } else {
                    const float inv = l[u] > 0.0f || l[u] != l[u] ? 1.0f / l[u] : 0.0f;
                    if (WIDE)
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow[u] * D + at) =
                            make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    else
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow[u] * D + at) =
                            make_uint2(bf16_pair(v.x * inv, v.y * inv), bf16_pair(v.z * inv, v.w * inv));
                }
            }
        }
    if (wave == 0 && g == 0)
#pragma unroll
        for (int u = 0; u < RT; ++u)
            if (live[u]) {
                if (a.splits > 1)
                    a.part_ml[(long long)split * a.total * a.heads + orow[u]] = make_float2(m[u], l[u]);
                else if (a.lse)
                    a.lse[orow[u]] = log_of_sum(m[u], l[u]);
            }
}

// ---- many rows ------------------------------------------------------------------------
// Prompts and chunks of prompts: bound by the matrix cores and by the softmax's
// VALU work, not by the cache's bytes, so the four wavefronts of a workgroup
// (16 RT rows each) share every chunk: it is converted to the products' 16-bit
// types once, a quarter by each wavefront, and the operands come from LDS, two
// chunks alternating. A
// thread's codes of the next chunk are loaded before the current one is used
// and converted after it.
// LDS: a key is a row of D values in 16-byte pieces, a value row (one d) has its 64
// tokens in eight, those of step 0 first. Pieces are stored at piece ^ key, where
// the key of a token is its row in the first product and that of a value row half
// its number, so that the sixteen lanes that a 16-byte read serves at once, which
// come from two lane groups, fall on different banks.
// Two chunks of 1024 tokens, 32 heads over 8, up to 4096 keys: 148 us, 0.6
// PFLOP/s. Counters: VALU 32%, matrix cores 21% of the time, the two wavefronts of
// a SIMD (244 registers each) wait for each other and for LDS in the rest.
// Scores stay unscaled in their registers: the factor ks * qs is the same for
// all 16 of a lane, so it enters as a multiply-add with the running reference.

template <int D>
struct ManyLds {
    static constexpr int K = CHUNK * D * 2, V = D * CHUNK * 2, STAGE = K + V;
};

template <int FMT, int D, int RT, bool WIDE>
__global__ __launch_bounds__(256, D == 64 || (D == 128 && !WIDE) ? 2 : 1) void kv8_many_kernel(Kv8 c, Attend a) {
    constexpr int KS = D / 32, DT = D / 16;
    constexpr int HALVES = WIDE ? 2 : 1;
    using S2 = Second<WIDE>;
    constexpr int KP = D / 16;              // 16-code pieces of a key
    constexpr int LK = CHUNK * KP / 256;    // pieces a thread loads of K, and of V
    constexpr int ROWS = 64 * RT;
    using L = ManyLds<D>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int b = blockIdx.x / c.H, h = blockIdx.x - b * c.H;
    const int split = blockIdx.y, tile = (int)(gridDim.z - 1 - blockIdx.z);  // the rows that see most first

    const Kv8Span s = kv8_span(c, b, a.total, a.max_new);
    const int rows = (s.end - s.begin) * a.group;
    if (tile * ROWS >= rows) return;
    const int row0 = tile * ROWS + wave * 16 * RT;

    int qpos[RT];
    long long orow[RT];
    bool live[RT];
    float qs[RT];
    h8 qf[RT][KS][HALVES];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rho = row0 + 16 * t + r;
        live[t] = rho < rows;
        load_query<D, WIDE, true>(c, a, s, h, min(rho, rows - 1), g, qpos[t], orow[t], qs[t], qf[t]);
    }

    // chunks that some row of the workgroup sees, and what this wavefront's rows see
    const int hi_row = min((tile + 1) * ROWS, rows) - 1;
    const int last = min(s.begin + hi_row / a.group, a.max_kv - 1);
    const int first = a.window > 0 ? max(0, s.begin + tile * ROWS / a.group - a.window + 1) : 0;
    const int chunk_end = last >= 0 ? last / CHUNK + 1 : 0;
    const int from = first / CHUNK + split * a.chunks_per_split;
    const int to = min(chunk_end, from + a.chunks_per_split);
    const int pos_min = s.begin + min(row0, rows - 1) / a.group;
    const int pos_max = s.begin + min(row0 + 16 * RT - 1, rows - 1) / a.group;

    float m[RT], l[RT];
    v4f o[RT][DT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = NEG;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int32_t* table = c.table + (long long)b * c.max_pages;
    const int shift = 31 - __builtin_clz(c.P);
    // pages of a chunk's four groups of 16 tokens, -1 where there are none. Their numbers are asked for two
    // chunks ahead and looked at one chunk ahead, when they have arrived.
    int pages[4], asked[4];
    auto ask_pages = [&](int ch) {
#pragma unroll
        for (int j = 0; j < 4; ++j) asked[j] = table[min(ch * CHUNK + 16 * j, last) >> shift];
    };
    auto take_pages = [&](int ch) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pg = __builtin_amdgcn_readfirstlane(asked[j]);
            pages[j] = ch * CHUNK + 16 * j <= last && pg >= 0 && pg < c.pages ? pg : -1;
        }
    };
    auto page_of = [&](int j) { return j == 0 ? pages[0] : j == 1 ? pages[1] : j == 2 ? pages[2] : pages[3]; };

    uint4 kraw[LK], vraw[LK];
    float ks_next, vs_next;
    bool has_next, hole_next;
    // a thread's pieces: K piece i is (token, 16 d), V piece i is (d, 16 tokens); their places in a chunk's
    // page or, where pages are smaller than a chunk, in the page of their 16 tokens
    const bool one_page = c.P >= CHUNK;
    uint32_t koff[LK], voff[LK];
#pragma unroll
    for (int i = 0; i < LK; ++i) {
        const int at = tid + 256 * i;
        const int tk = at / KP, slot = one_page ? tk : ((tk & ~15) & (c.P - 1)) + (tk & 15);
        koff[i] = slot * D + 16 * (at % KP);
        const int first_slot = 16 * (at & 3);
        voff[i] = (at >> 2) * c.P + (one_page ? first_slot : first_slot & (c.P - 1));
    }
    auto load_raw = [&](int ch) {
        const long long page_bytes = (long long)c.P * D;
        if (one_page) {
            const int slot = (ch * CHUNK) & (c.P - 1);
            const long long at = ((long long)max(pages[0], 0) * c.H + h) * page_bytes;
            const uint8_t* kp = c.k_codes + at + slot * D;
            const uint8_t* vp = c.v_codes + at + slot;
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                kraw[i] = *reinterpret_cast<const uint4*>(kp + koff[i]);
                vraw[i] = *reinterpret_cast<const uint4*>(vp + voff[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                const int at = tid + 256 * i;
                const long long kat = ((long long)max(page_of(at / KP >> 4), 0) * c.H + h) * page_bytes;
                const long long vat = ((long long)max(page_of(at & 3), 0) * c.H + h) * page_bytes;
                kraw[i] = *reinterpret_cast<const uint4*>(c.k_codes + kat + koff[i]);
                vraw[i] = *reinterpret_cast<const uint4*>(c.v_codes + vat + voff[i]);
            }
        }
        const int pg = page_of(g);
        has_next = pg >= 0;
        hole_next = pages[0] < 0 || pages[1] < 0 || pages[2] < 0 || pages[3] < 0;
        // what lies behind the last token was never written: no NaN may meet a zero weight
        if (hole_next || ch * CHUNK + CHUNK > last + 1) {
            const int grp = tid & 3;
            const int left = page_of(grp) < 0 ? 0 : last + 1 - (ch * CHUNK + 16 * grp);
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                uint32_t w[4] = {vraw[i].x, vraw[i].y, vraw[i].z, vraw[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = left - 4 * q;
                    w[q] = n >= 4 ? w[q] : n <= 0 ? 0u : w[q] & ((1u << (8 * n)) - 1u);
                }
                vraw[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        const long long sat = (long long)max(pg, 0) * c.H + h;
        ks_next = has_next ? c.k_scale[sat] : 0.0f;
        vs_next = has_next ? c.v_scale[sat] : 0.0f;
    };
    auto key_of = [&](int tk) { return ((tk >> 4) << 2) | (tk & 3); };
    auto store_chunk = [&](int buf) {
        uint8_t* kl = lds + buf * L::STAGE;
        uint8_t* vl = kl + L::K;
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const int at = tid + 256 * i;
            const int tk = at / KP, pc = at % KP;
            const int key = key_of(tk) & (2 * KP - 1);
            *reinterpret_cast<h8*>(kl + tk * (2 * D) + 16 * ((2 * pc) ^ key)) = codes_f16<FMT>(kraw[i].x, kraw[i].y);
            *reinterpret_cast<h8*>(kl + tk * (2 * D) + 16 * ((2 * pc + 1) ^ key)) = codes_f16<FMT>(kraw[i].z, kraw[i].w);
            const int d = at >> 2, grp = at & 3;
            const int vkey = (d >> 1) & 7;
            using Op = typename S2::Op;
            *reinterpret_cast<Op*>(vl + d * 128 + 16 * (grp ^ vkey)) = S2::template values<FMT>(vraw[i].x, vraw[i].y);
            *reinterpret_cast<Op*>(vl + d * 128 + 16 * ((grp + 4) ^ vkey)) = S2::template values<FMT>(vraw[i].z, vraw[i].w);
        }
    };

    if (from < to) {
        ask_pages(from);
        take_pages(from);
        load_raw(from);
        ask_pages(from + 1);
        store_chunk(0);
    }
    for (int ch = from; ch < to; ++ch) {
        const int buf = (ch - from) & 1;
        const int base = ch * CHUNK, tok = base + 16 * g;
        const float ks = ks_next, vs = vs_next;
        const bool has = has_next, hole = hole_next;
        __syncthreads();  // this chunk is in LDS, and the other buffer has been read
        if (ch + 1 < to) {
            take_pages(ch + 1);
            load_raw(ch + 1);
            ask_pages(ch + 2);
        }
        // a wavefront whose rows see nothing of the chunk only helps to load
        if (base <= pos_max && (a.window <= 0 || base + CHUNK - 1 > pos_min - a.window)) {
            const uint8_t* kl = lds + buf * L::STAGE;
            const uint8_t* vl = kl + L::K;
            v4f st[RT][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int tk = 16 * (r >> 2) + 4 * t + (r & 3);
                const uint8_t* row = kl + tk * (2 * D);
                const int key = r & (2 * KP - 1);  // key_of(tk)
#pragma unroll
                for (int u = 0; u < RT; ++u) st[u][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const h8 kf = *reinterpret_cast<const h8*>(row + 16 * ((4 * k + g) ^ key));
#pragma unroll
                    for (int u = 0; u < RT; ++u)
#pragma unroll
                        for (int q = 0; q < HALVES; ++q)
                            st[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[u][k][q], st[u][t], 0, 0, 0);
                }
            }
            const bool masked = hole || base + CHUNK - 1 > min(pos_min, a.max_kv - 1) ||
                                (a.window > 0 && base <= pos_max - a.window);
            if (masked) {
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int pos = tok + 4 * t + e;
                            const bool see = has && pos <= qpos[u] && pos < a.max_kv &&
                                             (a.window <= 0 || pos > qpos[u] - a.window);
                            st[u][t][e] = see ? st[u][t][e] : NEG;
                        }
            }
            const float lvs = __builtin_amdgcn_logf(vs), lv = fmaxf(lvs, -80.0f);
            // for bfloat16 results the value scale enters through the exponent (its logarithm is good to 2^-21, against
            // the weights' 2^-12), and the plain sum takes it out again
            float unit = WIDE ? 1.0f : __builtin_amdgcn_exp2f(-lv);
            float fac[RT], less[RT];
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                // > 0, so that a hidden score stays -infinity in a page of zeros
                fac[u] = fmaxf(ks * qs[u], 1.175494351e-38f);
                float top = NEG;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, st[u][t][e]);
                move_reference<WIDE>(m[u], column_max(fmaf(top, fac[u], lv)), l[u], o[u]);
                const float ref = m[u] == NEG ? 0.0f : m[u];
                less[u] = WIDE ? -ref : lvs - ref;
            }
            // below 2^-80 (and without a page) a score's part of the plain sum cannot be had from its weight: summed
            // by itself (148 us for the two chunks of 1024; a factor on every weight instead 151)
            if (!WIDE && __any(lvs < lv)) {
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    const float ref = m[u] == NEG ? 0.0f : m[u];
                    float sum = 0.0f;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f(fmaf(st[u][t][e], fac[u], -ref));
                    l[u] += lvs < lv ? sum : 0.0f;
                }
                unit = lvs < lv ? 0.0f : unit;
            }
            // half of the tokens at a time: the products of the first half's weights run under the
            // exponentials of the second
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                typename S2::Op pf[RT][S2::PIECES];
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    float sum = 0.0f, x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(st[u][2 * w + j / 4][j % 4], fac[u], less[u]));
                        sum += p;
                        x[j] = WIDE ? p * vs : p;
                    }
                    S2::weights(x, pf[u]);
                    l[u] = fmaf(sum, unit, l[u]);
                }
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const auto v = *reinterpret_cast<const typename S2::Op*>(vl + (16 * d + r) * 128 + 16 * ((g + 4 * w) ^ (r >> 1)));
#pragma unroll
                    for (int u = 0; u < RT; ++u)
#pragma unroll
                        for (int q = 0; q < S2::PIECES; ++q) o[u][d] = S2::product(v, pf[u][q], o[u][d]);
                }
            }
        }
        if (ch + 1 < to) store_chunk(buf ^ 1);
    }

#pragma unroll
    for (int u = 0; u < RT; ++u) {
        l[u] += __shfl_xor(l[u], 16, 64);
        l[u] += __shfl_xor(l[u], 32, 64);
        if (!live[u]) continue;
        const float inv = a.splits > 1 ? 1.0f : (l[u] > 0.0f || l[u] != l[u] ? 1.0f / l[u] : 0.0f);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const int at = 16 * d + 4 * g;
            const float4 v = make_float4(o[u][d][0] * inv, o[u][d][1] * inv, o[u][d][2] * inv, o[u][d][3] * inv);
            if (a.splits > 1)
                *reinterpret_cast<float4*>(a.part_o + ((long long)split * a.total * a.heads + orow[u]) * D + at) = v;
            else if (WIDE)
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow[u] * D + at) = v;
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow[u] * D + at) =
                    make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
        }
        if (g == 0) {
            if (a.splits > 1)
                a.part_ml[(long long)split * a.total * a.heads + orow[u]] = make_float2(m[u], l[u]);
            else if (a.lse)
                a.lse[orow[u]] = log_of_sum(m[u], l[u]);
        }
    }
}

// Joins the splits of a row: one wavefront a row, whose lanes first hold the
// splits' factors (at most 64 of them), then sum the parts in split order.
constexpr int MOST_SPLITS = 64;

template <int D, bool WIDE>
__global__ __launch_bounds__(256) void kv8_join_kernel(Attend a) {
    const int lane = threadIdx.x & 63;
    const long long rows = (long long)a.total * a.heads;
    for (long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += 4LL * gridDim.x) {
        const float2 ml = lane < a.splits ? a.part_ml[lane * rows + row] : make_float2(NEG, 0.0f);
        float top = ml.x;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        const float f = __builtin_amdgcn_exp2f(ml.x - (top == NEG ? 0.0f : top));  // 0 for a split that saw nothing
        const float l = wave_sum(ml.y * f);
        constexpr int E = D / 64;
        float v[E] = {};
        const float* p = a.part_o + row * D + E * lane;
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float fs = __shfl(f, s, 64);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = fmaf(p[s * rows * D + e], fs, v[e]);
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (WIDE)
                static_cast<float*>(a.out)[row * D + E * lane + e] = v[e] * inv;
            else
                static_cast<uint16_t*>(a.out)[row * D + E * lane + e] = (uint16_t)bf16_bits(v[e] * inv);
        }
        if (a.lse && lane == 0) a.lse[row] = log_of_sum(top, l);
    }
}

struct Plan {
    int rt;
    bool share;
    int tiles, splits, chunks_per_split;
    int most_splits;  // of any window
};

// How a call is cut: from the sizes alone, so that the workspace is known
// before the launch. (std::min: HIP's own min for the host takes two ints.)
Plan plan_of(int B, int H, int D, int group, int max_new, int max_kv, int window) {
    Plan p;
    const long long rows = (long long)max_new * group;
    p.share = rows <= FEW_ROWS;
    p.rt = rows <= 16 || D == 256 ? 1 : 2;
    const int tile = (p.share ? 16 : 64) * p.rt;
    p.tiles = (int)((rows + tile - 1) / tile);
    // chunks that a row tile can see
    long long span = max_kv;
    if (window > 0) span = std::min(span, (long long)window + tile / group + 1);
    const int chunks = (int)((span + CHUNK - 1) / CHUNK) + (window > 0 ? 1 : 0);
    const long long wgs = (long long)p.tiles * H * B;
    // enough workgroups for the chip (three a CU for the memory-bound kernel, two for the other), no split below
    // two chunks (few rows: one sequence of 1000 tokens took 11 us with two or four, 13 with one) or eight
    const int least = p.share ? 2 : 8;
    const long long fill = std::min(p.share ? (768 + wgs - 1) / wgs : wgs < 256 ? (512 + wgs - 1) / wgs : 1LL, (long long)MOST_SPLITS);
    const long long want = std::max(1LL, std::min(fill, (long long)(chunks + least - 1) / least));
    const long long all = (max_kv + CHUNK - 1) / CHUNK + 1;
    p.most_splits = (int)std::max(1LL, std::min(fill, (all + least - 1) / least));
    p.chunks_per_split = (int)((chunks + want - 1) / want);
    p.splits = (chunks + p.chunks_per_split - 1) / p.chunks_per_split;
    return p;
}

template <int FMT, int D, bool WIDE>
hipError_t launch_attn(const Kv8& c, const Attend& a, const Plan& p, hipStream_t stream) {
    const dim3 grid(c.B * c.H, p.splits, p.tiles);
    hipError_t e = hipSuccess;
    auto go = [&](auto kernel, size_t lds) {
        if (lds) e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL(kernel, grid, dim3(256), lds, stream, c, a);
        e = hipGetLastError();
    };
    constexpr int MOST = D == 256 ? 1 : 2;  // row tiles of a wavefront
    if (!p.share)
        go(kv8_many_kernel<FMT, D, MOST, WIDE>, 2 * ManyLds<D>::STAGE);
    else if (p.rt == 1)
        go(kv8_attn_kernel<FMT, D, 1, WIDE>, 0);
    else
        go(kv8_attn_kernel<FMT, D, MOST, WIDE>, 0);
    if (e != hipSuccess || p.splits == 1) return e;
    const long long rows = (long long)a.total * a.heads;
    hipLaunchKernelGGL((kv8_join_kernel<D, WIDE>), dim3((unsigned)std::min((rows + 3) / 4, 1LL << 20)), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t kv8_attn_work_bytes(const Kv8& c, int total, int max_new, int max_kv, int heads) {
    const Plan p = plan_of(c.B, c.H, c.D, heads / c.H, max_new, max_kv, 0);
    const size_t rows = (size_t)p.most_splits * total * heads;
    return p.most_splits == 1 ? 256 : align256(rows * c.D * 4) + align256(rows * 8);
}

hipError_t launch_kv8_attention(const Kv8& c, int format, int total, int max_new, int max_kv, int heads, bool bf16,
                                const void* q, long long q_stride, float scale, int window, void* out, float* lse,
                                void* work, hipStream_t stream) {
    // positions lie below 2^30, so a longer window hides nothing; the kernels subtract it from positions in 32 bits
    if (window >= 1 << 30) window = 0;
    const Plan p = plan_of(c.B, c.H, c.D, heads / c.H, max_new, max_kv, window);
    Attend a;
    a.total = total;
    a.max_new = max_new;
    a.max_kv = max_kv;
    a.heads = heads;
    a.group = heads / c.H;
    a.window = window;
    a.chunks_per_split = p.chunks_per_split;
    a.splits = p.splits;
    a.q = q;
    a.q_stride = q_stride;
    a.q_vec = ((uintptr_t)q & 15) == 0 && (q_stride * (bf16 ? 2 : 4)) % 16 == 0;
    a.scale2 = scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float*>(work);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(work) +
                                          align256((size_t)p.splits * total * heads * c.D * 4));
    auto by_type = [&](auto fmt, auto d) {
        return bf16 ? launch_attn<decltype(fmt)::value, decltype(d)::value, false>(c, a, p, stream)
                    : launch_attn<decltype(fmt)::value, decltype(d)::value, true>(c, a, p, stream);
    };
    auto by_size = [&](auto fmt) {
        switch (c.D) {
            case 64: return by_type(fmt, std::integral_constant<int, 64>());
            case 128: return by_type(fmt, std::integral_constant<int, 128>());
            case 256: return by_type(fmt, std::integral_constant<int, 256>());
            default: return hipErrorInvalidValue;
        }
    };
    return format == KV8_INT8 ? by_size(std::integral_constant<int, KV8_INT8>())
                              : by_size(std::integral_constant<int, KV8_E4M3>());
}

}  // namespace q4
