// Product of e4m3 codes with a float32 scale for each block of 128:
//     y[m][n] = sum_b xs[b][m] * as(b, n) * (sum_{k in b} a[n][k] * x[m][k])
// as(b, n) is ws[n / 128][b] for weights scaled per 128 x 128 block and
// ats[b][n] for an operand scaled per row (the weight gradient, where both
// operands are activations cut along the tokens).
//
// The inner sum of a block is a matrix-core product into a zero accumulator
// (v_mfma_f32_16x16x128_f8f6f4: one a block), the outer sum a float32
// multiply-add on the VALU. The operand whose rows are n takes the A
// side, the rows m the B side: a lane of the result then holds one m and four
// n, so a block's factor xs * ws is one value a lane, and four
// consecutive n leave in one store. Both operands have k contiguous and give
// a lane the same 32 bytes of k, so the order of k inside a block, which the
// sum does not depend on, never has to match the instruction's.
//
// Precision. The 8-bit matrix instructions add a block's products with about
// 16 bits below the largest one (measured on e4m3 codes: relative RMS 1.6e-5
// for normal codes, 6e-5 where the codes of a block span seventeen powers of
// two; the same for 32x32x64, 16x16x128 and 16x16x32). That is far below the
// rounding of a bfloat16 result, so results in bfloat16 take them. Results in
// float32 (EXACT) take the f16 instructions instead: e4m3 values are exact in
// f16, the products exact in float32, and the measured error is 1e-8 to 6e-8,
// at half the matrix rate and one conversion for two codes.
#include "f8.h"
#include "kernels_wide.h"
#include "wide.h"

namespace q4 {

namespace {

__device__ __forceinline__ v8i join(uint4 a, uint4 b) {
    v8i v = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    return v;
}

// 8 codes -> 8 f16, exactly.
__device__ __forceinline__ h8 widen(uint32_t lo, uint32_t hi) {
    const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 codes as a matrix operand: themselves, or four times 8 f16.
template <bool EXACT>
struct Operand;
template <>
struct Operand<false> {
    v8i v;
    __device__ __forceinline__ void set(uint4 a, uint4 b) { v = join(a, b); }
};
template <>
struct Operand<true> {
    h8 v[4];
    __device__ __forceinline__ void set(uint4 a, uint4 b) {
        v[0] = widen(a.x, a.y);
        v[1] = widen(a.z, a.w);
        v[2] = widen(b.x, b.y);
        v[3] = widen(b.z, b.w);
    }
};
__device__ __forceinline__ v4f product16(const Operand<false>& a, const Operand<false>& b, v4f c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v4f product16(const Operand<true>& a, const Operand<true>& b, v4f c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

// Tile of a workgroup. Workgroups go to the eight XCDs in turn, each with its
// own L2: an XCD takes a contiguous run of tiles, and a run walks down bands of
// eight tile rows, so that the workgroups that an XCD has at once share rows
// of both operands.
__device__ __forceinline__ void tile_of(int id, int tiles_n, int tiles_m, int& tile_n, int& tile_m) {
    const int total = tiles_n * tiles_m, per = total / 8, more = total % 8;
    const int x = id % 8, i = id / 8;
    const int at = x * per + min(x, more) + i;
    constexpr int BAND = 8;
    const int band = at / (BAND * tiles_n), in = at - band * BAND * tiles_n;
    const int high = min(BAND, tiles_m - band * BAND);
    tile_n = in / high;
    tile_m = band * BAND + in - tile_n * high;
}

// Four consecutive outputs of a row.
template <bool YBF16>
__device__ __forceinline__ void store4(void* y, long long at, int left, bool vec, float a, float b, float c, float d) {
    if (left <= 0) return;
    if (YBF16) {
        uint16_t* p = static_cast<uint16_t*>(y) + at;
        if (vec) {
            *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(a, b), bf16_pair(c, d));
            return;
        }
        p[0] = (uint16_t)bf16_bits(a);
        if (left > 1) p[1] = (uint16_t)bf16_bits(b);
        if (left > 2) p[2] = (uint16_t)bf16_bits(c);
        if (left > 3) p[3] = (uint16_t)bf16_bits(d);
    } else {
        float* p = static_cast<float*>(y) + at;
        if (vec) {
            *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
            return;
        }
        p[0] = a;
        if (left > 1) p[1] = b;
        if (left > 2) p[2] = c;
        if (left > 3) p[3] = d;
    }
}

// ---- tiles ------------------------------------------------------------------------
// A workgroup computes TN x TM outputs; a stage is one block of 128 k: TN + TM
// rows of 128 bytes and their scales in LDS, written by the buffer loads
// themselves (16 bytes a lane). A row's eight 16-byte pieces are stored at
// piece ^ (row / 2 & 7), and lane group g takes pieces g and g + 4: the sixteen
// lanes that a 16-byte read serves at once, which come from two lane groups, then
// fall on different banks. Rows past the end repeat the last one and are not stored.
// NS stages are kept, NS - 1 of them being filled while one is used. Loads past
// the last block repeat it, which keeps their number, and with it the wait, the
// same in every turn.
// The small 16x16 result keeps few products waiting for their multiply-add, so
// that the sums of a wavefront (128 registers at the large tile) fit beside
// them, and lets the multiply-adds of one product run under the next one's
// matrix instruction.
// Bound: the matrix cores and the four multiply-adds that each product needs on
// the VALU (half its time). 4096 x 4096 x 14336: 260 us, 1.85 PFLOP/s, 79% of what
// a library product with one scale for each whole operand reaches here (207 us);
// 1040 us before the products were shrunk to 16x16 and the loads left in flight.
template <int WN, int WM, int FN, int FM, int NS, bool AROW>
struct Tile {
    static constexpr int WAVES = WN * WM, NT = 64 * WAVES;
    static constexpr int TN = WN * FN * 16, TM = WM * FM * 16;
    static constexpr int CODES = (TN + TM) * 128;
    static constexpr int SEGMENTS = TM / 64 + (AROW ? TN / 64 : 1);  // of 64 scales, one a wavefront
    static constexpr int STAGE = CODES + (SEGMENTS * 256 + 1023) / 1024 * 1024;
    static constexpr size_t LDS = (size_t)NS * STAGE;
    static_assert(LDS <= 160 * 1024, "LDS of a CU");
    static constexpr int LA = TN / 8 / WAVES, LX = TM / 8 / WAVES;  // load instructions of a wavefront: 8 rows each
    static_assert(SEGMENTS <= WAVES, "one segment of scales a wavefront");
    static_assert((NS - 2) * (LA + LX + 1) < 64, "loads in flight are counted in six bits");
};

template <int WN, int WM, int FN, int FM, int NS, bool AROW, bool YBF16>
__global__ __launch_bounds__(64 * WN* WM) void f8_tile_kernel(int M, int N, int KB, const uint8_t* __restrict__ xq,
                                                              const float* __restrict__ xs,
                                                              const uint8_t* __restrict__ aq,
                                                              const float* __restrict__ as, void* __restrict__ y,
                                                              int tiles_n, int tiles_m) {
    using T = Tile<WN, WM, FN, FM, NS, AROW>;
    constexpr int TN = T::TN, TM = T::TM, LA = T::LA, LX = T::LX;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];  // NS stages

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    int tile_n, tile_m;
    tile_of(blockIdx.x, tiles_n, tiles_m, tile_n, tile_m);
    const int n0 = tile_n * TN, m0 = tile_m * TM;
    const int Kp = KB * 128;

    const int rows_n = min(TN, N - n0), rows_m = min(TM, M - m0);
    const v4i ra = resource(aq + (long long)n0 * Kp, (uint32_t)rows_n * Kp);
    const v4i rx = resource(xq + (long long)m0 * Kp, (uint32_t)rows_m * Kp);
    // lane -> (row of eight, piece); the piece follows the row's number in sixteen
    const int lr = lane >> 3;
    auto piece = [&](int instruction) { return 16 * ((lane & 7) ^ ((8 * (instruction & 1) + lr) >> 1)); };
    uint32_t off_a[LA], off_x[LX];
#pragma unroll
    for (int i = 0; i < LA; ++i) off_a[i] = (uint32_t)min((wave * LA + i) * 8 + lr, rows_n - 1) * Kp + piece(wave * LA + i);
#pragma unroll
    for (int i = 0; i < LX; ++i) off_x[i] = (uint32_t)min((wave * LX + i) * 8 + lr, rows_m - 1) * Kp + piece(wave * LX + i);
    // this wavefront's 64 scales: of x rows, then of the A side's rows or blocks
    const int seg = wave % T::SEGMENTS, aseg = seg - TM / 64;
    const int nblk = (N + 127) / 128;
    const bool of_x = aseg < 0;
    const v4i rs = of_x ? resource(xs, (uint32_t)(KB * M) * 4) : resource(as, (uint32_t)(KB * (AROW ? N : nblk)) * 4);
    const uint32_t off_s = 4u * (of_x ? m0 + min(seg * 64 + lane, rows_m - 1)
                                      : AROW ? n0 + min(aseg * 64 + lane, rows_n - 1)
                                             : min(n0 / 128 + min(lane, (TN + 127) / 128 - 1), nblk - 1) * KB);
    const uint32_t step_s = 4u * (of_x ? M : AROW ? N : 1);

    const uint32_t lds0 = lds_address(lds);
    auto load_stage = [&](int kb, int buf) {
        const uint32_t base = lds0 + buf * T::STAGE;
#pragma unroll
        for (int i = 0; i < LA; ++i) load_to_lds16(ra, base + (wave * LA + i) * 1024, off_a[i], kb * 128);
#pragma unroll
        for (int i = 0; i < LX; ++i) load_to_lds16(rx, base + TN * 128 + (wave * LX + i) * 1024, off_x[i], kb * 128);
        load_to_lds4(rs, base + T::CODES + seg * 256, off_s, kb * step_s);
    };

    v4f acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const int r = lane & 15, g = lane >> 4;
    const int at0 = 16 * (g ^ (r >> 1)), at1 = 16 * ((g + 4) ^ (r >> 1));
    auto use_stage = [&](const uint8_t* base) {
        const uint8_t* la = base + (wn * FN * 16 + r) * 128;
        const uint8_t* lx = base + TN * 128 + (wm * FM * 16 + r) * 128;
        const float* sc = reinterpret_cast<const float*>(base + T::CODES);
        Operand<!YBF16> b[FM];
        float sx[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            b[j].set(*reinterpret_cast<const uint4*>(lx + j * 2048 + at0),
                     *reinterpret_cast<const uint4*>(lx + j * 2048 + at1));
            sx[j] = sc[wm * FM * 16 + 16 * j + r];
            if (!AROW) sx[j] *= sc[TM + wn * FN * 16 / 128];
        }
        // one row tile at a time, the next one's operand being read meanwhile; the scheduler may not
        // gather the reads of several, whose registers would not fit beside the sums
        uint4 raw[2][2];
        raw[0][0] = *reinterpret_cast<const uint4*>(la + at0);
        raw[0][1] = *reinterpret_cast<const uint4*>(la + at1);
        v4f p[2][FM];
#pragma unroll
        for (int i = 0; i <= FN; ++i) {
            if (i + 1 < FN) {
                raw[(i + 1) & 1][0] = *reinterpret_cast<const uint4*>(la + (i + 1) * 2048 + at0);
                raw[(i + 1) & 1][1] = *reinterpret_cast<const uint4*>(la + (i + 1) * 2048 + at1);
            }
            if (i < FN) {
                Operand<!YBF16> a;
                a.set(raw[i & 1][0], raw[i & 1][1]);
#pragma unroll
                for (int j = 0; j < FM; ++j) p[i & 1][j] = product16(a, b[j], v4f{0.0f, 0.0f, 0.0f, 0.0f});
            }
            if (i > 0) {
                const int q = i - 1;
                float4 sa;
                if (AROW) sa = *reinterpret_cast<const float4*>(sc + TM + (wn * FN + q) * 16 + 4 * g);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const v4f d = p[q & 1][j];
                    acc[q][j][0] = fmaf(d[0], AROW ? sx[j] * sa.x : sx[j], acc[q][j][0]);
                    acc[q][j][1] = fmaf(d[1], AROW ? sx[j] * sa.y : sx[j], acc[q][j][1]);
                    acc[q][j][2] = fmaf(d[2], AROW ? sx[j] * sa.z : sx[j], acc[q][j][2]);
                    acc[q][j][3] = fmaf(d[3], AROW ? sx[j] * sa.w : sx[j], acc[q][j][3]);
                    __asm__ volatile("" : "+v"(acc[q][j]));  // here, not behind the last product
                }
            }
            // order: the reads, then a product and the multiply-adds of an earlier one in turn
            if (i > 0 && i < FN && YBF16) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, AROW ? 8 : 4, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

#pragma unroll
    for (int u = 0; u < NS - 1; ++u) load_stage(min(u, KB - 1), u);
    for (int kb = 0; kb < KB; kb += NS) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            if (kb + u >= KB) break;
            // stage kb + u has landed in every wavefront, and all have read the one before, which is filled again
            join_with_loads_left<(NS - 2) * (LA + LX + 1)>();
            load_stage(min(kb + u + NS - 1, KB - 1), (u + NS - 1) % NS);
            use_stage(lds + u * T::STAGE);
        }
    }
    join_with_loads_left<0>();  // no load may outlive the workgroup's LDS

    const bool vec = N % 4 == 0;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = m0 + (wm * FM + j) * 16 + r;
        if (m >= M) continue;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int n = n0 + (wn * FN + i) * 16 + 4 * g;
            store4<YBF16>(y, (long long)m * N + n, N - n, vec, acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
    }
}

// ---- few rows ---------------------------------------------------------------------
// Up to 64 rows of x: bound by the weights' bytes. A workgroup takes 16 weight
// rows, its wavefronts every WAVES-th block of k; the codes go from memory to
// the operand registers (32 bytes a lane), CT column tiles of 16 rows of x
// share them, and the wavefronts' sums are added in LDS in a fixed order.
// QUANT: x itself comes in, and every workgroup quantizes it into LDS while
// its first weights are on their way (one launch; taken for a few rows only,
// since each workgroup repeats it).
// 1 x 4096 x 4096 with the quantization inside: 6.0 us a call, 2.8 TB/s, weights
// in the last-level cache (a kernel that only reads 16.8 MB takes 3.0 us there and
// 3.9 from memory). 16 rows 9.1 us, 64 rows 14.5, both with the quantizer's launch.
constexpr int ROWS_WAVES = 8;
constexpr int ROWS_U = 4;  // blocks of k whose weights a wavefront has in flight

template <int CT, bool YBF16, bool QUANT, bool XBF16>
__global__ __launch_bounds__(64 * ROWS_WAVES) void f8_rows_kernel(int M, int N, int K, int KB,
                                                                  const void* __restrict__ x, long long stride,
                                                                  const uint8_t* __restrict__ xq,
                                                                  const float* __restrict__ xs,
                                                                  const uint8_t* __restrict__ wq,
                                                                  const float* __restrict__ ws,
                                                                  void* __restrict__ y) {
    constexpr int NT = 64 * ROWS_WAVES;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int Kp = KB * 128;
    float* sums = reinterpret_cast<float*>(lds);  // [WAVES][CT][16 m][16 n]
    uint8_t* xq_l = lds + ROWS_WAVES * CT * 1024;                         // QUANT: [M][Kp]
    float* xs_l = reinterpret_cast<float*>(xq_l + (QUANT ? M * Kp : 0));  // QUANT: [KB][M]

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int rows = min(16, N - n0);
    const __amdgpu_buffer_rsrc_t rw = buffer_of(wq + (long long)n0 * Kp, (uint32_t)rows * Kp);
    const float* wsr = ws + (long long)(n0 / 128) * KB;
    const uint32_t woff = (uint32_t)min(r, rows - 1) * Kp + 32 * g;

    uint4 w[ROWS_U][2];
    auto load_w = [&](int kb0) {
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u) {
            const uint32_t at = woff + (uint32_t)min(kb0 + u * ROWS_WAVES, KB - 1) * 128;
            w[u][0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rw, at, 0, 2));
            w[u][1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rw, at + 16, 0, 2));
        }
    };
    load_w(wave);

    if (QUANT) {
        // 16 lanes a block of 128, 8 values a lane
        const int items = M * KB * 16;
        for (int t0 = 0; t0 < items; t0 += NT) {
            const int t = t0 + tid;
            const int blk = min(t >> 4, M * KB - 1);
            const int m = blk / KB, b = blk - m * KB;
            const int k0 = 128 * b + 8 * (t & 15);
            float v[8] = {};
            if (k0 < K) load8_aligned<XBF16>(x, m * stride + k0, v);
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
            amax = row_max16(amax);
            const float s = amax / F8_TOP;
            const float inv = f8_inverse(s);
            if (t < items) {
                *reinterpret_cast<uint2*>(xq_l + m * Kp + k0) = make_uint2(f8_codes4(v, s, inv), f8_codes4(v + 4, s, inv));
                if ((t & 15) == 0) xs_l[b * M + m] = s;
            }
        }
        __syncthreads();
    }

    v4f acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][e] = 0.0f;

    for (int kb0 = wave; kb0 < KB; kb0 += ROWS_U * ROWS_WAVES) {
        if (kb0 != wave) load_w(kb0);
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u) {
            const int kb = kb0 + u * ROWS_WAVES;
            if (kb >= KB) break;
            const float sw = wsr[kb];
            Operand<!YBF16> a;
            a.set(w[u][0], w[u][1]);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int m = min(16 * c + r, M - 1);
                const uint8_t* p = (QUANT ? xq_l + m * Kp : xq + (long long)m * Kp) + kb * 128 + 32 * g;
                Operand<!YBF16> b;
                b.set(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 16));
                const float s = (QUANT ? xs_l[kb * M + m] : xs[(long long)kb * M + m]) * sw;
                v4f d = {};
                d = product16(a, b, d);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[c][e] = fmaf(d[e], s, acc[c][e]);
            }
        }
    }

#pragma unroll
    for (int c = 0; c < CT; ++c)
        *reinterpret_cast<float4*>(sums + ((wave * CT + c) * 16 + r) * 16 + 4 * g) =
            make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
    __syncthreads();
    const bool vec = N % 4 == 0;
    for (int t = tid; t < CT * 64; t += NT) {
        const int m = t >> 2, q = t & 3;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < ROWS_WAVES; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(sums + (i * CT * 16 + m) * 16 + 4 * q);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        if (m < M)
            store4<YBF16>(y, (long long)m * N + n0 + 4 * q, N - n0 - 4 * q, vec, s.x, s.y, s.z, s.w);
    }
}

template <bool YBF16, bool QUANT, bool XBF16>
hipError_t launch_rows(int M, int N, int K, int KB, const void* x, long long stride, const uint8_t* xq,
                       const float* xs, const uint8_t* wq, const float* ws, void* y, hipStream_t stream) {
    const int ct = (M + 15) / 16;
    const dim3 grid((N + 15) / 16);
    auto go = [&](auto kernel, int c) -> hipError_t {
        const size_t lds = (size_t)ROWS_WAVES * c * 1024 + (QUANT ? (size_t)M * KB * 132 : 0);
        const hipError_t e = lds > 65536 ? ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds) : hipSuccess;
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, grid, dim3(64 * ROWS_WAVES), lds, stream, M, N, K, KB, x, stride, xq, xs, wq, ws, y);
        return hipGetLastError();
    };
    if (QUANT || ct == 1) return go(f8_rows_kernel<1, YBF16, QUANT, XBF16>, 1);
    if constexpr (!QUANT) {
        if (ct == 2) return go(f8_rows_kernel<2, YBF16, false, XBF16>, 2);
        return go(f8_rows_kernel<4, YBF16, false, XBF16>, 4);
    }
    return hipErrorInvalidValue;
}

template <int WN, int WM, int FN, int FM, int NS, bool AROW, bool YBF16>
hipError_t launch_tile(int M, int N, int KB, const uint8_t* xq, const float* xs, const uint8_t* aq, const float* as,
                       void* y, hipStream_t stream) {
    using T = Tile<WN, WM, FN, FM, NS, AROW>;
    auto kernel = f8_tile_kernel<WN, WM, FN, FM, NS, AROW, YBF16>;
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), T::LDS);
    if (e != hipSuccess) return e;
    const int tn = (N + T::TN - 1) / T::TN, tm = (M + T::TM - 1) / T::TM;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long long)tn * tm)), dim3(T::NT), T::LDS, stream, M, N, KB, xq, xs, aq,
                       as, y, tn, tm);
    return hipGetLastError();
}

template <bool AROW, bool YBF16>
hipError_t launch_tiles(int M, int N, int KB, const uint8_t* xq, const float* xs, const uint8_t* aq, const float* as,
                        void* y, hipStream_t stream) {
    // The largest tile that still gives every CU work: 256 x 256 moves the fewest bytes a product (4096 x 4096 x
    // 14336: 260 us), 128 x 128 fills the chip from 200 tiles on (1024 x 4096 x 4096: 25 us, against 34 with four
    // wavefronts a tile), 64 x 64 serves the rest (515 x 1500 x 1000 in float32: 7.7 us, against 15 with 128 x 128).
    // The large and the middle tile take a CU's LDS, so 257 tiles are two waves of workgroups: 4096 x 4096 x 4096 (256
    // tiles, quantizer included) 83 us, x 4352 (272 tiles) 128 us. The rule does not look at that.
    auto tiles = [&](long long tn, long long tm) { return ((N + tn - 1) / tn) * ((M + tm - 1) / tm); };
    // float32 results hold their operands as f16, twice the registers: no large tile
    if constexpr (YBF16)
        if (tiles(256, 256) >= 256)
            return launch_tile<2, 4, 8, 4, 2, AROW, YBF16>(M, N, KB, xq, xs, aq, as, y, stream);
    if (tiles(128, 128) >= 200)
        return launch_tile<2, 4, 4, 2, 4, AROW, YBF16>(M, N, KB, xq, xs, aq, as, y, stream);
    return launch_tile<2, 2, 2, 2, 4, AROW, YBF16>(M, N, KB, xq, xs, aq, as, y, stream);
}

}  // namespace

constexpr int F8_ROWS_MOST = 64;       // rows of x that the few-row kernel takes: four column tiles of 16
constexpr int F8_FUSED_ROWS = 4;       // rows whose quantization every workgroup repeats,
constexpr int F8_FUSED_BYTES = 65536;  // and values, which its LDS holds as codes

bool f8_linear_fused(int M, int K, bool bf16, const void* x, long long stride) {
    const int size = bf16 ? 2 : 4;
    return M <= F8_FUSED_ROWS && (long long)M * K <= F8_FUSED_BYTES && K % 8 == 0 && (stride * size) % 16 == 0 &&
           ((uintptr_t)x & 15) == 0;
}

hipError_t launch_f8_gemm(int M, int N, int KB, bool ybf16, const uint8_t* xq, const float* xs, const uint8_t* wq,
                          const float* ws, void* y, hipStream_t stream) {
    if (M <= F8_ROWS_MOST)
        return ybf16 ? launch_rows<true, false, true>(M, N, 0, KB, nullptr, 0, xq, xs, wq, ws, y, stream)
                     : launch_rows<false, false, true>(M, N, 0, KB, nullptr, 0, xq, xs, wq, ws, y, stream);
    return ybf16 ? launch_tiles<false, true>(M, N, KB, xq, xs, wq, ws, y, stream)
                 : launch_tiles<false, false>(M, N, KB, xq, xs, wq, ws, y, stream);
}

hipError_t launch_f8_linear_fused(int M, int K, int N, bool bf16, const void* x, long long stride, const uint8_t* wq,
                                  const float* ws, void* y, hipStream_t stream) {
    const int KB = (K + 127) / 128;
    return bf16 ? launch_rows<true, true, true>(M, N, K, KB, x, stride, nullptr, nullptr, wq, ws, y, stream)
                : launch_rows<false, true, false>(M, N, K, KB, x, stride, nullptr, nullptr, wq, ws, y, stream);
}

hipError_t launch_f8_gemm_rowscales(int M, int N, int KB, bool ybf16, const uint8_t* xq, const float* xs,
                                    const uint8_t* aq, const float* as, void* y, hipStream_t stream) {
    return ybf16 ? launch_tiles<true, true>(M, N, KB, xq, xs, aq, as, y, stream)
                 : launch_tiles<true, false>(M, N, KB, xq, xs, aq, as, y, stream);
}

}  // namespace q4
