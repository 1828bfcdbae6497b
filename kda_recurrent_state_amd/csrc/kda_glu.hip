// kda_glu.hip -- the gated half of a feed-forward block and its gradient:
//   g = x Wg^T, u = x Wu^T, h = act(g) u                         (x [T, D], W [F, D])
//   dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x.
// Three products of matrices on the matrix cores, with what surrounds them in their epilogues.
//
// bf16 operands are read where they lie.  fp32 operands are first split into three bf16 planes whose sum they
// are (24 bits), and the product runs over the six pairs of planes above 2^-24, smallest first, into
// the same accumulators.  Six products at the peak of 2.5 PFLOP/s are 2.7 times the fp32 matrix instructions' 157 TFLOP/s;
// measured are 94 TFLOP/s of fp32 products at 777 x 1000 x 2731, where a library's fp32 product makes 74, and 149 at
// 1024 x 4096 x 10240 for the library's 144.
#include "kda_glu.hpp"

#include "kda_rows.hpp"

namespace kda {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- activations

// act(z) and its slope.  sigmoid(-z) is formed by itself: 1 - sigmoid(z) would lose it for large z.
template <int ACT> __device__ __forceinline__ void activation(float z, float& a, float& slope) {
    if constexpr (ACT == GLU_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678118654752f * z);
        a = z * cdf;
        slope = cdf + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    } else {
        const float e = __expf(-fabsf(z)), big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
        const float s = z >= 0.f ? big : small, sn = z >= 0.f ? small : big;
        if constexpr (ACT == GLU_SILU) {
            a = z * s;
            slope = s * (1.f + z * sn);
        } else {
            a = s;
            slope = s * sn;
        }
    }
}
template <int ACT> __device__ __forceinline__ float gated(float g, float u) {
    float a, slope;
    activation<ACT>(g, a, slope);
    return a * u;
}

// ---------------------------------------------------------------- tiled product
//
// out[m][n] = sum over segments s and k of A_s[m][k] B_s[n][k].  An operand is either stored with k
// contiguous (KR false: [rows][k]) or with k along the rows (KR true: [k][rows]); k is a multiple of 64 in the
// first form, and there are a multiple of 64 columns in the second.  Rows past the last are the last again, and their
// results are not stored; k rows past the last meet zeros of the other operand.

constexpr int KI = 32;    // k of a matrix instruction
constexpr int PAD = 64;   // what k and padded columns are a multiple of
constexpr int MAX_SEGS = 12;

struct Segment { const bf16 *a, *b, *b2; };
struct GemmArgs {
    Segment seg[MAX_SEGS];
    int64_t lda, ldb;          // elements between rows
    int64_t M, N;              // rows of A and B (of each of the two B where there are two)
    int64_t kA, kB, colsA, colsB;  // k rows that exist, and their columns, a multiple of 64 (KR)
    int32_t segs, ksteps;      // stages of a segment
    int32_t mt, nt, split;     // tiles, shares of the sum
    int32_t halves;            // outputs: seg[0..segs) and seg[segs..2 segs)
    // epilogue
    void* out;
    void* out2;
    float* part;
    const void* dh;
    float* saved;
    bf16 *dg, *du;
    int64_t ldo, hs, plane, T, Tpad;
    int32_t F, Fpad;
};

template <int V> struct Int { static constexpr int value = V; };

template <bool KR, int BK> struct Operand;
// [rows][k]: a row of BK k is 64 or 128 bytes in LDS, its 16-byte pieces exchanged by the row's number so that
// neighbouring rows' pieces of the same k lie in different banks.
template <int BK> struct Operand<false, BK> {
    static constexpr int P = BK / 8;
    static __device__ __forceinline__ int turn(int row) { return P == 8 ? row & 7 : (row >> 2) & 3; }
    static __device__ __forceinline__ int source(int at, int64_t rows_left, int64_t ld, int) {
        const int row = at / P, piece = (at % P) ^ turn(row);
        const int64_t r = row < rows_left ? row : rows_left - 1;
        return (int)(r * ld * 2) + piece * 16;
    }
    static __device__ __forceinline__ bf16x8 frag(const char* tile, int row0, int part, int lane, int) {
        const int row = row0 + (lane & 15), piece = (part * 4 + (lane >> 4)) ^ turn(row);
        return *reinterpret_cast<const bf16x8*>(tile + row * (BK * 2) + piece * 16);
    }
};
// [k][rows]: a k row of R columns is 2 R bytes, its 32-byte pieces (16 columns) exchanged so that the 8 k rows that
// half a wavefront reads at once lie in different banks.
template <int BK> struct Operand<true, BK> {
    static __device__ __forceinline__ int turn(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }
    static __device__ __forceinline__ int source(int at, int64_t rows_left, int64_t ld, int rows) {
        const int per = rows / 8, k = at / per, slot = at % per;
        const int c = ((((slot >> 1) ^ turn(k)) << 1) | (slot & 1)) * 8;
        const int64_t col = c + 8 <= rows_left ? c : rows_left - 8;
        return (int)(k * ld * 2 + col * 2);
    }
    static __device__ __forceinline__ bf16x8 frag(const char* tile, int row0, int part, int lane, int rows) {
        typedef __attribute__((address_space(3))) s16x4* lds;
        const int i = lane & 15, q = lane >> 4, k = part * KI + 8 * q + (i >> 2);
        const char* p = tile + k * rows * 2 + (((row0 >> 4) ^ turn(k)) * 32) + (i & 3) * 8;
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p)));
        const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + 4 * rows * 2)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

__device__ __forceinline__ void copy16(const char* base, int64_t offset, char* lds) {
    __builtin_amdgcn_global_load_lds((const void*)(base + offset), (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// The copies issued by this wavefront are done but for the last LEFT, and so are those of every other
// wavefront of the workgroup, and their reads of LDS.
template <int LEFT> __device__ __forceinline__ void wait_copies() {
    static_assert(LEFT < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// Epilogues: 4 neighbouring columns n .. n + 3 of row m, stored where they exist.
template <typename T> __device__ __forceinline__ void store_row(T* row, int64_t n, int64_t N, f32x4 v) {
    float f[4] = {v[0], v[1], v[2], v[3]};
    if (n + 4 <= N) store_v<4>(row + n, f);
    else
        for (int i = 0; i < 4; ++i)
            if (n + i < N) row[n + i] = from_f32<T>(f[i]);
}
// dg and du go to planes of [Tpad][Fpad], zero where a token or column does not exist.
template <int NP> __device__ __forceinline__ void store_planes(bf16* p, int64_t plane, float (&v)[4]) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        bf16x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = (bf16)(NP > 1 && n == 0 ? first_part(v[i]) : v[i]);
            v[i] -= (float)b[i];
        }
        *reinterpret_cast<bf16x4*>(p + n * plane) = b;
    }
}
template <typename DT, int ACT>
__device__ __forceinline__ void store_dgu(const GemmArgs& g, int64_t t, int64_t f, const float (&gv)[4], const float (&uv)[4]) {
    if (t >= g.Tpad || f >= g.Fpad) return;
    float dg[4], du[4];
    zero_v(dg);
    zero_v(du);
    if (t < g.T && f < g.F) {
        float d[4];
        zero_v(d);
        const DT* row = (const DT*)g.dh + t * g.hs;
        if (f + 4 <= g.F) get_v(load_v<4>(row + f), d);
        else
            for (int i = 0; i < 4; ++i)
                if (f + i < g.F) d[i] = to_f32(row[f + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, slope;
            activation<ACT>(gv[i], a, slope);
            const bool in = f + i < g.F;
            dg[i] = in ? d[i] * uv[i] * slope : 0.f;
            du[i] = in ? d[i] * a : 0.f;
        }
    }
    constexpr int NP = sizeof(DT) == 2 ? 1 : 3;
    store_planes<NP>(g.dg + t * g.Fpad + f, g.plane, dg);
    store_planes<NP>(g.du + t * g.Fpad + f, g.plane, du);
}

enum { EPI_OUT, EPI_H, EPI_DGU };

// BM x BN results a workgroup of WM x WN wavefronts.  Both operands come in stages of BK k, STAGES of them in LDS.
// The next 32 k are read from LDS into registers while 32 are multiplied out of others, and the stages after
// this one are on their way.  One barrier a stage, where its last 32 k are in everyone's registers: behind it
// the next stage's copies are complete, and this one's place takes new ones.  With two B (EPI_H, EPI_DGU) the
// first half of BN is of one and the second of the other, so that a lane holds both results of a column.
//
// What bounds it, 16384 x 4096 x 10240 bf16 (2.75 TFLOP, one tile of 256 x 256 a compute unit): 2180 us, 1260 TFLOP/s, where
// the matrix pipes alone take 1092 (168e6 instructions of 16 cycles on 1024 SIMDs at 2.4 GHz), vector issue 426 and LDS 410; a
// library product of these sizes runs at 1563.  The rest is the wait for a stage: 64 KB for 512 cycles of products.
// Two library products in bf16 and an elementwise tail (or one product over both weights), us, against this: 128 tokens
// of 4096 x 10240 70 (54), 68; 512 115 (94), 136; 1024 170 (175), 196; 2048 329 (418), 323; 8192 1043 (1064), 1089;
// 16384 2048 (2122), 2164.
// With fp32 the same loop runs over six pairs of planes: 777 x 1000 x 2731 91 us forward, 560 TFLOP/s of bf16 products, 94 of
// fp32 ones; 301 tiles of 128 on 256 compute units, two to some of them.
template <typename DT, int BM, int BN, int BK, int WM, int WN, int STAGES, bool AKR, bool BKR, int EPI, int ACT>
__global__ void __launch_bounds__(WM* WN * 64, 2) glu_gemm_kernel(GemmArgs g) {
    constexpr bool DUAL = EPI != EPI_OUT;
    constexpr int THREADS = WM * WN * 64, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int P = BK / 8, LA = BM * P / THREADS, LB = BN * P / THREADS, STAGE = (BM + BN) * BK * 2, PARTS = BK / KI;
    using OA = Operand<AKR, BK>;
    using OB = Operand<BKR, BK>;
    constexpr int BH = DUAL ? BN / 2 : BN;  // columns of one B in a tile
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wm = wave / WN, wn = wave % WN;

    // Every eighth workgroup runs on the same die: a die takes a run of neighbouring tiles, which share
    // operands in its cache, in strips of 8 tiles along m.
    auto uniform = [](unsigned v) { return (int)__builtin_amdgcn_readfirstlane(v); };
    const unsigned tiles = (unsigned)g.mt * g.nt, total = tiles * g.split * g.halves, run = (total + 7) / 8;
    const unsigned b = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= run || b >= total) return;
    const int half = uniform(b / tiles / g.split), share = uniform(b / tiles % g.split), tile = uniform(b % tiles);
    const int strip = uniform((unsigned)tile / (8u * g.nt)), in = tile - strip * 8 * g.nt;
    const int tall = min(g.mt - strip * 8, 8);
    const int ntile = uniform((unsigned)in / (unsigned)tall), mtile = strip * 8 + (in - ntile * tall);
    const int64_t m0 = (int64_t)mtile * BM, n0 = (int64_t)ntile * BH;

    int offa[LA], offb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) offa[i] = OA::source(i * THREADS + tid, (AKR ? g.colsA : g.M) - m0, g.lda, BM);
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int at = i * THREADS + tid;
        if (DUAL) offb[i] = OB::source(at % (BH * P), g.N - n0, g.ldb, BH);
        else offb[i] = OB::source(at, (BKR ? g.colsB : g.N) - n0, g.ldb, BN);
    }
    // this share's stages, whole pairs of 32 k
    constexpr int PAIR = 2 / PARTS;
    const int all = g.segs * g.ksteps / PAIR, k0 = (int)((int64_t)share * all / g.split) * PAIR;
    const int stages = (int)((int64_t)(share + 1) * all / g.split) * PAIR - k0;

    // What is fetched next: its operands' addresses, moved on by a stage each time and looked up where a segment
    // begins, and its place in LDS.
    int fs = uniform((unsigned)k0 / (unsigned)max(g.ksteps, 1)), fk = k0 - fs * g.ksteps, fslot = 0;
    const char *pa = nullptr, *pb = nullptr, *pb2 = nullptr;
    const int64_t stepa = (AKR ? g.lda : 1) * BK * 2, stepb = (BKR ? g.ldb : 1) * BK * 2;
    auto segment = [&]() {
        const Segment sg = g.seg[half * g.segs + fs];
        pa = (const char*)(sg.a + (AKR ? m0 : m0 * g.lda)) + fk * stepa;
        pb = (const char*)(sg.b + (BKR ? n0 : n0 * g.ldb)) + fk * stepb;
        if (DUAL) pb2 = (const char*)(sg.b2 + n0 * g.ldb) + fk * stepb;
    };
    auto fetch = [&]() {
        char* at = smem + fslot * STAGE + wave * 1024;
        const int64_t k = (int64_t)fk * BK;
        if ((AKR && g.kA - k < BK) || (BKR && g.kB - k < BK)) {
            // k rows past the last are the last again; the stage may lie behind it whole
            const int la = AKR ? (int)(g.kA - k) : BK, lb = BKR ? (int)(g.kB - k) : BK;
#pragma unroll
            for (int i = 0; i < LA; ++i) {
                const int row = (i * THREADS + tid) / (BM / 8);
                copy16(pa, offa[i] - (AKR && row >= la ? (int)((row - la + 1) * g.lda * 2) : 0), at + i * THREADS * 16);
            }
#pragma unroll
            for (int i = 0; i < LB; ++i) {
                const int row = (i * THREADS + tid) / (BN / 8);
                copy16(pb, offb[i] - (BKR && row >= lb ? (int)((row - lb + 1) * g.ldb * 2) : 0),
                       at + BM * BK * 2 + i * THREADS * 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < LA; ++i) copy16(pa, (unsigned)offa[i], at + i * THREADS * 16);
#pragma unroll
            for (int i = 0; i < LB; ++i)
                copy16(DUAL && i * THREADS >= BH * P ? pb2 : pb, (unsigned)offb[i], at + BM * BK * 2 + i * THREADS * 16);
        }
        if (++fslot == STAGES) fslot = 0;
        pa += stepa;
        pb += stepb;
        if (DUAL) pb2 += stepb;
        if (++fk == g.ksteps) {
            fk = 0;
            ++fs;
            if (fs < g.segs) segment();
        }
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = zero4();
    bf16x8 fa[2][TM], fb[2][TN];
    int rslot = 0;
    auto read = [&](int part, bf16x8 (&xa)[TM], bf16x8 (&xb)[TN]) {
        const char* ta = smem + rslot * STAGE;
        const char* tb = ta + BM * BK * 2;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int row = DUAL ? (j >= TN / 2 ? BH : 0) + wn * (BH / WN) + j % (TN / 2) * 16 : wn * (BN / WN) + j * 16;
            xb[j] = OB::frag(tb, row, part, lane, BN);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) xa[i] = OA::frag(ta, wm * (BM / WM) + i * 16, part, lane, BM);
        if (part == PARTS - 1 && ++rslot == STAGES) rslot = 0;
    };
    auto multiply = [&](const bf16x8 (&xa)[TM], const bf16x8 (&xb)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j], xa[i], acc[i][j], 0, 0, 0);
    };
    // the first 32 k of the next stage, of which at most LEFT copies are still on their way behind it
    auto next = [&](auto left, bool more, bf16x8 (&xa)[TM], bf16x8 (&xb)[TN]) {
        wait_copies<decltype(left)::value>();
        read(0, xa, xb);
        if (more) fetch();
    };
    constexpr int LEFT = (STAGES - 2) * (LA + LB);
    if (stages > 0) {
        segment();
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < stages) fetch();
        if (stages >= STAGES) wait_copies<(STAGES - 1) * (LA + LB)>(); else wait_copies<0>();
        read(0, fa[0], fb[0]);
        int j = 0;
        // the next stages exist: no conditions in the loop
        for (; j + PAIR - 1 + STAGES < stages; j += PAIR) {
            if constexpr (PARTS == 1) next(Int<LEFT>(), true, fa[1], fb[1]);
            else read(1, fa[1], fb[1]);
            multiply(fa[0], fb[0]);
            next(Int<LEFT>(), true, fa[0], fb[0]);
            multiply(fa[1], fb[1]);
        }
        for (; j < stages; j += PAIR) {
            if constexpr (PARTS == 1) {
                if (j + 1 < stages) next(Int<0>(), j + STAGES < stages, fa[1], fb[1]);
            } else {
                read(1, fa[1], fb[1]);
            }
            multiply(fa[0], fb[0]);
            if (j + PAIR < stages) next(Int<0>(), j + PAIR - 1 + STAGES < stages, fa[0], fb[0]);
            multiply(fa[1], fb[1]);
        }
    }

    // a lane holds columns 4 (lane / 16) .. + 3 of row lane % 16 of each 16 x 16 tile
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + wm * (BM / WM) + i * 16 + (lane & 15);
        if constexpr (DUAL) {
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                const int64_t n = n0 + wn * (BH / WN) + j * 16 + 4 * (lane >> 4);
                const f32x4 gv = acc[i][j], uv = acc[i][j + TN / 2];
                if constexpr (EPI == EPI_H) {
                    if (m < g.M && n < g.N) {
                        f32x4 h;
#pragma unroll
                        for (int r = 0; r < 4; ++r) h[r] = gated<ACT>(gv[r], uv[r]);
                        store_row((DT*)g.out + m * g.N, n, g.N, h);
                        if (g.saved) {
                            store_row(g.saved + m * g.N, n, g.N, gv);
                            store_row(g.saved + (g.T + m) * g.N, n, g.N, uv);
                        }
                    }
                } else {
                    const float ga[4] = {gv[0], gv[1], gv[2], gv[3]}, ua[4] = {uv[0], uv[1], uv[2], uv[3]};
                    store_dgu<DT, ACT>(g, m, n, ga, ua);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t n = n0 + wn * (BN / WN) + j * 16 + 4 * (lane >> 4);
                if (m >= g.M || n >= g.N) continue;
                if (g.split > 1) store_row(g.part + ((int64_t)(half * g.split + share) * g.M + m) * g.N, n, g.N, acc[i][j]);
                else store_row((DT*)(half ? g.out2 : g.out) + m * g.N, n, g.N, acc[i][j]);
            }
        }
    }
}

// One output or two, each the sum of its shares, in order.  (777 x 1000 x 2731: 6 + 7 us of 300.)
template <typename DT>
__global__ void __launch_bounds__(256) glu_shares_kernel(const float* part, int split, int64_t n, DT* one, DT* two) {
    DT* const out = blockIdx.y ? two : one;
    part += blockIdx.y * split * n;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
        if (i + 4 <= n) {
            f32x4 s = zero4();
            for (int k = 0; k < split; ++k) {
                const Pack<float, 4> p = load_v<4>(part + k * n + i);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] += p[r];
            }
            float f[4] = {s[0], s[1], s[2], s[3]};
            store_v<4>(out + i, f);
        } else {
            for (int64_t j = i; j < n; ++j) {
                float s = 0.f;
                for (int k = 0; k < split; ++k) s += part[k * n + j];
                out[j] = from_f32<DT>(s);
            }
        }
    }
}

// Up to three matrices, [rows][cols] each, as NP planes of [rows][pad] bf16, zero past the columns.
struct PackArgs {
    const void* src[3];
    bf16* dst[3];
    int64_t stride[3], rows[3];
    int cols, pad;
};
template <typename DT, int NP> __global__ void __launch_bounds__(256) glu_pack_kernel(PackArgs a) {
    const DT* src = (const DT*)a.src[blockIdx.y];
    bf16* dst = a.dst[blockIdx.y];
    const int64_t stride = a.stride[blockIdx.y], rows = a.rows[blockIdx.y], plane = rows * a.pad;
    const int per = a.pad / 4, cols = a.cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per;
        const int c = (int)(i % per) * 4;
        float v[4];
        zero_v(v);
        if (c + 4 <= cols) get_v(load_v<4>(src + r * stride + c), v);
        else
            for (int k = 0; k < 4; ++k)
                if (c + k < cols) v[k] = to_f32(src[r * stride + c + k]);
        store_planes<NP>(dst + r * a.pad + c, plane, v);
    }
}

// dg and du from the products that the forward kept (fp32, 8 bytes a value, and dh): bound by memory.  8192 x 10240 bf16 moves
// 1.17 GB in 246 us, 4.8 TB/s.
template <typename DT, int ACT> __global__ void __launch_bounds__(256) glu_saved_kernel(GemmArgs g) {
    const int per = g.Fpad / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < g.Tpad * per; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per;
        const int f = (int)(i % per) * 4;
        float gv[4], uv[4];
        zero_v(gv);
        zero_v(uv);
        if (t < g.T && f < g.F) {
            const float *pg = g.saved + t * g.F + f, *pu = g.saved + (g.T + t) * g.F + f;
            if (f + 4 <= g.F) {
                get_v(load_nt<4>(pg), gv);
                get_v(load_nt<4>(pu), uv);
            } else {
                for (int k = 0; k < 4; ++k)
                    if (f + k < g.F) {
                        gv[k] = pg[k];
                        uv[k] = pu[k];
                    }
            }
        }
        store_dgu<DT, ACT>(g, t, f, gv, uv);
    }
}

// ---------------------------------------------------------------- few tokens
//
// Few tokens: the weights are what there is to read.  4 tokens of 4096 x 10240 bf16: 168 MB in 34.5 us, 4.9 TB/s.
// fp32, 336 MB: 92 us up to 16 tokens, 3.7 TB/s, and 198 for 64 (two library products and a tail: 76 and 134); x is
// split into its parts again by every workgroup, and its products are six.
// A workgroup takes 16 columns of both weights, its wavefronts a part of the sum each; weights come straight from
// memory into the operand's registers, x from the cache.
template <typename DT> struct Direct;
template <> struct Direct<bf16> {
    static constexpr int NP = 1;
    static __device__ __forceinline__ void split(const Pack<bf16, 8>& p, bf16x8 (&o)[1]) { o[0] = p.part[0]; }
};
template <> struct Direct<float> {
    static constexpr int NP = 3;
    static __device__ __forceinline__ void split(const Pack<float, 8>& p, bf16x8 (&o)[3]) {
        float v[8];
        get_v(p, v);
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[n][i] = (bf16)(n == 0 ? first_part(v[i]) : v[i]);
                v[i] -= (float)o[n][i];
            }
    }
};

template <typename DT, int TT, int ACT>
__global__ void __launch_bounds__(256) glu_few_kernel(GluArgs a) {
    constexpr int NP = Direct<DT>::NP, U = sizeof(DT) == 2 ? (TT > 2 ? 4 : 8) : 2;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, l15 = lane & 15, q = lane >> 4;
    const int f0 = blockIdx.x * 16, f = min(f0 + l15, a.F - 1);
    const DT *wg = (const DT*)a.wg + (int64_t)f * a.D, *wu = (const DT*)a.wu + (int64_t)f * a.D;
    const DT* xr[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xr[t] = (const DT*)a.x + (int64_t)min((int64_t)(t * 16 + l15), a.T - 1) * a.xs;
    f32x4 ag[TT], au[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) ag[t] = au[t] = zero4();
    const int steps = (a.D + 31) / 32, s0 = steps * wave / 4, s1 = steps * (wave + 1) / 4;
    auto get = [&](const DT* row, int k) {
        if (k + 8 <= a.D) return load_v<8>(row + k);
        Pack<DT, 8> p;
        for (int i = 0; i < 8; ++i)
            p.part[i / Pack<DT, 8>::N][i % Pack<DT, 8>::N] = k + i < a.D ? row[k + i] : from_f32<DT>(0.f);
        return p;
    };
    for (int s = s0; s < s1; s += U) {
        Pack<DT, 8> pg[U], pu[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(s + u, s1 - 1) * 32 + 8 * q;
            pg[u] = get(wg, k);
            pu[u] = get(wu, k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            bf16x8 g[NP], w[NP];
            Direct<DT>::split(pg[u], g);
            Direct<DT>::split(pu[u], w);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                bf16x8 x[NP];
                Direct<DT>::split(get(xr[t], (s + u) * 32 + 8 * q), x);
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        if (i + j <= 2) {
                            ag[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(g[i], x[j], ag[t], 0, 0, 0);
                            au[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], x[j], au[t], 0, 0, 0);
                        }
            }
        }
    }
    __shared__ f32x4 part[3][2][TT][64];
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            part[wave - 1][0][t][lane] = ag[t];
            part[wave - 1][1][t][lane] = au[t];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            ag[t] += part[w][0][t][lane];
            au[t] += part[w][1][t][lane];
        }
        const int64_t m = t * 16 + l15;
        const int n = f0 + 4 * q;
        if (m >= a.T || n >= a.F) continue;
        f32x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = gated<ACT>(ag[t][r], au[t][r]);
        store_row((DT*)a.h + m * a.F, n, a.F, h);
        if (a.saved) {
            store_row(a.saved + m * a.F, n, a.F, ag[t]);
            store_row(a.saved + (a.T + m) * a.F, n, a.F, au[t]);
        }
    }
}

// ---------------------------------------------------------------- launches

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
size_t up256(int64_t x) { return (size_t)up(x, 256); }
int planes(const GluArgs& a) { return a.dtype == 1 ? 1 : 3; }

// The six pairs of planes above 2^-24, smallest first.
constexpr int PAIRS[6][2] = {{1, 1}, {0, 2}, {2, 0}, {0, 1}, {1, 0}, {0, 0}};

struct Mat { const bf16* p; int64_t ld, plane; };  // an operand, or its planes


// Tile shape and shares of a product of M x N results over `steps` steps.
struct Shape { bool big; int mt, nt, split; };
Shape shape_of(int64_t M, int64_t N, bool dual, int halves, int steps, bool may_split) {
    auto tiles = [&](int bm, int bn) {
        return ((M + bm - 1) / bm) * ((N + (dual ? bn / 2 : bn) - 1) / (dual ? bn / 2 : bn)) * halves;
    };
    Shape s;
    // A tile of 256 x 256 has half the reads of four of 128 x 128, but one has a compute unit to itself: taken where its
    // last round of workgroups is full enough, three quarters over all rounds.  bf16 forward, big and small, us:
    // 256 tiles 55, 67; 320 173, 156; 352 95, 94; 396 77, 86; 640 276, 305; 88 47, 34.
    const int64_t big = tiles(256, 256), rounds = (big + 255) / 256;
    s.big = rounds > 0 && big * 4 >= rounds * 256 * 3;
    const int bm = s.big ? 256 : 128, bn = bm;
    s.mt = (int)((M + bm - 1) / bm);
    s.nt = (int)((N + (dual ? bn / 2 : bn) - 1) / (dual ? bn / 2 : bn));
    s.split = 1;
    // Shares of the sum: two workgroups for every compute unit, rounded up, none shorter than 16 steps.  Whole, this way
    // and rounded down (one round of workgroups at most), us: 777 x 1000 x 2731 fp32, dx in 56 tiles 397, 97, 65, dW in 352 107,
    // 110, 107; bf16 70, 29, 23 and 35, 35, 35; 1024 x 1024 x 2816 bf16, 64 tiles 74, 26, 26, 352 34, 43, 33; 2048
    // tokens, 128 tiles 73, 36, 35, 352 54, 62, 53; 4096 x 512 x 1408 fp32, 128 tiles 212, 77, 79, 88 334, 154, 119.
    if (may_split && !s.big) {
        const int64_t t = tiles(bm, bn) > 0 ? tiles(bm, bn) : 1, want = (512 + t - 1) / t, most = steps / 16 > 0 ? steps / 16 : 1;
        s.split = (int)(want < most ? want : most);
    }
    return s;
}

template <typename DT, int SIDE, int BK, int STAGES, bool AKR, bool BKR, int EPI, int ACT>
hipError_t launch_gemm(GemmArgs g, int64_t blocks, hipStream_t st) {
    constexpr int lds = STAGES * 2 * SIDE * BK * 2, WN = SIDE / 64;
    static_assert(lds <= 160 * 1024, "the stages fit a compute unit");
    auto* k = glu_gemm_kernel<DT, SIDE, SIDE, BK, 2, WN, STAGES, AKR, BKR, EPI, ACT>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    g.ksteps /= BK;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(2 * WN * 64), lds, st, g);
    return hipGetLastError();
}

// (g.ksteps: k of a segment)
template <typename DT, bool AKR, bool BKR, int EPI, int ACT>
hipError_t run_gemm(GemmArgs g, const Shape& s, hipStream_t st) {
    g.mt = s.mt;
    g.nt = s.nt;
    g.split = s.split;
    const int64_t total = (int64_t)s.mt * s.nt * s.split * g.halves, blocks = (total + 7) / 8 * 8;
    // Stages of 64 k where both operands have k contiguous: their rows are then read in whole cache lines
    // (8192 x 4096 x 20480: 1160 us; of 32, half lines, 1314).  An operand with k along the rows is read in whole
    // lines either way, and five stages of 32 have more time to arrive than two of 64: 1154 us against 1672
    // for both such (dW), 1171 against 1184 for one (dx).  Small tiles: 64 (777 x 1000 x 2731 fp32, three
    // products: 82, 91, 75 us; of 32: 103, 104, 86).
    constexpr int BK = AKR || BKR ? 32 : 64;
    if (s.big) return launch_gemm<DT, 256, BK, BK == 32 ? 5 : 2, AKR, BKR, EPI, ACT>(g, blocks, st);
    return launch_gemm<DT, 128, 64, 2, AKR, BKR, EPI, ACT>(g, blocks, st);
}

template <typename DT>
hipError_t sum_shares(const float* part, int split, int64_t n, void* one, void* two, hipStream_t st) {
    const int64_t blocks = (n / 4 + 256) / 256;
    hipLaunchKernelGGL(glu_shares_kernel<DT>, dim3((unsigned)(blocks < 4096 ? blocks : 4096), two ? 2 : 1), dim3(256), 0, st, part,
                       split, n, (DT*)one, (DT*)two);
    return hipGetLastError();
}

#define GLU_TRY(call)                            \
    do {                                         \
        const hipError_t e_ = (call);            \
        if (e_ != hipSuccess) return e_;         \
    } while (0)

// The workspace's arrays, in order.
struct Work {
    size_t size = 0;
    bf16 *x = nullptr, *wg = nullptr, *wu = nullptr, *dg = nullptr, *du = nullptr;
    float* part = nullptr;
};
int pad_of(const GluArgs& a) { return (int)up(a.D, PAD); }
Shape dx_shape(const GluArgs& a) {
    const int np = planes(a);
    return shape_of(a.T, a.D, false, 1, (int)(up(a.F, PAD) / KI) * 2 * (np == 1 ? 1 : 6), true);
}
Shape dw_shape(const GluArgs& a) {
    const int np = planes(a);
    return shape_of(a.F, a.D, false, 2, (int)(up(a.T, PAD) / KI) * (np == 1 ? 1 : 6), true);
}
// Few tokens or tiles.  Inputs that tiles can read as they lie: tiles from 33 tokens on, where there are 96 of
// them.  bf16 forward of 33 and 64 tokens, few or tiles, us: 4096 x 10240 56, 68 or 45, 46; 2048 x 8192 26, 30 or 25, 25; 4096 x
// 5632 41, 47 or 43, 44; 2048 x 2816 15, 17 or 21, 21.  Others are packed for tiles, and fp32 has six products:
// 64 tokens 1000 x 2731 bf16 10 or 28, fp32 23 or 81; 4096 x 10240 fp32 191 or 508.  (Weights in the last-level cache; read
// from memory, bf16: 4096 x 10240 65, 75 or 65, 66; 2048 x 8192 31, 35 or 34, 35.)
bool is_few(const GluArgs& a) {
    return a.T <= (a.x_plain && a.w_plain && a.F > 95 * 64 ? GLU_FEW / 2 : GLU_FEW);
}
Work work_of(const GluArgs& a, bool backward, bool input_grad, uint8_t* base) {
    Work w;
    auto take = [&](int64_t bytes) {
        uint8_t* p = base + w.size;
        w.size += up256(bytes);
        return p;
    };
    const int64_t np = planes(a), pad = pad_of(a);
    if (!backward && is_few(a)) return w;
    if (!a.x_plain) w.x = (bf16*)take(a.T * pad * np * 2);
    if (!a.w_plain) {
        w.wg = (bf16*)take(a.F * pad * np * 2);
        w.wu = (bf16*)take(a.F * pad * np * 2);
    }
    if (backward) {
        const int64_t one = up(a.T, PAD) * up(a.F, PAD) * np * 2;
        w.dg = (bf16*)take(one);
        w.du = (bf16*)take(one);
        const Shape sx = dx_shape(a), sw = dw_shape(a);
        const int64_t px = input_grad && sx.split > 1 ? sx.split * a.T * a.D * 4 : 0;
        const int64_t pw = sw.split > 1 ? 2ll * sw.split * a.F * a.D * 4 : 0;
        if (px > 0 || pw > 0) w.part = (float*)take(px > pw ? px : pw);
    }
    return w;
}

struct Inputs { Mat x, wg, wu; };
template <typename DT> hipError_t inputs(const GluArgs& a, const Work& w, Inputs* in, hipStream_t st) {
    const int pad = pad_of(a);
    in->x = a.x_plain ? Mat{(const bf16*)a.x, a.xs, 0} : Mat{w.x, pad, a.T * pad};
    in->wg = a.w_plain ? Mat{(const bf16*)a.wg, a.D, 0} : Mat{w.wg, pad, (int64_t)a.F * pad};
    in->wu = a.w_plain ? Mat{(const bf16*)a.wu, a.D, 0} : Mat{w.wu, pad, (int64_t)a.F * pad};
    if (a.T == 0) return hipSuccess;
    PackArgs p = {};
    int n = 0;
    int64_t most = 0;
    auto add = [&](const void* src, int64_t stride, int64_t rows, bf16* dst) {
        p.src[n] = src;
        p.dst[n] = dst;
        p.stride[n] = stride;
        p.rows[n++] = rows;
        most = rows > most ? rows : most;
    };
    if (!a.x_plain) add(a.x, a.xs, a.T, w.x);
    if (!a.w_plain) {
        add(a.wg, a.D, a.F, w.wg);
        add(a.wu, a.D, a.F, w.wu);
    }
    if (n == 0) return hipSuccess;
    p.cols = a.D;
    p.pad = pad;
    const int64_t blocks = (most * (pad / 4) + 255) / 256;
    hipLaunchKernelGGL((glu_pack_kernel<DT, sizeof(DT) == 2 ? 1 : 3>), dim3((unsigned)(blocks < 8192 ? blocks : 8192), n),
                       dim3(256), 0, st, p);
    return hipGetLastError();
}

// x against both weights, with EPI
template <typename DT, int EPI, int ACT> hipError_t products(const GluArgs& a, const Inputs& in, GemmArgs g, hipStream_t st) {
    const int np = planes(a), n = np == 1 ? 1 : 6;
    for (int i = 0; i < n; ++i) {
        const int pa = np == 1 ? 0 : PAIRS[i][0], pb = np == 1 ? 0 : PAIRS[i][1];
        g.seg[i] = {in.x.p + pa * in.x.plane, in.wg.p + pb * in.wg.plane, in.wu.p + pb * in.wu.plane};
    }
    g.segs = n;
    g.ksteps = pad_of(a);
    g.lda = in.x.ld;
    g.ldb = in.wg.ld;
    g.M = a.T;
    g.N = a.F;
    g.halves = 1;
    return run_gemm<DT, false, false, EPI, ACT>(g, shape_of(a.T, a.F, true, 1, 0, false), st);
}

template <typename DT, int ACT> hipError_t few(const GluArgs& a, hipStream_t st) {
    const dim3 grid((a.F + 15) / 16);
    if (a.T <= 16) hipLaunchKernelGGL((glu_few_kernel<DT, 1, ACT>), grid, dim3(256), 0, st, a);
    else if (a.T <= 32) hipLaunchKernelGGL((glu_few_kernel<DT, 2, ACT>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((glu_few_kernel<DT, 4, ACT>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename DT, int ACT> hipError_t forward(const GluArgs& a, hipStream_t st) {
    if (is_few(a)) return few<DT, ACT>(a, st);
    const Work w = work_of(a, false, false, a.ws);
    Inputs in;
    GLU_TRY((inputs<DT>(a, w, &in, st)));
    GemmArgs g = {};
    g.out = a.h;
    g.saved = a.saved;
    g.T = a.T;
    return products<DT, EPI_H, ACT>(a, in, g, st);
}

template <typename DT, int ACT> hipError_t backward(const GluArgs& a, hipStream_t st) {
    const Work w = work_of(a, true, a.dx != nullptr, a.ws);
    Inputs in;
    GLU_TRY((inputs<DT>(a, w, &in, st)));
    const int np = planes(a), n = np == 1 ? 1 : 6;
    GemmArgs g = {};
    g.T = a.T;
    g.Tpad = up(a.T, PAD);
    g.F = a.F;
    g.Fpad = (int)up(a.F, PAD);
    g.plane = g.Tpad * g.Fpad;
    g.dh = a.dh;
    g.hs = a.hs;
    g.dg = w.dg;
    g.du = w.du;
    g.saved = a.saved;
    if (a.T == 0) {
        // nothing but the weights' gradients, which are zero
    } else if (a.saved) {
        const int64_t blocks = (g.plane / 4 + 255) / 256;
        hipLaunchKernelGGL((glu_saved_kernel<DT, ACT>), dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, g);
        GLU_TRY(hipGetLastError());
    } else {
        GLU_TRY((products<DT, EPI_DGU, ACT>(a, in, g, st)));
    }
    if (a.dx && a.T > 0) {
        GemmArgs p = {};
        for (int i = 0; i < n; ++i) {
            const int pa = np == 1 ? 0 : PAIRS[i][0], pb = np == 1 ? 0 : PAIRS[i][1];
            p.seg[2 * i] = {w.dg + pa * g.plane, in.wg.p + pb * in.wg.plane, nullptr};
            p.seg[2 * i + 1] = {w.du + pa * g.plane, in.wu.p + pb * in.wu.plane, nullptr};
        }
        p.segs = 2 * n;
        p.ksteps = g.Fpad;
        p.lda = g.Fpad;
        p.ldb = in.wg.ld;
        p.M = a.T;
        p.N = a.D;
        p.kB = a.F;
        p.colsB = pad_of(a);
        p.halves = 1;
        p.out = a.dx;
        p.part = w.part;
        const Shape s = dx_shape(a);
        GLU_TRY((run_gemm<DT, false, true, EPI_OUT, 0>(p, s, st)));
        if (s.split > 1) GLU_TRY((sum_shares<DT>(w.part, s.split, a.T * a.D, a.dx, nullptr, st)));
    }
    GemmArgs p = {};
    for (int i = 0; i < n; ++i) {
        const int pa = np == 1 ? 0 : PAIRS[i][0], pb = np == 1 ? 0 : PAIRS[i][1];
        p.seg[i] = {w.dg + pa * g.plane, in.x.p + pb * in.x.plane, nullptr};
        p.seg[n + i] = {w.du + pa * g.plane, in.x.p + pb * in.x.plane, nullptr};
    }
    p.segs = n;
    p.ksteps = (int)g.Tpad;
    p.lda = g.Fpad;
    p.ldb = in.x.ld;
    p.M = a.F;
    p.N = a.D;
    p.kA = g.Tpad;
    p.kB = a.T;
    p.colsA = g.Fpad;
    p.colsB = pad_of(a);
    p.halves = 2;
    p.out = a.dwg;
    p.out2 = a.dwu;
    p.part = w.part;
    const Shape s = dw_shape(a);
    GLU_TRY((run_gemm<DT, true, true, EPI_OUT, 0>(p, s, st)));
    if (s.split > 1) GLU_TRY((sum_shares<DT>(w.part, s.split, (int64_t)a.F * a.D, a.dwg, a.dwu, st)));
    return hipSuccess;
}

template <typename DT> hipError_t by_act(const GluArgs& a, bool bwd, hipStream_t st) {
    switch (a.act) {
        case GLU_SILU: return bwd ? backward<DT, GLU_SILU>(a, st) : forward<DT, GLU_SILU>(a, st);
        case GLU_SIGMOID: return bwd ? backward<DT, GLU_SIGMOID>(a, st) : forward<DT, GLU_SIGMOID>(a, st);
        default: return bwd ? backward<DT, GLU_GELU>(a, st) : forward<DT, GLU_GELU>(a, st);
    }
}

}  // namespace

size_t glu_fwd_workspace(const GluArgs& a) { return work_of(a, false, false, nullptr).size; }
size_t glu_bwd_workspace(const GluArgs& a, bool input_grad) { return work_of(a, true, input_grad, nullptr).size; }
int64_t glu_blocks(const GluArgs& a) {
    const int64_t t = (a.T + 127) / 128, d = ((int64_t)a.D + 127) / 128, f = ((int64_t)a.F + 63) / 64;
    const int64_t h = t * f, dx = t * d * dx_shape(a).split, dw = f * d * 2 * dw_shape(a).split;
    return (h > dx ? h > dw ? h : dw : dx > dw ? dx : dw) + 8;
}

hipError_t launch_glu_fwd(const GluArgs& a, hipStream_t st) {
    return a.dtype == 1 ? by_act<bf16>(a, false, st) : by_act<float>(a, false, st);
}
hipError_t launch_glu_bwd(const GluArgs& a, hipStream_t st) {
    return a.dtype == 1 ? by_act<bf16>(a, true, st) : by_act<float>(a, true, st);
}

}  // namespace kda
