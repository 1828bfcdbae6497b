// kda_ssm.hip -- selective state space scan: chunked walk over packed sequences.
//
// Per head, with d_t = softplus(dt_t + bias), l_t = d_t A log2(e) and a_t = 2^{l_t}:
//   h_t = a_t h_{t-1} + d_t B_t^T x_t,   y_t = C_t h_t + D x_t,   h [K, P].
// Inside a chunk of Q tokens, with c_t the running sum of l:
//   y_t   = 2^{c_t} C_t h + sum_{s <= t} (C_t . B_s) 2^{c_t - c_s} d_s x_s + D x_t
//   h'    = 2^{c_Q} h + sum_s 2^{c_Q - c_s} d_s B_s^T x_s.
// The gradient with respect to x' = d x walks the chunks from the end, with the chunk's tokens
// reversed, r_t = c_Q - c_t in place of c_t and (B, C, x) replaced by (C, B, dy):
//   dx'_s = 2^{r_s} B_s g + sum_{t >= s} (B_s . C_t) 2^{r_s - r_t} dy_t
//   g'    = 2^{c_Q} g + sum_t 2^{c_Q - r_t} C_t^T dy_t,
// the same map with other names, so one kernel does both.
//
// Exponents: c_t - c_s is the difference of two sums that may be large while it is small, so the
// sums are formed in fp64 and held as a multiple of 2^-8 and a rest; both differences are exact or
// nearly so.  (As single fp32 numbers, up to 9600 in a chunk, they put up to 2^-10 ln 2 on a weight; the second part
// is 2 us of the 750 of 2 x 32768 tokens.)  No exponent is positive, so nothing overflows whatever the decay; l is held above
// -300, below which 2^l is zero for every state that fp32 holds.
//
// Matrix cores take bf16 operands.  bf16 inputs go in as they are; what is computed in fp32 and is an operand again goes in as
// a sum of bf16 parts, each the rounding of what the parts before it left: three hold a value to 2^-26 of itself.
//   - states, and what the derivatives of dt, A and h0 are sums of: three parts;
//   - y and dx with bf16 inputs: the masked products and the state are rounded to bf16 once.  Every term of such a
//     result has one of them as a factor, so the result is off by at most 2^-8 of the sum of its terms' magnitudes,
//     about what its own rounding costs (measured against 64 bits 1.8e-3 to 2.2e-3, rounding alone 1.7e-3; with two
//     parts the forward of 2 x 32768 tokens took 1080 us where it took 846 with one);
//   - dB and dC with bf16 inputs: two parts of the masked products.  They sum heads whose terms cancel: with one part 2.7e-3
//     against 64 bits where rounding alone is 1.7e-3, and with two 1.7e-3 (gradient of 2 x 8192 980 us and 1025);
//   - fp32 inputs: everything in three parts, split as it is staged; products of parts below 2^-24 are left out.
//
// Per call: the segments' own states (ENDS), their join, and the walk proper.  The gradient does this in both directions side by
// side, forwards for the states before every chunk (EMIT) and backwards for dx and the derivatives behind every
// chunk, and then has a kernel over chunks for what needs both.  2 x 32768 tokens of 32 heads of 128 x 128, bf16: 735 to 753 us
// by the card (at 735 ENDS 185, join 18, OUT 535); gradient of 2 x 8192: 1025 us (below).
#include "kda_ssm.hpp"

#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int WAVES = 4;
constexpr int NT = WAVES * WAVE;
constexpr int WALK = 32;  // tokens of a chunk of the walk

template <typename DT> struct Cfg;
// QT: 16-token tiles of a chunk; parts of inputs (NP), of the masked products in the walk (MP) and in dB and dC (GP),
// of the state where it is an operand of a result (HP)
template <> struct Cfg<bf16> { static constexpr int QT = 4, NP = 1, MP = 1, HP = 1, GP = 2; };
template <> struct Cfg<float> { static constexpr int QT = 2, NP = 3, MP = 3, HP = 3, GP = 3; };

template <int V> struct Int { static constexpr int value = V; };
typedef short s16x4 __attribute__((ext_vector_type(4)));

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two values as bf16 in one register, one instruction; and back, exactly.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ float low_of(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_of(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The sum of N bf16 parts that stands for v.  WIDE: v may be above the largest bf16 (fp32 inputs, and what is formed of
// them; with bf16 inputs the 16 values a lane that a chunk's update splits cost 1.3 % of the long forward).
template <int N> struct Parts { bf16x8 p[N]; };
template <int N, bool WIDE> __device__ __forceinline__ Parts<N> split8(const float (&in)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    Parts<N> o;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = WIDE && n == 0 ? pack2(first_part(v[2 * i]), first_part(v[2 * i + 1])) : pack2(v[2 * i], v[2 * i + 1]);
            if (n + 1 < N) {
                v[2 * i] -= low_of(w[i]);
                v[2 * i + 1] -= high_of(w[i]);
            }
        }
        o.p[n] = __builtin_bit_cast(bf16x8, w);
    }
    return o;
}

// Part m of four values.
template <bool WIDE> __device__ __forceinline__ void pack4(const float (&v)[4], int m, uint32_t& a, uint32_t& b) {
    const bool first = WIDE && m == 0;
    a = first ? pack2(first_part(v[0]), first_part(v[1])) : pack2(v[0], v[1]);
    b = first ? pack2(first_part(v[2]), first_part(v[3])) : pack2(v[2], v[3]);
}

// acc += A B over the parts of both, without the products below 2^-24.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma_parts(const Parts<NA>& a, const Parts<NB>& b, f32x4 acc) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= 2) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], acc, 0, 0, 0);
    return acc;
}

// Operands of 32 contraction indices.  In the "paired" order lane group q = lane / 16 holds indices
// 4 q .. 4 q + 3 and 16 + 4 q .. 16 + 4 q + 3: the order in which two accumulator tiles, one
// above the other, hold their rows, so that they can be fed back without leaving the registers.
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// rows: the lane's row of a matrix whose contraction index is contiguous
__device__ __forceinline__ bf16x8 row_paired(const bf16* row, int lane) {
    const bf16* p = row + 4 * (lane >> 4);
    return join(*reinterpret_cast<const bf16x4*>(p), *reinterpret_cast<const bf16x4*>(p + 16));
}
__device__ __forceinline__ bf16x8 row_natural(const bf16* row, int lane) {
    return *reinterpret_cast<const bf16x8*>(row + 8 * (lane >> 4));
}
// a matrix stored with its contraction index along the rows: each group of 16 lanes reads 4 rows of 16
// columns and gets them transposed, 4 contraction indices of column lane % 16
__device__ __forceinline__ bf16x4 tr4(const bf16* m, int ld, int k0, int lane) {
    typedef __attribute__((address_space(3))) s16x4* lds;
    const bf16* p = m + (k0 + ((lane & 15) >> 2)) * ld + 4 * (lane & 3);
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p)));
}
__device__ __forceinline__ bf16x8 col_paired(const bf16* m, int ld, int lane) {
    const int k = 4 * (lane >> 4);
    return join(tr4(m, ld, k, lane), tr4(m, ld, k + 16, lane));
}
__device__ __forceinline__ bf16x8 col_natural(const bf16* m, int ld, int lane) {
    const int k = 8 * (lane >> 4);
    return join(tr4(m, ld, k, lane), tr4(m, ld, k + 4, lane));
}

// ROWS rows of up to COLS columns on their way from global memory to LDS, zero where a row or
// column does not exist: loads first, then (split into NP planes) the stores.  Where every column
// exists (the usual case) no lane branches: rows past the last read the last and are replaced by zeros.
template <typename DT, int ROWS, int COLS, int THREADS> struct Stage {
    static constexpr int NP = Cfg<DT>::NP, PER = COLS / 8, ALL = ROWS * PER, CNT = (ALL + THREADS - 1) / THREADS;
    Pack<DT, 8> v[CNT];
    // Row r is token t0 + r (reversed: the last of the n from t0 on minus r), r < n, n > 0.  Everything but tid is
    // uniform: offsets of lanes are 32 bits from a scalar address, where the stride allows it.
    __device__ __forceinline__ void load(const DT* src, int64_t stride, int cols, int t0, bool rev, int n, unsigned tid) {
        if (cols == COLS && stride < 1 << 22) {
            const char* base = reinterpret_cast<const char*>(src + (int64_t)t0 * stride);
#pragma unroll
            for (int i = 0; i < CNT; ++i) {
                const unsigned at = i * THREADS + tid, row = at / PER, c = at % PER * 8;
                const unsigned r = rev ? max((int)(n - 1 - row), 0) : min((int)row, n - 1);
                if (ALL % THREADS == 0 || at < ALL)
                    v[i] = load_v<8>(reinterpret_cast<const DT*>(base + (__umul24(r, (unsigned)stride) + c) * (unsigned)sizeof(DT)));
            }
            if (n < ROWS) {
#pragma unroll
                for (int i = 0; i < CNT; ++i)
                    if ((int)((i * THREADS + tid) / PER) >= n) clear(v[i]);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            const int at = i * THREADS + (int)tid, r = at / PER, c = at % PER * 8;
            clear(v[i]);
            if (r < n && c < cols && at < ALL) {
                const DT* p = src + (int64_t)(rev ? t0 + n - 1 - r : t0 + r) * stride + c;
                if (c + 8 <= cols) {
                    v[i] = load_v<8>(p);
                } else {  // one by one, and none waits for another: elements past the row are its last, then zero
                    DT e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] = p[min(k, cols - 1 - c)];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[i].part[k / Pack<DT, 8>::N][k % Pack<DT, 8>::N] = c + k < cols ? e[k] : from_f32<DT>(0.f);
                }
            }
        }
    }
    __device__ __forceinline__ void store(bf16* dst, int ld, int plane, unsigned tid) const {
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            const unsigned at = i * THREADS + tid, r = at / PER, c = at % PER * 8;
            if (ALL % THREADS != 0 && at >= ALL) continue;
            bf16* p = dst + r * ld + c;
            if constexpr (NP == 1) {
                *reinterpret_cast<bf16x8*>(p) = __builtin_bit_cast(bf16x8, v[i]);
            } else {
                float f[8];
                get_v(v[i], f);
                const Parts<NP> s = split8<NP, true>(f);
#pragma unroll
                for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8*>(p + n * plane) = s.p[n];
            }
        }
    }
    // the same with the byte of piece p of row r from `place`; plane in bytes
    template <typename F> __device__ __forceinline__ void store_to(char* dst, int plane, unsigned tid, F place) const {
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            const unsigned at = i * THREADS + tid;
            if (ALL % THREADS != 0 && at >= ALL) continue;
            char* p = dst + place(at / PER, at % PER);
            if constexpr (NP == 1) {
                *reinterpret_cast<bf16x8*>(p) = __builtin_bit_cast(bf16x8, v[i]);
            } else {
                float f[8];
                get_v(v[i], f);
                const Parts<NP> s = split8<NP, true>(f);
#pragma unroll
                for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8*>(p + n * plane) = s.p[n];
            }
        }
    }
    // the same into rows in the paired order
    template <typename TILE> __device__ __forceinline__ void store_paired(char* dst, int plane, unsigned tid) const {
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            const unsigned at = i * THREADS + tid;
            if (ALL % THREADS != 0 && at >= ALL) continue;
            const int r = at / PER, p = at % PER;
            Parts<NP> s;
            if constexpr (NP == 1) {
                s.p[0] = __builtin_bit_cast(bf16x8, v[i]);
            } else {
                float f[8];
                get_v(v[i], f);
                s = split8<NP, true>(f);
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                char* to = dst + n * plane + TILE::half(p) * 8;
                *reinterpret_cast<bf16x4*>(to + TILE::at(r, TILE::place(p))) = __builtin_shufflevector(s.p[n], s.p[n], 0, 1, 2, 3);
                *reinterpret_cast<bf16x4*>(to + TILE::at(r, TILE::place(p) + 1)) = __builtin_shufflevector(s.p[n], s.p[n], 4, 5, 6, 7);
            }
        }
    }
    static __device__ __forceinline__ void clear(Pack<DT, 8>& p) {
#pragma unroll
        for (int k = 0; k < 8; ++k) p.part[k / Pack<DT, 8>::N][k % Pack<DT, 8>::N] = from_f32<DT>(0.f);
    }
};

// d A in units of log 2, held above -300; a NaN stays one.
__device__ __forceinline__ double log2_decay(float d, float A) {
    const double l = (double)d * (double)A * 1.4426950408889634;
    return l < -300.0 ? -300.0 : l;
}
__device__ __forceinline__ float softplus_f(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

__device__ __forceinline__ double lanes_scan(double v, int lane) {
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
        const double t = __shfl_up(v, d);
        if (lane >= d) v += t;
    }
    return v;
}

// The decays of a chunk, one token a lane: c as hi + lo and what comes of it.
template <int Q> struct Decays {
    float hi[Q], lo[Q], src[Q], from[Q], to[Q], total, pad[15];  // total: 2^{total}
    // src: d; from: 2^{c}; to: 2^{total - c}
};
template <int Q>
__device__ __forceinline__ void decays(Decays<Q>& w, const SsmArgs& a, int h, int first, int n, int lane) {
    float d = 0.f;
    double l = 0.0;
    if (lane < n) {
        const float z = a.dt[(int64_t)(first + lane) * a.dts + h] + (a.bias ? a.bias[h] : 0.f);
        d = a.softplus ? softplus_f(z) : z;
        l = log2_decay(d, a.A[h]);
    }
    const double c = lanes_scan(l, lane), total = __shfl(c, WAVE - 1);
    if (lane < Q) {
        const double hi = rint(c * 256.0) * (1.0 / 256.0);
        w.hi[lane] = (float)hi;
        w.lo[lane] = (float)(c - hi);
        w.src[lane] = d;
        w.from[lane] = exp2f((float)c);
        w.to[lane] = exp2f((float)(total - c));
        if (lane == 0) w.total = exp2f((float)total);
    }
}

// Sums of four values over the 16 lanes of a group, the n-th in every lane with lane % 4 == n: neighbours
// exchange what they give up, so that 5 additions do what 16 would.  No trip through LDS.
template <int CTRL> __device__ __forceinline__ float lane_of(float v) {
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 15, 15, false));
}
__device__ __forceinline__ float sums16(f32x4 v, int lane) {
    const bool odd = lane & 1, high = lane & 2;
    const float a = (odd ? v[1] : v[0]) + lane_of<0xb1>(odd ? v[0] : v[1]);
    const float b = (odd ? v[3] : v[2]) + lane_of<0xb1>(odd ? v[2] : v[3]);
    float s = (high ? b : a) + lane_of<0x4e>(high ? a : b);
    s += lane_of<0x124>(s);
    return s + lane_of<0x128>(s);
}

// The n-th piece of `every` tokens of each sequence has the slot start / every + sequence + n: slots
// rise with the sequence, and a sequence of L tokens has room for ceil(L / every) of them.
struct Piece { int seq, n, start, len; bool live; };
__device__ __forceinline__ Piece find_piece(const Seqs& sq, int slot, int every) {
    const int lane = threadIdx.x % WAVE;
    int lo = 0, hi = sq.N;
    while (hi - lo > 1) {
        const int step = (hi - lo + WAVE - 1) / WAVE, n = lo + (lane + 1) * step;
        const bool in = n < hi;
        const int below = __popcll(__ballot(in && sq.start(in ? n : lo) / every + (in ? n : lo) <= slot));
        lo += below * step;
        hi = hi - lo < step ? hi : lo + step;
    }
    // the same in every lane: kept in scalar registers, and so is every address that comes of them
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    Piece p;
    p.seq = uniform(lo);
    p.start = uniform(sq.start(p.seq));
    p.len = max(uniform(sq.start(p.seq + 1)) - p.start, 0);
    p.n = slot - (p.start / every + p.seq);
    p.live = p.n >= 0 && (p.n == 0 || (int64_t)p.n * every < p.len);
    return p;
}

// A launch's workgroups by (slot, group) and by four units of the group.  Workgroups of a
// (slot, group) read the same B and C; every eighth workgroup runs on the same die, so they are
// given numbers 8 apart.
struct Place { int slot, group, quad; bool live; };
__device__ __forceinline__ Place place_of(unsigned b, int slots, int G, int quads) {
    auto uniform = [](unsigned v) { return (int)__builtin_amdgcn_readfirstlane(v); };
    const unsigned pair = (b & 7) + 8 * ((b >> 3) / (unsigned)quads);
    Place p;
    p.quad = uniform((b >> 3) % (unsigned)quads);
    p.slot = uniform(pair / (unsigned)G);
    p.group = uniform(pair % (unsigned)G);
    p.live = p.slot < slots;
    return p;
}
int64_t place_blocks(int64_t slots, int G, int quads) { return (slots * G + 7) / 8 * 8 * quads; }

constexpr int OUT = 1, EMIT = 2, ENDS = 4;

// What a walk takes and gives: the values, keys and queries (x, B, C; reversed dy, C, B) and their token strides, the
// states before the first token and behind the last, those before every chunk, and its segments' own states and decays.
struct Role {
    const void *val, *key, *query;
    int64_t vs, ks, qs;
    const float* first;
    float *last, *emit, *ends, *decay;
    int rev;
};

// A value the compiler takes for a new one.  Addresses that depend on it are formed where they are used
// and not kept in registers through the walk, where the state leaves no room for them.
__device__ __forceinline__ unsigned renewed(unsigned v) {
    asm volatile("" : "+v"(v));
    return v;
}

// ROWS rows of COLS bf16 in LDS, their 16-byte pieces exchanged by the row's number so that neither a column of
// pieces (16 rows at once) nor a block of 8 rows by 16 columns (half a transposing read) meets in a bank.
template <int COLS> struct Tile {
    static constexpr int ROW = COLS * 2, PIECES = COLS / 8;
    static __device__ __forceinline__ int turn(int row) {
        if constexpr (PIECES >= 16) return (row & 7) << 1 | ((row >> 3) & 1);
        else if constexpr (PIECES == 8) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
        else if constexpr (PIECES == 4) return ((row >> 2) & 1) << 1 | ((row >> 3) & 1);
        else return (row >> 3) & 1;
    }
    // byte of piece p of a row
    static __device__ __forceinline__ int at(int row, int p) { return row * ROW + (p ^ turn(row)) * 16; }
    // 32 contraction indices of a row in the paired order
    static __device__ __forceinline__ bf16x8 row_paired(const char* m, int row, int k32, int lane) {
        const int q = lane >> 4;
        return join(*reinterpret_cast<const bf16x4*>(m + at(row, 4 * k32 + (q >> 1)) + (q & 1) * 8),
                    *reinterpret_cast<const bf16x4*>(m + at(row, 4 * k32 + 2 + (q >> 1)) + (q & 1) * 8));
    }
    // the same of a row that is stored in the paired order: piece p's two halves go to half(p) of pieces place(p) and
    // place(p) + 1
    static __device__ __forceinline__ int place(int p) { return (p & ~3) + 2 * (p & 1); }
    static __device__ __forceinline__ int half(int p) { return (p >> 1) & 1; }
    static __device__ __forceinline__ bf16x8 row_stored(const char* m, int row, int k32, int lane) {
        return *reinterpret_cast<const bf16x8*>(m + at(row, 4 * k32 + (lane >> 4)));
    }
    // 32 rows as contraction indices of 16 columns in the paired order
    static __device__ __forceinline__ bf16x8 col_paired(const char* m, int c16, int lane) {
        typedef __attribute__((address_space(3))) s16x4* lds;
        const int i = lane & 15, row = 4 * (lane >> 4) + (i >> 2);
        const char* p = m + at(row, 2 * c16 + ((i & 3) >> 1)) + (i & 1) * 8;  // row + 16 has the same turn
        return join(__builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p))),
                    __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + 16 * ROW))));
    }
};

// The waits before this barrier are those for LDS only: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The decays of a chunk of the walk, for the wavefronts of a head.
struct WalkDecays {
    float from[WALK], into[WALK], scale[WALK], hi[WALK], lo[WALK], less[WALK];
    // from: 2^{c}; into: 2^{total - c} src, src the weight of a token's product (d, reversed 1); scale: that of its result
    // (1, reversed d); c is hi + lo; less: lo - log2(src), fp32 inputs: src
    float total, pad[3];  // 2^{total} (BEHIND: the log decay of the chunks behind this one)
};

// Two chunks at once, 32 tokens each, a token a lane; returns the sum of both chunks' log decays.
// BEHIND: `into` is the weight at the end of the segment, `behind` the log decay of the chunks behind these; `sign` is the
// sign of the sum it goes to.  Otherwise the state changes its sign with every chunk, and is negative before odd ones.
template <bool EXACT, bool BEHIND>
__device__ __forceinline__ double walk_decays(WalkDecays& w, float z, float A, int softplus, bool in,
                                              bool rev, double behind, float sign, int lane) {
    const int u = lane & (WALK - 1);
    const float d = in ? (softplus ? softplus_f(z) : z) : 0.f;
    const double l = in ? log2_decay(d, A) : 0.0;
    double incl = l;
#pragma unroll
    for (int m = 1; m < WALK; m <<= 1) {
        const double t = __shfl_up(incl, m, WALK);
        if (u >= m) incl += t;
    }
    const double c = rev ? incl - l : incl, total = __shfl(incl, WALK - 1, WALK);
    const float src = in ? (rev ? 1.f : d) : 0.f;
    if (BEHIND) {
        const double other = __shfl(total, 0);
        behind += lane >= WALK ? other : 0.0;
        w.into[u] = exp2f((float)(behind + (total - c))) * (src * sign);
        if (u == 0) w.total = (float)behind;
        return total + __shfl_xor(total, WALK);
    }
    const float odd = lane >= WALK ? -1.f : 1.f;
    w.from[u] = exp2f((float)c) * odd;
    w.into[u] = exp2f((float)(total - c)) * (src * -odd);
    w.scale[u] = rev ? d : 1.f;
    const double hi = rint(c * 256.0) * (1.0 / 256.0);
    const float lo = (float)(c - hi);
    w.hi[u] = (float)hi;
    w.lo[u] = lo;
    w.less[u] = EXACT ? src : lo - __log2f(src);
    if (u == 0) w.total = -exp2f((float)total);
    return total + __shfl_xor(total, WALK);
}

// One wavefront per unit walks the chunks of a segment, its state in accumulator tiles [k][p].
// OUT: writes the results; EMIT: the state before every chunk of a.chunk tokens; ENDS: starts from zero and
// writes the segment's own state and decay (not for a sequence's last segment).
//
// What bounds it: instruction issue.  For 65536 tokens of 32 heads OUT issues 177e6 vector and 19e6 matrix instructions, 288
// and 121 us on 1024 SIMDs at 2.4 GHz (4 and 16 cycles each), and takes 535; the two hardly overlap.  It moves
// 1.15 GB, 2.2 TB/s.  ENDS 42e6 and 7e6: 68 and 44 us of 185.  Vector instructions are the splitting of the state and the decayed rows into parts (3 instructions a pair and
// part), the scaling of the state, and a sixth the masked products.
//
// A unit is narrow, 64 registers of state, so that three wavefronts share a SIMD: with twice the columns two did,
// and waited for LDS and each other (with two of this size on a SIMD 764 us against 589, 2 x 32768 tokens of 32 heads).  The wavefronts of a
// workgroup that have the same head form the masked products once between them, in LDS.  Chunks of 32 tokens;
// with bf16 inputs the next chunk's rows are on their way in registers while one is multiplied.
//
// Heads of a workgroup, whose first unit's number in the group is a multiple of four: two of two blocks each, and any more
// blocks leave room for parts of two.  So two workgroups in fp32 share a compute unit (K <= 64: 70 KB, with room for
// four heads 90; forward and gradient of 6007 tokens of 10 heads of 40 x 50 242 us and 261).
__host__ __device__ constexpr int walk_heads(int blocks) { return blocks == 1 ? WAVES : 2; }

template <typename DT, int KT, int PT, int MODE>
__device__ __forceinline__ void walk_segment(const SsmArgs& a, const Role& role, int slots, int quads) {
    using C_ = Cfg<DT>;
    using TK = Tile<KT * 16>;
    using TP = Tile<PT * 16>;
    constexpr int Q = WALK, NP = C_::NP, MP = C_::MP, HP = C_::HP;
    constexpr bool AHEAD = NP == 1;
    const DT *const val = (const DT*)role.val, *const key = (const DT*)role.key, *const query = (const DT*)role.query;
    const int64_t vs = role.vs, ks = role.ks, qs = role.qs;
    const float* const first_state = role.first;
    float *const last_state = role.last, *const emit = role.emit;
    const int rev = role.rev;
    constexpr int PLK = Q * TK::ROW, PLP = Q * TP::ROW, PLM = Q * Q * 2;  // bytes of a plane
    constexpr int KEYS = NP * PLK, QUERIES = (MODE & OUT) ? KEYS : 0, VALS = NP * PLP, MASKED = (MODE & OUT) ? MP * PLM : 0;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char* const skey = smem;
    char* const squery = skey + KEYS;
    char* const svals = squery + QUERIES;
    char* const smasked = svals + WAVES * VALS;
    const int heads = walk_heads(a.wblocks);  // that a workgroup may have
    WalkDecays* const sdec = reinterpret_cast<WalkDecays*>(smasked + heads * MASKED);  // [head][chunk & 3]

    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int l15 = lane & 15, q4 = lane >> 4;
    const Place at = place_of(blockIdx.x, slots, a.G, quads);
    if (!at.live) return;
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const Piece pc = find_piece(sq, at.slot, a.seg);
    if (!pc.live) return;
    const int per = a.H / a.G, units = per * a.wblocks, unit_in = at.quad * WAVES + wave;
    const bool mine = unit_in < units;
    const int unit = at.group * units + (mine ? unit_in : 0);
    const int h = unit / a.wblocks, block = unit % a.wblocks, p0 = block * (PT * 16);
    // the workgroup's wavefronts with this head: `team` of them from `lead` on, this one the who-th
    const int lead = mine ? max(wave - block, 0) : wave, who = wave - lead;
    const int team = mine ? min(min(lead + a.wblocks - (block - who), WAVES), units - at.quad * WAVES) - lead : 1;
    const bool decides = mine && who == team - 1;  // forms the head's decays
    const int share = team == 1 ? 7 : team == 2 ? (who ? 2 : 5) : who < 3 ? 1 << who : 0;  // of the masked products' tiles
    // the leads of the workgroup's heads
    int leads = 0;
#pragma unroll
    for (int o = 0; o < WAVES; ++o) {
        const int u = at.quad * WAVES + o;
        if (u < units && (o == 0 || u % a.wblocks == 0)) leads |= 1 << o;
    }
    const int segs = max((pc.len + a.seg - 1) / a.seg, 1);
    const bool is_last = pc.n == (rev ? 0 : segs - 1), is_first = pc.n == (rev ? segs - 1 : 0);
    if ((MODE & ENDS) && is_last) return;
    const int t0 = pc.n * a.seg, t1 = min(t0 + a.seg, pc.len), chunks = (t1 - t0 + Q - 1) / Q;
    const int64_t frag = ((int64_t)at.slot * a.H * a.wblocks + unit) * (KT * PT * WAVE) + lane;

    char* const sval = svals + wave * VALS;
    const int own = mine ? __builtin_popcount(leads & ((1 << lead) - 1)) : 0;  // the head's number in the workgroup
    char* const sm = smasked + own * MASKED;
    WalkDecays* const dec = sdec + 4 * own;
    f32x4 st[KT][PT];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int p = 0; p < PT; ++p) st[k][p] = zero4();
    if (!(MODE & ENDS) && mine) {
        if (!is_first) {
            const f32x4* e = reinterpret_cast<const f32x4*>(role.ends);
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int p = 0; p < PT; ++p) st[k][p] = e[frag + (k * PT + p) * WAVE];
        } else if (first_state) {
            const float* f = first_state + ((int64_t)pc.seq * a.H + h) * a.K * a.P;
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int p = 0; p < PT; ++p)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int kk = 16 * k + 4 * q4 + r, pp = p0 + 16 * p + l15;
                        if (kk < a.K && pp < a.P) st[k][p][r] = f[kk * a.P + pp];
                    }
        }
    }
    if (MODE & OUT) {  // the tile above the diagonal stays zero
        for (int i = threadIdx.x * 16; i < heads * MASKED; i += NT * 16) *reinterpret_cast<f32x4*>(smasked + i) = zero4();
    }
    const float dskip = (MODE & OUT) && a.D && mine ? a.D[h] : 0.f;
    const float A = a.A[h], bias = a.bias ? a.bias[h] : 0.f;
    double log_decay = 0.0;

    // Chunk ci in the order of the walk: its first token in that order, and how many it has.  What a segment adds is
    // the sum of its tokens' products, each with the decay from there to the segment's end, so ENDS takes the chunks
    // from the end: weights come whole and the state is never scaled.
    struct Chunk { int index, t0, first, n; };
    auto chunk_at = [&](int ci) {
        Chunk c;
        c.index = (rev != 0) != ((MODE & ENDS) != 0) ? chunks - 1 - ci : ci;
        c.t0 = pc.start + t0 + c.index * Q;
        c.n = min(Q, pc.start + t1 - c.t0);
        c.first = rev ? c.t0 + c.n - 1 : c.t0;
        return c;
    };
    const int dir = rev ? -1 : 1;
    // A matrix instruction's additions are off towards one side, by a tenth of a unit in the last place, in every element
    // alike: little, but sums over the whole state gather it (dA).  So the state is held with the other sign half of the
    // time, where it is scaled anyway in every other chunk, in ENDS over the first half of the chunks.
    const int turn = chunks / 2;
    auto negate = [&]() {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int p = 0; p < PT; ++p) st[k][p] = -st[k][p];
    };
    bool positive = turn == 0;  // ENDS
    // dt of chunks ci and ci + 1, a token a lane
    auto steps_of = [&](int ci) {
        const Chunk c = chunk_at(ci + (lane >> 5));
        const bool in = ci + (lane >> 5) < chunks && (lane & 31) < c.n;
        return in ? a.dt[(int64_t)(c.first + (lane & 31) * dir) * a.dts + h] : 0.f;
    };
    auto decays_of = [&](int ci, float raw) {
        const Chunk c = chunk_at(ci + (lane >> 5));
        const bool in = ci + (lane >> 5) < chunks && (lane & 31) < c.n;
        const int to = (ci & 2) + (lane >> 5);
        const float sign = ci + (lane >> 5) < turn ? -1.f : 1.f;
        log_decay += walk_decays<NP != 1, (MODE & ENDS) != 0>(dec[to], raw + bias, A, a.softplus, in, rev, log_decay, sign, lane);
    };

    Stage<DT, Q, KT * 16, NT> bk, bq;
    Stage<DT, Q, PT * 16, WAVE> bv;
    auto load = [&](const Chunk& c) {
        const unsigned tid = renewed(threadIdx.x);
        bk.load(key + (int64_t)at.group * a.K, ks, a.K, c.t0, rev, c.n, tid);
        if (MODE & OUT) bq.load(query + (int64_t)at.group * a.K, qs, a.K, c.t0, rev, c.n, tid);
        bv.load(val + (int64_t)h * a.P + p0, vs, min(a.P - p0, PT * 16), c.t0, rev, c.n, tid % WAVE);
    };
    auto store = [&]() {
        const unsigned tid = renewed(threadIdx.x);
        bk.store_to(skey, PLK, tid, [](int r, int p) { return TK::at(r, p); });
        if (MODE & OUT) bq.template store_paired<TK>(squery, PLK, tid);
        bv.store_to(sval, PLP, tid % WAVE, [](int r, int p) { return TP::at(r, p); });
    };
    float raw = 0.f;
    if (chunks > 0) {
        if (AHEAD) load(chunk_at(0));
        if (decides) {
            raw = steps_of(0);
            decays_of(0, raw);
        }
    }

    for (int ci = 0; ci < chunks; ++ci) {
        const Chunk c = chunk_at(ci);
        const int n = c.n;
        if (!AHEAD) load(c);
        if (ci) lds_barrier();  // the last chunk's tiles are read
        store();
        lds_barrier();
        if (AHEAD && ci + 1 < chunks) load(chunk_at(ci + 1));
        if (decides && !(ci & 1)) raw = steps_of(ci + 2);
        const WalkDecays& w = dec[ci & 3];
        if (MODE & ENDS) {
            // Past 2^-150 every weight of this chunk and of those before it is zero in fp32: the sum is done, for
            // the workgroup where it is for each of its heads.
            float most = -INFINITY;
#pragma unroll
            for (int o = 0; o < WAVES; ++o)
                if (o < __builtin_popcount(leads)) most = fmaxf(most, sdec[4 * o + (ci & 3)].total);
            if (most < -152.f) break;
            if (ci == turn && turn) {
                negate();
                positive = true;
            }
        }

        if ((MODE & EMIT) && mine) {
            const int ev = a.chunk / Q;
            if (rev ? c.index % ev == ev - 1 || ci == 0 : c.index % ev == 0) {
                const int64_t cslot = pc.start / a.chunk + pc.seq + (t0 / a.chunk + c.index / ev);
                const int wide = a.blocks * a.cols;
                float* e = emit + (cslot * a.H + h) * ((int64_t)KT * 16 * wide) + p0;
                const int own = renewed(4 * q4 * wide + l15);
                const float sign = ci & 1 ? -1.f : 1.f;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int p = 0; p < PT; ++p) e[own + (16 * k + r) * wide + 16 * p] = st[k][p][r] * sign;
            }
        }

        f32x4 acc[2][PT];  // results transposed, [p][t]: a lane holds 4 neighbouring columns of token 16 j + l15
        if constexpr ((MODE & OUT) != 0) {
            if (mine) {
                // this wavefront's share of the masked products' three tiles
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    constexpr int J[3] = {1, 1, 0}, I[3] = {0, 1, 0};
                    if (!(share & 1 << x)) continue;
                    const int lane = renewed(threadIdx.x) % WAVE, l15 = lane & 15, q4 = lane >> 4;
                    const int t = 16 * J[x] + l15, s0 = 16 * I[x] + 4 * q4;
                    f32x4 s = zero4();
#pragma unroll
                    for (int kk = 0; kk < KT / 2; ++kk) {
                        Parts<NP> qf, kf;
#pragma unroll
                        for (int m = 0; m < NP; ++m) {
                            qf.p[m] = TK::row_stored(squery + m * PLK, t, kk, lane);
                            kf.p[m] = TK::row_paired(skey + m * PLK, 16 * I[x] + l15, kk, lane);
                        }
                        s = mma_parts(kf, qf, s);
                    }
                    float v[4];
                    const float hi_t = w.hi[t], lo_t = w.lo[t];
                    const f32x4 hi = *reinterpret_cast<const f32x4*>(&w.hi[s0]), less = *reinterpret_cast<const f32x4*>(&w.less[s0]);
                    if constexpr (NP == 1) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = s[r] * __builtin_amdgcn_exp2f((hi_t - hi[r]) + (lo_t - less[r]));
                    } else {
                        const f32x4 lo = *reinterpret_cast<const f32x4*>(&w.lo[s0]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[r] = s[r] * (__builtin_amdgcn_exp2f((hi_t - hi[r]) + (lo_t - lo[r])) * less[r]);
                    }
                    if (I[x] == J[x]) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = 4 * q4 + r <= l15 ? v[r] : 0.f;
                    }
                    char* to = sm + t * (Q * 2) + ((q4 ^ ((t >> 1) & 3)) * 16) + I[x] * 8;
#pragma unroll
                    for (int m = 0; m < MP; ++m) {
                        uint32_t a0, a1;
                        pack4<(NP > 1)>(v, m, a0, a1);
                        *reinterpret_cast<uint2*>(to + m * PLM) = make_uint2(a0, a1);
                        v[0] -= low_of(a0);
                        v[1] -= high_of(a0);
                        v[2] -= low_of(a1);
                        v[3] -= high_of(a1);
                    }
                }
                // the state's part of the results
                const int lane = renewed(threadIdx.x) % WAVE, l15 = lane & 15;
#pragma unroll
                for (int kk = 0; kk < KT / 2; ++kk) {
                    Parts<NP> qf[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int m = 0; m < NP; ++m) qf[j].p[m] = TK::row_stored(squery + m * PLK, 16 * j + l15, kk, lane);
#pragma unroll
                    for (int p = 0; p < PT; ++p) {
                        float v[8];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            v[r] = st[2 * kk][p][r];
                            v[4 + r] = st[2 * kk + 1][p][r];
                        }
                        const Parts<HP> hf = split8<HP, (NP > 1)>(v);
#pragma unroll
                        for (int j = 0; j < 2; ++j) acc[j][p] = mma_parts(hf, qf[j], kk ? acc[j][p] : zero4());
                    }
                }
            }
            lds_barrier();  // the masked products are there
        }
        if (mine) {
            Parts<NP> vf[PT];
#pragma unroll
            for (int p = 0; p < PT; ++p)
#pragma unroll
                for (int m = 0; m < NP; ++m) vf[p].p[m] = TP::col_paired(sval + m * PLP, p, lane);
            if constexpr ((MODE & OUT) != 0) {
                const int lane = renewed(threadIdx.x) % WAVE, l15 = lane & 15, q4 = lane >> 4;
                const int token = a.H * a.P;
                DT* const out = reinterpret_cast<DT*>(a.y) + ((int64_t)c.t0 * a.H + h) * a.P + p0;
                const bool whole = n == Q && p0 + PT * 16 <= a.P && token < 1 << 22;  // no conditions by lane
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int t = 16 * j + l15;
                    const float from = w.from[t], scale = w.scale[t];
                    Parts<MP> mf;
#pragma unroll
                    for (int m = 0; m < MP; ++m)
                        mf.p[m] = *reinterpret_cast<const bf16x8*>(sm + m * PLM + t * (Q * 2) + ((q4 ^ ((t >> 1) & 3)) * 16));
                    const unsigned row = rev ? n - 1 - t : t;
#pragma unroll
                    for (int p = 0; p < PT; ++p) {
                        acc[j][p] = mma_parts(vf[p], mf, acc[j][p] * from);
                        if (rev) acc[j][p] *= scale;
                        const int col = 16 * p + 4 * q4;
                        float o[4];
                        zero_v(o);
#pragma unroll
                        for (int m = NP - 1; m >= 0; --m) {
                            const uint2 v = *reinterpret_cast<const uint2*>(sval + m * PLP + TP::at(t, 2 * p + (q4 >> 1)) + (q4 & 1) * 8);
                            const float f[4] = {low_of(v.x), high_of(v.x), low_of(v.y), high_of(v.y)};
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[r] = m + 1 < NP ? o[r] + f[r] : f[r];
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[r] = acc[j][p][r] + dskip * o[r];
                        if (whole) {
                            store_v<4>(reinterpret_cast<DT*>(reinterpret_cast<char*>(out) + (__umul24(row, (unsigned)token) + col) * (unsigned)sizeof(DT)), o);
                        } else if (t < n) {
                            DT* to = out + (int64_t)row * token + col;
                            if (p0 + col + 4 <= a.P) {
                                store_v<4>(to, o);
                            } else {
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (p0 + col + r < a.P) to[r] = from_f32<DT>(o[r]);
                            }
                        }
                    }
                }
            }
            // the state behind the chunk
            const int lane = renewed(threadIdx.x) % WAVE, q4 = lane >> 4;
            const float total = w.total;
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(&w.into[4 * q4]), w1 = *reinterpret_cast<const f32x4*>(&w.into[16 + 4 * q4]);
            Parts<3> xf[PT];
#pragma unroll
            for (int p = 0; p < PT; ++p) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[r] = (float)vf[p].p[NP - 1][r];
#pragma unroll
                    for (int m = NP - 2; m >= 0; --m) v[r] += (float)vf[p].p[m][r];
                    v[r] *= r < 4 ? w0[r] : w1[r - 4];
                }
                xf[p] = split8<3, (NP > 1)>(v);
            }
            // products that add to one tile wait for each other: two tiles' rows side by side, a part at a time
#pragma unroll
            for (int k = 0; k < KT; k += 2) {
                Parts<NP> kf[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int m = 0; m < NP; ++m) kf[i].p[m] = TK::col_paired(skey + m * PLK, k + i, lane);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < PT; ++p)
                        if (!(MODE & ENDS)) st[k + i][p] *= total;
#pragma unroll
                for (int m = 0; m < NP; ++m)
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        if (m + x <= 2) {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int p = 0; p < PT; ++p)
                                    st[k + i][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i].p[m], xf[p].p[x], st[k + i][p], 0, 0, 0);
                        }
            }
            if (decides && (ci & 1) && ci + 1 < chunks) decays_of(ci + 1, raw);
        }
    }
    if (!mine) return;
    if (MODE & ENDS) {
        if (!positive) negate();
        f32x4* e = reinterpret_cast<f32x4*>(role.ends);
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int p = 0; p < PT; ++p) e[frag + (k * PT + p) * WAVE] = st[k][p];
        if (lane == 0 && decides && block == who) role.decay[(int64_t)at.slot * a.H + h] = exp2f((float)log_decay);
    } else if (is_last && last_state) {
        if (chunks & 1) negate();
        float* f = last_state + ((int64_t)pc.seq * a.H + h) * a.K * a.P;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int p = 0; p < PT; ++p)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kk = 16 * k + 4 * q4 + r, pp = p0 + 16 * p + l15;
                    if (kk < a.K && pp < a.P) f[kk * a.P + pp] = st[k][p][r];
                }
    }
}

// Two walks of one kind side by side, or (BOTH) the gradient's, which need nothing from each other: the longer first.  In one
// launch each the 6007 tokens take 216 us, one after another 242 (ENDS and join together 230); 2 x 8192 979 and 994.
constexpr int BOTH = 8;
template <typename DT, int KT, int PT, int MODE>
__global__ void __launch_bounds__(NT, sizeof(DT) == 2 ? 3 : 2)
ssm_walk_kernel(SsmArgs a, Role one, Role two, int slots, int quads) {
    if constexpr (MODE == BOTH) {
        if (blockIdx.y) walk_segment<DT, KT, PT, EMIT>(a, two, slots, quads);
        else walk_segment<DT, KT, PT, OUT | EMIT>(a, one, slots, quads);
    } else {
        walk_segment<DT, KT, PT, MODE>(a, (MODE & ENDS) && blockIdx.y ? two : one, slots, quads);
    }
}

// Joins the segments of a sequence: ends[slot] holds what the segment adds from a zero state and becomes
// the state it starts from.  Four elements a thread, the next segment's on their way.  One read and one write of the segments'
// states (92 MB in 18 us, 2 x 32768 tokens in 22 segments, 5.1 TB/s).
__global__ void __launch_bounds__(NT) ssm_join_kernel(SsmArgs a, Role one, Role two, int per_unit, int pieces) {
    const Role& role = blockIdx.y ? two : one;
    const float* const first_state = role.first;
    const int rev = role.rev;
    const int64_t units = (int64_t)a.H * a.wblocks;
    for (int64_t b = blockIdx.x; b < a.N * units * pieces; b += gridDim.x) {
    const int piece = (int)(b % pieces), unit = (int)(b / pieces % units), seq = (int)(b / pieces / units);
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int start = sq.start(seq), len = sq.start(seq + 1) - start;
    const int segs = (max(len, 0) + a.seg - 1) / a.seg;
    const int e = piece * NT + threadIdx.x;
    if (segs < 2 || e >= per_unit) continue;
    const int h = unit / a.wblocks, tiles = a.wcols / 16;
    const int lane = e % WAVE, tile = e / WAVE;
    f32x4 cur = zero4();
    if (first_state) {
        const int k0 = 16 * (tile / tiles) + 4 * (lane >> 4), p = unit % a.wblocks * a.wcols + 16 * (tile % tiles) + (lane & 15);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (k0 + r < a.K && p < a.P) cur[r] = first_state[(((int64_t)seq * a.H + h) * a.K + k0 + r) * a.P + p];
    }
    const int64_t slot = start / a.seg + seq;
    f32x4* ends = reinterpret_cast<f32x4*>(role.ends);
    auto at = [&](int j) { return ((slot + (rev ? segs - 1 - j : j)) * units + unit) * per_unit + e; };
    auto dec = [&](int j) { return role.decay[(slot + (rev ? segs - 1 - j : j)) * a.H + h]; };
    f32x4 nxt = ends[at(0)];
    float nd = dec(0);
    for (int j = 0; j + 1 < segs; ++j) {
        const f32x4 own = nxt;
        const float d = nd;
        if (j + 2 < segs) {
            nxt = ends[at(j + 1)];
            nd = dec(j + 1);
        }
        cur = cur * d + own;
        ends[at(j + 1)] = cur;
    }
    }
}

// row, col: of the products of two tiles, col also of a tile's with itself; near: a tile's own part of the derivative of
// its tokens' log decays; far: row of the tiles (3, 0) and (2, 0)
template <int Q> struct GradSums {
    float row[WAVES][Q], col[WAVES][Q], ui[WAVES][Q], vi[WAVES][Q], own[Q], near[Q + 1], far[2][16], xy[Q], hg[WAVES];
};

// The decays of every chunk and head, for the gradient: a wavefront each.
template <typename DT>
__global__ void __launch_bounds__(NT) ssm_decay_kernel(SsmArgs a, int slots) {
    constexpr int Q = Cfg<DT>::QT * 16;
    const int lane = threadIdx.x % WAVE;
    const int64_t i = (int64_t)blockIdx.x * WAVES + threadIdx.x / WAVE;
    if (i >= (int64_t)slots * a.H) return;
    const int slot = __builtin_amdgcn_readfirstlane((int)(i / a.H)), h = __builtin_amdgcn_readfirstlane((int)(i % a.H));
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const Piece pc = find_piece(sq, slot, Q);
    if (!pc.live || pc.len == 0) return;
    const int c0 = pc.start + pc.n * Q, n = min(Q, pc.len - pc.n * Q);
    decays<Q>(reinterpret_cast<Decays<Q>*>(a.dec)[i], a, h, c0, n, lane);
}

// The gradient that needs the states from both sides, a workgroup per chunk and share of a group's
// units.  With M[t][s] = (C_t . B_s) 2^{c_t - c_s} and E[t][s] = dy_t . x_s, s <= t, h the state
// before the chunk and g the derivative behind it:
//   dC_t = sum_s (E 2^{..} d_s)[t][s] B_s + 2^{c_t} dy_t h^T
//   dB_s = sum_t (E 2^{..} d_s)[t][s] C_t + d_s 2^{c_Q - c_s} x_s g^T
//   d(d_s) = sum_t (M E)[t][s] + 2^{c_Q - c_s} B_s . (x_s g^T)      (without the decays)
//   dl_t = sum of d_s (M E)[r][s] over r >= t > s + sum_{r >= t} 2^{c_r} C_r . (dy_r h^T)
//          + sum_{s < t} d_s 2^{c_Q - c_s} B_s . (x_s g^T) + 2^{c_Q} h . g
// dB and dC are summed over the group's heads in registers.  The wavefronts share a unit: each forms up to
// three 16 x 16 tiles of E and its products (in LDS as bf16 parts; C . B, the same for all heads, stays in
// registers), then a quarter of the columns of dB and dC, so no sum crosses wavefronts but those of single
// numbers a token, which ssm_tokens_kernel puts together.
//
// 2 x 8192 tokens of 32 heads of 128 x 128, bf16: 470 us of 1025 (walks 355, ENDS 140, joins 30, tokens 17, decays 9, sums 4).  Vector issue 179 us (110e6 instructions), matrix 54, LDS 107 (66e6 cycles on 256 compute units), and
// it reads 1.4 GB, most of it the chunks' states, 3.4 TB/s: no one resource, but the phases of a unit behind each other at
// two wavefronts a SIMD.
template <typename DT, int KT, int PT>
__global__ void __launch_bounds__(NT, 2) ssm_grad_kernel(SsmArgs a, int slots, int quads) {
    using C_ = Cfg<DT>;
    constexpr int QT = C_::QT, Q = QT * 16, NP = C_::NP, MP = C_::GP;
    constexpr int LDK = KT * 16 + 8, LDP = PT * 16 + 8, LDQ = Q + 8, PLK = Q * LDK, PLP = Q * LDP, PLQ = Q * LDQ;
    constexpr int KW = KT < WAVES ? 1 : KT / WAVES;  // column tiles of a wavefront
    using Sums = GradSums<Q>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    bf16* sb = reinterpret_cast<bf16*>(smem);
    bf16* sc = sb + NP * PLK;
    bf16* sx = sc + NP * PLK;
    bf16* sdy = sx + NP * PLP;
    bf16* sds = sdy + NP * PLP;
    Decays<Q>& dec = *reinterpret_cast<Decays<Q>*>(sds + MP * PLQ);
    Sums& sum = *reinterpret_cast<Sums*>(&dec + 1);

    const int tid = threadIdx.x, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int l15 = lane & 15, q4 = lane >> 4;
    const Place at = place_of(blockIdx.x, slots, a.G, quads);
    if (!at.live) return;
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const Piece pc = find_piece(sq, at.slot, Q);
    if (!pc.live || pc.len == 0) return;
    const int c0 = pc.start + pc.n * Q, n = min(Q, pc.len - pc.n * Q);
    const int units = a.H / a.G * a.blocks;
    const int u0 = (int)((int64_t)at.quad * units / quads), u1 = (int)((int64_t)(at.quad + 1) * units / quads);
    const int64_t all_units = (int64_t)a.H * a.blocks;

    Stage<DT, Q, PT * 16, NT> bx, by;  // the next unit's, on their way
    float nd[5];
    auto fetch = [&](int un, unsigned tid) {
        const int unit = at.group * units + un, h = unit / a.blocks, p0 = unit % a.blocks * (PT * 16);
        const int cols = min(a.P - p0, PT * 16);
        bx.load((const DT*)a.x + (int64_t)h * a.P + p0, a.xs, cols, c0, false, n, tid);
        by.load((const DT*)a.dy + (int64_t)h * a.P + p0, a.dys, cols, c0, false, n, tid);
        if (tid < Q) {
            const float* d = reinterpret_cast<const float*>(&reinterpret_cast<const Decays<Q>*>(a.dec)[(int64_t)at.slot * a.H + h]);
#pragma unroll
            for (int i = 0; i < 5; ++i) nd[i] = d[i * Q + tid];
        }
    };
    {
        Stage<DT, Q, KT * 16, NT> bk, bq;
        bk.load((const DT*)a.B + (int64_t)at.group * a.K, a.bs, a.K, c0, false, n, tid);
        bq.load((const DT*)a.C + (int64_t)at.group * a.K, a.cs, a.K, c0, false, n, tid);
        fetch(u0, tid);
        bk.store(sb, LDK, PLK, tid);
        bq.store(sc, LDK, PLK, tid);
        // what no tile writes stays zero: products above the diagonal, sums that a wavefront has no part in
        for (int i = tid; i < MP * PLQ / 2; i += NT) reinterpret_cast<uint32_t*>(sds)[i] = 0;
        for (int i = tid; i < (int)(sizeof(Sums) / 4); i += NT) reinterpret_cast<uint32_t*>(&sum)[i] = 0;
    }
    __syncthreads();

    // the wavefront's tiles (rows j, columns i), no two with the same columns
    constexpr int NTILE = QT == 4 ? 3 : 1;
    const int tiles = QT == 4 ? (wave == 0 || wave == 3 ? 2 : 3) : (wave < 3 ? 1 : 0);
    auto tile_j = [&](int x) { return QT == 4 ? (wave == 0 ? 3 : wave == 1 ? (x < 2 ? 3 : 0) : wave == 2 ? 2 : 1) : (wave < 2 ? 1 : 0); };
    auto tile_i = [&](int x) { return QT == 4 ? (wave == 1 ? (x < 2 ? 2 + x : 0) : x) : (wave == 1 ? 1 : 0); };
    f32x4 cb[NTILE];  // C . B
#pragma unroll
    for (int x = 0; x < NTILE; ++x) {
        cb[x] = zero4();
        if (x >= tiles) continue;
        const int t = 16 * tile_j(x) + l15, s = 16 * tile_i(x) + l15;
#pragma unroll
        for (int kk = 0; kk < KT / 2; ++kk) {
            Parts<NP> f, c;
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                f.p[m] = row_natural(sb + m * PLK + s * LDK + 32 * kk, lane);
                c.p[m] = row_natural(sc + m * PLK + t * LDK + 32 * kk, lane);
            }
            cb[x] = mma_parts(f, c, cb[x]);
        }
    }
    f32x4 dB[QT][KW], dC[QT][KW];
#pragma unroll
    for (int j = 0; j < QT; ++j)
#pragma unroll
        for (int k = 0; k < KW; ++k) dB[j][k] = dC[j][k] = zero4();

    for (int un = u0; un < u1; ++un) {
        const int unit = at.group * units + un, h = unit / a.blocks;
        // The last unit's products are read (its third barrier); the states are on their way through the first phase.
        {
            const unsigned tid = renewed(threadIdx.x);
            bx.store(sx, LDP, PLP, tid);
            by.store(sdy, LDP, PLP, tid);
            if (tid < Q) {
                float* d = reinterpret_cast<float*>(&dec);
#pragma unroll
                for (int i = 0; i < 5; ++i) d[i * Q + tid] = nd[i];
            }
            if (un + 1 < u1) fetch(un + 1, tid);
        }
        Pack<float, 8> hv[PT / 2], gv[PT / 2];
        auto states = [&](int k) {
            const int64_t cslot = pc.start / Q + pc.seq + pc.n;
            const int wide = a.blocks * (PT * 16);
            const int64_t state = (cslot * a.H + h) * ((int64_t)KT * 16 * wide) + (wave * KW + k) * 16 * wide + unit % a.blocks * (PT * 16);
            const int left = a.wblocks * a.wcols - unit % a.blocks * (PT * 16);
            const unsigned lane = renewed(threadIdx.x) % WAVE, own = (lane & 15) * wide + 8 * (lane >> 4);
            const float *ph = a.hs + state, *pg = a.gs + state;
#pragma unroll
            for (int pp = 0; pp < PT / 2; ++pp) {
                hv[pp] = load_v<8>(ph + (own + 32 * pp));
                gv[pp] = load_v<8>(pg + (own + 32 * pp));
            }
            if (left < PT * 16) {  // columns that no unit of the walk has written
#pragma unroll
                for (int pp = 0; pp < PT / 2; ++pp)
                    if ((int)(32 * pp + 8 * (lane >> 4)) >= left) {
                        hv[pp] = Pack<float, 8>{};
                        gv[pp] = Pack<float, 8>{};
                    }
            }
        };
        if (wave * KW < KT) states(0);
        __syncthreads();

        // tiles of E, transposed: a lane holds 4 s of one t
#pragma unroll
        for (int x = 0; x < NTILE; ++x) {
            if (x >= tiles) continue;
            const int j = tile_j(x), i = tile_i(x);
            const int lane = renewed(threadIdx.x) % WAVE, l15 = lane & 15, q4 = lane >> 4;
            const int t = 16 * j + l15, s0 = 16 * i + 4 * q4;
            f32x4 e = zero4();
#pragma unroll
            for (int pp = 0; pp < PT / 2; ++pp) {
                Parts<NP> f, y;
#pragma unroll
                for (int m = 0; m < NP; ++m) {
                    f.p[m] = row_natural(sx + m * PLP + (16 * i + l15) * LDP + 32 * pp, lane);
                    y.p[m] = row_natural(sdy + m * PLP + t * LDP + 32 * pp, lane);
                }
                e = mma_parts(f, y, e);
            }
            const float hi = dec.hi[t], lo = dec.lo[t];
            const f32x4 shi = *reinterpret_cast<const f32x4*>(&dec.hi[s0]);
            const f32x4 slo = *reinterpret_cast<const f32x4*>(&dec.lo[s0]);
            const f32x4 src = *reinterpret_cast<const f32x4*>(&dec.src[s0]);
            float row = 0.f, v[4];
            f32x4 zs, before;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = i < j || 4 * q4 + r <= l15;
                const float le = in ? __builtin_amdgcn_exp2f((hi - shi[r]) + (lo - slo[r])) * e[r] : 0.f;
                v[r] = le * src[r];
                float z = le * cb[x][r];
                if (i == j && 4 * q4 + r == l15) {
                    // a token's own product: in the derivative of its step, in no decay's
                    sum.xy[t] = e[r];
                    sum.own[t] = z;
                    z = 0.f;
                }
                row += z * src[r];
                before[r] = row;
                zs[r] = z;
            }
            if (i == j) {
                // token j + 1's decay is in the products of rows behind j with columns up to j: running sums over the
                // columns, added over the rows
                const float one = __shfl_up(row, 16), pair = row + (q4 >= 1 ? one : 0.f);
                const float two = __shfl_up(pair, 32), up = __shfl_up(pair + (q4 >= 2 ? two : 0.f), 16);
                const float left = q4 >= 1 ? up : 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) before[r] = 4 * q4 + r < l15 ? left + before[r] : 0.f;
                const float o = sums16(before, lane);
                if (l15 < 4) sum.near[s0 + l15 + 1] = o;
            }
            const float c = sums16(zs, lane);  // over the tile's 16 tokens t
            if (l15 < 4) sum.col[wave][s0 + l15] = c;
#pragma unroll
            for (int m = 0; m < MP; ++m) {
                uint32_t a0, a1;
                pack4<(NP > 1)>(v, m, a0, a1);
                *reinterpret_cast<uint2*>(sds + m * PLQ + t * LDQ + s0) = make_uint2(a0, a1);
                if (m + 1 < MP) {
                    v[0] -= low_of(a0);
                    v[1] -= high_of(a0);
                    v[2] -= low_of(a1);
                    v[3] -= high_of(a1);
                }
            }
            if (i == j) continue;
            row += __shfl_xor(row, 16);
            row += __shfl_xor(row, 32);
            if (q4 == 0) {
                // tiles of the same rows follow each other
                sum.row[wave][t] = x > 0 && tile_j(x) == tile_j(x - 1) ? sum.row[wave][t] + row : row;
                if (QT == 4 && x == 0 && i == 0 && j > 1) sum.far[j == 2][l15] = row;
            }
        }
        __syncthreads();

        // the wavefront's columns of dB and dC
        float hg = 0.f;
        if (wave * KW < KT) {
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const int lane = renewed(threadIdx.x) % WAVE, l15 = lane & 15, q4 = lane >> 4;
                const int kt = wave * KW + k;
                Parts<3> hf[PT / 2], gf[PT / 2];
#pragma unroll
                for (int pp = 0; pp < PT / 2; ++pp) {
                    float hx[8], gx[8];
                    get_v(hv[pp], hx);
                    get_v(gv[pp], gx);
#pragma unroll
                    for (int r = 0; r < 8; ++r) hg += hx[r] * gx[r];
                    hf[pp] = split8<3, (NP > 1)>(hx);
                }
                // sums over the wavefront's columns go to its own row: lane n of 4 holds row n's
                auto add = [&](float (&to)[Q], int t, f32x4 v) {
                    const float u = sums16(v, lane);
                    if (l15 < 4) to[t + l15] = k ? to[t + l15] + u : u;
                };
#pragma unroll
                for (int j = 0; j < QT; ++j) {
                    const int t = 16 * j + 4 * q4;
                    f32x4 tc = zero4(), cv = zero4();
#pragma unroll
                    for (int pp = 0; pp < PT / 2; ++pp) {
                        Parts<NP> f;
#pragma unroll
                        for (int m = 0; m < NP; ++m) f.p[m] = row_natural(sdy + m * PLP + (16 * j + l15) * LDP + 32 * pp, lane);
                        tc = mma_parts(f, hf[pp], tc);
                    }
                    tc *= *reinterpret_cast<const f32x4*>(&dec.from[t]);
                    dC[j][k] += tc;
#pragma unroll
                    for (int m = NP - 1; m >= 0; --m) {
                        const bf16x4 c = tr4(sc + m * PLK + 16 * kt, LDK, t, lane);
#pragma unroll
                        for (int r = 0; r < 4; ++r) cv[r] = m + 1 < NP ? cv[r] + (float)c[r] : (float)c[r];
                    }
                    add(sum.ui[wave], t, cv * tc);
                }
#pragma unroll
                for (int pp = 0; pp < PT / 2; ++pp) {
                    float gx[8];
                    get_v(gv[pp], gx);
                    gf[pp] = split8<3, (NP > 1)>(gx);
                }
                if (k + 1 < KW) states(k + 1);
#pragma unroll
                for (int j = 0; j < QT; ++j) {
                    const int t = 16 * j + 4 * q4;
                    f32x4 tb = zero4(), bv = zero4();
#pragma unroll
                    for (int pp = 0; pp < PT / 2; ++pp) {
                        Parts<NP> x;
#pragma unroll
                        for (int m = 0; m < NP; ++m) x.p[m] = row_natural(sx + m * PLP + (16 * j + l15) * LDP + 32 * pp, lane);
                        tb = mma_parts(x, gf[pp], tb);
                    }
                    tb *= *reinterpret_cast<const f32x4*>(&dec.to[t]);
                    dB[j][k] += tb * *reinterpret_cast<const f32x4*>(&dec.src[t]);
#pragma unroll
                    for (int m = NP - 1; m >= 0; --m) {
                        const bf16x4 b = tr4(sb + m * PLK + 16 * kt, LDK, t, lane);
#pragma unroll
                        for (int r = 0; r < 4; ++r) bv[r] = m + 1 < NP ? bv[r] + (float)b[r] : (float)b[r];
                    }
                    add(sum.vi[wave], t, bv * tb);
                }
#pragma unroll
                for (int i2 = 0; i2 < QT / 2; ++i2) {
                    Parts<NP> bf, cf;
#pragma unroll
                    for (int m = 0; m < NP; ++m) {
                        bf.p[m] = col_natural(sb + m * PLK + 32 * i2 * LDK + 16 * kt, LDK, lane);
                        cf.p[m] = col_natural(sc + m * PLK + 32 * i2 * LDK + 16 * kt, LDK, lane);
                    }
#pragma unroll
                    for (int j = 0; j < QT; ++j) {
                        Parts<MP> f;
                        if (i2 <= j / 2) {
#pragma unroll
                            for (int m = 0; m < MP; ++m)
                                f.p[m] = row_natural(sds + m * PLQ + (16 * j + l15) * LDQ + 32 * i2, lane);
                            dC[j][k] = mma_parts(f, bf, dC[j][k]);
                        }
                        if (i2 >= j / 2) {
#pragma unroll
                            for (int m = 0; m < MP; ++m)
                                f.p[m] = col_natural(sds + m * PLQ + 32 * i2 * LDQ + 16 * j, LDQ, lane);
                            dB[j][k] = mma_parts(f, cf, dB[j][k]);
                        }
                    }
                }
            }
        }
        hg = lanes_sum<WAVE>(hg);
        if (lane == 0) sum.hg[wave] = hg;
        __syncthreads();

        if (threadIdx.x < Q) {
            const int t = threadIdx.x, tile = t / 16;
            const int same = QT == 4 ? (tile == 1 ? 3 : tile == 2 ? 2 : 1) : 2 - tile;  // the wavefront of the tile's products with itself
            float row = 0.f, col = 0.f, ui = 0.f, vi = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                row += sum.row[w][t];
                if (w != same) col += sum.col[w][t];
                ui += sum.ui[w][t];
                vi += sum.vi[w][t];
            }
            // products of later tiles with earlier ones pass the whole of a tile between them
            float between = 0.f;
            if (QT == 4) {
                between = tile == 1 ? sum.far[0][t & 15] + sum.far[1][t & 15] : tile == 2 ? sum.row[0][t + 16] : 0.f;
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) between += __shfl_xor(between, m);
            }
            float* o = a.tok + ((int64_t)at.slot * all_units + unit) * ssm_token_floats(Q) + t;
            o[0] = ui;
            o[Q] = vi;
            o[2 * Q] = row;
            o[3 * Q] = col;
            o[4 * Q] = sum.near[t] + between;
            o[5 * Q] = sum.own[t] + sum.col[same][t];
            o[6 * Q] = sum.xy[t];
            if (t == 0) o[7 * Q] = (sum.hg[0] + sum.hg[1]) + (sum.hg[2] + sum.hg[3]);
        }
    }

    if (wave * KW >= KT) return;
#pragma unroll
    for (int j = 0; j < QT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * j + 4 * q4 + r;
            if (t >= n) continue;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const int kc = 16 * (wave * KW + k) + l15;
                if (kc >= a.K) continue;
                const int64_t o = ((int64_t)(c0 + t) * a.G + at.group) * a.K + kc;
                if (quads == 1) {
                    ((DT*)a.dB)[o] = from_f32<DT>(dB[j][k][r]);
                    ((DT*)a.dC)[o] = from_f32<DT>(dC[j][k][r]);
                } else {
                    const int64_t all = (int64_t)a.T * a.G * a.K, p = (int64_t)at.quad * 2 * all + o;
                    a.part[p] = dB[j][k][r];
                    a.part[p + all] = dC[j][k][r];
                }
            }
        }
}

// dB and dC from the shares' sums.
template <typename DT> __global__ void __launch_bounds__(NT) ssm_shares_kernel(SsmArgs a) {
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int64_t all = (int64_t)a.T * a.G * a.K, live = (int64_t)sq.end() * a.G * a.K;
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < live; i += (int64_t)gridDim.x * NT) {
        float b = 0.f, c = 0.f;
        for (int s = 0; s < a.split; ++s) {
            b += a.part[(int64_t)s * 2 * all + i];
            c += a.part[(int64_t)s * 2 * all + all + i];
        }
        ((DT*)a.dB)[i] = from_f32<DT>(b);
        ((DT*)a.dC)[i] = from_f32<DT>(c);
    }
}

// A wavefront per chunk and head: the units' numbers put together, ddt, and the chunk's parts of dA, dD and dbias.
template <typename DT>
__global__ void __launch_bounds__(NT) ssm_tokens_kernel(SsmArgs a, int slots) {
    constexpr int Q = Cfg<DT>::QT * 16;
    const int lane = threadIdx.x % WAVE;
    const int64_t i = (int64_t)blockIdx.x * WAVES + threadIdx.x / WAVE;
    if (i >= (int64_t)slots * a.H) return;
    const int slot = __builtin_amdgcn_readfirstlane((int)(i / a.H)), h = __builtin_amdgcn_readfirstlane((int)(i % a.H));
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const Piece pc = find_piece(sq, slot, Q);
    float* sums = a.sums + (int64_t)slot * 3 * a.H + h;
    if (!pc.live || pc.len == 0) {
        if (lane < 3) sums[lane * a.H] = 0.f;
        return;
    }
    const int c0 = pc.start + pc.n * Q, n = min(Q, pc.len - pc.n * Q);
    const Decays<Q>& dec = reinterpret_cast<const Decays<Q>*>(a.dec)[i];
    const float* tok = a.tok + i * a.blocks * ssm_token_floats(Q);
    double in = 0.0, out = 0.0, later = 0.0, sooner = 0.0, own = 0.0, dd = 0.0, xy = 0.0, hg = 0.0, d = 0.0;
    for (int b = 0; b < a.blocks; ++b) hg += tok[(int64_t)b * ssm_token_floats(Q) + 7 * Q];
    if (lane < n) {
        for (int b = 0; b < a.blocks; ++b) {
            const float* u = tok + (int64_t)b * ssm_token_floats(Q) + lane;
            in += u[0];
            out += u[Q];
            later += u[2 * Q];
            sooner += u[3 * Q];
            own += u[4 * Q];
            dd += u[5 * Q];
            xy += u[6 * Q];
        }
        d = dec.src[lane];
        dd += out + sooner;
        out *= d;
        sooner *= d;
    }
    // A log decay is in every product of a token not before it with one before it.  Each sum here is one of such products
    // only, with none that another takes away again: what enters (state before the chunk) with this or later tokens, what
    // leaves with earlier ones, this tile's rows from here on with earlier tiles, its columns before with later ones.
    double dl = own + (double)dec.total * hg;
    const double first = lanes_scan(in, lane), last = lanes_scan(out, lane);
    dl += __shfl(first, WAVE - 1) - first + in + (last - out);
    const double mine = sooner;
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        const double r = __shfl_down(later, m, 16), c = __shfl_up(sooner, m, 16);
        if ((lane & 15) + m < 16) later += r;
        if ((lane & 15) >= m) sooner += c;
    }
    dl += later + (sooner - mine);
    double dz = 0.0;
    if (lane < n) {
        const float z = a.dt[(int64_t)(c0 + lane) * a.dts + h] + (a.bias ? a.bias[h] : 0.f);
        // the slope of softplus is the logistic function
        dz = (dl * a.A[h] + dd) * (a.softplus ? 1.0 / (1.0 + exp(-(double)z)) : 1.0);
        a.ddt[(int64_t)(c0 + lane) * a.H + h] = (float)dz;
    }
    double dA = lane < n ? dl * d : 0.0;
#pragma unroll
    for (int m = 1; m < WAVE; m <<= 1) {
        dA += __shfl_xor(dA, m);
        xy += __shfl_xor(xy, m);
        dz += __shfl_xor(dz, m);
    }
    if (lane < 3) sums[lane * a.H] = (float)(lane == 0 ? dA : lane == 1 ? xy : dz);
}

// Last sums of dA, dD and dbias: a wavefront per value.
__global__ void __launch_bounds__(NT) ssm_sums_kernel(SsmArgs a, int rows) {
    const int lane = threadIdx.x % WAVE;
    const int64_t i = (int64_t)blockIdx.x * WAVES + threadIdx.x / WAVE;
    if (i >= 3ll * a.H) return;
    const int which = (int)(i / a.H), h = (int)(i % a.H);
    float* out = which == 0 ? a.dA : which == 1 ? a.dD : a.dbias;
    if (!out) return;
    double s = 0.0;
    for (int r = lane; r < rows; r += WAVE) s += a.sums[((int64_t)r * 3 + which) * a.H + h];
#pragma unroll
    for (int m = 1; m < WAVE; m <<= 1) s += __shfl_xor(s, m);
    if (lane == 0) out[h] = (float)s;
}

// ---------------------------------------------------------------- one token per sequence

// z = act(bias + sum_j w_j x_{W-1-j}) in fp32, and the taps moved on by a token.
template <typename DT> __global__ void __launch_bounds__(NT) ssm_conv_kernel(SsmConvArgs a) {
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= (int64_t)a.N * a.C) return;
    const int64_t n = i / a.C;
    const int c = (int)(i % a.C);
    const DT* in = (const DT*)a.state_in + n * (a.W - 1) * a.C + c;
    DT* out = (DT*)a.state_out + n * (a.W - 1) * a.C + c;
    const DT x = ((const DT*)a.x)[n * a.xs + c];
    const float* w = a.weight + (int64_t)c * a.W;
    DT s[3];
    for (int j = 0; j < a.W - 1; ++j) s[j] = in[(int64_t)j * a.C];
    float z = a.bias ? a.bias[c] : 0.f;
    for (int j = 0; j < a.W - 1; ++j) z += w[j] * to_f32(s[j]);
    z += w[a.W - 1] * to_f32(x);
    if (a.silu) z *= sigmoid_f(z);
    for (int j = 0; j + 1 < a.W - 1; ++j) out[(int64_t)j * a.C] = s[j + 1];
    out[(int64_t)(a.W - 2) * a.C] = x;
    a.z[i] = z;
}

// 256 sequences of 32 heads of 128 x 128: 189 us, 1.06 GB at 5.6 TB/s, bound by memory.  The convolution before it is a
// kernel of its own (10 us there): in this one every head of a group would convolve the group's B and C again, and its
// states move on in place under the other heads' reads.
// A workgroup per (sequence, head, COLS columns): the state is read and written once, V neighbouring
// columns and K / ROWS rows a thread.
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(NT) ssm_step_kernel(SsmStepArgs a, int lanes_log2, int cblocks) {
    const int cb = blockIdx.x % cblocks;
    const int64_t nh = blockIdx.x / cblocks;
    const int64_t n = nh / a.H;
    const int h = (int)(nh % a.H), g = h / (a.H / a.G);
    const int lanes = 1 << lanes_log2, cl = threadIdx.x & (lanes - 1), r0 = threadIdx.x >> lanes_log2, rs = NT >> lanes_log2;
    const int p = (cb * lanes + cl) * V;
    const bool in = p < a.P;
    const float z = a.dt[n * a.dts + h] + (a.bias ? a.bias[h] : 0.f);
    const float d = a.softplus ? softplus_f(z) : z;
    const float decay = expf(d * a.A[h]);
    const TI* B = (const TI*)a.B + n * a.bs + (int64_t)g * a.K;
    const TI* C = (const TI*)a.C + n * a.cs + (int64_t)g * a.K;
    float x[V], y[V];
    zero_v(x);
    zero_v(y);
    if (in) get_v(load_v<V>((const TI*)a.x + n * a.xs + (int64_t)h * a.P + p), x);
    float xd[V];
#pragma unroll
    for (int v = 0; v < V; ++v) xd[v] = d * x[v];
    const float* hin = a.h_in + nh * a.K * a.P + p;
    float* hout = a.h_out + nh * a.K * a.P + p;
    constexpr int U = 8;
    if (in) {
        for (int k0 = r0; k0 < a.K; k0 += U * rs) {
            Pack<float, V> s[U];
            float b[U], c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * rs;
                if (k < a.K) {
                    s[u] = load_nt<V>(hin + (int64_t)k * a.P);
                    b[u] = to_f32(B[k]);
                    c[u] = to_f32(C[k]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * rs;
                if (k >= a.K) break;
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o[v] = decay * s[u][v] + b[u] * xd[v];
                    y[v] += c[u] * o[v];
                }
                store_nt<V>(hout + (int64_t)k * a.P, o);
            }
        }
    }
    __shared__ float part[NT * V];
#pragma unroll
    for (int v = 0; v < V; ++v) part[threadIdx.x * V + v] = y[v];
    __syncthreads();
    if (r0 == 0 && in) {
        for (int r = 1; r < rs; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] += part[(r * lanes + cl) * V + v];
        const float dk = a.D ? a.D[h] : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] += dk * x[v];
        store_v<V>((TO*)a.y + nh * a.P + p, y);
    }
}

// ---------------------------------------------------------------- launches

template <typename DT, int KT, int PT, int MODE> constexpr int walk_lds(int heads) {
    constexpr int NP = Cfg<DT>::NP;
    return NP * WALK * ((MODE & OUT ? 2 : 1) * KT * 32 + WAVES * PT * 32) +
           heads * ((MODE & OUT ? Cfg<DT>::MP * WALK * WALK * 2 : 0) +
                    4 * (int)sizeof(WalkDecays));
}
template <typename DT, int KT, int PT> constexpr int grad_lds() {
    constexpr int Q = Cfg<DT>::QT * 16, NP = Cfg<DT>::NP;
    return (2 * NP * Q * (KT * 16 + 8) + 2 * NP * Q * (PT * 16 + 8) + Cfg<DT>::GP * Q * (Q + 8)) * 2 +
           (int)sizeof(Decays<Q>) + (int)sizeof(GradSums<Q>);
}

template <typename F> hipError_t allow_lds(F* kernel, int bytes) {
    return bytes > 65536 ? hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                         : hipSuccess;
}

template <typename DT, int KT, int PT, int MODE>
hipError_t walk(const SsmArgs& a, const Role& one, const Role* two, hipStream_t st) {
    const int64_t slots = ssm_slots(a, a.seg);
    const int quads = (a.H / a.G * a.wblocks + WAVES - 1) / WAVES;
    constexpr int LDS = MODE == BOTH ? OUT : MODE;
    static_assert(walk_lds<DT, KT, PT, LDS>(WAVES) <= 160 * 1024, "a chunk's tiles fit a compute unit");
    const int lds = walk_lds<DT, KT, PT, LDS>(walk_heads(a.wblocks));
    auto* kernel = ssm_walk_kernel<DT, KT, PT, MODE>;
    const hipError_t e = allow_lds(kernel, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)place_blocks(slots, a.G, quads), two ? 2 : 1), dim3(NT), lds, st, a, one,
                       two ? *two : one, (int)slots, quads);
    return hipGetLastError();
}

bool segmented(const SsmArgs& a) { return a.cu ? a.seg < a.T : a.seg < a.eq; }

#define SSM_TRY(call)                     \
    do {                                  \
        const hipError_t e_ = (call);     \
        if (e_ != hipSuccess) return e_;  \
    } while (0)

// The states that the segments of one walk, or of two at once, start from.
template <typename DT, int KT, int PT> hipError_t starts(const SsmArgs& a, const Role& one, const Role* two, hipStream_t st) {
    if (!segmented(a)) return hipSuccess;
    SSM_TRY((walk<DT, KT, PT, ENDS>(a, one, two, st)));
    const int per_unit = KT * PT * WAVE, pieces = (per_unit + NT - 1) / NT;
    const int64_t blocks = (int64_t)a.H * a.wblocks * a.N * pieces;
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20), two ? 2 : 1), dim3(NT), 0, st, a,
                       one, two ? *two : one, per_unit, pieces);
    return hipGetLastError();
}

template <typename DT, int KT, int PT> hipError_t forward(const SsmArgs& a, hipStream_t st) {
    constexpr int WT = PT / 2;
    const Role r{a.x, a.B, a.C, a.xs, a.bs, a.cs, a.h0, a.hT, nullptr, a.ends, a.decay, 0};
    SSM_TRY((starts<DT, KT, WT>(a, r, nullptr, st)));
    return walk<DT, KT, WT, OUT>(a, r, nullptr, st);
}

template <typename DT, int KT, int PT> hipError_t backward(const SsmArgs& a, hipStream_t st) {
    constexpr int WT = PT / 2;
    if (a.N > 0) {
        const Role f{a.x, a.B, a.C, a.xs, a.bs, a.cs, a.h0, nullptr, a.hs, a.ends, a.decay, 0};
        const Role b{a.dy, a.C, a.B, a.dys, a.cs, a.bs, a.dhT, a.dh0, a.gs, a.rends, a.rdecay, 1};
        SSM_TRY((starts<DT, KT, WT>(a, f, &b, st)));
        SSM_TRY((walk<DT, KT, WT, BOTH>(a, b, &f, st)));
    }
    const int64_t slots = ssm_slots(a, a.chunk);
    if (a.T > 0) {
        const dim3 each((unsigned)((slots * a.H + WAVES - 1) / WAVES));
        hipLaunchKernelGGL(ssm_decay_kernel<DT>, each, dim3(NT), 0, st, a, (int)slots);
        SSM_TRY(hipGetLastError());
        constexpr int lds = grad_lds<DT, KT, PT>();
        static_assert(lds <= 160 * 1024, "a chunk's tiles fit a compute unit");
        auto* kernel = ssm_grad_kernel<DT, KT, PT>;
        SSM_TRY(allow_lds(kernel, lds));
        hipLaunchKernelGGL(kernel, dim3((unsigned)place_blocks(slots, a.G, a.split)), dim3(NT), lds, st, a, (int)slots, a.split);
        SSM_TRY(hipGetLastError());
        if (a.split > 1) {
            const int64_t all = (int64_t)a.T * a.G * a.K, blocks = (all + NT - 1) / NT;
            hipLaunchKernelGGL(ssm_shares_kernel<DT>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(NT), 0, st, a);
            SSM_TRY(hipGetLastError());
        }
        hipLaunchKernelGGL(ssm_tokens_kernel<DT>, each, dim3(NT), 0, st, a, (int)slots);
        SSM_TRY(hipGetLastError());
    }
    if (!a.dA && !a.dD && !a.dbias) return hipSuccess;
    hipLaunchKernelGGL(ssm_sums_kernel, dim3((3 * a.H + WAVES - 1) / WAVES), dim3(NT), 0, st, a, a.T > 0 ? (int)slots : 0);
    return hipGetLastError();
}

template <typename DT> hipError_t by_state(const SsmArgs& a, bool bwd, hipStream_t st) {
    switch (a.rows) {
        case 32: return bwd ? backward<DT, 2, 4>(a, st) : forward<DT, 2, 4>(a, st);
        case 64: return bwd ? backward<DT, 4, 4>(a, st) : forward<DT, 4, 4>(a, st);
        case 128: return bwd ? backward<DT, 8, 4>(a, st) : forward<DT, 8, 4>(a, st);
        default: return bwd ? backward<DT, 16, 2>(a, st) : forward<DT, 16, 2>(a, st);
    }
}

}  // namespace

hipError_t launch_ssm_fwd(const SsmArgs& a, hipStream_t st) {
    return a.dtype == 1 ? by_state<bf16>(a, false, st) : by_state<float>(a, false, st);
}
hipError_t launch_ssm_bwd(const SsmArgs& a, hipStream_t st) {
    return a.dtype == 1 ? by_state<bf16>(a, true, st) : by_state<float>(a, true, st);
}

hipError_t launch_ssm_conv(const SsmConvArgs& a, hipStream_t st) {
    const int64_t blocks = ((int64_t)a.N * a.C + NT - 1) / NT;
    if (a.dtype == 1) hipLaunchKernelGGL(ssm_conv_kernel<bf16>, dim3((unsigned)blocks), dim3(NT), 0, st, a);
    else hipLaunchKernelGGL(ssm_conv_kernel<float>, dim3((unsigned)blocks), dim3(NT), 0, st, a);
    return hipGetLastError();
}

namespace {
template <typename TI, typename TO> hipError_t step(const SsmStepArgs& a, hipStream_t st) {
    // rows of whole float4 in four columns a lane; narrow blocks of columns where the heads do not fill the GPU
    const bool four = a.P % 4 == 0;
    const int wide = four ? (a.P + 3) / 4 : a.P;
    int log2 = 0;
    while ((1 << log2) < wide && log2 < 6) ++log2;
    const int64_t heads = (int64_t)a.N * a.H;
    while (log2 > 3 && heads * ((wide + (1 << log2) - 1) >> log2) < 512) --log2;
    const int cblocks = (wide + (1 << log2) - 1) >> log2;
    const dim3 grid((unsigned)(heads * cblocks));
    if (four) hipLaunchKernelGGL((ssm_step_kernel<TI, TO, 4>), grid, dim3(NT), 0, st, a, log2, cblocks);
    else hipLaunchKernelGGL((ssm_step_kernel<TI, TO, 1>), grid, dim3(NT), 0, st, a, log2, cblocks);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_ssm_step(const SsmStepArgs& a, hipStream_t st) {
    if (a.dtype != 1) return step<float, float>(a, st);
    return a.f32_in ? step<float, bf16>(a, st) : step<bf16, bf16>(a, st);
}

}  // namespace kda
