// kda_linscan.hip -- diagonal gated linear recurrence over packed sequences on gfx950.
//
//   h_t = a_t h_{t-1} + x_t,  a_t = e^{log a_t},  y_t = h_t            per channel
//   g_t = dy_t + a_{t+1} g_{t+1},  dx_t = g_t,  dlog a_t = g_t a_t h_{t-1}
//
// HBM-bound (2 x 32768 x 4096 bf16: 409 us, 5.25 TB/s of the bytes that have to move), so x and
// log a are read once.
// The packed axis is cut into tiles of 128 or 256 tokens whatever the sequences'
// edges; a workgroup holds one tile of 64 V channels, each of its wavefronts 16
// tokens in registers.  A run of tokens
// maps the state before it to P h + E (P the product of its a, E its end from a
// zero state), or, if a sequence starts in it, to E alone: that case is marked
// by P = -1 and chosen, never multiplied, so that nothing of an earlier
// sequence, infinities included, reaches the next one.
//
// Tiles of the same channels form a chain: each workgroup publishes its tile's
// (P, E), takes the state before the tile from the nearest tile behind whose
// state is known, folding in the (P, E) of those between, publishes its own end
// state as (-1, h), and only then walks its tokens.  A pair is one 64-bit word,
// read and written whole at agent scope, so no other ordering is needed, and
// written by the thread that owns the channel alone, so that a known state
// stays known.  The fold runs oldest to newest with the same operations that
// formed the published states, so the result does not depend on which of them
// were there.  Tiles are taken in the order of a ticket counter: a workgroup
// waits only for tiles whose workgroups have started, so every wait ends.
//
// The backward runs the same way from the end, with c_t = a_t g_t as what a
// token hands to the one before it, and takes the forward states from `states`.
#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int TW = 16;       // tokens per wavefront; a workgroup's NW wavefronts hold a tile (linscan_shape)
constexpr int SW = 64 / TW;  // wavefronts between two rows of states
constexpr uint32_t EMPTY = 0xffffffffu;  // P of a word not yet published
constexpr uint32_t KNOWN = 0xbf800000u;  // P = -1: E is the state itself
// Polls before a wait is given up (seconds; reached only if the workspace is
// written by something else meanwhile): the state is then NaN and the call ends.
constexpr int MAX_POLLS = 1 << 21;

// One run of tokens followed by another: (p, e) <- (p2, e2) after (p, e).  Fused
// multiply-adds by name: a state folded in by a waiting workgroup has to have the
// bits of the one that its owner publishes.  (-1 times a chosen 0 leaves e2 as it is.)
__device__ __forceinline__ void then(float& p, float& e, float p2, float e2) {
    e = fmaf(p2, p2 < 0.f ? 0.f : e, e2);
    p = p2 < 0.f ? -1.f : p < 0.f ? -1.f : p2 * p;
}
__device__ __forceinline__ float apply(float p, float e, float h) { return fmaf(p, p < 0.f ? 0.f : h, e); }

__device__ __forceinline__ void publish(uint64_t* word, float p, float e) {
    const uint32_t pb = p == p ? __float_as_uint(p) : 0x7fc00000u;  // no NaN reads as EMPTY
    __hip_atomic_store(word, (uint64_t)__float_as_uint(e) << 32 | pb, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint64_t read_word(const uint64_t* word) {
    return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state handed over by the tile behind: words at word, word + step, ...,
// nearest first, `behind` of them (>= 1; the last of them always becomes (-1, h)).
// The nearest LB are read together; after that a poll reads only the farthest
// again, whose state is the first to become known, and what was not there yet.
// Forwards LB = 4 keeps a wide chain ahead of the memory (2 x 32768 x 4096: 409 us;
// LB = 2: 415, 8: 416, 1: 473); narrow ones take 8 (60000 x 64 in one sequence: 44 us,
// 4: 56, 16: 39; 4096 x 2048: 20.6, 21.4, 21.1; 24571 x 1000 fp32: 72, 70, 76).
// Backwards 4, in float32 2 for its registers.
template <int LB>  // words of the chain read at once
__device__ __forceinline__ float look_back(const uint64_t* word, int64_t step, int behind) {
    const int far = (behind < LB ? behind : LB) - 1;
    uint64_t w[LB];
#pragma unroll
    for (int d = 0; d < LB; ++d) w[d] = read_word(word + (d < far ? d : far) * step);
    for (int poll = 0; poll < MAX_POLLS; ++poll) {
        bool have = false;
        float h = 0.f;
#pragma unroll
        for (int d = LB - 1; d >= 0; --d) {
            const uint32_t pb = (uint32_t)w[d];
            if (d > far) continue;
            have = pb == KNOWN || (have && pb != EMPTY);
            h = apply(__uint_as_float(pb), __uint_as_float((uint32_t)(w[d] >> 32)), h);
        }
        if (have) return h;
        __builtin_amdgcn_s_sleep(1);
#pragma unroll
        for (int d = 0; d < LB; ++d)
            if (d == far || (d < far && (uint32_t)w[d] == EMPTY)) w[d] = read_word(word + d * step);
    }
    return __uint_as_float(0x7fc00000u);
}

// No word published, no ticket taken (the counters follow the words).
__global__ __launch_bounds__(256) void linscan_clear_kernel(uint64_t* word, int64_t words, int64_t counters) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (i + k < words + counters) word[i + k] = i + k < words ? ~0ull : 0ull;
}

// The sequences of a wavefront's 16 tokens, and which of the tokens start and
// end one (bit i of first / last for token t0 + i), all uniform over the
// wavefront.  Every lane has to be active.
struct Edges {
    uint32_t first, last;
    int count;   // tokens of the run that exist
    int n0;      // sequence of token t0
    int next;    // this lane's: where sequence n0 + 1 + lane starts
    // sequence of token t (t0 <= t < t0 + count)
    __device__ __forceinline__ int seq(const Seqs& sq, int t) const {
        const uint64_t started = __ballot(next <= t);
        return ~started ? n0 + __popcll(started) : sq.find(t);  // more than 64 of them: look it up
    }
};
__device__ __forceinline__ Edges edges_of(const Seqs& sq, int t0, int tend) {
    Edges e{0u, 0u, tend - t0 < TW ? tend - t0 : TW, 0, 0x7fffffff};
    if (e.count <= 0) { e.count = 0; return e; }
    e.n0 = wave_find(sq, t0);
    if (sq.start(e.n0) == t0) e.first = 1u;
    if (sq.start(e.n0 + 1) > t0 + TW) return e;  // the usual run, inside one sequence
    const int n = e.n0 + 1 + (int)threadIdx.x % WAVE;
    if (n <= sq.N) e.next = sq.start(n);
#pragma unroll
    for (int i = 1; i <= TW; ++i)
        if (__ballot(e.next == t0 + i)) e.first |= 1u << i, e.last |= 1u << (i - 1);
    if (!~__ballot(e.next <= t0 + TW)) {  // more than 64 starts, empty sequences among them
        for (int i = 1; i <= e.count; ++i)
            if (sq.start(sq.find(t0 + i < tend ? t0 + i : tend - 1)) == t0 + i || t0 + i == tend)
                e.first |= 1u << i, e.last |= 1u << (i - 1);
    }
    const uint32_t there = (1u << e.count) - 1;
    e.first &= there;
    e.last &= there;
    return e;
}

// Rows t0 .. t0 + 15 of a [T, C] tensor at this lane's columns (rows past the
// tensor's end: its last one, unused).  The rows are the wavefront's, so their
// addresses stay in scalar registers.
template <int V, typename T>
__device__ __forceinline__ void load_rows(const T* base, int64_t stride, int t0, int T_, uint32_t c,
                                          Pack<T, V> (&r)[TW]) {
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        const T* row = base + (int64_t)(t0 + i < T_ ? t0 + i : T_ - 1) * stride;
        r[i] = load_v<V>(row + c);
    }
}

// e^{log a}, by the exponential instruction: within (|log a| + 3) 2^-24, which an exact one
// would take a dozen instructions per element to make 2^-24.  Tokens that do not exist keep
// the state (a = 1, and x = 0 below).
template <int V>
__device__ __forceinline__ void decays(const Pack<float, V> (&la)[TW], int count, float (&a)[TW][V]) {
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) a[i][v] = __expf(la[i][v]);
    if (count < TW) {
#pragma unroll
        for (int i = 0; i < TW; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) a[i][v] = i < count ? a[i][v] : 1.f;
    }
}
template <int V, typename T>
__device__ __forceinline__ float value(const Pack<T, V> (&x)[TW], int i, int v, int count) {
    return i < count ? x[i][v] : 0.f;
}

// Makes the rows new values to the compiler, which otherwise keeps the converted
// ones of the first walk for the second: twice the registers of the bf16 rows.
template <int V, typename T>
__device__ __forceinline__ void keep_packed(Pack<T, V> (&x)[TW]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        typedef Pack<T, V> XP;
        struct Words { uint32_t w[V / 2]; };
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            Words r = __builtin_bit_cast(Words, x[i]);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) asm volatile("" : "+v"(r.w[k]));
            x[i] = __builtin_bit_cast(XP, r);
        }
    }
}

template <int V>
__device__ __forceinline__ void load_state(const float* h0, int C, int n, int c, float (&h)[V]) {
    if (h0) get_v<V>(load_v<V>(h0 + (int64_t)n * C + c), h);
    else zero_v<V>(h);
}

// (P, E) of a wavefront's run, forwards
template <int V, typename T>
__device__ __forceinline__ void run_forward(const LinScanArgs& p, const Seqs& sq, const Edges& ed, int t0, int c,
                                            const float (&a)[TW][V], const Pack<T, V> (&x)[TW], float (&P)[V],
                                            float (&E)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, E[v] = 0.f;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (ed.first >> i & 1) {
            load_state<V>(p.h0, p.C, ed.seq(sq, t0 + i), c, E);
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = -1.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            E[v] = a[i][v] * E[v] + value<V>(x, i, v, ed.count);
            P[v] = P[v] < 0.f ? -1.f : P[v] * a[i][v];
        }
    }
}

// The same from the end: what a run hands to the token before it, P c + E for c
// handed to it from behind.
template <int V, typename T>
__device__ __forceinline__ void run_backward(const LinScanArgs& p, const Seqs& sq, const Edges& ed, int t0, int c,
                                             const float (&a)[TW][V], const Pack<T, V> (&dy)[TW], float (&P)[V],
                                             float (&E)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, E[v] = 0.f;
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
        if (ed.last >> i & 1) {
            load_state<V>(p.dhT, p.C, ed.seq(sq, t0 + i), c, E);
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = -1.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            E[v] = a[i][v] * (value<V>(dy, i, v, ed.count) + E[v]);
            P[v] = P[v] < 0.f ? -1.f : P[v] * a[i][v];
        }
    }
}

// An empty sequence's final state is its initial one (forward: hT from h0,
// backward: dh0 from dhT).
__device__ __forceinline__ void empty_seqs(const Seqs& sq, const float* from, float* to, int C, int block, int blocks) {
    for (int n = block; n < sq.N; n += blocks) {
        if (sq.start(n + 1) > sq.start(n)) continue;
        for (int c = threadIdx.x; c < C; c += (int)blockDim.x) to[(int64_t)n * C + c] = from ? from[(int64_t)n * C + c] : 0.f;
    }
}

// A workgroup's column block and tile (counted from the chain's start).  TG
// neighbouring column blocks share a ticket counter, in a line of its own, and
// take a tile's columns one after the other: with a counter for each they drift
// apart and rows are read in pieces (forward, bf16, 2 x 32768 x 4096: 446 us
// against 409), with one for all a short chain waits for its tickets (4096 x 2048:
// 27 us against 23).
// No counters: one tile in all.
constexpr int TG = 4;
__device__ __forceinline__ void take_tile(uint64_t* tickets, int cblocks, int* lds, int& tile, int& cb) {
    cb = (int)blockIdx.x % cblocks;
    tile = 0;
    if (!tickets) return;
    const int group = cb / TG, width = cblocks - group * TG < TG ? cblocks - group * TG : TG;
    if (threadIdx.x == 0)
        *lds = (int)atomicAdd(reinterpret_cast<unsigned long long*>(tickets + group * LINSCAN_LINE), 1ull);
    __syncthreads();
    const int ticket = __builtin_amdgcn_readfirstlane(*lds);
    tile = ticket / width;
    cb = group * TG + ticket - tile * width;
}

// The tile's (P, E) from its wavefronts', the state handed to it, and its own
// published: thread j < 64 V does channel j of the workgroup.  In: sp, se; out:
// sh, the state handed to the tile.  BACK: from the last wavefront to the first.
template <int V, int NW, bool BACK, int LB>
__device__ __forceinline__ void chain(const LinScanArgs& p, const float (&sp)[NW][WAVE * V],
                                      const float (&se)[NW][WAVE * V], float (&sh)[WAVE * V], int cb, int tile,
                                      int tiles) {
    const int j = threadIdx.x;
    if (j >= WAVE * V) return;
    const ChainColumn k = chain_column<V>(cb, j, p.C);
    float P = sp[BACK ? NW - 1 : 0][j], E = se[BACK ? NW - 1 : 0][j];
#pragma unroll
    for (int w = 1; w < NW; ++w) then(P, E, sp[BACK ? NW - 1 - w : w][j], se[BACK ? NW - 1 - w : w][j]);
    const int behind = BACK ? tiles - 1 - tile : tile;
    uint64_t* word = p.word + (int64_t)tile * p.C + k.c;
    float h = 0.f;
    if (tiles > 1) {
        if (behind > 0) {
            if (k.owner) publish(word, P, E);
            h = look_back<LB>(BACK ? word + p.C : word - p.C, BACK ? (int64_t)p.C : -(int64_t)p.C, behind);
        }
        if (k.owner && (P >= 0.f || behind == 0 || P != P)) publish(word, -1.f, apply(P, E, h));
    }
    sh[j] = h;
}

// OUT: y and hT too, else the states alone.
template <typename T, int V, int NW, bool OUT, int LB>
__global__ __launch_bounds__(NW* WAVE) void linscan_fwd_kernel(LinScanArgs p, int tiles, int cblocks, uint64_t* tickets) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V], sh[WAVE * V];
    __shared__ int s_tile;
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    const int jobs = tiles * cblocks;
    if ((int)blockIdx.x >= jobs) {
        if (OUT && p.hT) empty_seqs(sq, p.h0, p.hT, p.C, blockIdx.x - jobs, gridDim.x - jobs);
        return;
    }
    int tile, cb;
    take_tile(tickets, cblocks, &s_tile, tile, cb);
    if (tile >= tiles) return;
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = column<V>((cb * WAVE + lane) * V, p.C);  // lanes past the row's end: its last, once more
    const int t0 = (tile * NW + wv) * TW;
    Pack<float, V> la[TW];
    Pack<T, V> x[TW];
    load_rows<V>(p.la, p.ls, t0, p.T, c, la);
    load_rows<V>((const T*)p.x, p.xs, t0, p.T, c, x);
    const Edges ed = edges_of(sq, t0, sq.end());
    float a[TW][V], P[V], E[V], h[V];
    decays<V>(la, ed.count, a);
    run_forward<V>(p, sq, ed, t0, c, a, x, P, E);
    keep_packed<V>(x);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    __syncthreads();
    chain<V, NW, false, LB>(p, sp, se, sh, cb, tile, tiles);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sh[lane * V + v];
    for (int w = 0; w < wv; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(sp[w][lane * V + v], se[w][lane * V + v], h[v]);
    if (p.states && wv % SW == 0 && t0 < p.T) store_v<V>(p.states + (int64_t)(t0 / (SW * TW)) * p.C + c, h);
    if (!OUT) return;
    T* y = (T*)p.y + (int64_t)t0 * p.C;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (i >= ed.count) continue;
        if (ed.first >> i & 1) load_state<V>(p.h0, p.C, ed.seq(sq, t0 + i), c, h);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = a[i][v] * h[v] + x[i][v];
        store_nt<V>(y + (int64_t)i * p.C + (uint32_t)c, h);
        if ((ed.last >> i & 1) && p.hT) store_v<V>(p.hT + (int64_t)ed.seq(sq, t0 + i) * p.C + c, h);
    }
}

template <typename T, int V, int NW>
__global__ __launch_bounds__(NW* WAVE, 4) void linscan_bwd_kernel(LinScanArgs p, int tiles, int cblocks, uint64_t* tickets) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V], rp[NW][WAVE * V], re[NW][WAVE * V], sh[WAVE * V];
    __shared__ int s_tile;
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    const int jobs = tiles * cblocks;
    if ((int)blockIdx.x >= jobs) {
        if (p.hT) empty_seqs(sq, p.dhT, p.hT, p.C, blockIdx.x - jobs, gridDim.x - jobs);
        return;
    }
    int tile, cb;
    take_tile(tickets, cblocks, &s_tile, tile, cb);
    tile = tiles - 1 - tile;
    if (tile < 0) return;
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = column<V>((cb * WAVE + lane) * V, p.C);  // lanes past the row's end: its last, once more
    const int t0 = (tile * NW + wv) * TW;
    Pack<float, V> la[TW];
    Pack<T, V> x[TW], dy[TW];
    load_rows<V>(p.la, p.ls, t0, p.T, c, la);
    load_rows<V>((const T*)p.dy, p.ds, t0, p.T, c, dy);
    load_rows<V>((const T*)p.x, p.xs, t0, p.T, c, x);
    // the state before the 64 tokens that this wavefront's belong to
    const int row = (tile * NW + wv) / SW, rows = (p.T + SW * TW - 1) / (SW * TW);
    float h[V], g[V];
    get_v<V>(load_v<V>(p.states + (int64_t)(row < rows ? row : rows - 1) * p.C + c), h);
    const Edges ed = edges_of(sq, t0, sq.end());
    float a[TW][V], P[V], E[V];
    decays<V>(la, ed.count, a);
    run_backward<V>(p, sq, ed, t0, c, a, dy, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) rp[wv][lane * V + v] = P[v], re[wv][lane * V + v] = E[v];
    run_forward<V>(p, sq, ed, t0, c, a, x, P, E);
    keep_packed<V>(x);
    keep_packed<V>(dy);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    __syncthreads();
    chain<V, NW, true, sizeof(T) == 4 ? 2 : 4>(p, rp, re, sh, cb, tile, tiles);
    // the state before every token of the run
    for (int w = wv / SW * SW; w < wv; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(sp[w][lane * V + v], se[w][lane * V + v], h[v]);
    float hb[TW][V];
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (ed.first >> i & 1) load_state<V>(p.h0, p.C, ed.seq(sq, t0 + i), c, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hb[i][v] = h[v];
            h[v] = a[i][v] * h[v] + x[i][v];
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = sh[lane * V + v];
    for (int w = NW - 1; w > wv; --w)
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = apply(rp[w][lane * V + v], re[w][lane * V + v], g[v]);
    T* dx = (T*)p.y + (int64_t)t0 * p.C;
    float* dla = p.dla + (int64_t)t0 * p.C;
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
        if (i >= ed.count) continue;
        if (ed.last >> i & 1) load_state<V>(p.dhT, p.C, ed.seq(sq, t0 + i), c, g);
        float d[V], dl[V];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = dy[i][v] + g[v];
        store_nt<V>(dx + (int64_t)i * p.C + (uint32_t)c, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            g[v] = a[i][v] * d[v];
            dl[v] = g[v] * hb[i][v];
        }
        store_nt<V>(dla + (int64_t)i * p.C + (uint32_t)c, dl);
        if ((ed.first >> i & 1) && p.hT) store_v<V>(p.hT + (int64_t)ed.seq(sq, t0 + i) * p.C + c, g);
    }
}

// One token per sequence.  In place: a lane owns its columns alone, the row's
// last few one by one.
template <int V, typename T>
__device__ __forceinline__ void step_at(const LinScanArgs& p, int n, int c) {
    const Pack<float, V> la = load_v<V>(p.la + (int64_t)n * p.ls + c), h0 = load_v<V>(p.h0 + (int64_t)n * p.C + c);
    const Pack<T, V> x = load_v<V>((const T*)p.x + (int64_t)n * p.xs + c);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = __expf(la[v]) * h0[v] + x[v];
    store_v<V>(p.hT + (int64_t)n * p.C + c, h);
    store_v<V>((T*)p.y + (int64_t)n * p.C + c, h);
}
constexpr int BS = 256;
template <typename T, int V>
__global__ __launch_bounds__(BS) void linscan_step_kernel(LinScanArgs p) {
    const int ncv = (p.C + V - 1) / V;
    const int64_t id = (int64_t)blockIdx.x * BS + threadIdx.x;
    if (id >= (int64_t)p.N * ncv) return;
    const int n = (int)(id / ncv), c = (int)(id % ncv) * V;
    if (c + V <= p.C) {
        step_at<V, T>(p, n, c);
    } else {
        for (int i = c; i < p.C; ++i) step_at<1, T>(p, n, i);
    }
}

int empty_blocks(int N) { return N < LINSCAN_EMPTY ? N : LINSCAN_EMPTY; }

// Clears the chain (more than one tile) and gives the launch its grid.
template <typename K>
hipError_t run_chain(K kernel, const LinScanArgs& a, const LinScanShape& s, bool empties, hipStream_t st) {
    const int64_t blocks = (int64_t)s.tiles * s.cblocks + (empties ? empty_blocks(a.N) : 0);
    if (blocks == 0) return hipSuccess;
    uint64_t* tickets = nullptr;
    if (s.tiles > 1) {
        const int64_t words = (int64_t)s.tiles * a.C, counters = (int64_t)s.cblocks * LINSCAN_LINE;
        tickets = a.word + words;
        hipLaunchKernelGGL(linscan_clear_kernel, dim3((unsigned)((words + counters + 511) / 512)), dim3(256), 0, st,
                           a.word, words, counters);
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(s.waves * WAVE), 0, st, a, s.tiles, s.cblocks, tickets);
    return hipGetLastError();
}

template <typename T, int V, bool OUT>
hipError_t fwd(const LinScanArgs& a, const LinScanShape& s, hipStream_t st) {
    const bool empties = OUT && a.hT;
    if constexpr (V > 1)
        if (s.waves == 8) return run_chain(linscan_fwd_kernel<T, V, 8, OUT, 4>, a, s, empties, st);
    return run_chain(linscan_fwd_kernel<T, V, 16, OUT, 8>, a, s, empties, st);
}
template <typename T, int V>
hipError_t fwd(const LinScanArgs& a, const LinScanShape& s, bool out, hipStream_t st) {
    return out ? fwd<T, V, true>(a, s, st) : fwd<T, V, false>(a, s, st);
}
template <typename T, int V>
hipError_t bwd(const LinScanArgs& a, const LinScanShape& s, hipStream_t st) {
    const bool empties = a.hT != nullptr;
    if constexpr (V > 1)
        if (s.waves == 8) return run_chain(linscan_bwd_kernel<T, V, 8>, a, s, empties, st);
    return run_chain(linscan_bwd_kernel<T, V, 16>, a, s, empties, st);
}

}  // namespace

hipError_t launch_linscan_fwd(const LinScanArgs& a, bool out, hipStream_t st) {
    const LinScanShape s = linscan_shape(a.T, a.C);
    if (s.vec == 1) return a.dtype == 1 ? fwd<bf16, 1>(a, s, out, st) : fwd<float, 1>(a, s, out, st);
    return a.dtype == 1 ? fwd<bf16, 2>(a, s, out, st) : fwd<float, 2>(a, s, out, st);
}

hipError_t launch_linscan_bwd(const LinScanArgs& a, hipStream_t st) {
    const LinScanShape s = linscan_shape(a.T, a.C);
    if (s.vec == 1) return a.dtype == 1 ? bwd<bf16, 1>(a, s, st) : bwd<float, 1>(a, s, st);
    return a.dtype == 1 ? bwd<bf16, 2>(a, s, st) : bwd<float, 2>(a, s, st);
}

hipError_t launch_linscan_step(const LinScanArgs& a, hipStream_t st) {
    constexpr int V = 4;
    const int64_t work = (int64_t)a.N * ((a.C + V - 1) / V);
    const dim3 grid((unsigned)((work + BS - 1) / BS));
    if (a.dtype == 1) hipLaunchKernelGGL((linscan_step_kernel<bf16, V>), grid, dim3(BS), 0, st, a);
    else hipLaunchKernelGGL((linscan_step_kernel<float, V>), grid, dim3(BS), 0, st, a);
    return hipGetLastError();
}

}  // namespace kda
