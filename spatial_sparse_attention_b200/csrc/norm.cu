// ssa_group_norm and ssa_group_norm_backward: group normalisation over the tokens of a sequence and the
// channels of a group, weights and an activation, channels last, for packed sequences.
//
//   xhat = (x - mean) * rstd,  z = xhat * gamma + beta,  y = act(z),
//   mean, 1/rstd^2 - eps: mean and variance over the m = tokens * width values of a (sequence, group).
// With dz = dy * act'(z):  dbeta = sum dz,  dgamma = sum dz * xhat  (over tokens and sequences),
//   dx = rstd * (dz * gamma - S1 - xhat * S2),  S1 = sum(dz * gamma) / m,  S2 = sum(dz * gamma * xhat) / m
// over the sequence and group.
//
// Bound: HBM. Two launches: sums of every tile of tokens, and the pass that writes, whose CTAs first add up the
// tiles' sums of their own groups (a few KB from L2, while their first rows arrive). Both cut the rows into column
// blocks of 16-byte vectors, whatever the groups' width: a thread keeps one vector of channels and walks rows, so
// channel constants stay in registers; a group across column blocks has sums in each. Rows that are not aligned
// to 16 bytes are read in chunks of A elements. The second pass takes the tiles in reverse: what the
// first read last is still in L2. Measured (2112 channels in 32 groups, fp16, silu): 340,000 tokens 699 us, the gradient of
// 80,000 288 us: 6.2 and 5.9 TB/s over the three and five passes made. A forward whose rows all fit in shared
// memory is one cooperative launch that reads them once (20,000 x 512 bf16: 18 against 21 us; the gradient
// gained nothing from it).
// Inside a tile sums are fp32 (at most 48 rows of a thread, then up to 256 threads and 680 channels), from tile to tile fp64. (Tried and slower: column blocks or units of groups small enough to stay in L2
// between the passes, as one launch with tickets or as many launches, 913 us and more against 691 for 340,000 tokens x 2112
// fp16: pieces of rows, 128 to 528 bytes 4 KB apart, cost more than the third pass over memory.)
// Tile `t` of sequence s holds its tokens [t * R, ...) and has slot lo / R + s + t in the tables of sums: a sequence of n
// tokens owns hi / R - lo / R + 1 >= ceil(n / R) slots; the tiles beyond its end are empty.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>

#include "views.cuh"

namespace ssa {

namespace {

constexpr int kThreads = 256;
constexpr int kVecBytes = 16;
constexpr int kMaxChannels = 65536;
// Rows per thread of a full tile.
constexpr int kRowsPerThread = 48;
// The variance of a thread's rows comes from sums about its first row, and after kSettled of them about those rows' mean. With n rows
// the cancellation about one of them is at most a factor n (sq <= n D^2, D the largest deviation from it, and
// the squared deviations from the mean are at least D^2 / 2); about the mean of n0 of n rows it is n / n0, as
// what the others have in common off it counts n0 (n - n0) / n times in the variance. So a first row far from the others costs
// a factor 8 in place of 48. The merges after that take deviations from means.
constexpr int kSettled = 8;
constexpr int kTilesPerLane = 10;       // tiles of a column that one lane of a merge adds up,
constexpr int kMinTiles = 148;          // where that does not leave SMs without work
constexpr int kBlockBytes = 128;        // of a row that a column block's threads read together, at least
constexpr int kStages = 8;              // rows per thread in flight or in use: forward, gradient
static_assert(kStages == kSettled, "the sums' pivot moves after the ring's first round");
constexpr int kGradStages = 6;
constexpr int kKeptRows = 12;           // rows per thread and CTAs per SM of the one-launch forward: 198 KB of 227
constexpr int kKeptCtas = 3;

struct NormArgs {
    const void* x;
    const void* dy;
    void* out;
    int64_t x_ts, dy_ts, o_ts;
    const float* gamma;     // null: ones
    const float* beta;      // null: zeros
    float* mean;            // [B, G] (forward: null when not wanted)
    float* rstd;
    float2* group_part;     // [slots][over][G]: (mean, squared deviations); gradient: sums of gamma dz, gamma dz xhat
    float2* chan_part;      // gradient: [slots][C] sums of dz, dz xhat
    float* dgamma;
    float* dbeta;
    const SeqInfo* seqs;
    int64_t N;
    uint32_t R, slots;      // tokens per tile; slots of all sequences
    int32_t B, C, G, width;
    uint32_t magic;         // ceil(2^32 / width), see group_of
    int32_t nvt, nv, rl;    // vectors per row (the last may be partly filled); vectors and row lanes of a CTA
    int32_t blocks, over;   // column blocks; blocks that a group can touch
    int32_t clanes, glanes; // lanes that add a channel's rows, a group's channels (powers of two)
    float eps;
};

// c / width for 0 <= c < 65536: c * magic is off by less than c * width < 2^32, under the next quotient's step.
__device__ __forceinline__ int group_of(const NormArgs& a, int c) {
    return a.width == 1 ? c : (int)__umulhi((uint32_t)c, a.magic);
}

// A CTA's column block: vectors [v0, v0 + nvec), channels [c0, c1), groups [g0, g1]; this thread's vector and row lane.
struct Block {
    int index, v0, nvec, c0, c1, g0, g1, vec, lane;
    __device__ __forceinline__ Block(const NormArgs& a, int b, int V) {
        index = b;
        v0 = b * a.nv;
        nvec = min(a.nv, a.nvt - v0);
        c0 = v0 * V;
        c1 = min(a.C, c0 + nvec * V);
        g0 = group_of(a, c0);
        g1 = group_of(a, c1 - 1);
        lane = threadIdx.x / a.nv;
        vec = threadIdx.x - lane * a.nv;
    }
    __device__ __forceinline__ bool active(const NormArgs& a) const { return lane < a.rl && vec < nvec; }
    // Channel of element j of the thread's vector, relative to c0. Chunks of A elements go round the block's vectors:
    // what neighbouring threads read or write together is contiguous, whatever A.
    template <int A>
    __device__ __forceinline__ int relative(int j) const { return ((j / A) * nvec + vec) * A + j % A; }
    // the same, inside the block: elements beyond the row take the last channel's constants, nothing is made of them
    template <int A>
    __device__ __forceinline__ int channel(int j) const { return min(c0 + relative<A>(j), c1 - 1); }
    // chunks of the vector that lie in the row
    template <int A>
    __device__ __forceinline__ int chunks() const { return (c1 - c0 - vec * A + nvec * A - 1) / (nvec * A); }
};

// First column block of a group.
__device__ __forceinline__ int first_block(const NormArgs& a, int g, int V) { return g * a.width / (a.nv * V); }
__device__ __forceinline__ int last_block(const NormArgs& a, int g, int V) { return ((g + 1) * a.width - 1) / (a.nv * V); }

__device__ __forceinline__ uint32_t first_slot(const NormArgs& a, int s) { return (uint32_t)a.seqs[s].lo / a.R + s; }

// The tile of a slot: n tokens of sequence s from t0; tiles: of the sequence.
struct Tile {
    int s, n, tiles;
    int64_t t0;
    uint32_t slot;
    bool opens;     // the sequence's first
    __device__ __forceinline__ Tile(const NormArgs& a, uint32_t i) {
        int last = a.B - 1;
        s = 0;
        while (s < last) {
            const int mid = (s + last + 1) >> 1;
            if (first_slot(a, mid) <= i) s = mid; else last = mid - 1;
        }
        const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
        const uint32_t t = i - first_slot(a, s);
        slot = i;
        opens = t == 0;
        t0 = lo + (int64_t)t * a.R;
        n = (int)max((int64_t)0, min((int64_t)a.R, hi - t0));
        tiles = (int)(((uint32_t)(hi - lo) + a.R - 1) / a.R);
    }
};

// The vectors of this thread's rows, 16 bytes in chunks of A elements `hop` apart; `chunks` of them are inside the row.
template <typename T, int A>
struct Pieces {
    static constexpr int V = kVecBytes / (int)sizeof(T), N = V / A;
    using W = Vec<T, A>;
    using C = typename W::C;
    static __device__ __forceinline__ void unpack(const C& raw, int i, float (&e)[V]) {
        float v[A];
        W::unpack(raw, v);
#pragma unroll
        for (int j = 0; j < A; ++j) e[i * A + j] = v[j];
    }
    static __device__ __forceinline__ void store(T* at, const float (&e)[V], int chunks, int hop) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[A];
#pragma unroll
            for (int j = 0; j < A; ++j) v[j] = e[i * A + j];
            if (N == 1 || i < chunks) __stcs(reinterpret_cast<C*>(at + i * hop), W::pack(v));
        }
    }
};

// This thread's `count` rows of K arrays, `step` elements apart, its loads STAGES - 1 rows ahead in its own places of
// the ring: no barrier and no registers for what is in flight. Rows of 2-byte chunks, which the
// asynchronous copy does not take, come in batches through registers instead.
template <typename T, int A, int K, int STAGES>
struct Rows {
    using P = Pieces<T, A>;
    using C = typename P::C;
    static constexpr int V = P::V, N = P::N;
    static constexpr bool kRing = sizeof(C) >= 4;
    static constexpr size_t kBytes = kRing ? STAGES * K * kThreads * kVecBytes : 0;
    const T* at[K];
    int64_t step[K];
    int count, chunks, hop;
    char* ring;
    int left;           // rows not asked for yet

    __device__ __forceinline__ C* place(int stage, int k, int i) const {
        return (C*)ring + ((stage * K + k) * N + i) * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(int stage) {
        if (left > 0) {
            --left;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (N == 1 || i < chunks) cp_async<sizeof(C)>(place(stage, k, i), at[k] + i * hop);
                at[k] += step[k];
            }
        }
        cp_commit();
    }
    // sends off the first rows
    __device__ __forceinline__ void start() {
        left = count;
        if constexpr (kRing) {
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) fetch(i);
        }
    }
    // all rows at once, to be kept: count <= STAGES
    __device__ __forceinline__ void start_kept() {
        left = count;
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch(i);
        cp_wait<0>();
    }
    // channels beyond the row come out as anything: nothing is made of them
    __device__ __forceinline__ void read(int stage, int k, float (&e)[V]) {
#pragma unroll
        for (int i = 0; i < N; ++i) P::unpack(*place(stage, k, i), i, e);
    }
    __device__ __forceinline__ void load(const T* from, C (&raw)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (N == 1 || i < chunks) raw[i] = *reinterpret_cast<const C*>(from + i * hop);
    }
    // row 0, which stays to be read (count > 0)
    template <bool KEPT>
    __device__ __forceinline__ void peek(float (&e)[V]) {
        if constexpr (KEPT) {
            read(0, 0, e);
        } else if constexpr (kRing) {
            cp_wait<STAGES - 2>();
            read(0, 0, e);
        } else {
            C raw[N] = {};
            load(at[0], raw);
#pragma unroll
            for (int i = 0; i < N; ++i) P::unpack(raw[i], i, e);
        }
    }
    // f(e) for every row, e[k] being its vector of array k; f may write over the row (in place). g() once after the first
    // kSettled rows, where more follow (not for kept rows, which are few).
    template <bool KEPT, typename F, typename Then>
    __device__ __forceinline__ void each(F f, Then g) {
        float e[K][V];
        if constexpr (KEPT) {
#pragma unroll 4
            for (int i = 0; i < count; ++i) {
#pragma unroll
                for (int k = 0; k < K; ++k) read(i, k, e[k]);
                f(e);
            }
        } else if constexpr (kRing) {
            for (int i = 0; i < count; i += STAGES) {
#pragma unroll
                for (int j = 0; j < STAGES; ++j) {
                    if (i + j < count) {
                        fetch((j + STAGES - 1) % STAGES);
                        cp_wait<STAGES - 1>();
#pragma unroll
                        for (int k = 0; k < K; ++k) read(j, k, e[k]);
                        f(e);
                    }
                }
                if constexpr (STAGES == kSettled) {
                    if (i == 0 && count > kSettled) g();
                }
            }
        } else {
            constexpr int U = 4 / K;
            for (int i = 0; i < count; i += U) {
                C raw[U][K][N] = {};
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + u < count) {
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            load(at[k], raw[u][k]);
                            at[k] += step[k];
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + u < count) {
#pragma unroll
                        for (int k = 0; k < K; ++k) {
#pragma unroll
                            for (int n = 0; n < N; ++n) P::unpack(raw[u][k][n], n, e[k]);
                        }
                        f(e);
                    }
                }
                static_assert(kSettled % U == 0, "the rows of a batch come before or after g");
                if (i + U == kSettled && count > kSettled) g();
            }
        }
    }
    template <bool KEPT, typename F>
    __device__ __forceinline__ void each(F f) {
        each<KEPT>(f, [] {});
    }
};

__device__ __forceinline__ int row_count(const NormArgs& a, const Block& b, int n) {
    return b.active(a) && b.lane < n ? (n - b.lane + a.rl - 1) / a.rl : 0;
}

// The channels' sums of a CTA's row lanes: [rl][red_row], rows padded by 64 bytes so that threads which read the
// same channel of different rows meet in few banks; bytes, a multiple of 16.
__host__ __device__ inline int red_row(const NormArgs& a, int V) { return a.nv * V + 8; }
__host__ __device__ inline size_t red_bytes(const NormArgs& a, int V) { return (sizeof(float2) * a.rl * red_row(a, V) + 15) / 16 * 16; }

// Adds v over the `lanes` (a power of two) neighbouring lanes; every one gets it.
template <typename F>
__device__ __forceinline__ F lane_sum(F v, int lanes) {
    for (int h = lanes / 2; h > 0; h >>= 1) v += __shfl_xor_sync(0xffffffffu, v, h);
    return v;
}

// f(channel relative to c0, whether it is one, lane, lanes) for the block's channels, several neighbouring lanes to a
// channel; all threads take part, those beyond the last channel with channel 0. A channel is done by one warp at once.
template <typename F>
__device__ __forceinline__ void for_channels(const NormArgs& a, const Block& b, F f) {
    const int Q = a.clanes, n = b.c1 - b.c0;
    for (int base = 0; base < n; base += kThreads / Q) {
        const int c = base + threadIdx.x / Q;
        f(c < n ? c : 0, c < n, threadIdx.x % Q, Q);
    }
}

// f(group, channel range relative to c0, lane of the group, lanes) for the block's groups; all threads take part.
template <typename F>
__device__ __forceinline__ void for_groups(const NormArgs& a, const Block& b, F f) {
    const int L = a.glanes;
    for (int base = b.g0; base <= b.g1; base += kThreads / L) {
        const int g = base + threadIdx.x / L;
        const int lo = max(g * a.width, b.c0), hi = g <= b.g1 ? min((g + 1) * a.width, b.c1) : lo;
        f(g, lo - b.c0, hi - b.c0, threadIdx.x % L, L);
    }
}

// ---- activations -------------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^(c x) for a constant c = hi + lo, to the hardware's 2 ulp whatever the size of c x: what rounding takes from the
// product comes back as a factor. |c x| < 300.
__device__ __forceinline__ float ex2_scaled(float x, float hi, float lo) {
    const float y = x * hi, rest = fmaf(x, lo, fmaf(x, hi, -y)), e = ex2(y);
    return fmaf(e, rest * 0.6931472f, e);
}

// sigma(z), by the hardware's exponential and reciprocal. For the 16-bit types the exponent's product is rounded
// (|z| 2^-24 relative, far below a step of theirs; the weights' fp32 gradients are sums of such terms, whose 16-bit inputs are
// known to less than that); with expf and a division fp32 would wait for instructions, not memory.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 2) return rcp(1.0f + ex2(z * -1.4426950408889634f));
    return rcp(1.0f + ex2_scaled(fminf(fmaxf(z, -88.0f), 88.0f), -1.44269502f, -1.92596303e-8f));
}

// Phi(z) of the normal distribution, and e = exp(-z^2 / 2). Phi(-|z|) is t p(t) e with t = 1 / (1 + a |z|): p is fitted to
// the scaled complement erfc(x) exp(x^2) / 2 at x = |z| / sqrt(2) <= 10 for least relative error, of degree 7 (3.4e-7 in
// fp32) for the 16-bit types and 8 (2.3e-7, the fp32 evaluation's own) for fp32. normcdff, twice as many instructions, bounds the
// pass that writes in place of memory (570 against 242 us for 135,000 tokens x 1376 bf16).
template <typename T>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    float q;
    if constexpr (sizeof(T) == 2) {
        e = ex2(z * z * -0.72134752f);      // log2(e) / 2
        const float t = rcp(fmaf(fabsf(z), 0.3f, 1.0f));
        float p = fmaf(t, 0.035675015f, -0.157204f);
        p = fmaf(p, t, 0.20635495f);
        p = fmaf(p, t, -0.053684855f);
        p = fmaf(p, t, 0.12856221f);
        p = fmaf(p, t, 0.09991333f);
        p = fmaf(p, t, 0.12075398f);
        q = fmaf(p, t, 0.11962929f) * t * e;
    } else {
        const float y = fminf(fabsf(z), 20.0f), sq = y * y;     // exp(-200) = 0 in fp32
        e = ex2_scaled(sq, -0.72134751f, -9.6298151e-9f);
        e = fmaf(e, fmaf(y, y, -sq) * -0.5f, e);                // the square's own rounding
        const float t = rcp(fmaf(y, 0.35f, 1.0f));
        float p = fmaf(t, -0.029145656f, 0.14397046f);
        p = fmaf(p, t, -0.25571191f);
        p = fmaf(p, t, 0.15917169f);
        p = fmaf(p, t, -0.023108279f);
        p = fmaf(p, t, 0.1055074f);
        p = fmaf(p, t, 0.11983301f);
        p = fmaf(p, t, 0.13986185f);
        q = fmaf(p, t, 0.13962141f) * t * e;
    }
    return z > 0.0f ? 1.0f - q : q;
}

// z -> act(z)
template <typename T, int ACT>
__device__ __forceinline__ float activate(float z) {
    float e;
    if (ACT == SSA_ACT_SILU) return z * sigmoid<T>(z);
    if (ACT == SSA_ACT_GELU) return z * normal_cdf<T>(z, e);
    return z;
}

// z -> act'(z)
template <typename T, int ACT>
__device__ __forceinline__ float activate_grad(float z) {
    if (ACT == SSA_ACT_SILU) {
        const float t = sigmoid<T>(z);
        return t * fmaf(z, 1.0f - t, 1.0f);
    }
    if (ACT == SSA_ACT_GELU) {
        float e;
        const float c = normal_cdf<T>(z, e);
        return fmaf(z * 0.3989422804014327f, e, c);
    }
    return 1.0f;
}

// z -> act'(z) of two values.
template <typename T, int ACT>
__device__ __forceinline__ void activate_grad2(float& z0, float& z1) {
    if constexpr (ACT == SSA_ACT_SILU) {
        const float t0 = sigmoid<T>(z0), t1 = sigmoid<T>(z1);
        float u0, u1;       // t + z t (1 - t)
        fma2(u0, u1, -t0, -t1, t0, t1, t0, t1);
        fma2(z0, z1, z0, z1, u0, u1, t0, t1);
    } else {
        z0 = activate_grad<T, ACT>(z0);
        z1 = activate_grad<T, ACT>(z1);
    }
}

// The second launch of a call starts while the first one's last CTAs run, sends off its rows and waits here for the
// first to end.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- forward -----------------------------------------------------------------------------------

template <typename T, int A, int STAGES>
__device__ __forceinline__ Rows<T, A, 1, STAGES> norm_rows(const NormArgs& a, const Block& b, const Tile& tile, char* ring) {
    return {{(const T*)a.x + (tile.t0 + b.lane) * a.x_ts + b.c0 + b.vec * A}, {a.rl * a.x_ts}, row_count(a, b, tile.n),
            b.chunks<A>(), b.nvec * A, ring};
}

// Mean and squared deviations of a tile per group of the column block, from its rows.
template <typename T, int A, bool KEPT, typename ROWS>
__device__ __forceinline__ void sum_tile(const NormArgs& a, const Block& b, const Tile& tile, ROWS& rows, float2* red) {
    constexpr int V = Pieces<T, A>::V;
    const int n = tile.n, row_c = red_row(a, V), count = rows.count;
    const uint32_t slot = tile.slot;
    if (count) {
        float p[V], sum[V], sq[V];      // p: the pivot, negated
        rows.template peek<KEPT>(p);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = -p[j];
            sum[j] = sq[j] = 0.0f;
        }
        rows.template each<KEPT>([&](const float (&e)[1][V]) {
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                float d0, d1;
                add2(d0, d1, e[0][j], e[0][j + 1], p[j], p[j + 1]);
                add2(sum[j], sum[j + 1], sum[j], sum[j + 1], d0, d1);
                fma2(sq[j], sq[j + 1], d0, d1, d0, d1, sq[j], sq[j + 1]);
            }
        }, [&] {
            // on about the mean of the rows so far: p moves by delta
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float to = fmaf(sum[j], -1.0f / kSettled, p[j]), delta = p[j] - to, rest = fmaf(-(float)kSettled, delta, sum[j]);
                sq[j] = fmaf(-delta, sum[j] + rest, sq[j]);
                sum[j] = rest;
                p[j] = to;
            }
        });
        const float inv = 1.0f / (float)count;
        float2* mine = red + b.lane * row_c;
#pragma unroll
        for (int j = 0; j < V; ++j) mine[b.relative<A>(j)] = make_float2(fmaf(sum[j], inv, -p[j]), sq[j] - sum[j] * sum[j] * inv);
    }
    __syncthreads();
    // the channels' row lanes into row 0, then the groups' channels: the mean first, then the deviations from it, as one
    // lane or channel far from the others would cancel in a variance about it by their number (up to 256 and 680). What the
    // mean is off by comes back as the deviations' sum.
    const int less = n / a.rl, more = n - less * a.rl, lanes = min(a.rl, n);    // rows per lane; lanes with one more
    const float inv_n = 1.0f / (float)n;
    for_channels(a, b, [&](int c, bool valid, int q, int Q) {
        const float first = red[c].x;
        float sum = 0.0f, rest = 0.0f, sq = 0.0f;
        for (int l = q; l < lanes; l += Q) sum = fmaf(l < more ? less + 1.0f : (float)less, red[l * row_c + c].x - first, sum);
        const float mean = fmaf(lane_sum(sum, Q), inv_n, first);
        for (int l = q; l < lanes; l += Q) {
            const float2 v = red[l * row_c + c];
            const float k = l < more ? less + 1.0f : (float)less, d = v.x - mean;
            rest = fmaf(k, d, rest);
            sq += fmaf(k * d, d, v.y);
        }
        rest = lane_sum(rest, Q);
        sq = lane_sum(sq, Q);
        __syncwarp();       // row 0 is read by all lanes of the channel
        if (q == 0 && valid) red[c] = make_float2(fmaf(rest, inv_n, mean), sq);
    });
    __syncthreads();
    for_groups(a, b, [&](int g, int lo, int hi, int l, int L) {
        const float first = lo < hi ? red[lo].x : 0.0f, inv = lo < hi ? 1.0f / (float)(hi - lo) : 0.0f;
        float sum = 0.0f, rest = 0.0f, sq = 0.0f;
        for (int c = lo + l; c < hi; c += L) sum += red[c].x - first;
        const float mean = fmaf(lane_sum(sum, L), inv, first);
        for (int c = lo + l; c < hi; c += L) {
            const float d = red[c].x - mean;
            rest += d;
            sq += fmaf(n * d, d, red[c].y);
        }
        rest = lane_sum(rest, L);
        sq = lane_sum(sq, L);
        if (l == 0 && lo < hi)
            a.group_part[((int64_t)slot * a.over + b.index - first_block(a, g, V)) * a.G + g] = make_float2(fmaf(rest, inv, mean), sq);
    });
}

// Sequences without tokens have one empty tile.
__device__ __forceinline__ void write_empty(const NormArgs& a, const Block& b, const Tile& tile) {
    if (tile.tiles == 0 && a.mean)
        for (int g = b.g0 + threadIdx.x; g <= b.g1; g += kThreads)
            a.mean[(int64_t)tile.s * a.G + g] = a.rstd[(int64_t)tile.s * a.G + g] = 0.0f;
}

// Four CTAs per SM (64 registers); with 2-byte chunks three, whose batches of rows lie in registers (109,000 x 211 fp16: 86 us, with
// two 94).
template <typename T, int A>
__global__ void __launch_bounds__(kThreads, A * sizeof(T) == 2 ? 3 : 4) k_norm_stats(const __grid_constant__ NormArgs a) {
    constexpr int V = Pieces<T, A>::V;
    extern __shared__ __align__(16) char smem[];
    float2* red = (float2*)smem;        // [rl][red_row], then the ring
    let_next_launch_start();
    const uint32_t slot = blockIdx.x / a.blocks;
    const Block b(a, blockIdx.x - slot * a.blocks, V);
    const Tile tile(a, slot);
    if (tile.n == 0) return write_empty(a, b, tile);
    auto rows = norm_rows<T, A, kStages>(a, b, tile, smem + red_bytes(a, V));
    rows.start();
    sum_tile<T, A, false>(a, b, tile, rows, red);
}

// Lanes per group where a CTA adds up the tiles' sums.
__host__ __device__ inline int merge_lanes(int groups) {
    int L = 32;
    while (L > 4 && kThreads / L < groups) L /= 2;
    return L;
}

// f(g, lane, lanes) for the block's groups, several lanes of a warp to a group: all 32 for few groups, at least 4 for
// many; all threads take part, those beyond the last group with group g1 and `valid` false.
template <typename F>
__device__ __forceinline__ void for_merges(const Block& b, F f) {
    const int L = merge_lanes(b.g1 - b.g0 + 1);
    for (int base = b.g0; base <= b.g1; base += kThreads / L) {
        const int g = base + threadIdx.x / L;
        f(min(g, b.g1), g <= b.g1, threadIdx.x % L, L);
    }
}

// Mean and rstd of the block's groups in the tile's sequence into shared memory, from the tiles' in fp64 about the first
// tile's mean.
__device__ __forceinline__ void merge_stats(const NormArgs& a, const Block& b, const Tile& tile, int V, float2* stats) {
    const int s = tile.s;
    const int64_t tokens = a.seqs[s].hi - a.seqs[s].lo;
    const uint32_t slot0 = first_slot(a, s);
    for_merges(b, [&](int g, bool valid, int l, int L) {
        const int o0 = first_block(a, g, V), overlaps = last_block(a, g, V) - o0 + 1, cols = a.nv * V;
        const float2* part = a.group_part + (int64_t)slot0 * a.over * a.G + g;
        const double first = part->x;
        double sum = 0.0, sq = 0.0;
        for (int o = 0; o < overlaps; ++o) {
            const int from = (o0 + o) * cols;
            const int c = min((g + 1) * a.width, from + cols) - max(g * a.width, from);    // its channels in the block
#pragma unroll 8
            for (int i = l; i < tile.tiles; i += L) {
                const float2 v = part[((int64_t)i * a.over + o) * a.G];
                const double k = (double)((int)min((int64_t)a.R, tokens - (int64_t)i * a.R) * c), d = (double)v.x - first;
                sum += k * d;
                sq += (double)v.y + k * d * d;
            }
        }
        sum = lane_sum(sum, L);
        sq = lane_sum(sq, L);
        if (l == 0 && valid) {
            const double m = (double)tokens * a.width, d = sum / m, var = fmax(sq / m - d * d, 0.0);
            // a NaN or an infinity among the values leaves NaN here (fmax drops it)
            const float mean = (float)(first + d), rstd = sq == sq ? (float)(1.0 / sqrt(var + (double)a.eps)) : (float)sq;
            stats[g - b.g0] = make_float2(mean, rstd);
            if (tile.opens && a.mean && o0 == b.index) {
                a.mean[(int64_t)s * a.G + g] = mean;
                a.rstd[(int64_t)s * a.G + g] = rstd;
            }
        }
    });
}

// The outputs of a tile, with the groups' mean and rstd in `stats`.
template <typename T, int A, int ACT, bool KEPT, typename ROWS>
__device__ __forceinline__ void apply_tile(const NormArgs& a, const Block& b, const Tile& tile, ROWS& rows, const float2* stats) {
    constexpr int V = Pieces<T, A>::V;
    if (rows.count) {
        float mean[V], scale[V], beta[V];       // mean: negated
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = b.channel<A>(j);
            const float2 st = stats[group_of(a, c) - b.g0];
            mean[j] = -st.x;
            scale[j] = st.y * (a.gamma ? a.gamma[c] : 1.0f);
            beta[j] = a.beta ? a.beta[c] : 0.0f;
        }
        const int64_t out_step = a.rl * a.o_ts;
        T* out = (T*)a.out + (tile.t0 + b.lane) * a.o_ts + b.c0 + b.vec * A;
        rows.template each<KEPT>([&](const float (&e)[1][V]) {
            float z[V];
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                add2(z[j], z[j + 1], e[0][j], e[0][j + 1], mean[j], mean[j + 1]);
                fma2(z[j], z[j + 1], z[j], z[j + 1], scale[j], scale[j + 1], beta[j], beta[j + 1]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = activate<T, ACT>(z[j]);
            Pieces<T, A>::store(out, z, rows.chunks, rows.hop);
            out += out_step;
        });
    }
}

template <typename T, int A, int ACT>
__global__ void __launch_bounds__(kThreads, 4) k_norm_apply(const __grid_constant__ NormArgs a) {
    constexpr int V = Pieces<T, A>::V;
    extern __shared__ __align__(16) char smem[];
    float2* stats = (float2*)(smem + Rows<T, A, 1, kStages>::kBytes);     // the block's groups, after the ring
    const uint32_t i = gridDim.x - 1 - blockIdx.x, slot = i / a.blocks;
    const Block b(a, i - slot * a.blocks, V);
    const Tile tile(a, slot);
    if (tile.n == 0) return;
    auto rows = norm_rows<T, A, kStages>(a, b, tile, smem);
    rows.start();
    wait_for_last_launch();
    merge_stats(a, b, tile, V, stats);
    __syncthreads();
    apply_tile<T, A, ACT, false>(a, b, tile, rows, stats);
}

// Both passes in one cooperative launch, where all rows fit in the shared memory of the CTAs that run at once: read once,
// and the second pass waits for the grid instead of for a launch.
template <typename T, int A, int ACT>
__global__ void __launch_bounds__(kThreads, kKeptCtas) k_norm_kept(const __grid_constant__ NormArgs a) {
    constexpr int V = Pieces<T, A>::V;
    extern __shared__ __align__(16) char smem[];
    float2* red = (float2*)(smem + Rows<T, A, 1, kKeptRows>::kBytes);     // then the block's groups
    const uint32_t slot = blockIdx.x / a.blocks;
    const Block b(a, blockIdx.x - slot * a.blocks, V);
    const Tile tile(a, slot);
    auto rows = norm_rows<T, A, kKeptRows>(a, b, tile, smem);
    if (tile.n == 0) {
        write_empty(a, b, tile);
    } else {
        rows.start_kept();
        sum_tile<T, A, true>(a, b, tile, rows, red);
    }
    cooperative_groups::this_grid().sync();
    if (tile.n == 0) return;
    merge_stats(a, b, tile, V, red);
    __syncthreads();
    apply_tile<T, A, ACT, true>(a, b, tile, rows, red);
}

// ---- gradient ------------------------------------------------------------------------------------

// A thread's channel constants in one sequence: mean (negated), rstd * gamma, beta. The loops work on x - mean and
// leave the factors rstd to the sums.
template <int V>
struct Channels {
    float mean[V], scale[V], beta[V];
    template <int A>
    __device__ __forceinline__ void load(const NormArgs& a, const Block& b, int s) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = b.channel<A>(j);
            const int64_t at = (int64_t)s * a.G + group_of(a, c);
            mean[j] = -a.mean[at];
            scale[j] = a.rstd[at] * (a.gamma ? a.gamma[c] : 1.0f);
            beta[j] = a.beta ? a.beta[c] : 0.0f;
        }
    }
};

// x - mean and dz of one row's vector: e = {x, dy}.
template <typename T, int V, int ACT>
__device__ __forceinline__ void row_grad(const Channels<V>& ch, const float (&e)[2][V], float (&xc)[V], float (&dz)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        add2(xc[j], xc[j + 1], e[0][j], e[0][j + 1], ch.mean[j], ch.mean[j + 1]);
        if constexpr (ACT == SSA_ACT_NONE) {
            dz[j] = e[1][j];
            dz[j + 1] = e[1][j + 1];
        } else {
            float z0, z1;
            fma2(z0, z1, xc[j], xc[j + 1], ch.scale[j], ch.scale[j + 1], ch.beta[j], ch.beta[j + 1]);
            activate_grad2<T, ACT>(z0, z1);
            mul2(dz[j], dz[j + 1], e[1][j], e[1][j + 1], z0, z1);
        }
    }
}

template <typename T, int A>
__device__ __forceinline__ Rows<T, A, 2, kGradStages> grad_rows(const NormArgs& a, const Block& b, const Tile& tile, char* ring) {
    const int64_t row = tile.t0 + b.lane;
    const int c0 = b.c0 + b.vec * A;
    return {{(const T*)a.x + row * a.x_ts + c0, (const T*)a.dy + row * a.dy_ts + c0},
            {a.rl * a.x_ts, a.rl * a.dy_ts}, row_count(a, b, tile.n), b.chunks<A>(), b.nvec * A, ring};
}

// Sums of a tile: per channel dz and dz * xhat, per group of the column block the same times gamma.
template <typename T, int A, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_norm_grad_sums(const __grid_constant__ NormArgs a) {
    constexpr int V = Pieces<T, A>::V;
    extern __shared__ __align__(16) char smem[];
    float2* red = (float2*)smem;
    let_next_launch_start();
    const uint32_t slot = blockIdx.x / a.blocks;
    const Block b(a, blockIdx.x - slot * a.blocks, V);
    const Tile tile(a, slot);
    const int s = tile.s, n = tile.n, row_c = red_row(a, V), lanes = min(a.rl, n);
    if (n == 0) return;
    auto rows = grad_rows<T, A>(a, b, tile, smem + red_bytes(a, V));
    rows.start();
    if (rows.count) {
        Channels<V> ch;
        ch.template load<A>(a, b, s);
        float s0[V], s1[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s0[j] = s1[j] = 0.0f;
        rows.template each<false>([&](const float (&e)[2][V]) {
            float xc[V], dz[V];
            row_grad<T, V, ACT>(ch, e, xc, dz);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                add2(s0[j], s0[j + 1], s0[j], s0[j + 1], dz[j], dz[j + 1]);
                fma2(s1[j], s1[j + 1], dz[j], dz[j + 1], xc[j], xc[j + 1], s1[j], s1[j + 1]);
            }
        });
        float2* mine = red + b.lane * row_c;
#pragma unroll
        for (int j = 0; j < V; ++j) mine[b.relative<A>(j)] = make_float2(s0[j], s1[j]);
    }
    __syncthreads();
    for_channels(a, b, [&](int c, bool valid, int q, int Q) {
        float s0 = 0.0f, s1 = 0.0f;
        for (int l = q; l < lanes; l += Q) {
            const float2 v = red[l * row_c + c];
            s0 += v.x;
            s1 += v.y;
        }
        s0 = lane_sum(s0, Q);
        s1 = lane_sum(s1, Q);
        if (q == 0 && valid) {
            s1 *= a.rstd[(int64_t)s * a.G + group_of(a, b.c0 + c)];
            a.chan_part[(int64_t)slot * a.C + b.c0 + c] = make_float2(s0, s1);
            const float gamma = a.gamma ? a.gamma[b.c0 + c] : 1.0f;
            red[c] = make_float2(s0 * gamma, s1 * gamma);
        }
    });
    __syncthreads();
    for_groups(a, b, [&](int g, int lo, int hi, int l, int L) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = lo + l; c < hi; c += L) {
            s1 += red[c].x;
            s2 += red[c].y;
        }
        s1 = lane_sum(s1, L);
        s2 = lane_sum(s2, L);
        if (l == 0 && lo < hi)
            a.group_part[((int64_t)slot * a.over + b.index - first_block(a, g, V)) * a.G + g] = make_float2(s1, s2);
    });
}

// rstd * S1 and rstd^2 * S2, negated, of the block's groups in sequence s into shared memory.
__device__ __forceinline__ void merge_sums(const NormArgs& a, const Block& b, const Tile& tile, int V, float2* sums) {
    const int s = tile.s;
    const uint32_t slot0 = first_slot(a, s);
    for_merges(b, [&](int g, bool valid, int l, int L) {
        const int overlaps = last_block(a, g, V) - first_block(a, g, V) + 1;
        const float2* part = a.group_part + (int64_t)slot0 * a.over * a.G + g;
        double s1 = 0.0, s2 = 0.0;
        for (int o = 0; o < overlaps; ++o) {
#pragma unroll 8
            for (int i = l; i < tile.tiles; i += L) {
                const float2 v = part[((int64_t)i * a.over + o) * a.G];
                s1 += v.x;
                s2 += v.y;
            }
        }
        s1 = lane_sum(s1, L);
        s2 = lane_sum(s2, L);
        if (l == 0 && valid) {
            const double r = a.rstd[(int64_t)s * a.G + g], f = -r / ((double)(a.seqs[s].hi - a.seqs[s].lo) * a.width);
            sums[g - b.g0] = make_float2((float)(f * s1), (float)(f * r * s2));
        }
    });
}

// The weights' gradients of 32 channels: the sums of all tiles, in fp64.
__device__ __forceinline__ void merge_weights(const NormArgs& a, int c0, double2* red) {
    const int c = c0 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    double2 acc = make_double2(0.0, 0.0);
    if (c < a.C) {
        for (int s = 0; s < a.B; ++s) {
            const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
            if (hi <= lo) continue;
            const int64_t from = first_slot(a, s), to = from + (uint32_t)(hi - lo - 1) / a.R;
#pragma unroll 4
            for (int64_t i = from + w; i <= to; i += kThreads / 32) {
                const float2 v = a.chan_part[i * a.C + c];
                acc.x += v.x;
                acc.y += v.y;
            }
        }
    }
    red[threadIdx.x] = acc;
    __syncthreads();
    if (w == 0 && c < a.C) {
        for (int i = 1; i < kThreads / 32; ++i) {
            acc.x += red[i * 32 + threadIdx.x].x;
            acc.y += red[i * 32 + threadIdx.x].y;
        }
        a.dbeta[c] = (float)acc.x;
        a.dgamma[c] = (float)acc.y;
    }
}

// dx, the tiles in reverse; the first CTAs add up the weights' gradients, 32 channels each.
template <typename T, int A, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_norm_grad_apply(const __grid_constant__ NormArgs a) {
    constexpr int V = Pieces<T, A>::V;
    extern __shared__ __align__(16) char smem[];
    float2* sums = (float2*)(smem + Rows<T, A, 2, kGradStages>::kBytes);
    const uint32_t weights = (a.C + 31) / 32;
    if (blockIdx.x < weights) {
        wait_for_last_launch();
        merge_weights(a, blockIdx.x * 32, (double2*)smem);
        return;
    }
    const uint32_t i = gridDim.x - 1 - blockIdx.x, slot = i / a.blocks;
    const Block b(a, i - slot * a.blocks, V);
    const Tile tile(a, slot);
    const int s = tile.s;
    if (tile.n == 0) return;
    auto rows = grad_rows<T, A>(a, b, tile, smem);
    rows.start();
    wait_for_last_launch();
    merge_sums(a, b, tile, V, sums);
    __syncthreads();
    if (rows.count) {
        const int c0 = b.c0 + b.vec * A;
        Channels<V> ch;
        ch.template load<A>(a, b, s);
        float S1[V], S2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 v = sums[group_of(a, b.channel<A>(j)) - b.g0];
            S1[j] = v.x;
            S2[j] = v.y;
        }
        const int64_t out_step = a.rl * a.o_ts;
        T* out = (T*)a.out + (tile.t0 + b.lane) * a.o_ts + c0;
        rows.template each<false>([&](const float (&e)[2][V]) {
            float xc[V], dz[V];
            row_grad<T, V, ACT>(ch, e, xc, dz);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                fma2(dz[j], dz[j + 1], dz[j], dz[j + 1], ch.scale[j], ch.scale[j + 1], S1[j], S1[j + 1]);
                fma2(dz[j], dz[j + 1], xc[j], xc[j + 1], S2[j], S2[j + 1], dz[j], dz[j + 1]);
            }
            Pieces<T, A>::store(out, dz, rows.chunks, rows.hop);
            out += out_step;
        });
    }
}

// ---- host --------------------------------------------------------------------------------------

template <void (*K)(NormArgs)>
using Kernel = std::integral_constant<void (*)(NormArgs), K>;

struct Launch {
    bool grad;
    int act, A, device;     // A: elements per chunk
    bool kept;              // the one-launch forward
    cudaStream_t st;
};

template <typename T, int A, int ACT>
bool launch_act(const NormArgs& a, const Launch& l) {
    constexpr int V = Pieces<T, A>::V;
    const unsigned grid = a.slots * (unsigned)a.blocks;
    const size_t red = red_bytes(a, V), groups = sizeof(float2) * std::min(a.G, a.nv * V);    // at most 32 and 16 KB
    enum Mode { kPlain, kEarly, kCooperative };
    auto go = [&](auto tag, unsigned ctas, size_t smem, Mode mode) {
        constexpr auto kernel = decltype(tag)::value;
        if (!allow_smem<kernel>(l.device)) return false;
        cudaLaunchAttribute attr = {};
        if (mode == kCooperative) {
            attr.id = cudaLaunchAttributeCooperative;
            attr.val.cooperative = 1;
        } else {
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
        }
        cudaLaunchConfig_t config = {};
        config.gridDim = dim3(ctas);
        config.blockDim = dim3(kThreads);
        config.dynamicSmemBytes = smem;
        config.stream = l.st;
        config.attrs = &attr;
        config.numAttrs = mode == kPlain ? 0 : 1;
        if (cudaLaunchKernelEx(&config, kernel, a) != cudaSuccess) return false;
        note_launch();
        return true;
    };
    if (l.grad) {
        const size_t ring = Rows<T, A, 2, kGradStages>::kBytes;
        return go(Kernel<k_norm_grad_sums<T, A, ACT>>(), grid, red + ring, kPlain) &&
               go(Kernel<k_norm_grad_apply<T, A, ACT>>(), grid + (unsigned)cdiv(a.C, 32), std::max(ring + groups, sizeof(double2) * kThreads), kEarly);
    }
    if constexpr (Rows<T, A, 1, kStages>::kRing) {
        if (l.kept) {
            if (go(Kernel<k_norm_kept<T, A, ACT>>(), grid, Rows<T, A, 1, kKeptRows>::kBytes + std::max(red, groups), kCooperative))
                return true;
            // fewer SMs than the device has (a partition of it): the two launches do the same
            if (cudaGetLastError() != cudaErrorCooperativeLaunchTooLarge) return false;
        }
    }
    const size_t ring = Rows<T, A, 1, kStages>::kBytes;
    return go(Kernel<k_norm_stats<T, A>>(), grid, red + ring, kPlain) && go(Kernel<k_norm_apply<T, A, ACT>>(), grid, ring + groups, kEarly);
}

template <typename T, int A>
bool launch_chunk(const NormArgs& a, const Launch& l) {
    if (l.act == SSA_ACT_SILU) return launch_act<T, A, SSA_ACT_SILU>(a, l);
    if (l.act == SSA_ACT_GELU) return launch_act<T, A, SSA_ACT_GELU>(a, l);
    return launch_act<T, A, SSA_ACT_NONE>(a, l);
}

template <typename T>
bool launch_type(const NormArgs& a, const Launch& l) {
    if constexpr (sizeof(T) == 2) {
        if (l.A == 8) return launch_chunk<T, 8>(a, l);
    }
    if (l.A == 4) return launch_chunk<T, 4>(a, l);
    if (l.A == 2) return launch_chunk<T, 2>(a, l);
    return launch_chunk<T, 1>(a, l);
}

// Column blocks and tiles of a call; true where all rows can be kept on the SMs.
bool shape(NormArgs& a, int V, int chunk, int sms, int per_sm, bool may_keep) {
    a.nvt = (int32_t)cdiv(a.C, V);
    // vectors per block: at least kBlockBytes of a row in a round of chunks, the narrowest that keeps nine tenths of the threads on vectors
    const int least = std::min(a.nvt, kBlockBytes / chunk);
    int best = -1;
    for (int n = least; n <= std::min(a.nvt, 4 * least); ++n) {
        const int used = (int)((int64_t)100 * a.nvt * (kThreads / n) / (cdiv(a.nvt, n) * kThreads));
        if (used > best) {
            best = used;
            a.nv = n;
        }
        if (best >= 90) break;
    }
    a.rl = kThreads / a.nv;
    a.blocks = (int32_t)cdiv(a.nvt, a.nv);
    a.over = std::min<int32_t>(a.blocks, (a.width - 1 + a.nv * V - 1) / (a.nv * V) + 1);
    a.clanes = a.glanes = 1;
    while (a.clanes < 32 && a.clanes * 2 <= a.rl && a.clanes * 2 * a.nv * V <= kThreads) a.clanes *= 2;
    while (a.glanes < 32 && a.glanes < std::min(a.width, a.nv * V)) a.glanes *= 2;
    a.magic = (uint32_t)((((uint64_t)1 << 32) + a.width - 1) / a.width);
    // tokens per tile, a multiple of the row lanes: kRowsPerThread a thread; less where that leaves SMs without CTAs, but
    // not for so many tiles that adding up their sums, which every CTA of the second pass does, takes long
    const int groups = std::min(a.G, (a.nv * V + a.width - 2) / a.width + 1);
    const int64_t most = std::max<int64_t>(kTilesPerLane * merge_lanes(groups), kMinTiles);
    const size_t kept_smem = (size_t)kKeptRows * kThreads * kVecBytes + std::max(red_bytes(a, V), sizeof(float2) * a.nv * V);
    const int64_t kept_ctas = std::min<int64_t>(kKeptCtas, 227 * 1024 / (kept_smem + 1024)) * sms;
    const int64_t room = std::min(most, kept_ctas / a.blocks - a.B);      // slots: tiles and one for each sequence
    if (may_keep && room > 0 && cdiv(cdiv(a.N, room), a.rl) <= kKeptRows) {
        a.R = (uint32_t)(a.rl * cdiv(cdiv(a.N, room), a.rl));
        a.slots = (uint32_t)(a.N / a.R + a.B);
        return true;
    }
    const int64_t tiles = std::min(most, (int64_t)std::max(1, per_sm * sms / a.blocks));
    a.R = (uint32_t)(a.rl * std::min<int64_t>(kRowsPerThread, cdiv(cdiv(a.N, tiles), a.rl)));
    a.slots = (uint32_t)(a.N / a.R + a.B);
    return false;
}

struct Call {
    const ssa_rows_t* x;
    const ssa_rows_t* dy;
    const ssa_rows_t* out;
    const float* gamma;
    const float* beta;
    float* mean;
    float* rstd;
    float* dgamma;
    float* dbeta;
};

ssa_status_t run_norm(Plan* p, const Call& c, int32_t C, int32_t G, float eps, int act, ssa_dtype_t dt, cudaStream_t st) {
    const bool grad = c.dy != nullptr;
    if (!p || p->owned.empty() || !c.x || !c.out) return SSA_ERR_INVALID_ARG;
    if (C < 1 || G < 1 || C % G) return SSA_ERR_INVALID_ARG;
    if (C > kMaxChannels) return SSA_ERR_UNSUPPORTED;
    if (dt != SSA_F32 && dt != SSA_BF16 && dt != SSA_F16) return SSA_ERR_INVALID_ARG;
    if (act != SSA_ACT_NONE && act != SSA_ACT_SILU && act != SSA_ACT_GELU) return SSA_ERR_INVALID_ARG;
    if ((c.gamma == nullptr) != (c.beta == nullptr)) return SSA_ERR_INVALID_ARG;
    if (grad ? (!c.mean || !c.rstd || !c.dgamma || !c.dbeta) : !(eps >= 0.0f) || std::isinf(eps)) return SSA_ERR_INVALID_ARG;
    if ((c.mean == nullptr) != (c.rstd == nullptr)) return SSA_ERR_INVALID_ARG;
    if (!aligned4(c.gamma, c.beta, c.mean, c.rstd, c.dgamma, c.dbeta)) return SSA_ERR_INVALID_ARG;
    // the pass that writes reads the weights (and the gradient's the statistics) while other CTAs of it write these
    const int64_t stats = (int64_t)p->B * G;
    const Span gamma = {c.gamma, C}, beta = {c.beta, C}, mean = {c.mean, stats}, rstd = {c.rstd, stats};
    const Span outs[2] = {grad ? Span{c.dgamma, C} : mean, grad ? Span{c.dbeta, C} : rstd};
    if (!apart(outs[0], outs[1])) return SSA_ERR_INVALID_ARG;
    for (const Span& o : outs)
        if (!apart(o, gamma) || !apart(o, beta) || (grad && (!apart(o, mean) || !apart(o, rstd)))) return SSA_ERR_INVALID_ARG;
    const int64_t N = p->N;
    const size_t es = dt == SSA_F32 ? 4 : 2;
    auto view = [](const ssa_rows_t* r) { return ssa_heads_t{r->data, r->token_stride, 0, 1}; };
    const ssa_heads_t x = view(c.x), out = view(c.out), dy = grad ? view(c.dy) : x;
    if (!check_view(&x, N, C, es, false) || !check_view(&out, N, C, es, true) || !check_view(&dy, N, C, es, false))
        return SSA_ERR_INVALID_ARG;
    for (const ssa_heads_t* in : {&x, &dy})
        if (!same_view(out, *in, N) && !disjoint(out, *in, N, C, es)) return SSA_ERR_INVALID_ARG;

    int A = kVecBytes / (int)es;
    while (A > 1 && C % A) A >>= 1;
    for (const ssa_heads_t* v : {&x, &dy, &out}) A = view_vector(*v, N, es, A);
    NormArgs a = {};
    a.x = x.data;
    a.dy = dy.data;
    a.out = out.data;
    a.x_ts = x.token_stride;
    a.dy_ts = dy.token_stride;
    a.o_ts = out.token_stride;
    a.gamma = c.gamma;
    a.beta = c.beta;
    a.dgamma = c.dgamma;
    a.dbeta = c.dbeta;
    a.seqs = p->d_seqs;
    a.N = N;
    a.B = p->B;
    a.C = C;
    a.G = G;
    a.width = C / G;
    a.eps = eps;
    const DeviceScope on(p->device);
    if (!on.ok) return SSA_ERR_CUDA;
    const bool kept = shape(a, kVecBytes / (int)es, A * (int)es, sm_count(p->device), grad ? 2 : 4, !grad && A * es >= 4);
    if ((int64_t)a.slots * a.blocks >= ((int64_t)1 << 30)) return SSA_ERR_UNSUPPORTED;
    // one buffer of the tiles' sums
    const int64_t n_group = (int64_t)a.slots * a.over * G, n_chan = grad ? (int64_t)a.slots * C : 0;
    a.group_part = (float2*)p->alloc(sizeof(float2) * (size_t)(n_group + n_chan), st, p->alloc_ctx);
    if (!a.group_part) return SSA_ERR_ALLOC;
    a.chan_part = a.group_part + n_group;
    a.mean = c.mean;
    a.rstd = c.rstd;
    const char* name = grad ? "group_norm_backward" : "group_norm";
    ProfScope ps(name, st);
    const Launch l = {grad, act, A, p->device, kept, st};
    const bool ok = dt == SSA_F32    ? launch_type<float>(a, l)
                    : dt == SSA_BF16 ? launch_type<__nv_bfloat16>(a, l)
                                     : launch_type<__half>(a, l);
    p->release(a.group_part, st, p->alloc_ctx);
    trace_step(name, st);
    const bool clear = cudaGetLastError() == cudaSuccess;     // read in any case: the next call is not to find it
    return ok && clear ? SSA_OK : SSA_ERR_CUDA;
}

}  // namespace

}  // namespace ssa

using namespace ssa;

extern "C" {

ssa_status_t ssa_group_norm(ssa_plan_t plan, const ssa_rows_t* x, int32_t channels, int32_t groups, const float* gamma,
                            const float* beta, float eps, ssa_activation_t activation, ssa_dtype_t dtype,
                            const ssa_rows_t* y, float* mean, float* rstd, void* stream) {
    const Call c = {x, nullptr, y, gamma, beta, mean, rstd, nullptr, nullptr};
    return run_norm(plan, c, channels, groups, eps, activation, dtype, (cudaStream_t)stream);
}

ssa_status_t ssa_group_norm_backward(ssa_plan_t plan, const ssa_rows_t* dy, const ssa_rows_t* x, const float* mean,
                                     const float* rstd, int32_t channels, int32_t groups, const float* gamma,
                                     const float* beta, ssa_activation_t activation, ssa_dtype_t dtype,
                                     const ssa_rows_t* dx, float* dgamma, float* dbeta, void* stream) {
    if (!dy) return SSA_ERR_INVALID_ARG;
    const Call c = {x, dy, dx, gamma, beta, const_cast<float*>(mean), const_cast<float*>(rstd), dgamma, dbeta};
    return run_norm(plan, c, channels, groups, 0.0f, activation, dtype, (cudaStream_t)stream);
}

}  // extern "C"
