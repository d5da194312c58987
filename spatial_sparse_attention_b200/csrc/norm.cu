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
// blocks of whole vectors, whatever the groups' width: a thread keeps one vector of channels and walks rows, so
// channel constants stay in registers; a group across column blocks has sums in each. The second pass takes the
// tiles in reverse: what the first read last is still in L2.
// A tile that crosses sequences is cut at their borders: the part of tile t that lies in sequence s has slot
// t + s in the tables of sums, unique and increasing along the tokens.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "views.cuh"

namespace ssa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxChannels = 65536;
// Rows per thread of a full tile. The variance of a thread's rows comes from sums about its first row: with n rows
// the cancellation is at most a factor n, as the pivot is one of them (sq <= n D^2, D the largest deviation from it, and
// the squared deviations from the mean are at least D^2 / 2).
constexpr int kRowsPerThread = 48;
constexpr int kBlockBytes = 128;        // least width of a column block
constexpr int kStages = 8;              // rows per thread in flight or in use: forward, gradient
constexpr int kGradStages = 6;

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
    uint32_t R, tiles;      // tokens per tile; tiles
    int32_t B, C, G, width;
    uint32_t magic;         // ceil(2^32 / width), see group_of
    int32_t nvt, nv, rl;    // vectors per row; vectors and row lanes of a CTA
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
        c1 = c0 + nvec * V;
        g0 = group_of(a, c0);
        g1 = group_of(a, c1 - 1);
        lane = threadIdx.x / a.nv;
        vec = threadIdx.x - lane * a.nv;
    }
    __device__ __forceinline__ bool active(const NormArgs& a) const { return lane < a.rl && vec < nvec; }
    __device__ __forceinline__ int channel(int V) const { return c0 + vec * V; }
};

// First column block of a group.
__device__ __forceinline__ int first_block(const NormArgs& a, int g, int V) { return g * a.width / (a.nv * V); }
__device__ __forceinline__ int last_block(const NormArgs& a, int g, int V) { return ((g + 1) * a.width - 1) / (a.nv * V); }

// Calls f(s, first token, end) for every part of the tile that lies in one sequence.
template <typename F>
__device__ __forceinline__ void for_segments(const NormArgs& a, int64_t tile, F f) {
    int64_t t = tile * a.R;
    const int64_t end = min(a.N, t + a.R);
    for (int s = find_seq(a.seqs, a.B, t); t < end; ++s) {
        const int64_t e = min(a.seqs[s].hi, end);
        if (e <= t) continue;
        f(s, t, e);
        t = e;
    }
}

// This thread's `count` rows of K arrays, `step` elements apart, its loads STAGES - 1 rows ahead in its own places of
// the ring: no barrier and no registers for what is in flight. Rows of 2-byte loads, which the
// asynchronous copy does not take, come in batches through registers instead.
template <typename T, int V, int K, int STAGES>
struct Rows {
    using W = Vec<T, V>;
    using C = typename W::C;
    static constexpr bool kRing = sizeof(C) >= 4;
    static constexpr size_t kBytes = kRing ? STAGES * K * kThreads * sizeof(C) : 0;
    const T* at[K];
    int64_t step[K];
    int count, left;    // rows; those not asked for yet
    char* ring;

    __device__ __forceinline__ C* place(int stage, int k) const { return (C*)ring + (stage * K + k) * kThreads + threadIdx.x; }
    __device__ __forceinline__ void fetch(int stage) {
        if (left > 0) {
            --left;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                cp_async<sizeof(C)>(place(stage, k), at[k]);
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
    // row 0, which stays to be read (count > 0)
    __device__ __forceinline__ void peek(float (&e)[V]) {
        if constexpr (kRing) {
            cp_wait<STAGES - 2>();
            W::unpack(*place(0, 0), e);
        } else {
            W::unpack(*reinterpret_cast<const C*>(at[0]), e);
        }
    }
    // f(e) for every row, e[k] being its vector of array k; f may write over the row (in place)
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        if constexpr (kRing) {
            for (int i = 0; i < count; i += STAGES) {
#pragma unroll
                for (int j = 0; j < STAGES; ++j) {
                    if (i + j < count) {
                        fetch((j + STAGES - 1) % STAGES);
                        cp_wait<STAGES - 1>();
                        float e[K][V];
#pragma unroll
                        for (int k = 0; k < K; ++k) W::unpack(*place(j, k), e[k]);
                        f(e);
                    }
                }
            }
        } else {
            constexpr int U = 8;
            for (int i = 0; i < count; i += U) {
                C raw[U][K];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + u < count) {
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            raw[u][k] = *reinterpret_cast<const C*>(at[k]);
                            at[k] += step[k];
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + u < count) {
                        float e[K][V];
#pragma unroll
                        for (int k = 0; k < K; ++k) W::unpack(raw[u][k], e[k]);
                        f(e);
                    }
                }
            }
        }
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

// sigma(z). The 16-bit types take the hardware's exponential and reciprocal (2^-20 relative for |z| < 16, far
// below their rounding); fp32 the exact functions.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    return rcp(1.0f + ex2(z * -1.4426950408889634f));
}
template <>
__device__ __forceinline__ float sigmoid<float>(float z) {
    return 1.0f / (1.0f + expf(-z));
}

// z -> act(z)
template <typename T, int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == SSA_ACT_SILU) return z * sigmoid<T>(z);
    if (ACT == SSA_ACT_GELU) return z * normcdff(z);
    return z;
}

template <typename T, int ACT>
__device__ __forceinline__ float activate_grad(float z) {
    if (ACT == SSA_ACT_SILU) {
        const float t = sigmoid<T>(z);
        return t * fmaf(z, 1.0f - t, 1.0f);
    }
    if (ACT == SSA_ACT_GELU) return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
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

// Sums of the tile's segments: per group of the column block, mean and squared deviations.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) k_norm_stats(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) char smem[];
    float2* red = (float2*)smem;        // [rl][red_row], then the ring
    let_next_launch_start();
    const uint32_t tile = blockIdx.x / a.blocks;
    const Block b(a, blockIdx.x - tile * a.blocks, V);
    if (tile == 0 && a.mean) {      // sequences without tokens have no tile
        for (int s = threadIdx.x; s < a.B; s += kThreads)
            if (a.seqs[s].hi == a.seqs[s].lo)
                for (int g = b.g0; g <= b.g1; ++g) a.mean[(int64_t)s * a.G + g] = a.rstd[(int64_t)s * a.G + g] = 0.0f;
    }
    for_segments(a, tile, [&](int s, int64_t t, int64_t e) {
        const int n = (int)(e - t), row_c = red_row(a, V);
        Rows<T, V, 1, kStages> rows = {{(const T*)a.x + (t + b.lane) * a.x_ts + b.channel(V)}, {a.rl * a.x_ts},
                                       row_count(a, b, n), 0, smem + red_bytes(a, V)};
        rows.start();
        const int count = rows.count;
        if (count) {
            float p[V], sum[V], sq[V];      // p: the first row, negated
            rows.peek(p);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                p[j] = -p[j];
                sum[j] = sq[j] = 0.0f;
            }
            rows.each([&](const float (&e)[1][V]) {
                if constexpr (V > 1) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        float d0, d1;
                        add2(d0, d1, e[0][j], e[0][j + 1], p[j], p[j + 1]);
                        add2(sum[j], sum[j + 1], sum[j], sum[j + 1], d0, d1);
                        fma2(sq[j], sq[j + 1], d0, d1, d0, d1, sq[j], sq[j + 1]);
                    }
                } else {
                    const float d = e[0][0] + p[0];
                    sum[0] += d;
                    sq[0] = fmaf(d, d, sq[0]);
                }
            });
            const float inv = 1.0f / (float)count;
            float2* mine = red + b.lane * row_c + b.vec * V;
#pragma unroll
            for (int j = 0; j < V; ++j) mine[j] = make_float2(fmaf(sum[j], inv, -p[j]), sq[j] - sum[j] * sum[j] * inv);
        }
        __syncthreads();
        // the channels' row lanes into row 0, then the groups' channels
        const int less = n / a.rl, more = n - less * a.rl, lanes = min(a.rl, n);    // rows per lane; lanes with one more
        for_channels(a, b, [&](int c, bool valid, int q, int Q) {
            const float first = red[c].x;
            float sum = 0.0f, sq = 0.0f;
            for (int l = q; l < lanes; l += Q) {
                const float2 v = red[l * row_c + c];
                const float k = l < more ? less + 1.0f : (float)less, d = v.x - first;
                sum = fmaf(k, d, sum);
                sq += fmaf(k * d, d, v.y);
            }
            sum = lane_sum(sum, Q);
            sq = lane_sum(sq, Q);
            const float inv = 1.0f / (float)n;
            if (q == 0 && valid) red[c] = make_float2(fmaf(sum, inv, first), sq - sum * sum * inv);
        });
        __syncthreads();
        for_groups(a, b, [&](int g, int lo, int hi, int l, int L) {
            const float first = lo < hi ? red[lo].x : 0.0f;
            float sum = 0.0f, sq = 0.0f;
            for (int c = lo + l; c < hi; c += L) {
                const float d = red[c].x - first;
                sum += d;
                sq += fmaf(n * d, d, red[c].y);
            }
            sum = lane_sum(sum, L);
            sq = lane_sum(sq, L);
            if (l == 0 && lo < hi) {
                const float d = sum / (float)(hi - lo);
                a.group_part[((int64_t)(tile + s) * a.over + b.index - first_block(a, g, V)) * a.G + g] =
                    make_float2(first + d, sq - n * sum * d);
            }
        });
        __syncthreads();    // red is read
    });
}

// f(g, tile sums' table, first slot, slots, overlaps): one warp per group of the column block in sequence s.
template <typename F>
__device__ __forceinline__ void for_group_warps(const NormArgs& a, const Block& b, F f) {
    for (int g = b.g0 + (threadIdx.x >> 5); g <= b.g1; g += kThreads / 32) f(g);
}

// Mean and rstd of the block's groups in sequence s into shared memory, from the tiles' in fp64 about the first
// tile's mean.
__device__ __forceinline__ void merge_stats(const NormArgs& a, const Block& b, int s, int V, bool write, float2* stats) {
    const int lane = threadIdx.x & 31;
    const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
    const int ta = (int)((uint32_t)lo / a.R), tiles = (int)((uint32_t)(hi - 1) / a.R) - ta + 1;
    for_group_warps(a, b, [&](int g) {
        const int o0 = first_block(a, g, V), overlaps = last_block(a, g, V) - o0 + 1, cols = a.nv * V;
        const float2* part = a.group_part + (int64_t)(ta + s) * a.over * a.G + g;
        const double first = part->x;
        double sum = 0.0, sq = 0.0;
        for (int o = 0; o < overlaps; ++o) {
            const int from = (o0 + o) * cols;
            const int c = min((g + 1) * a.width, from + cols) - max(g * a.width, from);    // its channels in the block
#pragma unroll 4
            for (int i = lane; i < tiles; i += 32) {
                const float2 v = part[((int64_t)i * a.over + o) * a.G];
                const int64_t t = (int64_t)(ta + i) * a.R;
                const double k = (double)((int)(min(hi, t + a.R) - max(lo, t)) * c), d = (double)v.x - first;
                sum += k * d;
                sq += (double)v.y + k * d * d;
            }
        }
        sum = lane_sum(sum, 32);
        sq = lane_sum(sq, 32);
        const double m = (double)(hi - lo) * a.width, d = sum / m, var = fmax(sq / m - d * d, 0.0);
        // a NaN or an infinity among the values leaves NaN here (fmax drops it)
        const float mean = (float)(first + d), rstd = sq == sq ? (float)(1.0 / sqrt(var + (double)a.eps)) : (float)sq;
        if (lane == 0) {
            stats[g - b.g0] = make_float2(mean, rstd);
            if (write && a.mean && o0 == b.index) {
                a.mean[(int64_t)s * a.G + g] = mean;
                a.rstd[(int64_t)s * a.G + g] = rstd;
            }
        }
    });
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4) k_norm_apply(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) char smem[];
    float2* stats = (float2*)(smem + Rows<T, V, 1, kStages>::kBytes);     // the block's groups, after the ring
    const uint32_t i = gridDim.x - 1 - blockIdx.x, tile = i / a.blocks;
    const Block b(a, i - tile * a.blocks, V);
    for_segments(a, tile, [&](int s, int64_t t, int64_t e) {
        const int c0 = b.channel(V);
        Rows<T, V, 1, kStages> rows = {{(const T*)a.x + (t + b.lane) * a.x_ts + c0}, {a.rl * a.x_ts},
                                       row_count(a, b, (int)(e - t)), 0, smem};
        rows.start();
        wait_for_last_launch();
        merge_stats(a, b, s, V, t == a.seqs[s].lo, stats);
        __syncthreads();
        if (rows.count) {
            float mean[V], scale[V], beta[V];       // mean: negated
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 st = stats[group_of(a, c0 + j) - b.g0];
                mean[j] = -st.x;
                scale[j] = st.y * (a.gamma ? a.gamma[c0 + j] : 1.0f);
                beta[j] = a.beta ? a.beta[c0 + j] : 0.0f;
            }
            const int64_t out_step = a.rl * a.o_ts;
            T* out = (T*)a.out + (t + b.lane) * a.o_ts + c0;
            rows.each([&](const float (&e)[1][V]) {
                float z[V];
                if constexpr (V > 1) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        add2(z[j], z[j + 1], e[0][j], e[0][j + 1], mean[j], mean[j + 1]);
                        fma2(z[j], z[j + 1], z[j], z[j + 1], scale[j], scale[j + 1], beta[j], beta[j + 1]);
                    }
                } else {
                    z[0] = fmaf(e[0][0] + mean[0], scale[0], beta[0]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = activate<T, ACT>(z[j]);
                __stcs(reinterpret_cast<typename Vec<T, V>::C*>(out), Vec<T, V>::pack(z));
                out += out_step;
            });
        }
        __syncthreads();    // stats are read
    });
}

// ---- gradient ------------------------------------------------------------------------------------

// A thread's channel constants in one sequence: mean (negated), rstd * gamma, beta. The loops work on x - mean and
// leave the factors rstd to the sums.
template <int V>
struct Channels {
    float mean[V], scale[V], beta[V];
    __device__ __forceinline__ void load(const NormArgs& a, int s, int c0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t at = (int64_t)s * a.G + group_of(a, c0 + j);
            mean[j] = -a.mean[at];
            scale[j] = a.rstd[at] * (a.gamma ? a.gamma[c0 + j] : 1.0f);
            beta[j] = a.beta ? a.beta[c0 + j] : 0.0f;
        }
    }
};

// x - mean and dz of one row's vector: e = {x, dy}.
template <typename T, int V, int ACT>
__device__ __forceinline__ void row_grad(const Channels<V>& ch, const float (&e)[2][V], float (&xc)[V], float (&dz)[V]) {
    if constexpr (V > 1) {
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
    } else {
        xc[0] = e[0][0] + ch.mean[0];
        dz[0] = e[1][0] * activate_grad<T, ACT>(fmaf(xc[0], ch.scale[0], ch.beta[0]));
    }
}

template <typename T, int V>
__device__ __forceinline__ Rows<T, V, 2, kGradStages> grad_rows(const NormArgs& a, const Block& b, int64_t t, int n, char* ring) {
    return {{(const T*)a.x + (t + b.lane) * a.x_ts + b.channel(V), (const T*)a.dy + (t + b.lane) * a.dy_ts + b.channel(V)},
            {a.rl * a.x_ts, a.rl * a.dy_ts}, row_count(a, b, n), 0, ring};
}

// Sums of the tile's segments: per channel dz and dz * xhat, per group of the column block the same times gamma.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_norm_grad_sums(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) char smem[];
    float2* red = (float2*)smem;
    let_next_launch_start();
    const uint32_t tile = blockIdx.x / a.blocks;
    const Block b(a, blockIdx.x - tile * a.blocks, V);
    for_segments(a, tile, [&](int s, int64_t t, int64_t e) {
        const int n = (int)(e - t), row_c = red_row(a, V), lanes = min(a.rl, n);
        auto rows = grad_rows<T, V>(a, b, t, n, smem + red_bytes(a, V));
        rows.start();
        if (rows.count) {
            Channels<V> ch;
            ch.load(a, s, b.channel(V));
            float s0[V], s1[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s0[j] = s1[j] = 0.0f;
            rows.each([&](const float (&e)[2][V]) {
                float xc[V], dz[V];
                row_grad<T, V, ACT>(ch, e, xc, dz);
                if constexpr (V > 1) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        add2(s0[j], s0[j + 1], s0[j], s0[j + 1], dz[j], dz[j + 1]);
                        fma2(s1[j], s1[j + 1], dz[j], dz[j + 1], xc[j], xc[j + 1], s1[j], s1[j + 1]);
                    }
                } else {
                    s0[0] += dz[0];
                    s1[0] = fmaf(dz[0], xc[0], s1[0]);
                }
            });
            float2* mine = red + b.lane * row_c + b.vec * V;
#pragma unroll
            for (int j = 0; j < V; ++j) mine[j] = make_float2(s0[j], s1[j]);
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
                a.chan_part[(int64_t)(tile + s) * a.C + b.c0 + c] = make_float2(s0, s1);
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
                a.group_part[((int64_t)(tile + s) * a.over + b.index - first_block(a, g, V)) * a.G + g] = make_float2(s1, s2);
        });
        __syncthreads();
    });
}

// rstd * S1 and rstd^2 * S2, negated, of the block's groups in sequence s into shared memory.
__device__ __forceinline__ void merge_sums(const NormArgs& a, const Block& b, int s, int V, float2* sums) {
    const int lane = threadIdx.x & 31;
    const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
    const int ta = (int)((uint32_t)lo / a.R), tiles = (int)((uint32_t)(hi - 1) / a.R) - ta + 1;
    for_group_warps(a, b, [&](int g) {
        const int overlaps = last_block(a, g, V) - first_block(a, g, V) + 1;
        const float2* part = a.group_part + (int64_t)(ta + s) * a.over * a.G + g;
        double s1 = 0.0, s2 = 0.0;
        for (int o = 0; o < overlaps; ++o) {
#pragma unroll 4
            for (int i = lane; i < tiles; i += 32) {
                const float2 v = part[((int64_t)i * a.over + o) * a.G];
                s1 += v.x;
                s2 += v.y;
            }
        }
        s1 = lane_sum(s1, 32);
        s2 = lane_sum(s2, 32);
        if (lane == 0) {
            const double r = a.rstd[(int64_t)s * a.G + g], f = -r / ((double)(hi - lo) * a.width);
            sums[g - b.g0] = make_float2((float)(f * s1), (float)(f * r * s2));
        }
    });
}

// The weights' gradients of 32 channels: the sums of all slots, in fp64. Slots that no segment has (a tile without
// tokens of the sequence) are skipped: slot i belongs to sequence s where i - s is one of its tiles.
__device__ __forceinline__ void merge_weights(const NormArgs& a, int c0, double2* red) {
    const int c = c0 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    double2 acc = make_double2(0.0, 0.0);
    if (c < a.C) {
        for (int s = 0; s < a.B; ++s) {
            const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
            if (hi <= lo) continue;
            const int64_t from = (uint32_t)lo / a.R + s, to = (uint32_t)(hi - 1) / a.R + s;
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
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_norm_grad_apply(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) char smem[];
    float2* sums = (float2*)(smem + Rows<T, V, 2, kGradStages>::kBytes);
    const uint32_t weights = (a.C + 31) / 32;
    if (blockIdx.x < weights) {
        wait_for_last_launch();
        merge_weights(a, blockIdx.x * 32, (double2*)smem);
        return;
    }
    const uint32_t i = gridDim.x - 1 - blockIdx.x, tile = i / a.blocks;
    const Block b(a, i - tile * a.blocks, V);
    for_segments(a, tile, [&](int s, int64_t t, int64_t e) {
        auto rows = grad_rows<T, V>(a, b, t, (int)(e - t), smem);
        rows.start();
        wait_for_last_launch();
        merge_sums(a, b, s, V, sums);
        __syncthreads();
        if (rows.count) {
            const int c0 = b.channel(V);
            Channels<V> ch;
            ch.load(a, s, c0);
            float S1[V], S2[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 v = sums[group_of(a, c0 + j) - b.g0];
                S1[j] = v.x;
                S2[j] = v.y;
            }
            const int64_t out_step = a.rl * a.o_ts;
            T* out = (T*)a.out + (t + b.lane) * a.o_ts + c0;
            rows.each([&](const float (&e)[2][V]) {
                float xc[V], dz[V];
                row_grad<T, V, ACT>(ch, e, xc, dz);
                if constexpr (V > 1) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        fma2(dz[j], dz[j + 1], dz[j], dz[j + 1], ch.scale[j], ch.scale[j + 1], S1[j], S1[j + 1]);
                        fma2(dz[j], dz[j + 1], xc[j], xc[j + 1], S2[j], S2[j + 1], dz[j], dz[j + 1]);
                    }
                } else {
                    dz[0] = fmaf(dz[0], ch.scale[0], fmaf(xc[0], S2[0], S1[0]));
                }
                __stcs(reinterpret_cast<typename Vec<T, V>::C*>(out), Vec<T, V>::pack(dz));
                out += out_step;
            });
        }
        __syncthreads();
    });
}

// ---- host --------------------------------------------------------------------------------------

template <void (*K)(NormArgs)>
using Kernel = std::integral_constant<void (*)(NormArgs), K>;

struct Launch {
    bool grad;
    int act, V, device;
    cudaStream_t st;
};

template <typename T, int V, int ACT>
bool launch_act(const NormArgs& a, const Launch& l) {
    const unsigned grid = a.tiles * (unsigned)a.blocks;
    const size_t red = red_bytes(a, V), groups = sizeof(float2) * std::min(a.G, a.nv * V);    // at most 16 KB each
    auto go = [&](auto tag, unsigned ctas, size_t smem, bool second) {
        constexpr auto kernel = decltype(tag)::value;
        if (!allow_smem<kernel>(l.device)) return false;
        cudaLaunchAttribute early = {};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t config = {};
        config.gridDim = dim3(ctas);
        config.blockDim = dim3(kThreads);
        config.dynamicSmemBytes = smem;
        config.stream = l.st;
        config.attrs = &early;
        config.numAttrs = second ? 1 : 0;
        note_launch();
        return cudaLaunchKernelEx(&config, kernel, a) == cudaSuccess;
    };
    if (l.grad) {
        const size_t ring = Rows<T, V, 2, kGradStages>::kBytes;
        return go(Kernel<k_norm_grad_sums<T, V, ACT>>(), grid, red + ring, false) &&
               go(Kernel<k_norm_grad_apply<T, V, ACT>>(), grid + (unsigned)cdiv(a.C, 32), std::max(ring + groups, sizeof(double2) * kThreads), true);
    }
    const size_t ring = Rows<T, V, 1, kStages>::kBytes;
    return go(Kernel<k_norm_stats<T, V>>(), grid, red + ring, false) && go(Kernel<k_norm_apply<T, V, ACT>>(), grid, ring + groups, true);
}

template <typename T, int V>
bool launch_vec(const NormArgs& a, const Launch& l) {
    if (l.act == SSA_ACT_SILU) return launch_act<T, V, SSA_ACT_SILU>(a, l);
    if (l.act == SSA_ACT_GELU) return launch_act<T, V, SSA_ACT_GELU>(a, l);
    return launch_act<T, V, SSA_ACT_NONE>(a, l);
}

template <typename T>
bool launch_type(const NormArgs& a, const Launch& l) {
    if constexpr (sizeof(T) == 2) {
        if (l.V == 8) return launch_vec<T, 8>(a, l);
    }
    if (l.V == 4) return launch_vec<T, 4>(a, l);
    if (l.V == 2) return launch_vec<T, 2>(a, l);
    return launch_vec<T, 1>(a, l);
}

// Column blocks and tiles of a call.
void shape(NormArgs& a, int V, size_t es, int ctas) {
    a.nvt = a.C / V;
    // vectors per block: at least kBlockBytes of a row, the narrowest that keeps nine tenths of the threads on vectors
    const int least = std::min<int>(a.nvt, std::max<int>(1, kBlockBytes / (V * (int)es)));
    int best = -1;
    for (int n = least; n <= std::min(a.nvt, std::max(least, 4 * least)) && n <= kThreads; ++n) {
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
    // tokens per tile, a multiple of the row lanes: kRowsPerThread a thread, less where that leaves SMs without CTAs
    const int64_t even = cdiv(a.N, std::max<int64_t>(1, ctas / a.blocks));
    a.R = (uint32_t)(a.rl * std::min<int64_t>(kRowsPerThread, cdiv(even, a.rl)));
    a.tiles = (uint32_t)cdiv(a.N, a.R);
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
    const int64_t N = p->N;
    const size_t es = dt == SSA_F32 ? 4 : 2;
    auto view = [](const ssa_rows_t* r) { return ssa_heads_t{r->data, r->token_stride, 0, 1}; };
    const ssa_heads_t x = view(c.x), out = view(c.out), dy = grad ? view(c.dy) : x;
    if (!check_view(&x, N, C, es, false) || !check_view(&out, N, C, es, true) || !check_view(&dy, N, C, es, false))
        return SSA_ERR_INVALID_ARG;
    for (const ssa_heads_t* in : {&x, &dy})
        if (!same_view(out, *in, N) && !disjoint(out, *in, N, C, es)) return SSA_ERR_INVALID_ARG;

    int V = dt == SSA_F32 ? 4 : 8;
    while (V > 1 && C % V) V >>= 1;
    V = view_vector(x, N, es, V);
    V = view_vector(dy, N, es, V);
    V = view_vector(out, N, es, V);
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
    shape(a, V, es, (grad ? 2 : 4) * sm_count(p->device));
    if ((int64_t)a.tiles * a.blocks >= ((int64_t)1 << 30)) return SSA_ERR_UNSUPPORTED;
    // one buffer of the tiles' sums
    const int64_t slots = (int64_t)a.tiles + p->B, n_group = slots * a.over * G, n_chan = grad ? slots * C : 0;
    a.group_part = (float2*)p->alloc(sizeof(float2) * (size_t)(n_group + n_chan), st, p->alloc_ctx);
    if (!a.group_part) return SSA_ERR_ALLOC;
    a.chan_part = a.group_part + n_group;
    a.mean = c.mean;
    a.rstd = c.rstd;
    const Launch l = {grad, act, V, p->device, st};
    const bool ok = dt == SSA_F32    ? launch_type<float>(a, l)
                    : dt == SSA_BF16 ? launch_type<__nv_bfloat16>(a, l)
                                     : launch_type<__half>(a, l);
    p->release(a.group_part, st, p->alloc_ctx);
    return ok && cudaGetLastError() == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
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
