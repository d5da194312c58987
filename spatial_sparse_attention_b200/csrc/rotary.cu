// ssa_rotary and ssa_rotary_backward: RMS normalisation of queries and keys over the head dimension and
// rotary positions at the voxel coordinates, as operators of their own with gradients (Hi3D v1.0
// pipeline page, "Stage 3: sparse flow sampling").
//
// Per (token, head) row x, with n = x * inv, inv = rsqrt(mean x^2 + eps) and u = n * gamma:
//   (a, b) -> (a c - b s, a s + b c) * mscale   for every rotated pair (a, b) of u.
// The gradient turns back, du = R^T dy, and then dx = inv * (g - n * mean(g n)) with g = du * gamma, and
// dgamma = sum over rows of du * n.
//
// Bound: HBM. A row moves 2 (gradient with weights: 3) times head_dim elements for some 10 operations
// each. A lane keeps 32 bytes of a row (two 16-byte loads), two to sixteen lanes make a row. The loads of a
// lane's next rows are always in flight: they go to the lane's own places in shared memory (no barrier, no
// registers), several rows ahead. The cosines and sines are shared by all heads of a token: a CTA takes a
// tile of tokens, queries and keys, and computes them once into shared memory while its first loads fly.
// Measured (fp16, 44 heads x 96): 110,000 tokens 303 us, 6.1 TB/s; the gradient with weights of 80,000 tokens
// 350 us, 5.8 TB/s; a plain copy reaches 6.55. What is next to memory is instruction issue.
#include <algorithm>
#include <cmath>

#include "views.cuh"

namespace ssa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = 32;      // tokens per CTA tile, at most one per lane
constexpr int kMaxPairs = 64;     // head_dim <= 128
constexpr int kLane = 32;         // bytes of a row per lane
constexpr int kStages = 3;        // rows per lane in flight or in use, forward
constexpr int kStagedBelow = 2;   // half layout: loads of at most this many elements are staged
constexpr int kGradStages = 3;    // gradient (two rows each)
// Rows that a lane adds up in fp32 before the sums go on in fp64. Gradient of 80,000 tokens x 44 heads x 96 fp16: 342 us without,
// 345 every 128 rows, 350 every 32; the sums of equal terms, whose roundings point one way, are off by up to 30 and 8 units of 2^-24.
constexpr int kChain = 32;

struct RowsArg {
    const void* x;        // forward: input; gradient: the forward's input (weights) or unused
    const void* g;        // gradient: gradient of the output
    void* out;
    const float* gamma;
    double* part;         // gradient with weights: [CTAs of this tensor][D] partial sums
    int64_t x_ts, x_hs, g_ts, g_hs, o_ts, o_hs;
    int32_t H;
    int32_t tile;         // gradient: tokens per tile
};

// Frequencies as fractions of a turn in units of 2^-64: coordinate * turns wraps modulo one turn by
// itself, so the angle is reduced exactly at any coordinate.
struct RotArgs {
    RowsArg t[2];                  // queries, keys
    const int32_t* coords;
    int64_t N;
    int32_t D, G;                  // head dimension; lanes per row
    int32_t pairs;                 // rotated pairs
    int32_t tile;                  // tokens per tile (gradient: the larger of the two)
    int32_t device;                // host side
    int32_t ctas0;                 // gradient: CTAs [0, ctas0) work on t[0], the rest on t[1]
    float eps, inv_d, mscale, sgn; // inv_d = 1/D; sgn = -1 turns back
    uint64_t turns[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

// How a lane's 32 bytes of a row are cut. An item is P pairs: one load of V = 2P elements (interleaved,
// V >= 2), or two loads of V elements (half: the pairs' two sides; interleaved at V = 1). Item m of lane l
// is item m*G + l of the row, so neighbouring lanes read neighbouring items. In registers an item is its P
// first sides, then its P second sides, in both layouts.
template <typename T, int V_, bool HALF_>
struct Cut {
    static constexpr int V = V_;
    static constexpr bool HALF = HALF_;
    static constexpr int E = kLane / (int)sizeof(T);       // elements per lane
    static constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);
    static constexpr int M = E / (2 * P);                   // items per lane
    static constexpr int L = 2 * P / V;                     // loads per item
    static constexpr int N = M * L;                         // loads per lane
    static constexpr bool MIXED = !HALF && V > 2;           // sides alternate inside a load
    using C = typename Chunk<V * (int)sizeof(T)>::type;
    // register of element j of load i
    static __host__ __device__ constexpr int reg(int i, int j) {
        return MIXED ? i * V + (j & 1) * P + j / 2 : i * V + j;
    }
};

// Place of pair p in a token's table row: pairs that one lane reads as two float4 are kept four apart by
// the row's items, so that a warp's 16-byte reads are contiguous.
template <int P>
__device__ __forceinline__ int tab_pos(int p, int items) {
    if (P == 8) return (((p >> 2) & 1) * items + (p >> 3)) * 4 + (p & 3);
    return p;
}

// cos and sin of coordinate * turns (2^-64 of a turn), by quadrant plus a remainder of at most an
// eighth of a turn, which fp32 holds to 2^-28 of a turn. There x <= pi/4, and the Taylor series end with
// x^9 / 9! and x^10 / 10!: the next terms are below 2^-29 and 2^-32.
__device__ __forceinline__ void turn_cos_sin(int32_t coord, uint64_t turns, float& c, float& s) {
    const int32_t hi = (int32_t)(((uint64_t)(uint32_t)coord * turns) >> 32);   // signed, 2^-32 of a turn
    const int32_t q = (int32_t)((uint32_t)hi + 0x20000000u) >> 30;
    const float x = (float)(int32_t)((uint32_t)hi - ((uint32_t)q << 30)) * (0x1p-31f * 3.14159265358979f);
    const float y = x * x;
    const float ps = fmaf(fmaf(fmaf(y, 1.0f / 362880, -1.0f / 5040), y, 1.0f / 120), y, -1.0f / 6);
    const float pc = fmaf(fmaf(fmaf(fmaf(y, -1.0f / 3628800, 1.0f / 40320), y, -1.0f / 720), y, 1.0f / 24), y, -0.5f);
    const float s0 = fmaf(x * y, ps, x), c0 = fmaf(y, pc, 1.0f);
    c = (q & 1) ? s0 : c0;
    s = (q & 1) ? c0 : s0;
    if ((q & 3) == 1 || (q & 3) == 2) c = -c;
    if (q & 2) s = -s;
}

// Bytes of the rows that a CTA has in one stage. Staged rows are 16 bytes apart, so that the same element of a warp's
// rows (of up to 16) lies in different banks.
constexpr int kRowPad = 16;
__host__ __device__ constexpr int stage_bytes(bool staged) { return kThreads * kLane + (staged ? kWarps * 16 * kRowPad : 0); }

// A lane group's row in flight. Direct: a lane's loads lie in places of its own, neighbouring lanes side by side.
// STAGED (the half layout where the two sides of the pairs do not start at a vector): the row lies in its natural
// order, fetched and stored in 16-byte chunks, and the lanes pick their pairs' elements out of it and put them back.
template <typename T, typename CUT, bool STAGED>
struct Slot {
    using C = typename CUT::C;
    char* at;       // direct: this lane's first chunk; staged: the row
    int l, G;
    __device__ __forceinline__ Slot(char* ring, int stage, int sub, int l_, int G_) : l(l_), G(G_) {
        char* const base = ring + stage * stage_bytes(STAGED);
        at = STAGED ? base + (threadIdx.x >> 5) * (stage_bytes(true) / kWarps) + sub * (G * kLane + kRowPad)
                    : base + threadIdx.x * sizeof(C);
    }
    __device__ __forceinline__ C* place(int i) const { return (C*)(at + i * (kThreads * sizeof(C))); }
    __device__ __forceinline__ int chunk(int i) const { return (i * G + l) * 16; }
    __device__ __forceinline__ void fetch(const T* row, const int (&off)[CUT::N]) const {
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < kLane / 16; ++i) cp_async<16>(at + chunk(i), (const char*)row + chunk(i));
        } else {
#pragma unroll
            for (int i = 0; i < CUT::N; ++i) cp_async<sizeof(C)>(place(i), row + off[i]);
        }
    }
    // after the copies have landed (staged: and a __syncwarp)
    __device__ __forceinline__ void read(const int (&off)[CUT::N], float (&e)[CUT::E]) const {
#pragma unroll
        for (int i = 0; i < CUT::N; ++i) {
            float v[CUT::V];
            if constexpr (STAGED) v[0] = Elem<T>::to_f(((const T*)at)[off[i]]);
            else Vec<T, CUT::V>::unpack(*place(i), v);
#pragma unroll
            for (int j = 0; j < CUT::V; ++j) e[CUT::reg(i, j)] = v[j];
        }
    }
    // staged: the lane's elements back into the row; then, after a __syncwarp, `write` stores the row
    __device__ __forceinline__ void put_back(const int (&off)[CUT::N], const float (&e)[CUT::E]) const {
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < CUT::N; ++i) ((T*)at)[off[i]] = Elem<T>::from_f(e[i]);
        }
    }
    __device__ __forceinline__ void write(T* row, const int (&off)[CUT::N], const float (&e)[CUT::E]) const {
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < kLane / 16; ++i) *(uint4*)((char*)row + chunk(i)) = *(const uint4*)(at + chunk(i));
        } else {
#pragma unroll
            for (int i = 0; i < CUT::N; ++i) {
                float v[CUT::V];
#pragma unroll
                for (int j = 0; j < CUT::V; ++j) v[j] = e[CUT::reg(i, j)];
                *reinterpret_cast<C*>(row + off[i]) = Vec<T, CUT::V>::pack(v);
            }
        }
    }
};

// A lane's weights, from a table in register order: item `it` at it * 2P.
template <typename CUT>
__device__ __forceinline__ void read_gamma(const float* gamma, int l, int G, float (&g)[CUT::E]) {
    constexpr int W = 2 * CUT::P;
#pragma unroll
    for (int m = 0; m < CUT::M; ++m) {
        const float* at = gamma + (m * G + l) * W;
        if constexpr (W >= 4) {
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(at + j);
                g[m * W + j] = v.x; g[m * W + j + 1] = v.y; g[m * W + j + 2] = v.z; g[m * W + j + 3] = v.w;
            }
        } else {
            const float2 v = *reinterpret_cast<const float2*>(at);
            g[m * W] = v.x;
            g[m * W + 1] = v.y;
        }
    }
}

// Sum over the G lanes of a row (G = 2, 4, 6, 8, 12, 16; its first lane is `base`); all lanes of the warp
// call it. At G = 6 and 12 the lanes add the last three partial sums in orders of their own.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int G, int base, int l) {
    auto from = [&](int n) { return base + (l + n < G ? l + n : l + n - G); };
    auto add = [&](int src) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_sync(0xffffffffu, v[k], src);
    };
    if (G % 3 == 0) {
        if (G == 12) add(from(6));
        add(from(3));
        const int s1 = from(1), s2 = from(2);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float b = __shfl_sync(0xffffffffu, v[k], s1), c = __shfl_sync(0xffffffffu, v[k], s2);
            v[k] += b + c;
        }
    } else {
        if (G >= 16) add(from(8));
        if (G >= 8) add(from(4));
        if (G >= 4) add(from(2));
        add(from(1));
    }
}

// Turn the pairs of a lane's elements; cs, sn are the token's table rows. Channels that pass through are
// left as they are, whatever their neighbours hold.
template <typename CUT>
__device__ __forceinline__ void turn_row(float (&e)[CUT::E], const float* cs, const float* sn, int l, int G, int pairs) {
    constexpr int P = CUT::P;
#pragma unroll
    for (int m = 0; m < CUT::M; ++m) {
        const int it = m * G + l;
        const int turned = pairs - it * P;     // of the item's pairs
        if (turned <= 0) continue;
        float c[P], s[P];
        if constexpr (P >= 4) {
#pragma unroll
            for (int q = 0; q < P / 4; ++q) {
                const int at = tab_pos<P>(it * P + 4 * q, G * CUT::M);
                const float4 c4 = *reinterpret_cast<const float4*>(cs + at);
                const float4 s4 = *reinterpret_cast<const float4*>(sn + at);
                c[4 * q] = c4.x; c[4 * q + 1] = c4.y; c[4 * q + 2] = c4.z; c[4 * q + 3] = c4.w;
                s[4 * q] = s4.x; s[4 * q + 1] = s4.y; s[4 * q + 2] = s4.z; s[4 * q + 3] = s4.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                c[i] = cs[it * P + i];
                s[i] = sn[it * P + i];
            }
        }
        float* a = e + m * 2 * P;
        float* b = a + P;
        // in the half layout 2P divides the rotated width: an item is turned as a whole or not
        if (CUT::HALF || P == 1 || turned >= P) {
            if constexpr (P >= 2) {
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    float x0, x1, y0, y1;
                    mul2(x0, x1, b[i], b[i + 1], -s[i], -s[i + 1]);
                    mul2(y0, y1, b[i], b[i + 1], c[i], c[i + 1]);
                    fma2(b[i], b[i + 1], a[i], a[i + 1], s[i], s[i + 1], y0, y1);
                    fma2(a[i], a[i + 1], a[i], a[i + 1], c[i], c[i + 1], x0, x1);
                }
            } else {
                const float u = a[0], v = b[0];
                a[0] = u * c[0] - v * s[0];
                b[0] = u * s[0] + v * c[0];
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (i < turned) {
                    const float u = a[i], v = b[i];
                    a[i] = u * c[i] - v * s[i];
                    b[i] = u * s[i] + v * c[i];
                }
            }
        }
    }
}

// Floats per token in a table.
__host__ __device__ constexpr int tab_stride(int D) { return D / 2 + 4; }

// The tokens' cosines and sines, for ntok <= 32 tokens from tok0: a lane takes a token, a warp a pair.
template <int P>
__device__ __forceinline__ void fill_tables(const RotArgs& a, int64_t tok0, int ntok, float* cs, float* sn) {
    const int t = threadIdx.x & 31;
    if (t >= ntok) return;
    const int32_t* xyz = a.coords + 3 * (tok0 + t);
    const int32_t x = xyz[0], y = xyz[1], z = xyz[2];
    const int row = t * tab_stride(a.D), items = a.D / (2 * P);
    for (int p = threadIdx.x >> 5; p < a.pairs; p += kWarps) {
        float c, s;
        turn_cos_sin(a.axis[p] == 0 ? x : a.axis[p] == 1 ? y : z, a.turns[p], c, s);
        const int at = row + tab_pos<P>(p, items);
        cs[at] = c * a.mscale;
        sn[at] = s * (a.mscale * a.sgn);
    }
}

// First channel of load i of lane l. In the half layout a load holds one side of its item's pairs.
template <typename T, int V, bool HALF>
__device__ __forceinline__ int load_offset(const RotArgs& a, int G, int l, int i) {
    using CUT = Cut<T, V, HALF>;
    const int side = i % CUT::L, p = (i / CUT::L * G + l) * CUT::P;   // the item's first pair
    // 2P divides the rotated width: an item is turned as a whole or not
    if (HALF && p < a.pairs) return side * a.pairs + p;
    return 2 * p + side * CUT::P;
}

// Channel of register e (0..E-1) of lane l.
template <typename T, int V, bool HALF>
__device__ __forceinline__ int lane_channel(const RotArgs& a, int G, int l, int e) {
    using CUT = Cut<T, V, HALF>;
    const int i = e / V, j = e % V;     // a load's registers are its own, in the order of CUT::reg
    return load_offset<T, V, HALF>(a, G, l, i) + (CUT::MIXED ? (j % CUT::P) * 2 + j / CUT::P : j);
}

// The weights in register order (read_gamma).
template <typename T, int V, bool HALF>
__device__ __forceinline__ void fill_gamma(const RotArgs& a, const float* gamma, float* table) {
    using CUT = Cut<T, V, HALF>;
    for (int i = threadIdx.x; i < a.D; i += kThreads) {
        const int it = i / (2 * CUT::P), l = it % a.G, e = it / a.G * 2 * CUT::P + i % (2 * CUT::P);
        table[i] = gamma[lane_channel<T, V, HALF>(a, a.G, l, e)];
    }
}

template <typename T, int V, bool HALF>
__device__ __forceinline__ void lane_offsets(const RotArgs& a, int G, int l, int (&off)[Cut<T, V, HALF>::N]) {
#pragma unroll
    for (int i = 0; i < Cut<T, V, HALF>::N; ++i) off[i] = load_offset<T, V, HALF>(a, G, l, i);
}

// A lane group's place in the rows of a tile: row r is head h of token t.
struct Cursor {
    int r, t, h;
    __device__ __forceinline__ void advance(int step, int dt, int dh, int H) {
        r += step;
        t += dt;
        h += dh;
        if (h >= H) {
            h -= H;
            ++t;
        }
    }
};

// out = rotate(normalise(x)), or the rotation back (sgn = -1, no weights). One tile of tokens per CTA, the
// queries' heads then the keys'; warps take row after row.
template <typename T, int V, bool HALF, bool NORM, int LANES, bool STAGED>
__global__ void __launch_bounds__(kThreads, 4) k_rotary(const __grid_constant__ RotArgs a) {
    using CUT = Cut<T, V, HALF>;
    constexpr int E = CUT::E;
    extern __shared__ __align__(16) char smem[];    // ring, tables, weights
    float* cs = (float*)(smem + kStages * stage_bytes(STAGED));
    float* sn = cs + a.tile * tab_stride(a.D);
    float* gamma = sn + a.tile * tab_stride(a.D);
    const int64_t tok0 = (int64_t)blockIdx.x * a.tile;
    const int ntok = (int)min((int64_t)a.tile, a.N - tok0);

    const int lane = threadIdx.x & 31, G = LANES ? LANES : a.G, rpw = 32 / G;
    const int sub = lane / G, l = lane - sub * G, base = lane - l;
    int off[CUT::N];
    lane_offsets<T, V, HALF>(a, G, l, off);
    const int H0 = a.t[0].H, H = H0 + a.t[1].H;
    const int nrow = ntok * H, step = kWarps * rpw, dt = step / H, dh = step - dt * H;
    const int r0 = (threadIdx.x >> 5) * rpw;
    Cursor at = {r0 + sub, (r0 + sub) / H, (r0 + sub) % H};
    if (sub >= rpw) at.r = nrow;    // lanes beyond the last whole row of the warp
    Cursor ahead = at;
    auto fetch = [&](int stage) {
        if (ahead.r < nrow) {
            const bool second = ahead.h >= H0;
            const RowsArg& t = a.t[second];
            Slot<T, CUT, STAGED>(smem, stage, sub, l, G)
                .fetch((const T*)t.x + (tok0 + ahead.t) * t.x_ts + (ahead.h - (second ? H0 : 0)) * t.x_hs, off);
        }
        cp_commit();
        ahead.advance(step, dt, dh, H);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    if constexpr (NORM) {
        fill_gamma<T, V, HALF>(a, a.t[0].gamma, gamma);
        if (a.t[1].H) fill_gamma<T, V, HALF>(a, a.t[1].gamma, gamma + a.D);
    }
    fill_tables<CUT::P>(a, tok0, ntok, cs, sn);
    __syncthreads();

    int stage = 0;
    for (int w0 = r0; w0 < nrow; w0 += step) {
        fetch((stage + kStages - 1) % kStages);
        cp_wait<kStages - 1>();
        const bool mine = at.r < nrow, second = at.h >= H0;
        const Slot<T, CUT, STAGED> slot(smem, stage, sub, l, G);
        float e[E];
        if (STAGED) __syncwarp();
        if (mine) slot.read(off, e);
        if constexpr (NORM) {
            float ss[1] = {0.0f}, odd = 0.0f;
            if (mine) {
#pragma unroll
                for (int i = 0; i < E; i += 2) fma2(ss[0], odd, e[i], e[i + 1], e[i], e[i + 1], ss[0], odd);
                ss[0] += odd;
            }
            row_sum(ss, G, base, l);
            const float inv = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
            if (mine) {
                float gam[E];
                read_gamma<CUT>(gamma + (second ? a.D : 0), l, G, gam);
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    mul2(e[i], e[i + 1], e[i], e[i + 1], inv, inv);
                    mul2(e[i], e[i + 1], e[i], e[i + 1], gam[i], gam[i + 1]);
                }
            }
        }
        if (mine) {
            const int tab = at.t * tab_stride(a.D);
            turn_row<CUT>(e, cs + tab, sn + tab, l, G, a.pairs);
            slot.put_back(off, e);
        }
        if (STAGED) __syncwarp();
        if (mine) {
            const RowsArg& t = a.t[second];
            slot.write((T*)t.out + (tok0 + at.t) * t.o_ts + (at.h - (second ? H0 : 0)) * t.o_hs, off, e);
        }
        at.advance(step, dt, dh, H);
        stage = (stage + 1) % kStages;
    }
}

// The gradient with weights. Persistent: a CTA walks tiles of its tensor, its loads running ahead into the
// next tile, and keeps the weights' sums of its lanes' channels in registers, from which every kChain rows they go to fp64
// sums in the lane's own places in shared memory (no barrier): a sum of millions of rows loses nothing to its length.
// The CTA adds them up over its rows in a fixed order at the end.
template <typename T, int V, bool HALF, int LANES, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) k_rotary_grad(const __grid_constant__ RotArgs a) {
    using CUT = Cut<T, V, HALF>;
    constexpr int E = CUT::E, S = kGradStages;
    extern __shared__ __align__(16) char smem[];
    char* const ring_g = smem + S * stage_bytes(STAGED);
    float* cs = (float*)(smem + 2 * S * stage_bytes(STAGED));
    float* sn = cs + a.tile * tab_stride(a.D);
    float* gamma = sn + a.tile * tab_stride(a.D);
    double* sums64 = (double*)(gamma + a.D);    // [E][kThreads]
    const int which = blockIdx.x < a.ctas0 ? 0 : 1;
    const RowsArg& t = a.t[which];
    const int cta = blockIdx.x - (which ? a.ctas0 : 0), nctas = which ? gridDim.x - a.ctas0 : a.ctas0;

    const int lane = threadIdx.x & 31, G = LANES ? LANES : a.G, rpw = 32 / G;
    const int sub = lane / G, l = lane - sub * G, base = lane - l;
    int off[CUT::N];
    lane_offsets<T, V, HALF>(a, G, l, off);
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        acc[i] = 0.0f;
        sums64[i * kThreads + threadIdx.x] = 0.0;
    }
    int chain = 0;
    auto flush = [&] {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            sums64[i * kThreads + threadIdx.x] += (double)acc[i];
            acc[i] = 0.0f;
        }
        chain = 0;
    };
    const int H = t.H, step = kWarps * rpw, dt = step / H, dh = step - dt * H;
    const int r0 = (threadIdx.x >> 5) * rpw;
    const Cursor first = {r0 + sub, (r0 + sub) / H, (r0 + sub) % H};
    const int64_t stride = (int64_t)nctas * t.tile;
    // what is fetched next: row `ahead` of the tile at `ftok`, in steps of the whole CTA
    int64_t ftok = (int64_t)cta * t.tile;
    int frow = 0, fbase = 0;
    Cursor ahead = first;
    auto fetch = [&](int stage) {
        if (ftok < a.N) {
            if (fbase == 0) frow = (int)min((int64_t)t.tile, a.N - ftok) * H;
            if (ahead.r < frow && sub < rpw) {
                Slot<T, CUT, STAGED>(smem, stage, sub, l, G)
                    .fetch((const T*)t.x + (ftok + ahead.t) * t.x_ts + ahead.h * t.x_hs, off);
                Slot<T, CUT, STAGED>(ring_g, stage, sub, l, G)
                    .fetch((const T*)t.g + (ftok + ahead.t) * t.g_ts + ahead.h * t.g_hs, off);
            }
            ahead.advance(step, dt, dh, H);
            fbase += step;
            if (fbase >= frow) {
                fbase = 0;
                ahead = first;
                ftok += stride;
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    fill_gamma<T, V, HALF>(a, t.gamma, gamma);
    __syncthreads();
    float gam[E];
    read_gamma<CUT>(gamma, l, G, gam);
    int stage = 0;
    for (int64_t tok0 = (int64_t)cta * t.tile; tok0 < a.N; tok0 += stride) {
        const int ntok = (int)min((int64_t)t.tile, a.N - tok0);
        __syncthreads();    // the previous tile's tables are read
        fill_tables<CUT::P>(a, tok0, ntok, cs, sn);
        __syncthreads();
        const int nrow = ntok * H;
        Cursor at = first;
        T* out = (T*)t.out + tok0 * t.o_ts;
        for (int from = 0; from < nrow; from += kChain * step) {
            const int to = min(nrow, from + kChain * step), rows = (to - from + step - 1) / step;
            if (chain + rows > kChain) flush();
            chain += rows;
            for (int w0 = from; w0 < to; w0 += step) {
                fetch((stage + S - 1) % S);
                cp_wait<S - 1>();
                const bool mine = at.r < nrow && sub < rpw;
                float e[E], d[E], sums[2] = {0.0f, 0.0f};   // sum x^2, sum du gamma x
                const Slot<T, CUT, STAGED> slot(ring_g, stage, sub, l, G);
                if (STAGED) __syncwarp();
                if (mine) {
                    Slot<T, CUT, STAGED>(smem, stage, sub, l, G).read(off, e);
                    slot.read(off, d);
                    const int tab = at.t * tab_stride(a.D);
                    turn_row<CUT>(d, cs + tab, sn + tab, l, G, a.pairs);
                    float odd0 = 0.0f, odd1 = 0.0f;
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        float g0, g1;
                        mul2(g0, g1, d[i], d[i + 1], gam[i], gam[i + 1]);
                        fma2(sums[0], odd0, e[i], e[i + 1], e[i], e[i + 1], sums[0], odd0);
                        fma2(sums[1], odd1, g0, g1, e[i], e[i + 1], sums[1], odd1);
                    }
                    sums[0] += odd0;
                    sums[1] += odd1;
                }
                row_sum(sums, G, base, l);
                if (mine) {
                    const float inv = rsqrtf(fmaf(sums[0], a.inv_d, a.eps));
                    const float dot = -sums[1] * inv * a.inv_d;      // - mean of g n
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        float n0, n1;
                        mul2(n0, n1, e[i], e[i + 1], inv, inv);
                        fma2(acc[i], acc[i + 1], d[i], d[i + 1], n0, n1, acc[i], acc[i + 1]);
                        mul2(d[i], d[i + 1], d[i], d[i + 1], gam[i], gam[i + 1]);
                        fma2(d[i], d[i + 1], n0, n1, dot, dot, d[i], d[i + 1]);
                        mul2(d[i], d[i + 1], d[i], d[i + 1], inv, inv);
                    }
                    slot.put_back(off, d);
                }
                if (STAGED) __syncwarp();
                if (mine) slot.write(out + at.t * t.o_ts + at.h * t.o_hs, off, d);
                at.advance(step, dt, dh, H);
                stage = (stage + 1) % S;
            }
        }
    }
    // one thread per element adds the sums of all warps and rows
    flush();
    __syncthreads();
    if (threadIdx.x < a.D) {    // D = G * E
        const int i = threadIdx.x / G, ll = threadIdx.x - i * G;   // element i of lane ll
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w)
            for (int q = 0; q < rpw; ++q) s += sums64[i * kThreads + w * 32 + q * G + ll];
        t.part[(int64_t)cta * a.D + lane_channel<T, V, HALF>(a, G, ll, i)] = s;
    }
}

// dgamma[c] = sum over CTAs of part[cta][c], 32 channels per CTA, in a fixed order.
__global__ void __launch_bounds__(1024) k_rotary_dgamma(const double* __restrict__ part0, const double* __restrict__ part1,
                                                        int n0, int n1, int D, float* out0, float* out1) {
    __shared__ double red[32][33];
    const double* part = blockIdx.y ? part1 : part0;
    const int n = blockIdx.y ? n1 : n0, c = blockIdx.x * 32 + threadIdx.x;
    double s = 0.0;
    for (int i = threadIdx.y; i < n; i += 32) s += part[(int64_t)i * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        s = 0.0;
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
        (blockIdx.y ? out1 : out0)[c] = (float)s;
    }
}

// ---- host --------------------------------------------------------------------------------------

ssa_status_t check_rotary(const ssa_rotary_t* r, int32_t D) {
    if (!r) return SSA_ERR_INVALID_ARG;
    if (D != 32 && D != 64 && D != 96 && D != 128) return SSA_ERR_UNSUPPORTED;
    if (!(r->theta > 1.0) || !std::isfinite(r->theta) || !(r->mscale > 0.0f) || !std::isfinite(r->mscale))
        return SSA_ERR_INVALID_ARG;
    if (r->dim < 0 || r->dim > D || (r->dim & 1)) return SSA_ERR_INVALID_ARG;
    if (r->layout != SSA_ROTARY_INTERLEAVED && r->layout != SSA_ROTARY_HALF) return SSA_ERR_INVALID_ARG;
    if (r->scaling < SSA_ROTARY_SCALE_NONE || r->scaling > SSA_ROTARY_SCALE_YARN) return SSA_ERR_INVALID_ARG;
    if (r->scaling != SSA_ROTARY_SCALE_NONE && (!(r->scale > 0.0) || !std::isfinite(r->scale)))
        return SSA_ERR_INVALID_ARG;
    if (r->scaling == SSA_ROTARY_SCALE_YARN &&
        (!(r->extent > 0.0) || !std::isfinite(r->extent) || !(r->beta_slow >= 0.0) ||
         !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast)))
        return SSA_ERR_INVALID_ARG;
    return SSA_OK;
}

// Axis and angular frequency of the rotated pairs (the formulas of ssa_rotary_t); returns their count.
int rotary_frequencies(const ssa_rotary_t& r, int32_t D, int32_t* axis, double* freq) {
    const int R = r.dim ? r.dim : D, c = 2 * (R / 6);
    const int width[3] = {R - 2 * c, c, c};
    const double two_pi = 6.28318530717958647692;
    int p = 0;
    for (int a = 0; a < 3; ++a) {
        const int w = width[a];
        for (int j = 0; j < w / 2; ++j, ++p) {
            axis[p] = a;
            if (a && w == width[a - 1]) {   // the same frequencies as the axis before
                freq[p] = freq[p - w / 2];
                continue;
            }
            double f = std::pow(r.theta, -2.0 * j / w);
            if (r.scaling == SSA_ROTARY_SCALE_LINEAR) {
                f /= r.scale;
            } else if (r.scaling == SSA_ROTARY_SCALE_NTK && w > 2) {
                f = std::pow(r.theta * std::pow(r.scale, w / (w - 2.0)), -2.0 * j / w);
            } else if (r.scaling == SSA_ROTARY_SCALE_YARN) {
                double g = (r.extent * f / two_pi - r.beta_slow) / (r.beta_fast - r.beta_slow);
                g = std::min(1.0, std::max(0.0, g));
                f *= g + (1.0 - g) / r.scale;
            }
            freq[p] = f;
        }
    }
    return p;
}

template <void (*KERNEL)(RotArgs)>
bool launch_one(const RotArgs& a, unsigned grid, size_t smem, cudaStream_t st) {
    if (!allow_smem<KERNEL>(a.device)) return false;
    KERNEL<<<grid, kThreads, smem, st>>>(a);
    return true;
}

template <typename T, int V, bool HALF, int LANES, bool STAGED>
bool launch_lanes(const RotArgs& a, unsigned grid, bool grad, cudaStream_t st) {
    const size_t ring = stage_bytes(STAGED), tables = sizeof(float) * 2 * ((size_t)a.tile * tab_stride(a.D) + a.D);
    const size_t sums64 = sizeof(double) * Cut<T, V, HALF>::E * kThreads;
    if (grad) return launch_one<k_rotary_grad<T, V, HALF, LANES, STAGED>>(a, grid, 2 * kGradStages * ring + tables + sums64, st);
    if (a.t[0].gamma) return launch_one<k_rotary<T, V, HALF, true, LANES, STAGED>>(a, grid, kStages * ring + tables, st);
    return launch_one<k_rotary<T, V, HALF, false, LANES, STAGED>>(a, grid, kStages * ring + tables, st);
}

// Full vectors (half layout: halves of one too) with the lanes per row known at compile time (a shuffle tree and offsets without branches: 350
// against 437 us for the gradient of 80,000 tokens x 44 heads x 96); rows aligned to less with them at run time.
template <typename T, int V, bool HALF, bool STAGED>
bool launch_cut(const RotArgs& a, unsigned grid, bool grad, cudaStream_t st) {
    constexpr int D32 = 32 * (int)sizeof(T) / kLane;    // lanes of 32 channels
    if constexpr (STAGED || V * sizeof(T) == 16 || (HALF && V * sizeof(T) == 8)) {
        if (a.D == 32) return launch_lanes<T, V, HALF, D32, STAGED>(a, grid, grad, st);
        if (a.D == 64) return launch_lanes<T, V, HALF, 2 * D32, STAGED>(a, grid, grad, st);
        if (a.D == 96) return launch_lanes<T, V, HALF, 3 * D32, STAGED>(a, grid, grad, st);
        return launch_lanes<T, V, HALF, 4 * D32, STAGED>(a, grid, grad, st);
    } else {
        return launch_lanes<T, V, HALF, 0, STAGED>(a, grid, grad, st);
    }
}

template <typename T, int V>
bool launch_layout(const RotArgs& a, unsigned grid, bool half, bool grad, cudaStream_t st) {
    note_launch();
    return half ? launch_cut<T, V, true, false>(a, grid, grad, st) : launch_cut<T, V, false, false>(a, grid, grad, st);
}

// V: elements per load; 0: staged.
bool launch_rows(const RotArgs& a, unsigned grid, ssa_dtype_t dt, int V, bool half, bool grad, cudaStream_t st) {
    if (V == 0) {
        note_launch();
        if (dt == SSA_F32) return launch_cut<float, 1, true, true>(a, grid, grad, st);
        if (dt == SSA_BF16) return launch_cut<__nv_bfloat16, 1, true, true>(a, grid, grad, st);
        return launch_cut<__half, 1, true, true>(a, grid, grad, st);
    }
    if (dt == SSA_F32) {
        if (V >= 4) return launch_layout<float, 4>(a, grid, half, grad, st);
        if (V == 2) return launch_layout<float, 2>(a, grid, half, grad, st);
        return launch_layout<float, 1>(a, grid, half, grad, st);
    }
    auto pick = [&](auto tag) {
        using T = decltype(tag);
        if (V >= 8) return launch_layout<T, 8>(a, grid, half, grad, st);
        if (V == 4) return launch_layout<T, 4>(a, grid, half, grad, st);
        if (V == 2) return launch_layout<T, 2>(a, grid, half, grad, st);
        return launch_layout<T, 1>(a, grid, half, grad, st);
    };
    return dt == SSA_BF16 ? pick(__nv_bfloat16()) : pick(__half());
}

struct Call {
    const ssa_heads_t* x[2];    // forward inputs (null in a gradient without weights)
    const ssa_heads_t* g[2];    // gradients of the outputs (null in the forward)
    const ssa_heads_t* out[2];
    const float* gamma[2];
    float* dgamma[2];
};

ssa_status_t run_rotary(Plan* p, const Call& c, float eps, const ssa_rotary_t* rot, int32_t D, ssa_dtype_t dt,
                        bool backward, cudaStream_t st) {
    if (!p || p->owned.empty()) return SSA_ERR_INVALID_ARG;
    const ssa_status_t rc = check_rotary(rot, D);
    if (rc != SSA_OK) return rc;
    if (dt != SSA_F32 && dt != SSA_BF16 && dt != SSA_F16) return SSA_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return SSA_ERR_INVALID_ARG;
    if (!aligned4(c.gamma[0], c.gamma[1], c.dgamma[0], c.dgamma[1])) return SSA_ERR_INVALID_ARG;
    const int64_t N = p->N;
    const size_t es = dt == SSA_F32 ? 4 : 2;
    const int nt = c.out[1] ? 2 : 1;
    const bool norm = c.gamma[0] != nullptr;
    const ssa_heads_t* in[4] = {};     // what each tensor reads, x and g
    for (int i = 0; i < nt; ++i) {
        if (norm != (c.gamma[i] != nullptr)) return SSA_ERR_INVALID_ARG;
        in[2 * i] = (!backward || norm) ? c.x[i] : nullptr;
        in[2 * i + 1] = backward ? c.g[i] : nullptr;
        if ((!backward || norm) && !check_view(c.x[i], N, D, es, false)) return SSA_ERR_INVALID_ARG;
        if (backward && !check_view(c.g[i], N, D, es, false)) return SSA_ERR_INVALID_ARG;
        if (!check_view(c.out[i], N, D, es, true)) return SSA_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j)
            if (in[2 * i + j] && in[2 * i + j]->heads != c.out[i]->heads) return SSA_ERR_INVALID_ARG;
        if (backward && norm && !c.dgamma[i]) return SSA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < nt; ++i)
        for (int j = 0; j < 2 * nt; ++j)
            if (in[j] && !(j / 2 == i && same_view(*c.out[i], *in[j], N)) && !disjoint(*c.out[i], *in[j], N, D, es))
                return SSA_ERR_INVALID_ARG;
    if (nt == 2 && !disjoint(*c.out[0], *c.out[1], N, D, es)) return SSA_ERR_INVALID_ARG;
    if (nt == 2 && !apart({c.dgamma[0], D}, {c.dgamma[1], D})) return SSA_ERR_INVALID_ARG;

    RotArgs a = {};
    int32_t axis[kMaxPairs];
    double freq[kMaxPairs];
    a.pairs = rotary_frequencies(*rot, D, axis, freq);
    for (int i = 0; i < a.pairs; ++i) {
        if (!std::isfinite(freq[i])) return SSA_ERR_INVALID_ARG;
        const long double turn = (long double)freq[i] * 0.15915494309189533576888376337251436L;   // 1 / (2 pi)
        const long double frac = turn - std::floor(turn);
        a.turns[i] = (uint64_t)(frac * 18446744073709551616.0L);   // 2^64
        a.axis[i] = (uint8_t)axis[i];
    }
    const bool half = rot->layout == SSA_ROTARY_HALF, grad = backward && norm;
    const int full = dt == SSA_F32 ? 4 : 8;
    int V = full;
    for (int i = 0; i < nt; ++i) {
        V = view_vector(*c.out[i], N, es, V);
        for (int j = 0; j < 2; ++j)
            if (in[2 * i + j]) V = view_vector(*in[2 * i + j], N, es, V);
        RowsArg& t = a.t[i];
        // without weights the gradient is the rotation back: the forward's kernel reads it as its input
        const ssa_heads_t* x = backward && !norm ? c.g[i] : c.x[i];
        const ssa_heads_t* g = grad ? c.g[i] : x;
        t = RowsArg{x->data, g->data, c.out[i]->data, norm ? c.gamma[i] : nullptr, nullptr,
                    x->token_stride, x->head_stride, g->token_stride, g->head_stride,
                    c.out[i]->token_stride, c.out[i]->head_stride, x->heads, 0};
    }
    // in the half layout a vector holds one side of V pairs, so 2V has to divide the rotated width; where that leaves short
    // loads of aligned rows, the rows go through shared memory whole
    int side = V;
    while (half && side > 1 && a.pairs % side) side >>= 1;
    V = V == full && side <= kStagedBelow ? 0 : side;     // (kStagedBelow < full)
    a.coords = p->coords;
    a.N = N;
    a.D = D;
    a.G = D * (int)es / 32;
    a.eps = eps;
    a.inv_d = 1.0f / (float)D;
    a.device = p->device;
    a.mscale = rot->mscale;
    a.sgn = backward ? -1.0f : 1.0f;

    const DeviceScope on(p->device);
    if (!on.ok) return SSA_ERR_CUDA;
    const int sms = sm_count(p->device);
    // tokens per tile: some 1280 rows, so that the start of a CTA is a small part of it, but eight CTAs per SM; and
    // the rows that the CTA's warps take at once
    const int once = kWarps * (32 / a.G);
    auto tile_of = [&](int heads) {
        return (int)std::min<int64_t>({(int64_t)kMaxTile, cdiv(1280, heads), std::max(cdiv(once, heads), cdiv(N, 8 * sms))});
    };
    if (grad) {
        a.t[0].tile = tile_of(a.t[0].H);
        a.t[1].tile = nt == 2 ? tile_of(a.t[1].H) : 0;
        a.tile = std::max(a.t[0].tile, a.t[1].tile);
    } else {
        a.tile = tile_of(a.t[0].H + a.t[1].H);
    }
    const int64_t tiles = cdiv(N, a.tile);
    const char* name = backward ? "rotary_backward" : "rotary";
    ProfScope ps(name, st);
    ssa_status_t out = SSA_OK;
    if (!grad) {
        if (!launch_rows(a, (unsigned)tiles, dt, V, half, false, st)) out = SSA_ERR_CUDA;
    } else {
        // persistent CTAs, shared out by the tensors' heads
        const int64_t most = 2 * sms, hq = a.t[0].H, hk = a.t[1].H;
        const int n0 = (int)std::min(cdiv(N, a.t[0].tile), std::max<int64_t>(1, most * hq / (hq + hk)));
        const int n1 = nt == 2 ? (int)std::min(cdiv(N, a.t[1].tile), std::max<int64_t>(1, most * hk / (hq + hk))) : 0;
        double* part = (double*)p->alloc(sizeof(double) * (size_t)(n0 + n1) * D, st, p->alloc_ctx);
        if (!part) {
            out = SSA_ERR_ALLOC;
        } else {
            a.ctas0 = n0;
            a.t[0].part = part;
            a.t[1].part = part + (size_t)n0 * D;
            if (!launch_rows(a, (unsigned)(n0 + n1), dt, V, half, true, st)) out = SSA_ERR_CUDA;
            k_rotary_dgamma<<<dim3(D / 32, nt), dim3(32, 32), 0, st>>>(a.t[0].part, a.t[1].part, n0, n1, D, c.dgamma[0],
                                                                       nt == 2 ? c.dgamma[1] : nullptr);
            note_launch();
            p->release(part, st, p->alloc_ctx);
        }
    }
    const bool clear = cudaGetLastError() == cudaSuccess;     // read in any case: the next call is not to find it
    if (out == SSA_OK && !clear) out = SSA_ERR_CUDA;
    trace_step(name, st);
    return out;
}

}  // namespace

}  // namespace ssa

using namespace ssa;

extern "C" {

ssa_status_t ssa_rotary_frequencies(const ssa_rotary_t* rotary, int32_t head_dim, int32_t* axis, double* freq) {
    const ssa_status_t rc = check_rotary(rotary, head_dim);
    if (rc != SSA_OK) return rc;
    int32_t ax[kMaxPairs];
    double f[kMaxPairs];
    const int n = rotary_frequencies(*rotary, head_dim, ax, f);
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(f[i])) return SSA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (axis) axis[i] = ax[i];
        if (freq) freq[i] = f[i];
    }
    return SSA_OK;
}

ssa_status_t ssa_rotary(ssa_plan_t plan, const ssa_heads_t* q, const ssa_heads_t* k, const float* q_gamma,
                        const float* k_gamma, float eps, const ssa_rotary_t* rotary, int32_t head_dim,
                        ssa_dtype_t dtype, const ssa_heads_t* q_out, const ssa_heads_t* k_out, void* stream) {
    if ((k == nullptr) != (k_out == nullptr)) return SSA_ERR_INVALID_ARG;
    const Call c = {{q, k}, {nullptr, nullptr}, {q_out, k_out}, {q_gamma, k_gamma}, {nullptr, nullptr}};
    return run_rotary(plan, c, eps, rotary, head_dim, dtype, false, (cudaStream_t)stream);
}

ssa_status_t ssa_rotary_backward(ssa_plan_t plan, const ssa_heads_t* dq_out, const ssa_heads_t* dk_out,
                                 const ssa_heads_t* q, const ssa_heads_t* k, const float* q_gamma, const float* k_gamma,
                                 float eps, const ssa_rotary_t* rotary, int32_t head_dim, ssa_dtype_t dtype,
                                 const ssa_heads_t* dq, const ssa_heads_t* dk, float* dq_gamma, float* dk_gamma,
                                 void* stream) {
    if ((dk_out == nullptr) != (dk == nullptr)) return SSA_ERR_INVALID_ARG;
    const Call c = {{q, k}, {dq_out, dk_out}, {dq, dk}, {q_gamma, k_gamma}, {dq_gamma, dk_gamma}};
    return run_rotary(plan, c, eps, rotary, head_dim, dtype, true, (cudaStream_t)stream);
}

}  // extern "C"
