// ssa_rotary and ssa_rotary_backward: RMS normalisation of queries and keys over the head dimension and
// rotary positions at the voxel coordinates, as operators of their own with gradients (Hi3D v1.0
// pipeline page, "Stage 3: sparse flow sampling").
//
// Per (token, head) row x, with n = x * inv, inv = rsqrt(mean x^2 + eps) and u = n * gamma:
//   (a, b) -> (a c - b s, a s + b c) * mscale   for every rotated pair (a, b) of u.
// The gradient turns back, du = R^T dy, and then dx = inv * (g - n * mean(g n)) with g = du * gamma, and
// dgamma = sum over rows of du * n.
//
// Bound: HBM. A row moves 2 (gradient with weights: 3) times head_dim elements for some 10
// operations each. So a lane keeps 32 bytes of a row (two 16-byte loads), two to sixteen lanes make
// a row, and every lane has the loads of several rows in flight before it uses the first. The
// cosines and sines are shared by all heads of a token: a CTA takes a tile of tokens and computes
// them once into shared memory.
#include <algorithm>
#include <cmath>

#include "views.cuh"

namespace ssa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = 16;      // tokens per CTA tile
constexpr int kMaxPairs = 64;     // head_dim <= 128
constexpr int kTabStride = kMaxPairs + 4;   // floats per token in a table (16-byte aligned rows)

struct RowsArg {
    const void* x;        // forward: input; gradient: the forward's input (weights) or unused
    const void* g;        // gradient: gradient of the output
    void* out;
    const float* gamma;
    float* part;          // gradient with weights: [CTAs of this tensor][D] partial sums
    int64_t x_ts, x_hs, g_ts, g_hs, o_ts, o_hs;
    int32_t H;
};

// Frequencies as fractions of a turn in units of 2^-64: coordinate * turns wraps modulo one turn by
// itself, so the angle is reduced exactly at any coordinate.
struct RotArgs {
    RowsArg t[2];                  // queries, keys
    const int32_t* coords;
    int64_t N;
    int32_t D, G;                  // head dimension; lanes per row
    int32_t pairs;                 // rotated pairs
    int32_t tile;                  // tokens per tile
    int32_t ctas0;                 // CTAs [0, ctas0) work on t[0], the rest on t[1]
    float eps, mscale, sgn;        // sgn = -1 turns back
    uint64_t turns[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

// How a lane's 32 bytes of a row are cut. An item is P pairs: one load of V = 2P elements (interleaved,
// V >= 2), or two loads of V elements (half: the pairs' two sides; interleaved at V = 1). Item m of lane l
// is item m*G + l of the row, so neighbouring lanes read neighbouring items.
template <typename T, int V, bool HALF>
struct Cut {
    static constexpr int E = 32 / (int)sizeof(T);          // elements per lane
    static constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);
    static constexpr int M = E / (2 * P);                   // items per lane
    static constexpr int L = 2 * P / V;                     // loads per item
    using C = typename Chunk<V * (int)sizeof(T)>::type;
};

// Place of pair p in a token's table row: pairs that one lane reads as two float4 are kept four apart by
// the row's items, so that a warp's 16-byte reads are contiguous.
template <int P>
__device__ __forceinline__ int tab_pos(int p, int items) {
    if (P == 8) return (((p >> 2) & 1) * items + (p >> 3)) * 4 + (p & 3);
    return p;
}

// cos and sin of coordinate * turns (2^-64 of a turn), by quadrant plus a remainder of at most an
// eighth of a turn, which fp32 holds to 2^-28 of a turn.
__device__ __forceinline__ void turn_cos_sin(int32_t coord, uint64_t turns, float& c, float& s) {
    const int32_t hi = (int32_t)(((uint64_t)(uint32_t)coord * turns) >> 32);   // signed, 2^-32 of a turn
    const int32_t q = (int32_t)((uint32_t)hi + 0x20000000u) >> 30;
    const float r = (float)(int32_t)((uint32_t)hi - ((uint32_t)q << 30)) * 0x1p-31f;   // half turns
    float c0, s0;
    sincospif(r, &s0, &c0);
    c = (q & 1) ? s0 : c0;
    s = (q & 1) ? c0 : s0;
    if ((q & 3) == 1 || (q & 3) == 2) c = -c;
    if (q & 2) s = -s;
}

template <typename CUT, typename T>
__device__ __forceinline__ void load_row(const T* row, const int (&off)[CUT::M * CUT::L],
                                         typename CUT::C (&raw)[CUT::M * CUT::L]) {
#pragma unroll
    for (int i = 0; i < CUT::M * CUT::L; ++i) raw[i] = *reinterpret_cast<const typename CUT::C*>(row + off[i]);
}

template <typename CUT, typename T, int N>
__device__ __forceinline__ void unpack(const typename CUT::C (&raw)[N], float (&e)[CUT::E]) {
    constexpr int V = CUT::E / N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        T v[V];
        memcpy(v, &raw[i], sizeof(v));
#pragma unroll
        for (int j = 0; j < V; ++j) e[i * V + j] = Elem<T>::to_f(v[j]);
    }
}

template <typename CUT, typename T, int N>
__device__ __forceinline__ void store_row(T* row, const int (&off)[N], const float (&e)[CUT::E]) {
    constexpr int V = CUT::E / N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        T v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = Elem<T>::from_f(e[i * V + j]);
        typename CUT::C raw;
        memcpy(&raw, v, sizeof(v));
        *reinterpret_cast<typename CUT::C*>(row + off[i]) = raw;
    }
}

// Sum over the G lanes of a row (G = 2, 4, 6, 8, 12, 16; its first lane is `base`); all lanes of the warp
// call it. G = 6 and 12 end with three partial sums added in one order, so that the lanes of a row agree.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int G, int base, int l) {
    int n = G;
    while (!(n & 1)) {
        n >>= 1;
        const int src = base + (l + n < G ? l + n : l + n - G);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_sync(0xffffffffu, v[k], src);
    }
    if (n == 3) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float a = __shfl_sync(0xffffffffu, v[k], base);
            const float b = __shfl_sync(0xffffffffu, v[k], base + 1);
            const float c = __shfl_sync(0xffffffffu, v[k], base + 2);
            v[k] = (a + b) + c;
        }
    }
}

// Turn the pairs of a lane's elements; cs, sn are the token's table rows. Channels that pass through are
// left as they are, whatever their neighbours hold.
template <typename CUT, int V, bool HALF>
__device__ __forceinline__ void turn_row(float (&e)[CUT::E], const float* cs, const float* sn, int l, int G, int pairs) {
    constexpr int P = CUT::P;
#pragma unroll
    for (int m = 0; m < CUT::M; ++m) {
        const int it = m * G + l;
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
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int ia = m * 2 * P + (HALF ? i : 2 * i), ib = m * 2 * P + (HALF ? P + i : 2 * i + 1);
            const float a = e[ia], b = e[ib];
            const bool turned = it * P + i < pairs;
            e[ia] = turned ? a * c[i] - b * s[i] : a;
            e[ib] = turned ? a * s[i] + b * c[i] : b;
        }
    }
}

// The tokens' cosines and sines, for ntok tokens from tok0. Neighbouring threads take neighbouring
// tokens of one pair, so that the pair's frequency is one constant per warp.
template <int P>
__device__ __forceinline__ void fill_tables(const RotArgs& a, int64_t tok0, int ntok, float (*cs)[kTabStride],
                                            float (*sn)[kTabStride]) {
    for (int i = threadIdx.x; i < a.pairs * kMaxTile; i += kThreads) {
        const int p = i / kMaxTile, t = i % kMaxTile;
        if (t >= ntok) continue;
        float c, s;
        turn_cos_sin(a.coords[3 * (tok0 + t) + a.axis[p]], a.turns[p], c, s);
        const int at = tab_pos<P>(p, a.D / (2 * P));
        cs[t][at] = c * a.mscale;
        sn[t][at] = s * (a.mscale * a.sgn);
    }
}

// First channel of load i of lane l. In the half layout a load holds one side of its item's pairs.
template <typename T, int V, bool HALF>
__device__ __forceinline__ int load_offset(const RotArgs& a, int l, int i) {
    using CUT = Cut<T, V, HALF>;
    const int side = i % CUT::L, p = (i / CUT::L * a.G + l) * CUT::P;   // the item's first pair
    // 2P divides the rotated width: an item is turned as a whole or not
    if (HALF && p < a.pairs) return side * a.pairs + p;
    return 2 * p + side * CUT::P;
}

// Channel of element i (0..E-1) of lane l.
template <typename T, int V, bool HALF>
__device__ __forceinline__ int lane_channel(const RotArgs& a, int l, int i) {
    return load_offset<T, V, HALF>(a, l, i / V) + i % V;
}

template <typename T, int V, bool HALF>
__device__ __forceinline__ void lane_offsets(const RotArgs& a, int l, int (&off)[Cut<T, V, HALF>::M * Cut<T, V, HALF>::L]) {
#pragma unroll
    for (int i = 0; i < Cut<T, V, HALF>::M * Cut<T, V, HALF>::L; ++i) off[i] = load_offset<T, V, HALF>(a, l, i);
}

// out = rotate(normalise(x)), or the rotation back (sgn = -1, no weights). One tile of tokens of one
// tensor per CTA; warps take row after row, U of them with their loads in flight.
template <typename T, int V, bool HALF, bool NORM>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ RotArgs a) {
    using CUT = Cut<T, V, HALF>;
    constexpr int E = CUT::E, NL = CUT::M * CUT::L, U = 4;
    __shared__ __align__(16) float cs[kMaxTile][kTabStride];
    __shared__ __align__(16) float sn[kMaxTile][kTabStride];
    const int which = blockIdx.x < a.ctas0 ? 0 : 1;
    const RowsArg& t = a.t[which];
    const int64_t tok0 = (int64_t)(blockIdx.x - (which ? a.ctas0 : 0)) * a.tile;
    const int ntok = (int)min((int64_t)a.tile, a.N - tok0);
    fill_tables<CUT::P>(a, tok0, ntok, cs, sn);

    const int lane = threadIdx.x & 31, G = a.G, rpw = 32 / G;
    const int sub = lane / G, l = lane - sub * G, base = lane - l;
    int off[NL];
    lane_offsets<T, V, HALF>(a, l, off);
    float gam[E];
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < E; ++i) gam[i] = t.gamma[off[i / V] + i % V];
    }
    __syncthreads();

    const int nrow = ntok * t.H, step = kWarps * rpw;
    const int dt = step / t.H, dh = step - dt * t.H;
    int r = (threadIdx.x >> 5) * rpw + sub;
    int tt = r / t.H, hh = r - tt * t.H;
    if (sub >= rpw) r = nrow;    // lanes beyond the last whole row of the warp
    const T* x = (const T*)t.x + tok0 * t.x_ts;
    T* out = (T*)t.out + tok0 * t.o_ts;
    for (int w0 = (threadIdx.x >> 5) * rpw; w0 < nrow; w0 += U * step) {
        typename CUT::C raw[U][NL];
        int rt[U], rh[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rt[u] = r < nrow ? tt : -1;
            rh[u] = hh;
            if (rt[u] >= 0) load_row<CUT, T>(x + tt * t.x_ts + hh * t.x_hs, off, raw[u]);
            r += step;
            tt += dt;
            hh += dh;
            if (hh >= t.H) {
                hh -= t.H;
                ++tt;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float e[E];
            if (rt[u] >= 0) unpack<CUT, T>(raw[u], e);
            if constexpr (NORM) {
                float ss[1] = {0.0f};
                if (rt[u] >= 0) {
#pragma unroll
                    for (int i = 0; i < E; ++i) ss[0] = fmaf(e[i], e[i], ss[0]);
                }
                row_sum(ss, G, base, l);
                const float inv = rsqrtf(ss[0] / (float)a.D + a.eps);
#pragma unroll
                for (int i = 0; i < E; ++i) e[i] = e[i] * inv * gam[i];
            }
            if (rt[u] >= 0) {
                turn_row<CUT, V, HALF>(e, cs[rt[u]], sn[rt[u]], l, G, a.pairs);
                store_row<CUT, T>(out + rt[u] * t.o_ts + rh[u] * t.o_hs, off, e);
            }
        }
    }
}

// The gradient with weights. Persistent: a CTA walks tiles of its tensor and keeps the weights' sums
// of its lanes' channels in registers; it adds them up over its rows in a fixed order at the end.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rotary_grad(const __grid_constant__ RotArgs a) {
    using CUT = Cut<T, V, HALF>;
    constexpr int E = CUT::E, NL = CUT::M * CUT::L, U = 2;
    __shared__ __align__(16) float cs[kMaxTile][kTabStride];
    __shared__ __align__(16) float sn[kMaxTile][kTabStride];
    __shared__ float red[kThreads * E];
    const int which = blockIdx.x < a.ctas0 ? 0 : 1;
    const RowsArg& t = a.t[which];
    const int cta = blockIdx.x - (which ? a.ctas0 : 0), nctas = which ? gridDim.x - a.ctas0 : a.ctas0;

    const int lane = threadIdx.x & 31, G = a.G, rpw = 32 / G;
    const int sub = lane / G, l = lane - sub * G, base = lane - l;
    int off[NL];
    lane_offsets<T, V, HALF>(a, l, off);
    float gam[E], acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        gam[i] = t.gamma[off[i / V] + i % V];
        acc[i] = 0.0f;
    }
    const int step = kWarps * rpw;
    const int dt = step / t.H, dh = step - dt * t.H;
    for (int64_t tok0 = (int64_t)cta * a.tile; tok0 < a.N; tok0 += (int64_t)nctas * a.tile) {
        const int ntok = (int)min((int64_t)a.tile, a.N - tok0);
        __syncthreads();    // the previous tile's tables are read
        fill_tables<CUT::P>(a, tok0, ntok, cs, sn);
        __syncthreads();
        const int nrow = ntok * t.H;
        int r = (threadIdx.x >> 5) * rpw + sub;
        int tt = r / t.H, hh = r - tt * t.H;
        if (sub >= rpw) r = nrow;
        const T* x = (const T*)t.x + tok0 * t.x_ts;
        const T* g = (const T*)t.g + tok0 * t.g_ts;
        T* out = (T*)t.out + tok0 * t.o_ts;
        for (int w0 = (threadIdx.x >> 5) * rpw; w0 < nrow; w0 += U * step) {
            typename CUT::C xr[U][NL], gr[U][NL];
            int rt[U], rh[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                rt[u] = r < nrow ? tt : -1;
                rh[u] = hh;
                if (rt[u] >= 0) {
                    load_row<CUT, T>(x + tt * t.x_ts + hh * t.x_hs, off, xr[u]);
                    load_row<CUT, T>(g + tt * t.g_ts + hh * t.g_hs, off, gr[u]);
                }
                r += step;
                tt += dt;
                hh += dh;
                if (hh >= t.H) {
                    hh -= t.H;
                    ++tt;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[E], d[E], sums[2] = {0.0f, 0.0f};   // sum x^2, sum du gamma x
                if (rt[u] >= 0) {
                    unpack<CUT, T>(xr[u], e);
                    unpack<CUT, T>(gr[u], d);
                    turn_row<CUT, V, HALF>(d, cs[rt[u]], sn[rt[u]], l, G, a.pairs);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sums[0] = fmaf(e[i], e[i], sums[0]);
                        sums[1] = fmaf(d[i] * gam[i], e[i], sums[1]);
                    }
                }
                row_sum(sums, G, base, l);
                if (rt[u] >= 0) {
                    const float inv = rsqrtf(sums[0] / (float)a.D + a.eps);
                    const float dot = sums[1] * inv / (float)a.D;      // mean of g n
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float n = e[i] * inv;
                        acc[i] = fmaf(d[i], n, acc[i]);
                        d[i] = inv * (d[i] * gam[i] - n * dot);
                    }
                    store_row<CUT, T>(out + rt[u] * t.o_ts + rh[u] * t.o_hs, off, d);
                }
            }
        }
    }
    // every lane's sums to shared memory; then one thread per element adds those of all warps and rows
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) red[i * kThreads + threadIdx.x] = acc[i];
    __syncthreads();
    if (threadIdx.x < a.D) {
        const int i = threadIdx.x / G, ll = threadIdx.x - i * G;   // element i of lane ll
        float s = 0.0f;
        for (int w = 0; w < kWarps; ++w)
            for (int q = 0; q < rpw; ++q) s += red[i * kThreads + w * 32 + q * G + ll];
        t.part[(int64_t)cta * a.D + lane_channel<T, V, HALF>(a, ll, i)] = s;
    }
}

// dgamma[c] = sum over CTAs of part[cta][c], 32 channels per CTA, in a fixed order.
__global__ void __launch_bounds__(1024) k_rotary_dgamma(const float* __restrict__ part0, const float* __restrict__ part1,
                                                        int n0, int n1, int D, float* out0, float* out1) {
    __shared__ float red[32][33];
    const float* part = blockIdx.y ? part1 : part0;
    const int n = blockIdx.y ? n1 : n0, c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    for (int i = threadIdx.y; i < n; i += 32) s += part[(int64_t)i * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
        (blockIdx.y ? out1 : out0)[c] = s;
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
            axis[p] = a;
            freq[p] = f;
        }
    }
    return p;
}

template <typename T, int V, bool HALF>
void launch_cut(const RotArgs& a, unsigned grid, bool grad, cudaStream_t st) {
    if (grad)
        k_rotary_grad<T, V, HALF><<<grid, kThreads, 0, st>>>(a);
    else if (a.t[0].gamma)
        k_rotary<T, V, HALF, true><<<grid, kThreads, 0, st>>>(a);
    else
        k_rotary<T, V, HALF, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename T, int V>
void launch_layout(const RotArgs& a, unsigned grid, bool half, bool grad, cudaStream_t st) {
    if (half) launch_cut<T, V, true>(a, grid, grad, st);
    else launch_cut<T, V, false>(a, grid, grad, st);
    note_launch();
}

void launch_rows(const RotArgs& a, unsigned grid, ssa_dtype_t dt, int V, bool half, bool grad, cudaStream_t st) {
    if (dt == SSA_F32) {
        if (V >= 4) launch_layout<float, 4>(a, grid, half, grad, st);
        else if (V == 2) launch_layout<float, 2>(a, grid, half, grad, st);
        else launch_layout<float, 1>(a, grid, half, grad, st);
        return;
    }
    auto pick = [&](auto tag) {
        using T = decltype(tag);
        if (V >= 8) launch_layout<T, 8>(a, grid, half, grad, st);
        else if (V == 4) launch_layout<T, 4>(a, grid, half, grad, st);
        else if (V == 2) launch_layout<T, 2>(a, grid, half, grad, st);
        else launch_layout<T, 1>(a, grid, half, grad, st);
    };
    if (dt == SSA_BF16) pick(__nv_bfloat16());
    else pick(__half());
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
    if (!(eps >= 0.0f)) return SSA_ERR_INVALID_ARG;
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

    RotArgs a = {};
    int32_t axis[kMaxPairs];
    double freq[kMaxPairs];
    a.pairs = rotary_frequencies(*rot, D, axis, freq);
    for (int i = 0; i < a.pairs; ++i) {
        const long double turn = (long double)freq[i] * 0.15915494309189533576888376337251436L;   // 1 / (2 pi)
        const long double frac = turn - std::floor(turn);
        a.turns[i] = (uint64_t)(frac * 18446744073709551616.0L);   // 2^64
        a.axis[i] = (uint8_t)axis[i];
    }
    const bool half = rot->layout == SSA_ROTARY_HALF, grad = backward && norm;
    int V = dt == SSA_F32 ? 4 : 8;
    // in the half layout a vector holds one side of V pairs, so 2V has to divide the rotated width
    while (half && V > 1 && 2 * a.pairs % (2 * V)) V >>= 1;
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
                    c.out[i]->token_stride, c.out[i]->head_stride, x->heads};
    }
    a.coords = p->coords;
    a.N = N;
    a.D = D;
    a.G = D * (int)es / 32;
    a.eps = eps;
    a.mscale = rot->mscale;
    a.sgn = backward ? -1.0f : 1.0f;

    const DeviceScope on(p->device);
    if (!on.ok) return SSA_ERR_CUDA;
    const int sms = sm_count(p->device);
    // tokens per tile: the most that still gives every SM several CTAs
    a.tile = (int)std::min<int64_t>(kMaxTile, std::max<int64_t>(1, N / (4 * sms)));
    const int64_t tiles = cdiv(N, a.tile);
    ssa_status_t out = SSA_OK;
    if (!grad) {
        a.ctas0 = (int)tiles;
        launch_rows(a, (unsigned)(nt * tiles), dt, V, half, false, st);
    } else {
        // persistent CTAs, shared out by the tensors' heads
        const int64_t most = 3 * sms, hq = a.t[0].H, hk = nt == 2 ? a.t[1].H : 0;
        const int n0 = (int)std::min(tiles, std::max<int64_t>(1, most * hq / (hq + hk)));
        const int n1 = nt == 2 ? (int)std::min(tiles, std::max<int64_t>(1, most * hk / (hq + hk))) : 0;
        float* part = (float*)p->alloc(sizeof(float) * (size_t)(n0 + n1) * D, st, p->alloc_ctx);
        if (!part) {
            out = SSA_ERR_ALLOC;
        } else {
            a.ctas0 = n0;
            a.t[0].part = part;
            a.t[1].part = part + (size_t)n0 * D;
            launch_rows(a, (unsigned)(n0 + n1), dt, V, half, true, st);
            k_rotary_dgamma<<<dim3(D / 32, nt), dim3(32, 32), 0, st>>>(a.t[0].part, a.t[1].part, n0, n1, D, c.dgamma[0],
                                                                       nt == 2 ? c.dgamma[1] : nullptr);
            note_launch();
            p->release(part, st, p->alloc_ctx);
        }
    }
    if (out == SSA_OK && cudaGetLastError() != cudaSuccess) out = SSA_ERR_CUDA;
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
