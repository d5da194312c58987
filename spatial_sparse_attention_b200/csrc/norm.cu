// ssa_group_norm and ssa_group_norm_backward: group normalisation over the tokens of a sequence and the
// channels of a group, weights and an activation, channels last, for packed sequences.
//
//   xhat = (x - mean) * rstd,  z = xhat * gamma + beta,  y = act(z),
//   mean, 1/rstd^2 - eps: mean and variance over the m = tokens * width values of a (sequence, group).
// With dz = dy * act'(z):  dbeta = sum dz,  dgamma = sum dz * xhat  (over tokens and sequences),
//   dx = rstd * (dz * gamma - S1 - xhat * S2),  S1 = sum(dz * gamma) / m,  S2 = sum(dz * gamma * xhat) / m
// over the sequence and group.
//
// Bound: HBM. Three launches: sums per channel of every tile of tokens, their merge to groups, and the pass
// that writes. A thread keeps one vector of channels and walks rows, so channel constants stay in registers
// whatever the groups' width. A tile that crosses sequences is cut at their borders: part t of
// the tokens' tiles that lies in sequence s is slot t + s, unique and increasing along the tokens.
#include <algorithm>
#include <cmath>

#include "views.cuh"

namespace ssa {

namespace {

constexpr int kMaxChannels = 65536;
constexpr int kMergeThreads = 256;
// Rows per thread and tile. The variance of a thread's rows comes from sums about its first row: with n rows
// the cancellation is at most a factor n, as the pivot is one of them; 64 keeps it under 2^-18.
constexpr int kMaxRowsPerThread = 64;

struct NormArgs {
    const void* x;
    const void* dy;
    void* out;
    int64_t x_ts, dy_ts, o_ts;
    const float* gamma;     // null: ones
    const float* beta;      // null: zeros
    float* mean;            // [B, G]
    float* rstd;
    float2* part;           // [slots][C]: (mean, sum of squared deviations); gradient: (sum dz, sum dz xhat)
    float2* chan;           // gradient: [B][C] sums per sequence
    float2* s12;            // gradient: [B][G] (S1, S2)
    float* dgamma;
    float* dbeta;
    const SeqInfo* seqs;
    int64_t N, R;           // tokens; tokens per tile
    int32_t B, C, G, width;
    int32_t nvt, nv, rl;    // vectors per row; vectors and row lanes of a CTA
    float eps;
};

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

// sigma(z). The 16-bit types take the fast exponential (2^-21 relative for |z| < 16); fp32 the exact one.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    return __fdividef(1.0f, 1.0f + __expf(-z));
}
template <>
__device__ __forceinline__ float sigmoid<float>(float z) {
    return 1.0f / (1.0f + expf(-z));
}

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

// Per-channel (mean, sum of squared deviations) of every segment of a tile.
template <typename T, int V>
__global__ void k_norm_stats(const __grid_constant__ NormArgs a) {
    using W = Vec<T, V>;
    extern __shared__ float2 red[];     // [rl][nv * V]
    const int vec = threadIdx.x % a.nv, lane = threadIdx.x / a.nv;
    const int v0 = blockIdx.y * a.nv, row_c = a.nv * V;
    const bool active = lane < a.rl && v0 + vec < a.nvt;
    for_segments(a, blockIdx.x, [&](int s, int64_t t, int64_t e) {
        const int n = (int)(e - t), rl = a.rl;
        if (active && lane < n) {
            const T* row = (const T*)a.x + (t + lane) * a.x_ts + (v0 + vec) * V;
            float p[V], sum[V], sq[V];
            W::unpack(*reinterpret_cast<const typename W::C*>(row), p);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] = sq[j] = 0.0f;
            int k = 0;
#pragma unroll 4
            for (int r = lane; r < n; r += rl, ++k) {
                float v[V];
                W::unpack(*reinterpret_cast<const typename W::C*>(row + (int64_t)(r - lane) * a.x_ts), v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[j] - p[j];
                    sum[j] += d;
                    sq[j] = fmaf(d, d, sq[j]);
                }
            }
            const float inv = 1.0f / (float)k;
#pragma unroll
            for (int j = 0; j < V; ++j)
                red[lane * row_c + vec * V + j] = make_float2(fmaf(sum[j], inv, p[j]), sq[j] - sum[j] * sum[j] * inv);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < row_c && v0 * V + c < a.C; c += blockDim.x) {
            const float first = red[c].x;
            float sum = 0.0f, sq = 0.0f;
            for (int l = 0; l < rl && l < n; ++l) {
                const float k = (float)((n - l + rl - 1) / rl), d = red[l * row_c + c].x - first;
                sum = fmaf(k, d, sum);
                sq += fmaf(k * d, d, red[l * row_c + c].y);
            }
            const float inv = 1.0f / (float)n;
            a.part[(blockIdx.x + s) * (int64_t)a.C + v0 * V + c] =
                make_float2(fmaf(sum, inv, first), sq - sum * sum * inv);
        }
        __syncthreads();
    });
}

// Sum of two doubles over the CTA, in a fixed order; every thread gets it.
__device__ __forceinline__ double2 block_sum(double2 v, double2* red) {
    red[threadIdx.x] = v;
    __syncthreads();
    for (int h = kMergeThreads / 2; h > 0; h >>= 1) {
        if (threadIdx.x < h) {
            red[threadIdx.x].x += red[threadIdx.x + h].x;
            red[threadIdx.x].y += red[threadIdx.x + h].y;
        }
        __syncthreads();
    }
    const double2 r = red[0];
    __syncthreads();
    return r;
}

// mean and rstd of group blockIdx.x of sequence blockIdx.y, in fp64 about the first channel's mean.
__global__ void __launch_bounds__(kMergeThreads) k_norm_merge(const __grid_constant__ NormArgs a) {
    __shared__ double2 red[kMergeThreads];
    const int g = blockIdx.x, s = blockIdx.y;
    const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
    if (hi <= lo) {
        if (threadIdx.x == 0) a.mean[(int64_t)s * a.G + g] = a.rstd[(int64_t)s * a.G + g] = 0.0f;
        return;
    }
    const int64_t ta = lo / a.R, tb = (hi - 1) / a.R;
    const int cl = min(a.width, kMergeThreads), sl = kMergeThreads / cl;
    const int l = threadIdx.x / cl;
    const float2* part = a.part + (int64_t)s * a.C + g * a.width;
    const double first = part[ta * a.C].x;
    double2 acc = make_double2(0.0, 0.0);
    if (l < sl) {
        for (int c = threadIdx.x % cl; c < a.width; c += cl) {
            for (int64_t t = ta + l; t <= tb; t += sl) {
                const float2 v = part[t * a.C + c];
                const double k = (double)(min(hi, (t + 1) * a.R) - max(lo, t * a.R)), d = (double)v.x - first;
                acc.x += k * d;
                acc.y += (double)v.y + k * d * d;
            }
        }
    }
    acc = block_sum(acc, red);
    if (threadIdx.x == 0) {
        const double m = (double)(hi - lo) * a.width, d = acc.x / m;
        const double var = fmax(acc.y / m - d * d, 0.0);
        a.mean[(int64_t)s * a.G + g] = (float)(first + d);
        // a NaN or an infinity among the values leaves NaN here (fmax drops it)
        const double r = 1.0 / sqrt(var + (double)a.eps);
        a.rstd[(int64_t)s * a.G + g] = acc.y == acc.y ? (float)r : (float)acc.y;
    }
}

// A thread's channel constants in one sequence.
template <int V>
struct Channels {
    float mean[V], rstd[V], gamma[V], beta[V];
    __device__ __forceinline__ void load(const NormArgs& a, int s, int c0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t at = (int64_t)s * a.G + (c0 + j) / a.width;
            mean[j] = a.mean[at];
            rstd[j] = a.rstd[at];
            gamma[j] = a.gamma ? a.gamma[c0 + j] : 1.0f;
            beta[j] = a.beta ? a.beta[c0 + j] : 0.0f;
        }
    }
};

template <typename T, int V, int ACT>
__global__ void k_norm_apply(const __grid_constant__ NormArgs a) {
    using W = Vec<T, V>;
    const int vec = blockIdx.y * a.nv + threadIdx.x % a.nv, lane = threadIdx.x / a.nv;
    if (lane >= a.rl || vec >= a.nvt) return;
    for_segments(a, blockIdx.x, [&](int s, int64_t t, int64_t e) {
        Channels<V> ch;
        ch.load(a, s, vec * V);
        float scale[V];
#pragma unroll
        for (int j = 0; j < V; ++j) scale[j] = ch.rstd[j] * ch.gamma[j];
        const T* x = (const T*)a.x + vec * V;
        T* out = (T*)a.out + vec * V;
#pragma unroll 4
        for (int64_t r = t + lane; r < e; r += a.rl) {
            float v[V];
            W::unpack(*reinterpret_cast<const typename W::C*>(x + r * a.x_ts), v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = activate<T, ACT>(fmaf(v[j] - ch.mean[j], scale[j], ch.beta[j]));
            *reinterpret_cast<typename W::C*>(out + r * a.o_ts) = W::pack(v);
        }
    });
}

// Per-channel sums of dz and dz * xhat of every segment of a tile.
template <typename T, int V, int ACT>
__global__ void k_norm_grad_sums(const __grid_constant__ NormArgs a) {
    using W = Vec<T, V>;
    extern __shared__ float2 red[];
    const int vec = threadIdx.x % a.nv, lane = threadIdx.x / a.nv;
    const int v0 = blockIdx.y * a.nv, row_c = a.nv * V;
    const bool active = lane < a.rl && v0 + vec < a.nvt;
    for_segments(a, blockIdx.x, [&](int s, int64_t t, int64_t e) {
        if (active) {
            Channels<V> ch;
            ch.load(a, s, (v0 + vec) * V);
            float s0[V], s1[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s0[j] = s1[j] = 0.0f;
            const T* x = (const T*)a.x + (v0 + vec) * V;
            const T* dy = (const T*)a.dy + (v0 + vec) * V;
#pragma unroll 2
            for (int64_t r = t + lane; r < e; r += a.rl) {
                float v[V], d[V];
                W::unpack(*reinterpret_cast<const typename W::C*>(x + r * a.x_ts), v);
                W::unpack(*reinterpret_cast<const typename W::C*>(dy + r * a.dy_ts), d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xhat = (v[j] - ch.mean[j]) * ch.rstd[j];
                    const float dz = d[j] * activate_grad<T, ACT>(fmaf(xhat, ch.gamma[j], ch.beta[j]));
                    s0[j] += dz;
                    s1[j] = fmaf(dz, xhat, s1[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) red[lane * row_c + vec * V + j] = make_float2(s0[j], s1[j]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < row_c && v0 * V + c < a.C; c += blockDim.x) {
            float2 sum = make_float2(0.0f, 0.0f);
            for (int l = 0; l < a.rl; ++l) {
                sum.x += red[l * row_c + c].x;
                sum.y += red[l * row_c + c].y;
            }
            a.part[(blockIdx.x + s) * (int64_t)a.C + v0 * V + c] = sum;
        }
        __syncthreads();
    });
}

// The channels' sums over sequence blockIdx.y, and S1, S2 of group blockIdx.x.
__global__ void __launch_bounds__(kMergeThreads) k_norm_grad_merge(const __grid_constant__ NormArgs a) {
    __shared__ double2 red[kMergeThreads];
    const int g = blockIdx.x, s = blockIdx.y;
    const int64_t lo = a.seqs[s].lo, hi = a.seqs[s].hi;
    const int cl = min(a.width, kMergeThreads), sl = kMergeThreads / cl;
    const int col = threadIdx.x % cl, l = threadIdx.x / cl;
    float2* chan = a.chan + (int64_t)s * a.C + g * a.width;
    if (hi <= lo) {
        for (int c = threadIdx.x; c < a.width; c += kMergeThreads) chan[c] = make_float2(0.0f, 0.0f);
        return;
    }
    const int64_t ta = lo / a.R, tb = (hi - 1) / a.R;
    const float2* part = a.part + (int64_t)s * a.C + g * a.width;
    double2 total = make_double2(0.0, 0.0);
    for (int c0 = 0; c0 < a.width; c0 += cl) {
        const int c = c0 + col;
        double2 acc = make_double2(0.0, 0.0);
        if (l < sl && c < a.width) {
            for (int64_t t = ta + l; t <= tb; t += sl) {
                const float2 v = part[t * a.C + c];
                acc.x += v.x;
                acc.y += v.y;
            }
        }
        red[threadIdx.x] = acc;
        __syncthreads();
        if (l == 0 && c < a.width) {
            for (int i = 1; i < sl; ++i) {
                acc.x += red[i * cl + col].x;
                acc.y += red[i * cl + col].y;
            }
            chan[c] = make_float2((float)acc.x, (float)acc.y);
            const double gamma = a.gamma ? (double)a.gamma[g * a.width + c] : 1.0;
            total.x += gamma * acc.x;
            total.y += gamma * acc.y;
        }
        __syncthreads();
    }
    total = block_sum(total, red);
    if (threadIdx.x == 0) {
        const double m = (double)(hi - lo) * a.width;
        a.s12[(int64_t)s * a.G + g] = make_float2((float)(total.x / m), (float)(total.y / m));
    }
}

// dx; and the weights' gradients, the channels' sums over the sequences, by the first tile's CTAs.
template <typename T, int V, int ACT>
__global__ void k_norm_grad_apply(const __grid_constant__ NormArgs a) {
    using W = Vec<T, V>;
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < a.nv * V; i += blockDim.x) {
            const int c = blockIdx.y * a.nv * V + i;
            if (c >= a.C) break;
            double b = 0.0, g = 0.0;
            for (int s = 0; s < a.B; ++s) {
                const float2 v = a.chan[(int64_t)s * a.C + c];
                b += v.x;
                g += v.y;
            }
            a.dbeta[c] = (float)b;
            a.dgamma[c] = (float)g;
        }
    }
    const int vec = blockIdx.y * a.nv + threadIdx.x % a.nv, lane = threadIdx.x / a.nv;
    if (lane >= a.rl || vec >= a.nvt) return;
    for_segments(a, blockIdx.x, [&](int s, int64_t t, int64_t e) {
        Channels<V> ch;
        ch.load(a, s, vec * V);
        float S1[V], S2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 v = a.s12[(int64_t)s * a.G + (vec * V + j) / a.width];
            S1[j] = v.x;
            S2[j] = v.y;
        }
        const T* x = (const T*)a.x + vec * V;
        const T* dy = (const T*)a.dy + vec * V;
        T* out = (T*)a.out + vec * V;
#pragma unroll 2
        for (int64_t r = t + lane; r < e; r += a.rl) {
            float v[V], d[V];
            W::unpack(*reinterpret_cast<const typename W::C*>(x + r * a.x_ts), v);
            W::unpack(*reinterpret_cast<const typename W::C*>(dy + r * a.dy_ts), d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xhat = (v[j] - ch.mean[j]) * ch.rstd[j];
                const float dz = d[j] * activate_grad<T, ACT>(fmaf(xhat, ch.gamma[j], ch.beta[j]));
                v[j] = ch.rstd[j] * (fmaf(dz, ch.gamma[j], -S1[j]) - xhat * S2[j]);
            }
            *reinterpret_cast<typename W::C*>(out + r * a.o_ts) = W::pack(v);
        }
    });
}

// ---- host --------------------------------------------------------------------------------------

struct Launch {
    dim3 grid;
    int threads;
    size_t smem;
    bool grad;
    int act;
    cudaStream_t st;
};

template <typename T, int V, int ACT>
void launch_act(const NormArgs& a, const Launch& l) {
    if (l.grad) {
        k_norm_grad_sums<T, V, ACT><<<l.grid, l.threads, l.smem, l.st>>>(a);
        k_norm_grad_merge<<<dim3(a.G, a.B), kMergeThreads, 0, l.st>>>(a);
        k_norm_grad_apply<T, V, ACT><<<l.grid, l.threads, 0, l.st>>>(a);
    } else {
        k_norm_stats<T, V><<<l.grid, l.threads, l.smem, l.st>>>(a);
        k_norm_merge<<<dim3(a.G, a.B), kMergeThreads, 0, l.st>>>(a);
        k_norm_apply<T, V, ACT><<<l.grid, l.threads, 0, l.st>>>(a);
    }
    note_launch(3);
}

template <typename T, int V>
void launch_vec(const NormArgs& a, const Launch& l) {
    if (l.act == SSA_ACT_SILU) launch_act<T, V, SSA_ACT_SILU>(a, l);
    else if (l.act == SSA_ACT_GELU) launch_act<T, V, SSA_ACT_GELU>(a, l);
    else launch_act<T, V, SSA_ACT_NONE>(a, l);
}

template <typename T>
void launch_type(const NormArgs& a, const Launch& l, int V) {
    if constexpr (sizeof(T) == 2) {
        if (V == 8) return launch_vec<T, 8>(a, l);
    }
    if (V == 4) launch_vec<T, 4>(a, l);
    else if (V == 2) launch_vec<T, 2>(a, l);
    else launch_vec<T, 1>(a, l);
}

// Vectors per CTA and row lanes: the split of a row's vectors that keeps most threads of a CTA of up to 288
// busy, wide CTAs first.
void shape_cta(int nvt, int* nv, int* rl, int* threads) {
    double best = 0.0;
    const int least = (nvt + 287) / 288;
    for (int n = least; n < least + 64; ++n) {
        const int w = (nvt + n - 1) / n;
        if (w < 4 && n > least) break;
        const int r = std::max(1, 288 / w), th = (w * r + 31) / 32 * 32;
        const double use = (double)nvt / ((double)((nvt + w - 1) / w) * w) * (w * r) / th;
        if (use > best + 0.02) {
            best = use;
            *nv = w;
            *rl = r;
            *threads = th;
        }
    }
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
    a.nvt = C / V;
    Launch l = {};
    shape_cta(a.nvt, &a.nv, &a.rl, &l.threads);
    const int ncol = (int)cdiv(a.nvt, a.nv);

    const DeviceScope on(p->device);
    if (!on.ok) return SSA_ERR_CUDA;
    // tokens per tile: eight CTAs per SM, between 4 and 64 rows a thread
    const int64_t even = cdiv(N * ncol, 8 * sm_count(p->device));
    a.R = std::min<int64_t>(std::max<int64_t>(even, 4 * a.rl), (int64_t)kMaxRowsPerThread * a.rl);
    const int64_t tiles = cdiv(N, a.R), slots = tiles + p->B;
    l.grid = dim3((unsigned)tiles, (unsigned)ncol);
    l.smem = sizeof(float2) * a.nv * V * a.rl;
    l.grad = grad;
    l.act = act;
    l.st = st;

    // one buffer: partial sums, and the sequences' sums or the statistics that the caller does not want
    const int64_t BG = (int64_t)p->B * G, extra = grad ? (int64_t)p->B * C + BG : (c.mean ? 0 : BG);
    a.part = (float2*)p->alloc(sizeof(float2) * (size_t)(slots * C + extra), st, p->alloc_ctx);
    if (!a.part) return SSA_ERR_ALLOC;
    a.mean = c.mean;
    a.rstd = c.rstd;
    float2* rest = a.part + slots * C;
    if (grad) {
        a.chan = rest;
        a.s12 = rest + (int64_t)p->B * C;
    } else if (!c.mean) {
        a.mean = (float*)rest;
        a.rstd = a.mean + BG;
    }
    if (dt == SSA_F32) launch_type<float>(a, l, V);
    else if (dt == SSA_BF16) launch_type<__nv_bfloat16>(a, l, V);
    else launch_type<__half>(a, l, V);
    p->release(a.part, st, p->alloc_ctx);
    return cudaGetLastError() == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
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
