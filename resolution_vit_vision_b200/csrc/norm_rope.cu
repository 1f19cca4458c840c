// norm_rope.cu -- per-head RMS norm of q and k with the 3-D M-RoPE rotation in the same pass, and
// its gradient.
//
// Mathematics, for one head vector x of D dims at a token with positions (t, h, w):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,  y = R n,
// R turning the pairs (j, j + D/2) by pos[axis(j)] theta^(-2j/D), as mrope_apply ("Qwen2-VL", intro
// and Qwen2VLModel table). Gradient, with dn = R^T dy and g = dn w:
//   dx = r (g - x r^2 mean(g x)),  dw = sum over tokens and heads of dn x r.
// Both sums of a head (x^2 and g x) are taken in one round of shuffles, since r factors out.
//
// Bound by HBM: the forward reads and writes every element once, the gradient reads x and dy and
// writes dx. A lane owns one 16-byte vector of the lower half of a head and the matching one of the
// upper half, so a head is D / (2 kVec) lanes (8 for 128 16-bit dims), its sums are shuffles inside
// that group and a pair never leaves its lane. Heads whose lane count is not a power of two (D = 80,
// 96) leave the group's last lanes idle. A CTA takes a tile of tokens; cos / sin and the weights sit
// in shared memory in an order that gives the lanes of a group consecutive 16-byte words. All
// arithmetic is fp32 (angles fp64), rounded once to the element type on the way out.
#include <algorithm>
#include <cmath>

#include "dtype.cuh"
#include "internal.h"

namespace vitk {

constexpr int kNormMaxFreq = 128;       // head_dim <= 256
constexpr int kNormThreads = 256;
constexpr int kNormMaxTile = 8;         // tokens per tile
constexpr int kNormGradCtas = 592;      // at most this many CTAs write partial weight gradients

struct NormRopeArgs {
    const void *x[2];                   // q, k
    void *y[2];                         // outputs (dq, dk in the gradient)
    const void *dy[2];                  // gradient only
    const void *w[2];                   // may be null: ones
    int64_t xs[2], ys[2], dys[2];       // token strides in elements
    int heads[2];
    int D;
    float eps;
    const int32_t *pos;
    int64_t L;
    int tile;                           // tokens per tile
    float *dw_part;                     // [grid][2][D], gradient only, may be null
    int n_freq, axis_end0, axis_end1;
    double inv_freq[kNormMaxFreq];
};

// Shared arrays hold element e of lane g at [e / 4][g][e % 4]: a group's lanes read consecutive
// 16-byte words.
template <int V>
__device__ __forceinline__ int lane_slot(int j, int lanes) {   // j: dim inside a half
    const int g = j / V, e = j % V;
    return ((e >> 2) * lanes + g) * 4 + (e & 3);
}
template <int V>
__device__ __forceinline__ void lane_read(const float *s, int g, int lanes, float *f) {
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
        const float4 v = *reinterpret_cast<const float4 *>(s + (c * lanes + g) * 4);
        f[4 * c] = v.x;
        f[4 * c + 1] = v.y;
        f[4 * c + 2] = v.z;
        f[4 * c + 3] = v.w;
    }
}

// cos and sin of a tile's angles: position x frequency formed and reduced modulo 2 pi in double
// (positions reach 10^5, where an fp32 angle is off by 10^-2 rad), then fp32
template <int V>
__device__ __forceinline__ void tile_angles(const NormRopeArgs &a, int64_t l0, int tokens, float *s_cos, float *s_sin) {
    const int lanes = a.D / (2 * V);
    for (int i = threadIdx.x; i < tokens * a.n_freq; i += blockDim.x) {
        const int tt = i / a.n_freq, j = i - tt * a.n_freq;
        const int axis = j < a.axis_end0 ? 0 : (j < a.axis_end1 ? 1 : 2);
        const double ang = static_cast<double>(a.pos[axis * a.L + l0 + tt]) * a.inv_freq[j];
        const double r = ang - 6.283185307179586476925 * rint(ang * 0.159154943091895335768883763);
        float sv, cv;
        sincosf(static_cast<float>(r), &sv, &cv);
        const int at = tt * a.n_freq + lane_slot<V>(j, lanes);
        s_cos[at] = cv;
        s_sin[at] = sv;
    }
}

// weights of q and k, lower and upper half, in lane order: [2][2][D/2]
template <typename T, int V>
__device__ __forceinline__ void load_weights(const NormRopeArgs &a, float *s_w) {
    const int half = a.D / 2, lanes = half / V;
    for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
        const int qk = i / a.D, d = i - qk * a.D, up = d >= half;
        const T *w = static_cast<const T *>(a.w[qk]);
        s_w[(qk * 2 + up) * half + lane_slot<V>(d - up * half, lanes)] = w ? to_float(w[d]) : 1.0f;
    }
}

template <int GL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct NormItem {
    bool live;
    int tt, qk, head;
};
// item i of a tile -> token and head; the q heads of a token first, then its k heads
__device__ __forceinline__ NormItem norm_item(const NormRopeArgs &a, int i, int tokens, bool lane_live) {
    const int H = a.heads[0] + a.heads[1];
    NormItem it;
    it.tt = i / H;
    const int h = i - it.tt * H;
    it.qk = h >= a.heads[0];
    it.head = it.qk ? h - a.heads[0] : h;
    it.live = lane_live && it.tt < tokens;
    return it;
}

constexpr int kNormHeld = 2;   // items a thread has in flight

template <typename T, int GL>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int V = Vec<T>::kVec;
    extern __shared__ float4 s_raw[];
    float *s_cos = reinterpret_cast<float *>(s_raw);
    float *s_sin = s_cos + a.tile * a.n_freq;
    float *s_w = s_sin + a.tile * a.n_freq;
    const int half = a.D / 2, lanes = half / V;
    const int g = threadIdx.x % GL, slot = threadIdx.x / GL;
    constexpr int kSlots = kNormThreads / GL;
    const int64_t l0 = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int tokens = static_cast<int>(a.L - l0 < a.tile ? a.L - l0 : a.tile);
    const int n = tokens * (a.heads[0] + a.heads[1]);
    const bool lane_live = g < lanes;

    auto src = [&](const NormItem &it) {
        return static_cast<const T *>(a.x[it.qk]) + (l0 + it.tt) * a.xs[it.qk] + it.head * a.D + g * V;
    };
    bool ready = false;
    for (int base = 0; base < n; base += kNormHeld * kSlots) {
        NormItem it[kNormHeld];
        uint4 lo[kNormHeld], hi[kNormHeld];
#pragma unroll
        for (int u = 0; u < kNormHeld; ++u) {
            it[u] = norm_item(a, base + u * kSlots + slot, tokens, lane_live);
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (it[u].live) {
                const T *p = src(it[u]);
                lo[u] = *reinterpret_cast<const uint4 *>(p);
                hi[u] = *reinterpret_cast<const uint4 *>(p + half);
            }
        }
        if (!ready) {   // the first vectors are in flight while the angles are formed
            load_weights<T, V>(a, s_w);
            tile_angles<V>(a, l0, tokens, s_cos, s_sin);
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kNormHeld; ++u) {
            float xl[V], xh[V];
            Vec<T>::unpack(lo[u], xl);
            Vec<T>::unpack(hi[u], xh);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) ss += xl[e] * xl[e] + xh[e] * xh[e];
            ss = group_sum<GL>(ss);
            const float r = rsqrtf(ss / a.D + a.eps);
            if (it[u].live) {
                float c[V], s[V], wl[V], wh[V];
                lane_read<V>(s_cos + it[u].tt * a.n_freq, g, lanes, c);
                lane_read<V>(s_sin + it[u].tt * a.n_freq, g, lanes, s);
                lane_read<V>(s_w + it[u].qk * a.D, g, lanes, wl);
                lane_read<V>(s_w + it[u].qk * a.D + half, g, lanes, wh);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float nl = xl[e] * r * wl[e], nh = xh[e] * r * wh[e];
                    xl[e] = nl * c[e] - nh * s[e];
                    xh[e] = nh * c[e] + nl * s[e];
                }
                T *p = static_cast<T *>(a.y[it[u].qk]) + (l0 + it[u].tt) * a.ys[it[u].qk] + it[u].head * a.D + g * V;
                *reinterpret_cast<uint4 *>(p) = Vec<T>::pack(xl);
                *reinterpret_cast<uint4 *>(p + half) = Vec<T>::pack(xh);
            }
        }
    }
}

// Gradient. Persistent CTAs, each a fixed set of tiles (tile blockIdx.x, + gridDim.x, ...), so that
// the weight gradients are few partial rows, summed in one fixed order whatever the scheduling.
template <typename T, int GL>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_grad_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int V = Vec<T>::kVec;
    extern __shared__ float4 s_raw[];
    float *s_cos = reinterpret_cast<float *>(s_raw);
    float *s_sin = s_cos + a.tile * a.n_freq;
    float *s_w = s_sin + a.tile * a.n_freq;
    const int half = a.D / 2, lanes = half / V;
    const int g = threadIdx.x % GL, slot = threadIdx.x / GL;
    constexpr int kSlots = kNormThreads / GL;
    const bool lane_live = g < lanes;
    float acc[2][2][V];                 // [q, k][lower, upper]
#pragma unroll
    for (int qk = 0; qk < 2; ++qk)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[qk][0][e] = acc[qk][1][e] = 0.f;
    load_weights<T, V>(a, s_w);

    const int64_t n_tiles = (a.L + a.tile - 1) / a.tile;
    for (int64_t tl = blockIdx.x; tl < n_tiles; tl += gridDim.x) {
        const int64_t l0 = tl * a.tile;
        const int tokens = static_cast<int>(a.L - l0 < a.tile ? a.L - l0 : a.tile);
        const int n = tokens * (a.heads[0] + a.heads[1]);
        bool ready = false;
        for (int base = 0; base < n; base += kSlots) {
            const NormItem it = norm_item(a, base + slot, tokens, lane_live);
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = make_uint4(0, 0, 0, 0);
            if (it.live) {
                const T *p = static_cast<const T *>(a.x[it.qk]) + (l0 + it.tt) * a.xs[it.qk] + it.head * a.D + g * V;
                const T *d = static_cast<const T *>(a.dy[it.qk]) + (l0 + it.tt) * a.dys[it.qk] + it.head * a.D + g * V;
                v[0] = *reinterpret_cast<const uint4 *>(p);
                v[1] = *reinterpret_cast<const uint4 *>(p + half);
                v[2] = *reinterpret_cast<const uint4 *>(d);
                v[3] = *reinterpret_cast<const uint4 *>(d + half);
            }
            if (!ready) {
                __syncthreads();        // the previous tile's angles have been read
                tile_angles<V>(a, l0, tokens, s_cos, s_sin);
                __syncthreads();
                ready = true;
            }
            float xl[V], xh[V], dl[V], dh[V], wl[V], wh[V];
            Vec<T>::unpack(v[0], xl);
            Vec<T>::unpack(v[1], xh);
            Vec<T>::unpack(v[2], dl);
            Vec<T>::unpack(v[3], dh);
            float ss = 0.f, gx = 0.f;
            if (it.live) {
                float c[V], s[V];
                lane_read<V>(s_cos + it.tt * a.n_freq, g, lanes, c);
                lane_read<V>(s_sin + it.tt * a.n_freq, g, lanes, s);
                lane_read<V>(s_w + it.qk * a.D, g, lanes, wl);
                lane_read<V>(s_w + it.qk * a.D + half, g, lanes, wh);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float nl = dl[e] * c[e] + dh[e] * s[e], nh = dh[e] * c[e] - dl[e] * s[e];
                    dl[e] = nl;
                    dh[e] = nh;
                    ss += xl[e] * xl[e] + xh[e] * xh[e];
                    gx += nl * wl[e] * xl[e] + nh * wh[e] * xh[e];
                }
            }
            ss = group_sum<GL>(ss);
            gx = group_sum<GL>(gx);
            if (it.live) {
                const float r = rsqrtf(ss / a.D + a.eps);
                const float k = gx / a.D * r * r;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float tl_ = dl[e] * xl[e] * r, th_ = dh[e] * xh[e] * r;
                    if (it.qk) {
                        acc[1][0][e] += tl_;
                        acc[1][1][e] += th_;
                    } else {
                        acc[0][0][e] += tl_;
                        acc[0][1][e] += th_;
                    }
                    xl[e] = r * (dl[e] * wl[e] - xl[e] * k);
                    xh[e] = r * (dh[e] * wh[e] - xh[e] * k);
                }
                T *p = static_cast<T *>(a.y[it.qk]) + (l0 + it.tt) * a.ys[it.qk] + it.head * a.D + g * V;
                *reinterpret_cast<uint4 *>(p) = Vec<T>::pack(xl);
                *reinterpret_cast<uint4 *>(p + half) = Vec<T>::pack(xh);
            }
        }
    }
    if (a.dw_part == nullptr) return;
    // the CTA's partial: groups of a warp by shuffles, warps through shared memory, in warp order
    __syncthreads();
    float *s_red = reinterpret_cast<float *>(s_raw);               // [warps][2][D]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int qk = 0; qk < 2; ++qk)
#pragma unroll
        for (int up = 0; up < 2; ++up)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = acc[qk][up][e];
#pragma unroll
                for (int o = 16; o >= GL; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane < GL && lane_live) s_red[(warp * 2 + qk) * a.D + up * half + g * V + e] = v;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kNormThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kNormThreads / 32; ++w) v += s_red[w * 2 * a.D + i];
        a.dw_part[static_cast<int64_t>(blockIdx.x) * 2 * a.D + i] = v;
    }
}

// dw[qk][d] = sum of the CTAs' partials: 32 columns x 32 strided row groups per CTA, then the row
// groups in order
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *__restrict__ part, int n_part, int D,
                                                       float *__restrict__ dqw, float *__restrict__ dkw) {
    __shared__ float s[32][33];
    const int c = threadIdx.x & 31, rg = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float v = 0.f;
    if (col < 2 * D)
        for (int p = rg; p < n_part; p += 32) v += part[static_cast<int64_t>(p) * 2 * D + col];
    s[rg][c] = v;
    __syncthreads();
    if (rg == 0 && col < 2 * D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][c];
        if (col < D) {
            if (dqw) dqw[col] = t;
        } else if (dkw) {
            dkw[col - D] = t;
        }
    }
}

}  // namespace vitk

namespace vith {

namespace {

// lanes of a head, rounded up to a power of two
int group_lanes(int D, int dtype) {
    const int v = dtype == VIT_DTYPE_F32 ? 4 : 8, lanes = D / (2 * v);
    int gl = 1;
    while (gl < lanes) gl *= 2;
    return gl;
}

// Tokens per tile: enough (token, head) items for every lane group of a CTA to hold `held`, at most
// kNormMaxTile (rows of few heads would otherwise leave most of a CTA idle).
int tile_tokens(int gl, int heads, int held) {
    const int want = vitk::kNormThreads / gl * held;
    return std::max(1, std::min(vitk::kNormMaxTile, want / std::max(1, heads)));
}

template <typename T>
cudaError_t forward(const vitk::NormRopeArgs &a, int gl, unsigned grid, size_t smem, cudaStream_t s) {
    switch (gl) {
        case 1:   // 16 dims of a 16-bit type; 32-bit heads have two lanes or more
            if constexpr (sizeof(T) == 2) vitk::norm_rope_kernel<T, 1><<<grid, vitk::kNormThreads, smem, s>>>(a);
            break;
        case 2: vitk::norm_rope_kernel<T, 2><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 4: vitk::norm_rope_kernel<T, 4><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 8: vitk::norm_rope_kernel<T, 8><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 16: vitk::norm_rope_kernel<T, 16><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        default:  // 32 lanes: fp32 heads of more than 128 dims
            if constexpr (sizeof(T) == 4) vitk::norm_rope_kernel<T, 32><<<grid, vitk::kNormThreads, smem, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const vitk::NormRopeArgs &a, int gl, unsigned grid, size_t smem, cudaStream_t s) {
    switch (gl) {
        case 1:   // 16 dims of a 16-bit type; 32-bit heads have two lanes or more
            if constexpr (sizeof(T) == 2) vitk::norm_rope_grad_kernel<T, 1><<<grid, vitk::kNormThreads, smem, s>>>(a);
            break;
        case 2: vitk::norm_rope_grad_kernel<T, 2><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 4: vitk::norm_rope_grad_kernel<T, 4><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 8: vitk::norm_rope_grad_kernel<T, 8><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        case 16: vitk::norm_rope_grad_kernel<T, 16><<<grid, vitk::kNormThreads, smem, s>>>(a); break;
        default:  // 32 lanes: fp32 heads of more than 128 dims
            if constexpr (sizeof(T) == 4) vitk::norm_rope_grad_kernel<T, 32><<<grid, vitk::kNormThreads, smem, s>>>(a);
    }
    return cudaGetLastError();
}

void fill(vitk::NormRopeArgs &a, const NormRopeCall &c, int tile) {
    for (int i = 0; i < 2; ++i) {
        a.x[i] = c.x[i];
        a.y[i] = c.y[i];
        a.dy[i] = c.dy[i];
        a.w[i] = c.w[i];
        a.xs[i] = c.x_stride[i];
        a.ys[i] = c.y_stride[i];
        a.dys[i] = c.dy_stride[i];
        a.heads[i] = c.heads[i];
    }
    a.D = c.head_dim;
    a.eps = c.eps;
    a.pos = c.pos;
    a.L = c.L;
    a.tile = tile;
    a.dw_part = nullptr;
    a.n_freq = c.head_dim / 2;
    a.axis_end0 = c.sections[0];
    a.axis_end1 = c.sections[0] + c.sections[1];
    // powers of theta^(-2/D), one product each: j roundings of 2^-53, under 2e-14 relative at j = 128
    // (10^-9 rad at position 10^5), where one pow per frequency would cost a call 2 us on the host
    const double step = std::pow(c.theta, -2.0 / c.head_dim);
    double f = 1.0;
    for (int j = 0; j < a.n_freq; ++j, f *= step) a.inv_freq[j] = f;
}

size_t angle_bytes(int tile, int D) { return sizeof(float) * (static_cast<size_t>(tile) * D + 2 * D); }

}  // namespace

int norm_rope_launch(const NormRopeCall &c, cudaStream_t s) {
    const int H = c.heads[0] + c.heads[1];
    if (c.L <= 0 || H <= 0) return VIT_OK;
    const int gl = group_lanes(c.head_dim, c.dtype);
    vitk::NormRopeArgs a;
    fill(a, c, tile_tokens(gl, H, vitk::kNormHeld));
    const unsigned grid = static_cast<unsigned>((c.L + a.tile - 1) / a.tile);
    const size_t smem = angle_bytes(a.tile, c.head_dim);
    const cudaError_t e = c.dtype == VIT_DTYPE_BF16   ? forward<__nv_bfloat16>(a, gl, grid, smem, s)
                          : c.dtype == VIT_DTYPE_F16 ? forward<__half>(a, gl, grid, smem, s)
                                                     : forward<float>(a, gl, grid, smem, s);
    return e == cudaSuccess ? VIT_OK : VIT_ERR_CUDA;
}

int64_t norm_rope_grad_workspace(int head_dim) {
    return static_cast<int64_t>(vitk::kNormGradCtas) * 2 * head_dim * sizeof(float);
}

int norm_rope_grad_launch(const NormRopeCall &c, float *dqw, float *dkw, void *workspace, cudaStream_t s) {
    const int H = c.heads[0] + c.heads[1];
    unsigned grid = 0;
    if (c.L > 0 && H > 0) {
        const int gl = group_lanes(c.head_dim, c.dtype);
        vitk::NormRopeArgs a;
        fill(a, c, tile_tokens(gl, H, 1));
        a.dw_part = dqw || dkw ? static_cast<float *>(workspace) : nullptr;
        const int64_t tiles = (c.L + a.tile - 1) / a.tile;
        grid = static_cast<unsigned>(std::min<int64_t>(tiles, vitk::kNormGradCtas));
        const size_t smem = std::max(angle_bytes(a.tile, c.head_dim),
                                     sizeof(float) * (vitk::kNormThreads / 32) * 2 * c.head_dim);
        const cudaError_t e = c.dtype == VIT_DTYPE_BF16   ? backward<__nv_bfloat16>(a, gl, grid, smem, s)
                              : c.dtype == VIT_DTYPE_F16 ? backward<__half>(a, gl, grid, smem, s)
                                                         : backward<float>(a, gl, grid, smem, s);
        if (e != cudaSuccess) return VIT_ERR_CUDA;
    }
    if (dqw || dkw) {   // no tokens: the sums over nothing are written as zeros
        vitk::norm_dw_kernel<<<(2 * c.head_dim + 31) / 32, 1024, 0, s>>>(static_cast<const float *>(workspace),
                                                                         static_cast<int>(grid), c.head_dim, dqw, dkw);
        if (cudaGetLastError() != cudaSuccess) return VIT_ERR_CUDA;
    }
    return VIT_OK;
}

}  // namespace vith
