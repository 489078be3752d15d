// Carried states kept in 8 bits: quantised as they are written to a cache, and read back.
//
// A state is a matrix of `rows` rows (all heads) of `cols` fp32 values.  Each row is cut into groups of 32 from its
// start (the last may be shorter), and a group keeps one fp32 scale:
//   scale = max |x| (1 / 127),   code = rint(x / scale) in [-127, 127],   read back as code * scale,
// in fp32: the product with the rounded 1 / 127, and an IEEE division, so that the format says which code a value on a
// border gets.  The error of a value is at most half a step, max |x| / 254, and three roundings.  Rounding to 8 bits is
// the purpose of the cache; the recurrences themselves keep their states in fp32.  In a [K, dv + 1] mixture memory whose
// dv is a multiple of 32 the normaliser column is a group of its own and comes back to within three roundings.
//
// Bound by memory: 5.125 bytes an element (at cols a multiple of 32).  A thread takes four neighbouring elements (one
// float4, one char4), eight threads a group, and kUnroll such pieces at a time so that enough loads are in flight.
// Measured, 96 states of 32 x 128 x 128: store 62 us (258 MB, 4.1 TB/s; bound by issue, 71 % of its slots: a group's
// maximum, its divisions and four roundings for each 20 bytes a thread moves), load 39 us (6.6 TB/s).
#include <cstdint>

#include "gma_delta.h"

namespace gma {
namespace {

constexpr int kThreads = 256, kGroup = 32, kSub = kGroup / 4, kUnroll = 4;

struct CopyArgs {
    StateCopy p;
    float *state;
    signed char *codes;
    float *scales;
    int groups;                       // groups of a row
    int pieces, per_cta;              // (row, group, sub) pieces of four elements: of a state, of one CTA
    int ctas;                         // CTAs of one state
};

// The entry's source and destination, or false where there is nothing to copy: a negative index marks an absent entry, an index
// outside its pool is an error, and of several entries with one destination the last one counts.
__device__ bool copy_pair(const CopyArgs &a, int n_src, int n_dst, int i, int &src, int &dst) {
    src = a.p.src ? a.p.src[i] : i;
    dst = a.p.dst ? a.p.dst[i] : i;
    bool later = false;
    if (a.p.dst)
        for (int j = i + 1 + threadIdx.x; j < a.p.n; j += kThreads)
            later |= a.p.dst[j] == dst && (!a.p.src || (a.p.src[j] >= 0 && a.p.src[j] < n_src));
    later = __syncthreads_or(later);
    if (src >= n_src || dst >= n_dst) {
        if (threadIdx.x == 0) atomicOr(a.p.status, (unsigned)kDevErrBounds);
        return false;
    }
    return src >= 0 && dst >= 0 && !later;
}

// Where piece w lies: its element offset in the state, its group and how many of its four elements exist.  FULL: whole
// groups only, so that pieces and elements run alike and nothing is divided.
template <bool FULL>
__device__ __forceinline__ void locate(const CopyArgs &a, int w, bool in, int &off, int &grp, int &n) {
    grp = w / kSub;
    if (FULL) {
        off = 4 * w;
        n = in ? 4 : 0;
    } else {
        const int row = grp / a.groups, col = (grp - row * a.groups) * kGroup + (w % kSub) * 4;
        off = row * a.p.cols + col;
        n = in ? min(max(a.p.cols - col, 0), 4) : 0;
    }
}

template <bool VEC, bool FULL>
__global__ void __launch_bounds__(kThreads) state_store_kernel(const CopyArgs a) {
    int src, dst;
    const int i = blockIdx.x / a.ctas;
    if (!copy_pair(a, a.p.n_states, a.p.n_cache, i, src, dst)) return;
    const float *from = a.state + (size_t)src * a.p.rows * a.p.cols;
    signed char *codes = a.codes + (size_t)dst * a.p.rows * a.p.cols;
    float *scales = a.scales + (size_t)dst * a.p.rows * a.groups;
    const int first = (blockIdx.x % a.ctas) * a.per_cta, count = min(a.per_cta, a.pieces - first);
    // `first` and `count` are multiples of kSub: the eight threads of a group are there together
    for (int at = 0; at < count; at += kThreads * kUnroll) {
        float x[kUnroll][4];
        int off[kUnroll], grp[kUnroll], n[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int w = at + u * kThreads + threadIdx.x;
            locate<FULL>(a, first + w, w < count, off[u], grp[u], n[u]);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[u][j] = 0.f;
            if (VEC) {
                if (n[u]) *reinterpret_cast<float4 *>(x[u]) = __ldcs(reinterpret_cast<const float4 *>(from + off[u]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < n[u]) x[u][j] = from[off[u] + j];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float m = 0.f;                               // infinite where the group holds a NaN or an infinity
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fabsf(x[u][j]) <= 3.402823466e38f ? fmaxf(m, fabsf(x[u][j])) : __int_as_float(0x7f800000);
#pragma unroll
            for (int o = 1; o < kSub; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            const bool odd = m > 3.402823466e38f;
            const float scale = __fmul_rn(m, 1.f / 127.f);
            // The quotient by way of 1 / scale is off by 127 * 2^-23 = 1.6e-5 at most: the same code as the division's
            // unless a border is that near, where (and where 1 / scale may overflow) the division itself is taken.
            const float inv = __fdiv_rn(1.f, scale);
            bool near = scale < 1e-30f;
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float q = x[u][j] * inv;
                y[j] = rintf(q);
                near |= !(fabsf(fabsf(q - y[j]) - 0.5f) > 1e-4f);
            }
            if (near)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = scale == 0.f ? 0.f : rintf(__fdiv_rn(x[u][j], scale));
            signed char q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)                  // a scale that was rounded down as a subnormal is why codes are held
                q[j] = odd ? 0 : (signed char)(int)fminf(fmaxf(y[j], -127.f), 127.f);
            if (VEC) {
                if (n[u]) *reinterpret_cast<char4 *>(codes + off[u]) = make_char4(q[0], q[1], q[2], q[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < n[u]) codes[off[u] + j] = q[j];
            }
            if (n[u] && threadIdx.x % kSub == 0) scales[grp[u]] = odd ? __int_as_float(0x7fffffff) : scale;
        }
    }
}

template <bool VEC, bool FULL>
__global__ void __launch_bounds__(kThreads) state_load_kernel(const CopyArgs a) {
    int src, dst;
    const int i = blockIdx.x / a.ctas;
    if (!copy_pair(a, a.p.n_cache, a.p.n_states, i, src, dst)) return;
    const signed char *codes = a.codes + (size_t)src * a.p.rows * a.p.cols;
    const float *scales = a.scales + (size_t)src * a.p.rows * a.groups;
    float *to = a.state + (size_t)dst * a.p.rows * a.p.cols;
    const int first = (blockIdx.x % a.ctas) * a.per_cta, count = min(a.per_cta, a.pieces - first);
    for (int at = 0; at < count; at += kThreads * kUnroll) {
        char4 q[kUnroll];
        float scale[kUnroll];
        int off[kUnroll], n[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int w = at + u * kThreads + threadIdx.x;
            int grp;
            locate<FULL>(a, first + w, w < count, off[u], grp, n[u]);
            q[u] = make_char4(0, 0, 0, 0);
            if (VEC) {
                if (n[u]) q[u] = *reinterpret_cast<const char4 *>(codes + off[u]);
            } else {
                if (n[u] > 0) q[u].x = codes[off[u]];
                if (n[u] > 1) q[u].y = codes[off[u] + 1];
                if (n[u] > 2) q[u].z = codes[off[u] + 2];
                if (n[u] > 3) q[u].w = codes[off[u] + 3];
            }
            scale[u] = n[u] ? scales[grp] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const float4 x = make_float4(q[u].x * scale[u], q[u].y * scale[u], q[u].z * scale[u], q[u].w * scale[u]);
            if (VEC) {
                if (n[u]) __stcs(reinterpret_cast<float4 *>(to + off[u]), x);
            } else {
                if (n[u] > 0) to[off[u]] = x.x;
                if (n[u] > 1) to[off[u] + 1] = x.y;
                if (n[u] > 2) to[off[u] + 2] = x.z;
                if (n[u] > 3) to[off[u] + 3] = x.w;
            }
        }
    }
}

CopyArgs copy_args(const StateCopy &p, float *state, signed char *codes, float *scales) {
    CopyArgs a{p, state, codes, scales, (p.cols + kGroup - 1) / kGroup, 0, 0, 0};
    a.pieces = (int)(p.rows * a.groups * kSub);
    // two rounds of the unrolled loop to a CTA; one where that would leave part of the GPU idle
    const int round = kThreads * kUnroll;
    a.per_cta = (long long)p.n * ((a.pieces + 2 * round - 1) / (2 * round)) < 1216 ? round : 2 * round;
    a.ctas = (a.pieces + a.per_cta - 1) / a.per_cta;
    return a;
}

}  // namespace

cudaError_t state_store(const StateCopy &p, const float *state, signed char *codes, float *scales, cudaStream_t s) {
    const CopyArgs a = copy_args(p, const_cast<float *>(state), codes, scales);
    const unsigned grid = (unsigned)((long long)a.ctas * p.n);
    if (p.cols % kGroup == 0) state_store_kernel<true, true><<<grid, kThreads, 0, s>>>(a);
    else if (p.cols % 4 == 0) state_store_kernel<true, false><<<grid, kThreads, 0, s>>>(a);
    else state_store_kernel<false, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t state_load(const StateCopy &p, const signed char *codes, const float *scales, float *state,
                       cudaStream_t s) {
    const CopyArgs a = copy_args(p, state, const_cast<signed char *>(codes), const_cast<float *>(scales));
    const unsigned grid = (unsigned)((long long)a.ctas * p.n);
    if (p.cols % kGroup == 0) state_load_kernel<true, true><<<grid, kThreads, 0, s>>>(a);
    else if (p.cols % 4 == 0) state_load_kernel<true, false><<<grid, kThreads, 0, s>>>(a);
    else state_load_kernel<false, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gma
