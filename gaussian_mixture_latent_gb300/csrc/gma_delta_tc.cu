// The gated delta rule in chunks of 64 rows on the tensor cores (bf16 inputs, d <= 128, d and dv multiples of 8).
//
// Within a chunk, with G the running sum of the log decays, D_ij = e^{G_i - G_j} (i >= j), L_ij = D_ij k_i.k_j below
// the diagonal and S the state [d, dv] before the chunk:
//   U = T (diag(beta) (V - diag(e^G) K S)),  T = (I + diag(beta) L)^-1
//   O = scale (diag(e^G) Q S + (D o Q K^T) U),  S <- e^{G_C} S + (diag(e^{G_C - G}) K)^T U.
// Every exponent is a difference that is <= 0 for decays <= 0.
//
// Two kernels.  delta_prep: what does not depend on the state, all chunks in parallel: T, P = scale D o Q K^T and the
// row factors, to the workspace.  delta_chain: the chunks of a head one after another.
//
// Precision.  K, Q, V are bf16 as given and exact.  fp32 values that enter a product (S, R, U, T) are split into
// NT bf16 terms: three (24 bits) when the state is returned, two (16 bits, 2^-17) when only the bf16 output is; P has
// two.  Q S alone takes S in one term: half a bf16 step of that product, which the output's own rounding equals.
#include <cstdint>

#include "gma_delta.h"
#include "gma_delta_mma.cuh"

namespace gma {
namespace {

using namespace dmma;

constexpr int C = kTcRows;

template <int V>
struct Int { static constexpr int value = V; };

struct Vec {                           // one chunk's row factors
    float2 G[C];                       // running sum of the log2 decays, hi + lo
    float e[C], f[C], beta[C];         // e^G, e^{G_C - G}
    float last, pad[3];                // e^{G_C}
};
// One chunk in the workspace: T's NT terms and P's two, as packed triangles, then the factors.
template <int NT>
struct Chunk {
    static constexpr int oP = NT * kTriBytes, oVec = oP + 2 * kTriBytes, bytes = oVec + (int)sizeof(Vec);
    static_assert(bytes % 16 == 0, "copied in pieces of 16 bytes");
};

// -------------------------------------------------------------------------------------------------- delta_prep
// One CTA of eight warps to a chunk.  Warps 0-3 take a row block of K K^T each and the inverse, warps 4-7 Q K^T.
// T is inverted in fp32: 16 x 16 diagonal blocks by substitution (a product of powers would overflow for repeated
// keys), joined to 32 and 64 by X21 = -T22 (A21 T11) with products of NT terms.  Bound by the latency of that chain of small
// steps: three CTAs share an SM.
constexpr int kPrepThreads = 256;
enum { kBarInv = 1, kBarPair = 2 };    // named barriers; the pairs use 2..5

struct PrepArgs {
    DeltaProblem p;
    char *chunks;
    int nc;
    bool held;                         // for the backward: no beta below 2^-64 in size (see delta_chain)
};

template <int D>
struct PrepSmem {
    static constexpr int kRow = 2 * D, kKey = C * kRow;
    static constexpr int oQ = kKey, oA = 2 * kKey, oI = oA + C * kFp * 4, oX = oI + C * kFp * 4;
    static constexpr int oVec = oX + 4 * 32 * 12 * 4, total = oVec + (int)sizeof(Vec);
};

template <int D, int NT>
__global__ void __launch_bounds__(kPrepThreads, 2) delta_prep_kernel(const PrepArgs a) {
    using L = PrepSmem<D>;
    using W = Chunk<NT>;
    constexpr int kRow = L::kRow;
    extern __shared__ __align__(128) char sm[];
    const uint32_t sb = smem_u32(sm);
    const DeltaProblem &p = a.p;
    const int pt = threadIdx.x, lane = pt & 31, pw = (pt >> 5) & 3;
    const bool inv = pt < 128;
    const int rb = inv ? pw : 3 - pw;                    // row block: each tensor unit gets five of the ten block pairs
    const int c = blockIdx.x % a.nc, bh = blockIdx.x / a.nc;
    const int b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.Hk);
    const int len = delta_len(p.lengths, b, p.N);
    if (c * C >= len) return;
    const size_t vrow = (size_t)bh * p.N, krow = ((size_t)b * p.Hk + hk) * p.N;
    char *to_ws = a.chunks + (size_t)blockIdx.x * W::bytes;
    const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.Kx), *Q = static_cast<const __nv_bfloat16 *>(p.Qx);
    for (int i = pt; i < C * (D / 8); i += kPrepThreads) {
        const int r = i / (D / 8), col = i % (D / 8), row = c * C + r;
        const bool ok = row < len && col * 8 < p.d;
        const size_t off = ok ? (krow + row) * p.d + col * 8 : 0;
        copy16(sb + at<kRow>(r, col), K + off, ok);
        copy16(sb + L::oQ + at<kRow>(r, col), Q + off, ok);
    }
    copy_commit();
    float *A = reinterpret_cast<float *>(sm + L::oA), *I = reinterpret_cast<float *>(sm + L::oI);
    float *X = reinterpret_cast<float *>(sm + L::oX) + pw * 32 * 12;
    Vec &vec = *reinterpret_cast<Vec *>(sm + L::oVec);
    const int r0 = lane >> 2, q0 = 2 * (lane & 3);
    if (pt < 32) {
        float gn[2], bn[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = c * C + 2 * lane + j;
            gn[j] = row < len ? delta_floor(delta_gate(p.g, vrow + row, p.gate_bf16)) : 0.f;
            bn[j] = row < len ? delta_gate(p.beta, vrow + row, p.gate_bf16) : 0.f;
            if (a.held && fabsf(bn[j]) < 0x1p-64f) bn[j] = copysignf(0x1p-64f, bn[j]);
        }
        const unsigned nan = __ballot_sync(~0u, gn[0] != gn[0] || gn[1] != gn[1]);
        const long long x0 = fixed_log2(gn[0]), x1 = fixed_log2(gn[1]);
        long long run = x0 + x1;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += y;
        }
        const long long end = __shfl_sync(~0u, run, 31);
        const bool bad = nan & (0xffffffffu >> (31 - lane));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const long long q = j ? run : run - x1;
            float2 G = fixed_pair(q);
            if (bad) G.x = __int_as_float(0x7fffffff);
            vec.G[2 * lane + j] = G;
            vec.e[2 * lane + j] = ex2(G.x);
            vec.f[2 * lane + j] = nan ? __int_as_float(0x7fffffff) : ex2(fixed_pair(end - q).x);
            vec.beta[2 * lane + j] = bn[j];
        }
        if (lane == 31) vec.last = vec.e[C - 1];
    }
    copy_wait<0>();
    __syncthreads();
    if (pt < (int)sizeof(Vec) / 16)
        reinterpret_cast<uint4 *>(to_ws + W::oVec)[pt] = reinterpret_cast<const uint4 *>(&vec)[pt];
    const uint32_t kt = sb, xt = inv ? sb : sb + L::oQ;
    char *P = to_ws + W::oP;
    const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ac = lane >> 4;      // A operand: row, 16-byte piece
    const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;      // B operand of two n tiles
                // rows 16 rb.. of K K^T (Q K^T), up to the diagonal
    float x[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t fa[4];
        ldsm(fa, xt + at<kRow>(rb * 16 + ar, 2 * ks + ac));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > rb) continue;
            uint32_t fb[4];
            ldsm(fb, kt + at<kRow>(np * 16 + br, 2 * ks + bc));
            mma(x[2 * np], fa, fb[0], fb[1]);
            mma(x[2 * np + 1], fa, fb[2], fb[3]);
        }
    }
    const int i0 = rb * 16 + r0, i1 = i0 + 8;
    const float2 g0 = vec.G[i0], g1 = vec.G[i1];
    const float m0 = inv ? vec.beta[i0] : p.scale, m1 = inv ? vec.beta[i1] : p.scale;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        if (n / 2 > rb) continue;
        const int j = 8 * n + q0;
        const float4 gj = *reinterpret_cast<const float4 *>(vec.G + j);      // hi, lo of rows j and j + 1
        x[n][0] *= ex2((g0.x - gj.x) + (g0.y - gj.y)) * m0;
        x[n][1] *= ex2((g0.x - gj.z) + (g0.y - gj.w)) * m0;
        x[n][2] *= ex2((g1.x - gj.x) + (g1.y - gj.y)) * m1;
        x[n][3] *= ex2((g1.x - gj.z) + (g1.y - gj.w)) * m1;
        if (n / 2 == rb) {                       // the diagonal block: below (and, for P, on) the diagonal
            const int on = inv ? 0 : 1;
            if (j >= i0 + on) x[n][0] = 0.f;
            if (j + 1 >= i0 + on) x[n][1] = 0.f;
            if (j >= i1 + on) x[n][2] = 0.f;
            if (j + 1 >= i1 + on) x[n][3] = 0.f;
        }
        if (inv) {
            *reinterpret_cast<float2 *>(A + i0 * kFp + j) = make_float2(x[n][0], x[n][1]);
            *reinterpret_cast<float2 *>(A + i1 * kFp + j) = make_float2(x[n][2], x[n][3]);
        } else {
            uint32_t t[2];
            const uint32_t o = tri(rb, n / 2) + 4 * (lane & 3);
            split<2>(x[n][0], x[n][1], t);
            *reinterpret_cast<uint32_t *>(P + o + at<32>(r0, n & 1)) = t[0];
            *reinterpret_cast<uint32_t *>(P + o + at<32>(r0, n & 1) + kTriBytes) = t[1];
            split<2>(x[n][2], x[n][3], t);
            *reinterpret_cast<uint32_t *>(P + o + at<32>(r0 + 8, n & 1)) = t[0];
            *reinterpret_cast<uint32_t *>(P + o + at<32>(r0 + 8, n & 1) + kTriBytes) = t[1];
        }
    }
    if (inv) {
        __syncwarp();
        {   // diagonal block pw: column `lane` of its inverse by substitution (both half-warps do the same)
            const int j = lane & 15;
            const float *row = A + pw * 16 * kFp + pw * 16;
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == j ? 1.f : 0.f;
#pragma unroll
                for (int m = 0; m < 16; m += 4) {
                    if (m >= i) break;
                    const float4 l = *reinterpret_cast<const float4 *>(row + i * kFp + m);
                    s = fmaf(-l.x, y[m], s);
                    if (m + 1 < i) s = fmaf(-l.y, y[m + 1], s);
                    if (m + 2 < i) s = fmaf(-l.z, y[m + 2], s);
                    if (m + 3 < i) s = fmaf(-l.w, y[m + 3], s);
                }
                y[i] = s;
            }
            if (lane < 16)
#pragma unroll
                for (int i = 0; i < 16; ++i) I[(pw * 16 + i) * kFp + pw * 16 + j] = y[i];
        }
        bar<128>(kBarInv);
        {   // 32 x 32 blocks: block (1, 0) by warps 0 and 1 (eight columns each), block (3, 2) by 2 and 3
            const int lo = (pw >> 1) * 32, col = lo + (pw & 1) * 8;
            uint32_t fa[NT][4], fb[NT][2];
            float y[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
            frag_a32<NT>(A + (lo + 16) * kFp + lo, kFp, lane, fa);
            frag_b32<NT>(I + lo * kFp + col, kFp, lane, fb);
            mma32<NT>(y, fa, fb);
            *reinterpret_cast<float2 *>(X + r0 * 12 + q0) = make_float2(y[0], y[1]);
            *reinterpret_cast<float2 *>(X + (r0 + 8) * 12 + q0) = make_float2(y[2], y[3]);
            __syncwarp();
            frag_a32<NT>(I + (lo + 16) * kFp + lo + 16, kFp, lane, fa);
            frag_b32<NT>(X, 12, lane, fb);
            mma32<NT>(z, fa, fb);
            float *to = I + (lo + 16 + r0) * kFp + col + q0;
            *reinterpret_cast<float2 *>(to) = make_float2(-z[0], -z[1]);
            *reinterpret_cast<float2 *>(to + 8 * kFp) = make_float2(-z[2], -z[3]);
        }
    }
    __syncthreads();
    {   // the 64 x 64 inverse: rows 32 + 16 m.., eight columns, to each of the eight warps
        const int col = pw * 8, m = inv ? 0 : 1;
        uint32_t fa[NT][4], fb[NT][2];
        float y[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 0 && col >= 16) continue;   // I is lower triangular: columns 16.. have no rows 0..15
            frag_a32<NT>(A + (32 + 16 * m) * kFp + 16 * k, kFp, lane, fa);
            frag_b32<NT>(I + 16 * k * kFp + col, kFp, lane, fb);
            mma32<NT>(y, fa, fb);
        }
        float *to = X + (16 * m + r0) * 12 + q0;
        *reinterpret_cast<float2 *>(to) = make_float2(y[0], y[1]);
        *reinterpret_cast<float2 *>(to + 8 * 12) = make_float2(y[2], y[3]);
        bar<64>(kBarPair + pw);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k > m) continue;
            frag_a32<NT>(I + (32 + 16 * m) * kFp + 32 + 16 * k, kFp, lane, fa);
            frag_b32<NT>(X + 16 * k * 12, 12, lane, fb);
            mma32<NT>(z, fa, fb);
        }
        to = I + (32 + 16 * m + r0) * kFp + col + q0;
        *reinterpret_cast<float2 *>(to) = make_float2(-z[0], -z[1]);
        *reinterpret_cast<float2 *>(to + 8 * kFp) = make_float2(-z[2], -z[3]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 10 * 128 / kPrepThreads; ++u) {  // pairs of the ten blocks
        const int e = pt + u * kPrepThreads, blk = e >> 7, r = (e >> 3) & 15, pc = e & 7;
        const int ib = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, jb = blk - ib * (ib + 1) / 2;
        const float2 y = *reinterpret_cast<const float2 *>(I + (16 * ib + r) * kFp + 16 * jb + 2 * pc);
        uint32_t t[NT];
        split<NT>(y.x, y.y, t);
#pragma unroll
        for (int k = 0; k < NT; ++k)
            *reinterpret_cast<uint32_t *>(to_ws + k * kTriBytes + blk * 512 + at<32>(r, pc >> 2) + 4 * (pc & 3)) = t[k];
    }
}

// -------------------------------------------------------------------------------------------------- delta_chain
// The state never leaves registers.  KS warps share 16 columns of dv; each holds its part of S^T, [16, D / KS], as fp32
// accumulator tiles.  Written transposed, every product of a chunk has such a tile on its left:
//   (K S)^T = S^T K^T,  U^T = R^T T^T,  O^T = S^T Q^T + U^T P^T,  S^T += (f U)^T K,
// and an accumulator tile is the next product's A operand as it stands.  The right sides (K, Q, T, P) are read from
// shared memory with ldmatrix; four loader warps copy chunk c + kStages - 1 while chunk c is worked on.
// The KS warps split the first product's sum (their parts of d), then the 64 rows (eight-row tiles r, 7 - r, ..: the
// same work under the triangles), then the columns of S^T; in between they exchange partial sums, R and U through shared
// memory, lane by lane.
//
// Checkpoint form (for the backward): no O; writes S before each chunk and W = U / beta, with |beta| held to at least
// 2^-64 (a beta of 0 then adds 2^-64 W to the state, nothing in fp32).
//
// Bound by the chain: mma.sync issues one m16n8k16 each 8.0 cycles on each of the SM's four tensor units (measured,
// 1 to 16 warps; latency 21), and the products of a chunk depend on one another.  tcgen05 has four times that rate,
// but its accumulators are in TMEM: three dependent products a chunk would each pay a round trip (load, split, store,
// fence, issue) of about a chunk's time here.
constexpr int kChainThreads = 256, kLoadThreads = 128, kAllThreads = kChainThreads + kLoadThreads;
// Registers: the block is launched with 168 a thread (384 x 168 = 64512); 256 x 232 + 128 x 40 = 64512.
constexpr int kChainRegs = 232, kLoadRegs = 40;
enum { kBarAll = 1, kBarSlice = 2 };   // named barriers; the slices use 2..5

struct ChainArgs {
    DeltaProblem p;
    const char *chunks;
    int nc, groups;                    // chunks of a head; CTAs of a head
    const float *state_in;
    float *state_out;
    void *out;
    float *w;                          // checkpoint form: [G, N, dv]
    __nv_bfloat16 *s0;                 // checkpoint form: [G, nc, dv, d], S before each chunk
};

template <int D, int NT, int SL>
struct ChainSmem {
    static constexpr int KS = 8 / SL;
    static constexpr int kRow = 2 * D, kKey = C * kRow, kValRow = 32 * SL, kVal = C * kValRow;
    static constexpr int oQ = kKey, oV = 2 * kKey, oW = oV + kVal, kStage = oW + Chunk<NT>::bytes;
    static constexpr int kSum = KS * 4096, kRows = 2048 * (NT > 2 ? NT : 2);    // of one slice
    static constexpr int kShared = SL * (kSum + kRows);
    static constexpr int kStages = 3 * kStage + kShared <= 227 * 1024 ? 3 : 2;
    static constexpr int oSum = kStages * kStage, oRows = oSum + SL * kSum, total = oRows + SL * kRows;
    static_assert(total <= 227 * 1024, "shared memory");
};

template <int D, int NT, int SL, bool CKPT>
__global__ void __launch_bounds__(kAllThreads, 1) delta_chain_kernel(const ChainArgs a) {
    using L = ChainSmem<D, NT, SL>;
    using W = Chunk<NT>;
    constexpr int KS = L::KS, DK = D / KS, OWN = 8 / KS;
    extern __shared__ __align__(128) char sm[];
    const uint32_t sb = smem_u32(sm);
    const DeltaProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = blockIdx.x / a.groups, grp = blockIdx.x % a.groups;
    const int b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.Hk);
    const int len = delta_len(p.lengths, b, p.N);
    const int nc = (len + C - 1) / C;
    const int c0 = grp * 16 * SL;                        // first column of the CTA
    const size_t vrow = (size_t)bh * p.N, krow = ((size_t)b * p.Hk + hk) * p.N;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);

    if (tid >= kChainThreads) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        const int lt = tid - kChainThreads;
        const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.Kx), *Q = static_cast<const __nv_bfloat16 *>(p.Qx);
        const __nv_bfloat16 *V = static_cast<const __nv_bfloat16 *>(p.V);
        auto load = [&](int c) {
            if (c < nc) {
                const uint32_t st = sb + (c % L::kStages) * L::kStage;
                for (int i = lt; i < C * (D / 8); i += kLoadThreads) {
                    const int r = i / (D / 8), col = i % (D / 8), row = c * C + r;
                    const bool ok = row < len && col * 8 < p.d;
                    const size_t off = ok ? (krow + row) * p.d + col * 8 : 0;
                    copy16(st + at<L::kRow>(r, col), K + off, ok);
                    if (!CKPT) copy16(st + L::oQ + at<L::kRow>(r, col), Q + off, ok);
                }
                for (int i = lt; i < C * 2 * SL; i += kLoadThreads) {
                    const int r = i / (2 * SL), col = i % (2 * SL), row = c * C + r;
                    const bool ok = row < len && c0 + col * 8 < p.dv;
                    const size_t off = ok ? (vrow + row) * p.dv + c0 + col * 8 : 0;
                    copy16(st + L::oV + at<L::kValRow>(r, col), V + off, ok);
                }
                const char *ws = a.chunks + ((size_t)bh * a.nc + c) * W::bytes;
                for (int i = lt; i < W::bytes / 16; i += kLoadThreads) copy16(st + L::oW + 16 * i, ws + 16 * i, true);
            }
            copy_commit();
        };
        for (int c = 0; c < L::kStages - 1; ++c) load(c);
        copy_wait<L::kStages - 2>();
        bar<kAllThreads>(kBarAll);
        for (int c = 0; c < nc; ++c) {
            load(c + L::kStages - 1);
            copy_wait<L::kStages - 2>();
            bar<kAllThreads>(kBarAll);
        }
        copy_wait<0>();
        if (!CKPT) {                                     // rows that do not exist
            const int w = min(16 * SL, p.dv - c0) / 8;
            for (size_t i = lt; i < (size_t)(p.N - len) * w; i += kLoadThreads)
                *reinterpret_cast<uint4 *>(out + (vrow + len + i / w) * p.dv + c0 + (int)(i % w) * 8) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChainRegs));
    const int slice = warp % SL, rank = warp / SL;
    const int col = c0 + 16 * slice + (lane >> 2), q0 = 2 * (lane & 3), k0 = rank * DK;
    const size_t sbase = (size_t)bh * p.d * p.dv;
    float S[DK / 8][4];                                  // S^T: rows col, col + 8; columns k0 + 8 n + q0, + 1
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = k0 + 8 * n + q0 + (j & 1), cc = col + 8 * (j >> 1);
            S[n][j] = a.state_in && r < p.d && cc < p.dv ? a.state_in[sbase + (size_t)r * p.dv + cc] : 0.f;
        }
    const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;              // B operand: rows n, pieces k
    const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, tc = lane >> 4;              // transposed: rows k, pieces n
    // the warp's eight-row tiles: r, 7 - r (and r + 2, 5 - r of two warps)
    auto own = [&](int j) { return j == 0 ? rank : j == 1 ? 7 - rank : j == 2 ? rank + 2 : 5 - rank; };
    float4 *sums = reinterpret_cast<float4 *>(sm + L::oSum + slice * L::kSum);      // [KS][8 tiles][32 lanes]
    char *rows = sm + L::oRows + slice * L::kRows;
    auto put_sums = [&](const float (&x)[8][4]) {
#pragma unroll
        for (int n = 0; n < 8; ++n) sums[(rank * 8 + n) * 32 + lane] = make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
    };
    auto get_sum = [&](int n, float (&x)[4]) {
        float4 y = sums[n * 32 + lane];
#pragma unroll
        for (int k = 1; k < KS; ++k) {
            const float4 z = sums[(k * 8 + n) * 32 + lane];
            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    };
    // x[j] += (rows of F^T) (triangle)^T for the warp's tiles: FT terms of F, TT of the triangle, the products that matter
    auto triangle = [&](auto &x, const auto &f, uint32_t t0, auto ft, auto tt, auto most) {
        constexpr int FT = decltype(ft)::value, TT = decltype(tt)::value, MOST = decltype(most)::value;
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const int n = own(j), ib = n >> 1;
#pragma unroll
            for (int jb = 0; jb < 4; jb += 2) {
                if (jb > ib) continue;
                // two blocks of the row at a time (the second one is the first again past the diagonal)
                const uint32_t blk = t0 + tri(ib, min(jb + (lane >> 4), ib)) + at<32>((n & 1) * 8 + (lane & 7), bc);
#pragma unroll
                for (int t = TT - 1; t >= 0; --t) {
                    uint32_t fb[4];
                    ldsm(fb, blk + t * kTriBytes);
#pragma unroll
                    for (int s = FT - 1; s >= 0; --s) {
                        if (s + t > MOST) continue;
                        mma(x[j], f[jb][s], fb[0], fb[1]);
                        if (jb + 1 <= ib) mma(x[j], f[jb + 1][s], fb[2], fb[3]);
                    }
                }
            }
        }
    };
    bar<kAllThreads>(kBarAll);
    for (int c = 0; c < nc; ++c) {
        char *st = sm + (c % L::kStages) * L::kStage;
        const uint32_t kt = smem_u32(st), qt = kt + L::oQ, vt = kt + L::oV, tt = kt + L::oW, pt = tt + W::oP;
        const Vec &vec = *reinterpret_cast<const Vec *>(st + L::oW + W::oVec);
        if (CKPT) {
            // S^T as it is held: [dv, d] in bf16
#pragma unroll
            for (int n = 0; n < DK / 8; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = k0 + 8 * n + q0, cc = col + 8 * j;
                    if (r < p.d && cc < p.dv)
                        *reinterpret_cast<uint32_t *>(a.s0 + (((size_t)bh * a.nc + c) * p.dv + cc) * p.d + r) =
                            pack(S[n][2 * j], S[n][2 * j + 1]);
                }
        }
        float y[8][4], o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[n][j] = o[n][j] = 0.f;
        // y = (K S)^T in NT terms of S, o = (Q S)^T in one: this warp's part of the sum
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
            uint32_t fs[NT][4];
            split_a<NT>(S[2 * ks], S[2 * ks + 1], fs);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t fb[4], fq[4];
                ldsm(fb, kt + at<L::kRow>(np * 16 + br, k0 / 8 + 2 * ks + bc));
                if (!CKPT) ldsm(fq, qt + at<L::kRow>(np * 16 + br, k0 / 8 + 2 * ks + bc));
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) {
                    mma(y[2 * np], fs[t], fb[0], fb[1]);
                    mma(y[2 * np + 1], fs[t], fb[2], fb[3]);
                }
                if (!CKPT) {
                    mma(o[2 * np], fs[0], fq[0], fq[1]);
                    mma(o[2 * np + 1], fs[0], fq[2], fq[3]);
                }
            }
        }
        put_sums(y);
        bar<32 * KS>(kBarSlice + slice);
        // R = beta (V - e^G K S), the left operand of T
#pragma unroll
        for (int j = 0; j < OWN; j += 2) {
            uint32_t fv[4];
            ldsm_t(fv, vt + at<L::kValRow>((lane >> 4 ? own(j + 1) : own(j)) * 8 + (lane & 7), 2 * slice + bc));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int n = own(j + m);
                float x[4];
                get_sum(n, x);
                const float2 e = *reinterpret_cast<const float2 *>(vec.e + 8 * n + q0);
                const float2 be = *reinterpret_cast<const float2 *>(vec.beta + 8 * n + q0);
                x[0] = be.x * fmaf(-e.x, x[0], low(fv[2 * m]));
                x[1] = be.y * fmaf(-e.y, x[1], high(fv[2 * m]));
                x[2] = be.x * fmaf(-e.x, x[2], low(fv[2 * m + 1]));
                x[3] = be.y * fmaf(-e.y, x[3], high(fv[2 * m + 1]));
                uint32_t t0[NT], t1[NT];
                split<NT>(x[0], x[1], t0);
                split<NT>(x[2], x[3], t1);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    reinterpret_cast<uint2 *>(rows)[(t * 8 + n) * 32 + lane] = make_uint2(t0[t], t1[t]);
            }
        }
        bar<32 * KS>(kBarSlice + slice);
        if (!CKPT) put_sums(o);
        uint32_t fr[4][NT][4];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint2 u0 = reinterpret_cast<const uint2 *>(rows)[(t * 8 + 2 * kb) * 32 + lane];
                const uint2 u1 = reinterpret_cast<const uint2 *>(rows)[(t * 8 + 2 * kb + 1) * 32 + lane];
                fr[kb][t][0] = u0.x; fr[kb][t][1] = u0.y; fr[kb][t][2] = u1.x; fr[kb][t][3] = u1.y;
            }
        bar<32 * KS>(kBarSlice + slice);
        // U^T = R^T T^T over the blocks at and below the diagonal
        float u[OWN][4];
#pragma unroll
        for (int j = 0; j < OWN; ++j)
#pragma unroll
            for (int m = 0; m < 4; ++m) u[j][m] = 0.f;
        triangle(u, fr, tt, Int<NT>{}, Int<NT>{}, Int<NT - 1>{});
#pragma unroll
        for (int j = 0; j < OWN; ++j)
            reinterpret_cast<float4 *>(rows)[own(j) * 32 + lane] = make_float4(u[j][0], u[j][1], u[j][2], u[j][3]);
        bar<32 * KS>(kBarSlice + slice);
        float z[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float4 x = reinterpret_cast<const float4 *>(rows)[n * 32 + lane];
            z[n][0] = x.x; z[n][1] = x.y; z[n][2] = x.z; z[n][3] = x.w;
        }
        if (!CKPT) {
            // O = scale e^G Q S + P U
            uint32_t fu[4][2][4];
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) split_a<2>(z[2 * kb], z[2 * kb + 1], fu[kb]);
            float x[OWN][4];
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                get_sum(own(j), x[j]);
                const float2 e = *reinterpret_cast<const float2 *>(vec.e + 8 * own(j) + q0);
#pragma unroll
                for (int m = 0; m < 4; ++m) x[j][m] *= p.scale * ((m & 1) ? e.y : e.x);
            }
            triangle(x, fu, pt, Int<2>{}, Int<2>{}, Int<1>{});
            // through the chunk's own V columns to memory
#pragma unroll
            for (int j = 0; j < OWN; j += 2) {
                const int r = (lane >> 4 ? own(j + 1) : own(j)) * 8 + (lane & 7);
                stsm_t(vt + at<L::kValRow>(r, 2 * slice + bc), pack(x[j][0], x[j][1]), pack(x[j][2], x[j][3]),
                       pack(x[j + 1][0], x[j + 1][1]), pack(x[j + 1][2], x[j + 1][3]));
                __syncwarp();
                const int cc = c0 + 16 * slice + bc * 8, row = c * C + r;
                if (row < len && cc < p.dv)
                    *reinterpret_cast<uint4 *>(out + (vrow + row) * p.dv + cc) =
                        *reinterpret_cast<const uint4 *>(st + L::oV + at<L::kValRow>(r, 2 * slice + bc));
            }
        } else {
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const float2 be = *reinterpret_cast<const float2 *>(vec.beta + 8 * own(j) + q0);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int row = c * C + 8 * own(j) + q0 + (m & 1), cc = col + 8 * (m >> 1);
                    if (row < len && cc < p.dv) a.w[(vrow + row) * p.dv + cc] = u[j][m] / ((m & 1) ? be.y : be.x);
                }
            }
        }
        // S <- e^{G_C} S + (f U)^T K
        const float last = vec.last;
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[n][j] *= last;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 f = *reinterpret_cast<const float2 *>(vec.f + 16 * kb + 8 * m + q0);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[2 * kb + m][j] *= (j & 1) ? f.y : f.x;
            }
            uint32_t fs[NT][4];
            split_a<NT>(z[2 * kb], z[2 * kb + 1], fs);
#pragma unroll
            for (int nd = 0; nd < DK / 16; ++nd) {
                uint32_t fb[4];
                ldsm_t(fb, kt + at<L::kRow>(kb * 16 + tr, k0 / 8 + 2 * nd + tc));
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) {
                    mma(S[2 * nd], fs[t], fb[0], fb[1]);
                    mma(S[2 * nd + 1], fs[t], fb[2], fb[3]);
                }
            }
        }
        bar<kAllThreads>(kBarAll);
    }
    if (a.state_out)
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = k0 + 8 * n + q0 + (j & 1), cc = col + 8 * (j >> 1);
                if (r < p.d && cc < p.dv) a.state_out[sbase + (size_t)r * p.dv + cc] = S[n][j];
            }
}

template <int D, int NT>
cudaError_t prep(const DeltaProblem &p, char *chunks, bool held, cudaStream_t s) {
    const PrepArgs a{p, chunks, (p.N + C - 1) / C, held};
    const cudaError_t e = set_dyn_smem((const void *)delta_prep_kernel<D, NT>, PrepSmem<D>::total);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<D, NT><<<(unsigned)((size_t)p.B * p.H * a.nc), kPrepThreads, PrepSmem<D>::total, s>>>(a);
    return cudaGetLastError();
}

template <int D, int NT, int SL, bool CKPT>
cudaError_t chain(ChainArgs a, cudaStream_t s) {
    a.groups = (a.p.dv + 16 * SL - 1) / (16 * SL);
    constexpr int smem = ChainSmem<D, NT, SL>::total;
    const cudaError_t e = set_dyn_smem((const void *)delta_chain_kernel<D, NT, SL, CKPT>, smem);
    if (e != cudaSuccess) return e;
    delta_chain_kernel<D, NT, SL, CKPT><<<(unsigned)(a.p.B * a.p.H * a.groups), kAllThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D, int NT, bool CKPT>
cudaError_t forward(const ChainArgs &a, cudaStream_t s) {
    const cudaError_t e = prep<D, NT>(a.p, const_cast<char *>(a.chunks), CKPT, s);
    if (e != cudaSuccess) return e;
    // Eight chain warps to a CTA, one CTA to an SM: four warps to each 16 columns while that fits one wave of CTAs, two
    // beyond (measured at 32 heads of 128 x 128: ... and 96 heads of 64 x 64: ...).
    const long long heads = (long long)a.p.B * a.p.H;
    return heads * ((a.p.dv + 31) / 32) <= 152 ? chain<D, NT, 2, CKPT>(a, s) : chain<D, NT, 4, CKPT>(a, s);
}

}  // namespace

bool delta_tc_supported(const DeltaProblem &p) {
    return p.bf16 && p.d <= 128 && p.d % 8 == 0 && p.dv % 8 == 0;
}

size_t delta_tc_workspace(const DeltaProblem &p) {
    return align_up((size_t)p.B * p.H * ((p.N + C - 1) / C) * Chunk<3>::bytes);
}

cudaError_t delta_tc_forward(const DeltaProblem &p, const float *state_in, void *out, float *state_out, char *ws,
                             cudaStream_t s) {
    const ChainArgs a{p, ws, (p.N + C - 1) / C, 0, state_in, state_out, out, nullptr, nullptr};
    if (p.d <= 64) return state_out ? forward<64, 3, false>(a, s) : forward<64, 2, false>(a, s);
    return state_out ? forward<128, 3, false>(a, s) : forward<128, 2, false>(a, s);
}

}  // namespace gma
